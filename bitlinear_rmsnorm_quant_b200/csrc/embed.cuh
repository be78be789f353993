// embed.cuh -- the embedding of the model: lookup with scaling (the bf16 x of
// the first BitLinear layer) and its gradient by sorted tokens.
//   x[m][k]      = bf16(scale * table[id_m][k])
//   dtable[v][k] = (dtable[v][k] +) scale * sum over m with id_m = v of dx[m][k]
// An id outside [0, V) (a padded place) gives a row of zeros and no gradient.
#pragma once
#include "common.cuh"

namespace mmf {

constexpr int kEmbedThreads = 256;

// The id at place m, or -1 when it is outside [0, V).
template <typename Id>
__device__ __forceinline__ int64_t embed_id(const Id* __restrict__ ids, int64_t m, int64_t V) {
    const int64_t v = static_cast<int64_t>(__ldg(ids + m));
    return v >= 0 && v < V ? v : -1;
}

// One CTA per token, 8 columns (16 bytes of x) per thread and step.
template <typename Id, bool BF16>
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const Id* __restrict__ ids,
                                                                  const void* __restrict__ table, int64_t V, int64_t M,
                                                                  int K, float scale, uint16_t* __restrict__ x) {
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const int64_t id = embed_id(ids, m, V);
        for (int k = 8 * threadIdx.x; k < K; k += 8 * kEmbedThreads) {
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (id >= 0) {
                if (BF16) {
                    unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(table) + id * K + k)), v);
                } else {
                    const float4* row = reinterpret_cast<const float4*>(static_cast<const float*>(table) + id * K + k);
                    const float4 a = __ldg(row), b = __ldg(row + 1);
                    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
                    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(v[2 * i], scale), __fmul_rn(v[2 * i + 1], scale));
                w[i] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *reinterpret_cast<uint4*>(x + m * K + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// Rows of dtable that no token names.  embed_count_kernel marks the others in
// used[]; the sorting and summing launches behind it have CTAs of their own
// that write zeros to a share of the unmarked rows, a warp to a row, so that
// the writes (most of the work of a small batch and a large table) run beside
// the sort and the sums.
// ---------------------------------------------------------------------------
struct ZeroParams {
    float* dtable;
    const uint8_t* used;
    int begin, end;  // rows of this launch
    int ctas;        // CTAs of this launch that zero; 0: none
    int K;
};

__device__ __forceinline__ void embed_zero(const ZeroParams& z, int cta) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int stride = z.ctas * warps;
    for (int row = z.begin + cta * warps + warp; row < z.end; row += stride) {
        if (z.used[row]) continue;
        float4* to = reinterpret_cast<float4*>(z.dtable + static_cast<int64_t>(row) * z.K);
        for (int i = lane; i < z.K / 4; i += 32) __stcs(to + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    }
}

// ---------------------------------------------------------------------------
// The tokens in the order of their ids, equal ids in the order of the tokens:
// a least-significant-digit radix sort of (id, token) with at most 8 bits a
// pass.  The places are split over at most kSortCtas CTAs; a CTA counts the
// digits of its places (embed_count_kernel), and places them behind those of
// the CTAs before it (embed_place_kernel).  Ids outside [0, V) sort as V,
// behind all rows.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 128;
constexpr int kSortBins = 256;
constexpr int kSortMaxPasses = 4;   // keys of 31 bits

struct SortParams {
    const void* ids;        // first pass: the caller's ids
    const uint32_t* key_in; // later passes
    const uint32_t* pos_in;
    uint32_t* key_out;
    uint32_t* pos_out;
    int* count;             // [CTA][kSortBins]
    int64_t V;
    int M;
    int per;                // places per CTA, a multiple of kSortThreads
    int ctas;
    int shift, mask;        // digit = (key >> shift) & mask
    int* next_count;        // the next pass's counts, taken while placing; null in the last pass
    int later_counts;       // first pass: how many later passes' counts, one behind another, to zero
    int next_shift;
    uint8_t* used;          // first pass, may be null: marks the rows that tokens name
};

template <typename Id, bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int i) {
    if (!FIRST) return p.key_in[i];
    const int64_t id = embed_id(static_cast<const Id*>(p.ids), i, p.V);
    return static_cast<uint32_t>(id < 0 ? p.V : id);
}

// The first pass's counts, and zeros for the later ones'.
template <typename Id>
__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const SortParams p) {
    __shared__ int bins[kSortBins];
    pdl_launch_dependents();
    bins[threadIdx.x] = 0;
    __syncthreads();
    const int begin = blockIdx.x * p.per, end = min(p.M, begin + p.per);
    for (int i = begin + threadIdx.x; i < end; i += kSortThreads) {
        const uint32_t key = sort_key<Id, true>(p, i);
        atomicAdd(&bins[(key >> p.shift) & p.mask], 1);
        if (p.used && key < p.V) p.used[key] = 1;
    }
    __syncthreads();
    p.count[blockIdx.x * kSortBins + threadIdx.x] = bins[threadIdx.x];
    for (int i = 0; i < p.later_counts; ++i)
        p.next_count[(i * kSortCtas + blockIdx.x) * kSortBins + threadIdx.x] = 0;
}

template <typename Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) embed_place_kernel(const SortParams p, const ZeroParams z) {
    __shared__ int base[kSortBins];                  // where this CTA's next place with a digit goes
    __shared__ int wcount[kSortWarps][kSortBins];    // a round's digits per warp, then the places before each warp's
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= p.ctas) {
        embed_zero(z, blockIdx.x - p.ctas);
        return;
    }
    {
        // digit t: places of all CTAs, and of the CTAs before this one
        int before = 0, all = 0;
#pragma unroll 16
        for (int b = 0; b < p.ctas; ++b) {
            const int c = p.count[b * kSortBins + t];
            all += c;
            if (b < static_cast<int>(blockIdx.x)) before += c;
        }
        // exclusive sum of the totals over the digits: 8 warps of 32, then the warps before
        int v = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) wcount[0][warp] = v;
        __syncthreads();
        for (int w = 0; w < warp; ++w) v += wcount[0][w];
        base[t] = v - all + before;
        __syncthreads();
    }
    const int begin = blockIdx.x * p.per, end = min(p.M, begin + p.per);
    for (int round = begin; round < end; round += kSortThreads) {
        const int i = round + t;
        const bool there = i < end;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) wcount[w][t] = 0;
        __syncthreads();
        const uint32_t active = __ballot_sync(0xffffffffu, there);
        uint32_t key = 0, pos = 0, peers = 0;
        int digit = 0;
        if (there) {
            key = sort_key<Id, FIRST>(p, i);
            pos = FIRST ? static_cast<uint32_t>(i) : p.pos_in[i];
            digit = static_cast<int>((key >> p.shift) & static_cast<uint32_t>(p.mask));
            peers = __match_any_sync(active, digit);  // the warp's lanes with the same digit
            if ((peers & ((1u << lane) - 1)) == 0) wcount[warp][digit] = __popc(peers);
        }
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = wcount[w][t];
            wcount[w][t] = sum;
            sum += c;
        }
        __syncthreads();
        if (there) {
            const int to = base[digit] + wcount[warp][digit] + __popc(peers & ((1u << lane) - 1));
            p.key_out[to] = key;
            p.pos_out[to] = pos;
            if (p.next_count)
                atomicAdd(&p.next_count[to / p.per * kSortBins + static_cast<int>((key >> p.next_shift) & static_cast<uint32_t>(p.mask))], 1);
        }
        __syncthreads();
        base[t] += sum;
    }
}

// ---------------------------------------------------------------------------
// Sums of equal ids.  A CTA takes `per` consecutive places of the sorted order
// and 8 columns per thread; it adds the rows of dx in order, in fp32, and at
// the end of a run of equal ids writes the row of dtable.  A run that crosses
// the CTA's places leaves its part in the workspace (the part up to the CTA's
// last place in tail[], the part from its first place, when the run began
// earlier, in head[]), and embed_join_kernel adds the parts in order, in fp64.
// So the order of additions depends on the ids alone.
// ---------------------------------------------------------------------------
struct SumParams {
    const uint32_t* key;
    const uint32_t* pos;
    const uint16_t* dx;
    float* dtable;
    float* head;  // [CTA][K]
    float* tail;  // [CTA][K]
    int64_t V;
    int M, K, per;
    float scale;
    int accumulate;
};

__device__ __forceinline__ void embed_store8(float* dst, const float (&a)[8], float scale, bool accumulate) {
    float4 lo = make_float4(a[0] * scale, a[1] * scale, a[2] * scale, a[3] * scale);
    float4 hi = make_float4(a[4] * scale, a[5] * scale, a[6] * scale, a[7] * scale);
    float4* d = reinterpret_cast<float4*>(dst);
    if (accumulate) {
        const float4 l = d[0], h = d[1];
        lo = make_float4(l.x + lo.x, l.y + lo.y, l.z + lo.z, l.w + lo.w);
        hi = make_float4(h.x + hi.x, h.y + hi.y, h.z + hi.z, h.w + hi.w);
    }
    d[0] = lo;
    d[1] = hi;
}

constexpr int kSumMaxPer = 256;
constexpr int kSumBatch = 8;  // rows of dx in flight per thread

__global__ void __launch_bounds__(kEmbedThreads) embed_sum_kernel(const SumParams p, const ZeroParams z) {
    __shared__ uint32_t key[kSumMaxPer + 1], pos[kSumMaxPer];
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) < z.ctas) {  // these first: they write all the while
        if (blockIdx.y == 0) embed_zero(z, blockIdx.x);
        return;
    }
    const int cta = blockIdx.x - z.ctas;
    const int begin = cta * p.per, n = min(p.M - begin, p.per);
    for (int i = threadIdx.x; i <= n; i += blockDim.x) {
        key[i] = begin + i < p.M ? p.key[begin + i] : 0xffffffffu;
        if (i < n) pos[i] = p.pos[begin + i];
    }
    const bool began_before = begin > 0 && p.key[begin - 1] == p.key[begin];
    __syncthreads();
    const int k = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
    if (k >= p.K) return;
    float a[8] = {};
    bool from_before = began_before;
    for (int i0 = 0; i0 < n; i0 += kSumBatch) {
        uint4 row[kSumBatch];
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u)
            if (i0 + u < n && key[i0 + u] < p.V)
                row[u] = __ldcs(reinterpret_cast<const uint4*>(p.dx + static_cast<int64_t>(pos[i0 + u]) * p.K + k));
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
            const int i = i0 + u;
            if (i >= n) break;
            const uint32_t run = key[i], next = key[i + 1];
            if (run >= p.V) return;  // the places without a row come last
            float v[8];
            unpack_bf16x8(row[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += v[j];
            if (next == run && i + 1 < n) continue;
            if (from_before || next == run) {
                float* to = (from_before ? p.head : p.tail) + static_cast<int64_t>(cta) * p.K + k;
                reinterpret_cast<float4*>(to)[0] = make_float4(a[0], a[1], a[2], a[3]);
                reinterpret_cast<float4*>(to)[1] = make_float4(a[4], a[5], a[6], a[7]);
            } else {
                embed_store8(p.dtable + static_cast<int64_t>(run) * p.K + k, a, p.scale, p.accumulate);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = 0.0f;
            from_before = false;
        }
    }
}

// CTA b joins the run that begins among its places and goes on behind them.
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(const SumParams p) {
    pdl_wait();
    const int begin = blockIdx.x * p.per, end = min(p.M, begin + p.per);
    if (end >= p.M) return;
    const uint32_t run = p.key[end - 1];
    if (run >= p.V || p.key[end] != run) return;                              // it ends here
    if (p.key[begin] == run && begin > 0 && p.key[begin - 1] == run) return;  // it began earlier
    const int k = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
    if (k >= p.K) return;
    double a[8];
    const float* part = p.tail + static_cast<int64_t>(blockIdx.x) * p.K + k;
    for (int b = blockIdx.x;;) {
        const float4 lo = reinterpret_cast<const float4*>(part)[0], hi = reinterpret_cast<const float4*>(part)[1];
        const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        const bool first = b == static_cast<int>(blockIdx.x);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = first ? static_cast<double>(v[j]) : a[j] + v[j];
        ++b;
        const int64_t at = static_cast<int64_t>(b) * p.per;
        if (at >= p.M || p.key[at] != run) break;
        part = p.head + static_cast<int64_t>(b) * p.K + k;
    }
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = static_cast<float>(a[j]);
    embed_store8(p.dtable + static_cast<int64_t>(run) * p.K + k, s, p.scale, p.accumulate);
}

// ---------------------------------------------------------------------------
// A few tokens: one launch, nothing sorted.  A CTA per token (and 8 columns
// per thread) reads all ids; the first token of an id lists the others in
// order and adds their rows, in fp32 up to 64 at a time and those in fp64; the
// CTAs of the later ones leave at once.
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 1024;
constexpr int kFewGroup = 64;

template <typename Id>
__global__ void __launch_bounds__(kEmbedThreads) embed_few_kernel(const Id* __restrict__ ids,
                                                                 const uint16_t* __restrict__ dx, int64_t V, int M,
                                                                 int K, float scale, float* __restrict__ dtable,
                                                                 int accumulate) {
    __shared__ int key[kFewTokens];
    __shared__ int pos[kFewTokens];
    __shared__ int count;
    const int m = blockIdx.x;
    for (int i = threadIdx.x; i < M; i += blockDim.x) key[i] = static_cast<int>(embed_id(ids, i, V));
    __syncthreads();
    const int mine = key[m];
    bool later = mine < 0;
    for (int i = threadIdx.x; i < m; i += blockDim.x) later |= key[i] == mine;
    if (__syncthreads_or(later)) return;
    if (threadIdx.x < 32) {
        int n = 0;
        for (int i0 = m; i0 < M; i0 += 32) {
            const int i = i0 + static_cast<int>(threadIdx.x);
            const bool same = i < M && key[i] == mine;
            const uint32_t who = __ballot_sync(0xffffffffu, same);
            if (same) pos[n + __popc(who & ((1u << threadIdx.x) - 1))] = i;
            n += __popc(who);
        }
        if (threadIdx.x == 0) count = n;
    }
    __syncthreads();
    const int k = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
    if (k >= K) return;
    double total[8] = {};
    for (int g = 0; g < count; g += kFewGroup) {
        const int end = min(count, g + kFewGroup);
        float a[8] = {};
        for (int i0 = g; i0 < end; i0 += kSumBatch) {
            uint4 row[kSumBatch];
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u)
                if (i0 + u < end) row[u] = __ldg(reinterpret_cast<const uint4*>(dx + static_cast<int64_t>(pos[i0 + u]) * K + k));
#pragma unroll
            for (int u = 0; u < kSumBatch; ++u) {
                if (i0 + u >= end) break;
                float v[8];
                unpack_bf16x8(row[u], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += v[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) total[j] += a[j];
    }
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = static_cast<float>(total[j]);
    embed_store8(dtable + static_cast<int64_t>(mine) * K + k, s, scale, accumulate);
}

}  // namespace mmf
