// embed.cuh -- the embedding of the model: lookup with scaling (the bf16 x of
// the first BitLinear layer) and its gradient by sorted tokens.
//   x[m][k]      = bf16(scale * table[id_m][k])
//   dtable[v][k] = (dtable[v][k] +) scale * sum over m with id_m = v of dx[m][k]
// An id outside [0, V) (a padded place) gives a row of zeros and no gradient.
//
// Bound by HBM and, for small batches, by launches.  Measured: lookup of 131072
// rows of 2048 from a bf16 table of 50257, 109 us on the device (5.9 TB/s
// counting each row of the table once), 117 where calls follow one another;
// gradient of 8192 tokens for a table of 32000 x 2560, 75 us, 60 of them the sums
// and zeros at 5.5 TB/s behind the sort's 14; of 131072 tokens for 50257 x 2048,
// 190 us, 144 of them at 5.9 TB/s, 30 the sort's and 14 the join's; 511 tokens
// added to a table, 5 us (9 us a call on the host).
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

// The rows of x laid end to end in groups of 8 columns (16 bytes), kFwdItems
// groups per thread, kEmbedThreads apart: all of a thread's ids, then all of
// its table reads are in flight before the first is used, and any K and M fill
// the CTAs alike.  x is written past L2 so that the frequent words' rows stay
// there.  Index is what numbers the groups: 32 bits where they fit.  A thread
// divides once and steps from group to group by kEmbedThreads' quotient and
// remainder (131072 x 2048: 109 us on the device; with a division for each, 116 us at three
// instructions a cycle).
constexpr int kFwdItems = 4;

template <typename Id, bool BF16, typename Index>
__global__ void __launch_bounds__(kEmbedThreads) embed_fwd_kernel(const Id* __restrict__ ids,
                                                                  const void* __restrict__ table, int64_t V, int64_t M,
                                                                  int K, unsigned step_rows, unsigned step_cols, float scale,
                                                                  uint16_t* __restrict__ x) {
    const unsigned lanes = static_cast<unsigned>(K) / 8;
    const Index first = static_cast<Index>(blockIdx.x) * (kFwdItems * kEmbedThreads) + threadIdx.x;
    const Index row0 = first / lanes;
    int64_t m = static_cast<int64_t>(row0);
    unsigned col[kFwdItems];
    int64_t id[kFwdItems];
    bool there[kFwdItems];
    col[0] = static_cast<unsigned>(first - row0 * lanes);
#pragma unroll
    for (int u = 0; u < kFwdItems; ++u) {
        if (u > 0) {
            const unsigned c = col[u - 1] + step_cols;
            const bool over = c >= lanes;
            col[u] = over ? c - lanes : c;
            m += step_rows + (over ? 1 : 0);
        }
        there[u] = m < M;
        id[u] = there[u] ? embed_id(ids, m, V) : -1;
    }
    uint4 lo[kFwdItems], hi[kFwdItems];  // 8 bf16, or 8 fp32
#pragma unroll
    for (int u = 0; u < kFwdItems; ++u) {
        lo[u] = hi[u] = make_uint4(0u, 0u, 0u, 0u);
        const unsigned c = col[u];
        if (id[u] < 0) continue;
        if (BF16) {
            lo[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(table) + id[u] * K) + c);
        } else {
            const uint4* row = reinterpret_cast<const uint4*>(static_cast<const float*>(table) + id[u] * K) + 2 * c;
            lo[u] = __ldg(row);
            hi[u] = __ldg(row + 1);
        }
    }
#pragma unroll
    for (int u = 0; u < kFwdItems; ++u) {
        if (!there[u]) continue;
        float v[8];
        if (BF16) {
            unpack_bf16x8(lo[u], v);
        } else {
            v[0] = __uint_as_float(lo[u].x), v[1] = __uint_as_float(lo[u].y), v[2] = __uint_as_float(lo[u].z);
            v[3] = __uint_as_float(lo[u].w), v[4] = __uint_as_float(hi[u].x), v[5] = __uint_as_float(hi[u].y);
            v[6] = __uint_as_float(hi[u].z), v[7] = __uint_as_float(hi[u].w);
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(v[2 * i], scale), __fmul_rn(v[2 * i + 1], scale));
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        __stcs(reinterpret_cast<uint4*>(x) + first + u * kEmbedThreads, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// ---------------------------------------------------------------------------
// Rows of dtable that no token names.  The first placing launch marks the
// others in used[]; the launches behind it have CTAs of their own that write
// zeros to a share of the unmarked rows, so that the writes (most of the work
// of a small batch and a large table) run beside the sort and the sums.  The
// launches up to the marking, which cannot know, zero all rows of a share: the
// sums come later.  A warp writes kZeroUnits pieces of a row of at most 2 KB and
// is done: many short CTAs write 6.4 TB/s, 296 that stay 5.9 TB/s (32000 rows
// of 2560 fp32, 12% of them marked).
// ---------------------------------------------------------------------------
constexpr int kZeroUnits = 2;
constexpr int kZeroPiece = 128;  // 16-byte stores of a piece

struct ZeroParams {
    float* dtable;
    const uint8_t* used;  // null: all rows
    int begin, end;       // rows of this launch
    int K;
};

__host__ __device__ __forceinline__ int64_t embed_zero_ctas(const ZeroParams& z, int threads) {
    const int64_t pieces = (z.K / 4 + kZeroPiece - 1) / kZeroPiece, warps = threads / 32;
    return (static_cast<int64_t>(z.end - z.begin) * pieces + warps * kZeroUnits - 1) / (warps * kZeroUnits);
}

__device__ __forceinline__ void embed_zero(const ZeroParams& z, int cta) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const unsigned per_row = z.K / 4, pieces = (per_row + kZeroPiece - 1) / kZeroPiece;
    const unsigned first = (static_cast<unsigned>(cta) * warps + warp) * kZeroUnits;  // pieces of a table fit 32 bits
#pragma unroll
    for (int u = 0; u < kZeroUnits; ++u) {
        const unsigned of = (first + u) / pieces;
        const unsigned from = (first + u - of * pieces) * kZeroPiece;
        const int64_t row = z.begin + static_cast<int64_t>(of);
        if (row >= z.end || (z.used && z.used[row])) continue;
        float4* to = reinterpret_cast<float4*>(z.dtable + row * z.K);
#pragma unroll
        for (unsigned i = 0; i < kZeroPiece; i += 32)
            if (from + i + lane < per_row) __stcs(to + from + i + lane, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    }
}

// ---------------------------------------------------------------------------
// The tokens in the order of their ids, equal ids in the order of the tokens:
// a least-significant-digit radix sort of (id, token) with at most 8 bits a
// pass.  The places are split over at most kSortCtas CTAs; a CTA counts the
// digits of its places (embed_count_kernel), and places them behind those of
// the CTAs before it (embed_place_kernel; counting the next pass's digits there
// with atomics took 16 us more at 131072 tokens than the launch it saved).  Ids outside [0, V) sort as V,
// behind all rows.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 128;
constexpr int kSortBins = 256;

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
    uint8_t* used;          // first pass, may be null: the rows that tokens name, cleared while counting, marked while placing
};

template <typename Id, bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int i) {
    if (!FIRST) return __ldcg(p.key_in + i);
    const int64_t id = embed_id(static_cast<const Id*>(p.ids), i, p.V);
    return static_cast<uint32_t>(id < 0 ? p.V : id);
}

template <typename Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const SortParams p, const ZeroParams z) {
    __shared__ int bins[kSortBins];
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= p.ctas) {
        embed_zero(z, blockIdx.x - p.ctas);
        return;
    }
    if (threadIdx.x < kSortBins) bins[threadIdx.x] = 0;
    __syncthreads();
    const int begin = blockIdx.x * p.per, end = min(p.M, begin + p.per);
    for (int i = begin + threadIdx.x; i < end; i += kSortThreads) {
        const uint32_t key = sort_key<Id, FIRST>(p, i);
        atomicAdd(&bins[(key >> p.shift) & p.mask], 1);
    }
    if (FIRST && p.used)  // for the placing launch to mark (the buffer is whole 16-byte words)
        for (int64_t i = 16 * (static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x); i < p.V;
             i += int64_t(16) * kSortThreads * p.ctas)
            *reinterpret_cast<uint4*>(p.used + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    if (threadIdx.x < kSortBins) p.count[blockIdx.x * kSortBins + threadIdx.x] = bins[threadIdx.x];
}

// What placing works with in shared memory.
struct SortShared {
    int base[kSortBins];                 // where the CTA's next place with a digit goes
    int wcount[kSortWarps][kSortBins];   // a round's digits per warp, then the places before each warp's
    int wsum[kSortBins / 32];
};

// base[] from each digit's places in all CTAs and in those before this one
// (thread t's digit t): those of the smaller digits come first.
__device__ __forceinline__ void sort_base(SortShared& sh, int all, int before) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    int v = all;
    if (t < kSortBins) {  // inclusive sum over the digits: 8 warps of 32, then the warps before
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) sh.wsum[warp] = v;
    }
    __syncthreads();
    if (t < kSortBins) {
        for (int w = 0; w < warp; ++w) v += sh.wsum[w];
        sh.base[t] = v - all + before;
    }
}

// Places begin .. end - 1 behind base[], a thread each per round; key and pos
// are this thread's of the first round.
template <typename Id, bool FIRST>
__device__ __forceinline__ void sort_place(const SortParams& p, SortShared& sh, int begin, int end, uint32_t key,
                                           uint32_t pos) {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    for (int round = begin; round < end; round += kSortThreads) {
        const bool there = round + t < end;
        for (int i = t; i < kSortWarps * kSortBins; i += kSortThreads) sh.wcount[0][i] = 0;
        __syncthreads();
        const uint32_t active = __ballot_sync(0xffffffffu, there);
        uint32_t peers = 0;
        const int digit = static_cast<int>((key >> p.shift) & static_cast<uint32_t>(p.mask));
        if (there) {
            peers = __match_any_sync(active, digit);  // the warp's lanes with the same digit
            if ((peers & ((1u << lane) - 1)) == 0) sh.wcount[warp][digit] = __popc(peers);
        }
        __syncthreads();
        int sum = 0;
        if (t < kSortBins) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = sh.wcount[w][t];
                sh.wcount[w][t] = sum;
                sum += c;
            }
        }
        __syncthreads();
        if (there) {
            const int to = sh.base[digit] + sh.wcount[warp][digit] + __popc(peers & ((1u << lane) - 1));
            p.key_out[to] = key;
            p.pos_out[to] = pos;
            if (FIRST && p.used && key < p.V) p.used[key] = 1;
        }
        const int i = round + kSortThreads + t;
        if (i < end) {
            key = sort_key<Id, FIRST>(p, i);
            pos = FIRST ? static_cast<uint32_t>(i) : __ldcg(p.pos_in + i);
        }
        __syncthreads();
        if (t < kSortBins) sh.base[t] += sum;
    }
}

template <typename Id, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) embed_place_kernel(const SortParams p, const ZeroParams z) {
    __shared__ SortShared sh;
    __shared__ int part[2][4][kSortBins];  // a quarter of the CTAs' places: all, and before this one
    const int t = threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= p.ctas) {
        embed_zero(z, blockIdx.x - p.ctas);
        return;
    }
    const int begin = blockIdx.x * p.per, end = min(p.M, begin + p.per);
    uint32_t key = 0, pos = 0;
    if (begin + t < end) {
        key = sort_key<Id, FIRST>(p, begin + t);
        pos = FIRST ? static_cast<uint32_t>(begin + t) : __ldcg(p.pos_in + begin + t);
    }
    {
        const int d = t & (kSortBins - 1), quarter = t / kSortBins;
        int count[kSortCtas / 4];
#pragma unroll
        for (int i = 0; i < kSortCtas / 4; ++i) {
            const int b = 4 * i + quarter;
            count[i] = b < p.ctas ? p.count[b * kSortBins + d] : 0;
        }
        int before = 0, all = 0;
#pragma unroll
        for (int i = 0; i < kSortCtas / 4; ++i) {
            all += count[i];
            if (4 * i + quarter < static_cast<int>(blockIdx.x)) before += count[i];
        }
        part[0][quarter][d] = all;
        part[1][quarter][d] = before;
    }
    __syncthreads();
    int all = 0, before = 0;
    if (t < kSortBins) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            all += part[0][q][t];
            before += part[1][q][t];
        }
    }
    sort_base(sh, all, before);
    sort_place<Id, FIRST>(p, sh, begin, end, key, pos);
}

// The whole sort of up to kClusterTokens places in one launch of one cluster:
// the CTAs read one another's counts from shared memory, and the passes are
// kept apart by cluster barriers (which also make the placed keys visible).
// Two launches a pass cost the host 14 us at two passes, this one 3.5.
constexpr int kSortCluster = 8;
constexpr int kClusterTokens = 16384;

struct SortPasses {
    int passes, digit_bits;
    uint32_t* key[2];
    uint32_t* pos[2];
};

template <typename Id, bool FIRST>
__device__ __forceinline__ void sort_cluster_pass(const SortParams& p, SortShared& sh, int* bins) {
    const int t = threadIdx.x, rank = blockIdx.x;
    if (t < kSortBins) bins[t] = 0;
    __syncthreads();
    const int begin = min(p.M, rank * p.per), end = min(p.M, begin + p.per);
    uint32_t key = 0, pos = 0;
    for (int i = begin + t; i < end; i += kSortThreads) {
        const uint32_t k = sort_key<Id, FIRST>(p, i);
        atomicAdd(&bins[(k >> p.shift) & p.mask], 1);
        if (i == begin + t) {
            key = k;
            pos = FIRST ? static_cast<uint32_t>(i) : __ldcg(p.pos_in + i);
        }
    }
    if (FIRST && p.used)
        for (int64_t i = 16 * (static_cast<int64_t>(rank) * kSortThreads + t); i < p.V; i += int64_t(16) * kSortThreads * kSortCluster)
            *reinterpret_cast<uint4*>(p.used + i) = make_uint4(0u, 0u, 0u, 0u);
    cluster_sync_all();
    int all = 0, before = 0;
    if (t < kSortBins) {
#pragma unroll
        for (int b = 0; b < kSortCluster; ++b) {
            int c;
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(dsmem_addr(smem_u32(bins + t), b)) : "memory");
            all += c;
            if (b < rank) before += c;
        }
    }
    sort_base(sh, all, before);
    sort_place<Id, FIRST>(p, sh, begin, end, key, pos);
    cluster_sync_all();
}

template <typename Id>
__global__ void __launch_bounds__(kSortThreads) embed_sort_cluster_kernel(SortParams p, const SortPasses s, const ZeroParams z) {
    __shared__ SortShared sh;
    __shared__ int bins[kSortBins];
    pdl_launch_dependents();
    if (blockIdx.x >= kSortCluster) {  // the clusters behind the first zero a share
        embed_zero(z, blockIdx.x - kSortCluster);
        return;
    }
    for (int i = 0; i < s.passes; ++i) {
        p.shift = i * s.digit_bits;
        p.key_in = s.key[(i + 1) & 1];
        p.pos_in = s.pos[(i + 1) & 1];
        p.key_out = s.key[i & 1];
        p.pos_out = s.pos[i & 1];
        if (i == 0)
            sort_cluster_pass<Id, true>(p, sh, bins);
        else
            sort_cluster_pass<Id, false>(p, sh, bins);
    }
}

// ---------------------------------------------------------------------------
// Sums of equal ids.  A CTA takes `per` consecutive places of the sorted order
// and 8 columns per thread; it adds the rows of dx in order, in fp32, and at
// the end of a run of equal ids writes the row of dtable.  A run of at most
// `per` places is summed by the CTA it begins in, also behind the CTA's own
// places (and skipped by the next).  Of a longer one each CTA leaves its part
// in the workspace (the part up to the CTA's last place in tail[], the part
// from its first place, where the run began earlier, in head[]), and
// embed_join_kernel adds the parts in order, in fp64.  So the order of
// additions depends on the ids alone.
// ---------------------------------------------------------------------------
struct SumParams {
    const uint32_t* key;
    const uint32_t* pos;
    const uint16_t* dx;
    float* dtable;
    float* head;         // [CTA][K]
    float* tail;         // [CTA][K]
    uint32_t* crossing;  // [CTA] the long run that begins in the CTA and goes on behind it, or kNoRun
    int64_t V;
    int M, K, per, ctas;
    float scale;
    int accumulate;
};
constexpr uint32_t kNoRun = 0xffffffffu;

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
    __shared__ uint32_t keys[3 * kSumMaxPer + 1];  // of places begin - per .. begin + 2 per
    __shared__ uint32_t pos[2 * kSumMaxPer];
    __shared__ int head_start, head_end, tail_start, tail_end;
    pdl_launch_dependents();
    pdl_wait();
    const int cta = blockIdx.x;  // the summing CTAs first: they wait for memory most of their time
    if (cta >= p.ctas) {
        if (blockIdx.y == 0) embed_zero(z, cta - p.ctas);
        return;
    }
    const int begin = cta * p.per, n = min(p.M - begin, p.per), per = p.per;
    if (threadIdx.x == 0) {
        head_start = -per;
        head_end = 2 * per + 1;
        tail_start = 0;
        tail_end = 2 * per + 1;
    }
    for (int i = threadIdx.x; i <= 3 * per; i += blockDim.x) {
        const int at = begin - per + i;
        keys[i] = at >= 0 && at < p.M ? p.key[at] : kNoRun;
        if (i >= per && i < 3 * per && at < p.M) pos[i - per] = p.pos[at];
    }
    __syncthreads();
    // The runs over the CTA's first and last place, by places counted from
    // `begin`: where they begin (looked for as far as `per` places before the
    // CTA) and end (as far as the places loaded).
    const uint32_t* key = keys + per;
    const uint32_t first = key[0], last = key[n - 1];
    for (int i = static_cast<int>(threadIdx.x) - per; i <= 2 * per; i += blockDim.x) {
        if (i < 0 && key[i] != first) atomicMax(&head_start, i + 1);
        if (i >= 0 && key[i] != first) atomicMin(&head_end, i);
        if (i >= 0 && i < n && key[i] != last) atomicMax(&tail_start, i + 1);
        if (i >= n && key[i] != last) atomicMin(&tail_end, i);
    }
    __syncthreads();
    // the run over the first place began earlier; it is long if it is more than `per` places
    const bool before = begin > 0 && head_start < 0;
    const bool head_long = before && head_end - head_start > per;
    int i0 = before && !head_long ? head_end : 0;
    // the run over the last place goes on; one that covers the CTA and began earlier is the head's
    const bool covers = before && tail_start == 0;
    const bool goes_on = tail_end > n;
    const bool tail_long = goes_on && (covers ? head_long : tail_end - tail_start > per);
    const int end = goes_on && !tail_long && !covers ? tail_end : n;
    if (threadIdx.x == 0 && blockIdx.y == 0) p.crossing[cta] = tail_long && !covers && last < p.V ? last : kNoRun;
    const int k = 8 * (blockIdx.y * blockDim.x + threadIdx.x);
    if (k >= p.K) return;
    float a[8] = {};
    bool from_before = head_long;
    for (; i0 < end; i0 += kSumBatch) {
        uint4 row[kSumBatch];
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u)
            if (i0 + u < end && key[i0 + u] < p.V)
                row[u] = __ldcs(reinterpret_cast<const uint4*>(p.dx + static_cast<int64_t>(pos[i0 + u]) * p.K + k));
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
            const int i = i0 + u;
            if (i >= end) break;
            const uint32_t run = key[i], next = key[i + 1];
            if (run >= p.V) return;  // the places without a row come last
            float v[8];
            unpack_bf16x8(row[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += v[j];
            if (next == run && i + 1 < end) continue;
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

// Joins the parts of the long runs in fp64, a warp for each summing CTA that one
// begins in (the others have nothing to do) and for 256 columns.  The parts were
// written up to a whole summing launch ago and are read from HBM behind its last
// writes, so only those of the run are, and how many they are comes first.  A run
// of more than kJoinAlone parts, as of a padding id, is divided among the CTA's
// warps, and their sums are added in order (131072 tokens of 2048 columns, half
// of them of one id: 212 us a call added, 518 when one warp's columns read all
// parts in turn).  Eight parts in flight take 118 registers and 19 us instead of
// 16 where no run is that long.
constexpr int kJoinBatch = 4;  // parts in flight per warp
constexpr int kJoinAlone = 16;
constexpr int kJoinWarps = 8;
constexpr int kJoinColumns = 256;
static_assert(kJoinAlone >= kJoinWarps, "at most one divided run begins in the places of a CTA");

// How many CTAs from `first` on begin in the run; sorted, so they are the first ones.
__device__ __forceinline__ int embed_run_parts(const SumParams& p, int first, uint32_t run) {
    const int lane = threadIdx.x & 31;
    const auto matches = [&](int64_t b, int end) {
        return __popc(__ballot_sync(0xffffffffu, b < end && p.key[b * p.per] == run));
    };
    int n = matches(first + lane, p.ctas);
    if (n < 32) return n;
    int lo = first + 32, hi = p.ctas;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        n = matches(lo + static_cast<int64_t>(lane) * step, hi);
        if (n == 0) break;
        hi = static_cast<int>(min(static_cast<int64_t>(hi), lo + static_cast<int64_t>(n) * step));
        lo += (n - 1) * step + 1;
    }
    return lo - first;
}

__device__ __forceinline__ void embed_add_parts(double (&a)[8], const SumParams& p, int from, int to, int k) {
    for (int b = from; b < to; b += kJoinBatch) {
        float4 part[kJoinBatch][2];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (b + i >= to) continue;
            const float4* head = reinterpret_cast<const float4*>(p.head + static_cast<int64_t>(b + i) * p.K + k);
            part[i][0] = head[0];
            part[i][1] = head[1];
        }
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            if (b + i >= to) continue;
            a[0] += part[i][0].x, a[1] += part[i][0].y, a[2] += part[i][0].z, a[3] += part[i][0].w;
            a[4] += part[i][1].x, a[5] += part[i][1].y, a[6] += part[i][1].z, a[7] += part[i][1].w;
        }
    }
}

__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const SumParams p) {
    __shared__ double sums[kJoinWarps][kJoinColumns];  // column 8 lane + j at 32 j + lane
    __shared__ int divided_cta, divided_parts;
    __shared__ uint32_t divided_run;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = blockIdx.x * kJoinWarps, cta = first + warp;
    const int k = kJoinColumns * blockIdx.y + 8 * lane;
    const uint32_t run = cta < p.ctas ? p.crossing[cta] : kNoRun;
    float4 tail[2] = {};
    if (run != kNoRun && k < p.K) {
        const float4* from = reinterpret_cast<const float4*>(p.tail + static_cast<int64_t>(cta) * p.K + k);
        tail[0] = from[0], tail[1] = from[1];
    }
    const int parts = run != kNoRun ? embed_run_parts(p, cta + 1, run) : 0;
    const bool divided = parts > kJoinAlone;
    if (divided && lane == 0) {
        divided_cta = cta;
        divided_parts = parts;
        divided_run = run;
    }
    if (run != kNoRun && !divided && k < p.K) {
        double a[8] = {tail[0].x, tail[0].y, tail[0].z, tail[0].w, tail[1].x, tail[1].y, tail[1].z, tail[1].w};
        float s[8];
        embed_add_parts(a, p, cta + 1, cta + 1 + parts, k);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = static_cast<float>(a[j]);
        embed_store8(p.dtable + static_cast<int64_t>(run) * p.K + k, s, p.scale, p.accumulate);
    }
    if (!__syncthreads_or(divided)) return;
    const int n = divided_parts, share = (n + kJoinWarps - 1) / kJoinWarps, begin = divided_cta + 1;
    double a[8] = {};
    if (k < p.K) embed_add_parts(a, p, begin + min(n, warp * share), begin + min(n, (warp + 1) * share), k);
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[warp][32 * j + lane] = a[j];
    __syncthreads();
    const int column = threadIdx.x, at = kJoinColumns * blockIdx.y + column;
    if (at >= p.K) return;
    double total = p.tail[static_cast<int64_t>(divided_cta) * p.K + at];
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) total += sums[i][32 * (column & 7) + (column >> 3)];
    float* to = p.dtable + static_cast<int64_t>(divided_run) * p.K + at;
    const float s = static_cast<float>(total) * p.scale;
    *to = p.accumulate ? *to + s : s;
}
static_assert(kJoinColumns == kJoinWarps * 32);

// ---------------------------------------------------------------------------
// A few tokens: one launch, nothing sorted.  A CTA per token (and up to
// 8 kFewLanes columns) reads all ids; the first token of an id lists the others
// in order and adds their rows, in fp32 up to 64 at a time and those in fp64; the
// CTAs of the later ones leave at once.  A long list, as of a padding id, is
// divided among as many slices of 8 columns a thread as fit the CTA, and their
// sums are added in order.  1000 tokens of 2560 columns added: 14.4 us a call, 31
// with half of the tokens of one id; 12.3 and 43 with twice the columns per CTA,
// 20.5 and 27 with half of them.
// ---------------------------------------------------------------------------
constexpr int kFewTokens = 1024;
constexpr int kFewThreads = 256;
constexpr int kFewLanes = 128;  // of 8 columns
constexpr int kFewGroup = 64;
constexpr int kFewBatch = 8;   // rows of dx in flight per thread
constexpr int kFewAlone = 16;  // rows that one slice adds

template <typename Id>
__global__ void __launch_bounds__(kFewThreads, 4) embed_few_kernel(const Id* __restrict__ ids,
                                                                  const uint16_t* __restrict__ dx, int64_t V, int M,
                                                                  int K, int lanes, float scale,
                                                                  float* __restrict__ dtable, int accumulate) {
    __shared__ int key[kFewTokens];
    __shared__ int pos[kFewTokens];
    __shared__ double sums[8][kFewThreads];
    __shared__ int count;
    const int m = blockIdx.x;
    for (int i = threadIdx.x; i < M; i += kFewThreads) key[i] = static_cast<int>(embed_id(ids, i, V));
    __syncthreads();
    const int mine = key[m];
    bool later = mine < 0, more = false;
    for (int i = threadIdx.x; i < M; i += kFewThreads) {
        later |= i < m && key[i] == mine;
        more |= i > m && key[i] == mine;
    }
    if (__syncthreads_or(later)) return;
    const bool several = __syncthreads_or(more);
    if (!several) {
        if (threadIdx.x == 0) pos[0] = m, count = 1;
    } else if (threadIdx.x < 32) {
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
    const int slices = count <= kFewAlone ? 1 : kFewThreads / lanes;
    const int slice = threadIdx.x / lanes, share = (count + slices - 1) / slices;
    const int k = 8 * (blockIdx.y * lanes + threadIdx.x - slice * lanes);
    const int from = min(count, slice * share), to = slice < slices && k < K ? min(count, from + share) : from;
    float a[8] = {};
    if (slices > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[j][threadIdx.x] = 0.0;
    }
    for (int i0 = from; i0 < to;) {
        const int end = min(to, i0 + kFewGroup);
        for (; i0 < end; i0 += kFewBatch) {
            uint4 row[kFewBatch];
#pragma unroll
            for (int u = 0; u < kFewBatch; ++u)
                if (i0 + u < end)
                    row[u] = __ldg(reinterpret_cast<const uint4*>(dx + static_cast<int64_t>(pos[i0 + u]) * K + k));
#pragma unroll
            for (int u = 0; u < kFewBatch; ++u) {
                if (i0 + u >= end) break;
                float v[8];
                unpack_bf16x8(row[u], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += v[j];
            }
        }
        if (slices > 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sums[j][threadIdx.x] += a[j];
                a[j] = 0.0f;
            }
        }
    }
    if (slices > 1) {
        __syncthreads();
        if (slice == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                double total = 0.0;
                for (int i = 0; i < slices; ++i) total += sums[j][i * lanes + threadIdx.x];
                a[j] = static_cast<float>(total);
            }
        }
    }
    if (slice == 0 && k < K) embed_store8(dtable + static_cast<int64_t>(mine) * K + k, a, scale, accumulate);
}

}  // namespace mmf
