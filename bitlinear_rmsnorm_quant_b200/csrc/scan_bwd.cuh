// scan_bwd.cuh -- gradient of the MLGRU recurrence (scan.cuh).  With
//   f = sigma(f_pre), s = sigma(c_pre), c = c_pre s, g = sigma(g_pre),
//   h_t = f_t h_{t-1} + (1 - f_t) c_t,  o_t = g_t h_t
// the state's gradient runs backwards through the tokens,
//   dh_t = do_t g_t + f_{t+1} dh_{t+1}   (dh_T also gets dh_last), dh0 = f_1 dh_1,
// and every token gives
//   dg_pre = do h_t g (1 - g)
//   df_pre = dh_t (h_{t-1} - c_t) f (1 - f)
//   dc_pre = dh_t (1 - f) s (1 + c_pre (1 - s)).
// 1 - sigma(v) is taken as e^-v sigma(v), which keeps its precision where
// sigma(v) is close to 1.
//
// Both recurrences are linear, so a run of tokens acts on them as
//   h -> A h + P  (forward)  and  dh -> A dh + R  (backward), A = prod f,
// and P and R both come out of one forward walk (R = sum A_t do_t g_t with A_t
// the product up to token t).  The tokens of a sequence are split into
// segments; mlgru_scan_bwd_maps_kernel walks each and leaves its (A, P, R),
// and on the way the (A, P) of the tokens before every kSbSub-th one.
// mlgru_scan_bwd_kernel folds the segments before and behind its own into the
// state and the gradient that enter it, and takes it backwards, kSbSub tokens
// at a time: their gates once, their states forward from the kept map, their
// gradients backward.  A warp works alone, on 64 channels (a bf16 pair per
// lane) of one segment: no barriers, and any number of channels, segments and
// sequences fills the GPU alike.
//
// Bound and measured: 14 bytes a token and channel (f, c, g, do read, the
// gradients written) are the least; the second launch reads the first four
// again, from L2 where they fit, and the kept maps are a byte written and read,
// 24 in all.  16 x 2048 x 2048: 262 us on the device, 1.55 GB at 5.9 TB/s (276
// where calls follow one another).  4 x 2048 x 2048: 68 us, 29 for the maps (4.8
// TB/s) and 39 for the gradients, which a quarter of the reads find in L2 and 76
// instructions a channel pair at two a cycle bind (73 where calls follow one
// another; 16 warps of 122 registers an SM; 24 of 80, with half the tokens at a
// time, took 72 us).
#pragma once
#include "common.cuh"
#include "scan.cuh"

namespace mmf {

constexpr int kSbSub = 8;      // tokens taken backwards at a time
constexpr int kSbWarps = 4;    // warps per CTA, each on a segment of its own

// a bf16 pair -> fp32 pair
__device__ __forceinline__ f2 f2_bf16(uint32_t w) {
    return f2_make(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// a bf16 pair raised to at least kScanClamp (-28 is a bf16 value); a NaN stays, or (floor) becomes kScanClamp too
__device__ __forceinline__ uint32_t clamp_bf16x2(uint32_t w) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xC1E0C1E0u));
    return r;
}
__device__ __forceinline__ uint32_t floor_bf16x2(uint32_t w) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0xC1E0C1E0u));
    return r;
}
__device__ __forceinline__ f2 f2_exp_neg(f2 v) {  // e^-v
    const float2 a = f2_get(f2_mul(v, f2_set(-kLog2e)));
    return f2_make(ex2_ftz(a.x), ex2_ftz(a.y));
}
// e^-v of a v at least kScanClamp; of a NaN e^28
__device__ __forceinline__ f2 f2_exp_neg_number(f2 v) {
    const float2 a = f2_get(f2_mul(v, f2_set(-kLog2e)));
    return f2_make(ex2_ftz(fminf(a.x, -kLog2e * kScanClamp)), ex2_ftz(fminf(a.y, -kLog2e * kScanClamp)));
}
// do g of a gate from ScanGates, a NaN where its pre-activation is one
__device__ __forceinline__ f2 f2_gated(uint32_t wd, uint32_t wg, f2 g) {
    uint32_t nan;
    asm("set.nan.u32.bf16x2 %0, %1, %1;" : "=r"(nan) : "r"(wg));
    return f2_mul(f2_bf16(wd | nan), g);
}
__device__ __forceinline__ uint32_t f2_to_bf16(f2 v) {
    const float2 a = f2_get(v);
    const __nv_bfloat162 b = __floats2bfloat162_rn(a.x, a.y);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// The gates of one token from its (clamped) pre-activations: one reciprocal
// gives all three sigmoids (scan.cuh).  A NaN of f_pre makes the token's gates
// NaN, which every output it has a part in is; one of c_pre or g_pre must not
// reach the others (a NaN of f would spread over the whole sequence), so s and g
// are numbers then: cp keeps the NaN of c_pre, and f2_gated puts back that of g_pre.
struct ScanGates {
    f2 cp, ef, ec, eg, f, s, g;
    __device__ __forceinline__ ScanGates(uint32_t wf, uint32_t wc, uint32_t wg) {
        cp = f2_bf16(clamp_bf16x2(wc));
        ef = f2_exp_neg(f2_bf16(clamp_bf16x2(wf)));
        ec = f2_exp_neg_number(cp);
        eg = f2_exp_neg(f2_bf16(floor_bf16x2(wg)));
        const f2 one = f2_set(1.0f);
        const f2 df = f2_add(one, ef), dc = f2_add(one, ec), dg = f2_add(one, eg);
        const f2 dfc = f2_mul(df, dc);
        const float2 all = f2_get(f2_mul(dfc, dg));
        const f2 r = f2_make(rcp_ftz(all.x), rcp_ftz(all.y));
        const f2 rg = f2_mul(r, dg);  // 1 / (df dc)
        f = f2_mul(rg, dc);
        s = f2_mul(rg, df);
        g = f2_mul(r, dfc);
    }
};

struct ScanBwdParams {
    const uint16_t *f_pre, *c_pre, *g_pre, *d_o;
    const float *h0, *dh_last;
    uint16_t *df_pre, *dc_pre, *dg_pre;
    float* dh0;
    float4* part;  // [B][subs][D / 2] (A, A, P, P) of the segment's tokens before each kSbSub-th
    float4* seg;   // [B][S][D / 2] (A, A, P, P) of a segment
    float2* seg_r; // [B][S][D / 2] R of a segment
    int T, D, S, subs, subs_per_seg, tiles;
    int64_t items; // B * S * tiles
};

// Which segment a warp takes, and where its data begins.
struct ScanItem {
    int64_t b;
    int seg, k;      // k: this lane's first channel
    bool valid;      // D is even, so k + 1 < D too
    __device__ __forceinline__ ScanItem(const ScanBwdParams& p, int64_t item) {
        const int tile = static_cast<int>(item % p.tiles);
        const int64_t bs = item / p.tiles;
        seg = static_cast<int>(bs % p.S);
        b = bs / p.S;
        k = tile * 64 + 2 * (threadIdx.x & 31);
        valid = k < p.D;
    }
};

__device__ __forceinline__ uint32_t ld_pair(const uint16_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); }

__global__ void __launch_bounds__(kSbWarps * 32) mlgru_scan_bwd_maps_kernel(const ScanBwdParams p) {
    pdl_launch_dependents();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kSbWarps + (threadIdx.x >> 5);
    if (item >= p.items) return;
    const ScanItem it(p, item);
    if (!it.valid) return;
    const int sub0 = it.seg * p.subs_per_seg, sub1 = min(p.subs, sub0 + p.subs_per_seg);
    const int64_t half = p.D / 2;
    f2 A = f2_set(1.0f), P = f2_set(0.0f), R = f2_set(0.0f);
    for (int sub = sub0; sub < sub1; ++sub) {
        const int t0 = sub * kSbSub;
        const int64_t at = (it.b * p.T + t0) * p.D + it.k;
        const float2 a = f2_get(A), q = f2_get(P);
        p.part[(it.b * p.subs + sub) * half + it.k / 2] = make_float4(a.x, a.y, q.x, q.y);
        const int n = min(kSbSub, p.T - t0);
        uint32_t wf[kSbSub], wc[kSbSub], wg[kSbSub], wd[kSbSub];
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) {
            const int64_t o = at + static_cast<int64_t>(i) * p.D;
            const bool there = i < n;
            wf[i] = there ? ld_pair(p.f_pre + o) : 0u;
            wc[i] = there ? ld_pair(p.c_pre + o) : 0u;
            wg[i] = there ? ld_pair(p.g_pre + o) : 0u;
            wd[i] = there ? ld_pair(p.d_o + o) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) {
            if (i >= n) break;
            const ScanGates t(wf[i], wc[i], wg[i]);
            A = f2_mul(A, t.f);
            P = f2_fma(t.f, P, f2_mul(f2_mul(t.ef, t.f), f2_mul(t.cp, t.s)));
            R = f2_fma(A, f2_gated(wd[i], wg[i], t.g), R);
        }
    }
    const float2 a = f2_get(A), q = f2_get(P), r = f2_get(R);
    const int64_t to = (it.b * p.S + it.seg) * half + it.k / 2;
    p.seg[to] = make_float4(a.x, a.y, q.x, q.y);
    p.seg_r[to] = r;
}

// n (at most kSbSub) tokens from element `at` on, taken backwards: hs is the
// state before them, dh the gradient of the state behind them and then of hs.
__device__ __forceinline__ void scan_back(const ScanBwdParams& p, int64_t at, int n, f2 hs, f2& dh) {
    uint32_t wf[kSbSub], wc[kSbSub], wg[kSbSub], wd[kSbSub];
#pragma unroll
    for (int i = 0; i < kSbSub; ++i) {
        const int64_t o = at + static_cast<int64_t>(i) * p.D;
        const bool there = i < n;
        wf[i] = there ? ld_pair(p.f_pre + o) : 0u;
        wc[i] = there ? ld_pair(p.c_pre + o) : 0u;
        wg[i] = there ? ld_pair(p.g_pre + o) : 0u;
        wd[i] = there ? ld_pair(p.d_o + o) : 0u;
    }
    // of each token: what dh is multiplied with for df_pre, dc_pre and the token before, and do g
    f2 xf[kSbSub], xc[kSbSub], fg[kSbSub], dg[kSbSub];
#pragma unroll
    for (int i = 0; i < kSbSub; ++i) {
        if (i >= n) break;
        const ScanGates t(wf[i], wc[i], wg[i]);
        const f2 omf = f2_mul(t.ef, t.f);   // 1 - f
        const f2 c = f2_mul(t.cp, t.s);
        xf[i] = f2_mul(f2_fma(c, f2_set(-1.0f), hs), f2_mul(t.f, omf));
        xc[i] = f2_mul(omf, f2_mul(t.s, f2_fma(t.cp, f2_mul(t.ec, t.s), f2_set(1.0f))));
        hs = f2_fma(t.f, hs, f2_mul(omf, c));
        fg[i] = t.f;
        dg[i] = f2_gated(wd[i], wg[i], t.g);
        *reinterpret_cast<uint32_t*>(p.dg_pre + at + static_cast<int64_t>(i) * p.D) =
            f2_to_bf16(f2_mul(f2_mul(dg[i], hs), f2_mul(t.eg, t.g)));
    }
#pragma unroll
    for (int i = kSbSub - 1; i >= 0; --i) {
        if (i >= n) continue;
        const int64_t o = at + static_cast<int64_t>(i) * p.D;
        const f2 d = f2_add(dg[i], dh);
        *reinterpret_cast<uint32_t*>(p.df_pre + o) = f2_to_bf16(f2_mul(d, xf[i]));
        *reinterpret_cast<uint32_t*>(p.dc_pre + o) = f2_to_bf16(f2_mul(d, xc[i]));
        dh = f2_mul(d, fg[i]);
    }
}

__global__ void __launch_bounds__(kSbWarps * 32, 3) mlgru_scan_bwd_kernel(const ScanBwdParams p) {
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kSbWarps + (threadIdx.x >> 5);
    if (item >= p.items) return;
    // the last segments first: the maps kernel has just read them
    const ScanItem it(p, p.items - 1 - item);
    if (!it.valid) return;
    const int sub0 = it.seg * p.subs_per_seg, sub1 = min(p.subs, sub0 + p.subs_per_seg);
    const int64_t half = p.D / 2;
    f2 h = f2_set(0.0f), dh = f2_set(0.0f);
    if (p.h0) h = *reinterpret_cast<const f2*>(p.h0 + it.b * p.D + it.k);
    if (p.dh_last) dh = *reinterpret_cast<const f2*>(p.dh_last + it.b * p.D + it.k);
    pdl_wait();
    {
        const float4* seg = p.seg + it.b * p.S * half + it.k / 2;
        const float2* seg_r = p.seg_r + it.b * p.S * half + it.k / 2;
#pragma unroll 4
        for (int s = 0; s < it.seg; ++s) {
            const float4 m = seg[s * half];
            h = f2_fma(f2_make(m.x, m.y), h, f2_make(m.z, m.w));
        }
#pragma unroll 4
        for (int s = p.S - 1; s > it.seg; --s) {
            const float4 m = seg[s * half];
            const float2 r = seg_r[s * half];
            dh = f2_fma(f2_make(m.x, m.y), dh, f2_make(r.x, r.y));
        }
    }
    for (int sub = sub1 - 1; sub >= sub0; --sub) {
        const int t0 = sub * kSbSub;
        const float4 m = p.part[(it.b * p.subs + sub) * half + it.k / 2];
        scan_back(p, (it.b * p.T + t0) * p.D + it.k, min(kSbSub, p.T - t0),
                  f2_fma(f2_make(m.x, m.y), h, f2_make(m.z, m.w)), dh);
    }
    if (p.dh0 && it.seg == 0) *reinterpret_cast<float2*>(p.dh0 + it.b * p.D + it.k) = f2_get(dh);
}

// Short sequences (kSbShort tokens at most) in one launch: a warp walks its 64
// channels' tokens forward, keeping the state before every kSbSub-th in shared
// memory, and takes them backwards from there.
constexpr int kSbShort = 40;

__global__ void __launch_bounds__(kSbWarps * 32, 3) mlgru_scan_bwd_short_kernel(const ScanBwdParams p) {
    __shared__ float2 kept[kSbWarps][kSbShort / kSbSub][32];
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kSbWarps + (threadIdx.x >> 5);
    if (item >= p.items) return;
    const ScanItem it(p, item);  // S = 1
    if (!it.valid) return;
    const int lane = threadIdx.x & 31;
    float2(*keep)[32] = kept[threadIdx.x >> 5];
    f2 h = f2_set(0.0f), dh = f2_set(0.0f);
    if (p.h0) h = *reinterpret_cast<const f2*>(p.h0 + it.b * p.D + it.k);
    if (p.dh_last) dh = *reinterpret_cast<const f2*>(p.dh_last + it.b * p.D + it.k);
    const int64_t base = it.b * p.T * p.D + it.k;
    for (int sub = 0; sub < p.subs; ++sub) {
        keep[sub][lane] = f2_get(h);
        const int n = min(kSbSub, p.T - sub * kSbSub);
        const int64_t at = base + static_cast<int64_t>(sub) * kSbSub * p.D;
        uint32_t wf[kSbSub], wc[kSbSub];
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) {
            wf[i] = i < n ? ld_pair(p.f_pre + at + static_cast<int64_t>(i) * p.D) : 0u;
            wc[i] = i < n ? ld_pair(p.c_pre + at + static_cast<int64_t>(i) * p.D) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) {
            if (i >= n) break;
            const f2 cp = f2_bf16(clamp_bf16x2(wc[i])), ef = f2_exp_neg(f2_bf16(clamp_bf16x2(wf[i])));
            const f2 df = f2_add(f2_set(1.0f), ef), dc = f2_add(f2_set(1.0f), f2_exp_neg(cp));
            const float2 d = f2_get(f2_mul(df, dc));
            const f2 r = f2_make(rcp_ftz(d.x), rcp_ftz(d.y));
            const f2 f = f2_mul(r, dc);
            h = f2_fma(f, h, f2_mul(f2_mul(ef, f), f2_mul(cp, f2_mul(r, df))));
        }
    }
    for (int sub = p.subs - 1; sub >= 0; --sub) {
        const float2 hs = keep[sub][lane];
        scan_back(p, base + static_cast<int64_t>(sub) * kSbSub * p.D, min(kSbSub, p.T - sub * kSbSub),
                  f2_make(hs.x, hs.y), dh);
    }
    if (p.dh0) *reinterpret_cast<float2*>(p.dh0 + it.b * p.D + it.k) = f2_get(dh);
}

// ---------------------------------------------------------------------------
// The same two kernels with the tensors moved by tensor copies.  A CTA of GW
// warps takes GW * 64 neighbouring channels of one segment, a warp 64 of them;
// kSbSub tokens of f, c, g and do at a time come into a ring of kSbStages
// stages in shared memory; a lane leaves df, dc and dg where it read f, c and g,
// and they are copied out from there.  After the one barrier per kSbSub tokens
// the first thread starts the copies out of this stage and, once those of the
// stage before have been read, the copies in for the stage after the next.  The
// maps are [B][T][D] bf16, so a copy stops at the sequence's end (what it reads
// beyond is zeros, what it would write beyond is dropped).  Needs D % 8 == 0
// (16-byte row pitch) and D >= 64; other shapes take the kernels above.
// ---------------------------------------------------------------------------
constexpr int kSbStages = 3;
constexpr int kSbMaxGw = 4;
__host__ __device__ constexpr uint32_t sb_tile(int gw) { return kSbSub * 128u * gw; }  // one tensor's kSbSub tokens
__host__ __device__ constexpr uint32_t sb_stage(int gw) { return 4 * sb_tile(gw); }    // f, c, g, do
__host__ __device__ constexpr size_t sb_smem(int gw) { return kSbStages * size_t(sb_stage(gw)); }

struct ScanBwdMaps {
    CUtensorMap f, c, g, d_o, df, dc, dg;
};

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// at most N of this thread's groups of copies are still reading shared memory
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// The CTA's place: its sequence, segment and first channel.
struct ScanPlace {
    int b, seg, x, sub0, sub1;
    __device__ __forceinline__ ScanPlace(const ScanBwdParams& p, unsigned item, int gw) {
        const unsigned groups = static_cast<unsigned>(p.tiles);
        const unsigned bs = item / groups;
        x = static_cast<int>(item - bs * groups) * 64 * gw;
        b = static_cast<int>(bs / static_cast<unsigned>(p.S));
        seg = static_cast<int>(bs - static_cast<unsigned>(b) * static_cast<unsigned>(p.S));
        sub0 = seg * p.subs_per_seg;
        sub1 = min(p.subs, sub0 + p.subs_per_seg);
    }
};

template <int GW>
__device__ __forceinline__ void scan_stage_load(const ScanBwdMaps& maps, uint8_t* dst, uint64_t* full, int x, int sub, int b) {
    mbar_arrive_expect_tx(full, sb_stage(GW));
    tma_load_3d(dst, &maps.f, x, sub * kSbSub, b, full);
    tma_load_3d(dst + sb_tile(GW), &maps.c, x, sub * kSbSub, b, full);
    tma_load_3d(dst + 2 * sb_tile(GW), &maps.g, x, sub * kSbSub, b, full);
    tma_load_3d(dst + 3 * sb_tile(GW), &maps.d_o, x, sub * kSbSub, b, full);
}

// Waits for stage j of the CTA's ring.  A thread whose wait gives up (and sets
// the abort flag, so every other's does) waits for the copies still in flight,
// bounded too, and leaves; a barrier does not count threads that have left.
template <int IN_FLIGHT>
__device__ __forceinline__ bool scan_stage_wait(uint64_t* full, int j, int count, volatile int* abort_flag) {
    if (mbar_wait(&full[j % kSbStages], (j / kSbStages) & 1, abort_flag)) return true;
    for (int i = j; i < j + IN_FLIGHT && i < count; ++i) {
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[i % kSbStages], (i / kSbStages) & 1) && globaltimer_ns() - t0 <= kWaitLimitNs) {
        }
    }
    return false;
}

template <int GW>
__device__ __forceinline__ uint32_t tile_pair(const uint8_t* mine, int tensor, int i) {
    return *reinterpret_cast<const uint32_t*>(mine + tensor * sb_tile(GW) + i * (128 * GW));
}

template <int GW>
__global__ void __launch_bounds__(GW * 32) mlgru_scan_bwd_maps_tma_kernel(const ScanBwdParams p,
                                                                         const __grid_constant__ ScanBwdMaps maps) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kSbStages];
    __shared__ int abort_flag;
    pdl_launch_dependents();
    const ScanPlace at(p, blockIdx.x, GW);
    const int count = at.sub1 - at.sub0;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kSbStages; ++i) mbar_init(&full[i], 1);
        mbar_fence_init();
        for (int i = 0; i < kSbStages && i < count; ++i)
            scan_stage_load<GW>(maps, smem + i * sb_stage(GW), &full[i], at.x, at.sub0 + i, at.b);
    }
    __syncthreads();
    const int k = at.x + 2 * static_cast<int>(threadIdx.x);  // this lane's channels k, k + 1
    const bool valid = k < p.D;                              // D is even, so k + 1 < D too
    const int64_t half = p.D / 2;
    f2 A = f2_set(1.0f), P = f2_set(0.0f), R = f2_set(0.0f);
    float4* part = p.part + (static_cast<int64_t>(at.b) * p.subs + at.sub0) * half + k / 2;
    for (int j = 0; j < count; ++j) {
        if (valid) {
            const float2 a = f2_get(A), q = f2_get(P);
            *part = make_float4(a.x, a.y, q.x, q.y);
        }
        part += half;
        if (!scan_stage_wait<kSbStages>(full, j, count, &abort_flag)) return;  // the others find the abort flag set
        const uint8_t* mine = smem + (j % kSbStages) * sb_stage(GW) + 4 * threadIdx.x;
        // the gates of kBatch tokens side by side (their chains of dependent
        // instructions overlap), then their turns in the recurrences
        constexpr int kBatch = 4;
        const int n = p.T - (at.sub0 + j) * kSbSub;
#pragma unroll
        for (int i0 = 0; i0 < kSbSub; i0 += kBatch) {
            f2 f[kBatch], q[kBatch], x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t wg = tile_pair<GW>(mine, 2, i0 + i);
                const ScanGates t(tile_pair<GW>(mine, 0, i0 + i), tile_pair<GW>(mine, 1, i0 + i), wg);
                f[i] = t.f;
                q[i] = f2_mul(f2_mul(t.ef, t.f), f2_mul(t.cp, t.s));
                x[i] = f2_gated(tile_pair<GW>(mine, 3, i0 + i), wg, t.g);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i0 + i >= n) break;
                A = f2_mul(A, f[i]);
                P = f2_fma(f[i], P, q[i]);
                R = f2_fma(A, x[i], R);
            }
        }
        __syncthreads();  // the stage has been read
        if (threadIdx.x == 0 && j + kSbStages < count)
            scan_stage_load<GW>(maps, smem + (j % kSbStages) * sb_stage(GW), &full[j % kSbStages], at.x,
                                at.sub0 + j + kSbStages, at.b);
    }
    if (!valid) return;
    const float2 a = f2_get(A), q = f2_get(P), r = f2_get(R);
    const int64_t to = (static_cast<int64_t>(at.b) * p.S + at.seg) * half + k / 2;
    p.seg[to] = make_float4(a.x, a.y, q.x, q.y);
    p.seg_r[to] = r;
}

template <int GW>
__global__ void __launch_bounds__(GW * 32, 16 / GW) mlgru_scan_bwd_tma_kernel(const ScanBwdParams p,
                                                                             const __grid_constant__ ScanBwdMaps maps) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kSbStages];
    __shared__ int abort_flag;
    // the last segments first: the maps kernel has just read them
    const ScanPlace at(p, gridDim.x - 1 - blockIdx.x, GW);
    const int count = at.sub1 - at.sub0;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int i = 0; i < kSbStages; ++i) mbar_init(&full[i], 1);
        mbar_fence_init();
        for (int i = 0; i < kSbStages - 1 && i < count; ++i)
            scan_stage_load<GW>(maps, smem + i * sb_stage(GW), &full[i], at.x, at.sub1 - 1 - i, at.b);
    }
    __syncthreads();
    const int k = at.x + 2 * static_cast<int>(threadIdx.x);
    const bool valid = k < p.D;
    const int64_t half = p.D / 2;
    f2 h = f2_set(0.0f), dh = f2_set(0.0f);
    if (p.h0 && valid) h = *reinterpret_cast<const f2*>(p.h0 + static_cast<int64_t>(at.b) * p.D + k);
    if (p.dh_last && valid) dh = *reinterpret_cast<const f2*>(p.dh_last + static_cast<int64_t>(at.b) * p.D + k);
    pdl_wait();
    if (valid) {
        const float4* seg = p.seg + static_cast<int64_t>(at.b) * p.S * half + k / 2;
        const float2* seg_r = p.seg_r + static_cast<int64_t>(at.b) * p.S * half + k / 2;
#pragma unroll 8
        for (int s = 0; s < at.seg; ++s) {
            const float4 m = seg[s * half];
            h = f2_fma(f2_make(m.x, m.y), h, f2_make(m.z, m.w));
        }
#pragma unroll 8
        for (int s = p.S - 1; s > at.seg; --s) {
            const float4 m = seg[s * half];
            const float2 r = seg_r[s * half];
            dh = f2_fma(f2_make(m.x, m.y), dh, f2_make(r.x, r.y));
        }
    }
    const float4* part = p.part + (static_cast<int64_t>(at.b) * p.subs + at.sub1 - 1) * half + k / 2;
    float4 next = valid ? *part : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    bool ok = true;
    for (int j = 0; j < count; ++j) {
        const int sub = at.sub1 - 1 - j;
        const float4 m = next;
        if (valid && j + 1 < count) next = *(part -= half);
        f2 hs = f2_fma(f2_make(m.x, m.y), h, f2_make(m.z, m.w));  // the state before these tokens
        ok = scan_stage_wait<kSbStages - 1>(full, j, count, &abort_flag);
        if (!ok) break;  // the others find the abort flag set
        uint8_t* mine = smem + (j % kSbStages) * sb_stage(GW) + 4 * threadIdx.x;
        // of each token: what dh is multiplied with for df_pre, dc_pre and the token before, and do g
        f2 xf[kSbSub], xc[kSbSub], fg[kSbSub], dg[kSbSub];
        const auto ahead = [&](int i) {
            const uint32_t wg = tile_pair<GW>(mine, 2, i);
            const ScanGates t(tile_pair<GW>(mine, 0, i), tile_pair<GW>(mine, 1, i), wg);
            const f2 omf = f2_mul(t.ef, t.f);   // 1 - f
            const f2 c = f2_mul(t.cp, t.s);
            xf[i] = f2_mul(f2_fma(c, f2_set(-1.0f), hs), f2_mul(t.f, omf));
            xc[i] = f2_mul(omf, f2_mul(t.s, f2_fma(t.cp, f2_mul(t.ec, t.s), f2_set(1.0f))));
            hs = f2_fma(t.f, hs, f2_mul(omf, c));
            fg[i] = t.f;
            dg[i] = f2_gated(tile_pair<GW>(mine, 3, i), wg, t.g);
            *reinterpret_cast<uint32_t*>(mine + 2 * sb_tile(GW) + i * (128 * GW)) =
                f2_to_bf16(f2_mul(f2_mul(dg[i], hs), f2_mul(t.eg, t.g)));
        };
        const auto back = [&](int i) {
            const f2 d = f2_add(dg[i], dh);
            *reinterpret_cast<uint32_t*>(mine + i * (128 * GW)) = f2_to_bf16(f2_mul(d, xf[i]));
            *reinterpret_cast<uint32_t*>(mine + sb_tile(GW) + i * (128 * GW)) = f2_to_bf16(f2_mul(d, xc[i]));
            dh = f2_mul(d, fg[i]);
        };
        const int n = p.T - sub * kSbSub;
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) ahead(i);  // tokens past the end read zeros and are not written
        constexpr int ahead_by = kSbStages - 1;
        if (threadIdx.x == 0 && j + ahead_by < count) {
            const int slot = (j + ahead_by) % kSbStages;
            bulk_wait_read<0>();  // the copies out of this slot, a stage ago, have been read
            scan_stage_load<GW>(maps, smem + slot * sb_stage(GW), &full[slot], at.x, sub - ahead_by, at.b);
        }
        if (n >= kSbSub) {
#pragma unroll
            for (int i = kSbSub - 1; i >= 0; --i) back(i);
        } else {
#pragma unroll
            for (int i = kSbSub - 1; i >= 0; --i)
                if (i < n) back(i);
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            const uint8_t* from = smem + (j % kSbStages) * sb_stage(GW);
            tma_store_3d(&maps.df, from, at.x, sub * kSbSub, at.b);
            tma_store_3d(&maps.dc, from + sb_tile(GW), at.x, sub * kSbSub, at.b);
            tma_store_3d(&maps.dg, from + 2 * sb_tile(GW), at.x, sub * kSbSub, at.b);
            bulk_commit();
        }
    }
    if (threadIdx.x == 0) bulk_wait_read<0>();
    if (ok && p.dh0 && valid && at.seg == 0)
        *reinterpret_cast<float2*>(p.dh0 + static_cast<int64_t>(at.b) * p.D + k) = f2_get(dh);
}

}  // namespace mmf
