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
#pragma once
#include "common.cuh"
#include "scan.cuh"

namespace mmf {

// max(v, kScanClamp) that passes a NaN on (fmaxf would return the clamp).
__device__ __forceinline__ float clamp_nan(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(kScanClamp));
    return r;
}

// e^-v, 1 + e^-v of the clamped pre-activation
__device__ __forceinline__ float sig_exp(float v) { return ex2_ftz(-kLog2e * clamp_nan(v)); }

constexpr int kSbSub = 8;      // tokens between two kept states
constexpr int kSbWarps = 4;    // warps per CTA, each on 64 channels of its own

// h -> f h + (1 - f) c of one token and channel
__device__ __forceinline__ float scan_step(float fp, float cp, float h) {
    const float ef = sig_exp(fp), ec = sig_exp(cp);
    const float df = 1.0f + ef, dc = 1.0f + ec;
    const float r = rcp_ftz(df * dc);
    const float f = r * dc;
    return fmaf(f, h, ef * f * (cp * (r * df)));
}

// A warp takes 64 channels (a bf16 pair per lane) of one sequence: forward
// through the tokens, keeping the state before every kSbSub-th token in `kept`
// ([B][ceil(T / kSbSub)][D] fp32), then backwards, kSbSub tokens at a time,
// their states recomputed from the kept one.
__global__ void __launch_bounds__(kSbWarps * 32) mlgru_scan_bwd_kernel(
    const uint16_t* __restrict__ f_pre, const uint16_t* __restrict__ c_pre, const uint16_t* __restrict__ g_pre,
    const uint16_t* __restrict__ d_o, const float* __restrict__ h0, const float* __restrict__ dh_last, int T, int D,
    float* __restrict__ kept, uint16_t* __restrict__ df_pre, uint16_t* __restrict__ dc_pre,
    uint16_t* __restrict__ dg_pre, float* __restrict__ dh0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t b = blockIdx.y;
    const int k = (blockIdx.x * kSbWarps + warp) * 64 + 2 * lane;  // this lane's channels k, k + 1
    if (k >= D) return;                                            // D is even, so k + 1 < D too
    const int subs = (T + kSbSub - 1) / kSbSub;
    const int64_t base = b * T * static_cast<int64_t>(D) + k;
    float* keep = kept + b * subs * static_cast<int64_t>(D) + k;
    float2 h = make_float2(0.0f, 0.0f);
    if (h0) h = *reinterpret_cast<const float2*>(h0 + b * D + k);
    for (int t = 0; t < T; ++t) {
        if (t % kSbSub == 0) *reinterpret_cast<float2*>(keep + (t / kSbSub) * static_cast<int64_t>(D)) = h;
        float fp0, fp1, cp0, cp1;
        const int64_t at = base + t * static_cast<int64_t>(D);
        bf16x2_to_f(__ldg(reinterpret_cast<const uint32_t*>(f_pre + at)), fp0, fp1);
        bf16x2_to_f(__ldg(reinterpret_cast<const uint32_t*>(c_pre + at)), cp0, cp1);
        h.x = scan_step(fp0, cp0, h.x);
        h.y = scan_step(fp1, cp1, h.y);
    }
    float dh[2] = {0.0f, 0.0f};
    if (dh_last) {
        const float2 v = *reinterpret_cast<const float2*>(dh_last + b * D + k);
        dh[0] = v.x;
        dh[1] = v.y;
    }
    for (int s = subs - 1; s >= 0; --s) {
        const float2 hv = *reinterpret_cast<const float2*>(keep + s * static_cast<int64_t>(D));
        float hp[kSbSub + 1][2];   // hp[i]: the state before token i of these
        hp[0][0] = hv.x;
        hp[0][1] = hv.y;
        const int n = min(kSbSub, T - s * kSbSub);
        const int64_t at0 = base + static_cast<int64_t>(s) * kSbSub * D;
        uint32_t rf[kSbSub], rc[kSbSub];
#pragma unroll
        for (int i = 0; i < kSbSub; ++i) {
            if (i < n) {
                rf[i] = __ldg(reinterpret_cast<const uint32_t*>(f_pre + at0 + i * static_cast<int64_t>(D)));
                rc[i] = __ldg(reinterpret_cast<const uint32_t*>(c_pre + at0 + i * static_cast<int64_t>(D)));
                float fp[2], cp[2];
                bf16x2_to_f(rf[i], fp[0], fp[1]);
                bf16x2_to_f(rc[i], cp[0], cp[1]);
                hp[i + 1][0] = scan_step(fp[0], cp[0], hp[i][0]);
                hp[i + 1][1] = scan_step(fp[1], cp[1], hp[i][1]);
            } else {
                rf[i] = rc[i] = 0;
                hp[i + 1][0] = hp[i + 1][1] = 0.0f;
            }
        }
#pragma unroll
        for (int i = kSbSub - 1; i >= 0; --i) {
            if (i < n) {
                const int64_t at = at0 + i * static_cast<int64_t>(D);
                float fp[2], cp[2], gp[2], dov[2], ov[3][2];
                bf16x2_to_f(rf[i], fp[0], fp[1]);
                bf16x2_to_f(rc[i], cp[0], cp[1]);
                bf16x2_to_f(__ldg(reinterpret_cast<const uint32_t*>(g_pre + at)), gp[0], gp[1]);
                bf16x2_to_f(__ldg(reinterpret_cast<const uint32_t*>(d_o + at)), dov[0], dov[1]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float ef = sig_exp(fp[j]), ec = sig_exp(cp[j]), eg = sig_exp(gp[j]);
                    const float df = 1.0f + ef, dc = 1.0f + ec, dg = 1.0f + eg;
                    const float dfc = df * dc;
                    const float r = rcp_ftz(dfc * dg);
                    const float rg = r * dg;                      // 1 / (df dc)
                    const float f = rg * dc, sc = rg * df, g = r * dfc;
                    const float omf = ef * f, omc = ec * sc, omg = eg * g;  // 1 - f, 1 - sigma(c_pre), 1 - g
                    const float d = fmaf(dov[j], g, dh[j]);
                    ov[2][j] = dov[j] * hp[i + 1][j] * (g * omg);
                    ov[0][j] = d * (hp[i][j] - cp[j] * sc) * (f * omf);
                    ov[1][j] = d * omf * (sc * fmaf(cp[j], omc, 1.0f));
                    dh[j] = d * f;
                }
                *reinterpret_cast<__nv_bfloat162*>(df_pre + at) = __floats2bfloat162_rn(ov[0][0], ov[0][1]);
                *reinterpret_cast<__nv_bfloat162*>(dc_pre + at) = __floats2bfloat162_rn(ov[1][0], ov[1][1]);
                *reinterpret_cast<__nv_bfloat162*>(dg_pre + at) = __floats2bfloat162_rn(ov[2][0], ov[2][1]);
            }
        }
    }
    if (dh0) *reinterpret_cast<float2*>(dh0 + b * D + k) = make_float2(dh[0], dh[1]);
}

}  // namespace mmf
