// adamw.cuh -- one AdamW step over many tensors in one launch, with the two
// moments held in fp32 or in 8 bits.  Per element, each product and sum of the
// moments rounded to fp32 in this order (their bits decide the 8-bit codes):
//   g' = g * grad_scale
//   m  = m * beta1 + g' * (1 - beta1)
//   v  = v * beta2 + (g' * g') * (1 - beta2)
//   p  = p * (1 - lr * weight_decay) - alpha * (m / (sqrt(v) * r + eps)),
//        alpha = lr / (1 - beta1^step),  r = 1 / sqrt(1 - beta2^step)
// (square root and division by the hardware's approximations, a few ulp of the
// update).  8-bit moments: blocks of 256 elements share a power of two each,
//   m = e4m3 code * m_scale, the block's largest |m| / m_scale in [2^7, 2^8),
//   v = e5m2 code * v_scale, the block's largest  v  / v_scale in [2^14, 2^15),
// so both span 2^14 below the block's largest (v, read as sqrt(v)).  A
// moment's change of 1 - beta per step is far below an 8-bit code's step, so
// rounding to nearest would stop it from moving; the codes are rounded up or
// down at random with the right mean instead, by 16 bits a moment of the
// SplitMix64 stream (seed, tensor).  The update takes the moments before they
// are rounded.  |m| below the smallest normal code becomes 0; a positive v is
// kept at least at the smallest normal code, so it never reads as 0.
#pragma once
#include "common.cuh"

namespace mmf {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = 256;                              // elements that share the scales
constexpr int kAdamRounds = 2;                               // blocks per warp
constexpr int kAdamChunk = kAdamWarps * kAdamRounds * kAdamBlock;  // elements per CTA

// One tensor as the kernel sees it.
struct AdamTensor {
    float* p;
    const void* g;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    uint16_t* p_bf16;
    int64_t n;
    unsigned long long key;  // of the tensor's noise stream
    float weight_decay;
    int flags;               // kAdam8, kAdamGradBf16
};
constexpr int kAdam8 = 1, kAdamGradBf16 = 2;

struct AdamScalars {
    float lr, alpha, r, grad_scale;
};

template <int CAP>
struct AdamParams {
    AdamTensor t[CAP];
    unsigned chunk_start[CAP + 1];  // first chunk of each tensor; [count] = all chunks
    int count;
    float beta1, omb1, beta2, omb2, eps;
    AdamScalars host;
    const AdamScalars* device;  // taken instead of host when not null, with the seed behind it
    int64_t first;              // this launch's first tensor among the call's
};

__host__ __device__ __forceinline__ unsigned long long splitmix_mix(unsigned long long z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
constexpr unsigned long long kSplitmixGolden = 0x9E3779B97F4A7C15ull;

__host__ __device__ __forceinline__ unsigned long long adam_key(unsigned long long seed, unsigned long long tensor) {
    return splitmix_mix((seed << 32) + tensor);
}

// two 8-bit floats -> fp32 (exact)
template <bool E5M2>
__device__ __forceinline__ float2 fp8x2_to_f(uint32_t two) {
    uint32_t h;
    if (E5M2)
        asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e5m2x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
    else
        asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(h) : "r"(two));
    float2 f;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// The power of two a block is held with: from the largest |value|'s bits,
// 2^e <= largest < 2^(e+1), e at least -90, scale = 2^(e - LOW) and
// inv = 2^(LOW - e).  A largest value of 2^127 or more, an infinity or a NaN
// cannot be held: the scale is NaN then, so the whole block reads as NaN.
template <int LOW>
__device__ __forceinline__ bool adam_scale(uint32_t top, float& scale, float& inv) {
    const int e = max(static_cast<int>(top >> 23) - 127, -90);
    const bool held = top < 0x7F000000u;
    scale = __uint_as_float(held ? static_cast<uint32_t>(127 + e - LOW) << 23 : 0x7FC00000u);
    inv = held ? __uint_as_float(static_cast<uint32_t>(127 + LOW - e) << 23) : 0.0f;
    return held;
}

// e4m3: 3 mantissa bits, codes 8 .. 126 normal, exponent bias 7 (127 - 7 = 120, 120 << 3 = 960)
__device__ __forceinline__ uint32_t adam_code_m(float m, float inv, bool held, uint32_t rnd16) {
    const uint32_t y = __float_as_uint(__fmul_rn(m, inv));
    const int c = static_cast<int>(((y & 0x7FFFFFFFu) + (rnd16 << 4) + 8u) >> 20) - 960;
    return held ? static_cast<uint32_t>(c < 8 ? 0 : c) | ((y >> 24) & 0x80u) : 0u;
}

// e5m2: 2 mantissa bits, codes 4 .. 123 normal, exponent bias 15 (127 - 15 = 112, 112 << 2 = 448)
__device__ __forceinline__ uint32_t adam_code_v(float v, float inv, bool held, uint32_t rnd16) {
    const uint32_t y = __float_as_uint(__fmul_rn(v, inv));
    const int c = static_cast<int>((y + (rnd16 << 5) + 16u) >> 21) - 448;
    return held && v > 0.0f ? static_cast<uint32_t>(max(c, 4)) : 0u;
}

struct AdamStep {
    float beta1, omb1, beta2, omb2, eps, decay, alpha, r, grad_scale;
    __device__ __forceinline__ void operator()(float& p, float g, float& m, float& v) const {
        g = __fmul_rn(g, grad_scale);
        m = __fadd_rn(__fmul_rn(m, beta1), __fmul_rn(g, omb1));
        v = __fadd_rn(__fmul_rn(v, beta2), __fmul_rn(__fmul_rn(g, g), omb2));
        float root;
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
        p = fmaf(-alpha, __fdividef(m, fmaf(root, r, eps)), p * decay);
    }
};

// A block of 256 elements by one warp: lane l has elements 4l .. 4l + 3 of
// each half, so every access of a full block is one vector per lane over
// consecutive memory.
template <bool STATE8, bool GRAD_BF16, bool FULL>
__device__ __forceinline__ void adam_block(const AdamTensor& t, const AdamStep& step, unsigned long long key,
                                           int64_t at, int lane) {
    float p[8], g[8], m[8], v[8];
    const int left = FULL ? kAdamBlock : static_cast<int>(t.n - at);
    float ms = 0.0f, vs = 0.0f;
    if (STATE8) {
        ms = t.m_scale[at / kAdamBlock];
        vs = t.v_scale[at / kAdamBlock];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = 128 * h + 4 * lane;
        const int64_t i = at + j;
        float* P = p + 4 * h;
        float* G = g + 4 * h;
        float* Mo = m + 4 * h;
        float* V = v + 4 * h;
        if (FULL || j + 4 <= left) {
            const float4 pv = *reinterpret_cast<const float4*>(t.p + i);
            P[0] = pv.x, P[1] = pv.y, P[2] = pv.z, P[3] = pv.w;
            if (GRAD_BF16) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t.g) + i);
                G[0] = __uint_as_float(w.x << 16), G[1] = __uint_as_float(w.x & 0xFFFF0000u);
                G[2] = __uint_as_float(w.y << 16), G[3] = __uint_as_float(w.y & 0xFFFF0000u);
            } else {
                const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(t.g) + i);
                G[0] = w.x, G[1] = w.y, G[2] = w.z, G[3] = w.w;
            }
            if (STATE8) {
                const uint32_t mc = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i);
                const uint32_t vc = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i);
                const float2 a = fp8x2_to_f<false>(mc & 0xFFFFu), b = fp8x2_to_f<false>(mc >> 16);
                const float2 c = fp8x2_to_f<true>(vc & 0xFFFFu), d = fp8x2_to_f<true>(vc >> 16);
                Mo[0] = a.x * ms, Mo[1] = a.y * ms, Mo[2] = b.x * ms, Mo[3] = b.y * ms;
                V[0] = c.x * vs, V[1] = c.y * vs, V[2] = d.x * vs, V[3] = d.y * vs;
            } else {
                const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(t.m) + i);
                const float4 c = *reinterpret_cast<const float4*>(static_cast<const float*>(t.v) + i);
                Mo[0] = a.x, Mo[1] = a.y, Mo[2] = a.z, Mo[3] = a.w;
                V[0] = c.x, V[1] = c.y, V[2] = c.z, V[3] = c.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                P[e] = G[e] = Mo[e] = V[e] = 0.0f;
                if (j + e < left) {
                    P[e] = t.p[i + e];
                    G[e] = GRAD_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(t.g)[i + e])
                                     : static_cast<const float*>(t.g)[i + e];
                    if (STATE8) {
                        Mo[e] = fp8x2_to_f<false>(static_cast<const uint8_t*>(t.m)[i + e]).x * ms;
                        V[e] = fp8x2_to_f<true>(static_cast<const uint8_t*>(t.v)[i + e]).x * vs;
                    } else {
                        Mo[e] = static_cast<const float*>(t.m)[i + e];
                        V[e] = static_cast<const float*>(t.v)[i + e];
                    }
                }
            }
        }
    }
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        step(p[e], g[e], m[e], v[e]);
        if (STATE8 && (FULL || (e / 4) * 128 + 4 * lane + (e & 3) < left)) {
            mtop = max(mtop, __float_as_uint(m[e]) & 0x7FFFFFFFu);
            vtop = max(vtop, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
    }
    float minv = 0.0f, vinv = 0.0f;
    bool mheld = true, vheld = true;
    if (STATE8) {
        mtop = __reduce_max_sync(0xffffffffu, mtop);
        vtop = __reduce_max_sync(0xffffffffu, vtop);
        mheld = adam_scale<7>(mtop, ms, minv);
        vheld = adam_scale<14>(vtop, vs, vinv);
        if (lane == 0) {
            t.m_scale[at / kAdamBlock] = ms;
            t.v_scale[at / kAdamBlock] = vs;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = 128 * h + 4 * lane;
        const int64_t i = at + j;
        const float* P = p + 4 * h;
        uint32_t mc = 0, vc = 0;
        if (STATE8) {
            // draws i / 2 and i / 2 + 1 of the stream: 32 bits per element, m below v
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const unsigned long long z =
                    splitmix_mix(key + (static_cast<unsigned long long>(i / 2) + d + 1) * kSplitmixGolden);
                const uint32_t lo = static_cast<uint32_t>(z), hi = static_cast<uint32_t>(z >> 32);
                const int e = 4 * h + 2 * d;
                mc |= (adam_code_m(m[e], minv, mheld, lo & 0xFFFFu) | (adam_code_m(m[e + 1], minv, mheld, hi & 0xFFFFu) << 8))
                      << (16 * d);
                vc |= (adam_code_v(v[e], vinv, vheld, lo >> 16) | (adam_code_v(v[e + 1], vinv, vheld, hi >> 16) << 8))
                      << (16 * d);
            }
        }
        if (FULL || j + 4 <= left) {
            *reinterpret_cast<float4*>(t.p + i) = make_float4(P[0], P[1], P[2], P[3]);
            if (t.p_bf16) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(P[0], P[1]), hi = __floats2bfloat162_rn(P[2], P[3]);
                *reinterpret_cast<uint2*>(t.p_bf16 + i) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
            if (STATE8) {
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i) = mc;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i) = vc;
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(t.m) + i) =
                    make_float4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
                *reinterpret_cast<float4*>(static_cast<float*>(t.v) + i) =
                    make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (j + e >= left) continue;
                t.p[i + e] = P[e];
                if (t.p_bf16) {
                    const __nv_bfloat16 q = __float2bfloat16_rn(P[e]);
                    t.p_bf16[i + e] = *reinterpret_cast<const uint16_t*>(&q);
                }
                if (STATE8) {
                    static_cast<uint8_t*>(t.m)[i + e] = static_cast<uint8_t>(mc >> (8 * e));
                    static_cast<uint8_t*>(t.v)[i + e] = static_cast<uint8_t>(vc >> (8 * e));
                } else {
                    static_cast<float*>(t.m)[i + e] = m[4 * h + e];
                    static_cast<float*>(t.v)[i + e] = v[4 * h + e];
                }
            }
        }
    }
}

template <bool STATE8, bool GRAD_BF16>
__device__ __forceinline__ void adam_chunk(const AdamTensor& t, const AdamStep& step, unsigned long long key,
                                           int64_t chunk) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < kAdamRounds; ++r) {
        const int64_t at = chunk * kAdamChunk + (r * kAdamWarps + warp) * kAdamBlock;
        if (at + kAdamBlock <= t.n)
            adam_block<STATE8, GRAD_BF16, true>(t, step, key, at, lane);
        else if (at < t.n)
            adam_block<STATE8, GRAD_BF16, false>(t, step, key, at, lane);
    }
}

// CTA c takes chunk c of the call's tensors laid end to end, each tensor's
// chunks beginning with its first element.
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamParams<CAP> p) {
    int lo = 0, hi = p.count;  // chunk_start[lo] <= blockIdx.x < chunk_start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.chunk_start[mid] <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const AdamTensor& t = p.t[lo];
    AdamScalars s = p.host;
    unsigned long long key = t.key;
    if (p.device) {
        s = *p.device;
        key = adam_key(*reinterpret_cast<const unsigned long long*>(p.device + 1),
                       static_cast<unsigned long long>(p.first + lo));
    }
    AdamStep step;
    step.beta1 = p.beta1, step.omb1 = p.omb1, step.beta2 = p.beta2, step.omb2 = p.omb2, step.eps = p.eps;
    step.decay = __fsub_rn(1.0f, __fmul_rn(s.lr, t.weight_decay));
    step.alpha = s.alpha, step.r = s.r, step.grad_scale = s.grad_scale;
    const int64_t chunk = blockIdx.x - p.chunk_start[lo];
    switch (t.flags) {
        case 0: adam_chunk<false, false>(t, step, key, chunk); break;
        case kAdamGradBf16: adam_chunk<false, true>(t, step, key, chunk); break;
        case kAdam8: adam_chunk<true, false>(t, step, key, chunk); break;
        default: adam_chunk<true, true>(t, step, key, chunk); break;
    }
}

}  // namespace mmf
