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
// SplitMix64 stream (seed, tensor); the caller's seed is another at every step,
// or the bits would be fixed thresholds.  The update takes the moments before they
// are rounded.  |m| below the smallest normal code becomes 0; a positive v is
// kept at least at the smallest normal code, so it never reads as 0.
//
// Bound and measured: 28 bytes an element with fp32 moments and gradients, 14
// with 8-bit moments and bf16 gradients.  One 1.3B layer set (51.4 M elements,
// fp32): 213 us, 6.7 TB/s, the copy rate.  Two 2.7B layer sets (158.6 M, 8
// bits, bf16 gradients and copy, 16 bytes): 430 us in a short run, 5.9 TB/s,
// 487 us where calls follow one another for long; there the noise and the
// packing of the codes bind, 71 instructions an element, the ALU pipe 71% busy.
#pragma once
#include "common.cuh"

namespace mmf {

constexpr int kAdamThreads = 256;
constexpr int kAdamWarps = kAdamThreads / 32;
constexpr int kAdamBlock = 256;                              // elements that share the scales
constexpr int kAdamRow = kAdamWarps * kAdamBlock;            // elements a CTA takes at once
// and how often, where there is work for all SMs: 8-bit moments ask for their
// later rows ahead, 32-bit ones gain nothing from it or from longer chunks
// (51.4 M elements: 214 us at 2 rounds, 221 at 8, 269 with rows asked for ahead)
constexpr int kAdamRounds8 = 8, kAdamRounds32 = 2;

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
    int rounds;              // a CTA's chunk of it: rounds * kAdamRow elements
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

// z >> S (S above 16): the upper word's two parts by one multiplication, since
// the shifts' pipe is the busy one here
template <int S>
__host__ __device__ __forceinline__ unsigned long long shift_right(unsigned long long z) {
#ifdef __CUDA_ARCH__
    const uint32_t lo = static_cast<uint32_t>(z), hi = static_cast<uint32_t>(z >> 32);
    return static_cast<unsigned long long>(hi) * (1u << (32 - S)) + (lo >> S);
#else
    return z >> S;
#endif
}

__host__ __device__ __forceinline__ unsigned long long splitmix_mix(unsigned long long z) {
    z = (z ^ shift_right<30>(z)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ shift_right<27>(z)) * 0x94D049BB133111EBull;
    return z ^ shift_right<31>(z);
}
constexpr unsigned long long kSplitmixGolden = 0x9E3779B97F4A7C15ull;

// The key of a tensor's stream, from all 64 bits of the seed: of a seed below
// 2^32 it is mix(seed 2^32 + tensor), as of the input streams, since mix(0) = 0.
__host__ __device__ __forceinline__ unsigned long long adam_key(unsigned long long seed, unsigned long long tensor) {
    return splitmix_mix((seed << 32) + tensor + splitmix_mix(seed >> 32));
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

// |a|, |b| and c's largest; NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Bits SHIFT .. SHIFT + 7 (SHIFT 20 or 21) of four words as four bytes.
template <int SHIFT>
__device__ __forceinline__ uint32_t pack_bytes(const uint32_t (&t)[4]) {
    const uint32_t even = __byte_perm(t[0], t[2], 0x7632), odd = __byte_perm(t[1], t[3], 0x7632);  // the upper halves
    return ((even >> (SHIFT - 16)) & 0x00FF00FFu) | ((odd << (24 - SHIFT)) & 0xFF00FF00u);
}

// Four e4m3 codes, each the bits of |m| / scale cut to 3 mantissa bits after a
// random number below a step was added (16 of its 20 bits random, the rest a
// half).  Bits 20 and up are then the code plus 960 (120, the bias' difference,
// times 8): its low 7 bits are the code's with bit 6 flipped.  Codes 8 .. 126
// are normal; below them the code is 0, which few elements are, so a warp looks
// for them once and not each.
__device__ __forceinline__ uint32_t adam_codes_m(const float (&m)[4], float inv, const uint32_t (&rnd)[4]) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        t[e] = __float_as_uint(__fmul_rn(fabsf(m[e]), inv)) + (((rnd[e] << 4) & 0xFFFF0u) | 8u);
    if (__any_sync(0xffffffffu, min(min(t[0], t[1]), min(t[2], t[3])) < (968u << 20))) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t[e] < (968u << 20)) t[e] = 0x40u << 20;
    }
    const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(m[0]), __float_as_uint(m[1]), 0x0073),
                                       __byte_perm(__float_as_uint(m[2]), __float_as_uint(m[3]), 0x0073), 0x5410);
    return ((pack_bytes<20>(t) & 0x7F7F7F7Fu) | (signs & 0x80808080u)) ^ 0x40404040u;
}

// Four e5m2 codes, the same with 2 mantissa bits: bits 21 and up are the code
// plus 448 (112 times 4).  Codes 4 .. 123 are normal; a positive v has at least
// 4, and 0 is looked for once a warp.
__device__ __forceinline__ uint32_t adam_codes_v(const float (&v)[4], float inv, const uint32_t (&rnd)[4]) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        t[e] = max(__float_as_uint(__fmul_rn(v[e], inv)) + (((rnd[e] >> 11) & 0x1FFFE0u) | 16u), 452u << 21);
    if (__any_sync(0xffffffffu, v[0] == 0.0f || v[1] == 0.0f || v[2] == 0.0f || v[3] == 0.0f)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (v[e] == 0.0f) t[e] = 448u << 21;
    }
    return (pack_bytes<21>(t) & 0x7F7F7F7Fu) ^ 0x40404040u;
}

// a + b of both halves by scalar additions: a packed product and a packed sum
// behind it come out as one fused operation, which rounds once, not twice
__device__ __forceinline__ f2 f2_add_unfused(f2 a, f2 b) {
    const float2 x = f2_get(a), y = f2_get(b);
    return f2_make(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
}

// One step of two elements.
struct AdamStep {
    f2 beta1, omb1, beta2, omb2, eps, decay, alpha, r, grad_scale;  // alpha negated
    __device__ __forceinline__ void operator()(f2& p, f2 g, f2& m, f2& v) const {
        g = f2_mul(g, grad_scale);
        m = f2_add_unfused(f2_mul(m, beta1), f2_mul(g, omb1));
        v = f2_add_unfused(f2_mul(v, beta2), f2_mul(f2_mul(g, g), omb2));
        float2 root = f2_get(v);
        asm("sqrt.approx.f32 %0, %0;" : "+f"(root.x));
        asm("sqrt.approx.f32 %0, %0;" : "+f"(root.y));
        const float2 d = f2_get(f2_fma(f2_make(root.x, root.y), r, eps));  // at least eps, a normal number
        float ix, iy;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ix) : "f"(d.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(iy) : "f"(d.y));
        p = f2_fma(f2_mul(m, f2_make(ix, iy)), alpha, f2_mul(p, decay));
    }
};

// A block of 256 elements by one warp: lane l has elements 4l .. 4l + 3 of
// each half, so every access of a full block is one vector per lane over
// consecutive memory.  AdamRaw is such a block as it lies in memory.
template <bool STATE8, bool GRAD_BF16>
struct AdamRaw {
    float4 p[2];
    uint4 g[2];  // fp32, or bf16 in x and y
    uint4 m[2];  // fp32, or 8-bit codes in x
    uint4 v[2];
    float ms, vs;

    __device__ __forceinline__ void load(const AdamTensor& t, int64_t at, int lane) {
        if (STATE8) {
            ms = t.m_scale[at / kAdamBlock];
            vs = t.v_scale[at / kAdamBlock];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t i = at + 128 * h + 4 * lane;
            p[h] = *reinterpret_cast<const float4*>(t.p + i);
            if (GRAD_BF16) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(t.g) + i);
                g[h].x = w.x, g[h].y = w.y;
            } else {
                g[h] = *reinterpret_cast<const uint4*>(static_cast<const float*>(t.g) + i);
            }
            if (STATE8) {
                m[h].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + i);
                v[h].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i);
            } else {
                m[h] = *reinterpret_cast<const uint4*>(static_cast<const float*>(t.m) + i);
                v[h] = *reinterpret_cast<const uint4*>(static_cast<const float*>(t.v) + i);
            }
        }
    }
};

// Its elements as fp32 pairs, two of each half.
struct AdamValues {
    f2 p[4], g[4], m[4], v[4];

    template <bool STATE8, bool GRAD_BF16>
    __device__ __forceinline__ void unpack(const AdamRaw<STATE8, GRAD_BF16>& r) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            p[2 * h] = f2_make(r.p[h].x, r.p[h].y), p[2 * h + 1] = f2_make(r.p[h].z, r.p[h].w);
            if (GRAD_BF16) {
                g[2 * h] = f2_make(__uint_as_float(r.g[h].x << 16), __uint_as_float(r.g[h].x & 0xFFFF0000u));
                g[2 * h + 1] = f2_make(__uint_as_float(r.g[h].y << 16), __uint_as_float(r.g[h].y & 0xFFFF0000u));
            } else {
                words(g + 2 * h, r.g[h]);
            }
            if (STATE8) {
                const float2 a = fp8x2_to_f<false>(r.m[h].x & 0xFFFFu), b = fp8x2_to_f<false>(r.m[h].x >> 16);
                const float2 c = fp8x2_to_f<true>(r.v[h].x & 0xFFFFu), d = fp8x2_to_f<true>(r.v[h].x >> 16);
                const f2 ms = f2_set(r.ms), vs = f2_set(r.vs);
                m[2 * h] = f2_mul(f2_make(a.x, a.y), ms), m[2 * h + 1] = f2_mul(f2_make(b.x, b.y), ms);
                v[2 * h] = f2_mul(f2_make(c.x, c.y), vs), v[2 * h + 1] = f2_mul(f2_make(d.x, d.y), vs);
            } else {
                words(m + 2 * h, r.m[h]);
                words(v + 2 * h, r.v[h]);
            }
        }
    }
    static __device__ __forceinline__ void words(f2* to, const uint4& w) {
        to[0] = f2_make(__uint_as_float(w.x), __uint_as_float(w.y));
        to[1] = f2_make(__uint_as_float(w.z), __uint_as_float(w.w));
    }

    // a tensor's last, short block: `left` elements, the others zeros
    template <bool STATE8, bool GRAD_BF16>
    __device__ __forceinline__ void load_short(const AdamTensor& t, int64_t at, int left, int lane) {
        const float ms = STATE8 ? t.m_scale[at / kAdamBlock] : 0.0f, vs = STATE8 ? t.v_scale[at / kAdamBlock] : 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e[4][2] = {};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int j = 128 * (q / 2) + 4 * lane + 2 * (q & 1) + s;
                if (j >= left) continue;
                e[0][s] = t.p[at + j];
                e[1][s] = GRAD_BF16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(t.g)[at + j])
                                    : static_cast<const float*>(t.g)[at + j];
                e[2][s] = STATE8 ? fp8x2_to_f<false>(static_cast<const uint8_t*>(t.m)[at + j]).x * ms
                                 : static_cast<const float*>(t.m)[at + j];
                e[3][s] = STATE8 ? fp8x2_to_f<true>(static_cast<const uint8_t*>(t.v)[at + j]).x * vs
                                 : static_cast<const float*>(t.v)[at + j];
            }
            p[q] = f2_make(e[0][0], e[0][1]);
            g[q] = f2_make(e[1][0], e[1][1]);
            m[q] = f2_make(e[2][0], e[2][1]);
            v[q] = f2_make(e[3][0], e[3][1]);
        }
    }
};

// The step of a block's elements, and their way back to memory.
template <bool STATE8, bool FULL>
__device__ __forceinline__ void adam_block(const AdamTensor& t, const AdamStep& step, unsigned long long key,
                                           AdamValues& x, int64_t at, int left, int lane) {
    float me[8], ve[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        step(x.p[q], x.g[q], x.m[q], x.v[q]);
        const float2 a = f2_get(x.m[q]), b = f2_get(x.v[q]);
        me[2 * q] = a.x, me[2 * q + 1] = a.y;
        ve[2 * q] = b.x, ve[2 * q + 1] = b.y;
    }
    float minv = 0.0f, vinv = 0.0f;
    bool mheld = true, vheld = true;
    unsigned long long draw = 0;
    if (STATE8) {
        if (!FULL) {  // the places behind the end count for nothing, whatever 0 * grad_scale is
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((e / 4) * 128 + 4 * lane + (e & 3) >= left) me[e] = ve[e] = 0.0f;
        }
        float ml = 0.0f, vl = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            ml = max3_abs(me[e], me[e + 1], ml);
            vl = max3_abs(ve[e], ve[e + 1], vl);
        }
        const uint32_t mtop = __reduce_max_sync(0xffffffffu, __float_as_uint(ml));
        const uint32_t vtop = __reduce_max_sync(0xffffffffu, __float_as_uint(vl));
        float ms, vs;
        mheld = adam_scale<7>(mtop, ms, minv);
        vheld = adam_scale<14>(vtop, vs, vinv);
        if (lane == 0) {
            t.m_scale[at / kAdamBlock] = ms;
            t.v_scale[at / kAdamBlock] = vs;
        }
        // element i takes half of draw i / 2 of the stream, m the low 16 bits of it
        draw = key + (static_cast<unsigned long long>(at / 2) + 2 * lane + 1) * kSplitmixGolden;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = 128 * h + 4 * lane;
        const int64_t i = at + j;
        const float2 p0 = f2_get(x.p[2 * h]), p1 = f2_get(x.p[2 * h + 1]);
        const float M4[4] = {me[4 * h], me[4 * h + 1], me[4 * h + 2], me[4 * h + 3]};
        const float V4[4] = {ve[4 * h], ve[4 * h + 1], ve[4 * h + 2], ve[4 * h + 3]};
        uint32_t mc = 0, vc = 0;
        if (STATE8) {
            const unsigned long long z0 = splitmix_mix(draw + (64 * h) * kSplitmixGolden);
            const unsigned long long z1 = splitmix_mix(draw + (64 * h + 1) * kSplitmixGolden);
            const uint32_t rnd[4] = {static_cast<uint32_t>(z0), static_cast<uint32_t>(z0 >> 32), static_cast<uint32_t>(z1),
                                     static_cast<uint32_t>(z1 >> 32)};
            mc = mheld ? adam_codes_m(M4, minv, rnd) : 0u;
            vc = vheld ? adam_codes_v(V4, vinv, rnd) : 0u;
        }
        if (FULL || j + 4 <= left) {
            *reinterpret_cast<float4*>(t.p + i) = make_float4(p0.x, p0.y, p1.x, p1.y);
            if (t.p_bf16) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(p0.x, p0.y), hi = __floats2bfloat162_rn(p1.x, p1.y);
                *reinterpret_cast<uint2*>(t.p_bf16 + i) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
            if (STATE8) {
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + i) = mc;
                *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i) = vc;
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(t.m) + i) = make_float4(M4[0], M4[1], M4[2], M4[3]);
                *reinterpret_cast<float4*>(static_cast<float*>(t.v) + i) = make_float4(V4[0], V4[1], V4[2], V4[3]);
            }
        } else {
            const float P4[4] = {p0.x, p0.y, p1.x, p1.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (j + e >= left) continue;
                t.p[i + e] = P4[e];
                if (t.p_bf16) {
                    const __nv_bfloat16 q = __float2bfloat16_rn(P4[e]);
                    t.p_bf16[i + e] = *reinterpret_cast<const uint16_t*>(&q);
                }
                if (STATE8) {
                    static_cast<uint8_t*>(t.m)[i + e] = static_cast<uint8_t>(mc >> (8 * e));
                    static_cast<uint8_t*>(t.v)[i + e] = static_cast<uint8_t>(vc >> (8 * e));
                } else {
                    static_cast<float*>(t.m)[i + e] = M4[e];
                    static_cast<float*>(t.v)[i + e] = V4[e];
                }
            }
        }
    }
}

// Brings a row of kAdamRow elements into L2, by one thread.  A CTA's later rows
// are asked for kAdamAhead rows before they are worked on: the loads then wait
// for L2 only, and HBM is kept busy whatever the warps do.
constexpr int kAdamAhead = 1;

template <bool STATE8, bool GRAD_BF16>
__device__ __forceinline__ void adam_prefetch(const AdamTensor& t, int64_t at) {
    if (at + kAdamRow > t.n) return;
    bulk_prefetch_l2(t.p + at, 4 * kAdamRow);
    bulk_prefetch_l2(static_cast<const uint8_t*>(t.g) + (GRAD_BF16 ? 2 : 4) * at, (GRAD_BF16 ? 2 : 4) * kAdamRow);
    bulk_prefetch_l2(static_cast<const uint8_t*>(t.m) + (STATE8 ? 1 : 4) * at, (STATE8 ? 1 : 4) * kAdamRow);
    bulk_prefetch_l2(static_cast<const uint8_t*>(t.v) + (STATE8 ? 1 : 4) * at, (STATE8 ? 1 : 4) * kAdamRow);
}

// A CTA's chunk: `rounds` blocks per warp, kAdamRow apart.
template <bool STATE8, bool GRAD_BF16>
__device__ __forceinline__ void adam_chunk(const AdamTensor& t, const AdamStep& step, unsigned long long key,
                                           int64_t chunk, int rounds) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = chunk * rounds * kAdamRow;
    if (STATE8 && threadIdx.x == 0)
        for (int r = 1; r <= kAdamAhead && r < rounds; ++r) adam_prefetch<STATE8, GRAD_BF16>(t, row + r * kAdamRow);
    for (int r = 0; r < rounds; ++r) {
        if (STATE8 && threadIdx.x == 0 && r + 1 + kAdamAhead < rounds)
            adam_prefetch<STATE8, GRAD_BF16>(t, row + (r + 1 + kAdamAhead) * kAdamRow);
        const int64_t at = row + r * kAdamRow + warp * kAdamBlock;
        AdamValues x;
        if (at + kAdamBlock <= t.n) {
            AdamRaw<STATE8, GRAD_BF16> raw;
            raw.load(t, at, lane);
            x.unpack(raw);
            adam_block<STATE8, true>(t, step, key, x, at, kAdamBlock, lane);
        } else if (at < t.n) {
            const int left = static_cast<int>(t.n - at);
            x.load_short<STATE8, GRAD_BF16>(t, at, left, lane);
            adam_block<STATE8, false>(t, step, key, x, at, left, lane);
        }
    }
}

// CTA c takes chunk c of the call's tensors laid end to end, each tensor's
// chunks beginning with its first element.
template <int CAP>
__global__ void __launch_bounds__(kAdamThreads, 4) adamw_kernel(const __grid_constant__ AdamParams<CAP> p) {
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
    step.beta1 = f2_set(p.beta1), step.omb1 = f2_set(p.omb1);
    step.beta2 = f2_set(p.beta2), step.omb2 = f2_set(p.omb2), step.eps = f2_set(p.eps);
    step.decay = f2_set(__fsub_rn(1.0f, __fmul_rn(s.lr, t.weight_decay)));
    step.alpha = f2_set(-s.alpha), step.r = f2_set(s.r), step.grad_scale = f2_set(s.grad_scale);
    const int64_t chunk = blockIdx.x - p.chunk_start[lo];
    switch (t.flags) {
        case 0: adam_chunk<false, false>(t, step, key, chunk, t.rounds); break;
        case kAdamGradBf16: adam_chunk<false, true>(t, step, key, chunk, t.rounds); break;
        case kAdam8: adam_chunk<true, false>(t, step, key, chunk, t.rounds); break;
        default: adam_chunk<true, true>(t, step, key, chunk, t.rounds); break;
    }
}

}  // namespace mmf
