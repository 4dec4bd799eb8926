// norm_rope.cuh -- rotary tables, and the RMS norm and rotation of queries and keys in one
// pass over them, written as bf16 or as head-major FP4 operands; decoding of such operands.
//
// For a token's head x[0..D-1] (bf16), weights w (fp32), and a table row of R / 2 pairs
// (c_j, s_j) (fp32):
//   y = x w / sqrt(mean(x^2) + eps)      the mean over the head or over the token's H D values
//   (u, v) -> (u c_j - v s_j, u s_j + v c_j)     for the pairs j of the first R elements:
//       interleaved: elements 2j, 2j + 1;  half: elements j, j + R / 2.
//
// The output is the nearest bf16 of that value (rot_pair), so the FP4 form, which quantizes
// that bf16, gives the codes and scales that the head quantizer gives for the bf16 form's output,
// and neither depends on how the fp32 arithmetic in between is ordered.  The sum of squares is
// taken in fp32 for two elements at a time (their squares are exact there, the sum of two is
// rounded once) and in fp64 above that, so the root is within a relative 2^-24 in every case.
//
// Work unit: 16 elements of one head, as two 16-byte chunks -- consecutive ones, or (half
// layout) the two that rotate together.  D / 16 consecutive lanes hold a head.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace fp4 {

// ------------------------------------------------------------------------------- rotary table
constexpr int ROPE_MAX_PAIRS = 128;
struct RopeFreqs {
    double turns[ROPE_MAX_PAIRS];  // frequency / (2 pi): turns per position
    int8_t axis[ROPE_MAX_PAIRS];   // position axis of each pair
};

// table[t][j] = amplitude (cos, sin)(2 pi frac(p turns_j)).  The turn count x = p turns_j is taken
// and reduced in fp64: |x| < 2^28.4, so it is within 2^-24 of the exact count (its own rounding
// and turns_j's), and twice its fraction, at most 1, within 2^-25 more in fp32.  With sincospif's
// last-place errors a value is within 2^-20 amplitude at positions near 2^31, 2^-22 below 2^24.
__global__ void __launch_bounds__(256) rope_table_kernel(const int32_t* __restrict__ pos, int64_t T, int axes,
                                                         int pairs, float amplitude,
                                                         const __grid_constant__ RopeFreqs f,
                                                         float2* __restrict__ table) {
    const int64_t n = T * pairs;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / pairs;
        const int j = (int)(i - t * pairs);
        const double x = (double)pos[t * axes + f.axis[j]] * f.turns[j];
        float s, c;
        sincospif((float)(2.0 * (x - rint(x))), &s, &c);
        table[i] = make_float2(__fmul_rn(amplitude, c), __fmul_rn(amplitude, s));
    }
}

// ------------------------------------------------------------------------------- norm + rotation
enum NormKind { NORM_NONE = 0, NORM_HEAD = 1, NORM_TOKEN = 2 };
enum NormOut { NR_BF16 = 0, NR_MXFP4 = 1, NR_NVFP4 = 2 };

struct NormRopeTensor {
    const __nv_bfloat16* x;  // [T][H][D], `stride` elements from token to token
    int64_t stride;
    int H;
    const float* weight;     // [D] (head) or [H D] (token), or null: ones
    __nv_bfloat16* out;      // bf16 form
    int64_t out_stride;
    uint8_t* codes;          // FP4 form: head-major codes and scale atoms
    uint8_t* sf;
    const float* g;          // NVFP4: the tensor's global
};
struct NormRopeParams {
    NormRopeTensor t[2];     // queries, keys (blockIdx.y)
    int64_t T;
    int norm;
    float eps;
    const float* table;      // [T][rot]
    int rot;
};

// One value rounded to bf16 exactly: fp64 -> fp32 towards zero with the discarded part kept as
// a sticky last bit, then to nearest even.
FP4_DEV uint32_t bf16_bits_exact(double v) {
    float f = __double2float_rz(v);
    if ((double)f != v) f = __uint_as_float(__float_as_uint(f) | 1u);
    return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f));
}
FP4_DEV uint32_t bf16_pack(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
FP4_DEV float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
FP4_DEV float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two rotated pairs in fp32 with a bound on their error, to bf16.  In fp32 a and b carry three
// roundings each (x w, the reciprocal root, their product) and u = a c - b s two more, so u is
// within 5 2^-24 (|a c| + |b s|) of the exact value; m = 2^-21 max(|a|, |b|) (|c| + |s|) covers
// that and the roundings of u - m and u + m.  Where both ends round to the same bf16 that is the
// answer, elsewhere (about 2 in 10,000 values) the value is taken again in fp64.
struct RotPair {
    float u, v, m;
};
FP4_DEV RotPair rot_pair(float x0, float x1, float w0, float w1, float r, float c, float s, bool turned) {
    const float a = x0 * w0 * r, b = x1 * w1 * r;
    RotPair p;
    p.m = fmaxf(fabsf(a), fabsf(b)) * ((fabsf(c) + fabsf(s)) * 0x1p-21f);
    p.u = turned ? a * c - b * s : a;
    p.v = turned ? a * s + b * c : b;
    return p;
}
FP4_DEV double rot_exact(float x0, float x1, float w0, float w1, double r, float c, float s, bool turned, bool second) {
    const double a = (double)x0 * (double)w0, b = (double)x1 * (double)w1;
    if (!turned) return (second ? b : a) * r;
    return (second ? a * (double)s + b * (double)c : a * (double)c - b * (double)s) * r;
}

// r = 1 / sqrt(m): the fp32 approximation and one Newton step in fp64 (relative error < 2^-40).
FP4_DEV double rsqrt_fp64(double m) {
    const double y = (double)rsqrtf((float)m);
    return y * (1.5 - 0.5 * m * y * y);
}

template <bool TOKEN, int OUT, bool HALF, int D>
__global__ void __launch_bounds__(TOKEN ? 1024 : 256) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LPH = D / 16;  // lanes (units) per head
    __shared__ float nv_rcp[OUT == NR_NVFP4 ? 128 : 1];
    __shared__ double red[2][32];
    const NormRopeTensor& q = p.t[blockIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float six_g = 6.0f;
    if (OUT == NR_NVFP4) {
        // 1 / (e4m3(sf) g) for every scale byte, by the activation quantizer's operations
        const float g = *q.g;
        six_g = __fmul_rn(6.0f, g);
        for (int i = threadIdx.x; i < 128; i += blockDim.x) {
            const float d = __fmul_rn(e4m3_to_f32((uint32_t)i), g);
            nv_rcp[i] = d == 0.0f ? 0.0f : __frcp_rn(d);
        }
        __syncthreads();
    }
    const int units = q.H * LPH;
    const int64_t T = p.T;
    const int64_t rows = OUT == NR_BF16 ? T : (T + 127) / 128 * 128;  // FP4: padding tokens are written too
    const int part = threadIdx.x % LPH;  // this thread's unit of its head: the same for all its units
    // its two chunks of eight elements, and whether they rotate
    const bool turned = part * 16 < p.rot;
    const int e0 = HALF ? (turned ? 8 * part : p.rot + 8 * (part - p.rot / 16)) : 16 * part;
    const int e1 = HALF ? e0 + (turned ? p.rot / 2 : (D - p.rot) / 2) : e0 + 8;
    // TOKEN: a block per token, unit threadIdx.x; otherwise units are numbered over all tokens
    const int64_t step = TOKEN ? gridDim.x : (int64_t)gridDim.x * blockDim.x;
    const int64_t limit = TOKEN ? rows : rows * units;
    const bool active = !TOKEN || threadIdx.x < units;

    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.0f;
    if (q.weight && active) {
        const float* wp = q.weight + (TOKEN ? (threadIdx.x / LPH) * D : 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 f = *reinterpret_cast<const float4*>(wp + (c < 2 ? e0 : e1 - 8) + 4 * c);
            w[4 * c] = f.x, w[4 * c + 1] = f.y, w[4 * c + 2] = f.z, w[4 * c + 3] = f.w;
        }
    }
    // where unit index i lies, and its two chunks
    auto place = [&](int64_t i, int64_t& t, int& h) {
        if (TOKEN) {
            t = i;
            h = threadIdx.x / LPH;
        } else {
            const uint32_t tt = (uint32_t)i / (uint32_t)units;
            t = tt;
            h = (int)(((uint32_t)i - tt * (uint32_t)units) / LPH);
        }
    };
    auto fetch = [&](int64_t i, uint4& c0, uint4& c1) {
        c0 = c1 = make_uint4(0, 0, 0, 0);
        if (i >= limit || !active) return;
        int64_t t;
        int h;
        place(i, t, h);
        if (t >= T) return;
        const __nv_bfloat16* src = q.x + t * q.stride + h * D;
        c0 = __ldcs(reinterpret_cast<const uint4*>(src + e0));
        c1 = __ldcs(reinterpret_cast<const uint4*>(src + e1));
    };

    int64_t i = TOKEN ? blockIdx.x : (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    uint4 n0, n1;
    fetch(i, n0, n1);
    for (int phase = 0; TOKEN ? i < limit : __any_sync(0xffffffffu, i < limit); i += step, phase ^= 1) {
        const uint32_t x[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
        int64_t t = 0;
        int h = 0;
        const bool mine = i < limit && active;
        if (mine) place(i, t, h);
        float cs[16];  // eight (cos, sin) pairs
        if (mine && turned && t < T) {
            const float4* row = reinterpret_cast<const float4*>(p.table + t * p.rot + 16 * part);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 f = row[c];
                cs[4 * c] = f.x, cs[4 * c + 1] = f.y, cs[4 * c + 2] = f.z, cs[4 * c + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) cs[2 * c] = 1.0f, cs[2 * c + 1] = 0.0f;
        }
        fetch(i + step, n0, n1);  // the next unit is on its way while this one is worked on

        double r = 1.0;
        if (p.norm != NORM_NONE) {
            double sum = 0.0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float a = bf16_lo(x[k]), b = bf16_hi(x[k]);
                sum += (double)fmaf(a, a, b * b);
            }
            // (TOKEN: over the warp, then over the block's warps in order; else over the head's lanes)
#pragma unroll
            for (int o = TOKEN ? 16 : LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (TOKEN) {
                if (lane == 0) red[phase][warp] = sum;
                __syncthreads();
                sum = 0.0;
                for (int k = 0; k < (int)blockDim.x / 32; ++k) sum += red[phase][k];
                r = rsqrt_fp64(sum / (double)(q.H * D) + (double)p.eps);
            } else {
                r = rsqrt_fp64(sum * (1.0 / D) + (double)p.eps);
            }
        }
        const float rf = (float)r;

        // the unit's sixteen values as bf16: y[k] = pairs of neighbours of chunk 0, then of chunk 1
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            // two rotation pairs, j = k and k + 1, each (x0, x1)
            float x0[2], x1[2], w0[2], w1[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (HALF) {
                    x0[e] = e ? bf16_hi(x[k / 2]) : bf16_lo(x[k / 2]);
                    x1[e] = e ? bf16_hi(x[4 + k / 2]) : bf16_lo(x[4 + k / 2]);
                    w0[e] = w[k + e], w1[e] = w[8 + k + e];
                } else {
                    x0[e] = bf16_lo(x[k + e]), x1[e] = bf16_hi(x[k + e]);
                    w0[e] = w[2 * (k + e)], w1[e] = w[2 * (k + e) + 1];
                }
            }
            RotPair z[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                z[e] = rot_pair(x0[e], x1[e], w0[e], w1[e], rf, cs[2 * (k + e)], cs[2 * (k + e) + 1], turned);
            // word 0 and 1 of the result: HALF neighbours are the two pairs' u (and v), else a pair's u, v
            uint32_t lo[2], hi[2];
            if (HALF) {
                lo[0] = bf16_pack(z[0].u - z[0].m, z[1].u - z[1].m), hi[0] = bf16_pack(z[0].u + z[0].m, z[1].u + z[1].m);
                lo[1] = bf16_pack(z[0].v - z[0].m, z[1].v - z[1].m), hi[1] = bf16_pack(z[0].v + z[0].m, z[1].v + z[1].m);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    lo[e] = bf16_pack(z[e].u - z[e].m, z[e].v - z[e].m);
                    hi[e] = bf16_pack(z[e].u + z[e].m, z[e].v + z[e].m);
                }
            }
            if ((lo[0] != hi[0]) | (lo[1] != hi[1])) {
                uint32_t b[2][2];  // [pair][u, v]
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int o = 0; o < 2; ++o)
                        b[e][o] = bf16_bits_exact(rot_exact(x0[e], x1[e], w0[e], w1[e], r, cs[2 * (k + e)],
                                                            cs[2 * (k + e) + 1], turned, o == 1));
                lo[0] = b[0][0] | (HALF ? b[1][0] : b[0][1]) << 16;
                lo[1] = (HALF ? b[0][1] : b[1][0]) | b[1][1] << 16;
            }
            if (HALF)
                y[k / 2] = lo[0], y[4 + k / 2] = lo[1];
            else
                y[k] = lo[0], y[k + 1] = lo[1];
        }

        if constexpr (OUT == NR_BF16) {
            if (mine) {
                __nv_bfloat16* dst = q.out + t * q.out_stride + h * D;
                *reinterpret_cast<uint4*>(dst + e0) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(dst + e1) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        } else {
            // ---- FP4: blocks of G consecutive elements, as the activation quantizer
            constexpr int G = OUT == NR_NVFP4 ? 16 : 32;
            float v[16], top[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                // padding tokens hold zero codes and scales
                v[2 * k] = t < T ? bf16_lo(y[k]) : 0.0f, v[2 * k + 1] = t < T ? bf16_hi(y[k]) : 0.0f;
                top[k / 4] = fmaxf(top[k / 4], fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
            }
            // a block's lanes: interleaved units are consecutive (one lane or two); in the half
            // layout a chunk's neighbours lie in the next lanes (two or four)
            if (HALF) {
#pragma unroll
                for (int o = 1; o < G / 8; o <<= 1) {
                    top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
                    top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
                }
            } else {
                top[0] = fmaxf(top[0], top[1]);
                if (G == 32) top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], 1));
                top[1] = top[0];
            }
            uint32_t cw[2], words[2] = {0u, 0u};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float z[8];
                uint32_t sfb;
                if (OUT == NR_NVFP4) {
                    sfb = cvt_e4m3x2(__fdiv_rn(top[c], six_g), 0.0f) & 0xFFu;
                    const float rr = nv_rcp[sfb & 0x7Fu];
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[k] = rr == 0.0f ? 0.0f : __fmul_rn(v[8 * c + k], rr);
                } else {
                    sfb = mx_scale_byte<2>(top[c]);
                    const float inv = mx_inv_scale(sfb);
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[k] = __fmul_rn(v[8 * c + k], inv);
                }
                cw[c] = cvt_e2m1x8(z);
                const int block = (c ? e1 : e0) / G;
                if (G == 16) {
                    words[0] |= block < 4 ? sfb << (8 * block) : 0u;
                    words[1] |= block >= 4 ? sfb << (8 * (block - 4)) : 0u;
                } else {
                    words[0] |= sfb << (8 * block);
                }
            }
#pragma unroll
            for (int o = 1; o < LPH; o <<= 1) {
                words[0] |= __shfl_xor_sync(0xffffffffu, words[0], o);
                if (G == 16) words[1] |= __shfl_xor_sync(0xffffffffu, words[1], o);
            }
            if (mine) {
                uint8_t* crow = q.codes + ((int64_t)h * rows + t) * 64;
                if (HALF) {
                    *reinterpret_cast<uint32_t*>(crow + e0 / 2) = cw[0];
                    *reinterpret_cast<uint32_t*>(crow + e1 / 2) = cw[1];
                } else {
                    *reinterpret_cast<uint2*>(crow + e0 / 2) = make_uint2(cw[0], cw[1]);
                }
                constexpr int APR = G == 16 ? 2 : 1;  // scale atoms per 128 tokens of a head
                uint8_t* srow = q.sf + (int64_t)h * rows * (128 / G);
                if (part < APR) *reinterpret_cast<uint32_t*>(srow + sf_word_offset(t, part, APR)) = words[part];
            }
        }
    }
}

// ------------------------------------------------------------------------------- decode
// Head-major FP4 heads (codes [H][Tpad][64], scale atoms) to bf16 [T][H][128]: the value of a code
// times its scale (NVFP4: the scale times the global, rounded to fp32), rounded once more.  A thread
// takes 16 elements: 8 code bytes in, 32 bytes out.
template <bool NV>
__global__ void __launch_bounds__(256) dequant_heads_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ sf, int64_t T, int H,
                                                            const float* __restrict__ g, __nv_bfloat16* __restrict__ out,
                                                            int64_t out_stride) {
    const int64_t tpad = (T + 127) / 128 * 128;
    const uint32_t units = (uint32_t)H * 8u, n = (uint32_t)T * units;
    const float gs = NV ? *g : 1.0f;
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < n; i += gridDim.x * 256u) {
        const uint32_t t = i / units, u = i - t * units;
        const int h = (int)(u >> 3), part = (int)(u & 7);
        const uint2 c = *reinterpret_cast<const uint2*>(codes + ((int64_t)h * tpad + t) * 64 + part * 8);
        constexpr int G = NV ? 16 : 32, APR = NV ? 2 : 1;
        const int block = part * 16 / G;
        const uint32_t sfb = sf[(int64_t)h * tpad * (128 / G) + sf_word_offset(t, block / 4, APR) + block % 4];
        // 2^(byte - 127); byte 0 marks a block of zeros or of values below 2^-125, 2^-127 as a subnormal
        const float d = NV ? __fmul_rn(e4m3_to_f32(sfb), gs)
                           : (sfb ? __uint_as_float(sfb << 23) : __uint_as_float(0x00400000u));
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t b = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t m = (b >> (4 * e)) & 7u, sign = (b >> (4 * e) & 8u) << 28;
                // 0, .5, 1, 1.5, 2, 3, 4, 6: exponent m / 2, one bit of mantissa, .5 the subnormal
                const uint32_t bits = m < 2 ? (m ? 0x3F000000u : 0u) : ((126u + (m >> 1)) << 23) | ((m & 1u) << 22);
                v[e] = __fmul_rn(__uint_as_float(bits | sign), d);
            }
            w[k] = bf16_pack(v[0], v[1]);
        }
        uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)t * out_stride + h * 128 + part * 16);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

}  // namespace fp4
