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
// Work unit: 16 elements of one head, as two 16-byte chunks half a head apart (half layout: the
// two that rotate together).  D / 16 consecutive lanes hold a head, so each load and store of a
// warp covers whole 32-byte sectors; with the two chunks next to each other in memory the bf16
// form took 1.4 times as long.
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace fp4 {

// ------------------------------------------------------------------------------- rotary table
constexpr int ROPE_MAX_PAIRS = 128;
struct RopeFreqs {
    uint64_t turns[ROPE_MAX_PAIRS];  // turns per position, frequency / (2 pi), in units of 2^-64
    int8_t axis[ROPE_MAX_PAIRS];     // position axis of each pair
};

// table[t][j] = amplitude (cos, sin)(2 pi frac(p turns_j)).  The fraction of the turn count is
// the low 64 bits of the integer product, within 2^-34 of a turn for every position (turns_j is
// within 2^-65, |p| at most 2^31, and the host's frequency within a few 2^-53 of itself: 2^-24 of
// a turn at the far end for the fastest pair); its upper 32 bits, a signed number of half turns,
// are rounded to fp32 (2^-25) and go to sincospif.  Integer arithmetic instead of fp64 products:
// 75600 x 64 pairs took 74 us with those.  A thread keeps its pair and walks over the tokens.
__global__ void __launch_bounds__(256) rope_table_kernel(const int32_t* __restrict__ pos, int64_t T, int axes,
                                                         int pairs, float amplitude,
                                                         const __grid_constant__ RopeFreqs f,
                                                         float2* __restrict__ table) {
    const int per = 256 / pairs;  // tokens a block takes at a time; threads beyond per * pairs idle
    const int j = threadIdx.x % pairs, row = threadIdx.x / pairs;
    if (row >= per) return;
    const uint64_t turns = f.turns[j];
    const int axis = f.axis[j];
    for (int64_t t = (int64_t)blockIdx.x * per + row; t < T; t += (int64_t)gridDim.x * per) {
        const uint64_t x = (uint64_t)(int64_t)pos[t * axes + axis] * turns;
        float s, c;
        sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &s, &c);
        __stcs(table + t * pairs + j, make_float2(__fmul_rn(amplitude, c), __fmul_rn(amplitude, s)));
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

// A pair (u, v) rotated in fp32, to bf16 by both ends of its error.  In fp32 a = x0 (w0 r) carries
// three roundings and so does b; u = a c - b s carries two more, so u is within
// 2^-24 (3 (|a c| + |b s|) + |b s| + |u|) of the exact value, where |a c| + |b s| <= sqrt(u^2 + v^2)
// since (c, s) is a scaled rotation: with t = max(|u|, |v|) at most 2^-24 (4 sqrt(2) t + |u|).
// m = 2^-21 t covers that and the rounding of u - m and u + m (2^-24 |u|); the same holds for v.
// Where both round to the same bf16 that is the answer; elsewhere (some 3 in 10,000 values) the
// pair is taken again in fp64 (rot_exact).  Unrotated values have the bound of a alone.
FP4_DEV uint32_t low_high(float u, float v, uint32_t& high) {
    const float t = fmaxf(fabsf(u), fabsf(v));
    const uint64_t uv = f2_pack(u, v), tt = f2_pack(t, t);
    float a, b;
    f2_unpack(f2_fma(tt, f2_splat(0x1p-21f), uv), a, b);
    high = bf16_pack(a, b);
    f2_unpack(f2_fma(tt, f2_splat(-0x1p-21f), uv), a, b);
    return bf16_pack(a, b);
}
// The same pair in fp64: (u, v) as two bf16 in one word.  (c, s) = (1, 0) leaves it unrotated.
FP4_DEV uint32_t rot_exact(float x0, float x1, float w0, float w1, double r, float c, float s) {
    const double a = (double)x0 * (double)w0, b = (double)x1 * (double)w1;
    const double u = s == 0.0f ? a * (double)c : a * (double)c - b * (double)s;
    const double v = s == 0.0f ? b * (double)c : a * (double)s + b * (double)c;
    return bf16_bits_exact(u * r) | bf16_bits_exact(v * r) << 16;
}

// r = 1 / sqrt(m): the fp32 approximation and one Newton step in fp64 (relative error < 2^-40).
FP4_DEV double rsqrt_fp64(double m) {
    const double y = (double)rsqrtf((float)m);
    return y * (1.5 - 0.5 * m * y * y);
}

// `wpt` (1, 2 or 4) warps take a token together; a lane holds `iters` units of it, unit number
// warp * 32 + lane + 32 wpt i, whose place within their heads is the same for all i.  A token's
// values come to shared memory by asynchronous copies, all issued at once, each lane its own
// 32 bytes a unit (so no barrier is needed) and are read there twice, for the sum and for the
// result: held in registers (160 values a lane at 40 heads) they spilled.
// TOKEN: the norm runs over the token, else over each head or not at all (p.norm).
constexpr int NR_THREADS = 128;
FP4_DEV void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
FP4_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <bool TOKEN, int OUT, bool HALF, int D>
__global__ void __launch_bounds__(NR_THREADS, 5)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p, int wpt, int iters) {
    constexpr int LPH = D / 16;  // lanes (units) per head
    extern __shared__ __align__(16) uint4 stage[];  // [warp][iters][chunk][lane]
    __shared__ float nv_rcp[OUT == NR_NVFP4 ? 128 : 1];
    __shared__ double red[NR_THREADS / 32];
    const NormRopeTensor& q = p.t[blockIdx.y];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = q.H * LPH;
    const int64_t rows = OUT == NR_BF16 ? p.T : (p.T + 127) / 128 * 128;  // FP4: padding tokens are written too
    const int64_t t = (int64_t)blockIdx.x * (NR_THREADS / 32 / wpt) + warp / wpt;
    const bool real = t < p.T;
    const int first = (warp % wpt) * 32 + lane, stride = 32 * wpt;
    const int part = lane % LPH;
    // this lane's two chunks of each of its heads, and whether they rotate
    const bool head_turned = HALF && part * 16 < p.rot;
    const int e0 = !HALF || head_turned ? 8 * part : p.rot + 8 * (part - p.rot / 16);
    const int e1 = e0 + (!HALF ? D / 2 : head_turned ? p.rot / 2 : (D - p.rot) / 2);
    const bool turned0 = HALF ? head_turned : e0 < p.rot, turned1 = HALF ? head_turned : e1 < p.rot;
    // its pairs' places in a table row: half layout pairs 8 part .., else each chunk's own four
    const int c0 = HALF ? 16 * part : e0, c1 = HALF ? 16 * part + 8 : e1;
    uint4* const mine_at = stage + warp * iters * 64 + lane;

    if (real) {
        const __nv_bfloat16* src = q.x + t * q.stride + (first / LPH) * D;
        for (int i = 0; first + i * stride < units; ++i, src += (stride / LPH) * D) {
            cp_async_16(mine_at + i * 64, src + e0);
            cp_async_16(mine_at + i * 64 + 32, src + e1);
        }
    }
    float six_g = 6.0f;
    if (OUT == NR_NVFP4) {
        // 1 / (e4m3(sf) g) for every scale byte, by the activation quantizer's operations
        const float g = *q.g;
        six_g = __fmul_rn(6.0f, g);
        const float d = __fmul_rn(e4m3_to_f32(threadIdx.x), g);
        nv_rcp[threadIdx.x] = d == 0.0f ? 0.0f : __frcp_rn(d);
        __syncthreads();
    }
    const float* const row = p.table + t * p.rot;
    float cs[16];  // eight (cos, sin) pairs
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float4 f = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        if (real && (c < 2 ? turned0 : turned1))
            f = __ldg(reinterpret_cast<const float4*>(row + (c < 2 ? c0 : c1 - 8) + 4 * c));
        cs[4 * c] = f.x, cs[4 * c + 1] = f.y, cs[4 * c + 2] = f.z, cs[4 * c + 3] = f.w;
    }
    cp_async_wait_all();
    // a unit's sum of squares: four squares at a time in fp32, the rest in fp64
    auto squares = [](const uint32_t (&x)[8]) {
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const uint64_t a = f2_pack(bf16_lo(x[k]), bf16_hi(x[k]));
            const uint64_t b = f2_pack(bf16_lo(x[k + 1]), bf16_hi(x[k + 1]));
            float s0, s1;
            f2_unpack(f2_fma(a, a, f2_mul(b, b)), s0, s1);
            sum += (double)(s0 + s1);
        }
        return sum;
    };
    auto unit = [&](int i, uint32_t (&x)[8]) {
        const uint4 a = mine_at[i * 64], b = mine_at[i * 64 + 32];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    };
    double r = 1.0;
    if (TOKEN) {
        double sum = 0.0;
        if (real)
            for (int i = 0; first + i * stride < units; ++i) {
                uint32_t x[8];
                unit(i, x);
                sum += squares(x);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (wpt > 1) {  // the token's warps in order
            if (lane == 0) red[warp] = sum;
            __syncthreads();
            sum = 0.0;
            for (int k = 0; k < wpt; ++k) sum += red[warp / wpt * wpt + k];
        }
        r = rsqrt_fp64(sum / (double)(q.H * D) + (double)p.eps);
    }
    if (t >= rows) return;

#pragma unroll 1
    for (int i = 0; i < iters; ++i) {
        const int u = first + i * stride;
        // whole warps leave together (the shuffles below): the first lane's unit is the lowest
        if (u - lane >= units) break;
        const bool mine = u < units;
        const int h = u / LPH;
        uint32_t x[8];
        if (mine && real) {
            unit(i, x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = 0u;
        }
        if (!TOKEN && p.norm == NORM_HEAD) {
            double sum = squares(x);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrt_fp64(sum * (1.0 / D) + (double)p.eps);
        }
        const uint64_t r2 = f2_splat((float)r);
        const float* const wp = q.weight && mine ? q.weight + (TOKEN ? h * D : 0) : nullptr;
        uint64_t w[8];  // the weights of chunk 0 and chunk 1 as fp32 pairs
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = f2_splat(1.0f);
        if (wp) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(wp + (c < 2 ? e0 : e1 - 8) + 4 * c));
                w[2 * c] = f2_pack(f.x, f.y), w[2 * c + 1] = f2_pack(f.z, f.w);
            }
        }

        // the unit's sixteen values as bf16, y[k] in memory order: chunk 0, then chunk 1
        uint32_t y[8], again = 0u;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            // rotation pairs j = k and k + 1 are (a, b); in memory order these four values are
            // a b a b (interleaved), or the two a's in chunk 0 and the two b's in chunk 1
            float a[2], b[2];
            if (HALF) {
                f2_unpack(f2_mul(f2_pack(bf16_lo(x[k / 2]), bf16_hi(x[k / 2])), f2_mul(w[k / 2], r2)), a[0], a[1]);
                f2_unpack(f2_mul(f2_pack(bf16_lo(x[4 + k / 2]), bf16_hi(x[4 + k / 2])), f2_mul(w[4 + k / 2], r2)), b[0],
                          b[1]);
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    f2_unpack(f2_mul(f2_pack(bf16_lo(x[k + e]), bf16_hi(x[k + e])), f2_mul(w[k + e], r2)), a[e], b[e]);
            }
            uint32_t z[2];  // (u, v) of each pair
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float c = cs[2 * (k + e)], sn = cs[2 * (k + e) + 1];
                float uu = __fmaf_rn(a[e], c, -__fmul_rn(b[e], sn));
                float vv = __fmaf_rn(a[e], sn, __fmul_rn(b[e], c));
                if (!(k < 4 ? turned0 : turned1)) uu = a[e], vv = b[e];  // (not by c = 1, s = 0: an infinity stays alone)
                uint32_t high;
                z[e] = low_high(uu, vv, high);
                again |= z[e] != high ? 1u << (k + e) : 0u;
            }
            y[HALF ? k / 2 : k] = HALF ? __byte_perm(z[0], z[1], 0x5410) : z[0];
            y[HALF ? 4 + k / 2 : k + 1] = HALF ? __byte_perm(z[0], z[1], 0x7632) : z[1];
        }
        while (again) {
            const int j = __ffs((int)again) - 1;
            again &= again - 1;
            // pair j's elements within the head, its table entry, and its values in shared memory
            const int i0 = HALF ? e0 + j : (j < 4 ? e0 : e1 - 8) + 2 * j, i1 = HALF ? e1 + j : i0 + 1;
            const uint16_t* xs = reinterpret_cast<const uint16_t*>(mine_at + i * 64 + (!HALF && j >= 4 ? 32 : 0));
            const uint32_t b0 = xs[HALF ? j : 2 * (j & 3)], b1 = HALF ? xs[32 * 8 + j] : xs[2 * (j & 3) + 1];
            float2 csj = make_float2(1.0f, 0.0f);
            if (j < 4 ? turned0 : turned1)
                csj = __ldg(reinterpret_cast<const float2*>(row + (HALF ? c0 : j < 4 ? c0 : c1 - 8) + 2 * j));
            const uint32_t z = rot_exact(__uint_as_float(b0 << 16), __uint_as_float(b1 << 16), wp ? __ldg(wp + i0) : 1.0f,
                                         wp ? __ldg(wp + i1) : 1.0f, r, csj.x, csj.y);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!HALF && k == j) y[k] = z;
                if (HALF && k < 4 && k == j / 2) {
                    y[k] = __byte_perm(y[k], z, j & 1 ? 0x5410 : 0x3254);
                    y[4 + k] = __byte_perm(y[4 + k], z, j & 1 ? 0x7610 : 0x3276);
                }
            }
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
                v[2 * k] = real ? bf16_lo(y[k]) : 0.0f, v[2 * k + 1] = real ? bf16_hi(y[k]) : 0.0f;
                top[k / 4] = fmaxf(top[k / 4], fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
            }
            // a block's values lie in the same chunk of two or four neighbouring lanes
#pragma unroll
            for (int o = 1; o < G / 8; o <<= 1) {
                top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
                top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
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
                *reinterpret_cast<uint32_t*>(crow + e0 / 2) = cw[0];
                *reinterpret_cast<uint32_t*>(crow + e1 / 2) = cw[1];
                constexpr int APR = G == 16 ? 2 : 1;  // scale atoms per 128 tokens of a head
                uint8_t* srow = q.sf + (int64_t)h * rows * (128 / G);
                if (part < APR) *reinterpret_cast<uint32_t*>(srow + sf_word_offset(t, part, APR)) = words[part];
            }
        }
    }
}

// ------------------------------------------------------------------------------- decode
// Head-major FP4 heads (codes [H][Tpad][64], scale atoms) to bf16 [T][H][128]: the value of a code
// times its scale (NVFP4: the scale times the global, rounded to fp32), rounded once more.  A block
// takes 64 tokens of one head, a thread 8 values (4 code bytes in, 16 bytes out) of four tokens.
// The code's value in bf16 comes out of two byte tables by prmt: its high byte (sign apart) is one
// of 00 3f 3f 3f 40 40 40 40, its low byte one of 00 00 80 c0 00 40 80 c0.
template <bool NV>
__global__ void __launch_bounds__(256) dequant_heads_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ sf, int64_t T,
                                                            const float* __restrict__ g, __nv_bfloat16* __restrict__ out,
                                                            int64_t out_stride) {
    constexpr int G = NV ? 16 : 32, APR = NV ? 2 : 1, ROWS = 4;
    const int64_t tpad = (T + 127) / 128 * 128;
    const int h = blockIdx.y, part = threadIdx.x & 15, block = part * 8 / G;
    const int64_t t0 = (int64_t)blockIdx.x * (16 * ROWS) + (threadIdx.x >> 4);
    const uint8_t* crow = codes + ((int64_t)h * tpad + t0) * 64 + part * 4;
    const uint8_t* srow = sf + (int64_t)h * tpad * (128 / G) + block % 4;
    const float gs = NV ? *g : 1.0f;
    uint32_t c[ROWS], sfb[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {  // (padding tokens up to tpad are there to be read)
        c[r] = __ldcs(reinterpret_cast<const uint32_t*>(crow + r * 16 * 64));
        sfb[r] = srow[sf_word_offset(t0 + 16 * r, block / 4, APR)];
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t t = t0 + 16 * r;
        if (t >= T) break;
        // 2^(byte - 127); byte 0 marks a block of zeros or of values below 2^-125, 2^-127 as a subnormal
        const float d = NV ? __fmul_rn(e4m3_to_f32(sfb[r]), gs)
                           : (sfb[r] ? __uint_as_float(sfb[r] << 23) : __uint_as_float(0x00400000u));
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // four codes, two words
            const uint32_t four = c[r] >> (16 * k), pick = four & 0x7777u;
            const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, pick);
            const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, pick);
            w[2 * k] = __byte_perm(lo, hi, 0x5140) | (four & 8u) << 12 | (four & 0x80u) << 24;
            w[2 * k + 1] = __byte_perm(lo, hi, 0x7362) | (four & 0x800u) << 4 | (four & 0x8000u) << 16;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = bf16_pack(__fmul_rn(bf16_lo(w[k]), d), __fmul_rn(bf16_hi(w[k]), d));
        __stcs(reinterpret_cast<uint4*>(out + t * out_stride + h * 128 + part * 8), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

}  // namespace fp4
