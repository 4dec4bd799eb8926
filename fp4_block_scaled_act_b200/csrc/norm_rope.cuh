// norm_rope.cuh -- rotary tables, and the RMS norm and rotation of queries and keys in one
// pass over them, written as bf16 or as head-major FP4 operands; decoding of such operands.
//
// For a token's head x[0..D-1] (bf16), weights w (fp32), and a table row of R / 2 pairs
// (c_j, s_j) (fp32):
//   y = x w / sqrt(mean(x^2) + eps)      the mean over the head or over the token's H D values
//   (u, v) -> (u c_j - v s_j, u s_j + v c_j)     for the pairs j of the first R elements:
//       interleaved: elements 2j, 2j + 1;  half: elements j, j + R / 2.
//
// The output is the nearest bf16 of that value (low_high, rot_exact), so the FP4 form, which quantizes
// that bf16, gives the codes and scales that the head quantizer gives for the bf16 form's output,
// and neither depends on how the fp32 arithmetic in between is ordered.  The sum of squares is
// taken in fp32 for eight elements at a time (their squares are exact there) and in fp64 above
// that: four roundings of positive terms, so the root is within a relative 2^-23.  Where squares leave
// fp32's range (seen from the root) they are summed in fp64, and all pairs are rotated in fp64.
//
// What bounds it: instructions.  75600 tokens of 40 + 40 heads of 128 move 3.1 GB in the bf16 form, 477 us
// at the copy rate, and take 622 (5.0 TB/s); with NVFP4 out 2.0 GB, 302 us, and 790, at 395 warp
// instructions for 512 elements and 0.65 of the issue slots.  Of those 395 the fp64 path of the
// pairs that fp32 leaves open takes some 80 (and finding them, low_high, comes on top), quantization 90, the
// sum of squares 26, the rotation 16, the check that the root is one for fp32 some 10.
// What was taken out: the root goes into the table's entries, once a token instead of once a weight;
// pairs of pairs are rotated in packed fp32; scale bytes are stored one by one instead of gathered by
// shuffles; the interleaved layout multiplies its weights singly, since packed products would
// first need them regrouped.  Persistent blocks with the weights in shared memory were slower (975).
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
// the low 64 bits of the integer product.  turns_j comes from an fp64 quotient of the host's frequency e^-x,
// which is within (3 x + 1) 2^-53 of itself; with the quotient's own rounding and that of 2 pi it is within
// (3 x + 3) e^-x 2^-53 / (2 pi), at most 2^-54.  So the angle is within 2^-30 of a turn for |p| below 2^24 and
// within 2^-23 for all; its upper 32 bits, a signed number of half turns, are rounded to fp32 (2^-25) and go
// to sincospif.  Integer arithmetic instead of fp64 products: 75600 x 64 pairs took 74 us with those and
// take 14 (38.7 MB written, 6 us at the copy rate); what bounds the rest has not been counted.  A
// thread keeps its pair and walks over the tokens.
__global__ void __launch_bounds__(256) rope_table_kernel(const int32_t* __restrict__ pos, int64_t T, int axes,
                                                         int pairs, float amplitude,
                                                         const __grid_constant__ RopeFreqs f,
                                                         float2* __restrict__ table) {
    const int per = 256 / pairs;  // tokens a block takes at a time; threads beyond per * pairs idle
    const int j = threadIdx.x % pairs, row = threadIdx.x / pairs;
    if (row >= per) return;
    const uint64_t turns = f.turns[j];
    const int axis = f.axis[j];
    const int64_t t0 = (int64_t)blockIdx.x * per + row, step = (int64_t)gridDim.x * per;
    const int32_t* src = pos + t0 * axes + axis;
    float2* dst = table + t0 * pairs + j;
    int left = t0 < T ? (int)((T - 1 - t0) / step) + 1 : 0;  // this thread's tokens
    int32_t next = left ? *src : 0;
    for (; left > 0; --left, dst += step * pairs) {
        const uint64_t x = (uint64_t)(int64_t)next * turns;
        src += step * axes;
        if (left > 1) next = *src;  // (while this one is worked on)
        float s, c;
        sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &s, &c);
        __stcs(dst, make_float2(__fmul_rn(amplitude, c), __fmul_rn(amplitude, s)));
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
// Larger magnitudes of two pairs of bf16 (the signs become the exclusive or of both); a NaN
// beside a number drops out.
FP4_DEV uint32_t bf16_absmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two pairs (u, v) rotated in fp32, to bf16 by both ends of their errors.  In fp32
// a = x0 w0 carries one rounding (where it is no subnormal) and so does b, c r and s r carry two;
// u = a (c r) - b (s r) carries two more, so u is, with r in c and s, within
// 2^-24 (3 (|a c| + |b s|) + |b s| + |u|) of the exact value, where |a c| + |b s| <= sqrt(u^2 + v^2)
// since (c, s) is a scaled rotation: with t = max(|u|, |v|) at most 2^-24 (4 sqrt(2) t + |u|).
// m = 2^-21 t covers that and the rounding of u - m and u + m (2^-24 |u|); the same holds for v.
// Where both round to the same bf16 that is the answer; elsewhere (some 2 in 1000 pairs) the pair is
// taken again in fp64 (rot_exact).  Unrotated values have the bound of a alone.
// SIDE: the words are (u, u') and (v, v'), else (u, v) and (u', v'); bit 0 / 1 of
// the result: the first / second pair differs.
template <bool SIDE>
FP4_DEV uint32_t low_high(uint64_t u2, uint64_t v2, uint32_t& w0, uint32_t& w1) {
    float u[2], v[2], lu[2], lv[2], hu[2], hv[2];
    f2_unpack(u2, u[0], u[1]);
    f2_unpack(v2, v[0], v[1]);
    const uint64_t t = f2_pack(fmaxf(fabsf(u[0]), fabsf(v[0])), fmaxf(fabsf(u[1]), fabsf(v[1])));
    f2_unpack(f2_fma(t, f2_splat(-0x1p-21f), u2), lu[0], lu[1]);
    f2_unpack(f2_fma(t, f2_splat(-0x1p-21f), v2), lv[0], lv[1]);
    f2_unpack(f2_fma(t, f2_splat(0x1p-21f), u2), hu[0], hu[1]);
    f2_unpack(f2_fma(t, f2_splat(0x1p-21f), v2), hv[0], hv[1]);
    w0 = SIDE ? bf16_pack(lu[0], lu[1]) : bf16_pack(lu[0], lv[0]);
    w1 = SIDE ? bf16_pack(lv[0], lv[1]) : bf16_pack(lu[1], lv[1]);
    const uint32_t h0 = SIDE ? bf16_pack(hu[0], hu[1]) : bf16_pack(hu[0], hv[0]);
    const uint32_t h1 = SIDE ? bf16_pack(hv[0], hv[1]) : bf16_pack(hu[1], hv[1]);
    if (SIDE) {
        const uint32_t d = (w0 ^ h0) | (w1 ^ h1);
        return ((d & 0xFFFFu) ? 1u : 0u) | ((d >> 16) ? 2u : 0u);
    }
    return (w0 != h0 ? 1u : 0u) | (w1 != h1 ? 2u : 0u);
}
// The same pair in fp64: (u, v) as two bf16 in one word.
FP4_DEV uint32_t rot_exact(float x0, float x1, float w0, float w1, double r, bool turned, float c, float s) {
    const double a = (double)x0 * (double)w0, b = (double)x1 * (double)w1;
    double u = a, v = b;
    if (turned) u = a * (double)c - b * (double)s, v = a * (double)s + b * (double)c;
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
    float six_g = 6.0f, per_six_g = 0.0f;
    if (OUT == NR_NVFP4) {
        // 1 / (e4m3(sf) g) for every scale byte, by the activation quantizer's operations
        const float g = *q.g;
        six_g = __fmul_rn(6.0f, g);
        per_six_g = six_g >= 0x1p-100f && six_g <= 0x1p100f ? __frcp_rn(six_g) : 0.0f;
        const float d = __fmul_rn(e4m3_to_f32(threadIdx.x), g);
        nv_rcp[threadIdx.x] = d == 0.0f ? 0.0f : __frcp_rn(d);
        __syncthreads();
    }
    const float* const row = p.table + t * p.rot;
    // its eight pairs' cosines and sines, two pairs to a word pair
    uint64_t cs[4], sn[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float4 f = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        if (real && (c < 2 ? turned0 : turned1))
            f = __ldg(reinterpret_cast<const float4*>(row + (c < 2 ? c0 : c1 - 8) + 4 * c));
        cs[c] = f2_pack(f.x, f.z), sn[c] = f2_pack(f.y, f.w);
    }
    // r is plain within 2^+-40: squares were then no subnormals and did not overflow, and r in fp32 is good.
    // Elsewhere the norm is taken again in fp64, and all pairs are rotated in fp64 (low_high's bound needs
    // products that are no subnormals and do not overflow).
    constexpr uint32_t PLAIN_FROM = (127 - 40) << 23, PLAIN_SPAN = 80 << 23;
    auto plain = [](double r) { return __float_as_uint((float)r) - PLAIN_FROM < PLAIN_SPAN; };
    cp_async_wait_all();
    // a unit's sum of squares: eight squares at a time in fp32, the rest in fp64
    auto squares = [](const uint32_t (&x)[8]) {
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
            uint64_t s = f2_pack(bf16_lo(x[k]), bf16_hi(x[k]));
            s = f2_mul(s, s);
#pragma unroll
            for (int e = 1; e < 4; ++e) {
                const uint64_t a = f2_pack(bf16_lo(x[k + e]), bf16_hi(x[k + e]));
                s = f2_fma(a, a, s);
            }
            float s0, s1;
            f2_unpack(s, s0, s1);
            sum += (double)(s0 + s1);
        }
        return sum;
    };
    auto squares_fp64 = [&](int i) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(mine_at + i * 64);
        double sum = 0.0;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = x[k < 4 ? k : 32 * 4 + k - 4];
            const double a = bf16_lo(w), b = bf16_hi(w);
            sum += a * a + b * b;
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
        // a lane whose sum is not within 2^-90 .. 2^120 takes it again in fp64, before the token's lanes meet
        if (real && (uint32_t)__double2hiint(sum) - ((1023 - 90) << 20) >= (210 << 20)) {
            sum = 0.0;
            for (int i = 0; first + i * stride < units; ++i) sum += squares_fp64(i);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (wpt > 1) {  // the token's warps in order
            if (lane == 0) red[warp] = sum;
            __syncthreads();
            sum = 0.0;
            for (int k = 0; k < wpt; ++k) sum += red[warp / wpt * wpt + k];
        }
        const double m = sum / (double)(q.H * D) + (double)p.eps;
        r = rsqrt_fp64(m);
        if (!plain(r)) r = 1.0 / sqrt(m);
    }
    if (t >= rows) return;
    // r c, r s and -r s: once a token, or once a head's unit
    uint64_t cr[4], sr[4], nr[4];
    auto scale_table = [&]() {
        const uint64_t r2 = f2_splat((float)r), m2 = f2_splat(-(float)r);
#pragma unroll
        for (int k = 0; k < 4; ++k) cr[k] = f2_mul(cs[k], r2), sr[k] = f2_mul(sn[k], r2), nr[k] = f2_mul(sn[k], m2);
    };
    uint32_t all = 0u;  // the pairs to be taken in fp64 whatever their values
    if (TOKEN) scale_table(), all = plain(r) ? 0u : 0xFFu;

    constexpr int G = OUT == NR_NVFP4 ? 16 : 32;  // FP4: elements a scale
    constexpr int APR = OUT == NR_NVFP4 ? 2 : 1;  // and scale atoms per 128 tokens of a head
    const int h0 = first / LPH, dh = stride / LPH;
    const float* const weight = q.weight;
    // where a lane's results go, moved on by `dh` heads from unit to unit
    __nv_bfloat16* dst = OUT == NR_BF16 ? q.out + t * q.out_stride + h0 * D : nullptr;
    uint8_t *crow = nullptr, *srow = nullptr;
    int64_t crow_step = 0, srow_step = 0;
    if (OUT != NR_BF16) {
        crow = q.codes + (h0 * rows + t) * 64;
        crow_step = dh * rows * 64;
        // (a scale block's first two lanes write a byte each, of chunk 0 and of chunk 1)
        const int block = (part & 1 ? e1 : e0) / G;
        srow = q.sf + h0 * rows * (128 / G) + sf_word_offset(t, block / 4, APR) + block % 4;
        srow_step = dh * rows * (128 / G);
    }

#pragma unroll 1
    for (int i = 0; i < iters; ++i, dst += dh * D, crow += crow_step, srow += srow_step) {
        const int u = first + i * stride;
        // whole warps leave together (the shuffles below): the first lane's unit is the lowest
        if (u - lane >= units) break;
        const bool mine = u < units;
        const int h = h0 + i * dh;
        if (OUT != NR_BF16 && !real) {  // padding tokens hold zero codes and scales
            if (mine) {
                *reinterpret_cast<uint32_t*>(crow + e0 / 2) = 0u;
                *reinterpret_cast<uint32_t*>(crow + e1 / 2) = 0u;
                if (part % (G / 8) < 2) *srow = 0u;
            }
            continue;
        }
        uint32_t x[8];
        if (mine) {
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
        if (!TOKEN) {
            all = 0u;  // (without a norm r is 1)
            if (__any_sync(0xffffffffu, !plain(r))) {
                all = plain(r) ? 0u : 0xFFu;
                double sum = squares_fp64(i);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (all) r = 1.0 / sqrt(sum * (1.0 / D) + (double)p.eps);
            }
            scale_table();
        }
        const float* const wp = weight ? weight + (TOKEN && mine ? h * D : 0) : nullptr;
        // Rotation pairs j = 2k and 2k + 1 are (a, b), times their weights.  In memory order their four
        // values are a b a b (interleaved), or the two a's in chunk 0 and the two b's in chunk 1 (half).
        uint64_t a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (HALF) {
                a[k] = f2_pack(bf16_lo(x[k]), bf16_hi(x[k]));
                b[k] = f2_pack(bf16_lo(x[4 + k]), bf16_hi(x[4 + k]));
            } else {
                a[k] = f2_pack(bf16_lo(x[2 * k]), bf16_lo(x[2 * k + 1]));
                b[k] = f2_pack(bf16_hi(x[2 * k]), bf16_hi(x[2 * k + 1]));
            }
        }
        if (wp) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(wp + (c < 2 ? e0 : e1 - 8) + 4 * c));
                if (HALF) {
                    uint64_t* const to = c < 2 ? a + 2 * c : b + 2 * c - 4;
                    to[0] = f2_mul(to[0], f2_pack(f.x, f.y)), to[1] = f2_mul(to[1], f2_pack(f.z, f.w));
                } else {  // (in single products: pairs of weights would have to be put together first)
                    float x0, x1;
                    f2_unpack(a[c], x0, x1);
                    a[c] = f2_pack(__fmul_rn(x0, f.x), __fmul_rn(x1, f.z));
                    f2_unpack(b[c], x0, x1);
                    b[c] = f2_pack(__fmul_rn(x0, f.y), __fmul_rn(x1, f.w));
                }
            }
        }
        auto turn = [&](int k) {
            const uint64_t u = f2_fma(a[k], cr[k], f2_mul(b[k], nr[k]));
            b[k] = f2_fma(a[k], sr[k], f2_mul(b[k], cr[k]));
            a[k] = u;
        };
        auto keep = [&](int k) { a[k] = f2_mul(a[k], cr[k]), b[k] = f2_mul(b[k], cr[k]); };
        // (unrotated pairs do not take c = 1, s = 0: an infinity stays alone)
        if (p.rot == D) {
            turn(0), turn(1), turn(2), turn(3);
        } else {
            if (turned0) turn(0), turn(1);
            else keep(0), keep(1);
            if (turned1) turn(2), turn(3);
            else keep(2), keep(3);
        }

        // the unit's sixteen values as bf16, y[k] in memory order: chunk 0, then chunk 1
        uint32_t y[8], again = all;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            again |= low_high<HALF>(a[k], b[k], y[HALF ? k : 2 * k], y[HALF ? 4 + k : 2 * k + 1]) << (2 * k);
        while (again) {
            const int j = __ffs((int)again) - 1;
            again &= again - 1;
            // pair j's elements within the head, its table entry, and its values in shared memory
            const int i0 = HALF ? e0 + j : (j < 4 ? e0 : e1 - 8) + 2 * j, i1 = HALF ? e1 + j : i0 + 1;
            const uint16_t* xs = reinterpret_cast<const uint16_t*>(mine_at + i * 64 + (!HALF && j >= 4 ? 32 : 0));
            const uint32_t b0 = xs[HALF ? j : 2 * (j & 3)], b1 = HALF ? xs[32 * 8 + j] : xs[2 * (j & 3) + 1];
            const bool turned = j < 4 ? turned0 : turned1;
            float2 csj = make_float2(1.0f, 0.0f);
            if (turned) csj = __ldg(reinterpret_cast<const float2*>(row + (HALF ? c0 : j < 4 ? c0 : c1 - 8) + 2 * j));
            const float w0 = wp ? __ldg(wp + i0) : 1.0f, w1 = wp ? __ldg(wp + i1) : 1.0f;
            const uint32_t z = rot_exact(__uint_as_float(b0 << 16), __uint_as_float(b1 << 16), w0, w1, r, turned, csj.x,
                                         csj.y);
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
                *reinterpret_cast<uint4*>(dst + e0) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(dst + e1) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        } else {
            // ---- FP4: blocks of G consecutive elements, as the activation quantizer
            // A block's values lie in the same chunk of two or four neighbouring lanes: the largest of
            // chunk 0 in the low half of a word, of chunk 1 in the high half (a NaN beside others drops
            // out, as in fmaxf).
            uint32_t m0 = y[0], m1 = y[4];
#pragma unroll
            for (int k = 1; k < 4; ++k) m0 = bf16_absmax2(m0, y[k]), m1 = bf16_absmax2(m1, y[4 + k]);
            uint32_t both = bf16_absmax2(__byte_perm(m0, m1, 0x5410), __byte_perm(m0, m1, 0x7632));
#pragma unroll
            for (int o = 1; o < G / 8; o <<= 1)
                both = bf16_absmax2(both, __shfl_xor_sync(0xffffffffu, both, o));
            both &= 0x7FFF7FFFu;
            const float top[2] = {fmaxf(bf16_lo(both), 0.0f), fmaxf(bf16_hi(both), 0.0f)};
            uint32_t cw[2], sfb[2];
            if (OUT == NR_NVFP4) {
                // top / (6 g) rounded to e4m3: within 2^-23 from the reciprocal, so where both ends of a
                // wider band give one byte that is it, else (and for extreme g) the division
                const float f0 = top[0] * per_six_g, f1 = top[1] * per_six_g;
                const uint32_t low = cvt_e4m3x2(f0 * (1.0f - 0x1p-21f), f1 * (1.0f - 0x1p-21f));
                uint32_t two = cvt_e4m3x2(f0 * (1.0f + 0x1p-21f), f1 * (1.0f + 0x1p-21f));
                if (low != two || per_six_g == 0.0f)
                    two = cvt_e4m3x2(__fdiv_rn(top[0], six_g), __fdiv_rn(top[1], six_g));
                sfb[0] = two & 0xFFu, sfb[1] = two >> 8;
            } else {
                sfb[0] = mx_scale_byte<2>(top[0]), sfb[1] = mx_scale_byte<2>(top[1]);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float rr = OUT == NR_NVFP4 ? nv_rcp[sfb[c] & 0x7Fu] : mx_inv_scale(sfb[c]);
                float z[8];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    f2_unpack(f2_mul(f2_pack(bf16_lo(y[4 * c + k]), bf16_hi(y[4 * c + k])), f2_splat(rr)), z[2 * k],
                              z[2 * k + 1]);
                cw[c] = rr == 0.0f ? 0u : cvt_e2m1x8(z);  // (NVFP4: scale zero)
            }
            if (mine) {
                *reinterpret_cast<uint32_t*>(crow + e0 / 2) = cw[0];
                *reinterpret_cast<uint32_t*>(crow + e1 / 2) = cw[1];
                if (part % (G / 8) < 2) *srow = (uint8_t)(part & 1 ? sfb[1] : sfb[0]);
            }
        }
    }
}

// ------------------------------------------------------------------------------- decode
// Head-major FP4 heads (codes [H][Tpad][64], scale atoms) to bf16 [T][H][128]: the value of a code
// times its scale (NVFP4: the scale times the global, rounded to fp32), rounded once more.  A block
// takes 64 tokens of one head, a thread 8 values (4 code bytes in, 16 bytes out) of four tokens.
// The code's value in bf16 comes out of two byte tables by prmt: its high byte (sign apart) is one
// of 00 3f 3f 3f 40 40 40 40, its low byte one of 00 00 80 c0 00 40 80 c0.  Bound by the writes: 75600
// tokens x 40 heads take 199 us for 1.0 GB (5.0 TB/s, 151 us at the copy rate).
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
