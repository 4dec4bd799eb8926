// attn_bf16.cuh -- attention in bf16 with masks given as one range of keys per query row, capped
// scores, a distance bias and shared key heads; streaming softmax, S, P and O in TMEM.
//
//   s_ij = scale (q_i . k_j);  s_ij = cap tanh(s_ij / cap)  (cap > 0);
//   s_ij -= slope_h |pos_i - j|  (slopes given);  keys j with start_i <= j < end_i;
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(s_ij - m_i);   lse_i = log sum_j exp(s_ij).
// A row without keys gives o = 0 and lse = -inf.
//
// One CTA takes two tiles of up to 128 rows and one key head.  A row is a (token, query head) pair:
// the g = H / H_kv query heads that share the key head are rows of the same tile (g consecutive
// rows a token, floor(128 / g) tokens), so K and V are read once for all of them.  384 threads:
//   warp 0      TMA producer: Q once, then K_j, V_j tiles of 128 keys through one ring
//   warp 1      TMEM owner and MMA issuer
//   warps 2-3   V guards (below)
//   warps 4-7   softmax of tile 0, warps 8-11 of tile 1: a thread is one row
// Per key tile and row tile: S = Q K^T (kind::f16, fp32 in TMEM); a softmax thread reads its row of
// S into registers, takes the maximum, writes P = 2^(s c - m) in bf16 over S in TMEM and adds the
// fp32 weights (before rounding) to its sum; O += P V with P as the TMEM operand.  The MMA warp
// issues O += P V and the next S of one row tile while the other tile's softmax runs.  The running
// maximum that P and O refer to is replaced only when the row's maximum has grown past it by more
// than 2^8 (P then stays below 2^8, O and the sum far below overflow); only then O is rescaled in
// TMEM, by the softmax warps themselves, which know from S's arrival that the last P V is done.
// The exponent rate bounds it: a 128 x 128 tile needs 16384 exponentials, 1024 cycles of the SM's
// 16 a cycle, against 2 x 256 cycles of MMA (head_dim 128).
//
// Masks cost only where they cut: tiles outside every row's range are not visited, a warp whose
// 32 rows see a whole tile does not test keys.  Within a tile that some row does not see whole,
// a value of V that is infinite or NaN would reach rows that exclude its key (0 * inf in P V):
// the V guards look through such tiles in shared memory, put zeros in place of such values, and
// the rows that do attend them get them added at the end (rare and slow, see `repair`).
//
// With few row tiles the key tiles are split over gridDim.z; each part writes its unnormalized O,
// maximum and sum, and a second kernel joins them in a fixed order.  Every wait is bounded
// (status FP4_ERR_TIMEOUT).
#pragma once
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace fp4 {

struct AttnBfParams {
    int T_q, T_kv, H, H_kv, g;   // g = H / H_kv query heads a key head
    int tokens;                  // tokens of one row tile: 128 / g
    int q_tiles, splits;
    bool heads_first;            // block order: key heads fastest, row tiles from the last (masked calls)
    float c;                     // scale log2(e), or (capped) 2 scale log2(e) / cap
    float cap;                   // capped: cap log2(e)
    const float* slopes;         // [H] or null
    int64_t q_pos;               // position of query row 0 against key 0 (slopes)
    const int32_t* key_start;    // [T_q] or null (0)
    const int32_t* key_end;      // [T_q] or null (T_kv)
    const __nv_bfloat16* v;      // for `repair`
    int64_t v_stride;
    __nv_bfloat16* o;
    int64_t o_stride;
    float* lse;                  // [T_q][H] or null
    float* part_o;               // splits > 1: [splits][T_q H][D]
    float2* part_ml;             //   [splits][T_q H] (maximum in log2 units, sum)
    uint64_t timeout_ns;
    int* status;
};

constexpr int AB_THREADS = 384;
// registers: launched with 168 a thread; the control warpgroup gives some to the two softmax ones
constexpr uint32_t AB_REG_LAUNCH = 168, AB_REG_LO = 72, AB_REG_HI = 216;
static_assert(AB_REG_LO + 2 * AB_REG_HI == 3 * AB_REG_LAUNCH, "register split must match the launch");
constexpr float AB_LAZY = 8.0f;  // log2 of how far P may exceed 1

template <int D>
struct AttnBfCfg {
    static constexpr int TILE = 128 * D * 2;       // bytes of 128 rows: D / 64 blocks of 128 x 128 bytes
    static constexpr int BLK = 128 * 128;          // one 64-column block
    static constexpr int SLOTS = D == 128 ? 5 : 8;
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_MISC = OFF_KV + SLOTS * TILE;
    static constexpr int SMEM = OFF_MISC + 1024;
    static constexpr uint32_t T_S = 0, T_O = 256;  // TMEM columns: S (and P over it) of tile w at 128 w, O at 256 + 128 w
    // instruction descriptors: fp32 accumulator, bf16 x bf16, M = 128; V is read MN-major (bit 16)
    static constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(128 >> 4) << 24);
    static constexpr uint32_t IDESC_S = IDESC | ((uint32_t)(128 >> 3) << 17);
    static constexpr uint32_t IDESC_PV = IDESC | (1u << 16) | ((uint32_t)(D >> 3) << 17);
    static_assert(SMEM <= 232448, "shared memory");
};

FP4_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
FP4_DEV float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// D[tmem] (+)= A B^T, bf16: A from shared memory, or from TMEM (two values a column)
FP4_DEV void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
FP4_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
FP4_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
FP4_DEV void attn_bf_fail(const AttnBfParams& p, volatile int* abort) {
    *abort = 1;
    atomicCAS(p.status, 0, STATUS_TIMEOUT);
}

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(AB_THREADS, 1)
    attn_bf16_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnBfParams p) {
    using C = AttnBfCfg<D>;
    constexpr int NS = C::SLOTS;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint32_t dyn_smem;
    asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_smem));
    if ((smem_u32(sm) & 1023u) != 0 || dyn_smem < (uint32_t)C::SMEM) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, STATUS_LAYOUT);
        return;
    }
    uint8_t* sKV = sm + C::OFF_KV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);
    uint64_t* full = bars;            // [NS] ring slot loaded
    uint64_t* empty = bars + NS;      // [NS] ring slot's MMAs done
    uint64_t* q_full = bars + 2 * NS;
    uint64_t* s_full = q_full + 1;    // [2] S_j of row tile w in TMEM, and its O up to j - 1 (MMA commit)
    uint64_t* p_full = q_full + 3;    // [2] P_j of row tile w written (4 softmax warps)
    uint64_t* o_full = q_full + 5;    // [2] O of row tile w complete
    uint64_t* v_ok = q_full + 7;      // [4] V tile i has passed the guards (2 warps): barrier i % 4.  They pass
                                      // every tile in order and the MMA warp waits for each, so neither
                                      // side laps the other: the ring holds 4 V tiles at most
    uint64_t* mma_done = q_full + 11;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(q_full + 12);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* bad_v = abort + 1;  // a guarded V tile held an infinity or a NaN
    int* red = reinterpret_cast<int*>(sm + C::OFF_MISC + 512);  // [8 warps][4] row ranges

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // which rows and which key head
    int qt, hk;
    if (p.heads_first) {
        hk = blockIdx.x % p.H_kv;
        qt = p.q_tiles - 1 - blockIdx.x / p.H_kv;
    } else {
        qt = blockIdx.x % p.q_tiles;
        hk = blockIdx.x / p.q_tiles;
    }
    const int t0 = qt * 2 * p.tokens;                        // first token
    const int nsub = p.T_q - t0 > p.tokens ? 2 : 1;          // row tiles with rows

    // a softmax thread's row: w = row tile, r = row in it
    const int w = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const int tok = t0 + w * p.tokens + r / p.g, head = hk * p.g + r % p.g;
    const bool row_real = warp >= 4 && r < p.tokens * p.g && tok < p.T_q;
    int ks = 0, ke = p.T_kv;
    if (row_real) {
        if (p.key_start) ks = max(p.key_start[tok], 0);
        if (p.key_end) ke = min(p.key_end[tok], p.T_kv);
    }
    const bool row_some = row_real && ks < ke;
    if (!row_some) ks = 0, ke = p.T_kv;  // masks nothing; its output is not taken from O
    // ranges over the warp: where the first row begins and the last ends, and the keys that all see
    int lo = row_some ? ks : p.T_kv, hi = row_some ? ke : 0, all_lo = ks, all_hi = ke;
    if (warp >= 4) {
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        all_lo = __reduce_max_sync(0xffffffffu, all_lo);
        all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        if (lane == 0) {
            int* e = red + (warp - 4) * 4;
            e[0] = lo, e[1] = hi, e[2] = all_lo, e[3] = all_hi;
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&v_ok[i], 2);
        mbar_init(mma_done, 1);
        *abort = 0;
        *bad_v = 0;
        fence_mbar_init();
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // the CTA's key tiles: those that some row sees, of them this split's share
    int cta_lo = p.T_kv, cta_hi = 0, see_lo = 0, see_hi = p.T_kv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cta_lo = min(cta_lo, red[4 * i]);
        cta_hi = max(cta_hi, red[4 * i + 1]);
        see_lo = max(see_lo, red[4 * i + 2]);
        see_hi = min(see_hi, red[4 * i + 3]);
    }
    int jb = 0, je = 0;
    if (cta_lo < cta_hi) {
        const int first = cta_lo / 128, n = (cta_hi + 127) / 128 - first;
        jb = first + (int)((int64_t)n * blockIdx.z / p.splits);
        je = first + (int)((int64_t)n * (blockIdx.z + 1) / p.splits);
    }
    const int n = je - jb;
    // tiles that some row does not see whole (keys beyond T_kv are zeros already)
    auto guarded = [&](int j) { return j * 128 < see_lo || min(j * 128 + 128, p.T_kv) > see_hi; };

    const bool guarding = p.key_start || p.key_end;

    if (warp < 4) {
        setmaxnreg_dec<AB_REG_LO>();
        if (warp == 0) {
            // ======================================================== producer
            if (lane == 0 && n > 0) {
                const uint64_t pol = policy_evict_normal();
                mbar_arrive_expect_tx(q_full, (uint32_t)(nsub * p.tokens * p.g * D * 2));
                for (int s = 0; s < nsub; ++s)
                    for (int b = 0; b < D / 64; ++b)
                        tma_load_3d(sm + s * C::TILE + b * C::BLK, &tmQ, q_full, b * 64, hk * p.g, t0 + s * p.tokens, pol);
                int it = 0;
                for (; it < 2 * n; ++it) {  // K_j, V_j in turn
                    const int s = it % NS;
                    if (!mbar_wait(&empty[s], (uint32_t)((it / NS) & 1) ^ 1u, p.timeout_ns, abort)) {
                        attn_bf_fail(p, abort);
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], C::TILE);
                    const CUtensorMap* map = it & 1 ? &tmV : &tmK;
                    for (int b = 0; b < D / 64; ++b)
                        tma_load_3d(sKV + s * C::TILE + b * C::BLK, map, &full[s], b * 64, hk, (jb + (it >> 1)) * 128, pol);
                }
                // every copy issued must land before the CTA exits
                for (int i = max(0, it - NS); i < it; ++i)
                    if (!mbar_wait_drain(&full[i % NS], (uint32_t)((i / NS) & 1), p.timeout_ns)) attn_bf_fail(p, abort);
                if (!mbar_wait_drain(q_full, 0, p.timeout_ns)) attn_bf_fail(p, abort);
            }
        } else if (warp == 1) {
            // ======================================================== MMA issuer
            if (lane == 0 && n > 0) {
                bool ok = mbar_wait(q_full, 0, p.timeout_ns, abort);
                tc_fence_after();
                uint64_t qd[2];
                for (int s = 0; s < 2; ++s) qd[s] = smem_desc(smem_u32(sm + s * C::TILE), 0, 1024, 2);
                auto wait_slot = [&](int it) {
                    const bool got = mbar_wait(&full[it % NS], (uint32_t)((it / NS) & 1), p.timeout_ns, abort);
                    tc_fence_after();
                    return got;
                };
                // S of row tile s and key tile number i (ring item 2 i)
                auto issue_s = [&](int s, int i) {
                    const uint64_t kd = smem_desc(smem_u32(sKV + (2 * i % NS) * C::TILE), 0, 1024, 2);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t off = (uint64_t)((k >> 2) * (C::BLK >> 4) + (k & 3) * 2);
                        mma_f16_ss(tmem + C::T_S + 128 * s, qd[s] + off, kd + off, C::IDESC_S, k > 0 ? 1u : 0u);
                    }
                    tc_commit(&s_full[s]);
                };
                bool issued = false;
                if (ok) ok = wait_slot(0);
                if (ok) {
                    issued = true;
                    for (int s = 0; s < nsub; ++s) issue_s(s, 0);
                    tc_commit(&empty[0]);
                }
                for (int i = 0; ok && i < n; ++i) {
                    const int vi = 2 * i + 1;
                    for (int s = 0; ok && s < nsub; ++s) {
                        if (s == 0) {
                            ok = wait_slot(vi);
                            if (ok && guarding)
                                ok = mbar_wait(&v_ok[i & 3], (uint32_t)((i >> 2) & 1), p.timeout_ns, abort);
                        }
                        if (ok) ok = mbar_wait(&p_full[s], (uint32_t)(i & 1), p.timeout_ns, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd =
                            smem_desc(smem_u32(sKV + (vi % NS) * C::TILE), D == 128 ? C::BLK : 0, 1024, 2);
#pragma unroll
                        for (int k = 0; k < 8; ++k)  // 16 keys each: 8 columns of P, two groups of 8 rows of V
                            mma_f16_ts(tmem + C::T_O + 128 * s, tmem + C::T_S + 128 * s + 8 * k, vd + (uint64_t)(k * 128),
                                       C::IDESC_PV, (i > 0 || k > 0) ? 1u : 0u);
                        if (i + 1 < n) {
                            if (s == 0) ok = wait_slot(vi + 1);
                            if (ok) issue_s(s, i + 1);
                        } else {
                            tc_commit(&o_full[s]);
                        }
                    }
                    if (!ok) break;
                    tc_commit(&empty[vi % NS]);
                    if (i + 1 < n) tc_commit(&empty[(vi + 1) % NS]);
                }
                if (!ok) attn_bf_fail(p, abort);
                if (issued) {
                    tc_commit(mma_done);
                    if (!mbar_wait_drain(mma_done, 0, p.timeout_ns)) attn_bf_fail(p, abort);
                }
            }
            __syncwarp();
        } else if (guarding) {
            // ======================================================== V guards
            const int tid = threadIdx.x - 64;
            for (int i = 0; i < n; ++i) {
                const int vi = 2 * i + 1;
                bool ok = mbar_wait(&full[vi % NS], (uint32_t)((vi / NS) & 1), p.timeout_ns, abort);
                if (!__all_sync(0xffffffffu, ok)) break;  // (the MMA warp's own wait reports it)
                uint4* tile = reinterpret_cast<uint4*>(sKV + (vi % NS) * C::TILE);
                bool wrote = false;
                const int end = guarded(jb + i) ? C::TILE / 16 : 0;
#pragma unroll 4
                for (int e = tid; e < end; e += 64) {
                    uint4 x = tile[e];
                    uint32_t* word = reinterpret_cast<uint32_t*>(&x);
                    bool bad = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool b0 = (word[k] & 0x7F80u) == 0x7F80u, b1 = (word[k] & 0x7F800000u) == 0x7F800000u;
                        bad |= b0 | b1;
                        if (b0) word[k] &= 0xFFFF0000u;
                        if (b1) word[k] &= 0x0000FFFFu;
                    }
                    if (bad) {
                        tile[e] = x;
                        wrote = true;
                    }
                }
                if (wrote) *bad_v = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_ok[i & 3]);
            }
        }
    } else {
        setmaxnreg_inc<AB_REG_HI>();
        // ============================================================ softmax
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = tl + C::T_S + 128 * w, t_o = tl + C::T_O + 128 * w;
        float m = -INFINITY, l = 0.0f;  // the maximum that P and O refer to (log2 units), the sum
        const float slope = BIAS && row_real ? -1.44269504f * p.slopes[head] : 0.0f;
        const float pos = BIAS ? (float)(p.q_pos + tok - (int64_t)jb * 128) : 0.0f;
        bool ok = w < nsub;
        for (int i = 0; ok && i < n; ++i) {
            ok = __all_sync(0xffffffffu, mbar_wait(&s_full[w], (uint32_t)(i & 1), p.timeout_ns, abort));
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(t_s + 32 * q, v[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_tie(v[q]);
            const int k0 = (jb + i) * 128;
            if (CAP) {
                // cap log2(e) tanh(s / cap), tanh(x) = 1 - 2 / (1 + 2^(2 x log2 e)): within 2^-21 of cap
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float y = rcp_approx(1.0f + ex2(__uint_as_float(v[q][e]) * p.c));
                        v[q][e] = __float_as_uint(__fmaf_rn(-2.0f * p.cap, y, p.cap));
                    }
            }
            if (BIAS) {
                const float at = pos - (float)(i * 128);
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float b = fabsf(at - (float)(32 * q + e)) * slope, s = __uint_as_float(v[q][e]);
                        v[q][e] = __float_as_uint(CAP ? s + b : __fmaf_rn(s, p.c, b));
                    }
            }
            // the multiplier still to be applied
            const float c = CAP || BIAS ? 1.0f : p.c;
            if (k0 < all_lo || k0 + 128 > all_hi) {
                const int a = ks - k0, b = ke - k0;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (32 * q + e < a || 32 * q + e >= b) v[q][e] = 0xFF800000u;
            }
            float mx[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mx[q] = __uint_as_float(v[q][0]);
#pragma unroll
                for (int e = 1; e < 31; e += 2)
                    mx[q] = fmaxf(fmaxf(mx[q], __uint_as_float(v[q][e])), __uint_as_float(v[q][e + 1]));
                mx[q] = fmaxf(mx[q], __uint_as_float(v[q][31]));
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            const bool grow = top > m + AB_LAZY || (m == -INFINITY && top > m);
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2(m - top) : 1.0f;
                if (grow) m = top;
                l *= f;
                if (i > 0) {
#pragma unroll
                    for (int b = 0; b < D / 32; ++b) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(t_o + 32 * b, o);
                        tmem_wait_ld();
                        tmem_tie(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_32x32b_x16(t_o + 32 * b, *reinterpret_cast<const uint32_t(*)[16]>(o));
                        tmem_st_32x32b_x16(t_o + 32 * b + 16, *reinterpret_cast<const uint32_t(*)[16]>(o + 16));
                    }
                }
            }
            const uint64_t c2 = f2_splat(c), m2 = f2_splat(m == -INFINITY ? 0.0f : -m);
            uint64_t sum[2] = {f2_splat(0.0f), f2_splat(0.0f)};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[q][2 * e]), __uint_as_float(v[q][2 * e + 1])), c2, m2), a, b);
                    a = ex2(a), b = ex2(b);
                    sum[e & 1] = f2_add(sum[e & 1], f2_pack(a, b));
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                    pk[e] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                tmem_st_32x32b_x16(t_s + 16 * q, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[w]);
            float a, b;
            f2_unpack(f2_add(sum[0], sum[1]), a, b);
            l += a + b;
        }
        // ---------------------------------------------------------------- the rows' outputs
        if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&o_full[w], 0, p.timeout_ns, abort));
        if (w < nsub && !ok && lane == 0) attn_bf_fail(p, abort);
        if (ok) {
            tc_fence_after();
            const bool some = row_some && n > 0;
            const float inv = some && p.splits == 1 ? 1.0f / l : 1.0f;
            const size_t row = (size_t)tok * p.H + head;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(t_o + 32 * b, o);
                    tmem_wait_ld();
                    tmem_tie(o);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = some ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
                if (*bad_v && some) {
                    // repair: the values that the guards took out, for the rows that attend their keys
#pragma unroll 1
                    for (int j = jb; j < je; ++j) {
                        if (!guarded(j)) continue;
#pragma unroll 1
                        for (int key = max(ks, j * 128); key < min(ke, j * 128 + 128); ++key) {
                            const __nv_bfloat16* src = p.v + key * p.v_stride + hk * D + 32 * b;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float x = __bfloat162float(src[e]);
                                if (!(fabsf(x) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + x);
                            }
                        }
                    }
                }
                if (row_real && p.splits > 1) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + ((size_t)blockIdx.z * p.T_q * p.H + row) * D + 32 * b);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                             __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                } else if (row_real) {
                    uint4* dst = reinterpret_cast<uint4*>(p.o + (size_t)tok * p.o_stride + head * D + 32 * b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * k]),
                                                                            __uint_as_float(o[8 * e + 2 * k + 1]));
                            y[k] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        dst[e] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                __syncwarp();  // (the next TMEM load is for the whole warp)
            }
            if (row_real) {
                if (p.splits > 1)
                    p.part_ml[(size_t)blockIdx.z * p.T_q * p.H + row] =
                        some ? make_float2(m, l) : make_float2(-INFINITY, 0.0f);
                else if (p.lse)
                    p.lse[row] = some ? (m + log2f(l)) * 0.693147181f : -INFINITY;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The splits of a row joined in order: o = sum_z 2^(m_z - m) O_z / sum_z 2^(m_z - m) l_z.  A part without
// keys (l = 0) is passed over.  A warp takes a row, D / 32 values a lane.
template <int D>
__global__ void __launch_bounds__(128) attn_bf16_join_kernel(const __grid_constant__ AttnBfParams p) {
    constexpr int V = D / 32;
    const int64_t rows = (int64_t)p.T_q * p.H, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float m = -INFINITY;
    for (int z = 0; z < p.splits; ++z) m = fmaxf(m, p.part_ml[z * rows + row].x);
    float l = 0.0f, acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    bool some = false;
    for (int z = 0; z < p.splits; ++z) {
        const float2 ml = p.part_ml[z * rows + row];
        if (ml.y == 0.0f) continue;
        some = true;
        const float f = exp2f(ml.x - m);
        l += ml.y * f;
        const float* src = p.part_o + (z * rows + row) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += src[e] * f;
    }
    const int64_t tok = row / p.H;
    __nv_bfloat16* dst = p.o + tok * p.o_stride + (row - tok * p.H) * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + e) =
            some ? __floats2bfloat162_rn(acc[e] / l, acc[e + 1] / l) : __floats2bfloat162_rn(0.0f, 0.0f);
    if (p.lse && lane == 0) p.lse[row] = some ? (m + log2f(l)) * 0.693147181f : -INFINITY;
}

// Key ranges of query rows of packed documents: row i of document d (q_offsets[d] <= i <
// q_offsets[d + 1]) sees k_offsets[d] .. + n - 1, n the document's keys, or in causal order the
// larger of its own place, counted back from the document's end, and the document's prefix.
__global__ void __launch_bounds__(256) attn_ranges_kernel(const int32_t* __restrict__ q_off,
                                                          const int32_t* __restrict__ k_off, int docs, int T_q, int T_kv,
                                                          bool causal, const int32_t* __restrict__ prefix,
                                                          int32_t* __restrict__ start, int32_t* __restrict__ end) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= T_q) return;
    int lo = 0, hi = docs;  // the last document that begins at or before row i
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (q_off[mid] <= i)
            lo = mid + 1;
        else
            hi = mid;
    }
    int a = 0, b = 0;
    if (lo > 0 && i < q_off[lo]) {
        const int q0 = q_off[lo - 1], q1 = q_off[lo];
        const int k0 = min(max(k_off[lo - 1], 0), T_kv), k1 = min(max(k_off[lo], k0), T_kv);
        int n = k1 - k0;
        if (causal) n = max(0, min(n, max(i - q0 + 1 + n - (q1 - q0), prefix ? prefix[lo - 1] : 0)));
        a = k0, b = k0 + n;
    }
    start[i] = a, end[i] = b;
}

}  // namespace fp4
