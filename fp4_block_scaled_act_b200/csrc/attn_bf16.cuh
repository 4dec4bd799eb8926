// attn_bf16.cuh -- attention in bf16 with masks given as one range of keys per query row, capped
// scores, a distance bias and shared key heads; streaming softmax, S, P and O in TMEM.
//
//   s_ij = scale (q_i . k_j);  s_ij = cap tanh(s_ij / cap)  (cap > 0);
//   s_ij -= slope_h |pos_i - j|  (slopes given);  keys j with start_i <= j < end_i;
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(s_ij - m_i);   lse_i = log sum_j exp(s_ij).
// A row without keys gives o = 0 and lse = -inf.
//
// Work items: two tiles of up to 128 rows and one key head; a persistent CTA per SM takes them
// in turn.  A row is a (token, query head) pair: the g = H / H_kv query heads that share the key
// head are rows of the same tile (g consecutive rows a token, floor(128 / g) tokens), so K and V
// are read once for all of them.  384 threads:
//   warp 0      planner and TMA producer: an item's key range, Q, then K_j, V_j tiles of 128 keys
//               through one ring, running ahead into the next item
//   warp 1      TMEM owner and MMA issuer
//   warps 2-3   V guards (below)
//   warps 4-7   softmax of tile 0, warps 8-11 of tile 1: a thread is one row
// Per key tile and row tile: S = Q K^T (kind::f16, fp32 in TMEM); a softmax thread reads its row of
// S into registers and writes P = 2^(s c - m) in bf16 over S in TMEM, in two halves of 64 keys, each
// handed to the MMA warp as it is done; the fp32 weights (before rounding) are added to its sum.
// O += P V with P as the TMEM operand, the first half while the second is being made, then the
// next S.  m is a running reference, not the row's maximum (lazy rescaling, a published method of
// streaming attention): it is replaced only when the maximum has grown past it by more than 2^8 (P then
// stays below 2^8, the sum below 2^38, O within it for values below 2^88); only then O is rescaled in TMEM,
// by the softmax warps, which know from S's arrival that the last P V is done.
// What bounds it: per 128 x 128 scores 512 cycles of MMA for S and for P V each (head_dim 128), and
// 16384 exponentials at 16 a cycle, 1024 cycles, in turn for a row tile, in parallel for the two.
// Measured, head_dim 128: 8192 rows x 8192 keys x 16 heads 553 us (994 TFLOP/s, 0.60 of the library
// GEMM's rate), causal 277 (993), capped 841 (1400 where tiles hold scores beyond the cap), with a bias
// 729, both 1098; head_dim 64 494.  An SM that works has its tensor pipe busy 0.53 of the cycles, the
// exponentials' pipe as much.  Part of the rest is the schedule: items go to the CTAs in a fixed order,
// and 512 equal ones on 148 CTAs make a last round that is half empty (256 key tiles on the longest CTA,
// 221 in the mean).  The rest is each row tile's chain from S over its maximum and exponentials to P V,
// which the other tile covers only in part.  Tried and no
// faster: 64-key tiles, a reference maximum guessed ahead, exponentials by polynomial for a share of
// the keys, P handed over whole, a second MMA warp, O staged through shared memory.
// The kernels spill 100 to 300 bytes a thread (136 bytes of loads in the plain one, 356 MB a call above,
// out of L1); a split of 56 / 224 registers would spill less and has not been timed.
// Documents: an item has one key range for both its row tiles, and its length does not decide where it
// runs.  Three clips of 4290 tokens x 24 heads, 179 us: 54 key tiles on the longest CTA, 37 in the mean, 34
// if each row tile took its own range.
// Few keys: 32760 rows x 40 heads over 512 keys 420 us, over 256 281 (104 us of bytes): an item of
// one key tile takes a softmax warp some 7000 cycles in turn, most of it the wait for S, its
// exponentials, the wait for P V, and reading and storing O.  One token x 40 heads (8 key heads) over 100001
// keys: 107 us (62 of bytes).
//
// Masks cost only where they cut: tiles outside every row's range are not visited, a warp whose
// 32 rows see a whole tile does not test keys.  Within a tile that some row does not see whole,
// a value of V that is infinite or NaN would reach rows that exclude its key (0 * inf in P V):
// the V guard looks through such tiles in shared memory, puts zeros in place of such values, and
// the rows that do attend them get them added at the end (`repair`).  That is slow, also where no row
// attends them: one token over 100001 keys 112 us with zeros behind the last key and 167 with NaN there, over
// 1000 keys 30 and 185; 8192 rows x 8100 keys 569 and 918.
//
// With few row tiles the key tiles are split into parts, each an item of its own; each part
// writes its unnormalized O, maximum and sum, and a second kernel joins them in a fixed order.
// Where a key head has one row tile only (`alt`, calls of one or a few tokens) the item's two tiles
// are the same rows, over the even and the odd key tiles, as two parts: one's softmax still runs
// beside the other's MMAs.  Every wait is bounded (status FP4_ERR_TIMEOUT).
#pragma once
#include <cuda_bf16.h>

#include <climits>

#include "ptx.cuh"

namespace fp4 {

struct AttnBfParams {
    int T_q, T_kv, H, H_kv, g;   // g = H / H_kv query heads a key head
    int tokens;                  // tokens of one row tile: 128 / g
    int q_tiles, splits;         // row tile pairs; parts of the keys that are items
    int items;                   // q_tiles H_kv splits
    bool alt;                    // one row tile, even and odd key tiles (two parts an item)
    bool heads_first;            // item order: key heads fastest, row tiles from the last (masked calls)
    float c;                     // scale log2(e), or (capped) scale / cap
    float cap;                   // capped: cap log2(e)
    float tanh[6];               //   and the coefficients of tanh_near
    const float* slopes;         // [H] or null
    int64_t q_pos;               // position of query row 0 against key 0 (slopes)
    const int32_t* key_start;    // [T_q] or null (0)
    const int32_t* key_end;      // [T_q] or null (T_kv)
    const __nv_bfloat16* v;      // for `repair`
    int64_t v_stride;
    __nv_bfloat16* o;
    int64_t o_stride;
    bool o_32;                   // o's rows are 32-byte aligned: stored by whole sectors
    float* lse;                  // [T_q][H] or null
    int parts;                   // splits, or twice that (alt); > 1: partial results
    float* part_o;               //   [parts][T_q H][D]
    float2* part_ml;             //   [parts][T_q H] (maximum in log2 units, sum; -1: no keys)
    uint64_t timeout_ns;
    int* status;
};

constexpr int AB_THREADS = 384;
// registers: launched with 168 a thread; the control warpgroup gives some to the two softmax ones
constexpr uint32_t AB_REG_LAUNCH = 168, AB_REG_LO = 72, AB_REG_HI = 216;
static_assert(AB_REG_LO + 2 * AB_REG_HI == 3 * AB_REG_LAUNCH, "register split must match the launch");
constexpr int AB_KEYS = 128;  // keys of a tile
constexpr int AB_ITEMS = 4;   // items in flight between the planner and the slowest warp
constexpr float AB_LAZY = 8.0f;  // log2 of how far P may exceed 1

template <int D>
struct AttnBfCfg {
    static constexpr int TILE = 128 * D * 2;       // bytes of 128 rows: D / 64 blocks of 128 x 128 bytes
    static constexpr int BLK = 128 * 128;          // one 64-column block
    static constexpr int PAIR = 2 * TILE;          // a ring slot: K_u, then V_{u - lag}
    static constexpr int SLOTS = D == 128 ? 2 : 4;
    static constexpr int OFF_KV = 2 * TILE;
    static constexpr int OFF_MISC = OFF_KV + SLOTS * PAIR;
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
// Groups of four MMAs, D[tmem] (+)= A B^T in bf16, issued by one elected lane of a converged warp: K
// steps of 16 over 64 columns of K-major operands in shared memory (32 bytes a step), and over 64
// keys with A in TMEM (two values a column, 8 columns a step) and B MN-major (2048 bytes a step).
// Called by the whole warp with warp-uniform operands, so that descriptors stay in uniform
// registers: from a single lane's branch an MMA took 139 cycles to issue beside eight busy warps,
// so takes 49, below the 64 that the tensor core needs for it.
FP4_DEV void mma4_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b64 x, y;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.s64 x, %1, 2;\n\tadd.s64 y, %2, 2;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
        "add.s64 x, %1, 4;\n\tadd.s64 y, %2, 4;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t"
        "add.s64 x, %1, 6;\n\tadd.s64 y, %2, 6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
FP4_DEV void mma4_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
        "add.s32 x, %1, 8;\n\tadd.s64 y, %2, 128;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t"
        "add.s32 x, %1, 16;\n\tadd.s64 y, %2, 256;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t"
        "add.s32 x, %1, 24;\n\tadd.s64 y, %2, 384;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// tc_commit by the lane that issues the groups
FP4_DEV void tc_commit_elect(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}
FP4_DEV void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
// mbar_wait by a whole warp: one lane polls
FP4_DEV bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort) {
    bool got = true;
    if ((threadIdx.x & 31) == 0) got = mbar_wait(bar, parity, limit_ns, abort);
    return __shfl_sync(0xffffffffu, (int)got, 0) != 0;
}
FP4_DEV void attn_bf_fail(const AttnBfParams& p, volatile int* abort) {
    *abort = 1;
    atomicCAS(p.status, 0, STATUS_TIMEOUT);
}

// The capped score of |s / cap| <= 1: cap log2(e) tanh(x), x = s / cap, as an odd polynomial x P(x^2), without
// a transcendental: tanh(x) = x sum_i t_i x^2i fitted here on [0, 1] (minimax by reweighted least squares,
// degree 11, within 2^-20.6 of its value: relative, so that small scores keep their accuracy under a large
// cap), cap log2(e) folded into its coefficients on the host.  Folding the scale in too would save the product
// s / cap, 4 % of the time, but its powers overflow fp32 for small caps and underflow for large ones (2 %
// of the score at a cap of 1e6 times the scale).
constexpr double AB_TANH[6] = {0x1.ffffecp-1, -0x1.554a16p-2, 0x1.1000f6p-3, -0x1.a6c0f0p-5, 0x1.1251b4p-6, -0x1.92016cp-9};
FP4_DEV uint64_t tanh_near(uint64_t x, const float (&t)[6]) {
    const uint64_t y = f2_mul(x, x);
    uint64_t e = f2_splat(t[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) e = f2_fma(e, y, f2_splat(t[i]));
    return f2_mul(x, e);
}

// Distance bias.  A query may stand far from the keys of its range ks .. ke - 1, where fp32 holds neither its
// distances (beyond 2^24) nor their differences in a large bias.  Keys are therefore counted from `pos`, the
// query's own place if that is within the range, else the range's nearest key: |q_pos + i - j| is |pos - j| and a
// part that all keys share.  The latter cancels in o and is added to lse.  A slope below 0 makes far keys the
// heavy ones; for those distances are taken less the largest (`far`), so that biases are 0 at the heaviest key.
struct AttnBfBias {
    int pos;
    float slope, far;  // bias in log2 units: (|pos - j| - far) slope
    FP4_DEV AttnBfBias(const AttnBfParams& p, int tok, int head, int ks, int ke) {
        const int64_t at = p.q_pos + tok;
        pos = (int)(at < ks ? ks : at >= ke ? ke - 1 : at);
        slope = -1.44269504f * p.slopes[head];
        far = slope > 0.0f ? (float)max(pos - ks, ke - 1 - pos) : 0.0f;
    }
    // lse of biases as above, to that of the whole distances
    FP4_DEV float lse(const AttnBfParams& p, int tok, int head, float log2_sum) const {
        const int64_t apart = p.q_pos + tok - pos;
        return (log2_sum + far * slope) * 0.693147181f - p.slopes[head] * fabsf((float)apart);
    }
};

// An item as the planner gives it to the other warps
struct AttnBfItem {
    int t0, hk, z, subs; // first token, key head, part; row tiles
    int t0_next;         // first token of the CTA's next item (T_q: none)
    int jb, n;           // its key tiles
    int see_lo, see_hi;  // the keys that all its rows see
    int bad;             // set by the guard: a guarded V tile held an infinity or a NaN
    // tiles that some row does not see whole (keys beyond T_kv are zeros already)
    FP4_DEV bool guarded(int j, int T_kv) const { return j * 128 < see_lo || min(j * 128 + 128, T_kv) > see_hi; }
};

template <int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(AB_THREADS, 1)
    attn_bf16_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnBfParams p) {
    using C = AttnBfCfg<D>;
    constexpr uint32_t NS = C::SLOTS;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint32_t dyn_smem;
    asm volatile("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_smem));
    if ((smem_u32(sm) & 1023u) != 0 || dyn_smem < (uint32_t)C::SMEM) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0, STATUS_LAYOUT);
        return;
    }
    uint8_t* sKV = sm + C::OFF_KV;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_MISC);
    uint64_t* full = bars;             // [NS] ring slot loaded
    uint64_t* empty = bars + NS;       // [NS] ring slot's MMAs done
    uint64_t* q_full = bars + 2 * NS;  // an item's Q loaded
    uint64_t* q_empty = q_full + 1;    // its last S done
    uint64_t* s_full = q_full + 2;     // [2] S of row tile w in TMEM, and its O up to the tile before (MMA commit)
    uint64_t* p_full = q_full + 4;     // [row tile][half] P written (4 softmax warps)
    uint64_t* o_full = q_full + 10;    // [2] an item's O of row tile w complete
    uint64_t* o_free = q_full + 12;    // [2] and read (4 softmax warps)
    uint64_t* v_ok = q_full + 14;      // [4] ring slot number i has passed the guards (2 warps): barrier i % 4.  They
                                       // pass every slot in order and the MMA warp waits for each, so neither
                                       // side laps the other: the ring holds 4 at most
    uint64_t* item_full = q_full + 18;             // [AB_ITEMS] item planned
    uint64_t* item_empty = item_full + AB_ITEMS;   // [AB_ITEMS] all warps are done with it
    uint64_t* mma_done = item_empty + AB_ITEMS;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile AttnBfItem* info = reinterpret_cast<volatile AttnBfItem*>(sm + C::OFF_MISC + 512);  // [AB_ITEMS]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool guarding = p.key_start || p.key_end;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 4);
            mbar_init(&p_full[2 * i + 1], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_free[i], 4);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&v_ok[i], 2);
        for (int i = 0; i < AB_ITEMS; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], guarding ? 11 : 9);  // MMA, 8 softmax warps, 2 guards
        }
        mbar_init(mma_done, 1);
        *abort = 0;
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

    // the CTA's k-th item: rounds over the CTAs in turn, every second one backwards (the items of a
    // masked call come longest first)
    const int G = gridDim.x;
    auto item_of = [&](int k) { return k * G + (k & 1 ? G - 1 - (int)blockIdx.x : (int)blockIdx.x); };
    struct Place {
        int t0, hk, z;  // first token, key head, part
    };
    auto place = [&](int item) {
        const int per = p.q_tiles * p.H_kv, z = item / per, at = item - z * per;
        int qt, hk;
        if (p.heads_first) {
            qt = p.q_tiles - 1 - at / p.H_kv;
            hk = at % p.H_kv;
        } else {
            hk = at / p.q_tiles;
            qt = at - hk * p.q_tiles;
        }
        return Place{qt * 2 * p.tokens, hk, z};
    };
    auto subs_of = [&](const Place& at) { return p.alt || p.T_q - at.t0 > p.tokens ? 2 : 1; };
    // key tiles of an item that row tile s takes: all n, or every second
    auto tiles_of = [&](int n, int s) { return p.alt ? (n + 1 - s) >> 1 : n; };
    // ring slot u of an item holds K_u and V_{u - lag}, what the MMA warp needs at a time: a row tile's
    // P V and its next S (alt: the row tile's next tile but one)
    const int lag = p.alt ? 2 : 1;

    if (warp < 4) {
        setmaxnreg_dec<AB_REG_LO>();
        if (warp == 0) {
            // ======================================================== planner and producer
            const uint64_t pol = policy_evict_normal();
            uint32_t it = 0, nq = 0;  // ring items and Q loads so far
            bool ok = true;
            // the ranges of an item's rows: lane l takes tokens l, l + 32, ...
            constexpr int PER = 8;
            int ks[PER], ke[PER];
            auto fetch = [&](int item) {
                const int t0 = item < p.items ? place(item).t0 : p.T_q;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int off = lane + 32 * i, t = t0 + off;
                    const bool in = off < (p.alt ? p.tokens : 2 * p.tokens) && t < p.T_q;
                    ks[i] = in ? (p.key_start ? p.key_start[t] : 0) : INT_MAX;
                    ke[i] = in ? (p.key_end ? p.key_end[t] : p.T_kv) : INT_MIN;
                }
                return t0;
            };
            fetch(item_of(0));
            for (int k = 0; ok; ++k) {
                const int item = item_of(k);
                if (item >= p.items) break;
                const Place at = place(item);
                int lo = p.T_kv, hi = 0, all_lo = 0, all_hi = p.T_kv;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int a = max(ks[i], 0), b = min(ke[i], p.T_kv);
                    if (a < b) {  // rows without keys take no part
                        lo = min(lo, a), hi = max(hi, b);
                        all_lo = max(all_lo, a), all_hi = min(all_hi, b);
                    }
                }
                lo = __reduce_min_sync(0xffffffffu, lo);
                hi = __reduce_max_sync(0xffffffffu, hi);
                all_lo = __reduce_max_sync(0xffffffffu, all_lo);
                all_hi = __reduce_min_sync(0xffffffffu, all_hi);
                int jb = 0, n = 0;
                if (lo < hi) {
                    const int first = lo / 128, all = (hi + 127) / 128 - first;
                    jb = first + (int)((int64_t)all * at.z / p.splits);
                    n = first + (int)((int64_t)all * (at.z + 1) / p.splits) - jb;
                }
                const int e = k % AB_ITEMS;
                ok = mbar_wait_warp(&item_empty[e], (uint32_t)((k / AB_ITEMS) & 1) ^ 1u, p.timeout_ns, abort);
                const int t0_next = fetch(item_of(k + 1));
                if (lane == 0) {
                    if (ok) {
                        info[e].t0 = at.t0, info[e].hk = at.hk, info[e].z = at.z, info[e].subs = subs_of(at);
                        info[e].t0_next = t0_next;
                        info[e].jb = jb, info[e].n = n, info[e].see_lo = all_lo, info[e].see_hi = all_hi, info[e].bad = 0;
                        mbar_arrive(&item_full[e]);
                    }
                    if (ok && n > 0) {
                        ok = mbar_wait(q_empty, (nq & 1u) ^ 1u, p.timeout_ns, abort);
                        if (ok) {
                            const int loads = p.alt ? 1 : subs_of(at);
                            mbar_arrive_expect_tx(q_full, (uint32_t)(loads * p.tokens * p.g * D * 2));
                            for (int s = 0; s < loads; ++s)
                                for (int b = 0; b < D / 64; ++b)
                                    tma_load_3d(sm + s * C::TILE + b * C::BLK, &tmQ, q_full, b * 64, at.hk * p.g,
                                                at.t0 + s * p.tokens, pol);
                            ++nq;
                        }
                        for (int u = 0; ok && u < n + lag; ++u, ++it) {
                            const uint32_t at_s = it % NS;
                            ok = mbar_wait(&empty[at_s], ((it / NS) & 1u) ^ 1u, p.timeout_ns, abort);
                            if (!ok) break;
                            const bool has_k = u < n, has_v = u >= lag;  // (alt with one key tile: slot 1 is empty)
                            mbar_arrive_expect_tx(&full[at_s], (uint32_t)(((int)has_k + (int)has_v) * C::TILE));
                            for (int b = 0; b < D / 64; ++b) {
                                uint8_t* dst = sKV + at_s * C::PAIR + b * C::BLK;
                                if (has_k) tma_load_3d(dst, &tmK, &full[at_s], b * 64, at.hk, (jb + u) * 128, pol);
                                if (has_v)
                                    tma_load_3d(dst + C::TILE, &tmV, &full[at_s], b * 64, at.hk, (jb + u - lag) * 128, pol);
                            }
                        }
                    }
                    if (!ok) attn_bf_fail(p, abort);
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            // every copy issued must land before the CTA exits
            if (lane == 0) {
                for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i)
                    if (!mbar_wait_drain(&full[i % NS], (i / NS) & 1u, p.timeout_ns)) attn_bf_fail(p, abort);
                if (nq && !mbar_wait_drain(q_full, (nq - 1) & 1u, p.timeout_ns)) attn_bf_fail(p, abort);
            }
        } else if (warp == 1) {
            // ======================================================== MMA issuer
            // The whole warp runs this, converged (mma4_f16_ss).  It serves the row tiles in turn, each to
            // the end of its step, which keeps them half a step apart: one's exponentials then run beside
            // the other's MMAs.  (With a warp for each they fell into step, and both waited.)
            const uint64_t qd0 = smem_desc(smem_u32(sm), 0, 1024, 2);
            const uint64_t kd0 = smem_desc(smem_u32(sKV), 0, 1024, 2);
            const uint64_t vd0 = smem_desc(smem_u32(sKV + C::TILE), D == 128 ? C::BLK : 0, 1024, 2);
            uint32_t slot = 0, phase = 0;             // the ring item next in turn
            uint32_t nq = 0, nv = 0;                  // Q loads and ring slots so far
            uint32_t np[2] = {0, 0}, no[2] = {0, 0};  // P tiles and O results of each row tile so far
            bool ok = true, issued = false;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.timeout_ns, abort)) != 0;
            };
            auto issue_s = [&](int s, uint32_t at) {
                const uint64_t qd = qd0 + (p.alt ? 0 : (uint64_t)(s * (C::TILE >> 4)));
                const uint64_t kd = kd0 + (uint64_t)(at * (C::PAIR >> 4));
#pragma unroll
                for (int b = 0; b < D / 64; ++b)
                    mma4_f16_ss(tmem + C::T_S + 128 * s, qd + (uint64_t)(b * (C::BLK >> 4)),
                                kd + (uint64_t)(b * (C::BLK >> 4)), C::IDESC_S, b > 0 ? 1u : 0u);
                tc_commit_elect(&s_full[s]);
            };
            // O += P V of row tile s with the V in ring slot `at`, as P's halves come
            auto issue_pv = [&](int s, uint32_t at, bool first) {
                const uint64_t vd = vd0 + (uint64_t)(at * (C::PAIR >> 4));
                if (first && !wait(&o_free[s], (no[s]++ & 1u) ^ 1u)) return false;
                if (!wait(&p_full[2 * s], np[s] & 1u)) return false;
                tc_fence_after();
                mma4_f16_ts(tmem + C::T_O + 128 * s, tmem + C::T_S + 128 * s, vd, C::IDESC_PV, first ? 0u : 1u);
                if (!wait(&p_full[2 * s + 1], np[s]++ & 1u)) return false;
                tc_fence_after();
                mma4_f16_ts(tmem + C::T_O + 128 * s, tmem + C::T_S + 128 * s + 32, vd + 512u, C::IDESC_PV, 1u);
                return true;
            };
            for (int k = 0; ok; ++k) {
                const int e = k % AB_ITEMS;
                if (item_of(k) >= p.items) break;
                ok = wait(&item_full[e], (uint32_t)((k / AB_ITEMS) & 1));
                if (!ok) break;
                const int n = __reduce_max_sync(0xffffffffu, info[e].n), nsub = __reduce_max_sync(0xffffffffu, info[e].subs);
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[e]);
                __syncwarp();
                if (n == 0) continue;
                ok = wait(q_full, nq++ & 1u);
                for (int u = 0; ok && u < n + lag; ++u) {
                    const uint32_t at_s = slot;
                    ok = wait(&full[slot], phase);
                    if (++slot == NS) slot = 0, phase ^= 1u;
                    if (ok && guarding) {
                        ok = wait(&v_ok[nv & 3], (nv >> 2) & 1u);
                        ++nv;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const int s1 = p.alt ? (u & 1) + 1 : nsub;
                    for (int s = p.alt ? u & 1 : 0; ok && s < s1; ++s) {
                        if (u >= lag) ok = issue_pv(s, at_s, u < 2 * lag);
                        if (!ok) break;
                        if (u < n)
                            issue_s(s, at_s);
                        else if (u >= lag)
                            tc_commit_elect(&o_full[s]);
                    }
                    if (!ok) break;
                    issued = true;
                    tc_commit_elect(&empty[at_s]);
                    if (u == n - 1) tc_commit_elect(q_empty);
                }
            }
            if (!ok && lane == 0) attn_bf_fail(p, abort);
            __syncwarp();
            if (issued) {
                tc_commit_elect(mma_done);
                const bool done = mbar_wait_drain(mma_done, 0, p.timeout_ns);
                if (!__all_sync(0xffffffffu, done) && lane == 0) attn_bf_fail(p, abort);
            }
            __syncwarp();
        } else if (guarding) {
            // ======================================================== V guard
            const int tid = threadIdx.x - 64;
            uint32_t it = 0, nv = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const int e = k % AB_ITEMS;
                if (item_of(k) >= p.items) break;
                ok = mbar_wait_warp(&item_full[e], (uint32_t)((k / AB_ITEMS) & 1), p.timeout_ns, abort);
                if (!ok) break;
                AttnBfItem w;
                w.jb = info[e].jb, w.n = info[e].n, w.see_lo = info[e].see_lo, w.see_hi = info[e].see_hi;
                for (int u = 0; u < (w.n ? w.n + lag : 0); ++u, ++it) {
                    ok = mbar_wait_warp(&full[it % NS], (it / NS) & 1u, p.timeout_ns, abort);
                    if (!ok) break;  // (the MMA warp's own wait reports it)
                    const int j = u - lag;
                    if (j >= 0 && w.guarded(w.jb + j, p.T_kv)) {
                        // 0 * x + sum stays 0 unless some x is infinite or NaN
                        uint4* tile = reinterpret_cast<uint4*>(sKV + (it % NS) * C::PAIR + C::TILE);
                        __nv_bfloat162 sum[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) sum[c] = __floats2bfloat162_rn(0.0f, 0.0f);
                        const __nv_bfloat162 zero = sum[0];
#pragma unroll 8
                        for (int i = tid; i < C::TILE / 16; i += 64) {
                            uint4 v = tile[i];
                            const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
                            for (int c = 0; c < 4; ++c) sum[c] = __hfma2(b[c], zero, sum[c]);
                        }
                        const float2 f = __bfloat1622float2(__hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3])));
                        if (f.x != 0.0f || f.y != 0.0f) {  // (also where it is NaN)
                            info[e].bad = 1;
#pragma unroll 1
                            for (int i = tid; i < C::TILE / 16; i += 64) {
                                uint4 v = tile[i];
                                uint32_t* word = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    if ((word[c] & 0x7F80u) == 0x7F80u) word[c] &= 0xFFFF0000u;
                                    if ((word[c] & 0x7F800000u) == 0x7F800000u) word[c] &= 0x0000FFFFu;
                                }
                                tile[i] = v;
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_ok[nv & 3]);
                    ++nv;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&item_empty[e]);
            }
        }
    } else {
        setmaxnreg_inc<AB_REG_HI>();
        // ============================================================ softmax
        const int w = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;  // row tile, row in it
        const int row_tok = r / p.g, row_head = r - row_tok * p.g;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = tl + C::T_S + 128 * w, t_o = tl + C::T_O + 128 * w;
        uint32_t ns = 0, no = 0;  // S tiles and O results so far
        bool ok = true;
        // a row's token in an item, or -1, and its range
        auto token_of = [&](int t0) {
            const int t = t0 + (p.alt ? 0 : w * p.tokens) + row_tok;
            return row_tok < p.tokens && t < p.T_q ? t : -1;
        };
        int ks_next = 0, ke_next = p.T_kv;
        auto fetch = [&](int t0) {
            if (!guarding) return;
            const int t = token_of(t0);
            ks_next = t >= 0 && p.key_start ? p.key_start[t] : 0;
            ke_next = t >= 0 && p.key_end ? p.key_end[t] : p.T_kv;
        };
        if (item_of(0) < p.items) fetch(place(item_of(0)).t0);
        for (int k = 0; ok; ++k) {
            const int e = k % AB_ITEMS;
            if (item_of(k) >= p.items) break;
            ok = mbar_wait_warp(&item_full[e], (uint32_t)((k / AB_ITEMS) & 1), p.timeout_ns, abort);
            if (!ok) break;
            const int tok = token_of(info[e].t0), head = info[e].hk * p.g + row_head;
            int ks = max(ks_next, 0), ke = min(ke_next, p.T_kv);
            const bool row_some = tok >= 0 && ks < ke;
            if (!row_some) ks = 0, ke = p.T_kv;  // masks nothing; its output is not taken from O
            fetch(info[e].t0_next);
            // the keys that all rows of the warp see
            const int all_lo = __reduce_max_sync(0xffffffffu, ks), all_hi = __reduce_min_sync(0xffffffffu, ke);
            const int jb = info[e].jb, n = w < info[e].subs ? tiles_of(info[e].n, w) : 0;
            float m = -INFINITY, l = 0.0f;  // the maximum that P and O refer to (log2 units), the sum
            int bias_pos = 0;
            float slope = 0.0f, bias_far = 0.0f;
            if (BIAS && tok >= 0) {
                const AttnBfBias b(p, tok, head, ks, ke);
                bias_pos = b.pos, slope = b.slope, bias_far = b.far;
            }
            for (int i = 0; ok && i < n; ++i, ++ns) {
                ok = mbar_wait_warp(&s_full[w], ns & 1u, p.timeout_ns, abort);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[4][32];
                tmem_ld_32x32b_x32(t_s, v[0]);
                tmem_ld_32x32b_x32(t_s + 32, v[1]);
                tmem_wait_ld();
                tmem_tie(v[0]);
                tmem_tie(v[1]);
                tmem_ld_32x32b_x32(t_s + 64, v[2]);
                tmem_ld_32x32b_x32(t_s + 96, v[3]);
                float mx[4];
                auto row_max = [&](int q) {
                    float x = __uint_as_float(v[q][0]), y = __uint_as_float(v[q][1]);
#pragma unroll
                    for (int i = 2; i < 30; i += 4) {
                        x = fmaxf(fmaxf(x, __uint_as_float(v[q][i])), __uint_as_float(v[q][i + 1]));
                        y = fmaxf(fmaxf(y, __uint_as_float(v[q][i + 2])), __uint_as_float(v[q][i + 3]));
                    }
                    mx[q] = fmaxf(fmaxf(x, y), fmaxf(__uint_as_float(v[q][30]), __uint_as_float(v[q][31])));
                };
                // the first half's maximum while the second half is on its way, unless the scores change first
                if (!CAP && !BIAS) row_max(0), row_max(1);
                tmem_wait_ld();
                tmem_tie(v[2]);
                tmem_tie(v[3]);
                const int k0 = (jb + (p.alt ? 2 * i + w : i)) * 128;
                if (CAP) {
                    float far = 0.0f;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int y = 0; y < 32; y += 2)
                            far = fmaxf(fmaxf(far, fabsf(__uint_as_float(v[q][y]))), fabsf(__uint_as_float(v[q][y + 1])));
                    // Each value takes the form of its own size.  The warp's vote, in which masked keys and other
                    // rows take part, only skips the other form where no value takes it: one form a tile by that
                    // vote made the far one 1.2 times as fast, but a row's bits then hung on what it does not see.
                    // (a NaN is passed over by the maximum and stays one in either form)
                    const uint64_t cc = f2_splat(p.c);
                    if (__all_sync(0xffffffffu, far * p.c <= 1.0f || tok < 0)) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int y = 0; y < 32; y += 2) {
                                const uint64_t x = f2_mul(f2_pack(__uint_as_float(v[q][y]), __uint_as_float(v[q][y + 1])), cc);
                                float a, b;
                                f2_unpack(tanh_near(x, p.tanh), a, b);
                                v[q][y] = __float_as_uint(a), v[q][y + 1] = __float_as_uint(b);
                            }
                    } else {
                        // tanh(x) = 1 - 2 / (1 + 2^(2 x log2 e)): within 2^-21 of cap
                        auto far_form = [&](float x) {
                            return __fmaf_rn(-2.0f * p.cap, rcp_approx(1.0f + ex2(x * (2.0f * 1.44269504f))), p.cap);
                        };
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int y = 0; y < 32; y += 2) {
                                const uint64_t x = f2_mul(f2_pack(__uint_as_float(v[q][y]), __uint_as_float(v[q][y + 1])), cc);
                                float x0, x1, a, b;
                                f2_unpack(x, x0, x1);
                                f2_unpack(tanh_near(x, p.tanh), a, b);
                                v[q][y] = __float_as_uint(fabsf(x0) <= 1.0f ? a : far_form(x0));
                                v[q][y + 1] = __float_as_uint(fabsf(x1) <= 1.0f ? b : far_form(x1));
                            }
                    }
                }
                if (BIAS) {
                    const float from = (float)(bias_pos - k0);
                    if (!CAP) {
                        const float off = -bias_far * slope;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                const float b = __fmaf_rn(fabsf(from - (float)(32 * q + y)), slope, off);
                                v[q][y] = __float_as_uint(__fmaf_rn(__uint_as_float(v[q][y]), p.c, b));
                            }
                    } else if (__any_sync(0xffffffffu, bias_far != 0.0f)) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                v[q][y] = __float_as_uint(__fmaf_rn(fabsf(from - (float)(32 * q + y)) - bias_far, slope,
                                                                    __uint_as_float(v[q][y])));
                    } else {  // (the same where nothing is taken off)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                v[q][y] = __float_as_uint(__fmaf_rn(fabsf(from - (float)(32 * q + y)), slope,
                                                                    __uint_as_float(v[q][y])));
                    }
                }
                // the multiplier still to be applied
                const float c = CAP || BIAS ? 1.0f : p.c;
                const bool cut = k0 < all_lo || k0 + 128 > all_hi;
                if (cut) {
                    const int a = ks - k0, b = ke - k0;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (32 * q + y < a || 32 * q + y >= b) v[q][y] = 0xFF800000u;
                }
                if (CAP || BIAS || cut) row_max(0), row_max(1);
                row_max(2), row_max(3);
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
                            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st_32x32b_x16(t_o + 32 * b, *reinterpret_cast<const uint32_t(*)[16]>(o));
                            tmem_st_32x32b_x16(t_o + 32 * b + 16, *reinterpret_cast<const uint32_t(*)[16]>(o + 16));
                        }
                    }
                }
                const uint64_t c2 = f2_splat(c), m2 = f2_splat(m == -INFINITY ? 0.0f : -m);
                uint64_t sum[2] = {f2_splat(0.0f), f2_splat(0.0f)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int q = 2 * half; q < 2 * half + 2; ++q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            float a, b;
                            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[q][2 * y]), __uint_as_float(v[q][2 * y + 1])), c2, m2), a,
                                      b);
                            a = ex2(a), b = ex2(b);
                            sum[y & 1] = f2_add(sum[y & 1], f2_pack(a, b));
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
                            pk[y] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        tmem_st_32x32b_x16(t_s + 16 * q, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * w + half]);
                }
                float a, b;
                f2_unpack(f2_add(sum[0], sum[1]), a, b);
                l += a + b;
            }
            // ------------------------------------------------------------ the rows' outputs
            if (ok && n > 0) {
                ok = mbar_wait_warp(&o_full[w], no & 1u, p.timeout_ns, abort);
                ++no;
            }
            if (!ok) break;
            tc_fence_after();
            const bool some = row_some && n > 0, bad = info[e].bad != 0;
            const float inv = some && p.parts == 1 ? 1.0f / l : 1.0f;
            const size_t row = (size_t)tok * p.H + head;
            const size_t part = (size_t)(p.alt ? 2 * info[e].z + w : info[e].z) * p.T_q * p.H + row;
            // (a loop, whose code is a quarter: 32760 rows over 512 keys took 451 us unrolled and 423 so; but capped
            // and biased scores, 812 and 706 us at 8192 x 8192, took 842 and 727 with it)
#pragma unroll (CAP || BIAS ? D / 32 : 1)
            for (int b = 0; b < D / 32; ++b) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld_32x32b_x32(t_o + 32 * b, o);
                    tmem_wait_ld();
                    tmem_tie(o);
                    if (b == D / 32 - 1) {  // O is read: the next item may write it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_free[w]);
                    }
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = some ? __float_as_uint(__uint_as_float(o[y]) * inv) : 0u;
                if (bad && some) {
                    // repair: the values that the guard took out, for the rows that attend their keys
                    AttnBfItem wk;
                    wk.see_lo = info[e].see_lo, wk.see_hi = info[e].see_hi;
#pragma unroll 1
                    for (int i = 0; i < n; ++i) {
                        const int j = jb + (p.alt ? 2 * i + w : i);
                        if (!wk.guarded(j, p.T_kv)) continue;
#pragma unroll 1
                        for (int key = max(ks, j * 128); key < min(ke, j * 128 + 128); ++key) {
                            const __nv_bfloat16* src = p.v + key * p.v_stride + info[e].hk * D + 32 * b;
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                const float x = __bfloat162float(src[y]);
                                if (!(fabsf(x) < INFINITY)) o[y] = __float_as_uint(__uint_as_float(o[y]) + x);
                            }
                        }
                    }
                }
                if (tok >= 0 && p.parts > 1) {
                    float4* dst = reinterpret_cast<float4*>(p.part_o + part * D + 32 * b);
#pragma unroll
                    for (int y = 0; y < 8; ++y)
                        dst[y] = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                             __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
                } else if (tok >= 0) {
                    __nv_bfloat16* dst = p.o + (size_t)tok * p.o_stride + head * D + 32 * b;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t h[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[16 * y + 2 * c]),
                                                                            __uint_as_float(o[16 * y + 2 * c + 1]));
                            h[c] = *reinterpret_cast<const uint32_t*>(&h2);
                        }
                        if (p.o_32) {
                            st_global_v8(dst + 16 * y, h);
                        } else {
                            *reinterpret_cast<uint4*>(dst + 16 * y) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(dst + 16 * y + 8) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                    }
                }
                __syncwarp();  // (the next TMEM load is for the whole warp)
            }
            if (tok >= 0) {
                if (p.parts > 1)
                    p.part_ml[part] = some ? make_float2(m, l) : make_float2(-INFINITY, -1.0f);
                else if (p.lse && !some)
                    p.lse[row] = -INFINITY;
                else if (p.lse)
                    p.lse[row] = BIAS ? AttnBfBias(p, tok, head, ks, ke).lse(p, tok, head, m + log2f(l))
                                      : (m + log2f(l)) * 0.693147181f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[e]);
        }
        if (!ok && lane == 0) attn_bf_fail(p, abort);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of a row joined in order: o = sum_z 2^(m_z - m) O_z / sum_z 2^(m_z - m) l_z.  A part without
// keys (l < 0) is passed over; where all keys score -infinity (m too, l = 0) the division gives NaN, as in one part.  A warp takes a row, D / 32 values a lane.
template <int D>
__global__ void __launch_bounds__(128) attn_bf16_join_kernel(const __grid_constant__ AttnBfParams p) {
    constexpr int V = D / 32;
    const int64_t rows = (int64_t)p.T_q * p.H, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    float m = -INFINITY;
    for (int z = 0; z < p.parts; ++z) m = fmaxf(m, p.part_ml[z * rows + row].x);
    float l = 0.0f, acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    bool some = false;
    for (int z = 0; z < p.parts; ++z) {
        const float2 ml = p.part_ml[z * rows + row];
        if (ml.y < 0.0f) continue;
        some = true;
        const float f = ml.x == m ? 1.0f : exp2f(ml.x - m);
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
    if (p.lse && lane == 0) {
        float y = some ? (m + log2f(l)) * 0.693147181f : -INFINITY;
        if (some && p.slopes) {
            const int ks = p.key_start ? max(p.key_start[tok], 0) : 0;
            const int ke = p.key_end ? min(p.key_end[tok], p.T_kv) : p.T_kv;
            const int head = (int)(row - tok * p.H);
            y = AttnBfBias(p, (int)tok, head, ks, ke).lse(p, (int)tok, head, m + log2f(l));
        }
        p.lse[row] = y;
    }
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
