// cache_attn_wide.cuh -- attention over a paged cache of 8 or 4 bits, units of 33 to 128 rows (see cache_attn.cu,
// cache4_attn.cu).
//
// The mathematics is cache_attn.cu's with the operands' roles swapped: the unit's (token, head) rows are the rows of the
// products, S = Q K^T and O = P V, keys and dims their columns.  A softmax thread owns one row: maximum, sum and fades are
// its own registers, and nothing crosses lanes or waits at a barrier.  A tile of 128 x 128 takes 5.7k warp instructions
// instead of the 10.2k of a thread for each key, but lanes without a row have no work, so units of up to 32 rows stay
// with the other kernel.  The weights are written over the tile's scores in TMEM and are the A operand of P V: 64 KB of
// shared memory less than as a shared operand, which holds four more K and V tiles (1.41 -> 1.33 ms on the chunk below).
//
// Tensor memory holds the scores of three tiles and one O: S runs two tiles ahead of O, so a softmax group that ends a
// tile finds the scores of its next.
//
// What bounds it.  Chunks: the softmax groups' issue and latencies.  2048 queries over 16384 keys, 64 heads on 8, take
// 1.00 ms, 1027 TFLOP/s of the products (4 FLOP a pair and dim) or twice that as executed in 8-bit pieces; the tensor pipe
// is active 36 % of the time, issue slots 49 %, and without the softmax it takes 0.68 ms.  Selected keys: loading them.  4096
// rows of 512 keys, 64 heads on one, take 238 us where all of them are seen and 285 us in the causal prompt of 1024
// compressed keys, whose first rows see few (unseen tiles are walked like others).  Of the 238 us, 151 us are left without softmax,
// joining, output and conversion of queries.
//
// The register split leaves the four kernels of the 8-bit cache 260 to 412 bytes of spills, those of the 4-bit cache 360 to 468
// (-Xptxas -v).  A second group of widening warps there takes registers from the others: 32 decode rows of 2048 selected keys 32.0
// us instead of 30.0, 4 sequences of 131072 keys with 64 heads on one 64.0 us instead of 61.7.
//
// Units of at most 64 rows (one selected row of 64 heads, a decode step on a shared key head) are laid out twice: row r
// again as row r + 64.  Of a tile's keys the first copy's weights hold the first 64, the second copy's the others (zeros
// elsewhere), so all four warps of a softmax group work, on half of the keys each, with the scores kept in registers;
// each copy has its own maximum and sum, and the joining warps add the copies when a segment ends.
#pragma once
#include "cache_attn.cuh"

namespace lidx {

// TWICE: units of at most 64 rows.
template <int BITS, bool TWICE>
struct WideCfg {
    static constexpr int N = 128, QB = 2;
    using RING = AttnSlots<BITS, BITS == 8 ? 4 : 2, BITS == 8 ? 4 : 3>;
    static constexpr int SLOTS = RING::ALL, PACKED = BITS == 8 ? 0 : (TWICE ? 5 : 7);
    static constexpr int Q_BYTES = 2 * N * 128;  // hi and lo
    static constexpr int OFF_Q = SLOTS * kASlotBytes;
    static constexpr int OFF_META = OFF_Q + QB * Q_BYTES;                // [3][kAMeta][128] of the keys
    static constexpr int OFF_SEEN = OFF_META + 3 * kAMeta * kATile * 4;  // [kAMeta][4], then [kAMeta] flags
    static constexpr int OFF_QS = OFF_SEEN + 128;                        // [QB][N] query scales
    static constexpr int OFF_MT = OFF_QS + QB * N * 4;                   // [4][N] tile maxima
    static constexpr int OFF_L = OFF_MT + 4 * N * 4;                     // [2][N] float2: a group's sum, its reference
    static constexpr int OFF_GATHER = OFF_L + 2 * N * 8;                 // [4][128] cache rows of a tile's keys
    static constexpr int OFF_X = OFF_GATHER + 4 * kATile * 4;                // [32][128] dims that the copies exchange
    static constexpr int OFF_PACKED = OFF_X + (TWICE ? 32 * 128 * 4 : 0);  // 4 bits: packed tiles
    static constexpr int OFF_BAR = OFF_PACKED + PACKED * kAPackedBytes;
    static constexpr int NBAR = 2 * SLOTS + 2 * kAMeta + 2 * 2 + 3 + 4 + 2 + 2 + 1 + 2 * PACKED;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int TOTAL = OFF_MISC + 288 + 1024;
    static_assert(TOTAL <= 232448 && kAMeta * 20 <= 128, "shared memory");
    static_assert(OFF_QS % 16 == 0 && OFF_GATHER % 16 == 0 && OFF_MISC % 8 == 0, "16-byte reads");
    static constexpr int TMEM = 512;  // three tiles of S (and the weights over them), one of O
    // Warpgroups: MMA and queries (4 bits: and the producers); two of softmax that take the tiles in turn; joining; producers
    // (4 bits: four warps that widen).
    static constexpr int THREADS = 640, PRODUCERS = BITS == 8 ? 4 : 2, QWARPS = BITS == 8 ? 3 : 1;
    static constexpr int W_SOFT = 4, W_JOIN = 12, W_PROD = 16;
    static constexpr int R_LAUNCH = 96, R_MMA = BITS == 8 ? 56 : 64, R_SOFT = 96, R_JOIN = 176, R_PROD = BITS == 8 ? 56 : 48;
    static_assert(R_LAUNCH == 65536 / THREADS / 8 * 8 && R_MMA + 2 * R_SOFT + R_JOIN + R_PROD <= R_LAUNCH * 5,
                  "register split");
    static_assert(R_MMA <= R_LAUNCH && R_PROD <= R_LAUNCH && R_SOFT >= R_LAUNCH && R_JOIN >= R_LAUNCH, "directions");
};

// Products of 32 keys of this thread's row.  vis: bits of the keys the row sees (MASK; others become -inf).
template <bool MASK>
__device__ __forceinline__ void wide_products(uint32_t s_addr, uint32_t vis, float (&x)[32]) {
    uint32_t r[32];
    tmem_ld32(s_addr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = !MASK || ((vis >> i) & 1) ? __uint_as_float(r[i]) : -INFINITY;
}

// Scores from products, in log2 units: S * (key's factor * row's factor) + log2(v scale) (+ sh with SHIFT).  a, lv: of the 32 keys.
// UNI: the keys of a block of 16 share their page's factors.
template <bool MASK, bool UNI, bool SHIFT>
__device__ __forceinline__ void wide_scores(const float* a, const float* lv, float qs, float sh, uint32_t vis,
                                            float (&x)[32]) {
    const uint64_t q2 = pack2(qs, qs), sh2 = pack2(sh, sh);
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        uint64_t f0, f1, v0, v1;
        if constexpr (UNI) {
            const float f = a[i & 16] * qs, v = SHIFT ? lv[i & 16] + sh : lv[i & 16];
            f0 = f1 = pack2(f, f);
            v0 = v1 = pack2(v, v);
        } else {
            const float4 f = *reinterpret_cast<const float4*>(a + i);
            const float4 v = *reinterpret_cast<const float4*>(lv + i);
            f0 = mul2(pack2(f.x, f.y), q2);
            f1 = mul2(pack2(f.z, f.w), q2);
            v0 = pack2(v.x, v.y);
            v1 = pack2(v.z, v.w);
        }
        v0 = fma2(pack2(x[i], x[i + 1]), f0, v0);
        v1 = fma2(pack2(x[i + 2], x[i + 3]), f1, v1);
        unpack2(UNI || !SHIFT ? v0 : add2(v0, sh2), x[i], x[i + 1]);
        unpack2(UNI || !SHIFT ? v1 : add2(v1, sh2), x[i + 2], x[i + 3]);
    }
    if constexpr (MASK) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = (vis >> i) & 1 ? x[i] : -INFINITY;
    }
}

// SEL: selected keys.  TWICE: units of at most 64 rows.
template <bool SEL, bool TWICE, int BITS>
__global__ void __launch_bounds__(WideCfg<BITS, TWICE>::THREADS, 1)
    cache_attn_wide_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ AttnParams p) {
    using C = WideCfg<BITS, TWICE>;
    using RING = typename C::RING;
    constexpr int N = C::N, SLOTS = C::SLOTS, QB = C::QB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* const sQ = smem + C::OFF_Q;
    float* const sMt = (float*)(smem + C::OFF_MT);
    float2* const sL = (float2*)(smem + C::OFF_L);
    uint64_t* bars = (uint64_t*)(smem + C::OFF_BAR);
    AttnPipe x;
    x.kv = smem;
    x.q = sQ;
    x.q_scale = (float*)(smem + C::OFF_QS);
    x.key_a = (float*)(smem + C::OFF_META);
    x.key_lv = x.key_a + kAMeta * kATile;
    x.key_iv = x.key_lv + kAMeta * kATile;
    x.seen = (uint32_t*)(smem + C::OFF_SEEN);
    x.flag = x.seen + 4 * kAMeta;
    x.rows = (int*)(smem + C::OFF_GATHER);
    x.packed = smem + C::OFF_PACKED;
    uint64_t* const kv_full = x.kv_full = bars;
    uint64_t* const kv_empty = x.kv_empty = kv_full + SLOTS;
    uint64_t* const meta_full = x.meta_full = kv_empty + SLOTS;
    uint64_t* const meta_empty = x.meta_empty = meta_full + kAMeta;
    uint64_t* const q_full = x.q_full = meta_empty + kAMeta;
    uint64_t* const q_empty = x.q_empty = q_full + 2;
    uint64_t* s_full = q_empty + 2;  // [3] S of a tile in TMEM
    uint64_t* p_full = s_full + 3;   // [4] weights and tile maxima written (and S read)
    uint64_t* o_full = p_full + 4;   // O of a tile in TMEM (and the weights read)
    uint64_t* o_empty = o_full + 1;  // O read
    uint64_t* l_full = o_empty + 1;  // sums of a segment written
    uint64_t* l_empty = l_full + 1;
    uint64_t* drain = l_empty + 1;
    uint64_t* const pk_full = x.pk_full = drain + 1;
    uint64_t* const pk_empty = x.pk_empty = pk_full + C::PACKED;
    uint32_t* tmem_slot = (uint32_t*)(smem + C::OFF_MISC);
    int64_t* const scan = (int64_t*)(smem + C::OFF_MISC + 8);  // [34]

    // the warp's number by a shuffle: known to be uniform, so a role's counters and descriptors live in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(kv_full + i, BITS == 8 ? 1 : 4);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < kAMeta; ++i) {
            mbar_init(meta_full + i, 1);
            mbar_init(meta_empty + i, 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, C::QWARPS);
            mbar_init(q_empty + i, 1 + 8);
        }
        for (int i = 0; i < 3; ++i) mbar_init(s_full + i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(p_full + i, 4);
        mbar_init(o_full, 1);
        mbar_init(o_empty, 4);
        mbar_init(l_full, 8);
        mbar_init(l_empty, 4);
        mbar_init(drain, 1);
        for (int i = 0; i < C::PACKED; ++i) {
            mbar_init(pk_full + i, SEL ? 33 : 1);  // copies of the lanes arrive by themselves
            mbar_init(pk_empty + i, 4);
        }
        fence_mbar_init();
        if constexpr (BITS == 8) {
            tma_prefetch_desc(&tmk);
            tma_prefetch_desc(&tmv);
        }
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, C::TMEM);
        tmem_relinquish();
    }
    AttnWalk wk;
    int64_t W;
    tc_fence_before();
    const int nc = attn_begin<C::THREADS>(p, wk, W, scan), c = blockIdx.x;
    grid_dependency_launch();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int rows = p.TS * p.G;  // of a unit

    if (warp < 4) {
        regs_dec<C::R_MMA>();
        if (warp == 0) {
            // ------------------------------------------------------- MMA issuer
            // The whole warp walks and waits; one lane issues.
            const bool issuer = elect_one();
            const uint32_t id_s = idesc_e4m3_f32(128, kATile);
            const uint32_t id_o = idesc_e4m3_f32(128, (uint32_t)p.D) | kIdescBMn;
            const int nk = (p.D + 31) / 32;
            const uint64_t dk0 = smem_desc_kmajor(smem_u32(smem), 128);
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(smem), kASlotBytes);
            const uint64_t dq0 = smem_desc_kmajor(smem_u32(sQ), 128);
            bool ok = true;
            int tc = 0, sc = 0;
            // O of tile t: (hi + lo) V
            auto second = [&](int t) {
                const int sl = RING::at(t, 1);
                ok = ok && mbar_wait(kv_full + sl, RING::phase(t, 1), p.wait_ns);
                ok = ok && mbar_wait(o_empty, (t & 1) ^ 1, p.wait_ns);
                ok = ok && mbar_wait(p_full + (t & 3), (t >> 2) & 1, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                const uint32_t a = tmem + t % 3 * 128;  // the weights, in the columns of the tile's S
                const uint64_t b = dv0 + (uint64_t)(sl * (kASlotBytes >> 4));
                const uint32_t d = tmem + 384;
                if (issuer) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 32 keys a step
                        umma_f8_ts(d, a + 16 * k, b + k * (32 * 128 >> 4), id_o, k > 0);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_f8_ts(d, a + 16 * k + 8, b + k * (32 * 128 >> 4), id_o, 1);
                    umma_commit(o_full);
                    umma_commit(kv_empty + sl);
                }
                __syncwarp();
            };
            while (ok && wk.next(p)) {
                if (wk.gr.n == 0) continue;
                const int qb = sc % QB;
                ok = ok && mbar_wait(q_full + qb, (sc / QB) & 1, p.wait_ns);
                for (int t = wk.t0; ok && t < wk.t1; ++t, ++tc) {
                    const int sl = RING::at(tc, 0);
                    ok = mbar_wait(kv_full + sl, RING::phase(tc, 0), p.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = dq0 + (uint64_t)(qb * (C::Q_BYTES >> 4));
                    const uint64_t b = dk0 + (uint64_t)(sl * (kASlotBytes >> 4));
                    const uint32_t d = tmem + tc % 3 * 128;  // (its last tile's weights are read by a product before)
                    if (issuer) {
                        // 32 dims a step, hi then lo
                        if (nk == 4) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, a + (N * 128 >> 4) + 2 * k, b + 2 * k, id_s, 1);
                        } else {
                            // (the places past D are zero: a narrower head takes fewer steps)
#pragma unroll 1
                            for (int k = 0; k < nk; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll 1
                            for (int k = 0; k < nk; ++k) umma_f8(d, a + (N * 128 >> 4) + 2 * k, b + 2 * k, id_s, 1);
                        }
                        umma_commit(s_full + tc % 3);
                        umma_commit(kv_empty + sl);
                        if (t == wk.t1 - 1) umma_commit(q_empty + qb);
                    }
                    __syncwarp();
                    // S two tiles ahead of O: a softmax group that ends a tile finds the scores of its next
                    if (tc > 1) second(tc - 2);
                }
                ++sc;
            }
            if (ok && tc > 1) second(tc - 2);
            if (ok && tc > 0) second(tc - 1);
            if (!__all_sync(0xffffffffu, ok)) {  // products in flight end before the memory is given up
                if (issuer) umma_commit(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        } else if (warp <= C::QWARPS) {
            attn_queries<N, QB, C::QWARPS>(p, wk, x, warp - 1, lane, TWICE);
        } else if constexpr (BITS == 4) {
            attn_produce4<C::PACKED, C::PRODUCERS, SEL>(p, wk, x, warp - 1 - C::QWARPS, lane);
        }
    } else if (warp < C::W_JOIN) {
        // -------------------------------------------------------------- softmax
        regs_inc<C::R_SOFT>();
        const int grp = (warp - C::W_SOFT) >> 2, row = tid & 127, wg_warp = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16);
        const int n = TWICE ? row & 63 : row;                                 // row of the unit
        const bool works = (TWICE ? wg_warp & 1 : wg_warp) * 32 < rows;       // the warp has a row
        const int st = attn_token(p, n);
        bool ok = true;
        int tc = 0, sc = 0;
        while (wk.next(p)) {
            if (wk.gr.n == 0) continue;
            const int qb = sc % QB, s = wk.gr.st * p.TS + st;
            int end = INT_MAX, least = INT_MAX;  // keys this row sees; keys every row sees
            if (!SEL) {
                end = n < rows && s < p.S ? attn_end(p, wk.gr.b, s) : 0;
                least = attn_end(p, wk.gr.b, wk.gr.st * p.TS);
            }
            ok = ok && mbar_wait(q_full + qb, (sc / QB) & 1, p.wait_ns);
            const float qs = x.q_scale[qb * N + row];
            float l = 0.f, m = -INFINITY;
            for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                if ((tc & 1) != grp) continue;
                const int bf = tc % 3, ph = (tc / 3) & 1, ms = tc % kAMeta;
                ok = ok && mbar_wait(x.meta_full + ms, (tc / kAMeta) & 1, p.wait_ns);
                const float* const ka = x.key_a + ms * kATile;
                const float* const kl = x.key_lv + ms * kATile;
                const float* const ki = x.key_iv + ms * kATile;
                const bool flag = x.flag[ms] != 0;
                const bool masked = flag || t * kATile + kATile > least;
                // S of this tile is done, and with it the O of three tiles ago, which was issued before it when the tile
                // before that was joined: the maxima of four tiles ago have been read
                ok = ok && mbar_wait(s_full + bf, ph, p.wait_ns);
                tc_fence_after();
                const uint32_t s_addr = lane_addr + bf * 128;

                // TWICE: chunks of 32 keys [2 half, 2 half + 2), products kept (scores, where not UNI); else all four, read twice.
                // UNI (a cache page's keys follow each other, a positive softmax scale): the largest score of a block is
                // that of its largest product, so the first pass has no scores to compute (chunk: 1.14 -> 1.05 ms).  The
                // second adds the shift to the factor log2(v scale) first, which is only done where scores are below
                // 2^20, so that no weight comes out above 2^8.3: returns false where they are not.
                auto one_tile = [&](auto mask_c, auto uni_c) {
                    constexpr bool MASK = decltype(mask_c)::value, UNI = decltype(uni_c)::value;
                    constexpr int NCH = TWICE ? 2 : 4, KEEP = TWICE ? 2 : 1;
                    const int c0 = TWICE && row >= 64 ? 2 : 0;
                    uint32_t vis[NCH];
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        vis[i] = ~0u;
                        if constexpr (MASK) {
                            const int left = end - (t * kATile + 32 * (c0 + i));  // keys of the word below the row's end
                            vis[i] = x.seen[ms * 4 + c0 + i] & (left >= 32 ? ~0u : (left > 0 ? (1u << left) - 1 : 0u));
                        }
                    }
                    float v[KEEP][32], top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const int at = 32 * (c0 + i);
                        float(&u)[32] = v[TWICE ? i : 0];
                        wide_products<MASK && UNI>(s_addr + at, vis[i], u);
                        if constexpr (UNI) {
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {
                                float b = u[h];
#pragma unroll
                                for (int k = 1; k < 15; k += 2) b = max3_nan(b, u[h + k], u[h + k + 1]);
                                b = max_nan(b, u[h + 15]);
                                if (b != -INFINITY) top = max_nan(top, fmaf(b, ka[at + h] * qs, kl[at + h]));
                            }
                        } else {
                            wide_scores<MASK, UNI, false>(ka + at, kl + at, qs, 0.f, vis[i], u);
#pragma unroll
                            for (int k = 0; k < 32; k += 2) top = max3_nan(top, u[k], u[k + 1]);
                        }
                    }
                    if constexpr (UNI)
                        if (__any_sync(0xffffffffu, fabsf(top) > 0x1p20f && top != -INFINITY)) return false;
                    const float sh = top == -INFINITY ? kATop : kATop - top;
                    uint64_t sum0 = pack2(0.f, 0.f), sum1 = sum0;
#pragma unroll
                    for (int i = 0; i < NCH; ++i) {
                        const int at = 32 * (c0 + i);
                        float(&u)[32] = v[TWICE ? i : 0];
                        if constexpr (!TWICE) wide_products<false>(s_addr + at, 0, u);
                        if constexpr (UNI || !TWICE) {
                            wide_scores<MASK, UNI, true>(ka + at, kl + at, qs, sh, vis[i], u);
                        } else {
                            const uint64_t sh2 = pack2(sh, sh);
#pragma unroll
                            for (int k = 0; k < 32; k += 2) unpack2(add2(pack2(u[k], u[k + 1]), sh2), u[k], u[k + 1]);
                        }
                        uint32_t w[16];  // hi and lo of 32 keys
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float w0 = exp2_approx(u[k]), w1 = exp2_approx(u[k + 1]);
                            const float w2 = exp2_approx(u[k + 2]), w3 = exp2_approx(u[k + 3]);
                            if constexpr (UNI) {
                                const float iv = ki[at + (k & 16)];
                                sum0 = fma2(pack2(w0, w1), pack2(iv, iv), sum0);
                                sum1 = fma2(pack2(w2, w3), pack2(iv, iv), sum1);
                            } else {
                                const float4 iv = *reinterpret_cast<const float4*>(ki + at + k);
                                sum0 = fma2(pack2(w0, w1), pack2(iv.x, iv.y), sum0);
                                sum1 = fma2(pack2(w2, w3), pack2(iv.z, iv.w), sum1);
                            }
                            uint32_t h0, l0, h1, l1;
                            split_e4m3(w0, w1, h0, l0);
                            split_e4m3(w2, w3, h1, l1);
                            w[k / 4] = h0 | (h1 << 16);
                            w[8 + k / 4] = l0 | (l1 << 16);
                        }
                        tmem_st16(s_addr + at / 2, w);  // columns whose scores have been read
                    }
                    if constexpr (TWICE) {  // the other half of the keys has no weight in this copy
                        uint32_t z[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) z[k] = 0;
                        tmem_st16(s_addr + (c0 ^ 2) * 16, z);
                        tmem_st16(s_addr + (c0 ^ 2) * 16 + 16, z);
                    }
                    tmem_st_wait();
                    float a0, a1, b0, b1;
                    unpack2(sum0, a0, a1);
                    unpack2(sum1, b0, b1);
                    const float mn = max_nan(m, top);
                    if (top != -INFINITY) {
                        l = (m == -INFINITY ? 0.f : l * exp2_approx(m - mn)) + ((a0 + a1) + (b0 + b1)) * exp2_approx(top - mn);
                        m = mn;
                    }
                    sMt[(tc & 3) * N + row] = top;
                    return true;
                };
                if (works) {
                    const std::true_type yes{};
                    const std::false_type no{};
                    if constexpr (SEL) {
                        masked ? one_tile(yes, no) : one_tile(no, no);
                    } else {
                        const bool done = p.scale_log2 > 0.f && (masked ? one_tile(yes, yes) : one_tile(no, yes));
                        if (!done) one_tile(yes, no);
                    }
                }
                if (BITS == 8 && flag) {  // (4 bits: the producers write zeros there)
                    // unseen slots may hold anything (NaN codes): a zero weight alone would not keep them out.
                    // Thread i clears V's row i.
                    const int sl = RING::at(tc, 1);
                    ok = ok && mbar_wait(kv_full + sl, RING::phase(tc, 1), p.wait_ns);
                    if (ok && !((x.seen[ms * 4 + wg_warp] >> lane) & 1)) {
                        uint4* vrow = reinterpret_cast<uint4*>(smem + sl * kASlotBytes + row * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) vrow[i] = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(x.meta_empty + ms);
                    mbar_arrive(p_full + (tc & 3));
                }
            }
            ok = ok && mbar_wait(l_empty, (sc & 1) ^ 1, p.wait_ns);
            sL[grp * N + row] = make_float2(l, m);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(l_full);
                mbar_arrive(q_empty + qb);
            }
            ++sc;
        }
    } else if (warp < C::W_JOIN + 4) {
        // ---------------------------------------------------------------- joining
        // A thread has one row: its D outputs, maximum and sum.
        regs_inc<C::R_JOIN>();
        const int row = tid & 127, wg_warp = warp & 3;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + 384;
        const int n = TWICE ? row & 63 : row;
        const bool works = (TWICE ? wg_warp & 1 : wg_warp) * 32 < rows;
        const int d0 = TWICE && row >= 64 ? 64 : 0;    // dims this thread writes: [d0, dz)
        const int dz = TWICE ? min(p.D, d0 + 64) : p.D;
        const int st = attn_token(p, n);
        float* const sX = (float*)(smem + C::OFF_X);
        bool ok = true;
        int tc = 0, sc = 0;
        AttnHeader hd{0, 0, 0, 0};
        AttnHeader* const heads = reinterpret_cast<AttnHeader*>(p.ws);
        float* const parts = (float*)(p.ws + (size_t)gridDim.x * sizeof(AttnHeader));
        while (wk.next(p)) {
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.f;
            float m = -INFINITY, l = 0.f;
            if (wk.gr.n > 0) {
                for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                    // (four barriers: the softmax may be three tiles ahead of the joining)
                    ok = ok && mbar_wait(p_full + (tc & 3), (tc >> 2) & 1, p.wait_ns);
                    const float top = works ? sMt[(tc & 3) * N + row] : -INFINITY, mn = max_nan(m, top);
                    const float fa = m == -INFINITY ? 1.f : exp2_approx(m - mn);  // (acc is zero before a row's first key)
                    const float fb = top == -INFINITY ? 0.f : exp2_approx(top - mn);
                    m = mn;
                    // what there is fades before O is awaited, and only if a row's maximum grew
                    if (__any_sync(0xffffffffu, fa != 1.f)) {
                        const uint64_t fa2 = pack2(fa, fa);
#pragma unroll
                        for (int i = 0; i < 128; i += 2) unpack2(mul2(pack2(acc[i], acc[i + 1]), fa2), acc[i], acc[i + 1]);
                    }
                    ok = ok && mbar_wait(o_full, tc & 1, p.wait_ns);
                    tc_fence_after();
                    if (works) {
                        const uint64_t fb2 = pack2(fb, fb);
#pragma unroll
                        for (int cc = 0; cc < 128; cc += 32) {
                            if (cc < p.D) {  // (columns past D are never used)
                                uint32_t r[32];
                                tmem_ld32(lane_addr + cc, r);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 32; i += 2)
                                    unpack2(fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), fb2,
                                                 pack2(acc[cc + i], acc[cc + i + 1])),
                                            acc[cc + i], acc[cc + i + 1]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_empty);
                }
                ok = ok && mbar_wait(l_full, sc & 1, p.wait_ns);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float2 lm = sL[g * N + row];
                    if (lm.y != -INFINITY) l += lm.x * exp2_approx(lm.y - m);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(l_empty);
                ++sc;
            }
            if (TWICE && wk.gr.n > 0) {
                // The copies' maxima and sums; then the first copy takes dims 0 .. 63 of both, the second the others, 32
                // at a time, into acc[0 .. 63].
                sX[row] = m;
                sX[128 + row] = l;
                named_bar_sync(1, 128);
                const float mo = sX[row ^ 64], lo = sX[128 + (row ^ 64)], mm = fmaxf(m, mo);
                const float f = m == -INFINITY ? 0.f : exp2_approx(m - mm), fo = mo == -INFINITY ? 0.f : exp2_approx(mo - mm);
                l = l * f + lo * fo;
                m = mm;
                const bool one = row < 64;
#pragma unroll
                for (int r = 0; r < 64; r += 32) {
                    named_bar_sync(1, 128);  // what was there is read
#pragma unroll
                    for (int i = 0; i < 32; ++i) sX[i * 128 + row] = (one ? acc[64 + r + i] : acc[r + i]) * f;
                    named_bar_sync(1, 128);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        acc[r + i] = (one ? acc[r + i] : acc[64 + r + i]) * f + sX[i * 128 + (row ^ 64)];
                }
                named_bar_sync(1, 128);
            }
            const bool whole = wk.t0 == 0 && wk.t1 == wk.gr.w;
            if (whole) {
                const int s = wk.gr.st * p.TS + st;
                if (n < rows && s < p.S) {
                    const int at = (wk.gr.b * p.S + s) * p.Hq + wk.h * p.G + n - st * p.G;
                    const float inv = l > 0.f ? 1.f / l : 0.f;
                    uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)at * p.D + d0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (d0 + 8 * i < dz) {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const __nv_bfloat162 h =
                                    __floats2bfloat162_rn(acc[8 * i + 2 * k] * inv, acc[8 * i + 2 * k + 1] * inv);
                                w[k] = *reinterpret_cast<const uint32_t*>(&h);
                            }
                            out[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (p.lse && d0 == 0) p.lse[at] = attn_lse(m, l);
                }
            } else {
                const int slot = 2 * c + (wk.first ? 0 : 1);
                float* part = parts + slot * attn_part_floats(N);
                if (n < rows) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (d0 + 4 * i < dz)
                            reinterpret_cast<float4*>(part + n * 128 + d0)[i] =
                                make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
                    if (d0 == 0) {
                        part[N * 128 + n] = m;
                        part[N * 128 + N + n] = l;
                    }
                }
                if (wk.t0 == 0)  // place unit_end - 1 is in the share of the last CTA that begins at or before it
                    hd = AttnHeader{(int32_t)((wk.unit_end * nc - 1) / W), wk.g, wk.h, slot};
            }
            if (p.by_unit && wk.t0 == 0 && row == 0)
                heads[wk.g * p.Hkv + wk.h] = whole ? AttnHeader{0, 0, 0, 0} : hd;
        }
        if (!p.by_unit && row == 0) heads[c] = hd;
    } else {
        regs_dec<C::R_PROD>();
        if constexpr (BITS == 8)
            attn_produce<SLOTS, C::PRODUCERS, SEL>(p, wk, x, &tmk, &tmv, warp - C::W_PROD, lane);
        else
            attn_widen<RING, C::PACKED, 1>(p, wk, x, 0, warp & 3, lane);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

template <bool SEL, bool TWICE, int BITS>
static cudaError_t wide_launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid, cudaStream_t st) {
    auto* kernel = cache_attn_wide_kernel<SEL, TWICE, BITS>;
    cudaError_t e = set_smem_attr((const void*)kernel, WideCfg<BITS, TWICE>::TOTAL);
    if (e != cudaSuccess) return e;
    kernel<<<grid, WideCfg<BITS, TWICE>::THREADS, WideCfg<BITS, TWICE>::TOTAL, st>>>(mk, mv, p);
    return cudaGetLastError();
}
template <int BITS>
static cudaError_t wide_launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid,
                                    cudaStream_t st) {
    const bool twice = p.TS * p.G <= 64;
    if (p.idx) return twice ? wide_launch<true, true, BITS>(mk, mv, p, grid, st) : wide_launch<true, false, BITS>(mk, mv, p, grid, st);
    return twice ? wide_launch<false, true, BITS>(mk, mv, p, grid, st) : wide_launch<false, false, BITS>(mk, mv, p, grid, st);
}

}  // namespace lidx
