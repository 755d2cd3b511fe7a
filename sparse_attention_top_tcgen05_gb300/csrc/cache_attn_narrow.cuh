// cache_attn_narrow.cuh -- the attention kernel of units of up to 32 rows over a paged cache of 8 or 4 bits (see
// cache_attn.cu, cache4_attn.cu).
#pragma once
#include "cache_attn.cuh"

namespace lidx {

// Configuration of the kernel with room for N rows, N = 16 or 32, of which a softmax thread has NC, over a cache of BITS bits.
//
// 4 bits, slots and packed tiles in shared memory (64 ragged sequences to 32768 keys): 3 + 3 slots and 8 packed tiles 339 us, 2 +
// 3 and 11 348 us.
//
// The products' columns are the rows' hi and lo parts.  8 bits: a product for the hi part and one for the lo part into the
// same columns.  4 bits, where shared memory also serves the widening: one product of twice the columns, which
// reads K and V once (363 us with two, 356 us with one); whoever reads its columns adds the two.
template <int N, int NC_, int BITS>
struct AttnCfg {
    static_assert((N == 16 && (NC_ == 8 || NC_ == 16)) || (N == 32 && NC_ == 16), "columns");
    // Two softmax groups of four warps, NC columns each.  At N = 16 they take the tiles in turn, at N = 32 they share each
    // tile's columns: a thread keeps its scores and sums in registers either way.
    static constexpr bool SPLIT = N == 32;
    static constexpr int COLS = SPLIT ? N : NC_;       // columns that hold rows
    static constexpr int SG = 2, NC = NC_, QB = 2;
    using RING = AttnSlots<BITS, BITS == 8 ? 4 : 3, BITS == 8 ? 4 : 3>;
    static constexpr int SLOTS = RING::ALL, PACKED = BITS == 8 ? 0 : 8;
    static constexpr int MN = BITS == 8 ? N : 2 * COLS;  // columns of a product
    static constexpr int Q_BYTES = 2 * COLS * 128;     // hi and lo
    // Weights, a key 128 bytes, two buffers: 8 bits, hi and lo in a tile each; 4 bits, whose packed tiles need the room, hi
    // and lo columns of both buffers beside each other in one tile
    static constexpr int P_BYTES = BITS == 8 ? 2 * kASlotBytes : MN;
    static constexpr int OFF_P = SLOTS * kASlotBytes;
    static constexpr int OFF_Q = OFF_P + (BITS == 8 ? 2 * P_BYTES : kASlotBytes);
    static constexpr int OFF_META = OFF_Q + QB * Q_BYTES;              // [3][kAMeta][128] of the keys
    static constexpr int OFF_SEEN = OFF_META + 3 * kAMeta * kATile * 4;  // [kAMeta][4], then [kAMeta] flags
    static constexpr int OFF_QS = OFF_SEEN + 128;                      // [QB][COLS] query scales
    static constexpr int OFF_W = OFF_QS + QB * N * 4;                  // [2][SG][4][NC] warp maxima of a tile
    static constexpr int OFF_MB = OFF_W + 2 * SG * 4 * NC * 4;         // [4 SG][3][NC] of a warp: 8 - M, fades
    static constexpr int OFF_END = OFF_MB + 4 * SG * 3 * NC * 4;       // [SG][NC] keys a column sees
    static constexpr int OFF_MT = OFF_END + SG * NC * 4;               // [4][N] tile maxima
    static constexpr int OFF_AB = OFF_MT + 4 * N * 4;                  // [2][2][N] fades of acc and tile
    static constexpr int OFF_L = OFF_AB + 2 * N * 8;                   // [SG][4][NC] sums of the warps
    static constexpr int OFF_MW = OFF_L + SG * 4 * NC * 4;             // [SG][NC] their reference
    static constexpr int OFF_INV = OFF_MW + SG * NC * 4;               // [N] 1 / l
    static constexpr int OFF_ROW = OFF_INV + N * 4;                    // [N] output rows
    static constexpr int OFF_GATHER = OFF_ROW + N * 4;                 // [4][128] cache rows of a tile's keys
    static constexpr int OFF_PACKED = OFF_GATHER + 4 * kATile * 4;     // 4 bits: packed tiles
    static constexpr int OFF_BAR = OFF_PACKED + PACKED * kAPackedBytes;
    static constexpr int NBAR = 2 * SLOTS + 2 * kAMeta + 2 * 2 + 3 * 2 + 4 + 2 + 1 + 2 * PACKED;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;                // start of the share, TMEM address
    static constexpr int TOTAL = OFF_MISC + 288 + 1024;                // + alignment of the base
    static_assert(TOTAL <= 232448 && kAMeta * 20 <= 128, "shared memory");
    static_assert(OFF_QS % 16 == 0 && OFF_MB % 16 == 0 && OFF_END % 16 == 0 && OFF_AB % 16 == 0 && OFF_W % 16 == 0 &&
                      OFF_GATHER % 16 == 0 && OFF_MISC % 8 == 0,
                  "16-byte reads");
    static constexpr int TMEM = 4 * MN;                                // columns: two tiles of S and of O
    // Warpgroups: MMA and queries (4 bits: and the producers); two of softmax; joining; producers (4 bits: two that widen, K
    // tiles and V tiles).
    static constexpr int THREADS = BITS == 8 ? 640 : 768, PRODUCERS = BITS == 8 ? 4 : 2, QWARPS = BITS == 8 ? 3 : 1;
    static constexpr int W_QUERY = 1, W_SOFT = 4, W_JOIN = 12, W_PROD = 16;  // first warps
    // registers a thread of each group: their sum is at most what the launch has
    static constexpr int R_LAUNCH = BITS == 8 ? 96 : 80, R_MMA = BITS == 8 ? 64 : (SPLIT ? 72 : 80);
    static constexpr int R_SOFT = BITS == 8 ? 112 : (NC == 8 ? 88 : 96), R_JOIN = BITS == 8 || SPLIT ? 104 : 80;
    static constexpr int R_PROD = BITS == 8 ? 88 : (SPLIT ? 56 : 64);
    static_assert(R_LAUNCH == 65536 / THREADS / 8 * 8 &&
                      R_MMA + SG * R_SOFT + R_JOIN + R_PROD * (THREADS / 32 - W_PROD) / 4 <= R_LAUNCH * (THREADS / 128),
                  "register split");
    static_assert(R_MMA <= R_LAUNCH && R_PROD <= R_LAUNCH && R_SOFT >= R_LAUNCH && R_JOIN >= R_LAUNCH, "directions");
};

// Sums over the warp's lanes of NC columns: lane i returns column i % NC's.
template <int NC>
__device__ __forceinline__ float warp_sum_columns(float (&v)[NC], int lane) {
#pragma unroll
    for (int s = 16; s >= NC; s >>= 1) {
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
    }
#pragma unroll
    for (int step = NC / 2; step > 0; step >>= 1) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float send = up ? v[i] : v[i + step], keep = up ? v[i + step] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
        }
    }
    return v[0];
}

// x of the columns of this thread's key: (S^T * key's factor) * column's factor + log2(v scale); unseen -inf.  LO > 0: the lo
// parts' products are LO columns on.
template <bool MASK, int NC, int LO>
__device__ __forceinline__ void attn_scores(uint32_t s_addr, const float* qs, const int* ends, uint64_t a2,
                                            uint64_t lv2, int key, bool seen, float (&x)[NC]) {
    uint32_t r[NC];
    if constexpr (NC == 8) {
        uint32_t both[16];
        tmem_ld16(s_addr, both);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(both[i]) + __uint_as_float(both[8 + i]));
    } else {
        tmem_ld16(s_addr, r);
        if constexpr (LO > 0) {
            uint32_t lo[16];
            tmem_ld16(s_addr + LO, lo);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(lo[i]));
        } else {
            tmem_ld_wait();
        }
    }
#pragma unroll
    for (int i = 0; i < NC; i += 4) {
        const float4 q4 = *reinterpret_cast<const float4*>(qs + i);
        const uint64_t x0 = fma2(mul2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), a2),
                                 pack2(q4.x, q4.y), lv2);
        const uint64_t x1 = fma2(mul2(pack2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), a2),
                                 pack2(q4.z, q4.w), lv2);
        unpack2(x0, x[i], x[i + 1]);
        unpack2(x1, x[i + 2], x[i + 3]);
        if constexpr (MASK) {
            const int4 e4 = *reinterpret_cast<const int4*>(ends + i);
            x[i] = seen && key < e4.x ? x[i] : -INFINITY;
            x[i + 1] = seen && key < e4.y ? x[i + 1] : -INFINITY;
            x[i + 2] = seen && key < e4.z ? x[i + 2] : -INFINITY;
            x[i + 3] = seen && key < e4.w ? x[i + 3] : -INFINITY;
        }
    }
}

template <int N, int NC_, int BITS>
__global__ void __launch_bounds__(AttnCfg<N, NC_, BITS>::THREADS, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ AttnParams p) {
    using C = AttnCfg<N, NC_, BITS>;
    using RING = typename C::RING;
    constexpr int NC = C::NC, SLOTS = C::SLOTS, QB = C::QB, COLS = C::COLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* const sP = smem + C::OFF_P;
    uint8_t* const sQ = smem + C::OFF_Q;
    float* const sMt = (float*)(smem + C::OFF_MT);
    float* const sL = (float*)(smem + C::OFF_L);
    float* const sMw = (float*)(smem + C::OFF_MW);
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
    uint64_t* s_full = q_empty + 2;         // [2] S^T of a tile in TMEM
    uint64_t* p_full = s_full + 2;          // [4] weights and tile maxima written (and S^T read)
    uint64_t* o_full = p_full + 4;          // [2] O^T of a tile in TMEM (and the weights read)
    uint64_t* o_empty = o_full + 2;         // [2] O^T read
    uint64_t* l_full = o_empty + 2;         // sums of a segment written
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
            mbar_init(meta_empty + i, C::SPLIT ? 8 : 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, C::QWARPS);
            mbar_init(q_empty + i, 1 + 8);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, C::SPLIT ? 8 : 4);
            mbar_init(p_full + 2 + i, C::SPLIT ? 8 : 4);
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 4);
        }
        mbar_init(l_full, 8);
        mbar_init(l_empty, 4);
        mbar_init(drain, 1);
        for (int i = 0; i < C::PACKED; ++i) {
            mbar_init(pk_full + i, p.idx ? 33 : 1);  // copies of the lanes arrive by themselves
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

    if (warp < 4) {
        regs_dec<C::R_MMA>();
        if (warp == 0) {
            // ------------------------------------------------------- MMA issuer
            // The whole warp walks and waits; one lane issues.
            const bool issuer = elect_one();
            const uint32_t id_s = idesc_e4m3_f32(128, C::MN);
            const uint32_t id_o = idesc_e4m3_f32(128, C::MN) | kIdescAMn | kIdescBMn;
            const int nk = (p.D + 31) / 32;
            const uint64_t dk0 = smem_desc_kmajor(smem_u32(smem), 128);
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(smem), kASlotBytes);
            const uint64_t dq0 = smem_desc_kmajor(smem_u32(sQ), 128);
            const uint64_t dp0 = smem_desc_mn_sw128(smem_u32(sP), kASlotBytes);
            bool ok = true;
            int tc = 0, sc = 0;
            // O^T of tile t: V^T (hi + lo)
            auto second = [&](int t) {
                const int bf = t & 1, ph = (t >> 1) & 1, sl = RING::at(t, 1);
                ok = ok && mbar_wait(kv_full + sl, RING::phase(t, 1), p.wait_ns);
                ok = ok && mbar_wait(o_empty + bf, ph ^ 1, p.wait_ns);
                ok = ok && mbar_wait(p_full + (t & 3), (t >> 2) & 1, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                if (issuer) {
                    const uint64_t a = dv0 + (uint64_t)(sl * (kASlotBytes >> 4));
                    const uint64_t b = dp0 + (uint64_t)(bf * (C::P_BYTES >> 4));
                    const uint32_t d = tmem + 2 * C::MN + bf * C::MN;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // 32 keys a step
                        umma_f8(d, a + k * (32 * 128 >> 4), b + k * (32 * 128 >> 4), id_o, k > 0);
                        if (BITS == 8)
                            umma_f8(d, a + k * (32 * 128 >> 4), b + (kASlotBytes >> 4) + k * (32 * 128 >> 4), id_o, 1);
                    }
                    umma_commit(o_full + bf);
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
                    if (issuer) {
                        const uint64_t a = dk0 + (uint64_t)(sl * (kASlotBytes >> 4));
                        const uint64_t b = dq0 + (uint64_t)(qb * (C::Q_BYTES >> 4));
                        const uint32_t d = tmem + (tc & 1) * C::MN;
                        // 32 dims a step, hi then lo
                        if (nk == 4) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (BITS == 8) umma_f8(d, a + 2 * k, b + (N * 128 >> 4) + 2 * k, id_s, 1);
                        } else {
                            // (the places past D are zero: a narrower head takes fewer steps)
#pragma unroll 1
                            for (int k = 0; k < nk; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll 1
                            for (int k = 0; k < nk; ++k)
                                if (BITS == 8) umma_f8(d, a + 2 * k, b + (N * 128 >> 4) + 2 * k, id_s, 1);
                        }
                        umma_commit(s_full + (tc & 1));
                        umma_commit(kv_empty + sl);
                        if (t == wk.t1 - 1) umma_commit(q_empty + qb);
                    }
                    __syncwarp();
                    if (tc > 0) second(tc - 1);
                }
                ++sc;
            }
            if (ok && tc > 0) second(tc - 1);
            if (!__all_sync(0xffffffffu, ok)) {  // products in flight end before the memory is given up
                if (issuer) umma_commit(drain);
                mbar_wait(drain, 0, p.wait_ns);
            }
        } else if (warp <= C::QWARPS) {
            attn_queries<COLS, QB, C::QWARPS>(p, wk, x, warp - C::W_QUERY, lane);
        } else if constexpr (BITS == 4) {
            if (p.idx)
                attn_produce4<C::PACKED, C::PRODUCERS, true>(p, wk, x, warp - 1 - C::QWARPS, lane);
            else
                attn_produce4<C::PACKED, C::PRODUCERS, false>(p, wk, x, warp - 1 - C::QWARPS, lane);
        }
    } else if (warp < C::W_JOIN) {
        // -------------------------------------------------------------- softmax
        // A thread has one key of a tile and the columns [c0, c0 + NC).
        regs_inc<C::R_SOFT>();
        const int grp = (warp - C::W_SOFT) >> 2, wtid = tid & 127, wg_warp = warp & 3;
        const int c0 = C::SPLIT ? grp * NC : 0;
        const uint32_t bar_id = 1 + grp;
        float* const sW = (float*)(smem + C::OFF_W) + grp * 4 * NC;  // + parity of the group's tiles * SG * 4 * NC
        float* const sSh = (float*)(smem + C::OFF_MB) + (grp * 4 + wg_warp) * 3 * NC;  // 8 - M, of this warp alone
        float* const sBe = sSh + NC;                                                   // fade of the tile
        float* const sAl = sBe + NC;                                                   // fade of the sum
        int* const sEnd = (int*)(smem + C::OFF_END) + grp * NC;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + c0;
        bool ok = true;
        int tc = 0, sc = 0, odd = 0;
        if (p.idx) {
            if (wtid < NC) sEnd[wtid] = INT_MAX;
            named_bar_sync(bar_id, 128);
        }
        while (wk.next(p)) {
            if (wk.gr.n == 0) continue;
            const int qb = sc % QB;
            int least = INT_MAX;  // keys that every column sees
            if (!p.idx) {
                const int st0 = wk.gr.st * p.TS;
                named_bar_sync(bar_id, 128);  // the last segment's ends are read
                if (wtid < NC) {
                    const int st = attn_token(p, c0 + wtid);
                    sEnd[wtid] = st < p.TS && st0 + st < p.S ? attn_end(p, wk.gr.b, st0 + st) : 0;
                }
                least = attn_end(p, wk.gr.b, st0);
                named_bar_sync(bar_id, 128);
            }
            ok = ok && mbar_wait(q_full + qb, (sc / QB) & 1, p.wait_ns);
            const float* const qs = x.q_scale + qb * COLS + c0;
            float l[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) l[i] = 0.f;
            float mw = -INFINITY;  // running maximum of column lane (of NC), the same in the group's four warps
            for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                if (!C::SPLIT && (tc & 1) != grp) continue;
                const int bf = tc & 1, ph = (tc >> 1) & 1, ms = tc % kAMeta;
                ok = ok && mbar_wait(meta_full + ms, (tc / kAMeta) & 1, p.wait_ns);
                const float key_a = x.key_a[ms * kATile + wtid], key_lv = x.key_lv[ms * kATile + wtid];
                const float key_iv = x.key_iv[ms * kATile + wtid];
                const bool flag = x.flag[ms] != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(meta_empty + ms);
                const int key = t * kATile + wtid;
                const bool seen = key_lv != -INFINITY;
                const bool masked = flag || t * kATile + kATile > least;
                const uint64_t a2 = pack2(key_a, key_a), lv2 = pack2(key_lv, key_lv);
                // S^T of this tile is done, and with it all products issued before: those of O^T of the tile before
                // last, so its weights' buffer is free, and so are the maxima of four tiles ago (a tile's O^T waits for the
                // joining of the tile two before it)
                ok = ok && mbar_wait(s_full + bf, ph, p.wait_ns);
                tc_fence_after();
                const uint32_t s_addr = lane_addr + bf * C::MN;
                uint8_t* const prow = sP + (BITS == 8 ? bf * C::P_BYTES : 0) + wtid * 128;

                float* const sWt = sW + odd * C::SG * 4 * NC;
                odd ^= 1;
                auto one_tile = [&](auto mask_c) {
                    constexpr bool MASK = decltype(mask_c)::value;
                    float score[NC], top[NC];
                    attn_scores<MASK, NC, BITS == 8 ? 0 : COLS>(s_addr, qs, sEnd, a2, lv2, key, seen, score);
#pragma unroll
                    for (int i = 0; i < NC; ++i) top[i] = warp_max_nan(score[i]);
                    if (lane == 0) {
#pragma unroll
                        for (int i = 0; i < NC; i += 4)
                            *reinterpret_cast<float4*>(sWt + wg_warp * NC + i) =
                                make_float4(top[i], top[i + 1], top[i + 2], top[i + 3]);
                    }
                    named_bar_sync(bar_id, 128);
                    // every warp takes the tile's maxima by itself: no second barrier.  (The next tile's go to the other
                    // half of sW, and a warp reads these before it reaches the next tile's barrier.)
                    bool fade = false;
                    if (lane < NC) {
                        const float M = max_nan(max3_nan(sWt[lane], sWt[NC + lane], sWt[2 * NC + lane]), sWt[3 * NC + lane]);
                        const float mn = max_nan(mw, M);
                        fade = mn > mw && mw != -INFINITY;
                        sAl[lane] = fade ? exp2_approx(mw - mn) : 1.f;
                        sSh[lane] = M == -INFINITY ? kATop : kATop - M;
                        sBe[lane] = M == -INFINITY ? 0.f : exp2_approx(M - mn);
                        if (wg_warp == 0) sMt[(tc & 3) * N + c0 + lane] = M;
                        mw = mn;
                    }
                    __syncwarp();  // the writes above are seen by all lanes (a vote orders no memory)
                    if (__any_sync(0xffffffffu, fade)) {
#pragma unroll
                        for (int i = 0; i < NC; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sAl + i);
                            l[i] *= f.x, l[i + 1] *= f.y, l[i + 2] *= f.z, l[i + 3] *= f.w;
                        }
                    }
                    const uint64_t iv2 = seen ? pack2(key_iv, key_iv) : pack2(0.f, 0.f);
                    uint32_t hi[NC / 4], lo[NC / 4];
#pragma unroll
                    for (int i = 0; i < NC; i += 4) {
                        const float4 sh = *reinterpret_cast<const float4*>(sSh + i);
                        const float4 be = *reinterpret_cast<const float4*>(sBe + i);
                        float e0, e1, e2, e3;
                        unpack2(add2(pack2(score[i], score[i + 1]), pack2(sh.x, sh.y)), e0, e1);
                        unpack2(add2(pack2(score[i + 2], score[i + 3]), pack2(sh.z, sh.w)), e2, e3);
                        const float w0 = exp2_approx(e0), w1 = exp2_approx(e1);
                        const float w2 = exp2_approx(e2), w3 = exp2_approx(e3);
                        unpack2(fma2(mul2(pack2(w0, w1), iv2), pack2(be.x, be.y), pack2(l[i], l[i + 1])), l[i], l[i + 1]);
                        unpack2(fma2(mul2(pack2(w2, w3), iv2), pack2(be.z, be.w), pack2(l[i + 2], l[i + 3])), l[i + 2],
                                l[i + 3]);
                        uint32_t h0, l0, h1, l1;
                        split_e4m3(w0, w1, h0, l0);
                        split_e4m3(w2, w3, h1, l1);
                        hi[i / 4] = h0 | (h1 << 16);
                        lo[i / 4] = l0 | (l1 << 16);
                    }
                    // 128-byte swizzle
                    const int j = (c0 >> 4) + (BITS == 8 ? 0 : bf * (C::MN >> 4));
                    uint8_t* const ph = prow + ((j ^ (wtid & 7)) << 4);
                    if constexpr (NC == 16) {
                        uint8_t* const pl = prow + (BITS == 8 ? kASlotBytes : 0) + (((j + (BITS == 8 ? 0 : COLS >> 4)) ^ (wtid & 7)) << 4);
                        *reinterpret_cast<uint4*>(ph) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(pl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    } else {
                        *reinterpret_cast<uint4*>(ph) = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                    }
                };
                if (masked)
                    one_tile(std::true_type{});
                else
                    one_tile(std::false_type{});
                if (BITS == 8 && flag && c0 == 0) {  // (4 bits: the producers write zeros there)
                    // unseen slots may hold anything (NaN codes): a zero weight alone would not keep them out
                    const int sl = RING::at(tc, 1);
                    ok = ok && mbar_wait(kv_full + sl, RING::phase(tc, 1), p.wait_ns);
                    if (!seen && ok) {
                        uint4* vrow = reinterpret_cast<uint4*>(smem + sl * kASlotBytes + wtid * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) vrow[i] = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + (tc & 3));
            }
            // the segment's sums: lanes, then (by the joining warps) warps and groups
            ok = ok && mbar_wait(l_empty, (sc & 1) ^ 1, p.wait_ns);
            const float sum = warp_sum_columns<NC>(l, lane);
            if (lane < NC) {
                sL[(grp * 4 + wg_warp) * NC + lane] = sum;
                if (wg_warp == 0) sMw[grp * NC + lane] = mw;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(l_full);
                mbar_arrive(q_empty + qb);
            }
            ++sc;
        }
    } else if (warp < C::W_JOIN + 4) {
        // ---------------------------------------------------------------- joining
        // A thread has one output dim (TMEM lane) of every column; thread i < COLS also keeps column i's maximum.
        regs_inc<C::R_JOIN>();
        const int d = tid & 127, wg_warp = warp & 3;
        constexpr uint32_t bar_id = 1 + C::SG;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + 2 * C::MN;
        float* const sA = (float*)(smem + C::OFF_AB);  // [2][N] fade of acc
        float* const sB = sA + 2 * N;                  // [2][N] of the tile
        float* const sInv = (float*)(smem + C::OFF_INV);
        int* const sRow = (int*)(smem + C::OFF_ROW);
        bool ok = true;
        int tc = 0, sc = 0;
        AttnHeader hd{0, 0, 0, 0};
        AttnHeader* const heads = reinterpret_cast<AttnHeader*>(p.ws);
        float* const parts = (float*)(p.ws + (size_t)gridDim.x * sizeof(AttnHeader));
        while (wk.next(p)) {
            float acc[COLS];
#pragma unroll
            for (int i = 0; i < COLS; ++i) acc[i] = 0.f;
            float m = -INFINITY, l = 0.f;
            if (wk.gr.n > 0) {
                for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                    const int bf = tc & 1, ph = (tc >> 1) & 1;
                    // (four barriers: the softmax may be three tiles ahead of the joining)
                    ok = ok && mbar_wait(p_full + (tc & 3), (tc >> 2) & 1, p.wait_ns);
                    if (d < COLS) {
                        const float M = sMt[(tc & 3) * N + d], mn = max_nan(m, M);
                        sA[bf * N + d] = m == -INFINITY ? 0.f : exp2_approx(m - mn);
                        sB[bf * N + d] = M == -INFINITY ? 0.f : exp2_approx(M - mn);
                        m = mn;
                    }
                    named_bar_sync(bar_id, 128);
                    ok = ok && mbar_wait(o_full + bf, ph, p.wait_ns);
                    tc_fence_after();
                    uint32_t r[COLS];
                    if constexpr (BITS == 8) {
                        if constexpr (COLS == 32)
                            tmem_ld32(lane_addr + bf * C::MN, r);
                        else
                            tmem_ld16(lane_addr + bf * C::MN, r);
                        tmem_ld_wait();
                    } else if constexpr (COLS == 8) {
                        uint32_t both[16];
                        tmem_ld16(lane_addr + bf * C::MN, both);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(both[i]) + __uint_as_float(both[8 + i]));
                    } else {
#pragma unroll
                        for (int c = 0; c < COLS; c += 16) {
                            uint32_t h[16], l[16];
                            tmem_ld16(lane_addr + bf * C::MN + c, h);
                            tmem_ld16(lane_addr + bf * C::MN + COLS + c, l);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) r[c + i] = __float_as_uint(__uint_as_float(h[i]) + __uint_as_float(l[i]));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < COLS; i += 4) {
                        const float4 fa = *reinterpret_cast<const float4*>(sA + bf * N + i);
                        const float4 fb = *reinterpret_cast<const float4*>(sB + bf * N + i);
                        const uint64_t o0 = mul2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), pack2(fb.x, fb.y));
                        const uint64_t o1 =
                            mul2(pack2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), pack2(fb.z, fb.w));
                        unpack2(fma2(pack2(acc[i], acc[i + 1]), pack2(fa.x, fa.y), o0), acc[i], acc[i + 1]);
                        unpack2(fma2(pack2(acc[i + 2], acc[i + 3]), pack2(fa.z, fa.w), o1), acc[i + 2], acc[i + 3]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(o_empty + bf);
                }
                ok = ok && mbar_wait(l_full, sc & 1, p.wait_ns);
                if (d < COLS) {
#pragma unroll
                    for (int gi = 0; gi < C::SG; ++gi) {
                        if (C::SPLIT && gi != d / NC) continue;
                        const int col = C::SPLIT ? d % NC : d;
                        const float* s = sL + gi * 4 * NC + col;
                        const float mg = sMw[gi * NC + col];
                        if (mg != -INFINITY) l += ((s[0] + s[NC]) + (s[2 * NC] + s[3 * NC])) * exp2_approx(mg - m);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(l_empty);
                ++sc;
            }
            const bool whole = wk.t0 == 0 && wk.t1 == wk.gr.w;
            if (whole) {
                if (d < COLS) {
                    const int st = attn_token(p, d), s = wk.gr.st * p.TS + st;
                    const int row = st < p.TS && s < p.S
                                        ? (wk.gr.b * p.S + s) * p.Hq + wk.h * p.G + d - st * p.G
                                        : -1;
                    sRow[d] = row;
                    sInv[d] = l > 0.f ? 1.f / l : 0.f;
                    if (p.lse && row >= 0) p.lse[row] = attn_lse(m, l);
                }
                named_bar_sync(bar_id, 128);
                if (d < p.D) {
                    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + d;
#pragma unroll
                    for (int i = 0; i < COLS; ++i) {
                        const int row = sRow[i];
                        if (row >= 0) out[(int64_t)row * p.D] = __float2bfloat16_rn(acc[i] * sInv[i]);
                    }
                }
                named_bar_sync(bar_id, 128);
            } else {
                const int slot = 2 * c + (wk.first ? 0 : 1);
                float* part = parts + slot * attn_part_floats(N);
#pragma unroll
                for (int i = 0; i < COLS; ++i) part[i * 128 + d] = acc[i];
                if (d < COLS) {
                    part[N * 128 + d] = m;
                    part[N * 128 + N + d] = l;
                }
                if (wk.t0 == 0)  // place unit_end - 1 is in the share of the last CTA that begins at or before it
                    hd = AttnHeader{(int32_t)((wk.unit_end * nc - 1) / W), wk.g, wk.h, slot};
            }
            if (p.by_unit && wk.t0 == 0 && d == 0)
                heads[wk.g * p.Hkv + wk.h] = whole ? AttnHeader{0, 0, 0, 0} : hd;
        }
        if (!p.by_unit && d == 0) heads[c] = hd;
    } else {
        regs_dec<C::R_PROD>();
        if constexpr (BITS == 8) {
            if (p.idx)
                attn_produce<SLOTS, C::PRODUCERS, true>(p, wk, x, &tmk, &tmv, warp - C::W_PROD, lane);
            else
                attn_produce<SLOTS, C::PRODUCERS, false>(p, wk, x, &tmk, &tmv, warp - C::W_PROD, lane);
        } else {
            attn_widen<RING, C::PACKED, 2>(p, wk, x, (warp - C::W_PROD) >> 2, warp & 3, lane);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

template <int N, int NC, int BITS>
static cudaError_t attn_launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid,
                               cudaStream_t st) {
    using C = AttnCfg<N, NC, BITS>;
    auto* kernel = cache_attn_kernel<N, NC, BITS>;
    cudaError_t e = set_smem_attr((const void*)kernel, C::TOTAL);
    if (e != cudaSuccess) return e;
    kernel<<<grid, C::THREADS, C::TOTAL, st>>>(mk, mv, p);
    return cudaGetLastError();
}

}  // namespace lidx
