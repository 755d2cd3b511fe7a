// cache_attn.cu -- attention over a paged cache of 8-bit keys and values.
//
//     o = sum_t p_t v_t,  p = softmax over the row's keys of softmax_scale * q . k_t
// with k_t = code * scale of its page and head, v_t likewise.  One pass over the keys with the running
// maximum m and sum l of the softmax.
//
// Mathematics on the tensor cores.  A bf16 number has 8 significant bits and e4m3 has 4, so a query row,
// scaled by a power of two to at most 256, is exactly hi + lo with hi = e4m3(q), lo = e4m3(q - hi)
// (elements below 2^-10 of the row's largest keep an error of 2^-17 of it).  The cache's codes then
// go to tcgen05 kind::f8f6f4 as they are stored, without conversion, two passes for q.  The weights are held
// as hi + lo the same way (relative error 2^-8).  e4m3 spans few powers of two, so the weights of each tile
// of 128 keys are scaled to the tile's own largest, every tile's product is taken by itself, and the
// products are joined in fp32 registers with the running maximum: a key that takes nearly all the weight
// costs the tiles behind it nothing.  With x_t = log2(e) softmax_scale q.k_t + log2(v scale):
//     M = max_t x_t of the tile;  w_t = 2^(x_t - M + 8) -> hi + lo;  O = sum_t w_t code_t
//     m' = max(m, M);  acc = acc 2^(m - m') + O 2^(M - m');  l likewise with w_t / v scale;  o = acc / l.
//
// Keys are the rows of both products (S^T = K Q^T, O^T = V^T P^T): 128 keys fill the tensor core's rows however
// few queries there are.  The N columns are (query token, head of the group), N = 16 or 32; units of more rows go to
// the kernel in cache_attn_wide.cu.
//
// What bounds it: reading the cache once.  8 sequences x 65536 keys, 64 heads on 8: 165 us, 6.5 TB/s.
// One shared head does 8 x 65536 keys in 33 us with 16 query heads and 35 us with 32; one
// sequence of 1024 keys takes 10 us, which are two launches and one tile's latencies.
//
// Work.  The units (sequence, tile of query tokens, kv head) have as many tiles of 128 keys as their last row
// sees.  All tiles form one line that is cut into equal shares, one a CTA, found on the device from the
// lengths.  A CTA that holds only part of a unit writes (m, l, acc) to the workspace, and cache_attn_join_kernel
// joins the parts in order.  No atomics: two calls give the same bits.
#include <string.h>

#include "cache_attn.cuh"

namespace lidx {

constexpr int kACols = 16;  // columns of a softmax thread

// Configuration of the kernel with N columns, N = 16 or 32.
template <int N>
struct AttnCfg {
    static_assert(N == 16 || N == 32, "columns");
    // Two softmax groups of four warps, 16 columns each.  At N = 16 they take the tiles in turn, at N = 32 they share each
    // tile's columns: a thread keeps its 16 scores and sums in registers either way.
    static constexpr bool SPLIT = N == 32;
    static constexpr int SG = 2, NC = kACols, QB = 2, SLOTS = 8;
    static constexpr int Q_BYTES = 2 * N * 128;        // hi and lo
    static constexpr int P_BYTES = 2 * kASlotBytes;    // hi and lo
    static constexpr int OFF_P = SLOTS * kASlotBytes;
    static constexpr int OFF_Q = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_META = OFF_Q + QB * Q_BYTES;              // [3][kAMeta][128] of the keys
    static constexpr int OFF_SEEN = OFF_META + 3 * kAMeta * kATile * 4;  // [kAMeta][4], then [kAMeta] flags
    static constexpr int OFF_QS = OFF_SEEN + 128;                      // [QB][N] query scales
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
    static constexpr int OFF_BAR = OFF_GATHER + 4 * kATile * 4;
    static constexpr int NBAR = 2 * SLOTS + 2 * kAMeta + 2 * 2 + 3 * 2 + 4 + 2 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;                // start of the share, TMEM address
    static constexpr int TOTAL = OFF_MISC + 288 + 1024;                // + alignment of the base
    static_assert(TOTAL <= 232448 && kAMeta * 20 <= 128, "shared memory");
    static_assert(OFF_QS % 16 == 0 && OFF_MB % 16 == 0 && OFF_END % 16 == 0 && OFF_AB % 16 == 0 && OFF_W % 16 == 0 &&
                      OFF_GATHER % 16 == 0 && OFF_MISC % 8 == 0,
                  "16-byte reads");
    static constexpr int TMEM = 4 * N;                                 // columns: two tiles of S and of O
    // Warpgroups: MMA and queries; two of softmax; joining; producers.
    static constexpr int THREADS = 640, PRODUCERS = 4, QWARPS = 3;
    static constexpr int W_QUERY = 1, W_SOFT = 4, W_JOIN = 12, W_PROD = 16;  // first warps
    // registers a thread of each group: their sum is at most what the launch has
    static constexpr int R_LAUNCH = 96, R_MMA = 64, R_SOFT = 112, R_JOIN = 104, R_PROD = 88;
    static_assert(R_LAUNCH == 65536 / THREADS / 8 * 8 && R_MMA + SG * R_SOFT + R_JOIN + R_PROD <= R_LAUNCH * 5,
                  "register split");
    static_assert(R_MMA <= R_LAUNCH && R_PROD <= R_LAUNCH && R_SOFT >= R_LAUNCH && R_JOIN >= R_LAUNCH, "directions");
};

// Sums over the warp's lanes of 16 columns: lanes i and i + 16 return column i's.
__device__ __forceinline__ float warp_sum_columns(float (&v)[kACols], int lane) {
#pragma unroll
    for (int i = 0; i < kACols; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
#pragma unroll
    for (int step = 8; step > 0; step >>= 1) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float send = up ? v[i] : v[i + step], keep = up ? v[i + step] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
        }
    }
    return v[0];
}

// x of the columns of this thread's key: (S^T * key's factor) * column's factor + log2(v scale); unseen -inf.
template <bool MASK>
__device__ __forceinline__ void attn_scores(uint32_t s_addr, const float* qs, const int* ends, uint64_t a2,
                                            uint64_t lv2, int key, bool seen, float (&x)[kACols]) {
    uint32_t r[kACols];
    tmem_ld16(s_addr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < kACols; i += 4) {
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

template <int N>
__global__ void __launch_bounds__(AttnCfg<N>::THREADS, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                      const __grid_constant__ AttnParams p) {
    using C = AttnCfg<N>;
    constexpr int NC = C::NC, SLOTS = C::SLOTS, QB = C::QB;
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
    uint32_t* tmem_slot = (uint32_t*)(smem + C::OFF_MISC);
    int64_t* const scan = (int64_t*)(smem + C::OFF_MISC + 8);  // [34]

    // the warp's number by a shuffle: known to be uniform, so a role's counters and descriptors live in uniform registers
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(kv_full + i, 1);
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
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
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
            const uint32_t id_s = idesc_e4m3_f32(128, N);
            const uint32_t id_o = idesc_e4m3_f32(128, N) | kIdescAMn | kIdescBMn;
            const int nk = (p.D + 31) / 32;
            const uint64_t dk0 = smem_desc_kmajor(smem_u32(smem), 128);
            const uint64_t dv0 = smem_desc_mn_sw128(smem_u32(smem), kASlotBytes);
            const uint64_t dq0 = smem_desc_kmajor(smem_u32(sQ), 128);
            const uint64_t dp0 = smem_desc_mn_sw128(smem_u32(sP), kASlotBytes);
            bool ok = true;
            int tc = 0, sc = 0;
            // O^T of tile t: V^T (hi + lo)
            auto second = [&](int t) {
                const int bf = t & 1, ph = (t >> 1) & 1, seq = 2 * t + 1, sl = seq % SLOTS;
                ok = ok && mbar_wait(kv_full + sl, (seq / SLOTS) & 1, p.wait_ns);
                ok = ok && mbar_wait(o_empty + bf, ph ^ 1, p.wait_ns);
                ok = ok && mbar_wait(p_full + (t & 3), (t >> 2) & 1, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                tc_fence_after();
                if (issuer) {
                    const uint64_t a = dv0 + (uint64_t)(sl * (kASlotBytes >> 4));
                    const uint64_t b = dp0 + (uint64_t)(bf * (C::P_BYTES >> 4));
                    const uint32_t d = tmem + 2 * N + bf * N;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // 32 keys a step
                        umma_f8(d, a + k * (32 * 128 >> 4), b + k * (32 * 128 >> 4), id_o, k > 0);
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
                    const int seq = 2 * tc, sl = seq % SLOTS;
                    ok = mbar_wait(kv_full + sl, (seq / SLOTS) & 1, p.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (issuer) {
                        const uint64_t a = dk0 + (uint64_t)(sl * (kASlotBytes >> 4));
                        const uint64_t b = dq0 + (uint64_t)(qb * (C::Q_BYTES >> 4));
                        const uint32_t d = tmem + (tc & 1) * N;
                        // 32 dims a step, hi then lo
                        if (nk == 4) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll
                            for (int k = 0; k < 4; ++k) umma_f8(d, a + 2 * k, b + (N * 128 >> 4) + 2 * k, id_s, 1);
                        } else {
                            // (the places past D are zero: a narrower head takes fewer steps)
#pragma unroll 1
                            for (int k = 0; k < nk; ++k) umma_f8(d, a + 2 * k, b + 2 * k, id_s, k > 0);
#pragma unroll 1
                            for (int k = 0; k < nk; ++k) umma_f8(d, a + 2 * k, b + (N * 128 >> 4) + 2 * k, id_s, 1);
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
        } else {
            attn_queries<N, QB, C::QWARPS>(p, wk, x, warp - C::W_QUERY, lane);
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
            const float* const qs = x.q_scale + qb * N + c0;
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
                const uint32_t s_addr = lane_addr + bf * N;
                uint8_t* const prow = sP + bf * C::P_BYTES + wtid * 128;

                float* const sWt = sW + odd * C::SG * 4 * NC;
                odd ^= 1;
                auto one_tile = [&](auto mask_c) {
                    constexpr bool MASK = decltype(mask_c)::value;
                    float score[NC], top[NC];
                    attn_scores<MASK>(s_addr, qs, sEnd, a2, lv2, key, seen, score);
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
                    const int j = (c0 >> 4) ^ (wtid & 7);  // 128-byte swizzle
                    *reinterpret_cast<uint4*>(prow + (j << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(prow + kASlotBytes + (j << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                };
                if (masked)
                    one_tile(std::true_type{});
                else
                    one_tile(std::false_type{});
                if (flag && c0 == 0) {
                    // unseen slots may hold anything (NaN codes): a zero weight alone would not keep them out
                    const int seq = 2 * tc + 1, sl = seq % SLOTS;
                    ok = ok && mbar_wait(kv_full + sl, (seq / SLOTS) & 1, p.wait_ns);
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
            const float sum = warp_sum_columns(l, lane);
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
        // A thread has one output dim (TMEM lane) of every column; thread i < N also keeps column i's maximum.
        regs_inc<C::R_JOIN>();
        const int d = tid & 127, wg_warp = warp & 3;
        constexpr uint32_t bar_id = 1 + C::SG;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + 2 * N;
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
            float acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = 0.f;
            float m = -INFINITY, l = 0.f;
            if (wk.gr.n > 0) {
                for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                    const int bf = tc & 1, ph = (tc >> 1) & 1;
                    // (four barriers: the softmax may be three tiles ahead of the joining)
                    ok = ok && mbar_wait(p_full + (tc & 3), (tc >> 2) & 1, p.wait_ns);
                    if (d < N) {
                        const float M = sMt[(tc & 3) * N + d], mn = max_nan(m, M);
                        sA[bf * N + d] = m == -INFINITY ? 0.f : exp2_approx(m - mn);
                        sB[bf * N + d] = M == -INFINITY ? 0.f : exp2_approx(M - mn);
                        m = mn;
                    }
                    named_bar_sync(bar_id, 128);
                    ok = ok && mbar_wait(o_full + bf, ph, p.wait_ns);
                    tc_fence_after();
                    uint32_t r[N];
                    if constexpr (N == 32)
                        tmem_ld32(lane_addr + bf * N, r);
                    else
                        tmem_ld16(lane_addr + bf * N, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
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
                if (d < N) {
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
                if (d < N) {
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
                    for (int i = 0; i < N; ++i) {
                        const int row = sRow[i];
                        if (row >= 0) out[(int64_t)row * p.D] = __float2bfloat16_rn(acc[i] * sInv[i]);
                    }
                }
                named_bar_sync(bar_id, 128);
            } else {
                const int slot = 2 * c + (wk.first ? 0 : 1);
                float* part = parts + slot * attn_part_floats(N);
#pragma unroll
                for (int i = 0; i < N; ++i) part[i * 128 + d] = acc[i];
                if (d < N) {
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
        if (p.idx)
            attn_produce<SLOTS, C::PRODUCERS, true>(p, wk, x, &tmk, &tmv, warp - C::W_PROD, lane);
        else
            attn_produce<SLOTS, C::PRODUCERS, false>(p, wk, x, &tmk, &tmv, warp - C::W_PROD, lane);
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// Joins the parts of the units that were cut, block (x, y) rows of the unit of header x.  The parts follow each other in the
// workspace (two slots a CTA).  W warps share a row, each takes every W-th part with a running maximum, a lane four
// dims; eight parts are loaded at a time, and the warps' results are added in order.
// Its bytes are few (two parts a CTA): its time is its launch, two dependent reads and the start of its blocks.
constexpr int kJoinWarps = 16;
constexpr int kJoinBatch = 8;
template <int N>
__global__ void __launch_bounds__(kJoinWarps * 32, 1) cache_attn_join_kernel(const __grid_constant__ AttnParams p, int nc,
                                                                          int W) {
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ float4 s_o[kJoinWarps][32];
    grid_dependency_wait();
    const AttnHeader hd = reinterpret_cast<const AttnHeader*>(p.ws)[blockIdx.x];
    if (hd.last == 0) return;
    const float* parts = (const float*)(p.ws + (size_t)nc * sizeof(AttnHeader));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp & (W - 1);
    const int c0 = hd.slot >> 1, P = hd.last - c0 + 1, b = hd.g / p.ST, st0 = (hd.g - b * p.ST) * p.TS;
    const int rows = min(p.TS, p.S - st0) * p.G, n = (blockIdx.y * kJoinWarps + warp) / W;
    const bool some = 4 * lane < p.D;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto take = [&](float pm, float pl, const float4& po, float top) {
        const float f = pm == -INFINITY ? 0.f : exp2_approx(pm - top);
        l += pl * f;
        o.x += po.x * f, o.y += po.y * f, o.z += po.z * f, o.w += po.w * f;
    };
    auto fade = [&](float top) {
        const float f = m == -INFINITY ? 0.f : exp2_approx(m - top);
        l *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
        m = top;
    };
    if (n < rows)
        for (int i0 = sub; i0 < P; i0 += kJoinBatch * W) {
            float pm[kJoinBatch], pl[kJoinBatch], top = m;
            float4 po[kJoinBatch];
#pragma unroll
            for (int j = 0; j < kJoinBatch; ++j) {
                const int i = i0 + j * W, k = i < P ? i : i0;
                const float* part = parts + (size_t)(k == 0 ? hd.slot : 2 * (c0 + k)) * attn_part_floats(N);
                pm[j] = i < P ? part[N * 128 + n] : -INFINITY;
                pl[j] = part[N * 128 + N + n];
                po[j] = some ? reinterpret_cast<const float4*>(part + n * 128)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                top = fmaxf(top, pm[j]);
            }
            fade(top);
#pragma unroll
            for (int j = 0; j < kJoinBatch; ++j) take(pm[j], pl[j], po[j], top);
        }
    if (W > 1) {
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
        s_o[warp][lane] = o;
        __syncthreads();
        if (sub > 0) return;
        for (int i = 1; i < W; ++i) {
            const float pm = s_m[warp + i], top = fmaxf(m, pm);
            fade(top);
            take(pm, s_l[warp + i], s_o[warp + i][lane], top);
        }
    }
    if (n >= rows) return;
    const int st = attn_token(p, n);
    const int64_t row = ((int64_t)b * p.S + st0 + st) * p.Hq + hd.h * p.G + n - st * p.G;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    if (some) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        reinterpret_cast<uint2*>(p.out + row * p.D)[lane] =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    if (p.lse && lane == 0) p.lse[row] = attn_lse(m, l);
}

// ------------------------------------------------------------------- host

// Columns of the configuration for a call: the fewest that hold a row's group of heads and, without
// indices, as many of the sequence's query tokens as fit.  8 x 65536 keys of one head: 32 rows take 36 us with keys as
// the products' rows and 41 us in the wide kernel; 64 rows took 64 us and 55 us when both had them (43 us now).
static int attn_columns(int64_t S, int G, bool selected) {
    const int64_t want = selected ? G : (S * G < 128 ? S * G : 128);
    return want <= 16 ? 16 : (want <= 32 ? 32 : 128);
}

static int attn_cache_map(CUtensorMap* m, const void* cache, int64_t rows, int D, int box_rows) {
    const cuuint64_t dim[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t str[1] = {(cuuint64_t)D};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void*)cache, dim, str, box, es,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int N>
static cudaError_t attn_launch(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid,
                               cudaStream_t st) {
    cudaError_t e = set_smem_attr((const void*)cache_attn_kernel<N>, AttnCfg<N>::TOTAL);
    if (e != cudaSuccess) return e;
    cache_attn_kernel<N><<<grid, AttnCfg<N>::THREADS, AttnCfg<N>::TOTAL, st>>>(mk, mv, p);
    return cudaGetLastError();
}

template <int N>
static cudaError_t attn_join(const AttnParams& p, int grid, cudaStream_t st) {
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    // Warps a row: eight parts each, by the parts that a unit has on average.  A header's blocks that find no cut unit
    // cost 1.5 ns each, so a block takes as many rows as that leaves it warps for.
    const int rows = p.TS * p.G, units = p.by_unit ? p.B * p.ST * p.Hkv : grid;
    int W = 1;
    while (W < kJoinWarps && W * kJoinBatch < grid / units + 2) W *= 2;
    cfg.gridDim = dim3(units, (rows * W + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    // the join is set up while the main kernel runs; it waits for its end itself
    cudaLaunchAttribute at;
    memset(&at, 0, sizeof at);
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<N>, p, grid, W);
}

LIDX_STATUS_READER(status_cache_attn)

}  // namespace lidx

using namespace lidx;

extern "C" {

size_t lidx_cache_attn_workspace_bytes(int64_t B, int64_t S, int Hq, int Hkv, int D, int topk) {
    (void)B, (void)D;
    if (S < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv || Hq / Hkv > 128) return 0;
    int sms = sm103_sms();
    if (sms <= 0) sms = 256;  // no device: an upper bound
    return attn_ws_bytes(attn_columns(S, Hq / Hkv, topk > 0), sms);
}

int lidx_cache_attn(const void* q, const int64_t* qs, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    const int32_t* kv_len, const int32_t* q_pos, const int32_t* topk_indices,
                    int64_t B, int64_t S, int Hq, int Hkv, int D, int page, int64_t max_pages,
                    int64_t num_pages, int compress_ratio, int topk, float softmax_scale, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !qs || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_len || !out)
        return LIDX_ERR_NULL;
    const int rc = check_cache(B, S, Hkv, D, page, max_pages, num_pages);
    if (rc) return rc;
    if (Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || B * S > INT_MAX || B * S * Hq > INT_MAX) return LIDX_ERR_SHAPE;
    if (compress_ratio < 1 || !isfinite(softmax_scale) || (topk_indices && (topk < 1 || topk > (1 << 20))))
        return LIDX_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15u) return LIDX_ERR_ALIGN;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale | (uintptr_t)block_table | (uintptr_t)kv_len |
         (uintptr_t)q_pos | (uintptr_t)topk_indices | (uintptr_t)lse) & 3u)
        return LIDX_ERR_ALIGN;
    if ((qs[0] | qs[1] | qs[2]) & 7) return LIDX_ERR_ALIGN;
    const int sms = sm103_sms();
    if (sms <= 0) return LIDX_ERR_NO_DEVICE;
    AttnParams p;
    memset(&p, 0, sizeof p);
    p.q = (const uint16_t*)q;
    for (int i = 0; i < 3; ++i) p.qs[i] = qs[i];
    p.ks = k_scale;
    p.vs = v_scale;
    p.table = block_table;
    p.kv_len = kv_len;
    p.q_pos = q_pos;
    p.idx = topk_indices;
    p.num_pages = num_pages;
    p.B = (int)B;
    p.S = (int)S;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.D = D;
    p.page = page;
    p.max_pages = (int)max_pages;
    p.ratio = compress_ratio;
    p.topk = topk;
    const int N = attn_columns(S, p.G, topk_indices != nullptr);
    p.TS = topk_indices ? 1 : (int)(N / p.G < S ? N / p.G : S);
    p.ST = (int)((S + p.TS - 1) / p.TS);
    p.page_shift = page == 16 ? 4 : (page == 32 ? 5 : (page == 64 ? 6 : 7));
    p.inv_g = (65536 + p.G - 1) / p.G;
    p.scale_log2 = softmax_scale * 1.44269504088896341f;
    p.out = (uint16_t*)out;
    p.lse = lse;
    p.wait_ns = wait_limit_ns();
    p.debug_stall = debug_stall();
    // no more CTAs than the line can have places
    const int64_t tiles = topk_indices ? (topk + kATile - 1) / kATile : (max_pages * page + kATile - 1) / kATile;
    const int64_t most = tiles * B * p.ST * Hkv;
    const int grid = most < sms ? (int)most : sms;
    p.by_unit = B * p.ST * Hkv <= grid;
    const size_t need = attn_ws_bytes(N, grid);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)) return LIDX_ERR_WORKSPACE;
    p.ws = (uint8_t*)workspace;
    CUtensorMap mk, mv;
    const int box = topk_indices ? 1 : page;  // rows of a copy
    if (attn_cache_map(&mk, k_cache, num_pages * Hkv * page, D, box) ||
        attn_cache_map(&mv, v_cache, num_pages * Hkv * page, D, box))
        return LIDX_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    switch (N) {
        case 16: e = attn_launch<16>(mk, mv, p, grid, st); break;
        case 32: e = attn_launch<32>(mk, mv, p, grid, st); break;
        default: e = attn_launch_wide(mk, mv, p, grid, st); break;
    }
    if (e == cudaSuccess && grid > 1) switch (N) {
            case 16: e = attn_join<16>(p, grid, st); break;
            case 32: e = attn_join<32>(p, grid, st); break;
            default: e = attn_join<128>(p, grid, st); break;
        }
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
