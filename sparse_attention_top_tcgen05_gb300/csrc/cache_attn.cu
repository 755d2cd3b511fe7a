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
// few queries there are.  The N columns are (query token, head of the group), N = 16, 32, 64 or 128.
//
// Work.  The units (sequence, tile of query tokens, kv head) have as many tiles of 128 keys as their last row
// sees.  All tiles form one line that is cut into equal shares, one a CTA, found on the device from the
// lengths.  A CTA that holds only part of a unit writes (m, l, acc) to the workspace, and cache_attn_join_kernel
// joins the parts in order.  No atomics: two calls give the same bits.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <climits>
#include <type_traits>

#include "cache.cuh"
#include "kernels.h"
#include "lidx.h"
#include "ptx.cuh"

namespace lidx {

struct AttnParams {
    const uint16_t* q;
    int64_t qs[3];
    const float* ks;
    const float* vs;
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_pos;  // nullable
    const int32_t* idx;    // nullable
    int64_t num_pages;
    int B, S, Hq, Hkv, G, D, page, max_pages, ratio, topk;
    int TS, ST;            // query tokens of a unit; units of a sequence
    int page_shift;        // page = 1 << page_shift
    uint32_t inv_g;        // ceil(2^16 / G): n / G = n * inv_g >> 16 for n < 128
    float scale_log2;      // softmax_scale * log2(e)
    uint16_t* out;
    float* lse;            // nullable
    uint8_t* ws;
    uint64_t wait_ns;
    int debug_stall;       // 1: the producer issues nothing (failure-detection tests)
};

constexpr int kATile = 128;                     // keys of a tile
constexpr int kASlotBytes = kATile * 128;       // one K or V tile: 128 bytes a key (zero past D)
constexpr int kAMeta = 5;                       // stages of per-key scales
constexpr float kATop = 8.f;                    // weights are scaled to 2^8
constexpr float kALn2 = 0.693147180559945309f;

// Shared memory of the configuration with N columns.
template <int N>
struct AttnCfg {
    // Softmax groups of four warps.  At N = 16 two groups take the tiles in turn; from N = 32 on the groups share each
    // tile's columns, 16 a group, so that a thread keeps its 16 scores and sums in registers (at N = 64 two groups of
    // 64 columns took 7.7k cycles a tile, most of it exposed latency and spills).  N = 128 has two groups of 64 columns:
    // four groups would not leave the registers that joining 128 columns takes.
    static constexpr int SG = N == 64 ? 4 : 2;
    static constexpr bool SPLIT = N > 16;
    static constexpr int NC = SPLIT ? N / SG : N;      // columns of a group
    static constexpr int QB = N == 128 ? 1 : 2;        // query buffers
    static constexpr int SLOTS = N <= 32 ? 8 : (N == 64 ? 7 : 6);
    static constexpr int Q_BYTES = 2 * N * 128;        // hi and lo
    static constexpr int P_BYTES = 2 * kASlotBytes;    // hi and lo
    static constexpr int OFF_P = SLOTS * kASlotBytes;
    static constexpr int OFF_Q = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_META = OFF_Q + QB * Q_BYTES;              // [kAMeta][128] float2
    static constexpr int OFF_FLAG = OFF_META + kAMeta * kATile * 8;    // [kAMeta] four bytes, one a producer
    static constexpr int OFF_QS = OFF_FLAG + 128;                      // [2][N] query scales
    static constexpr int OFF_W = OFF_QS + 2 * N * 4;                   // [2][SG][4][NC] warp maxima of a tile
    static constexpr int OFF_MB = OFF_W + 2 * SG * 4 * NC * 4;         // [4 SG][3][NC] of a warp: 8 - M, fades
    static constexpr int OFF_END = OFF_MB + 4 * SG * 3 * NC * 4;       // [SG][NC] keys a column sees
    static constexpr int OFF_MT = OFF_END + SG * NC * 4;               // [4][N] tile maxima
    static constexpr int OFF_AB = OFF_MT + 4 * N * 4;                  // [2][2][N] fades of acc and tile
    static constexpr int OFF_L = OFF_AB + 2 * N * 8;                   // [SG][4][NC] sums of the warps
    static constexpr int OFF_MW = OFF_L + SG * 4 * NC * 4;             // [SG][NC] their reference
    static constexpr int OFF_INV = OFF_MW + SG * NC * 4;               // [N] 1 / l
    static constexpr int OFF_ROW = OFF_INV + N * 4;                    // [N] output rows
    static constexpr int OFF_GATHER = OFF_ROW + N * 4;                 // [128] cache rows of a tile's keys
    static constexpr int OFF_BAR = OFF_GATHER + kATile * 4;
    static constexpr int NBAR = 2 * SLOTS + 2 * kAMeta + 2 * 2 + 3 * 2 + 4 + 2 + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;                // start of the share, TMEM address
    static constexpr int TOTAL = OFF_MISC + 256 + 1024;                // + alignment of the base
    static_assert(TOTAL <= 232448 && kAMeta * 4 <= 128, "shared memory");
    static_assert(OFF_QS % 16 == 0 && OFF_MB % 16 == 0 && OFF_END % 16 == 0 && OFF_AB % 16 == 0 && OFF_W % 16 == 0 &&
                      OFF_GATHER % 16 == 0,
                  "16-byte reads");
    static constexpr int TMEM = 4 * N;                                 // columns: two tiles of S and of O
    // Warpgroups: MMA and queries; SG of softmax; joining; up to N = 64 four producers (N = 128, whose joining group holds
    // 128 sums a thread, has no registers for them: one warp of the first group produces).
    static constexpr bool OWN_PROD = N < 128;
    static constexpr int THREADS = 128 * (2 + SG + (OWN_PROD ? 1 : 0));
    static constexpr int W_SOFT = 4, W_JOIN = 4 + 4 * SG;  // first warps
    static constexpr int PRODUCERS = OWN_PROD ? 4 : 1, W_PROD = OWN_PROD ? W_JOIN + 4 : 1;
    static constexpr int QWARPS = OWN_PROD ? 3 : 2, W_QUERY = OWN_PROD ? 1 : 2;
    // registers a thread of each group; their sum is at most what the launch has
    static constexpr int R_LAUNCH = 65536 / THREADS / 8 * 8;
    static constexpr int R_MMA = N == 128 ? 80 : (N == 64 ? 56 : 64), R_PROD = N == 64 ? 56 : 88, R_JOIN = N == 128 ? 160 : 104;
    static constexpr int R_SOFT = N == 128 ? 136 : (N == 64 ? 72 : 112);
    static_assert(R_MMA + SG * R_SOFT + R_JOIN + (OWN_PROD ? R_PROD : 0) <= R_LAUNCH * (THREADS / 128), "register split");
    static_assert(R_MMA < R_LAUNCH && (!OWN_PROD || R_PROD < R_LAUNCH) && R_JOIN > R_LAUNCH && R_SOFT >= R_LAUNCH,
                  "groups that give registers, groups that take them");
};

// Row (b, s) sees keys [0, end).
__device__ __forceinline__ int attn_end(const AttnParams& p, int b, int s) {
    int n = p.kv_len[b];
    const int cap = p.max_pages * p.page;
    n = n < 0 ? 0 : (n > cap ? cap : n);
    if (p.q_pos) {
        const int64_t seen = (int64_t)p.q_pos[b] + s + 1;  // below 2^32
        const uint32_t e = seen > 0 ? (uint32_t)seen / (uint32_t)p.ratio : 0;
        n = e < (uint32_t)n ? (int)e : n;
    }
    return n;
}

// ---- the line of tiles.  Group g = (sequence, tile of query tokens); its Hkv units follow each other.
struct AttnGroup {
    int b, st, limit;  // limit: keys its last row sees
    int n;             // tiles of a unit (0: nothing to see)
    int w;             // places of a unit on the line: at least one
};
__device__ __forceinline__ void attn_group_size(const AttnParams& p, AttnGroup& r) {
    if (!p.idx) r.limit = attn_end(p, r.b, min(r.st * p.TS + p.TS, p.S) - 1);  // (selected keys: the producers look)
    r.n = ((p.idx ? p.topk : r.limit) + kATile - 1) / kATile;
    r.w = max(r.n, 1);
}
__device__ __forceinline__ AttnGroup attn_group(const AttnParams& p, int g) {
    AttnGroup r;
    r.b = g / p.ST;
    r.st = g - r.b * p.ST;
    r.limit = 0;
    attn_group_size(p, r);
    return r;
}
// Query token of column n within a unit.
__device__ __forceinline__ int attn_token(const AttnParams& p, int n) { return (int)(n * p.inv_g >> 16); }
__device__ __forceinline__ int64_t attn_share(int64_t W, int c, int n) { return W * c / n; }

// The segments [t0, t1) of units that make up a CTA's share; every role walks them alike.
struct AttnWalk {
    int64_t pos, end;   // places not walked yet
    int64_t unit_end;   // place behind the segment's unit
    int g, h, t0, t1;
    AttnGroup gr;
    bool first, fresh;  // first: the segment is the CTA's first

    // pos lies in group g, whose first unit's place is base
    __device__ void begin(const AttnParams& p, int64_t pos_, int64_t end_, int g_, int64_t base) {
        pos = pos_;
        end = end_;
        g = g_;
        t1 = 0;
        fresh = true;
        if (pos >= end) return;
        gr = attn_group(p, g);
        const int64_t at = pos - base;
        h = at < INT_MAX ? (int)((uint32_t)at / (uint32_t)gr.w) : (int)(at / gr.w);
        t0 = (int)(at - (int64_t)h * gr.w);
    }
    __device__ bool next(const AttnParams& p) {
        if (pos >= end) return false;
        first = fresh;
        if (fresh) {
            fresh = false;
        } else {
            t0 = 0;
            if (++h == p.Hkv) {
                h = 0;
                ++g;
                if (++gr.st == p.ST) gr.st = 0, ++gr.b;
                attn_group_size(p, gr);
            }
        }
        unit_end = pos - t0 + gr.w;
        const int64_t e = unit_end < end ? unit_end : end;
        t1 = t0 + (int)(e - pos);
        pos = e;
        return true;
    }
};

// Workspace: a header for each CTA, then two parts for each (its first segment, its last).
struct AttnHeader {
    // last > 0: the CTA holds the first tiles (in part `slot`) of a unit that ends with CTA `last`'s first segment
    int32_t last, g, h, slot;
};
__host__ __device__ inline size_t attn_part_floats(int N) { return (size_t)N * 128 + 2 * N; }
__host__ __device__ inline size_t attn_ws_bytes(int N, int grid) {
    return (size_t)grid * sizeof(AttnHeader) + (size_t)grid * 2 * attn_part_floats(N) * 4;
}

// Two floats (at most 256 in size) -> e4m3 hi and lo pairs in the low halves.
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    uint32_t f, b, r;
    uint16_t h, l;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(f));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(h));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(f), "r"(b));  // exact
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(r));
    hi = h;
    lo = l;
}

// Sums over the warp's lanes of 32 columns: lane i returns column i's.
__device__ __forceinline__ float warp_sum_columns(float (&v)[32], int lane) {
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) {
        const bool up = lane & step;
#pragma unroll
        for (int i = 0; i < step; ++i) {
            const float send = up ? v[i] : v[i + step], keep = up ? v[i + step] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, step);
        }
    }
    return v[0];
}

// x of CH columns of this thread's key: (S^T * key's factor) * column's factor + log2(v scale); unseen -inf.
template <bool MASK, int CH>
__device__ __forceinline__ void attn_scores(uint32_t s_addr, const float* qs, const int* ends, uint64_t a2,
                                            uint64_t lv2, int key, bool seen, float (&x)[CH]) {
    uint32_t r[CH];
    if constexpr (CH == 32)
        tmem_ld32(s_addr, r);
    else
        tmem_ld16(s_addr, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < CH; i += 4) {
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
    constexpr int CH = NC < 32 ? NC : 32;  // columns of a chunk in registers
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* const sP = smem + C::OFF_P;
    uint8_t* const sQ = smem + C::OFF_Q;
    float2* const sMeta = (float2*)(smem + C::OFF_META);
    uint32_t* const sFlag = (uint32_t*)(smem + C::OFF_FLAG);  // not 0: a key of the tile is not seen
    float* const sQs = (float*)(smem + C::OFF_QS);
    float* const sMt = (float*)(smem + C::OFF_MT);
    float* const sL = (float*)(smem + C::OFF_L);
    float* const sMw = (float*)(smem + C::OFF_MW);
    uint64_t* bars = (uint64_t*)(smem + C::OFF_BAR);
    uint64_t* kv_full = bars;               // [SLOTS] K or V tile landed
    uint64_t* kv_empty = kv_full + SLOTS;   // [SLOTS] its product is done
    uint64_t* meta_full = kv_empty + SLOTS;     // [kAMeta] scales of a tile's keys written
    uint64_t* meta_empty = meta_full + kAMeta;  // [kAMeta] read by the softmax warps
    uint64_t* q_full = meta_empty + kAMeta;     // [2]
    uint64_t* q_empty = q_full + 2;             // [2]
    uint64_t* s_full = q_empty + 2;         // [2] S^T of a tile in TMEM
    uint64_t* p_full = s_full + 2;          // [4] weights and tile maxima written (and S^T read)
    uint64_t* o_full = p_full + 4;          // [2] O^T of a tile in TMEM (and the weights read)
    uint64_t* o_empty = o_full + 2;         // [2] O^T read
    uint64_t* l_full = o_empty + 2;         // sums of a segment written
    uint64_t* l_empty = l_full + 1;
    uint64_t* drain = l_empty + 1;
    int64_t* sScan = (int64_t*)(smem + C::OFF_MISC);  // [28]
    int64_t* sBase = sScan + 28;
    int* sGroup = (int*)(sBase + 1);
    uint32_t* tmem_slot = (uint32_t*)(sGroup + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(kv_full + i, p.idx ? C::PRODUCERS : 1);
            mbar_init(kv_empty + i, 1);
        }
        for (int i = 0; i < kAMeta; ++i) {
            mbar_init(meta_full + i, p.idx ? C::PRODUCERS : 1);
            mbar_init(meta_empty + i, C::SPLIT ? 4 * C::SG : 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, C::QWARPS);
            mbar_init(q_empty + i, 1 + 4 * C::SG);
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, C::SPLIT ? 4 * C::SG : 4);
            mbar_init(p_full + 2 + i, C::SPLIT ? 4 * C::SG : 4);
            mbar_init(o_full + i, 1);
            mbar_init(o_empty + i, 4);
        }
        mbar_init(l_full, 4 * C::SG);
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

    // ---- this CTA's share of the line
    const int c = blockIdx.x;
    int nc = gridDim.x;  // CTAs with a share
    int64_t W, pos0, pos1, base0 = 0;
    int g0 = 0;
    if (p.idx) {
        // every unit has the same places
        const int64_t w = (int64_t)((p.topk + kATile - 1) / kATile) * p.Hkv;
        W = w * p.B * p.ST;
        nc = W < nc ? (int)W : nc;
        pos0 = attn_share(W, min(c, nc), nc);
        pos1 = attn_share(W, min(c + 1, nc), nc);
        g0 = (int)(pos0 / w);
        base0 = g0 * w;
    } else {
        const int NG = p.B * p.ST, per = (NG + C::THREADS - 1) / C::THREADS;
        const int ga = min(tid * per, NG), gz = min(ga + per, NG);
        int64_t sum = 0;
        for (int g = ga; g < gz; ++g) sum += (int64_t)attn_group(p, g).w * p.Hkv;
        int64_t incl = sum;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, i);
            if (lane >= i) incl += o;
        }
        if (lane == 31) sScan[warp] = incl;
        __syncthreads();
        W = 0;
        int64_t before = 0;
#pragma unroll
        for (int i = 0; i < C::THREADS / 32; ++i) {
            if (i == warp) before = W;
            W += sScan[i];
        }
        nc = W < nc ? (int)W : nc;
        pos0 = attn_share(W, min(c, nc), nc);
        pos1 = attn_share(W, min(c + 1, nc), nc);
        int64_t at = before + incl - sum;
        if (pos0 >= at && pos0 < at + sum) {
            int g = ga;
            for (; g < gz; ++g) {
                const int64_t w = (int64_t)attn_group(p, g).w * p.Hkv;
                if (pos0 < at + w) break;
                at += w;
            }
            *sGroup = g;
            *sBase = at;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!p.idx && pos0 < pos1) {
        g0 = *sGroup;
        base0 = *sBase;
    }
    const uint32_t tmem = *tmem_slot;
    AttnWalk wk;
    wk.begin(p, pos0, pos1, g0, base0);

    auto produce = [&]() {
        // --------------------------------------------------------- producer
        // Three steps ahead: indices of tile i + 2, page ids of tile i + 1, scales of tile i, so that a
        // step waits for one memory latency at most.  A lane has four keys.
        bool ok = !p.debug_stall;
        struct Ref {
            bool live;
            int b, h, tile, limit;
            int64_t row;  // of topk_indices
        };
        int tile = 0;
        bool more = true;
        auto next_ref = [&]() {
            Ref r{false, 0, 0, 0, 0, 0};
            while (more && (tile >= wk.t1 || wk.gr.n == 0)) {
                more = wk.next(p);
                tile = wk.t0;
                if (more && p.idx) wk.gr.limit = attn_end(p, wk.gr.b, wk.gr.st);
            }
            if (more) r = Ref{true, wk.gr.b, wk.h, tile++, wk.gr.limit, (int64_t)wk.gr.b * p.S + wk.gr.st};
            return r;
        };
        int tc = 0;
        const int page_mask = p.page - 1;
        // waits for the slots of tile tc's K and V and its stage of scales
        auto claim = [&]() {
            const int sk = 2 * tc, ms = tc % kAMeta;
#pragma unroll
            for (int w = 0; w < 2; ++w)
                ok = ok && mbar_wait(kv_empty + (sk + w) % SLOTS, (((sk + w) / SLOTS) & 1) ^ 1, p.wait_ns);
            ok = ok && mbar_wait(meta_empty + ms, ((tc / kAMeta) & 1) ^ 1, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
        };
        const int pw = warp - C::W_PROD;  // of the producers
        if (!p.idx) {
            if (pw > 0) return;
            // Pages: the four keys of a lane share one; the lane with a page's first key loads it.
            auto page_id = [&](const Ref& r) {
                const int k0 = r.tile * kATile + 4 * lane;
                return r.live && k0 < r.limit ? p.table[(int64_t)r.b * p.max_pages + (k0 >> p.page_shift)] : -1;
            };
            Ref r0 = next_ref();
            int pid0 = page_id(r0);
            Ref r1 = next_ref();
            while (ok && r0.live) {
                const bool good = pid0 >= 0 && pid0 < p.num_pages;
                const int64_t cell = (int64_t)(good ? pid0 : 0) * p.Hkv + r0.h;
                const float a = p.ks[cell], v = p.vs[cell];
                const int pid1 = page_id(r1);
                const Ref r2 = next_ref();
                claim();
                if (!ok) break;
                const int sk = 2 * tc, ms = tc % kAMeta, s0 = sk % SLOTS, s1 = (sk + 1) % SLOTS;
                const bool lead = good && ((4 * lane) & page_mask) == 0;
                const uint32_t bytes = (128u << p.page_shift) * __popc(__ballot_sync(0xffffffffu, lead));
                if (lane == 0) {
                    mbar_arrive_expect_tx(kv_full + s0, bytes);
                    mbar_arrive_expect_tx(kv_full + s1, bytes);
                }
                __syncwarp();
                if (lead) {
                    const int row = (int)(cell << p.page_shift);
                    tma_load_2d(smem + s0 * kASlotBytes + lane * 512, &tmk, kv_full + s0, 0, row);
                    tma_load_2d(smem + s1 * kASlotBytes + lane * 512, &tmv, kv_full + s1, 0, row);
                }
                const int left = good ? r0.limit - (r0.tile * kATile + 4 * lane) : 0;  // keys of the lane that count
                const float x = a * p.scale_log2, y = __log2f(fmaxf(v, 0x1p-60f));
                float4* m4 = reinterpret_cast<float4*>(sMeta + ms * kATile + 4 * lane);
                m4[0] = make_float4(x, left > 0 ? y : -INFINITY, x, left > 1 ? y : -INFINITY);
                m4[1] = make_float4(x, left > 2 ? y : -INFINITY, x, left > 3 ? y : -INFINITY);
                const bool all = __all_sync(0xffffffffu, left > 3);
                if (lane == 0) {
                    sFlag[ms] = all ? 0 : 1;
                    mbar_arrive(meta_full + ms);
                }
                r0 = r1;
                r1 = r2;
                pid0 = pid1;
                ++tc;
            }
            if (!ok && !p.debug_stall)  // loads in flight end before the memory is given up
                for (int seq = max(0, 2 * tc - SLOTS); seq < 2 * tc; ++seq)
                    mbar_wait(kv_full + seq % SLOTS, (seq / SLOTS) & 1, p.wait_ns);
        } else {
            // Selected keys: TMA gathers of four rows.  A producer has NQ quarters of 32 keys of each tile, a lane one key of
            // each.  Unseen keys gather row 0 with the other three (or nothing); the softmax clears their V rows.
            constexpr int NQ = 4 / C::PRODUCERS;
            auto keys = [&](const Ref& r, int (&t)[NQ]) {
                const int32_t* src = p.idx + r.row * p.topk;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    const int k = r.tile * kATile + 32 * (pw + i) + lane;
                    t[i] = r.live && k < p.topk ? src[k] : -1;
                }
            };
            auto pages = [&](const Ref& r, const int (&t)[NQ], int (&pid)[NQ]) {
                const int32_t* tab = p.table + (int64_t)r.b * p.max_pages;
#pragma unroll
                for (int i = 0; i < NQ; ++i) pid[i] = t[i] >= 0 && t[i] < r.limit ? tab[t[i] >> p.page_shift] : -1;
            };
            int* const sRows = (int*)(smem + C::OFF_GATHER) + 32 * pw;
            Ref r0 = next_ref();
            int t0[NQ], t1[NQ], t2[NQ], pid0[NQ], pid1[NQ];
            keys(r0, t0);
            Ref r1 = next_ref();
            keys(r1, t1);
            pages(r0, t0, pid0);
            while (ok && r0.live) {
                float a[NQ], v[NQ];
                bool good[NQ];
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    good[i] = pid0[i] >= 0 && pid0[i] < p.num_pages;
                    const int cell = (good[i] ? pid0[i] : 0) * p.Hkv + r0.h;  // num_pages * Hkv * page < 2^31
                    a[i] = p.ks[cell];
                    v[i] = p.vs[cell];
                    sRows[32 * i + lane] = good[i] ? (cell << p.page_shift) + (t0[i] & page_mask) : -1;
                }
                pages(r1, t1, pid1);
                const Ref r2 = next_ref();
                keys(r2, t2);
                claim();
                if (!ok) break;
                __syncwarp();
                const int sk = 2 * tc, ms = tc % kAMeta, s0 = sk % SLOTS, s1 = (sk + 1) % SLOTS;
                // four keys a lane
                const int4 r = *reinterpret_cast<const int4*>(sRows + 4 * (lane & (8 * NQ - 1)));
                const bool any = lane < 8 * NQ && (r.x & r.y & r.z & r.w) >= 0;  // one of them is seen
                const uint32_t bytes = 512u * __popc(__ballot_sync(0xffffffffu, any));
                if (lane == 0) {
                    mbar_arrive_expect_tx(kv_full + s0, bytes);
                    mbar_arrive_expect_tx(kv_full + s1, bytes);
                }
                __syncwarp();
                if (any) {
                    const uint32_t to = pw * 4096 + lane * 512;
                    tma_gather4(smem + s0 * kASlotBytes + to, &tmk, kv_full + s0, 0, max(r.x, 0), max(r.y, 0),
                                max(r.z, 0), max(r.w, 0));
                    tma_gather4(smem + s1 * kASlotBytes + to, &tmv, kv_full + s1, 0, max(r.x, 0), max(r.y, 0),
                                max(r.z, 0), max(r.w, 0));
                }
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    sMeta[ms * kATile + 32 * (pw + i) + lane] =
                        good[i] ? make_float2(a[i] * p.scale_log2, __log2f(fmaxf(v[i], 0x1p-60f)))
                                : make_float2(0.f, -INFINITY);
                    const bool all = __all_sync(0xffffffffu, good[i]);
                    if (lane == 0) reinterpret_cast<uint8_t*>(sFlag + ms)[pw + i] = all ? 0 : 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(meta_full + ms);
                r0 = r1;
                r1 = r2;
#pragma unroll
                for (int i = 0; i < NQ; ++i) {
                    t0[i] = t1[i];
                    t1[i] = t2[i];
                    pid0[i] = pid1[i];
                }
                ++tc;
            }
            if (!ok && !p.debug_stall)  // loads in flight end before the memory is given up
                for (int seq = max(0, 2 * tc - SLOTS); seq < 2 * tc; ++seq)
                    mbar_wait(kv_full + seq % SLOTS, (seq / SLOTS) & 1, p.wait_ns);
        }
    };

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
                            // (with `if (k < nk)` around unrolled products the N = 128 build took wrong operands)
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
        } else if (warp >= C::W_QUERY && warp < C::W_QUERY + C::QWARPS) {
            // ------------------------------------- queries: bf16 rows -> e4m3 hi and lo
            // Eight lanes a row, 16 dims each, four rows a warp at a time.
            bool ok = true;
            int sc = 0;
            const int sub = lane & 7;
            while (wk.next(p)) {
                if (wk.gr.n == 0) continue;
                const int qb = sc % QB;
                ok = ok && mbar_wait(q_empty + qb, ((sc / QB) & 1) ^ 1, p.wait_ns);
                uint8_t* dst = sQ + qb * C::Q_BYTES;
                // the next row's loads are in flight while a row is converted
                auto load = [&](int n, uint4& u0, uint4& u1) {
                    const int st = attn_token(p, n), s = wk.gr.st * p.TS + st;
                    u0 = u1 = make_uint4(0, 0, 0, 0);
                    if (n < N && st < p.TS && s < p.S && sub * 16 < p.D) {
                        const uint4* src = reinterpret_cast<const uint4*>(
                            p.q + wk.gr.b * p.qs[0] + s * p.qs[1] + (wk.h * p.G + n - st * p.G) * p.qs[2] + sub * 16);
                        u0 = src[0];
                        u1 = src[1];
                    }
                };
                uint4 n0, n1, f0, f1;
                constexpr int step = 4 * C::QWARPS;
                const int first = (warp - C::W_QUERY) * 4 + (lane >> 3);
                load(first, n0, n1);
                load(first + step, f0, f1);
#pragma unroll 1
                for (int n = first; n < N; n += step) {
                    const uint32_t w[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
                    n0 = f0, n1 = f1;
                    load(n + 2 * step, f0, f1);
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
                    top = max(top & 0xffffu, top >> 16);
#pragma unroll
                    for (int i = 1; i < 8; i <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
                    // 2^(7 - exponent) brings the largest to [128, 256); exponents are kept where both the
                    // factor and its inverse are normal numbers
                    int ex = (int)(top >> 7);
                    ex = top == 0 ? 127 + 7 : (ex < 16 ? 16 : ex);
                    const float up = __int_as_float((254 + 7 - ex) << 23);
                    if (sub == 0) sQs[qb * N + n] = __int_as_float((ex - 7) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h0, l0, h1, l1;
                        split_e4m3(__uint_as_float(w[2 * i] << 16) * up, __uint_as_float(w[2 * i] & 0xffff0000u) * up, h0,
                                   l0);
                        split_e4m3(__uint_as_float(w[2 * i + 1] << 16) * up,
                                   __uint_as_float(w[2 * i + 1] & 0xffff0000u) * up, h1, l1);
                        hi[i] = h0 | (h1 << 16);
                        lo[i] = l0 | (l1 << 16);
                    }
                    uint8_t* at = dst + n * 128 + ((sub ^ (n & 7)) << 4);  // 128-byte swizzle
                    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(at + N * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full + qb);
                ++sc;
            }
        } else if constexpr (!C::OWN_PROD) {
            produce();
        }
    } else if (warp < C::W_JOIN) {
        // -------------------------------------------------------------- softmax
        // A thread has one key of a tile and the columns [c0, c0 + NC).
        if constexpr (C::R_SOFT > C::R_LAUNCH) regs_inc<C::R_SOFT>();
        const int grp = (warp - C::W_SOFT) >> 2, wtid = tid & 127, wg_warp = warp & 3;
        const int c0 = C::SPLIT ? grp * NC : 0;
        const uint32_t bar_id = 1 + grp;
        float* const sW = (float*)(smem + C::OFF_W) + grp * 4 * NC;  // + parity of the group's tiles * SG * 4 * NC
        float* const sSh = (float*)(smem + C::OFF_MB) + (grp * 4 + wg_warp) * 3 * NC;  // 8 - M, of this warp alone
        float* const sBe = sSh + NC;                                                   // fade of the tile
        float* const sAl = sBe + NC;                                                   // fade of the sum
        int* const sEnd = (int*)(smem + C::OFF_END) + grp * NC;
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + c0;
        constexpr int MC = (NC + 31) / 32;  // columns of a lane where a warp looks at all NC maxima
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
            const float* const qs = sQs + qb * N + c0;
            float l[NC];
#pragma unroll
            for (int i = 0; i < NC; ++i) l[i] = 0.f;
            float mw[MC];  // running maxima of columns lane, lane + 32, the same in the group's four warps
#pragma unroll
            for (int i = 0; i < MC; ++i) mw[i] = -INFINITY;
            for (int t = wk.t0; t < wk.t1; ++t, ++tc) {
                if (!C::SPLIT && (tc & 1) != grp) continue;
                const int bf = tc & 1, ph = (tc >> 1) & 1, ms = tc % kAMeta;
                ok = ok && mbar_wait(meta_full + ms, (tc / kAMeta) & 1, p.wait_ns);
                const float2 mv = sMeta[ms * kATile + wtid];
                const bool flag = sFlag[ms] != 0;
                __syncwarp();
                if (lane == 0) mbar_arrive(meta_empty + ms);
                const int key = t * kATile + wtid;
                const bool seen = mv.y != -INFINITY;
                const bool masked = flag || t * kATile + kATile > least;
                const uint64_t a2 = pack2(mv.x, mv.x), lv2 = pack2(mv.y, mv.y);
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
                    float x[CH];
#pragma unroll
                    for (int cc = 0; cc < NC; cc += CH) {
                        attn_scores<MASK, CH>(s_addr + cc, qs + cc, sEnd + cc, a2, lv2, key, seen, x);
                        float top[CH];
#pragma unroll
                        for (int i = 0; i < CH; ++i) top[i] = warp_max(x[i]);
                        if (lane == 0) {
#pragma unroll
                            for (int i = 0; i < CH; i += 4)
                                *reinterpret_cast<float4*>(sWt + wg_warp * NC + cc + i) =
                                    make_float4(top[i], top[i + 1], top[i + 2], top[i + 3]);
                        }
                    }
                    named_bar_sync(bar_id, 128);
                    // every warp takes the tile's maxima by itself: no second barrier.  (The next tile's go to the other
                    // half of sW, and a warp reads these before it reaches the next tile's barrier.)
                    bool fade = false;
#pragma unroll
                    for (int i = 0; i < MC; ++i) {
                        const int col = lane + 32 * i;
                        if (col < NC) {
                            const float M = fmaxf(fmaxf(sWt[col], sWt[NC + col]), fmaxf(sWt[2 * NC + col], sWt[3 * NC + col]));
                            const float mn = fmaxf(mw[i], M);
                            const bool f = mn > mw[i] && mw[i] != -INFINITY;
                            sAl[col] = f ? exp2_approx(mw[i] - mn) : 1.f;
                            sSh[col] = M == -INFINITY ? kATop : kATop - M;
                            sBe[col] = M == -INFINITY ? 0.f : exp2_approx(M - mn);
                            if (wg_warp == 0) sMt[(tc & 3) * N + c0 + col] = M;
                            mw[i] = mn;
                            fade = fade || f;
                        }
                    }
                    if (__any_sync(0xffffffffu, fade)) {  // (orders the writes above for the warp, too)
#pragma unroll
                        for (int i = 0; i < NC; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sAl + i);
                            l[i] *= f.x, l[i + 1] *= f.y, l[i + 2] *= f.z, l[i + 3] *= f.w;
                        }
                    }
                    const float ivs = exp2_approx(-mv.y);
                    const uint64_t iv2 = seen ? pack2(ivs, ivs) : pack2(0.f, 0.f);
#pragma unroll
                    for (int cc = 0; cc < NC; cc += CH) {
                        if constexpr (NC > CH)
                            attn_scores<MASK, CH>(s_addr + cc, qs + cc, sEnd + cc, a2, lv2, key, seen, x);
                        uint32_t hi[CH / 4], lo[CH / 4];
#pragma unroll
                        for (int i = 0; i < CH; i += 4) {
                            const float4 sh = *reinterpret_cast<const float4*>(sSh + cc + i);
                            const float4 be = *reinterpret_cast<const float4*>(sBe + cc + i);
                            float e0, e1, e2, e3;
                            unpack2(add2(pack2(x[i], x[i + 1]), pack2(sh.x, sh.y)), e0, e1);
                            unpack2(add2(pack2(x[i + 2], x[i + 3]), pack2(sh.z, sh.w)), e2, e3);
                            const float w0 = exp2_approx(e0), w1 = exp2_approx(e1);
                            const float w2 = exp2_approx(e2), w3 = exp2_approx(e3);
                            unpack2(fma2(mul2(pack2(w0, w1), iv2), pack2(be.x, be.y), pack2(l[cc + i], l[cc + i + 1])),
                                    l[cc + i], l[cc + i + 1]);
                            unpack2(fma2(mul2(pack2(w2, w3), iv2), pack2(be.z, be.w),
                                         pack2(l[cc + i + 2], l[cc + i + 3])),
                                    l[cc + i + 2], l[cc + i + 3]);
                            uint32_t h0, l0, h1, l1;
                            split_e4m3(w0, w1, h0, l0);
                            split_e4m3(w2, w3, h1, l1);
                            hi[i / 4] = h0 | (h1 << 16);
                            lo[i / 4] = l0 | (l1 << 16);
                        }
#pragma unroll
                        for (int k = 0; k < CH / 16; ++k) {
                            const int j = (((c0 + cc) >> 4) + k) ^ (wtid & 7);  // 128-byte swizzle
                            *reinterpret_cast<uint4*>(prow + (j << 4)) =
                                make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                            *reinterpret_cast<uint4*>(prow + kASlotBytes + (j << 4)) =
                                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                        }
                    }
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
#pragma unroll
            for (int cc = 0; cc < NC; cc += CH) {
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = i < CH ? l[cc + (i < CH ? i : 0)] : 0.f;
                const float sum = warp_sum_columns(v, lane);
                if (lane < CH) sL[(grp * 4 + wg_warp) * NC + cc + lane] = sum;
            }
            if (wg_warp == 0) {
#pragma unroll
                for (int i = 0; i < MC; ++i)
                    if (lane + 32 * i < NC) sMw[grp * NC + lane + 32 * i] = mw[i];
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
        constexpr int JC = N == 32 || N == 64 ? 32 : 16;  // columns read at a time
        const uint32_t lane_addr = tmem + ((uint32_t)(wg_warp * 32) << 16) + 2 * N;
        float* const sA = (float*)(smem + C::OFF_AB);  // [2][N] fade of acc
        float* const sB = sA + 2 * N;                  // [2][N] of the tile
        float* const sInv = (float*)(smem + C::OFF_INV);
        int* const sRow = (int*)(smem + C::OFF_ROW);
        bool ok = true;
        int tc = 0, sc = 0;
        AttnHeader hd{0, 0, 0, 0};
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
                        const float M = sMt[(tc & 3) * N + d], mn = fmaxf(m, M);
                        sA[bf * N + d] = m == -INFINITY ? 0.f : exp2_approx(m - mn);
                        sB[bf * N + d] = M == -INFINITY ? 0.f : exp2_approx(M - mn);
                        m = mn;
                    }
                    named_bar_sync(bar_id, 128);
                    ok = ok && mbar_wait(o_full + bf, ph, p.wait_ns);
                    tc_fence_after();
#pragma unroll
                    for (int cc = 0; cc < N; cc += JC) {
                        uint32_t r[JC];
                        if constexpr (JC == 32)
                            tmem_ld32(lane_addr + bf * N + cc, r);
                        else
                            tmem_ld16(lane_addr + bf * N + cc, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < JC; i += 4) {
                            const float4 fa = *reinterpret_cast<const float4*>(sA + bf * N + cc + i);
                            const float4 fb = *reinterpret_cast<const float4*>(sB + bf * N + cc + i);
                            const uint64_t o0 = mul2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                                     pack2(fb.x, fb.y));
                            const uint64_t o1 = mul2(pack2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])),
                                                     pack2(fb.z, fb.w));
                            unpack2(fma2(pack2(acc[cc + i], acc[cc + i + 1]), pack2(fa.x, fa.y), o0), acc[cc + i],
                                    acc[cc + i + 1]);
                            unpack2(fma2(pack2(acc[cc + i + 2], acc[cc + i + 3]), pack2(fa.z, fa.w), o1),
                                    acc[cc + i + 2], acc[cc + i + 3]);
                        }
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
                    if (p.lse && row >= 0) p.lse[row] = l > 0.f ? (m + log2f(l) - kATop) * kALn2 : -INFINITY;
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
        }
        if (d == 0) reinterpret_cast<AttnHeader*>(p.ws)[c] = hd;
    } else if constexpr (C::OWN_PROD) {
        regs_dec<C::R_PROD>();
        produce();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// Joins the parts of the units that were cut: block (c, y) takes rows y, y + gridDim.y, ... of the unit whose first
// tiles CTA c had.  The parts follow each other in the workspace (two slots a CTA).  Four groups of 128 threads take
// every fourth part and are added in order.
constexpr int kJoinThreads = 512;
constexpr int kJoinMaxParts = 1024;  // more than SMs of a device
template <int N>
__global__ void __launch_bounds__(kJoinThreads) cache_attn_join_kernel(const __grid_constant__ AttnParams p, int nc) {
    __shared__ float s_f[kJoinMaxParts], s_o[3][128], s_red[2][kJoinThreads / 32];
    grid_dependency_wait();
    const AttnHeader hd = reinterpret_cast<const AttnHeader*>(p.ws)[blockIdx.x];
    if (hd.last == 0) return;
    const float* parts = (const float*)(p.ws + (size_t)nc * sizeof(AttnHeader));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = tid & 127, quarter = tid >> 7;
    const int P = hd.last - blockIdx.x + 1, b = hd.g / p.ST, st0 = (hd.g - b * p.ST) * p.TS;
    auto part_of = [&](int i) {
        return parts + (size_t)(i == 0 ? hd.slot : 2 * (blockIdx.x + i)) * attn_part_floats(N);
    };
    for (int n = blockIdx.y; n < p.TS * p.G; n += gridDim.y) {
        const int st = attn_token(p, n), s = st0 + st;
        if (s >= p.S) break;  // uniform
        float m = -INFINITY;
        for (int i = tid; i < P; i += kJoinThreads) m = fmaxf(m, part_of(i)[N * 128 + n]);
        m = warp_max(m);
        if (lane == 0) s_red[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) m = fmaxf(m, s_red[0][i]);
        float l = 0.f;
        for (int i = tid; i < P; i += kJoinThreads) {
            const float* part = part_of(i) + N * 128 + n;
            const float f = m == -INFINITY ? 0.f : exp2_approx(part[0] - m);
            s_f[i] = f;
            l += part[N] * f;
        }
#pragma unroll
        for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
        if (lane == 0) s_red[1][warp] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) l += s_red[1][i];
        float o = 0.f;
#pragma unroll 4
        for (int i = quarter; i < P; i += 4) o += part_of(i)[n * 128 + d] * s_f[i];
        if (quarter > 0) s_o[quarter - 1][d] = o;
        __syncthreads();
        const int64_t row = ((int64_t)b * p.S + s) * p.Hq + hd.h * p.G + n - st * p.G;
        if (tid < p.D) {
            o = ((o + s_o[0][d]) + s_o[1][d]) + s_o[2][d];
            reinterpret_cast<__nv_bfloat16*>(p.out)[row * p.D + d] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
        }
        if (p.lse && tid == 0) p.lse[row] = l > 0.f ? (m + log2f(l) - kATop) * kALn2 : -INFINITY;
        __syncthreads();
    }
}

// ------------------------------------------------------------------- host

// Columns of the configuration for a call: the fewest that hold a row's group of heads and, without
// indices, as many of the sequence's query tokens as fit.
static int attn_columns(int64_t S, int G, bool selected) {
    const int64_t want = selected ? G : (S * G < 128 ? S * G : 128);
    return want <= 16 ? 16 : (want <= 32 ? 32 : (want <= 64 ? 64 : 128));
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
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    const int rows = p.TS * p.G;
    cfg.gridDim = dim3(grid, rows < 16 ? rows : 16);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    // the join is set up while the main kernel runs; it waits for its end itself
    cudaLaunchAttribute at;
    memset(&at, 0, sizeof at);
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_attn_join_kernel<N>, p, grid);
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
    if (sms <= 0 || sms > kJoinMaxParts) return LIDX_ERR_NO_DEVICE;
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
        case 64: e = attn_launch<64>(mk, mv, p, grid, st); break;
        default: e = attn_launch<128>(mk, mv, p, grid, st); break;
    }
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
