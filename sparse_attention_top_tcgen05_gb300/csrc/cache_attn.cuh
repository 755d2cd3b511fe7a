// cache_attn.cuh -- what the two kernels of the attention over the paged 8-bit cache share (see cache_attn.cu):
// parameters, the line of tiles and its shares, the producer of keys and values and the conversion of queries.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

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
    int by_unit;           // not more units than CTAs: headers belong to units, not to CTAs
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
constexpr int kAMeta = 6;                       // stages of per-key scales
constexpr float kATop = 8.f;                    // weights are scaled to 2^8
constexpr float kALn2 = 0.693147180559945309f;
// Smallest value scale.  A row's sum adds weights of at most 2^8.3 divided by their value scales: 2^30 keys of this one stay
// below 2^119.  At the other end, 2^100, the largest weight is 2^-92 there, and fp32 has 2^34 normal steps below it.
constexpr float kAMinScale = 0x1p-80f;

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

// Workspace: a header for each unit or CTA, then two parts for each CTA (its first segment, its last).
struct AttnHeader {
    // last > 0: a unit's first tiles are in part `slot`, of CTA slot / 2, and it ends with CTA `last`'s first segment
    int32_t last, g, h, slot;
};
__host__ __device__ inline size_t attn_part_floats(int N) { return (size_t)N * 128 + 2 * N; }
__host__ __device__ inline size_t attn_ws_bytes(int N, int grid) {
    return (size_t)grid * sizeof(AttnHeader) + (size_t)grid * 2 * attn_part_floats(N) * 4;
}

// log of the sum of exp(score) from a row's maximum and sum.  The largest key adds 2^8 / (its value scale), so only a row
// without keys has a sum of zero.  A NaN score makes its row's maximum and sum NaN.
__device__ __forceinline__ float attn_lse(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l) - kATop) * kALn2;
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


// One pipeline of a CTA in shared memory.
struct AttnPipe {
    uint8_t* kv;            // [SLOTS] K or V tiles, in turn
    uint8_t* q;             // [QB] query rows: hi, lo
    float* q_scale;         // [QB][N]
    float* key_a;           // [kAMeta][128] key scale * softmax_scale * log2(e)
    float* key_lv;          // [kAMeta][128] log2 of the value scale; -inf: the key is not seen
    float* key_iv;          // [kAMeta][128] its inverse
    uint32_t* seen;         // [kAMeta][4] bits of the keys that are seen
    uint32_t* flag;         // [kAMeta] not 0: a key of the tile is not seen
    int* rows;              // [PRODUCERS][128] cache rows of gathered keys
    uint64_t *kv_full;      // [SLOTS] K or V tile landed
    uint64_t *kv_empty;     // [SLOTS] its product is done
    uint64_t *meta_full;    // [kAMeta] what belongs to a tile's keys is written
    uint64_t *meta_empty;   // [kAMeta] and read
    uint64_t *q_full, *q_empty;  // [QB]
};

// This CTA's share of the line.  All THREADS threads call it; scan: 34 words of 64 bits.  Returns the number of CTAs
// that have a share; total: places of the line.
template <int THREADS>
__device__ __forceinline__ int attn_begin(const AttnParams& p, AttnWalk& wk, int64_t& total, int64_t* scan) {
    int64_t* const sScan = scan;
    int64_t* const sBase = scan + 32;
    int* const sGroup = (int*)(scan + 33);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    static_assert(THREADS / 32 <= 32, "scan");
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
        const int NG = p.B * p.ST, per = (NG + THREADS - 1) / THREADS;
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
        for (int i = 0; i < THREADS / 32; ++i) {
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
    __syncthreads();
    if (!p.idx && pos0 < pos1) {
        g0 = *sGroup;
        base0 = *sBase;
    }
    wk.begin(p, pos0, pos1, g0, base0);
    total = W;
    return nc;
}

// Loads keys and values: warp pw of PRODUCERS.  The warps take the tiles in turn: the lookups of several tiles are then in
// flight at once, and no tile's keys wait for the slot of an earlier tile's values.  (With one warp for all pages, 8
// sequences x 65536 keys took 178 us instead of 169, in pages of 16 tokens 228 us instead of 169.)
template <int SLOTS, int PRODUCERS, bool SEL>
__device__ __forceinline__ void attn_produce(const AttnParams& p, AttnWalk& wk, const AttnPipe& x, const CUtensorMap* tmk,
                                             const CUtensorMap* tmv, int pw, int lane) {
    static_assert(SLOTS <= 2 * PRODUCERS, "a warp's tile before has been used when its next one is loaded");
    // Three steps ahead: indices of the warp's tile after next, page ids of its next tile, scales of this one, so that a
    // step waits for one memory latency at most.
    bool ok = !p.debug_stall;
    int last_k = -1, last_v = -1;  // tiles of the last loads
    struct Ref {
        bool live;
        int b, h, tile, limit;
        int tc;       // tiles of the CTA before it
        int64_t row;  // of topk_indices
    };
    int tile = 0, count = 0;
    bool more = true;
    auto next_ref = [&]() {
        Ref r{false, 0, 0, 0, 0, 0, 0};
        while (more) {
            if (tile >= wk.t1 || wk.gr.n == 0) {
                more = wk.next(p);
                tile = wk.t0;
                continue;
            }
            // on to the first tile of this segment that is the warp's
            const int skip = (pw - count % PRODUCERS + PRODUCERS) % PRODUCERS, left = wk.t1 - tile;
            if (skip >= left) {
                count += left;
                tile = wk.t1;
                continue;
            }
            count += skip;
            tile += skip;
            const int limit = SEL ? attn_end(p, wk.gr.b, wk.gr.st) : wk.gr.limit;
            r = Ref{true, wk.gr.b, wk.h, tile, limit, count, (int64_t)wk.gr.b * p.S + wk.gr.st};
            ++count;
            ++tile;
            break;
        }
        return r;
    };
    const int page_mask = p.page - 1;
    // waits for the slot of tile tc's K (which = 0) or V
    auto claim = [&](int tc, int which) {
        const int seq = 2 * tc + which;
        ok = ok && mbar_wait(x.kv_empty + seq % SLOTS, ((seq / SLOTS) & 1) ^ 1, p.wait_ns);
        if (which == 0) ok = ok && mbar_wait(x.meta_empty + tc % kAMeta, ((tc / kAMeta) & 1) ^ 1, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
    };
    if constexpr (!SEL) {
        // Pages: a lane has four keys, which share one; the lane with a page's first key loads it.
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
            const int tc = r0.tc, sk = 2 * tc, ms = tc % kAMeta, s0 = sk % SLOTS, s1 = (sk + 1) % SLOTS;
            const bool lead = good && ((4 * lane) & page_mask) == 0;
            const uint32_t bytes = (128u << p.page_shift) * __popc(__ballot_sync(0xffffffffu, lead));
            const int row = (int)(cell << p.page_shift);
            claim(tc, 0);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(x.kv_full + s0, bytes);
            __syncwarp();
            if (lead) tma_load_2d(x.kv + s0 * kASlotBytes + lane * 512, tmk, x.kv_full + s0, 0, row);
            last_k = tc;
            const int left = good ? r0.limit - (r0.tile * kATile + 4 * lane) : 0;  // keys of the lane that count
            const float f = a * p.scale_log2, y = __log2f(fmaxf(v, kAMinScale)), iv = exp2_approx(-y);
            const float none = -INFINITY;
            const int at = ms * kATile + 4 * lane;
            *reinterpret_cast<float4*>(x.key_a + at) = make_float4(f, f, f, f);
            *reinterpret_cast<float4*>(x.key_lv + at) = make_float4(left > 0 ? y : none, left > 1 ? y : none,
                                                                    left > 2 ? y : none, left > 3 ? y : none);
            *reinterpret_cast<float4*>(x.key_iv + at) = make_float4(iv, iv, iv, iv);
            uint32_t seen = (left > 3 ? 15u : (left > 0 ? (1u << left) - 1 : 0u)) << (4 * (lane & 7));
#pragma unroll
            for (int i = 1; i < 8; i <<= 1) seen |= __shfl_xor_sync(0xffffffffu, seen, i);
            if ((lane & 7) == 0) x.seen[ms * 4 + (lane >> 3)] = seen;
            const bool all = __all_sync(0xffffffffu, left > 3);
            if (lane == 0) x.flag[ms] = all ? 0 : 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(x.meta_full + ms);
            claim(tc, 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(x.kv_full + s1, bytes);
            __syncwarp();
            if (lead) tma_load_2d(x.kv + s1 * kASlotBytes + lane * 512, tmv, x.kv_full + s1, 0, row);
            last_v = tc;
            r0 = r1;
            r1 = r2;
            pid0 = pid1;
        }
    } else {
        // Selected keys: TMA gathers of four rows.  A lane has a key of each quarter of the tile.  Unseen keys gather row 0
        // with the other three (or nothing); the softmax clears their V rows.
        auto keys = [&](const Ref& r, int (&t)[4]) {
            const int32_t* src = p.idx + r.row * p.topk;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = r.tile * kATile + 32 * i + lane;
                t[i] = r.live && k < p.topk ? src[k] : -1;
            }
        };
        auto pages = [&](const Ref& r, const int (&t)[4], int (&pid)[4]) {
            const int32_t* tab = p.table + (int64_t)r.b * p.max_pages;
#pragma unroll
            for (int i = 0; i < 4; ++i) pid[i] = t[i] >= 0 && t[i] < r.limit ? tab[t[i] >> p.page_shift] : -1;
        };
        int* const sRows = x.rows + kATile * pw;
        Ref r0 = next_ref();
        int t0[4], t1[4], t2[4], pid0[4], pid1[4];
        keys(r0, t0);
        Ref r1 = next_ref();
        keys(r1, t1);
        pages(r0, t0, pid0);
        while (ok && r0.live) {
            float a[4], v[4];
            bool good[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                good[i] = pid0[i] >= 0 && pid0[i] < p.num_pages;
                const int cell = (good[i] ? pid0[i] : 0) * p.Hkv + r0.h;  // num_pages * Hkv * page < 2^31
                a[i] = p.ks[cell];
                v[i] = p.vs[cell];
                sRows[32 * i + lane] = good[i] ? (cell << p.page_shift) + (t0[i] & page_mask) : -1;
            }
            pages(r1, t1, pid1);
            const Ref r2 = next_ref();
            keys(r2, t2);
            __syncwarp();
            const int tc = r0.tc, sk = 2 * tc, ms = tc % kAMeta, s0 = sk % SLOTS, s1 = (sk + 1) % SLOTS;
            // four keys a lane
            const int4 r = *reinterpret_cast<const int4*>(sRows + 4 * lane);
            const bool any = (r.x & r.y & r.z & r.w) >= 0;  // one of them is seen
            const uint32_t bytes = 512u * __popc(__ballot_sync(0xffffffffu, any));
            const int y0 = max(r.x, 0), y1 = max(r.y, 0), y2 = max(r.z, 0), y3 = max(r.w, 0);
            claim(tc, 0);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(x.kv_full + s0, bytes);
            __syncwarp();
            if (any) tma_gather4(x.kv + s0 * kASlotBytes + lane * 512, tmk, x.kv_full + s0, 0, y0, y1, y2, y3);
            last_k = tc;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = ms * kATile + 32 * i + lane;
                const float y = __log2f(fmaxf(v[i], kAMinScale));
                x.key_a[at] = good[i] ? a[i] * p.scale_log2 : 0.f;
                x.key_lv[at] = good[i] ? y : -INFINITY;
                x.key_iv[at] = exp2_approx(-y);
                const uint32_t seen = __ballot_sync(0xffffffffu, good[i]);
                if (lane == 0) {
                    x.seen[ms * 4 + i] = seen;
                    reinterpret_cast<uint8_t*>(x.flag + ms)[i] = seen == 0xffffffffu ? 0 : 1;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(x.meta_full + ms);
            claim(tc, 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(x.kv_full + s1, bytes);
            __syncwarp();
            if (any) tma_gather4(x.kv + s1 * kASlotBytes + lane * 512, tmv, x.kv_full + s1, 0, y0, y1, y2, y3);
            last_v = tc;
            r0 = r1;
            r1 = r2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                t0[i] = t1[i];
                t1[i] = t2[i];
                pid0[i] = pid1[i];
            }
        }
    }
    if (!ok) {  // loads in flight end before the memory is given up
        const int sk = 2 * last_k, sv = 2 * last_v + 1;
        if (last_k >= 0) mbar_wait(x.kv_full + sk % SLOTS, (sk / SLOTS) & 1, p.wait_ns);
        if (last_v >= 0) mbar_wait(x.kv_full + sv % SLOTS, (sv / SLOTS) & 1, p.wait_ns);
    }
}

// Query rows of a unit, bf16 -> e4m3 hi and lo: one of QWARPS warps.  twice: rows 0 .. 63 are repeated as 64 .. 127.
template <int N, int QB, int QWARPS>
__device__ __forceinline__ void attn_queries(const AttnParams& p, AttnWalk& wk, const AttnPipe& x, int qw, int lane,
                                             bool twice = false) {
    // Eight lanes a row, 16 dims each, four rows a warp at a time.
    bool ok = true;
    int sc = 0;
    const int sub = lane & 7;
    while (wk.next(p)) {
        if (wk.gr.n == 0) continue;
        const int qb = sc % QB;
        ok = ok && mbar_wait(x.q_empty + qb, ((sc / QB) & 1) ^ 1, p.wait_ns);
        uint8_t* dst = x.q + qb * (2 * N * 128);
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
        constexpr int step = 4 * QWARPS;
        const int first = qw * 4 + (lane >> 3);
        load(first, n0, n1);
        load(first + step, f0, f1);
        const int last = twice ? 64 : N;
#pragma unroll 1
        for (int n = first; n < last; n += step) {
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
            // (a row with an infinity or a NaN is NaN as a whole, as its scores are: e4m3 would take infinity for 448)
            const float up = __int_as_float(ex == 255 ? 0x7fffffff : (254 + 7 - ex) << 23);
            if (sub == 0) x.q_scale[qb * N + n] = __int_as_float((ex - 7) << 23);
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
            if (twice) {
                if (sub == 0) x.q_scale[qb * N + n + 64] = __int_as_float((ex - 7) << 23);
                *reinterpret_cast<uint4*>(at + 64 * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(at + (N + 64) * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(x.q_full + qb);
        ++sc;
    }
}

// Kernels of at most 32 and of at most 128 columns; the parts of either are joined by one kernel.
cudaError_t attn_launch_wide(const CUtensorMap& mk, const CUtensorMap& mv, const AttnParams& p, int grid, cudaStream_t st);

}  // namespace lidx
