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

#include "cache_attn_narrow.cuh"

namespace lidx {

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

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// 4 bits: whether a call widens the sequences' pages first (see cache4_attn.cu), and into how many bytes.  A tile costs an SM
// about 2.6 us where a kernel of 128 rows widens it and 1.25 us where it is widened already; to write and read the copy costs
// it 1.1 us once (chunk of 2048 queries over 16384 keys, 128 units a key: 2.1 ms and 1.0 ms).  So two units a key, or two
// selections of it on average, are enough.  kCopyMost: a copy beyond that is taken for too much memory.  Both go by the table's
// places, since lengths are on the device: a chunk of 2048 over 2048 keys (8 heads of 128, pages of 16) takes 518 us with a
// table of as many, 582 us with 2^18 places and 797 us with 2^20, the most, and 767 us without a copy; over 16384 keys 1045,
// 1108 and 1309 us, and 2305 us without.
constexpr size_t kCopyMost = (size_t)2 << 30;
static size_t attn4_copy_bytes(int64_t B, int64_t S, int G, int Hkv, int D, int page, int64_t max_pages, int topk) {
    const int64_t keys = max_pages * page;
    if (topk > 0 ? S * topk < 2 * keys : S * G <= 128) return 0;
    if (B * max_pages > INT_MAX / page / Hkv || Hkv > 65535) return 0;  // as num_pages; blocks of the widening launch
    const size_t pages = (size_t)(B * max_pages), bytes = 2 * pages * Hkv * page * D;
    if (bytes > kCopyMost) return 0;
    return round256(bytes) + round256(2 * pages * Hkv * sizeof(float)) + round256(pages * sizeof(int32_t));
}

// Both entries; bits 8: exps NULL.
static int attn_call(int bits, const void* q, const int64_t* qs, const void* k_cache, const void* v_cache,
                    const int32_t* k_exps, const int32_t* v_exps,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    const int32_t* kv_len, const int32_t* q_pos, const int32_t* topk_indices,
                    int64_t B, int64_t S, int Hq, int Hkv, int D, int page, int64_t max_pages,
                    int64_t num_pages, int compress_ratio, int topk, float softmax_scale, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !qs || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !kv_len || !out ||
        (bits == 4 && (!k_exps || !v_exps)))
        return LIDX_ERR_NULL;
    const int rc = check_cache(B, S, Hkv, D, page, max_pages, num_pages);
    if (rc) return rc;
    if (Hq < 1 || Hq % Hkv || Hq / Hkv > 128 || B * S > INT_MAX || B * S * Hq > INT_MAX) return LIDX_ERR_SHAPE;
    if (compress_ratio < 1 || !isfinite(softmax_scale) || (topk_indices && (topk < 1 || topk > (1 << 20))))
        return LIDX_ERR_SHAPE;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out | (uintptr_t)k_exps | (uintptr_t)v_exps) & 15u)
        return LIDX_ERR_ALIGN;
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
    const size_t copy = bits == 4 ? attn4_copy_bytes(B, S, p.G, Hkv, D, page, max_pages, topk_indices ? topk : 0) : 0;
    const size_t need = copy + attn_ws_bytes(N, grid);
    if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)) return LIDX_ERR_WORKSPACE;
    p.ws = (uint8_t*)workspace + copy;
    p.codes[0] = (const uint8_t*)k_cache;
    p.codes[1] = (const uint8_t*)v_cache;
    p.exps[0] = k_exps;
    p.exps[1] = v_exps;
    CUtensorMap mk, mv;
    const int box = topk_indices ? 1 : page;  // rows of a copy
    Attn4Copy to;
    if (copy) {
        const int64_t pages = B * max_pages;
        uint8_t* at = (uint8_t*)workspace;
        to.cache[0] = at;
        to.cache[1] = at + pages * Hkv * page * D;
        at += round256((size_t)2 * pages * Hkv * page * D);
        to.scale[0] = (float*)at;
        to.scale[1] = to.scale[0] + pages * Hkv;
        to.table = (int32_t*)(at + round256((size_t)2 * pages * Hkv * sizeof(float)));
        k_cache = to.cache[0];
        v_cache = to.cache[1];
        num_pages = pages;
    }
    if ((bits == 8 || copy) && (attn_cache_map(&mk, k_cache, num_pages * Hkv * page, D, box) ||
                                attn_cache_map(&mv, v_cache, num_pages * Hkv * page, D, box)))
        return LIDX_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (copy) {
        e = attn4_widen_pages(p, to, st);
        if (e != cudaSuccess) return LIDX_ERR_CUDA;
        p.ks = to.scale[0];
        p.vs = to.scale[1];
        p.table = to.table;
        p.num_pages = num_pages;
        bits = 8;
    }
    if (bits == 4)
        e = N <= 32 ? attn4_launch(N, p, grid, st) : attn4_launch_wide(p, grid, st);
    else if (N == 16)
        e = attn_launch<16, 16, 8>(mk, mv, p, grid, st);
    else
        e = N == 32 ? attn_launch<32, 16, 8>(mk, mv, p, grid, st) : attn_launch_wide(mk, mv, p, grid, st);
    if (e == cudaSuccess && grid > 1) switch (N) {
            case 16: e = attn_join<16>(p, grid, st); break;
            case 32: e = attn_join<32>(p, grid, st); break;
            default: e = attn_join<128>(p, grid, st); break;
        }
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
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

size_t lidx_cache4_attn_workspace_bytes(int64_t B, int64_t S, int Hq, int Hkv, int D, int page, int64_t max_pages, int topk) {
    if (check_cache(B, S, Hkv, D, page, max_pages, 1) || topk < 0) return 0;
    const size_t parts = lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk);
    return parts ? parts + attn4_copy_bytes(B, S, Hq / Hkv, Hkv, D, page, max_pages, topk) : 0;
}

int lidx_cache_attn(const void* q, const int64_t* qs, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const int32_t* block_table,
                    const int32_t* kv_len, const int32_t* q_pos, const int32_t* topk_indices,
                    int64_t B, int64_t S, int Hq, int Hkv, int D, int page, int64_t max_pages,
                    int64_t num_pages, int compress_ratio, int topk, float softmax_scale, void* out,
                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_call(8, q, qs, k_cache, v_cache, nullptr, nullptr, k_scale, v_scale, block_table, kv_len, q_pos, topk_indices,
                     B, S, Hq, Hkv, D, page, max_pages, num_pages, compress_ratio, topk, softmax_scale, out, lse, workspace,
                     workspace_bytes, stream);
}

int lidx_cache4_attn(const void* q, const int64_t* qs, const void* k_cache, const void* v_cache, const int32_t* k_exps,
                     const int32_t* v_exps, const float* k_scale, const float* v_scale, const int32_t* block_table,
                     const int32_t* kv_len, const int32_t* q_pos, const int32_t* topk_indices, int64_t B, int64_t S, int Hq,
                     int Hkv, int D, int page, int64_t max_pages, int64_t num_pages, int compress_ratio, int topk,
                     float softmax_scale, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_call(4, q, qs, k_cache, v_cache, k_exps, v_exps, k_scale, v_scale, block_table, kv_len, q_pos, topk_indices, B,
                     S, Hq, Hkv, D, page, max_pages, num_pages, compress_ratio, topk, softmax_scale, out, lse, workspace,
                     workspace_bytes, stream);
}

}  // extern "C"
