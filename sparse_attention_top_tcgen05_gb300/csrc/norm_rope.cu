// norm_rope.cu -- root-mean-square norms of queries and keys for each head, with the rotary positions in the same pass,
// forward and backward.
//
// Forward: with r = (mean_d x^2 + eps)^-1/2 a head's n = x r w turns as in rope.cu; y = turn(n).
// Backward, from g = dL/dy: u = turn^T(g) (the inverse turn), t = u w, and with h = x r
//     dx = r (t - h mean_d(t h)),    dw_d = sum over rows of u_d h_d.
// The backward takes r from x again: reading a saved r would cost what it saves.  All of it is computed in fp32 from the
// inputs as they are, and rounded once; weights' gradients are fp32.  dw: a thread adds its rows in order, a block its
// threads, a second launch the blocks, all in fixed orders: two calls give the same bits.
//
// What bounds it: reading and writing each element once.  2 x 8192 tokens of 72 bf16 heads of 128: 107 us, 5.6 TB/s;
// backward of 4095 tokens of 40 fp32 heads: 44 us, 5.7 TB/s with the second launch; 16 tokens: 2.5 us, a launch.  In bf16 the
// same backward takes 34 us, 3.7 TB/s: two blocks an SM have half the bytes in flight.  (2 x 4096 tokens of 72 heads: 103 us.)
#include <string.h>

#include "ptx.cuh"
#include "rope.cuh"

namespace lidx {

struct NormTensor {
    const void* x;
    const void* g;  // backward
    void* y;        // output, or gradient of x
    int64_t xs[3], gs[3], ys[3];
    const void* w;  // nullable
    float* dw;      // nullable
    int64_t all;    // rows
    int H, blocks;  // blocks of this tensor
    RopeDiv heads;
    uint32_t step_tok, step_row;  // backward: rows from a block's chunk to its next, as tokens and rows
};
struct NormParams {
    NormTensor t[2];
    RopeTurn r;
    int64_t T0, T1;
    int D, w32;  // w32: weights are fp32, else bf16
    float eps, inv_d;
    RopeDiv tokens1, pairs;
    float* part;  // backward: [blocks][D] sums of u h
};

constexpr int kNormThreads = 256;
// Rows a thread, blocks an SM.  Forward (2 x 8192 tokens of 72 bf16 heads): two rows and five blocks 107 us, two and four 110 us,
// two and six 109 us, one and six 117 us; four and three 105 us, but 9.3 us for 1024 tokens (8.8 us) and 50.3 us for 4096 of fp32
// (48.8 us).  Five blocks leave 48 registers, and kernels of two rows spill 16 to 32 bytes (-Xptxas -v), but for interleaved fp32; with
// four nothing spills, and that is the 110 us.  A call with fewer than two such blocks an SM takes one row.
// Backward, whose blocks go over all rows (4095 tokens of 40 fp32 heads): one row and four blocks 45 us, two and three 51 us.
constexpr int kNormPer = 2;
constexpr int kNormAngles = 4096;   // of a block's tokens: 32 KB
constexpr int kNormBlocks = 4;
template <class T>
constexpr int norm_bwd_blocks() { return sizeof(T) == 4 ? kNormBlocks : 2; }  // (without spills)

__device__ __forceinline__ float norm_weight(const NormParams& p, const void* w, int d) {
    if (!w) return 1.f;
    return p.w32 ? ((const float*)w)[d] : __bfloat162float(((const __nv_bfloat16*)w)[d]);
}

// ------------------------------------------------------------------ aligned tensors
// A row (token, head) belongs to LANES neighbouring lanes, each with two 16-byte vectors: in the half layout the two that
// hold its pairs, so that no element crosses lanes; sums over the row are a few shuffles.
struct NormLane {
    int n;       // vectors of the lane: 0 .. 2
    int d0, d1;  // their first dims
    int c0, c1;  // their items among the rotated ones, -1: not rotated
};
template <bool HALF, int V>
__device__ __forceinline__ NormLane norm_lane(const RopeTurn& r, int D, int l) {
    NormLane o{0, 0, 0, -1, -1};
    if constexpr (HALF) {
        const int np = r.R / 2 / V;
        if (l < np) {
            o = NormLane{2, r.off + l * V, r.off + l * V + r.R / 2, l, l};
        } else {
            const int q = 2 * (l - np), nc = (D - r.R) / V;
            o.n = max(0, min(2, nc - q));
            o.d0 = q * V < r.off ? q * V : q * V + r.R;
            o.d1 = (q + 1) * V < r.off ? (q + 1) * V : (q + 1) * V + r.R;
        }
    } else {
        const int nv = D / V, half = (nv + 1) / 2;
        o.n = l >= half ? 0 : (l + half < nv ? 2 : 1);
        o.d0 = l * V;
        o.d1 = (l + half) * V;
        if (o.d0 >= r.off && o.d0 < r.off + r.R) o.c0 = (o.d0 - r.off) / V;
        if (o.d1 >= r.off && o.d1 < r.off + r.R) o.c1 = (o.d1 - r.off) / V;
    }
    return o;
}
static int norm_lanes(const RopeTurn& r, int D, int V) {
    return r.half ? r.R / 2 / V + ((D - r.R) / V + 1) / 2 : (D / V + 1) / 2;
}

// A lane's elements as P and Q: element i of P and element i of Q are a pair (half layout: of the two vectors; interleaved:
// neighbours, the first vector's and then the second's).  Two neighbouring elements of either are an operand of packed
// arithmetic.
template <bool HALF, class T, int V>
__device__ __forceinline__ void norm_unpack(const uint4& a, const uint4& b, float (&P)[V], float (&Q)[V]) {
    float f[V], g[V];
    rope_unpack(a, f);
    rope_unpack(b, g);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        P[i] = HALF ? f[i] : (i < V / 2 ? f[2 * i] : g[2 * i - V]);
        Q[i] = HALF ? g[i] : (i < V / 2 ? f[2 * i + 1] : g[2 * i + 1 - V]);
    }
}
template <bool HALF, int V>
__device__ __forceinline__ void norm_pack(const float (&P)[V], const float (&Q)[V], uint4& a, uint4& b) {
    float f[V], g[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        f[i] = HALF ? P[i] : (i % 2 ? Q[i / 2] : P[i / 2]);
        g[i] = HALF ? Q[i] : (i % 2 ? Q[V / 2 + i / 2] : P[V / 2 + i / 2]);
    }
    a = rope_pack(f);
    b = rope_pack(g);
}
// Place of element i of P (q: of Q) among the lane's dims.
template <bool HALF, int V>
__device__ __forceinline__ int norm_dim(const NormLane& o, int i, bool q) {
    if (HALF) return (q ? o.d1 : o.d0) + i;
    return (i < V / 2 ? o.d0 + 2 * i : o.d1 + 2 * i - V) + q;
}
template <bool HALF, int V>
__device__ __forceinline__ bool norm_has(const NormLane& o, int i, bool q) {
    return o.n > (HALF ? q : i >= V / 2);
}

// Pairs turn.  cs: angles of the row's token; items: rotated items of a head.
template <bool HALF, int V>
__device__ __forceinline__ void norm_turn(const NormLane& o, const float2* cs, int items, float (&P)[V], float (&Q)[V]) {
    auto turn = [&](int i0, int n, int item) {
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const int i = i0 + 2 * k;
            const float4 v = reinterpret_cast<const float4*>(cs)[k * items + item];
            const uint64_t c = pack2(v.x, v.y), s = pack2(v.z, v.w), m = pack2(-v.z, -v.w);
            const uint64_t a = pack2(P[i], P[i + 1]), b = pack2(Q[i], Q[i + 1]);
            unpack2(fma2(b, m, mul2(a, c)), P[i], P[i + 1]);
            unpack2(fma2(a, s, mul2(b, c)), Q[i], Q[i + 1]);
        }
    };
    if constexpr (HALF) {
        if (o.c0 >= 0) turn(0, V, o.c0);
    } else {
        if (o.c0 >= 0) turn(0, V / 2, o.c0);
        if (o.c1 >= 0) turn(V / 2, V / 2, o.c1);
    }
}

// Weights in shared memory as the lanes' P and Q, words of 16 bytes: the lanes' k-th words follow each other.
template <bool HALF, int LANES, int V>
__device__ __forceinline__ void norm_load_weights(const NormParams& p, const void* w, const NormLane& o, float* s_w) {
    for (int e = threadIdx.x / LANES; e < 2 * V; e += kNormThreads / LANES) {
        const int i = e % V;
        const bool q = e >= V;
        s_w[(e / 4 * LANES + threadIdx.x % LANES) * 4 + e % 4] =
            norm_has<HALF, V>(o, i, q) ? norm_weight(p, w, norm_dim<HALF, V>(o, i, q)) : 0.f;
    }
}
// P (or Q) times weights and r; returns the pairs.
template <int LANES, int V>
__device__ __forceinline__ void norm_weights(const float* s_w, int l, int part, uint64_t (&w)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 a = reinterpret_cast<const float4*>(s_w)[(part * V + i) / 4 * LANES + l];
        w[i / 2] = pack2(a.x, a.y);
        w[i / 2 + 1] = pack2(a.z, a.w);
    }
}
template <int V>
__device__ __forceinline__ float norm_dot(const float (&a)[V], const float (&b)[V], const float (&c)[V], const float (&d)[V]) {
    uint64_t s = pack2(0.f, 0.f), t = s;  // a . b + c . d
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        s = fma2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1]), s);
        t = fma2(pack2(c[i], c[i + 1]), pack2(d[i], d[i + 1]), t);
    }
    float x, y;
    unpack2(add2(s, t), x, y);
    return x + y;
}

template <int LANES>
__device__ __forceinline__ float norm_sum(float v) {
#pragma unroll
    for (int i = 1; i < LANES; i <<= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

// Rows [first, first + n) of a tensor: where row e of a block is.
struct NormRows {
    uint32_t tok0;
    int skip, n;
    __device__ NormRows(const NormTensor& t, int64_t first, int rows) {
        tok0 = t.all < INT_MAX ? rope_quot((uint32_t)first, t.heads) : (uint32_t)(first / t.H);
        skip = (int)(first - (int64_t)tok0 * t.H);
        n = (int)max((int64_t)0, min((int64_t)rows, t.all - first));
    }
    // on by a step of t.step_tok tokens and t.step_row rows; n rows there
    __device__ NormRows after(const NormTensor& t, int rows) const {
        NormRows r = *this;
        r.tok0 += t.step_tok;
        r.skip += t.step_row;
        if (r.skip >= t.H) r.skip -= t.H, ++r.tok0;
        r.n = rows;
        return r;
    }
    // token of the block, and places of row e with strides s and z
    __device__ int token(const NormTensor& t, int e) const { return (int)rope_quot(skip + e, t.heads); }
    __device__ void at(const NormParams& p, const NormTensor& t, const int64_t (&s)[3], const int64_t (&z)[3], int e, int tok,
                       int64_t (&out)[2]) const {
        const uint32_t k = tok0 + tok, t0 = rope_quot(k, p.tokens1), t1 = k - t0 * (uint32_t)p.T1;
        const int h = skip + e - tok * t.H;
        out[0] = t0 * s[0] + t1 * s[1] + h * s[2];
        out[1] = t0 * z[0] + t1 * z[1] + h * z[2];
    }
    // angles of the block's tokens; A of an item
    template <int A>
    __device__ void angles(const NormParams& p, const NormTensor& t, float2* s_cs) const {
        const int R2 = p.r.R / 2, all = (token(t, n - 1) + 1) * R2;
        for (int i = threadIdx.x; i < all; i += kNormThreads) {
            const int k = rope_quot(i, p.pairs);
            const uint32_t tok = tok0 + k, t0 = rope_quot(tok, p.tokens1), t1 = tok - t0 * (uint32_t)p.T1;
            rope_put_angle<A>(s_cs + k * R2, i - k * R2, R2 / A, rope_cs(p.r, t0, t1, i - k * R2));
        }
    }
};

template <class T, bool HALF, int LANES, int PER>
__global__ void __launch_bounds__(kNormThreads, 5) norm_rope_kernel(const __grid_constant__ NormParams p) {
    constexpr int V = 16 / sizeof(T), G = kNormThreads / LANES, A = HALF ? V : V / 2;
    extern __shared__ __align__(16) float s_norm[];
    float* const s_w = s_norm;                               // [2 V / 4][LANES] words
    float2* const s_cs = (float2*)(s_norm + 2 * V * LANES);
    const int which = (int)blockIdx.x >= p.t[0].blocks;
    const NormTensor& t = p.t[which];
    const int64_t first = (int64_t)(blockIdx.x - (which ? p.t[0].blocks : 0)) * (G * PER);
    const NormRows rows(t, first, G * PER);
    const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES;
    const NormLane o = norm_lane<HALF, V>(p.r, p.D, l);
    uint4 a[PER], b[PER];
    int tok[PER];
    T* y[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = grp + k * G;
        a[k] = b[k] = make_uint4(0, 0, 0, 0);
        tok[k] = 0;
        y[k] = nullptr;
        if (e < rows.n) {
            int64_t at[2];
            tok[k] = rows.token(t, e);
            rows.at(p, t, t.xs, t.ys, e, tok[k], at);
            const T* x = (const T*)t.x + at[0];
            y[k] = (T*)t.y + at[1];
            if (o.n > 0) a[k] = *reinterpret_cast<const uint4*>(x + o.d0);
            if (o.n > 1) b[k] = *reinterpret_cast<const uint4*>(x + o.d1);
        }
    }
    norm_load_weights<HALF, LANES, V>(p, t.w, o, s_w);
    rows.angles<A>(p, t, s_cs);
    __syncthreads();
    const int R2 = p.r.R / 2;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        float P[V], Q[V];
        norm_unpack<HALF, T, V>(a[k], b[k], P, Q);
        const float r = __frsqrt_rn(norm_sum<LANES>(norm_dot(P, P, Q, Q)) * p.inv_d + p.eps);
        if (!y[k] || o.n == 0) continue;
        const uint64_t r2 = pack2(r, r);
        uint64_t w[V / 2];
        norm_weights<LANES, V>(s_w, l, 0, w);
#pragma unroll
        for (int i = 0; i < V; i += 2) unpack2(mul2(pack2(P[i], P[i + 1]), mul2(r2, w[i / 2])), P[i], P[i + 1]);
        norm_weights<LANES, V>(s_w, l, 1, w);
#pragma unroll
        for (int i = 0; i < V; i += 2) unpack2(mul2(pack2(Q[i], Q[i + 1]), mul2(r2, w[i / 2])), Q[i], Q[i + 1]);
        norm_turn<HALF, V>(o, s_cs + tok[k] * R2, R2 / A, P, Q);
        norm_pack<HALF, V>(P, Q, a[k], b[k]);
        *reinterpret_cast<uint4*>(y[k] + o.d0) = a[k];
        if (o.n > 1) *reinterpret_cast<uint4*>(y[k] + o.d1) = b[k];
    }
}

// A block goes over its rows in chunks.  A chunk's loads are issued as the chunk before is computed, and its angles go to the
// other half of their buffer, so that a chunk has one barrier.
template <class T, bool HALF, int LANES>
__global__ void __launch_bounds__(kNormThreads, norm_bwd_blocks<T>()) norm_rope_bwd_kernel(const __grid_constant__ NormParams p,
                                                                                int half_angles) {
    constexpr int V = 16 / sizeof(T), G = kNormThreads / LANES, A = HALF ? V : V / 2;
    extern __shared__ __align__(16) float s_norm[];
    float* const s_w = s_norm;
    float2* const s_cs = (float2*)(s_norm + 2 * V * LANES);  // two halves of half_angles
    const int which = (int)blockIdx.x >= p.t[0].blocks;
    const NormTensor& t = p.t[which];
    const int l = threadIdx.x % LANES, grp = threadIdx.x / LANES, R2 = p.r.R / 2;
    const NormLane o = norm_lane<HALF, V>(p.r, p.D, l);
    grid_dependency_launch();
    norm_load_weights<HALF, LANES, V>(p, t.w, o, s_w);
    float sp[V], sq[V];  // sums of u h
#pragma unroll
    for (int i = 0; i < V; ++i) sp[i] = sq[i] = 0.f;
    const int64_t step = (int64_t)t.blocks * G;
    uint4 xa, xb, ga, gb;
    auto load = [&](const NormRows& rows) {
        xa = xb = ga = gb = make_uint4(0, 0, 0, 0);
        if (grp < rows.n) {
            int64_t at[2];
            rows.at(p, t, t.xs, t.gs, grp, rows.token(t, grp), at);
            const T* x = (const T*)t.x + at[0];
            const T* g = (const T*)t.g + at[1];
            if (o.n > 0) {
                xa = *reinterpret_cast<const uint4*>(x + o.d0);
                ga = *reinterpret_cast<const uint4*>(g + o.d0);
            }
            if (o.n > 1) {
                xb = *reinterpret_cast<const uint4*>(x + o.d1);
                gb = *reinterpret_cast<const uint4*>(g + o.d1);
            }
        }
    };
    int64_t first = (int64_t)(blockIdx.x - (which ? p.t[0].blocks : 0)) * G;
    NormRows rows(t, first, G);
    load(rows);
    for (int odd = 0; first < t.all; first += step, odd ^= 1) {
        float2* const cs = s_cs + odd * half_angles;
        rows.angles<A>(p, t, cs);
        __syncthreads();
        const NormRows next = rows.after(t, (int)max((int64_t)0, min((int64_t)G, t.all - (first + step))));
        const int tok = grp < rows.n ? rows.token(t, grp) : 0;
        float xp[V], xq[V], up[V], uq[V], tp[V], tq[V];
        norm_unpack<HALF, T, V>(xa, xb, xp, xq);
        norm_unpack<HALF, T, V>(ga, gb, up, uq);
        load(next);
        norm_turn<HALF, V>(o, cs + tok * R2, R2 / A, up, uq);
        uint64_t w[V / 2];
        norm_weights<LANES, V>(s_w, l, 0, w);
#pragma unroll
        for (int i = 0; i < V; i += 2) unpack2(mul2(pack2(up[i], up[i + 1]), w[i / 2]), tp[i], tp[i + 1]);
        norm_weights<LANES, V>(s_w, l, 1, w);
#pragma unroll
        for (int i = 0; i < V; i += 2) unpack2(mul2(pack2(uq[i], uq[i + 1]), w[i / 2]), tq[i], tq[i + 1]);
        const float r = __frsqrt_rn(norm_sum<LANES>(norm_dot(xp, xp, xq, xq)) * p.inv_d + p.eps);
        const uint64_t r2 = pack2(r, r);
        // x becomes h, which is at most D^1/2 whatever the row's size: the mean of t x overflows with large x, and r r with small
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            unpack2(mul2(pack2(xp[i], xp[i + 1]), r2), xp[i], xp[i + 1]);
            unpack2(mul2(pack2(xq[i], xq[i + 1]), r2), xq[i], xq[i + 1]);
        }
        const float c = -(norm_sum<LANES>(norm_dot(tp, xp, tq, xq)) * p.inv_d);
        if (grp < rows.n && o.n > 0) {
            const uint64_t c2 = pack2(c, c);
            auto grad = [&](const float (&h)[V], const float (&u)[V], float (&t)[V], float (&sum)[V]) {
#pragma unroll
                for (int i = 0; i < V; i += 2) {
                    const uint64_t h2 = pack2(h[i], h[i + 1]);
                    unpack2(fma2(pack2(u[i], u[i + 1]), h2, pack2(sum[i], sum[i + 1])), sum[i], sum[i + 1]);
                    unpack2(mul2(r2, fma2(h2, c2, pack2(t[i], t[i + 1]))), t[i], t[i + 1]);
                }
            };
            grad(xp, up, tp, sp);
            grad(xq, uq, tq, sq);
            int64_t at[2];
            rows.at(p, t, t.ys, t.ys, grp, tok, at);
            T* y = (T*)t.y + at[0];
            uint4 a, b;
            norm_pack<HALF, V>(tp, tq, a, b);
            *reinterpret_cast<uint4*>(y + o.d0) = a;
            if (o.n > 1) *reinterpret_cast<uint4*>(y + o.d1) = b;
        }
        rows = next;
    }
    // the block's sums: one row of smem a group, added in order
    __syncthreads();
    float* const s_sum = (float*)s_cs;  // [G][D]
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (norm_has<HALF, V>(o, i, false)) s_sum[grp * p.D + norm_dim<HALF, V>(o, i, false)] = sp[i];
        if (norm_has<HALF, V>(o, i, true)) s_sum[grp * p.D + norm_dim<HALF, V>(o, i, true)] = sq[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
        float s = 0.f;
        for (int i = 0; i < G; ++i) s += s_sum[i * p.D + d];
        p.part[(int64_t)blockIdx.x * p.D + d] = s;
    }
}

// ------------------------------------------------------------------ any alignment, any rotated part
// A warp a row; a lane has pairs (or two copied dims) and recomputes their angles, in the backward twice: what bounds it.  4095
// tokens of 24 bf16 heads of 80 dims, of which half layouts turn 40: 46 us, backward 85 us (their bytes 4.6 and 7 us).
__device__ __forceinline__ void norm_unit(const RopeTurn& r, int u, int& ia, int& ib) {
    if (u < r.R / 2) {
        ia = r.half ? r.off + u : r.off + 2 * u;
        ib = r.half ? ia + r.R / 2 : ia + 1;
    } else {  // the dims that are not rotated, those before the rotated part first
        const int d = 2 * (u - r.R / 2);
        ia = d < r.off ? d : d + r.R;
        ib = d + 1 < r.off ? d + 1 : d + 1 + r.R;
    }
}
template <class T, bool BWD>
__global__ void __launch_bounds__(kNormThreads) norm_rope_any_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ __align__(16) float s_norm[];  // backward: [warps][D] sums of u h
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, units = p.D / 2;
    const int which = (int)blockIdx.x >= p.t[0].blocks;
    const NormTensor& t = p.t[which];
    float* const sum = s_norm + warp * p.D;
    if constexpr (BWD) {
        grid_dependency_launch();
        for (int d = lane; d < p.D; d += 32) sum[d] = 0.f;
        __syncwarp();
    }
    for (int64_t row = (int64_t)(blockIdx.x - (which ? p.t[0].blocks : 0)) * (kNormThreads / 32) + warp; row < t.all;
         row += (int64_t)t.blocks * (kNormThreads / 32)) {
        const int64_t tok = row / t.H, t0 = tok / p.T1, t1 = tok - t0 * p.T1;
        const int h = (int)(row - tok * t.H);
        const T* x = (const T*)t.x + t0 * t.xs[0] + t1 * t.xs[1] + h * t.xs[2];
        const T* g = BWD ? (const T*)t.g + t0 * t.gs[0] + t1 * t.gs[1] + h * t.gs[2] : nullptr;
        T* y = (T*)t.y + t0 * t.ys[0] + t1 * t.ys[1] + h * t.ys[2];
        // gradients of the pair before the turn
        auto grad = [&](int u, int ia, int ib, float& a, float& b) {
            a = rope_get(g + ia), b = rope_get(g + ib);
            if (u < p.r.R / 2) {
                const float2 c = rope_cs(p.r, t0, t1, u);
                const float s = a;
                a = s * c.x - b * c.y;
                b = b * c.x + s * c.y;
            }
        };
        float s2 = 0.f, s3 = 0.f;
        for (int u = lane; u < units; u += 32) {
            int ia, ib;
            norm_unit(p.r, u, ia, ib);
            const float a = rope_get(x + ia), b = rope_get(x + ib);
            s2 += a * a + b * b;
            if constexpr (BWD) {
                float ga, gb;
                grad(u, ia, ib, ga, gb);
                s3 += ga * norm_weight(p, t.w, ia) * a + gb * norm_weight(p, t.w, ib) * b;
            }
        }
        const float r = __frsqrt_rn(norm_sum<32>(s2) * p.inv_d + p.eps);
        float c = 0.f;  // mean of t h
        if constexpr (BWD) {
            s3 = norm_sum<32>(s3);
            c = r * (s3 * p.inv_d);
            if (!(fabsf(s3) > 0x1p-100f && fabsf(s3) < INFINITY)) {
                // products t x beyond fp32's range, or behind it: those of h, which is at most D^1/2, are not (a pass more in every
                // row costs an eighth of the time)
                s3 = 0.f;
                for (int u = lane; u < units; u += 32) {
                    int ia, ib;
                    norm_unit(p.r, u, ia, ib);
                    float ga, gb;
                    grad(u, ia, ib, ga, gb);
                    s3 += ga * norm_weight(p, t.w, ia) * (rope_get(x + ia) * r) + gb * norm_weight(p, t.w, ib) * (rope_get(x + ib) * r);
                }
                c = norm_sum<32>(s3) * p.inv_d;
            }
        }
        for (int u = lane; u < units; u += 32) {
            int ia, ib;
            norm_unit(p.r, u, ia, ib);
            const float a = rope_get(x + ia), b = rope_get(x + ib);
            const float wa = norm_weight(p, t.w, ia), wb = norm_weight(p, t.w, ib);
            if constexpr (BWD) {
                float ga, gb;
                grad(u, ia, ib, ga, gb);
                const float ha = a * r, hb = b * r;
                sum[ia] += ga * ha;
                sum[ib] += gb * hb;
                rope_put(y + ia, r * (ga * wa - ha * c));
                rope_put(y + ib, r * (gb * wb - hb * c));
            } else {
                const float na = a * (r * wa), nb = b * (r * wb);
                if (u < p.r.R / 2) {
                    const float2 cs = rope_cs(p.r, t0, t1, u);
                    rope_put(y + ia, na * cs.x - nb * cs.y);
                    rope_put(y + ib, nb * cs.x + na * cs.y);
                } else {
                    rope_put(y + ia, na);
                    rope_put(y + ib, nb);
                }
            }
        }
    }
    if constexpr (BWD) {
        __syncthreads();
        for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
            float s = 0.f;
            for (int i = 0; i < kNormThreads / 32; ++i) s += s_norm[i * p.D + d];
            p.part[(int64_t)blockIdx.x * p.D + d] = s;
        }
    }
}

// dw of a tensor: block x has 32 dims, block y the tensor; 32 runs of blocks, then those, in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const __grid_constant__ NormParams p) {
    __shared__ float s[32][33];
    const NormTensor& t = p.t[blockIdx.y];
    grid_dependency_wait();
    if (!t.dw) return;
    const int c = threadIdx.x & 31, run = threadIdx.x >> 5, d = blockIdx.x * 32 + c;
    const float* part = p.part + (blockIdx.y ? (int64_t)p.t[0].blocks * p.D : 0);
    float v = 0.f;
    if (d < p.D)
        for (int b = run; b < t.blocks; b += 32) v += part[(int64_t)b * p.D + d];
    s[run][c] = v;
    __syncthreads();
    if (run == 0 && d < p.D) {
        v = 0.f;
        for (int i = 0; i < 32; ++i) v += s[i][c];
        t.dw[d] = v;
    }
}

// ------------------------------------------------------------------- host

static bool norm_vectors(const NormParams& p, int nt, int V, int es, bool bwd) {
    const RopeTurn& r = p.r;
    if (p.D % V || r.off % V || (r.half ? (r.R / 2) % V : r.R % V) || norm_lanes(r, p.D, V) > 32) return false;
    uintptr_t bits = 0;
    for (int i = 0; i < nt; ++i) {
        const NormTensor& t = p.t[i];
        bits |= (uintptr_t)t.x | (uintptr_t)t.y | (bwd ? (uintptr_t)t.g : 0);
        for (int k = 0; k < 3; ++k)
            bits |= (uintptr_t)(t.xs[k] * es) | (uintptr_t)(t.ys[k] * es) | (bwd ? (uintptr_t)(t.gs[k] * es) : 0);
    }
    return (bits & 15) == 0;
}

// Blocks of the backward, shared out by the tensors' rows.
static void norm_share(NormParams& p, int nt, int rows, int per_sm) {
    int64_t chunks[2] = {0, 0}, all = 0;
    for (int i = 0; i < nt; ++i) all += chunks[i] = (p.T0 * p.T1 * p.t[i].H + rows - 1) / rows;
    const int64_t most = (int64_t)per_sm * current_sms();
    for (int i = 0; i < nt; ++i) {
        int64_t n = all <= most ? chunks[i] : chunks[i] * (most - 1) / all;
        p.t[i].blocks = (int)(n < 1 ? 1 : n);
        const int64_t step = (int64_t)p.t[i].blocks * rows;
        p.t[i].step_tok = (uint32_t)(step / p.t[i].H);
        p.t[i].step_row = (uint32_t)(step % p.t[i].H);
    }
}

template <class T, bool HALF, int LANES>
static cudaError_t norm_launch_lanes(NormParams& p, int nt, bool bwd, cudaStream_t st) {
    constexpr int G = kNormThreads / LANES;
    constexpr int V = 16 / (int)sizeof(T), weights = 2 * V * LANES * 4;
    // A head has at most 2 V LANES dims, all of them turned, and a row may be a token: every launch stays within what any kernel may
    // have (two halves of angles of G + 1 tokens backward; forward one of G + 1, or kNormAngles).
    static_assert(2 * 8 * (G + 1) * V * LANES + weights <= 48 * 1024 && G * 2 * V * LANES * 4 + weights <= 48 * 1024 &&
                      8 * kNormAngles + weights <= 48 * 1024,
                  "shared memory");
    auto smem = [&](int rows) {  // angles of the tokens of `rows` rows
        int64_t angles = 0;
        for (int i = 0; i < nt; ++i) {
            const int64_t n = (int64_t)((rows - 1) / p.t[i].H + 2) * (p.r.R / 2);
            angles = n > angles ? n : angles;
        }
        return angles;
    };
    if (bwd) {
        norm_share(p, nt, G, norm_bwd_blocks<T>());
        const int64_t angles = smem(G) + (smem(G) & 1), a = 2 * angles * 8, s = (int64_t)G * p.D * 4;
        const int bytes = (int)(a > s ? a : s) + weights;
        norm_rope_bwd_kernel<T, HALF, LANES><<<p.t[0].blocks + p.t[1].blocks, kNormThreads, bytes, st>>>(p, (int)angles);
        return cudaGetLastError();
    }
    constexpr int big = G * kNormPer;
    int64_t rows = 0, n[2] = {0, 0};
    for (int i = 0; i < nt; ++i) rows += p.T0 * p.T1 * p.t[i].H;
    const int per = rows / big >= 2 * current_sms() && smem(big) <= kNormAngles ? kNormPer : 1;
    for (int i = 0; i < nt; ++i) {
        n[i] = (p.T0 * p.T1 * p.t[i].H + G * per - 1) / (G * per);
        p.t[i].blocks = (int)n[i];
    }
    if (n[0] + n[1] > INT_MAX) return cudaErrorInvalidValue;
    const int bytes = (int)smem(G * per) * 8 + weights;
    if (per == kNormPer)
        norm_rope_kernel<T, HALF, LANES, kNormPer><<<(unsigned)(n[0] + n[1]), kNormThreads, bytes, st>>>(p);
    else
        norm_rope_kernel<T, HALF, LANES, 1><<<(unsigned)(n[0] + n[1]), kNormThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

template <class T, bool HALF>
static cudaError_t norm_launch_vec(NormParams& p, int nt, bool bwd, cudaStream_t st) {
    const int lanes = norm_lanes(p.r, p.D, 16 / sizeof(T));
    if (lanes <= 4) return norm_launch_lanes<T, HALF, 4>(p, nt, bwd, st);
    if (lanes <= 8) return norm_launch_lanes<T, HALF, 8>(p, nt, bwd, st);
    if (lanes <= 16) return norm_launch_lanes<T, HALF, 16>(p, nt, bwd, st);
    return norm_launch_lanes<T, HALF, 32>(p, nt, bwd, st);
}

template <class T>
static cudaError_t norm_launch(NormParams& p, int nt, bool bwd, cudaStream_t st) {
    if (norm_vectors(p, nt, 16 / sizeof(T), sizeof(T), bwd))
        return p.r.half ? norm_launch_vec<T, true>(p, nt, bwd, st) : norm_launch_vec<T, false>(p, nt, bwd, st);
    constexpr int rows = kNormThreads / 32;
    if (bwd) {
        norm_share(p, nt, rows, kNormBlocks);
        norm_rope_any_kernel<T, true>
            <<<p.t[0].blocks + p.t[1].blocks, kNormThreads, rows * p.D * 4, st>>>(p);
        return cudaGetLastError();
    }
    const int64_t cap = (int64_t)current_sms() * 32;
    for (int i = 0; i < nt; ++i) {
        const int64_t n = (p.T0 * p.T1 * p.t[i].H + rows - 1) / rows;
        p.t[i].blocks = (int)(n < cap ? n : cap);
    }
    norm_rope_any_kernel<T, false><<<p.t[0].blocks + p.t[1].blocks, kNormThreads, 0, st>>>(p);
    return cudaGetLastError();
}

static size_t norm_ws_bytes(int nt, int D, int sms) { return (size_t)(kNormBlocks * sms + nt) * D * sizeof(float); }

// Checks of both directions; fills p.
static int norm_params(const lidx_norm_tensor* t, int nt, const lidx_rope_turn* r, float eps, int64_t T0, int64_t T1, int D,
                       int dtype, int w_dtype, bool bwd, NormParams& p) {
    if (!t) return LIDX_ERR_NULL;
    memset(&p, 0, sizeof p);
    int rc = rope_turn(r, D, bwd, p.r);
    if (rc) return rc;
    if (nt < 1 || nt > 2 || (dtype != 0 && dtype != 1) || (w_dtype != 0 && w_dtype != 1)) return LIDX_ERR_SHAPE;
    for (int i = 0; i < nt; ++i)
        if (!t[i].x || !t[i].y || (bwd && !t[i].g)) return LIDX_ERR_NULL;
    if (!(eps >= 0.f) || !isfinite(eps)) return LIDX_ERR_SHAPE;
    if (T0 < 1 || T1 < 1 || T0 > (1 << 30) || T1 > (1 << 30) || T0 * T1 > INT_MAX) return LIDX_ERR_SHAPE;
    const uintptr_t es = dtype == 0 ? 4 : 2, ws = w_dtype == 0 ? 4 : 2;
    for (int i = 0; i < nt; ++i) {
        NormTensor& o = p.t[i];
        if (t[i].H < 1 || t[i].H > (1 << 15)) return LIDX_ERR_SHAPE;
        if (((uintptr_t)t[i].x | (uintptr_t)t[i].y | (bwd ? (uintptr_t)t[i].g : 0)) % es || (uintptr_t)t[i].w % ws ||
            (bwd && (uintptr_t)t[i].dw % 4))
            return LIDX_ERR_ALIGN;
        o.x = t[i].x;
        o.g = t[i].g;
        o.y = t[i].y;
        for (int k = 0; k < 3; ++k) {
            o.xs[k] = t[i].xs[k];
            o.gs[k] = t[i].gs[k];
            o.ys[k] = t[i].ys[k];
        }
        o.w = t[i].w;
        o.dw = bwd ? t[i].dw : nullptr;
        o.H = t[i].H;
        o.heads = rope_div(o.H);
        o.all = T0 * T1 * o.H;
    }
    rc = rope_turn_aligned(*r);
    if (rc) return rc;
    p.T0 = T0;
    p.T1 = T1;
    p.D = D;
    p.w32 = w_dtype == 0;
    p.eps = eps;
    p.inv_d = 1.f / D;
    p.tokens1 = rope_div((uint32_t)T1);
    p.pairs = rope_div(p.r.R / 2);
    return sm103_sms() <= 0 ? LIDX_ERR_NO_DEVICE : LIDX_OK;
}

}  // namespace lidx

using namespace lidx;

extern "C" {

int lidx_norm_rope(const lidx_norm_tensor* t, int nt, const lidx_rope_turn* r, float eps, int64_t T0, int64_t T1, int D,
                   int dtype, int w_dtype, void* stream) {
    NormParams p;
    const int rc = norm_params(t, nt, r, eps, T0, T1, D, dtype, w_dtype, false, p);
    if (rc) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == 0 ? norm_launch<float>(p, nt, false, st) : norm_launch<__nv_bfloat16>(p, nt, false, st);
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

size_t lidx_norm_rope_bwd_workspace_bytes(int D) {
    if (D < 2 || D > 1024) return 0;
    const int sms = sm103_sms();
    return norm_ws_bytes(2, D, sms > 0 ? sms : 256);  // no device: an upper bound
}

int lidx_norm_rope_bwd(const lidx_norm_tensor* t, int nt, const lidx_rope_turn* r, float eps, int64_t T0, int64_t T1, int D,
                       int dtype, int w_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    NormParams p;
    const int rc = norm_params(t, nt, r, eps, T0, T1, D, dtype, w_dtype, true, p);
    if (rc) return rc;
    if (!workspace || workspace_bytes < norm_ws_bytes(2, D, current_sms()) || ((uintptr_t)workspace & 255u))
        return LIDX_ERR_WORKSPACE;
    p.part = (float*)workspace;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = dtype == 0 ? norm_launch<float>(p, nt, true, st) : norm_launch<__nv_bfloat16>(p, nt, true, st);
    if (e == cudaSuccess && (p.t[0].dw || p.t[1].dw)) {
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3((D + 31) / 32, nt);
        cfg.blockDim = dim3(1024);
        cfg.stream = st;
        // set up while the main kernel runs; it waits for its end itself
        cudaLaunchAttribute at;
        memset(&at, 0, sizeof at);
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, norm_dw_kernel, p);
    }
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
