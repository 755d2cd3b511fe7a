// rope.cu -- rotary positions of queries and keys, forward and backward.
//
// Pair (a, b) of a head turns by the angle of its position:
//     (a, b) -> (a c - b s, b c + a s),   c = m cos(2 pi t), s = m sin(2 pi t),
// with t the position times the pair's frequency in turns.  The backward is the same turn with -s.
// With several axes (time, height, width) a token has a position on each, and a pair turns by its axis's: only the lookup of
// the angle changes.
//
// What bounds it: reading and writing each element once.  2 x 8192 tokens of 65 bf16 heads of 128: 89 us, 6.1 TB/s (with
// the divisions by sizes as divisions, a third of the instructions, 105 us); 4095 tokens of 40 fp32 heads: 27 us, 6.2
// TB/s.  16 tokens take 2.2 us, a launch.
#include "rope.cuh"

namespace lidx {

struct RopeTensor {
    const void* x;
    void* y;
    int64_t xs[3], ys[3];
    int H;
};
struct RopeParams {
    RopeTensor t[2];
    RopeTurn r;
    int64_t T0, T1;
    int heads;  // of both tensors
    int D;
    RopeDiv row, items, tokens1, pairs;  // items of a token and of a head, T1, R / 2 (vector kernel)
};

// Any alignment, any rotated part: one thread per pair or copied pair of elements, which recomputes its angle (the prompt
// above: 428 us, bound by instructions).
template <class T>
__global__ void rope_any_kernel(const RopeParams p) {
    const int units = p.D / 2;  // R/2 rotated pairs, then (D - R)/2 copied pairs
    const int64_t n = p.T0 * p.T1 * p.heads * (int64_t)units;
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int u = (int)(e % units);
        const int64_t r = e / units;
        const int hh = (int)(r % p.heads);
        const int64_t tok = r / p.heads, t0 = tok / p.T1, t1 = tok % p.T1;
        const int which = hh >= p.t[0].H;
        const RopeTensor& t = p.t[which];
        const int h = which ? hh - p.t[0].H : hh;
        const T* x = (const T*)t.x + t0 * t.xs[0] + t1 * t.xs[1] + h * t.xs[2];
        T* y = (T*)t.y + t0 * t.ys[0] + t1 * t.ys[1] + h * t.ys[2];
        if (u < p.r.R / 2) {
            const int ia = p.r.half ? p.r.off + u : p.r.off + 2 * u;
            const int ib = p.r.half ? ia + p.r.R / 2 : ia + 1;
            const float2 cs = rope_cs(p.r, t0, t1, u);
            const float a = rope_get(x + ia), b = rope_get(x + ib);
            rope_put(y + ia, a * cs.x - b * cs.y);
            rope_put(y + ib, b * cs.x + a * cs.y);
        } else {
            int d = 2 * (u - p.r.R / 2);  // the copied dims, those before the rotated part first
            for (int k = 0; k < 2; ++k, ++d) {
                const int at = d < p.r.off ? d : d + p.r.R;
                y[at] = x[at];
            }
        }
    }
}

// Aligned tensors.  The items of all (token, head) rows form one line; a block takes PER * 256 of them, a thread PER.  An
// item is a 16-byte vector, or (half layout, rotated part) the two vectors that hold its pairs.  A thread's loads are all
// in flight while the block computes the cosines and sines of its few tokens into shared memory.
constexpr int kRopeThreads = 256;
constexpr int kRopePer = 4;
constexpr int kRopeAngles = 4096;  // of a block's tokens: 32 KB

template <class T, bool HALF, bool AXES, int PER>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const __grid_constant__ RopeParams p) {
    constexpr int V = 16 / sizeof(T);
    // The half layout's items have V angles, which lie as rope_put_angle puts them (8191 tokens of 72 heads, all of 128 dims
    // turned: 53 -> 46 us); the interleaved layout's V / 2 lie side by side, where fewer lanes meet in a bank.
    extern __shared__ __align__(16) float2 s_cs[];
    const int R2 = p.r.R / 2;
    const int rot = HALF ? R2 / V : p.r.R / V;      // rotated items of a head
    const int items = rot + (p.D - p.r.R) / V;      // then its copied vectors
    const int row = items * p.heads;              // items of a token
    const int64_t all = p.T0 * p.T1 * (int64_t)row;
    const int64_t first = (int64_t)blockIdx.x * (PER * kRopeThreads);
    const uint32_t tok0 = (uint32_t)(first / row);
    const int skip = (int)(first - (int64_t)tok0 * row);
    const int n = (int)min((int64_t)(PER * kRopeThreads), all - first);
    uint4 a[PER], b[PER];
    T* dst[PER];
    int cs[PER];  // place of the item's first angles (half layout: in 16-byte words), -1: copied
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int e = threadIdx.x + k * kRopeThreads;
        if (e >= n) break;
        const uint32_t at = skip + e, t = rope_quot(at, p.row), r = at - t * row;
        const int hh = rope_quot(r, p.items), it = r - hh * items;
        const int which = hh >= p.t[0].H, h = which ? hh - p.t[0].H : hh;
        const uint32_t tok = tok0 + t, t0 = rope_quot(tok, p.tokens1), t1 = tok - t0 * (uint32_t)p.T1;
        int d;
        if (it < rot) {
            d = p.r.off + it * V;
            cs[k] = HALF ? t * (R2 / 2) + it : t * R2 + it * (V / 2);
        } else {
            d = (it - rot) * V;
            if (d >= p.r.off) d += p.r.R;
            cs[k] = -1;
        }
        const RopeTensor& x = p.t[which];
        const T* src = (const T*)x.x + t0 * x.xs[0] + t1 * x.xs[1] + h * x.xs[2] + d;
        dst[k] = (T*)x.y + t0 * x.ys[0] + t1 * x.ys[1] + h * x.ys[2] + d;
        a[k] = *reinterpret_cast<const uint4*>(src);
        if (HALF && it < rot) b[k] = *reinterpret_cast<const uint4*>(src + R2);
    }
    const int angles = ((skip + n - 1) / row + 1) * R2;
    for (int i = threadIdx.x; i < angles; i += kRopeThreads) {
        const int t = rope_quot(i, p.pairs);
        const uint32_t tok = tok0 + t, t0 = rope_quot(tok, p.tokens1), t1 = tok - t0 * (uint32_t)p.T1;
        const float2 c = AXES ? rope_cs(p.r, t0, t1, i - t * R2)
                              : rope_cs(p.r.pos[t0 * p.r.ps[1] + t1 * p.r.ps[2]], p.r.freqs[i - t * R2], p.r.mscale, p.r.sign);
        if constexpr (HALF)
            rope_put_angle<V>(s_cs + t * R2, i - t * R2, rot, c);
        else
            s_cs[i] = c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (threadIdx.x + k * kRopeThreads >= n) break;
        if (cs[k] >= 0) {
            float f[V];
            rope_unpack(a[k], f);
            if constexpr (HALF) {
                float2 c[V];
                rope_angles_of<V>(s_cs, cs[k], rot, c);
                float g[V];
                rope_unpack(b[k], g);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u = f[i], w = g[i];
                    f[i] = u * c[i].x - w * c[i].y;
                    g[i] = w * c[i].x + u * c[i].y;
                }
                *reinterpret_cast<uint4*>(dst[k] + R2) = rope_pack(g);
            } else {
                const float2* c = s_cs + cs[k];
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float u = f[2 * i], w = f[2 * i + 1];
                    f[2 * i] = u * c[i].x - w * c[i].y;
                    f[2 * i + 1] = w * c[i].x + u * c[i].y;
                }
            }
            a[k] = rope_pack(f);
        }
        *reinterpret_cast<uint4*>(dst[k]) = a[k];
    }
}

// Angles of the tokens that `n` items can touch.
static int64_t rope_angles(const RopeParams& p, int row, int n) { return (int64_t)((n - 1) / row + 2) * (p.r.R / 2); }

template <class T, bool HALF, bool AXES>
static cudaError_t rope_vec_launch(RopeParams p, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int items = (HALF ? p.r.R / 2 / V : p.r.R / V) + (p.D - p.r.R) / V, row = items * p.heads;
    p.row = rope_div(row);
    p.items = rope_div(items);
    p.tokens1 = rope_div((uint32_t)p.T1);
    p.pairs = rope_div(p.r.R / 2);
    const int64_t all = p.T0 * p.T1 * row;
    // Four items a thread share a block's angles and overlap their loads (2 x 8192 tokens: 89 us, with one item 129 us),
    // unless that leaves SMs without a block (16 tokens: 2.2 us with one) or there are too many angles (a single short head).
    constexpr int big = kRopePer * kRopeThreads;
    const int per = all / big >= 2 * current_sms() && rope_angles(p, row, big) <= kRopeAngles ? kRopePer : 1;
    const int64_t blocks = (all + per * kRopeThreads - 1) / (per * kRopeThreads);
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    const int smem = (int)rope_angles(p, row, per * kRopeThreads) * (int)sizeof(float2);
    if (per == kRopePer)
        rope_vec_kernel<T, HALF, AXES, kRopePer><<<(unsigned)blocks, kRopeThreads, smem, st>>>(p);
    else
        rope_vec_kernel<T, HALF, AXES, 1><<<(unsigned)blocks, kRopeThreads, smem, st>>>(p);
    return cudaGetLastError();
}

// Every vector of every head starts on 16 bytes and lies in or outside the rotated part as a whole.
static bool rope_vectors(const RopeParams& p, int V, int es) {
    if (p.D % V || p.r.off % V || (p.r.half ? (p.r.R / 2) % V : p.r.R % V)) return false;
    uintptr_t bits = 0;
    for (const RopeTensor& t : p.t) {
        bits |= (uintptr_t)t.x | (uintptr_t)t.y;
        for (int k = 0; k < 3; ++k) bits |= (uintptr_t)(t.xs[k] * es) | (uintptr_t)(t.ys[k] * es);
    }
    return (bits & 15) == 0;
}

// Rules of a rotation (see lidx.h), and its device form.
int rope_turn(const lidx_rope_turn* r, int D, int inverse, RopeTurn& out, bool own_pos) {
    if (!r || !r->freqs || (!r->pos && !own_pos)) return LIDX_ERR_NULL;
    if (D < 2 || D > 1024 || D % 2 || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_off < 0 ||
        r->rot_off + (int64_t)r->rot_dim > D)
        return LIDX_ERR_SHAPE;
    if ((r->layout != 0 && r->layout != 1) || (inverse != 0 && inverse != 1) || !isfinite(r->mscale)) return LIDX_ERR_SHAPE;
    if (r->axes < 1 || r->axes > 255 || (r->axes > 1 && !r->axis)) return LIDX_ERR_SHAPE;
    out.pos = r->pos;
    for (int i = 0; i < 3; ++i) out.ps[i] = r->ps[i];
    out.freqs = r->freqs;
    out.axis = r->axes > 1 ? r->axis : nullptr;
    out.axes = r->axes;
    out.R = r->rot_dim;
    out.off = r->rot_off;
    out.half = r->layout == LIDX_ROPE_HALF;
    out.mscale = r->mscale;
    out.sign = inverse ? -1.f : 1.f;
    return LIDX_OK;
}
int rope_turn_aligned(const lidx_rope_turn& r) {
    return (uintptr_t)r.pos % 4 || (uintptr_t)r.freqs % 8 ? LIDX_ERR_ALIGN : LIDX_OK;
}

template <class T>
static cudaError_t rope_launch(const RopeParams& p, cudaStream_t st) {
    if (rope_vectors(p, 16 / sizeof(T), sizeof(T)))
        return p.r.axis ? (p.r.half ? rope_vec_launch<T, true, true>(p, st) : rope_vec_launch<T, false, true>(p, st))
                        : (p.r.half ? rope_vec_launch<T, true, false>(p, st) : rope_vec_launch<T, false, false>(p, st));
    const int64_t n = p.T0 * p.T1 * p.heads * (int64_t)(p.D / 2);
    int64_t blocks = (n + 255) / 256;
    const int64_t cap = (int64_t)current_sms() * 32;
    if (blocks > cap) blocks = cap;
    rope_any_kernel<T><<<(unsigned)blocks, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lidx

using namespace lidx;

extern "C" {

int lidx_rope_freqs(int rot_dim, double theta, int scaling, double factor, double original_len,
                    double beta_fast, double beta_slow, uint64_t* freqs) {
    if (!freqs) return LIDX_ERR_NULL;
    if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2) return LIDX_ERR_SHAPE;
    if (!(theta > 1.0) || !(theta < 1e300) || scaling < LIDX_ROPE_PLAIN || scaling > LIDX_ROPE_YARN)
        return LIDX_ERR_SHAPE;
    if (scaling != LIDX_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < 1e30))) return LIDX_ERR_SHAPE;
    if (scaling == LIDX_ROPE_YARN &&
        (!(original_len > 0.0) || !(original_len < 1e30) || !(beta_fast > beta_slow) ||
         !isfinite(beta_fast) || !isfinite(beta_slow)))
        return LIDX_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    const double R = rot_dim;
    if (scaling == LIDX_ROPE_NTK && rot_dim > 2) theta *= pow(factor, R / (R - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = pow(theta, -2.0 * i / R);
        if (scaling == LIDX_ROPE_LINEAR || (scaling == LIDX_ROPE_NTK && rot_dim == 2)) w /= factor;
        if (scaling == LIDX_ROPE_YARN) {
            double g = (original_len * w / two_pi - beta_slow) / (beta_fast - beta_slow);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            w = w * ((1.0 - g) / factor + g);
        }
        freqs[i] = (uint64_t)rint(w / two_pi * 18446744073709551616.0);  // w <= 1: below 2^62
    }
    return LIDX_OK;
}

int lidx_rope_axes(const lidx_rope_tensor* t, int nt, const lidx_rope_turn* r, int64_t T0, int64_t T1, int D, int inverse,
                   int dtype, void* stream) {
    if (!t) return LIDX_ERR_NULL;
    RopeParams p;
    int rc = rope_turn(r, D, inverse, p.r);
    if (rc) return rc;
    if (nt < 1 || nt > 2 || (dtype != 0 && dtype != 1)) return LIDX_ERR_SHAPE;
    for (int i = 0; i < nt; ++i)
        if (!t[i].x || !t[i].y) return LIDX_ERR_NULL;
    if (T0 < 1 || T1 < 1 || T0 > (1 << 30) || T1 > (1 << 30) || T0 * T1 > INT_MAX) return LIDX_ERR_SHAPE;
    const uintptr_t es = dtype == 0 ? 4 : 2;
    p.heads = 0;
    for (int i = 0; i < 2; ++i) {
        const lidx_rope_tensor& s = t[i < nt ? i : 0];
        if (s.H < 1 || s.H > (1 << 15)) return LIDX_ERR_SHAPE;
        if (((uintptr_t)s.x | (uintptr_t)s.y) % es) return LIDX_ERR_ALIGN;
        p.t[i].x = s.x;
        p.t[i].y = s.y;
        for (int k = 0; k < 3; ++k) {
            p.t[i].xs[k] = s.xs[k];
            p.t[i].ys[k] = s.ys[k];
        }
        p.t[i].H = s.H;
        if (i < nt) p.heads += s.H;
    }
    rc = rope_turn_aligned(*r);
    if (rc) return rc;
    p.T0 = T0;
    p.T1 = T1;
    p.D = D;
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == 0 ? rope_launch<float>(p, st) : rope_launch<__nv_bfloat16>(p, st);
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

int lidx_rope(const lidx_rope_tensor* t, int nt, const int32_t* pos, const int64_t* ps,
              const uint64_t* freqs, int64_t T0, int64_t T1, int D, int rot_dim, int rot_off,
              int layout, int inverse, float mscale, int dtype, void* stream) {
    if (!ps) return LIDX_ERR_NULL;
    const lidx_rope_turn r = {pos, {0, ps[0], ps[1]}, freqs, nullptr, 1, rot_dim, rot_off, layout, mscale};
    return lidx_rope_axes(t, nt, &r, T0, T1, D, inverse, dtype, stream);
}

}  // extern "C"
