// rope.cu -- rotary positions of queries and keys, forward and backward.
//
// Pair (a, b) of a head turns by the angle of its position:
//     (a, b) -> (a c - b s, b c + a s),   c = m cos(2 pi t), s = m sin(2 pi t),
// with t the position times the pair's frequency in turns.  The backward is the same turn with -s.
//
// Frequencies are turns per position in 0.64 fixed point, so pos * freq mod 2^64 is the fraction of
// a turn exactly, whatever the position: a float angle would lose log2(pos) of its 24 bits.  The upper
// 32 bits of the product, read as signed, are the angle from half a turn back to half a turn.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <climits>

#include "kernels.h"
#include "lidx.h"

namespace lidx {

struct RopeTensor {
    const void* x;
    void* y;
    int64_t xs[3], ys[3];
    int H;
};
struct RopeParams {
    RopeTensor t[2];
    const int32_t* pos;
    int64_t ps[2];
    const uint64_t* freqs;
    int64_t T0, T1;
    int heads;  // of both tensors
    int D, R, off, half;
    float mscale, sign;
};

// Scaled cosine and sine of position pos of a pair.
__device__ __forceinline__ float2 rope_cs(int pos, uint64_t freq, float mscale, float sign) {
    const uint64_t t = (uint64_t)(int64_t)pos * freq;
    // half turns in [-1, 1): 32 bits of the fraction, rounded once
    const float h = (float)(int32_t)(t >> 32) * 0x1p-31f;
    float s, c;
    sincospif(h, &s, &c);
    return make_float2(c * mscale, s * mscale * sign);
}

__device__ __forceinline__ float rope_get(const float* p) { return *p; }
__device__ __forceinline__ float rope_get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rope_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void rope_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Any alignment, any rotated part: one thread per pair or copied pair of elements.
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
        if (u < p.R / 2) {
            const int ia = p.half ? p.off + u : p.off + 2 * u;
            const int ib = p.half ? ia + p.R / 2 : ia + 1;
            const float2 cs = rope_cs(p.pos[t0 * p.ps[0] + t1 * p.ps[1]], p.freqs[u], p.mscale, p.sign);
            const float a = rope_get(x + ia), b = rope_get(x + ib);
            rope_put(y + ia, a * cs.x - b * cs.y);
            rope_put(y + ib, b * cs.x + a * cs.y);
        } else {
            int d = 2 * (u - p.R / 2);  // the copied dims, those before the rotated part first
            for (int k = 0; k < 2; ++k, ++d) {
                const int at = d < p.off ? d : d + p.R;
                y[at] = x[at];
            }
        }
    }
}

template <class T>
static cudaError_t rope_launch(const RopeParams& p, cudaStream_t st) {
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

int lidx_rope(const lidx_rope_tensor* t, int nt, const int32_t* pos, const int64_t* ps,
              const uint64_t* freqs, int64_t T0, int64_t T1, int D, int rot_dim, int rot_off,
              int layout, int inverse, float mscale, int dtype, void* stream) {
    if (!t || !pos || !ps || !freqs) return LIDX_ERR_NULL;
    if (nt < 1 || nt > 2) return LIDX_ERR_SHAPE;
    for (int i = 0; i < nt; ++i)
        if (!t[i].x || !t[i].y) return LIDX_ERR_NULL;
    if (T0 < 1 || T1 < 1 || T0 > (1 << 30) || T1 > (1 << 30) || T0 * T1 > INT_MAX) return LIDX_ERR_SHAPE;
    if (D < 2 || D > 1024 || D % 2 || rot_dim < 2 || rot_dim % 2 || rot_off < 0 || rot_off + (int64_t)rot_dim > D)
        return LIDX_ERR_SHAPE;
    if ((layout != 0 && layout != 1) || (inverse != 0 && inverse != 1) || (dtype != 0 && dtype != 1) ||
        !isfinite(mscale))
        return LIDX_ERR_SHAPE;
    const uintptr_t es = dtype == 0 ? 4 : 2;
    RopeParams p;
    p.heads = 0;
    for (int i = 0; i < 2; ++i) {
        const lidx_rope_tensor& s = t[i < nt ? i : 0];
        if (s.H < 1 || s.H > (1 << 20)) return LIDX_ERR_SHAPE;
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
    if ((uintptr_t)pos % 4 || (uintptr_t)freqs % 8) return LIDX_ERR_ALIGN;
    p.pos = pos;
    p.ps[0] = ps[0];
    p.ps[1] = ps[1];
    p.freqs = freqs;
    p.T0 = T0;
    p.T1 = T1;
    p.D = D;
    p.R = rot_dim;
    p.off = rot_off;
    p.half = layout == LIDX_ROPE_HALF;
    p.mscale = mscale;
    p.sign = inverse ? -1.f : 1.f;
    if (sm103_sms() <= 0) return LIDX_ERR_NO_DEVICE;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == 0 ? rope_launch<float>(p, st) : rope_launch<__nv_bfloat16>(p, st);
    return e == cudaSuccess ? LIDX_OK : LIDX_ERR_CUDA;
}

}  // extern "C"
