// Rotary positions: every pair (x1, x2) of a head's first `rot` channels is turned by the
// angle position * freq[i] and scaled,
//   y1 = s (x1 cos a - x2 sin a),   y2 = s (x2 cos a + x1 sin a),
// pair i being channels (i, i + rot/2) or (2i, 2i+1); the channels from rot on are copied.
// The gradient is the same map with the angle negated (the matrix is s times a rotation).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace infini {
namespace paged {

__device__ __forceinline__ float ld_f(const float *p) { return *p; }
__device__ __forceinline__ float ld_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_f(float *p, float x) { *p = x; }
__device__ __forceinline__ void st_f(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// sigma(x) = ELU(x) + 1 with alpha = 1.
__device__ __forceinline__ float feature_map(float x) { return x > 0.f ? x + 1.f : expf(x); }

struct RotaryArgs {
    const double *freq;          // [rot / 2]
    const int64_t *positions;    // [B, L], or null: start + t
    int64_t start;
    int64_t sq[3], sk[3];        // input strides (batch, head, token), elements
    int64_t L;
    int H, Hkv, rot;
    int interleaved, backward;
    float scale;
};

// cos and sin of pos * freq, times `scale`.  The product is formed in 64 bits (positions near
// a million leave only about 4 bits of a 32-bit angle's fraction) and reduced there to
// half turns in [-1, 1], which 32 bits hold to 2^-24.
__device__ __forceinline__ float2 rotary_turn(double pos, double freq, float scale)
{
    const double half = pos * freq * 0.31830988618379067154;     // angle / pi
    const double r = half - 2.0 * rint(0.5 * half);
    float s, c;
    sincospif((float)r, &s, &c);
    return make_float2(c * scale, s * scale);
}

// One thread per (batch, token, pair or pair of copied channels); it forms the turn once and
// applies it to every head.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_rotary(const T *q, const T *k, T *q_out, T *k_out, RotaryArgs a, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int u = (int)(i % (D / 2));
    const int64_t bt = i / (D / 2), b = bt / a.L, t = bt % a.L;
    int c1, c2;
    float2 cs = make_float2(1.f, 0.f);
    if (u < a.rot / 2) {
        c1 = a.interleaved ? 2 * u : u;
        c2 = a.interleaved ? 2 * u + 1 : u + a.rot / 2;
        const double pos = (double)(a.positions ? a.positions[bt] : a.start + t);
        cs = rotary_turn(pos, a.freq[u], a.scale);
        if (a.backward) cs.y = -cs.y;
    } else {
        c1 = 2 * u;
        c2 = 2 * u + 1;
    }
    for (int h = 0; h < a.H + a.Hkv; ++h) {
        const bool isq = h < a.H;
        const int hh = isq ? h : h - a.H;
        const T *x = isq ? q + b * a.sq[0] + hh * a.sq[1] + t * a.sq[2]
                         : k + b * a.sk[0] + hh * a.sk[1] + t * a.sk[2];
        T *y = isq ? q_out + ((b * a.H + hh) * a.L + t) * D : k_out + ((b * a.Hkv + hh) * a.L + t) * D;
        if (u >= a.rot / 2) {
            const T x1 = x[c1], x2 = x[c2];
            y[c1] = x1;
            y[c2] = x2;
            continue;
        }
        const float x1 = ld_f(x + c1), x2 = ld_f(x + c2);
        st_f(y + c1, x1 * cs.x - x2 * cs.y);
        st_f(y + c2, x2 * cs.x + x1 * cs.y);
    }
}

}  // namespace paged
}  // namespace infini
