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
// a million leave only about 4 bits of a 32-bit angle's fraction) and reduced there to half turns in
// [-1, 1]; what their rounding to 32 bits leaves, up to 2^-25, turns the result by as much.
__device__ __forceinline__ float2 rotary_turn(double pos, double freq, float scale)
{
    const double half = pos * freq * 0.31830988618379067154;     // angle / pi
    const double r = half - 2.0 * rint(0.5 * half);
    const float t = (float)r, rest = (float)(r - (double)t) * 3.14159265358979f;
    float s, c;
    sincospif(t, &s, &c);
    return make_float2(fmaf(-s, rest, c) * scale, fmaf(c, rest, s) * scale);
}

// The turn of pair i at this thread's position.
__device__ __forceinline__ float2 turn_of(const RotaryArgs &a, int64_t bt, int64_t t, int i)
{
    const double pos = (double)(a.positions ? a.positions[bt] : a.start + t);
    float2 cs = rotary_turn(pos, a.freq[i], a.scale);
    if (a.backward) cs.y = -cs.y;
    return cs;
}

template <typename T>
__device__ __forceinline__ const T *rotary_in(const T *q, const T *k, const RotaryArgs &a, int64_t b, int64_t t, int h)
{
    return h < a.H ? q + b * a.sq[0] + h * a.sq[1] + t * a.sq[2]
                   : k + b * a.sk[0] + (h - a.H) * a.sk[1] + t * a.sk[2];
}

template <typename T, int D>
__device__ __forceinline__ T *rotary_out(T *q_out, T *k_out, const RotaryArgs &a, int64_t b, int64_t t, int h)
{
    return h < a.H ? q_out + ((b * a.H + h) * a.L + t) * D : k_out + ((b * a.Hkv + h - a.H) * a.L + t) * D;
}

// 16 bytes of a row as 32-bit values, and back.
template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
    static __device__ __forceinline__ void get(const uint4 &v, float (&x)[N])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[N])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                w[i] = __float_as_uint(x[i]);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Bandwidth is the bound: every element is read and written once (40 heads of 32768 tokens, d = 128,
// bf16, read token by token: 671 MB in 108 us, 6.2 TB/s; fp32 gradients at positions near a million
// 537 MB in 85 us, 6.3 TB/s; one element at a time took 260 and 131 us; 18 of 64 channels in halves of
// nine, 457 MB in 81 us, 5.6 TB/s, against 164 with partners fetched one by one).  A thread owns two 16-byte
// vectors of a token's row and applies its turns, formed once, to its heads, four heads' loads
// in flight at a time.  The vectors are
//   kHalves:  channels c and c + rot/2 (rot/2 a whole number of vectors), or two copied ones;
//   kPairs:   neighbours, each holding whole pairs (interleaved);
//   kRagged:  neighbours; rot/2 cuts a vector, so the turned ones pass through shared memory, where
//             the row's threads (of one warp: it may still be rotated in place) share its pairs.
enum RotaryForm { kHalves, kPairs, kRagged };

template <typename T, int D, int FORM>
__global__ void __launch_bounds__(256)
k_rotary_rows(const T *q, const T *k, T *q_out, T *k_out, RotaryArgs a, int64_t n, int per)
{
    constexpr int N = Vec<T>::N, U = D / (2 * N), NB = 4;
    static_assert(32 % U == 0, "a row lies in one warp");
    // rows of four heads; 16 bytes between rows put a warp's rows in different banks
    constexpr int ROW = 2 * U + 1, SLOT = 256 / U * ROW;
    __shared__ uint4 s_row[FORM == kRagged ? NB * SLOT : 1];
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;                                    // whole rows (n is a multiple of U)
    const int u = (int)(i % U), half = a.rot / 2;
    const int64_t bt = i / U, b = bt / a.L, t = bt % a.L;
    int c1 = 2 * u * N, c2 = c1 + N;
    bool turned = c1 < a.rot;
    if (FORM == kHalves) {
        turned = u < half / N;
        c1 = turned ? u * N : a.rot + 2 * (u - half / N) * N;
        c2 = turned ? c1 + half : c1 + N;
    }
    const int64_t rest = n - (i - (threadIdx.x & 31));     // this warp's threads that have a row
    const unsigned lanes = rest >= 32 ? 0xffffffffu : (1u << rest) - 1;
    float2 cs[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        cs[e] = make_float2(1.f, 0.f);
        if (FORM == kHalves) {
            if (turned) cs[e] = turn_of(a, bt, t, c1 + e);
        } else if (FORM == kPairs) {
            if (c1 + 2 * e < a.rot) cs[e] = turn_of(a, bt, t, c1 / 2 + e);
        } else if (u + e * U < half) {
            cs[e] = turn_of(a, bt, t, u + e * U);
        }
    }
    uint4 *row = s_row + (FORM == kRagged ? threadIdx.x / U * ROW : 0);
    const int h1 = min(((int)blockIdx.y + 1) * per, a.H + a.Hkv);
    for (int h0 = blockIdx.y * per; h0 < h1; h0 += NB) {
        uint4 v[NB][2];
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (h0 + j < h1) {
                const T *x = rotary_in(q, k, a, b, t, h0 + j);
                v[j][0] = *reinterpret_cast<const uint4 *>(x + c1);
                v[j][1] = *reinterpret_cast<const uint4 *>(x + c2);
            }
        if constexpr (FORM == kRagged) {
            __syncwarp(lanes);                             // the last heads' vectors have been read
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (h0 + j < h1 && c1 < a.rot) row[j * SLOT + 2 * u] = v[j][0];
                if (h0 + j < h1 && c2 < a.rot) row[j * SLOT + 2 * u + 1] = v[j][1];
            }
            __syncwarp(lanes);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int c = u + e * U;
                if (c < half)
#pragma unroll
                    for (int j = 0; j < NB; ++j) {
                        T *x = reinterpret_cast<T *>(row + j * SLOT) + c;
                        const float x1 = ld_f(x), x2 = ld_f(x + half);
                        st_f(x, x1 * cs[e].x - x2 * cs[e].y);
                        st_f(x + half, x2 * cs[e].x + x1 * cs[e].y);
                    }
            }
            __syncwarp(lanes);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (c1 < a.rot) v[j][0] = row[j * SLOT + 2 * u];
                if (c2 < a.rot) v[j][1] = row[j * SLOT + 2 * u + 1];
            }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j)
            if (h0 + j < h1) {
                if (FORM != kRagged && turned) {
                    float x1[N], x2[N], y1[N], y2[N];
                    Vec<T>::get(v[j][0], x1);
                    Vec<T>::get(v[j][1], x2);
                    if (FORM == kHalves) {
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            y1[e] = x1[e] * cs[e].x - x2[e] * cs[e].y;
                            y2[e] = x2[e] * cs[e].x + x1[e] * cs[e].y;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < N / 2; ++e) {
                            const float2 w1 = cs[e], w2 = cs[e + N / 2];
                            const bool on1 = c1 + 2 * e < a.rot, on2 = c2 + 2 * e < a.rot;
                            y1[2 * e] = on1 ? x1[2 * e] * w1.x - x1[2 * e + 1] * w1.y : x1[2 * e];
                            y1[2 * e + 1] = on1 ? x1[2 * e + 1] * w1.x + x1[2 * e] * w1.y : x1[2 * e + 1];
                            y2[2 * e] = on2 ? x2[2 * e] * w2.x - x2[2 * e + 1] * w2.y : x2[2 * e];
                            y2[2 * e + 1] = on2 ? x2[2 * e + 1] * w2.x + x2[2 * e] * w2.y : x2[2 * e + 1];
                        }
                    }
                    v[j][0] = Vec<T>::put(y1);
                    if (FORM == kHalves || c2 < a.rot) v[j][1] = Vec<T>::put(y2);
                }
                T *y = rotary_out<T, D>(q_out, k_out, a, b, t, h0 + j);
                *reinterpret_cast<uint4 *>(y + c1) = v[j][0];
                *reinterpret_cast<uint4 *>(y + c2) = v[j][1];
            }
    }
}

// Rows off 16-byte boundaries: one thread per (batch, token, pair or pair of copied channels), which
// alone reads and writes that pair in every head.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_rotary_pairs(const T *q, const T *k, T *q_out, T *k_out, RotaryArgs a, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int u = (int)(i % (D / 2));
    const int64_t bt = i / (D / 2), b = bt / a.L, t = bt % a.L;
    int c1 = 2 * u, c2 = 2 * u + 1;
    float2 cs = make_float2(1.f, 0.f);
    if (u < a.rot / 2) {
        if (!a.interleaved) {
            c1 = u;
            c2 = u + a.rot / 2;
        }
        cs = turn_of(a, bt, t, u);
    }
    for (int h = 0; h < a.H + a.Hkv; ++h) {
        const T *x = rotary_in(q, k, a, b, t, h);
        T *y = rotary_out<T, D>(q_out, k_out, a, b, t, h);
        const T v1 = x[c1], v2 = x[c2];
        if (u >= a.rot / 2) {
            y[c1] = v1;
            y[c2] = v2;
            continue;
        }
        const float x1 = ld_f(&v1), x2 = ld_f(&v2);
        st_f(y + c1, x1 * cs.x - x2 * cs.y);
        st_f(y + c2, x2 * cs.x + x1 * cs.y);
    }
}

}  // namespace paged
}  // namespace infini
