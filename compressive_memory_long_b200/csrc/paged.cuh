// A key/value cache in pages, and the attention of one new token over it.
//
// The pool holds P pages of `page` rows for every key/value head, [P, Hkv, page, d]; row r of
// sequence b lies in page table[b][r / page] at slot r % page.  A page number outside [0, P)
// or a row past the table is never followed: the row is skipped and the device's page record
// is set (take_page_status).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "rotary.cuh"

namespace infini {
namespace paged {

__device__ int g_page_status;

struct PageArgs {
    const int *table;            // [B, max_pages]
    const int *lens;             // [B] rows cached
    int64_t P;
    int max_pages, shift, Hkv;   // page = 1 << shift
};

// Rows of sequence b in the cache: no more than its table can hold; negative: a padding entry.
__device__ __forceinline__ int cached_rows(const PageArgs &a, int64_t b)
{
    const int n = a.lens[b];
    const int64_t most = (int64_t)a.max_pages << a.shift;
    if (n <= most) return n;
    g_page_status = 1;
    return (int)most;
}

// Row index of (b, kv head, r) within the pool, in rows of d elements; -1 for a bad page.
__device__ __forceinline__ int64_t pool_row(const PageArgs &a, const int *table_row, int64_t r, int kvh)
{
    const int64_t i = r >> a.shift;
    const int pg = i < a.max_pages ? table_row[i] : -1;
    if (pg < 0 || pg >= a.P) {
        g_page_status = 1;
        return -1;
    }
    return ((((int64_t)pg * a.Hkv + kvh) << a.shift) | (r & (((int64_t)1 << a.shift) - 1)));
}

// Rows lens[b] .. lens[b] + counts[b] - 1 of the pages from k / v [B, Hkv, T, d] (strided);
// their accumulated weights start at 0.  One thread per element.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_paged_append(const T *__restrict__ k, const T *__restrict__ v, T *k_pages, T *v_pages,
               float *weights, PageArgs a, const int *__restrict__ counts, int64_t sk0, int64_t sk1,
               int64_t sk2, int64_t sv0, int64_t sv1, int64_t sv2, int64_t Tn, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const int c = (int)(i % D);
    const int64_t t = i / D % Tn, bh = i / D / Tn, b = bh / a.Hkv;
    const int kvh = (int)(bh % a.Hkv), len = cached_rows(a, b);
    if (len < 0 || t >= (counts ? (int64_t)counts[b] : Tn)) return;
    const int64_t row = pool_row(a, a.table + b * a.max_pages, len + t, kvh);
    if (row < 0) return;
    k_pages[row * D + c] = k[b * sk0 + kvh * sk1 + t * sk2 + c];
    v_pages[row * D + c] = v[b * sv0 + kvh * sv1 + t * sv2 + c];
    if (weights && c == 0) weights[row] = 0.f;
}

struct DecodeArgs {
    const float *beta, *M, *z;   // all null: plain attention
    const double *freq;          // null: no rotation
    const int64_t *positions;    // [B], or null: lens
    int H, rot, interleaved;
    float rot_scale;
};

// Channel c of one rotated head row.
template <typename T>
__device__ __forceinline__ float rotated(const T *x, int c, double pos, const DecodeArgs &a)
{
    if (!a.freq || c >= a.rot) return ld_f(x + c);
    const int half = a.rot / 2, i = a.interleaved ? c / 2 : c % half;
    const bool second = a.interleaved ? (c & 1) : c >= half;
    const float2 cs = rotary_turn(pos, a.freq[i], a.rot_scale);
    const float x1 = ld_f(x + (a.interleaved ? 2 * i : i));
    const float x2 = ld_f(x + (a.interleaved ? 2 * i + 1 : i + half));
    return second ? x2 * cs.x + x1 * cs.y : x1 * cs.x - x2 * cs.y;
}

// One CTA per (batch, kv head): the new row is written, then the group's heads one after the
// other: eight warps split the rows, each with its own running maximum, sum and values.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_paged_decode(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, T *k_pages,
               T *v_pages, float *weights, T *__restrict__ out, PageArgs a, DecodeArgs dc)
{
    constexpr int NW = 8, PL = D / 32;
    __shared__ float sq[D], sk[D];
    __shared__ float s_m[NW], s_l[NW], s_o[NW][D], s_den;
    const int64_t b = blockIdx.x / a.Hkv;
    const int kvh = (int)(blockIdx.x % a.Hkv), G = dc.H / a.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = cached_rows(a, b);
    const int *table = a.table + b * a.max_pages;
    const int64_t h0 = b * dc.H + (int64_t)kvh * G;
    if (len < 0) {
        for (int i = tid; i < G * D; i += 256) st_f(out + h0 * D + i, 0.f);
        return;
    }
    const double pos = dc.positions ? (double)dc.positions[b] : (double)len;
    const int64_t n = (int64_t)len + (k ? 1 : 0);
    const T *vt = nullptr;
    if (k) {
        const T *kt = k + ((int64_t)b * a.Hkv + kvh) * D;
        vt = v + ((int64_t)b * a.Hkv + kvh) * D;
        const int64_t row = pool_row(a, table, len, kvh);
        for (int c = tid; c < D; c += 256) {
            T x;
            st_f(&x, rotated(kt, c, pos, dc));
            sk[c] = ld_f(&x);
            if (row >= 0) {
                k_pages[row * D + c] = x;
                v_pages[row * D + c] = vt[c];
            }
        }
        if (weights && row >= 0 && tid == 0) weights[row] = 0.f;
    }
    const float sl2 = rsqrtf((float)D) * 1.4426950408889634f;
    for (int g = 0; g < G; ++g) {
        __syncthreads();
        for (int c = tid; c < D; c += 256) sq[c] = rotated(q + (h0 + g) * D, c, pos, dc);
        __syncthreads();
        float o[PL], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int e = 0; e < PL; ++e) o[e] = 0.f;
        auto score = [&](int64_t j, int64_t &row) {
            row = j == len ? -1 : pool_row(a, table, j, kvh);
            if (row < 0 && j != len) return -INFINITY;
            float part = 0.f;
#pragma unroll
            for (int e = 0; e < PL; ++e)
                part = fmaf(sq[lane + 32 * e], j == len ? sk[lane + 32 * e] : ld_f(k_pages + row * D + lane + 32 * e), part);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            return part * sl2;
        };
        for (int64_t j = warp; j < n; j += NW) {
            int64_t row;
            const float x = score(j, row);
            if (x == -INFINITY) continue;
            const float mn = fmaxf(m, x), r = exp2f(m - mn), p = exp2f(x - mn);
            l = l * r + p;
            const T *vr = j == len ? vt : v_pages + row * D;
#pragma unroll
            for (int e = 0; e < PL; ++e) o[e] = fmaf(p, ld_f(vr + lane + 32 * e), o[e] * r);
            m = mn;
        }
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
#pragma unroll
        for (int e = 0; e < PL; ++e) s_o[warp][lane + 32 * e] = o[e];
        if (dc.M && warp == 0) {
            float part = 0.f;
            for (int f = lane; f < D; f += 32)
                part = fmaf(feature_map(sq[f]), dc.z[((int64_t)b * a.Hkv + kvh) * D + f], part);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            if (lane == 0) s_den = part;
        }
        __syncthreads();
        float mx = -INFINITY, ls = 0.f;
        for (int w = 0; w < NW; ++w) mx = fmaxf(mx, s_m[w]);
        for (int w = 0; w < NW; ++w)
            if (s_m[w] != -INFINITY) ls = fmaf(s_l[w], exp2f(s_m[w] - mx), ls);
        if (tid < D) {
            float os = 0.f;
            for (int w = 0; w < NW; ++w)
                if (s_m[w] != -INFINITY) os = fmaf(s_o[w][tid], exp2f(s_m[w] - mx), os);
            float y = ls > 0.f ? os / ls : 0.f;
            if (dc.M) {
                const float *Mc = dc.M + ((int64_t)b * a.Hkv + kvh) * D * D;
                float num = 0.f;
                for (int f = 0; f < D; ++f) num = fmaf(feature_map(sq[f]), Mc[f * D + tid], num);
                const float gt = 1.f / (1.f + expf(-dc.beta[kvh * G + g]));
                y = gt * (s_den == 0.f ? 0.f : num / s_den) + (1.f - gt) * y;
            }
            st_f(out + (h0 + g) * D + tid, y);
        }
        if (weights)
            for (int64_t j = warp; j < n; j += NW) {
                int64_t row;
                const float x = score(j, row);
                if (j == len) row = pool_row(a, table, len, kvh);
                if (lane == 0 && row >= 0) weights[row] += exp2f(x - mx) / ls;
            }
    }
}

}  // namespace paged
}  // namespace infini
