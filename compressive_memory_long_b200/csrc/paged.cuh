// A key/value cache in pages, and the attention of one new token over it.
//
// The pool holds P pages of `page` rows for every key/value head, [P, Hkv, page, d]; row r of
// sequence b lies in page table[b][r / page] at slot r % page.  A page number outside [0, P)
// or a row past the table is never followed: the row is skipped and the device's page record
// is set (infini_attn_device_status).
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

}  // namespace paged
}  // namespace infini
