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

// Row index of (b, kv head, r) within the pool, in rows of d elements; -1 for a bad page, noted
// in `bad`.  A caller with several rows reports once, after its loads: a store between them would
// put the loads one after the other.
__device__ __forceinline__ int64_t place_of(const PageArgs &a, const int *table_row, int64_t r, int kvh, bool &bad)
{
    const int64_t i = r >> a.shift;
    const int pg = i < a.max_pages ? table_row[i] : -1;
    const bool ok = pg >= 0 && pg < a.P;
    bad |= !ok;
    return ok ? ((((int64_t)pg * a.Hkv + kvh) << a.shift) | (r & (((int64_t)1 << a.shift) - 1))) : -1;
}

__device__ __forceinline__ void report(bool bad)
{
    if (bad) g_page_status = 1;
}

__device__ __forceinline__ uint32_t s_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared, zeros where !ok (the source is not read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}

// A block's rows when 16 bytes go to a thread and row: four rows of keys and values in flight.
template <typename T, int D>
struct RowTile {
    static constexpr int CPR = D * (int)sizeof(T) / 16, LINES = 256 / CPR, ROWS = 4 * LINES;
};

// Chunk c of a row, whose address needs an element's alignment only when !ALIGNED.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_chunk(const T *row, int c)
{
    if constexpr (ALIGNED) {
        return __ldcs(reinterpret_cast<const uint4 *>(row) + c);
    } else {
        constexpr int E = 16 / (int)sizeof(T);
        union {
            uint4 v;
            T x[E];
        } u;
#pragma unroll
        for (int i = 0; i < E; ++i) u.x[i] = row[c * E + i];
        return u.v;
    }
}

// Rows lens[b] .. lens[b] + counts[b] - 1 of the pages from k / v [B, Hkv, T, d] (strided);
// their accumulated weights start at 0.  A copy: bandwidth is the bound, and for one token a
// sequence the latency of lens, table and row one after the other (17,400 rows of 8 heads, d = 128,
// bf16: 143 MB in 25 us, 5.7 TB/s; one token of 64 sequences: 2 us).  A block takes ROWS (token,
// head) rows of one sequence, heads first (a token-major projection is read in one run); those
// past a sequence's count return at once.
template <typename T, int D, bool ALIGNED>
__global__ void __launch_bounds__(256)
k_paged_append(const T *__restrict__ k, const T *__restrict__ v, T *k_pages, T *v_pages,
               float *weights, PageArgs a, const int *__restrict__ counts, int64_t sk0, int64_t sk1,
               int64_t sk2, int64_t sv0, int64_t sv1, int64_t sv2, int Tn, uint32_t blocks)
{
    using Tile = RowTile<T, D>;
    constexpr int CPR = Tile::CPR, LINES = Tile::LINES;
    const int64_t b = blockIdx.x / blocks;
    const int i0 = (int)(blockIdx.x % blocks) * Tile::ROWS;   // (token, head) rows of a sequence fit 31 bits
    const int len = cached_rows(a, b);
    const int n = (counts ? min(max(counts[b], 0), Tn) : Tn) * a.Hkv;
    if (len < 0 || i0 >= n) return;
    const int c = threadIdx.x % CPR, line = threadIdx.x / CPR;
    uint4 *kp = reinterpret_cast<uint4 *>(k_pages), *vp = reinterpret_cast<uint4 *>(v_pages);
    uint4 x[4], y[4];
    int64_t row[4];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = i0 + line + u * LINES;
        row[u] = -1;
        if (i < n) {
            const int t = (int)((uint32_t)i / (uint32_t)a.Hkv), kvh = i - t * a.Hkv;
            x[u] = load_chunk<T, ALIGNED>(k + b * sk0 + kvh * sk1 + t * sk2, c);
            y[u] = load_chunk<T, ALIGNED>(v + b * sv0 + kvh * sv1 + t * sv2, c);
            row[u] = place_of(a, a.table + b * a.max_pages, (int64_t)len + t, kvh, bad);
        }
    }
    report(bad);
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (row[u] >= 0) {
            kp[row[u] * CPR + c] = x[u];
            vp[row[u] * CPR + c] = y[u];
            if (weights && c == 0) weights[row[u]] = 0.f;
        }
}

}  // namespace paged
}  // namespace infini
