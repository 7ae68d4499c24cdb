// Eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n rows, every key/value head keeps min(n, budget): the last `recent` ones
// and, of the others, those whose accumulated weight is highest, ties going to the lowest row.
// The kept rows, in their old order, are copied to the first rows of the sequence's
// destination pages.  With a memory the other rows are folded into it as one update of the
// linear rule, M += sum sigma(k) v^T and z += sum sigma(k).
#pragma once

#include "paged.cuh"

namespace infini {
namespace paged {

struct EvictArgs {
    const int *dst_table;        // [B, dst_pages]
    int dst_pages, budget, recent;
    int *lens_out, *kept;        // [B], [B, Hkv, budget]
    int *gone;                   // [B, Hkv, rows - budget] evicted rows (with a memory)
    int64_t gone_stride;
};

// Order-preserving image of a float: larger weight, larger key.  NaN sorts above everything,
// and the two zeros are one value.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One CTA per (batch, kv head).  The weight of rank m is found digit by digit from the top
// (four passes of 8 bits over the candidates, each a histogram of those that share the digits
// found so far); one more pass writes the kept rows, counting rows before each by a block
// prefix sum.
__global__ void __launch_bounds__(1024)
k_evict_select(const float *__restrict__ weights, PageArgs a, EvictArgs e)
{
    __shared__ int hist[256];
    __shared__ int s_scan[2][32];
    __shared__ int s_digit, s_rank;
    const int64_t unit = blockIdx.x, b = unit / a.Hkv;
    const int kvh = (int)(unit % a.Hkv), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = cached_rows(a, b);
    const int *table = a.table + b * a.max_pages;
    int *kept = e.kept + unit * e.budget;
    if (tid == 0 && kvh == 0) e.lens_out[b] = min(n, e.budget);
    if (n <= e.budget) {
        for (int i = tid; i < e.budget; i += 1024) kept[i] = i < n ? i : -1;
        return;
    }
    const int old = n - min(e.recent, n), m = e.budget - (n - old);   // keep m of rows 0..old-1
    auto key_of = [&](int r) {
        const int64_t row = pool_row(a, table, r, kvh);
        return row < 0 ? 0u : weight_key(weights[row]);
    };
    uint32_t thr = 0;
    int rank = m;                       // how many keys of the chosen prefix are kept
    if (m > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += 1024) hist[i] = 0;
            __syncthreads();
            for (int r = tid; r < old; r += 1024) {
                const uint32_t key = key_of(r);
                if (shift == 24 || (key >> (shift + 8)) == (thr >> (shift + 8)))
                    atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = rank, d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                s_digit = d;
                s_rank = left;
            }
            __syncthreads();
            thr |= (uint32_t)s_digit << shift;
            rank = s_rank;
        }
    }
    // keys above thr are kept, and the first `rank` of those equal to it
    int base_keep = 0, base_eq = 0;
    int *gone = e.gone ? e.gone + unit * e.gone_stride : nullptr;
    for (int r0 = 0; r0 < n; r0 += 1024) {
        const int r = r0 + tid;
        const uint32_t key = r < old ? key_of(r) : 0;
        const bool eq = m > 0 && r < old && key == thr;
        const unsigned be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) s_scan[0][warp] = __popc(be);
        __syncthreads();
        int before_eq = base_eq + __popc(be & ((1u << lane) - 1)), all_eq = 0;
        for (int w = 0; w < 32; ++w) {
            before_eq += w < warp ? s_scan[0][w] : 0;
            all_eq += s_scan[0][w];
        }
        const bool keep = r < n && (r >= old || (m > 0 && (key > thr || (eq && before_eq < rank))));
        const unsigned bk = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) s_scan[1][warp] = __popc(bk);
        __syncthreads();
        int before = base_keep + __popc(bk & ((1u << lane) - 1)), all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? s_scan[1][w] : 0;
            all += s_scan[1][w];
        }
        if (keep) kept[before] = r;
        if (gone && r < n && !keep) gone[r - before] = r;
        base_eq += all_eq;
        base_keep += all;
        __syncthreads();
    }
}

// Copies the kept rows: one warp per (unit, row).
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_evict_move(T *k_pages, T *v_pages, float *weights, PageArgs a, EvictArgs e, int64_t rows)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
    if (i >= rows) return;
    const int lane = threadIdx.x & 31, j = (int)(i % e.budget);
    const int64_t unit = i / e.budget, b = unit / a.Hkv;
    const int kvh = (int)(unit % a.Hkv), n = min(cached_rows(a, b), e.budget);
    if (j >= n) return;
    PageArgs dst = a;
    dst.table = e.dst_table;
    dst.max_pages = e.dst_pages;
    const int64_t from = pool_row(a, a.table + b * a.max_pages, e.kept[unit * e.budget + j], kvh);
    const int64_t to = pool_row(dst, e.dst_table + b * e.dst_pages, j, kvh);
    if (from < 0 || to < 0 || from == to) return;
    for (int c = lane; c < D; c += 32) {
        k_pages[to * D + c] = k_pages[from * D + c];
        v_pages[to * D + c] = v_pages[from * D + c];
    }
    if (lane == 0) weights[to] = weights[from];
}

// The evicted rows of one (batch, kv head) into its memory: one CTA, 32 rows at a time.
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_evict_fold(const T *__restrict__ k_pages, const T *__restrict__ v_pages, PageArgs a, EvictArgs e,
             float *M, float *z)
{
    constexpr int TK = 32, R = D / 16;
    __shared__ float sK[TK][D + 1];
    __shared__ float sV[TK][D + 1];
    const int64_t unit = blockIdx.x, b = unit / a.Hkv;
    const int kvh = (int)(unit % a.Hkv), tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int count = cached_rows(a, b) - e.budget;
    if (count <= 0) return;
    const int *table = a.table + b * a.max_pages, *gone = e.gone + unit * e.gone_stride;
    float acc[R][R], zacc = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) acc[i][j] = 0.f;
    for (int t0 = 0; t0 < count; t0 += TK) {
        for (int i = tid; i < TK * D; i += 256) {
            const int t = i / D, c = i % D;
            const int64_t row = t0 + t < count ? pool_row(a, table, gone[t0 + t], kvh) : -1;
            sK[t][c] = row >= 0 ? feature_map(ld_f(k_pages + row * D + c)) : 0.f;
            sV[t][c] = row >= 0 ? ld_f(v_pages + row * D + c) : 0.f;
        }
        __syncthreads();
        for (int t = 0; t < TK; ++t) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < R; ++j)
                    acc[i][j] = fmaf(sK[t][ty + 16 * i], sV[t][tx + 16 * j], acc[i][j]);
        }
        if (tid < D)
            for (int t = 0; t < TK; ++t) zacc += sK[t][tid];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) M[unit * D * D + (ty + 16 * i) * D + tx + 16 * j] += acc[i][j];
    if (tid < D) z[unit * D + tid] += zacc;
}

}  // namespace paged
}  // namespace infini
