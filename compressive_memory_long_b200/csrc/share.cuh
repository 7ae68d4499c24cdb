// Rows of a batch shared out evenly over a fixed number of CTAs, by the device.
//
// Every sequence b has rows(b) rows for each of KH heads; a (sequence, head) -- a unit -- is cut
// into tiles of TR rows, and the tiles of all units are numbered through, sequence by sequence,
// head by head.  CTA c of C = min(NC, tiles) takes tiles [c tiles / C, (c + 1) tiles / C): the
// lengths are known on the device alone, and a long sequence beside short ones leaves no SM idle.
// A unit's part in one CTA is a piece; along the numbering each new piece has a higher CTA or a
// higher unit, so c + unit names it uniquely (below NC + units).
//
// With LEAD = 1 every unit has one tile without rows before its own, which stands for what a
// piece costs besides its rows: a CTA of many short units would end last otherwise.
#pragma once

#include <stdint.h>

namespace infini {
namespace paged {

struct ShareScratch {
    int64_t red[64];             // two values per warp
    int64_t b, before;
};

template <int NC>
__device__ __forceinline__ int64_t share_from(int64_t c, int64_t total)
{
    const int64_t C = total < NC ? total : NC;
    if (c >= C) return total;
    if (total < (1 << 22)) return (uint32_t)c * (uint32_t)total / (uint32_t)C;   // a shorter division
    return c * total / C;
}

// The CTA whose range holds tile t: the largest c with c total / C < t + 1.
template <int NC>
__device__ __forceinline__ int64_t share_owner(int64_t t, int64_t total)
{
    const int64_t C = total < NC ? total : NC;
    if (total < (1 << 22)) return ((uint32_t)(t + 1) * (uint32_t)C - 1) / (uint32_t)total;
    return ((t + 1) * C - 1) / total;
}

template <int LEAD>
__device__ __forceinline__ int64_t share_tiles(int64_t rows, int TR)
{
    const int64_t t = (rows + TR - 1) / TR;
    return t > 0 ? t + LEAD : 0;
}

// Tiles per head of all sequences, and of those before sequence `want`.  The whole block calls.
template <int NT, int LEAD, class Rows>
__device__ __forceinline__ int64_t share_count(const Rows &rows, int64_t B, int TR, int64_t want, ShareScratch &s,
                                               int64_t &before)
{
    int64_t all = 0, pre = 0;
    for (int64_t b = threadIdx.x; b < B; b += NT) {
        const int64_t t = share_tiles<LEAD>(rows(b), TR);
        all += t;
        if (b < want) pre += t;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, off);
        pre += __shfl_xor_sync(0xffffffffu, pre, off);
    }
    if ((threadIdx.x & 31) == 0) {
        s.red[threadIdx.x / 32 * 2] = all;
        s.red[threadIdx.x / 32 * 2 + 1] = pre;
    }
    __syncthreads();
    all = pre = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        all += s.red[2 * w];
        pre += s.red[2 * w + 1];
    }
    __syncthreads();
    before = pre;
    return all;
}

// A tile of the walk through all units; walk_next says whether a new unit begins.
struct Walk {
    int b, kh;                   // sequence, head
    int tile, nt;                // tile of the unit, the unit's tiles
    int n;                       // its rows
};

template <int LEAD, class Rows>
__device__ __forceinline__ bool walk_next(Walk &w, const Rows &rows, int KH, int64_t B, int TR)
{
    if (++w.tile < w.nt) return false;
    w.tile = 0;
    if (++w.kh < KH) return true;
    w.kh = 0;
    for (++w.b; w.b < B; ++w.b) {
        w.n = (int)rows(w.b);
        w.nt = (int)share_tiles<LEAD>(w.n, TR);
        if (w.nt > 0) break;
    }
    return true;
}

// This CTA's tiles [t0, t1) and where the first one lies.  The whole block calls; with t0 >= t1
// there is nothing to do.
template <int NC, int NT, int LEAD, class Rows>
__device__ __forceinline__ void share_begin(const Rows &rows, int64_t B, int KH, int TR, ShareScratch &s, int64_t &t0,
                                            int64_t &t1, Walk &w)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t total = 0, none;
    const bool few = B <= NT;            // one look at the lengths serves both passes
    if (!few) total = KH * share_count<NT, LEAD>(rows, B, TR, 0, s, none);
    t0 = t1 = 0;
    int64_t base = 0, at = 0;
    for (int64_t b0 = 0; b0 < B; b0 += NT) {
        const int64_t b = b0 + threadIdx.x;
        const int64_t mine = b < B ? share_tiles<LEAD>(rows(b), TR) : 0;
        int64_t inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) s.red[warp] = inc;
        __syncthreads();
        int64_t upto = base + inc, sum = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < warp) upto += s.red[i];
            sum += s.red[i];
        }
        if (b0 == 0) {
            if (few) total = KH * sum;
            if (total == 0) return;
            t0 = share_from<NC>(blockIdx.x, total);
            t1 = share_from<NC>(blockIdx.x + 1, total);
            if (t0 >= t1) return;
            at = t0 / KH;    // of the sequence b with before <= at < before + tiles(b)
        }
        if (mine > 0 && upto - mine <= at && at < upto) {
            s.b = b;
            s.before = upto - mine;
        }
        __syncthreads();
        base += sum;
        if (base > at) break;
    }
    w.b = (int)s.b;
    w.n = (int)rows(w.b);
    w.nt = (int)share_tiles<LEAD>(w.n, TR);
    const int64_t in_b = t0 - s.before * KH;
    w.kh = (int)(in_b / w.nt);
    w.tile = (int)(in_b % w.nt);
}

}  // namespace paged
}  // namespace infini
