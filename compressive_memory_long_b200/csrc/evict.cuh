// Eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n rows, every key/value head keeps min(n, budget): the last `recent` ones
// and, of the others, those whose accumulated weight is highest, ties going to the lowest row.
// The kept rows, in their old order, are copied to the first rows of the sequence's
// destination pages.  With a memory the other rows are folded into it as one update of the
// linear rule, M += sum sigma(k) v^T and z += sum sigma(k).
//
// Three steps, each a kernel that may start while the one before drains: select (cluster of
// CTAs per head, the weights read once), fold (tensor cores, the evicted rows shared out over
// all SMs), finish (adds the fold's pieces to the memory and moves the kept rows).
#pragma once

#include "paged.cuh"
#include "share.cuh"
#include "tc_paged.cuh"

namespace infini {
namespace paged {

struct EvictArgs {
    const int *dst_table;        // [B, dst_pages]
    int dst_pages, budget, recent;
    int *lens_out, *kept;        // [B], [B, Hkv, budget]
    int *gone;                   // [B, Hkv, gone_stride] evicted rows (with a memory)
    int64_t gone_stride;
    int64_t B;
    int fold_rows;               // of a tile of the fold
    float *part_M, *part_z;      // [slots, D * D], [slots, kFoldLoaders, D]
};

// Rows of sequence b that leave each head (none of a padding entry, however negative its length).
__device__ __forceinline__ int64_t rows_leaving(const PageArgs &a, const EvictArgs &e, int64_t b)
{
    const int n = cached_rows(a, b);
    return n > e.budget ? n - e.budget : 0;
}

// Order-preserving image of a float: larger weight, larger key.  NaN sorts above everything,
// and the two zeros are one value.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    if (w != w) return 0xffffffffu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// ---- select -----------------------------------------------------------------------------------
//
// A cluster of CTAs per (batch, kv head); each holds the keys of its part of the rows in shared
// memory (rows past kSelectKeys are read again).  The key of rank m is found digit by digit from
// the top: 11, 11 and 10 bits, each a histogram of the keys that share the digits found so far,
// summed over the cluster.  Then every warp counts the keys above and equal to it in its own run
// of rows; prefix sums over warps and CTAs give each row its place.  11 bits for the first digit
// take the exponent and two bits more: attention weights spread over few exponents, and 8 bits
// would put most of them in a handful of bins.  The bound is latency: 65500 rows of 8 heads take
// 26 us on 64 CTAs (lens, page table and weights one after the other 7; per digit 1 to 2 for the
// histogram, 0.8 for the cluster's barrier and 1.5 for the digit; 5 for the places).  Clusters of
// 16 CTAs could not all be resident and took 38 us.
constexpr int kSelectThreads = 1024;
constexpr int kSelectKeys = 40960;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int peer_ld(const int *p, uint32_t rank)
{
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ int2 peer_ld2(const int *p, uint32_t rank)
{
    uint32_t at;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// Sum of the 32 warps' values before this warp's.
__device__ __forceinline__ int before_warp(const int *per_warp, int warp, int lane)
{
    return __reduce_add_sync(0xffffffffu, lane < warp ? per_warp[lane] : 0);
}

__global__ void __launch_bounds__(kSelectThreads)
k_evict_select(const float *__restrict__ weights, PageArgs a, EvictArgs e, int CS, int cap)
{
    constexpr int NT = kSelectThreads, NW = NT / 32;
    extern __shared__ int s_dyn[];
    int *hist = s_dyn;                                               // [3][kBins]
    uint32_t *keys = reinterpret_cast<uint32_t *>(s_dyn + 3 * kBins);   // [cap]
    __shared__ int s_gt[NW], s_eq[NW];
    __shared__ __align__(8) int s_tot[2], groups[3 * 64];
    __shared__ int s_digit, s_rank;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t unit = blockIdx.x / CS, b = unit / a.Hkv;
    const int kvh = (int)(unit % a.Hkv), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CS > 1 ? (int)cluster_rank() : 0;
    const int n = cached_rows(a, b);
    const int *table = a.table + b * a.max_pages;
    int *kept = e.kept + unit * e.budget;
    if (tid == 0 && kvh == 0 && rank == 0) e.lens_out[b] = min(n, e.budget);
    if (n <= e.budget) {
        for (int64_t i = rank * NT + tid; i < e.budget; i += CS * NT) kept[i] = i < n ? (int)i : -1;
        return;
    }
    const int old = n - min(e.recent, n), m = e.budget - (n - old);   // keep m of rows 0..old-1
    for (int i = rank * NT + tid; i < n - old; i += CS * NT) kept[m + i] = old + i;
    const int per = (old + CS - 1) / CS, r0 = min(rank * per, old), cnt = min(per, old - r0);
    bool bad = false;
    auto load_key = [&](int i) {        // a row without a page goes first
        const int64_t row = place_of(a, table, r0 + i, kvh, bad);
        return row < 0 ? 0u : weight_key(__ldcs(weights + row));
    };
    auto key_of = [&](int i) { return i < cap ? keys[i] : load_key(i); };
    for (int i = tid; i < 3 * kBins; i += NT) hist[i] = 0;
    {
        const int held = min(cnt, cap);
        for (int i0 = tid; i0 < held; i0 += 8 * NT) {
            uint32_t x[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) x[u] = i0 + u * NT < held ? load_key(i0 + u * NT) : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i0 + u * NT < held) keys[i0 + u * NT] = x[u];
        }
    }
    __syncthreads();
    uint32_t thr = 0;
    int left = m;                       // how many keys of the digits so far are kept
    if (m > 0) {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            int *h = hist + pass * kBins;
            for (int i = tid; i < cnt; i += NT) {
                const uint32_t key = key_of(i);
                if (pass == 0 || (key >> (shift + bits)) == (thr >> (shift + bits)))
                    atomicAdd(&h[(key >> shift) & ((1 << bits) - 1)], 1);
            }
            __syncthreads();
            // a warp's 64 bins are two groups
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int sum = __reduce_add_sync(0xffffffffu, h[warp * 64 + k * 32 + lane]);
                if (lane == 0) groups[pass * 64 + warp * 2 + k] = sum;
            }
            if (CS > 1) cluster_sync();
            else __syncthreads();
            // Warp 0 finds the digit: the bin where the count from the top reaches `left`.  First
            // among 64 groups of 32 bins (each CTA's sums), two to a lane, then among a group's.
            if (warp == 0) {
                const int *gr = groups + pass * 64;
                int x0 = 0, x1 = 0;
                const int hi = 62 - 2 * lane;              // groups hi + 1 and hi, from the top
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < CS) {
                        const int2 y = CS > 1 ? peer_ld2(gr + hi, c) : *reinterpret_cast<const int2 *>(gr + hi);
                        x0 += y.y;
                        x1 += y.x;
                    }
                int inc = x0 + x1;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off) inc += y;
                }
                int above = inc - x0 - x1;
                bool here = above < left && left <= inc;
                int g = left <= above + x0 ? hi + 1 : hi;
                if (g == hi) above += x0;
                const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
                g = __shfl_sync(0xffffffffu, g, src);
                above = __shfl_sync(0xffffffffu, above, src);
                int x = 0;
                const int bin = g * 32 + 31 - lane;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < CS) x += CS > 1 ? peer_ld(h + bin, c) : h[bin];
                inc = x;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, inc, off);
                    if (lane >= off) inc += y;
                }
                above += inc - x;
                if (above < left && left <= above + x) {
                    s_digit = bin;
                    s_rank = left - above;
                }
            }
            __syncthreads();
            thr |= (uint32_t)s_digit << shift;
            left = s_rank;
        }
    }
    // a warp's run of rows, 32 at a time
    const int run = ((cnt + NW - 1) / NW + 31) / 32 * 32, w0 = min(warp * run, cnt), w1 = min(w0 + run, cnt);
    int gt = 0, eq = 0;
    for (int i = w0; i < w1; i += 32) {
        const uint32_t key = i + lane < w1 ? key_of(i + lane) : 0;
        const bool in = i + lane < w1 && m > 0;
        gt += __popc(__ballot_sync(0xffffffffu, in && key > thr));
        eq += __popc(__ballot_sync(0xffffffffu, in && key == thr));
    }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    if (warp < 2) {
        const int sum = __reduce_add_sync(0xffffffffu, warp == 0 ? s_gt[lane] : s_eq[lane]);
        if (lane == 0) s_tot[warp] = sum;
    }
    if (CS > 1) cluster_sync();
    else __syncthreads();
    gt = before_warp(s_gt, warp, lane);
    eq = before_warp(s_eq, warp, lane);
#pragma unroll
    for (int c = 0; c < 7; ++c)
        if (c < rank) {
            const int2 y = peer_ld2(s_tot, c);
            gt += y.x;
            eq += y.y;
        }
    int *gone = e.gone ? e.gone + unit * e.gone_stride : nullptr;
    for (int i = w0; i < w1; i += 32) {
        const uint32_t key = i + lane < w1 ? key_of(i + lane) : 0;
        const bool in = i + lane < w1;
        const unsigned bg = __ballot_sync(0xffffffffu, in && m > 0 && key > thr);
        const unsigned be = __ballot_sync(0xffffffffu, in && m > 0 && key == thr);
        const unsigned low = (1u << lane) - 1;
        const int eq_before = eq + __popc(be & low);
        const int before = gt + __popc(bg & low) + min(eq_before, left);
        const bool keep = (bg >> lane & 1) || ((be >> lane & 1) && eq_before < left);
        const int r = r0 + i + lane;
        if (keep) kept[before] = r;
        else if (in && gone) gone[r - before] = r;
        gt += __popc(bg);
        eq += __popc(be);
    }
    report(bad);
    if (CS > 1) cluster_sync();         // no CTA leaves while another reads its counts
}

// ---- fold ---------------------------------------------------------------------------------------
//
// sum sigma(k) v^T over a head's evicted rows, on tcgen05: A = sigma(K)^T (M = the key features),
// B = V (N = the value features), both staged row by row (MN-major), 64 rows a stage (fp32: 32).
// M and z are 32-bit sums, so sigma(k) is split into three bf16 parts (24 bits; two would leave
// 2^-17 of it, more than the sum's own rounding), v into one (bf16, exact) or three (fp32: the six
// products down to 2^-24 are kept).  The tensor core's additions over a long axis lose about one
// unit each, all in one direction: the leading product and the others have accumulators of their
// own, and both are read out and added in registers every 256 rows (twice as many additions
// between two readings raised the error of a 63,000-row sum from 2e-7 to 7e-7).
//
// The evicted rows of all heads are shared out evenly over 148 CTAs (share.cuh).  In each, 16
// loader warps copy rows two stages ahead (64 KB in flight), form sigma and the parts and sum z;
// one thread issues the products; eight warps read the accumulators.  Reading K and V is the floor
// (4 d bytes a row against 2 d^2 operations), 1400 cycles for a stage (bf16, d = 128).  Shared
// memory is the bound: copies and parts move 96 KB through it and the products' operands 96 KB,
// 1500 cycles at 128 bytes, and a stage takes 2300 (65500 rows of 8 heads: 79 us, 3.3 TB/s).
// Tried without gain: sigma as max(k, 0) + e^min(k, 0) with the first term taken as a part (fewer
// instructions, the same time); z as a product with a column of ones (reads sigma's parts once
// more: 98 us).
constexpr int kFoldCtas = 148;
constexpr int kFoldLoaders = 16, kFoldReaders = 8;
// 28 warps, launched with 72 registers a thread (64512 in all); the loaders go down to 64 and the
// issuing warpgroup to 24, which gives the readers their 104.
constexpr int kFoldThreads = 32 * (kFoldLoaders + kFoldReaders + 4);
// Rows of a tile (one reading of the accumulators): many, or two stages where no head evicts more
// than kFoldFew, since a tile's stages pass through the pipeline whether they have rows or not (36
// evicted rows, fp32, the whole call: 16 us against 20).
constexpr int kFoldRows = 256, kFoldFew = 512;

template <typename T, int D, bool FEW>
struct FoldTile {
    static constexpr bool kWide = sizeof(T) == 4;
    static constexpr int VP = kWide ? 3 : 1;               // parts of v
    static constexpr int HALF = kWide ? 32 : 64;           // rows of a stage
    static constexpr int ROWS = FEW ? 2 * HALF : kFoldRows, SUB = ROWS / HALF;   // rows and stages of a tile
    static constexpr int KB = 2 * HALF * 128;              // bytes of a part: two blocks of 64 columns
    // Staged parts, two deep (fp32: v's parts with them; bf16: v as it is, four deep), then the
    // rows as they arrive, three deep.
    static constexpr int PART = kWide ? 6 * KB : 3 * KB;
    static constexpr int CPR = D * (int)sizeof(T) / 16;    // 16-byte chunks of a row
    static constexpr int LR = HALF / kFoldLoaders;         // rows of a loader warp and stage
    static constexpr int LD = (LR * CPR + 31) / 32;        // chunks per lane, tensor and stage
    static constexpr int RAW = kFoldLoaders * LD * 512 * (kWide ? 2 : 1);   // a chunk's place per lane
    static constexpr int V_AT = 2 * PART, RAW_AT = V_AT + (kWide ? 0 : 4 * KB);
    static constexpr int SMEM = RAW_AT + 3 * RAW + 1024;   // rounded up to 1024 inside
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static constexpr int E = 16 / (int)sizeof(T);          // channels of a chunk
    static constexpr uint32_t COLS = 4 * D;                // two buffers of two accumulators
};

__device__ __forceinline__ uint64_t f2_twice(float x) { return tc::f2_pack(x, x); }

__device__ __forceinline__ float max_nan(float x, float y)
{
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ float min_nan(float x, float y)
{
    float z;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

// sigma of two values.  e^x is 2^h (1 + r ln 2) with h + r = x log2(e): 2^(x log2(e)) alone would be off
// by the product's rounding, 0.7 |x| units, mostly to one side.  Keys below -200, whose e^x is 0, are
// taken as that, so that nothing here is infinite.  A NaN passes through the maximum.
//
// bf16 values: h is the product with 16 bits of log2(e), exact; x the rest of it r (r^2 / 4 is lost: one
// unit in 24 bits at x = -70).  sigma = max(x, 0) + min(e^x, 1); the saturating addition is the minimum,
// and off the pipe that the parts' conversions fill.
__device__ __forceinline__ uint64_t sigma2(uint32_t xy)
{
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(xy) : "r"(0xc348c348u));                     // -200
    const float x = __uint_as_float(xy << 16), y = __uint_as_float(xy & 0xffff0000u);
    const uint64_t v = tc::f2_pack(x, y);
    float h0, h1, e0, e1;
    tc::f2_unpack(tc::f2_mul(v, f2_twice(1.44268798828125f)), h0, h1);
    const uint64_t e = tc::f2_pack(tc::ex2(h0), tc::ex2(h1));
    tc::f2_unpack(tc::f2_fma(e, tc::f2_mul(v, f2_twice(4.88849518e-6f)), e), e0, e1);
    return tc::f2_add(tc::f2_pack(max_nan(x, 0.f), max_nan(y, 0.f)), tc::f2_pack(__saturatef(e0), __saturatef(e1)));
}

// fp32 values: h is the product with log2(e) rounded to 24 bits, r what either rounding left.
// sigma = max(x, 0) + e^min(x, 0).
__device__ __forceinline__ uint64_t sigma2(float x, float y)
{
    const uint64_t v = tc::f2_pack(max_nan(min_nan(x, 0.f), -200.f), max_nan(min_nan(y, 0.f), -200.f));
    const uint64_t nh = tc::f2_mul(v, f2_twice(-1.4426950408889634f));
    float h0, h1;
    tc::f2_unpack(nh, h0, h1);
    const uint64_t e = tc::f2_pack(tc::ex2(-h0), tc::ex2(-h1));
    const uint64_t r = tc::f2_fma(v, f2_twice(1.925963033e-8f), tc::f2_fma(v, f2_twice(1.4426950408889634f), nh));
    return tc::f2_add(tc::f2_pack(max_nan(x, 0.f), max_nan(y, 0.f)),
                      tc::f2_fma(e, tc::f2_mul(r, f2_twice(0.6931471805599453f)), e));
}

// x = h + m + l in bf16 parts, to 2^-25 of it; pairs packed.
__device__ __forceinline__ void split3(uint64_t xy, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        float x, y;
        tc::f2_unpack(xy, x, y);
        p[i] = tc::pack_bf16x2(x, y);
        if (i < 2) xy = tc::f2_sub(xy, tc::f2_pack(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u)));
    }
}

template <typename T, int D, bool FEW>
__global__ void __launch_bounds__(kFoldThreads, 1)
k_evict_fold(const T *__restrict__ k_pages, const T *__restrict__ v_pages, PageArgs a, EvictArgs e, float *M)
{
    using Tile = FoldTile<T, D, FEW>;
    constexpr int CPR = Tile::CPR, LD = Tile::LD, E = Tile::E, SUB = Tile::SUB, HALF = Tile::HALF, VP = Tile::VP, ST = 2;
    extern __shared__ unsigned char s_raw[];
    __shared__ __align__(8) uint64_t full[ST], empty[ST], tfull[2], tempty[2], drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ ShareScratch s_share;
    unsigned char *base = s_raw + ((1024 - (tc::smem_u32(s_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const bool given_up = tc::wait_status_set();           // (its latency lies beside that of the lengths)
    auto rows_of = [&](int64_t b) { return rows_leaving(a, e, b); };
    Walk first;
    int64_t t0, t1;
    share_begin<kFoldCtas, kFoldThreads, 0>(rows_of, e.B, a.Hkv, Tile::ROWS, s_share, t0, t1, first);
    // nothing to do, or a record of a wait that gave up has not been read yet (the whole CTA)
    if (__syncthreads_or(t0 >= t1 || given_up)) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(&full[i], kFoldLoaders);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&tfull[i], 1);
            tc::mbar_init(&tempty[i], kFoldReaders);
        }
        tc::mbar_init(&drained, 1);
        s_abort = 0;
        tc::fence_barrier_init();
    }
    if (D < 128)                        // columns that no row fills: features past D are 0
        for (int i = tid; i < Tile::RAW_AT / 16; i += kFoldThreads)
            reinterpret_cast<uint4 *>(base)[i] = make_uint4(0, 0, 0, 0);
    if (warp == 0) tc::tmem_alloc(&s_tmem, Tile::COLS);
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    asm volatile("griddepcontrol.wait;" ::: "memory");     // from here on the selection is read, M written
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int *abort = &s_abort;
    const int64_t steps = t1 - t0;
    // A whole warp waits: lanes that saw the barrier and lanes that gave up go on the same way.  A role
    // that gave up stops at once and signals nothing more, so that no other one takes a stage or an
    // accumulator that is not complete.
    auto wait_all = [&](uint64_t *bar, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort, where)) != 0;
    };

    if (warp < kFoldLoaders) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // Lane x looks up row x % LR of this warp in stage x / LR of a tile: the evicted row's number
        // two tiles ahead, its page one, its data two stages.
        constexpr int LR = Tile::LR;
        Walk ahead = first;
        int64_t t_ahead = t1 - t0;
        int r1 = -1, r2 = -1, kvh1 = 0, kvh2 = 0, pg2 = -1, b1 = 0;
        int64_t base3 = -1;
        auto take_row = [&] {
            r1 = -1;
            if (t_ahead <= 0) return;
            const int j = ahead.tile * Tile::ROWS + lane / LR * HALF + warp * LR + lane % LR;
            b1 = ahead.b;
            kvh1 = ahead.kh;
            if (lane < SUB * LR && j < ahead.n) r1 = e.gone[((int64_t)b1 * a.Hkv + kvh1) * e.gone_stride + j];
            walk_next<0>(ahead, rows_of, a.Hkv, e.B, Tile::ROWS);
            --t_ahead;
        };
        auto take_page = [&] {
            r2 = r1;
            kvh2 = kvh1;
            pg2 = -1;
            if (r2 >= 0) {
                const int i = r2 >> a.shift;
                pg2 = i < a.max_pages ? a.table[(int64_t)b1 * a.max_pages + i] : -1;
            }
        };
        auto take_base = [&] {
            base3 = -1;
            if (r2 >= 0) {
                if (pg2 >= 0 && pg2 < a.P)
                    base3 = ((((int64_t)pg2 * a.Hkv + kvh2) << a.shift) | (r2 & ((1 << a.shift) - 1)));
                else
                    g_page_status = 1;
            }
        };
        // Chunk i of a stage: row ci / CPR of this warp, column ci % CPR (the same in every stage);
        // a lane converts what it copied itself.  In a part: the column block, then the row's
        // swizzled 16-byte chunk of 8 channels.
        uint32_t spot[LD];
#pragma unroll
        for (int i = 0; i < LD; ++i) {
            const int ci = i * 32 + lane, r = warp * LR + ci / CPR, ch = ci % CPR * E;
            spot[i] = (ch >> 6) * (HALF * 128) + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4) + (ch & 7) * 2;
        }
        unsigned char *raw = base + Tile::RAW_AT + (warp * LD * 32 + lane) * 16;
        uint32_t ok = 0;                // bit 8 (stage % 4) + i: chunk i of a stage is a row's;
                                        // bit 7 of them: so are all of this warp's
        // stage q (h-th of its tile) into raw slot `slot`
        auto issue = [&](int h, int slot, uint32_t q) {
            if (h == 0) {
                take_base();
                take_page();
                take_row();
            }
            const uint32_t bit = (q & 3) * 8;
            ok &= ~(0xffu << bit);
            const bool all = (__ballot_sync(0xffffffffu, base3 >= 0) >> (h * LR) & ((1u << LR) - 1)) == (1u << LR) - 1 &&
                             LR * CPR >= 32;
            if (all) ok |= 0x80u << bit;
#pragma unroll
            for (int i = 0; i < LD; ++i) {
                const int ci = i * 32 + lane;
                const int64_t at = __shfl_sync(0xffffffffu, base3, h * LR + (ci / CPR) % LR);
                if (ci < LR * CPR) {
                    const bool on = at >= 0;
                    const int64_t off = ((on ? at : 0) * CPR + ci % CPR) * 16;
                    cp16(tc::smem_u32(raw + slot * Tile::RAW + i * 512),
                         reinterpret_cast<const char *>(k_pages) + off, on);
                    const uint32_t dv = Tile::kWide ? tc::smem_u32(raw + slot * Tile::RAW + Tile::RAW / 2 + i * 512)
                                                    : tc::smem_u32(base + Tile::V_AT + (q & 3) * Tile::KB + spot[i]);
                    cp16(dv, reinterpret_cast<const char *>(v_pages) + off, on);
                    if (!all) ok |= (on ? 1u : 0u) << (bit + i);
                }
            }
        };
        auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
        take_row();
        take_page();
        take_row();
        const int64_t stages = steps * SUB;
        issue(0, 0, 0);
        commit();
        issue(1, 1, 1);                 // (SUB >= 2)
        commit();
        uint64_t zs[E / 2];
#pragma unroll
        for (int x = 0; x < E / 2; ++x) zs[x] = 0;
        Walk at = first;
        int slot = 0;                   // s % 3
        uint32_t s = 0;                 // low bits of the stage's number
        bool alive = warp > 0 || tc::g_paged_test_withhold == 0;   // (a test hook: warp 0 fills no stage)
        int64_t rest = stages;
        for (int64_t left = steps; left > 0 && alive; --left) {
#pragma unroll
            for (int h = 0; h < SUB; ++h, ++s, --rest) {
                // the products of stage s - 2 are done: its parts and its v are free
                const int stage = s & 1;
                if (rest <= stages - 2 && !(alive = wait_all(&empty[stage], ((s >> 1) - 1) & 1, 90))) break;
                if (rest > 2) issue((h + 2) % SUB, slot == 0 ? 2 : slot - 1, s + 2);
                commit();
                asm volatile("cp.async.wait_group 2;" ::: "memory");
                unsigned char *sk = base + stage * Tile::PART, *sv = sk + 3 * Tile::KB;
                const uint32_t on_bits = ok >> ((s & 3) * 8);
#pragma unroll
                for (int i = 0; i < LD; ++i) {
                    const unsigned char *src = raw + slot * Tile::RAW + i * 512;
                    uint4 rk = *reinterpret_cast<const uint4 *>(src);
                    if (!(on_bits >> 7 & 1) && !(on_bits >> i & 1)) {   // no row: sigma(-inf) = 0
                        const uint32_t none = Tile::kWide ? 0xff800000u : 0xff80ff80u;
                        rk = make_uint4(none, none, none, none);
                    }
                    const uint32_t w[4] = {rk.x, rk.y, rk.z, rk.w};
                    uint32_t p[E / 2][3];
#pragma unroll
                    for (int x = 0; x < E / 2; ++x) {
                        uint64_t f;
                        if constexpr (Tile::kWide) f = sigma2(__uint_as_float(w[2 * x]), __uint_as_float(w[2 * x + 1]));
                        else f = sigma2(w[x]);
                        zs[x] = tc::f2_add(zs[x], f);
                        split3(f, p[x]);
                    }
                    if (i * 32 + lane < LR * CPR) {
                        if constexpr (!Tile::kWide) {
#pragma unroll
                            for (int y = 0; y < 3; ++y)
                                *reinterpret_cast<uint4 *>(sk + y * Tile::KB + spot[i]) =
                                    make_uint4(p[0][y], p[1][y], p[2][y], p[3][y]);
                        } else {
                            const uint4 rv = *reinterpret_cast<const uint4 *>(src + Tile::RAW / 2);
                            uint32_t q[2][3];
                            split3(tc::f2_pack(__uint_as_float(rv.x), __uint_as_float(rv.y)), q[0]);
                            split3(tc::f2_pack(__uint_as_float(rv.z), __uint_as_float(rv.w)), q[1]);
#pragma unroll
                            for (int y = 0; y < 3; ++y) {
                                *reinterpret_cast<uint2 *>(sk + y * Tile::KB + spot[i]) = make_uint2(p[0][y], p[1][y]);
                                *reinterpret_cast<uint2 *>(sv + y * Tile::KB + spot[i]) = make_uint2(q[0][y], q[1][y]);
                            }
                        }
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&full[stage]);
                slot = slot == 2 ? 0 : slot + 1;
            }
            if (!alive) break;
            if (left == 1 || at.tile == at.nt - 1) {   // a piece ends: this warp's part of z
                const int64_t slot = blockIdx.x + (int64_t)at.b * a.Hkv + at.kh;
#pragma unroll
                for (int x = 0; x < E / 2; ++x) {
                    float z0, z1;
                    tc::f2_unpack(zs[x], z0, z1);
#pragma unroll
                    for (int off = CPR; off < 32; off <<= 1) {
                        z0 += __shfl_xor_sync(0xffffffffu, z0, off);
                        z1 += __shfl_xor_sync(0xffffffffu, z1, off);
                    }
                    if (lane < CPR) {
                        float *z = e.part_z + (slot * kFoldLoaders + warp) * D + lane * E + 2 * x;
                        z[0] = z0;
                        z[1] = z1;
                    }
                    zs[x] = 0;
                }
            }
            walk_next<0>(at, rows_of, a.Hkv, e.B, Tile::ROWS);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp < kFoldLoaders + kFoldReaders) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // reader w: lanes 32 (w % 4) .. + 31 (key features), half w / 4 of the columns
        const int w = warp - kFoldLoaders, part = warp & 3, half = w >> 2, f = part * 32 + lane;
        constexpr int NC = D / 2;       // columns of a half
        uint64_t acc[NC / 2];           // pairs of columns
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
        Walk at = first;
        for (int64_t t = t0; t < t1; ++t) {
            const int64_t s = t - t0;
            const int buf = (int)(s & 1);
            if (!wait_all(&tfull[buf], (uint32_t)((s >> 1) & 1), 91)) break;
            tc::tc_fence_after();
            if (part * 32 < D) {
                const uint32_t col = tmem + ((uint32_t)(part * 32) << 16) + buf * 2 * D + half * NC;
#pragma unroll
                for (int c = 0; c < NC; c += 16) {
                    uint32_t x[16], y[16];
                    tc::tmem_ld16(col + c, x);
                    tc::tmem_ld16(col + D + c, y);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += 2)
                        acc[(c + i) / 2] = tc::f2_add(
                            acc[(c + i) / 2],
                            tc::f2_add(tc::f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                       tc::f2_pack(__uint_as_float(y[i]), __uint_as_float(y[i + 1]))));
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&tempty[buf]);
            if (t == t1 - 1 || at.tile == at.nt - 1) {
                if (part * 32 < D) {
                    const int64_t unit = (int64_t)at.b * a.Hkv + at.kh;
                    // a head that is this CTA's alone goes into its memory at once
                    const bool whole = t - t0 >= at.nt - 1 && at.tile == at.nt - 1;
                    float4 *dst = whole ? reinterpret_cast<float4 *>(M + unit * D * D + f * D + half * NC)
                                        : reinterpret_cast<float4 *>(e.part_M + (blockIdx.x + unit) * D * D +
                                                                     half * NC * D + f * 4);
#pragma unroll
                    for (int c = 0; c < NC; c += 4) {
                        float4 x;
                        tc::f2_unpack(acc[c / 2], x.x, x.y);
                        tc::f2_unpack(acc[c / 2 + 1], x.z, x.w);
                        float4 *p = dst + (whole ? c / 4 : c / 4 * D);   // pieces: [c / 4][f][4]
                        if (whole) {
                            const float4 y = *p;
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        *p = x;
                    }
                }
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
            }
            walk_next<0>(at, rows_of, a.Hkv, e.B, Tile::ROWS);
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 24;");
      if (warp == kFoldLoaders + kFoldReaders && lane == 0) {
        constexpr uint32_t idesc = tc::idesc_bf16(128, D, 1, 1);
        uint32_t q = 0;                 // the stage's number
        bool alive = true;
        for (int64_t s = 0; s < steps && alive; ++s) {
            const int buf = (int)(s & 1);
            if (s >= 2 && !tc::mbar_wait(&tempty[buf], (uint32_t)(((s >> 1) - 1) & 1), abort, 92)) break;
            const uint32_t d0 = tmem + buf * 2 * D, d1 = d0 + D;
            for (int h = 0; h < SUB; ++h, ++q) {
                if (!(alive = tc::mbar_wait(&full[q & 1], (q >> 1) & 1, abort, 93))) break;
                tc::tc_fence_after();
                const uint32_t sk = tc::smem_u32(base + (q & 1) * Tile::PART);
                const uint32_t sv = Tile::kWide ? sk + 3 * Tile::KB
                                                : tc::smem_u32(base + Tile::V_AT + (q & 3) * Tile::KB);
                uint32_t on = h;
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < VP; ++j) {
                        if (i + j > 2) continue;
                        for (int kk = 0; kk < HALF / 16; ++kk) {
                            const uint64_t da = tc::sdesc_sw128(sk + i * Tile::KB + kk * 2048, HALF * 128, 1024);
                            const uint64_t db = tc::sdesc_sw128(sv + j * Tile::KB + kk * 2048, HALF * 128, 1024);
                            if (i + j == 0) {
                                tc::mma_ss(d0, da, db, idesc, h + kk > 0);
                            } else {
                                tc::mma_ss(d1, da, db, idesc, on);
                                on = 1;
                            }
                        }
                    }
                tc::mma_commit(&empty[q & 1]);
            }
            if (alive) tc::mma_commit(&tfull[buf]);
        }
        // every product issued ends before TMEM is given back, whatever gave up before
        tc::mma_commit(&drained);
        const long long t_end = clock64();
        while (!tc::mbar_try_wait(&drained, 0) && clock64() - t_end < tc::kSpinLimitCycles) {
        }
      }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp == 0) tc::tmem_dealloc(tmem, Tile::COLS);
}

// ---- finish -------------------------------------------------------------------------------------
//
// One grid for what is left: blocks that copy the kept rows (16 bytes per thread and row, four
// rows of keys and values in flight: 207 MB of a batch in 32 us, 6.4 TB/s), and with a memory blocks
// that add the pieces of a head that several CTAs folded, in order, and z of every head.  (Copying
// the rows that need no selection before it ends, from blocks that stay resident, gained nothing:
// the selection leaves them too little of the SMs.)
template <typename T, int D>
__device__ __forceinline__ void move_rows(T *k_pages, T *v_pages, float *weights, const PageArgs &a, const EvictArgs &e,
                                          int64_t block, int blocks)
{
    using Tile = RowTile<T, D>;
    constexpr int CPR = Tile::CPR, LINES = Tile::LINES, ROWS = Tile::ROWS;
    __shared__ int64_t s_from[ROWS], s_to[ROWS];
    const int64_t unit = block / blocks, b = unit / a.Hkv;
    const int j0 = (int)(block % blocks) * ROWS;
    const int kvh = (int)(unit % a.Hkv), n = min(cached_rows(a, b), e.budget), tid = threadIdx.x;
    if (j0 >= n) return;
    PageArgs dst = a;
    dst.table = e.dst_table;
    dst.max_pages = e.dst_pages;
    bool bad = false;
    for (int i = tid; i < ROWS; i += 256) {
        int64_t from = -1, to = -1;
        if (j0 + i < n) {
            to = place_of(dst, e.dst_table + b * e.dst_pages, j0 + i, kvh, bad);
            from = place_of(a, a.table + b * a.max_pages, e.kept[unit * e.budget + j0 + i], kvh, bad);
            if (from < 0 || to < 0 || from == to) from = -1;
            else weights[to] = weights[from];
        }
        s_from[i] = from;
        s_to[i] = to;
    }
    report(bad);
    __syncthreads();
    const int c = tid % CPR, line = tid / CPR;
    uint4 *kp = reinterpret_cast<uint4 *>(k_pages), *vp = reinterpret_cast<uint4 *>(v_pages);
    uint4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t from = s_from[line + u * LINES];
        if (from >= 0) {
            x[u] = __ldcs(kp + from * CPR + c);
            y[u] = __ldcs(vp + from * CPR + c);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t to = s_to[line + u * LINES];
        if (s_from[line + u * LINES] >= 0) {
            kp[to * CPR + c] = x[u];
            vp[to * CPR + c] = y[u];
        }
    }
}

// Block `part` of `parts` of a head: its share of M's float4 columns (32 at a time, eight warps
// over the pieces), the last block z (a warp per eighth of the pieces' loader warps).
template <int D>
__device__ __forceinline__ void add_pieces(const PageArgs &a, const EvictArgs &e, float *M, float *z, int64_t unit,
                                           int64_t c0, int64_t c1, int part, int parts)
{
    // a fold that gave up left pieces unwritten: nothing is added then (threads whose views differ,
    // since another stream's fold gives up meanwhile, part at the stores alone)
    const bool complete = !tc::wait_status_set();
    __shared__ float4 s_sum[256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto total = [&](float4 x) {         // over the eight warps; lane's sum, in warp 0
        s_sum[threadIdx.x] = x;
        __syncthreads();
        if (warp == 0)
#pragma unroll
            for (int w = 1; w < 8; ++w) {
                const float4 y = s_sum[w * 32 + lane];
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
        __syncthreads();
        return x;
    };
    if (part == parts - 1) {
        const float4 *p = reinterpret_cast<const float4 *>(e.part_z) + (c0 + unit) * kFoldLoaders * (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < D / 4)
#pragma unroll 8
            for (int64_t w = warp; w < (c1 - c0 + 1) * kFoldLoaders; w += 8) {
                const float4 y = p[w * (D / 4) + lane];
                x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
        x = total(x);
        if (warp == 0 && lane < D / 4 && complete) {
            float4 *dst = reinterpret_cast<float4 *>(z + unit * D) + lane;
            const float4 y = *dst;
            *dst = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        return;
    }
    if (c0 == c1) return;                // folded in place
    for (int i0 = part * 32; i0 < D * D / 4; i0 += (parts - 1) * 32) {
        const int i = i0 + lane, f = i % D, c4 = i / D;    // [c / 4][f]
        const float4 *p = reinterpret_cast<const float4 *>(e.part_M) + i;
        float4 *dst = reinterpret_cast<float4 *>(M) + (unit * D + f) * (D / 4) + c4;
        float4 old = make_float4(0.f, 0.f, 0.f, 0.f), x = old;
        if (warp == 0) old = *dst;
#pragma unroll 4
        for (int64_t c = c0 + warp; c <= c1; c += 8) {
            const float4 y = p[(c + unit) * (D * D / 4)];
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        x = total(x);
        if (warp == 0 && complete) *dst = make_float4(x.x + old.x, x.y + old.y, x.z + old.z, x.w + old.w);
    }
}

// Blocks 0 .. units * parts - 1 add, the others move (parts = 0: no memory).
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_evict_finish(T *k_pages, T *v_pages, float *weights, PageArgs a, EvictArgs e, float *M, float *z, int64_t units,
               int parts, int blocks)
{
    __shared__ ShareScratch s_share;
    const int64_t adders = units * parts;
    if (blockIdx.x < adders) {
        const int64_t unit = blockIdx.x / parts, b = unit / a.Hkv;
        const int kvh = (int)(unit % a.Hkv);
        auto rows_of = [&](int64_t i) { return rows_leaving(a, e, i); };
        const int64_t nt = share_tiles<0>(rows_of(b), e.fold_rows);
        int64_t before;
        const int64_t total = a.Hkv * share_count<256, 0>(rows_of, e.B, e.fold_rows, b, s_share, before);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (nt == 0) return;
        const int64_t s = before * a.Hkv + kvh * nt;
        add_pieces<D>(a, e, M, z, unit, share_owner<kFoldCtas>(s, total), share_owner<kFoldCtas>(s + nt - 1, total),
                      (int)(blockIdx.x % parts), parts);
        return;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    move_rows<T, D>(k_pages, v_pages, weights, a, e, blockIdx.x - adders, blocks);
}

}  // namespace paged
}  // namespace infini
