// One new token's attention over a paged cache: split over the rows, then joined.
//
// For every query head of a (sequence, key/value head) with rows 0 .. n-1,
//   s_j = q . k_j / sqrt(d),   m = max_j s_j,   l = sum_j e^(s_j - m),   o = sum_j e^(s_j - m) v_j / l.
// A piece of the rows gives (m_i, l_i, o_i) of its own; pieces join by
//   m = max m_i,   l = sum l_i e^(m_i - m),   o = (sum o_i e^(m_i - m)) / l.
//
// The work is read bandwidth: 2 d elements per row against 4 d operations per query head.  So
// the split kernel is one resident wave of CTAs (two per SM) that share all rows of the batch
// evenly (share.cuh); a unit there is a (sequence, key/value head, tile of up to eight query
// heads).  Measured (8 key/value heads, d = 128, bf16): one sequence of 1,000,003 rows 590-605 us,
// 6.8-6.9 TB/s; 32 ragged sequences with memory and weights, 157 MB, 51 us: 7 until the first
// tiles are in, 27 for the rows, then the join; one sequence of 64 rows (d = 64) 8 us, all latency.
#pragma once

#include "paged.cuh"
#include "share.cuh"

namespace infini {
namespace paged {

struct DecodeArgs {
    const float *beta, *M, *z;   // all null: plain attention
    const double *freq;          // null: no rotation
    const int64_t *positions;    // [B], or null: lens
    int H, rot, interleaved;
    float rot_scale;
    int G, HT, hg;               // query heads per kv head; tiles of them; heads per full tile
    int64_t B;
    float *part_o, *part_ml;     // [slots, hg, D], [slots, hg, 2]
    float *scores;               // [P, Hkv, page, G], base-2 scaled (null without weights)
};

constexpr int kSplitCtas = 296;      // two on each of 148 SMs
constexpr int kSplitWarps = 4;
constexpr int kStages = 3;

// A warp stages 4 KB of keys and 4 KB of values at a time.
template <typename T, int D>
struct DecodeTile {
    static constexpr int CPR = D * (int)sizeof(T) / 16;   // 16-byte chunks of a row
    static constexpr int R = 256 / CPR;                   // rows a warp stages
    static constexpr int TR = kSplitWarps * R;            // rows of a tile
    static constexpr int RL = (R + 31) / 32;
    // Chunk c of row r sits at c ^ swz(r), so that eight rows' chunk c lie in eight different
    // groups of four banks.
    static __device__ __forceinline__ int swz(int r) { return CPR >= 8 ? (r & 7) : ((r >> 1) & 3); }
};

// Warps whose sums of a piece lie side by side: as many as the eight-head tile's shared memory holds.
template <typename T>
constexpr int decode_sums(int GT)
{
    return sizeof(T) == 2 && GT == 4 ? 4 : 2;
}

__device__ __forceinline__ int64_t unit_rows(const PageArgs &a, int64_t b, int extra)
{
    const int len = cached_rows(a, b);
    return len < 0 ? 0 : (int64_t)len + extra;
}

// ---- rotation and small pieces ----------------------------------------------------------------

// Rows 0 .. heads - 1 of q, rotated, into sq [heads][D] (rows up to `fill` are set to 0); with k,
// one more row, rotated and rounded to the cache's type, into new_k and v into new_v.  A thread
// turns one pair of channels of every GROUPS-th row.  Two halves: `load` puts all loads in flight,
// `store` uses them, so that other loads can be issued between.
template <typename T, int D, int NT>
struct RowLoad {
    static constexpr int GROUPS = NT / (D / 2), MOST = (9 + GROUPS - 1) / GROUPS;
    float x1[MOST], x2[MOST];
    double freq;
    int64_t pos;
    T y;
    int heads, c1, c2;
    bool fresh, turned;

    __device__ __forceinline__ void load(const T *__restrict__ q, int heads_, const T *k, const T *v, const int64_t *at,
                                         int64_t row, const DecodeArgs &a)
    {
        const int half = a.freq ? a.rot / 2 : 0, i = threadIdx.x % (D / 2), grp = threadIdx.x / (D / 2);
        heads = heads_;
        fresh = k != nullptr;
        turned = i < half;
        const bool cross = turned && !a.interleaved;
        c1 = cross ? i : 2 * i;
        c2 = cross ? i + half : 2 * i + 1;
        pos = at ? *at : row;
        freq = turned ? a.freq[i] : 0.0;
#pragma unroll
        for (int e = 0; e < MOST; ++e) {
            const int g = grp + e * GROUPS;
            const T *src = g < heads ? q + g * D : k;
            x1[e] = x2[e] = 0.f;
            if (g < heads || (g == heads && fresh)) {
                x1[e] = ld_f(src + c1);
                x2[e] = ld_f(src + c2);
            }
        }
        if (fresh && threadIdx.x < D) y = v[threadIdx.x];
    }

    __device__ __forceinline__ void store(int fill, const DecodeArgs &a, float *sq, T *new_k, T *new_v) const
    {
        const int grp = threadIdx.x / (D / 2);
        float2 cs = make_float2(1.f, 0.f);
        if (turned) cs = rotary_turn((double)pos, freq, a.rot_scale);
#pragma unroll
        for (int e = 0; e < MOST; ++e) {
            const int g = grp + e * GROUPS;
            // copied channels stay as they are (a product with 0 would spread infinities)
            const float y1 = turned ? x1[e] * cs.x - x2[e] * cs.y : x1[e];
            const float y2 = turned ? x2[e] * cs.x + x1[e] * cs.y : x2[e];
            const bool last = g == heads && fresh;
            if (last) {
                st_f(new_k + c1, y1);
                st_f(new_k + c2, y2);
            }
            if (g < fill) {                                // zeros past the heads
                sq[g * D + c1] = last ? 0.f : y1;
                sq[g * D + c2] = last ? 0.f : y2;
            }
        }
        if (fresh && threadIdx.x < D) new_v[threadIdx.x] = y;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two values as three bf16 pairs whose sum is x to 2^-25 of it.
__device__ __forceinline__ void parts3(float x, float y, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        p[i] = *reinterpret_cast<const uint32_t *>(&h);
        x -= __bfloat162float(h.x);
        y -= __bfloat162float(h.y);
    }
}

// ---- the split kernel ---------------------------------------------------------------------------
//
// Four warps; each stages its own rows with cp.async three deep (up to 24 KB a warp, 192 KB an
// SM, in flight) and needs no barrier inside a piece.  The stages run on across pieces, so a
// unit's end drains nothing.  Eight warps an SM are all that the accumulators leave room for, so
// instructions count: rows of one page are copied from one address (no shuffles; 1M rows 0.80 to
// 0.65 ms with 32-bit positions), and a piece's q, new row, frequencies and first pages travel
// together.
//
// bf16: products on mma.sync m16n8k16 with the query heads as the 16 rows.  q after rotation and the
// weights e^(s-m) are 32-bit values and enter as three bf16 parts each (two would leave 2^-17 of
// them, which turns the rounding of one output in a thousand and shows in the kept weights).  Up to
// four heads: rows 0-3 hold their first parts, 8-11 the second, 4-7 the third; a head's first two land
// in one thread, which adds the third from the lane 16 further (250000 rows of 8 key/value heads, d =
// 128: 157 us, 160 with two parts; d = 32, where rows are short, 4 million of 2 heads: 230, 209 with
// two).  Up to eight: rows 0-7 and 8-15 hold the first two, and a second product, its rows 8-15
// zero, adds the third (174 us, 163 with two parts).  The tensor rate is no bound here (104 TFLOP/s,
// all 16 rows counted, at full read bandwidth: 18% of the pipe), and a tcgen05 tile of 128 rows would be
// padding but for eight of them, with its operands' way through shared memory and TMEM on top.
//
// fp32: on the CUDA cores, exactly; GT query heads at a time.  A lane forms a quarter of one
// row's dot products, and a float4 column of the values' sum.
template <typename T, int D, int GT>
__global__ void __launch_bounds__(32 * kSplitWarps, 2)
k_paged_split(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v, T *k_pages,
               T *v_pages, PageArgs a, DecodeArgs dc)
{
    using Tile = DecodeTile<T, D>;
    constexpr bool kMma = sizeof(T) == 2;
    constexpr int CPR = Tile::CPR, R = Tile::R, TR = Tile::TR, RL = Tile::RL, NT = 32 * kSplitWarps;
    constexpr int NO = D / 8;                              // mma: accumulator tiles of 8 channels
    constexpr int SUMS = decode_sums<T>(GT);
    constexpr bool kPack = kMma && GT == 4;                // mma: a head's three parts in one product
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float s_m[kSplitWarps][8], s_l[kSplitWarps][8];
    __shared__ __align__(16) T s_new[2][D];
    __shared__ ShareScratch s_share;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    unsigned char *stages = smem;                                                // [warp][stage][8 KB]
    float *sq = reinterpret_cast<float *>(smem + kSplitWarps * kStages * 8192);   // [GT][D]
    float *s_o = sq;                                                             // [SUMS][GT][D], over sq at a piece's end
    int64_t *s_base = reinterpret_cast<int64_t *>(sq + SUMS * GT * D);             // [warp][stage][R]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int extra = k ? 1 : 0, KH = a.Hkv * dc.HT;
    const int64_t cta = blockIdx.x;

    int64_t t0, t1;
    Walk rd;
    auto rows_of = [&](int64_t b) { return unit_rows(a, b, extra); };
    share_begin<kSplitCtas, NT, 1>(rows_of, dc.B, KH, TR, s_share, t0, t1, rd);
    if (t0 >= t1) return;                // the whole CTA
    // tile 0 of a unit has no rows: skipped wherever it is met (`left` counts it all the same)
    int64_t left = t1 - t0;
    if (rd.tile == 0) {
        rd.tile = 1;
        --left;
    }
    if (left == 0) return;
    auto next = [&](Walk &w, int64_t &count) {
        const bool fresh = walk_next<1>(w, rows_of, KH, dc.B, TR);
        --count;
        if (fresh && count > 0) {
            w.tile = 1;
            --count;
        }
        return fresh;
    };
    Walk ld = rd;
    int64_t to_load = left;
    int ld_kvh = ld.kh / dc.HT;
    // a warp's rows of a tile lie in one page, one after the other
    const bool in_page = (1 << a.shift) >= R;

    unsigned char *my = stages + warp * kStages * 8192;
    int64_t *my_base = s_base + warp * kStages * R;
    int pg[RL];
    // page numbers of a tile to load, one tile ahead of their use
    auto fetch_pages = [&](const Walk &w, int64_t count, int (&pg)[RL]) {
        const int *table = a.table + (int64_t)w.b * a.max_pages;
#pragma unroll
        for (int e = 0; e < RL; ++e) {
            pg[e] = -1;
            const int r = (w.tile - 1) * TR + warp * R + lane + 32 * e;
            if (count > 0 && lane + 32 * e < R && r < w.n) {
                const int i = r >> a.shift;
                pg[e] = i < a.max_pages ? table[i] : -1;
            }
        }
    };
    uint32_t spot[8];            // where this lane's chunks of a stage go
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ci = i * 32 + lane, r = ci / CPR, c = ci % CPR;
        spot[i] = (r * CPR + (c ^ Tile::swz(r))) * 16;
    }
    auto issue = [&](int stage, const int (&pg)[RL]) {
        if (to_load > 0) {
            const int r0 = (ld.tile - 1) * TR + warp * R, len = ld.n - extra;
            int64_t base[RL];
#pragma unroll
            for (int e = 0; e < RL; ++e) {
                const int r = r0 + lane + 32 * e;
                base[e] = -1;
                if (lane + 32 * e < R && r < ld.n) {
                    if (pg[e] >= 0 && pg[e] < a.P)
                        base[e] = ((((int64_t)pg[e] * a.Hkv + ld_kvh) << a.shift) | (r & ((1 << a.shift) - 1)));
                    else
                        g_page_status = 1;
                }
                if (lane + 32 * e < R) my_base[stage * R + lane + 32 * e] = base[e];
                if (r >= len) base[e] = -1;                // the new row comes from k and v
            }
            const uint32_t dk = s_u32(my + stage * 8192);
            if (in_page) {
                const int64_t at = __shfl_sync(0xffffffffu, base[0], 0);
                const int64_t off = (at < 0 ? 0 : at * (CPR * 16)) + lane * 16;
                const char *ks = reinterpret_cast<const char *>(k_pages) + off;
                const char *vs = reinterpret_cast<const char *>(v_pages) + off;
                const int chunks = at < 0 ? 0 : min(len - r0, R) * CPR - lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool ok = i * 32 < chunks;
                    // (a chunk past the rows is not read; its address stays inside the pool)
                    cp16(dk + spot[i], ok ? ks + i * 512 : reinterpret_cast<const char *>(k_pages), ok);
                    cp16(dk + spot[i] + 4096, ok ? vs + i * 512 : reinterpret_cast<const char *>(v_pages), ok);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int ci = i * 32 + lane, r = ci / CPR, c = ci % CPR;
                    const int64_t at = __shfl_sync(0xffffffffu, base[RL == 1 ? 0 : (i * 32 / CPR) / 32], r & 31);
                    const int64_t off = (at < 0 ? 0 : at * D) + c * (16 / (int)sizeof(T));
                    cp16(dk + spot[i], k_pages + off, at >= 0);
                    cp16(dk + spot[i] + 4096, v_pages + off, at >= 0);
                }
            }
            if (next(ld, to_load)) ld_kvh = ld.kh / dc.HT;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int kvh = 0, ht = 0, heads = 0, len = 0;
    RowLoad<T, D, NT> rows;
    auto begin_piece = [&] {
        kvh = rd.kh / dc.HT;
        ht = rd.kh % dc.HT;
        heads = min(dc.G - ht * dc.hg, dc.hg);
        len = rd.n - extra;
        const bool fresh = extra && left >= rd.nt - rd.tile;   // the new row is in this piece
        const int64_t at = ((int64_t)rd.b * a.Hkv + kvh) * D;
        rows.load(q + ((int64_t)rd.b * dc.H + (int64_t)kvh * dc.G + ht * dc.hg) * D, heads, fresh ? k + at : nullptr,
                  v + at, dc.positions ? dc.positions + rd.b : nullptr, len, dc);
    };
    {   // the first two tiles' pages and the first piece's rows travel together
        static_assert(kStages == 3, "two tiles are issued ahead");
        int pg2[RL];
        Walk w = ld;
        int64_t count = to_load;
        fetch_pages(w, count, pg);
        next(w, count);
        fetch_pages(w, count, pg2);
        begin_piece();
        issue(0, pg);
        issue(1, pg2);
        fetch_pages(ld, to_load, pg);
    }

    const float sl2 = rsqrtf((float)D) * 1.4426950408889634f;
    float m[kMma ? 1 : GT], l[kMma ? 1 : GT];
    float o[kMma ? NO : GT][4];
    uint32_t qa[kMma ? D / 16 : 1][4], qc[kMma && !kPack ? D / 16 : 1][2];   // first two parts of q, the third
    const bool third = kPack && lane >= 16;                // this lane's rows: third parts, and none
    const uint32_t third_bits = third ? 0xffffffffu : 0u;
    auto place = [&](const uint32_t (&p)[3], uint32_t &top, uint32_t &bottom) {
        top = (p[2] & third_bits) | (p[0] & ~third_bits);
        bottom = p[1] & ~third_bits;
    };
    int stage = 0;

    for (bool begins = true, first = true; left > 0;) {
        issue(stage == 0 ? kStages - 1 : stage - 1, pg);
        fetch_pages(ld, to_load, pg);
        if (begins) {                                      // a piece begins
            if (!first) begin_piece();
            first = false;
            __syncthreads();                               // the last piece's sums have been read
            rows.store(GT, dc, sq, s_new[0], s_new[1]);
            __syncthreads();
            if constexpr (kMma) {
                const float *row = sq + ((lane >> 2) & (GT - 1)) * D + (lane & 3) * 2;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint32_t p[3];
                        parts3(row[i * 16 + 8 * e], row[i * 16 + 8 * e + 1], p);
                        place(p, qa[i][2 * e], qa[i][2 * e + 1]);
                        if constexpr (!kPack) qc[i][e] = p[2];
                    }
            }
#pragma unroll
            for (int g = 0; g < (kMma ? 1 : GT); ++g) {
                m[g] = -INFINITY;
                l[g] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < (kMma ? NO : GT); ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        unsigned char *sk = my + stage * 8192, *sv = sk + 4096;
        const int64_t *bs = my_base + stage * R;
        const int r0 = (rd.tile - 1) * TR + warp * R;
        const int mine = min(R, rd.n - r0);                // rows of this warp (none: <= 0)
        if (extra && r0 <= len && len < r0 + R) {
            // the new row into the stage and its page
            const int j = len - r0;
            const int64_t at = bs[j];
            if (lane < CPR) {
                const uint4 x = reinterpret_cast<const uint4 *>(s_new[0])[lane];
                const uint4 y = reinterpret_cast<const uint4 *>(s_new[1])[lane];
                const int p = j * CPR + (lane ^ Tile::swz(j));
                reinterpret_cast<uint4 *>(sk)[p] = x;
                reinterpret_cast<uint4 *>(sv)[p] = y;
                if (at >= 0 && ht == 0) {
                    reinterpret_cast<uint4 *>(k_pages)[at * CPR + lane] = x;
                    reinterpret_cast<uint4 *>(v_pages)[at * CPR + lane] = y;
                }
            }
            __syncwarp();
        }
        // the rows to attend to: on a good page, or the new one
        uint32_t okay[RL];
#pragma unroll
        for (int e = 0; e < RL; ++e) {
            const int j = lane + 32 * e;
            okay[e] = __ballot_sync(0xffffffffu, j < mine && (bs[j] >= 0 || r0 + j == len));
        }
        if constexpr (kMma) {
            const uint32_t ka = s_u32(sk), va = s_u32(sv);
            for (int rb = 0; rb < R && rb < mine; rb += 16) {
                float s[2][4] = {}, s2[2][4] = {};         // even and odd steps: four chains
                // keys: matrices (rows 0-7, k 0-7), (rows 0-7, k 8-15), (rows 8-15, ...) x 2
                const int kr = rb + ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];
                    ldsm4(ka + (kr * CPR + ((2 * i + kc) ^ Tile::swz(kr))) * 16, b);
                    mma16816(i & 1 ? s2[0] : s[0], qa[i], b[0], b[1]);
                    mma16816(i & 1 ? s2[1] : s[1], qa[i], b[2], b[3]);
                    if constexpr (!kPack) {
                        const uint32_t c[4] = {qc[i][0], 0u, qc[i][1], 0u};
                        mma16816(i & 1 ? s2[0] : s[0], c, b[0], b[1]);
                        mma16816(i & 1 ? s2[1] : s[1], c, b[2], b[3]);
                    }
                }
                const uint32_t live = (RL == 1 ? okay[0] : okay[rb >> 5]) >> (rb & 31);
                float x[2][2], mx = m[0];
#pragma unroll
                for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = n8 * 8 + (lane & 3) * 2 + e;
                        float y = (s[n8][e] + s2[n8][e]) + (s[n8][e + 2] + s2[n8][e + 2]);
                        if constexpr (kPack) y += __shfl_xor_sync(0xffffffffu, y, 16);
                        x[n8][e] = live >> j & 1 ? y * sl2 : -INFINITY;
                        mx = fmaxf(mx, x[n8][e]);
                    }
                if (dc.scores && (lane >> 2) < heads)
#pragma unroll
                    for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = n8 * 8 + (lane & 3) * 2 + e;
                            const int64_t at = bs[rb + j];
                            if ((live >> j & 1) && at >= 0) dc.scores[at * dc.G + ht * dc.hg + (lane >> 2)] = x[n8][e];
                        }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float at = mx == -INFINITY ? 0.f : mx, corr = exp2f(m[0] - at);
                uint32_t pa[4], pc[2];
                float p[2][2];
#pragma unroll
                for (int n8 = 0; n8 < 2; ++n8) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) p[n8][e] = exp2f(x[n8][e] - at);
                    uint32_t w[3];
                    parts3(p[n8][0], p[n8][1], w);
                    place(w, pa[2 * n8], pa[2 * n8 + 1]);
                    pc[n8] = w[2];
                }
                l[0] = l[0] * corr + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
                m[0] = mx;
                if (__any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll
                    for (int i = 0; i < NO; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][e] *= corr;
                }
                // values: matrices (rows 0-7, c 0-7), (rows 8-15, c 0-7), (rows 0-7, c 8-15), ...
                const int vr = rb + (lane & 15), vc = lane >> 4;
#pragma unroll
                for (int i = 0; i < NO / 2; ++i) {
                    uint32_t b[4];
                    ldsm4_t(va + (vr * CPR + ((2 * i + vc) ^ Tile::swz(vr))) * 16, b);
                    mma16816(o[2 * i], pa, b[0], b[1]);
                    mma16816(o[2 * i + 1], pa, b[2], b[3]);
                    if constexpr (!kPack) {
                        const uint32_t c[4] = {pc[0], 0u, pc[1], 0u};
                        mma16816(o[2 * i], c, b[0], b[1]);
                        mma16816(o[2 * i + 1], c, b[2], b[3]);
                    }
                }
            }
        } else {
            const float4 *kf = reinterpret_cast<const float4 *>(sk), *vf = reinterpret_cast<const float4 *>(sv);
            const float4 *qf = reinterpret_cast<const float4 *>(sq);
            const int r = lane & 7, part = lane >> 3;
            for (int rb = 0; rb < R && rb < mine; rb += 8) {
                float s[GT];
#pragma unroll
                for (int g = 0; g < GT; ++g) s[g] = 0.f;
#pragma unroll
                for (int i = 0; i < CPR / 4; ++i) {
                    const int c = 4 * i + part;
                    const float4 y = kf[(rb + r) * CPR + (c ^ r)];
#pragma unroll
                    for (int g = 0; g < GT; ++g) {
                        const float4 w = qf[g * CPR + c];
                        s[g] = fmaf(y.x, w.x, fmaf(y.y, w.y, fmaf(y.z, w.z, fmaf(y.w, w.w, s[g]))));
                    }
                }
                const bool ok = okay[0] >> (rb + r) & 1;          // (R <= 32 here)
                float p[GT];
#pragma unroll
                for (int g = 0; g < GT; ++g) {
                    s[g] += __shfl_xor_sync(0xffffffffu, s[g], 8);
                    s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
                    const float x = ok ? s[g] * sl2 : -INFINITY;
                    if (dc.scores && part == 0 && g < heads && ok && bs[rb + r] >= 0)
                        dc.scores[bs[rb + r] * dc.G + ht * dc.hg + g] = x;
                    float mx = x;
#pragma unroll
                    for (int off = 1; off < 8; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    mx = fmaxf(mx, m[g]);
                    const float at = mx == -INFINITY ? 0.f : mx, corr = exp2f(m[g] - at);
                    p[g] = exp2f(x - at);
                    l[g] = l[g] * corr + p[g];
                    m[g] = mx;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[g][e] *= corr;
                }
                constexpr int RW = 32 / CPR;               // rows of the values read at once
                const int c = lane % CPR, sub = lane / CPR;
#pragma unroll
                for (int j = 0; j < 8 / RW; ++j) {
                    const int row = j * RW + sub;
                    const float4 y = vf[(rb + row) * CPR + (c ^ row)];
#pragma unroll
                    for (int g = 0; g < GT; ++g) {
                        const float w = __shfl_sync(0xffffffffu, p[g], row);
                        o[g][0] = fmaf(w, y.x, o[g][0]);
                        o[g][1] = fmaf(w, y.y, o[g][1]);
                        o[g][2] = fmaf(w, y.z, o[g][2]);
                        o[g][3] = fmaf(w, y.w, o[g][3]);
                    }
                }
            }
        }
        __syncwarp();
        begins = rd.tile == rd.nt - 1;
        if (left == 1 || begins) {                         // a piece ends: join the warps
            if constexpr (kMma) {
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
                l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
                if ((lane & 3) == 0) {
                    s_m[warp][lane >> 2] = m[0];
                    s_l[warp][lane >> 2] = l[0];
                }
            } else {
#pragma unroll
                for (int g = 0; g < GT; ++g) {
#pragma unroll
                    for (int off = 1; off < 8; off <<= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], off);
#pragma unroll
                    for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[g][e] += __shfl_xor_sync(0xffffffffu, o[g][e], off);
                    if (lane == 0) {
                        s_m[warp][g] = m[g];
                        s_l[warp][g] = l[g];
                    }
                }
            }
            __syncthreads();
            auto top = [&](int g) {
                float mx = s_m[0][g];
#pragma unroll
                for (int w = 1; w < kSplitWarps; ++w) mx = fmaxf(mx, s_m[w][g]);
                return mx;
            };
            auto share = [&](int w, int g, float mx) {
                return mx == -INFINITY ? 0.f : exp2f(s_m[w][g] - mx);
            };
#pragma unroll
            for (int turn = 0; turn < kSplitWarps / SUMS; ++turn) {   // SUMS warps, then the others on top of them
                if (warp / SUMS == turn) {
                    float *dst = s_o + warp % SUMS * GT * D;
                    if constexpr (kMma) {
                        const int g = (lane >> 2) & (GT - 1);
                        const float f = share(warp, g, top(g));
#pragma unroll
                        for (int i = 0; i < NO; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float *y = dst + g * D + i * 8 + (lane & 3) * 2 + e;
                                float x = o[i][e] + o[i][e + 2];
                                if constexpr (kPack) x += __shfl_xor_sync(0xffffffffu, x, 16);
                                x *= f;
                                if (!third) *y = turn ? *y + x : x;
                            }
                    } else {
#pragma unroll
                        for (int g = 0; g < GT; ++g) {
                            const float f = share(warp, g, top(g));
                            if (lane < CPR)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float *y = dst + g * D + lane * 4 + e;
                                    *y = turn ? *y + o[g][e] * f : o[g][e] * f;
                                }
                        }
                    }
                }
                __syncthreads();
            }
            const int64_t slot = cta + (int64_t)rd.b * KH + rd.kh;
            float *po = dc.part_o + slot * dc.hg * D;
            for (int i = tid; i < heads * D; i += NT) {
                float y = s_o[i] + s_o[GT * D + i];
                if constexpr (SUMS == 4) y += s_o[2 * GT * D + i] + s_o[3 * GT * D + i];
                po[i] = y;
            }
            if (tid < heads) {
                const float mx = top(tid);
                float ls = 0.f;
#pragma unroll
                for (int w = 0; w < kSplitWarps; ++w) ls = fmaf(s_l[w][tid], share(w, tid, mx), ls);
                dc.part_ml[(slot * dc.hg + tid) * 2] = mx;
                dc.part_ml[(slot * dc.hg + tid) * 2 + 1] = ls;
            }
        }
        next(rd, left);
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
}

// ---- the join -----------------------------------------------------------------------------------
//
// One CTA per (sequence, key/value head) and chunk of rows.  What needs the inputs alone comes
// before the wait for the split kernel: the memory's part of chunk 0, and with weights the rows'
// places and what they have so far.  Then chunk 0 joins the pieces, gates and writes the output,
// and every chunk adds its rows' normalised weights from the kept scores.
// BLOCKS to an SM: two leave the registers that keep most loads in flight (d = 128, 256 units with
// memory and weights: 51 us for the step against 55 with three; 504 units of up to three rows, fp32:
// 28 against 34); three where a unit's memory is small and two would not hold all units at once
// (d = 64, 432 units of one or two rows: 17 against 20).
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 1024;      // rows of a chunk

template <typename T, int D, int BLOCKS>
__global__ void __launch_bounds__(kJoinThreads, BLOCKS)
k_paged_join(const T *__restrict__ q, float *weights, T *__restrict__ out, PageArgs a, DecodeArgs dc, int extra)
{
    constexpr int TR = DecodeTile<T, D>::TR, NT = kJoinThreads, NW = NT / 32, C4 = D / 4, PER = kJoinRows / NT;
    __shared__ __align__(16) float sq[1024];               // 8 rows of q, then the pieces' sums
    extern __shared__ __align__(16) float s_num[];         // [4][hg * D]
    __shared__ float s_den[8], s_mx[8], s_il[8];
    __shared__ ShareScratch s_share;
    const int64_t b = blockIdx.x / a.Hkv;
    const int kvh = (int)(blockIdx.x % a.Hkv), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int KH = a.Hkv * dc.HT;
    const int len = cached_rows(a, b);
    const int64_t n = len < 0 ? 0 : (int64_t)len + extra;
    const int64_t h0 = b * dc.H + (int64_t)kvh * dc.G;
    // every path waits for the split kernel, so that no grid of this stream ends before it
    auto wait_split = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (blockIdx.y > 0 && (int64_t)blockIdx.y * kJoinRows >= n) {
        wait_split();
        return;
    }
    if (len < 0) {
        for (int i = tid; i < dc.G * D; i += NT) st_f(out + h0 * D + i, 0.f);
        wait_split();
        return;
    }
    const int64_t unit_b = b * a.Hkv + kvh;
    const bool mem = dc.M && blockIdx.y == 0;
    RowLoad<T, D, NT> rows;
    auto load_q = [&](int ht, int heads) {
        rows.load(q + (h0 + ht * dc.hg) * D, heads, nullptr, nullptr, dc.positions ? dc.positions + b : nullptr, len, dc);
    };
    if (mem) {
        for (int i = tid; i < D * D / 32; i += NT)         // on its way while q is rotated
            asm volatile("prefetch.global.L2 [%0];" ::"l"(dc.M + unit_b * D * D + i * 32));
        load_q(0, min(dc.G, dc.hg));
    }
    // a thread's rows of a chunk: their places and weights
    int64_t place[PER];
    float so_far[PER];
    auto load_weights = [&](int64_t j0) {
        const int *table = a.table + b * a.max_pages;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int64_t j = j0 + e * NT + tid;
            place[e] = j < n ? place_of(a, table, j, kvh, bad) : -1;
        }
        report(bad);
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int64_t j = j0 + e * NT + tid;
            so_far[e] = place[e] >= 0 && j != len ? weights[place[e]] : 0.f;   // the new row starts at 0
        }
    };
    if (weights) load_weights((int64_t)blockIdx.y * kJoinRows);
    int64_t before;
    auto rows_of = [&](int64_t i) { return unit_rows(a, i, extra); };
    const int64_t total = KH * share_count<NT, 1>(rows_of, dc.B, TR, b, s_share, before);
    const int64_t nt = share_tiles<1>(n, TR);
    for (int ht = 0; ht < dc.HT; ++ht) {
        const int heads = min(dc.G - ht * dc.hg, dc.hg);
        const float beta = mem && tid < heads ? dc.beta[kvh * dc.G + ht * dc.hg + tid] : 0.f;
        if (mem) {
            // num_g = sigma(q_g) M, den_g = sigma(q_g) . z: a warp takes every NW-th row of M,
            // a lane four columns
            if (ht > 0) load_q(ht, heads);
            __syncthreads();
            rows.store(8, dc, sq, nullptr, nullptr);
            __syncthreads();
            for (int i = tid; i < 8 * D; i += NT) sq[i] = i < heads * D ? feature_map(sq[i]) : 0.f;
            __syncthreads();
            constexpr int RW = 32 / C4;                    // rows of M a warp reads at once
            float4 acc[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 *Mf = reinterpret_cast<const float4 *>(dc.M + unit_b * D * D);
            const int c = lane % C4, sub = lane / C4;
#pragma unroll 8
            for (int f = warp * RW + sub; f < D; f += NW * RW) {
                const float4 y = __ldcs(Mf + f * C4 + c);
#pragma unroll
                for (int g = 0; g < 8; ++g)
                    if (g < heads) {
                        const float w = sq[g * D + f];
                        acc[g].x = fmaf(w, y.x, acc[g].x);
                        acc[g].y = fmaf(w, y.y, acc[g].y);
                        acc[g].z = fmaf(w, y.z, acc[g].z);
                        acc[g].w = fmaf(w, y.w, acc[g].w);
                    }
            }
            if (warp < heads) {
                float part = 0.f;
#pragma unroll
                for (int f = lane; f < D; f += 32) part = fmaf(sq[warp * D + f], dc.z[unit_b * D + f], part);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
                if (lane == 0) s_den[warp] = part;
            }
#pragma unroll
            for (int g = 0; g < 8; ++g)
#pragma unroll
                for (int off = C4; off < 32; off <<= 1) {
                    acc[g].x += __shfl_xor_sync(0xffffffffu, acc[g].x, off);
                    acc[g].y += __shfl_xor_sync(0xffffffffu, acc[g].y, off);
                    acc[g].z += __shfl_xor_sync(0xffffffffu, acc[g].z, off);
                    acc[g].w += __shfl_xor_sync(0xffffffffu, acc[g].w, off);
                }
            // warps 4-7, then 0-3 on top of them; the four sums meet at the output
#pragma unroll
            for (int turn = 1; turn >= 0; --turn) {
                if (warp / 4 == turn && lane < C4)
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        if (g < heads) {
                            float4 *y = reinterpret_cast<float4 *>(s_num + (warp & 3) * dc.hg * D + g * D) + lane;
                            float4 x = acc[g];
                            if (turn == 0) {
                                const float4 z = *y;
                                x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
                            }
                            *y = x;
                        }
                __syncthreads();
            }
        }
        if (ht == 0) wait_split();
        // the unit's pieces: CTAs c0 .. c1 of the split kernel (its first tile has no rows)
        const int64_t unit = b * KH + kvh * dc.HT + ht;
        int64_t c0 = 0, c1 = -1;
        if (n > 0) {
            const int64_t s = before * KH + (kvh * dc.HT + ht) * nt;
            c0 = share_owner<kSplitCtas>(s + 1, total);
            c1 = share_owner<kSplitCtas>(s + nt - 1, total);
        }
        __syncthreads();
        if (warp < heads) {
            // (a maximum of -inf: no row, or NaN alone, which stays in the sums)
            float mx = -INFINITY, ls = 0.f;
            auto join = [&](float m, float l) {
                const float top = fmaxf(mx, m);
                ls = (mx == -INFINITY ? ls : ls * exp2f(mx - top)) + (m == -INFINITY ? l : l * exp2f(m - top));
                mx = top;
            };
            for (int64_t c = c0 + lane; c <= c1; c += 32) {
                const float2 ml = reinterpret_cast<const float2 *>(dc.part_ml)[(c + unit) * dc.hg + warp];
                join(ml.x, ml.y);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const float m = __shfl_xor_sync(0xffffffffu, mx, off), l = __shfl_xor_sync(0xffffffffu, ls, off);
                join(m, l);
            }
            if (lane == 0) {
                s_mx[warp] = mx;
                s_il[warp] = ls == 0.f ? 0.f : 1.f / ls;
            }
        }
        __syncthreads();
        if (blockIdx.y == 0) {
            // four columns to a thread; the threads left over take every groups-th piece
            const int cols = heads * C4, groups = NT / cols, col = tid % cols, grp = tid / cols, g = col / C4;
            if (grp < groups) {
                const float mx = s_mx[g];
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 *po = reinterpret_cast<const float4 *>(dc.part_o) + col;
#pragma unroll 8
                for (int64_t c = c0 + grp; c <= c1; c += groups) {
                    const float4 x = po[(c + unit) * dc.hg * C4];
                    const float w = mx == -INFINITY ? 0.f : exp2f(dc.part_ml[((c + unit) * dc.hg + g) * 2] - mx);
                    y = make_float4(fmaf(w, x.x, y.x), fmaf(w, x.y, y.y), fmaf(w, x.z, y.z), fmaf(w, x.w, y.w));
                }
                reinterpret_cast<float4 *>(sq)[grp * cols + col] = y;
            }
            __shared__ float s_gate[8];
            if (mem && tid < heads) s_gate[tid] = 1.f / (1.f + expf(-beta));
            __syncthreads();
            for (int i = tid; i < heads * D; i += NT) {
                const int h = i / D;
                float y = 0.f;
                for (int k = 0; k < groups; ++k) y += sq[k * cols * 4 + i];
                y *= s_il[h];
                if (mem) {
                    const float gt = s_gate[h];
                    const int w = dc.hg * D;
                    const float num = (s_num[i] + s_num[w + i]) + (s_num[2 * w + i] + s_num[3 * w + i]);
                    y = gt * (s_den[h] == 0.f ? 0.f : num / s_den[h]) + (1.f - gt) * y;
                }
                st_f(out + (h0 + ht * dc.hg) * D + i, y);
            }
        }
        if (weights)
            for (int64_t j0 = (int64_t)blockIdx.y * kJoinRows; j0 < n; j0 += (int64_t)gridDim.y * kJoinRows) {
                if (ht > 0 || j0 != (int64_t)blockIdx.y * kJoinRows || dc.HT > 1) load_weights(j0);
                float sum[PER] = {};
                for (int g = 0; g < heads; ++g) {
                    const float mx = s_mx[g], il = s_il[g];
#pragma unroll
                    for (int e = 0; e < PER; ++e)
                        if (place[e] >= 0) {
                            const float x = dc.scores[place[e] * dc.G + ht * dc.hg + g];
                            sum[e] = fmaf(mx == -INFINITY ? 0.f : exp2f(x - mx), il, sum[e]);
                        }
                }
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (place[e] >= 0) {
                        const bool later = ht > 0 && j0 + e * NT + tid == len;   // its other heads' part
                        weights[place[e]] = (later ? weights[place[e]] : so_far[e]) + sum[e];
                    }
            }
    }
}

}  // namespace paged
}  // namespace infini
