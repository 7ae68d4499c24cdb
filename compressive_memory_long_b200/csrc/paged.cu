// Host side of the paged serving entry points: rotary positions, filling the paged cache,
// one new token's attention over it, and eviction from it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>

#include "evict.cuh"
#include "host.h"
#include "infini_attn.h"
#include "paged.cuh"
#include "paged_decode.cuh"
#include "rotary.cuh"

namespace infini {

int take_paged_status(bool &waits, bool &pages)
{
    int v[2] = {0, 0};
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v[0], tc::g_paged_wait_status, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&v[1], paged::g_page_status, sizeof(int)) != cudaSuccess)
        return INFINI_ERR_CUDA;
    waits |= v[0] != 0;
    pages = v[1] != 0;
    if ((v[0] != 0 && cudaMemcpyToSymbol(tc::g_paged_wait_status, &zero, sizeof(int)) != cudaSuccess) ||
        (pages && !waits && cudaMemcpyToSymbol(paged::g_page_status, &zero, sizeof(int)) != cudaSuccess))
        return INFINI_ERR_CUDA;
    return INFINI_OK;
}

int set_paged_wait_limit(long long cycles)
{
    return cudaMemcpyToSymbol(tc::g_paged_spin_limit, &cycles, sizeof(cycles)) == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

int set_paged_withhold(int on)
{
    return cudaMemcpyToSymbol(tc::g_paged_test_withhold, &on, sizeof(on)) == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA;
}

namespace {

using namespace paged;

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

struct Range {
    const void *p;
    int64_t bytes;
    bool written;
};

// Whether some written range overlaps another one (empty and null ranges overlap nothing).
bool clash(std::initializer_list<Range> rs)
{
    for (const Range *x = rs.begin(); x != rs.end(); ++x)
        for (const Range *y = x + 1; y != rs.end(); ++y) {
            if (!(x->written || y->written) || !x->p || !y->p || x->bytes <= 0 || y->bytes <= 0)
                continue;
            const uintptr_t x0 = (uintptr_t)x->p, y0 = (uintptr_t)y->p;
            if (x0 < y0 + (uintptr_t)y->bytes && y0 < x0 + (uintptr_t)x->bytes) return true;
        }
    return false;
}

bool head_dim(int64_t d) { return d == 32 || d == 64 || d == 128; }

// Strides (batch, head, token) of a [B, H, L, d] input: contiguous when none are given.
bool take_strides(const int64_t *given, int64_t H, int64_t L, int64_t d, int64_t out[3])
{
    out[0] = H * L * d;
    out[1] = L * d;
    out[2] = d;
    if (!given) return true;
    for (int i = 0; i < 3; ++i) {
        if (given[i] < 0 || given[i] > ((int64_t)1 << 42)) return false;
        out[i] = given[i];
    }
    return true;
}

int64_t extent_bytes(const int64_t s[3], int64_t B, int64_t H, int64_t L, int64_t d, int64_t es)
{
    return ((B - 1) * s[0] + (H - 1) * s[1] + (L - 1) * s[2] + d) * es;
}

int launched(cudaError_t e = cudaGetLastError()) { return e == cudaSuccess ? INFINI_OK : INFINI_ERR_CUDA; }

// Lets `Kernel` use `bytes` of dynamic shared memory on the current device (asked once each).
template <auto Kernel>
bool opt_in_smem(size_t bytes)
{
    static std::atomic<uint64_t> done_mask{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done_mask.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return false;
    done_mask.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Launches a kernel that may start while the one before it on the stream still runs (it waits
// for that one's end itself).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ---- rotary positions ---------------------------------------------------------------------

bool row_aligned(const void *p, const int64_t s[3], int64_t es)
{
    return aligned(p, 16) && s[0] * es % 16 == 0 && s[1] * es % 16 == 0 && s[2] * es % 16 == 0;
}

template <typename T, int D>
int launch_rotary(const T *q, const T *k, T *q_out, T *k_out, const RotaryArgs &a, int64_t B, bool rows,
                  cudaStream_t st)
{
    TraceScope trace("rotary", st);
    constexpr int N = Vec<T>::N, U = D / (2 * N);
    const bool even = a.interleaved || a.rot / 2 % N == 0;
    if (!rows) {
        const int64_t n = B * a.L * (D / 2);
        k_rotary_pairs<T, D><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(q, k, q_out, k_out, a, n);
        return launched();
    }
    // a thread takes all heads of its token, or fewer, so that the card has threads enough
    const int64_t n = B * a.L * U, heads = a.H + a.Hkv;
    const int64_t groups = std::max<int64_t>(1, std::min((heads + 3) / 4, ((int64_t)148 * 2048 + n - 1) / n));
    const int per = (int)((heads + groups - 1) / groups);
    const dim3 grid((unsigned)((n + 255) / 256), (unsigned)((heads + per - 1) / per));
    if (a.interleaved) k_rotary_rows<T, D, kPairs><<<grid, 256, 0, st>>>(q, k, q_out, k_out, a, n, per);
    else if (even) k_rotary_rows<T, D, kHalves><<<grid, 256, 0, st>>>(q, k, q_out, k_out, a, n, per);
    else k_rotary_rows<T, D, kRagged><<<grid, 256, 0, st>>>(q, k, q_out, k_out, a, n, per);
    return launched();
}

template <typename T>
int rotary(const void *q, const void *k, void *q_out, void *k_out, const double *freq,
           const int64_t *positions, int64_t start, const int64_t *q_strides,
           const int64_t *k_strides, int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t d,
           int64_t rot, int interleaved, float scale, int backward, infini_stream_t stream)
{
    if (!q || !q_out || (k == nullptr) != (k_out == nullptr)) return INFINI_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || L <= 0 || d <= 0 || (k && Hkv <= 0)) return INFINI_ERR_INVALID_ARG;
    if (rot < 0 || rot > d || rot % 2 != 0 || (rot > 0 && !freq)) return INFINI_ERR_INVALID_ARG;
    if (!k) Hkv = 0;
    if (B > (1 << 20) || H > (1 << 16) || Hkv > (1 << 16) || L > ((int64_t)1 << 34) ||
        B * L > ((int64_t)1 << 34) || B * (H + Hkv) * L > ((int64_t)1 << 40))
        return INFINI_ERR_INVALID_ARG;
    const int64_t es = (int64_t)sizeof(T);
    RotaryArgs a{};
    if (!take_strides(q_strides, H, L, d, a.sq) || !take_strides(k_strides, Hkv, L, d, a.sk))
        return INFINI_ERR_INVALID_ARG;
    if (!aligned(q, es) || !aligned(k, es) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
        !aligned(freq, 16) || !aligned(positions, 8))
        return INFINI_ERR_INVALID_ARG;
    const int64_t qb = B * H * L * d * es, kb = B * Hkv * L * d * es;
    const int64_t qx = extent_bytes(a.sq, B, H, L, d, es), kx = k ? extent_bytes(a.sk, B, Hkv, L, d, es) : 0;
    int64_t cq[3], ck[3];
    take_strides(nullptr, H, L, d, cq);
    take_strides(nullptr, Hkv, L, d, ck);
    auto same = [](const int64_t *x, const int64_t *y) { return x[0] == y[0] && x[1] == y[1] && x[2] == y[2]; };
    // in place: a contiguous input that is its own output
    const bool q_in = q == q_out && same(a.sq, cq), k_in = k && k == k_out && same(a.sk, ck);
    if (clash({{q_out, qb, true}, {k_out, kb, true}, {q_in ? nullptr : q, qx, false},
               {k_in ? nullptr : k, kx, false}, {freq, rot / 2 * 8, false},
               {positions, B * L * 8, false}}))
        return INFINI_ERR_INVALID_ARG;
    if (!head_dim(d)) return INFINI_ERR_UNSUPPORTED;
    a.freq = freq;
    a.positions = positions;
    a.start = start;
    a.L = L;
    a.H = (int)H;
    a.Hkv = (int)Hkv;
    a.rot = (int)rot;
    a.interleaved = interleaved != 0;
    a.backward = backward;
    a.scale = scale;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaGetLastError();
    const T *tq = static_cast<const T *>(q), *tk = static_cast<const T *>(k);
    T *oq = static_cast<T *>(q_out), *ok = static_cast<T *>(k_out);
    const bool rows = row_aligned(q, a.sq, es) && (!k || row_aligned(k, a.sk, es));
    switch (d) {
    case 32: return launch_rotary<T, 32>(tq, tk, oq, ok, a, B, rows, st);
    case 64: return launch_rotary<T, 64>(tq, tk, oq, ok, a, B, rows, st);
    default: return launch_rotary<T, 128>(tq, tk, oq, ok, a, B, rows, st);
    }
}

// ---- the paged cache ------------------------------------------------------------------------

// Sizes of a paged cache; `shift` with page = 1 << shift.
int check_pool(int64_t B, int64_t Hkv, int64_t P, int64_t page, int64_t max_pages, int *shift)
{
    if (B <= 0 || Hkv <= 0 || P <= 0 || page <= 0 || max_pages <= 0) return INFINI_ERR_INVALID_ARG;
    if (B > (1 << 20) || Hkv > (1 << 16) || B * Hkv > ((int64_t)1 << 24) || P > ((int64_t)1 << 31) - 1 ||
        page > (1 << 20) || max_pages > ((int64_t)1 << 31) - 1 || max_pages * page > ((int64_t)1 << 30) ||
        B * max_pages > ((int64_t)1 << 40) || P * page * Hkv > ((int64_t)1 << 40))
        return INFINI_ERR_INVALID_ARG;
    if ((page & (page - 1)) != 0) return INFINI_ERR_UNSUPPORTED;
    *shift = 0;
    while (((int64_t)1 << *shift) < page) ++*shift;
    return INFINI_OK;
}

template <typename T>
int paged_append(const void *k, const void *v, const int64_t *k_strides, const int64_t *v_strides,
                 void *k_pages, void *v_pages, float *weights, const int *table, const int *lens,
                 const int *counts, int64_t B, int64_t Hkv, int64_t Tn, int64_t d, int64_t P,
                 int64_t page, int64_t max_pages, infini_stream_t stream)
{
    if (!k || !v || !k_pages || !v_pages || !table || !lens || Tn <= 0 || d <= 0)
        return INFINI_ERR_INVALID_ARG;
    PageArgs a{table, lens, P, (int)max_pages, 0, (int)Hkv};
    const int rc = check_pool(B, Hkv, P, page, max_pages, &a.shift);
    if (rc == INFINI_ERR_INVALID_ARG) return rc;
    if (Tn > ((int64_t)1 << 30) || Hkv * Tn > ((int64_t)1 << 30) || B * Hkv * Tn > ((int64_t)1 << 32))
        return INFINI_ERR_INVALID_ARG;
    const int64_t es = (int64_t)sizeof(T), pool = P * Hkv * page;
    int64_t sk[3], sv[3];
    if (!take_strides(k_strides, Hkv, Tn, d, sk) || !take_strides(v_strides, Hkv, Tn, d, sv))
        return INFINI_ERR_INVALID_ARG;
    if (!aligned(k, es) || !aligned(v, es) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(weights, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(counts, 4))
        return INFINI_ERR_INVALID_ARG;
    if (clash({{k_pages, pool * d * es, true}, {v_pages, pool * d * es, true}, {weights, pool * 4, true},
               {k, extent_bytes(sk, B, Hkv, Tn, d, es), false},
               {v, extent_bytes(sv, B, Hkv, Tn, d, es), false}, {table, B * max_pages * 4, false},
               {lens, B * 4, false}, {counts, B * 4, false}}))
        return INFINI_ERR_INVALID_ARG;
    if (rc != INFINI_OK || !head_dim(d)) return INFINI_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaGetLastError();
    const T *tk = static_cast<const T *>(k), *tv = static_cast<const T *>(v);
    T *kp = static_cast<T *>(k_pages), *vp = static_cast<T *>(v_pages);
    TraceScope trace("paged_append", st);
    const bool rows = row_aligned(k, sk, es) && row_aligned(v, sv, es);
#define APPEND(D, ALIGNED)                                                                          \
    do {                                                                                            \
        const int64_t blocks = (Tn * Hkv + RowTile<T, D>::ROWS - 1) / RowTile<T, D>::ROWS;          \
        if (B * blocks > ((int64_t)1 << 31) - 1) return INFINI_ERR_INVALID_ARG;                     \
        k_paged_append<T, D, ALIGNED><<<(unsigned)(B * blocks), 256, 0, st>>>(                      \
            tk, tv, kp, vp, weights, a, counts, sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], (int)Tn, \
            (uint32_t)blocks);                                                                      \
    } while (0)
    switch (d) {
    case 32: if (rows) APPEND(32, true); else APPEND(32, false); break;
    case 64: if (rows) APPEND(64, true); else APPEND(64, false); break;
    default: if (rows) APPEND(128, true); else APPEND(128, false); break;
    }
#undef APPEND
    return launched();
}

// Pieces' outputs and statistics, and with weights every cached row's scores.
int64_t decode_slots(int64_t B, int64_t H, int64_t Hkv)
{
    return kSplitCtas + B * Hkv * ((H / Hkv + 7) / 8);
}

int64_t decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t d, int64_t P, int64_t page,
                               int with_weights)
{
    const int64_t parts = decode_slots(B, H, Hkv) * std::min<int64_t>(H / Hkv, 8) * (d + 2);
    return (parts + 3) / 4 * 16 + (with_weights ? P * page * H * 4 : 0);
}

template <typename T, int D, int GT>
int launch_decode(const T *q, const T *k, const T *v, T *kp, T *vp, float *weights, T *out, const PageArgs &a,
                  const DecodeArgs &dc, int64_t most_rows, cudaStream_t st)
{
    constexpr size_t smem = kSplitWarps * kStages * (8192 + DecodeTile<T, D>::R * 8) + decode_sums<T>(GT) * GT * D * 4;
    if (!opt_in_smem<k_paged_split<T, D, GT>>(smem)) return INFINI_ERR_CUDA;
    {
        TraceScope trace("paged_split", st);
        k_paged_split<T, D, GT><<<kSplitCtas, 32 * kSplitWarps, smem, st>>>(q, k, v, kp, vp, a, dc);
    }
    const int rc = launched();
    if (rc != INFINI_OK) return rc;
    TraceScope trace("paged_join", st);
    const int64_t units = dc.B * a.Hkv;
    int64_t chunks = 1;
    if (weights)   // no more CTAs than are resident at once (they all wait); a chunk loops over its rows
        chunks = std::max<int64_t>(1, std::min((most_rows + kJoinRows - 1) / kJoinRows, kSplitCtas / units));
    const auto join = D < 128 && units > kSplitCtas ? k_paged_join<T, D, D < 128 ? 3 : 2> : k_paged_join<T, D, 2>;
    return launched(launch_early(join, dim3((unsigned)units, (unsigned)chunks), kJoinThreads,
                                 dc.M ? (size_t)4 * dc.hg * D * 4 : 0, st, q,
                                 weights, out, a, dc, k ? 1 : 0));
}

template <typename T, int D>
int pick_decode(const T *q, const T *k, const T *v, T *kp, T *vp, float *weights, T *out, const PageArgs &a,
                const DecodeArgs &dc, int64_t most_rows, cudaStream_t st)
{
    if constexpr (sizeof(T) == 4) {   // as many heads at a time as there are
        if (dc.hg == 1) return launch_decode<T, D, 1>(q, k, v, kp, vp, weights, out, a, dc, most_rows, st);
        if (dc.hg == 2) return launch_decode<T, D, 2>(q, k, v, kp, vp, weights, out, a, dc, most_rows, st);
    }
    // (bf16: the three parts of up to four heads fill one product's rows)
    if (dc.hg <= 4) return launch_decode<T, D, 4>(q, k, v, kp, vp, weights, out, a, dc, most_rows, st);
    return launch_decode<T, D, 8>(q, k, v, kp, vp, weights, out, a, dc, most_rows, st);
}

template <typename T>
int paged_decode_step(const void *q, const void *k, const void *v, void *k_pages, void *v_pages,
                      const int *table, const int *lens, const float *beta, const float *M,
                      const float *z, float *weights, const double *freq, const int64_t *positions,
                      void *out, void *workspace, int64_t workspace_bytes, int64_t B, int64_t H,
                      int64_t Hkv, int64_t d, int64_t P, int64_t page, int64_t max_pages,
                      int64_t rot, int interleaved, float scale, infini_stream_t stream)
{
    if (!q || !k_pages || !v_pages || !table || !lens || !out || (k == nullptr) != (v == nullptr))
        return INFINI_ERR_INVALID_ARG;
    if ((beta == nullptr) != (M == nullptr) || (beta == nullptr) != (z == nullptr))
        return INFINI_ERR_INVALID_ARG;
    PageArgs a{table, lens, P, (int)max_pages, 0, (int)Hkv};
    const int rc = check_pool(B, Hkv, P, page, max_pages, &a.shift);
    if (rc == INFINI_ERR_INVALID_ARG) return rc;
    if (H <= 0 || H % Hkv != 0 || H > (1 << 16) || B * H > ((int64_t)1 << 31) - 1 || d <= 0 || rot < 0 ||
        rot > d || rot % 2 != 0 || (rot > 0 && !freq))
        return INFINI_ERR_INVALID_ARG;
    const int64_t need = decode_workspace_bytes(B, H, Hkv, d, P, page, weights != nullptr);
    if (workspace_bytes < need || (need > 0 && !workspace)) return INFINI_ERR_INVALID_ARG;
    for (const void *p : {q, k, v, (const void *)k_pages, (const void *)v_pages, (const void *)M, (const void *)z,
                          (const void *)weights, (const void *)freq, (const void *)out, (const void *)workspace})
        if (!aligned(p, 16)) return INFINI_ERR_INVALID_ARG;
    // read one element at a time, and often slices: a layer's gates, a step's positions
    if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(beta, 4) || !aligned(positions, 8))
        return INFINI_ERR_INVALID_ARG;
    const int64_t es = (int64_t)sizeof(T), pool = P * Hkv * page;
    if (clash({{k_pages, pool * d * es, true}, {v_pages, pool * d * es, true}, {weights, pool * 4, true},
               {out, B * H * d * es, true}, {workspace, need, true}, {q, B * H * d * es, false},
               {k, B * Hkv * d * es, false}, {v, B * Hkv * d * es, false},
               {table, B * max_pages * 4, false}, {lens, B * 4, false}, {beta, H * 4, false},
               {M, B * Hkv * d * d * 4, false}, {z, B * Hkv * d * 4, false}, {freq, rot / 2 * 8, false},
               {positions, B * 8, false}}))
        return INFINI_ERR_INVALID_ARG;
    if (rc != INFINI_OK || !head_dim(d)) return INFINI_ERR_UNSUPPORTED;
    DecodeArgs dc{};
    dc.beta = beta;
    dc.M = M;
    dc.z = z;
    dc.freq = rot > 0 ? freq : nullptr;
    dc.positions = positions;
    dc.H = (int)H;
    dc.rot = (int)rot;
    dc.interleaved = interleaved != 0;
    dc.rot_scale = scale;
    dc.G = (int)(H / Hkv);
    dc.HT = (dc.G + 7) / 8;
    dc.hg = std::min(dc.G, 8);
    dc.B = B;
    const int64_t slots = decode_slots(B, H, Hkv);
    dc.part_o = static_cast<float *>(workspace);
    dc.part_ml = dc.part_o + slots * dc.hg * d;
    dc.scores = weights ? dc.part_o + (slots * dc.hg * (d + 2) + 3) / 4 * 4 : nullptr;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaGetLastError();
    const T *tq = static_cast<const T *>(q), *tk = static_cast<const T *>(k), *tv = static_cast<const T *>(v);
    T *kp = static_cast<T *>(k_pages), *vp = static_cast<T *>(v_pages), *to = static_cast<T *>(out);
    const int64_t most = max_pages * page + 1;
    switch (d) {
    case 32: return pick_decode<T, 32>(tq, tk, tv, kp, vp, weights, to, a, dc, most, st);
    case 64: return pick_decode<T, 64>(tq, tk, tv, kp, vp, weights, to, a, dc, most, st);
    default: return pick_decode<T, 128>(tq, tk, tv, kp, vp, weights, to, a, dc, most, st);
    }
}

// The evicted rows of every (batch, kv head), when they go into a memory, and the pieces of
// their sums.
struct EvictSpace {
    int64_t gone, part_M, part_z, bytes;   // offsets of 4-byte words; bytes of all
};

EvictSpace evict_space(int64_t B, int64_t Hkv, int64_t d, int64_t page, int64_t max_pages, int64_t budget,
                       int with_memory)
{
    EvictSpace s{0, 0, 0, 0};
    const int64_t most = max_pages * page - budget;
    if (!with_memory || most <= 0) return s;
    const int64_t slots = kFoldCtas + B * Hkv;
    s.part_M = (B * Hkv * most + 3) / 4 * 4;
    s.part_z = s.part_M + slots * d * d;
    s.bytes = (s.part_z + slots * kFoldLoaders * d) * 4;
    return s;
}

template <typename T, int D, bool FEW>
int launch_fold(const T *kp, const T *vp, const PageArgs &a, EvictArgs &e, float *M, cudaStream_t st)
{
    using Tile = FoldTile<T, D, FEW>;
    e.fold_rows = Tile::ROWS;
    if (!opt_in_smem<k_evict_fold<T, D, FEW>>(Tile::SMEM)) return INFINI_ERR_CUDA;
    TraceScope trace("evict_fold", st);
    return launched(launch_early(k_evict_fold<T, D, FEW>, dim3(kFoldCtas), kFoldThreads, Tile::SMEM, st, kp, vp, a, e, M));
}

template <typename T, int D>
int launch_evict(T *kp, T *vp, float *weights, const PageArgs &a, EvictArgs e, float *M, float *z,
                 int64_t units, int64_t most_rows, cudaStream_t st)
{
    // a cluster while that gives no more CTAs than SMs and each has 2048 rows at the least
    int CS = 1;
    while (CS < 8 && units * CS * 2 <= 148 && most_rows >= 2048 * 2 * CS) CS *= 2;
    const int cap = (int)std::min<int64_t>((most_rows + CS - 1) / CS, kSelectKeys);
    {
        TraceScope trace("evict_select", st);
        if (!opt_in_smem<k_evict_select>((3 * kBins + kSelectKeys) * 4)) return INFINI_ERR_CUDA;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units * CS));
        cfg.blockDim = dim3(kSelectThreads);
        cfg.dynamicSmemBytes = (size_t)(3 * kBins + cap) * 4;
        cfg.stream = st;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)CS;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const int rc = launched(cudaLaunchKernelEx(&cfg, k_evict_select, (const float *)weights, a, e, CS, cap));
        if (rc != INFINI_OK) return rc;
    }
    if (M && e.gone) {
        const int rc = most_rows - e.budget <= kFoldFew ? launch_fold<T, D, true>(kp, vp, a, e, M, st)
                                                         : launch_fold<T, D, false>(kp, vp, a, e, M, st);
        if (rc != INFINI_OK) return rc;
    }
    TraceScope trace("evict_finish", st);
    const int blocks = (e.budget + RowTile<T, D>::ROWS - 1) / RowTile<T, D>::ROWS;
    // adding blocks: some for every SM, at most one per 32 float4 columns, and one for z
    const int parts = M && e.gone ? 1 + (int)std::max<int64_t>(1, std::min<int64_t>(D * D / 128, 1184 / units)) : 0;
    return launched(launch_early(k_evict_finish<T, D>, dim3((unsigned)(units * (blocks + parts))), 256, 0, st, kp, vp,
                                 weights, a, e, M, z, units, parts, blocks));
}

template <typename T>
int paged_evict(void *k_pages, void *v_pages, float *weights, const int *table, const int *lens,
                const int *dst_table, int *lens_out, int *kept, float *M, float *z, void *workspace,
                int64_t workspace_bytes, int64_t B, int64_t Hkv, int64_t d, int64_t P, int64_t page,
                int64_t max_pages, int64_t dst_pages, int64_t budget, int64_t recent, int rule,
                infini_stream_t stream)
{
    if (!k_pages || !v_pages || !weights || !table || !lens || !dst_table || !lens_out || !kept ||
        (M == nullptr) != (z == nullptr))
        return INFINI_ERR_INVALID_ARG;
    if (rule != INFINI_UPDATE_LINEAR && rule != INFINI_UPDATE_DELTA) return INFINI_ERR_INVALID_ARG;
    PageArgs a{table, lens, P, (int)max_pages, 0, (int)Hkv};
    int rc = check_pool(B, Hkv, P, page, max_pages, &a.shift);
    if (rc == INFINI_ERR_INVALID_ARG) return rc;
    if (d <= 0 || budget <= 0 || recent < 0 || recent > budget || dst_pages <= 0 ||
        dst_pages > ((int64_t)1 << 31) - 1 || dst_pages * page < budget ||
        budget > ((int64_t)1 << 30) || B * Hkv * budget > ((int64_t)1 << 33))
        return INFINI_ERR_INVALID_ARG;
    const int64_t es = (int64_t)sizeof(T), pool = P * Hkv * page, units = B * Hkv;
    const EvictSpace space = evict_space(B, Hkv, d, page, max_pages, budget, M != nullptr);
    const int64_t need = space.bytes;
    if (workspace_bytes < need || (need > 0 && !workspace)) return INFINI_ERR_INVALID_ARG;
    for (const void *p : {(const void *)k_pages, (const void *)v_pages, (const void *)weights,
                          (const void *)M, (const void *)z, (const void *)workspace, (const void *)kept})
        if (!aligned(p, 16)) return INFINI_ERR_INVALID_ARG;
    for (const int *p : {table, lens, dst_table, (const int *)lens_out})
        if (!aligned(p, 4)) return INFINI_ERR_INVALID_ARG;
    // lens_out may not be lens: all three kernels still read lens after the first has written lens_out
    if (clash({{k_pages, pool * d * es, true}, {v_pages, pool * d * es, true}, {weights, pool * 4, true},
               {lens_out, B * 4, true}, {kept, units * budget * 4, true}, {M, units * d * d * 4, true},
               {z, units * d * 4, true}, {workspace, need, true}, {table, B * max_pages * 4, false},
               {lens, B * 4, false}, {dst_table, B * dst_pages * 4, false}}))
        return INFINI_ERR_INVALID_ARG;
    if (rc != INFINI_OK || !head_dim(d)) return INFINI_ERR_UNSUPPORTED;
    if (M && rule == INFINI_UPDATE_DELTA) return INFINI_ERR_UNSUPPORTED;
    float *ws = static_cast<float *>(workspace);
    EvictArgs e{};
    e.dst_table = dst_table;
    e.dst_pages = (int)dst_pages;
    e.budget = (int)budget;
    e.recent = (int)recent;
    e.lens_out = lens_out;
    e.kept = kept;
    e.B = B;
    e.gone_stride = max_pages * page - budget;
    if (need > 0) {
        e.gone = reinterpret_cast<int *>(ws);
        e.part_M = ws + space.part_M;
        e.part_z = ws + space.part_z;
    }
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaGetLastError();
    T *kp = static_cast<T *>(k_pages), *vp = static_cast<T *>(v_pages);
    switch (d) {
    case 32: return launch_evict<T, 32>(kp, vp, weights, a, e, M, z, units, max_pages * page, st);
    case 64: return launch_evict<T, 64>(kp, vp, weights, a, e, M, z, units, max_pages * page, st);
    default: return launch_evict<T, 128>(kp, vp, weights, a, e, M, z, units, max_pages * page, st);
    }
}

}  // namespace
}  // namespace infini

using bf16 = __nv_bfloat16;

extern "C" {

#define ROTARY_ENTRY(name, T, backward)                                                            \
    int name(const void *q, const void *k, void *q_out, void *k_out, const double *freq,           \
             const int64_t *positions, int64_t start, const int64_t *q_strides,                    \
             const int64_t *k_strides, int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t d,    \
             int64_t rot, int interleaved, float scale, infini_stream_t stream)                    \
    {                                                                                              \
        return infini::rotary<T>(q, k, q_out, k_out, freq, positions, start, q_strides, k_strides, \
                                 B, H, Hkv, L, d, rot, interleaved, scale, backward, stream);      \
    }
ROTARY_ENTRY(infini_attn_rotary, bf16, 0)
ROTARY_ENTRY(infini_attn_rotary_f32, float, 0)
ROTARY_ENTRY(infini_attn_rotary_bwd, bf16, 1)
ROTARY_ENTRY(infini_attn_rotary_bwd_f32, float, 1)
#undef ROTARY_ENTRY

#define APPEND_ENTRY(name, T)                                                                      \
    int name(const void *k, const void *v, const int64_t *k_strides, const int64_t *v_strides,     \
             void *k_pages, void *v_pages, float *weights, const int32_t *page_table,              \
             const int32_t *lens, const int32_t *counts, int64_t B, int64_t Hkv, int64_t T_new,    \
             int64_t d, int64_t P, int64_t page, int64_t max_pages, infini_stream_t stream)        \
    {                                                                                              \
        return infini::paged_append<T>(k, v, k_strides, v_strides, k_pages, v_pages, weights,      \
                                       page_table, lens, counts, B, Hkv, T_new, d, P, page,        \
                                       max_pages, stream);                                         \
    }
APPEND_ENTRY(infini_attn_paged_append, bf16)
APPEND_ENTRY(infini_attn_paged_append_f32, float)
#undef APPEND_ENTRY

#define DECODE_ENTRY(name, T)                                                                      \
    int name(const void *q, const void *k, const void *v, void *k_pages, void *v_pages,            \
             const int32_t *page_table, const int32_t *lens, const float *beta, const float *M,    \
             const float *z, float *weights, const double *freq, const int64_t *positions,         \
             void *out, void *workspace, int64_t workspace_bytes, int64_t B, int64_t H,            \
             int64_t Hkv, int64_t d, int64_t P, int64_t page, int64_t max_pages, int64_t rot,      \
             int interleaved, float scale, infini_stream_t stream)                                 \
    {                                                                                              \
        return infini::paged_decode_step<T>(q, k, v, k_pages, v_pages, page_table, lens, beta, M,  \
                                            z, weights, freq, positions, out, workspace,           \
                                            workspace_bytes, B, H, Hkv, d, P, page, max_pages,     \
                                            rot, interleaved, scale, stream);                      \
    }
DECODE_ENTRY(infini_attn_paged_decode_step, bf16)
DECODE_ENTRY(infini_attn_paged_decode_step_f32, float)
#undef DECODE_ENTRY

#define EVICT_ENTRY(name, T)                                                                       \
    int name(void *k_pages, void *v_pages, float *weights, const int32_t *page_table,              \
             const int32_t *lens, const int32_t *dst_table, int32_t *lens_out, int32_t *kept,      \
             float *M, float *z, void *workspace, int64_t workspace_bytes, int64_t B, int64_t Hkv, \
             int64_t d, int64_t P, int64_t page, int64_t max_pages, int64_t dst_pages,             \
             int64_t budget, int64_t recent, int update_rule, infini_stream_t stream)              \
    {                                                                                              \
        return infini::paged_evict<T>(k_pages, v_pages, weights, page_table, lens, dst_table,      \
                                      lens_out, kept, M, z, workspace, workspace_bytes, B, Hkv, d, \
                                      P, page, max_pages, dst_pages, budget, recent, update_rule,  \
                                      stream);                                                     \
    }
EVICT_ENTRY(infini_attn_paged_evict, bf16)
EVICT_ENTRY(infini_attn_paged_evict_f32, float)
#undef EVICT_ENTRY

int64_t infini_attn_paged_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t d, int64_t P,
                                                 int64_t page, int with_weights)
{
    if (B <= 0 || Hkv <= 0 || H <= 0 || d <= 0 || P <= 0 || page <= 0) return 0;
    return infini::decode_workspace_bytes(B, H, Hkv, d, P, page, with_weights);
}

int64_t infini_attn_paged_evict_workspace_bytes(int64_t B, int64_t Hkv, int64_t d, int64_t page,
                                                int64_t max_pages, int64_t budget, int with_memory)
{
    if (B <= 0 || Hkv <= 0 || d <= 0 || page <= 0 || max_pages <= 0 || budget <= 0) return 0;
    return infini::evict_space(B, Hkv, d, page, max_pages, budget, with_memory).bytes;
}

}  // extern "C"
