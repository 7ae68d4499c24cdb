"""Rotary positions and the paged cache on the GPU against plain fp64 loops.

Tolerances (u = 2^-24, half a step of fp32; h = half a step of the stored type, 2^-8 for bf16
and u for fp32).  With r = max |x1| + |x2| of a turned pair and s the scale:

* a turned channel: the angle reduced to half turns in [-1, 1] and rounded to fp32 is off by
  at most pi u / 2 < 2u rad, sine and cosine round within 2u, the scale, two products and the
  sum round once each: 8 u s r in all; then h |y| for the store.
* a score: q and k products summed in fp32, d + 2 roundings of at most sum |q k| each, q itself
  off by 8 u s r when rotated, or by 2^-17 of it where it is split into two bf16 parts; all
  multiplied by 1/sqrt(d).  A weight p then is off by a factor of e^(2 delta), delta the score
  error, by 2^-16 where it is split in the same way, and by n + 4 roundings of the sums.
* out: sum p v, so max |v| times the above, and h |out| for the store.
"""
import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
from compressive_memory_long_b200.positions import rotary_frequencies
from tests import _paged_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}


def f64(x):
    return x.detach().to(torch.float64).cpu().numpy()


def close(got, want, tol, what):
    got, want = f64(got), np.asarray(want)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = np.max(np.abs(got - want) - tol) if got.size else 0
    assert worst <= 0, f"{what}: {worst:.3e} over a tolerance of up to {np.max(tol):.3e}"


def ok():
    assert binding.infini_attn_device_status() == 0


def normal(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dt).cuda()


# ---- rotary ---------------------------------------------------------------------------------

def rotary_reference(x, pos, freq, inter, scale, back):
    """x [B, H, L, d] (fp64), pos [B, L]."""
    y = np.empty_like(x)
    for b in range(x.shape[0]):
        for t in range(x.shape[2]):
            y[b, :, t] = ref.rotate(x[b, :, t], pos[b, t], freq, inter, scale, back)
    return y


ROTARY = [  # d, rot, interleaved, L, layout, positions, scale
    (128, 128, False, 37, "heads", "start", 1.0),
    (128, 128, True, 5, "tokens", "start", 1.0),
    (128, 64, False, 9, "fused", "given", 1.25),
    (128, 34, True, 3, "tokens", "given", 1.0),
    (64, 64, True, 33, "fused", "start", 1.0),
    (64, 18, False, 1, "heads", "given", 1.0),
    (64, 2, False, 4, "odd", "given", 0.5),
    (32, 32, False, 130, "odd", "start", 1.0),
    (32, 16, True, 7, "tokens", "start", 1.0),
    (32, 0, False, 6, "heads", "start", 3.0),
]


def lay(x, layout):
    """The same values as a [B, H, L, d] view of another layout."""
    B, H, L, d = x.shape
    if layout == "heads":
        return x.contiguous()
    if layout == "tokens":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "fused":        # slices of one token-major projection of 3 H heads
        buf = torch.full((B, L, 3 * H, d), float("nan"), dtype=x.dtype, device=x.device)
        buf[:, :, H:2 * H] = x.transpose(1, 2)
        return buf[:, :, H:2 * H].transpose(1, 2)
    buf = torch.full((B, L, H * d + 3), float("nan"), dtype=x.dtype, device=x.device)   # rows off 16 bytes
    view = buf[:, :, 1:1 + H * d].unflatten(2, (H, d)).transpose(1, 2)
    view.copy_(x)
    return view


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("back", [False, True], ids=["fwd", "bwd"])
@pytest.mark.parametrize("d,rot,inter,L,layout,positions,scale", ROTARY)
def test_rotary(d, rot, inter, L, layout, positions, scale, back, dtype):
    B, H, Hkv, dt = 2, 6, 3, DT[dtype]
    q, k = normal((B, H, L, d), dt, 1), normal((B, Hkv, L, d), dt, 2)
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(0, rot, 2).double() / max(rot, 1))
    start, given = 1048570, None
    pos = start + np.arange(L)[None].repeat(B, 0)
    if positions == "given":
        given = torch.randint(-100, 1 << 21, (B, L), generator=torch.Generator().manual_seed(3))
        pos, given = given.numpy(), given.cuda()
    call = binding.rotary_backward if back else binding.rotary
    qo, ko = call(lay(q, layout), lay(k, layout), freq.cuda(), positions=given,
                  start=0 if positions == "given" else start, interleaved=inter, scale=scale)
    for name, x, y in (("q", q, qo), ("k", k, ko)):
        want = rotary_reference(f64(x), pos, freq.numpy(), inter, scale, back)
        r = 2 * np.abs(f64(x)).max()
        close(y, want, (8 * U * scale * r if rot else 0) + (HALF[dtype] * np.abs(want) if rot else 0), name)
        if rot < d:
            assert torch.equal(y[..., rot:], x[..., rot:])


def test_rotary_in_place_and_alone():
    q, k = normal((1, 4, 11, 64), torch.bfloat16, 4), normal((1, 2, 11, 64), torch.bfloat16, 5)
    freq, _ = rotary_frequencies(64)
    qo, ko = binding.rotary(q, k, freq)
    alone, none = binding.rotary(q, None, freq)
    assert none is None and torch.equal(alone, qo)
    q2, k2 = q.clone(), k.clone()
    binding.rotary(q2, k2, freq, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_rotary_gradient_against_differences():
    """The map is linear, so a difference quotient of any step is exact up to rounding: for
    g = sum(c y), each dg/dx is (g(x + e) - g(x)) with a unit step, formed in fp64 from outputs
    within 8u|r| each; the values stay below 8, so 2 * 64 channels * 8u * 8 bounds the error."""
    x, c = normal((1, 2, 3, 32), torch.float32, 6), normal((1, 2, 3, 32), torch.float32, 7)
    freq, scale = rotary_frequencies(32, scaling="yarn", factor=8, trained_length=2048)
    kw = dict(start=123456, scale=scale)
    got, _ = binding.rotary_backward(c, None, freq, **kw)
    base = f64(binding.rotary(x, None, freq, **kw)[0])
    for h, t, e in ((0, 0, 0), (1, 2, 5), (0, 1, 16), (1, 0, 31)):
        x2 = x.clone()
        x2[0, h, t, e] += 1
        step = float(x2[0, h, t, e].double() - x[0, h, t, e].double())
        diff = (f64(c) * (f64(binding.rotary(x2, None, freq, **kw)[0]) - base)).sum() / step
        assert abs(diff - float(got[0, h, t, e])) <= 2 * 64 * 8 * U * 8 * scale


def test_rotary_large_grid_and_stream():
    """More tokens than one grid dimension of blocks would hold at one token each, on a stream
    of its own."""
    L = 70001
    q = normal((1, 2, L, 32), torch.bfloat16, 8)
    freq, _ = rotary_frequencies(32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qo, _ = binding.rotary(q, None, freq, stream=s)
    s.synchronize()
    for t in (0, 1, L // 2, L - 1):
        want = ref.rotate(f64(q[0, :, t]), t, f64(freq), False)
        close(qo[0, :, t], want, 8 * U * 8 + HALF["bf16"] * np.abs(want), f"token {t}")


# ---- the paged cache --------------------------------------------------------------------------

class Cache:
    """A pool with more pages than needed, in a random order, every unwritten value NaN."""

    def __init__(self, B, Hkv, d, page, rows, dtype, seed=0, weights=True):
        g = torch.Generator().manual_seed(seed)
        self.per = -(-rows // page)
        self.P = B * self.per + 4
        self.page, self.B, self.Hkv, self.d, self.dtype = page, B, Hkv, d, dtype
        nan = float("nan")
        self.k = torch.full((self.P, Hkv, page, d), nan, dtype=DT[dtype], device="cuda")
        self.v = self.k.clone()
        self.w = torch.full((self.P, Hkv, page), nan, device="cuda") if weights else None
        perm = torch.randperm(self.P, generator=g)
        self.free = perm[B * self.per:].tolist()
        self.table_h = perm[:B * self.per].reshape(B, self.per).to(torch.int32)
        self.table = self.table_h.cuda()

    def fill(self, lens, seed, scale=1.0):
        """Random rows; returns dense [b][Hkv, n, d] fp64 copies of k and v, and weights."""
        rows = []
        for b, n in enumerate(lens):
            n = max(n, 0)
            kk = (normal((self.Hkv, n, self.d), torch.float32, seed + 2 * b) * scale).to(DT[self.dtype])
            vv = normal((self.Hkv, n, self.d), DT[self.dtype], seed + 2 * b + 1)
            ww = torch.rand((self.Hkv, n), generator=torch.Generator().manual_seed(seed + b)).cuda()
            r = torch.arange(n)
            pg, sl = self.table_h[b].long()[r // self.page].cuda(), (r % self.page).cuda()
            self.k[pg, :, sl] = kk.transpose(0, 1)
            self.v[pg, :, sl] = vv.transpose(0, 1)
            if self.w is not None:
                self.w[pg, :, sl] = ww.T
            rows.append((f64(kk), f64(vv), f64(ww)))
        return rows

    def dense(self, pool, b, n, table=None):
        r = torch.arange(n)
        t = (self.table_h if table is None else table)[b].long()
        return f64(pool[t[r // self.page].cuda(), :, (r % self.page).cuda()]).swapaxes(0, 1)


def same_bits(a, b):
    i = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(i), b.view(i))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,T,layout", [(128, 16, 1, "heads"), (128, 64, 70, "tokens"),
                                             (64, 1, 9, "odd"), (32, 8, 33, "fused"), (64, 32, 65, "odd")])
def test_append(d, page, T, layout, dtype):
    B, Hkv = 5, 3
    lens = [0, 5, 17, -1, 30]
    counts = [T, T // 2, 0, T, T + 5]            # a padding entry, a count beyond T
    c = Cache(B, Hkv, d, page, 30 + T + 3, dtype, seed=page)
    k, v = normal((B, Hkv, T, d), DT[dtype], 11), normal((B, Hkv, T, d), DT[dtype], 12)
    want = [x.clone() for x in (c.k, c.v, c.w)]
    for b in range(B):
        for t in range(min(counts[b], T) if lens[b] >= 0 else 0):
            pg, sl = ref.row_at(c.table_h[b].tolist(), lens[b] + t, page, c.P)
            want[0][pg, :, sl], want[1][pg, :, sl], want[2][pg, :, sl] = k[b, :, t], v[b, :, t], 0.0
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    binding.paged_append(lay(k, layout), lay(v, layout), c.k, c.v, c.table, n,
                         counts=torch.tensor(counts, dtype=torch.int32, device="cuda"), weights=c.w)
    for got, x in zip((c.k, c.v, c.w), want):
        assert same_bits(got, x)
    # all T, no weights
    c2 = Cache(B, Hkv, d, page, 30 + T + 3, dtype, seed=page, weights=False)
    binding.paged_append(k, v, c2.k, c2.v, c2.table, n)
    for b in (0, 1, 4):
        np.testing.assert_array_equal(c2.dense(c2.k, b, lens[b] + T)[:, lens[b]:], f64(k[b]))
        np.testing.assert_array_equal(c2.dense(c2.v, b, lens[b] + T)[:, lens[b]:], f64(v[b]))
    ok()


def test_append_leaves_out_bad_pages():
    """Numbers outside the pool and rows past the table are skipped and reported once."""
    c = Cache(2, 2, 32, 8, 24, "f32", seed=1)
    k = normal((2, 2, 30, 32), torch.float32, 13)
    table = c.table.clone()
    table[0, 1], table[1, 2] = -7, c.P
    before = [x.clone() for x in (c.k, c.v)]
    binding.paged_append(k, k, c.k, c.v, table, torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert binding.infini_attn_device_status() == 6
    ok()
    for b, i in ((0, 0), (0, 2), (1, 0), (1, 1)):
        pg = int(table[b, i])
        assert torch.equal(c.k[pg], k[b, :, 8 * i:8 * i + 8])
        before[0][pg] = before[1][pg] = k[b, :, 8 * i:8 * i + 8]
    assert same_bits(c.k, before[0]) and same_bits(c.v, before[1])


def run_decode(c, q, k, v, lens, table=None, **kw):
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return binding.paged_decode_step(q, k, v, c.k, c.v, c.table if table is None else table, n, **kw)


def check_decode(c, rows, q, k, v, lens, out, before_w=None, beta=None, M=None, z=None, freq=None,
                 positions=None, inter=False, scale=1.0):
    """Every head of every sequence against the definition; the cache's new rows; the weights."""
    B, H, d = q.shape
    G, dt = H // c.Hkv, c.dtype
    kr, vr = f64(q), None
    for b in range(B):
        n = lens[b]
        if n < 0:
            assert not out[b].any()
            continue
        pos = n if positions is None else int(positions[b])
        qb = f64(q[b])
        eq = 0.0
        if freq is not None:
            eq = 8 * U * scale * 2 * np.abs(qb).max()
            qb = ref.rotate(qb, pos, f64(freq), inter, scale)
        if dt == "bf16":
            eq += 2.0 ** -17 * np.abs(qb).max()
        K, V, W = rows[b]
        if k is not None:
            new_k, new_v = c.dense(c.k, b, n + 1)[:, n], c.dense(c.v, b, n + 1)[:, n]
            kb = f64(k[b])
            want = kb if freq is None else ref.rotate(kb, pos, f64(freq), inter, scale)
            tol = 0 if freq is None else 8 * U * scale * 2 * np.abs(kb).max() + HALF[dt] * np.abs(want)
            assert np.all(np.abs(new_k - want) <= tol)
            np.testing.assert_array_equal(new_v, f64(v[b]))
            K = np.concatenate([K, new_k[:, None]], 1)      # what the cache now holds
            V = np.concatenate([V, new_v[:, None]], 1)
            np.testing.assert_array_equal(c.dense(c.k, b, n), K[:, :n])
            np.testing.assert_array_equal(c.dense(c.v, b, n), V[:, :n])
        m = K.shape[1]
        acc = np.zeros((c.Hkv, m))
        p_tol = 0.0
        for h in range(H):
            g = h // G
            o, p = ref.attend(qb[h], K[g], V[g])
            acc[g] += p
            tol = 0.0
            if m:
                delta = ((d + 2) * U * np.abs(qb[h]) @ np.abs(K[g]).T + eq * np.abs(K[g]).sum(1)).max() / np.sqrt(d)
                p_tol = max(p_tol, 2.02 * delta + 2.0 ** -16 * (dt == "bf16") + (m + 4) * U)
                tol = np.abs(V[g]).max() * (2.02 * delta + 2.0 ** -16 * (dt == "bf16") + (m + 4) * U)
            if M is not None:
                f = ref.sigma(qb[h])
                den = f @ f64(z[b, g])
                mem = f @ f64(M[b, g]) / den if den != 0 else np.zeros(d)
                gate = 1 / (1 + np.exp(-float(beta[h])))
                o = gate * mem + (1 - gate) * o
                # sigma is off by eq + 3 roundings of at most 1 + |q|, the sums by d roundings
                tol = tol + gate * (d + 8 + (eq / U)) * U * 4 * np.abs(f64(M[b, g])).max() / \
                    max(f64(z[b, g]).min(), 1e-30) + 8 * U * np.abs(mem).max()
            close(out[b, h], o, tol + HALF[dt] * np.abs(o), f"out[{b}, {h}] of {m} rows")
        if before_w is not None:
            old = np.concatenate([W, np.zeros((c.Hkv, m - n))], 1) if m > n else W
            got = c.dense(c.w, b, m)
            assert np.all(np.abs(got - old - acc) <= p_tol * acc + 2 * U * (old + acc) + 1e-30)


DECODE = [  # d, H, Hkv, page, lens
    (128, 4, 1, 16, [0, 1, 15, 16, 17, 63, 64, 65]),
    (128, 8, 2, 64, [130, -1, 1000, 0, 333]),
    (128, 16, 1, 32, [77, 300]),                    # more query heads than one tile holds
    (128, 12, 4, 8, [40, 41]),                      # groups of three
    (64, 4, 4, 1, [9, 33, 0]),
    (64, 20, 2, 128, [127, 128, 129, 500]),         # groups of ten
    (64, 2, 2, 16, [2047]),
    (32, 2, 2, 32, [31, 4, 95, 1500]),
    (32, 24, 1, 64, [200]),
    (128, 1, 1, 16, [5000]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,H,Hkv,page,lens", DECODE)
def test_decode_step(d, H, Hkv, page, lens, dtype):
    """New row, attention, weights, memory and rotation together, odd lengths and groups, with
    NaN in every row that is not the sequence's own."""
    B = len(lens)
    c = Cache(B, Hkv, d, page, max(lens) + 1, dtype, seed=d + H)
    rows = c.fill(lens, 100)
    q, k, v = (normal((B, n, d), DT[dtype], 20 + i) for i, n in enumerate((H, Hkv, Hkv)))
    M = torch.rand((B, Hkv, d, d), generator=torch.Generator().manual_seed(4)).cuda()
    z = 1 + torch.rand((B, Hkv, d), generator=torch.Generator().manual_seed(5)).cuda()
    beta = normal((H,), torch.float32, 6)
    freq, scale = rotary_frequencies(d // 2, scaling="yarn", factor=4, trained_length=2048)
    positions = torch.arange(B, dtype=torch.int64).cuda() * 100003 + 7
    kw = dict(beta=beta, M=M, z=z, freq=freq, positions=positions, scale=scale)
    out = run_decode(c, q, k, v, lens, weights=c.w, interleaved=True, **kw)
    ok()
    check_decode(c, rows, q, k, v, lens, out, before_w=True, inter=True, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,H,Hkv,page,lens", DECODE)
def test_decode_plain_and_read_only(d, H, Hkv, page, lens, dtype):
    """No memory, rotation or weights; then the same rows read again without a new token."""
    B = len(lens)
    c = Cache(B, Hkv, d, page, max(lens) + 1, dtype, seed=d, weights=False)
    rows = c.fill(lens, 200)
    q, k, v = (normal((B, n, d), DT[dtype], 30 + i) for i, n in enumerate((H, Hkv, Hkv)))
    before = c.k.clone()
    out = run_decode(c, q, None, None, lens)
    assert same_bits(before, c.k)
    check_decode(c, rows, q, None, None, lens, out)
    out = run_decode(c, q, k, v, lens)
    check_decode(c, rows, q, k, v, lens, out)
    more = [n + 1 if n >= 0 else -1 for n in lens]
    assert torch.equal(run_decode(c, q, None, None, more), out)    # the appended row reads the same
    ok()


def test_decode_without_rows_or_memory():
    """No rows: 0, and with a memory the gated retrieval alone; an empty memory reads 0."""
    c = Cache(2, 2, 64, 16, 16, "f32", weights=False)
    q = normal((2, 4, 64), torch.float32, 40)
    assert not run_decode(c, q, None, None, [0, -1]).any()
    beta = normal((4,), torch.float32, 41)
    M, z = torch.rand((2, 2, 64, 64)).cuda(), torch.rand((2, 2, 64)).cuda() + 1
    kw = dict(beta=beta, M=M, z=z)
    check_decode(c, [(np.zeros((2, 0, 64)),) * 2 + (None,)] * 2, q, None, None, [0, 0],
                 run_decode(c, q, None, None, [0, 0], **kw), **kw)
    zero = dict(beta=beta, M=torch.zeros_like(M), z=torch.zeros_like(z))
    rows = c.fill([5, 9], 300)
    check_decode(c, rows, q, None, None, [5, 9], run_decode(c, q, None, None, [5, 9], **zero), **zero)
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_large_scores(dtype):
    """Scores up to several hundred: the running maximum carries them."""
    lens = [300, 64]
    c = Cache(2, 2, 64, 16, 301, dtype, weights=False)
    rows = c.fill(lens, 400, scale=30.0)
    q = normal((2, 8, 64), DT[dtype], 42)
    out = run_decode(c, q, None, None, lens)
    check_decode(c, rows, q, None, None, lens, out)


def test_decode_leaves_out_bad_pages():
    """Rows on pages outside the pool carry no weight; a new row without a place is attended
    but not stored; both are reported."""
    c = Cache(2, 2, 64, 8, 32, "f32", weights=False)
    rows = c.fill([30, 32], 500)
    q, k, v = (normal((2, n, 64), torch.float32, 50 + n) for n in (4, 2, 2))
    table = c.table.clone()
    table[0, 1] = 1 << 30
    before = c.k.clone()
    out = run_decode(c, q, k, v, [30, 32], table=table)
    assert binding.infini_attn_device_status() == 6
    ok()
    for b, drop in ((0, range(8, 16)), (1, ())):
        for h in range(4):
            g = h // 2
            K, V = (np.concatenate([np.delete(x[g], list(drop), 0), f64(y[b, g])[None]])
                    for x, y in zip(rows[b], (k, v)))
            close(out[b, h], ref.attend(f64(q[b, h]), K, V)[0], 64 * U * 40, f"{b} {h}")
    pg, sl = int(table[0, 3]), 30 % 8
    before[pg, :, sl] = k[0]
    assert same_bits(before, c.k)
    # a length beyond the table: the rows that exist
    out = run_decode(c, q, None, None, [30, 1000000])
    assert binding.infini_attn_device_status() == 6
    close(out[1, 0], ref.attend(f64(q[1, 0]), rows[1][0][0], rows[1][1][0])[0], 64 * U * 40, "long")


def test_decode_shared_pages():
    """Two sequences with a common prefix on the same pages."""
    c = Cache(2, 2, 128, 16, 80, "bf16", weights=False)
    rows = c.fill([70, 32], 600)
    table = c.table.clone()
    table[1, :2] = table[0, :2]
    q = normal((2, 8, 128), torch.bfloat16, 60)
    out = run_decode(c, q, None, None, [70, 32], table=table)
    check_decode(c, [rows[0], tuple(x[:, :32] for x in rows[0])], q, None, None, [70, 32], out)


def test_decode_captured_and_two_at_once():
    """A captured step replayed with other lengths, tables and inputs in the same buffers; then
    two steps of different batches at once on two streams, many times, against their own."""
    def make(seed, lens):
        c = Cache(len(lens), 2, 128, 16, 700, "bf16", seed=seed)
        rows = c.fill([700] * len(lens), seed)
        q, k, v = (normal((len(lens), n, 128), torch.bfloat16, seed + n) for n in (8, 2, 2))
        return c, rows, q, k, v, torch.tensor(lens, dtype=torch.int32, device="cuda")

    c, rows, q, k, v, lens = make(700, [5, 600, 0])
    out = torch.empty_like(q)
    step = lambda: binding.paged_decode_step(q, k, v, c.k, c.v, c.table, lens, weights=c.w, out=out)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for new in ([5, 600, 0], [650, 1, 99], [-1, 300, 301]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(normal(q.shape, torch.bfloat16, sum(new)))
        rows = c.fill(new, 900)
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_decode(c, rows, q, k, v, new, out, before_w=True)
    a, b = make(710, [690, 5]), make(720, [300, 400])
    want = [binding.paged_decode_step(*x[2:5], x[0].k, x[0].v, x[0].table, x[5]) for x in (a, b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[binding.paged_decode_step(*x[2:5], x[0].k, x[0].v, x[0].table, x[5], stream=st)
            for x, st in zip((a, b), s)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])
    ok()


# ---- eviction -----------------------------------------------------------------------------------

def evict_case(lens, Hkv, d, page, budget, recent, dtype, weights="random", fold=False, seed=0):
    B = len(lens)
    c = Cache(B, Hkv, d, page, max(max(lens), 1), dtype, seed=seed)
    rows = c.fill(lens, 1000 + seed)
    extra = -(-budget // page)
    # destination pages of their own at the pool's end
    more = torch.full((B * extra, Hkv, page, d), float("nan"), dtype=DT[dtype], device="cuda")
    c.k, c.v = torch.cat([c.k, more]), torch.cat([c.v, more])
    c.w = torch.cat([c.w, torch.full((B * extra, Hkv, page), float("nan"), device="cuda")])
    dst = torch.randperm(B * extra, generator=torch.Generator().manual_seed(seed)).reshape(B, extra) + c.P
    c.P += B * extra
    dst = dst.to(torch.int32)
    if weights != "random":
        for b, n in enumerate(lens):
            w = torch.zeros((Hkv, max(n, 0)))
            if weights == "ties":
                w = torch.randint(0, 3, w.shape, generator=torch.Generator().manual_seed(b)).float()
            elif weights == "odd" and n > 8:
                w = torch.randn(w.shape, generator=torch.Generator().manual_seed(b))
                w[:, 1], w[:, 3], w[:, 5], w[:, 6], w[:, 7] = float("nan"), float("inf"), -float("inf"), 0.0, -0.0
            r = torch.arange(max(n, 0))
            c.w[c.table_h[b].long()[r // page].cuda(), :, (r % page).cuda()] = w.T.cuda()
            rows[b] = rows[b][:2] + (w.double().numpy(),)
    M = z = None
    if fold:
        M = torch.rand((B, Hkv, d, d), generator=torch.Generator().manual_seed(8)).cuda()
        z = torch.rand((B, Hkv, d), generator=torch.Generator().manual_seed(9)).cuda()
    before = [x.clone() for x in (c.k, c.v, c.w)]
    M0, z0 = (None, None) if M is None else (f64(M), f64(z))
    n_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
    lens_out, kept = binding.paged_evict(c.k, c.v, c.w, c.table, n_dev, dst.cuda(), budget=budget,
                                         recent=recent, M=M, z=z)
    ok()
    assert lens_out.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        for h in range(Hkv):
            K, V, W = (x[h] for x in rows[b])
            want = ref.select(W, budget, recent)
            m = len(want)
            assert kept[b, h].tolist() == want + [-1] * (budget - m)
            for i, r in enumerate(want):         # bit for bit into the destination rows
                (pg, sl), (po, so) = (int(dst[b, i // page]), i % page), ref.row_at(c.table_h[b].tolist(), r, page, c.P)
                for x in before:
                    x[pg, h, sl] = x[po, h, so]
            if fold:
                gone = [r for r in range(max(n, 0)) if r not in set(want)]
                f = ref.sigma(K[gone])
                # sigma rounds within 4u (2^-17 more where it is split in two bf16 parts), the
                # products are summed with at most count + 2 roundings
                e = 4 * U + 2.0 ** -17 * (dtype == "bf16") + (len(gone) + 2) * U
                dM = f.T @ V[gone]
                close(M[b, h], M0[b, h] + dM, e * (f.T @ np.abs(V[gone])) + U * (2 * np.abs(M0[b, h]) + np.abs(dM)), "M")
                close(z[b, h], z0[b, h] + f.sum(0), e * f.sum(0) + 2 * U * (z0[b, h] + f.sum(0)), "z")
    for got, x in zip((c.k, c.v, c.w), before):
        assert same_bits(got, x)                 # every other row as it was


EVICT = [  # lens, Hkv, d, page, budget, recent
    ([100, 33, 32, 31, 0, -1], 2, 64, 8, 32, 8),
    ([1000, 5], 3, 128, 64, 130, 0),
    ([513], 1, 32, 1, 100, 100),             # the recent rows alone
    ([2050, 2049], 2, 128, 16, 2048, 7),     # one or two rows leave
    ([5000], 1, 64, 128, 1, 0),
    ([3001, 1200], 2, 32, 32, 1025, 1),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weights", ["random", "ties", "zero", "odd"])
@pytest.mark.parametrize("lens,Hkv,d,page,budget,recent", EVICT)
def test_evict(lens, Hkv, d, page, budget, recent, weights, dtype):
    evict_case(lens, Hkv, d, page, budget, recent, dtype, weights)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hkv,d,page,budget,recent", EVICT)
def test_evict_into_the_memory(lens, Hkv, d, page, budget, recent, dtype):
    evict_case(lens, Hkv, d, page, budget, recent, dtype, fold=True, seed=3)


def test_evict_short_sequences_keep_their_pages():
    """Destination pages that are the sequence's own: nothing moves while it fits."""
    c = Cache(2, 2, 64, 8, 24, "bf16")
    c.fill([20, 24], 50)
    before = [x.clone() for x in (c.k, c.v, c.w)]
    lens = torch.tensor([20, 24], dtype=torch.int32, device="cuda")
    lens_out, kept = binding.paged_evict(c.k, c.v, c.w, c.table, lens, c.table, budget=24, recent=3)
    assert lens_out.tolist() == [20, 24] and kept[0, 0].tolist() == list(range(20)) + [-1] * 4
    for x, y in zip(before, (c.k, c.v, c.w)):
        assert same_bits(x, y)
    ok()


def test_evict_leaves_out_bad_pages():
    """A source or destination page outside the pool is skipped and reported."""
    c = Cache(1, 1, 32, 8, 32, "f32")
    c.fill([32], 60)
    table, dst = c.table.clone(), torch.tensor([[c.free[0], -1]], dtype=torch.int32, device="cuda")
    table[0, 0] = c.P + 3
    before = c.k.clone()
    lens = torch.tensor([32], dtype=torch.int32, device="cuda")
    _, kept = binding.paged_evict(c.k, c.v, c.w, table, lens, dst, budget=16, recent=0)
    assert binding.infini_attn_device_status() == 6
    ok()
    rows = kept[0, 0].tolist()
    assert min(rows) >= 8                       # rows without a page go first
    for i in range(8):
        pg, sl = ref.row_at(table[0].tolist(), rows[i], 8, c.P)
        before[c.free[0], 0, i] = before[pg, 0, sl]
    assert same_bits(before, c.k)


# ---- together -------------------------------------------------------------------------------

@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 2)])
def test_prefill_pages_and_steps_give_the_forward(d, H, Hkv):
    """A prompt through rotary, the forward (one segment) and the pages, then tokens one at a
    time with their own rotation: each step gives the forward's output of that token, and the
    weights sum to the group's size per step.  Both sides round their output to bf16 (2^-8 each)
    and the forward rounds its softmax weights and the memory's part to bf16 before the products
    (2^-8 of max |v| each): 4 * 2^-8 * max |v| in all."""
    L, L0, page = 128, 100, 16
    x = [normal((1, L, n, d), torch.bfloat16, 80 + i) for i, n in enumerate((H, Hkv, Hkv))]
    q, k, v = (t.transpose(1, 2) for t in x)
    freq, _ = rotary_frequencies(d)
    qr, kr = binding.rotary(q, k, freq)
    beta = torch.full((H,), -30.0, device="cuda")          # the gate closed: local attention alone
    out, _, _ = binding.forward(qr, kr, v.contiguous(), beta, N=L)
    c = Cache(1, Hkv, d, page, L, "bf16")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.paged_append(kr[:, :, :L0], v[:, :, :L0], c.k, c.v, c.table, lens, weights=c.w)
    lens += L0
    for t in range(L0, L):
        got = binding.paged_decode_step(q[:, :, t].contiguous(), k[:, :, t].contiguous(), v[:, :, t].contiguous(),
                                        c.k, c.v, c.table, lens, weights=c.w, freq=freq)
        lens += 1
        assert float((got.float() - out[:, :, t].float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    np.testing.assert_array_equal(c.dense(c.k, 0, L), f64(kr[0]))
    w = c.dense(c.w, 0, L).sum(1)
    np.testing.assert_allclose(w, (L - L0) * H // Hkv, rtol=(L + 8) * 2 * U + 2.0 ** -16)
    ok()


def test_steps_with_eviction_into_the_memory():
    """A stream decoded with a budget: whenever a sequence reaches 40 rows it is cut to 24 on
    other pages, the rest going into the memory its later steps read.  Every step is checked
    against fp64 on the cache and memory as they stand, every cut against the definition."""
    B, H, Hkv, d, page, cap, budget, recent = 2, 4, 2, 64, 8, 40, 24, 8
    per = cap // page
    P = 2 * B * per
    kp = torch.full((P, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp, wp = kp.clone(), torch.full((P, Hkv, page), float("nan"), device="cuda")
    tables = [torch.arange(B * per, dtype=torch.int32).reshape(B, per) + i * B * per for i in (0, 1)]
    M, z = torch.zeros((B, Hkv, d, d), device="cuda"), torch.zeros((B, Hkv, d), device="cuda")
    beta, (freq, _) = normal((H,), torch.float32, 90), rotary_frequencies(d)
    n, lens = 0, torch.zeros(B, dtype=torch.int32, device="cuda")
    c = Cache.__new__(Cache)
    c.page, c.B, c.Hkv, c.d, c.dtype, c.k, c.v, c.w, c.P = page, B, Hkv, d, "bf16", kp, vp, wp, P
    for t in range(75):
        c.table_h = tables[0]
        q, k, v = (normal((B, m, d), torch.bfloat16, 1000 + 3 * t + i) for i, m in enumerate((H, Hkv, Hkv)))
        rows = [(c.dense(kp, b, n), c.dense(vp, b, n), c.dense(wp, b, n)) for b in range(B)]
        pos = torch.full((B,), t, dtype=torch.int64, device="cuda")
        kw = dict(beta=beta, M=M, z=z, freq=freq, positions=pos)
        out = binding.paged_decode_step(q, k, v, kp, vp, tables[0].cuda(), lens, weights=wp, **kw)
        if t % 8 == 0 or n in (0, budget, cap - 1):
            check_decode(c, rows, q, k, v, [n] * B, out, before_w=True, **kw)
        n, lens = n + 1, lens + 1
        if n == cap:
            old = [(c.dense(kp, b, n), c.dense(vp, b, n), c.dense(wp, b, n)) for b in range(B)]
            M0, z0 = f64(M), f64(z)
            lens, kept = binding.paged_evict(kp, vp, wp, tables[0].cuda(), lens, tables[1].cuda(),
                                             budget=budget, recent=recent, M=M, z=z)
            tables.reverse()
            n = budget
            assert lens.tolist() == [n] * B
            for b in range(B):
                for h in range(Hkv):
                    want = ref.select(old[b][2][h], budget, recent)
                    assert kept[b, h].tolist() == want
                    np.testing.assert_array_equal(c.dense(kp, b, n, tables[0])[h], old[b][0][h][want])
                    gone = sorted(set(range(cap)) - set(want))
                    f, V = ref.sigma(old[b][0][h][gone]), old[b][1][h][gone]
                    e = 4 * U + 2.0 ** -17 + 18 * U
                    close(M[b, h], M0[b, h] + f.T @ V, e * (f.T @ np.abs(V)) + 2 * U * np.abs(M0[b, h]) + U * np.abs(f.T @ V), "M")
                    close(z[b, h], z0[b, h] + f.sum(0), e * f.sum(0) + 2 * U * (z0[b, h] + f.sum(0)), "z")
    ok()
