"""The paged operators where their work is shared out or laid out differently: batches larger than
a block, more tiles than CTAs, selection over clusters and past shared memory, pools past 32-bit
offsets, captured chains, refusals.  Tolerances as in test_gpu_paged."""
import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
from compressive_memory_long_b200.positions import rotary_frequencies
from tests import _paged_reference as ref
from tests.test_gpu_paged import DT, Cache, check_decode, evict_case, f64, normal, ok, run_decode, same_bits

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_more_tiles_than_ctas(dtype):
    """Long and short sequences together: every CTA has several tiles, long units span CTAs, one
    CTA holds many short units."""
    lens = [3000, 1, 0, 2500, -1, 2, 2047, 64, 63, 3500]
    c = Cache(len(lens), 4, 128, 32, max(lens) + 1, dtype, seed=3)
    rows = c.fill(lens, 40)
    q, k, v = (normal((len(lens), n, 128), DT[dtype], 50 + n) for n in (8, 4, 4))
    k = k + 0.5
    out = run_decode(c, q, k, v, lens, weights=c.w)
    check_decode(c, rows, q, k, v, lens, out, before_w=True)
    ok()


def test_decode_batch_larger_than_a_block():
    """More sequences than threads look at the lengths at once, padding entries among them."""
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(-1, 40, (700,), generator=g).tolist()
    c = Cache(700, 2, 32, 8, 41, "bf16", seed=6)
    rows = c.fill(lens, 60)
    q, k, v = (normal((700, n, 32), torch.bfloat16, 70 + n) for n in (4, 2, 2))
    M = torch.rand((700, 2, 32, 32), generator=torch.Generator().manual_seed(4)).cuda()
    z = 1 + torch.rand((700, 2, 32), generator=torch.Generator().manual_seed(5)).cuda()
    kw = dict(beta=normal((4,), torch.float32, 7), M=M, z=z)
    out = run_decode(c, q, k, v, lens, weights=c.w, **kw)
    check_decode(c, rows, q, k, v, lens, out, before_w=True, **kw)
    ok()


@pytest.mark.parametrize("B,n", [(300, 30), (950, 9)])
def test_evict_batch_larger_than_a_block(B, n):
    lens = torch.randint(-1, n, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    lens[B // 2] = n
    evict_case(lens, 1, 32, 4, n // 3, 2, "f32", fold=True, seed=9)


def dense_evict(n, units, budget, recent, weights, seed):
    """Selection alone, against a stable sort: one sequence whose rows lie in order in the pool."""
    page, d = 16, 32
    pages, dst_pages = -(-n // page), -(-budget // page)
    k = torch.zeros((pages + dst_pages, units, page, d), dtype=torch.bfloat16, device="cuda")
    w = weights(torch.Generator(device="cuda").manual_seed(seed), (pages, units, page))
    pool = torch.cat([w, torch.full((dst_pages, units, page), 7.0, device="cuda")])
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    dst = torch.arange(pages, pages + dst_pages, dtype=torch.int32, device="cuda")[None]
    lens, kept = binding.paged_evict(k, k.clone(), pool, table, i32([n]), dst, budget=budget, recent=recent)
    ok()
    assert lens.tolist() == [min(n, budget)]
    flat = w.transpose(0, 1).reshape(units, -1)[:, :n - recent]
    best = flat.sort(dim=1, descending=True, stable=True).indices[:, :budget - recent].sort(dim=1).values
    want = torch.cat([best, torch.arange(n - recent, n, device="cuda").expand(units, -1)], 1)
    assert torch.equal(kept[0], want.to(torch.int32))
    got = pool[pages:].transpose(0, 1).reshape(units, -1)[:, :budget]
    assert torch.equal(got, w.transpose(0, 1).reshape(units, -1).gather(1, want))


@pytest.mark.parametrize("weights", ["spread", "ties", "equal"])
@pytest.mark.parametrize("n,units,budget,recent", [
    (40000, 2, 3000, 100),          # eight CTAs a head
    (20011, 18, 20010, 5),          # four, one row leaves
    (9000, 37, 1, 1),               # two, the recent row alone
    (42001, 75, 500, 0),            # one CTA a head, more rows than its shared memory holds
    (330001, 1, 70000, 12),         # eight, and more rows than they hold
])
def test_select_over_clusters(n, units, budget, recent, weights):
    make = {"spread": lambda g, s: torch.rand(s, device="cuda", generator=g).pow(6) * 8,
            "ties": lambda g, s: torch.randint(0, 4, s, device="cuda", generator=g).float(),
            "equal": lambda g, s: torch.full(s, 0.25, device="cuda")}[weights]
    dense_evict(n, units, budget, recent, make, n % 97)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,Hkv,n", [(128, 2, 20001), (64, 3, 9000), (32, 1, 30000)])
def test_fold_of_many_rows(d, Hkv, n, dtype):
    """Heads folded by several CTAs each: the sum of sigma(k) v^T of all rows but the recent ones, in
    fp64.  Error as in test_gpu_paged: sigma 4u (2^-25 more for its parts), count + 2 roundings."""
    budget = recent = 64
    page, pages, dst = 64, -(-n // 64), 1
    k = normal((pages + dst, Hkv, page, d), DT[dtype], 21)
    v = normal((pages + dst, Hkv, page, d), DT[dtype], 22)
    w = torch.rand((pages + dst, Hkv, page), device="cuda")
    M, z = torch.zeros((1, Hkv, d, d), device="cuda"), torch.zeros((1, Hkv, d), device="cuda")
    rows = lambda x: f64(x[:pages].transpose(0, 1).reshape(Hkv, -1, d)[:, :n - recent])
    K, V = rows(k), rows(v)
    binding.paged_evict(k, v, w, torch.arange(pages, dtype=torch.int32, device="cuda")[None], i32([n]),
                        i32([[pages]]), budget=budget, recent=recent, M=M, z=z)
    ok()
    f = ref.sigma(K)
    u = 2.0 ** -24
    for h in range(Hkv):
        e = (6 + n) * u
        assert np.all(np.abs(f64(M[0, h]) - f[h].T @ V[h]) <= e * (f[h].T @ np.abs(V[h])))
        assert np.all(np.abs(f64(z[0, h]) - f[h].sum(0)) <= e * f[h].sum(0))
        # and far below the bound as a whole: the sums' own rounding, not a lost part of sigma
        d_m = f64(M[0, h]) - f[h].T @ V[h]
        assert np.linalg.norm(d_m) <= 2.0 ** -20 * np.linalg.norm(f[h].T @ V[h])


def test_pools_past_32_bit_offsets():
    """The same rows in a small pool and in the last pages of one of more than 2^32 bytes and 2^31
    elements give the same bits."""
    Hkv, page, d, H = 2, 64, 128, 8
    P = (1 << 31) // (Hkv * page * d) + 9
    lens, B, per = [200, 129], 2, 4
    small = Cache(B, Hkv, d, page, 256, "bf16", seed=8)
    small.fill(lens, 10)
    big = [torch.empty((P, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    bw = torch.empty((P, Hkv, page), device="cuda")
    table = torch.arange(P - B * per, P, dtype=torch.int32).reshape(B, per)
    at, src = table.flatten().long().cuda(), small.table.flatten().long()
    big[0][at], big[1][at], bw[at] = small.k[src], small.v[src], small.w[src]
    q, k, v = (normal((B, n, d), torch.bfloat16, 30 + n) for n in (H, Hkv, Hkv))
    one = run_decode(small, q, k, v, lens, weights=small.w)
    two = binding.paged_decode_step(q, k, v, *big, table.cuda(), i32(lens), weights=bw)
    assert torch.equal(one, two)
    more = i32([n + 1 for n in lens])
    kk = normal((B, Hkv, 3, d), torch.bfloat16, 33)
    binding.paged_append(kk, kk, small.k, small.v, small.table, more, weights=small.w)
    binding.paged_append(kk, kk, *big, table.cuda(), more, weights=bw)
    for x, y in zip((small.k, small.v, small.w), (*big, bw)):
        assert same_bits(x[src], y[at])
    n = i32([m + 4 for m in lens])
    M, z = torch.rand((B, Hkv, d, d), device="cuda"), torch.rand((B, Hkv, d), device="cuda")
    M2, z2 = M.clone(), z.clone()
    dst_small = torch.tensor(small.free[:2], dtype=torch.int32).reshape(2, 1).cuda()
    dst_big = i32([[3], [P - B * per - 1]])
    a = binding.paged_evict(small.k, small.v, small.w, small.table, n, dst_small, budget=60, recent=9, M=M, z=z)
    b = binding.paged_evict(*big, bw, table.cuda(), n, dst_big, budget=60, recent=9, M=M2, z=z2)
    assert all(torch.equal(x, y) for x, y in zip((*a, M, z), (*b, M2, z2)))
    for x, y in zip((small.k, small.v, small.w), (*big, bw)):
        assert same_bits(x[dst_small[:, 0].long()][:, :, :60], y[dst_big[:, 0].long()][:, :, :60])
    ok()


def test_a_captured_chain_replays():
    """rotary, append, a decode step and an eviction into the memory in one graph, replayed on other
    inputs in the same buffers, against the same calls made one by one on a second stream."""
    B, H, Hkv, d, page, T, L = 3, 8, 2, 128, 16, 90, 200
    freq, scale = rotary_frequencies(d, scaling="ntk", factor=4)

    def state(seed):
        x = dict(q=normal((B, T, H, d), torch.bfloat16, seed), k=normal((B, T, Hkv, d), torch.bfloat16, seed + 1),
                 v=normal((B, T, Hkv, d), torch.bfloat16, seed + 2), q1=normal((B, H, d), torch.bfloat16, seed + 3),
                 k1=normal((B, Hkv, d), torch.bfloat16, seed + 4), lens=i32([0, seed % 70, 100]),
                 M=torch.rand((B, Hkv, d, d), device="cuda"), z=torch.rand((B, Hkv, d), device="cuda") + 1,
                 beta=normal((H,), torch.float32, seed + 5))
        n, m = L // page + 1, 2
        x["pages"] = normal((B * (n + m), Hkv, page, d), torch.bfloat16, seed + 6)
        x["v_pages"] = normal(x["pages"].shape, torch.bfloat16, seed + 7)
        x["w"] = torch.rand(x["pages"].shape[:3], generator=torch.Generator().manual_seed(seed)).cuda()
        order = torch.randperm(B * (n + m), generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        x["table"], x["dst"] = order[:B * n].reshape(B, n).cuda(), order[B * n:].reshape(B, m).cuda()
        return x

    def chain(x, stream=None):
        kw = dict(stream=stream)
        _, kr = binding.rotary(x["q"].transpose(1, 2), x["k"].transpose(1, 2), freq, start=7, scale=scale, **kw)
        binding.paged_append(kr, x["v"].transpose(1, 2), x["pages"], x["v_pages"], x["table"], x["lens"],
                             weights=x["w"], **kw)
        x["lens"] += T
        out = binding.paged_decode_step(x["q1"], x["k1"], x["k1"], x["pages"], x["v_pages"], x["table"], x["lens"],
                                        beta=x["beta"], M=x["M"], z=x["z"], weights=x["w"], freq=freq, **kw)
        x["lens"] += 1
        n, kept = binding.paged_evict(x["pages"], x["v_pages"], x["w"], x["table"], x["lens"], x["dst"], budget=30,
                                      recent=5, M=x["M"], z=x["z"], **kw)
        return out, n, kept

    x = state(100)
    chain(state(90))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(x)
    for seed in (200, 301, 333):
        y = state(seed)
        for name, t in y.items():
            x[name].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = chain(y, s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("pages", "v_pages"):
            assert same_bits(x[name], y[name])
        assert torch.equal(x["w"], y["w"]) and torch.equal(x["M"], y["M"]) and torch.equal(x["z"], y["z"])
    ok()


def test_steps_on_two_streams_with_weights_and_evictions():
    """Two batches, each with its own cache, stepped and cut at the same time on two streams, give
    what they give alone."""
    def make(seed):
        c = Cache(3, 2, 64, 8, 64, "f32", seed=seed)
        c.fill([50, 33, 64 - 1], seed)
        dst = Cache(3, 2, 64, 8, 24, "f32", seed=seed)          # pages of their own behind the pool
        pool = [torch.cat([a, b]) for a, b in ((c.k, dst.k), (c.v, dst.v), (c.w, dst.w))]
        q, k = normal((3, 4, 64), torch.float32, seed), normal((3, 2, 64), torch.float32, seed + 1)
        return pool, c.table, dst.table + c.P, q, k, i32([50, 33, 63])

    def go(x, stream):
        (kp, vp, w), t, dst, q, k, n = x
        M, z = torch.ones((3, 2, 64, 64), device="cuda"), torch.ones((3, 2, 64), device="cuda")
        stream.wait_stream(torch.cuda.current_stream())
        out = binding.paged_decode_step(q, k, k, kp, vp, t, n, weights=w, stream=stream)
        with torch.cuda.stream(stream):
            more = n + 1
        _, kept = binding.paged_evict(kp, vp, w, t, more, dst, budget=20, recent=4, M=M, z=z, stream=stream)
        return out, kept, M, z

    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    want = []
    for seed in (1, 2):
        want.append(go(make(seed), one))
        torch.cuda.synchronize()
    for _ in range(5):
        xs = [make(1), make(2)]
        got = [go(xs[0], one), go(xs[1], two)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    ok()


def test_refusals_with_tensors():
    c = Cache(2, 2, 64, 8, 24, "bf16")
    n = i32([3, 4])
    q, k = normal((2, 4, 64), torch.bfloat16, 1), normal((2, 2, 64), torch.bfloat16, 2)
    step = lambda **kw: binding.paged_decode_step(**{**dict(q=q, k=k, v=k, k_pages=c.k, v_pages=c.v,
                                                            page_table=c.table, lens=n), **kw})
    for bad in (dict(q=q.float()), dict(k=k[:, :1]), dict(lens=n.long()), dict(lens=n.cpu()), dict(lens=None),
                dict(page_table=c.table[0]), dict(weights=c.w.double()), dict(positions=n.long()),
                dict(q=q.transpose(1, 2)), dict(freq=torch.ones(8, device="cuda")), dict(k_pages=c.k[0]),
                dict(out=torch.empty((2, 4, 32), dtype=torch.bfloat16, device="cuda")), dict(q="q"),
                dict(k_pages=c.k.half(), v_pages=c.v.half())):
        with pytest.raises(ValueError):
            step(**bad)
    for bad in (dict(v=None), dict(beta=torch.zeros(4, device="cuda")), dict(out=q)):
        with pytest.raises(binding.InfiniError) as e:
            step(**bad)
        assert e.value.status == 1
    odd = torch.zeros((4, 2, 24, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.InfiniError) as e:
        step(k_pages=odd, v_pages=odd.clone())
    assert e.value.status == 2
    with pytest.raises(ValueError):
        binding.paged_evict(c.k, c.v, c.w, c.table, n, c.table[:1], budget=4)
    with pytest.raises(ValueError):
        binding.paged_evict(c.k, c.v, None, c.table, n, c.table, budget=4)
    with pytest.raises(binding.InfiniError) as e:
        binding.paged_evict(c.k, c.v, c.w, c.table, n, c.table, budget=4, recent=5)
    assert e.value.status == 1
    M, z = torch.zeros((2, 2, 64, 64), device="cuda"), torch.zeros((2, 2, 64), device="cuda")
    with pytest.raises(binding.InfiniError) as e:
        binding.paged_evict(c.k, c.v, c.w, c.table, n, c.table, budget=4, M=M, z=z, rule="delta")
    assert e.value.status == 2
    with pytest.raises(ValueError):
        binding.paged_append(k[:, :, None, ::2], k[:, :, None, ::2], c.k, c.v, c.table, n)
    with pytest.raises(ValueError):
        binding.rotary(q, None, torch.ones(32, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        binding.rotary(q[:, :, None], None, torch.ones(32, dtype=torch.float64, device="cuda"),
                       k_out=q[:, :, None])
    ok()


def test_rotary_copies_channels_that_no_pair_has():
    """Infinities and NaN in channels past rot stay where they are and spread to none."""
    for inter in (False, True):
        for rot, dt in ((34, torch.bfloat16), (32, torch.bfloat16), (18, torch.float32), (0, torch.bfloat16)):
            q = normal((1, 3, 5, 64), dt, 5)
            q[..., rot + 1], q[..., rot + 2], q[..., 63] = float("inf"), float("nan"), -float("inf")
            freq, _ = rotary_frequencies(rot)
            y, _ = binding.rotary(q, None, freq, start=9, interleaved=inter)
            assert torch.equal(y[..., rot:].nan_to_num(5.0), q[..., rot:].nan_to_num(5.0))
            assert torch.isfinite(y[..., :rot]).all()
    k, v = (normal((1, 1, 32), torch.float32, 6 + i) for i in range(2))
    k[..., 20] = float("inf")                  # in the cache's new row as well
    c = Cache(1, 1, 32, 8, 8, "f32", weights=False)
    freq, _ = rotary_frequencies(16)
    binding.paged_decode_step(normal((1, 1, 32), torch.float32, 8), k, v, c.k, c.v, c.table, i32([0]), freq=freq)
    row = c.dense(c.k, 0, 1)[0, 0]
    assert np.isinf(row[20]) and np.isfinite(np.delete(row, 20)).all()


@pytest.mark.parametrize("d,rot,L,dt", [(64, 34, 7, torch.bfloat16), (128, 34, 301, torch.bfloat16),
                                        (64, 18, 5, torch.float32), (32, 10, 1, torch.bfloat16),
                                        (128, 6, 33, torch.float32)])
def test_ragged_halves_in_place(d, rot, L, dt):
    """Halves that cut a vector: in place as out of place, and against the definition."""
    q, k = normal((2, 5, L, d), dt, 1), normal((2, 2, L, d), dt, 2)
    freq, _ = rotary_frequencies(rot)
    qo, ko = binding.rotary(q, k, freq, start=77)
    for b, h, t in ((0, 0, 0), (1, 4, L - 1), (0, 2, L // 2)):
        want = ref.rotate(f64(q[b, h, t]), 77 + t, f64(freq), False)
        half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
        assert np.all(np.abs(f64(qo[b, h, t]) - want) <= 8 * 2.0 ** -24 * 12 + half * np.abs(want))
    q2, k2 = q.clone(), k.clone()
    binding.rotary(q2, k2, freq, start=77, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_nan_in_a_cached_row_reaches_its_head_alone():
    c = Cache(2, 2, 64, 8, 40, "bf16", weights=False)
    c.fill([30, 35], 11)
    q = normal((2, 4, 64), torch.bfloat16, 12)
    clean = run_decode(c, q, None, None, [30, 35])
    pg, sl = ref.row_at(c.table_h[0].tolist(), 17, 8, c.P)
    c.k[pg, 1, sl, 5] = float("nan")
    out = run_decode(c, q, None, None, [30, 35])
    assert torch.equal(out[1], clean[1]) and torch.equal(out[0, :2], clean[0, :2])
    assert out[0, 2:].isnan().all()
    only = run_decode(c, q, None, None, [0, 35])
    assert not only[0].any()
    ok()
