"""What the paged operators keep of their 32-bit values, at inputs whose other roundings are few, so
that the bound is far below 16 bits (u = 2^-24)."""
import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
from compressive_memory_long_b200.positions import rotary_frequencies
from tests import _paged_reference as ref
from tests.test_gpu_paged import Cache, f64, normal, ok, run_decode

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HEADS = [(2, 2), (4, 1), (5, 1), (8, 1), (12, 1)]


def one_channel(B, H, Hkv, d, n, seed):
    """A cache of n rows whose keys, like q, have one channel that is not 0: a score is one product."""
    c = Cache(B, Hkv, d, 16, n, "bf16", seed=seed)
    c.k.zero_(), c.w.zero_()
    q = torch.zeros((B, H, d), dtype=torch.bfloat16, device="cuda")
    q[..., 1] = 1 + torch.rand((B, H), generator=torch.Generator().manual_seed(seed)).cuda()
    K = torch.zeros((B, Hkv, n, d), dtype=torch.bfloat16)
    K[..., 1] = torch.rand((B, Hkv, n), generator=torch.Generator().manual_seed(seed + 1)) * 2 - 1
    V = torch.randn((B, Hkv, n, d), generator=torch.Generator().manual_seed(seed + 2)).to(torch.bfloat16)
    for b in range(B):
        for r in range(n):
            pg, sl = ref.row_at(c.table_h[b].tolist(), r, 16, c.P)
            c.k[pg, :, sl], c.v[pg, :, sl] = K[b, :, r].cuda(), V[b, :, r].cuda()
    return c, q, K.double().numpy(), V.double().numpy()


@pytest.mark.parametrize("d", [128, 64, 32])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_scores_of_a_rotated_q_keep_32_bits(H, Hkv, d):
    """Position 0 turns by no angle, so q is q * scale, rounded once or twice (2u); its product with a
    key of one channel is summed of three parts (2 additions of up to 2u each), the factor
    log2(e) / sqrt(d) is off by at most 5u and multiplies with 1u: 12u of a score, which reaches |x|;
    x - max and the exponential's own argument 2u of it more.  A weight's relative error is twice that and
    n + 12 roundings of the sums and functions."""
    B, n, scale = 16, 3, 4.7123889 * d ** 0.5
    c, q, K, _ = one_channel(B, H, Hkv, d, n, 3 * d + H)
    run_decode(c, q, None, None, [n] * B, weights=c.w, freq=torch.ones(1, dtype=torch.float64, device="cuda"),
               positions=torch.zeros(B, dtype=torch.int64, device="cuda"), scale=scale)
    ok()
    s = float(torch.tensor(scale, dtype=torch.float32))
    for b in range(B):
        got = c.dense(c.w, b, n)
        for g in range(Hkv):
            want, most = np.zeros(n), 0.0
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                x = f64(q[b, h])[1] * s * K[b, g, :, 1] / np.sqrt(d)
                p = np.exp(x - x.max())
                want += p / p.sum()
                most = max(most, np.abs(x).max())
            assert np.all(np.abs(got[g] - want) <= (2.02 * 14 * U * most + (n + 12) * U) * want)


@pytest.mark.parametrize("d", [128, 64, 32])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_softmax_weights_keep_32_bits(H, Hkv, d):
    """Every output is the exact one's bf16 rounding unless that lies next to a border: off by half a
    step and by what 32-bit sums leave of s = sum p |v|.  Scores, one exact product of at most 1/4 in size,
    are off by 2u (as above), a weight by twice that and 4u of its exponential; the row of the highest
    score has the weight 1 and no value.  Numerator: 8u and 5 additions of parts of up to 2u.
    Denominator: 8u of two weights in three, 3 additions, a reciprocal and a product: 30u in all."""
    B, n = 256, 3
    c, q, K, V = one_channel(B, H, Hkv, d, n, 5 * d + H)
    q *= 0.5
    first, slot = c.table_h[:, 0].long().cuda(), slice(0, n)
    K *= 0.25 * d ** 0.5
    K[:, :, 0, 1], V[:, :, 0] = 0.25 * d ** 0.5, 0.0
    K = torch.from_numpy(K).to(torch.bfloat16)
    c.k[first, :, slot], c.v[first, :, slot] = K.cuda(), torch.from_numpy(V).to(torch.bfloat16).cuda()
    out = f64(run_decode(c, q, None, None, [n] * B)).reshape(B, Hkv, -1, d)
    ok()
    x = f64(q)[..., 1].reshape(B, Hkv, -1, 1) * K.double().numpy()[:, :, None, :, 1] / np.sqrt(d)
    assert np.abs(x).max() <= 0.26
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    want, s = p @ V, p @ np.abs(V)
    half = 2.0 ** (np.floor(np.log2(np.abs(want) + 1e-300)) - 8)
    assert np.all(np.abs(out - want) <= half + 30 * U * s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 64, 32])
def test_fold_of_negative_keys_channel_by_channel(d, dtype):
    """One evicted row, keys from 3 down to -60, so M and z are sigma(k) v and sigma(k) of a channel.
    sigma: the exponential is off by 2^-22 (4u) of it, its argument's remainder and the square of that
    by 2u, the product with it or x + 1 by 1u: 7u.  M: parts to u/2, the lower ones' products and the two
    accumulators add with 3u, and fp32 values come in parts to u/2 as well: 4u more."""
    B, Hkv, n = 48, 2, 2
    c = Cache(B, Hkv, d, 16, n, dtype, seed=d)
    extra = Cache(B, Hkv, d, 16, 1, dtype, seed=d + 1)
    dt = c.k.dtype
    g = torch.Generator().manual_seed(d)
    K = (3 - 63 * torch.rand((B, Hkv, d), generator=g)).to(dt)
    V = torch.randn((B, Hkv, d), generator=g).to(dt)
    first = c.table[:, 0].long()
    c.k[first, :, 0], c.v[first, :, 0] = K.cuda(), V.cuda()
    c.k[first, :, 1] = c.v[first, :, 1] = 1.0
    c.w[first, :, :2] = 1.0
    pool = [torch.cat([x, y]) for x, y in zip((c.k, c.v, c.w), (extra.k, extra.v, extra.w))]
    M, z = torch.zeros((B, Hkv, d, d), device="cuda"), torch.zeros((B, Hkv, d), device="cuda")
    binding.paged_evict(*pool, c.table, torch.full((B,), n, dtype=torch.int32, device="cuda"),
                        extra.table + c.P, budget=1, recent=1, M=M, z=z)
    ok()
    f = ref.sigma(f64(K))
    assert np.all(np.abs(f64(z) - f) <= 7 * U * f)
    want = f[..., :, None] * f64(V)[..., None, :]
    assert np.all(np.abs(f64(M) - want) <= 11 * U * np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fold_of_the_largest_keys(dtype):
    """sigma is 0 of keys far below, the key plus 1 of keys far above, and 0 of -inf; V beside them."""
    keys = [-1e4, -3e38, float("-inf"), 1e4, 1e30, -87.0, 0.0, -0.0]
    d, n = 32, 2
    c, extra = Cache(1, 1, d, 16, n, dtype), Cache(1, 1, d, 16, 1, dtype)
    k = torch.zeros(d)
    k[:len(keys)] = torch.tensor(keys)
    first = c.table[:, 0].long()
    c.k[first, :, 0], c.v[first, :, 0] = k.to(c.k.dtype).cuda(), torch.tensor(0.5).to(c.k.dtype).cuda()
    c.k[first, :, 1] = c.v[first, :, 1] = 1.0
    c.w[first, :, :2] = 1.0
    pool = [torch.cat([x, y]) for x, y in zip((c.k, c.v, c.w), (extra.k, extra.v, extra.w))]
    M, z = torch.zeros((1, 1, d, d), device="cuda"), torch.zeros((1, 1, d), device="cuda")
    binding.paged_evict(*pool, c.table, torch.tensor([n], dtype=torch.int32, device="cuda"), extra.table + c.P,
                        budget=1, recent=1, M=M, z=z)
    ok()
    f = ref.sigma(f64(k.to(c.k.dtype)))
    # e^-87 is 1.6e-38, next to the smallest number that is not subnormal: its parts are 0
    assert np.all(np.abs(f64(z[0, 0]) - f) <= 7 * U * f)
    assert np.all(np.abs(f64(M[0, 0]) - 0.5 * f[:, None]) <= 11 * U * 0.5 * f[:, None] + 2e-38)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 18), (32, 32)])
def test_rotary_keeps_the_angle_s_last_bits(d, rot, inter):
    """Pairs (1, 0) turn into cosine and sine themselves, both of the angle formed in 64 bits: off by one
    unit in the last place of a 32-bit function's value (u below 1) and half of one of its correction."""
    L, start = 4000, 1048000
    x = torch.zeros((1, 1, L, d), device="cuda")
    first = slice(0, rot, 2) if inter else slice(0, rot // 2)
    second = slice(1, rot, 2) if inter else slice(rot // 2, rot)
    x[..., first] = 1.0
    freq, _ = rotary_frequencies(rot)
    y, _ = binding.rotary(x, None, freq, start=start, interleaved=inter)
    odd = torch.zeros((1, 1, L, d + 1), device="cuda")[..., 1:]            # rows off 16 bytes as well
    odd.copy_(x)
    assert torch.equal(binding.rotary(odd, None, freq, start=start, interleaved=inter)[0], y)
    a = (start + np.arange(L))[:, None] * f64(freq)
    y = f64(y[0, 0])
    assert np.abs(y[:, first] - np.cos(a)).max() <= 1.5 * U
    assert np.abs(y[:, second] - np.sin(a)).max() <= 1.5 * U
