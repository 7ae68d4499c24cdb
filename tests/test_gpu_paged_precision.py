"""What the paged operators keep of their 32-bit values, at inputs whose other roundings are few, so
that the bound is far below 16 bits (u = 2^-24)."""
import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
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
