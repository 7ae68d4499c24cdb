"""Calls of the paged operators at the ends of what they take."""
import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
from compressive_memory_long_b200.positions import rotary_frequencies
from tests.test_gpu_paged import Cache, check_decode, normal, ok, run_decode, same_bits

pytestmark = pytest.mark.gpu

LOWEST = -2 ** 31


@pytest.mark.parametrize("lens", [[LOWEST, 40], [40, LOWEST + 1], [LOWEST]])
def test_the_lowest_length_is_a_padding_entry(lens):
    """Any negative length marks one: no row of it is read, folded or written."""
    B, Hkv, d = len(lens), 2, 64
    c = Cache(B, Hkv, d, 8, 48, "bf16", seed=1)
    rows = c.fill([max(n, 0) for n in lens], 10)
    q, k = normal((B, 4, d), torch.bfloat16, 3), normal((B, Hkv, d), torch.bfloat16, 4)
    out = run_decode(c, q, k, k, lens, weights=c.w)
    check_decode(c, rows, q, k, k, lens, out, before_w=True)
    binding.paged_append(k[:, :, None], k[:, :, None], c.k, c.v, c.table,
                         torch.tensor([n + 1 if n > 0 else n for n in lens], dtype=torch.int32, device="cuda"),
                         weights=c.w)
    extra = Cache(B, Hkv, d, 8, 8, "bf16", seed=2)
    pool = [torch.cat([x, y]) for x, y in zip((c.k, c.v, c.w), (extra.k, extra.v, extra.w))]
    M, z = torch.ones((B, Hkv, d, d), device="cuda"), torch.ones((B, Hkv, d), device="cuda")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in pool]
    lens_out, kept = binding.paged_evict(*pool, c.table, n, extra.table + c.P, budget=8, recent=2, M=M, z=z)
    ok()
    assert lens_out.tolist() == [min(n, 8) for n in lens]
    for b, n in enumerate(lens):
        if n < 0:
            assert (kept[b] == -1).all() and (M[b] == 1).all() and (z[b] == 1).all()
            dst = (extra.table[b] + c.P).long()
            assert all(same_bits(x[dst], y[dst]) for x, y in zip(pool, before))
        else:
            assert (z[b] > 1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hkv,d,edges", [
    (40, 16, 8, 32, [1022, 1023, 1024, 1025, 2047, 2048, 2500, 0, -1, 3100]),   # 320 units, one chunk each
    (76, 48, 4, 32, [1023, 1024, 1025, 2049, 1, 2500]),                         # groups of twelve, 304 units
    (3, 12, 1, 64, [5000, 1024, 1023]),                                         # chunks of several blocks
])
def test_weights_of_rows_past_a_block_s_first_chunk(B, H, Hkv, d, edges, dtype):
    """The rows of a (sequence, key/value head) are weighted a thousand at a time; where there are as many of
    these as blocks fit the card, one block goes on to the next thousand itself."""
    lens = [edges[i % len(edges)] for i in range(B)]
    c = Cache(B, Hkv, d, 64, max(lens) + 1, dtype, seed=B)
    rows = c.fill(lens, 20)
    q, k, v = (normal((B, n, d), c.k.dtype, 30 + n) for n in (H, Hkv, Hkv))
    out = run_decode(c, q, k, v, lens, weights=c.w)
    ok()
    few = [b for b in range(B) if b < len(edges)] + [B - 1]      # the loops in 64 bits take their time
    check_decode(c, rows, q, k, v, [n if b in few else -1 for b, n in enumerate(lens)],
                 torch.where(torch.tensor([b in few for b in range(B)], device="cuda")[:, None, None], out, 0),
                 before_w=True)


def test_slices_of_positions_and_gates():
    """A step's positions and a layer's gates may be slices off 16 bytes, in the rotary call as well."""
    lens, H, d = [5, 20, 33], 4, 64
    c = Cache(3, 2, d, 16, 34, "f32", seed=7)
    c.fill(lens, 40)
    q, k = normal((3, H, d), torch.float32, 1), normal((3, 2, d), torch.float32, 2)
    freq, _ = rotary_frequencies(d)
    M, z = torch.rand((3, 2, d, d)).cuda(), torch.rand((3, 2, d)).cuda() + 1
    positions, beta = torch.arange(4, device="cuda") * 1001, normal((H + 1,), torch.float32, 3)
    assert positions[1:].data_ptr() % 16 == 8 and beta[1:].data_ptr() % 16 == 4
    outs = [run_decode(c, q, k, k, lens, M=M, z=z, freq=freq, positions=p, beta=g)
            for p, g in ((positions[1:], beta[1:]), (positions[1:].clone(), beta[1:].clone()))]
    assert torch.equal(*outs)
    x = normal((1, 2, 3, d), torch.float32, 4)
    one, two = (binding.rotary(x, None, freq, positions=p)[0] for p in (positions[1:][None], positions[1:].clone()[None]))
    assert torch.equal(one, two)
    ok()


def test_a_flag_without_a_truth_value_is_refused():
    q = normal((1, 2, 3, 32), torch.float32, 1)
    before = q.clone()
    freq, _ = rotary_frequencies(32)
    with pytest.raises(ValueError):
        binding.rotary(q, None, freq, start=5, interleaved=np.zeros(2), q_out=q)
    assert torch.equal(q, before)
    c = Cache(1, 2, 32, 8, 8, "f32")
    with pytest.raises(ValueError):
        run_decode(c, q[:, :, 0].contiguous(), None, None, [0], freq=freq, interleaved=np.zeros(2))
    ok()
