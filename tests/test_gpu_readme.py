"""The README's serving example, run as it is written."""
import os
import re

import pytest
import torch

from tests.test_gpu_paged import normal, ok

pytestmark = pytest.mark.gpu


def test_the_serving_example():
    """A prompt, a step and a cut: the step's row follows the prompt's, and the cut sees them all."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(root, "README.md")).read(), re.S)
    (code,) = [b for b in blocks if "paged_append" in b]
    B, H, Hkv, L, d, page = 2, 4, 2, 2300, 128, 64
    per, new = L // page + 1, 2048 // page
    q, k, v = (normal((B, n, L, d), torch.bfloat16, n) for n in (H, Hkv, Hkv))
    q1, k1, v1 = (normal((B, n, d), torch.bfloat16, 10 + n) for n in (H, Hkv, Hkv))
    order = torch.randperm(B * (per + new), generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    s = dict(q=q, k=k, v=v, q1=q1, k1=k1, v1=v1, beta=torch.zeros(H, device="cuda"),
             k_pages=torch.zeros((B * (per + new), Hkv, page, d), dtype=torch.bfloat16, device="cuda"),
             weights=torch.full((B * (per + new), Hkv, page), 9.0, device="cuda"),
             page_table=order[:B * per].reshape(B, per), new_pages=order[B * per:].reshape(B, new),
             lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
             positions=torch.full((B,), L, dtype=torch.int64, device="cuda"),
             M=torch.zeros((B, Hkv, d, d), device="cuda"), z=torch.zeros((B, Hkv, d), device="cuda"),
             M0=None, z0=None, dout=q, dM=None, dz=None)
    s["v_pages"] = s["k_pages"].clone()
    exec(code, s)
    ok()
    assert s["lens"].tolist() == [2048] * B
    last = torch.arange(L + 1 - 256, L + 1, dtype=torch.int32, device="cuda")
    assert (s["kept"][..., -256:] == last).all()
    table, r = s["new_pages"].long(), 2047                     # the step's own row, where it went
    got = s["v_pages"][table[:, r // page], :, r % page]
    assert torch.equal(got, v1)
    # one step's weights of the kept rows: what the group's heads gave, less what left
    w = s["weights"][table].transpose(1, 2).sum((2, 3))
    assert ((w > 0) & (w <= H // Hkv + 1e-3)).all()
    assert (s["z"] > 0).all() and s["out"].isfinite().all()
