"""The paged serving entry points on the host: refusals by status before any CUDA call (fake
addresses that argument checking never dereferences), the binding's own checks, and the
rotary frequency tables."""
import ctypes
import math

import pytest
import torch

from compressive_memory_long_b200 import binding
from compressive_memory_long_b200.positions import rotary_frequencies

BASE, GAP = 1 << 40, 1 << 36
INVALID, UNSUPPORTED = 1, 2


def at(i, off=0):
    return BASE + i * GAP + off


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def pointers(names, over):
    p = {n: at(i) for i, n in enumerate(names)}
    p.update(over)
    return [None if p[n] is None else ctypes.c_void_p(p[n]) for n in names]


ROT = ["q", "k", "q_out", "k_out", "freq", "positions"]
BOTH = [("", ""), ("_f32", "")]


def call_rotary(entry, B=1, H=4, Hkv=2, L=8, d=64, rot=64, start=0, sq=None, sk=None, **ptr):
    f = getattr(binding.LIB, entry)
    return f(*pointers(ROT, ptr), start, sq, sk, B, H, Hkv, L, d, rot, 0, 1.0, None)


@pytest.mark.parametrize("entry", ["infini_attn_rotary", "infini_attn_rotary_f32",
                                   "infini_attn_rotary_bwd", "infini_attn_rotary_bwd_f32"])
@pytest.mark.parametrize("kw,status", [
    *[(dict({n: None}), INVALID) for n in ("q", "k", "q_out", "k_out", "freq")],
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(L=0), INVALID),
    (dict(rot=-2), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID),
    (dict(q=at(0, 1)), INVALID), (dict(q_out=at(2, 8)), INVALID), (dict(freq=at(4, 8)), INVALID),
    (dict(sq=strides(-1, 64, 64)), INVALID),
    (dict(q_out=at(0, 64)), INVALID),                            # part of q
    (dict(q_out=at(0), sq=strides(4096, 64, 256)), INVALID),     # in place, but not contiguous
    (dict(k_out=at(0)), INVALID), (dict(k_out=at(2, 64)), INVALID),
    (dict(positions=at(2)), INVALID),
    (dict(d=48, rot=32), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
])
def test_rotary_argument_errors(entry, kw, status):
    assert call_rotary(entry, **kw) == status


APP = ["k", "v", "sk", "sv", "k_pages", "v_pages", "weights", "page_table", "lens", "counts"]


def call_append(entry, B=2, Hkv=2, T=3, d=64, P=10, page=16, max_pages=4, sk=None, sv=None, **ptr):
    a = pointers(APP, dict(ptr, sk=None, sv=None))
    a[2], a[3] = sk, sv
    return getattr(binding.LIB, entry)(*a, B, Hkv, T, d, P, page, max_pages, None)


@pytest.mark.parametrize("entry", ["infini_attn_paged_append", "infini_attn_paged_append_f32"])
@pytest.mark.parametrize("kw,status", [
    *[(dict({n: None}), INVALID) for n in ("k", "v", "k_pages", "v_pages", "page_table", "lens")],
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(T=0), INVALID), (dict(P=0), INVALID),
    (dict(page=0), INVALID), (dict(max_pages=0), INVALID), (dict(max_pages=1 << 30), INVALID),
    (dict(k=at(0, 1)), INVALID), (dict(k_pages=at(4, 8)), INVALID), (dict(lens=at(8, 2)), INVALID),
    (dict(v_pages=at(4, 64)), INVALID), (dict(k=at(4)), INVALID), (dict(weights=at(5)), INVALID),
    (dict(page_table=at(6, 16)), INVALID), (dict(sv=strides(64, -64, 64)), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(d=48), UNSUPPORTED),
])
def test_append_argument_errors(entry, kw, status):
    assert call_append(entry, **kw) == status


DEC = ["q", "k", "v", "k_pages", "v_pages", "page_table", "lens", "beta", "M", "z", "weights", "freq",
       "positions", "out", "workspace"]


def call_decode(entry, B=2, H=4, Hkv=2, d=64, P=10, page=16, max_pages=4, rot=64, nbytes=None, **ptr):
    need = binding.LIB.infini_attn_paged_decode_workspace_bytes(B, H, Hkv, d, P, page, 1)
    return getattr(binding.LIB, entry)(*pointers(DEC, ptr), need if nbytes is None else nbytes, B, H,
                                       Hkv, d, P, page, max_pages, rot, 0, 1.0, None)


@pytest.mark.parametrize("entry", ["infini_attn_paged_decode_step",
                                   "infini_attn_paged_decode_step_f32"])
@pytest.mark.parametrize("kw,status", [
    *[(dict({n: None}), INVALID) for n in ("q", "k", "v", "k_pages", "v_pages", "page_table", "lens",
                                           "beta", "M", "z", "freq", "out")],
    (dict(B=0), INVALID), (dict(H=3), INVALID), (dict(H=0), INVALID), (dict(P=0), INVALID),
    (dict(rot=5), INVALID), (dict(rot=128), INVALID), (dict(nbytes=-1), INVALID),
    (dict(q=at(0, 8)), INVALID), (dict(out=at(13, 4)), INVALID), (dict(lens=at(6, 2)), INVALID),
    (dict(out=at(0)), INVALID), (dict(out=at(3, 64)), INVALID), (dict(k=at(3)), INVALID),
    (dict(weights=at(4)), INVALID), (dict(M=at(10)), INVALID), (dict(page_table=at(3)), INVALID),
    (dict(page=12), UNSUPPORTED), (dict(d=48, rot=32), UNSUPPORTED),
])
def test_paged_decode_argument_errors(entry, kw, status):
    assert call_decode(entry, **kw) == status


EVI = ["k_pages", "v_pages", "weights", "page_table", "lens", "dst_table", "lens_out", "kept", "M", "z",
       "workspace"]


def call_evict(entry, B=2, Hkv=2, d=64, P=10, page=16, max_pages=4, dst_pages=2, budget=32, recent=8,
               rule=0, nbytes=None, **ptr):
    need = binding.LIB.infini_attn_paged_evict_workspace_bytes(B, Hkv, d, page, max_pages, budget, 1)
    return getattr(binding.LIB, entry)(*pointers(EVI, ptr), need if nbytes is None else nbytes, B, Hkv,
                                       d, P, page, max_pages, dst_pages, budget, recent, rule, None)


@pytest.mark.parametrize("entry", ["infini_attn_paged_evict", "infini_attn_paged_evict_f32"])
@pytest.mark.parametrize("kw,status", [
    *[(dict({n: None}), INVALID) for n in EVI],
    (dict(B=0), INVALID), (dict(budget=0), INVALID), (dict(recent=-1), INVALID),
    (dict(recent=33), INVALID), (dict(budget=33, recent=0), INVALID),      # past dst_table
    (dict(rule=2), INVALID), (dict(nbytes=8), INVALID),
    (dict(kept=at(7, 4)), INVALID), (dict(lens_out=at(6, 1)), INVALID),
    (dict(lens_out=at(4)), INVALID), (dict(v_pages=at(0)), INVALID), (dict(M=at(9)), INVALID),
    (dict(workspace=at(7)), INVALID), (dict(dst_table=at(7)), INVALID),
    (dict(page=24), UNSUPPORTED), (dict(d=16), UNSUPPORTED), (dict(rule=1), UNSUPPORTED),
])
def test_evict_argument_errors(entry, kw, status):
    assert call_evict(entry, **kw) == status


def test_workspace_sizes():
    f, e = (binding.LIB.infini_attn_paged_decode_workspace_bytes,
            binding.LIB.infini_attn_paged_evict_workspace_bytes)
    assert f(0, 1, 1, 64, 1, 16, 0) == 0 and e(0, 1, 64, 16, 1, 16, 1) == 0
    assert f(2, 8, 2, 64, 100, 16, 1) >= f(2, 8, 2, 64, 100, 16, 0)
    assert e(2, 2, 64, 16, 4, 64, 0) >= 0 and e(2, 2, 64, 16, 4, 32, 1) > 0


def test_page_status_has_a_description():
    assert "page" in binding.infini_attn_status_string(6)
    assert binding.STATUS[6] == "INFINI_ERR_PAGE"


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 4, 32)
    f = torch.ones(16, dtype=torch.float64)
    pages = torch.zeros(2, 2, 8, 32)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(2, 2, 8)
    for call in (lambda: binding.rotary(q, q, f), lambda: binding.rotary_backward(q, q, f),
                 lambda: binding.paged_append(q, q, pages, pages, t, n),
                 lambda: binding.paged_decode_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], pages, pages, t, n),
                 lambda: binding.paged_evict(pages, pages, w, t, n, t, budget=4)):
        with pytest.raises(ValueError):
            call()


def test_frequencies():
    f, s = rotary_frequencies(8, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64
    assert f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert rotary_frequencies(0, device="cpu")[0].numel() == 0
    lin, _ = rotary_frequencies(8, scaling="linear", factor=4, device="cpu")
    assert lin.tolist() == pytest.approx([x / 4 for x in f.tolist()], rel=1e-15)
    ntk, _ = rotary_frequencies(8, scaling="ntk", factor=4, device="cpu")
    assert ntk[0] == 1 and ntk[-1].item() == pytest.approx(f[-1].item() / 4, rel=1e-12)
    assert rotary_frequencies(2, scaling="ntk", factor=4, device="cpu")[0].tolist() == [1.0]


def test_yarn_frequencies():
    """Fast pairs keep their frequency, slow ones are divided, the ramp lies between."""
    rot, n, k = 128, 2048, 16.0
    f, _ = rotary_frequencies(rot, device="cpu")
    y, s = rotary_frequencies(rot, scaling="yarn", factor=k, trained_length=n, device="cpu")
    assert s == pytest.approx(0.1 * math.log(k) + 1)
    ratio = (y / f).tolist()
    for r, t in zip(ratio, (f * n / (2 * math.pi)).tolist()):
        if t > 40:
            assert r == pytest.approx(1)
        elif t < 0.8:
            assert r == pytest.approx(1 / k)
        else:
            assert 1 / k - 1e-12 <= r <= 1 + 1e-12
    assert all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=-2), dict(rot=8, scaling="other"),
                                dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, scaling="yarn")])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rotary_frequencies(device="cpu", **kw)


def test_declared_and_bound_argument_counts_agree():
    """Every paged prototype of the header has as many parameters as its binding."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "infini_attn.h")).read()
    seen = 0
    for name, args in re.findall(r"INFINI_API\s+\w+\s+(infini_attn_(?:rotary|paged)\w*)\s*\(([^)]*)\)", src):
        types = binding.SIGNATURES[name][0]
        kinds = ["P" if "*" in a or "stream" in a else "F" if "float" in a else
                 "Q" if "int64_t" in a else "I" for a in args.split(",")]
        want = {ctypes.c_void_p: "P", ctypes.c_float: "F", ctypes.c_int64: "Q", ctypes.c_int: "I"}
        assert kinds == [want[t] for t in types], name
        seen += 1
    assert seen == 12
