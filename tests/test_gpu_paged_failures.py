"""A bounded wait of the eviction's fold runs out, made to happen without a real failure: a test hook
lets one loading warp fill no stage and the wait limit is short; every role gives up and the kernel
returns."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

from compressive_memory_long_b200 import binding
from tests.test_gpu_paged import Cache, evict_case, f64, ok, same_bits

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@contextlib.contextmanager
def withheld():
    assert binding.infini_attn_test_wait_limit(1 << 20) == 0      # about half a millisecond
    assert binding.infini_attn_test_withhold_publish(True) == 0
    try:
        yield
        torch.cuda.synchronize()
    finally:
        binding.infini_attn_test_withhold_publish(False)
        binding.infini_attn_test_wait_limit(0)


class Cut:
    """Sequences of a few tiles and of many, to be cut to `budget` rows; the workspace is NaN."""

    def __init__(self, dtype="bf16", lens=(3000, 130, 70, 20), Hkv=2, d=64, page=16, budget=64, recent=9):
        self.lens, self.budget, self.recent = lens, budget, recent
        B, extra = len(lens), -(-budget // page)
        c = self.c = Cache(B, Hkv, d, page, max(lens), dtype, seed=4)
        self.rows = c.fill(lens, 70)
        more = Cache(B, Hkv, d, page, budget, dtype, seed=5)
        self.dst = (more.table + c.P).contiguous()
        c.k, c.v, c.w = torch.cat([c.k, more.k]), torch.cat([c.v, more.v]), torch.cat([c.w, more.w])
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.M, self.z = torch.rand((B, Hkv, d, d)).cuda(), torch.rand((B, Hkv, d)).cuda()
        self.kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda")
        self.lens_out = torch.empty(B, dtype=torch.int32, device="cuda")
        self.sizes = (B, Hkv, d, c.k.shape[0], page, c.table.shape[1], extra, budget, recent, 0)
        need = binding.LIB.infini_attn_paged_evict_workspace_bytes(B, Hkv, d, page, c.table.shape[1], budget, 1)
        self.ws = torch.full((need // 4,), float("nan"), device="cuda")
        self.fn = binding.LIB.infini_attn_paged_evict if dtype == "bf16" else binding.LIB.infini_attn_paged_evict_f32

    def __call__(self):
        p = lambda t: ctypes.c_void_p(t.data_ptr())
        c = self.c
        assert self.fn(p(c.k), p(c.v), p(c.w), p(c.table), p(self.n), p(self.dst), p(self.lens_out), p(self.kept),
                       p(self.M), p(self.z), p(self.ws), self.ws.numel() * 4, *self.sizes,
                       ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_fold_that_gives_up_ends_and_is_reported(dtype):
    """The call ends, its selection and copies are those of any call, the status is read once, and the
    same call afterwards is correct."""
    x, y = Cut(dtype), Cut(dtype)
    with withheld():
        x()
        status = binding.infini_attn_device_status()
    assert status == TIMEOUT
    ok()
    y()
    ok()
    assert torch.equal(x.kept, y.kept) and torch.equal(x.lens_out, y.lens_out)
    for a, b in ((x.c.k, y.c.k), (x.c.v, y.c.v), (x.c.w, y.c.w)):
        assert same_bits(a, b)
    evict_case([3000, 130, 70, 20], 2, 64, 16, 64, 9, dtype, fold=True, seed=4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_fold_that_gives_up_adds_no_unwritten_piece(dtype):
    """No block completes a tile here, so M and z keep their bits (the workspace's pieces are NaN)."""
    x = Cut(dtype)
    M, z = x.M.clone(), x.z.clone()
    with withheld():
        x()
        assert binding.infini_attn_device_status() == TIMEOUT
    assert same_bits(x.M, M) and same_bits(x.z, z)
    x()                                    # the same rows again, from M and z as they were
    ok()
    for b, n in enumerate(x.lens):
        for h in range(2):
            K, V, _ = (r[h] for r in x.rows[b])
            gone = sorted(set(range(n)) - set(x.kept[b, h].tolist()))
            f = np.where(K[gone] > 0, K[gone] + 1, np.exp(np.minimum(K[gone], 0)))
            for got, old, add, size in ((x.M, M, f.T @ V[gone], f.T @ np.abs(V[gone])),
                                        (x.z, z, f.sum(0), f.sum(0))):
                assert np.all(np.abs(f64(got[b, h]) - f64(old[b, h]) - add)
                              <= (2.0 ** -17 + (n + 8) * 2.0 ** -24) * (size + np.abs(f64(old[b, h]))))


def test_an_unread_record_stops_later_folds():
    """Until the record is read, a call without any fault folds nothing; then it folds as ever."""
    x, y, z = Cut(), Cut(), Cut()
    M, zz = y.M.clone(), y.z.clone()
    with withheld():
        x()
    y()
    assert binding.infini_attn_device_status() == TIMEOUT
    ok()
    assert same_bits(y.M, M) and same_bits(y.z, zz)
    z.M.copy_(M), z.z.copy_(zz)
    y(), z()
    ok()
    assert torch.equal(y.M, z.M) and torch.equal(y.z, z.z) and not torch.equal(y.M, M)


def test_a_bad_page_is_reported_after_a_timeout():
    """Both records of one call reach the caller, one at a time."""
    x = Cut()
    x.c.table[0, 3] = x.c.k.shape[0]                   # past the pool
    with withheld():
        x()
        first = binding.infini_attn_device_status()
    assert (first, binding.infini_attn_device_status()) == (TIMEOUT, 6)
    ok()
