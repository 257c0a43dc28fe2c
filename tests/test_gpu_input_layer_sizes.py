"""The input layer's largest calls: more workgroups or threads than one launch holds.

HIP refuses a launch of 2^32 threads or more, and the launches here are divided
or strided well below that; each test says how many it takes.  Values are small
integers, whose fp32 sums are exact, so results are compared for equality.
"""
import numpy as np
import pytest
import torch

from gpu_harness import say
from zero_sharded_mixed_plan_amd import input_layer as L

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _free_gib():
    return torch.cuda.mem_get_info()[0] / 2 ** 30


def _parts(n, step=1 << 28):
    for lo in range(0, n, step):
        yield lo, min(n, lo + step)


def _nonzero_rows(m):
    """Rows of a matrix that hold anything but zeros (part by part: torch's own
    calls on more than 2^31 elements are not what is tested here)."""
    return [lo + int(r) for lo, hi in _parts(m.shape[0], 1 << 25)
            for r in torch.nonzero((m[lo:hi] != 0).any(1)).flatten().tolist()]


def _pattern(n, dim, mod):
    """dy[t, c] = (t + c) % mod - mod // 2 in bf16."""
    out = torch.empty(n, dim, dtype=torch.bfloat16, device="cuda")
    for lo, hi in _parts(n, 1 << 24):
        t = torch.arange(lo, hi, device="cuda")[:, None] + torch.arange(dim, device="cuda")
        out[lo:hi] = (t % mod - mod // 2).to(torch.bfloat16)
    return out


@pytest.mark.parametrize("rows,ids", [
    (1 << 27, True), (1 << 27, False),                 # 2^21 workgroups of 64 rows that zero
    ((1 << 30) + (1 << 22), True)])                    # 2^32 threads of them
def test_zeroing_in_several_launches(rows, ids):
    say(f"zeroing {rows} rows, ids {ids}")
    grad = torch.ones(rows, 8, dtype=torch.bfloat16, device="cuda")
    dy = _pattern(100, 8, 7)
    at = torch.arange(100, device="cuda") % 50 * (rows // 50) + 17 if ids else None
    L.embedding_grad(dy, at, grad, period=50)
    want = dy[:50].float() + dy[50:].float()
    touched = [int(v) for v in at[:50]] if ids else list(range(50))
    assert torch.equal(grad[torch.tensor(touched, device="cuda")].float(), want)
    nz = [touched[i] for i in torch.nonzero((want != 0).any(1)).flatten().tolist()]
    assert _nonzero_rows(grad) == nz


def _check_sums(dy, grad, period):
    n = dy.shape[0] // period * period
    want = torch.zeros(period, dy.shape[1], dtype=torch.float64, device="cuda")
    for lo, hi in _parts(n, period * 10000):
        want += dy[lo:hi].view(-1, period, dy.shape[1]).sum(0, dtype=torch.float64)
    want[:dy.shape[0] - n] += dy[n:].double()
    assert want.abs().max() < 2 ** 24 and want.abs().max() > 1000
    assert torch.equal(grad.double(), want)


def test_sums_and_joins_in_several_launches():
    """2^23 workgroups that sum, 2^20 and more that join: the position form, whose
    rows recur half a million times."""
    if _free_gib() < 130:
        pytest.skip("needs 130 GiB of free device memory")
    n, period = (1 << 29) + (1 << 20), 1000
    dy = _pattern(n, 8, 8)                              # the mean is -1/2
    say(f"{n} rows of dy")
    grad = L.embedding_grad(dy, None, torch.empty(period, 8, device="cuda"), period=period)
    _check_sums(dy, grad, period)


def test_sorted_sums_in_several_launches():
    """2^20 and more workgroups that sum; 2^22 and more positions per wave of the
    order pass, which then keeps no list and reads the ids again."""
    n, period = (1 << 26) + (1 << 20), 1000
    dy = _pattern(n, 8, 8)
    ids = (torch.arange(n, device="cuda") % period).int()
    say(f"{n} ids")
    grad = L.embedding_grad(dy, ids, torch.empty(period, 8, device="cuda"))
    _check_sums(dy, grad, period)


def test_element_kernels_beyond_one_launch():
    """Tensors of fewer than 8 elements beside results of more than 2^32."""
    n, dim = 1_500_000_000, 3
    table = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]], dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(n, dtype=torch.int32, device="cuda")
    for lo, hi in _parts(n):
        ids[lo:hi] = torch.arange(lo, hi, device="cuda") % 5 - 1
    say(f"lookup of {n} x {dim}")
    out = L.embedding(ids, table, scale=2.0)
    rows = torch.cat([torch.zeros_like(table[:1]), 2 * table, torch.zeros_like(table)])      # ids -1 .. 3
    for lo, hi in _parts(n, 1 << 27):
        assert torch.equal(out[lo:hi], rows[ids[lo:hi].long() + 1]), lo
    del ids
    grad = out.fill_(7.0)
    say(f"gradient of {n} x {dim}")
    at = torch.tensor([n - 2, 5], device="cuda")
    L.embedding_grad(table, at, grad)
    assert torch.equal(grad[at], table) and _nonzero_rows(grad) == [5, n - 2]
