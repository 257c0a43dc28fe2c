"""The input layer's largest calls: the lookup's form of two units a lane, and more
workgroups, threads or units than one launch holds.

HIP refuses a launch of 2^32 threads or more, and the launches here are divided
or strided well below that; each test says how many it takes.  Values of sums are
small integers, whose fp32 sums are exact, so results are compared for equality.
"""
import numpy as np
import pytest
import torch

from gpu_harness import say
from oracle import input_layer as OI
from test_gpu_input_layer import PAIRS, T, close, drop_of
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


def _check_lookup_rows(out, lo, hi, ids, table, pos, period, drop, scale):
    """Rows lo .. hi - 1 of a lookup against the oracle."""
    at = np.arange(lo, hi) % period
    i = ids[lo:hi].cpu().numpy()
    ts, ps = table.cpu().double().numpy(), pos.cpu().double().numpy()
    d = dict(drop, row0=drop["row0"] + lo) if drop else None
    want = OI.lookup(i, ts, scale=scale, pos_table=ps, pos=at, drop=d)
    mag = OI.lookup(i, np.abs(ts), scale=scale, pos_table=np.abs(ps), pos=at)
    close(out[lo:hi], want, mag * OI.keep_scale(drop["p"] if drop else 0.0), 5, f"rows {lo} .. {hi}")


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("n,dim", [(16387, 4096), (41951, 1600), (86001, 777)])
@pytest.mark.parametrize("tt,ot", PAIRS)
def test_lookup_of_two_units_a_lane(tt, ot, n, dim, p):
    """From 2^23 units of 8 columns on some types and forms take two; one row a wave (4096),
    whole groups (1600) and an odd width, each with a last wave in part.  Every element equals that of the same
    rows looked up by halves, which take one unit a lane; some rows are checked
    against the oracle."""
    assert n * ((dim + 7) // 8) >= 1 << 23 > (n // 2 + 1) * ((dim + 7) // 8)
    say(f"lookup {n} of 301x{dim} {tt}->{ot} p={p}")
    g = torch.Generator(device="cuda").manual_seed(dim)
    flat = torch.randn(301 * dim + 3, generator=g, device="cuda").to(T[tt])
    table = flat[3:].view(301, dim)
    pos = torch.randn(97, dim, generator=g, device="cuda").to(T[tt])
    ids = torch.randint(-2, 304, (n,), generator=g, device="cuda")
    drop = drop_of(p, rows_at=70) if p else None
    period, scale = 101, 1.5                            # positions 97 .. 100 have no row
    whole = L.embedding(ids, table, scale=scale, pos_table=pos, pos_period=period,
                        drop=L.Dropout(**drop) if p else None, out_dtype=T[ot])
    half = n // 2
    for lo, hi in ((0, half), (half, n)):
        at = torch.arange(lo, hi, device="cuda") % period
        part = L.embedding(ids[lo:hi], table, scale=scale, pos_table=pos, pos=at,
                           drop=L.Dropout(**dict(drop, row0=70 + lo)) if p else None, out_dtype=T[ot])
        assert torch.equal(whole[lo:hi], part)
    for lo in (0, n // 3, n - 6):
        _check_lookup_rows(whole, lo, lo + 6, ids, table, pos, period, drop, scale)
    # without positions
    whole = L.embedding(ids, table, scale=scale, drop=L.Dropout(**drop) if p else None, out_dtype=T[ot])
    _check_lookup_rows(whole, n - 6, n, ids, table, torch.zeros_like(pos), period, drop, scale)


def test_dropout_of_more_units_than_a_launch_holds():
    """2^31 - 1 rows of one column in the first launch, the others in a second one."""
    rows = (1 << 31) + 1000
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    for lo, hi in _parts(rows):
        x[lo:hi, 0] = (torch.arange(lo, hi, device="cuda") % 251 - 125).to(torch.bfloat16)
    say(f"dropout {rows} x 1")
    d = drop_of(0.3, rows_at=5)
    out = L.dropout(x, L.Dropout(**d))
    for lo in (0, (1 << 31) - 51, rows - 100):
        xs = x[lo:lo + 100].cpu().double().numpy()
        close(out[lo:lo + 100], OI.dropout(xs, dict(d, row0=5 + lo)), np.abs(xs) * OI.keep_scale(0.3), 5, str(lo))
    for lo, hi in _parts(rows):
        assert torch.equal(L.dropout(x[lo:hi], L.Dropout(**dict(d, row0=5 + lo))), out[lo:hi]), lo
    # in place
    L.dropout(x, L.Dropout(**d), out=x)
    for lo, hi in _parts(rows):
        assert torch.equal(x[lo:hi], out[lo:hi]), lo


def test_lookup_of_more_units_than_a_launch_holds():
    """2^30 - 1 rows of two groups of columns in the first launch."""
    n, dim, period, border = (1 << 30) + 1000, 9, 777, (1 << 30) - 1
    g = torch.Generator(device="cuda").manual_seed(4)
    table = torch.randn(50, dim, generator=g, device="cuda").bfloat16()
    pos = torch.randn(period, dim, generator=g, device="cuda").bfloat16()
    ids = torch.randint(-1, 51, (n,), generator=g, device="cuda", dtype=torch.int32)
    say(f"lookup {n} of 50 x {dim}")
    d = drop_of(0.25, rows_at=11)
    out = L.embedding(ids, table, scale=2.0, pos_table=pos, pos_period=period, drop=L.Dropout(**d))
    for lo in (0, border - 50, n - 100):
        _check_lookup_rows(out, lo, lo + 100, ids, table, pos, period, d, 2.0)
    for lo in (border - 100000, n - 100000):
        at = (torch.arange(lo, lo + 100000, device="cuda") % period).int()
        part = L.embedding(ids[lo:lo + 100000], table, scale=2.0, pos_table=pos, pos=at,
                           drop=L.Dropout(**dict(d, row0=11 + lo)))
        assert torch.equal(out[lo:lo + 100000], part[:n - lo]), lo
