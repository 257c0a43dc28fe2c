"""The input layer on the GPU against the float64 oracle: embedding lookup, its
gradient, dropout, and a run of them around the sharded step.

Error bounds (u = half a step of a type relative to the value, e = 2^-24):
  lookup / dropout  scale * w, + pos, * ks, + residual and the rounded ks are at
                    most 5 fp32 roundings of numbers no larger than the sum of the
                    terms' magnitudes: 5 e mag + u |y|
  gradient          a sum of n terms (fewer than n roundings of partial sums, each
                    at most the sum of magnitudes), the factor and its product,
                    the addition to the old value: (n + 4) e mag + u |y|
plus half the smallest subnormal of the output type.  Products of the two
bounds are covered by a factor of 1.01.
"""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_plan_amd as Z
from oracle import input_layer as OI
from oracle import step as OS
from gpu_harness import say, storage
from zero_sharded_mixed_plan_amd import input_layer as L
from zero_sharded_mixed_plan_amd.optim import ZeroAdam

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24
SUB = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
GUARD = 77.0


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def close(got: torch.Tensor, want: np.ndarray, mag: np.ndarray, ops, what=""):
    u = torch.finfo(got.dtype).eps / 2
    tol = 1.01 * (ops * E * mag + u * np.abs(want)) + SUB[got.dtype]
    g = got.detach().cpu().double().numpy().reshape(want.shape)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} wrong, first {np.argwhere(bad)[:3].tolist()}: " \
                          f"{g[bad][:3]} for {want[bad][:3]}, tolerance {tol[bad][:3]}"


class Mat:
    """[rows, cols] of a type inside a guarded flat buffer: element offset
    `off`, rows `ld` apart; the elements around and between must not change."""

    def __init__(self, rows, cols, dt, off=0, ld=None, data=None, fill=GUARD):
        self.ld = ld or cols
        self.flat = torch.full((off + max(rows, 1) * self.ld + 16,), fill, dtype=T[dt], device="cuda")
        self.v = self.flat[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]
        if data is not None:
            self.v.copy_(torch.as_tensor(data))
        inside = torch.zeros_like(self.flat, dtype=torch.bool)
        inside[off:off + rows * self.ld].view(rows, self.ld)[:, :cols] = True
        self.outside = ~inside
        self.fill = fill

    def check(self):
        assert bool((self.flat[self.outside] == self.fill).all()), "written outside the matrix"

    def f64(self):
        return self.v.cpu().double().numpy()


def drop_of(p, rows_at=0, step=5, seed=0xABCDEF0123456789, site=4):
    return dict(p=p, seed=seed, site=site, step=step, row0=rows_at)


def L_drop(d):
    return None if d is None else L.Dropout(**d)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

DROPOUT = [  # rows, cols, x type, out type, residual, p, offset, ld - cols
    (1, 1, "f32", "f32", False, 0.5, 0, 0),
    (3, 7, "bf16", "bf16", True, 0.1, 1, 0),
    (5, 8, "f16", "f16", False, 0.25, 3, 5),
    (17, 777, "f16", "f32", True, 0.1, 3, 2),
    (33, 1600, "bf16", "bf16", True, 0.1, 0, 0),
    (9, 2049, "f32", "bf16", True, 0.9, 1, 7),
    (64, 513, "f32", "f16", False, 0.0, 1, 0),
    (4, 100, "bf16", "f32", True, 1.0, 0, 0),
    (1, 300001, "bf16", "f16", False, 0.5, 5, 0),
    (70000, 9, "f16", "bf16", True, 0.3, 1, 1),
]


@pytest.mark.parametrize("rows,cols,xt,ot,res,p,off,pad", DROPOUT)
def test_dropout(rows, cols, xt, ot, res, p, off, pad):
    say(f"dropout {rows}x{cols} {xt}->{ot} p={p}")
    g = np.random.default_rng(rows * 7 + cols)
    x = Mat(rows, cols, xt, off, cols + pad, g.normal(size=(rows, cols)))
    r = Mat(rows, cols, ot, off + 2, cols + pad, g.normal(size=(rows, cols))) if res else None
    out = Mat(rows, cols, ot, off, cols + 2 * pad)
    d = drop_of(p, rows_at=123)
    L.dropout(x.v, L_drop(d), residual=r.v if res else None, out=out.v)
    xs, rs = x.f64(), (r.f64() if res else None)
    want = OI.dropout(xs, d, rs)
    mag = np.abs(xs) * OI.keep_scale(p) + (np.abs(rs) if res else 0)
    close(out.v, want, mag, 5)
    for m in (x, out):
        m.check()
    if p == 1.0 or p == 0.0:
        assert np.array_equal(want, (rs if p else xs + (rs if res else 0)))


@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_dropout_in_place_and_backward(xt):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(31, 250, generator=g, device="cuda").to(T[xt])
    d = L.Dropout(0.4, seed=9, site=1, step=2)
    want = L.dropout(x, d)
    a = x.clone()
    assert L.dropout(a, d, out=a) is a and torch.equal(a, want)
    r = torch.randn(31, 250, generator=g, device="cuda").to(T[xt])
    want_r = L.dropout(x, d, residual=r)
    b = r.clone()
    L.dropout(x, d, residual=b, out=b)
    assert torch.equal(b, want_r)
    # the backward pass keeps what the forward pass kept: ones come back as 0 or ks
    ks = np.float32(OI.keep_scale(0.4))
    back = L.dropout(torch.ones(31, 250, device="cuda"), d)
    assert set(back.unique().tolist()) == {0.0, float(ks)}
    assert torch.equal(back == 0, want == 0)
    # a matrix, and the same rows as a batch of sequences
    assert torch.equal(L.dropout(x[:30].view(5, 6, 250), d).view(30, 250), want[:30])


def test_dropped_elements_hide_infinities_and_nan():
    keep = torch.from_numpy(OI.keep(40, 90, **drop_of(0.5))).cuda()
    x = torch.randn(40, 90, device="cuda")
    bad = torch.where(keep, x, torch.full_like(x, float("nan")))
    bad[::2] = torch.where(keep[::2], x[::2], torch.full_like(x[::2], float("inf")))
    d = L.Dropout(**drop_of(0.5))
    assert torch.equal(L.dropout(bad, d), L.dropout(x, d))
    # a kept one stays what it is
    x[~keep] = 0
    r, c = torch.nonzero(keep)[5].tolist()
    x[r, c] = float("inf")
    y = L.dropout(x, d)
    assert torch.isinf(y).sum() == 1 and torch.isinf(y[r, c])
    # p = 1 drops everything, whatever it is
    assert not L.dropout(torch.full((3, 9), float("nan"), device="cuda"), L.Dropout(1.0)).any()


def test_dropout_empty_and_host_step_against_device_step():
    assert L.dropout(torch.empty(0, 5, device="cuda"), L.Dropout(0.5)).shape == (0, 5)
    assert L.dropout(torch.empty(4, 0, device="cuda"), L.Dropout(0.5)).shape == (4, 0)
    x = torch.randn(12, 200, device="cuda")
    s = torch.tensor([0x1_0000_0007], device="cuda")      # the low 32 bits count
    assert torch.equal(L.dropout(x, L.Dropout(0.3, seed=1, step=s)), L.dropout(x, L.Dropout(0.3, seed=1, step=7)))


# ---------------------------------------------------------------------------
# lookup
# ---------------------------------------------------------------------------

LOOKUP = [  # n, rows, dim, table, out, id type, scale, positions, p, offset, pad, id0
    (1, 10, 4096, "bf16", "bf16", torch.int64, 1.0, 0, 0.0, 0, 0, 0),
    (1, 1, 1, "f32", "f32", torch.int32, 3.0, 1, 0.0, 1, 0, 0),
    (7, 3, 9, "f16", "f32", torch.int64, 0.5, 2, 0.2, 1, 3, 0),
    (300, 50, 777, "f16", "bf16", torch.int32, 28.0, 33, 0.25, 3, 1, -7),
    (129, 1000, 1600, "bf16", "bf16", torch.int64, 40.0, 64, 0.1, 0, 0, 5),
    (1000, 257, 520, "f32", "f16", torch.int32, 1.0, 0, 0.5, 1, 0, 1 << 20),
    (5000, 31, 130, "bf16", "f32", torch.int64, 2.0, 5000, 0.0, 7, 0, 0),
    (64, 9, 8192, "f32", "bf16", torch.int32, 1.0, 10, 1.0, 0, 8, 0),
]


@pytest.mark.parametrize("n,rows,dim,tt,ot,it,scale,period,p,off,pad,id0", LOOKUP)
def test_lookup(n, rows, dim, tt, ot, it, scale, period, p, off, pad, id0):
    say(f"lookup {n} of {rows}x{dim} {tt}->{ot} p={p}")
    g = np.random.default_rng(n + dim)
    table = Mat(rows, dim, tt, off, dim + pad, g.normal(size=(rows, dim)))
    ids = g.integers(id0 - 2, id0 + rows + 2, size=n)           # some outside
    ids[:2] = [id0, id0 + rows - 1][:n]
    out = Mat(n, dim, ot, off, dim + pad)
    pos = Mat(period, dim, tt, off + 2, dim, g.normal(size=(period, dim))) if period else None
    d = drop_of(p, rows_at=77) if p else None
    ti = torch.from_numpy(ids).to(it).cuda()
    L.embedding(ti, table.v, scale=scale, id0=id0, pos_table=pos.v if pos else None, pos_period=period,
                drop=L_drop(d), out=out.v)
    ts, ps = table.f64(), pos.f64() if pos else None
    kw = dict(scale=scale, id0=id0, pos_period=period)
    want = OI.lookup(ids, ts, pos_table=ps, drop=d, **kw)
    mag = OI.lookup(ids, np.abs(ts), pos_table=np.abs(ps) if period else None, **kw) * OI.keep_scale(p)
    close(out.v, want, mag, 5)
    out.check()
    # explicit positions, some outside the table
    if period:
        at = g.integers(-1, period + 2, size=n)
        got = L.embedding(ti, table.v, scale=scale, id0=id0, pos_table=pos.v,
                          pos=torch.from_numpy(at).to(it).cuda(), drop=L_drop(d), out_dtype=torch.float32)
        want = OI.lookup(ids, ts, scale=scale, id0=id0, pos_table=ps, pos=at, drop=d)
        close(got, want, mag + np.abs(ps).max() * OI.keep_scale(p), 5)


def test_lookup_ids_far_outside_and_unread_rows():
    """Ids anywhere in their type read zeros; rows that no id names may hold NaN."""
    table = torch.full((6, 24), float("nan"), device="cuda")
    table[2] = 3.0
    far = torch.tensor([2**63 - 1, -2**63, -1, 6, 2, 2**40, -2**62], device="cuda")
    y = L.embedding(far, table)
    want = torch.zeros(7, 24, device="cuda")
    want[4] = 3.0
    assert torch.equal(y, want)
    # the table of another rank's rows: ids around 2^63 do not wrap into it
    y = L.embedding(torch.tensor([-2**63, 2**63 - 4], device="cuda"), table, id0=2**63 - 6)
    assert torch.equal(y, want[3:5])
    # a table with no rows here
    assert not L.embedding(torch.tensor([[0, 1]], device="cuda"), table[:0]).any()
    assert L.embedding(torch.empty(0, dtype=torch.int32, device="cuda"), table).shape == (0, 24)


def test_lookup_split_by_rows_adds_up():
    """A table split over ranks by rows (the dim-0 layout): the parts' outputs
    sum to the whole table's."""
    table = torch.randn(103, 65, device="cuda")
    ids = torch.randint(0, 103, (50,), device="cuda")
    whole = L.embedding(ids, table, scale=2.0)
    parts = sum(L.embedding(ids, table[a:a + 26], scale=2.0, id0=a) for a in range(0, 103, 26))
    assert torch.equal(whole, parts)


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------

def _ids(kind, n, rows, rng):
    if kind == "uniform":
        return rng.integers(0, rows, size=n)
    if kind == "zipf":
        w = 1 / (np.arange(rows) + 2.7)
        return rng.choice(rows, size=n, p=w / w.sum())
    if kind == "one":
        return np.full(n, rows - 1)
    if kind == "two":                                 # a border inside a tile, not in its middle
        return np.where(np.arange(n) < n // 3 + 1, rows // 2, 0)
    if kind == "outside":
        return rng.integers(-5, rows + 5, size=n)
    if kind == "in turn":                             # every row equally often
        return rng.permutation(np.arange(n) % rows)
    if kind == "none inside":
        return np.full(n, -1)
    if kind == "each once":
        return rng.permutation(rows)[:n]
    raise KeyError(kind)


GRAD = [  # n, rows, dim, dy, grad, ids, kind, scale, p, offset, pad, id0
    (0, 5, 16, "f32", "f32", torch.int64, "uniform", 1.0, 0.0, 0, 0, 0),
    (1, 1, 1, "f32", "f32", torch.int32, "one", 1.0, 0.0, 0, 0, 0),
    (1, 300, 4096, "bf16", "bf16", torch.int64, "one", 1.0, 0.1, 0, 0, 0),
    (64, 256, 64, "f32", "f32", torch.int64, "zipf", 8.0, 0.0, 0, 0, 0),
    (15, 40, 7, "f16", "f32", torch.int32, "uniform", 0.5, 0.3, 1, 3, 0),
    (16, 40, 8, "f16", "f16", torch.int32, "two", 0.5, 0.0, 1, 0, 0),
    (17, 16, 9, "f32", "bf16", torch.int64, "one", 2.0, 0.5, 3, 0, 0),
    (100, 700, 513, "bf16", "f32", torch.int64, "each once", 1.0, 0.0, 0, 1, 0),
    (1000, 9, 40, "bf16", "f32", torch.int32, "two", 1.0, 0.25, 5, 0, 3),
    (3000, 500, 777, "f16", "f32", torch.int64, "zipf", 28.0, 0.25, 3, 2, 0),
    (4096, 1000, 72, "bf16", "bf16", torch.int64, "one", 1.0, 0.0, 0, 0, 0),
    (5000, 300, 100, "f32", "f32", torch.int32, "outside", 1.0, 0.1, 1, 0, 0),
    (777, 300, 100, "f32", "f32", torch.int32, "none inside", 1.0, 0.1, 1, 0, 0),
    (20000, 50, 24, "f32", "f32", torch.int64, "uniform", 1.0, 0.0, 0, 0, -4),
    (70001, 2000, 16, "bf16", "f32", torch.int32, "zipf", 1.0, 0.1, 0, 0, 0),
    (300, 300000, 24, "bf16", "bf16", torch.int64, "uniform", 1.0, 0.0, 0, 0, 0),
    (200, 64, 1100, "f32", "f32", torch.int64, "zipf", 1.0, 1.0, 0, 0, 0),
    # the most rows a workgroup of the order pass counts, with its longest lists
    (20000, 262144, 8, "f32", "f32", torch.int32, "zipf", 1.0, 0.0, 0, 0, 0),
    # three launches and one, on either side of the rule between them
    (1024, 900, 512, "bf16", "f32", torch.int64, "two", 1.0, 0.1, 0, 0, 0),
    (1025, 900, 512, "bf16", "f32", torch.int64, "two", 1.0, 0.1, 0, 0, 0),
    # few ids into many rows, past the one-launch form
    (60, 70000, 130, "bf16", "f32", torch.int32, "zipf", 1.0, 0.1, 3, 0, 0),
    (1, 33000, 260, "f32", "f32", torch.int64, "one", 1.0, 0.0, 0, 1, 0),
    # runs of exactly a chunk, and one more
    (8 * 41, 41, 600, "f32", "f32", torch.int64, "uniform", 1.0, 0.0, 0, 0, 0),
    (40000, 1250, 24, "bf16", "f32", torch.int64, "in turn", 1.0, 0.0, 0, 0, 0),
    (41250, 1250, 24, "bf16", "f32", torch.int64, "in turn", 1.0, 0.0, 0, 0, 0),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,rows,dim,dt,gt,it,kind,scale,p,off,pad,id0", GRAD)
def test_gradient(n, rows, dim, dt, gt, it, kind, scale, p, off, pad, id0, accumulate):
    say(f"gradient {n} -> {rows}x{dim} {dt}->{gt} {kind} p={p} accumulate={accumulate}")
    rng = np.random.default_rng(n + dim)
    ids = _ids(kind, n, rows, rng) + id0
    dy = Mat(n, dim, dt, off, dim + pad, rng.normal(size=(n, dim)))
    grad = Mat(rows, dim, gt, off, dim + pad, rng.normal(size=(rows, dim)) if accumulate else None)
    old = grad.f64() if accumulate else np.zeros((rows, dim))
    d = drop_of(p, rows_at=31) if p else None
    got = L.embedding_grad(dy.v, torch.from_numpy(ids).to(it).cuda(), grad.v, scale=scale, id0=id0,
                           drop=L_drop(d), accumulate=accumulate)
    assert got is grad.v
    want, cnt, mag = OI.lookup_grad(dy.f64(), ids, rows, scale=scale, id0=id0, drop=d)
    if accumulate:                                    # rows without an id keep their bits
        idle = torch.from_numpy(cnt == 0).cuda()
        assert np.array_equal(grad.v[idle].cpu().double().numpy(), old[cnt == 0])
    else:
        assert not grad.v[torch.from_numpy(cnt == 0).cuda()].any()
    close(grad.v, want + old, mag + np.abs(old), (cnt + 4)[:, None])
    grad.check()
    # the same call again gives the same bits
    again = Mat(rows, dim, gt, off, dim + pad, old if accumulate else None)
    L.embedding_grad(dy.v, torch.from_numpy(ids).to(it).cuda(), again.v, scale=scale, id0=id0, drop=L_drop(d),
                     accumulate=accumulate)
    assert torch.equal(again.v, grad.v)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,rows,dim,period,id0,p", [
    (1, 1, 8, 1, 0, 0.0), (10, 4, 9, 4, 0, 0.1), (10, 7, 33, 4, 0, 0.0), (8192, 1024, 40, 1024, 0, 0.1),
    (1000, 3, 520, 1, 0, 0.0), (5003, 1, 24, 1, 0, 0.3), (50, 100, 16, 99, 0, 0.0), (37, 20, 16, 1 << 40, 0, 0.0),
    (999, 30, 17, 100, 50, 0.1), (999, 30, 17, 100, 90, 0.0), (999, 30, 17, 100, -10, 0.0), (999, 30, 17, 100, 200, 0.0),
    (70000, 17, 16, 23, 3, 0.0), (0, 5, 8, 3, 0, 0.0), (999, 30, 17, 3, 50, 0.0)])
def test_gradient_of_positions(n, rows, dim, period, id0, p, accumulate):
    say(f"positions {n} -> {rows}x{dim} period {period} id0 {id0}")
    rng = np.random.default_rng(n + dim)
    dy = Mat(n, dim, "bf16", 1, dim, rng.normal(size=(n, dim)))
    grad = Mat(rows, dim, "f32", 3, dim + 1, rng.normal(size=(rows, dim)) if accumulate else None)
    old = grad.f64() if accumulate else np.zeros((rows, dim))
    d = drop_of(p) if p else None
    L.embedding_grad(dy.v, None, grad.v, period=period, id0=id0, drop=L_drop(d), accumulate=accumulate)
    want, cnt, mag = OI.lookup_grad(dy.f64(), None, rows, id0=id0, period=period, drop=d)
    if accumulate:
        assert np.array_equal(grad.f64()[cnt == 0], old[cnt == 0])
    close(grad.v, want + old, mag + np.abs(old), (cnt + 4)[:, None])
    grad.check()


def test_gradient_against_differences():
    """The lookup is linear in its tables, so a central difference with a power
    of two step is the gradient up to the fp32 roundings of the two outputs."""
    rng = np.random.default_rng(8)
    table = torch.from_numpy(rng.normal(size=(11, 20)).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.normal(size=(6, 20)).astype(np.float32)).cuda()
    ids = torch.tensor([3, 3, 7, 0, 12, 3, 10, -1, 7], device="cuda")
    c = torch.from_numpy(rng.normal(size=(9, 20))).cuda()
    d = L.Dropout(0.25, seed=4, site=1, step=9)

    def f(tab, ps):
        return (L.embedding(ids, tab, scale=3.0, pos_table=ps, pos_period=6, drop=d).double() * c).sum().item()

    g = L.embedding_grad(c.float(), ids, torch.empty_like(table), scale=3.0, drop=d)
    gp = L.embedding_grad(c.float(), None, torch.empty_like(pos), period=6, drop=d)
    h = 0.5
    # nine outputs at most change, each off by 5 roundings of at most |y| < 64
    tol = 2 * 9 * 5 * E * 64 * c.abs().max().item() / (2 * h) + 1e-5
    for which, grad in ((0, g), (1, gp)):
        for r, col in ((0, 0), (3, 5), (3, 19), (5, 7), (2, 11)):
            lo, hi = [table.clone(), pos.clone()], [table.clone(), pos.clone()]
            lo[which][r, col] -= h
            hi[which][r, col] += h
            diff = (f(*hi) - f(*lo)) / (2 * h)
            assert abs(diff - grad[r, col].item()) <= tol


def test_gradient_hides_dropped_infinities_and_padding():
    n, dim = 60, 130
    keep = torch.from_numpy(OI.keep(n, dim, **drop_of(0.5))).cuda()
    x = torch.randn(n, dim, device="cuda")
    ids = torch.arange(n, device="cuda") % 7
    ids[::5] = -1
    bad = torch.where(keep, x, torch.full_like(x, float("inf")))
    bad[::5] = float("nan")                           # rows of padding ids
    d = L.Dropout(**drop_of(0.5))
    a = L.embedding_grad(x, ids, torch.empty(7, dim, device="cuda"), drop=d)
    b = L.embedding_grad(bad, ids, torch.empty(7, dim, device="cuda"), drop=d)
    assert torch.equal(a, b)


def test_empty_batch_zeroes_the_gradient():
    """No ids: every row is zero, with an id array and without, through the C call."""
    for rows, dim in ((5, 40), (3000, 600)):
        for accumulate in (0, 1):
            grad = torch.full((rows, dim), 3.0, device="cuda")
            ws = torch.empty(Z.zero_embed_grad_ws_bytes(0, rows, dim), dtype=torch.uint8, device="cuda")
            a = Z.zero_embed_grad_args_t()
            a.dy, a.ids, a.id_bytes = ws.data_ptr(), ws.data_ptr(), 8
            a.dim, a.rows, a.ld_grad, a.ld_dy = dim, rows, dim, dim
            a.scale, a.grad, a.accumulate = 1.0, grad.data_ptr(), accumulate
            a.ws, a.ws_bytes = ws.data_ptr(), ws.numel()
            Z.zero_embed_grad(a, torch.cuda.current_stream().cuda_stream)
            assert bool((grad == (3.0 if accumulate else 0.0)).all())
            ids = torch.empty(0, dtype=torch.int64, device="cuda")
            L.embedding_grad(torch.empty(0, dim, device="cuda"), ids, grad, accumulate=bool(accumulate))
            assert bool((grad == (3.0 if accumulate else 0.0)).all())


def test_workspace_of_a_larger_call_serves_a_smaller_one():
    ws = L.embedding_grad_workspace(5000, 400, 100)
    ws.fill_(0xFF)
    for n in (5000, 17, 900):
        dy = torch.randn(n, 100, device="cuda")
        ids = torch.randint(0, 400, (n,), device="cuda")
        a = L.embedding_grad(dy, ids, torch.empty(400, 100, device="cuda"), workspace=ws)
        assert torch.equal(a, L.embedding_grad(dy, ids, torch.empty(400, 100, device="cuda")))
    with pytest.raises(RuntimeError, match="workspace"):
        L.embedding_grad(torch.randn(6000, 100, device="cuda"), torch.zeros(6000, dtype=torch.int64, device="cuda"),
                         torch.empty(400, 100, device="cuda"), workspace=ws)


def test_offsets_past_32_bits():
    """Tables, gradients and activations of more than 2^32 bytes."""
    rows, dim = 540_000, 4096                          # 4.4 GB in bf16
    table = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    table[-1] = 5.0
    table[rows // 2] = 3.0
    ids = torch.tensor([rows - 1, 0, rows // 2], device="cuda")
    y = L.embedding(ids, table)
    assert (y[0] == 5).all() and (y[1] == 0).all() and (y[2] == 3).all()
    say("wide table read")
    grad = table
    grad.fill_(1.0)
    L.embedding_grad(y, ids, grad)
    assert (grad[-1] == 5).all() and (grad[rows // 2] == 3).all()
    assert grad.count_nonzero().item() == 2 * dim
    say("wide gradient written")
    dy = table                                        # 540000 tokens, one of them the only one of row 1
    dy.fill_(0.0)
    dy[-1] = 2.0
    dy[-2] = 4.0
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ids[-1] = 1
    g = L.embedding_grad(dy, ids, torch.empty(3, dim, device="cuda"))
    assert (g[0] == 4).all() and (g[1] == 2).all() and not g[2].any()
    say("wide activations summed")
    z = L.dropout(dy, None)
    assert torch.equal(z[-2:], dy[-2:]) and z.count_nonzero().item() == 2 * dim


# ---------------------------------------------------------------------------
# streams, graphs, and the run around the step
# ---------------------------------------------------------------------------

def test_calls_on_two_streams_at_once():
    g = torch.Generator(device="cuda").manual_seed(1)
    work = []
    for i in range(2):
        n, rows, dim = 6000 + i, 2000 + 3 * i, 512 + 8 * i
        dy = torch.randn(n, dim, generator=g, device="cuda")
        ids = torch.randint(0, rows, (n,), generator=g, device="cuda")
        work.append((dy, ids, rows, dim))
    serial = [L.embedding_grad(dy, ids, torch.empty(r, d, device="cuda")) for dy, ids, r, d in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    outs = [[torch.empty(r, d, device="cuda") for _ in range(5)] for _, _, r, d in work]
    torch.cuda.synchronize()
    for k in range(5):
        for s, (dy, ids, r, d), o in zip(streams, work, outs):
            with torch.cuda.stream(s):
                L.embedding_grad(dy, ids, o[k])
    torch.cuda.synchronize()
    for want, got in zip(serial, outs):
        assert all(torch.equal(want, x) for x in got)


def test_graph_draws_a_new_mask_at_every_replay():
    """Lookup, dropout and gradients captured in one graph, the step number in
    device memory: each replay equals the eager calls at that step."""
    g = torch.Generator(device="cuda").manual_seed(2)
    n, rows, dim, ctx = 500, 300, 136, 100
    table = torch.randn(rows, dim, generator=g, device="cuda")
    pos = torch.randn(ctx, dim, generator=g, device="cuda")
    ids = torch.randint(-1, rows, (n,), generator=g, device="cuda")
    dy = torch.randn(n, dim, generator=g, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(s):
        d0, d1 = L.Dropout(0.2, seed=7, site=0, step=s), L.Dropout(0.2, seed=7, site=1, step=s)
        h = L.embedding(ids, table, pos_table=pos, pos_period=ctx, drop=d0)
        r = L.dropout(dy, d1, residual=h)
        gt = L.embedding_grad(dy, ids, torch.empty_like(table), drop=d0)
        gp = L.embedding_grad(dy, None, torch.empty_like(pos), period=ctx, drop=d0)
        return h, r, gt, gp

    run(step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(step)
    seen = []
    for replay in range(4):
        step.fill_(replay + 3)
        graph.replay()
        torch.cuda.synchronize()
        eager = run(replay + 3)                       # eager work between replays
        torch.cuda.synchronize()
        for a, b in zip(outs, eager):
            assert torch.equal(a, b), f"replay {replay}"
        seen.append(outs[0].clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("captured", [False, True])
def test_training_steps_of_an_input_layer(captured):
    """GPT-2's input layer, tied output head, trained by the sharded step (one
    rank): lookup of words and positions with dropout, a residual dropout, the
    word gradient added to the head's, the position gradient, the AdamW step with
    control in device memory; eager, and as a captured graph of two steps."""
    V, D, CTX, B, STEPS = 211, 72, 24, 3, 6
    rng = np.random.default_rng(5)
    n = B * CTX
    master = torch.from_numpy(rng.normal(0, 0.05, V * D + CTX * D).astype(np.float32))
    opt = ZeroAdam([V * D, CTX * D], 1, 0, lr=1e-2, weight_decay=0.1, grad_dtype=torch.bfloat16,
                   param_dtype=torch.bfloat16, master=master.cuda(), device_control=True)
    wte, wpe = opt.param(0, (V, D)), opt.param(1, (CTX, D))
    opt.gather.copy_(master[:opt.gather.numel()].cuda())
    flat = torch.zeros(1, opt.plan.padded_numel, dtype=torch.bfloat16, device="cuda")
    g_wte, g_wpe = opt.grad_view(flat[0], 0, (V, D)), opt.grad_view(flat[0], 1, (CTX, D))
    ids = torch.from_numpy(rng.integers(0, V, size=(B, CTX))).cuda()
    head = torch.from_numpy(rng.normal(0, 1e-2, (V, D)).astype(np.float32)).cuda().to(torch.bfloat16)
    target = torch.from_numpy(rng.normal(0, 1, (B, CTX, D)).astype(np.float32)).cuda()
    d0, d1 = opt.dropout(0.1, seed=11, site=0), opt.dropout(0.1, seed=11, site=1)
    hs = []

    def step():
        h = L.embedding(ids, wte, pos_table=wpe, pos_period=CTX, drop=d0, out_dtype=torch.float32)
        y = L.dropout(h, d1, residual=h)
        dy = (y - target) * 1e-2
        dh = L.dropout(dy, d1, residual=dy)           # through the branch and the residual
        g_wte.copy_(head)                             # what the tied head's backward pass left
        L.embedding_grad(dh, ids, g_wte, drop=d0, accumulate=True)
        L.embedding_grad(dh, None, g_wpe, period=CTX, drop=d0)
        opt.step(flat, full=True)
        return h, dh

    if captured:
        state0 = [b.clone() for b in opt._state[0]]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):                    # warm-up of both parities, then back to the start
            step()
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for b, b0 in zip(opt._state[0], state0):
            b.copy_(b0)
        c = opt.ctl.read()
        c.step = 0
        opt.ctl.write(c)
        opt.gather.copy_(master[:opt.gather.numel()].cuda())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = []
            for _ in range(2):
                h, dh = step()
                kept.append((h, dh, flat.clone(), opt.gather.clone()))
        torch.cuda.synchronize()

    p, m, v = (master.numpy().copy(), np.zeros(master.numel(), np.float32), np.zeros(master.numel(), np.float32))
    w16 = master.to(torch.bfloat16)
    for t in range(STEPS):
        if captured:
            if t % 2 == 0:
                graph.replay()
                torch.cuda.synchronize()
                torch.randn(1 << 18, device="cuda").sum()          # eager work between replays
            h, dh, fl, gath = kept[t % 2]
        else:
            h, dh = step()
            fl, gath = flat, opt.gather
        torch.cuda.synchronize()
        hs.append(h.clone())
        # the forward pass from the parameters before this step
        tab, pos = w16[:V * D].double().numpy().reshape(V, D), w16[V * D:].double().numpy().reshape(CTX, D)
        drop = dict(p=0.1, seed=11, site=0, step=t, row0=0)
        flat_ids = ids.cpu().numpy().reshape(-1)
        want = OI.lookup(flat_ids, tab, pos_table=pos, pos_period=CTX, drop=drop)
        mag = OI.lookup(flat_ids, np.abs(tab), pos_table=np.abs(pos), pos_period=CTX) * OI.keep_scale(0.1)
        close(h, want, mag, 5, f"step {t} forward")
        # the gradients from the device's own dh
        dhs = dh.cpu().double().numpy().reshape(n, D)
        hd = head.cpu().double().numpy()
        want, cnt, mag = OI.lookup_grad(dhs, flat_ids, V, drop=drop)
        got = fl[0, :V * D].view(V, D)
        close(got, want + hd, mag + np.abs(hd), (cnt + 4)[:, None], f"step {t} words")
        assert torch.equal(got[torch.from_numpy(cnt == 0).cuda()], head[torch.from_numpy(cnt == 0).cuda()])
        want, cnt, mag = OI.lookup_grad(dhs, None, CTX, period=CTX, drop=drop)
        close(fl[0, V * D:].view(CTX, D), want, mag, (cnt + 4)[:, None], f"step {t} positions")
        # the step from the device's own gradients, bit for bit
        res = OS.shard_step([storage(fl[0])], "bf16", "bf16", 1, p, m, v, lr=1e-2, weight_decay=0.1, t=t + 1)
        assert not res.flag
        p, m, v = res.master, res.m, res.v
        assert np.array_equal(storage(gath), res.params)
        w16 = torch.from_numpy(res.params.view(np.int16).copy()).view(torch.bfloat16)
    assert opt.t == STEPS
    say(f"input layer trained {STEPS} steps, captured={captured}")


def test_step_views():
    opt = ZeroAdam([(10, 6), (7,), (4, 3)], 2, 1, lr=1e-3, layout="dim0")
    assert opt.param(0).shape == (10, 6) and opt.param(2).shape == (4, 3) and opt.param(1).shape == (7,)
    assert opt.param(0).data_ptr() == opt.gather.data_ptr()
    off = opt.plan.tensor(2)[1]
    assert opt.param(2).data_ptr() == opt.gather.data_ptr() + 2 * off
    g = torch.zeros(opt.plan.padded_numel, device="cuda")
    assert opt.grad_view(g, 2).data_ptr() == g.data_ptr() + 4 * off
    with pytest.raises(ValueError, match="flat gradient"):
        opt.grad_view(g[1:], 0)
    assert opt.dropout(0.1).p == 0.1


@pytest.mark.parametrize("n,dim", [(1, 1), (1, 7), (1, 8), (1, 9), (2, 3), (3, 3), (7, 1), (8, 1), (9, 1), (4, 2),
                                   (40, 3), (5, 15), (33, 12)])
@pytest.mark.parametrize("dt,gt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_tensors_of_a_few_elements_at_the_end_of_memory(n, dim, dt, gt):
    """The vector accesses near the ends of the smallest tensors: every operator at the
    end of its own allocation's used part, with NaN right behind every tensor."""
    rng = np.random.default_rng(n * 100 + dim)
    d = drop_of(0.3, rows_at=2)
    x = Mat(n, dim, dt, 3, dim, rng.normal(size=(n, dim)), fill=float("nan"))
    r = Mat(n, dim, gt, 1, dim, rng.normal(size=(n, dim)), fill=float("nan"))
    y = L.dropout(x.v, L_drop(d), residual=r.v)
    close(y, OI.dropout(x.f64(), d, r.f64()), np.abs(x.f64()) * OI.keep_scale(0.3) + np.abs(r.f64()), 5)
    ids = rng.integers(-1, n + 1, size=19)
    ti = torch.from_numpy(ids).cuda()
    y = L.embedding(ti, x.v, scale=2.0, pos_table=x.v, pos_period=4, drop=L_drop(d), out_dtype=T[gt])
    kw = dict(scale=2.0, pos_period=4)
    close(y, OI.lookup(ids, x.f64(), pos_table=x.f64(), drop=d, **kw),
          OI.lookup(ids, np.abs(x.f64()), pos_table=np.abs(x.f64()), **kw) * OI.keep_scale(0.3), 5)
    ids = rng.integers(-1, 4, size=n)
    for it in (torch.int32, torch.int64):
        for accumulate in (False, True):
            grad = Mat(3, dim, gt, 1, dim, rng.normal(size=(3, dim)))
            old = grad.f64() if accumulate else np.zeros((3, dim))
            L.embedding_grad(x.v, torch.from_numpy(ids).to(it).cuda(), grad.v, scale=0.5, drop=L_drop(d),
                             accumulate=accumulate)
            want, cnt, mag = OI.lookup_grad(x.f64(), ids, 3, scale=0.5, drop=d)
            close(grad.v, want + old, mag + np.abs(old), (cnt + 4)[:, None])
            grad.check()
    grad = Mat(4, dim, gt, 1, dim)
    L.embedding_grad(x.v, None, grad.v, period=3, drop=L_drop(d))
    want, cnt, mag = OI.lookup_grad(x.f64(), None, 4, period=3, drop=d)
    close(grad.v, want, mag, (cnt + 4)[:, None])
    grad.check()


def test_workspace_of_a_full_batch_serves_its_shorter_last_one():
    """Across the steps of the chunk length, where a shorter batch uses more partial rows."""
    rows, dim = 700, 1600
    ws = L.embedding_grad_workspace(8192, rows, dim)
    ws.fill_(0xFF)
    for n in (8192, 8191, 5000, 4097):
        say(f"workspace of 8192 ids, {n} ids")
        dy = torch.randn(n, dim, device="cuda").bfloat16()
        ids = torch.randint(0, rows, (n,), device="cuda") // 40 * 40      # long runs: every chunk a partial row
        a = L.embedding_grad(dy, ids, torch.empty(rows, dim, device="cuda"), workspace=ws)
        assert torch.equal(a, L.embedding_grad(dy, ids, torch.empty(rows, dim, device="cuda")))


class _Embed(torch.autograd.Function):
    """Embedding with dropout as a torch model's own function: the calls' place in autograd."""

    @staticmethod
    def forward(ctx, ids, table, drop):
        ctx.save_for_backward(ids)
        ctx.shape, ctx.drop = table.shape, drop
        return L.embedding(ids, table, drop=drop)

    @staticmethod
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        return None, L.embedding_grad(dy.contiguous(), ids, dy.new_empty(ctx.shape), drop=ctx.drop), None


class _Drop(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, drop):
        ctx.drop = drop
        return L.dropout(x, drop)

    @staticmethod
    def backward(ctx, dy):
        return L.dropout(dy.contiguous(), ctx.drop), None


def test_inside_autograd_functions():
    """Called directly on what requires grad they are refused; from a Function they
    give autograd the gradients of the oracle."""
    rng = np.random.default_rng(12)
    table = torch.from_numpy(rng.normal(size=(13, 40)).astype(np.float32)).cuda().requires_grad_()
    ids = torch.from_numpy(rng.integers(0, 13, size=30)).cuda()
    c = torch.from_numpy(rng.normal(size=(30, 40)).astype(np.float32)).cuda()
    with pytest.raises(ValueError, match="requires grad"):
        L.embedding(ids, table)
    with pytest.raises(ValueError, match="requires grad"):
        L.dropout(table, None)
    d0, d1 = drop_of(0.2), dict(drop_of(0.3), site=5)
    (_Drop.apply(_Embed.apply(ids, table, L_drop(d0)), L_drop(d1)) * c).sum().backward()
    cs = c.cpu().double().numpy()
    inner = OI.dropout(cs, d1)
    want, cnt, mag = OI.lookup_grad(inner, ids.cpu().numpy(), 13, drop=d0)
    close(table.grad, want, mag, (cnt + 6)[:, None])       # and the outer dropout's factor, rounded twice


@pytest.mark.parametrize("device_control", [False, True])
def test_the_optimizers_dropout_follows_its_steps(device_control):
    """One Dropout object kept over a loop draws each step's own mask, with the step
    count on the host or on the device, and repeats it after a skipped step."""
    opt = ZeroAdam([4096], 1, 0, lr=1e-3, grad_dtype=torch.bfloat16, device_control=device_control)
    d = opt.dropout(0.5, seed=3, site=2)
    x = torch.randn(16, 100, device="cuda")
    grads = torch.ones(1, opt.plan.padded_numel, dtype=torch.bfloat16, device="cuda")
    t = 0
    for skipped in (False, False, True, False):
        assert torch.equal(L.dropout(x, d), L.dropout(x, L.Dropout(0.5, seed=3, site=2, step=t))), t
        grads.fill_(float("inf") if skipped else 1.0)
        opt.step(grads, full=True)
        t += not skipped
    assert opt.t == t == 3


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_rows_that_are_not_there_are_positive_zeros(dt):
    """A gradient's row without an id is +0 in every form, with a scale below zero too;
    a lookup of an id outside the table is scale * (+0) in both forms, and + 0 where
    a position has no row."""
    def plus_zero(x):
        return not x.any() and not torch.signbit(x.float()).any()

    for rows, dim in ((3, 2), (6, 40), (5, 512)):
        table = torch.ones(rows, dim, device="cuda").to(T[dt])
        ids = torch.tensor([0, -1, rows, rows - 1], device="cuda")
        y = L.embedding(ids, table, scale=-2.0)
        assert (y[0] == -2).all() and (y[3] == -2).all()
        assert not y[1:3].any() and torch.signbit(y[1:3].float()).all()
        assert plus_zero(L.embedding(ids, table)[1:3])
        pos = torch.full((2, dim), 0.5, device="cuda").to(T[dt])
        y = L.embedding(ids, table, scale=-2.0, pos_table=pos, pos_period=4)
        assert (y[1] == 0.5).all() and plus_zero(y[2])
    # element by element; one launch; sorted; by period
    for n, rows, dim in ((2, 9, 3), (10, 300, 40), (3000, 900, 40), (3000, 900, 1024)):
        dy = torch.ones(n, dim, device="cuda").to(T[dt])
        for ids, period in ((torch.arange(n, device="cuda") % 3 * 2, 0), (None, 4)):
            for out in (torch.float32, T[dt]):
                grad = torch.full((rows, dim), 3.0, device="cuda", dtype=out)
                L.embedding_grad(dy, ids, grad, scale=-0.5, period=period)
                there = [0, 2, 4] if ids is not None else [0, 1, 2, 3]
                there = there[:n]
                idle = torch.ones(rows, dtype=torch.bool, device="cuda")
                idle[there] = False
                assert plus_zero(grad[idle]) and (grad[there] < 0).all(), (n, rows, dim, period)


def test_lookup_with_a_position_table_without_rows():
    """Every position is outside it and reads zeros, given one by one or by a period,
    through the torch layer and with an address through the C call."""
    table = torch.randn(9, 136, device="cuda").bfloat16()
    ids, at = torch.arange(-1, 10, device="cuda"), torch.arange(11, device="cuda")
    want = L.embedding(ids, table)
    assert torch.equal(L.embedding(ids, table, pos_table=table[:0], pos=at), want)
    assert torch.equal(L.embedding(ids, table, pos_table=table[:0], pos_period=4), want)
    out = torch.empty_like(want)
    a = Z.zero_embed_args_t()
    a.table, a.ld_table, a.rows, a.table_dtype = table.data_ptr(), 136, 9, Z.ZERO_BF16
    a.ids, a.id_bytes, a.n_ids, a.dim, a.scale = ids.data_ptr(), 8, 11, 136, 1.0
    a.pos_table, a.ld_pos, a.pos_rows, a.pos = table.data_ptr(), 136, 0, at.data_ptr()
    a.out, a.ld_out, a.out_dtype = out.data_ptr(), 136, Z.ZERO_BF16
    Z.zero_embed_lookup(a, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, want)


@pytest.mark.parametrize("ot", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [1031, 1600, 4096])
def test_every_element_is_rounded_alike(cols, ot):
    """Each operation in fp32, its result rounded to the output's type: the same bits
    wherever an element stands.  2^21 fp32 values and more, so that hundreds lie where
    one rounding of the exact product to 16 bits and two roundings differ."""
    rows = (1 << 21) // cols + 1
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    r = torch.randn(rows, cols, generator=g, device="cuda").to(T[ot])
    d = drop_of(0.1, rows_at=3)
    keep = torch.from_numpy(OI.keep(rows, cols, **d)).cuda()
    ks = torch.tensor(OI.keep_scale(0.1), dtype=torch.float32, device="cuda")
    zero = torch.zeros((), device="cuda")

    def same(got, want32):
        return torch.equal(got, want32.to(T[ot]))

    kept = torch.where(keep, x * ks, zero)
    assert same(L.dropout(x, L_drop(d), out_dtype=T[ot]), kept)
    assert same(L.dropout(x, L_drop(d), residual=r), kept + r.float())
    ids = torch.randperm(rows, generator=g, device="cuda")
    assert same(L.embedding(ids, x, scale=1.3, out_dtype=T[ot]), x[ids] * 1.3)
    y = L.embedding(ids, x, scale=1.3, pos_table=x, pos_period=rows, drop=L_drop(d), out_dtype=T[ot])
    assert same(y, torch.where(keep, (x[ids] * 1.3 + x) * ks, zero))
    # each id once: many ids; few, in one launch; by period
    for n in (rows, 200):
        grad = torch.empty(rows, cols, dtype=T[ot], device="cuda")
        L.embedding_grad(x[:n], ids[:n], grad, scale=1.3)
        assert same(grad[ids[:n]], x[:n] * 1.3)
        L.embedding_grad(x[:n], None, grad[:n], scale=1.3, period=n)
        assert same(grad[:n], x[:n] * 1.3)
        grad.copy_(r)
        L.embedding_grad(x[:n], ids[:n], grad, scale=1.3, accumulate=True)
        assert same(grad[ids[:n]], x[:n] * 1.3 + r[ids[:n]].float())


# ---------------------------------------------------------------------------
# rows of a multiple of 512 columns, where a wave has one row
# ---------------------------------------------------------------------------

PAIRS = [(a, b) for a in ("f32", "bf16", "f16") for b in ("f32", "bf16", "f16")]


@pytest.mark.parametrize("cols", [512, 4096])
@pytest.mark.parametrize("xt,ot", PAIRS)
def test_dropout_of_whole_wave_rows(xt, ot, cols):
    say(f"dropout 21x{cols} {xt}->{ot}")
    g = np.random.default_rng(cols + len(xt))
    for off, pad, res in ((0, 0, True), (1, 3, True), (5, 0, False)):
        x = Mat(21, cols, xt, off, cols + pad, g.normal(size=(21, cols)))
        r = Mat(21, cols, ot, off, cols + 2 * pad, g.normal(size=(21, cols))) if res else None
        out = Mat(21, cols, ot, off, cols + pad)
        d = drop_of(0.1, rows_at=2**32 - 30, step=2**32 - 1)
        L.dropout(x.v, L_drop(d), residual=r.v if res else None, out=out.v)
        xs, rs = x.f64(), r.f64() if res else None
        close(out.v, OI.dropout(xs, d, rs), np.abs(xs) * OI.keep_scale(0.1) + (np.abs(rs) if res else 0), 5)
        out.check()


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("dim", [512, 4096])
@pytest.mark.parametrize("tt,ot", PAIRS)
def test_lookup_of_whole_wave_rows(tt, ot, dim, p):
    say(f"lookup 37 of 11x{dim} {tt}->{ot} p={p}")
    g = np.random.default_rng(dim + len(ot))
    table = Mat(11, dim, tt, 1, dim + 2, g.normal(size=(11, dim)))
    pos = Mat(6, dim, tt, 3, dim, g.normal(size=(6, dim)))
    ids, at = g.integers(-2, 13, size=37), g.integers(-1, 8, size=37)
    ti, tp = torch.from_numpy(ids).cuda(), torch.from_numpy(at).cuda()
    d = drop_of(p, rows_at=9) if p else None
    for kw, okw in ((dict(), dict()),
                    (dict(pos_table=pos.v, pos_period=7), dict(pos_table=pos.f64(), pos_period=7)),
                    (dict(pos_table=pos.v, pos=tp), dict(pos_table=pos.f64(), pos=at))):
        out = Mat(37, dim, ot, 1, dim + 1)
        L.embedding(ti, table.v, scale=3.0, drop=L_drop(d), out=out.v, **kw)
        want = OI.lookup(ids, table.f64(), scale=3.0, drop=d, **okw)
        mag = dict(okw, **({"pos_table": np.abs(okw["pos_table"])} if okw else {}))
        close(out.v, want, OI.lookup(ids, np.abs(table.f64()), scale=3.0, **mag) * OI.keep_scale(p), 5)
        out.check()


@pytest.mark.parametrize("rows,cols", [(64, 513), (9, 512), (3, 2)])
@pytest.mark.parametrize("xt,ot", PAIRS)
def test_dropout_of_nothing_and_of_everything(rows, cols, xt, ot):
    """p = 0 (and no drop) passes x on, p = 1 leaves the residual, bit for bit: one
    fp32 addition, or none, and one rounding."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(T[xt])
    r = torch.randn(rows, cols, generator=g, device="cuda").to(T[ot])
    for d in (None, L.Dropout(0.0), L.Dropout(2.0 ** -18)):
        assert torch.equal(L.dropout(x, d, out_dtype=T[ot]), x.to(T[ot]))
        assert torch.equal(L.dropout(x, d, residual=r), (x.float() + r.float()).to(T[ot]))
    assert torch.equal(L.dropout(x, L.Dropout(1.0), residual=r), r)
    assert not L.dropout(x, L.Dropout(1.0), out_dtype=T[ot]).any()
