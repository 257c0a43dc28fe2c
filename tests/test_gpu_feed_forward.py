"""The feed-forward sub-layer on the GPU against the float64 oracle: 8-bit checkpoints, RMS
norm, the gated projections, their backward passes, and a run of them around the
sharded step.

Error bounds (u = half a step of a type relative to the value, e = 2^-24; SUB = half the
smallest subnormal of the result's type):
  codes, totals, unpacked values   equal bits
  y           computed in pairs of fp32 (an error of some 2^-44, covered by 1.01), rounded to
              fp32, then to its type: (e + u) |y|
  dh          s = w dy and n = h rstd: 1 rounding each; their products' sum over a row is made of at
              most 16 terms a lane, 6 steps over the lanes, 8 waves: 30 additions on any path, each
              off by at most e times the sum of magnitudes A = mean |s n|; the division, and the
              product n * mean inside one fma: 36 e A |n|; then rstd * and + dres:
              e rstd (3 |s| + 40 A |n|) + e |dh| + u |dh|
  dweight     n: 1, the sum over rows at most `rows` fma: (rows + 3) e sum |dy n| + u |dw|
  products    sums of k terms.  A matrix instruction adds its terms in an order and with roundings
              of its own, each taken as at most a whole step, 2 e: 2 k e sum |x w|, and k more e
              where fp32 products are rounded
  activation  p = 1 / (1 + exp(-z)): the exponent's argument is off by at most 6 e |z| (for GELU the
              polynomial's 4 roundings, the factor log2(e) and the product), exp2, the addition and
              the reciprocal by at most 8 e: relative to p by (6 |z| + 8) e, or it is a subnormal that reads
              0: r = (6 |z| + 8) e p + 2^-126; 1 - p then is off by r + e.
              a = g p u: r |g u| + 3 e |a|;  act' = p + g p (1 - p) slope:
              D = r + |g| slope (r + 12 e p) + 2 e |act'|
Tests with whole numbers have sums below 2^24, which are exact in any order: there the
results are equal to the last bit.
"""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_plan_amd as Z
from gpu_harness import say
from oracle import feed_forward as OF
from zero_sharded_mixed_plan_amd import feed_forward as F
from zero_sharded_mixed_plan_amd.optim import ZeroAdam

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24
SUB = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def f64(t):
    return t.detach().cpu().double().numpy()


def rounded(v, dt):
    """float64 values rounded once to a type (through fp32 where fp32 holds them)."""
    with np.errstate(over="ignore"):
        return f64(torch.from_numpy(np.asarray(v, dtype=np.float64)).float().to(T[dt]))


def close(got, want, err, what=""):
    """|got - want| <= 1.01 (err + u |want|) + SUB."""
    u = torch.finfo(got.dtype).eps / 2
    tol = 1.01 * (err + u * np.abs(want)) + SUB[got.dtype]
    g = f64(got).reshape(want.shape)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} wrong, first {np.argwhere(bad)[:3].tolist()}: " \
                          f"{g[bad][:3]} for {want[bad][:3]}, tolerance {tol[bad][:3]}"


def same(got, want, what=""):
    g = f64(got).reshape(want.shape)
    bad = ~((g == want) | (np.isnan(g) & np.isnan(want)))
    assert not bad.any(), f"{what}: {bad.sum()} differ, first {np.argwhere(bad)[:3].tolist()}: {g[bad][:3]} for {want[bad][:3]}"


class Mat:
    """[rows, cols] of a type inside a guarded flat buffer: element offset `off`, rows
    `ld` apart; the elements around and between must not change.  fill: what they hold (NaN
    shows a read that has an effect)."""

    def __init__(self, rows, cols, dt, off=0, ld=None, data=None, fill=float("nan")):
        dtype = T[dt] if isinstance(dt, str) else dt
        self.ld = ld or cols
        n = off + max(rows, 1) * self.ld + 16
        self.flat = torch.full((n,), 255, dtype=torch.uint8, device="cuda").view(dtype) if dtype.itemsize == 1 else \
            torch.full((n,), fill, dtype=dtype, device="cuda")
        self.v = self.flat[off:off + rows * self.ld].view(rows, self.ld)[:, :cols]
        if data is not None:
            self.v.copy_(torch.as_tensor(np.asarray(data)))
        inside = torch.zeros(n, dtype=torch.bool, device="cuda")
        inside[off:off + rows * self.ld].view(rows, self.ld)[:, :cols] = True
        self.outside = ~inside
        self.bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[dtype.itemsize]
        self.before = self.flat.view(self.bits)[self.outside].clone()

    def check(self):
        assert torch.equal(self.flat.view(self.bits)[self.outside], self.before), "written outside the matrix"


class Held:
    """Guarded codes and scales."""

    def __init__(self, rows, cols, off=0, pad=0):
        self.c = Mat(rows, cols, torch.float8_e4m3fn, off, cols + pad)
        self.s = Mat(rows, OF.blocks(cols), torch.float8_e8m0fnu, off, OF.blocks(cols) + pad)
        self.p = F.Packed8(self.c.v, self.s.v)

    def check(self):
        self.c.check()
        self.s.check()


def codes_of(p):
    """(values of the codes, exponents) of a Packed8."""
    q = OF.e4m3_value(p.codes.contiguous().view(torch.uint8).cpu().numpy())
    return q, p.scales.contiguous().view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def same_codes(p, want, what=""):
    q, e = codes_of(p)
    wq, we = want
    assert np.array_equal(e, we.reshape(e.shape)), f"{what}: scales differ at {np.argwhere(e != we.reshape(e.shape))[:3].tolist()}"
    wq = wq.reshape(q.shape)
    bad = ~((q == wq) | (np.isnan(q) & np.isnan(wq)))
    assert not bad.any(), f"{what}: {bad.sum()} codes differ, {np.argwhere(bad)[:3].tolist()}: {q[bad][:3]} for {wq[bad][:3]}"


def stream(g, rows, cols):
    """Rows of different size, a few large columns, zeros."""
    v = g.normal(size=(rows, cols)) * np.exp2(g.integers(-3, 4, size=(rows, 1)))
    v[:, ::61] *= 16
    v[g.random(size=v.shape) < 0.02] = 0
    return v


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------

HOLD = [  # rows, cols, type, offset, padding
    (1, 1, "f32", 0, 0), (3, 7, "bf16", 1, 0), (2, 8, "f16", 3, 5), (5, 31, "f16", 0, 1), (5, 32, "bf16", 1, 0),
    (4, 33, "f32", 1, 3), (17, 777, "f16", 3, 2), (33, 1600, "bf16", 0, 0), (9, 2049, "f32", 1, 7),
    (64, 512, "bf16", 0, 64), (1, 100001, "bf16", 5, 0), (40000, 9, "f32", 1, 1), (300, 64, "f32", 0, 0),
]


@pytest.mark.parametrize("rows,cols,dt,off,pad", HOLD)
def test_pack_and_unpack(rows, cols, dt, off, pad):
    say(f"pack {rows}x{cols} {dt} off {off} pad {pad}")
    g = np.random.default_rng(rows * 7 + cols)
    x = Mat(rows, cols, dt, off, cols + pad, stream(g, rows, cols))
    h = Held(rows, cols, off, pad)
    assert F.pack8(x.v, out=h.p) is h.p
    want = OF.hold(f64(x.v))
    same_codes(h.p, want)
    for m in (x, h):
        m.check()
    value = OF.held_value(*want)
    for out in ("f32", "bf16", "f16"):
        y = Mat(rows, cols, out, off, cols + 2 * pad)
        F.unpack8(h.p, out=y.v)
        y.check()
        same(y.v, rounded(value, out), out)
        if out != "f16":
            assert np.array_equal(rounded(value, out), value)
    new = F.pack8(x.v)
    same_codes(new, want)
    same(F.unpack8(new, torch.float32), value)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_pack_special_values(dt):
    """Borders of the scale, ties, subnormals, the largest numbers, infinities and NaN."""
    fi = torch.finfo(T[dt])
    v = np.zeros((12, 64))
    g = np.random.default_rng(5)
    v[1, :3] = [448.0, -448.0, 1.0]
    v[2, :3] = [450.0, -3.0, 17.0]             # just past 448: the scale doubles (450 is a bf16)
    v[3, :8] = [17, 19, 21, 23, 25, 27, 29, 448]  # ties of e4m3
    v[4, :4] = [fi.max, -fi.max, fi.max / 2, 1]
    v[5, :4] = [fi.tiny, fi.tiny / 2, -fi.smallest_normal, fi.tiny * 1.5]
    v[6] = fi.smallest_normal * g.normal(size=64) * 2.0 ** -3
    v[7, :4] = [np.inf, 3.0, -np.inf, np.nan]
    v[8, :] = np.inf
    v[9, :40] = np.nan
    v[10] = g.normal(size=64)
    v[10, 5] = -0.0
    v[11] = np.exp2(g.uniform(-12, 12, size=64))
    x = torch.from_numpy(v).float().to(T[dt]).cuda()
    p = F.pack8(x)
    want = OF.hold(f64(x))
    same_codes(p, want)
    y = F.unpack8(p, torch.float32)
    # the largest fp32 and bf16 numbers round up to 2^128, which in fp32 is an infinity
    same(y, rounded(OF.held_value(*want), "f32"))
    assert torch.isfinite(y[10]).all() and not torch.signbit(y[0]).any() and bool(torch.signbit(y[10, 5]))
    assert int(p.scales.view(torch.uint8).max()) < 255


def test_pack_bytes_and_batches():
    """uint8 tensors in place of torch's 8-bit types; batches of sequences are rows."""
    x = torch.randn(3, 5, 70, device="cuda").bfloat16()
    p = F.pack8(x)
    b = F.Packed8(torch.empty(3, 5, 70, dtype=torch.uint8, device="cuda"), torch.empty(3, 5, 3, dtype=torch.uint8, device="cuda"))
    F.pack8(x, out=b)
    assert torch.equal(b.codes, p.codes.view(torch.uint8)) and torch.equal(b.scales, p.scales.view(torch.uint8))
    y = F.unpack8(b)
    assert y.shape == x.shape and torch.equal(y, F.unpack8(F.pack8(x.view(15, 70))).view(3, 5, 70))
    # held once more, a checkpoint is the same
    q = F.pack8(y)
    assert torch.equal(F.unpack8(q), y)
    for shape in ((0, 5), (4, 0)):
        assert F.unpack8(F.pack8(torch.empty(shape, device="cuda"))).shape == shape


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

NORM = [  # rows, cols, x, residual (or None), weight (or None), y, packed, offset, padding
    (1, 1, "f32", None, "f32", "f32", True, 0, 0), (3, 7, "bf16", "bf16", "bf16", "bf16", True, 1, 0),
    (5, 31, "f16", "f32", "f32", "f16", True, 3, 5), (130, 64, "bf16", "bf16", None, "f32", False, 0, 0),
    (9, 511, "bf16", None, "bf16", "bf16", True, 1, 1), (6, 512, "f32", "f32", "bf16", "bf16", True, 0, 0),
    (7, 513, "f16", "f16", "f16", "f32", True, 0, 0), (33, 777, "f16", None, "f16", "f32", False, 3, 2),
    (4, 1024, "bf16", "f32", "f32", "bf16", True, 0, 8), (5, 1025, "f32", "f32", "f32", "f32", False, 1, 0),
    (21, 1600, "bf16", "bf16", "bf16", "bf16", True, 0, 0), (3, 2049, "f16", "f16", None, "f16", True, 1, 1),
    (1, 4096, "bf16", "bf16", "bf16", "bf16", False, 0, 0), (300, 4096, "bf16", "bf16", "bf16", "bf16", True, 0, 0),
    (5, 4097, "bf16", "f32", "f32", "bf16", True, 1, 0), (3, 8191, "f32", "f32", "bf16", "f16", True, 0, 3),
    (4, 8192, "f16", "f16", "f32", "f32", True, 0, 0), (2000, 40, "bf16", "bf16", "f32", "bf16", True, 0, 0),
]


@pytest.mark.parametrize("rows,cols,xt,rt,wt,yt,packed,off,pad", NORM)
def test_rms_norm(rows, cols, xt, rt, wt, yt, packed, off, pad):
    say(f"norm {rows}x{cols} {xt}+{rt} w {wt} -> {yt}")
    g = np.random.default_rng(rows + cols)
    x = Mat(rows, cols, xt, off, cols + pad, stream(g, rows, cols))
    r = Mat(rows, cols, rt, off + 1, cols + pad, g.normal(size=(rows, cols))) if rt else None
    w = Mat(1, cols, wt, off, data=1 + 0.2 * g.normal(size=(1, cols))) if wt else None
    total = Mat(rows, cols, rt, off, cols + 2 * pad) if rt else None
    y, h = Mat(rows, cols, yt, off, cols + pad), Held(rows, cols, off, pad)
    rstd = Mat(1, rows, "f32", 1)
    n = F.rms_norm(x.v, w.v[0] if wt else None, eps=1e-5, residual=r.v if rt else None, total=total.v if rt else None,
                   out=y.v, packed=h.p if packed else False, rstd=rstd.v[0])
    assert n.y is y.v and n.rstd.data_ptr() == rstd.v.data_ptr()
    hs = f64(x.v)
    if rt:  # one fp32 addition, one rounding
        hs = f64((x.v.float() + r.v.float()).cpu().to(T[rt]))
        same(total.v, hs, "total")
    want, scale = OF.rms_norm(hs, f64(w.v)[0] if wt else None, 1e-5)
    close(rstd.v, scale[None], np.zeros((1, rows)), "rstd")
    close(y.v, want, E * np.abs(want), "y")
    if packed:
        same_codes(n.packed, OF.hold(want.astype(np.float32).astype(np.float64)), "codes")
    for m in [x, y, h, rstd] + ([r, total] if rt else []):
        m.check()
    # only the codes, and nothing but y
    only = F.rms_norm(x.v, w.v[0] if wt else None, eps=1e-5, residual=r.v if rt else None, out=False, packed=True, rstd=False)
    assert only.y is None and only.rstd is None
    if packed:
        assert torch.equal(only.packed.codes.view(torch.uint8), n.packed.codes.contiguous().view(torch.uint8))
    alone = F.rms_norm(x.v, w.v[0] if wt else None, eps=1e-5, residual=r.v if rt else None, out_dtype=T[yt])
    assert alone.packed is None and torch.equal(alone.y, y.v)


def test_rms_norm_in_place_and_batches():
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(6, 50, 300, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(300, generator=g, device="cuda")
    ref = F.rms_norm(x, w, eps=1e-6, residual=r, packed=True)
    assert ref.y.shape == x.shape and ref.rstd.shape == (6, 50) and ref.total.shape == x.shape
    for which in (0, 1):
        a, b = x.clone(), r.clone()
        into = (a, b)[which]
        n = F.rms_norm(a, w, eps=1e-6, residual=b, total=into, packed=True)
        assert n.total is into and torch.equal(into, ref.total) and torch.equal(n.y, ref.y)
        assert torch.equal(n.packed.codes.view(torch.uint8), ref.packed.codes.view(torch.uint8))
    # a row's results do not hang on its place in the batch, nor on its neighbours
    one = F.rms_norm(x[2, 7:8], w, eps=1e-6, residual=r[2, 7:8])
    assert torch.equal(one.y, ref.y[2, 7:8]) and torch.equal(one.rstd, ref.rstd[2, 7:8])


@pytest.mark.parametrize("cols", [40, 700, 1500, 4096, 8192])
def test_rms_norm_far_magnitudes(cols):
    """Rows whose rstd, or whose products with the weight, lie near the ends of fp32 or beyond: y is the value in
    64 bits rounded once, whatever the factors' sizes; what does not fit is an infinity.  Of y below 2^-100 the
    second part of the pair is a multiple of 2^-149, after two roundings of at most 2^-150 each, and so is
    the result below 2^-126: 3 * 2^-150 beside E |y|."""
    least = 3 * 2.0 ** -150
    g = torch.Generator(device="cuda").manual_seed(cols)
    size = torch.tensor([1e-44, 1e-38, 1e-33, 1e-20, 1.0, 1e20, 1e33, 1e36], device="cuda")
    x = torch.randn(len(size), cols, generator=g, device="cuda") * size[:, None]
    x[:, 1] = 0
    w = torch.randn(cols, generator=g, device="cuda") + 3
    for k, factor in ((0, 1.0), (1, 1e-6), (2, 1e30), (3, 1e-38), (4, 2e38)):
        v = w * factor
        if k == 0:
            v[3] = float("inf")
            v[5] = float("nan")
        with np.errstate(all="ignore"):
            want, scale = OF.rms_norm(f64(x), f64(v), 0.0)
            once = torch.from_numpy(want).float().double().numpy()
        n = F.rms_norm(x, v, eps=0.0, packed=True)
        got = f64(n.y)
        assert np.array_equal(np.isnan(got), np.isnan(once))
        assert np.array_equal(np.isinf(got) & ~np.isnan(once), np.isinf(once) & ~np.isnan(once)), factor
        fits = np.isfinite(once)
        assert (np.abs(got[fits] - want[fits]) <= 1.01 * E * np.abs(want[fits]) + least).all(), factor
        same_codes(n.packed, OF.hold(got), "codes")
        assert np.array_equal(f64(n.rstd), torch.from_numpy(scale).float().double().numpy())
    alone = F.rms_norm(x, None, eps=0.0).y
    want, _ = OF.rms_norm(f64(x), None, 0.0)
    assert (np.abs(f64(alone) - want) <= 1.01 * E * np.abs(want) + least).all()


def test_rms_norm_special_rows():
    """A row of zeros, one with an infinity, one with NaN, very large and very small
    ones: each on its own."""
    x = torch.randn(6, 700, device="cuda")
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 6] = float("nan")
    x[3] *= 1e30
    x[4] *= 1e-30
    n = F.rms_norm(x, None, eps=1e-12, packed=True)
    assert (n.y[0] == 0).all() and (n.packed.codes[0].float() == 0).all()
    assert n.rstd[1] == 0 and torch.isnan(n.y[1, 5]) and (n.y[1, 6:] == 0).all()
    assert torch.isnan(n.y[2]).all()
    want, scale = OF.rms_norm(f64(x[3:]), None, 1e-12)
    close(n.y[3:], want, E * np.abs(want))
    close(n.rstd[3:], scale, np.zeros(3))
    same_codes(F.Packed8(n.packed.codes[3:], n.packed.scales[3:]), OF.hold(want.astype(np.float32).astype(np.float64)))
    assert torch.isnan(F.rms_norm(torch.zeros(1, 9, device="cuda"), None, eps=0.0).y).all()
    e = F.rms_norm(torch.empty(0, 64, device="cuda"), None, eps=1e-5, packed=True)
    assert e.y.shape == (0, 64) and e.packed.scales.shape == (0, 2)


NORM_GRAD = [  # rows, cols, dy, h, held, weight, residual's gradient, dweight, offset, padding
    (1, 1, "f32", "f32", False, "f32", True, "f32", 0, 0), (3, 7, "bf16", "bf16", True, "bf16", True, "bf16", 1, 0),
    (5, 31, "f16", "f32", False, "f32", True, "f32", 3, 5), (300, 64, "bf16", "bf16", False, None, False, "f32", 0, 0),
    (9, 512, "bf16", "f32", True, "f32", True, "bf16", 0, 0), (65, 513, "f16", "f16", True, "f16", False, "f16", 1, 1),
    (130, 777, "f16", "f16", False, "f16", False, "f32", 3, 2), (7, 1024, "f32", "f32", True, "bf16", True, "f32", 0, 0),
    (40, 1025, "f32", "f32", False, "f32", False, None, 1, 0), (50, 1600, "bf16", "bf16", True, "bf16", True, "bf16", 0, 0),
    (1500, 2048, "bf16", "bf16", True, "bf16", True, "f32", 0, 0), (20, 2049, "f16", "f16", False, None, True, None, 1, 1),
    (40, 4096, "bf16", "bf16", True, "bf16", True, "bf16", 0, 0), (11, 4097, "bf16", "f32", False, "f32", True, "f32", 1, 0),
    (9, 8191, "f32", "f32", True, "bf16", False, "f16", 0, 3), (600, 8192, "f16", "f16", True, "f32", True, "f32", 0, 0),
    (5000, 40, "bf16", "bf16", False, "f32", True, "bf16", 0, 0),
]


@pytest.mark.parametrize("rows,cols,yt,ht,packed,wt,res,dwt,off,pad", NORM_GRAD)
def test_rms_norm_grad(rows, cols, yt, ht, packed, wt, res, dwt, off, pad):
    say(f"norm grad {rows}x{cols} {yt} {ht} held {packed} -> {dwt}")
    g = np.random.default_rng(rows + cols)
    dy = Mat(rows, cols, yt, off, cols + pad, g.normal(size=(rows, cols)))
    h = Mat(rows, cols, ht, off, cols + pad, stream(g, rows, cols))
    if packed:
        held = Held(rows, cols, off, pad)
        F.pack8(h.v, out=held.p)
        hs = OF.held_value(*codes_of(held.p))
    else:
        hs = f64(h.v)
    w = Mat(1, cols, wt, off, data=1 + 0.2 * g.normal(size=(1, cols))) if wt else None
    d = Mat(rows, cols, ht, off, cols + pad, g.normal(size=(rows, cols))) if res else None
    rstd = Mat(1, rows, "f32", 1, data=1 / np.sqrt((f64(h.v) ** 2).mean(axis=1) + 1e-5)[None])
    dh = Mat(rows, cols, ht, off, cols + 2 * pad)
    old = g.normal(size=(1, cols))
    dw = Mat(1, cols, dwt, off + 1, data=old) if dwt else None
    out = F.rms_norm_grad(dy.v, held.p if packed else h.v, rstd.v[0], w.v[0] if wt else None,
                          residual_grad=d.v if res else None, out=dh.v, weight_grad=dw.v[0] if dwt else None)
    assert out is dh.v
    dys, rs, ws = f64(dy.v), f64(rstd.v)[0], f64(w.v)[0] if wt else None
    want, want_dw = OF.rms_norm_grad(dys, hs, rs, ws, f64(d.v) if res else None)
    n, s = hs * rs[:, None], dys * (1 if ws is None else ws)
    A = np.abs(s * n).mean(axis=1, keepdims=True)
    err = E * rs[:, None] * (3 * np.abs(s) + 40 * A * np.abs(n)) + E * np.abs(want)
    close(dh.v, want, err, "dh")
    for m in [dy, h, dh] + ([d] if res else []):
        m.check()
    if dwt:
        mag = np.abs(dys * n).sum(axis=0)
        close(dw.v, want_dw[None], ((rows + 3) * E * mag)[None], "dweight")
        dw.check()
        # added to what is there
        dw.v.copy_(torch.from_numpy(old))
        before = f64(dw.v)
        again = F.rms_norm_grad(dy.v, held.p if packed else h.v, rstd.v[0], w.v[0] if wt else None,
                                residual_grad=d.v if res else None, out_dtype=T[ht], weight_grad=dw.v[0], accumulate=True)
        assert torch.equal(again, dh.v)
        close(dw.v, before + want_dw[None], ((rows + 3) * E * mag)[None] + E * np.abs(before), "accumulated")
        dw.check()


def test_rms_norm_grad_in_place_workspace_and_empty():
    g = torch.Generator(device="cuda").manual_seed(4)
    dy, h, d = (torch.randn(4, 70, 520, generator=g, device="cuda").bfloat16() for _ in range(3))
    w, dw = torch.randn(520, generator=g, device="cuda"), torch.zeros(520, device="cuda")
    rstd = F.rms_norm(h, w, eps=1e-5).rstd
    ref = F.rms_norm_grad(dy, h, rstd, w, residual_grad=d, weight_grad=dw)
    ws = F.rms_norm_grad_workspace(1000, 1000)
    for which in range(3):
        a = [dy.clone(), h.clone(), d.clone()]
        dw2 = torch.zeros_like(dw)
        F.rms_norm_grad(a[0], a[1], rstd, w, residual_grad=a[2], weight_grad=dw2, out=a[which], workspace=ws)
        assert torch.equal(a[which], ref) and torch.equal(dw2, dw)
    e = torch.empty(0, 520, device="cuda").bfloat16()
    dw.fill_(3)
    F.rms_norm_grad(e, e, torch.empty(0, device="cuda"), w, weight_grad=dw, accumulate=True)
    assert (dw == 3).all()
    F.rms_norm_grad(e, e, torch.empty(0, device="cuda"), w, weight_grad=dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("cols", [300, 1000, 2000, 4000, 7001])
@pytest.mark.parametrize("at,st", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
def test_norm_forms(at, st, cols):
    """Every pair of types at every width of a row's share of a workgroup, with and without 8 bits, against
    64 bits on the GPU; an odd number of rows."""
    say(f"norm forms {at} {st} {cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    rows = 69
    r = lambda *s, k=1.0, dt=at: (torch.randn(*s, generator=g, device="cuda") * k).to(T[dt])  # noqa: E731
    x, res, w, dy, dres = r(rows, cols), r(rows, cols, k=2.0, dt=st), r(cols, dt="f32"), r(rows, cols), r(rows, cols, dt=st)
    total = (x.float() + res.float()).to(T[st])
    h = total.double()
    rstd = 1 / (h.square().mean(1, keepdim=True) + 1e-5).sqrt()
    y = h * rstd * w.double()
    plain = F.rms_norm(x, w, eps=1e-5, residual=res, out_dtype=T[at])
    both = F.rms_norm(x, w, eps=1e-5, residual=res, out_dtype=T[at], packed=True)
    assert torch.equal(plain.total, total) and torch.equal(both.total, total) and torch.equal(plain.y, both.y)
    close(plain.y, f64(y), E * np.abs(f64(y)), "y")
    close(plain.rstd, f64(rstd)[:, 0], np.zeros(rows), "rstd")
    want = F.pack8(F.rms_norm(x, w, eps=1e-5, residual=res, out_dtype=torch.float32).y)
    assert torch.equal(both.packed.codes.view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(both.packed.scales.view(torch.uint8), want.scales.view(torch.uint8))
    kept = F.pack8(total)
    for source, hs in ((total, h), (kept, F.unpack8(kept, torch.float32).double())):
        n = hs * plain.rstd.double()[:, None]
        s = dy.double() * w.double()
        dh = plain.rstd.double()[:, None] * (s - n * (s * n).mean(1, keepdim=True)) + dres.double()
        size = (s * n).abs().mean(1, keepdim=True) * n.abs()
        err = E * plain.rstd.double()[:, None] * (3 * s.abs() + 40 * size) + E * dh.abs()
        dw = torch.empty(cols, device="cuda")
        got = F.rms_norm_grad(dy, source, plain.rstd, w, residual_grad=dres, out_dtype=T[st] if source is kept else None,
                              weight_grad=dw)
        close(got, f64(dh), f64(err), "dh")
        close(dw, f64((dy.double() * n).sum(0)), (rows + 3) * E * f64((dy.double() * n).abs().sum(0)), "dw")


def test_rms_norm_grad_against_differences():
    """The kernels' forward pass in fp32, differenced along a direction, against the
    kernels' gradient: y is off by at most 2^-24 |y|, which a step of 2^-6 turns into 2^-18 sum |y c|;
    the differences' own error is of the step's third order, below 1e-4 of the result here."""
    g = torch.Generator(device="cuda").manual_seed(6)
    h, c, v = (torch.randn(5, 300, generator=g, device="cuda") for _ in range(3))
    w = torch.randn(300, generator=g, device="cuda")
    y = F.rms_norm(h, w, eps=1e-5)
    dh = F.rms_norm_grad(c, h, y.rstd, w)
    s = 2.0 ** -6
    up, dn = (F.rms_norm(h + k * s * v, w, eps=1e-5).y.double() for k in (1, -1))
    got = float((dh.double() * v.double()).sum())
    num = float(((up - dn) * c.double()).sum()) / (2 * s)
    # the third order: bound it by a second, twice larger step (its error is four times as large)
    up2, dn2 = (F.rms_norm(h + 2 * k * s * v, w, eps=1e-5).y.double() for k in (1, -1))
    num2 = float(((up2 - dn2) * c.double()).sum()) / (4 * s)
    noise = 2.0 ** -18 * float((y.y.double() * c.double()).abs().sum()) + 2.0 ** -18 * float((dh * v).abs().sum())
    assert abs(got - num) <= abs(num2 - num) + noise


# ---------------------------------------------------------------------------
# the gated projections
# ---------------------------------------------------------------------------

GATED = [  # tokens, dim, hidden, type, offset, padding
    (1, 1, 1, "f32", 0, 0), (1, 8, 16, "bf16", 0, 0), (2, 7, 5, "f16", 1, 0), (3, 33, 31, "f32", 3, 2),
    (1, 64, 256, "bf16", 0, 0), (4, 100, 36, "bf16", 0, 4), (5, 128, 40, "f16", 0, 8), (16, 256, 64, "bf16", 0, 0),
    (17, 72, 200, "f16", 0, 0), (33, 136, 264, "bf16", 8, 8), (64, 64, 128, "f32", 0, 0), (65, 97, 129, "bf16", 1, 1),
    (100, 1024, 24, "f16", 0, 0), (130, 200, 392, "bf16", 0, 0), (256, 64, 128, "bf16", 0, 0), (257, 72, 136, "f16", 0, 0),
    (300, 520, 648, "bf16", 0, 0), (513, 64, 8, "f16", 0, 0), (70, 2048, 1000, "bf16", 0, 0), (1, 4096, 1376, "bf16", 0, 0),
    (9, 1600, 700, "f16", 0, 0), (31, 777, 130, "bf16", 0, 0),
]


def whole(g, shape, most=3):
    return g.integers(-most, most + 1, size=shape).astype(np.float64)


def gated_case(t, d, f, dt, off, pad, g):
    """Whole numbers with |sums| < 2^24: x and weights of -3 .. 3."""
    x = Mat(t, d, dt, off, d + pad, whole(g, (t, d)))
    wg, wu = (Mat(f, d, dt, off, d + pad, whole(g, (f, d))) for _ in range(2))
    return x, wg, wu


def act_errors(kind, g):
    v, d, p, z, dz = OF.act(kind, g)
    r = (6 * np.abs(z) + 8) * E * p + 2.0 ** -126
    D = r + np.abs(g) * dz * (r + 12 * E * p) + 2 * E * np.abs(d)
    return v, d, r * np.abs(g), D


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f,dt,off,pad", GATED)
def test_gated_whole_numbers(t, d, f, dt, off, pad, kind):
    """Sums are exact, so gate and up come back to the last bit."""
    say(f"gated {t}x{d}x{f} {dt} {kind} off {off} pad {pad}")
    g = np.random.default_rng(t * 31 + d + f)
    x, wg, wu = gated_case(t, d, f, dt, off, pad, g)
    wg.v.mul_(2.0 ** -4)  # gates within the activation's range
    a, gate, up = (Mat(t, f, dt, off, f + pad) for _ in range(3))
    F.gated(x.v, wg.v, wu.v, act=kind, out=a.v, keep=(gate.v, up.v))
    xs, gs, us = f64(x.v), f64(wg.v), f64(wu.v)
    want, wgate, wup = OF.gated(xs, gs, us, kind)
    same(gate.v, rounded(wgate, dt), "gate")
    same(up.v, rounded(wup, dt), "up")
    rg = act_errors(kind, wgate)[2]
    close(a.v, want, rg * np.abs(wup) + 3 * E * np.abs(want), "a")
    hg, hu = Held(t, f, off, pad), Held(t, f, off, pad)
    b = F.gated(x.v, wg.v, wu.v, act=kind, keep=(hg.p, hu.p))
    assert torch.equal(b.a, a.v)
    same_codes(hg.p, OF.hold(wgate), "held gate")
    same_codes(hu.p, OF.hold(wup), "held up")
    assert torch.equal(F.gated(x.v, wg.v, wu.v, act=kind).a, a.v)
    for m in (x, wg, wu, a, gate, up, hg, hu):
        m.check()


@pytest.mark.parametrize("t,d,f,dt", [(3, 1600, 700, "bf16"), (70, 640, 136, "f16"), (40, 333, 77, "f32"), (300, 512, 264, "bf16")])
def test_gated_random(t, d, f, dt):
    g = np.random.default_rng(t + d)
    x = torch.from_numpy(g.normal(size=(t, d))).to(T[dt]).cuda()
    wg, wu = (torch.from_numpy(g.normal(size=(f, d)) / np.sqrt(d)).to(T[dt]).cuda() for _ in range(2))
    for kind in ("silu", "gelu"):
        r = F.gated(x, wg, wu, act=kind, keep="tensors")
        xs, gs, us = f64(x), f64(wg), f64(wu)
        want, wgate, wup = OF.gated(xs, gs, us, kind)
        k = 3 * d * E
        eg, eu = k * (np.abs(xs) @ np.abs(gs).T), k * (np.abs(xs) @ np.abs(us).T)
        close(r.gate, wgate, eg, "gate")
        close(r.up, wup, eu, "up")
        v, _, rg, _ = act_errors(kind, wgate)
        # act is Lipschitz: |act'| <= 1.13
        err = (rg + 1.13 * eg) * (np.abs(wup) + eu) + np.abs(v) * eu + 3 * E * np.abs(want)
        close(r.a, want, err, "a")


def test_gated_packed_random_stands_for_the_sums():
    """Codes of sums that are not exact: each within half a step of e4m3 (2^-4, or 2^-10 of the
    scale) of the exact sum, the scale that of a maximum within the sums' bound."""
    g = np.random.default_rng(8)
    x = torch.from_numpy(g.normal(size=(70, 640))).bfloat16().cuda()
    wg, wu = (torch.from_numpy(g.normal(size=(100, 640)) / 25).bfloat16().cuda() for _ in range(2))
    r = F.gated(x, wg, wu, keep="packed")
    for p, w in ((r.gate, wg), (r.up, wu)):
        s = f64(x) @ f64(w).T
        err = 3 * 640 * E * (np.abs(f64(x)) @ np.abs(f64(w)).T)
        q, e = codes_of(p)
        scale = np.exp2(e.astype(float)).repeat(32, axis=1)[:, :100]
        assert (np.abs(q * scale - s) <= 1.01 * (err + np.maximum(np.abs(s) * 2.0 ** -4, scale * 2.0 ** -10))).all()
        assert np.abs(q).max() <= 448


def test_gated_batches_and_special_values():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 3, 96, generator=g, device="cuda").bfloat16()
    wg, wu = (torch.randn(64, 96, generator=g, device="cuda").bfloat16() * 0.1 for _ in range(2))
    r = F.gated(x, wg, wu, keep="packed")
    assert r.a.shape == (2, 3, 64) and r.gate.codes.shape == (2, 3, 64) and r.up.scales.shape == (2, 3, 2)
    assert torch.equal(r.a.view(6, 64), F.gated(x.view(6, 96), wg, wu).a)
    for keep in (None, "tensors", "packed"):
        e = F.gated(x[:0], wg, wu, keep=keep)
        assert e.a.shape == (0, 3, 64)
    # one token's NaN stays in its row, and a NaN weight row in its column
    y = x.clone()
    y[0, 1, 3] = float("nan")
    n = F.gated(y, wg, wu, keep="packed")
    bad = torch.isnan(n.a)
    assert bad[0, 1].all() and int(bad.sum()) == 64 and torch.isnan(n.gate.codes.float()).sum() == 64
    v = wg.clone()
    v[7, 0] = float("inf")
    n = F.gated(x, v, wu, keep="packed")
    ok = [c for c in range(64) if c != 7]
    assert torch.equal(n.a[..., ok], r.a[..., ok]) and torch.isnan(n.gate.codes[..., 7].float()).all()
    # the block's other codes are those of its finite values
    same = F.gated(x, torch.cat([wg[:7], torch.zeros_like(wg[:1]), wg[8:]]), wu, keep="packed")
    assert torch.equal(n.gate.scales.view(torch.uint8), same.gate.scales.view(torch.uint8))
    assert torch.equal(n.gate.codes[..., ok].view(torch.uint8), same.gate.codes[..., ok].view(torch.uint8))


GRAD = [  # tokens, hidden, type, held, offset, padding
    (1, 1, "f32", False, 0, 0), (3, 7, "bf16", True, 1, 0), (5, 31, "f16", False, 3, 5), (4, 64, "bf16", True, 0, 0),
    (17, 777, "f16", True, 3, 2), (33, 1376, "bf16", False, 0, 0), (9, 2049, "f32", True, 1, 7), (50, 2001, "f32", False, 0, 0),
    (3000, 40, "bf16", True, 0, 8),
]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,f,dt,packed,off,pad", GRAD)
def test_gated_grad(t, f, dt, packed, off, pad, kind):
    say(f"gated grad {t}x{f} {dt} {kind} held {packed}")
    g = np.random.default_rng(t + f)
    da = Mat(t, f, dt, off, f + pad, g.normal(size=(t, f)))
    gate, up = (Mat(t, f, dt, off, f + pad, 3 * g.normal(size=(t, f))) for _ in range(2))
    if packed:
        hg, hu = Held(t, f, off, pad), Held(t, f, off + 1, pad)
        F.pack8(gate.v, out=hg.p)
        F.pack8(up.v, out=hu.p)
        gs, us = OF.held_value(*codes_of(hg.p)), OF.held_value(*codes_of(hu.p))
        kept = hg.p, hu.p
    else:
        gs, us = f64(gate.v), f64(up.v)
        kept = gate.v, up.v
    dg, du, a = (Mat(t, f, dt, off, f + 2 * pad) for _ in range(3))
    r = F.gated_grad(da.v, *kept, act=kind, out_gate=dg.v, out_up=du.v, again=a.v)
    assert r.gate is dg.v and r.up is du.v and r.a is a.v
    ds = f64(da.v)
    wdg, wdu, wa = OF.gated_grad(ds, gs, us, kind)
    v, d, rg, D = act_errors(kind, gs)
    close(dg.v, wdg, np.abs(ds * us) * (D + 2 * E * np.abs(d)), "dg")
    close(du.v, wdu, rg * np.abs(ds) + 3 * E * np.abs(wdu), "du")
    close(a.v, wa, rg * np.abs(us) + 3 * E * np.abs(wa), "a")
    for m in (da, gate, up, dg, du, a):
        m.check()
    lean = F.gated_grad(da.v, *kept, act=kind)
    assert lean.a is None and torch.equal(lean.gate, dg.v) and torch.equal(lean.up, du.v)
    # on da itself, and on what was kept
    b, c = da.v.clone(), da.v.clone()
    F.gated_grad(b, *kept, act=kind, out_gate=b)
    assert torch.equal(b, dg.v)
    if not packed:
        x, y = gate.v.clone(), up.v.clone()
        F.gated_grad(c, x, y, act=kind, out_gate=x, out_up=y, again=c)
        assert torch.equal(x, dg.v) and torch.equal(y, du.v) and torch.equal(c, a.v)


def test_gated_grad_far_gates():
    """Far out the gates are 0 or 1 and nothing turns into NaN, up to the largest finite numbers."""
    g = torch.tensor([[-3e38, -1e20, -200.0, -88.0, 88.0, 200.0, 1e20, 3e38]], device="cuda")
    one = torch.ones_like(g)
    for kind in ("silu", "gelu"):
        r = F.gated_grad(one, g, one, act=kind, again=True)
        assert torch.isfinite(r.a).all() and torch.isfinite(r.gate).all()
        assert (r.gate[0, 4:] == 1).all() and (r.a[0, 4:] == g[0, 4:]).all() and (r.a[0, :3].abs() < 1e-30).all()


# ---------------------------------------------------------------------------
# the backward pass's products
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("wt", ["same", "f32", "bf16"])
@pytest.mark.parametrize("t,d,f,dt,off,pad", GATED + [(1000, 64, 72, "bf16", 0, 0), (2048, 128, 64, "f16", 0, 0),
                                                     (3001, 40, 24, "bf16", 0, 0), (4096, 256, 264, "bf16", 0, 0)])
def test_products_whole_numbers(t, d, f, dt, off, pad, wt):
    say(f"products {t}x{d}x{f} {dt} -> {wt} off {off} pad {pad}")
    wt = dt if wt == "same" else wt
    g = np.random.default_rng(t * 31 + d + f)
    x, wg, wu = gated_case(t, d, f, dt, off, pad, g)
    dg, du = (Mat(t, f, dt, off, f + pad, whole(g, (t, f))) for _ in range(2))
    dx = Mat(t, d, dt, off, d + 2 * pad)
    F.gated_input_grad(dg.v, du.v, wg.v, wu.v, out=dx.v)
    wdx, wdwg, wdwu = OF.products(f64(dg.v), f64(du.v), f64(x.v), f64(wg.v), f64(wu.v))
    same(dx.v, rounded(wdx, dt), "dx")
    old = whole(g, (2, f, d))
    gg, gu = (Mat(f, d, wt, off + 1, d + pad, old[i]) for i in range(2))
    r = F.gated_weight_grad(dg.v, du.v, x.v, gg.v, gu.v)
    assert r[0] is gg.v and r[1] is gu.v
    same(gg.v, rounded(wdwg, wt), "dw_gate")
    same(gu.v, rounded(wdwu, wt), "dw_up")
    for m, o in ((gg, old[0]), (gu, old[1])):
        m.check()
        m.v.copy_(torch.from_numpy(o))
    ws = F.gated_workspace(t + 5, d + 3, f)
    F.gated_weight_grad(dg.v, du.v, x.v, gg.v, gu.v, accumulate=True, workspace=ws)
    same(gg.v, rounded(wdwg + old[0], wt), "dw_gate added")
    same(gu.v, rounded(wdwu + old[1], wt), "dw_up added")
    for m in (x, wg, wu, dg, du, dx, gg, gu):
        m.check()


@pytest.mark.parametrize("t,d,f,dt", [(300, 64, 200, "bf16"), (777, 136, 72, "f16"), (130, 33, 77, "f32"), (2500, 256, 264, "bf16")])
def test_products_random(t, d, f, dt):
    g = np.random.default_rng(t + d)
    x, dg, du = (torch.from_numpy(g.normal(size=(t, c))).to(T[dt]).cuda() for c in (d, f, f))
    wg, wu = (torch.from_numpy(g.normal(size=(f, d)) / 8).to(T[dt]).cuda() for _ in range(2))
    want = OF.products(*(f64(v) for v in (dg, du, x, wg, wu)))
    mag = OF.products(*(np.abs(f64(v)) for v in (dg, du, x, wg, wu)))
    close(F.gated_input_grad(dg, du, wg, wu), want[0], 3 * 2 * f * E * mag[0], "dx")
    gg, gu = (torch.empty(f, d, device="cuda") for _ in range(2))
    F.gated_weight_grad(dg, du, x, gg, gu)
    close(gg, want[1], 3 * t * E * mag[1], "dw_gate")
    close(gu, want[2], 3 * t * E * mag[2], "dw_up")
    # equal calls give equal bits
    a, b = (torch.empty(f, d, device="cuda") for _ in range(2))
    F.gated_weight_grad(dg, du, x, a, b)
    assert torch.equal(a, gg) and torch.equal(b, gu)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f", [(20, 48, 64), (130, 33, 77), (3, 260, 129)])
def test_products_against_differences(t, d, f, kind):
    """The gradients of x and both weights along a direction in all of them, from kept tensors, against central
    differences of the forward pass; their third-order error is bounded by that of twice the step."""
    g = torch.Generator(device="cuda").manual_seed(t)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, wg, wu, c = r(t, d), r(f, d) * d ** -0.5, r(f, d) * d ** -0.5, r(t, f)
    v, vg, vu = r(t, d), r(f, d) * d ** -0.5, r(f, d) * d ** -0.5
    k = F.gated(x, wg, wu, act=kind, keep="tensors")
    b = F.gated_grad(c, k.gate, k.up, act=kind)
    dx = F.gated_input_grad(b.gate, b.up, wg, wu)
    gg, gu = torch.empty_like(wg), torch.empty_like(wu)
    F.gated_weight_grad(b.gate, b.up, x, gg, gu)
    terms = [(p.double() * q.double()) for p, q in ((dx, v), (gg, vg), (gu, vu))]
    got = float(sum(p.sum() for p in terms))
    loss = lambda s: float((F.gated(x + s * v, wg + s * vg, wu + s * vu, act=kind).a.double() * c.double()).sum())  # noqa: E731
    s = 2.0 ** -8
    num, num2 = ((loss(i * s) - loss(-i * s)) / (2 * i * s) for i in (1, 2))
    # a is off by some (3 d + 20) e of the sums of magnitudes, here of size d^(1/2) at most 4 each, at random
    size = float((k.a.double() * c.double()).abs().sum() + c.double().abs().sum())
    noise = (3 * d + 20) * E * size / s + 3 * (d + f + t) * E * float(sum(p.abs().sum() for p in terms))
    assert abs(got - num) <= abs(num2 - num) + noise
    assert noise <= 0.1 * abs(got) + 0.02 * float(sum(p.abs().sum() for p in terms))  # it says something


def test_products_empty_and_special():
    e = torch.empty(0, 24, device="cuda").bfloat16()
    w = torch.randn(24, 40, device="cuda").bfloat16()
    assert F.gated_input_grad(e, e, w, w).shape == (0, 40)
    gg, gu = (torch.full((24, 40), 3.0, device="cuda") for _ in range(2))
    x = torch.empty(0, 40, device="cuda").bfloat16()
    F.gated_weight_grad(e, e, x, gg, gu, accumulate=True)
    assert (gg == 3).all() and (gu == 3).all()
    F.gated_weight_grad(e, e, x, gg, gu)
    assert (gg == 0).all() and (gu == 0).all()
    # a NaN token spoils every gradient that it takes part in, and no other token's dx
    dg, du = (torch.randn(50, 24, device="cuda").bfloat16() for _ in range(2))
    clean = F.gated_input_grad(dg, du, w, w)
    bad = dg.clone()
    bad[3, 5] = float("nan")
    dx = F.gated_input_grad(bad, du, w, w)
    assert torch.isnan(dx[3]).all() and torch.equal(dx[4:], clean[4:]) and torch.equal(dx[:3], clean[:3])
    y = torch.randn(50, 40, device="cuda").bfloat16()
    F.gated_weight_grad(bad, du, y, gg, gu)
    assert torch.isnan(gg[5]).all() and torch.isfinite(gg[[i for i in range(24) if i != 5]]).all() and torch.isfinite(gu).all()
    # a weight's infinity reaches its column of dx alone
    v = w.clone()
    v[3, 7] = float("inf")
    dx = F.gated_input_grad(dg, du, v, w)
    ok = [c for c in range(40) if c != 7]
    assert torch.equal(dx[:, ok], clean[:, ok]) and not torch.isfinite(dx[:, 7]).any()


# Every variant that a rule on sizes chooses, with whole numbers on the GPU: dense and padded operands,
# aligned ones and others.
def on_gpu(gen, rows, cols, dt, off=0, pad=0, most=2):
    """Whole numbers of -most .. most in a padded matrix; NaN in the padding."""
    flat = torch.full((off + rows * (cols + pad),), float("nan"), dtype=T[dt], device="cuda")
    v = flat[off:].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.randint(-most, most + 1, (rows, cols), generator=gen, device="cuda", dtype=torch.int8))
    return v


FORMS = [  # tokens, dim, hidden, type, offset, padding
    (4000, 200, 2040, "bf16", 0, 0), (4001, 72, 2041, "f16", 0, 8), (2100, 136, 1000, "bf16", 0, 0), (65, 328, 9000, "bf16", 0, 0),
    (16384, 64, 520, "bf16", 0, 0),
    (1, 840, 8300, "bf16", 0, 0), (5, 64, 8200, "f16", 0, 0), (17, 136, 8300, "bf16", 0, 0), (32, 72, 200, "bf16", 0, 0),
    (33, 840, 300, "f16", 0, 0), (64, 200, 8300, "bf16", 0, 0), (64, 8, 31, "f16", 0, 0),
    (1, 841, 8301, "bf16", 0, 0), (2, 63, 33, "f16", 1, 0), (17, 137, 300, "bf16", 0, 1), (33, 300, 77, "f32", 1, 3),
    (64, 129, 1000, "f16", 3, 0), (64, 7, 65, "bf16", 0, 0), (12, 1000, 500, "f32", 0, 0),
    (200, 2200, 600, "f16", 0, 0), (130, 2304, 1000, "bf16", 0, 0), (20, 72, 8320, "f16", 0, 0), (20, 72, 8320, "bf16", 0, 0),
    (40, 72, 8320, "f16", 0, 0), (20, 65, 40, "f16", 0, 0), (29, 260, 200, "f32", 0, 0),
    (65, 9, 31, "bf16", 0, 0), (300, 515, 190, "bf16", 0, 0), (1025, 191, 333, "f16", 5, 3), (257, 512, 640, "f32", 0, 0),
    (129, 31, 65, "f32", 1, 1), (130, 64, 66, "bf16", 4, 0),
    (3, 16, (1 << 18) + 40, "bf16", 0, 0), ((1 << 18) + 5, 8, 16, "f16", 0, 0), (3, 5, (1 << 18) + 33, "f32", 0, 0),
]


@pytest.mark.parametrize("t,d,f,dt,off,pad", FORMS)
def test_gated_forms(t, d, f, dt, off, pad):
    say(f"gated {t}x{d}x{f} {dt} off {off} pad {pad}")
    gen = torch.Generator(device="cuda").manual_seed(t + d + f)
    x = on_gpu(gen, t, d, dt, off, pad)
    wg, wu = (on_gpu(gen, f, d, dt, off, pad) for _ in range(2))
    gate, up = ((x.float() @ w.float().t()).contiguous() for w in (wg, wu))  # exact
    kept = F.gated(x, wg, wu, act="gelu", keep="tensors")
    assert torch.equal(kept.gate, gate.to(T[dt])) and torch.equal(kept.up, up.to(T[dt]))
    held = F.gated(x, wg, wu, act="gelu", keep="packed")
    for got, v in ((held.gate, gate), (held.up, up)):
        want = F.pack8(v)
        assert torch.equal(got.codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(got.scales.view(torch.uint8), want.scales.view(torch.uint8))
    lean = F.gated(x, wg, wu, act="gelu").a
    assert torch.equal(lean, kept.a) and torch.equal(lean, held.a)
    # a = g p u with p = 1 / (1 + exp(-z)): z off by 6 e |z| moves p by p (1 - p) 6 e |z|, the rest by 8 e p (or
    # p reads 0 below 2^-126); the two products and what else is rounded 3 e
    g, u = gate.double(), up.double()
    z = 2 * 0.7978845608028654 * (g + 0.044715 * g ** 3)
    p = 1 / (1 + torch.exp(-z))
    want = g * p * u
    err = (6 * z.abs() * (1 - p) + 11) * E * want.abs() + 2.0 ** -126 * (g * u).abs()
    tol = 1.01 * (err + torch.finfo(T[dt]).eps / 2 * want.abs()) + SUB[T[dt]]
    fits = want.abs() <= 65000 if dt == "f16" else torch.ones_like(want, dtype=torch.bool)
    assert ((lean.double() - want).abs() <= tol)[fits].all()


PRODUCT_FORMS = [  # tokens, dim, hidden, type, offset, padding
    (4096, 4096, 72, "bf16", 0, 0), (4100, 2048, 200, "f16", 0, 8), (100, 4096, 2048, "bf16", 0, 0), (100, 4096, 2048, "f16", 0, 0),
    (1024, 1024, 1024, "f32", 0, 0), (1000, 2040, 2304, "bf16", 0, 0), (1000, 2040, 2304, "f16", 0, 0),
    (300, 512, 5000, "bf16", 0, 0), (9000, 136, 72, "bf16", 0, 0), (9000, 136, 72, "f16", 0, 8), (1, 512, 5000, "bf16", 0, 0),
    (1, 513, 5001, "bf16", 0, 0), (1, 300, 700, "f32", 0, 0), (9001, 137, 71, "bf16", 0, 0), (9001, 66, 130, "f16", 1, 0),
    (2500, 100, 60, "f32", 0, 0), (2501, 130, 129, "f32", 3, 1), (700, 260, 390, "bf16", 4, 0), (3, 5, 4099, "f16", 0, 3),
    (64, 7, 33, "bf16", 0, 0), (129, 3, 1000, "bf16", 0, 0), (40, 1000, 6, "f32", 0, 0), (63, 129, 127, "f16", 0, 0),
    (65, 8, 8, "bf16", 0, 0), (1, 1, 1, "f16", 0, 0),
    ((1 << 18) + 9, 8, 16, "bf16", 0, 0), (5, (1 << 18) + 8, 16, "bf16", 0, 0), (5, 8, (1 << 18) + 24, "f16", 0, 0),
    (6, (1 << 18) + 7, 5, "f32", 0, 0),
]


@pytest.mark.parametrize("t,d,f,dt,off,pad", PRODUCT_FORMS)
def test_product_forms(t, d, f, dt, off, pad):
    say(f"products {t}x{d}x{f} {dt} off {off} pad {pad}")
    gen = torch.Generator(device="cuda").manual_seed(t + d + f)
    x, dg, du = (on_gpu(gen, t, c, dt, off, pad) for c in (d, f, f))
    wg, wu = (on_gpu(gen, f, d, dt, off, pad) for _ in range(2))
    dx = F.gated_input_grad(dg, du, wg, wu)
    want = dg.double() @ wg.double() + du.double() @ wu.double()
    assert torch.equal(dx, want.float().to(T[dt]))
    for wt in ("f32", "bf16", "f16"):
        sums = [(v.double().t() @ x.double()).float() for v in (dg, du)]
        grads = [Mat(f, d, wt, off, d + pad) for _ in range(2)]
        F.gated_weight_grad(dg, du, x, grads[0].v, grads[1].v)
        for m, w in zip(grads, sums):
            assert torch.equal(m.v, w.to(T[wt])), wt
            m.v.fill_(3.0)
        F.gated_weight_grad(dg, du, x, grads[0].v, grads[1].v, accumulate=True)
        for m, w in zip(grads, sums):
            assert torch.equal(m.v, (w + 3.0).to(T[wt])), wt
            m.check()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_products_keep_apart_what_is_not_finite(dt):
    """NaN and infinities reach the results whose sums they are part of, in every form: aligned tiles,
    others, few tokens, split sums."""
    for t, d, f in ((300, 136, 200), (300, 137, 201), (5, 136, 200), (5, 137, 201), (2049, 72, 72), (2049, 71, 73)):
        say(f"not finite {t}x{d}x{f} {dt}")
        gen = torch.Generator(device="cuda").manual_seed(t + d)
        x, dg, du = (on_gpu(gen, t, c, dt) for c in (d, f, f))
        wg, wu = (on_gpu(gen, f, d, dt) for _ in range(2))
        clean = F.gated(x, wg, wu, keep="tensors")
        y, v = x.clone(), wg.clone()
        y[-1, -1] = float("nan")
        v[-1, 0] = float("inf")
        got = F.gated(y, wg, wu, keep="tensors")
        for a, b in zip(got, clean):
            assert torch.isnan(a[-1]).all() and torch.equal(a[:-1], b[:-1])
        got = F.gated(x, v, wu, keep="tensors")
        assert torch.equal(got.a[:, :-1], clean.a[:, :-1]) and torch.equal(got.gate[:, :-1], clean.gate[:, :-1])
        assert torch.equal(got.up, clean.up) and not torch.isfinite(got.gate[:, -1]).any()
        dx = F.gated_input_grad(dg, du, wg, wu)
        bad = du.clone()
        bad[-1, -1] = float("nan")
        got = F.gated_input_grad(dg, bad, wg, wu)
        assert torch.isnan(got[-1]).all() and torch.equal(got[:-1], dx[:-1])
        v = wu.clone()
        v[-1, -1] = float("nan")
        got = F.gated_input_grad(dg, du, wg, v)
        assert torch.isnan(got[:, -1]).all() and torch.equal(got[:, :-1], dx[:, :-1])
        one, two = ([torch.empty(f, d, device="cuda") for _ in range(2)] for _ in range(2))
        F.gated_weight_grad(dg, du, x, *one)
        F.gated_weight_grad(dg, bad, y, *two)
        assert torch.isnan(two[1][-1]).all() and torch.isnan(two[0][:, -1]).all()
        assert torch.equal(two[0][:, :-1], one[0][:, :-1]) and torch.equal(two[1][:-1, :-1], one[1][:-1, :-1])


@pytest.mark.parametrize("t,d,f,dt", [(5, 33, 40, "f32"), (37, 64, 136, "bf16"), (70, 65, 33, "f16"), (300, 128, 264, "bf16")])
def test_column_ranges_of_one_buffer(t, d, f, dt):
    """Matrices that lie side by side in the rows of one buffer, read and written: what a call gives is what
    it gives apart, and the columns between are left as they were."""
    gen = torch.Generator(device="cuda").manual_seed(t)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(T[dt])  # noqa: E731

    def beside(rows, *cols):
        m = Mat(rows, sum(cols) + 3 * len(cols), dt)
        at, out = 0, []
        for c in cols:
            out.append(m.v[:, at:at + c])
            at += c + 3
        return m, out

    x, res, w, wg, wu = r(t, d), r(t, d), r(d), r(f, d), r(f, d)
    m, (xs, rs, ts, ys) = beside(t, d, d, d, d)
    xs.copy_(x), rs.copy_(res)
    a, b = F.rms_norm(x, w, eps=1e-5, residual=res), F.rms_norm(xs, w, eps=1e-5, residual=rs, total=ts, out=ys)
    assert torch.equal(ys, a.y) and torch.equal(ts, a.total) and torch.equal(b.rstd, a.rstd)
    assert torch.equal(xs, x) and torch.equal(rs, res)
    assert torch.isnan(m.v[:, d:d + 3]).all() and torch.isnan(m.v[:, -3:]).all()
    dn, dres = r(t, d), r(t, d)
    gw, hw = (torch.empty(d, device="cuda") for _ in range(2))
    want = F.rms_norm_grad(dn, a.total, a.rstd, w, residual_grad=dres, weight_grad=gw)
    xs.copy_(dn), rs.copy_(dres)
    F.rms_norm_grad(xs, ts, a.rstd, w, residual_grad=rs, out=ys, weight_grad=hw)
    assert torch.equal(ys, want) and torch.equal(gw, hw)
    # weights in one [f, 2 d] buffer, gate, up and a in one [t, 3 f]
    m, (gs, us) = beside(f, d, d)
    gs.copy_(wg), us.copy_(wu)
    m2, (as_, gate, up) = beside(t, f, f, f)
    one, two = F.gated(x, wg, wu, keep="tensors"), F.gated(x, gs, us, out=as_, keep=(gate, up))
    for p, q in zip(one, two):
        close(q, f64(p), np.maximum(np.abs(f64(p)), 1.0) * (d + 40) * 8 * E + (0 if dt == "f32" else 2.0 ** -7 * np.abs(f64(p))))
    assert torch.isnan(m2.v[:, f:f + 3]).all() and torch.isnan(m2.v[:, 2 * f + 3:2 * f + 6]).all()
    da = r(t, f)
    m3, (dg, du) = beside(t, f, f)
    ref = F.gated_grad(da, gate.contiguous(), up.contiguous())
    F.gated_grad(da, gate, up, out_gate=dg, out_up=du, again=as_)
    assert torch.equal(dg, ref.gate) and torch.equal(du, ref.up)
    # whole numbers: exact on every path
    for v in (dg, du):
        v.copy_(torch.randint(-2, 3, v.shape, generator=gen, device="cuda"))
    xi, gi, ui = (torch.randint(-2, 3, s, generator=gen, device="cuda").to(T[dt]) for s in ((t, d), (f, d), (f, d)))
    gs.copy_(gi), us.copy_(ui)
    m4, (dx, other) = beside(t, d, d)
    F.gated_input_grad(dg, du, gs, us, out=dx)
    assert torch.equal(dx, (dg.double() @ gi.double() + du.double() @ ui.double()).to(T[dt]))
    assert torch.isnan(other).all()
    m5, (wgrad, ugrad) = beside(f, d, d)
    F.gated_weight_grad(dg, du, xi, wgrad, ugrad)
    assert torch.equal(wgrad, (dg.double().t() @ xi.double()).to(T[dt]))
    assert torch.equal(ugrad, (du.double().t() @ xi.double()).to(T[dt]))
    assert torch.isnan(m5.v[:, d:d + 3]).all()
    codes = torch.zeros(t, 2 * f, dtype=torch.float8_e4m3fn, device="cuda")
    blocks = OF.blocks(f)
    scales = torch.zeros(t, 2 * blocks, dtype=torch.uint8, device="cuda")
    for k, v in enumerate((dg, du)):
        p = F.pack8(v, out=F.Packed8(codes[:, k * f:(k + 1) * f], scales[:, k * blocks:(k + 1) * blocks]))
        assert torch.equal(F.unpack8(p, T[dt]), F.unpack8(F.pack8(v), T[dt]))


# ---------------------------------------------------------------------------
# streams, graphs, and a run of them together
# ---------------------------------------------------------------------------

def block(x, res, w_norm, wg, wu, wd, dout, grads, ws, kind="silu"):
    """Forward and backward of one sub-layer from 8-bit checkpoints: out = total + gated(...) w_down^T.
    Returns (out, dres); the weights' gradients go to `grads`."""
    n = F.rms_norm(x, w_norm, eps=1e-5, residual=res, packed=True)
    kept = F.pack8(n.total)
    f = F.gated(n.y, wg, wu, act=kind, keep="packed")
    out = n.total + f.a @ wd.t()
    b = F.gated_grad(dout @ wd, f.gate, f.up, act=kind, again=True)
    grads["wd"].copy_(dout.t() @ b.a)
    dn = F.gated_input_grad(b.gate, b.up, wg, wu, workspace=ws[0])
    F.gated_weight_grad(b.gate, b.up, F.unpack8(n.packed, x.dtype), grads["wg"], grads["wu"], workspace=ws[0])
    dres = F.rms_norm_grad(dn, kept, n.rstd, w_norm, residual_grad=dout, weight_grad=grads["norm"], workspace=ws[1])
    return out, dres


def make_block(t, d, f, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(T[dt])  # noqa: E731
    p = dict(x=r(t, d), res=r(t, d), w_norm=(1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(T[dt]),
             wg=r(f, d, k=d ** -0.5), wu=r(f, d, k=d ** -0.5), wd=r(d, f, k=f ** -0.5), dout=r(t, d, k=0.1))
    grads = dict(wd=torch.empty_like(p["wd"]), wg=torch.empty_like(p["wg"]), wu=torch.empty_like(p["wu"]),
                 norm=torch.empty_like(p["w_norm"]))
    ws = F.gated_workspace(t, d, f), F.rms_norm_grad_workspace(t, d)
    return p, grads, ws


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_block_against_float64(kind):
    """The whole sub-layer in bf16 from 8-bit checkpoints against the float64 gradients of
    the exact block, norm-wise.  What differs: y, gate and up are held with 2^-4 relative error at most
    (uniform over a step: rms 2^-4 / sqrt(3) = 0.036 at the worst place in the binade, of which the
    activations' checkpoint enters once in dW (y), and twice in dg (gate and up) through factors of
    size one; h once in n; bf16 results add 2^-9 each.  Root of the sum of squares of four such
    errors of 0.036: 0.072."""
    p, grads, ws = make_block(200, 256, 512, "bf16")
    out, dres = block(p["x"], p["res"], p["w_norm"], p["wg"], p["wu"], p["wd"], p["dout"], grads, ws, kind)
    q = {k: f64(v) for k, v in p.items()}
    h = f64(p["x"].float() + p["res"].float())
    y, rstd = OF.rms_norm(h, q["w_norm"], 1e-5)
    a, gate, up = OF.gated(y, q["wg"], q["wu"], kind)
    want_out = h + a @ q["wd"].T
    da = q["dout"] @ q["wd"]
    dg, du, _ = OF.gated_grad(da, gate, up, kind)
    dy, dwg, dwu = OF.products(dg, du, y, q["wg"], q["wu"])
    dh, dw = OF.rms_norm_grad(dy, h, rstd, q["w_norm"], q["dout"])
    off = lambda got, want: np.linalg.norm(f64(got) - want) / np.linalg.norm(want)  # noqa: E731
    assert off(out, want_out) <= 2.0 ** -7
    for name, got, want in (("dres", dres, dh), ("wd", grads["wd"], q["dout"].T @ a), ("wg", grads["wg"], dwg),
                            ("wu", grads["wu"], dwu), ("norm", grads["norm"], dw)):
        assert off(got, want) <= 0.072, (name, off(got, want))


def test_side_stream():
    p, grads, ws = make_block(130, 128, 264, "bf16")
    want = block(**{k: v for k, v in p.items()}, grads=grads, ws=ws)
    ref = {k: v.clone() for k, v in grads.items()}
    for v in grads.values():
        v.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = block(**p, grads=grads, ws=ws)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for k in ref:
        assert torch.equal(grads[k], ref[k]), k


def test_graph_replays():
    """Forward and backward captured once and replayed with new inputs, eager work between the
    replays: every replay equals the eager result.  Two graphs that run in turn share the workspaces."""
    sizes = [(70, 128, 264), (300, 64, 72)]
    graphs = []
    big = F.gated_workspace(300, 128, 264), F.rms_norm_grad_workspace(300, 128)
    for t, d, f in sizes:
        p, grads, _ = make_block(t, d, f, "bf16")
        block(**p, grads=grads, ws=big)  # warm up
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            block(**p, grads=grads, ws=big)
        s.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = block(**p, grads=grads, ws=big)
        graphs.append((gr, p, grads, out, (t, d, f)))
    for turn in range(4):
        for gr, p, grads, out, size in graphs:
            fresh = make_block(*size, "bf16", seed=10 + turn)[0]
            for k in p:
                p[k].copy_(fresh[k])
            gr.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in out] + [grads[k].clone() for k in sorted(grads)]
            other = {k: torch.empty_like(v) for k, v in grads.items()}
            want = list(block(**fresh, grads=other, ws=big)) + [other[k] for k in sorted(other)]
            for a, b in zip(got, want):
                assert torch.equal(a, b), turn
            torch.cuda.synchronize()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_graph_replays_of_other_forms(dt):
    """Odd widths, few tokens, split sums and accumulated gradients, captured together on one workspace."""
    sizes = [(33, 137, 201), (300, 64, 3000), (5, 96, 1040), (700, 130, 66)]
    ws = F.gated_workspace(700, 137, 3000), F.rms_norm_grad_workspace(700, 137)

    def run(p, grads, acc):
        n = F.rms_norm(p["x"], p["w_norm"], eps=1e-5, residual=p["res"], packed=True)
        f = F.gated(n.y, p["wg"], p["wu"], act="gelu", keep="packed")
        b = F.gated_grad(f.a, f.gate, f.up, act="gelu", again=True)
        dn = F.gated_input_grad(b.gate, b.up, p["wg"], p["wu"], workspace=ws[0])
        F.gated_weight_grad(b.gate, b.up, n.y, grads["wg"], grads["wu"], accumulate=acc, workspace=ws[0])
        dh = F.rms_norm_grad(dn, n.total, n.rstd, p["w_norm"], residual_grad=p["dout"], weight_grad=grads["norm"],
                             accumulate=acc, workspace=ws[1])
        return [f.a, b.a, dn, dh]

    ps, gs = zip(*(make_block(*s, dt)[:2] for s in sizes))
    for p, g in zip(ps, gs):
        run(p, g, False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = []
        for p, g in zip(ps, gs):
            run(p, g, False)
            outs.append(run(p, g, True))
    for turn in range(4):
        fresh = [make_block(*s, dt, seed=20 + turn)[0] for s in sizes]
        for p, q in zip(ps, fresh):
            for k in p:
                p[k].copy_(q[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] + [g[k].clone() for k in ("wg", "wu", "norm")] for o, g in zip(outs, gs)]
        for q, g, have in zip(fresh, gs, got):
            other = {k: torch.empty_like(v) for k, v in g.items()}
            run(q, other, False)
            want = run(q, other, True) + [other[k] for k in ("wg", "wu", "norm")]
            for a, b in zip(have, want):
                assert torch.equal(a, b), turn


def test_two_streams_at_once():
    """Calls of two streams at the same time, each with a workspace of its own, give what they give alone."""
    sizes = [(300, 512, 1376), (2000, 136, 264)]
    jobs = [make_block(*s, "bf16", seed=i) for i, s in enumerate(sizes)]
    want = []
    for p, grads, ws in jobs:
        out = [t.clone() for t in block(**p, grads=grads, ws=ws)]
        want.append(out + [grads[k].clone() for k in sorted(grads)])
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (p, grads, ws), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(list(block(**p, grads=grads, ws=ws)))
        torch.cuda.synchronize()
        for (p, grads, ws), have, w in zip(jobs, got, want):
            for a, b in zip(have + [grads[k] for k in sorted(grads)], w):
                assert torch.equal(a, b)


def test_training_with_the_sharded_step():
    """The sub-layer's weights live in the gather buffer and their gradients in the flat gradient that
    the step reads: four steps, eager, and as a captured graph of two replayed twice, end with
    the same weights; the first step moves every weight as Adam's rule says for its gradient."""
    t, d, f, lr = 120, 40, 88, 1e-2
    shapes = [(d,), (f, d), (f, d), (d, f)]
    sizes = [int(np.prod(s)) for s in shapes]
    g = torch.Generator(device="cuda").manual_seed(1)
    master = torch.cat([torch.randn(n, generator=g, device="cuda") * 0.2 + (i == 0) for i, n in enumerate(sizes)])
    x, res, dout = (torch.randn(t, d, generator=g, device="cuda").bfloat16() for _ in range(3))
    ws = F.gated_workspace(t, d, f), F.rms_norm_grad_workspace(t, d)

    def run(graph):
        opt = ZeroAdam(sizes, 1, 0, lr=lr, grad_dtype=torch.bfloat16, param_dtype=torch.bfloat16, master=master,
                       device_control=True)
        opt.gather.copy_(master[:opt.gather.numel()])
        flat = torch.zeros(1, opt.plan.padded_numel, dtype=torch.bfloat16, device="cuda")
        w = [opt.param(i, s) for i, s in enumerate(shapes)]
        gr = dict(zip(("norm", "wg", "wu", "wd"), (opt.grad_view(flat[0], i, s) for i, s in enumerate(shapes))))

        def step():
            block(x, res, *w, dout, gr, ws)
            opt.step(flat, full=True)

        first = None
        if graph:
            side = torch.cuda.Stream()
            cg = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                block(x, res, *w, dout, gr, ws)  # warm up the libraries
            side.synchronize()
            with torch.cuda.graph(cg):
                step()
                step()
            for _ in range(2):
                cg.replay()
                torch.cuda.synchronize()
        else:
            for i in range(4):
                step()
                if i == 0:
                    torch.cuda.synchronize()
                    first = flat[0].clone(), opt.gather.clone()
        torch.cuda.synchronize()
        assert opt.t == 4 and opt.skipped == 0
        return opt.gather.clone(), flat.clone(), first

    gather, flat, (g0, p0) = run(False)
    gather2, flat2, _ = run(True)
    assert torch.equal(gather, gather2) and torch.equal(flat, flat2)
    assert int((g0 != 0).sum()) > 0.99 * sum(sizes)
    gd = f64(g0)[:sum(sizes)]
    want = f64(master) - lr * gd / (np.abs(gd) + 1e-8)  # the first step's m and v are g and g^2 after their corrections
    # fp32 steps: under 20 roundings of numbers of size |p| + lr; one to bf16
    close(p0[:sum(sizes)], want, 20 * E * (np.abs(f64(master)) + lr), "first step")
