"""Where digits of the feed-forward sub-layer's results could be lost without a sign: gates far out,
sums rounded twice, far magnitudes, scales.

Error bounds beside those of test_gpu_feed_forward.py (e = 2^-24):
  gates of fp32   t = exp(-|z|) = 2^n exp2(f): an ulp, 2 e, and what f, below 1/2, is off, e / 2; or 2^-149 where
              t is a subnormal.  1 + t, its reciprocal and t times that: e each, and t's error divided by 1 + t.
              p and 1 - p are off by at most P = 6 e of themselves, whatever z (GELU: z in fp64, whose
              part beyond fp32 costs one more rounding, P = 7 e), and by 2^-148 where they are subnormals.
              With r = P p + 2^-148:  a = g p u: |g u| r + e |a|,  du = da g p: |g da| r + e |du|,
              act' = p + g p (1 - p) slope, slope off by 5 e: D = r + |g| slope ((2 P + 8 e) p (1 - p) + 2^-147)
              + e |act'|, and dg = da u act': |da u| (D + e |act'|)
"""
import numpy as np
import pytest
import torch

from oracle import feed_forward as OF
from test_gpu_feed_forward import E, close, codes_of, f64
from zero_sharded_mixed_plan_amd import feed_forward as F

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---------------------------------------------------------------------------
# gates
# ---------------------------------------------------------------------------

def far_gates():
    """Gates of both signs, to where silu's are subnormals and gelu's are 0."""
    g = np.concatenate([np.linspace(-103, 103, 4001), np.linspace(-11, 11, 4001), np.exp2(np.linspace(-40, -1, 79)),
                        -np.exp2(np.linspace(-40, -1, 79))])
    return torch.from_numpy(g).float().cuda()


def gate_errors(kind, g):
    """act(g), act'(g), r and D of the bounds above, float64."""
    v, d, p, z, dz = OF.act(kind, g)
    with np.errstate(over="ignore"):
        less = np.where(z >= 0, np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))), 1 / (1 + np.exp(-np.abs(z))))
    rel = (6 if kind == "silu" else 7) * E
    r = rel * p + 2.0 ** -148
    return v, d, r, r + np.abs(g) * dz * ((2 * rel + 8 * E) * p * less + 2.0 ** -147) + E * np.abs(d)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_fp32_gates_keep_their_digits(kind):
    g = far_gates()
    gen = torch.Generator(device="cuda").manual_seed(3)
    da, u = (torch.rand(g.shape, generator=gen, device="cuda") + 0.5 for _ in range(2))
    r = F.gated_grad(da[None], g[None], u[None], act=kind, again=True)
    gs, ds, us = f64(g), f64(da), f64(u)
    v, d, err, D = gate_errors(kind, gs)
    close(r.a[0], v * us, np.abs(gs * us) * err + E * np.abs(v * us), "a")
    close(r.up[0], v * ds, np.abs(gs * ds) * err + E * np.abs(v * ds), "du")
    close(r.gate[0], ds * us * d, np.abs(ds * us) * (D + E * np.abs(d)), "dg")
    # a product of one term gives the gates as they are; few tokens and tiles
    for tokens in (1, 70):
        f = F.gated(torch.ones(tokens, 1, device="cuda"), g[:, None], u[:, None], act=kind).a
        close(f, np.broadcast_to(v * us, f.shape), np.abs(gs * us) * err + E * np.abs(v * us), f"a of {tokens} tokens")


# ---------------------------------------------------------------------------
# scales
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_a_scale_of_255_is_not_a_number(dt):
    """e8m0's NaN, which no call here writes but other programs may: its block reads as NaN, no other does."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(5, 100, generator=g, device="cuda").to(dt)
    x[2, 40] = 0
    p = F.pack8(x)
    want = F.unpack8(p, dt)
    bytes_ = p.scales.view(torch.uint8).clone()
    bytes_[2, 1] = 255
    bad = F.Packed8(p.codes.view(torch.uint8), bytes_)
    got = F.unpack8(bad, dt)
    nan = torch.zeros(5, 100, dtype=torch.bool, device="cuda")
    nan[2, 32:64] = True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], want[~nan])
    one = torch.ones(5, 100, dtype=dt, device="cuda")
    r = F.gated_grad(one, bad, p, again=True)
    assert torch.equal(torch.isnan(r.a), nan) and torch.equal(torch.isnan(r.gate), nan)
    dh = F.rms_norm_grad(one, bad, torch.ones(5, device="cuda"))
    assert torch.equal(torch.isnan(dh).any(1), nan.any(1))


# ---------------------------------------------------------------------------
# the norm's gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt,half", [(torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)])
def test_weight_gradient_is_rounded_once(dt, half):
    """Sums next to the middle of two 16-bit numbers: fp32 in between would put them on it.  Rows of 2500
    columns are a workgroup each, whose sums are joined in fp64."""
    tiny = 2.0 ** -40
    one = torch.ones(2, 2500, device="cuda")

    def grad(first, second, held=None):
        dy = torch.tensor([[first], [second]], device="cuda").expand(2, 2500).contiguous()
        dw = torch.full((2500,), held or 0.0, dtype=dt, device="cuda")
        F.rms_norm_grad(dy, one, torch.ones(2, device="cuda"), weight_grad=dw, accumulate=held is not None)
        return dw

    for held in (None, 1.0):
        base = 0.0 if held else 1.0  # written: all of it in the sum; added: 1 lies there
        for sign in (1.0, -1.0):
            h = None if held is None else sign
            assert (grad(sign * (base + half), sign * tiny, h) == sign * (1 + 2 * half)).all()
            assert (grad(sign * (base + half), 0.0, h) == sign).all()  # the middle: to even
            assert (grad(sign * (base + 3 * half), -sign * tiny, h) == sign * (1 + 2 * half)).all()
            assert (grad(sign * (base + 3 * half), 0.0, h) == sign * (1 + 4 * half)).all()
    big = torch.finfo(dt).max
    assert torch.isinf(grad(3e38, 3e38)).all() and (grad(big, 0.0) == big).all()
    assert torch.isnan(grad(float("nan"), 1.0)).all() and (grad(0.0, 0.0) == 0).all()


@pytest.mark.parametrize("cols", [40, 1500, 8192])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_rms_norm_grad_far_magnitudes(dt, cols):
    """Rows over the whole range in which rstd is a number of fp32: from 1e-38, whose rstd is 1e38, on."""
    g = np.random.default_rng(cols)
    size = np.array([1e-38, 1e-33, 1e-20, 1e-5, 1.0, 1e20, 1e36, 3e37])
    sign = np.where(g.random((8, cols)) < 0.5, -1.0, 1.0)
    h = torch.from_numpy(size[:, None] * sign * (0.5 + g.random((8, cols)))).to(dt).cuda()
    dy = torch.from_numpy(0.25 * g.normal(size=(8, cols))).to(dt).cuda()
    w = torch.from_numpy(1 + 0.1 * g.normal(size=cols)).to(dt).cuda()
    rstd = F.rms_norm(h, w, eps=0.0).rstd
    assert torch.isfinite(rstd).all()
    dw = torch.empty(cols, device="cuda")
    dh = F.rms_norm_grad(dy, h, rstd, w, weight_grad=dw)
    hs, ds, ws, rs = f64(h), f64(dy), f64(w), f64(rstd)
    want, want_dw = OF.rms_norm_grad(ds, hs, rs, ws)
    n, s = hs * rs[:, None], ds * ws
    A = np.abs(s * n).mean(1, keepdims=True)
    close(dh, want, E * rs[:, None] * (3 * np.abs(s) + 40 * A * np.abs(n)) + E * np.abs(want), "dh")
    close(dw, want_dw, (8 + 3) * E * np.abs(ds * n).sum(0), "dweight")
    # a row whose rstd fp32 does not hold spoils no other row's gradient
    tiny = h.clone()
    tiny[3] = 0 if dt == torch.bfloat16 else 1e-44
    rs2 = rstd.clone()
    rs2[3] = float("inf")
    other = F.rms_norm_grad(dy, tiny, rs2, w)
    rest = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(other[rest], dh[rest]) and torch.isnan(other[3]).any()


@pytest.mark.parametrize("t,d,f,dt", [(70, 640, 100, torch.bfloat16), (3, 1600, 700, torch.bfloat16), (300, 512, 264, torch.float16),
                                      (40, 333, 77, torch.float32), (130, 333, 77, torch.bfloat16), (2000, 256, 1376, torch.bfloat16)])
def test_scales_of_sums_are_the_smallest_that_saturate_nothing(t, d, f, dt):
    """Gate and up held in 8 bits: with the block's largest magnitude known within b, the bound of the sums' errors,
    the scale 2^e lets it pass, top - b <= 448 * 2^e, and half of it would not, top + b > 448 * 2^(e - 1)."""
    g = np.random.default_rng(t)
    x = torch.from_numpy(g.normal(size=(t, d))).to(dt).cuda()
    for weights in [[torch.from_numpy(g.normal(size=(f, d)) / d ** 0.5 * size).to(dt).cuda() for size in sizes]
                    for sizes in ((1.0, 30.0), (2.0 ** -9, 0.1))]:
        r = F.gated(x, *weights, keep="packed")
        for p, w in zip((r.gate, r.up), weights):
            s = f64(x) @ f64(w).T
            err = 1.01 * 3 * d * E * (np.abs(f64(x)) @ np.abs(f64(w)).T)
            _, e = codes_of(p)
            for b in range(e.shape[1]):
                part = slice(32 * b, 32 * b + 32)
                top, off = np.abs(s[:, part]).max(1), err[:, part].max(1)
                limit = 448 * np.exp2(e[:, b].astype(float))
                assert (top - off <= limit).all()
                assert ((top + off > limit / 2) | (e[:, b] == -127)).all()
