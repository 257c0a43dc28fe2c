"""The feed-forward sub-layer on the host: the float64 oracle against first principles
and differences, and every refusal of the C ABI and of the torch layer (nothing here
touches a GPU: bad arguments are rejected before anything is enqueued)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import zero_sharded_mixed_plan_amd as Z
from oracle import feed_forward as OF
from zero_sharded_mixed_plan_amd import feed_forward as F

P = 1 << 20            # addresses that are never read: validation comes first
BIG = 1 << 24          # apart from each other


def at(i):
    return P + i * BIG


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------

def test_e4m3_is_the_nearest_number():
    """Against all finite e4m3 numbers, ties to the one with an even fraction; and torch's
    own conversion on fp32 values."""
    codes = np.array([c for c in range(127)])
    vals = OF.e4m3_value(codes)
    assert vals[-1] == 448.0 and vals[1] == 2.0 ** -9 and vals[8] == 2.0 ** -6
    g = np.random.default_rng(0)
    v = np.concatenate([vals, (vals[1:] + vals[:-1]) / 2, g.uniform(0, 448, 400), np.exp2(g.uniform(-12, 8.8, 400))])
    d = np.abs(v[:, None] - vals[None, :])
    best = d.min(axis=1)
    near = [[c for c in codes if d[i, c] == best[i]] for i in range(len(v))]
    want = np.array([vals[n[0] if len(n) == 1 or n[0] % 2 == 0 else n[1]] for n in near])
    assert np.array_equal(OF.e4m3(v), want) and np.array_equal(OF.e4m3(-v), -want)
    f = torch.from_numpy(v.astype(np.float32))
    assert np.array_equal(OF.e4m3(f.double().numpy()), f.to(torch.float8_e4m3fn).double().numpy())


def test_held_scale_is_the_smallest_that_saturates_nothing():
    g = np.random.default_rng(1)
    v = g.normal(size=(50, 70)) * np.exp2(g.integers(-30, 30, size=(50, 1)))
    v[0] = 0
    v[1, :32], v[2, :32], v[3, :32] = 448.0, np.nextafter(448.0, 449), 0.875
    v[4, 5] = np.inf
    v[5, 6] = np.nan
    q, e = OF.hold(v)
    assert np.array_equal(e[:4, 0], [-127, 0, 1, -9])
    fin = np.isfinite(v)
    assert np.array_equal(np.isnan(q), ~fin) and np.nanmax(np.abs(q)) <= 448
    for b in range(3):
        top = np.where(fin, np.abs(v), 0)[:, 32 * b:32 * b + 32].max(axis=1)
        live = top > 0
        assert (top[live] <= 448 * np.exp2(e[live, b])).all() and (top[live] > 448 * np.exp2(e[live, b] - 1.0)).all()
    err = np.abs(OF.held_value(q, e) - v)[fin]
    top = np.repeat(np.exp2(e.astype(float)), 32, axis=1)[:, :70][fin]
    assert (err <= np.maximum(np.abs(v[fin]) * 2.0 ** -4, top * 2.0 ** -10)).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_gradients_against_differences(kind):
    """One block in float64: every formula of the backward pass against central
    differences of the forward pass."""
    g = np.random.default_rng(2)
    t, d, f, eps = 5, 6, 7, 1e-5
    x, res, w = g.normal(size=(t, d)), g.normal(size=(t, d)), g.normal(size=d)
    wg, wu, c = g.normal(size=(f, d)), g.normal(size=(f, d)), g.normal(size=(t, f))
    dpast = g.normal(size=(t, d))

    def loss(res=res, w=w, wg=wg, wu=wu):
        h = x + res
        y, _ = OF.rms_norm(h, w, eps)
        return (OF.gated(y, wg, wu, kind)[0] * c).sum() + (h * dpast).sum()

    h = x + res
    y, rstd = OF.rms_norm(h, w, eps)
    a, gate, up = OF.gated(y, wg, wu, kind)
    dg, du, again = OF.gated_grad(c, gate, up, kind)
    assert np.allclose(again, a, rtol=1e-14)
    dy, dwg, dwu = OF.products(dg, du, y, wg, wu)
    dh, dw = OF.rms_norm_grad(dy, h, rstd, w, dpast)
    for name, v, grad in (("res", res, dh), ("w", w, dw), ("wg", wg, dwg), ("wu", wu, dwu)):
        num = np.empty_like(v)
        for i in np.ndindex(v.shape):
            s = 1e-5
            p, m = v.copy(), v.copy()
            p[i] += s
            m[i] -= s
            num[i] = (loss(**{name: p}) - loss(**{name: m})) / (2 * s)
        assert np.allclose(num, grad, rtol=1e-6, atol=1e-7), name


# ---------------------------------------------------------------------------
# the C ABI
# ---------------------------------------------------------------------------

def held(i, cols=40, **kw):
    h = Z.zero_held_t(at(i), cols, at(i + 1), OF.blocks(cols))
    for k, v in kw.items():
        setattr(h, k, v or None)
    return h


def fill(struct, base, kw, pointers):
    a = struct()
    a._keep = []
    for k, v in {**base, **kw}.items():
        if isinstance(v, Z.zero_held_t):
            a._keep.append(v)
            v = ctypes.addressof(v)
        setattr(a, k, (v or None) if k in pointers else v)
    return a


def refused(call, code, name):
    with pytest.raises(Z.ZeroError) as e:
        call()
    assert e.value.code == code and name in Z.zero_last_error()


IN, AL = Z.ZERO_EINVAL, Z.ZERO_EALIGN


@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), IN), (dict(rows=1 << 40), IN), (dict(cols=0), IN), (dict(cols=1 << 31), IN), (dict(x=0), IN), (dict(x=at(0) + 1), AL),
    (dict(ld=39), IN), (dict(ld=1 << 62), IN), (dict(dtype=3), IN), (dict(h=held(1, codes=0)), IN),
    (dict(h=held(1, scales=0)), IN), (dict(h=held(1, ld_codes=39)), IN), (dict(h=held(1, ld_scales=1)), IN),
    (dict(h=held(1, ld_codes=1 << 41)), IN), (dict(h=held(1, codes=at(0) + 100)), IN),
    (dict(h=held(1, scales=at(0) + 799)), IN),
    (dict(h=None), IN)])
def test_hold_refuses(pack, kw, code):
    a = dict(x=at(0), ld=40, dtype=Z.ZERO_BF16, rows=10, cols=40, h=held(1))
    a.update(kw)
    h = ctypes.addressof(a["h"]) if a["h"] is not None else None
    L = Z.lib()
    if pack:
        rc = L.zero_pack8(a["x"] or None, a["ld"], a["dtype"], a["rows"], a["cols"], h, None)
    else:
        rc = L.zero_unpack8(h, a["rows"], a["cols"], a["x"] or None, a["ld"], a["dtype"], None)
    assert rc == code and ("zero_pack8" if pack else "zero_unpack8") in Z.zero_last_error()


def test_codes_and_scales_that_overlap_are_refused_where_they_are_written():
    h = held(1, scales=at(1) + 5)
    assert Z.lib().zero_pack8(at(0), 40, Z.ZERO_F32, 10, 40, ctypes.addressof(h), None) == IN


RMS_PTR = ("x", "residual", "total", "weight", "out", "held", "rstd")


def rms_args(**kw):
    base = dict(x=at(0), ld_x=40, x_dtype=Z.ZERO_BF16, res_dtype=Z.ZERO_BF16, residual=at(1), ld_res=40, total=at(2),
                ld_total=40, weight=at(3), weight_dtype=Z.ZERO_BF16, out_dtype=Z.ZERO_BF16, out=at(4), ld_out=40,
                held=held(5), rstd=at(7), rows=10, cols=40, eps=1e-5)
    return fill(Z.zero_rms_args_t, base, kw, RMS_PTR)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), IN), (dict(rows=1 << 40), IN), (dict(cols=0), IN), (dict(cols=8193), IN), (dict(eps=-1e-9), IN),
    (dict(eps=float("nan")), IN), (dict(eps=float("inf")), IN), (dict(x=0), IN), (dict(x=at(0) + 1), AL),
    (dict(x_dtype=5), IN), (dict(ld_x=39), IN), (dict(residual=0), IN), (dict(total=0), IN), (dict(ld_res=39), IN),
    (dict(ld_total=39), IN), (dict(total=at(2) + 1), AL), (dict(res_dtype=Z.ZERO_F16), IN),
    (dict(x_dtype=Z.ZERO_F32), IN), (dict(weight=at(3) + 1), AL), (dict(weight_dtype=7), IN),
    (dict(out_dtype=-1), IN), (dict(out=at(4) + 1), AL), (dict(ld_out=39), IN), (dict(rstd=at(7) + 2), AL),
    (dict(out=0, held=None), IN), (dict(held=held(5, codes=0)), IN), (dict(held=held(5, ld_scales=1)), IN),
    (dict(total=at(1) + 2), IN), (dict(total=at(1), ld_total=48), IN),
    (dict(total=at(0), res_dtype=Z.ZERO_F32), IN),                       # in place with another type
    (dict(out=at(0)), IN), (dict(out=at(1)), IN), (dict(out=at(2)), IN), (dict(out=at(3)), IN),
    (dict(rstd=at(4) + 8), IN), (dict(held=held(5, codes=at(4))), IN), (dict(held=held(5, scales=at(7))), IN)])
def test_rms_norm_refuses(kw, code):
    refused(lambda: Z.zero_rms_norm(rms_args(**kw)), code, "zero_rms_norm")


RG_PTR = ("dy", "h", "held", "rstd", "weight", "dres", "dh", "dweight", "ws")


def rms_grad_args(**kw):
    base = dict(dy=at(0), ld_dy=40, dy_dtype=Z.ZERO_BF16, h_dtype=Z.ZERO_BF16, h=at(1), ld_h=40, held=None, rstd=at(2),
                weight=at(3), weight_dtype=Z.ZERO_F32, dweight_dtype=Z.ZERO_BF16, dres=at(4), ld_dres=40, dh=at(5),
                ld_dh=40, dweight=at(6), accumulate=0, reserved=0, rows=10, cols=40, ws=at(7),
                ws_bytes=Z.zero_rms_grad_ws_bytes(10, 40))
    return fill(Z.zero_rms_grad_args_t, base, kw, RG_PTR)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), IN), (dict(cols=0), IN), (dict(cols=8193), IN), (dict(reserved=1), IN), (dict(dy=0), IN),
    (dict(dy_dtype=9), IN), (dict(h_dtype=9), IN), (dict(h_dtype=Z.ZERO_F16), IN), (dict(dy_dtype=Z.ZERO_F32), IN),
    (dict(dy=at(0) + 1), AL), (dict(ld_dy=39), IN), (dict(h=0), IN), (dict(held=held(8)), IN),
    (dict(h=0, held=held(8, scales=0)), IN), (dict(ld_h=39), IN), (dict(rstd=0), IN), (dict(rstd=at(2) + 2), AL),
    (dict(weight=at(3) + 2), AL), (dict(weight_dtype=4), IN), (dict(dres=at(4) + 1), AL), (dict(ld_dres=39), IN),
    (dict(dh=0), IN), (dict(ld_dh=39), IN), (dict(dweight=at(6) + 1), AL), (dict(dweight_dtype=4), IN),
    (dict(ws=0), IN), (dict(ws_bytes=100), IN), (dict(ws=at(7) + 8), AL), (dict(dh=at(0) + 2), IN),
    (dict(dh=at(0), ld_dh=48), IN), (dict(dh=at(0), h_dtype=Z.ZERO_F32), IN), (dict(dh=at(2)), IN),
    (dict(dh=at(3)), IN), (dict(dweight=at(0)), IN), (dict(dweight=at(3)), IN), (dict(ws=at(0)), IN),
    (dict(ws=at(5)), IN), (dict(h=0, held=held(8), dh=at(8)), IN)])
def test_rms_norm_grad_refuses(kw, code):
    refused(lambda: Z.zero_rms_norm_grad(rms_grad_args(**kw)), code, "zero_rms_norm_grad")


G_PTR = ("x", "w_gate", "w_up", "a", "g", "u", "g8", "u8", "da", "dg", "du", "dx", "dw_gate", "dw_up", "ws")


def gated_args(**kw):
    base = dict(tokens=10, dim=24, hidden=40, dtype=Z.ZERO_BF16, act=0, x=at(0), ld_x=24, w_gate=at(1), ld_w_gate=24,
                w_up=at(2), ld_w_up=24, a=at(3), ld_a=40, g=0, ld_g=40, u=0, ld_u=40, g8=held(6), u8=held(8), da=at(10),
                ld_da=40, dg=at(11), ld_dg=40, du=at(12), ld_du=40, dx=at(13), ld_dx=24, dw_gate=at(14), ld_dw_gate=24,
                dw_up=at(15), ld_dw_up=24, dw_dtype=Z.ZERO_F32, accumulate=0, ws=at(16),
                ws_bytes=Z.zero_gated_ws_bytes(10, 24, 40))
    return fill(Z.zero_gated_args_t, base, kw, G_PTR)


SIZES = [(dict(tokens=-1), IN), (dict(tokens=1 << 31), IN), (dict(hidden=0), IN), (dict(hidden=1 << 31), IN),
         (dict(dtype=6), IN)]
DIMS = [(dict(dim=0), IN), (dict(dim=1 << 31), IN)]
KEPT = [(dict(g=at(4)), IN), (dict(u=at(5)), IN), (dict(g8=None), IN), (dict(g=at(4), u=at(5)), IN),
        (dict(g8=held(6, codes=0)), IN), (dict(u8=held(8, ld_codes=39)), IN),
        (dict(g8=None, u8=None, g=at(4), u=at(5) + 1), AL), (dict(g8=None, u8=None, g=at(4), u=at(5), ld_g=39), IN)]


@pytest.mark.parametrize("kw,code", SIZES + DIMS + KEPT + [
    (dict(act=2), IN), (dict(act=-1), IN), (dict(x=0), IN), (dict(x=at(0) + 1), AL), (dict(ld_x=23), IN),
    (dict(w_gate=0), IN), (dict(w_up=0), IN), (dict(ld_w_gate=23), IN), (dict(w_up=at(2) + 1), AL), (dict(a=0), IN),
    (dict(ld_a=39), IN), (dict(a=at(0)), IN), (dict(a=at(1)), IN), (dict(a=at(2) + 2), IN),
    (dict(u8=held(8, codes=at(6))), IN), (dict(g8=held(6, codes=at(3))), IN),
    (dict(g8=None, u8=None, g=at(4), u=at(4)), IN), (dict(g8=None, u8=None, g=at(4), u=at(3)), IN)])
def test_gated_refuses(kw, code):
    refused(lambda: Z.zero_gated(gated_args(**kw)), code, "zero_gated")


@pytest.mark.parametrize("kw,code", SIZES + KEPT + [
    (dict(act=2), IN), (dict(da=0), IN), (dict(dg=0), IN), (dict(du=0), IN), (dict(da=at(10) + 1), AL),
    (dict(ld_dg=39), IN), (dict(ld_a=39), IN), (dict(g8=None, u8=None), IN), (dict(dg=at(10) + 2), IN),
    (dict(dg=at(10), ld_dg=48), IN), (dict(du=at(11)), IN), (dict(a=at(12)), IN), (dict(dg=at(6)), IN),
    (dict(du=at(9)), IN)])
def test_gated_grad_refuses(kw, code):
    refused(lambda: Z.zero_gated_grad(gated_args(**kw)), code, "zero_gated_grad")


@pytest.mark.parametrize("kw,code", SIZES + DIMS + [
    (dict(dg=0), IN), (dict(du=0), IN), (dict(w_gate=0), IN), (dict(w_up=0), IN), (dict(dx=0), IN),
    (dict(dx=at(13) + 1), AL), (dict(ld_dx=23), IN), (dict(ld_du=39), IN), (dict(dx=at(11)), IN), (dict(dx=at(2)), IN),
    (dict(ws=0), IN), (dict(ws_bytes=100), IN), (dict(ws=at(16) + 8), AL), (dict(ws=at(13)), IN), (dict(ws=at(1)), IN)])
def test_gated_input_grad_refuses(kw, code):
    refused(lambda: Z.zero_gated_input_grad(gated_args(**kw)), code, "zero_gated_input_grad")


@pytest.mark.parametrize("kw,code", SIZES + DIMS + [
    (dict(dg=0), IN), (dict(du=0), IN), (dict(x=0), IN), (dict(dw_gate=0), IN), (dict(dw_up=0), IN),
    (dict(dw_dtype=3), IN), (dict(dw_gate=at(14) + 2), AL), (dict(ld_dw_up=23), IN), (dict(ld_x=23), IN),
    (dict(dw_up=at(14) + 4), IN), (dict(dw_gate=at(0)), IN), (dict(dw_up=at(12)), IN), (dict(ws=0), IN),
    (dict(ws_bytes=100), IN), (dict(ws=at(16) + 8), AL), (dict(ws=at(15)), IN), (dict(ws=at(0)), IN)])
def test_gated_weight_grad_refuses(kw, code):
    refused(lambda: Z.zero_gated_weight_grad(gated_args(**kw)), code, "zero_gated_weight_grad")


@pytest.mark.parametrize("kw", [
    dict(dg=at(11), ld_dg=79, du=at(11) + 80, ld_du=79),          # the second's last column wraps onto the first's
    dict(dg=at(11), ld_dg=80, du=at(11) + 78, ld_du=80),          # begins in the first's last column
    dict(dg=at(11), ld_dg=80, du=at(11) + 160 * 3 + 82, ld_du=80),  # the same rows further down, and past the row
    dict(dg=at(11) + 160, ld_dg=80, du=at(11) + 82, ld_du=80),
    dict(dg=at(11), ld_dg=80, du=at(11) + 80, ld_du=81),          # strides that differ
    dict(dg=at(10) + 82, ld_dg=80, ld_da=80)])
def test_column_ranges_that_meet_are_refused(kw):
    refused(lambda: Z.zero_gated_grad(gated_args(**kw)), IN, "zero_gated_grad")


def test_null_arguments():
    L = Z.lib()
    for fn in (L.zero_rms_norm, L.zero_rms_norm_grad, L.zero_gated, L.zero_gated_grad, L.zero_gated_input_grad,
               L.zero_gated_weight_grad):
        assert fn(None, None) == IN


def test_empty_calls_do_nothing():
    """No rows: nothing is read, launched or checked for overlap."""
    Z.zero_rms_norm(rms_args(rows=0, x=0, residual=0, total=0, out=0, held=None))
    Z.zero_rms_norm_grad(rms_grad_args(rows=0, dy=0, h=0, dres=0, dh=0, dweight=0, rstd=0))
    none = dict(tokens=0, x=0, a=0, da=0, dg=0, du=0, dx=0, g8=None, u8=None)
    for fn in (Z.zero_gated, Z.zero_gated_grad, Z.zero_gated_input_grad):
        fn(gated_args(**none))
    h = Z.zero_held_t()
    Z.zero_pack8(0, 40, Z.ZERO_BF16, 0, 40, h)
    Z.zero_unpack8(h, 0, 40, 0, 40, Z.ZERO_BF16)


def test_workspaces_never_shrink():
    sizes = [0, 1, 2, 7, 63, 64, 255, 256, 257, 1000, 1023, 1024, 1025, 8191, 8192, 100000]
    for cols in (1, 40, 512, 513, 4096, 4097, 8192):
        need = [Z.zero_rms_grad_ws_bytes(n, cols) for n in sizes]
        assert min(need) > 0 and need == sorted(need)
    for n in sizes:
        need = [Z.zero_rms_grad_ws_bytes(n, c) for c in range(1, 8193, 7)]
        assert need == sorted(need)
    for bad in ((-1, 5), (1, 0), (1, 8193), (1 << 40, 5)):
        assert Z.zero_rms_grad_ws_bytes(*bad) == 0
    dims = [1, 8, 63, 64, 65, 127, 128, 129, 256, 257, 511, 512, 513, 1376, 1600, 4096, 11008, 14336, 20000]
    f = Z.zero_gated_ws_bytes
    for d in dims:
        for h in dims:
            need = [f(n, d, h) for n in sizes]
            assert min(need) > 0 and need == sorted(need), (d, h)
    for n in (0, 1, 100, 8192):
        for d in dims:
            need = [f(n, d, h) for h in range(1, 9000, 31)]
            assert need == sorted(need), (n, d)
            need = [f(n, h, d) for h in range(1, 9000, 31)]
            assert need == sorted(need), (n, d)
    top = (1 << 31) - 1
    assert f(top, top, top) > 0
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 31, 1, 1), (1, 1 << 31, 1), (1, 1, 1 << 31)):
        assert f(*bad) == 0


def test_structs_match_the_header(tmp_path):
    """Sizes and every field's place as the C compiler lays the header's structs out."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    types = {n: getattr(Z, n) for n in ("zero_held_t", "zero_rms_args_t", "zero_rms_grad_args_t", "zero_gated_args_t")}
    body = "".join(f'printf("%zu\\n", sizeof({n}));' +
                   "".join(f'printf("%zu\\n", offsetof({n}, {f[0]}));' for f in t._fields_)
                   for n, t in types.items())
    src = tmp_path / "layout.c"
    src.write_text(f"#include <stdio.h>\n#include <zero_shard.h>\nint main(void) {{ {body} return 0; }}\n")
    cc = shutil.which("gcc") or shutil.which("cc")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "layout")],
                   check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "layout")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    want = [x for t in types.values() for x in [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]]
    assert got == want


# ---------------------------------------------------------------------------
# the torch layer
# ---------------------------------------------------------------------------

def z(*shape, dtype=torch.float32, **kw):
    return torch.zeros(*shape, dtype=dtype, **kw)


B = torch.bfloat16
X, W, WF = z(4, 8), z(8), z(6, 8)


@pytest.mark.parametrize("call,error,text", [
    (lambda: F.pack8(X), ValueError, "GPU"),
    (lambda: F.pack8(z(4, 8, dtype=torch.float64)), TypeError, "dtype"),
    (lambda: F.pack8(z(8, 4).t()), ValueError, "adjacent"),
    (lambda: F.rms_norm(z(4, 0), eps=1e-5), ValueError, "no columns"),
    (lambda: F.pack8(X, out=F.packed8_empty((4, 9), "cpu")), ValueError, "codes must be"),
    (lambda: F.pack8(X, out=F.Packed8(z(4, 8), z(4, 1))), TypeError, "float8"),
    (lambda: F.pack8(X, out=F.Packed8(z(4, 8, dtype=torch.uint8), z(4, 2, dtype=torch.uint8))), ValueError, "one for each"),
    (lambda: F.unpack8(F.packed8_empty((4, 8), "cpu")), ValueError, "GPU"),
    (lambda: F.unpack8(F.packed8_empty((4, 8), "cpu"), B, out=X), ValueError, "out must be"),
    (lambda: F.rms_norm(X, W, eps=1e-5), ValueError, "GPU"),
    (lambda: F.rms_norm(X, z(9), eps=1e-5), ValueError, "vector of 8"),
    (lambda: F.rms_norm(X, z(16)[::2], eps=1e-5), ValueError, "contiguous vector"),
    (lambda: F.rms_norm(X, W, eps=1e-5, residual=z(4, 9)), ValueError, "one shape"),
    (lambda: F.rms_norm(X, W, eps=1e-5, total=X), ValueError, "without a residual"),
    (lambda: F.rms_norm(X, W, eps=1e-5, residual=X, total=z(4, 8, dtype=B)), ValueError, "total must be"),
    (lambda: F.rms_norm(X, W, eps=1e-5, out=False), ValueError, "neither"),
    (lambda: F.rms_norm(X, W, eps=1e-5, out=X, out_dtype=B), ValueError, "out must be"),
    (lambda: F.rms_norm(X, W, eps=1e-5, rstd=z(5)), ValueError, "rstd"),
    (lambda: F.rms_norm(X, W, eps=1e-5, rstd=z(4, dtype=B)), ValueError, "rstd"),
    (lambda: F.rms_norm_grad(X, X, z(4), W), ValueError, "GPU"),
    (lambda: F.rms_norm_grad(X, z(4, 9), z(4), W), ValueError, "one shape"),
    (lambda: F.rms_norm_grad(X, X, z(5), W), ValueError, "rstd"),
    (lambda: F.rms_norm_grad(X, X, z(4), W, residual_grad=z(4, 8, dtype=B)), ValueError, "residual_grad must be"),
    (lambda: F.rms_norm_grad(X, X, z(4), W, out_dtype=B), ValueError, "another type"),
    (lambda: F.rms_norm_grad(X, X, z(4), W, accumulate=True), ValueError, "without a weight_grad"),
    (lambda: F.rms_norm_grad(X, X, z(4), W, weight_grad=z(7)), ValueError, "vector of 8"),
    (lambda: F.rms_norm_grad(X, F.packed8_empty((4, 9), "cpu"), z(4), W), ValueError, "codes must be"),
    (lambda: F.rms_norm_grad_workspace(1, 9000), ValueError, "out of range"),
    (lambda: F.gated(X, WF, WF), ValueError, "GPU"),
    (lambda: F.gated(X, WF, z(7, 8)), ValueError, "must be"),
    (lambda: F.gated(X, WF, WF.to(B)), ValueError, "must be"),
    (lambda: F.gated(X, z(6, 9), z(6, 9)), ValueError, "one width"),
    (lambda: F.gated(X, WF, WF, act="relu"), ValueError, "act must be"),
    (lambda: F.gated(X, WF, WF, keep="all"), ValueError, "keep"),
    (lambda: F.gated(X, WF, WF, keep=(z(4, 6), F.packed8_empty((4, 6), "cpu"))), ValueError, "one form"),
    (lambda: F.gated(X, WF, WF, keep=(z(4, 6), z(4, 7))), ValueError, "up must be"),
    (lambda: F.gated(X, WF, WF, out=z(4, 6, dtype=B)), ValueError, "out must be"),
    (lambda: F.gated_grad(X, X, X), ValueError, "GPU"),
    (lambda: F.gated_grad(X, X, F.packed8_empty((4, 8), "cpu")), ValueError, "one form"),
    (lambda: F.gated_grad(X, X, z(4, 8, dtype=B)), ValueError, "up must be"),
    (lambda: F.gated_input_grad(z(4, 6), z(4, 6), WF, WF), ValueError, "GPU"),
    (lambda: F.gated_input_grad(z(4, 6), z(4, 7), WF, WF), ValueError, "one shape"),
    (lambda: F.gated_input_grad(z(4, 5), z(4, 5), WF, WF), ValueError, "hidden size"),
    (lambda: F.gated_input_grad(z(4, 6), z(4, 6), WF, WF, out=z(4, 9)), ValueError, "out must be"),
    (lambda: F.gated_weight_grad(z(4, 6), z(4, 6), X, WF, WF.clone()), ValueError, "GPU"),
    (lambda: F.gated_weight_grad(z(4, 6), z(4, 6), z(5, 8), WF, WF), ValueError, "same rows"),
    (lambda: F.gated_weight_grad(z(4, 6), z(4, 6), X.to(B), WF, WF), ValueError, "same rows and type"),
    (lambda: F.gated_weight_grad(z(4, 6), z(4, 6), X, WF, z(6, 9)), ValueError, "grad_up must be"),
    (lambda: F.gated_weight_grad(z(4, 6), z(4, 6), X, WF, WF.to(B)), ValueError, "one type"),
    (lambda: F.gated_workspace(1, 0, 1), ValueError, "out of range"),
])
def test_torch_layer_refuses(call, error, text):
    with pytest.raises(error, match=text):
        call()


def test_torch_layer_refuses_to_lose_a_gradient():
    w = z(4, 8, requires_grad=True)
    wf = z(6, 8, requires_grad=True)
    calls = [lambda: F.pack8(w), lambda: F.rms_norm(w, W, eps=0.0), lambda: F.rms_norm(X, w[0], eps=0.0),
             lambda: F.rms_norm(X, W, eps=0.0, residual=w), lambda: F.rms_norm_grad(w, X, z(4), W),
             lambda: F.gated(w, WF, WF), lambda: F.gated(X, wf, WF), lambda: F.gated_grad(w, X, X),
             lambda: F.gated_input_grad(z(4, 6), z(4, 6), WF, wf),
             lambda: F.gated_weight_grad(z(4, 6), z(4, 6), w, WF, WF.clone())]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("half", [z(4, 6), F.packed8_empty((4, 6), "cpu")])
def test_gate_and_up_go_together(half):
    """One of the two would be neither read nor written, without a sign."""
    for keep in ((None, half), (half, None)):
        with pytest.raises(ValueError, match="both or neither"):
            F.gated(X, WF, WF, keep=keep)
        with pytest.raises(ValueError, match="both or neither"):
            F.gated_grad(z(4, 6), *keep)
    with pytest.raises(ValueError, match="GPU"):
        F.gated(X, WF, WF, keep=(None, None))


def test_torch_layer_refuses_to_lose_a_tangent():
    """A dual tensor of forward-mode differentiation does not require grad; its primal, and a dual inside a
    Function, get on to the next check (no GPU here)."""
    p = F.packed8_empty((4, 8), "cpu")
    calls = [lambda w, v, m: F.pack8(w), lambda w, v, m: F.unpack8(p, out=w), lambda w, v, m: F.rms_norm(w, W, eps=0.0),
             lambda w, v, m: F.rms_norm(X, v, eps=0.0), lambda w, v, m: F.rms_norm(X, W, eps=0.0, residual=w),
             lambda w, v, m: F.rms_norm_grad(w, X, z(4), W), lambda w, v, m: F.rms_norm_grad(X, w, z(4), W),
             lambda w, v, m: F.rms_norm_grad(X, p, z(4), W, residual_grad=w),
             lambda w, v, m: F.gated(w, WF, WF), lambda w, v, m: F.gated(X, m, WF), lambda w, v, m: F.gated_grad(w, X, X),
             lambda w, v, m: F.gated_grad(X, w, X), lambda w, v, m: F.gated_grad(X, X, w),
             lambda w, v, m: F.gated_input_grad(z(4, 6), z(4, 6), WF, m),
             lambda w, v, m: F.gated_weight_grad(z(4, 6), z(4, 6), w, WF, WF.clone())]
    for call in calls:
        class Through(torch.autograd.Function):
            @staticmethod
            def forward(ctx, *duals):
                call(*duals)

            @staticmethod
            def jvp(ctx, *tangents):
                pass

        with torch.autograd.forward_ad.dual_level():
            duals = [torch.autograd.forward_ad.make_dual(torch.zeros_like(t), torch.ones_like(t)) for t in (X, W, WF)]
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match="tangent"):
                    call(*duals)
            with pytest.raises(ValueError, match="GPU"):
                call(*[torch.autograd.forward_ad.unpack_dual(d).primal for d in duals])
            with pytest.raises(ValueError, match="GPU"):
                Through.apply(*duals)
