"""The input layer on the host: the oracle's generator against published test
vectors, and arguments that the library and the torch layer refuse before
anything is enqueued (no GPU is touched here)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import zero_sharded_mixed_plan_amd as Z
from oracle import input_layer as OI
from zero_sharded_mixed_plan_amd import input_layer as L

P = 1 << 40          # plausible device addresses; nothing reads them
FAR = 1 << 44


# published known answers of Philox4x32-10: counter, key, output
KAT = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


@pytest.mark.parametrize("ctr,key,want", KAT)
def test_generator_known_answers(ctr, key, want):
    got = OI.philox4x32([np.array([c]) for c in ctr], key)
    assert tuple(int(w[0]) for w in got) == want


def test_keep_is_a_function_of_place():
    a = OI.keep(9, 37, p=0.3, seed=5 << 33 | 7, site=2, step=11, row0=4)
    b = OI.keep(3, 21, p=0.3, seed=5 << 33 | 7, site=2, step=11, row0=6)
    assert np.array_equal(a[2:5, :21], b)
    for other in (dict(seed=8), dict(site=3), dict(step=12), dict(row0=5)):
        kw = dict(p=0.3, seed=5 << 33 | 7, site=2, step=11, row0=4)
        kw.update(other)
        assert not np.array_equal(a, OI.keep(9, 37, **kw))
    # share kept: 4 standard deviations of n Bernoulli trials
    n = 400 * 400
    q = 1 - OI.threshold(0.1) / 65536
    k = OI.keep(400, 400, p=0.1, seed=1, site=0, step=0)
    assert abs(k.mean() - q) < 4 * np.sqrt(q * (1 - q) / n)
    assert OI.keep(5, 9, p=0.0, seed=1, site=0, step=0).all()
    assert not OI.keep(5, 9, p=1.0, seed=1, site=0, step=0).any()


def test_oracle_gradient_is_the_lookups_adjoint():
    rng = np.random.default_rng(0)
    table = rng.normal(size=(7, 5))
    ids = [3, 0, 9, 3, -1, 6, 3, 2]
    drop = dict(p=0.4, seed=9, site=1, step=3)
    dy = rng.normal(size=(8, 5))
    g, cnt, _ = OI.lookup_grad(dy, ids, 7, scale=1.5, drop=drop)
    y = OI.lookup(ids, table, scale=1.5, drop=drop)
    assert abs((y * dy).sum() - (table * g).sum()) < 1e-12
    assert list(cnt) == [1, 0, 1, 3, 0, 0, 1]


def _drop(**kw):
    d = Z.zero_drop_t()
    d.p = 0.1
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_DROPS = [(dict(p=-0.1), Z.ZERO_EINVAL), (dict(p=1.5), Z.ZERO_EINVAL), (dict(p=float("nan")), Z.ZERO_EINVAL),
             (dict(reserved=1), Z.ZERO_EINVAL), (dict(step=-1), Z.ZERO_EINVAL), (dict(step=1 << 32), Z.ZERO_EINVAL),
             (dict(row0=-1), Z.ZERO_EINVAL), (dict(row0=(1 << 32) - 3), Z.ZERO_EINVAL),
             (dict(step_dev=FAR + 4), Z.ZERO_EALIGN)]


def _dropout(drop=None, **kw):
    a = dict(x=P, ld_x=40, x_dtype=Z.ZERO_BF16, residual=0, ld_res=0, out=FAR, ld_out=40, out_dtype=Z.ZERO_BF16,
             rows=10, cols=40)
    a.update(kw)
    Z.zero_dropout(drop=drop, **a)


@pytest.mark.parametrize("kw,code", [
    (dict(x=0), Z.ZERO_EINVAL), (dict(out=0), Z.ZERO_EINVAL), (dict(rows=-1), Z.ZERO_EINVAL),
    (dict(cols=0), Z.ZERO_EINVAL), (dict(cols=1 << 31), Z.ZERO_EINVAL), (dict(x_dtype=7), Z.ZERO_EINVAL),
    (dict(out_dtype=-1), Z.ZERO_EINVAL), (dict(ld_x=39), Z.ZERO_EINVAL), (dict(ld_out=39), Z.ZERO_EINVAL),
    (dict(ld_x=1 << 62), Z.ZERO_EINVAL), (dict(x=P + 1), Z.ZERO_EALIGN), (dict(out=FAR + 1), Z.ZERO_EALIGN),
    (dict(residual=P, ld_res=12), Z.ZERO_EINVAL), (dict(residual=P + 1, ld_res=40), Z.ZERO_EALIGN),
    (dict(out=P + 2), Z.ZERO_EINVAL),                               # overlaps x, not in place
    (dict(out=P, ld_out=48), Z.ZERO_EINVAL),                        # in place with another stride
    (dict(out=P, out_dtype=Z.ZERO_F32), Z.ZERO_EINVAL),             # in place with another type
    (dict(out=P, out_dtype=Z.ZERO_F16), Z.ZERO_EINVAL),
    (dict(residual=FAR + 80, ld_res=40), Z.ZERO_EINVAL),            # overlaps the residual
    (dict(drop=_drop(step_dev=FAR + 8)), Z.ZERO_EINVAL),            # step inside out
] + [(dict(drop=_drop(**d)), c) for d, c in BAD_DROPS])
def test_dropout_refuses(kw, code):
    with pytest.raises(Z.ZeroError) as e:
        _dropout(**kw)
    assert e.value.code == code and "zero_dropout" in Z.zero_last_error()


def test_empty_calls_do_nothing():
    _dropout(rows=0, x=0, out=0)
    a = _embed_args(n_ids=0, ids=0, out=0)
    Z.zero_embed_lookup(a)
    Z.zero_embed_grad(_grad_args(rows=0, grad=0))


def _embed_args(**kw):
    a = Z.zero_embed_args_t()
    base = dict(table=P, ld_table=64, rows=100, id0=0, table_dtype=Z.ZERO_BF16, id_bytes=8, ids=2 * P, n_ids=10,
                dim=64, scale=1.0, out=FAR, ld_out=64, out_dtype=Z.ZERO_BF16)
    base.update(kw)
    drop = base.pop("drop", None)
    for k, v in base.items():
        setattr(a, k, v or None if k in ("table", "ids", "out", "pos", "pos_table") else v)
    if drop is not None:
        a.drop = ctypes.addressof(drop)
        a._keep = drop
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(n_ids=-1), Z.ZERO_EINVAL), (dict(n_ids=1 << 31), Z.ZERO_EINVAL), (dict(dim=0), Z.ZERO_EINVAL),
    (dict(rows=-1), Z.ZERO_EINVAL), (dict(id_bytes=2), Z.ZERO_EINVAL), (dict(scale=float("inf")), Z.ZERO_EINVAL),
    (dict(scale=float("nan")), Z.ZERO_EINVAL), (dict(table=0), Z.ZERO_EINVAL), (dict(table=P + 1), Z.ZERO_EALIGN),
    (dict(ld_table=63), Z.ZERO_EINVAL), (dict(ids=0), Z.ZERO_EINVAL), (dict(ids=2 * P + 4), Z.ZERO_EALIGN),
    (dict(out=0), Z.ZERO_EINVAL), (dict(out=FAR + 1), Z.ZERO_EALIGN), (dict(out=P + 128), Z.ZERO_EINVAL),
    (dict(out=2 * P + 16), Z.ZERO_EINVAL), (dict(table_dtype=3), Z.ZERO_EINVAL), (dict(out_dtype=9), Z.ZERO_EINVAL),
    (dict(pos=3 * P), Z.ZERO_EINVAL),
    (dict(pos_table=3 * P, ld_pos=64, pos_rows=8), Z.ZERO_EINVAL),          # no period
    (dict(pos_table=3 * P, ld_pos=64, pos_rows=-8, pos_period=8), Z.ZERO_EINVAL),
    (dict(pos_table=3 * P, ld_pos=60, pos_rows=8, pos_period=8), Z.ZERO_EINVAL),
    (dict(pos_table=3 * P, ld_pos=64, pos_rows=8, pos=4 * P + 4), Z.ZERO_EALIGN),
    (dict(pos_table=FAR, ld_pos=64, pos_rows=8, pos_period=8), Z.ZERO_EINVAL),   # out overlaps it
] + [(dict(drop=_drop(**d)), c) for d, c in BAD_DROPS])
def test_lookup_refuses(kw, code):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_embed_lookup(_embed_args(**kw))
    assert e.value.code == code and "zero_embed_lookup" in Z.zero_last_error()


def _grad_args(**kw):
    a = Z.zero_embed_grad_args_t()
    base = dict(dy=P, ld_dy=64, dy_dtype=Z.ZERO_BF16, id_bytes=8, ids=2 * P, n_ids=10, dim=64, id0=0, rows=100,
                scale=1.0, grad_dtype=Z.ZERO_BF16, grad=FAR, ld_grad=64, ws=5 * P,
                ws_bytes=Z.zero_embed_grad_ws_bytes(10, 100, 64))
    base.update(kw)
    drop = base.pop("drop", None)
    for k, v in base.items():
        setattr(a, k, v or None if k in ("dy", "ids", "grad", "ws") else v)
    if drop is not None:
        a.drop = ctypes.addressof(drop)
        a._keep = drop
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(n_ids=-1), Z.ZERO_EINVAL), (dict(n_ids=1 << 31), Z.ZERO_EINVAL), (dict(rows=-1), Z.ZERO_EINVAL),
    (dict(rows=1 << 31), Z.ZERO_EINVAL), (dict(dim=0), Z.ZERO_EINVAL), (dict(dim=1 << 31), Z.ZERO_EINVAL),
    (dict(n_ids=(1 << 31) - 1, dim=(1 << 31) - 1), Z.ZERO_EINVAL),
    (dict(id_bytes=1), Z.ZERO_EINVAL), (dict(ids=0), Z.ZERO_EINVAL), (dict(ids=2 * P + 4), Z.ZERO_EALIGN),
    (dict(scale=float("nan")), Z.ZERO_EINVAL), (dict(scale=3e38, drop=_drop(p=0.5)), Z.ZERO_EINVAL),
    (dict(dy=0), Z.ZERO_EINVAL), (dict(dy=P + 1), Z.ZERO_EALIGN), (dict(ld_dy=2), Z.ZERO_EINVAL),
    (dict(grad=0), Z.ZERO_EINVAL), (dict(grad=FAR + 1), Z.ZERO_EALIGN), (dict(ld_grad=2), Z.ZERO_EINVAL),
    (dict(dy_dtype=5), Z.ZERO_EINVAL), (dict(grad_dtype=5), Z.ZERO_EINVAL),
    (dict(ws=0), Z.ZERO_EINVAL), (dict(ws_bytes=100), Z.ZERO_EINVAL), (dict(ws=5 * P + 8), Z.ZERO_EALIGN),
    (dict(grad=P), Z.ZERO_EINVAL), (dict(grad=2 * P), Z.ZERO_EINVAL), (dict(ws=FAR + 64), Z.ZERO_EINVAL),
    (dict(ws=P + 16), Z.ZERO_EINVAL),
] + [(dict(drop=_drop(**d)), c) for d, c in BAD_DROPS])
def test_gradient_refuses(kw, code):
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_embed_grad(_grad_args(**kw))
    assert e.value.code == code and "zero_embed_grad" in Z.zero_last_error()


def test_null_arguments():
    for fn in (Z._abi.lib().zero_embed_lookup, Z._abi.lib().zero_embed_grad):
        assert fn(None, None) == Z.ZERO_EINVAL


def test_workspace_bytes():
    f = Z.zero_embed_grad_ws_bytes
    assert f(0, 10, 8) > 0
    assert f(8192, 50257, 1600) >= 2 * 4 * 8192
    assert f(8192, 50257, 1600) <= f(8193, 50257, 1600) <= f(70000, 50257, 1600)
    for bad in ((-1, 1, 1), (1 << 31, 1, 1), (1, -1, 1), (1, 1 << 31, 1), (1, 1, 0), (1, 1, 1 << 31)):
        assert f(*bad) == 0


def test_structs_match_the_header(tmp_path):
    """Sizes and every field's place as the C compiler lays the header's structs out."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    types = {"zero_drop_t": Z.zero_drop_t, "zero_embed_args_t": Z.zero_embed_args_t,
             "zero_embed_grad_args_t": Z.zero_embed_grad_args_t}
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


def test_torch_layer_refuses():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        L.dropout(x, None)
    with pytest.raises(ValueError, match="GPU"):
        L.embedding(torch.zeros(3, dtype=torch.int64), x)
    with pytest.raises(ValueError, match="GPU"):
        L.embedding_grad(x, torch.zeros(4, dtype=torch.int64), torch.zeros(3, 8))
    with pytest.raises(TypeError, match="int32 or int64"):
        L.embedding(torch.zeros(3, dtype=torch.int16), x)
    with pytest.raises(ValueError, match="contiguous"):
        L.embedding(torch.zeros(6, dtype=torch.int64)[::2], x)
    with pytest.raises(ValueError, match="adjacent"):
        L.embedding(torch.zeros(3, dtype=torch.int64), torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="one width"):
        L.embedding_grad(x, torch.zeros(4, dtype=torch.int64), torch.zeros(3, 9))
    with pytest.raises(ValueError, match="ids.shape"):
        L.embedding_grad(x, torch.zeros(5, dtype=torch.int64), torch.zeros(3, 8))
    with pytest.raises(ValueError, match="period"):
        L.embedding_grad(x, None, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="pos_period"):
        L.embedding(torch.zeros(3, dtype=torch.int64), x, pos_table=x)
    with pytest.raises(ValueError, match="one shape"):
        L.dropout(x, None, residual=torch.zeros(4, 9))
    with pytest.raises(ValueError, match="one type"):
        L.dropout(x, None, residual=torch.zeros(4, 8, dtype=torch.bfloat16), out_dtype=torch.float32)
    with pytest.raises(ValueError, match="out of range"):
        L.Dropout(0.1, site=1 << 33)
    with pytest.raises(ValueError, match="int64 tensor"):
        L.Dropout(0.1, step=torch.zeros(1, dtype=torch.int64))


def test_workspace_never_shrinks_as_the_call_grows():
    """A workspace of the largest sizes serves every smaller call: on both sides of
    each step of the chunk length, and over widths and rows."""
    f = Z.zero_embed_grad_ws_bytes
    steps = [n for k in range(3, 22) for n in (2 ** k - 1, 2 ** k, 2 ** k + 1, 5 * 2 ** (k - 2), 5000 + k)]
    for dim in (1, 8, 511, 512, 513, 777, 1600, 2048, 4096, 8192, 70000):
        need = [f(n, 50257, dim) for n in sorted(steps)]
        assert min(need) > 0 and need == sorted(need), dim
    for n in (1, 7, 500, 4096, 8191, 8192, 32768, 40000):
        need = [f(n, 1000, dim) for dim in range(1, 9000, 41)]
        assert min(need) > 0 and need == sorted(need), n
        need = [f(n, rows, 512) for rows in (0, 1, 255, 256, 257, 100000, (1 << 31) - 9000, (1 << 31) - 1)]
        assert min(need) > 0 and need == sorted(need), n
    # a width at which the chunk length steps
    assert f(4096, 1000, 3584) <= f(4096, 1000, 3585)


def test_a_shorter_batch_is_not_refused_the_largest_ones_workspace():
    """The last batch of a loop that allocated for 8192 ids; it gets as far as the
    overlap check."""
    big = Z.zero_embed_grad_ws_bytes(8192, 50257, 1600)
    for n in (8191, 5000, 4097, 1):
        with pytest.raises(Z.ZeroError, match="overlaps an input"):
            Z.zero_embed_grad(_grad_args(n_ids=n, rows=50257, dim=1600, ld_dy=1600, ld_grad=1600, ids=5 * P,
                                         ws_bytes=big))


def test_torch_layer_refuses_to_lose_a_gradient():
    """No history is recorded, so with grad mode on a tensor that requires grad is
    refused; without, the calls get on to the next check (no GPU here)."""
    w = torch.zeros(4, 8, requires_grad=True)
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    calls = [lambda w: L.dropout(w, None), lambda w: L.dropout(x, None, residual=w),
             lambda w: L.dropout(x, None, out=w), lambda w: L.dropout(w * 2, L.Dropout(0.5)),
             lambda w: L.embedding(ids, w), lambda w: L.embedding(ids, x, pos_table=w, pos_period=4),
             lambda w: L.embedding(ids, x, out=w), lambda w: L.embedding_grad(w, ids, x),
             lambda w: L.embedding_grad(x, ids, w)]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call(w)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
            call(w)
        with pytest.raises(ValueError, match="GPU"):
            call(w.detach())


def test_a_dropouts_step_can_be_a_function():
    """Asked at every call; what it gives is checked like any step number."""
    n = [4]
    d = L.Dropout(0.5, step=lambda: n[0])
    assert d.c.step == 4
    n[0] = 7
    assert L._drop(d, 0) == ctypes.addressof(d.c) and d.c.step == 7
    n[0] = 1 << 32
    L._drop(d, 0)
    with pytest.raises(Z.ZeroError, match="step must lie in"):
        _dropout(drop=d.c)
    with pytest.raises(ValueError, match="out of range"):
        L.Dropout(0.5, step=lambda: -1)


def test_torch_layer_refuses_to_lose_a_tangent():
    """As of a tensor that requires grad, of a dual one of forward-mode differentiation; its primal gets on to the
    next check (no GPU here)."""
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    calls = [lambda w: L.dropout(w, None), lambda w: L.dropout(x, None, residual=w), lambda w: L.dropout(x, None, out=w),
             lambda w: L.embedding(ids, w), lambda w: L.embedding(ids, x, pos_table=w, pos_period=4),
             lambda w: L.embedding_grad(w, ids, x), lambda w: L.embedding_grad(x, ids, w)]
    for call in calls:
        with torch.autograd.forward_ad.dual_level():
            w = torch.autograd.forward_ad.make_dual(torch.zeros(4, 8), torch.ones(4, 8))
            with pytest.raises(ValueError, match="tangent"):
                call(w)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                call(w)
            with pytest.raises(ValueError, match="GPU"):
                call(torch.autograd.forward_ad.unpack_dual(w).primal)
