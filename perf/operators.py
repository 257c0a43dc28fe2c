"""The embedding and dropout operators on the sizes they are used at.

`listed()` names the measured cases, `draw(rng)` gives more of the same ranges,
`prepare` makes a case's inputs on the GPU, `run` passes once through the
operator: in plain torch operations, or with `own` set through the package.
`exact` computes the same outputs in float64 from the definition.

Definitions (t a token position, c a column):
  keep(r, c)   the 16-bit number u(r, c) >= rne(65536 p); u comes from
               Philox4x32-10 (Salmon et al., SC'11) with key = seed and counter
               (c div 8, r + first_row, step, site): the low, then the high half
               of the four output words serve columns 8*(c div 8) .. + 7
  ks           65536 / (65536 - rne(65536 p))
  lookup       keep ? (scale * table[id_t] + positions[t mod period]) * ks : 0,
               with a row of zeros for an id outside the table
  gradient     row v of the table: scale * ks * sum of the kept dy[t] with id_t = v
  dropout      keep ? x * ks : 0, plus the residual
"""
import math

import numpy as np
import torch

own = False
_layer = None  # the package's module, imported where `own` is true

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_I = {"i32": torch.int32, "i64": torch.int64}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a 7B decoder as it generates: a single row, latency only
        dict(name="lookup_one_token", op="lookup", tokens=1, rows=32000, dim=4096, dtype="bf16", out="bf16",
             ids="i64", scale=1.0, period=0, p=0.0, pad=0.0, offset=0, device_step=False),
        # GPT-2 1.5B training input: 8 sequences of 1024, positions added, dropout 0.1
        dict(name="lookup_gpt2", op="lookup", tokens=8192, rows=50257, dim=1600, dtype="bf16", out="bf16",
             ids="i64", scale=1.0, period=1024, p=0.1, pad=0.0, offset=0, device_step=True),
        # Llama-3-8B training input: long packed sequences, no positions, no dropout
        dict(name="lookup_llama3", op="lookup", tokens=32768, rows=128256, dim=4096, dtype="bf16", out="bf16",
             ids="i32", scale=1.0, period=0, p=0.0, pad=0.0, offset=0, device_step=False),
        # a padded batch over a table at an odd place of the flat parameters, odd width, fp16 to fp32
        dict(name="lookup_ragged", op="lookup", tokens=5003, rows=9973, dim=777, dtype="f16", out="f32",
             ids="i32", scale=28.0, period=509, p=0.25, pad=0.2, offset=3, device_step=False),
        # a toy model over bytes in fp32: launches only
        dict(name="grad_bytes", op="grad", tokens=64, rows=256, dim=64, dtype="f32", out="f32",
             ids="i64", scale=8.0, period=0, p=0.0, pad=0.0, offset=0, device_step=False),
        # GPT-2 1.5B: the whole word table's gradient of one rank's micro-batch
        dict(name="grad_gpt2", op="grad", tokens=8192, rows=50257, dim=1600, dtype="bf16", out="bf16",
             ids="i64", scale=1.0, period=0, p=0.1, pad=0.0, offset=0, device_step=True),
        # GPT-2 1.5B: the position table's gradient of the same batch
        dict(name="grad_gpt2_positions", op="grad", tokens=8192, rows=1024, dim=1600, dtype="bf16", out="bf16",
             ids="none", scale=1.0, period=1024, p=0.1, pad=0.0, offset=0, device_step=True),
        # Llama-3-8B: a large batch into the largest table
        dict(name="grad_llama3", op="grad", tokens=65536, rows=128256, dim=4096, dtype="bf16", out="bf16",
             ids="i32", scale=1.0, period=0, p=0.0, pad=0.0, offset=0, device_step=False),
        # a padded batch, odd width, fp16 activations into an fp32 gradient at an odd place
        dict(name="grad_ragged", op="grad", tokens=3001, rows=9973, dim=777, dtype="f16", out="f32",
             ids="i64", scale=28.0, period=0, p=0.25, pad=0.2, offset=3, device_step=False),
        # a short fine-tuning batch between two layers
        dict(name="dropout_short", op="dropout", rows=32, dim=1600, dtype="f16", out="f16", residual=False,
             p=0.1, offset=0, device_step=False),
        # GPT-2 1.5B: the end of a block, added to the residual stream
        dict(name="dropout_gpt2_residual", op="dropout", rows=8192, dim=1600, dtype="bf16", out="bf16",
             residual=True, p=0.1, offset=0, device_step=True),
        # a long batch in fp32, odd width: the backward pass of a wide layer
        dict(name="dropout_long_f32", op="dropout", rows=16384, dim=4097, dtype="f32", out="f32", residual=False,
             p=0.5, offset=1, device_step=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    d = _log_int(rng, 64, 8192)
    return d if rng.random() < 0.3 else max(64, d // 8 * 8)


def draw(rng):
    """One more case: one token to 65536, 256 to 128256 rows, widths 64 to 8192
    (three in ten odd), every type, padded batches, tables at odd places."""
    op = rng.choice(["lookup", "grad", "grad", "dropout"])
    types = ["bf16", "bf16", "f16", "f32"]
    dim = _width(rng)
    c = dict(op=op, dim=dim, dtype=rng.choice(types), out=rng.choice(types), p=rng.choice([0.0, 0.1, 0.1, 0.5]),
             offset=rng.choice([0, 0, 8, rng.randrange(1, 64)]), device_step=rng.random() < 0.5)
    # no more elements than the largest listed cases hold
    tokens = min(_log_int(rng, 1, 65536), (65536 * 2048 if c["p"] == 0.0 else 16384 * 4097) // dim)
    if op == "dropout":
        c.update(rows=min(tokens, (16384 * 4097) // dim), residual=rng.random() < 0.5)
        if c["p"] == 0.0:
            c["p"] = 0.2
        return c
    rows = min(_log_int(rng, 256, 128256), (128256 * 2048) // dim)
    positions = rng.random() < 0.25
    c.update(tokens=tokens, rows=rows, ids=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, 1.0, 8.0, 0.5]),
             period=0, pad=rng.choice([0.0, 0.0, 0.3]))
    if positions:
        if op == "lookup":
            c["period"] = _log_int(rng, 1, 4096)
        else:
            c["rows"] = min(rows, _log_int(rng, 1, 8192))
            c.update(ids="none", pad=0.0, period=_log_int(rng, 1, c["rows"]))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _zipf(rows):
    """Shares of the ids of a vocabulary: frequent ids first, Zipf's law with
    Mandelbrot's shift."""
    w = 1.0 / (np.arange(rows, dtype=np.float64) + 2.7)
    return w / w.sum()


def _ids(case, gen):
    n, dev = case["tokens"], gen.device
    cdf = torch.from_numpy(np.cumsum(_zipf(case["rows"]))).to(dev)
    u = torch.rand(n, generator=gen, device=dev, dtype=torch.float64) * cdf[-1]
    t = torch.searchsorted(cdf, u, right=True).clamp_(max=case["rows"] - 1)
    if case["pad"] > 0:  # the tails of padded sequences
        t = torch.where(torch.rand(n, generator=gen, device=dev) < case["pad"], torch.full_like(t, -1), t)
    return t.to(_I[case["ids"]])


def _matrix(gen, rows, cols, dtype, sigma, offset):
    """[rows, cols] view at element `offset` of a flat buffer, N(0, sigma)."""
    flat = torch.empty(offset + rows * cols, dtype=_T[dtype], device=gen.device)
    step = 1 << 26
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=gen, device=gen.device) * sigma)
    return flat[offset:].view(rows, cols)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dim = case["op"], case["dim"]
    s = dict(case=case)
    if op == "lookup":
        s["table"] = _matrix(gen, case["rows"], dim, case["dtype"], 0.02, case["offset"])
        s["ids"] = _ids(case, gen)
        if case["period"]:
            s["positions"] = _matrix(gen, case["period"], dim, case["dtype"], 0.01, case["offset"])
    elif op == "grad":
        s["dy"] = _matrix(gen, case["tokens"], dim, case["dtype"], 1e-2, 0)
        s["ids"] = None if case["ids"] == "none" else _ids(case, gen)
        flat = torch.empty(case["offset"] + case["rows"] * dim, dtype=_T[case["out"]], device="cuda")
        s["grad"] = flat[case["offset"]:].view(case["rows"], dim)
    else:
        s["x"] = _matrix(gen, case["rows"], dim, case["dtype"], 1.0, case["offset"])
        if case["residual"]:
            s["residual"] = _matrix(gen, case["rows"], dim, case["out"], 1.0, 0)
    s["seed"] = 0x9D2C5680_0000_0000 + 977 * seed
    s["site"] = 3
    s["first_row"] = 4096 * (seed % 5)  # the place of this micro-batch in the whole batch
    s["step"] = 1000 + seed % 1000
    if case["device_step"]:  # the step count of a captured training loop
        s["step_tensor"] = torch.tensor([s["step"]], dtype=torch.int64, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

_M32 = 0xFFFFFFFF


def _threshold(p):
    return int(np.rint(p * 65536.0))


def _keep_plain(s, rows, cols):
    """Truth values [rows, cols]; 32-bit words held in int64 (products wrap)."""
    dev = "cuda"
    groups = (cols + 7) // 8
    shape = (rows, groups)
    c0 = torch.arange(groups, dtype=torch.int64, device=dev).expand(shape)
    c1 = ((torch.arange(rows, dtype=torch.int64, device=dev) + s["first_row"]) & _M32)[:, None].expand(shape)
    if "step_tensor" in s:
        c2 = (s["step_tensor"] & _M32).expand(shape)
    else:
        c2 = torch.full(shape, s["step"] & _M32, dtype=torch.int64, device=dev)
    c3 = torch.full(shape, s["site"], dtype=torch.int64, device=dev)
    k0, k1 = s["seed"] & _M32, s["seed"] >> 32 & _M32
    for _ in range(10):
        a = c0 * 0xD2511F53
        b = c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    halves = [h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)]
    u = torch.stack(halves, dim=-1).view(rows, groups * 8)[:, :cols]
    return u >= _threshold(s["case"]["p"])


def _drop_plain(s, y):
    """Dropout of an fp32 [rows, cols] tensor."""
    p = s["case"]["p"]
    if _threshold(p) == 0:
        return y
    ks = 65536.0 / (65536 - _threshold(p))
    return torch.where(_keep_plain(s, *y.shape), y * ks, torch.zeros_like(y))


def _plain(s):
    c = s["case"]
    out = _T[c["out"]]
    if c["op"] == "lookup":
        ids = s["ids"].long()
        inside = (ids >= 0) & (ids < c["rows"])
        y = s["table"][ids.clamp(0, c["rows"] - 1)].float() * c["scale"]
        y = torch.where(inside[:, None], y, torch.zeros_like(y))
        if c["period"]:
            y = y + s["positions"][torch.arange(c["tokens"], device="cuda") % c["period"]].float()
        return _drop_plain(s, y).to(out)
    if c["op"] == "grad":
        if s["ids"] is None:
            ids = torch.arange(c["tokens"], device="cuda") % c["period"]
        else:
            ids = s["ids"].long()
        g = _drop_plain(s, s["dy"].float()) * c["scale"]
        ids = torch.where((ids >= 0) & (ids < c["rows"]), ids, torch.full_like(ids, c["rows"]))
        acc = torch.zeros(c["rows"] + 1, c["dim"], dtype=torch.float32, device="cuda")
        acc.index_add_(0, ids, g)
        s["grad"].copy_(acc[:c["rows"]])
        return s["grad"]
    y = _drop_plain(s, s["x"].float())
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(out)


def run(state):
    if not own:
        return _plain(state)
    global _layer
    if _layer is None:
        from zero_sharded_mixed_plan_amd import input_layer as _layer
    L, s, c = _layer, state, state["case"]
    drop = None
    if c["p"] > 0:
        drop = L.Dropout(c["p"], seed=s["seed"], site=s["site"], step=s.get("step_tensor", s["step"]),
                         row0=s["first_row"])
    if c["op"] == "lookup":
        return L.embedding(s["ids"], s["table"], scale=c["scale"], pos_table=s.get("positions"),
                           pos_period=c["period"], drop=drop, out_dtype=_T[c["out"]])
    if c["op"] == "grad":
        return L.embedding_grad(s["dy"], s["ids"], s["grad"], scale=c["scale"], period=c["period"], drop=drop)
    return L.dropout(s["x"], drop, residual=s.get("residual"), out_dtype=_T[c["out"]])


def work(case):
    """Each input once, each output once; of a table the rows that this many
    tokens are expected to touch."""
    dim, es, os_ = case["dim"], _BYTES[case["dtype"]], _BYTES[case["out"]]
    if case["op"] == "dropout":
        n = case["rows"] * dim
        return {"bytes": n * (es + os_ * (2 if case["residual"] else 1)), "flops": n * (2 if case["residual"] else 1)}
    n = case["tokens"]
    id_bytes = {"i32": 4, "i64": 8, "none": 0}[case["ids"]] * n
    live = n * (1.0 - case["pad"])
    if case["op"] == "lookup":
        touched = float((1.0 - (1.0 - _zipf(case["rows"])) ** live).sum())
        positions = min(case["period"], n)
        return {"bytes": int((touched + positions) * dim * es + id_bytes + n * dim * os_), "flops": 2 * n * dim}
    return {"bytes": int(live * dim * es + id_bytes + case["rows"] * dim * os_), "flops": int(2 * live * dim)}


# ---------------------------------------------------------------------------
# float64, from the definition
# ---------------------------------------------------------------------------

def _mul_hi_lo(m, x):
    """High and low 32 bits of m * x, from 16-bit limbs."""
    m0, m1, x0, x1 = m % 65536, m // 65536, x % 65536, x // 65536
    low = m0 * x0
    mid = m1 * x0 + low // 65536
    mid2 = m0 * x1 + mid % 65536
    return m1 * x1 + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + low % 65536


def _uniform16(seed, site, step, row, cols, dev):
    """u(r, c) of the rows in `row` (int64 tensor), as int64 [len(row), cols]."""
    g = (cols + 7) // 8
    n = row.numel()
    ctr = [torch.arange(g, device=dev).repeat(n), row.repeat_interleave(g) % 2**32,
           torch.full((n * g,), step % 2**32, device=dev), torch.full((n * g,), site, device=dev)]
    key = [seed % 2**32, seed // 2**32 % 2**32]
    for r in range(10):
        rk = [(key[0] + r * 0x9E3779B9) % 2**32, (key[1] + r * 0xBB67AE85) % 2**32]
        h0, l0 = _mul_hi_lo(0xD2511F53, ctr[0])
        h1, l1 = _mul_hi_lo(0xCD9E8D57, ctr[2])
        ctr = [h1.bitwise_xor(ctr[1]).bitwise_xor(rk[0]), l1, h0.bitwise_xor(ctr[3]).bitwise_xor(rk[1]), l0]
    u = torch.empty(n * g, 8, dtype=torch.int64, device=dev)
    for j in range(4):
        u[:, 2 * j] = ctr[j] % 65536
        u[:, 2 * j + 1] = ctr[j] // 65536
    return u.view(n, g * 8)[:, :cols]


def _mask64(s, lo, hi):
    """Multiplier 0 or ks of rows lo .. hi - 1 in float64, and the keep flags."""
    c = s["case"]
    drop = int(np.rint(c["p"] * 65536.0))
    rows = torch.arange(lo, hi, device="cuda") + s["first_row"]
    if drop == 0:
        return None, 1.0
    return _uniform16(s["seed"], s["site"], s["step"], rows, c["dim"], "cuda") >= drop, 65536.0 / (65536.0 - drop)


def exact(case, seed):
    s = prepare(case, seed)
    c, dim = case, case["dim"]
    n = c["rows"] if c["op"] == "dropout" else c["tokens"]
    chunk = max(1, (1 << 25) // dim)
    if c["op"] == "grad":
        out = torch.zeros(c["rows"], dim, dtype=torch.float64, device="cuda")
    else:
        out = torch.empty(n, dim, dtype=torch.float64, device="cuda")
    for lo in range(0, n, chunk):
        hi = min(n, lo + chunk)
        keep, ks = _mask64(s, lo, hi)
        if c["op"] == "lookup":
            ids = s["ids"][lo:hi].to(torch.int64)
            y = torch.zeros(hi - lo, dim, dtype=torch.float64, device="cuda")
            live = torch.nonzero((ids >= 0) & (ids < c["rows"])).flatten()
            y[live] = s["table"][ids[live]].double() * float(c["scale"])
            if c["period"]:
                y += s["positions"].double()[torch.arange(lo, hi, device="cuda").remainder(c["period"])]
        elif c["op"] == "grad":
            y = s["dy"][lo:hi].double()
        else:
            y = s["x"][lo:hi].double()
        y = y * ks
        if keep is not None:
            y = y.masked_fill(~keep, 0.0)
        if c["op"] == "grad":
            ids = (torch.arange(lo, hi, device="cuda").remainder(c["period"]) if s["ids"] is None
                   else s["ids"][lo:hi].to(torch.int64))
            live = torch.nonzero((ids >= 0) & (ids < c["rows"])).flatten()
            out.index_put_((ids[live],), y[live] * float(c["scale"]), accumulate=True)
            continue
        if c["op"] == "dropout" and c["residual"]:
            y = y + s["residual"][lo:hi].double()
        out[lo:hi] = y
    return out
