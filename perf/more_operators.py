"""Operators around a block whose linear layers run on 8-bit integers, as cases that can be run and timed: the linear
layer with its gradients, the norms before and after a block with its gate and residual scale, and activations kept in 8
bits.

`run` computes an operator in plain torch operations, or, where `own` is true, through the library."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
GROUP = 128  # columns to a scale, where a row has more than one
LEAST = 2.0**-126  # the smallest scale of values that are not zero


# ---------------------------------------------------------------- cases
def _linear(mode, T, H, N, dtype, group=0, pad=0):
    return {"op": "linear", "mode": mode, "T": T, "H": H, "N": N, "dtype": dtype, "group": group, "pad": pad}


def _norm(mode, rows, cols, dtype, x8=False, gate=True, pad=0):
    return {"op": "norm", "mode": mode, "rows": rows, "cols": cols, "dtype": dtype, "x8": x8, "gate": gate, "pad": pad}


def _pack(mode, rows, cols, dtype, group, pad=0):
    return {"op": mode, "rows": rows, "cols": cols, "dtype": dtype, "group": group, "pad": pad}


def listed():
    named = [
        # one generated token under a dense head of the layer's ordinary width
        ("linear one row", _linear("fwd", 1, 768, 32000, "bf16")),
        # a serving batch against a large head
        ("linear 48 rows", _linear("fwd", 48, 2048, 128000, "bf16")),
        # sizes off every tile, rows that start anywhere
        ("linear ragged f32", _linear("fwd", 777, 1001, 5003, "f32")),
        # a prompt through a block's wide layer
        ("linear 4096 rows", _linear("fwd", 4096, 4096, 16384, "bf16")),
        # the layer's ordinary batch, back, in the type with the short range
        ("linear backward 128 rows f16", _linear("bwd", 128, 768, 5003, "f16", pad=5)),
        # a large step's gradients; the input was kept in 8 bits with a scale for 128 columns
        ("linear backward 8192 rows", _linear("bwd", 8192, 4096, 4096, "bf16", GROUP)),
        # decoding
        ("norm one row", _norm("fwd", 1, 4096, "bf16")),
        # a training batch; the block's output is kept in 8 bits for the backward pass
        ("norm 16384 rows", _norm("fwd", 16384, 4096, "bf16", x8=True)),
        # odd width, rows of a wider buffer
        ("norm backward odd f32", _norm("bwd", 1023, 769, "f32", pad=3)),
        # the training step's gradient, from what was kept in 8 bits
        ("norm backward 16384 rows", _norm("bwd", 16384, 4096, "bf16", x8=True)),
        # activations of a large step, to be kept
        ("pack 32768 rows", _pack("pack", 32768, 4096, "bf16", GROUP)),
        # odd width, rows of a wider buffer, one scale for a row
        ("unpack odd f16", _pack("unpack", 4097, 1001, "f16", 0, pad=7)),
    ]
    return [{"name": n, **c} for n, c in named]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row's width: a usual one, an odd multiple of 8, or any odd number."""
    kind = rng.random()
    if kind < 0.5:
        return rng.choice([n for n in (64, 128, 256, 512, 768, 1024, 2048, 4096, 8192, 16384) if lo <= n <= hi])
    n = _log_int(rng, lo, hi)
    return max(lo, n // 16 * 16 - 8) if kind < 0.8 else n | 1 if n < hi else n - 1


def draw(rng):
    op = rng.choice(["linear fwd", "linear fwd", "linear fwd", "linear bwd", "linear bwd", "norm fwd", "norm bwd",
                     "norm bwd", "pack", "unpack"])
    while op == "linear fwd":
        T, H, N, pad = _log_int(rng, 1, 8192), _width(rng, 64, 8192), _log_int(rng, 64, 262144), rng.choice([0, 0, 16, 5])
        if T * N * H <= 4096 * 16384 * 4096 and N * H <= 128000 * 2048 and T * N <= 4096 * 16384:
            return _linear("fwd", T, H, N, rng.choice(["bf16", "bf16", "f16", "f32"]), 0, pad)
    while op == "linear bwd":
        T, H, N, pad = _log_int(rng, 1, 16384), _width(rng, 64, 8192), _log_int(rng, 64, 65536), rng.choice([0, 0, 16, 5])
        if T * N * H <= 8192 * 4096 * 4096 and N * H <= 1 << 26 and T * N <= 1 << 26 and T * H <= 1 << 26:
            return _linear("bwd", T, H, N, rng.choice(["bf16", "f16"]), rng.choice([0, GROUP]), pad)
    while True:
        rows, cols, pad = _log_int(rng, 1, 32768), _width(rng, 64, 16384), rng.choice([0, 0, 8, 5])
        dtype = rng.choice(["bf16", "f16", "f32"])
        if op in ("pack", "unpack") and rows * cols <= 32768 * 4096 * 2 // SIZES[dtype]:
            return _pack(op, rows, cols, dtype, rng.choice([0, GROUP]), pad)
        if op in ("norm fwd", "norm bwd") and rows * cols <= 16384 * 4096 * 2 // SIZES[dtype]:
            return _norm(op[5:], rows, cols, dtype, rng.random() < 0.5, rng.random() < 0.7, pad)


# ---------------------------------------------------------------- inputs
def _groups(cols, group):
    return -(-cols // group) if group else 1


def _rows(g, rows, cols, dtype, pad=0, std=1.0, spread=0.0):
    """Normal values; with `pad`, the first columns of rows that are `pad` wider; with `spread`, some columns larger than
    others, as a residual stream has them."""
    x = torch.randn((rows, cols + pad), generator=g, device="cuda", dtype=torch.float32)
    if spread:
        x.mul_(torch.exp(spread * torch.randn(cols + pad, generator=g, device="cuda")))
    return x.mul_(std).to(DTYPES[dtype])[:, :cols]


def _rows8(g, rows, cols, std, group=0, pad=0):
    """Normal values in 8 bits, with their scales."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32).mul_(std)
    wide = torch.nn.functional.pad(x, (0, _groups(cols, group) * (group or cols) - cols))
    top = wide.reshape(rows, -1, group or cols).abs().amax(2)
    n = _groups(cols, group)
    inv = (127.0 / top).repeat_interleave(group or cols, 1)[:, :cols] if n > 1 else 127.0 / top
    q = torch.empty((rows, cols + pad), dtype=torch.int8, device="cuda")
    q[:, :cols] = x.mul_(inv).round_().clamp_(-127, 127)
    q[:, cols:] = 99
    scale = top / 127.0
    return q[:, :cols], scale if group else scale[:, 0].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) + 1)
    s = dict(case)
    dt, pad = case["dtype"], case["pad"]
    if case["op"] == "linear":
        T, H, N = case["T"], case["H"], case["N"]
        # features as a norm leaves them, weights that give outputs of about one
        s["x8"], s["x_scale"] = _rows8(g, T, H, 1.0, case["group"], pad)
        s["W8"], s["W_scale"] = _rows8(g, N, H, 1.0 / math.sqrt(H), 0, pad)
        if case["mode"] == "bwd":
            # a mean over the rows leaves small gradients
            s["dout"] = _rows(g, T, N, dt, pad, 1.0 / math.sqrt(T))
        return s
    rows, cols = case["rows"], case["cols"]
    if case["op"] == "pack":
        s["x"] = _rows(g, rows, cols, dt, pad, spread=0.5)
        return s
    if case["op"] == "unpack":
        s["q"], s["scale"] = _rows8(g, rows, cols, 1.0, case["group"], pad)
        return s

    def vec():
        return (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DTYPES[dt])

    s["post"], s["pre"] = vec(), vec()
    s["gate_w"] = (0.5 * vec().float()).to(DTYPES[dt]) if case["gate"] else None
    s["alpha"] = 1.25  # the residual's scale
    if case["mode"] == "fwd":
        s["x"] = _rows(g, rows, cols, dt, pad, spread=0.5)
        s["residual"] = _rows(g, rows, cols, dt, pad, 2.0, 0.5)
        return s
    s["dy"] = _rows(g, rows, cols, dt, pad)
    s["du_in"] = _rows(g, rows, cols, dt, pad)
    x, u = _rows(g, rows, cols, "f32", 0, 1.0, 0.5), _rows(g, rows, cols, "f32", 0, 2.0, 0.5)
    if case["x8"]:
        for k, v in (("x", x), ("u", u)):
            q, scale = _plain_pack(v, GROUP)
            s[k] = torch.empty((rows, cols + pad), dtype=torch.int8, device="cuda")[:, :cols].copy_(q)
            s[k + "_scale"] = scale
    else:
        for k, v in (("x", x), ("u", u)):
            s[k] = torch.empty((rows, cols + pad), dtype=DTYPES[dt], device="cuda")[:, :cols].copy_(v)
            s[k + "_scale"] = None
    s["rstd_x"] = torch.rsqrt(x.square().mean(1) + EPS)
    s["rstd_u"] = torch.rsqrt(u.square().mean(1) + EPS)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_pack(x, group):
    rows, cols = x.shape
    n, w = _groups(cols, group), group or cols
    x = torch.nn.functional.pad(x.float(), (0, n * w - cols)).reshape(rows, n, w)
    top = x.abs().amax(2)
    small = top < 127.0 * LEAST
    inv = torch.where(small, 1.0 / LEAST, 127.0 / top)
    scale = torch.where(small, torch.where(top > 0, LEAST, 0.0), top / 127.0)
    q = (x * inv[:, :, None]).round().clamp(-127, 127).to(torch.int8)
    return q.reshape(rows, n * w)[:, :cols], scale if group else scale[:, 0]


def _plain_unpack(q, scale, group):
    if group:
        scale = scale.repeat_interleave(group, 1)[:, :q.shape[1]]
    else:
        scale = scale[:, None]
    return q.float() * scale


def _plain_linear(s):
    if s["mode"] == "fwd":
        z = s["x8"].float() @ s["W8"].float().t()
        return (z * s["x_scale"][:, None] * s["W_scale"]).to(DTYPES[s["dtype"]])
    d = s["dout"].float()
    dx = d @ _plain_unpack(s["W8"], s["W_scale"], 0)
    dW = d.t() @ _plain_unpack(s["x8"], s["x_scale"], s["group"])
    return {"dx": dx.to(s["dout"].dtype), "dW": dW.to(s["dout"].dtype)}


def _plain_norm_fwd(s):
    x, n = s["x"].float(), s["cols"]
    rx = 1.0 / torch.sqrt((x * x).sum(1) / n + EPS)
    v = x * rx[:, None] * s["post"].float()
    if s["gate_w"] is not None:
        v = v * s["gate_w"].float()
    u = (s["alpha"] * s["residual"].float() + v).to(s["x"].dtype)
    f = u.float()
    ru = 1.0 / torch.sqrt((f * f).sum(1) / n + EPS)
    out = {"u": u, "rstd_x": rx, "rstd_u": ru, "y": (f * ru[:, None] * s["pre"].float()).to(u.dtype)}
    if s["x8"]:
        out["x8"], out["x_scale"] = _plain_pack(s["x"], GROUP)
    return out


def _plain_norm_bwd(s):
    n, dt = s["cols"], s["dy"].dtype
    x, u = ((_plain_unpack(s[k], s[k + "_scale"], GROUP) if s["x8"] else s[k].float()) for k in ("x", "u"))
    rx, ru, dy = s["rstd_x"][:, None], s["rstd_u"][:, None], s["dy"].float()
    m, g = u * ru, dy * s["pre"].float()
    du = ru * (g - m * ((g * m).sum(1) / n)[:, None]) + s["du_in"].float()
    h, post = x * rx, s["post"].float()
    gate = s["gate_w"].float() if s["gate_w"] is not None else torch.ones_like(post)
    k = du * gate * post
    dx = rx * (k - h * ((k * h).sum(1) / n)[:, None])
    sums = (du * h).sum(0)
    out = {"dresidual": (s["alpha"] * du).to(dt), "dx": dx.to(dt), "dpost": gate * sums, "dpre": (dy * m).sum(0)}
    if s["gate_w"] is not None:
        out["dgate"] = post * sums
    return out


# ---------------------------------------------------------------- through the library
def _own_linear(s):
    import extreme_label_sparse_gb300 as sg

    T, H, N, dt = s["T"], s["H"], s["N"], DTYPES[s["dtype"]]
    if s["mode"] == "fwd":
        out = torch.empty((T, N), dtype=dt, device="cuda")
        sg.sg_linear8_fwd(s["x8"], s["x_scale"], s["W8"], s["W_scale"], out)
        return out
    out = {"dx": torch.empty((T, H), dtype=dt, device="cuda"), "dW": torch.empty((N, H), dtype=dt, device="cuda")}
    sg.sg_linear8_bwd(s["x8"], s["x_scale"], s["W8"], s["W_scale"], s["dout"], dx=out["dx"], dW=out["dW"])
    return out


def _own_norm_fwd(s):
    import extreme_label_sparse_gb300 as sg

    x = s["x"]
    rows, cols = x.shape
    out = {k: torch.empty((rows, cols), dtype=x.dtype, device="cuda") for k in ("u", "y")}
    out.update({k: torch.empty(rows, dtype=torch.float32, device="cuda") for k in ("rstd_x", "rstd_u")})
    if s["x8"]:
        out["x8"] = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
        out["x_scale"] = torch.empty((rows, _groups(cols, GROUP)), dtype=torch.float32, device="cuda")
    sg.sg_block_norm_fwd(x, s["post"], s["pre"], EPS, residual=s["residual"], gate=s["gate_w"],
                         residual_scale=s["alpha"], **out)
    return out


def _own_norm_bwd(s):
    import extreme_label_sparse_gb300 as sg

    dy = s["dy"]
    rows, cols = dy.shape
    out = {k: torch.empty((rows, cols), dtype=dy.dtype, device="cuda") for k in ("dresidual", "dx")}
    names = ("dpost", "dpre", "dgate") if s["gate_w"] is not None else ("dpost", "dpre")
    out.update({k: torch.empty(cols, dtype=torch.float32, device="cuda") for k in names})
    sg.sg_block_norm_bwd(dy, s["u"], s["x"], s["post"], s["pre"], s["rstd_x"], s["rstd_u"], u_scale=s["u_scale"],
                         x_scale=s["x_scale"], gate=s["gate_w"], residual_scale=s["alpha"], du_in=s["du_in"], **out)
    return out


def _own_pack(s):
    import extreme_label_sparse_gb300 as sg

    x, group = s["x"], s["group"]
    q = torch.empty(x.shape, dtype=torch.int8, device="cuda")
    n = _groups(s["cols"], group)
    scale = torch.empty((s["rows"], n) if group else s["rows"], dtype=torch.float32, device="cuda")
    sg.sg_pack8(x, q, scale)
    return {"q": q, "scale": scale}


def _own_unpack(s):
    import extreme_label_sparse_gb300 as sg

    y = torch.empty(s["q"].shape, dtype=DTYPES[s["dtype"]], device="cuda")
    sg.sg_unpack8(s["q"], s["scale"], y)
    return y


def run(s):
    if s["op"] == "linear":
        return _own_linear(s) if own else _plain_linear(s)
    if s["op"] == "norm":
        if s["mode"] == "fwd":
            return _own_norm_fwd(s) if own else _plain_norm_fwd(s)
        return _own_norm_bwd(s) if own else _plain_norm_bwd(s)
    if s["op"] == "pack":
        if own:
            return _own_pack(s)
        q, scale = _plain_pack(s["x"], s["group"])
        return {"q": q, "scale": scale}
    if own:
        return _own_unpack(s)
    return _plain_unpack(s["q"], s["scale"], s["group"]).to(DTYPES[s["dtype"]])


# ---------------------------------------------------------------- work
def work(case):
    size = SIZES[case["dtype"]]
    if case["op"] == "linear":
        T, H, N = case["T"], case["H"], case["N"]
        held = (T + N) * H + 4 * (T * _groups(H, case["group"]) + N)
        if case["mode"] == "fwd":
            return {"bytes": held + T * N * size, "flops": 2 * T * N * H}
        return {"bytes": held + (T * N + (T + N) * H) * size, "flops": 4 * T * N * H}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] in ("pack", "unpack"):
        return {"bytes": n * (size + 1) + 4 * rows * _groups(cols, case["group"]), "flops": 2 * n}
    kept = 4 * rows * _groups(cols, GROUP)
    vecs = (3 if case["gate"] else 2) * cols
    if case["mode"] == "fwd":
        return {"bytes": 4 * n * size + 8 * rows + vecs * size + (n + kept if case["x8"] else 0), "flops": 9 * n}
    held = 2 * n + 2 * kept if case["x8"] else 2 * n * size
    return {"bytes": 4 * n * size + held + 8 * rows + vecs * (size + 4), "flops": 18 * n}


# ---------------------------------------------------------------- in 64 bits
def _values(q, scale, group):
    """What rows held in 8 bits stand for."""
    v = q.double()
    if not group:
        return v * scale.double().unsqueeze(1)
    for i in range(scale.shape[1]):
        v[:, i * group:(i + 1) * group] *= scale[:, i:i + 1].double()
    return v


def _tops(x, group):
    """The largest magnitude of each group of columns."""
    return torch.stack([c.abs().max(1).values for c in x.double().split(group or x.shape[1], 1)], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        W = _values(s["W8"], s["W_scale"], 0)
        if case["mode"] == "fwd":
            return torch.mm(_values(s["x8"], s["x_scale"], 0), W.transpose(0, 1))
        d = s["dout"].double()
        return {"dx": torch.mm(d, W), "dW": torch.mm(d.transpose(0, 1), _values(s["x8"], s["x_scale"], case["group"]))}
    if case["op"] == "pack":
        scale = _tops(s["x"], case["group"]) / 127
        return {"q": None, "scale": scale if case["group"] else scale[:, 0]}
    if case["op"] == "unpack":
        return _values(s["q"], s["scale"], case["group"])
    post, pre = s["post"].double(), s["pre"].double()
    gate = 1.0 if s["gate_w"] is None else s["gate_w"].double()
    if case["mode"] == "fwd":
        x = s["x"].double()
        rx = x.square().mean(1).add(EPS).rsqrt()
        total = s["residual"].double() * s["alpha"] + gate * (x * rx.unsqueeze(1) * post)
        # the second norm is defined on the sum as it is stored
        u = total.to(torch.float32).to(s["x"].dtype).double()
        ru = u.square().mean(1).add(EPS).rsqrt()
        out = {"u": total, "rstd_x": rx, "rstd_u": ru, "y": u * ru.unsqueeze(1) * pre}
        if case["x8"]:
            out["x8"], out["x_scale"] = None, _tops(s["x"], GROUP) / 127
        return out
    held = case["x8"]
    x = _values(s["x"], s["x_scale"], GROUP) if held else s["x"].double()
    u = _values(s["u"], s["u_scale"], GROUP) if held else s["u"].double()
    rx, ru, dy = s["rstd_x"].double().unsqueeze(1), s["rstd_u"].double().unsqueeze(1), s["dy"].double()
    du = dy.mul(pre).mul(ru) - u * ru**3 * (dy * pre * u).mean(1, keepdim=True) + s["du_in"].double()
    back = du * (post * gate)
    out = {"dresidual": du * s["alpha"], "dx": back * rx - x * rx**3 * (back * x).mean(1, keepdim=True),
           "dpre": (dy * u * ru).sum(0)}
    total = (du * x * rx).sum(0)
    out["dpost"] = total * gate
    if s["gate_w"] is not None:
        out["dgate"] = total * post
    return out
