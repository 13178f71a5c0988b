"""Blocks on 8-bit integers at sizes where a CTA has much to do: several units of
both products of the linear layer's backward pass, and many rows to a row group of
the norms.  Everything is compared, with 64-bit results worked out on the GPU."""
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import ALPHA, E, EPS, HALF, LEAST, TYPES, backward_inputs, rand, rand8, scales, weights
from test_linear8_turns import PATHS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def near(got, want, dtype, slack, what):
    """As test_gpu_blocks8.close, on the GPU."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), what
    err = (got - want).abs() - (HALF[dtype] * want.abs() * 1.001 + LEAST[dtype] + slack)
    assert float(err.max()) <= 0, (what, float(err.max()), divmod(int(err.argmax()), got.shape[-1]))


def values(q, scale):
    s = scale.double()
    return q.double() * (s[:, None] if s.dim() == 1 else s.repeat_interleave(128, 1)[:, :q.shape[1]])


# ---------------------------------------------------------------- linear layer
@pytest.mark.parametrize("dtype,group", [("bf16", 128), ("f16", 0)])
@pytest.mark.parametrize("T,H,N", [p[:3] for p in PATHS])
def test_linear_backward_of_several_units_to_a_cluster(T, H, N, dtype, group):
    """Bounds of single elements: those of test_gpu_blocks8 (the values' rounding,
    HALF of each term, 2^-16 for sums of 1024 terms in the tensor cores, fp32 sums of
    parts; fp16's smallest step).

    Of the root mean square: a rounding is off by an even spread of up to half a
    step, HALF / sqrt(3) of the bottom of the value's binade, and so by no more than
    that of the value.  Errors of independent terms add up as their squares do,
    so those of the values are HALF / sqrt(3) of the result, and its own as much
    again: sqrt(2 / 3) HALF = 0.817 HALF where there are many terms, whatever the
    values."""
    x8, W8, ws = rand8(T, H, 1, (-H) % 16), rand8(N, H, 2, (-H) % 16), scales(N, 4)
    xs = scales(T * -(-H // 128), 3).reshape(T, -1) if group else scales(T, 3)
    dout = rand(T, N, dtype, 5, (-N) % 8, std=0.1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for _ in range(2):
        dx, dW = (torch.full(s, float("nan"), dtype=TYPES[dtype], device="cuda") for s in ((T, H), (N, H)))
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
        got.append((dx, dW))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and int(status) == 0
    d = dout.double()
    for out, a, b, top, what in ((dx, d, values(W8, ws), ws, "dx"), (dW, d.t(), values(x8, xs), xs, "dW")):
        want, terms = a @ b, a.abs() @ b.abs()
        parts = (a.shape[1] / 1024 + 67) * 2.0 ** -24
        low = a.abs().sum(1, keepdim=True) * float(top.max()) * 127 * 2.0 ** -39 if dtype == "f16" else 0.0
        near(out, want, dtype, (HALF[dtype] + 2.0 ** -16 + parts) * terms + low, what)
        if a.shape[1] >= 64:
            rel = float((out.double() - want).norm() / want.norm())
            assert rel <= 0.82 * HALF[dtype], (what, rel / HALF[dtype])


# ---------------------------------------------------------------- norms around a block
# row groups of the forward and backward kernels on 152 SMs: 2432 of one warp, 1216
# of two, 608 of four, 304 of eight, 152 of more.  The forward kernel has up to four
# rows of a group under way, the backward kernel two batches of up to four: the rows
# below are more than twice that for each group, and a remainder.
FORWARD = [(21893, 256), (21893, 512), (10951, 768), (5479, 2048), (2743, 4096), (1375, 8192), (1375, 16384)]
FORWARD_ANY = [(21893, 255), (10951, 1001), (2743, 4001), (1375, 9001)]  # rows that start anywhere
BACKWARD = [(41349, 256), (20681, 512), (10343, 1024), (5175, 2048), (2591, 4096), (2591, 8192), (1211, 16384)]
BACKWARD_ANY = [(20001, 255), (10343, 500), (5175, 1001), (2591, 2001), (1300, 4001), (1300, 9001)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols,shift", [s + (0,) for s in FORWARD] + [s + (1,) for s in FORWARD_ANY])
def test_block_norm_forward_of_many_rows_to_a_group(rows, cols, shift, dtype):
    x, res = rand(rows, cols, dtype, 1, 8 - shift, shift), rand(rows, cols, dtype, 2, 8 - shift, shift, 2.0)
    post, gate, pre = weights(cols, dtype)
    n = -(-cols // 128)
    mats = {k: torch.empty((rows, cols), dtype=t, device="cuda") for k, t in
            (("u", x.dtype), ("y", x.dtype), ("y8", torch.int8), ("x8", torch.int8), ("u8", torch.int8))}
    vecs = {k: torch.full((rows,), float("nan"), device="cuda") for k in ("rstd_x", "rstd_u", "y8_scale")}
    groups = {k: torch.full((rows, n), float("nan"), device="cuda") for k in ("x_scale", "u_scale")}
    sg.sg_block_norm_fwd(x, post, pre, EPS, residual=res, gate=gate, residual_scale=ALPHA, **mats, **vecs, **groups)
    rx = (x.double().square().mean(1) + EPS).rsqrt()
    v = x.double() * rx[:, None] * post.double() * gate.double()
    near(vecs["rstd_x"][:, None], rx[:, None], "f32", E * rx[:, None], "rstd_x")
    near(mats["u"], v + ALPHA * res.double(), dtype, E * (v.abs() + (ALPHA * res.double()).abs()), "u")
    u = mats["u"].double()
    ru = (u.square().mean(1) + EPS).rsqrt()
    y = u * ru[:, None] * pre.double()
    near(vecs["rstd_u"][:, None], ru[:, None], "f32", E * ru[:, None], "rstd_u")
    near(mats["y"], y, dtype, E * y.abs(), "y")
    top, s = y.abs().amax(1), vecs["y8_scale"].double()
    assert bool(((s - top / 127).abs() <= 2 * E * top / 127).all())
    assert bool(((mats["y8"].double() * s[:, None] - y).abs() <= s[:, None] * (0.5 + 127 * 4 * E)).all())
    for k, m in (("x", x), ("u", mats["u"])):  # the operator of their own, whose tests are by the definition
        q, scale = torch.empty_like(mats["y8"]), torch.empty_like(groups["x_scale"])
        sg.sg_pack8(m, q, scale)
        assert torch.equal(mats[k + "8"], q) and torch.equal(groups[k + "_scale"], scale), k


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols,shift", [s + (0,) for s in BACKWARD] + [s + (1,) for s in BACKWARD_ANY])
def test_block_norm_backward_of_many_rows_to_a_group(rows, cols, shift, dtype, held):
    dy, u, x, us, xs, di, rx, ru = backward_inputs((rows, cols), dtype, 16 - shift, shift, held)
    post, gate, pre = weights(cols, dtype)
    dx, dres = (torch.full((rows, cols), float("nan"), dtype=dy.dtype, device="cuda") for _ in range(2))
    sums = {k: torch.full((cols,), float("nan"), device="cuda") for k in ("dpost", "dpre", "dgate")}
    sg.sg_block_norm_bwd(dy, u, x, post, pre, rx, ru, dx, dresidual=dres, gate=gate, residual_scale=ALPHA, du_in=di,
                         u_scale=us, x_scale=xs, **sums)
    post, gate, pre, rx, ru = (t.double() for t in (post, gate, pre, rx[:, None], ru[:, None]))
    m = (values(u, us) if held else u.double()).mul_(ru)
    h = (values(x, xs) if held else x.double()).mul_(rx)
    g = dy.double() * pre
    du = ru * (g - m * (g * m).mean(1, keepdim=True)) + di.double()
    terms = ru * (g.abs() + m.abs() * (g * m).abs().mean(1, keepdim=True)) + di.double().abs()
    near(dres, ALPHA * du, dtype, E * ALPHA * terms, "dresidual")
    # a thread adds its rows one after the other, then the parts are joined
    chain = (rows + 100) * 2.0 ** -24 + 2 * E
    near(sums["dpre"][None], (dy.double() * m).sum(0)[None], "f32", chain * (dy.double() * m).abs().sum(0)[None], "dpre")
    s, t = (du * h).sum(0)[None], (terms * h.abs()).sum(0)[None]
    near(sums["dpost"][None], gate * s, "f32", chain * gate.abs() * t, "dpost")
    near(sums["dgate"][None], post * s, "f32", chain * post.abs() * t, "dgate")
    del m, g
    k, kt = du * gate * post, terms * (gate * post).abs()
    near(dx, rx * (k - h * (k * h).mean(1, keepdim=True)), dtype,
         3 * E * rx * (kt + h.abs() * (kt * h.abs()).mean(1, keepdim=True)), "dx")


@pytest.mark.parametrize("rows,cols,shift", [(21893, 256, 0), (10951, 768, 0), (2743, 4096, 0), (611, 16384, 0), (10951, 1001, 1)])
def test_block_norm_over_its_inputs_with_many_rows_to_a_group(rows, cols, shift):
    """Rows on their way to the chip are others than those that are written."""
    x, res = rand(rows, cols, "bf16", 1, 8 - shift, shift), rand(rows, cols, "bf16", 2, 8 - shift, shift)
    w = weights(cols, "bf16")
    u, y, rx, ru = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def fwd(x, res, u, y):
        sg.sg_block_norm_fwd(x, w[0], w[2], EPS, residual=res, gate=w[1], residual_scale=ALPHA, u=u, y=y, rstd_x=rx, rstd_u=ru)

    fwd(x, res, u, y)
    for u_at, y_at in ((0, 1), (1, 0)):
        b = [x.clone(), res.clone()]
        fwd(b[0], b[1], b[u_at], b[y_at])
        assert torch.equal(b[u_at], u) and torch.equal(b[y_at], y)
    dx, dres = torch.empty_like(x), torch.empty_like(x)

    def bwd(b, dx, dres):
        sums = torch.empty((3, cols), device="cuda")
        sg.sg_block_norm_bwd(b["dy"], b["u"], b["x"], w[0], w[2], rx, ru, dx, dresidual=dres, gate=w[1], residual_scale=ALPHA,
                             du_in=b["di"], dpost=sums[0], dpre=sums[1], dgate=sums[2])
        return sums

    given = {"dy": y, "u": u, "x": x, "di": res}
    ref = bwd(given, dx, dres)
    for res_at, dx_at in (("dy", "di"), ("di", "dy"), ("u", "x")):
        b = {k: v.clone() for k, v in given.items()}
        assert torch.equal(bwd(b, b[dx_at], b[res_at]), ref)
        assert torch.equal(b[dx_at], dx) and torch.equal(b[res_at], dres)
