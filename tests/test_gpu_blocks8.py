"""8-bit rows, the norms around a block and the linear layer on 8-bit integers
against their 64-bit restatements.

Tolerances.  HALF is half a unit in the last place of the output type, relative
to the value (2^-8 for bf16, 2^-11 for f16, never below half its smallest step;
2^-24 for fp32).  Packing and unpacking are fp32 operations rounded as they are
defined: equal bits.  E = 1e-5 of the terms of a result is for arithmetic in 32
bits along a row: a lane adds at most 32 terms and the warps join in 10 steps, a
sum of squares is halved by the root, and 160 roundings of 2^-24 are 1e-5.  The
linear layer: see its tests.
"""
import numpy as np
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from oracle import blocks8 as orc

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
E = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(rows, cols, dtype, seed, pad=0, shift=0, std=1.0):
    """Normal values as a slice of a wider buffer: `pad` more columns a row,
    starting at element `shift`."""
    x = torch.randn((rows, cols + pad + shift), generator=gen(seed), device="cuda") * std
    return x.to(TYPES[dtype])[:, shift:shift + cols]


def rand8(rows, cols, seed, pad=0, shift=0):
    return torch.randint(-128, 128, (rows, cols + pad + shift), generator=gen(seed), device="cuda",
                         dtype=torch.int8)[:, shift:shift + cols]


def guarded(rows, cols, dtype, pad=5, shift=0):
    """(whole buffer, its part for the result): what lies around is checked
    with `untouched`."""
    whole = torch.full((rows + 1, cols + pad + shift), 77, dtype=dtype, device="cuda")
    return whole, whole[:rows, shift:shift + cols]


def untouched(whole, part):
    r, c = part.shape
    s = part.storage_offset()
    assert bool((whole[r:] == 77).all()) and bool((whole[:, s + c:] == 77).all()) and bool((whole[:, :s] == 77).all())


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def close(got, want, dtype, slack, what=""):
    got = f64(got)
    assert np.all(np.isfinite(got)), what
    err = np.abs(got - want) - (HALF[dtype] * np.abs(want) * 1.001 + LEAST[dtype] + slack)
    assert err.max() <= 0, (what, err.max(), np.unravel_index(err.argmax(), err.shape))


# ---------------------------------------------------------------- 8-bit rows
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 255), (9, 256), (17, 264), (4, 1001), (2, 4096), (130, 768), (3, 8200),
          (2, 20001), (2, 32768)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_pack_and_unpack(shape, dtype, pad, shift):
    rows, cols = shape
    x = rand(*shape, dtype, 1, pad, shift, 3.0)
    for group in (0, 128):
        whole, q = guarded(rows, cols, torch.int8, pad + (1 if shift else 8), shift)
        scale = torch.full((rows + 1, -(-cols // 128)) if group else (rows + 1,), 77.0, device="cuda")
        sg.sg_pack8(x, q, scale[:rows])
        want_q, want_s = orc.pack8(f32(x), group)
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(scale[:rows].cpu().numpy(), want_s)
        untouched(whole, q)
        assert bool((scale[rows:] == 77).all())
        back, y = guarded(rows, cols, x.dtype, pad + (1 if shift else 8), shift)
        sg.sg_unpack8(q, scale[:rows], y)
        s32 = np.repeat(want_s, 128, axis=1)[:, :cols] if group else want_s[:, None]
        assert torch.equal(y.cpu(), torch.from_numpy(want_q.astype(np.float32) * s32).to(x.dtype))
        untouched(back, y)


def test_unpack_of_every_byte():
    q = torch.arange(-128, 128, device="cuda").to(torch.int8).reshape(2, 128)
    y = torch.empty((2, 128), device="cuda")
    sg.sg_unpack8(q, torch.tensor([0.5, 2.0], device="cuda"), y)
    assert torch.equal(y, q.float() * torch.tensor([[0.5], [2.0]], device="cuda"))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_pack_of_extreme_values(dtype, shift):
    """Infinities and NaN cost their own group alone, the smallest and largest
    values and zeros keep theirs."""
    big, small = float(torch.finfo(TYPES[dtype]).max), float(torch.finfo(TYPES[dtype]).tiny)
    x = rand(12, 400, dtype, 3, shift=shift)
    x[0, 5] = float("inf")
    x[1, 130] = float("-inf")
    x[2, 399] = float("nan")
    x[3, :] = 0
    x[4, 128:256] = 0
    x[5, 7] = big
    x[6, 7] = -big
    x[7] *= small
    x[8, :] = 0
    x[8, 200] = small
    x[9, :] = -0.0
    for group in (0, 128):
        q = torch.empty((12, 400), dtype=torch.int8, device="cuda")
        scale = torch.empty((12, 4) if group else (12,), device="cuda")
        sg.sg_pack8(x, q, scale)
        want_q, want_s = orc.pack8(f32(x), group)
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(scale.cpu().numpy(), want_s, equal_nan=True)
        y = torch.empty((12, 400), device="cuda")
        sg.sg_unpack8(q, scale, y)
        bad = ~np.isfinite(f32(y))
        assert bad[0].sum() == (128 if group else 400) and bad[2].sum() == (16 if group else 400) and not bad[3:].any()


def test_pack_beyond_2_31_elements():
    """Offsets pass 32 bits: the last rows of a matrix of more than 2^31 elements."""
    rows, cols = (1 << 18) + 3, 8192 + 64
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(3, cols, "bf16", 4)
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    for group in (0, 128):
        scale = torch.empty((rows, -(-cols // 128)) if group else (rows,), device="cuda")
        sg.sg_pack8(x, q, scale)
        want_q, want_s = orc.pack8(f32(x[-3:]), group)
        assert np.array_equal(q[-3:].cpu().numpy(), want_q) and np.array_equal(scale[-3:].cpu().numpy(), want_s)
        assert not bool(q[:-3].any())
        y = x.fill_(1)
        sg.sg_unpack8(q, scale, y)
        got = f32(y[-3:])
        assert not bool(y[:-3].any()) and np.abs(got - orc.values8(want_q, want_s)).max() <= 2.0 ** -8 * np.abs(got).max()
        x.zero_()
        x[-3:] = rand(3, cols, "bf16", 4)


# ---------------------------------------------------------------- norms around a block
ALPHA, EPS = 1.25, 1e-5
NORM_SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 255), (70, 256), (17, 264), (9, 512), (4, 1001), (600, 1024),
               (700, 768), (3, 2048), (330, 4096), (5, 4104), (3, 8192), (2, 9001), (2, 16384)]


def weights(cols, dtype, gate=True):
    post, g, pre = (rand(1, cols, dtype, s, std=0.3)[0] + 1 for s in (11, 12, 13))
    return post, g if gate else None, pre


def block(x, res, post, gate, pre, pad, shift, held=True):
    """One forward call with every output, and checks of what lies around."""
    rows, cols = x.shape
    dt = x.dtype
    n = -(-cols // 128)
    mats = {k: guarded(rows, cols, t, pad + (1 if shift else 8), shift)
            for k, t in (("u", dt), ("y", dt), ("y8", torch.int8), ("x8", torch.int8), ("u8", torch.int8))}
    vecs = {k: torch.full((rows + 1,), 77.0, device="cuda") for k in ("rstd_x", "rstd_u", "y8_scale")}
    vecs.update({k: torch.full((rows + 1, n), 77.0, device="cuda") for k in ("x_scale", "u_scale")})
    if not held:
        for k in ("x8", "u8", "x_scale", "u_scale"):
            mats.pop(k, None)
            vecs.pop(k, None)
    sg.sg_block_norm_fwd(x, post, pre, EPS, residual=res, gate=gate, residual_scale=ALPHA,
                         **{k: v[1] for k, v in mats.items()}, **{k: v[:rows] for k, v in vecs.items()})
    for whole, part in mats.values():
        untouched(whole, part)
    assert all(bool((v[rows:] == 77).all()) for v in vecs.values())
    return {**{k: v[1] for k, v in mats.items()}, **{k: v[:rows] for k, v in vecs.items()}}


def check_block(x, res, post, gate, pre, dtype, out):
    w = [None if v is None else f64(v) for v in (post, gate, pre)]
    want_u, rx = orc.block_norm_u(f64(x), None if res is None else f64(res), w[0], w[1], ALPHA, EPS)
    v = want_u - (0 if res is None else ALPHA * f64(res))
    close(out["rstd_x"][:, None], rx[:, None], "f32", E * rx[:, None], "rstd_x")
    close(out["u"], want_u, dtype, E * (np.abs(v) + np.abs(want_u - v)), "u")
    # the second norm is that of u as it was stored
    u = f64(out["u"])
    ru = orc.rms(u, EPS)
    y = u * ru[:, None] * w[2]
    close(out["rstd_u"][:, None], ru[:, None], "f32", E * ru[:, None], "rstd_u")
    close(out["y"], y, dtype, E * np.abs(y), "y")
    top = np.abs(y).max(1)
    scale = f64(out["y8_scale"])
    assert np.all(np.abs(scale - top / 127) <= 2 * E * top / 127)
    # half a step, and fp32's errors of a value of up to 127 steps
    assert np.all(np.abs(f64(out["y8"]) * scale[:, None] - y) <= scale[:, None] * (0.5 + 127 * 4 * E))
    for k in ("x", "u"):
        q, s = orc.pack8(f32(x if k == "x" else out["u"]), 128)
        assert np.array_equal(out[k + "8"].cpu().numpy(), q) and np.array_equal(out[k + "_scale"].cpu().numpy(), s), k


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_block_norm_forward(shape, dtype, pad, shift):
    x = rand(*shape, dtype, 1, pad, shift)
    res = rand(*shape, dtype, 2, pad, shift, 2.0)
    w = weights(shape[1], dtype)
    check_block(x, res, *w, dtype, block(x, res, *w, pad, shift))


@pytest.mark.parametrize("shape", [(9, 264), (5, 1001), (40, 4096)], ids=str)
def test_block_norm_without_gate_or_residual(shape):
    x, res = rand(*shape, "bf16", 1), rand(*shape, "bf16", 2)
    for r, g in ((None, True), (res, False), (None, False)):
        w = weights(shape[1], "bf16", g)
        check_block(x, r, *w, "bf16", block(x, r, *w, 0, 0))


@pytest.mark.parametrize("shape", [(33, 264), (5, 1001)], ids=str)
def test_block_norm_outputs_over_inputs_and_single_outputs(shape):
    x, res = rand(*shape, "bf16", 1), rand(*shape, "bf16", 2)
    w = weights(shape[1], "bf16")
    ref = block(x, res, *w, 0, 0)
    for u_at, y_at in ((0, 1), (1, 0), (1, 1)):
        bufs = [x.clone(), res.clone()]
        u, y = bufs[u_at], bufs[y_at]
        kw = {} if u_at == y_at else {"u": u}
        sg.sg_block_norm_fwd(bufs[0], w[0], w[2], EPS, residual=bufs[1], gate=w[1], residual_scale=ALPHA, y=y, **kw)
        assert torch.equal(y, ref["y"]) and (u_at == y_at or torch.equal(u, ref["u"]))
    y8, s = torch.empty(shape, dtype=torch.int8, device="cuda"), torch.empty(shape[0], device="cuda")
    sg.sg_block_norm_fwd(x, w[0], w[2], EPS, residual=res, gate=w[1], residual_scale=ALPHA, y8=y8, y8_scale=s)
    assert torch.equal(y8, ref["y8"]) and torch.equal(s, ref["y8_scale"])


@pytest.mark.parametrize("cols", [264, 1001])
def test_block_norm_rows_that_are_not_finite(cols):
    """They are lost alone: NaN scales for their 8-bit rows, and the other rows
    as without them."""
    x, res = rand(7, cols, "bf16", 1), rand(7, cols, "bf16", 2)
    w = weights(cols, "bf16")
    ref = block(x, res, *w, 0, 0)
    x[1, 3], x[4, 200], res[5, cols - 1] = float("inf"), float("nan"), float("nan")
    out = block(x, res, *w, 0, 0)
    fine = [0, 2, 3, 6]
    for k, v in ref.items():
        assert torch.equal(out[k][fine], v[fine]), k
    # an infinity in x leaves rstd_x = 0, and 0 times infinity in its place
    assert bool(torch.isnan(out["y8_scale"][[1, 4, 5]]).all()) and not bool(out["y8"][[1, 4, 5]].any())
    assert bool(torch.isnan(out["x_scale"][1, 0])) and bool(torch.isnan(out["u_scale"][5, -1]))


def backward_inputs(shape, dtype, pad, shift, held):
    rows, cols = shape
    x, u = rand(*shape, dtype, 1, pad, shift), rand(*shape, dtype, 2, pad, shift, 2.0)
    dy, di = rand(*shape, dtype, 3, pad, shift), rand(*shape, dtype, 4, pad, shift)
    rx = torch.rsqrt(x.float().square().mean(1) + EPS)
    ru = torch.rsqrt(u.float().square().mean(1) + EPS)
    if not held:
        return dy, u, x, None, None, di, rx, ru
    n = -(-cols // 128)
    kept = []
    for v in (u, x):
        q = torch.empty((rows, cols + pad + shift), dtype=torch.int8, device="cuda")[:, shift:shift + cols]
        s = torch.empty((rows, n), device="cuda")
        sg.sg_pack8(v, q, s)
        kept.append((q, s))
    return dy, kept[0][0], kept[1][0], kept[0][1], kept[1][1], di, rx, ru


def check_backward(inputs, w, dtype, out, alpha=ALPHA):
    dy, u, x, us, xs, di, rx, ru = inputs
    u64 = f64(u) if us is None else orc.values8(u.cpu().numpy(), us.cpu().numpy())
    x64 = f64(x) if xs is None else orc.values8(x.cpu().numpy(), xs.cpu().numpy())
    post, gate, pre = (None if v is None else f64(v) for v in w)
    rx64, ru64 = f64(rx)[:, None], f64(ru)[:, None]
    want = orc.block_norm_grad(f64(dy), u64, x64, post, gate, pre, alpha, f64(rx), f64(ru), None if di is None else f64(di))
    g, m = np.abs(f64(dy) * pre), np.abs(u64 * ru64)
    terms = ru64 * (g + m * (g * m).mean(1, keepdims=True)) + (0 if di is None else np.abs(f64(di)))
    if "dresidual" in out:
        close(out["dresidual"], want["dresidual"], dtype, E * abs(alpha) * terms, "dresidual")
    gp = np.abs(post if gate is None else post * gate)
    h, k = np.abs(x64 * rx64), gp * terms
    close(out["dx"], want["dx"], dtype, 3 * E * rx64 * (k + h * (k * h).mean(1, keepdims=True)), "dx")
    # a thread adds its rows one after the other, then the parts are joined
    chain = (dy.shape[0] + 100) * 2.0 ** -24
    for name, t in (("dpre", (g / np.abs(pre) * m).sum(0)),
                    ("dpost", (terms * h).sum(0) * (1 if gate is None else np.abs(gate))),
                    ("dgate", (terms * h).sum(0) * np.abs(post))):
        if out.get(name) is not None:
            close(out[name][None], want[name][None], "f32", (chain + 2 * E) * t[None], name)


def backward(inputs, w, pad, shift, gate=True, alpha=ALPHA):
    dy, u, x, us, xs, di, rx, ru = inputs
    rows, cols = dy.shape
    mats = {k: guarded(rows, cols, dy.dtype, pad + (1 if shift else 8), shift) for k in ("dresidual", "dx")}
    vecs = {k: torch.full((cols + 1,), 77.0, device="cuda") for k in ("dpost", "dpre") + (("dgate",) if gate else ())}
    sg.sg_block_norm_bwd(dy, u, x, w[0], w[2], rx, ru, gate=w[1], residual_scale=alpha, du_in=di, u_scale=us, x_scale=xs,
                         **{k: v[1] for k, v in mats.items()}, **{k: v[:cols] for k, v in vecs.items()})
    for whole, part in mats.values():
        untouched(whole, part)
    assert all(float(v[cols]) == 77 for v in vecs.values())
    return {**{k: v[1] for k, v in mats.items()}, **{k: v[:cols] for k, v in vecs.items()}}


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_block_norm_backward(shape, dtype, pad, shift, held):
    inputs = backward_inputs(shape, dtype, pad, shift, held)
    w = weights(shape[1], dtype)
    check_backward(inputs, w, dtype, backward(inputs, w, pad, shift))


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("shape", [(9, 264), (5, 1001)], ids=str)
def test_block_norm_backward_without_some(shape, held):
    """No gate, no du_in, no sums, no dresidual, and outputs over inputs."""
    inputs = list(backward_inputs(shape, "bf16", 0, 0, held))
    inputs[5] = None
    w = weights(shape[1], "bf16", False)
    ref = backward(inputs, w, 0, 0, gate=False)
    check_backward(inputs, w, "bf16", ref)
    dy, u, x, us, xs, di, rx, ru = inputs
    dx = torch.empty_like(dy)
    sg.sg_block_norm_bwd(dy, u, x, w[0], w[2], rx, ru, dx, residual_scale=ALPHA, u_scale=us, x_scale=xs)
    assert torch.equal(dx, ref["dx"])
    over = [("dy", "du_in"), ("du_in", "dy")] + ([] if held else [("u", "x")])
    di = rand(*shape, "bf16", 4)
    inputs[5] = di
    ref = backward(inputs, w, 0, 0, gate=False)
    for res_at, dx_at in over:
        b = {"dy": dy.clone(), "du_in": di.clone(), "u": u.clone(), "x": x.clone()}
        sg.sg_block_norm_bwd(b["dy"], b["u"], b["x"], w[0], w[2], rx, ru, b[dx_at], dresidual=b[res_at],
                             residual_scale=ALPHA, du_in=b["du_in"], u_scale=us, x_scale=xs)
        assert torch.equal(b[res_at], ref["dresidual"]) and torch.equal(b[dx_at], ref["dx"])


def test_block_norm_backward_of_small_and_large_rows():
    """Rows of any scale that fp32 holds: the gradient's parts do not overflow
    or vanish on their way."""
    shape = (6, 512)
    inputs = list(backward_inputs(shape, "f32", 0, 0, False))
    # the first rows' x, the others' u (and with it the size of du)
    size = torch.tensor([1e-30, 1e-20, 1e15, 1e-20, 1e15, 1e30], device="cuda")[:, None]
    first = torch.tensor([1, 1, 1, 0, 0, 0], device="cuda")[:, None] == 1
    for at, r, rows in ((2, 6, first), (1, 7, ~first)):
        inputs[at] = torch.where(rows, inputs[at] * size, inputs[at])
        inputs[r] = torch.rsqrt(inputs[at].double().square().mean(1)).float()
    inputs[5] = torch.where(first, inputs[5], inputs[5] / size)
    w = weights(512, "f32")
    out = backward(inputs, w, 0, 0)
    want = orc.block_norm_grad(f64(inputs[0]), f64(inputs[1]), f64(inputs[2]), *(f64(v) for v in w), ALPHA, f64(inputs[6]),
                               f64(inputs[7]), f64(inputs[5]))
    for k in ("dresidual", "dx"):
        top = np.abs(want[k]).max(1, keepdims=True)
        assert np.isfinite(f64(out[k])).all() and (np.abs(f64(out[k]) - want[k]) <= 20 * E * top).all(), k


def test_block_norm_without_rows():
    w = weights(64, "bf16")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    r = torch.empty(0, device="cuda")
    sg.sg_block_norm_fwd(x, w[0], w[2], EPS, y=torch.empty_like(x))
    sums = {k: torch.full((64,), 5.0, device="cuda") for k in ("dpost", "dgate", "dpre")}
    sg.sg_block_norm_bwd(x, x, x, w[0], w[2], r, r, torch.empty_like(x), gate=w[1], **sums)
    assert not any(bool(v.any()) for v in sums.values())


def test_block_norm_many_rows_are_the_same_bits_each_time():
    shape = (5000, 1024)
    inputs = backward_inputs(shape, "bf16", 0, 0, True)
    w = weights(1024, "bf16")
    a, b = backward(inputs, w, 0, 0), backward(inputs, w, 0, 0)
    assert all(torch.equal(a[k], b[k]) for k in a)
    check_backward(inputs, w, "bf16", a)


# ---------------------------------------------------------------- linear layer
# Forward: sums of 1024 products of integers are exact, and those are added in
# fp32, one rounding each, which a part of a split sum adds once more; then two
# products with the scales.  So at most (H / 1024 + 64 + 3) 2^-24 of the terms,
# and the output's rounding (exact below 2^24 in all, which random values are).
# Backward: the values enter the products rounded to the type (HALF of each
# term), sums of 1024 terms are rounded toward zero by the tensor cores (64 steps
# of 16 terms, 2^-23 each: below 2^-16 of the terms), parts are added in fp32.
LINEAR = [(1, 1, 1), (1, 3, 5), (1, 16, 16), (1, 768, 3000), (2, 64, 128), (3, 100, 7), (7, 1001, 129), (8, 128, 1000),
          (16, 2048, 515), (17, 4096, 260), (31, 130, 96), (33, 64, 1), (48, 1500, 1000), (64, 2064, 256),
          (65, 100, 300), (100, 768, 1000), (127, 5000, 33), (128, 96, 513), (129, 256, 256), (200, 1001, 1003),
          (256, 8200, 130), (300, 64, 3000), (385, 4096, 700), (512, 300, 1000), (777, 1000, 500), (1030, 2000, 260), (2100, 520, 72)]


def scales(n, seed):
    return torch.rand(n, generator=gen(seed), device="cuda") * 0.02 + 1e-4


def check_forward(x8, xs, W8, ws, out, dtype):
    x, W = x8.double(), W8.double()
    want = f64((x @ W.t()) * xs.double()[:, None] * ws.double())
    terms = f64((x.abs() @ W.abs().t()) * xs.double()[:, None] * ws.double())
    close(out, want, dtype, (x8.shape[1] / 1024 + 67) * 2.0 ** -24 * terms, "out")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,H,N", LINEAR)
def test_linear_forward(T, H, N, dtype):
    # rows that start on 16 bytes, and rows that start anywhere
    for pad, shift in (((-H) % 16, 0), (3, 1)):
        x8, W8 = rand8(T, H, 1, pad, shift), rand8(N, H, 2, pad, shift)
        xs, ws = scales(T, 3), scales(N, 4)
        whole, out = guarded(T, N, TYPES[dtype], (-N) % 8 + 8 if not shift else 3, shift)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sg.sg_linear8_fwd(x8, xs, W8, ws, out, status=status)
        check_forward(x8, xs, W8, ws, out, dtype)
        untouched(whole, out)
        assert int(status) == 0


@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_forward_of_extreme_integers(T):
    """All -128 or 127, whose sums of 1024 are as large as they can be: equal
    to the integers where those are below 2^24, rounded to fp32 beyond."""
    for H in (1024, 1023, 5000):
        x8 = torch.full((T, H), -128, dtype=torch.int8, device="cuda")
        W8 = torch.full((260, H), -128, dtype=torch.int8, device="cuda")
        W8[1::2] = 127
        x8[1::2] = 127
        out = torch.empty((T, 260), device="cuda")
        sg.sg_linear8_fwd(x8, torch.ones(T, device="cuda"), W8, torch.ones(260, device="cuda"), out)
        want = x8.double() @ W8.double().t()
        if H <= 1024:
            assert torch.equal(out.double(), want)
        else:
            assert bool(((out.double() - want).abs() <= 5 * 2.0 ** -24 * want.abs()).all())


def test_linear_forward_of_integers_is_exact():
    """Random integers: sums below 2^24, so the result is the integer."""
    for T, H, N in ((5, 4096, 700), (50, 3000, 300), (400, 4096, 300)):
        x8, W8 = rand8(T, H, 5), rand8(N, H, 6)
        out = torch.empty((T, N), device="cuda")
        sg.sg_linear8_fwd(x8, torch.ones(T, device="cuda"), W8, torch.ones(N, device="cuda"), out)
        assert torch.equal(out.double(), x8.double() @ W8.double().t())


@pytest.mark.parametrize("T", [1, 33, 300])
def test_linear_scales_that_are_nan_or_zero(T):
    x8, W8 = rand8(T, 200, 1), rand8(300, 200, 2)
    xs, ws = scales(T, 3), scales(300, 4)
    ws[7], ws[299], ws[8] = float("nan"), 0.0, 0.0
    out = torch.empty((T, 300), device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out)
    assert bool(torch.isnan(out[:, 7]).all()) and not bool(out[:, [8, 299]].any())
    assert bool(torch.isfinite(out[:, torch.arange(300, device="cuda") != 7]).all())
    xs[T - 1] = float("nan")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out)
    assert bool(torch.isnan(out[T - 1]).all())


def check_gradients(x8, xs, W8, ws, dout, dx, dW, dtype):
    d = dout.double()
    W = torch.from_numpy(orc.values8(W8.cpu().numpy(), ws.cpu().numpy())).cuda()
    x = torch.from_numpy(orc.values8(x8.cpu().numpy(), xs.cpu().numpy())).cuda()
    for got, a, b, what in ((dx, d, W, "dx"), (dW, d.t(), x, "dW")):
        if got is None:
            continue
        want, terms = f64(a @ b), f64(a.abs() @ b.abs())
        parts = (a.shape[1] / 1024 + 67) * 2.0 ** -24
        # fp16's smallest step is 2^-24, half of it 2^-40 of the largest value
        # that 8 bits may stand for (its scale is brought to at least 2^8)
        top = float((ws if what == "dx" else xs).max()) * 127
        low = f64(a.abs().sum(1, keepdim=True)) * top * 2.0 ** -39 if dtype == "f16" else 0.0
        close(got, want, dtype, (HALF[dtype] + 2.0 ** -16 + parts) * terms + low, what)
        # roundings of independent terms add up as squares do: as many as the
        # result has, so 1.5 times its own rounding where there are many
        if got.numel() >= 1000 and a.shape[1] >= 64 and np.abs(want).max() > 1e-3:
            rel = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
            assert rel <= 1.5 * HALF[dtype], (what, rel)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,N", LINEAR)
def test_linear_backward(T, H, N, dtype, group):
    for pad, shift in (((-H) % 16, 0), (3, 1)):
        x8, W8 = rand8(T, H, 1, pad, shift), rand8(N, H, 2, pad, shift)
        ws = scales(N, 4)
        xs = scales(T * -(-H // 128), 3).reshape(T, -1) if group else scales(T, 3)
        dout = rand(T, N, dtype, 5, (-N) % 8 if not shift else 3, shift)
        wx, dx = guarded(T, H, TYPES[dtype], (-H) % 8 + 8 if not shift else 3, shift)
        ww, dW = guarded(N, H, TYPES[dtype], (-H) % 8 + 8 if not shift else 3, shift)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
        check_gradients(x8, xs, W8, ws, dout, dx, dW, dtype)
        untouched(wx, dx)
        untouched(ww, dW)
        assert int(status) == 0


@pytest.mark.parametrize("T,H,N", [(40, 300, 500), (300, 520, 1000)])
def test_linear_backward_of_one_gradient(T, H, N):
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    dout = rand(T, N, "bf16", 5)
    dx, dW = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((T, H), (N, H)))
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx)
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dW=dW)
    check_gradients(x8, xs, W8, ws, dout, dx, dW, "bf16")


@pytest.mark.parametrize("T,H,N", [
    (200, 1500, 3000),   # dx in parts, first
    (64, 2048, 4096),    # dW first, of which each cluster has some
    (600, 2048, 2200),   # pairs of CTAs, dx first
    (1100, 1000, 1200),
    (128, 1024, 4864),   # 152 tiles of dW, as many as clusters
    (3000, 300, 700),    # dW in parts
])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_backward_units_of_both_products(T, H, N, dtype):
    """Every tile of either product is computed, by the cluster whose turn it is;
    outputs that held NaN before."""
    x8, W8, xs, ws = rand8(T, H, 1, (-H) % 16), rand8(N, H, 2, (-H) % 16), scales(T, 3), scales(N, 4)
    dout = rand(T, N, dtype, 5, (-N) % 8)
    dx, dW = (torch.full(s, float("nan"), dtype=TYPES[dtype], device="cuda") for s in ((T, H), (N, H)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, status=status)
    check_gradients(x8, xs, W8, ws, dout, dx, dW, dtype)
    assert int(status) == 0


@pytest.mark.parametrize("T", [50, 300])
def test_linear_backward_f16_of_small_and_uneven_scales(T):
    """fp16's range is that of the scales' ratios, not of the scales."""
    x8, W8 = rand8(T, 200, 1), rand8(300, 200, 2)
    for size, std in ((1e-9, 1e4), (1e-4, 1.0), (1e3, 1e-3)):
        xs, ws = scales(T, 3) * size, scales(300, 4) * size
        ws[::3] *= 2.0 ** -12
        dout = rand(T, 300, "f16", 5, std=std)
        dx, dW = (torch.empty(s, dtype=torch.float16, device="cuda") for s in ((T, 200), (300, 200)))
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW)
        check_gradients(x8, xs, W8, ws, dout, dx, dW, "f16")


def test_linear_backward_of_many_tokens_of_one_sign():
    """Terms of one sign: parts of 1024 are added in fp32, so that the tensor
    cores' rounding toward zero does not grow with their number."""
    T = 40000
    x8 = torch.full((T, 128), 100, dtype=torch.int8, device="cuda")
    W8 = rand8(256, 128, 2)
    dout = (rand(T, 256, "f16", 5).float().abs() * 1e-3).half()
    dW = torch.empty((256, 128), dtype=torch.float16, device="cuda")
    sg.sg_linear8_bwd(x8, torch.full((T,), 0.01, device="cuda"), W8, scales(256, 4), dout, dW=dW)
    want = f64(dout.double().sum(0))[:, None] * 100 * float(np.float32(0.01))
    # the common scale's value in fp16 is off by the same half step for all; the
    # rest is that of sums of 1024 terms
    assert (np.abs(f64(dW) - want) <= (2 * HALF["f16"] + 2.0 ** -16) * want).all()


def test_two_graphs_that_share_work_memory_in_turn():
    """Its contents need not survive between calls: two captured calls of other
    sizes and types over the same memory, replayed one after the other."""
    calls = []
    for T, H, N, dtype in ((300, 512, 700, "bf16"), (40, 4096, 500, "f16"), (700, 300, 900, "f16")):
        x8, W8, xs, ws = rand8(T, H, T, (-H) % 16), rand8(N, H, 2, (-H) % 16), scales(T, 3), scales(N, 4)
        dout = rand(T, N, dtype, 5)
        outs = [torch.empty(s, dtype=TYPES[dtype], device="cuda") for s in ((T, N), (T, H), (N, H))]
        calls.append((x8, xs, W8, ws, dout, outs, max(sg.sg_linear8_work(x8, W8), sg.sg_linear8_work(x8, W8, dout))))
    work = torch.empty(max(c[6] for c in calls), dtype=torch.uint8, device="cuda")

    def run(c):
        x8, xs, W8, ws, dout, (out, dx, dW), _ = c
        sg.sg_linear8_fwd(x8, xs, W8, ws, out, work=work)
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, work=work)

    ref = []
    for c in calls:
        run(c)
        ref.append([t.clone() for t in c[5]])
    graphs = []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            run(c)
        graphs.append(g)
    for i in (0, 1, 2, 1, 0, 2, 2, 0, 1):
        for t in calls[i][5]:
            t.zero_()
        work.fill_(255)
        graphs[i].replay()
        assert all(torch.equal(a, b) for a, b in zip(calls[i][5], ref[i])), i


def test_linear_without_tokens():
    x8, W8 = rand8(0, 64, 1), rand8(30, 64, 2)
    xs, ws = scales(0, 3), scales(30, 4)
    sg.sg_linear8_fwd(x8, xs, W8, ws, torch.empty((0, 30), device="cuda"))
    whole, dW = guarded(30, 64, torch.bfloat16)
    sg.sg_linear8_bwd(x8, xs, W8, ws, torch.empty((0, 30), dtype=torch.bfloat16, device="cuda"),
                      dx=torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), dW=dW)
    assert not bool(dW.any())
    untouched(whole, dW)


@pytest.mark.parametrize("T", [1, 4, 40, 128, 200, 600])
def test_linear_work_memory_may_hold_anything(T):
    x8, W8, xs, ws = rand8(T, 1000, 1, 8), rand8(900, 1000, 2, 8), scales(T, 3), scales(900, 4)
    dout = rand(T, 900, "bf16", 5, 4)
    out = torch.empty((T, 900), device="cuda")
    dx, dW = (torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in ((T, 1000), (900, 1000)))
    got = []
    for fill in (0, 255):
        work = [torch.full((n,), fill, dtype=torch.uint8, device="cuda")
                for n in (sg.sg_linear8_work(x8, W8), sg.sg_linear8_work(x8, W8, dout))]
        sg.sg_linear8_fwd(x8, xs, W8, ws, out, work=work[0])
        sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, work=work[1])
        got.append([t.clone() for t in (out, dx, dW)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("T,H,N", [(600, 4096, 40000), (2, 4099, 70000), (7, 4099, 70000), (100, 4099, 70000)])
def test_linear_channels_in_pieces(T, H, N):
    """More weights than one piece of work memory holds: 256 MB in 16 bits, or of
    rows that do not start on 16 bytes in 8."""
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    out = torch.empty((T, N), device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out)
    at = torch.cat([torch.arange(0, 40), torch.arange(32700, 32800), torch.arange(65200, 65400) % N,
                    torch.arange(N - 40, N)]).cuda()
    check_forward(x8, xs, W8[at], ws[at], out[:, at], "f32")


# ---------------------------------------------------------------- together
def train_step(x, res, w, W8, ws, dz, di):
    """A block's end and the next one's first layer, forward and back, from
    what is kept in 8 bits."""
    rows, cols = x.shape
    N, n = W8.shape[0], -(-cols // 128)
    i8, f = torch.int8, torch.float32
    new = lambda *s, dtype=f: torch.empty(s, dtype=dtype, device=x.device)  # noqa: E731
    u, y8, x8, u8 = new(rows, cols, dtype=x.dtype), *(new(rows, cols, dtype=i8) for _ in range(3))
    rx, ru, ys, x_s, u_s = new(rows), new(rows), new(rows), new(rows, n), new(rows, n)
    z, dy, dW = new(rows, N, dtype=x.dtype), new(rows, cols, dtype=x.dtype), new(N, cols, dtype=x.dtype)
    dx, dres, dpost, dgate, dpre = (*(new(rows, cols, dtype=x.dtype) for _ in range(2)), *(new(cols) for _ in range(3)))
    sg.sg_block_norm_fwd(x, w[0], w[2], EPS, residual=res, gate=w[1], residual_scale=ALPHA, u=u, rstd_x=rx, rstd_u=ru,
                         y8=y8, y8_scale=ys, x8=x8, x_scale=x_s, u8=u8, u_scale=u_s)
    sg.sg_linear8_fwd(y8, ys, W8, ws, z)
    sg.sg_linear8_bwd(y8, ys, W8, ws, dz, dx=dy, dW=dW)
    sg.sg_block_norm_bwd(dy, u8, x8, w[0], w[2], rx, ru, dx, dresidual=dres, dpost=dpost, dpre=dpre, dgate=dgate,
                         gate=w[1], residual_scale=ALPHA, du_in=di, u_scale=u_s, x_scale=x_s)
    return {"u": u, "z": z, "dW": dW, "dx": dx, "dres": dres, "dpost": dpost, "dgate": dgate, "dpre": dpre}


def step_inputs(rows, cols, N, seed=0, device="cuda"):
    x, res = rand(rows, cols, "bf16", seed + 1), rand(rows, cols, "bf16", seed + 2, std=2.0)
    w = weights(cols, "bf16")
    master = rand(N, cols, "bf16", seed + 3, std=cols ** -0.5)
    W8, ws = torch.empty((N, cols), dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    sg.sg_pack8(master, W8, ws)
    return [x, res, w, W8, ws, rand(rows, N, "bf16", seed + 4, std=0.1), rand(rows, cols, "bf16", seed + 5)], master


@pytest.mark.parametrize("rows,cols,N", [(3, 256, 500), (100, 520, 1000), (400, 768, 2000)])
def test_a_training_step_from_8_bit_rows_is_near_the_one_in_64_bits(rows, cols, N):
    """Eight bits are off by half of 1 / 127 of a group's largest value, which
    for normal values of 128 to 768 columns (largest 2.5 to 4 sigma) is a root
    mean square of 4 / 127 / sqrt(12) = 0.9 % of the values at most.  Results
    take that from two roundings each at most (x and u, y and W), du and dx through
    two factors of the row: 4 % with room."""
    args, master = step_inputs(rows, cols, N)
    got = train_step(*args)
    x, res, w, _, _, dz, di = args
    post, gate, pre = (f64(v) for v in w)
    u, rx = orc.block_norm_u(f64(x), f64(res), post, gate, ALPHA, EPS)
    ru = orc.rms(u, EPS)
    y = u * ru[:, None] * pre
    W = f64(master)
    dy = f64(dz) @ W
    want = orc.block_norm_grad(dy, u, f64(x), post, gate, pre, ALPHA, rx, ru, f64(di))
    want.update(u=u, z=y @ W.T, dW=f64(dz).T @ y, dres=want["dresidual"])
    for k, v in got.items():
        rel = np.linalg.norm(f64(v) - want[k]) / np.linalg.norm(want[k])
        assert rel <= 0.04, (k, rel)


@pytest.mark.parametrize("rows", [1, 20, 100, 300, 600])
def test_a_step_captured_and_replayed_with_other_inputs(rows):
    args, _ = step_inputs(rows, 512, 600)
    other, _ = step_inputs(rows, 512, 600, 50)
    eager = train_step(*other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train_step(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = train_step(*args)
    torch.cuda.current_stream().wait_stream(side)
    for i in (0, 1, 3, 4, 5, 6):
        args[i].copy_(other[i])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], eager[k]) for k in eager)


@pytest.mark.parametrize("rows", [4, 60, 300, 600])
def test_steps_on_two_streams_at_once(rows):
    sets = [step_inputs(rows, 512, 1500, s)[0] for s in (0, 50)]
    ref = [train_step(*a) for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i] = train_step(*sets[i])
    torch.cuda.synchronize()
    assert all(torch.equal(outs[i][k], ref[i][k]) for i in (0, 1) for k in ref[i])
    assert sg.sg_linear8_status() == 0 and sg.sg_device_status() == 0


def test_binding_refuses_what_the_library_cannot_see():
    x = rand(4, 256, "bf16", 1)
    q, s = torch.empty((4, 256), dtype=torch.int8, device="cuda"), torch.empty((4, 2), device="cuda")
    for bad in (lambda: sg.sg_pack8(x, q, torch.empty((4, 3), device="cuda")),
                lambda: sg.sg_pack8(x, q, torch.empty(5, device="cuda")),
                lambda: sg.sg_pack8(x, q[:3], s), lambda: sg.sg_pack8(x.t(), q, s),
                lambda: sg.sg_pack8(x, q, torch.empty((2, 4), device="cuda").t()),
                lambda: sg.sg_unpack8(q.cpu(), s, x),
                lambda: sg.sg_linear8_fwd(q, s, q, torch.empty(4, device="cuda"), torch.empty((4, 4), device="cuda")),
                lambda: sg.sg_linear8_fwd(q, s[:, 0], q, s[:, 1], torch.empty((4, 4), device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(TypeError):
        sg.sg_pack8(x, q.to(torch.uint8), s)
    r = torch.ones(4, device="cuda")
    w = x[0]
    with pytest.raises(TypeError):  # x in 8 bits, u not
        sg.sg_block_norm_bwd(x, x, q, w, w, r, r, x.clone(), x_scale=s)
    with pytest.raises(sg.SGError):  # both in 8 bits, one without scales
        sg.sg_block_norm_bwd(x, q, q, w, w, r, r, x.clone(), x_scale=s)
    with pytest.raises(ValueError):  # one scale for a row
        sg.sg_block_norm_bwd(x, q, q, w, w, r, r, x.clone(), x_scale=r, u_scale=r)


@pytest.mark.parametrize("T", [16, 33, 48, 64, 100, 300])
def test_linear_of_many_channels_again_and_again(T):
    """W from memory rather than the L2 cache, whose loads complete out of
    order: each launch gives the same result."""
    H, N = 2048, 90000
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    out = torch.empty((T, N), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out, status=status)
    at = torch.randint(0, N, (200,), generator=gen(7), device="cuda")
    check_forward(x8, xs, W8[at], ws[at], out[:, at], "f32")
    first = out.clone()
    for _ in range(60):
        sg.sg_linear8_fwd(x8, xs, W8, ws, out.zero_(), status=status)
        assert torch.equal(out, first)
    assert int(status) == 0


@pytest.mark.parametrize("T", [2, 20, 100, 200, 520])
def test_linear_weights_beyond_2_31_bytes(T):
    """Offsets pass 32 bits: the last channels of 2.2e9 weights."""
    H, N = 2048, (1 << 20) + 40001
    x8, xs = rand8(T, H, 1), scales(T, 3)
    W8 = torch.zeros((N, H), dtype=torch.int8, device="cuda")
    at = torch.tensor([0, 5, N // 2, N - 300, N - 2, N - 1], device="cuda")
    W8[at] = rand8(6, H, 2)
    ws = scales(N, 4)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out)
    check_forward(x8, xs, W8[at], ws[at], out[:, at], "bf16")
    out[:, at] = 0
    assert not bool(out.any())


def test_linear_output_beyond_2_31_elements():
    T, H, N = 140, 64, (1 << 24) - 5
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    sg.sg_linear8_fwd(x8, xs, W8, ws, out)
    at = torch.cat([torch.randint(0, N, (300,), generator=gen(7), device="cuda"), torch.arange(N - 3, N, device="cuda")])
    check_forward(x8, xs, W8[at], ws[at], out[:, at], "bf16")


def test_block_norm_beyond_2_31_elements():
    rows, cols = (1 << 17) + 300, 16384
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(3, cols, "bf16", 1)
    w = weights(cols, "bf16")
    y, x8 = torch.empty_like(x), torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    s, rx, ru = torch.empty((rows, 128), device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    u = torch.empty_like(x)
    sg.sg_block_norm_fwd(x, w[0], w[2], EPS, gate=w[1], u=u, rstd_x=rx, rstd_u=ru, y=y, x8=x8, x_scale=s)
    want = block(x[-3:].contiguous(), None, *w, 0, 0)
    assert all(torch.equal(a[-3:], want[k]) for a, k in ((u, "u"), (y, "y"), (x8, "x8"), (s, "x_scale"), (rx, "rstd_x")))
    assert not bool(y[:-3].any()) and not bool(x8[:-3].any())
    dx, dres = y, torch.empty_like(x)
    dpre = torch.empty(cols, device="cuda")
    sg.sg_block_norm_bwd(x, u, x, w[0], w[2], rx, ru, dx, dresidual=dres, gate=w[1], dpre=dpre)
    last = [t[-3:].contiguous() for t in (x, u, x)] + [None, None, None, rx[-3:].contiguous(), ru[-3:].contiguous()]
    check_backward(last, w, "bf16", {"dx": dx[-3:], "dresidual": dres[-3:], "dpre": dpre}, alpha=1.0)
    assert not bool(dres[:-3].any()) and not bool(dx[:-3].any())
