"""Dropout and residual RMS norm against their 64-bit restatements.

Tolerances: half a unit in the last place of the output type (at most 2^-8 of
the value for the 8 significant bits of bf16, 2^-11 for the 11 of f16 and never
below half its smallest step, 2^-24 for fp32); on top, 1e-5 of the terms
summed, for arithmetic in 32 bits (a lane adds at most 32 terms of a row, and
160 * 2^-24 is 1e-5).
Dropout itself and u are a product and a sum in fp32 rounded once: equal bits.
"""
import numpy as np
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from oracle import rows as orc

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
LEAST = {"bf16": 0.0, "f16": 2.0 ** -25, "f32": 0.0}
SEED, OFFSET = 0x1234567890ABCDEF, 0x0000000700000003


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def rand(rows, cols, dtype, seed, pad=0, shift=0, std=1.0):
    """Normal values as a slice of a wider buffer: `pad` more columns a row,
    starting at element `shift`."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((rows, cols + pad + shift), generator=g, device="cuda") * std
    return x.to(TYPES[dtype])[:, shift:shift + cols]


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def f32(t):
    return t.detach().float().cpu().numpy()


def close(got, want, dtype, slack):
    got = f64(got)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want) - (HALF_ULP[dtype] * np.abs(want) * 1.001 + LEAST[dtype] + 1e-5 * slack)
    assert err.max() <= 0, (err.max(), np.unravel_index(err.argmax(), err.shape))


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 255), (9, 256), (17, 264), (4, 1001), (2, 4096), (130, 768)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 0), (3, 1)])
def test_dropout(shape, dtype, pad, shift):
    x = rand(*shape, dtype, 1, pad, shift)
    out = torch.full((shape[0], shape[1] + 5), 7.0, dtype=x.dtype, device="cuda")
    y = out[:, :shape[1]]
    for p in (0.0, 0.1, 0.5, 1.0):
        sg.sg_dropout(x, p, SEED, OFFSET, y)
        want = torch.from_numpy(orc.dropout(f32(x), p, SEED, OFFSET)).to(x.dtype)
        assert torch.equal(y.cpu(), want)
        assert bool((out[:, shape[1]:] == 7.0).all())


def test_dropout_in_place_and_what_a_dropped_element_holds():
    x = rand(64, 512, "bf16", 2)
    keep = torch.from_numpy(orc.dropout_keep(64, 512, 0.5, 5, 6)).cuda()
    x = torch.where(keep, x, torch.tensor(float("nan"), dtype=x.dtype, device="cuda"))
    want = torch.from_numpy(orc.dropout(f32(torch.nan_to_num(x)), 0.5, 5, 6)).bfloat16()
    sg.sg_dropout(x, 0.5, 5, 6, x)
    assert torch.equal(x.cpu(), want)


def test_dropout_masks_differ_by_seed_and_offset():
    x = torch.ones((128, 1024), dtype=torch.bfloat16, device="cuda")
    got = []
    for seed, offset in ((1, 1), (2, 1), (1, 2), (1 + 2 ** 32, 1), (1, 1 + 2 ** 32)):
        y = torch.empty_like(x)
        sg.sg_dropout(x, 0.5, seed, offset, y)
        got.append(y != 0)
    for i in range(len(got)):
        for j in range(i):
            assert 0.45 < float((got[i] == got[j]).float().mean()) < 0.55


def fwd_inputs(shape, dtype, pad, shift):
    x, res = rand(*shape, dtype, 1, pad, shift), rand(*shape, dtype, 2, pad, 0, 2.0)
    w = (1 + 0.2 * rand(1, shape[1], "f32", 3)).to(TYPES[dtype]).reshape(-1)
    return x, res, w


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES + [(3, 16384), (2, 20001), (2, 32768)], ids=str)
@pytest.mark.parametrize("pad,shift,p", [(0, 0, 0.0), (8, 0, 0.3), (3, 1, 0.3)])
def test_norm_forward(shape, dtype, pad, shift, p):
    x, res, w = fwd_inputs(shape, dtype, pad, shift)
    u, y = torch.empty_like(res), torch.empty(shape, dtype=x.dtype, device="cuda")
    rstd, scale = (torch.empty(shape[0], device="cuda") for _ in range(2))
    y8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    sg.sg_add_rmsnorm_fwd(x, w, 1e-5, residual=res, u=u, rstd=rstd, y=y, y8=y8, y8_scale=scale, drop_p=p, seed=SEED,
                          offset=OFFSET)
    dropped = orc.dropout(f32(x), p, SEED, OFFSET) if p else f32(x)
    want_u = torch.from_numpy(dropped + f32(res)).to(x.dtype)
    assert torch.equal(u.cpu(), want_u)
    want, r = orc.add_rmsnorm(f64(u), f64(w), 1e-5)
    assert np.all(np.abs(f64(rstd) - r) <= 1e-5 * r)
    close(y, want, dtype, np.abs(want))
    top = np.abs(want).max(1)
    assert np.all(np.abs(f64(scale) - top / 448) <= 1e-5 * top / 448)
    # half a step of e4m3: 2^-4 of a normal value, 2^-10 below the least normal
    got8 = f64(y8) * f64(scale)[:, None]
    assert np.all(np.abs(got8 - want) <= np.abs(want) * (2.0 ** -4 + 1e-5) + top[:, None] / 448 * 2.0 ** -10)
    # fewer outputs, no residual, and u written over x
    y2 = torch.empty_like(y)
    sg.sg_add_rmsnorm_fwd(u, w, 1e-5, y=y2)
    close(y2, want, dtype, np.abs(want))
    q2, s2 = torch.empty_like(y8), torch.empty_like(scale)
    sg.sg_add_rmsnorm_fwd(x, w, 1e-5, residual=res, u=x, y8=q2, y8_scale=s2, drop_p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(x, u) and torch.equal(s2, scale) and torch.equal(q2.view(torch.uint8), y8.view(torch.uint8))


def test_norm_of_zero_rows_and_of_values_that_are_not_numbers():
    x = rand(4, 512, "bf16", 4)
    x[1] = 0
    x[2, 5] = float("inf")
    w = torch.ones(512, dtype=x.dtype, device="cuda")
    y, y8 = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(4, device="cuda")
    sg.sg_add_rmsnorm_fwd(x, w, 1e-6, y=y, y8=y8, y8_scale=scale)
    assert not y[1].any() and float(scale[1]) == 0 and not y8[1].float().any()
    assert torch.isnan(y[2, 5]) and torch.isnan(y8[2, 5].float()) and torch.isnan(scale[2])
    for r in (0, 3):  # the other rows do not see them
        assert torch.isfinite(y[r]).all() and torch.isfinite(y8[r].float()).all()
    sg.sg_add_rmsnorm_fwd(x[1:2], w, 0.0, y=y[1:2])  # 0 / 0
    assert torch.isnan(y[1]).all()


def test_norm_to_8_bits_of_the_smallest_rows():
    # y of 2^-137 to 2^-107: where max |y| / 448 or its inverse leave fp32's normal numbers
    x = rand(31, 512, "f32", 5)
    x[:, 7] = 0
    y, y8 = torch.empty_like(x), torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(31, device="cuda")
    for i in range(31):
        w = torch.full((512,), 2.0 ** (i - 137), device="cuda")
        sg.sg_add_rmsnorm_fwd(x[i:i + 1], w, 1e-6, y=y[i:i + 1], y8=y8[i:i + 1], y8_scale=scale[i:i + 1])
    # y itself is rounded to a multiple of 2^-149
    got, want, s = f64(y8) * f64(scale)[:, None], f64(y), f64(scale)[:, None]
    assert np.all(s >= 2.0 ** -126)
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -4 + 1e-5) + s * 2.0 ** -10 + 2.0 ** -148)


@pytest.mark.parametrize("unit", (1e-15, 1e15))
def test_norm_backward_of_rows_of_other_scales(unit):
    dy, u = rand(8, 520, "f32", 1), unit * rand(8, 520, "f32", 2)
    w = torch.ones(520, device="cuda")
    rstd = (1 / np.sqrt((f64(u) ** 2).mean(1))).astype(np.float32)
    rstd = torch.from_numpy(rstd).cuda()
    du = torch.empty_like(dy)
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du)
    want, _ = orc.add_rmsnorm_grad(f64(dy), f64(u), f64(w), f64(rstd), 0 * f64(dy))
    r = f64(rstd)[:, None]
    g, n = np.abs(f64(dy)), np.abs(f64(u)) * r
    close(du, want, "f32", r * (g + n * (g * n).mean(1, keepdims=True)))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES + [(700, 264), (5000, 40), (1300, 2056), (3, 16384), (2, 20001)], ids=str)
@pytest.mark.parametrize("pad,shift,p", [(0, 0, 0.0), (8, 0, 0.3), (3, 1, 0.3)])
def test_norm_backward(shape, dtype, pad, shift, p):
    rows, cols = shape
    dy, u = rand(*shape, dtype, 1, pad, shift), rand(*shape, dtype, 2, pad, 0, 2.0)
    du_in = rand(*shape, dtype, 3)
    w = (1 + 0.2 * rand(1, cols, "f32", 4)).to(TYPES[dtype]).reshape(-1)
    rstd = torch.rsqrt(u.float().square().mean(1) + 1e-5)
    du, dx = torch.empty_like(dy), torch.empty(shape, dtype=dy.dtype, device="cuda")
    dw = torch.empty(cols, device="cuda")
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw, du_in=du_in, dx=dx, drop_p=p, seed=SEED, offset=OFFSET)
    want, want_w = orc.add_rmsnorm_grad(f64(dy), f64(u), f64(w), f64(rstd), f64(du_in))
    r = f64(rstd)[:, None]
    g, n = np.abs(f64(dy) * f64(w)), np.abs(f64(u)) * r
    slack = r * (g + n * (g * n).mean(1, keepdims=True)) + np.abs(f64(du_in))
    close(du, want, dtype, slack)
    keep = orc.dropout_keep(rows, cols, p, SEED, OFFSET) if p else np.ones(shape, bool)
    factor = float(orc.dropout_scale(p))
    close(dx, np.where(keep, want * factor, 0), dtype, slack * factor)
    assert not f64(dx)[~keep].any()
    close(dw, want_w, "f32", (np.abs(f64(dy)) * n).sum(0) * 2)
    # without the optional parts, written over dy; and once more, the same bits
    dw2 = torch.empty_like(dw)
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw2, du_in=du_in, drop_p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(dw, dw2)
    plain, _ = orc.add_rmsnorm_grad(f64(dy), f64(u), f64(w), f64(rstd))
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, dy)
    close(dy, plain, dtype, slack)


def test_norm_gradient_against_differences():
    """The kernels' gradient along a direction, against central differences of
    the 64-bit forward (fp32 rows: the gradient is good to about 1e-6)."""
    shape, eps, step = (37, 301), 1e-3, 1e-5
    x, res, w = fwd_inputs(shape, "f32", 0, 0)
    c = rand(*shape, "f32", 9)
    u, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(shape[0], device="cuda")
    sg.sg_add_rmsnorm_fwd(x, w, eps, residual=res, u=u, rstd=rstd, y=y, drop_p=0.25, seed=1, offset=2)
    du, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(shape[1], device="cuda")
    sg.sg_add_rmsnorm_bwd(c, u, w, rstd, du, dw, dx=dx, drop_p=0.25, seed=1, offset=2)
    keep = orc.dropout_keep(*shape, 0.25, 1, 2) * (1 / 0.75)

    def loss(xx, rr, ww):
        return (orc.add_rmsnorm(rr + xx * keep, ww, eps)[0] * f64(c)).sum()

    r = np.random.RandomState(1)
    at = [f64(x), f64(res), f64(w)]
    for k, grad in enumerate((dx, du, dw)):
        d = r.randn(*at[k].shape)
        hi, lo = [a.copy() for a in at], [a.copy() for a in at]
        hi[k] += step * d
        lo[k] -= step * d
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        got = (f64(grad) * d).sum()
        assert abs(got - want) <= 1e-5 * np.abs(f64(grad) * d).sum()


def test_no_rows_and_another_stream():
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    sg.sg_dropout(e, 0.5, 1, 2, e)
    sg.sg_add_rmsnorm_fwd(e, w, 1e-6, y=e)
    dw = torch.full((64,), 3.0, device="cuda")
    sg.sg_add_rmsnorm_bwd(e, e, w, torch.empty(0, device="cuda"), e, dw)
    assert not dw.any()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        x = rand(2048, 4096, "bf16", 5)
        y, z = torch.empty_like(x), torch.empty_like(x)
        sg.sg_dropout(x, 0.5, 1, 2, y)
        sg.sg_dropout(y, 0.0, 1, 2, z)
    st.synchronize()
    assert torch.equal(y, z)


def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    r = torch.zeros(4, device="cuda")
    y = torch.empty_like(x)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(sg.SGError) as e:
            sg.sg_dropout(x, p, 1, 2, y)
        assert e.value.status == sg.SG_ERR_INVALID
    with pytest.raises(TypeError):
        sg.sg_dropout(x, 0.5, 1, 2, y.half())
    with pytest.raises(ValueError):
        sg.sg_dropout(x, 0.5, 1, 2, y[:, :32])
    with pytest.raises(ValueError):
        sg.sg_dropout(x, 0.5, 1, 2, torch.empty((64, 4), dtype=x.dtype, device="cuda").t())
    with pytest.raises(ValueError):
        sg.sg_dropout(x.cpu(), 0.5, 1, 2, y)
    with pytest.raises(sg.SGError):
        sg.sg_add_rmsnorm_fwd(x, w, 1e-6)  # neither y nor y8
    with pytest.raises(sg.SGError):
        sg.sg_add_rmsnorm_fwd(x, w, 1e-6, y8=torch.empty(x.shape, dtype=torch.float8_e4m3fn, device="cuda"))
    for eps in (-1.0, float("inf"), float("nan")):
        with pytest.raises(sg.SGError):
            sg.sg_add_rmsnorm_fwd(x, w, eps, y=y)
    with pytest.raises(TypeError):
        sg.sg_add_rmsnorm_fwd(x, w.float(), 1e-6, y=y)
    with pytest.raises(sg.SGError):
        sg.sg_add_rmsnorm_bwd(x, x, w, r, y, torch.empty(64, device="cuda"),
                              work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros((1, 32769), device="cuda")
    with pytest.raises(sg.SGError) as e:
        sg.sg_add_rmsnorm_fwd(wide, wide[0], 1e-6, y=wide)
    assert e.value.status == sg.SG_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(5003, 768), (4999, 520), (10001, 1024)], ids=str)
def test_norm_of_many_rows(shape, dtype):
    """Enough rows that every row group takes several, and (513 to 768 columns)
    the shape of one warp to a row."""
    x, res, w = fwd_inputs(shape, dtype, 0, 0)
    u, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(shape[0], device="cuda")
    sg.sg_add_rmsnorm_fwd(x, w, 1e-5, residual=res, u=u, rstd=rstd, y=y, drop_p=0.3, seed=SEED, offset=OFFSET)
    want_u = torch.from_numpy(orc.dropout(f32(x), 0.3, SEED, OFFSET) + f32(res)).to(x.dtype)
    assert torch.equal(u.cpu(), want_u)
    want, r = orc.add_rmsnorm(f64(u), f64(w), 1e-5)
    assert np.all(np.abs(f64(rstd) - r) <= 1e-5 * r)
    close(y, want, dtype, np.abs(want))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(16501, 512), (11003, 768), (2050, 4096)], ids=str)
def test_norm_of_many_rows_in_16_bits_without_dropout(shape, dtype):
    x, res, w = fwd_inputs(shape, dtype, 0, 0)
    u, y = torch.empty_like(x), torch.empty_like(x)
    sg.sg_add_rmsnorm_fwd(x, w, 1e-5, residual=res, u=u, y=y)
    assert torch.equal(u, (x.float() + res.float()).to(x.dtype))
    want, _ = orc.add_rmsnorm(f64(u), f64(w), 1e-5)
    close(y, want, dtype, np.abs(want))


def test_norm_backward_of_many_wide_rows():
    """More than 32 rows to a row group of four segments to a warp."""
    rows, cols = 5003, 8200
    dy, u = rand(rows, cols, "bf16", 1), rand(rows, cols, "bf16", 2)
    w = (1 + 0.2 * rand(1, cols, "f32", 3)).bfloat16().reshape(-1)
    rstd = (1 + torch.rand(rows, device="cuda")) / 2
    du, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw)
    r, n = rstd.double()[:, None], u.double() * rstd.double()[:, None]
    g = dy.double() * w.double()
    want = r * (g - n * (g * n).mean(1, keepdim=True))
    slack = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    close(du, want.cpu().numpy(), "bf16", slack.cpu().numpy())
    t = dy.double() * n
    close(dw, t.sum(0).cpu().numpy(), "f32", 2 * t.abs().sum(0).cpu().numpy())


def test_dropout_beyond_two_to_the_31_elements():
    """The mask goes by row and column alone: the first columns as a matrix of
    their own get the same one."""
    rows, cols = (1 << 21) + 5, 1032
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    y, part = torch.zeros_like(x), torch.zeros((rows, 8), dtype=x.dtype, device="cuda")
    sg.sg_dropout(x, 0.5, SEED, OFFSET, y)
    sg.sg_dropout(x[:, :8], 0.5, SEED, OFFSET, part)
    assert torch.equal(y[:, :8], part)
    assert torch.equal(part[:4].cpu(), torch.from_numpy(orc.dropout(np.ones((4, 8), np.float32), 0.5, SEED,
                                                                    OFFSET)).bfloat16())
    # standard deviation of the mean of 10^6 of them: 5e-4
    for at in (0, rows // 2, rows - 1000):
        assert abs(float((y[at:at + 1000] != 0).float().mean()) - 0.5) < 5e-3


@pytest.mark.parametrize("unit", (1e-36, 1e-30, 1e-20, 1e20, 1e30, 1e34))
@pytest.mark.parametrize("dtype,cols", [("f32", 520), ("f32", 301), ("bf16", 520), ("bf16", 8200)])
def test_norm_backward_of_rows_of_extreme_scales(dtype, cols, unit):
    """Rows whose squares fp32 cannot hold, but whose rstd it can."""
    dy, u = rand(5, cols, dtype, 1), (unit * rand(5, cols, "f32", 2)).to(TYPES[dtype])
    w = (1 + 0.2 * rand(1, cols, "f32", 3)).to(TYPES[dtype]).reshape(-1)
    rstd = torch.from_numpy((1 / np.sqrt((f64(u) ** 2).mean(1))).astype(np.float32)).cuda()
    du, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw)
    want, want_w = orc.add_rmsnorm_grad(f64(dy), f64(u), f64(w), f64(rstd))
    r = f64(rstd)[:, None]
    g, n = np.abs(f64(dy) * f64(w)), np.abs(f64(u)) * r
    close(du, want, dtype, r * (g + n * (g * n).mean(1, keepdims=True)))
    close(dw, want_w, "f32", (np.abs(f64(dy)) * n).sum(0) * 2)


@pytest.mark.parametrize("dtype,cols", [("f32", 520), ("f32", 301), ("bf16", 301), ("bf16", 700), ("bf16", 32768)])
def test_norm_forward_of_rows_at_the_ends_of_its_range(dtype, cols):
    """Root mean squares of 1e-18 and 1e19 / sqrt(cols); a row beyond keeps to
    itself, with the rstd that its fp32 sum gives."""
    far = 1e19 / np.sqrt(cols)
    units = np.array([1.0, 1e-18, 1e-17, far / 2, far, 1.0, 1e21, 1e-30, 1.0])
    x = rand(9, cols, "f32", 1)
    x = x / x.square().mean(1, keepdim=True).sqrt() * torch.tensor(units, device="cuda").float()[:, None]
    x = x.to(TYPES[dtype])
    w = (1 + 0.2 * rand(1, cols, "f32", 3)).to(TYPES[dtype]).reshape(-1)
    y, rstd = torch.empty_like(x), torch.empty(9, device="cuda")
    for eps in (0.0, 1e-30):
        sg.sg_add_rmsnorm_fwd(x, w, eps, rstd=rstd, y=y)
        ok = np.array([True] * 6 + [False, False, True])
        want, r = orc.add_rmsnorm(f64(x), f64(w), float(np.float32(eps)))
        assert np.all(np.abs(f64(rstd) - r)[ok] <= 1e-5 * r[ok])
        close(y[torch.from_numpy(ok).cuda()], want[ok], dtype, np.abs(want[ok]))
        assert float(rstd[6]) == 0 and not y[6].any()
        assert eps > 0 or float(rstd[7]) == float("inf")


@pytest.mark.parametrize("dtype,shape", [("bf16", (700, 1024)), ("f32", (300, 4096)), ("f16", (501, 333)),
                                         ("bf16", (40, 20000))])
def test_outputs_written_over_inputs(dtype, shape):
    """The same bits as with outputs of their own, for every input that an output
    may be."""
    rows, cols = shape
    x, res, w = fwd_inputs(shape, dtype, 0, 0)
    drop = dict(drop_p=0.25, seed=SEED, offset=OFFSET)
    u, y = torch.empty_like(x), torch.empty_like(x)
    sg.sg_add_rmsnorm_fwd(x, w, 1e-5, residual=res, u=u, y=y, **drop)
    for over_u, over_y in (("x", "residual"), ("residual", "x"), ("residual", "own"), ("x", "own"), ("own", "x"),
                           ("own", "residual")):
        t = {"x": x.clone(), "residual": res.clone()}
        own = torch.empty_like(x)
        a, b = t.get(over_u, own), t.get(over_y, own)
        sg.sg_add_rmsnorm_fwd(t["x"], w, 1e-5, residual=t["residual"], u=a, y=b, **drop)
        assert torch.equal(a, u) and torch.equal(b, y)
    for over in ("x", "residual"):  # u not asked for
        t = {"x": x.clone(), "residual": res.clone()}
        sg.sg_add_rmsnorm_fwd(t["x"], w, 1e-5, residual=t["residual"], y=t[over], **drop)
        assert torch.equal(t[over], y)
    dy, du_in = rand(*shape, dtype, 3), rand(*shape, dtype, 4)
    rstd = torch.rsqrt(u.float().square().mean(1) + 1e-5)
    du, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(cols, device="cuda")
    sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw, du_in=du_in, dx=dx, **drop)
    for over_du, over_dx in (("dy", "du_in"), ("du_in", "dy"), ("dy", "own"), ("du_in", "own"), ("own", "dy"),
                             ("own", "du_in")):
        t = {"dy": dy.clone(), "du_in": du_in.clone()}
        own, dw2 = torch.empty_like(x), torch.empty_like(dw)
        a, b = t.get(over_du, own), t.get(over_dx, own)
        sg.sg_add_rmsnorm_bwd(t["dy"], u, w, rstd, a, dw2, du_in=t["du_in"], dx=b, **drop)
        assert torch.equal(a, du) and torch.equal(b, dx) and torch.equal(dw2, dw)


def test_rows_on_two_streams_at_once():
    """Each stream's outputs are those of its calls alone."""
    cases = []
    for seed in (1, 2):
        dy, u = rand(4000, 2048, "bf16", seed), rand(4000, 2048, "bf16", seed + 2)
        rstd, w = torch.rand(4000, device="cuda") + 0.5, rand(1, 2048, "bf16", 5).reshape(-1)
        outs = [[torch.empty_like(u), torch.empty(2048, device="cuda"), torch.empty_like(u), torch.empty_like(u)]
                for _ in range(2)]
        cases.append((dy, u, rstd, w, outs, torch.cuda.Stream()))

    def step(case, i):
        dy, u, rstd, w, outs, _ = case
        du, dw, y, d = outs[i]
        sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw)
        sg.sg_add_rmsnorm_fwd(dy, w, 1e-6, residual=u, y=y)
        sg.sg_dropout(dy, 0.5, SEED, OFFSET, d)

    for case in cases:
        step(case, 0)
    torch.cuda.synchronize()
    for _ in range(10):
        for case in cases:
            with torch.cuda.stream(case[5]):
                step(case, 1)
    torch.cuda.synchronize()
    for case in cases:
        assert all(torch.equal(a, b) for a, b in zip(*case[4]))


@pytest.mark.parametrize("shape", [(1, 8), (3, 768), (1000, 264), (4001, 1001), (700, 20000)], ids=str)
def test_what_work_memory_of_dweight_holds_does_not_matter(shape):
    rows, cols = shape
    dy, u = rand(*shape, "bf16", 1), rand(*shape, "bf16", 2)
    w, rstd = torch.ones(cols, dtype=dy.dtype, device="cuda"), torch.rand(rows, device="cuda") + 0.5
    got = []
    for fill in (0, 255):
        work = torch.full((sg.sg_add_rmsnorm_bwd_work(rows, cols),), fill, dtype=torch.uint8, device="cuda")
        du, dw = torch.empty_like(dy), torch.empty(cols, device="cuda")
        sg.sg_add_rmsnorm_bwd(dy, u, w, rstd, du, dw, work=work)
        got.append((du, dw))
    for a, b in zip(*got):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
