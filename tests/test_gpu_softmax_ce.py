"""Softmax cross entropy of a dense head against its 64-bit restatement.

Tolerances.  A logit is a sum of H products, exact in fp32, added in fp32 in
steps of 16 or more: (H / 16 + 4) 2^-23 of its terms' absolute sum.  lse moves
by no more than the largest logit error, loss by twice that; the exponentials,
their sum and the logarithm add 1e-5 (1e-6 of a loss of a few units, several
times).  g, the sum of three parts that may cancel, is off by (2 e_z + 3e-5) of
its parts' absolute values and rounded to dtype (u = 2^-8 for bf16, 2^-11 for
f16, half a unit in the last place): an element of dh and dW is off by u of its
terms' absolute sum, by (2 e_z + 3e-5) of the sum with g's parts in its place,
and by u from its own rounding, and by what the types cannot hold (half of
f16's smallest step; an exponential below fp32's 2^-126 is taken as zero, times
features below 2^6).
Roundings that are independent of one another make less of it: over
a whole matrix, whose two roundings have a root mean square of at most
u / sqrt(3) each, the 2-norm of the error is below u of the 2-norm, plus the
other parts of the bound.
"""
import numpy as np
import pytest
import torch

import extreme_label_sparse_gb300 as sg
from oracle.softmax_ce import softmax_ce

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"bf16": 2.0 ** -120, "f16": 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rand(rows, cols, dtype, seed, std=1.0, pad=0, shift=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((rows, cols + pad + shift), generator=g, device="cuda") * std
    return x.to(TYPES[dtype])[:, shift:shift + cols]


def draw_targets(T, V, seed, ignored=0.1):
    r = np.random.RandomState(seed)
    y = r.randint(0, V, T)
    y[r.rand(T) < ignored] = -100
    return torch.tensor(y, dtype=torch.int32, device="cuda")


def logit_error(h, W):
    """Bound on a logit's error, row by row."""
    H = h.shape[1]
    return (H / 16 + 4) * 2.0 ** -23 * (np.abs(h) @ np.abs(W).T).max(1)


def check(h, W, y, dloss, dtype, smoothing=0.0, ignore=-100, want_dh=True, want_dW=True, dW_out=None, status=None):
    (T, H), V = h.shape, W.shape[0]
    loss, lse = torch.full((T,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda")
    dh = torch.full((T, H), 9.0, dtype=h.dtype, device="cuda") if want_dh else None
    dW = (torch.full((V, H), 9.0, dtype=h.dtype, device="cuda") if dW_out is None else dW_out) if want_dW else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(ignore_index=ignore, smoothing=smoothing, status=st)
    sg.sg_softmax_ce_fwd(h, W, y, loss, lse, **kw)
    sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, **kw)
    ref = softmax_ce(f64(h), f64(W), y.cpu().numpy(), f64(dloss), ignore, smoothing)
    e = logit_error(f64(h), f64(W))
    assert int(st) == (0 if status is None else status)
    assert np.all(np.abs(f64(lse) - ref["lse"]) <= e + 1e-5)
    assert np.all(np.abs(f64(loss) - ref["loss"]) <= 2 * e + 1e-5)
    u = U[dtype]
    for name, got in (("dh", dh), ("dW", dW)):
        if got is None:
            continue
        got, want, terms, mag = f64(got), ref[name], ref[name + "_abs"], ref[name + "_mag"]
        assert np.all(np.isfinite(got))
        err = np.abs(got - want)
        bound = u * terms + (2 * e.max() + 3e-5) * mag + u * np.abs(want) + LEAST[dtype] * (1 + 2.0 ** -14)
        assert np.all(err <= bound), (name, (err - bound).max(), np.unravel_index((err - bound).argmax(), err.shape))
        if dtype == "bf16" or np.sqrt(np.mean(want ** 2)) > 2.0 ** -10:  # f16: above its subnormal range
            rest = (2 * e.max() + 3e-5) * np.linalg.norm(mag)
            assert np.linalg.norm(err) <= u * np.linalg.norm(want) + rest, (name, np.linalg.norm(err))
    return loss, lse, dh, dW


SIZES = [(1, 8, 1), (1, 64, 300), (2, 72, 255), (5, 768, 256), (31, 64, 257), (64, 128, 20000), (127, 256, 1000),
         (128, 768, 4096), (129, 64, 1000), (130, 1032, 777), (256, 320, 5003), (300, 768, 2500), (1025, 128, 1300)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_against_64_bits(size, dtype, smoothing):
    T, H, V = size
    h, W = rand(T, H, dtype, 1), rand(V, H, dtype, 2, 2.0 / np.sqrt(H))
    dloss = torch.rand(T, device="cuda") + 0.5
    check(h, W, draw_targets(T, V, 3), dloss, dtype, smoothing)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(1, 1, 5), (3, 7, 300), (50, 100, 1000), (140, 1001, 700), (200, 333, 1025),
                                  (130, 1005, 600), (20, 333, 600)], ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1), (3, 0)])
def test_odd_widths_strides_and_alignment(size, dtype, pad, shift):
    T, H, V = size
    h, W = rand(T, H, dtype, 1, 1.0, pad, shift), rand(V, H, dtype, 2, 2.0 / np.sqrt(H), pad, 0)
    out = torch.full((V + 2, H + 3), 5.0, dtype=h.dtype, device="cuda")
    check(h, W, draw_targets(T, V, 3), torch.ones(T, device="cuda"), dtype, 0.0, dW_out=out[1:V + 1, :H])
    assert bool((out[0] == 5).all()) and bool((out[V + 1] == 5).all()) and bool((out[:, H:] == 5).all())


@pytest.mark.parametrize("size", [(4096, 64, 70000), (4500, 72, 1000), (2100, 520, 66000)], ids=str)
def test_pieces_of_the_vocabulary_and_bands_of_rows(size):
    """More than one piece (256 MB of g hold 32768 labels of 4096 rows), more
    than one band of 4096 rows."""
    T, H, V = size
    h, W = rand(T, H, "bf16", 1), rand(V, H, "bf16", 2, 3.0 / np.sqrt(H))
    check(h, W, draw_targets(T, V, 3), torch.full((T,), 1.0 / T, device="cuda"), "bf16", 0.1)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [40, 200])
def test_ignored_rows_and_small_weights(dtype, T):
    """Rows without a target have no loss and no gradient; dloss of 1e-7 is
    below what fp16 holds times a probability."""
    h, W = rand(T, 128, dtype, 1), rand(900, 128, dtype, 2, 0.2)
    y = draw_targets(T, 900, 3, 0.5)
    dloss = torch.rand(T, device="cuda") * 1e-7
    loss, lse, dh, dW = check(h, W, y, dloss, dtype)
    assert not loss[y == -100].any() and not dh[y == -100].any() and bool((lse != 9).all())
    y[:] = -100
    loss, _, dh, dW = check(h, W, y, dloss, dtype)
    assert not loss.any() and not dh.any() and not dW.any()
    # another ignore_index, one of the labels
    y = draw_targets(T, 900, 3, 0.0)
    loss, _, dh, _ = check(h, W, y, dloss, dtype, ignore=int(y[0]))
    assert not loss[y == y[0]].any() and not dh[y == y[0]].any()


def test_targets_that_are_no_labels():
    T, V = 20, 500
    h, W = rand(T, 64, "bf16", 1), rand(V, 64, "bf16", 2, 0.25)
    for bad in (-1, V, 2 ** 31 - 1, -2 ** 31):
        y = draw_targets(T, V, 3)
        y[7] = bad
        loss, _, dh, _ = check(h, W, y, torch.ones(T, device="cuda"), "bf16", status=sg.SG_ERR_DATA)
        assert float(loss[7]) == 0 and not dh[7].any()


def test_large_logits_and_values_that_are_not_numbers():
    """Logits of hundreds (exp overflows), a row with an infinity, a row with a
    NaN: the other rows do not see them."""
    h, W = rand(40, 64, "bf16", 1, 8.0), rand(1000, 64, "bf16", 2, 8.0)
    y = draw_targets(40, 1000, 3, 0.0)
    one = torch.ones(40, device="cuda")
    check(h, W, y, one, "bf16")
    h2 = h.clone()
    h2[3, 5], h2[9, 0] = float("inf"), float("nan")
    a, b = ([torch.empty(40, device="cuda") for _ in range(2)] for _ in range(2))
    sg.sg_softmax_ce_fwd(h, W, y, *a)
    sg.sg_softmax_ce_fwd(h2, W, y, *b)
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[3] = keep[9] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])
    assert torch.isnan(b[1][9]) and not torch.isfinite(b[1][3])
    dh, dh2 = torch.empty_like(h), torch.empty_like(h)
    sg.sg_softmax_ce_bwd(h, W, y, a[1], one, dh)
    sg.sg_softmax_ce_bwd(h2, W, y, b[1], one, dh2)
    assert torch.equal(dh[keep], dh2[keep])
    # an ignored row's values reach no gradient of W that is not 0 x infinity
    y[3] = y[9] = -100
    z = h2.clone()
    z[3], z[9] = 1e30, -1e30
    dW, dW0 = torch.empty_like(W), torch.empty_like(W)
    sg.sg_softmax_ce_bwd(z, W, y, a[1], one, None, dW)
    sg.sg_softmax_ce_bwd(h, W, y, a[1], one, None, dW0)
    assert torch.equal(dW, dW0)


@pytest.mark.parametrize("size", [(1, 16, 10), (1, 768, 32000), (48, 2048, 3001), (77, 100, 999), (200, 1000, 5000)],
                         ids=str)
@pytest.mark.parametrize("smoothing", [0.0, 0.2])
def test_8_bit_rows(size, smoothing):
    T, H, V = size
    e4m3 = torch.float8_e4m3fn

    def rows8(x):
        top = x.abs().amax(1).clamp_min(1e-20)
        return (x * (448 / top)[:, None]).to(e4m3), top / 448

    h, hs = rows8(rand(T, H, "bf16", 1).float())
    W, Ws = rows8(rand(V, H, "bf16", 2, 2.0 / np.sqrt(H)).float())
    if T > 1:
        hs[1] = 0  # a row of zeros
    y = draw_targets(T, V, 3)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    for use_h, use_W in ((True, True), (False, True), (True, False)):
        # without its scales the rows are taken as they are: small ones
        hh = h if use_h else (h.float() / 512).to(e4m3)
        WW = W if use_W else (W.float() / 512).to(e4m3)
        sg.sg_softmax_ce_fwd(hh, WW, y, loss, lse, h_scale=hs if use_h else None, W_scale=Ws if use_W else None,
                             smoothing=smoothing)
        h6 = f64(hh) * (f64(hs)[:, None] if use_h else 1)
        W6 = f64(WW) * (f64(Ws)[:, None] if use_W else 1)
        ref = softmax_ce(h6, W6, y.cpu().numpy(), smoothing=smoothing)
        e = logit_error(h6, W6)
        assert np.all(np.abs(f64(lse) - ref["lse"]) <= e + 1e-5)
        assert np.all(np.abs(f64(loss) - ref["loss"]) <= 2 * e + 1e-5)


def test_gradient_against_differences():
    """Along a direction, against central differences of the 64-bit loss: each
    gradient element is off by at most 2^-9 of its absolute terms (two
    roundings to f16), so the sum by 2^-9 of theirs."""
    T, H, V, step = 33, 72, 700, 1e-6
    h, W = rand(T, H, "f16", 1), rand(V, H, "f16", 2, 0.3)
    y, c = draw_targets(T, V, 3), torch.rand(T, device="cuda")
    _, _, dh, dW = check(h, W, y, c, "f16", 0.1)
    r, at = np.random.RandomState(4), [f64(h), f64(W)]
    ref = softmax_ce(*at, y.cpu().numpy(), f64(c), smoothing=0.1)
    for k, (got, terms) in enumerate(((dh, ref["dh_abs"]), (dW, ref["dW_abs"]))):
        d = r.randn(*at[k].shape)
        lo, hi = list(at), list(at)
        lo[k], hi[k] = at[k] - step * d, at[k] + step * d
        diff = sum(s * (softmax_ce(*a, y.cpu().numpy(), smoothing=0.1)["loss"] * f64(c)).sum()
                   for s, a in ((1, hi), (-1, lo))) / (2 * step)
        assert abs((f64(got) * d).sum() - diff) <= 2.0 ** -9 * (terms * np.abs(d)).sum()


def test_parts_of_the_gradient_and_the_same_bits_twice():
    for T in (60, 260):
        h, W = rand(T, 200, "bf16", 1), rand(3000, 200, "bf16", 2, 0.2)
        y, c = draw_targets(T, 3000, 3), torch.rand(T, device="cuda")
        a = check(h, W, y, c, "bf16")
        b = check(h, W, y, c, "bf16")
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        only = check(h, W, y, c, "bf16", want_dW=False)
        assert np.abs(f64(only[2]) - f64(a[2])).max() <= 2.0 ** -7 * np.abs(f64(a[2])).max()
        assert torch.equal(check(h, W, y, c, "bf16", want_dh=False)[3], a[3])


def test_no_rows_another_stream_and_a_graph():
    W = rand(300, 64, "bf16", 2)
    e, n = torch.empty((0, 64), dtype=W.dtype, device="cuda"), torch.empty(0, device="cuda")
    dW = torch.full_like(W, 4.0)
    sg.sg_softmax_ce_fwd(e, W, n.int(), n, n.clone())
    sg.sg_softmax_ce_bwd(e, W, n.int(), n, n, e, dW)
    assert not dW.any()
    T = 150
    h, y = rand(T, 64, "bf16", 1), draw_targets(T, 300, 3)
    loss, lse, dh, dW = check(h, W, y, torch.ones(T, device="cuda"), "bf16")
    out = [torch.empty_like(t) for t in (loss, lse, dh, dW)]
    one = torch.ones(T, device="cuda")
    work = torch.empty(max(sg.sg_softmax_ce_work(h, W, b) for b in (False, True)), dtype=torch.uint8, device="cuda")

    def step():
        sg.sg_softmax_ce_fwd(h, W, y, out[0], out[1], work=work)
        sg.sg_softmax_ce_bwd(h, W, y, out[1], one, out[2], out[3], work=work)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, (loss, lse, dh, dW)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in out:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, (loss, lse, dh, dW)))


def test_refusals():
    h, W = rand(4, 64, "bf16", 1), rand(10, 64, "bf16", 2)
    y, v = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    for s in (-0.1, 1.5, float("nan")):
        with pytest.raises(sg.SGError) as e:
            sg.sg_softmax_ce_fwd(h, W, y, v, v.clone(), smoothing=s)
        assert e.value.status == sg.SG_ERR_INVALID
    with pytest.raises(sg.SGError):  # scales without 8-bit rows
        sg.sg_softmax_ce_fwd(h, W, y, v, v.clone(), h_scale=v)
    with pytest.raises(sg.SGError):
        sg.sg_softmax_ce_bwd(h, W, y, v, v)  # no gradient asked for
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    with pytest.raises(sg.SGError):
        sg.sg_softmax_ce_fwd(h, W, y, v, v.clone(), work=small)
    with pytest.raises(sg.SGError):
        big = torch.empty(sg.sg_softmax_ce_work(h, W, False) + 512, dtype=torch.uint8, device="cuda")
        sg.sg_softmax_ce_fwd(h, W, y, v, v.clone(), work=big[16:])
    with pytest.raises(TypeError):
        sg.sg_softmax_ce_fwd(h, W.half(), y, v, v.clone())
    with pytest.raises(TypeError):
        sg.sg_softmax_ce_fwd(h, W, y.long(), v, v.clone())
    with pytest.raises(TypeError):
        sg.sg_softmax_ce_fwd(h.float(), W.float(), y, v, v.clone())
    with pytest.raises(TypeError):
        e4 = torch.float8_e4m3fn
        sg.sg_softmax_ce_bwd(h.to(e4), W.to(e4), y, v, v, torch.empty_like(h.to(e4)))
    with pytest.raises(ValueError):
        sg.sg_softmax_ce_fwd(h, W[:, :32], y, v, v.clone())
    with pytest.raises(ValueError):
        sg.sg_softmax_ce_fwd(h, W, y[:3], v, v.clone())


def test_weights_of_more_than_two_to_the_31_elements():
    """A block of 512 labels, many times over: every copy has the block's
    logits, so lse is the block's plus the logarithm of their number."""
    T, H, V0, n = 5, 2048, 512, 2051
    V = V0 * n
    h, block = rand(T, H, "bf16", 1), rand(V0, H, "bf16", 2, 2.0 / np.sqrt(H))
    W = block.repeat(n, 1)
    y = torch.tensor([3, V - 1, V - V0, -100, V // 2], dtype=torch.int32, device="cuda")
    dloss = torch.rand(T, device="cuda") + 0.5
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dh, dW = torch.empty_like(h), torch.empty_like(W)
    sg.sg_softmax_ce_fwd(h, W, y, loss, lse)
    sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW)
    hd, bd = f64(h), f64(block)
    e = logit_error(hd, bd)
    z = hd @ bd.T
    want = np.log(np.exp(z).sum(1)) + np.log(n)
    at = y.cpu().numpy()
    live = at >= 0
    assert np.all(np.abs(f64(lse) - want) <= e + 1e-5)
    zt = z[np.arange(T), np.where(live, at % V0, 0)]
    assert np.all(np.abs(f64(loss) - np.where(live, want - zt, 0)) <= 2 * e + 1e-5)
    c = np.where(live, f64(dloss), 0)[:, None]
    p = c * np.exp(z - want[:, None])  # g, but for the targets' part
    rel = 2 * e.max() + 3e-5
    u = U["bf16"]
    # dW: in every copy the same but for the targets' rows
    plain = p.T @ hd
    bound = (2 * u + rel) * (p.T @ np.abs(hd)) + LEAST["bf16"] * 2
    rows = dW.view(n, V0, H)
    other = torch.ones((n, V0), dtype=torch.bool, device="cuda")
    for t in np.flatnonzero(live):
        other[at[t] // V0, at[t] % V0] = False
        want_row = plain[at[t] % V0] - c[t] * hd[t]
        row_bound = bound[at[t] % V0] + (2 * u + rel) * c[t] * np.abs(hd[t])
        assert np.all(np.abs(f64(dW[int(at[t])]) - want_row) <= row_bound)
    for i in (0, 1, n // 2, n - 2, n - 1):
        err = np.abs(f64(rows[i]) - plain)
        assert np.all((err <= bound)[other[i].cpu().numpy()])
    for i in range(1, n):  # and the same bits
        same = (rows[i].view(torch.int16) == rows[1].view(torch.int16)).all(1)
        assert bool((same | ~other[i] | ~other[1]).all())
    # dh: the sum over all copies
    wt = bd[np.where(live, at % V0, 0)]
    want_h = n * (p @ bd) - c * wt
    terms = n * (p @ np.abs(bd)) + c * np.abs(wt)
    assert np.all(np.abs(f64(dh) - want_h) <= (2 * u + rel) * terms + LEAST["bf16"] * 2)


@pytest.mark.parametrize("T", [64, 96, 200])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_dloss_of_rows_without_a_target_has_no_effect(dtype, T):
    """Whatever dloss holds where a row is ignored or its target is no label,
    the gradients are the same bits."""
    V = 5000
    h, W = rand(T, 128, dtype, 1), rand(V, 128, dtype, 2, 0.2)
    y = draw_targets(T, V, 3, 0.3)
    y[1], y[2] = -100, V  # ignored, no label
    dead = (y < 0) | (y >= V)
    base = torch.full((T,), 1.0 / T, device="cuda")
    lse, status = torch.empty(T, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_softmax_ce_fwd(h, W, y, torch.empty_like(lse), lse, status=status)
    got = []
    for left in (0.0, 1e6, 1e20, -1e9, float("inf"), float("nan")):
        dh, dW = torch.empty_like(h), torch.empty_like(W)
        sg.sg_softmax_ce_bwd(h, W, y, lse, torch.where(dead, left, base), dh, dW, status=status)
        got.append((dh, dW))
    assert got[0][0][~dead].any() and not got[0][0][dead].any()
    for dh, dW in got[1:]:
        assert torch.equal(dh, got[0][0]) and torch.equal(dW, got[0][1])


@pytest.mark.parametrize("T", [96, 300])
@pytest.mark.parametrize("weights", ["mean", "spread"])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_f16_gradients_of_small_weights(T, weights, smoothing):
    """dloss of 1 / T, or over three orders of magnitude, where a probability
    times dloss is below what f16 holds well: with a factor that brings the
    largest dloss to 2^13 at least, an element of g is off by at most u of its
    value and half a subnormal step, 2^-25, over the factor.  Rounding errors
    that lie anywhere in such an interval have 1 / sqrt(3) of it as root mean
    square, and those of different elements are independent, so the squares of
    the sums' errors add up.  The output's own rounding is measured; features
    and weights are scaled so that it is one of normal numbers.  A tenth more
    for what a sample of errors differs from its mean."""
    H, V = 64, 2000
    y = draw_targets(T, V, 3)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    if weights == "spread":
        g = torch.Generator(device="cuda")
        g.manual_seed(4)
        dloss = dloss * 10.0 ** (-3 * torch.rand(T, generator=g, device="cuda"))
    for up in (2.0 ** -6, 2.0 ** 6):  # dh of normal numbers, dW of normal numbers
        h, W = rand(T, H, "f16", 1, up), rand(V, H, "f16", 2, 2.0 / np.sqrt(H) / up)
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dh, dW = torch.empty_like(h), torch.empty_like(W)
        sg.sg_softmax_ce_fwd(h, W, y, loss, lse, smoothing=smoothing)
        sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, smoothing=smoothing)
        hd, Wd, at, c = f64(h), f64(W), y.cpu().numpy(), f64(dloss)
        ref = softmax_ce(hd, Wd, at, c, smoothing=smoothing)
        z = hd @ Wd.T
        p = np.exp(z - ref["lse"][:, None]) - smoothing / V
        live = at >= 0
        p[live, at[live]] -= 1 - smoothing
        p *= np.where(live, c, 0)[:, None]
        off2 = (U["f16"] ** 2 * p ** 2 + (2.0 ** -25 * c.max() / 2 ** 13) ** 2) / 3 * live[:, None]
        e = 2 * logit_error(hd, Wd).max() + 3e-5
        name, got, mean2 = (("dh", dh, (off2 @ Wd ** 2).sum()), ("dW", dW, (off2.T @ hd ** 2).sum()))[up > 1]
        want = ref[name]
        own = np.linalg.norm(want.astype(np.float16).astype(np.float64) - want)
        err = np.linalg.norm(f64(got) - want)
        assert err <= 1.1 * np.sqrt(own ** 2 + mean2) + e * np.linalg.norm(ref[name + "_mag"]), (name, err, own)


@pytest.mark.parametrize("T", [20, 300])
def test_backward_call_reports_targets_that_are_no_labels(T):
    """By itself: its status word is another than the forward call's."""
    V = 500
    h, W, v = rand(T, 64, "bf16", 1), rand(V, 64, "bf16", 2, 0.25), torch.ones(T, device="cuda")
    for bad in (-1, V, 2 ** 31 - 1, -2 ** 31):
        y = draw_targets(T, V, 3)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sg.sg_softmax_ce_bwd(h, W, y, v, v, torch.empty_like(h), status=status)
        assert int(status) == 0
        y[T - 1] = bad
        sg.sg_softmax_ce_bwd(h, W, y, v, v, torch.empty_like(h), status=status)
        assert int(status) == sg.SG_ERR_DATA


def forward64(h, W, y, smoothing, hs=None, Ws=None, piece=16384):
    """loss, lse and the bound on a logit's error of each row, in 64 bits on the
    device, a piece of the vocabulary at a time."""
    h = h.double() if hs is None else h.float().double() * hs.double()[:, None]
    T, V = h.shape[0], W.shape[0]
    lse = torch.full((T,), -float("inf"), dtype=torch.float64, device="cuda")
    total, top, at = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(3))
    for v0 in range(0, V, piece):
        w = W[v0:v0 + piece].float().double()
        if Ws is not None:
            w = w * Ws[v0:v0 + piece].double()[:, None]
        z = h @ w.t()
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
        total += z.sum(1)
        here = (y >= v0) & (y < v0 + piece)
        at = torch.where(here, z.gather(1, (y.long() - v0).clamp(0, z.shape[1] - 1)[:, None])[:, 0], at)
        top = torch.maximum(top, (h.abs() @ w.abs().t()).amax(1))
    loss = lse - (1 - smoothing) * at - smoothing * total / V
    return torch.where(y >= 0, loss, 0.0), lse, (h.shape[1] / 16 + 4) * 2.0 ** -23 * top


@pytest.mark.parametrize("T,H,V,dtype", [(45000, 64, 66000, "bf16"), (5000, 16, 768100, "e4m3"),
                                         (4300, 8, 710000, "f16"), (600, 16, 3900000, "e4m3")])
def test_forward_in_bands_of_rows_and_pieces_of_the_vocabulary(T, H, V, dtype):
    """Sizes whose partial results do not fit the work memory at once: bands of
    rows (the last one short), pieces of the vocabulary, and both."""
    y = draw_targets(T, V, 3)
    y[:2] = torch.tensor([0, V - 1])
    hs = Ws = None
    if dtype == "e4m3":
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        h, W = (rand(n, H, "f16", s, 16.0).float().to(torch.float8_e4m3fn) for n, s in ((T, 1), (V, 2)))
        hs, Ws = ((0.5 + torch.rand(n, generator=g, device="cuda")) / 24 for n in (T, V))
    else:
        h, W = rand(T, H, dtype, 1), rand(V, H, dtype, 2, 2.0 / np.sqrt(H))
    assert sg.sg_softmax_ce_work(h, W, False) <= (256 << 20) + 16 * T + 4096
    loss, lse, status = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                                                  device="cuda")
    for smoothing in (0.0, 0.1):
        sg.sg_softmax_ce_fwd(h, W, y, loss, lse, h_scale=hs, W_scale=Ws, smoothing=smoothing, status=status)
        want, want_lse, e = forward64(h, W, y, smoothing, hs, Ws)
        assert int(status) == 0
        assert bool(((lse.double() - want_lse).abs() <= e + 1e-5).all())
        assert bool(((loss.double() - want).abs() <= 2 * e + 1e-5).all())


@pytest.mark.parametrize("T", [20, 300])
def test_errors_of_calls_without_a_status_word_are_kept(T):
    """In the device's word, by both calls, until it is cleared."""
    V = 500
    h, W, v = rand(T, 64, "bf16", 1), rand(V, 64, "bf16", 2, 0.25), torch.ones(T, device="cuda")
    good = draw_targets(T, V, 3)
    bad = good.clone()
    bad[T // 2] = V
    out = [torch.empty(T, device="cuda") for _ in range(2)]
    sg.sg_softmax_ce_status()
    for call in (lambda y: sg.sg_softmax_ce_fwd(h, W, y, *out), lambda y: sg.sg_softmax_ce_bwd(h, W, y, v, v, torch.empty_like(h))):
        call(good)
        assert sg.sg_softmax_ce_status() == 0
        call(bad)
        call(good)
        assert sg.sg_device_status() == sg.SG_ERR_DATA  # which does not clear it
        assert sg.sg_softmax_ce_status(clear=False) == sg.SG_ERR_DATA
        assert sg.sg_softmax_ce_status() == sg.SG_ERR_DATA and sg.sg_softmax_ce_status() == 0
    own = torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_softmax_ce_fwd(h, W, bad, *out, status=own)
    assert int(own) == sg.SG_ERR_DATA and sg.sg_softmax_ce_status() == 0


# width of the forward pass's tiles: (labels at which it is taken with one row
# tile of a pair of CTAs, with two, with one row tile of one CTA)
WIDTHS = {144: (9753, 4886, 19550), 160: (11014, 5515, 21975), 176: (12178, 6107, 24400), 192: (13439, 6736, 26825),
          208: (14603, 7328, 29250), 224: (15864, 7957, 31675), 240: (17028, 8549, 34100)}


@pytest.mark.parametrize("width", list(WIDTHS))
@pytest.mark.parametrize("place,T", [(0, 130), (1, 300), (2, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3"])
def test_forward_tiles_between_128_and_256_columns(width, place, T, dtype):
    """Where a warp's half of a tile is no whole number of its 32-column chunks;
    targets on both sides of the halves' ends, in the first tiles and the last."""
    V, H = WIDTHS[width][place], 72
    y = draw_targets(T, V, 3)
    ends = np.array([0, width // 2 - 1, width // 2, width - 1])
    ends = np.concatenate([ends, ends + width, ends + V // width * width, [V - 1]])
    y[:len(ends)] = torch.tensor(np.where(ends < V, ends, 0), dtype=torch.int32)
    hs = Ws = None
    if dtype == "e4m3":
        h, W = (rand(n, 80, "f16", s, 16.0).float().to(torch.float8_e4m3fn) for n, s in ((T, 1), (V, 2)))
        hs, Ws = ((0.5 + torch.rand(n, device="cuda")) / 48 for n in (T, V))
    else:
        h, W = rand(T, H, dtype, 1), rand(V, H, dtype, 2, 2.0 / np.sqrt(H))
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    for smoothing in (0.0, 0.1):
        sg.sg_softmax_ce_fwd(h, W, y, loss, lse, h_scale=hs, W_scale=Ws, smoothing=smoothing)
        want, want_lse, e = forward64(h, W, y, smoothing, hs, Ws)
        assert bool(((lse.double() - want_lse).abs() <= e + 1e-5).all())
        assert bool(((loss.double() - want).abs() <= 2 * e + 1e-5).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(65, 72, 1000), (72, 333, 600), (80, 256, 3000), (96, 768, 2500), (105, 64, 257),
                                  (112, 320, 5003), (113, 128, 700)], ids=str)
def test_two_boxes_of_fewer_than_64_rows(size, dtype):
    T, H, V = size
    h, W = rand(T, H, dtype, 1), rand(V, H, dtype, 2, 2.0 / np.sqrt(H))
    check(h, W, draw_targets(T, V, 3), torch.rand(T, device="cuda") + 0.5, dtype, 0.1)


def test_two_streams_at_once():
    """Calls with work memory of their own, on the GPU together."""
    cases = []
    for T, H, V, seed in ((100, 512, 30000, 1), (600, 512, 30000, 2)):
        h, W = rand(T, H, "bf16", seed), rand(V, H, "bf16", seed + 2, 2.0 / np.sqrt(H))
        y, dloss = draw_targets(T, V, seed), torch.rand(T, device="cuda")
        outs = [[torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(h), torch.empty_like(W)]
                for _ in range(2)]
        cases.append((h, W, y, dloss, outs, torch.cuda.Stream()))

    def step(case, i):
        h, W, y, dloss, outs, _ = case
        loss, lse, dh, dW = outs[i]
        sg.sg_softmax_ce_fwd(h, W, y, loss, lse, smoothing=0.1)
        sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, smoothing=0.1)

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


@pytest.mark.parametrize("size", [(1, 64, 3000), (17, 1001, 5000), (96, 256, 20000), (128, 768, 131072), (777, 1000, 9001),
                                  (4096, 128, 70000), (5000, 16, 768100)], ids=str)
def test_what_work_memory_holds_does_not_matter(size):
    """Zeros or NaNs, also between the calls: the same bits."""
    T, H, V = size
    h, W = rand(T, H, "bf16", 1), rand(V, H, "bf16", 2, 2.0 / np.sqrt(H))
    y, dloss = draw_targets(T, V, 3), torch.rand(T, device="cuda")
    got = []
    for fill in (0, 255):
        out = [torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(h), torch.empty_like(W)]
        for backward in (False, True):
            work = torch.full((sg.sg_softmax_ce_work(h, W, backward),), fill, dtype=torch.uint8, device="cuda")
            if backward:
                sg.sg_softmax_ce_bwd(h, W, y, out[1], dloss, out[2], out[3], smoothing=0.1, work=work)
            else:
                sg.sg_softmax_ce_fwd(h, W, y, out[0], out[1], smoothing=0.1, work=work)
        got.append(out)
    for a, b in zip(*got):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


def gradients64(h, W, y, lse, dloss, smoothing, rows, labels):
    """dh, dW in 64 bits on the device, in pieces of that many rows and labels,
    and their sums with the absolute values of g's parts."""
    T, V = h.shape[0], W.shape[0]
    dh, dhm = (torch.zeros(h.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    dW, dWm = (torch.zeros(W.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for t0 in range(0, T, rows):
        t = slice(t0, t0 + rows)
        hd, yt = h[t].double(), y[t].long()
        c = torch.where(yt >= 0, dloss[t].double(), 0.0)[:, None]
        for v0 in range(0, V, labels):
            v = slice(v0, v0 + labels)
            w = W[v].double()
            p = torch.exp(hd @ w.t() - lse[t][:, None])
            hit = torch.zeros_like(p)
            here = (yt >= v0) & (yt < v0 + labels)
            hit.scatter_(1, (yt - v0).clamp(0, p.shape[1] - 1)[:, None], here.double()[:, None] * (1 - smoothing))
            g, mag = (p - hit - smoothing / V) * c, (p + hit + smoothing / V) * c
            dh[t] += g @ w
            dW[v] += g.t() @ hd
            dhm[t] += mag @ w.abs()
            dWm[v] += mag.t() @ hd.abs()
    return dh, dW, dhm, dWm


def test_weight_gradients_of_very_many_rows():
    """Sums of 2^21 products of one sign.  The tensor cores' accumulator rounds
    toward zero, by 2^-24 of the sum so far on average for a step of 16 of them;
    the sum so far is half the sum on average: 2^-13 where 65536 are summed
    there (fewer are), 2^-8 if all of them were."""
    T, H, V, targets = (1 << 21) + 77, 64, 100, 5
    h, W = rand(T, H, "f16", 1).abs(), rand(V, H, "f16", 2, 2.0 / np.sqrt(H))
    y = draw_targets(T, targets, 3)
    loss, lse, dloss = (torch.full((T,), 64.0 / T, device="cuda") for _ in range(3))
    dh, dW, status = torch.empty_like(h), torch.empty_like(W), torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_softmax_ce_fwd(h, W, y, loss, lse, status=status)
    sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, status=status)
    _, lse64, e = forward64(h, W, y, 0.0)
    want_h, want, mag_h, mag = gradients64(h, W, y, lse64, dloss, 0.0, 1 << 18, V)
    assert int(status) == 0
    rest = 2 * float(e.max()) + 3e-5
    err = (dW.double() - want)[targets:].norm() / want[targets:].norm()
    assert float(err) <= U["f16"] + rest + 2.0 ** -13
    # dh is below f16's normal numbers: half its smallest step
    err, least = (dh.double() - want_h).norm(), LEAST["f16"] * np.sqrt(want_h.numel())
    assert float(err) <= U["f16"] * float(want_h.norm()) + rest * float(mag_h.norm()) + least


@pytest.mark.parametrize("T,H,V", [(1, 64, 4861730), (300, 1024, 417619), (1000, 2048, 136845)])
def test_feature_gradients_of_long_sums(T, H, V):
    """More than 65536 labels to a piece of dh's sum; the last size with a second
    piece of the vocabulary."""
    h, W = rand(T, H, "f16", 1), rand(V, H, "f16", 2, 2.0 / np.sqrt(H))
    y = draw_targets(T, V, 3, 0.0)
    loss, lse, dloss = (torch.full((T,), 1.0 / T, device="cuda") for _ in range(3))
    dh, dW, status = torch.empty_like(h), torch.empty_like(W), torch.zeros(1, dtype=torch.int32, device="cuda")
    sg.sg_softmax_ce_fwd(h, W, y, loss, lse, smoothing=0.1, status=status)
    sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, smoothing=0.1, status=status)
    _, lse64, e = forward64(h, W, y, 0.1)
    want_h, want_W, mag_h, mag_W = gradients64(h, W, y, lse64, dloss, 0.1, T, 1 << 16)
    assert int(status) == 0
    rest = 2 * float(e.max()) + 3e-5 + 2.0 ** -13
    for got, want, mag in ((dh, want_h, mag_h), (dW, want_W, mag_W)):
        # an element of dW may be below f16's normal numbers
        bound = U["f16"] * want.norm() + rest * mag.norm() + LEAST["f16"] * np.sqrt(want.numel())
        assert float((got.double() - want).norm()) <= float(bound)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("size", [(1, 1600, 300), (20, 2048, 5000), (100, 4096, 1300), (128, 1544, 3001), (130, 2048, 9753),
                                  (300, 3080, 2500), (700, 5000, 777), (9, 1601, 1000), (200, 2049, 600)], ids=str)
def test_many_features(size, dtype):
    T, H, V = size
    h, W = rand(T, H, dtype, 1), rand(V, H, dtype, 2, 2.0 / np.sqrt(H))
    check(h, W, draw_targets(T, V, 3), torch.rand(T, device="cuda") + 0.5, dtype, 0.1)
