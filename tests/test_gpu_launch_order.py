"""A call's first kernel begins when all that the program has put on the stream
before it has ended.

Kernels of one call may overlap: each waits for the one before it, which waited
for its own.  Behind a kernel of the program's nothing says that it waited for
what came before it, so the first one has to be launched in plain order.  A captured
graph shows the order: the program's kernel is its root, and the edges that leave it
are full dependencies.
"""
import ctypes as C

import pytest
import torch

import extreme_label_sparse_gb300 as sg
from test_gpu_blocks8 import rand, rand8, scales, weights

pytestmark = pytest.mark.gpu

FULL, PROGRAMMATIC = 0, 1  # CUgraphDependencyType


class EdgeData(C.Structure):
    _fields_ = [("from_port", C.c_ubyte), ("to_port", C.c_ubyte), ("type", C.c_ubyte), ("reserved", C.c_ubyte * 5)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    sg.build()


def edges(call):
    """(type of each edge from the graph's root, types of all) of a captured
    kernel of the program's and `call` behind it; nothing is run of either but
    `call` once before."""
    call()
    x = torch.ones(64, device="cuda")
    x.add_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        x.add_(1)
        call()
    cuda = C.CDLL("libcuda.so.1")
    handle, n = C.c_void_p(graph.raw_cuda_graph()), C.c_size_t(0)
    assert cuda.cuGraphGetEdges_v2(handle, None, None, None, C.byref(n)) == 0 and n.value > 0
    first, last, data = (C.c_void_p * n.value)(), (C.c_void_p * n.value)(), (EdgeData * n.value)()
    assert cuda.cuGraphGetEdges_v2(handle, first, last, data, C.byref(n)) == 0
    roots = set(first) - set(last)
    assert len(roots) == 1
    return [d.type for f, d in zip(first, data) if f in roots], [d.type for d in data]


def linear_fwd(T, H, N, shift):
    x8, W8, xs, ws = rand8(T, H, 1, -(H + shift) % 16, shift), rand8(N, H, 2, -(H + shift) % 16, shift), scales(T, 3), scales(N, 4)
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    work = torch.empty(max(1, sg.sg_linear8_work(x8, W8)), dtype=torch.uint8, device="cuda")
    return lambda: sg.sg_linear8_fwd(x8, xs, W8, ws, out, work=work)


def linear_bwd(T, H, N, dtype, shift):
    x8, W8, xs, ws = rand8(T, H, 1), rand8(N, H, 2), scales(T, 3), scales(N, 4)
    dout = rand(T, N, dtype, 5, -(N + shift) % 8, shift)
    dx, dW = (torch.empty(s, dtype=dout.dtype, device="cuda") for s in ((T, H), (N, H)))
    work = torch.empty(sg.sg_linear8_work(x8, W8, dout), dtype=torch.uint8, device="cuda")
    return lambda: sg.sg_linear8_bwd(x8, xs, W8, ws, dout, dx=dx, dW=dW, work=work)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T", [1, 2, 4, 16, 50, 100, 300, 600])
def test_linear_forward(T, shift):
    first, _ = edges(linear_fwd(T, 1024, 700, shift))
    assert set(first) == {FULL}


def test_linear_forward_in_pieces():
    """Later pieces' kernels follow the call's own."""
    first, all_ = edges(linear_fwd(600, 4096, 40000, 0))
    assert set(first) == {FULL} and PROGRAMMATIC in all_


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,N", [(40, 300, 500), (600, 520, 1000), (100, 256, 7000)])
def test_linear_backward(T, H, N, dtype, shift):
    first, all_ = edges(linear_bwd(T, H, N, dtype, shift))
    assert set(first) == {FULL} and PROGRAMMATIC in all_


def test_rows_and_norms():
    x, w = rand(300, 512, "bf16", 1), weights(512, "bf16")
    y, q, s = torch.empty_like(x), torch.empty((300, 512), dtype=torch.int8, device="cuda"), torch.empty((300, 4), device="cuda")
    r, sums = torch.empty((2, 300), device="cuda"), torch.empty((3, 512), device="cuda")
    work = torch.empty(max(sg.sg_block_norm_bwd_work(300, 512), sg.sg_add_rmsnorm_bwd_work(300, 512)), dtype=torch.uint8,
                       device="cuda")
    for call in (lambda: sg.sg_pack8(x, q, s), lambda: sg.sg_unpack8(q, s, y), lambda: sg.sg_dropout(x, 0.1, 1, 2, y),
                 lambda: sg.sg_block_norm_fwd(x, w[0], w[2], 1e-5, gate=w[1], rstd_x=r[0], rstd_u=r[1], y=y),
                 lambda: sg.sg_block_norm_bwd(x, x, x, w[0], w[2], r[0], r[1], y, dpost=sums[0], dpre=sums[1],
                                              dgate=sums[2], gate=w[1], work=work),
                 lambda: sg.sg_add_rmsnorm_fwd(x, w[0], 1e-5, y=y, rstd=r[0]),
                 lambda: sg.sg_add_rmsnorm_bwd(x, x, w[0], r[0], y, dweight=sums[0], work=work)):
        assert set(edges(call)[0]) == {FULL}


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T,V", [(40, 3000), (600, 3000)])
def test_softmax_cross_entropy(T, V, shift):
    h, W = rand(T, 256, "bf16", 1, 8 - shift, shift), rand(V, 256, "bf16", 2, 8 - shift, shift, std=0.1)
    y = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    loss, lse, dloss = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.ones(T, device="cuda")
    dh, dW = torch.empty((T, 256), dtype=h.dtype, device="cuda"), torch.empty((V, 256), dtype=h.dtype, device="cuda")
    work = torch.empty(max(sg.sg_softmax_ce_work(h, W, backward=b) for b in (False, True)), dtype=torch.uint8, device="cuda")
    for call in (lambda: sg.sg_softmax_ce_fwd(h, W, y, loss, lse, work=work),
                 lambda: sg.sg_softmax_ce_bwd(h, W, y, lse, dloss, dh, dW, work=work)):
        assert set(edges(call)[0]) == {FULL}
