"""Both gradients of a large layer in one launch: that they are where the estimate says so
(kernels are counted in a captured graph), that each has the bits that it has alone, and
every element against 64 bits, in widths of whole 16-byte pieces and odd ones.

A term of dx and dw has dpre rounded to bfloat16, half a step, and the sums are those of the
linear layer: 16 terms at a time on a float32 sum, a step (2 U) of the magnitudes each and
24 for the parts.  Then the output's own half step.  dpre's own value has the logistic
function's error, 2^-19 (1 + |p|)^2 of dout (test_slopes_gpu)."""
import ctypes

import pytest
import torch

import block_ref as ref
import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U, HALF = ref.U, ref.HALF[torch.bfloat16]


def kernels(fn):
    """how many kernels a call launches"""
    fn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        fn()
    driver = ctypes.CDLL("libcuda.so.1")
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert driver.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes, kind = (ctypes.c_void_p * n.value)(), ctypes.c_int()
    assert driver.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    count = 0
    for node in nodes:
        assert driver.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        count += kind.value == 0  # CU_GRAPH_NODE_TYPE_KERNEL
    return count


# what, M, N, K, and whether the two share a launch on 152 SMs
CASES = [("glu", 4096, 4096, 2048, True), ("glu", 2600, 3000, 5000, True), ("glu", 3001, 4100, 2571, True),
         ("glu", 9000, 2048, 1500, False), ("silu", 2601, 3001, 5001, True), ("silu", 2049, 8191, 2047, True),
         ("silu", 9001, 2048, 1501, True), ("silu", 5000, 1300, 4104, False), ("none", 4095, 4096, 2047, True),
         ("none", 2048, 8192, 2048, True)]


@pytest.mark.parametrize("what,M,N,K,joined", CASES)
def test_joined_gradients(what, M, N, K, joined):
    glu, act = what == "glu", "silu" if what == "glu" else what
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF)  # noqa: E731
    rows = 2 * N if glu else N
    x, do, w = r(M, K), r(M, N), r(rows, K)
    pre = None if act == "none" else r(M, rows)
    fn = wr.delta_glu_bwd if glu else wr.delta_linear_bwd
    call = lambda *want: fn(x, w, do, pre, act=act, want=want)  # noqa: E731
    got, dx, dw = call(True, True, False), call(True, False, False)[0], call(False, True, False)[1]
    wr.delta_check_device()
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        form = int(act != "none" or N % 8 != 0)  # the pass that forms dpre, once for both
        apart = kernels(lambda: call(True, False, False)) + kernels(lambda: call(False, True, False)) - form
        assert kernels(lambda: call(True, True, False)) == apart - joined
    d = do.double()
    if act == "none":
        dpre, loose = d, torch.zeros_like(d)
    else:
        p = pre.double().requires_grad_(True)
        value = ref.act(act, p[:, :N]) * p[:, N:] if glu else ref.act(act, p)
        (dpre,) = torch.autograd.grad(value, p, d)
        one = 2.0 ** -19 * (1.0 + p.detach()[:, :N].abs()) ** 2 * d.abs()
        loose = torch.cat([one * p.detach()[:, N:].abs(), one], 1) if glu else one
        loose = loose + 4 * U * dpre.abs()
        loose = loose + HALF * (dpre.abs() + loose)
    for name, g, a, e, b in (("dx", got[0], dpre, loose, w.double()), ("dw", got[1], dpre.T, loose.T, x.double())):
        want = a @ b
        bound = 2 * U * (a.shape[1] / 16 + 24) * (a.abs() @ b.abs()) + 1.01 * (e @ b.abs())
        bound += HALF * (want.abs() + bound)
        assert ((g.double() - want).abs() <= bound).all(), name
        del want, bound
