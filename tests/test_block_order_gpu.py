"""Calls that follow one another on a stream without a wait between them: a
kernel may start before the one in front has ended, but reads and writes only
after it.  Every call here reads what the one before wrote, and buffers are
written again at once; the same steps with a synchronize after each are the
comparison, bit by bit."""
import pytest
import torch

import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def steps(rows, D, count, pause):
    gen = torch.Generator().manual_seed(rows + D)
    r = lambda *s: torch.randn(*s, generator=gen)
    w = (r(D, D) / D ** 0.5).to(BF).cuda()
    w8 = w.to(torch.float8_e4m3fn)
    sw, norm = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    stream, state = r(rows, D).to(BF).cuda(), torch.zeros(rows, D, device="cuda")
    buf = torch.empty(rows, D, dtype=BF, device="cuda")
    grad = torch.zeros(D, device="cuda")
    for i in range(count):
        for call in range(6):
            if call == 0:
                buf.copy_(stream).mul_(0.5)
                y, total, rstd = wr.delta_add_rmsnorm_fwd(buf, norm, stream)
            elif call == 1:
                buf.fill_(float("nan"))  # (its old content has been read by now)
                torch.mul(y, 0.75, out=buf)
                h = wr.delta_scan_step(y, buf, state)
            elif call == 2:
                stream = wr.delta_linear_fwd(h, w, None, total, act="silu")
            elif call == 3:
                q, scale, _ = wr.delta_add_rmsnorm_quant(stream, norm)
                stream = wr.delta_linear_quant(q, scale, w8, sw, None, stream)
            elif call == 4:
                dx, dw, db = wr.delta_linear_bwd(h, w, stream)
                stream = wr.delta_add_rmsnorm_fwd(dx, norm, stream)[0]
            else:
                g, dn = wr.delta_add_rmsnorm_bwd(stream, total, norm, rstd)
                grad += dn + db
                buf.copy_(g)
                out, last = wr.delta_scan_fwd(stream.view(1, rows, D), buf.view(1, rows, D))
                stream = out.view(rows, D).add_(dw[0])
            if pause:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    wr.delta_check_device()
    return stream, state, grad


@pytest.mark.parametrize("rows,D,count", [(1, 256, 60), (4, 1024, 60), (16, 257, 40), (300, 512, 40),
                                          (2048, 1024, 10)])
def test_calls_in_a_row(rows, D, count):
    for a, b in zip(steps(rows, D, count, False), steps(rows, D, count, True)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_graph_of_calls():
    rows, D = 4, 512
    x, w = torch.randn(rows, D, device="cuda").to(BF), (torch.randn(D, D, device="cuda") / D ** 0.5).to(BF)
    norm, state = torch.ones(D, device="cuda"), torch.zeros(rows, D, device="cuda")

    def run():
        y, total, _ = wr.delta_add_rmsnorm_fwd(x, norm)
        h = wr.delta_scan_step(y, total, state)
        return wr.delta_linear_fwd(h, w, None, total, act="gelu")

    run()
    state.zero_()
    want = [run() for _ in range(20)][-1]
    end = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    state.zero_()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(state, end)
