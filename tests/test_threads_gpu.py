"""Calls from two host threads whose kernels are one instance with different
amounts of shared memory: the limit that a kernel is given is no call's own."""
import threading

import pytest
import torch

import weight_rnn_gb300 as wr

pytestmark = pytest.mark.gpu


def run_both(calls, n=1500):
    """each call over and over on a thread and a stream of its own"""
    errors, gate = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        gate.wait()
        try:
            for _ in range(n):
                call(stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_norm_of_two_odd_widths():
    # float32 rows of odd width: 16 elements a thread, 98 and 197 KB of rings
    def call(D):
        x, w = torch.randn(2, D, device="cuda"), torch.rand(D, device="cuda")
        return lambda stream: wr.delta_add_rmsnorm_fwd(x, w, x, stream=stream)
    run_both([call(4099), call(8191)])


def test_scans_in_two_cluster_sizes():
    def call(T):
        x, g = torch.randn(1, T, 64, device="cuda").to(torch.bfloat16), torch.rand(1, T, 64, device="cuda")
        return lambda stream: wr.delta_scan_fwd(x, g, form="linear", stream=stream)
    run_both([call(200), call(2200)])  # clusters of 2 and 16


def test_generic_chunks_and_diagnostics():
    def mixer(chunk):
        q, k, v = (torch.randn(1, 32, 1, 64, device="cuda") for _ in range(3))
        beta = torch.rand(1, 32, 1, device="cuda")
        return lambda stream: wr.delta_fwd(q, k / 8, v, beta, chunk=chunk, stream=stream)

    def rank(dk):
        s = torch.randn(1, 1, dk, dk, device="cuda")
        return lambda stream: wr.delta_state_erank(s, stream=stream)
    run_both([mixer(16), mixer(64)], 400)
    run_both([rank(64), rank(128)], 400)
