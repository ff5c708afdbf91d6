"""A scan's cluster whose exchange runs out of patience: the waiting CTA reports,
every CTA meets the others before it leaves, and the context stays usable."""
import pytest
import torch

import weight_rnn_gb300 as wr
from weight_rnn_gb300 import build as wbuild


def test_bad_poll_counts_are_refused():
    wbuild.build()
    lib = wr.load_library()
    for polls in (0, -1, (1 << 22) + 1):
        assert lib.delta_selftest_exchange(polls, None) == wr.DELTA_ERR_INVALID


@pytest.mark.gpu
def test_exchange_gives_up_and_reports():
    wr.delta_check_device()  # nothing pending
    x = torch.randn(1, 2000, 64, device="cuda")
    want = wr.delta_scan_fwd(x, x)
    wr.delta_selftest_exchange(polls=1000)
    with pytest.raises(wr.DeltaError, match="scan's cluster gave up") as ei:
        wr.delta_check_device()
    assert ei.value.status == wr.DELTA_ERR_CUDA
    wr.delta_check_device()  # the record was cleared
    got = wr.delta_scan_fwd(x, x)
    for p, q in zip(want, got):
        assert torch.equal(p, q)
