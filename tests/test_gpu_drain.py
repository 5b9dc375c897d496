"""A kernel that gives up drains what it has issued and no more: with the
loaders stalled by the test hook (2 ms limit) nothing is in flight that could
hold a kernel for its drain limit of 4 s."""
import time

import pytest
import torch

import block_sparse_linear_proj_b200 as S
from test_gpu_dense import backward, forward, make, ok, prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk,P", [(500, 900, 500), (1, 4000, 3000)])
def test_stalled_calls_end_soon(Nq, Nk, P, d, monkeypatch):
    x = make(2, 4, 2, Nq, Nk, d, grads=True)
    y = make(3, 4, 2, Nq, 200, d, P=P, diff=False)
    r = backward(x, forward(x, True))
    want = prefix(y, P, True)["out"]
    ok()
    monkeypatch.setenv("SLA_DEBUG_STALL", "1")
    monkeypatch.setenv("SLA_DEBUG_WAIT_LIMIT_NS", "2000000")
    copy = {n: t.clone() if torch.is_tensor(t) else t for n, t in r.items()}
    for call in (lambda: forward(x, True), lambda: backward(x, copy), lambda: prefix(y, P, True)):
        t = time.monotonic()
        call()
        assert S.sla_check_device_status() == S.sla.SLA_ERR_TIMEOUT
        assert time.monotonic() - t < 2.0
    monkeypatch.undo()
    again = backward(x, forward(x, True))
    assert torch.equal(prefix(y, P, True)["out"], want)
    ok()
    for n in ("out", "dq", "dk", "dv", "dlam"):
        assert torch.equal(again[n], r[n]), n
