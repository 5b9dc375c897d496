"""Dense attention at values beyond the usual: lambda far from (0, 1), logits in
the hundreds with their gradients, walks of thousands of queries."""
import pytest
import torch

import dense_ref as R
from test_gpu_dense import backward, forward, make, ok, prefix

pytestmark = pytest.mark.gpu

GRADS = ("out", "out2", "lse", "dq", "dk", "dv", "dlam")


@pytest.mark.parametrize("lam", [0.0, -0.7, 8.0, 900.0])
@pytest.mark.parametrize("d,dt", [(64, "fp16"), (128, "fp16"), (64, "bf16"), (128, "bf16")])
def test_lambda_of_any_size_and_sign(d, dt, lam):
    x = make(2, 4, 2, 150, 260, d, dt, grads=True)
    x["lam"] = torch.full_like(x["lam"], lam)
    x["lam"][1] = 0.5              # a head of the same group
    if abs(lam) > 100:
        x["dout"] = x["dout"] / 64     # (dq, dk of 900 times the usual stay within fp16)
    r = backward(x, forward(x, True, [150, 90], [260, 131]))
    ok()
    R.check(r, R.dense(**x, q_len=[150, 90], kv_len=[260, 131], causal=True), GRADS)
    y = {**make(3, 4, 2, 5, 90, d, dt, P=300), "lam": x["lam"]}
    R.check(prefix(y, 300, True), R.dense(**y, causal=True), ("out", "lse"))
    ok()


@pytest.mark.parametrize("d,dt", [(64, "fp16"), (128, "fp16"), (64, "bf16"), (128, "bf16")])
def test_gradients_at_large_logits(d, dt):
    """Logits of some +-100: a few keys take a row's weight, and log-sum-exps are far from 0."""
    x = make(1, 4, 2, 190, 260, d, dt, grads=True, std=12.0)
    r = backward(x, forward(x, True, sm_scale=0.3))
    ok()
    R.check(r, R.dense(**x, causal=True, sm_scale=0.3), GRADS)


@pytest.mark.parametrize("c", [(1, 2, 1, 5000, 5000, 64, "bf16", True), (1, 1, 1, 4500, 5100, 128, "bf16", False),
                               (1, 2, 1, 4100, 3000, 128, "fp16", True)], ids=lambda c: "-".join(map(str, c)))
def test_gradients_of_long_walks(c):
    x = make(*c[:7], grads=True)
    r = backward(x, forward(x, c[7]))
    ok()
    R.check(r, R.dense(**x, causal=c[7]), GRADS)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_gradients_without_keys(dt):
    """No own keys at all: zeros, and dlambda too."""
    x = make(3, 4, 2, 70, 0, 64, dt, grads=True)
    r = backward(x, forward(x, True))
    ok()
    for n in ("out", "out2", "dq", "dlam"):
        assert (r[n] == 0).all(), n
    assert torch.isneginf(r["lse"]).all() and r["dk"].numel() == 0
