"""Dense attention where fp16's range is what decides: small weights beside a
dominating one."""
import math

import pytest
import torch

import dense_ref as R
from test_gpu_dense import forward, ok, prefix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_fp16_small_weights_of_a_long_cache_count(d, diff):
    """One key of logit L and N of logit 0, as beside an attention sink: the others' weights are e^-17.5 = 2^-25.2
    each, their share of the result N e^-17.5.  A weight is rounded to half of 2^-24 of 2^7 at worst (2^-32), the
    result to u."""
    B, N, L, u = 150, 65536, 17.5, 2.0 ** -11
    e = d // 2 if diff else d
    q = torch.zeros(B, 1, 1, d, device="cuda", dtype=torch.float16)
    k = torch.zeros(1, 1, N + 1, d, device="cuda", dtype=torch.float16)
    v = torch.ones(1, 1, N + 1, d, device="cuda", dtype=torch.float16)
    q[..., 0] = 4.0
    k[:, :, 0, 0] = L * e ** 0.5 / 4.0
    v[:, :, 0] = 0.0
    x = {"q": q, "k": k.expand(B, -1, -1, -1), "v": v.expand(B, -1, -1, -1)}
    if diff:
        x["lam"] = torch.zeros(1, device="cuda", dtype=torch.float16)
    r = forward(x) if diff else prefix(x, 0)
    ok()
    ok()
    logit = 4.0 * float(k[0, 0, 0, 0]) * e ** -0.5
    rest = N * math.exp(-logit)
    want = rest / (1 + rest)
    assert (r["out"].double() - want).abs().max() <= N * 2.0 ** -32 + (u + R.SLACK) * want + 2.0 ** -25
    lse = r["lse"][:, :, 0] if diff else r["lse"]
    assert (lse.double() - (logit + math.log1p(rest))).abs().max() <= 2.0 ** -19 * 22
