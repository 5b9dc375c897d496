"""The 64-bit dense attention the GPU tests compare with, pinned on the CPU:
against torch's own softmax attention and autograd, and against differences."""
import math

import pytest
import torch

import dense_ref as R


def make(B, H, Hk, Nq, Nk, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return n(B, H, Nq, d), n(B, Hk, Nk, d), n(B, Hk, Nk, d), torch.rand(H, generator=g, dtype=torch.float64), n(B, H, Nq, d)


def by_torch(q, k, v, lam, ql, kl, causal):
    B, H, Nq, d = q.shape
    G, Nk, e = H // k.shape[1], k.shape[2], d // 2
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    i, j = torch.arange(Nq)[None, :, None], torch.arange(Nk)[None, None]
    qn, kn = torch.tensor(ql)[:, None, None], torch.tensor(kl)[:, None, None]
    see = (j < kn) & (i < qn) & ((j <= i + kn - qn) if causal else torch.ones(1, dtype=torch.bool))
    some = see.any(-1)[:, None, :, None]
    mask = torch.where(see | ~see.any(-1, keepdim=True), 0.0, -math.inf)[:, None].double()
    o = [torch.nn.functional.scaled_dot_product_attention(q[..., s], kk[..., s], vv, attn_mask=mask) * some
         for s in (slice(0, e), slice(e, d))]
    return o[0] - lam[:, None, None] * o[1]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("c", [(2, 4, 2, 5, 7, 8), (1, 2, 2, 6, 3, 4), (2, 3, 1, 1, 9, 8)])
def test_forward_and_gradients_against_torch(c, causal):
    q, k, v, lam, do = make(*c)
    ql, kl = [c[3], max(0, c[3] - 4)][:c[0]], [c[4], 2][:c[0]]
    leaves = [t.clone().requires_grad_() for t in (q, k, v, lam)]
    out = by_torch(*leaves, ql, kl, causal)
    for b in range(c[0]):
        do[b, :, ql[b]:] = 0
    g = torch.autograd.grad(out, leaves, do)
    r = R.dense(q, k, v, lam, q_len=ql, kv_len=kl, causal=causal, dout=do)
    for n, t in zip(("out", "dq", "dk", "dv", "dlam"), (out, *g)):
        assert torch.allclose(r[n], t, atol=1e-11), n


def test_gradients_against_differences():
    q, k, v, lam, do = make(1, 2, 1, 4, 5, 8)
    r = R.dense(q, k, v, lam, causal=True, dout=do)
    x = {"q": q, "k": k, "v": v, "lam": lam}
    for n in x:
        for at in range(0, x[n].numel(), 3):
            f = []
            for s in (1e-6, -1e-6):
                y = {**x, n: x[n].clone()}
                y[n].view(-1)[at] += s
                f.append((R.dense(**y, causal=True)["out"] * do).sum())
            assert abs((f[0] - f[1]) / 2e-6 - r["d" + n].view(-1)[at]) < 1e-7, (n, at)


def test_prefix_is_concatenation():
    q, k, v, lam, _ = make(2, 4, 2, 3, 6, 8)
    kp, vp = k[0, :, :4].clone(), v[0, :, :4].clone()
    cat = lambda a, b: torch.cat([a.expand(2, -1, -1, -1), b], 2)  # noqa: E731
    for la in (lam, None):
        a = R.dense(q, k, v, la, kp=kp, vp=vp, causal=True)
        b = R.dense(q, cat(kp, k), cat(vp, v), la, causal=True)
        assert torch.allclose(a["out"], b["out"], atol=1e-12) and torch.allclose(a["lse"], b["lse"], atol=1e-12)


def test_rows_that_see_nothing():
    q, k, v, lam, do = make(1, 2, 2, 5, 3, 8)
    r = R.dense(q, k, v, lam, causal=True, dout=do)
    assert (r["out"][:, :, :2] == 0).all() and torch.isinf(r["lse"][..., :2]).all() and (r["dq"][:, :, :2] == 0).all()
