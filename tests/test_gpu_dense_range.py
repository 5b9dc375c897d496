"""Dense attention where fp16's range is what decides: small gradients, small
weights beside a dominating one."""
import math

import pytest
import torch

import block_sparse_linear_proj_b200 as S

import dense_ref as R
from test_gpu_dense import backward, forward, make, ok, prefix

pytestmark = pytest.mark.gpu


def gradients_bound(x, sm_scale=0.0):
    """Gradients of one head in 64 bits, without masks, and how far the library's may be off.  u = 2^-11.
    dS_m, scaled so that the largest it can be lies between 2^14 and 2^15, is rounded relatively (u) or to half of
    2^-24 of that scale, 2^-39 of the bound |dout|_2 |v|_2 + |delta|; W to u or 2^-39 (|lambda| <= 1); delta_m moves
    by |dout| . (the roundings of out and out2: u of them, u of the weights' products, half a subnormal step);
    fp32 sums and exponentials as in dense_ref (SLACK); results to u or 2^-25."""
    u, half = 2.0 ** -11, 2.0 ** -25
    q, k, v, g = (x[n][0, 0].double() for n in ("q", "k", "v", "dout"))
    lam, e = float(x["lam"][0]), q.shape[1] // 2
    tau = sm_scale or e ** -0.5
    maps = [R.attend(q[:, s], k[:, s], v, 0, None, tau)[0] for s in (slice(0, e), slice(e, 2 * e))]
    o = [p @ v for p in maps]
    err = [(u + R.SLACK) * (p @ v.abs()) + u * y.abs() + half + 2.0 ** -32 * v.abs().sum(0) for p, y in zip(maps, o)]
    dP, gv = g @ v.T, g.abs() @ v.abs().T
    delta = [(g * y).sum(-1, keepdim=True) for y in o]
    e2 = (g.abs() * err[1]).sum(-1, keepdim=True) + R.SLACK * (g * o[1]).abs().sum(-1, keepdim=True)
    e1 = (g.abs() * (err[0] + lam * err[1] + u * (o[0] - lam * o[1]).abs())).sum(-1, keepdim=True) + lam * e2
    big = float(g.norm(dim=-1).max() * v.norm(dim=-1).max() + max(d.abs().max() for d in delta))
    W = maps[0] - lam * maps[1]
    r = {"dv": W.T @ g}
    tol = {"dv": (u * W.abs() + R.SLACK * (maps[0] + lam * maps[1]) + 2.0 ** -39).T @ g.abs()}
    dq, tq, dk, tk = [], [], [], []
    for p, dl, ed, w, s in ((maps[0], delta[0], e1, 1.0, slice(0, e)), (maps[1], delta[1], e2, -lam, slice(e, 2 * e))):
        ds = w * p * (dP - dl)
        es = u * ds.abs() + abs(w) * p * (ed + R.SLACK * (gv + dl.abs())) + 2.0 ** -39 * big
        dq.append(tau * (ds @ k[:, s]))
        tq.append(tau * (es @ k[:, s].abs()))
        dk.append(tau * (ds.T @ q[:, s]))
        tk.append(tau * (es.T @ q[:, s].abs()))
    for n, y, t in (("dq", dq, tq), ("dk", dk, tk)):
        r[n], tol[n] = torch.cat(y, -1), torch.cat(t, -1)
    for n in r:
        tol[n] = tol[n] + u * (r[n].abs() + tol[n]) + half
    return r, tol


def within(got, ref, tol, n):
    err = (got[n][0, 0].double() - ref[n]).abs()
    assert (err <= tol[n]).all(), "%s: relative error %.3g, %.3g of the bound" % (
        n, err.norm() / ref[n].norm(), (err / tol[n]).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gain", [2.0 ** -10, 2.0 ** -16])
def test_fp16_gradients_of_long_rows_keep_their_digits(d, gain):
    """4096 keys, so weights of some 2^-12, and a small dout: dS is far below fp16's normal range, dq (with large
    keys) and dk (with large queries) are not."""
    for of, by in (("dq", 16.0), ("dk", 1 / 16)):
        x = make(1, 1, 1, 4096, 4096, d, "fp16", grads=True, seed=3)
        x["q"], x["k"], x["dout"] = x["q"] / by, x["k"] * by, x["dout"] * gain
        r = backward(x, forward(x))
        ok()
        ref, tol = gradients_bound(x)
        assert ref[of].abs().median() > 2 * tol[of].median()     # the bound says something
        for n in ("dq", "dk", "dv"):
            within(r, ref, tol, n)


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_gradients_beside_a_dominating_key(d):
    """The first key takes all but 2^-29 or so of every other key's weight: dv of the others comes from weights far
    below fp16's smallest number."""
    x = make(1, 1, 1, 2048, 600, d, "fp16", grads=True, seed=4)
    e = d // 2
    x["q"] = x["q"] * 0.0625
    x["k"] = x["k"] * 0.0625
    for at in (0, e):
        x["q"][..., at] = 4.0
        x["k"][..., at] = 0.0
        x["k"][:, :, 0, at] = 20.0 * e ** 0.5 / 4.0
    x["dout"] = x["dout"] * 256 + 256
    r = backward(x, forward(x))
    ok()
    ref, tol = gradients_bound(x)
    assert ref["dv"][1:].abs().median() > 2 * tol["dv"][1:].median()
    # (dv of the first key itself is 2048 times 256 and more, past 65504)
    r["dv"], ref["dv"], tol["dv"] = r["dv"][:, :, 1:], ref["dv"][1:], tol["dv"][1:]
    for n in ("dq", "dk", "dv"):
        within(r, ref, tol, n)


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_gradients_of_logits_past_the_type(d):
    """dS of some 10^5 (large values, a large dout), its sums with a small scale within fp16."""
    x = make(1, 1, 1, 150, 200, d, "fp16", grads=True, seed=6)
    x["v"], x["dout"] = x["v"] * 256, x["dout"] * 16384
    r = backward(x, forward(x, sm_scale=2.0 ** -12))
    ok()
    ref, tol = gradients_bound(x, 2.0 ** -12)
    for n in ("dq", "dk", "dv"):
        within(r, ref, tol, n)


@pytest.mark.parametrize("d", [64, 128])
def test_fp16_lambda_past_1000(d):
    x = make(2, 4, 2, 150, 260, d, "fp16", grads=True)
    x["lam"] = torch.tensor([0.5, 12000.0, -5000.0, 0.0], device="cuda").half()
    x["dout"] = x["dout"] / 512
    r = backward(x, forward(x, True, [150, 90], [260, 131]))
    ok()
    R.check(r, R.dense(**x, q_len=[150, 90], kv_len=[260, 131], causal=True), ("out", "out2", "lse", "dq", "dk", "dv", "dlam"))


@pytest.mark.parametrize("of,size,code", [("q", 6000.0, S.sla.SLA_ERR_DEVICE_CHECK), ("q", 4000.0, S.sla.SLA_OK),
                                          ("v", 6000.0, S.sla.SLA_ERR_DEVICE_CHECK), ("v", 2800.0, S.sla.SLA_OK)])
def test_fp16_log_sum_exps_and_deltas_past_their_range_are_flagged(of, size, code):
    """2^29 = 5.4e8: 32 x 6000^2 (a map's q.k) and 64 x 6000^2 (dout.v) are past it, 32 x 4000^2 and 64 x 2800^2 not."""
    x = make(1, 1, 1, 70, 90, 64, "fp16", grads=True)
    for n in ("q", "k") if of == "q" else ("v", "dout"):
        x[n] = torch.full_like(x[n], size)
    r = forward(x, sm_scale=2.0 ** -18)
    assert S.sla_check_device_status() == S.sla.SLA_OK
    backward(x, r)
    assert S.sla_check_device_status() == code
    if code == S.sla.SLA_OK:
        assert all(torch.isfinite(r[n]).all() for n in ("dq", "dk"))


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
