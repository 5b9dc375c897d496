"""Differential attention, its gradients and shared-prefix attention on the GPU
against the 64-bit form in dense_ref.py, within the bounds derived there."""
import pytest
import torch

import block_sparse_linear_proj_b200 as S

import dense_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, dt, *shape, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)


def make(B, H, Hk, Nq, Nk, d, dt="bf16", P=0, diff=True, seed=1, std=1.0, grads=False):
    g, t = gen(seed), DT[dt]
    x = {"q": normal(g, t, B, H, Nq, d, std=std), "k": normal(g, t, B, Hk, Nk, d, mean=0.1),
         "v": normal(g, t, B, Hk, Nk, d)}
    if P:
        x["kp"], x["vp"] = normal(g, t, Hk, P, d), normal(g, t, Hk, P, d)
    if diff:
        x["lam"] = (torch.rand(H, generator=g, device="cuda") * 0.8 + 0.1).to(t)
    if grads:
        x["dout"] = normal(g, t, B, H, Nq, d)
    return x


def lengths(xs):
    return None if xs is None else torch.tensor(xs, dtype=torch.int32, device="cuda")


def par(x, P=0, causal=False, sm_scale=0.0, Nk=None):
    B, H, Nq, d = x["q"].shape
    Hk = x["k"].shape[1] if x.get("k") is not None else x["kp"].shape[0]
    Nk = x["k"].shape[2] if x.get("k") is not None else 0
    return S.dense_params(B, H, Hk, Nq, Nk, d, prefix=P, causal=causal, sm_scale=sm_scale,
                          differential=x.get("lam") is not None,
                          io_dtype=S.SLA_IO_FP16 if x["q"].dtype == torch.float16 else S.SLA_IO_BF16)


def filled(t):
    return torch.full(t.shape, float("nan"), dtype=t.dtype, device=t.device)


def results(p, x):
    return {"out": filled(x["q"]).contiguous(), "out2": filled(x["q"]).contiguous(),
            "lse": torch.full(S.sla._lse_shape(p), float("nan"), device="cuda")}


def forward(x, causal=False, q_len=None, kv_len=None, sm_scale=0.0, ws=None):
    p = par(x, causal=causal, sm_scale=sm_scale)
    r = results(p, x)
    r["p"], r["ws"] = p, S.dense_workspace(p) if ws is None else ws
    r["q_len"], r["kv_len"] = lengths(q_len), lengths(kv_len)
    S.sla_diff_forward(p, x["q"], x["k"], x["v"], x["lam"], r["out"], r["ws"], lse=r["lse"], out2=r["out2"],
                       q_len=r["q_len"], kv_len=r["kv_len"])
    return r


def backward(x, r):
    for n, of in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dlam", "lam")):
        r.setdefault(n, filled(x[of]).contiguous())
    S.sla_diff_backward(r["p"], x["q"], x["k"], x["v"], x["lam"], r["out"], r["out2"], r["lse"], x["dout"], r["dq"],
                        r["dk"], r["dv"], r["dlam"], r["ws"], q_len=r["q_len"], kv_len=r["kv_len"])
    return r


def prefix(x, P, causal=False, q_len=None, kv_len=None):
    p = par(x, P=P, causal=causal)
    r = results(p, x)
    S.sla_prefix_forward(p, x["q"], x.get("kp"), x.get("vp"), x.get("k"), x.get("v"), r["out"], S.dense_workspace(p),
                         lam=x.get("lam"), lse=r["lse"], q_len=lengths(q_len), kv_len=lengths(kv_len))
    return r


def ok():
    assert S.sla_check_device_status() == S.sla.SLA_OK


FWD = [  # B, H, Hk, Nq, Nk, d, dtype, causal, q_len, kv_len
    (1, 1, 1, 1, 1, 64, "bf16", False, None, None),
    (1, 2, 1, 1, 1, 128, "fp16", True, None, None),
    (2, 2, 2, 64, 64, 64, "bf16", False, None, None),
    (1, 2, 2, 128, 128, 128, "bf16", True, None, None),
    (1, 2, 1, 129, 127, 128, "fp16", False, None, None),
    (1, 2, 2, 200, 333, 64, "bf16", True, None, None),
    (1, 1, 1, 300, 200, 128, "bf16", True, None, None),       # the first 100 queries see nothing
    (3, 4, 2, 257, 257, 64, "fp16", True, [257, 100, 0], [257, 100, 0]),
    (3, 2, 2, 130, 500, 128, "bf16", False, [130, 129, 1], [1, 384, 385]),
    (2, 6, 2, 70, 300, 128, "bf16", True, [70, 3], [40, 299]),
    (1, 2, 2, 700, 900, 128, "bf16", False, None, None),
    # single tokens and a few of them against caches
    (1, 1, 1, 1, 5000, 128, "bf16", True, None, None),
    (3, 8, 2, 1, 4097, 64, "fp16", True, None, [4097, 1, 0]),
    (2, 12, 1, 3, 1025, 128, "bf16", True, [3, 2], [1025, 640]),
    (40, 6, 3, 1, 130, 64, "bf16", True, None, None),
]


@pytest.mark.parametrize("c", FWD, ids=lambda c: "-".join(map(str, c[:8])))
def test_diff_forward(c):
    B, H, Hk, Nq, Nk, d, dt, causal, ql, kl = c
    x = make(B, H, Hk, Nq, Nk, d, dt, std=1.5)
    r = forward(x, causal, ql, kl)
    ok()
    R.check(r, R.dense(**x, q_len=ql, kv_len=kl, causal=causal), ("out", "out2", "lse"))


BWD = [
    (1, 1, 1, 1, 1, 64, "bf16", False, None, None),
    (2, 2, 2, 64, 64, 64, "bf16", False, None, None),
    (1, 2, 2, 128, 128, 128, "bf16", True, None, None),
    (1, 2, 2, 256, 256, 128, "fp16", False, None, None),
    (1, 4, 2, 129, 127, 128, "bf16", False, None, None),
    (1, 2, 1, 200, 333, 64, "fp16", True, None, None),
    (1, 1, 1, 300, 200, 128, "bf16", True, None, None),
    (3, 4, 2, 257, 257, 64, "bf16", True, [257, 100, 0], [257, 100, 0]),
    (3, 3, 1, 130, 500, 128, "bf16", False, [130, 129, 1], [1, 384, 385]),
    (2, 6, 2, 70, 300, 128, "fp16", True, [70, 3], [40, 299]),
    (1, 2, 2, 700, 900, 128, "bf16", True, None, None),
    (1, 8, 1, 1, 1000, 64, "bf16", True, None, None),
    (1, 2, 1, 2500, 2500, 64, "fp16", True, None, None),      # long walks; weights near fp16's smallest
    (1, 2, 2, 3, 6000, 128, "fp16", False, None, None),
]


@pytest.mark.parametrize("dt,scale", [("fp16", 2.0 ** -20), ("fp16", 2.0), ("bf16", 2.0 ** -30), ("bf16", 3.0),
                                      ("fp16", 0.01)])
def test_diff_backward_at_scales(dt, scale):
    x = make(1, 2, 1, 150, 200, 64, dt, grads=True, std=0.3)
    r = backward(x, forward(x, True, sm_scale=scale))
    ok()
    R.check(r, R.dense(**x, causal=True, sm_scale=scale), ("out", "dq", "dk", "dv", "dlam"))


@pytest.mark.parametrize("gain", [2.0 ** -12, 2.0 ** 6])
def test_diff_backward_of_small_and_large_gradients(gain):
    """fp16 with dout far from 1: delta reaches some 2^-9 and 2^10, results stay below 65504."""
    x = make(1, 2, 1, 150, 200, 64, "fp16", grads=True, std=0.3)
    x["dout"] = (x["dout"].float() * gain).half()
    r = backward(x, forward(x, True))
    ok()
    R.check(r, R.dense(**x, causal=True), ("out", "dq", "dk", "dv", "dlam"))


@pytest.mark.parametrize("c", BWD, ids=lambda c: "-".join(map(str, c[:8])))
def test_diff_backward(c):
    B, H, Hk, Nq, Nk, d, dt, causal, ql, kl = c
    x = make(B, H, Hk, Nq, Nk, d, dt, grads=True)
    r = backward(x, forward(x, causal, ql, kl))
    ok()
    R.check(r, R.dense(**x, q_len=ql, kv_len=kl, causal=causal), ("out", "dq", "dk", "dv", "dlam"))


PREFIX = [  # B, H, Hk, Nq, Nk, P, d, dtype, causal, diff, q_len, kv_len
    (1, 1, 1, 1, 1, 1, 64, "bf16", False, False, None, None),
    (2, 2, 1, 1, 7, 130, 128, "bf16", True, True, None, None),
    (4, 8, 8, 1, 64, 777, 64, "bf16", True, False, None, None),
    (5, 8, 2, 1, 65, 4100, 128, "fp16", True, False, None, [65, 0, 1, 64, 30]),
    (16, 16, 2, 5, 333, 1000, 64, "fp16", True, False, None, None),
    (3, 6, 3, 40, 90, 300, 128, "bf16", True, True, [40, 1, 0], [90, 1, 0]),
    (2, 2, 2, 300, 300, 500, 128, "bf16", False, False, None, None),
    (2, 3, 3, 260, 260, 129, 64, "bf16", True, True, [260, 77], [260, 77]),
    (2, 4, 4, 400, 140, 128, 128, "bf16", True, False, None, None),
    (2, 2, 1, 150, 300, 0, 64, "bf16", True, False, None, [300, 10]),       # no prefix
    (3, 2, 2, 1, 200, 0, 128, "bf16", True, False, None, [200, 0, 3]),
    (2, 2, 1, 33, 0, 200, 64, "fp16", False, False, None, None),            # the prefix alone
    (2, 2, 2, 200, 0, 200, 128, "bf16", True, True, [200, 5], None),
    (2, 2, 2, 4, 0, 0, 64, "bf16", False, False, None, None),               # nothing at all
    (70, 4, 1, 2, 130, 2000, 128, "bf16", True, False, None, None),
    # few rows against few keys
    (3, 8, 1, 1, 1024, 0, 128, "bf16", True, True, None, [1024, 17, 0]),
    (2, 4, 4, 8, 100, 0, 64, "fp16", True, False, [8, 3], [100, 2]),
    (4, 4, 2, 1, 0, 1000, 128, "bf16", False, True, None, None),
    (3, 6, 3, 1, 15, 900, 64, "bf16", True, True, None, [15, 1, 0]),
    (64, 16, 2, 1, 700, 3000, 128, "fp16", True, True, None, [700 - 11 * i for i in range(64)]),
    (9, 1, 1, 1, 33, 1024, 128, "bf16", True, False, None, None),
    # long walks of a CTA over its keys, in each way the rows can be tiled
    (40, 12, 4, 1, 8192, 0, 128, "bf16", True, False, None, None),
    (50, 12, 4, 1, 6000, 0, 64, "fp16", True, False, None, [6000 - 97 * i for i in range(50)]),
    (2, 160, 160, 1, 100, 5000, 64, "bf16", True, False, None, None),
    (1, 80, 80, 129, 3000, 1000, 128, "bf16", True, False, None, None),
    (40, 12, 4, 1, 5000, 0, 128, "bf16", True, True, None, None),
]


@pytest.mark.parametrize("c", PREFIX, ids=lambda c: "-".join(map(str, c[:10])))
def test_prefix_forward(c):
    B, H, Hk, Nq, Nk, P, d, dt, causal, diff, ql, kl = c
    x = make(B, H, Hk, Nq, Nk, d, dt, P=P, diff=diff, std=1.5)
    if Nk == 0:
        x["kp"] = x.get("kp", torch.zeros((Hk, 0, d), dtype=DT[dt], device="cuda"))
        x["vp"] = x.get("vp", torch.zeros((Hk, 0, d), dtype=DT[dt], device="cuda"))
    r = prefix(x, P, causal, ql, kl)
    ok()
    R.check(r, R.dense(**x, q_len=ql, kv_len=kl, causal=causal), ("out", "lse"))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3.3e38])
@pytest.mark.parametrize("Nq", [200, 1])
def test_padding_is_never_read_into_a_result(bad, Nq):
    ql, kl = ([Nq, max(1, Nq - 77)], [200, 70]) if Nq > 1 else (None, [200, 70])
    x = make(2, 4, 2, Nq, 260, 128, grads=True)
    for b in range(2):
        for n in ("k", "v"):
            x[n][b, :, kl[b]:] = bad
        if ql:
            for n in ("q", "dout"):
                x[n][b, :, ql[b]:] = bad
    r = backward(x, forward(x, True, ql, kl))
    ok()
    R.check(r, R.dense(**x, q_len=ql, kv_len=kl, causal=True), ("out", "out2", "lse", "dq", "dk", "dv", "dlam"))
    y = {**make(2, 4, 2, Nq, 260, 128, P=140), "k": x["k"], "v": x["v"], "q": x["q"]}
    for lam in (y["lam"], None):
        y["lam"] = lam
        R.check(prefix(y, 140, True, ql, kl), R.dense(**y, q_len=ql, kv_len=kl, causal=True), ("out", "lse"))
    ok()


def test_strided_views_of_fused_projections():
    """q, k, v, and their gradients, as slices of [B, N, 3, H, d]; out and dout as [B, N, H, d]."""
    B, N, H, d = 2, 190, 3, 128
    g = gen(5)
    qkv = normal(g, torch.bfloat16, B, N, 3, H, d)
    grad = filled(qkv)
    x = {n: qkv[:, :, i].transpose(1, 2) for i, n in enumerate("qkv")}
    x["lam"] = torch.full((H,), 0.4, device="cuda").bfloat16()
    x["dout"] = normal(g, torch.bfloat16, B, N, H, d).transpose(1, 2)
    p = par(x, causal=True)
    r = results(p, x)
    r["out"] = filled(x["dout"]).contiguous().transpose(1, 2).contiguous().transpose(1, 2)
    r.update(p=p, ws=S.dense_workspace(p), q_len=None, kv_len=None)
    for i, n in enumerate(("dq", "dk", "dv")):
        r[n] = grad[:, :, i].transpose(1, 2)
    S.sla_diff_forward(p, x["q"], x["k"], x["v"], x["lam"], r["out"], r["ws"], lse=r["lse"], out2=r["out2"])
    backward(x, r)
    ok()
    R.check(r, R.dense(**x, causal=True), ("out", "dq", "dk", "dv", "dlam"))
    # the same values in dense tensors: the same bits
    y = {n: t.contiguous() for n, t in x.items()}
    s = backward(y, forward(y, True))
    for n in ("out", "dq", "dk", "dv", "dlam"):
        assert torch.equal(r[n], s[n]), n


def test_broadcast_inputs():
    """Keys and values shared by the batch through a stride of 0."""
    x = make(3, 4, 2, 100, 150, 64, grads=True)
    x["k"], x["v"] = (x[n][:1].expand(3, -1, -1, -1) for n in "kv")
    x["q"] = x["q"][:, :1].expand(-1, 4, -1, -1)
    r = backward(x, {**forward(x), "dk": filled(x["k"].contiguous()), "dv": filled(x["v"].contiguous()),
                     "dq": filled(x["q"].contiguous())})
    ok()
    R.check(r, R.dense(**x), ("out", "out2", "lse", "dq", "dk", "dv", "dlam"))


def test_large_logits_and_a_scale():
    x = make(1, 2, 2, 150, 260, 128, std=12.0)
    R.check(forward(x, sm_scale=0.3), R.dense(**x, sm_scale=0.3), ("out", "out2"))
    x = make(1, 2, 2, 1, 5000, 128, std=12.0)
    R.check(forward(x), R.dense(**x), ("out", "out2"))
    ok()


def test_equal_calls_give_equal_bits_and_streams_do_not_mix():
    xs = [make(2, 4, 2, 333, 400, 128, grads=True, seed=s) for s in (1, 2)]
    ref = [backward(x, forward(x, True)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, st in zip(xs, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(backward(x, forward(x, True)))
    torch.cuda.synchronize()
    ok()
    for a, b in zip(ref, got):
        for n in ("out", "out2", "lse", "dq", "dk", "dv", "dlam"):
            assert torch.equal(a[n], b[n]), n


def test_captured_step_replays_on_new_values():
    x = make(2, 4, 2, 150, 150, 64, grads=True)
    y = {**make(5, 8, 2, 1, 70, 64, P=600, diff=False)}
    p = par(y, P=600, causal=True)
    o, lse, ws = filled(y["q"]), torch.empty(5, 8, 1, device="cuda"), S.dense_workspace(p)

    def step(r):
        S.sla_diff_forward(r["p"], x["q"], x["k"], x["v"], x["lam"], r["out"], r["ws"], lse=r["lse"], out2=r["out2"],
                           q_len=r["q_len"], kv_len=r["kv_len"])
        backward(x, r)
        S.sla_prefix_forward(p, y["q"], y["kp"], y["vp"], y["k"], y["v"], o, ws, lse=lse)

    r = forward(x, True, [150, 60], [150, 60])
    step(backward(x, r))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(r)
    for t in (x["q"], y["q"]):
        t.mul_(-0.5)
    for t in (r["q_len"], r["kv_len"]):
        t.copy_(torch.tensor([90, 150], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    ok()
    R.check(r, R.dense(**x, q_len=[90, 150], kv_len=[90, 150], causal=True), ("out", "dq", "dk", "dv", "dlam"))
    R.check({"out": o, "lse": lse}, R.dense(**y, causal=True), ("out", "lse"))


def test_lengths_out_of_range_are_taken_in_and_flagged():
    x = make(3, 2, 2, 40, 90, 64, grads=True)
    r = forward(x, True, [41, -1, 40], [90, 91, -5])
    assert S.sla_check_device_status() == S.sla.SLA_ERR_DEVICE_CHECK
    backward(x, r)
    assert S.sla_check_device_status() == S.sla.SLA_ERR_DEVICE_CHECK
    R.check(r, R.dense(**x, q_len=[40, 0, 40], kv_len=[90, 90, 0], causal=True),
            ("out", "out2", "lse", "dq", "dk", "dv", "dlam"))


def test_training_and_serving_agree():
    """One differential layer: the whole sequence at once with its gradients; then the same rows served from a
    shared prefix, first as a chunk, then token by token from a growing cache."""
    B, H, Hk, P, N, d = 3, 4, 2, 300, 9, 128
    x = make(B, H, Hk, P + N, P + N, d, grads=True)
    for n in ("q", "k", "v"):      # the sequences begin alike
        x[n][:, :, :P] = x[n][:1, :, :P]
    full = backward(x, forward(x, True))
    ref = R.dense(**x, causal=True)
    R.check(full, ref, ("out", "dq", "dk", "dv", "dlam"))
    y = {"kp": x["k"][0, :, :P], "vp": x["v"][0, :, :P], "lam": x["lam"], "q": x["q"][:, :, P:], "k": x["k"][:, :, P:],
         "v": x["v"][:, :, P:]}
    tail = {"out": ref["out"][:, :, P:], "lse": ref["lse"][..., P:],
            "tol": {n: ref["tol"][n][:, :, P:] if n == "out" else ref["tol"][n][..., P:] for n in ("out", "lse")}}
    R.check(prefix(y, P, True), tail, ("out", "lse"))
    kv = torch.zeros(B, dtype=torch.int32, device="cuda")
    for t in range(N):
        one = {**y, "q": y["q"][:, :, t:t + 1]}
        p = par(one, P=P, causal=True)
        r = results(p, one)
        kv += 1
        S.sla_prefix_forward(p, one["q"], y["kp"], y["vp"], y["k"], y["v"], r["out"], S.dense_workspace(p),
                             lam=y["lam"], lse=r["lse"], kv_len=kv)
        row = {"out": tail["out"][:, :, t:t + 1], "lse": tail["lse"][..., t:t + 1],
               "tol": {"out": tail["tol"]["out"][:, :, t:t + 1], "lse": tail["tol"]["lse"][..., t:t + 1]}}
        R.check(r, row, ("out", "lse"))
    ok()


def test_gradients_against_differences():
    """fp16 forward differences along one direction: (f(x + h r) - f(x - h r)) / 2h with f = sum(out . dout).
    With |out| errors of u (P|v| + |out|) at both ends the quotient is off by at most sum |dout| tol / h, and by the
    third-order term, small against it for this h."""
    x = make(1, 2, 1, 90, 120, 64, "fp16", grads=True)
    x["dout"] = (x["dout"] * 0.25).half()
    r = backward(x, forward(x, True))
    tol = R.dense(**x, causal=True)["tol"]["out"]
    h, g = 2.0 ** -3, gen(9)
    for n, of in (("dq", "q"), ("dk", "k"), ("dv", "v")):
        step = torch.sign(torch.randn(x[of].shape, generator=g, device="cuda"))
        ends = []
        for s in (h, -h):
            y = {**x, of: (x[of].float() + s * step).half()}
            moved = y[of].double() - x[of].double()
            ends.append((y, moved))
        f = [(forward(y, True)["out"].double() * x["dout"].double()).sum() for y, _ in ends]
        want = ((ends[0][1] - ends[1][1]) * r[n].double()).sum()
        exact = [(R.dense(**y, causal=True)["out"] * x["dout"].double()).sum() for y, _ in ends]
        third = (exact[0] - exact[1] - ((ends[0][1] - ends[1][1]) * R.dense(**x, causal=True)[n]).sum()).abs()
        bound = 2.2 * (x["dout"].double().abs() * tol).sum() + third
        assert (f[0] - f[1] - want).abs() <= bound + 2.0 ** -10 * want.abs(), (n, f, want, bound)
    ok()


@pytest.mark.parametrize("Nq,Nk,P", [(300, 300, 500), (1, 1300, 1500)])
def test_waits_that_run_out_are_reported_and_the_context_survives(Nq, Nk, P, monkeypatch):
    """With the test hook the loaders issue no loads, so the consumers' bounded waits (2 ms here) run out: a
    status, no fault, and the next call is right."""
    x = make(2, 4, 2, Nq, Nk, 128, grads=True)
    y = make(3, 4, 2, Nq, 200, 64, P=P, diff=False)
    r = backward(x, forward(x, True))
    ok()
    monkeypatch.setenv("SLA_DEBUG_STALL", "1")
    monkeypatch.setenv("SLA_DEBUG_WAIT_LIMIT_NS", "2000000")
    forward(x, True)
    assert S.sla_check_device_status() == S.sla.SLA_ERR_TIMEOUT
    backward(x, dict(r))
    assert S.sla_check_device_status() == S.sla.SLA_ERR_TIMEOUT
    prefix(y, P, True)
    assert S.sla_check_device_status() == S.sla.SLA_ERR_TIMEOUT
    monkeypatch.undo()
    r = backward(x, forward(x, True))
    R.check(r, R.dense(**x, causal=True), ("out", "dq", "dk", "dv", "dlam"))
    R.check(prefix(y, P, True), R.dense(**y, causal=True), ("out", "lse"))
    ok()
