"""Cases of the dense attention operators: differential attention (training step,
inference forward, single tokens) and attention for a batch that shares a prefix.

Differential attention splits a head of dimension d into two halves, each with a
softmax map of its own, and weighs the second map by a learned lambda per head:
    O = softmax(tau q1 k1^T) v - lambda softmax(tau q2 k2^T) v,   tau = 1/sqrt(d/2).
Shared-prefix attention: every sequence of a batch attends to the same P prefix
keys and then to its own; tau = 1/sqrt(d) (or the differential form).
Own keys past kv_len[b] and queries past q_len[b] are padding; with the causal mask
the q_len[b] queries are the last q_len[b] of the kv_len[b] own keys.  A query that
sees no key, or is padding, has output 0 and log-sum-exp -inf.

A case holds the sizes; `run` is one pass in the plain form or, with `own` set,
through the library's calls.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases
def _case(name, op, B, H, Hk, Nq, Nk, d, dtype, P=0, causal=False, ragged=False, diff=True):
    c = {"op": op, "B": B, "H": H, "Hk": Hk, "Nq": Nq, "Nk": Nk, "P": P, "d": d, "dtype": dtype,
         "causal": causal, "ragged": ragged, "diff": diff}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a training step of a short clip or a text encoder's last layers: launches count
        _case("diff_train_small", "train", 1, 2, 2, 257, 257, 64, "bf16", causal=True),
        # a training step of a bidirectional video block, one latent frame pair per sample
        _case("diff_train_clip", "train", 2, 12, 12, 2048, 2048, 128, "bf16"),
        # a padded causal batch with shared key/value heads
        _case("diff_train_gqa", "train", 4, 16, 4, 1531, 1531, 64, "fp16", causal=True, ragged=True),
        # a training step over a quarter of the 21x30x52 latent grid
        _case("diff_train_large", "train", 1, 12, 12, 8192, 8192, 128, "bf16"),
        # inference over a third of that grid, a length that ends inside a tile
        _case("diff_forward_video", "forward", 1, 12, 12, 10400, 10400, 128, "bf16"),
        # single tokens against caches of different lengths
        _case("diff_decode", "forward", 32, 12, 4, 1, 8192, 128, "bf16", causal=True, ragged=True),
        # a handful of short continuations of one prompt: launches count
        _case("prefix_decode_small", "prefix", 4, 8, 8, 1, 64, 64, "bf16", P=777, causal=True, diff=False),
        # many samples of one long prompt, a token each
        _case("prefix_decode", "prefix", 64, 32, 8, 1, 512, 128, "bf16", P=16384, causal=True, ragged=True,
              diff=False),
        # the next 30x52 latent frame denoised in six variants that share the frames before it
        _case("prefix_frame", "prefix", 6, 12, 12, 1560, 1560, 128, "bf16", P=8190, diff=False),
        # a few drafted tokens per sequence, checked at once
        _case("prefix_draft", "prefix", 16, 16, 2, 5, 333, 64, "fp16", P=4099, causal=True, ragged=True,
              diff=False),
        # single tokens of a differential model on a shared context
        _case("prefix_diff_decode", "prefix", 24, 12, 12, 1, 700, 128, "bf16", P=12000, causal=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["train", "train", "forward", "decode", "prefix", "prefix", "prefix_decode", "prefix_decode"])
    d, dtype = rng.choice([64, 128]), rng.choice(["bf16", "bf16", "fp16"])
    Hk, G = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 1, 2, 3, 4, 8])
    causal, ragged = rng.random() < 0.5, rng.random() < 0.5
    if op in ("train", "forward"):
        N = _log(rng, 60, 5000)
        B = rng.randint(1, max(1, min(4, 150000000 // (Hk * G * N * N))))
        while G > 1 and B * Hk * G * N * N > 300000000:
            G -= 1
        return _case(None, op, B, Hk * G, Hk, N, N, d, dtype, causal=causal, ragged=ragged)
    if op == "decode":
        return _case(None, "forward", _log(rng, 1, 40), Hk * G, Hk, rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 9000), d,
                     dtype, causal=True, ragged=ragged)
    diff = rng.random() < 0.4
    P = _log(rng, 100, 16000)
    if op == "prefix":
        Nq = _log(rng, 7, 1600)
        B = rng.randint(1, max(1, min(8, 80000000 // (Hk * G * Nq * (P + Nq)))))
        return _case(None, "prefix", B, Hk * G, Hk, Nq, Nq + rng.choice([0, 0, 65, 300]), d, dtype, P=P,
                     causal=causal, ragged=ragged, diff=diff)
    return _case(None, "prefix", _log(rng, 1, 64), Hk * G, Hk, 1, _log(rng, 1, 600), d, dtype, P=P,
                 causal=True, ragged=ragged, diff=diff)


def _lens(c):
    """The queries and own keys of each sequence, from the sizes alone."""
    Nq, Nk = c["Nq"], c["Nk"]
    kv = [max(1, Nk - (b * 37 * Nk // 101) % max(1, 3 * Nk // 4)) if c["ragged"] else Nk for b in range(c["B"])]
    # a padded batch of whole sequences has as many queries as keys; a step on caches has all its queries
    qn = [min(Nq, x) for x in kv] if Nq == Nk else [min(Nq, x) if c["causal"] else Nq for x in kv]
    return qn, kv


def work(c):
    qn, kv = _lens(c)
    es, d, H, Hk = 2, c["d"], c["H"], c["Hk"]
    pairs = keys = 0
    for a, n in zip(qn, kv):
        keys += n
        pairs += a * c["P"]
        pairs += a * n - (a * (a - 1) // 2 if c["causal"] else 0)
    rows = sum(qn) * H
    kvb = 2 * (c["P"] + keys) * Hk * d * es
    if c["op"] == "train":     # q, dout in, out, dq out; k, v in, dk, dv out
        return {"bytes": 4 * rows * d * es + 2 * kvb, "flops": pairs * H * d * 16}
    return {"bytes": 2 * rows * d * es + kvb + rows * 4 * (2 if c["diff"] else 1),
            "flops": pairs * H * d * (6 if c["diff"] else 4)}


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    B, H, Hk, Nq, Nk, P, d = (c[x] for x in ("B", "H", "Hk", "Nq", "Nk", "P", "d"))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).add_(mean).to(dt)

    s = {"case": c}
    # a direction shared by the heads' queries and keys, as trained projections have: logits up to about 8
    s["q"] = normal(B, H, Nq, d, mean=0.15, std=1.2)
    s["k"] = normal(B, Hk, Nk, d, mean=0.15)
    s["v"] = normal(B, Hk, Nk, d)
    s["lam"] = (torch.rand(H, generator=g, device="cuda") * 0.6 + 0.2).to(dt) if c["diff"] else None
    s["kp"] = normal(Hk, P, d, mean=0.15) if P else None
    s["vp"] = normal(Hk, P, d) if P else None
    s["dout"] = normal(B, H, Nq, d) if c["op"] == "train" else None
    qn, kv = _lens(c)
    s["q_len"] = torch.tensor(qn, dtype=torch.int32, device="cuda") if min(qn) < Nq else None
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda") if min(kv) < Nk else None
    if own:
        _buffers(s)
    return s


def _buffers(s):
    """What a program that calls the library keeps: the parameters, the workspace and the results' buffers."""
    import block_sparse_linear_proj_b200 as S
    c = s["case"]
    p = S.dense_params(c["B"], c["H"], c["Hk"], c["Nq"], c["Nk"], c["d"], prefix=c["P"], causal=c["causal"],
                       differential=c["diff"], io_dtype=S.SLA_IO_BF16 if c["dtype"] == "bf16" else S.SLA_IO_FP16)
    s["p"], s["ws"] = p, S.dense_workspace(p)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((c["B"], c["H"], 2, c["Nq"]) if c["diff"] else (c["B"], c["H"], c["Nq"]), device="cuda")
    if c["op"] == "train":
        s["out2"] = torch.empty_like(s["q"])
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
        s["dlam"] = torch.empty_like(s["lam"])


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    o = _plain_forward(s, c)
    if c["op"] != "train":
        return {"out": o["out"].to(s["q"].dtype), "lse": o["lse"]}
    return _plain_backward(s, c, o)


def _run_own(s, c):
    import block_sparse_linear_proj_b200 as S
    if c["op"] == "prefix":
        S.sla_prefix_forward(s["p"], s["q"], s["kp"], s["vp"], s["k"], s["v"], s["out"], s["ws"], lam=s["lam"],
                             lse=s["lse"], q_len=s["q_len"], kv_len=s["kv_len"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "forward":
        S.sla_diff_forward(s["p"], s["q"], s["k"], s["v"], s["lam"], s["out"], s["ws"], lse=s["lse"],
                           q_len=s["q_len"], kv_len=s["kv_len"])
        return {"out": s["out"], "lse": s["lse"]}
    S.sla_diff_forward(s["p"], s["q"], s["k"], s["v"], s["lam"], s["out"], s["ws"], lse=s["lse"], out2=s["out2"],
                       q_len=s["q_len"], kv_len=s["kv_len"])
    S.sla_diff_backward(s["p"], s["q"], s["k"], s["v"], s["lam"], s["out"], s["out2"], s["lse"], s["dout"], s["dq"],
                        s["dk"], s["dv"], s["dlam"], s["ws"], q_len=s["q_len"], kv_len=s["kv_len"])
    return {"out": s["out"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dlambda": s["dlam"]}


# ------------------------------------------------------------------ the plain form, in 32 bits
def _rows(x, c):
    """[B, H, Nq, d] as [B, Hk, G * Nq, d]: the query heads of a key/value head side by side."""
    return x.float().reshape(c["B"], c["Hk"], c["H"] // c["Hk"] * c["Nq"], c["d"])


def _visible(s, c):
    """Which own keys a query sees, [B, 1, G * Nq, Nk], and which queries are no padding, [B, 1, G * Nq, 1]."""
    B, Nq, Nk, G = c["B"], c["Nq"], c["Nk"], c["H"] // c["Hk"]
    i, j = torch.arange(Nq, device="cuda")[None, :, None], torch.arange(Nk, device="cuda")[None, None, :]
    full = torch.ones(B, dtype=torch.int32, device="cuda")
    qn = (s["q_len"] if s["q_len"] is not None else full * Nq)[:, None, None]
    kv = (s["kv_len"] if s["kv_len"] is not None else full * Nk)[:, None, None]
    see = (j < kv) & (i < qn)
    if c["causal"]:
        see = see & (j <= i + kv - qn)
    return see.repeat(1, G, 1)[:, None], (i < qn).repeat(1, G, 1)[:, None]


def _map(q, k, kp, see, real, tau):
    """One softmax map over prefix and own keys: its weights and its log-sum-exp, 0 and -inf where nothing is seen."""
    s = (q * tau) @ k.transpose(-1, -2)
    s = s.masked_fill_(~see, -math.inf)
    if kp is not None:
        s = torch.cat([((q * tau) @ kp.transpose(-1, -2)).masked_fill_(~real, -math.inf), s], -1)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(torch.isfinite(m), m, torch.zeros_like(m))).exp_()
    l = p.sum(-1, keepdim=True)
    return p.div_(torch.where(l > 0, l, torch.ones_like(l))), torch.where(l > 0, m + l.log(), m)[..., 0]


def _halves(x, c):
    h = c["d"] // 2
    return (x[..., :h], x[..., h:]) if c["diff"] else (x,)


def _plain_forward(s, c):
    B, H, Nq, P = c["B"], c["H"], c["Nq"], c["P"]
    q, k, v = _rows(s["q"], c), s["k"].float(), s["v"].float()
    kp, vp = (s["kp"].float(), s["vp"].float()) if P else (None, None)
    see, real = _visible(s, c)
    tau = 1.0 / math.sqrt(c["d"] // (2 if c["diff"] else 1))
    kps = _halves(kp, c) if P else (None, None)
    maps = [_map(a, b, e, see, real, tau) for a, b, e in zip(_halves(q, c), _halves(k, c), kps)]
    outs = [p[..., P:] @ v + (p[..., :P] @ vp if P else 0.0) for p, _ in maps]
    lse = torch.stack([x.reshape(B, H, Nq) for _, x in maps], 2)
    if not c["diff"]:
        return {"out": outs[0].reshape(B, H, Nq, -1), "lse": lse[:, :, 0]}
    lam = _lam(s, c)
    return {"out": (outs[0] - lam * outs[1]).reshape(B, H, Nq, -1), "lse": lse, "maps": maps, "outs": outs}


def _lam(s, c):
    """lambda of each row, [1, Hk, G * Nq, 1]."""
    return s["lam"].float().repeat_interleave(c["Nq"]).reshape(1, c["Hk"], -1, 1)


def _plain_backward(s, c, o):
    B, H, Hk, Nq = c["B"], c["H"], c["Hk"], c["Nq"]
    dt, tau = s["q"].dtype, 1.0 / math.sqrt(c["d"] // 2)
    q, k, v, do = _rows(s["q"], c), s["k"].float(), s["v"].float(), _rows(s["dout"], c)
    lam = _lam(s, c)
    (p1, _), (p2, _) = o["maps"]
    do = do * _visible(s, c)[1]
    dp = do @ v.transpose(-1, -2)
    d1 = (do * o["outs"][0]).sum(-1, keepdim=True)
    d2 = (do * o["outs"][1]).sum(-1, keepdim=True)
    dv = (p1 - lam * p2).transpose(-1, -2) @ do
    ds1, ds2 = p1 * (dp - d1) * tau, -lam * p2 * (dp - d2) * tau
    (q1, q2), (k1, k2) = _halves(q, c), _halves(k, c)
    dq = torch.cat([ds1 @ k1, ds2 @ k2], -1).reshape(B, H, Nq, -1)
    dk = torch.cat([ds1.transpose(-1, -2) @ q1, ds2.transpose(-1, -2) @ q2], -1)
    dlam = -d2.double().reshape(B, H, Nq).sum((0, 2))
    return {"out": o["out"].to(dt), "dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt), "dlambda": dlam.to(dt)}


# ------------------------------------------------------------------ the definition, in 64 bits
def _attend(q, keys, values, offset, P, tau):
    """Softmax attention of the queries [G, n, e] over [m, e]; offset: own key i + offset is the last that query i
    sees (None: all)."""
    logits = torch.einsum("gne,me->gnm", q, keys) * tau
    if offset is not None:
        n, m = logits.shape[1:]
        own_key = torch.arange(m, device="cuda") - P
        late = own_key[None, :] > torch.arange(n, device="cuda")[:, None] + offset
        logits = torch.where(late, torch.full((), -math.inf, dtype=logits.dtype, device="cuda"), logits)
    return torch.einsum("gnm,me->gne", torch.softmax(logits, -1), values), torch.logsumexp(logits, -1)


def exact(c, seed):
    s = prepare(c, seed)
    B, H, Hk, Nq, P, d = (c[x] for x in ("B", "H", "Hk", "Nq", "P", "d"))
    G, h = H // Hk, d // 2
    train = c["op"] == "train"
    if sum(a * (n + P) for a, n in zip(*_lens(c))) * H * d > 2e12:
        return None
    x = {n: s[n].double() for n in ("q", "k", "v", "kp", "vp", "lam", "dout") if s[n] is not None}
    out = torch.zeros(B, H, Nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, 2, Nq), -math.inf, dtype=torch.float64, device="cuda")
    dq, dlam = torch.zeros_like(x["q"]), torch.zeros(H, dtype=torch.float64, device="cuda")
    dk, dv = torch.zeros_like(x["k"]), torch.zeros_like(x["v"])
    qn, kv = _lens(c)
    for b in range(B):
        for e in range(Hk):
            heads = slice(e * G, (e + 1) * G)
            n, m = qn[b], kv[b]
            q, k, v = x["q"][b, heads, :n], x["k"][b, e, :m], x["v"][b, e, :m]
            if P:
                k, v = torch.cat([x["kp"][e], k]), torch.cat([x["vp"][e], v])
            off = m - n if c["causal"] else None
            if not c["diff"]:
                out[b, heads, :n], lse[b, heads, 0, :n] = _attend(q, k, v, off, P, d ** -0.5)
                continue
            lam = x["lam"][heads].clone()
            leaves = [t.detach().requires_grad_(train) for t in (q, k, v, lam)]
            q, k, v, lam = leaves
            o1, l1 = _attend(q[..., :h], k[..., :h], v, off, P, h ** -0.5)
            o2, l2 = _attend(q[..., h:], k[..., h:], v, off, P, h ** -0.5)
            o = o1 - lam[:, None, None] * o2
            out[b, heads, :n], lse[b, heads, 0, :n], lse[b, heads, 1, :n] = o.detach(), l1.detach(), l2.detach()
            if train:
                gq, gk, gv, gl = torch.autograd.grad(o, leaves, x["dout"][b, heads, :n])
                dq[b, heads, :n], dk[b, e, :m], dv[b, e, :m] = gq, gk, gv
                dlam[heads] += gl
    if train:
        return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dlambda": dlam}
    return {"out": out, "lse": lse if c["diff"] else lse[:, :, 0]}
