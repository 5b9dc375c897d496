"""Dense attention in 64 bits, one (sequence, head) at a time over its valid
queries and keys, with a bound on what the library's roundings may change.

u = eps / 2 of the I/O type is the relative size of one rounding.  The library
rounds, in io_dtype:
  forward   the softmax weights (relative to their running maximum) and the
            results:  |d out| <= u sum_m |w_m| P_m |v| + u |out|,  w = (1, lambda)
  backward  W = P_1 - lambda P_2, dS_m and the results; and it reads the rounded
            out and out2, which moves delta_m by at most |dout| . (their errors);
            dlambda comes from the unrounded weights.
Everything else is fp32: sums of up to thousands of terms, exponentials and
log-sum-exps, taken as SLACK relative to the sums of magnitudes (2^-13, an
eighth of an fp16 rounding is 2^-14; logits of magnitude 30 alone put
30 * 2^-22 on an exponential, and a fp32 sum of n terms n * 2^-24 at most).
fp16 results below 2^-14 are subnormal: TINY covers half their step for each
rounded factor."""
import math

import torch

SLACK = 2.0 ** -13


def lens(x, B, full):
    return [full] * B if x is None else [int(v) for v in x]


def unit(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def attend(q, k, v, n_prefix, offset, tau):
    """Weights [n, m] and log-sum-exp [n] (0 and -inf where nothing is seen)."""
    s = q @ k.T * tau
    if offset is not None:
        j = torch.arange(k.shape[0], device=q.device) - n_prefix
        i = torch.arange(q.shape[0], device=q.device)
        s = s.masked_fill((j[None, :] > i[:, None] + offset) & (j[None, :] >= 0), -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full((q.shape[0],), -math.inf, dtype=q.dtype, device=q.device)
    p = torch.where(torch.isinf(lse)[:, None], torch.zeros((), dtype=q.dtype, device=q.device), torch.exp(s - lse[:, None]))
    return p, lse


def dense(q, k, v, lam=None, kp=None, vp=None, q_len=None, kv_len=None, causal=False, sm_scale=0.0, dout=None):
    """dict of results (out, out2, lse and, with dout, dq, dk, dv, dlam) and "tol" of the same names."""
    dt, dev = q.dtype, q.device
    u, t0 = unit(dt), tiny(dt)
    B, H, Nq, d = q.shape
    Hk = k.shape[1] if k is not None else kp.shape[0]
    Nk = k.shape[2] if k is not None else 0
    G, M = H // Hk, 2 if lam is not None else 1
    e = d // M
    tau = sm_scale if sm_scale > 0 else 1 / math.sqrt(e)
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=dev)  # noqa: E731
    r = {"out": z(B, H, Nq, d), "out2": z(B, H, Nq, d), "lse": torch.full((B, H, M, Nq), -math.inf, dtype=torch.float64, device=dev)}
    tol = {"out": z(B, H, Nq, d), "out2": z(B, H, Nq, d), "lse": z(B, H, M, Nq)}
    if dout is not None:
        for n, s in (("dq", q.shape), ("dk", k.shape), ("dv", v.shape), ("dlam", (H,))):
            r[n], tol[n] = z(*s), z(*s)
    qn, kn = lens(q_len, B, Nq), lens(kv_len, B, Nk)
    for b in range(B):
        for h in range(H):
            n, m, hk = qn[b], kn[b], h // G
            Q = q[b, h, :n].double()
            K = k[b, hk, :m].double() if Nk else z(0, d)
            V = v[b, hk, :m].double() if Nk else z(0, d)
            P0 = 0
            if kp is not None:
                K, V, P0 = torch.cat([kp[hk].double(), K]), torch.cat([vp[hk].double(), V]), kp.shape[1]
            off = m - n if causal else None
            w = [1.0] + ([float(lam[h])] if M == 2 else [])
            maps = [attend(Q[:, x * e:(x + 1) * e], K[:, x * e:(x + 1) * e], V, P0, off, tau) for x in range(M)]
            o = [p @ V for p, _ in maps]
            mag = [p @ V.abs() for p, _ in maps]
            out = o[0] - w[1] * o[1] if M == 2 else o[0]
            amag = mag[0] + abs(w[1]) * mag[1] if M == 2 else mag[0]
            r["out"][b, h, :n] = out
            tol["out"][b, h, :n] = (u + SLACK) * amag + u * out.abs() + t0 + 1e-30
            for x in range(M):
                r["lse"][b, h, x, :n] = maps[x][1]
                # fp32 logits of magnitude |s| and a sum of l: a few units of 2^-22 of |lse| and of 1
                tol["lse"][b, h, x, :n] = 2.0 ** -19 * (4 + maps[x][1].abs().nan_to_num(0, 0, 0))
            if M == 2:
                r["out2"][b, h, :n] = o[1]
                tol["out2"][b, h, :n] = (u + SLACK) * mag[1] + u * o[1].abs() + t0 + 1e-30
            if dout is None:
                continue
            g = dout[b, h, :n].double()
            (p1, _), (p2, _) = maps
            dP, lm = g @ V.T, w[1]
            gv = g.abs() @ V.abs().T
            d1, d2 = (g * o[0]).sum(-1, keepdim=True), (g * o[1]).sum(-1, keepdim=True)
            e2 = (g.abs() * tol["out2"][b, h, :n]).sum(-1, keepdim=True) + SLACK * (g * o[1]).abs().sum(-1, keepdim=True)
            e1 = (g.abs() * tol["out"][b, h, :n]).sum(-1, keepdim=True) + abs(lm) * e2
            W = p1 - lm * p2
            r["dv"][b, hk, :m] += W.T @ g
            tol["dv"][b, hk, :m] += (u * W.abs() + SLACK * (p1 + abs(lm) * p2) + t0).T @ g.abs()
            dq, tq, dk, tk = [], [], [], []
            for p, dl, ed, ww, x in ((p1, d1, e1, 1.0, 0), (p2, d2, e2, -lm, 1)):
                ds = ww * p * (dP - dl)
                es = u * ds.abs() + abs(ww) * p * (ed + SLACK * (gv + dl.abs())) + t0
                Kx, Qx = K[:, x * e:(x + 1) * e], Q[:, x * e:(x + 1) * e]
                dq.append(tau * (ds @ Kx))
                tq.append(tau * (es @ Kx.abs()))
                dk.append(tau * (ds.T @ Qx))
                tk.append(tau * (es.T @ Qx.abs()))
            r["dq"][b, h, :n] = torch.cat(dq, -1)
            tol["dq"][b, h, :n] = torch.cat(tq, -1)
            r["dk"][b, hk, :m] += torch.cat(dk, -1)
            tol["dk"][b, hk, :m] += torch.cat(tk, -1)
            r["dlam"][h] -= d2.sum()
            tol["dlam"][h] += SLACK * (p2 * gv).sum()
    for n in ("dq", "dk", "dv", "dlam"):
        if n in r:
            tol[n] += u * (r[n].abs() + tol[n]) + t0 + 1e-30
    if M == 1:
        r["lse"], tol["lse"] = r["lse"][:, :, 0], tol["lse"][:, :, 0]
    r["tol"] = tol
    return r


def check(got, ref, names):
    for n in names:
        x, y, t = got[n].double(), ref[n], ref["tol"][n]
        inf = torch.isinf(y)
        assert torch.equal(torch.isinf(x), inf) and not torch.isnan(x).any(), n
        err = torch.where(inf, torch.zeros_like(y), (x - torch.where(inf, torch.zeros_like(y), y)).abs())
        worst = (err - t).max() if err.numel() else 0.0
        at = int((err - t).argmax()) if err.numel() else 0
        assert worst <= 0, "%s: error %.3g, bound %.3g at %d" % (n, err.flatten()[at], t.flatten()[at], at)
        # zeros where nothing is seen are exact
        if n != "lse":
            z = (t <= 2 * max(1e-30, tiny(got[n].dtype))) & (y == 0)
            assert (x[z] == 0).all(), n
