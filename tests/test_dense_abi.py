"""Refusals of the dense attention calls: on the host, before anything is
enqueued (no GPU is touched)."""
import ctypes

import pytest
import torch

import block_sparse_linear_proj_b200 as S
from block_sparse_linear_proj_b200 import build
from block_sparse_linear_proj_b200 import sla as B

FAKE = 1 << 20          # aligned, never dereferenced: validation fails first
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    build.build()
    return S.sla.load()


def pd(**kw):
    a = dict(B=2, H=4, Hk=2, Nq=33, Nk=65, d=64, differential=True)
    a.update(kw)
    return S.dense_params(**a)


def i64(*xs):
    return (ctypes.c_int64 * len(xs))(*xs)


def fwd(lib, p, st=None, q=FAKE, k=FAKE, v=FAKE, lam=FAKE, ql=None, kl=None, out=FAKE, out2=None, lse=None, ws=FAKE,
        n=BIG):
    return lib.sla_diff_forward(ctypes.byref(p), st, q, k, v, lam, ql, kl, out, out2, lse, ws, n, None)


def bwd(lib, p, st=None, ws=FAKE, n=BIG, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, lam=FAKE, ql=None, kl=None, out=FAKE, out2=FAKE, lse=FAKE, dout=FAKE, dq=FAKE,
             dk=FAKE, dv=FAKE, dlam=FAKE)
    a.update(kw)
    return lib.sla_diff_backward(ctypes.byref(p), st, *a.values(), ws, n, None)


def pre(lib, p, st=None, ws=FAKE, n=BIG, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, k=FAKE, v=FAKE, lam=FAKE if p.differential else None, ql=None, kl=None,
             out=FAKE, lse=None)
    a.update(kw)
    return lib.sla_prefix_forward(ctypes.byref(p), st, *a.values(), ws, n, None)


INVALID, UNSUPPORTED, WORKSPACE = B.SLA_ERR_INVALID_ARG, B.SLA_ERR_UNSUPPORTED, B.SLA_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(Nq=0), INVALID), (dict(Nk=-1), INVALID),
    (dict(prefix=-1), INVALID), (dict(d=0), INVALID), (dict(H=5), INVALID), (dict(io_dtype=2), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(sm_scale=float("inf")), INVALID),
    (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(H=131072), UNSUPPORTED),
    (dict(Nq=1 << 28), UNSUPPORTED), (dict(Nk=1 << 30), UNSUPPORTED), (dict(Nk=1 << 29, prefix=1 << 29), UNSUPPORTED),
])
def test_parameters(lib, kw, code):
    p = pd(**kw)
    assert lib.sla_dense_workspace_size(ctypes.byref(p)) == 0
    assert fwd(lib, p) == code and bwd(lib, p) == code and pre(lib, p) == code
    with pytest.raises(S.SlaError):
        S.dense_workspace(p)


def test_gradients_of_more_keys_than_memory_has_room_for(lib):
    p = pd(B=4096, H=64, Hk=64, Nq=1, Nk=1 << 20)
    st = i64(*[64] * 24)
    assert bwd(lib, p, st=st) == UNSUPPORTED


def test_gradients_of_a_scale_beyond_range(lib):
    assert bwd(lib, pd(io_dtype=S.SLA_IO_FP16, sm_scale=2.0 ** -21), n=0) == UNSUPPORTED
    assert bwd(lib, pd(io_dtype=S.SLA_IO_FP16, sm_scale=2.0 ** -20), n=0) == WORKSPACE
    assert bwd(lib, pd(sm_scale=2.0 ** -99), n=0) == WORKSPACE
    assert bwd(lib, pd(sm_scale=2.0 ** -101), n=0) == UNSUPPORTED


def test_null_parameters_and_flags(lib):
    assert lib.sla_dense_workspace_size(None) == 0
    assert lib.sla_diff_forward(None, None, *[FAKE] * 10, BIG, None) == INVALID
    p = pd()
    for name in ("causal", "differential"):
        p = pd()
        setattr(p, name, 2)
        assert fwd(lib, p) == INVALID
    for p in (pd(differential=False), pd(prefix=5)):
        assert fwd(lib, p) == INVALID and bwd(lib, p) == INVALID


def test_pointers(lib):
    p = pd()
    for n in ("q", "k", "v", "lam", "out"):
        assert fwd(lib, p, **{n: None}) == INVALID
    for n in ("q", "k", "v", "out", "out2"):
        assert fwd(lib, p, **{n: FAKE + 8}) == INVALID
    assert fwd(lib, p, lam=FAKE + 1) == INVALID and fwd(lib, p, lse=FAKE + 2) == INVALID
    assert fwd(lib, p, ql=FAKE + 2) == INVALID and fwd(lib, p, kl=FAKE + 2) == INVALID
    for n in ("q", "k", "v", "lam", "out", "out2", "lse", "dout", "dq", "dk", "dv", "dlam"):
        assert bwd(lib, p, **{n: None}) == INVALID
        assert bwd(lib, p, **{n: FAKE + 1}) == INVALID
    pp = pd(prefix=9)
    for n in ("q", "kp", "vp", "k", "v", "lam", "out"):
        assert pre(lib, pp, **{n: None}) == INVALID
    plain = pd(prefix=9, differential=False)
    assert pre(lib, plain, lam=FAKE) == INVALID        # a lambda that would not be read
    for n in ("kp", "vp", "k", "v"):
        assert pre(lib, plain, **{n: FAKE + 4}) == INVALID


def test_workspace(lib):
    for p in (pd(), pd(prefix=100), pd(Nq=1, Nk=100000)):
        need = lib.sla_dense_workspace_size(ctypes.byref(p))
        assert need > 0
        calls = (pre,) if p.P else (fwd, bwd, pre)
        for call in calls:
            assert call(lib, p, n=need - 1) == WORKSPACE
            assert call(lib, p, ws=None) == WORKSPACE
            assert call(lib, p, ws=FAKE + 128) == WORKSPACE


def test_strides(lib):
    d, H, Hk, Nq, Nk = 64, 4, 2, 33, 65
    good = [H * Nq * d, Nq * d, d, Hk * Nk * d, Nk * d, d, Hk * Nk * d, Nk * d, d, H * Nq * d, Nq * d, d]
    p = pd()
    assert fwd(lib, p, st=i64(*good), n=0) == WORKSPACE        # the strides themselves are fine
    for at, bad in ((0, -8), (1, 12), (2, 0), (2, 4), (5, 0), (8, 1 << 36), (9, 0), (10, 0), (11, 0), (11, 56),
                    (10, Nq * d - 8), (9, (H - 1) * Nq * d)):
        st = list(good)
        st[at] = bad
        assert fwd(lib, p, st=i64(*st)) == INVALID, (at, bad)
    # broadcast batch and heads of inputs are fine; [B, N, H, d] outputs too
    st = [0, 0, d, 0, 0, d, 0, Nk * d, d, H * Nq * d, d, H * d]
    assert fwd(lib, p, st=i64(*st), n=0) == WORKSPACE
    # a dimension of one entry: its stride is not read
    one = pd(B=1, Nq=1)
    assert fwd(lib, one, st=i64(3, d, 5, 7, Nk * d, d, -1, Nk * d, d, 1, d, 1), n=0) == WORKSPACE
    b = good + [H * Nq * d, Nq * d, d] * 2 + [Hk * Nk * d, Nk * d, d] * 2
    assert bwd(lib, p, st=i64(*b), n=0) == WORKSPACE
    for at in range(15, 24):        # gradients may not overlap
        st = list(b)
        st[at] = 0
        assert bwd(lib, p, st=i64(*st)) == INVALID, at


def test_binding_refuses(lib):
    p = pd()
    q, k = torch.zeros(2, 4, 33, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 65, 64, dtype=torch.bfloat16)
    if not torch.cuda.is_available():
        a = B._DenseArgs.__new__(B._DenseArgs)
        a.dtype, a.dev, a.strides = torch.bfloat16, 0, []
        with pytest.raises(ValueError):
            a.strided(q, tuple(q.shape), "q")                     # a host tensor
        with pytest.raises(TypeError):
            a.strided(q.half(), tuple(q.shape), "q")
        with pytest.raises(ValueError):
            a.strided(q, (2, 4, 34, 64), "q")
        with pytest.raises(ValueError):
            a.strided(None, tuple(k.shape), "k")
        assert a.strided(None, (2, 0, 64), "k_prefix") is None and a.strides == [0, 0]
        assert B._lse_shape(p) == (2, 4, 2, 33)
