"""Dense attention calls on the host: what they take and refuse at the edges of
their sizes (no GPU is touched)."""
import ctypes

import pytest
import torch

import block_sparse_linear_proj_b200 as S
from block_sparse_linear_proj_b200 import sla as B
from test_dense_abi import INVALID, UNSUPPORTED, WORKSPACE, bwd, fwd, i64, lib, pd, pre  # noqa: F401


def test_no_own_keys(lib):  # noqa: F811
    """Nk = 0 is a size like any other: dense tensors (NULL strides), a missing tensor's zeros, whatever strides an
    empty tensor has."""
    p = pd(Nk=0)
    none = dict(k=None, v=None)
    H, Hk, Nq, d = p.H, p.Hk, p.Nq, p.d
    qs = [H * Nq * d, Nq * d, d]
    for e in ([0, 0, 0], [Hk * d, d, d], list(torch.empty(2, Hk, 0, d).stride()[:3]), [-1, 3, 5]):
        assert fwd(lib, p, st=i64(*qs, *e, *e, *qs), n=0, **none) == WORKSPACE
        assert bwd(lib, p, st=i64(*qs, *e, *e, *qs, *qs, *qs, *e, *e), n=0, dk=None, dv=None, **none) == WORKSPACE
    for q in (p, pd(Nk=0, B=1, Hk=1), pd(Nk=0, B=1)):
        assert fwd(lib, q, n=0, **none) == WORKSPACE
        assert bwd(lib, q, n=0, dk=None, dv=None, **none) == WORKSPACE
    # a gradient of queries still may not overlap
    assert bwd(lib, p, st=i64(*qs, *[0] * 6, *qs, *qs, 0, Nq * d, d, *[0] * 6), dk=None, dv=None, **none) == INVALID
