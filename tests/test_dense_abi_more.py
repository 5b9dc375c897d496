"""Dense attention calls on the host: what they take and refuse at the edges of
their sizes (no GPU is touched)."""
import ctypes

import torch

from test_dense_abi import INVALID, WORKSPACE, bwd, fwd, i64, lib, pd, pre  # noqa: F401


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


def test_workspace_of_a_prefix_call_holds_its_parts_only(lib):  # noqa: F811
    """The backward call refuses a prefix, so a differential prefix call needs its parts, twice the plain call's (a
    part a map), and nothing for gradients; without a prefix the size covers them."""
    for kw in (dict(B=1024, H=32, Hk=8, Nq=1, Nk=128, d=128, prefix=4096), dict(B=3, H=8, Hk=2, Nq=5, Nk=0, prefix=900),
               dict(B=2, H=4, Hk=4, Nq=300, Nk=300, prefix=500)):
        need = {x: lib.sla_dense_workspace_size(ctypes.byref(pd(differential=x, **kw))) for x in (False, True)}
        assert 0 < need[True] <= 2 * need[False] + 512
        assert pre(lib, pd(**kw), n=need[True] - 1) == WORKSPACE
    a, b = (lib.sla_dense_workspace_size(ctypes.byref(pd(B=40, H=4, Hk=4, Nq=300, Nk=300, prefix=x))) for x in (0, 1))
    assert b == 256 and bwd(lib, pd(B=40, H=4, Hk=4, Nq=300, Nk=300), n=a - 1) == WORKSPACE


def test_strides_whose_extent_passes_64_bits(lib):  # noqa: F811
    """2^29 tokens 2^35 elements apart span 2^64: no tensor, and no room below a batch stride of 2^33."""
    p = pd(B=2, H=1, Hk=1, Nq=1, Nk=1 << 29)
    d, big = p.d, 1 << 35
    st = [d, 0, 0, 0, 0, d, 0, 0, d, d, 0, 0, d, 0, 0, d, 0, 0]
    assert bwd(lib, p, st=i64(*st, 1 << 33, 0, big, 1 << 33, 0, big), n=0) == INVALID
    assert bwd(lib, p, st=i64(*st, p.Nk * d, 0, d, p.Nk * d, 0, d), n=0) == WORKSPACE


def test_three_key_tiles_are_not_split(lib):  # noqa: F811
    """A call in one part has no workspace beyond the least; four tiles of few rows are two ranges."""
    a, b = (pd(B=1, H=2, Hk=2, Nq=257, Nk=n, differential=False) for n in (3 * 128, 3 * 128 + 1))
    assert lib.sla_dense_workspace_size(ctypes.byref(a)) == 256 < lib.sla_dense_workspace_size(ctypes.byref(b))
