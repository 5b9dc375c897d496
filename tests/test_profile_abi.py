"""The tracing calls write as many entries as their caller has room for (host
side: without recorded launches no device is touched)."""
import ctypes
import os
import re

import pytest

from block_sparse_linear_proj_b200 import build
from block_sparse_linear_proj_b200 import sla as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def kinds(name):
    return int(re.search(r"\b%s = (\d+)" % name, open(os.path.join(ROOT, "include", "sla.h")).read()).group(1))


def arrays(n):
    return (ctypes.c_double * n)(*[-1.0] * n), (ctypes.c_int64 * n)(*[-1] * n)


def test_arrays_of_a_program_compiled_against_twelve_kinds(lib):
    ms, cnt = arrays(16)
    assert lib.sla_profile_read(ctypes.addressof(ms), ctypes.addressof(cnt)) == B.SLA_OK
    assert list(ms) == [0.0] * 12 + [-1.0] * 4 and list(cnt) == [0] * 12 + [-1] * 4
    assert kinds("SLA_KERNEL_KINDS") == 12 and lib.sla_version() >= 300


@pytest.mark.parametrize("n", [0, 1, 12, 14, 16])
def test_as_many_kinds_as_asked_for(lib, n):
    ms, cnt = arrays(20)
    assert lib.sla_profile_read_kinds(n, ctypes.addressof(ms), ctypes.addressof(cnt)) == B.SLA_OK
    assert list(ms) == [0.0] * n + [-1.0] * (20 - n) and list(cnt) == [0] * n + [-1] * (20 - n)
    assert lib.sla_profile_read_kinds(n, None, None) == B.SLA_OK


def test_binding_reads_every_kind(lib):
    assert len(B.KERNEL_KINDS) == kinds("SLA_KERNEL_KINDS_ALL")
    assert set(B.sla_profile_read()) == set(B.KERNEL_KINDS)
    assert lib.sla_profile_read_kinds(-1, None, None) == B.SLA_ERR_INVALID_ARG


@pytest.mark.gpu
def test_dense_launches_are_counted(lib):
    import torch

    import block_sparse_linear_proj_b200 as S
    p = S.dense_params(1, 2, 2, 40, 40, 64, differential=True)
    q, k, v, out = (torch.randn(1, 2, 40, 64, device="cuda").bfloat16() for _ in range(4))
    lam = torch.full((2,), 0.5, device="cuda").bfloat16()
    S.sla_profile_read()
    S.sla_profile_enable(True)
    try:
        S.sla_diff_forward(p, q, k, v, lam, out, S.dense_workspace(p))
    finally:
        S.sla_profile_enable(False)
    got = S.sla_profile_read()
    assert got["dense"][1] == 1 and got["dense"][0] > 0 and got["attn"][1] == 0
