"""The alias check of outputs that are columns of one wider buffer: tensors of the same stride in
bytes interleave row by row, whatever their widths and types, and are refused exactly where an
element is shared.  Addresses are made up, and without a workspace no call gets past the checks:
GNORM_ERR_WORKSPACE says that the alias check has passed.
"""
from __future__ import annotations

import random

import pytest

from gated_norm_b200._lib import GNORM_ERR_ALIAS, GNORM_ERR_WORKSPACE, lib
from test_block_delta_cpu import block_bwd, call, delta_bwd

BASE = 1 << 52
T = 5


def fused(width, **offsets):
    """A delta backward whose gradients are columns (from these byte offsets on) of rows of `width`
    bytes; 2 key heads and 4 value heads of 128, beta in FP32."""
    top = dict(workspace=None, workspace_bytes=0, dinitial_state=None)
    for n, at in offsets.items():
        top[n] = BASE + at
        top["ld" + n] = width // (4 if n in ("dg", "dbeta") else 2)
    return call(lib.gnorm_delta_bwd, delta_bwd(top, T=T, V=128))


COLS = dict(dq=512, dk=512, dv=1024, dg=16, dbeta=16)  # bytes of a row


def test_columns_of_one_buffer():
    """dq, dk and dv side by side where a row of v is twice as wide as one of q, and with dg and
    dbeta behind them."""
    assert fused(2048, dq=0, dk=512, dv=1024) == GNORM_ERR_WORKSPACE
    assert fused(2080, dv=0, dq=1024, dk=1536, dg=2048, dbeta=2064) == GNORM_ERR_WORKSPACE
    assert fused(2048, dq=0, dk=496, dv=1024) == GNORM_ERR_ALIAS
    assert fused(2048, dq=0, dk=512, dv=1008) == GNORM_ERR_ALIAS
    # v's rows run into q's next ones
    assert fused(1536, dq=0, dv=512) == GNORM_ERR_WORKSPACE
    assert fused(1536, dq=0, dv=528) == GNORM_ERR_ALIAS


def meet(width, x, nx, y, ny):
    return any(x + i * width < y + j * width + ny and y + j * width < x + i * width + nx
               for i in range(T) for j in range(T))


@pytest.mark.parametrize("seed", range(4))
def test_against_all_rows(seed):
    rng = random.Random(seed)
    seen = {GNORM_ERR_ALIAS: 0, GNORM_ERR_WORKSPACE: 0}
    for _ in range(400):
        names = rng.sample(sorted(COLS), 2)
        widest = max(COLS[n] for n in names)
        width = widest + 16 * rng.randrange(0, 100)
        at = {n: 16 * rng.randrange(0, T * width // 16) for n in names}
        a, b = names
        want = GNORM_ERR_ALIAS if meet(width, at[a], COLS[a], at[b], COLS[b]) else GNORM_ERR_WORKSPACE
        assert fused(width, **at) == want, (width, at)
        seen[want] += 1
    assert min(seen.values()) > 50


def test_other_strides_by_their_extents():
    d = block_bwd()
    d.da, d.ldda, d.dr, d.lddr = BASE, 512, BASE + 512, 520
    assert call(lib.gnorm_block_bwd, d) == GNORM_ERR_ALIAS
