"""Calls of the expert-layer entry points that are empty one way, and arguments that the foreign-function layer would cut
short (no GPU needed: fake device pointers, so only where nothing can launch)."""
import pytest
import torch
from test_layers_abi import A, EALIGN, EINVAL, ENODEV, NBACK, NO_GPU, NORM, OK, Stub, call, calls  # noqa: F401

from newton_schulz_quintic_gb300 import api


@NO_GPU
def test_block_norm_of_no_columns(call):  # noqa: F811
    n = lambda **k: call("ns_block_norm", {**NORM, "cols": 0}, **k)  # noqa: E731
    null = dict(x=None, y=None, post=None, pre=None, r=None, z=None)
    assert n() == OK and n(**null, gate=None) == OK and n(**null, gate=None, form=0) == OK and n(**null, form=2, ldg=1) == OK
    b = lambda **k: call("ns_block_norm_backward", {**NBACK, "cols": 0}, **k)  # noqa: E731
    null = dict(dr=None, dz=None, x=None, y=None, post=None, pre=None, dx=None, dy=None, dpost=None, dpre=None)
    assert b() == OK and b(**null, gate=None, dgate=None) == OK and b(**null, gate=None, form=0, dgate=None) == OK
    # one gate a row: its gradient is there to be written
    rows = dict(null, form=2, ldg=1, lddg=1)
    assert b(**rows) == ENODEV and b(**rows, rows=0, dgate=None) == OK and b(**rows, dgate=None) == EINVAL
    assert b(**rows, dgate=NBACK["gate"] + 2) == EINVAL and b(**rows, dgate=A + 1) == EALIGN and b(**dict(rows, lddg=0)) == EINVAL


def test_per_beyond_an_int_is_refused(calls):  # noqa: F811
    x, rows = Stub((6, 16), torch.bfloat16), Stub((9,), torch.int32)
    for per in (0, -1, 1 << 31, (1 << 32) + 1):
        with pytest.raises(ValueError):
            api.blocks_store(x, rows=rows, per=per)
    assert not calls
    api.blocks_store(x, rows=rows, per=(1 << 31) - 1)
    assert calls[0][1][4] == (1 << 31) - 1
