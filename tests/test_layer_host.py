"""Host-side checks of the operators around the scan that need no GPU: bad
arguments are refused, with a reason, before a device is touched, and the sizes
of the scratch that the calls ask for."""
import ctypes

import pytest

from linear_recurrence_scan_lrscan_gb300 import layer
from linear_recurrence_scan_lrscan_gb300 import lrscan as L

EINVAL, EDTYPE = -1, -2
F32, BF16 = 0, 1
P = 0x10000  # an address; no call here reaches a device with it


@pytest.fixture(scope="module")
def lib():
    return L.lib()


def rows(ptr=P, sb=1 << 20, st=64):
    return ctypes.byref(layer.Rows(ptr, sb, st))


def refused(lib, code, text, rc):
    assert rc == code
    assert text in lib.lrscan_last_error().decode()


GATES = dict(r=rows(), i=rows(), x=rows(), lam=P, c=8.0, out=rows(), last=None, saved=None, state=None, B=2, T=10, D=64,
             dtype=F32, stream=None, opts=None)


@pytest.mark.parametrize("change, code, text", [
    (dict(r=None), EINVAL, "NULL r"),
    (dict(x=rows(0)), EINVAL, "NULL x"),
    (dict(i=rows(P + 2)), EINVAL, "i is not aligned"),
    (dict(r=rows(sb=-64)), EINVAL, "negative stride"),
    (dict(x=rows(st=1 << 62)), EINVAL, "overflow"),
    (dict(out=rows(st=63)), EINVAL, "rows overlap"),
    (dict(out=rows(sb=0)), EINVAL, "rows overlap"),
    (dict(lam=None), EINVAL, "NULL lam"),
    (dict(lam=P + 1), EINVAL, "lam is not 4-byte aligned"),
    (dict(c=0.0), EINVAL, "not a positive number"),
    (dict(c=float("inf")), EINVAL, "not a positive number"),
    (dict(c=float("nan")), EINVAL, "not a positive number"),
    (dict(last=P + 2), EINVAL, "last is not 4-byte aligned"),
    (dict(T=-1), EINVAL, ""),
    (dict(B=1 << 40, T=1 << 40), EINVAL, ""),
    (dict(dtype=7), EDTYPE, ""),
])
def test_gates_refusals(lib, change, code, text):
    refused(lib, code, text, lib.lrscan_fwd_gates(*{**GATES, **change}.values()))


@pytest.mark.parametrize("K", [-1, 0, 1, 9])
def test_conv_refuses_its_taps(lib, K):
    assert lib.lrscan_fwd_conv(rows(), P, None, K, None, None, rows(), None, 2, 10, 64, F32, None) == EINVAL
    assert lib.lrscan_conv_workspace_bytes(2, 10, 64, K) == 0


def test_step_refuses_a_pool_too_small(lib):
    refused(lib, EINVAL, "requests without slots",
            lib.lrscan_step_gates(rows(), rows(), rows(), P, 8.0, P, None, rows(), 4, 3, 64, BF16, None))
    refused(lib, EINVAL, "requests without slots",
            lib.lrscan_step_conv(rows(), P, None, 4, P, None, rows(), 4, 3, 64, BF16, None))
    refused(lib, EINVAL, "NULL state",
            lib.lrscan_step_conv(rows(), P, None, 4, None, P, rows(), 4, 3, 64, BF16, None))


@pytest.mark.parametrize("change, text", [
    (dict(id_bytes=2), "ids of 2 bytes"),
    (dict(ids=None), "NULL ids"),
    (dict(out=None), "NULL output"),
    (dict(V=0), "empty table"),
    (dict(N=1 << 31), "above 2^31 - 2"),
    (dict(ids=P + 4), "not aligned"),
])
def test_embed_refusals(lib, change, text):
    a = dict(ids=P, id_bytes=8, weight=P, wdtype=F32, scale=1.0, out=P, odtype=BF16, N=10, V=100, D=64, stream=None)
    refused(lib, EINVAL, text, lib.lrscan_fwd_embed(*{**a, **change}.values()))


def test_scratch_sizes(lib):
    assert layer.lrscan_gates_workspace_bytes(2, 64, 64) == 0  # one tile of 64 tokens: nothing to publish
    assert layer.lrscan_gates_workspace_bytes(0, 64, 64) == 0
    assert layer.lrscan_gates_workspace_bytes(-1, 64, 64) == 0
    # a word a lane for each of 2 x 3 tiles
    assert layer.lrscan_gates_workspace_bytes(2, 129, 64) >= 8 * 64 * 6
    assert layer.lrscan_gates_workspace_bytes(2, 129, 64, direction="bwd") > layer.lrscan_gates_workspace_bytes(2, 129, 64)
    # an fp32 row of K + 1 sums a channel at least
    assert layer.lrscan_conv_workspace_bytes(2, 10, 64, 4) >= 2 * 5 * 64 * 4
    # ids and token numbers, twice
    assert layer.lrscan_embed_workspace_bytes(1000, 50, 64) >= 4 * 4 * 1000
    assert layer.lrscan_embed_workspace_bytes(0, 50, 64) == 0
    with pytest.raises(ValueError):
        layer.lrscan_gates_workspace_bytes(2, 64, 64, "f16")


def test_nothing_to_do_is_done(lib):
    assert lib.lrscan_fwd_gates(*{**GATES, **dict(B=0)}.values()) == 0
    assert lib.lrscan_fwd_gates(*{**GATES, **dict(D=0)}.values()) == 0
    assert lib.lrscan_fwd_embed(None, 8, None, F32, 1.0, None, F32, 0, 100, 64, None) == 0
