"""Host-side refusals of the layers' entry points at the ends of their ranges (no GPU: every call is refused)."""
import ctypes

import pytest

import lossless_draft_verification_spec_amd as pkg
from test_layers_host import BF, F8, MX, _gated, _linear, _weight

AT = [1 << 33 + i for i in range(7)]  # addresses far from each other


@pytest.fixture(scope="module")
def L():
    return pkg.lib()


def test_workspace_over_what_a_product_reads_or_writes(L):
    n, k, rows = 12288, 4096, 576
    x, out, bias, scales, w1, w2, ws = AT
    need = L.psispec_w4_workspace(rows, n, k, 1)
    assert need > 0 and need % 256 == 0
    sizes = dict(x=x, xs=k, rows=rows, out=out, os_=n, ws=ws, wsn=need)
    first = _weight(packed=w1, n=n, k=k)
    last = x + 2 * rows * k  # right behind the rows
    assert _linear(L, first, **{**sizes, "wsn": need - 256}) == -3
    for at in (x, last - 256, x + 256 - need, out, out + 2 * rows * n - 256, w1, bias, bias + 2 * n - 256):
        assert _linear(L, first, bias=bias, **{**sizes, "ws": at}) == -1, hex(at)
    second = _weight(packed=w2, n=n, k=k)
    sizes["wsn"] = L.psispec_w4_workspace(rows, n, k, 2)
    for at in (x, out, w1, w2, w2 + 256):
        assert _gated(L, first, second, **{**sizes, "ws": at}) == -1, hex(at)
    # rows of 8 bits in parts, which need one for their sums
    n, k, rows = 4096, 12288, 576
    need = L.psispec_w4_workspace(rows, n, k, 1)
    m = _weight(packed=w1, n=n, k=k, **MX)
    sizes = dict(x=x, xs=k, dtype=F8, sc=scales, ss=k // 32, rows=rows, out=out, os_=n, odtype=BF, wsn=need)
    for at in (x, scales, scales + rows * k // 32 - 256, out, w1):
        assert _linear(L, m, **{**sizes, "ws": at}) == -1, hex(at)


def test_workspace_by_format(L):
    """MX weights have no sums of rows: with uncut inputs nothing is needed, with cut ones the parts' sums alone."""
    def need(rows, mats=1, **kw):
        return L.psispec_w4_weight_workspace(ctypes.byref(_weight(**kw)), rows, mats)

    for n, k, rows, mats in ((2039, 160, 1601, 1), (4096, 16512, 131142, 1), (12288, 4096, 576, 2)):
        assert need(rows, mats, n=n, k=k, **MX) == 0
        assert need(rows, mats, n=n, k=k) == L.psispec_w4_workspace(rows, n, k, mats) > 0
    rows, n, k = 576, 4096, 12288  # three parts
    assert need(rows, n=n, k=k, **MX) == 3 * rows * n * 4
    assert need(rows, n=n, k=k) == L.psispec_w4_workspace(rows, n, k, 1) > 3 * rows * n * 4
    assert need(64, n=n, k=k) == need(64, n=n, k=k, **MX) == 0
    for bad in (dict(rows=0), dict(rows=1 << 24), dict(rows=576, mats=3), dict(rows=576, k=100), dict(rows=576, reserved=1)):
        assert need(**{"n": n, "k": k, **bad}) == 0
    assert L.psispec_w4_weight_workspace(None, 576, 1) == 0


def test_counts_beyond_32_bits_are_refused():
    assert pkg.w4_packed_bytes(48, 160, 32, "mx") > 0 and pkg.w4_workspace_bytes(576, 12288, 4096) > 0
    for wide in (1 << 31, (1 << 32) + 48, (1 << 32) + 160, (1 << 32) + 32):
        assert pkg.w4_packed_bytes(wide, 160, 32, "mx") == 0
        assert pkg.w4_packed_bytes(48, wide, 32, "mx") == 0
        assert pkg.w4_packed_bytes(48, 160, wide, "int") == 0
    for wide in (1 << 31, (1 << 32) + 576, (1 << 32) + 4096):
        assert pkg.w4_workspace_bytes(wide, 12288, 4096) == 0
        assert pkg.w4_workspace_bytes(576, wide, 4096) == 0
        assert pkg.w4_workspace_bytes(576, 12288, wide) == 0
