"""Host-side checks of the layers' entry points (no GPU: every call here is refused, or is empty)."""
import ctypes
import math

import pytest
import torch

import layers_ref as ref
import lossless_draft_verification_spec_amd as pkg

BF, FH, F32, F8, E8 = (pkg.PSISPEC_BF16, pkg.PSISPEC_F16, pkg.PSISPEC_F32, pkg.PSISPEC_F8E4M3, pkg.PSISPEC_E8M0)
X, W, R, RO, OUT, SC, PK, PK2, WS = (1 << 24 << i for i in range(9))  # addresses far from each other
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return pkg.lib()


def _norm(L, x=X, xs=256, dtype=BF, res=R, rs=256, ro=RO, ros=256, rdtype=BF, w=W, eps=1e-6, rows=4, dim=256, out=OUT,
          os_=256, odtype=BF, sc=None, ss=0, sdtype=F32):
    return L.psispec_add_rmsnorm(x, xs, dtype, res, rs, ro, ros, rdtype, w, eps, rows, dim, out, os_, odtype, sc, ss,
                                 sdtype, None)


def test_norm_checks(L):
    assert _norm(L, rows=0, x=None, out=None) == 0
    for kw in (dict(dtype=F32), dict(dtype=F8), dict(rdtype=FH), dict(rdtype=F8), dict(odtype=FH), dict(odtype=F32),
               dict(odtype=F8, sc=SC, sdtype=BF), dict(odtype=E8)):
        assert _norm(L, **kw) == -2, kw
    quant = dict(odtype=F8, sc=SC)
    mx = dict(odtype=F8, sc=SC, ss=8, sdtype=E8)
    for kw in (dict(rows=-1), dict(rows=1 << 24), dict(dim=0), dict(dim=32769), dict(eps=-1e-9), dict(eps=math.nan),
               dict(eps=math.inf), dict(eps=1e39), dict(x=None), dict(out=None), dict(x=X + 1), dict(out=OUT + 1),
               dict(w=W + 1), dict(res=R + 1), dict(ro=RO + 1), dict(rdtype=F32, ro=RO + 2), dict(xs=255), dict(rs=255),
               dict(ros=255), dict(os_=255), dict(xs=-256), dict(xs=1 << 40), dict(sc=SC), dict(quant, sc=None),
               dict(quant, sc=SC + 2), dict(mx, ss=7), dict(mx, dim=250)):
        assert _norm(L, **kw) == -1, kw
    # outputs over inputs or each other, other than the very rows of x or residual
    for kw in (dict(out=X + 2), dict(out=X + 512), dict(out=X, os_=512), dict(ro=X + 16), dict(ro=R + 512), dict(out=R - 2),
               dict(out=RO), dict(out=W), dict(ro=W + 256), dict(quant, out=X), dict(quant, sc=X), dict(quant, sc=OUT),
               dict(quant, sc=RO + 4), dict(mx, sc=R), dict(mx, sc=W), dict(rdtype=F32, out=R)):
        assert _norm(L, **kw) == -1, kw
    # rows between each other: parts of one wider row (refused only where they meet)
    assert _norm(L, xs=600, out=X + 2 * 100, os_=600) == -1
    assert _norm(L, xs=600, rows=0, out=X + 2 * 256, os_=600) == 0


def _weight(**kw):
    base = dict(packed=PK, n=64, k=256, group=128, format=pkg.PSISPEC_W4_INT, scale_dtype=BF, reserved=0)
    return pkg.psispec_w4_weight(**{**base, **kw})


MX = dict(group=32, format=pkg.PSISPEC_W4_MX, scale_dtype=E8)
BAD_WEIGHTS = [dict(n=0), dict(n=(1 << 20) + 1), dict(k=0), dict(k=31), dict(k=48), dict(k=(1 << 20) + 32), dict(group=0),
               dict(group=16), dict(group=96), dict(group=192), dict(group=-128), dict(group=1 << 21), dict(reserved=1),
               dict(MX, group=64), dict(packed=None), dict(packed=PK + 16)]


def _linear(L, w=None, x=X, xs=256, dtype=BF, sc=None, ss=0, rows=4, bias=None, out=OUT, os_=64, odtype=BF, ws=WS,
            wsn=BIG):
    w = _weight() if w is None else w
    return L.psispec_w4_linear(ctypes.byref(w), x, xs, dtype, sc, ss, rows, bias, out, os_, odtype, ws, wsn, None)


def _gated(L, g=None, u=None, act=0, x=X, xs=256, dtype=BF, sc=None, ss=0, rows=4, out=OUT, os_=64, odtype=BF, ws=WS,
           wsn=BIG):
    g, u = g or _weight(), u or _weight(packed=PK2)
    return L.psispec_w4_gated(ctypes.byref(g), ctypes.byref(u), act, x, xs, dtype, sc, ss, rows, out, os_, odtype, ws,
                              wsn, None)


def test_product_checks(L):
    assert _linear(L, rows=0, x=None, out=None, w=_weight(packed=None)) == 0
    assert _gated(L, rows=0, x=None, out=None) == 0
    for kw in BAD_WEIGHTS:
        assert _linear(L, _weight(**kw)) == -1, kw
        assert _gated(L, u=_weight(**kw)) == -1, kw
    assert _linear(L, _weight(format=2)) == -5
    assert L.psispec_w4_linear(None, X, 256, BF, None, 0, 4, None, OUT, 64, BF, WS, BIG, None) == -1
    for kw in (dict(scale_dtype=F32), dict(scale_dtype=E8), dict(MX, scale_dtype=BF)):
        assert _linear(L, _weight(**kw)) == -2, kw
    for kw in (dict(dtype=F32), dict(dtype=E8), dict(odtype=FH), dict(odtype=F32), dict(dtype=FH)):
        assert _linear(L, **kw) == -2, kw
    m = _weight(**MX)
    assert _linear(L, dtype=F8, sc=SC, ss=8) == -5                      # 8-bit rows with INT weights
    assert _linear(L, m, dtype=F8, sc=SC, ss=8, odtype=F32) == -2
    for kw in (dict(dtype=F8), dict(dtype=F8, sc=SC, ss=7), dict(sc=SC, ss=8)):
        assert _linear(L, m, **kw) == -1, kw
    for kw in (dict(rows=-1), dict(rows=1 << 24), dict(x=None), dict(out=None), dict(x=X + 8), dict(xs=248), dict(xs=260),
               dict(os_=63), dict(out=OUT + 1), dict(bias=W + 1), dict(xs=1 << 40), dict(xs=(1 << 23) + 8)):
        assert _linear(L, **kw) == -1, kw
    # 2^23 tiles of 16 rows x 16 outputs and more
    assert _linear(L, _weight(n=1 << 20), rows=2048, os_=1 << 20) == -1
    # the output over an input
    for kw in (dict(out=X), dict(out=X + 512 * 3 + 510), dict(out=X - 2, rows=1), dict(out=PK), dict(out=PK - 128),
               dict(out=W, bias=W), dict(out=X + 2 * 250, os_=256)):
        assert _linear(L, **kw) == -1, kw
    assert _linear(L, m, dtype=F8, sc=OUT, ss=8) == -1
    assert _gated(L, out=PK2) == -1
    for kw in (dict(act=-1), dict(act=3)):
        assert _gated(L, **kw) == -1, kw
    for kw in (dict(n=80), dict(k=128), dict(group=64), dict(scale_dtype=FH), MX):
        assert _gated(L, u=_weight(packed=PK2, **kw)) == -1, kw
    assert L.psispec_w4_gated(ctypes.byref(_weight()), None, 0, X, 256, BF, None, 0, 4, OUT, 64, BF, WS, BIG, None) == -1


def test_pack_checks(L):
    def pack(w=None, codes=X, cs=128, sc=SC, ss=2, nbytes=BIG):
        return L.psispec_w4_pack(codes, cs, sc, ss, ctypes.byref(w or _weight()), nbytes, None)

    for kw in BAD_WEIGHTS:
        assert pack(_weight(**kw)) == -1, kw
    assert pack(_weight(format=7)) == -5 and pack(_weight(scale_dtype=F32)) == -2
    need = L.psispec_w4_packed_bytes(64, 256, 128, pkg.PSISPEC_W4_INT)
    assert need >= 64 * 128 + 64 * 2 * 2 and pack(nbytes=need - 1) == -3
    for kw in (dict(codes=None), dict(sc=None), dict(cs=127), dict(ss=1), dict(sc=SC + 1), dict(codes=PK), dict(sc=PK)):
        assert pack(**kw) == -1, kw
    # 2^26 - 3 tiles of 16 outputs x 128 inputs and more
    big = dict(n=1 << 20, k=1 << 17)
    assert pack(_weight(**big), cs=1 << 16, ss=1 << 10) == -1 and L.psispec_w4_packed_bytes(1 << 20, 1 << 17, 128, 0) == 0
    assert L.psispec_w4_packed_bytes(1 << 20, (1 << 17) - 128, 128, 0) > 1 << 36
    for bad in ((0, 256, 128, 0), (64, 40, 32, 0), (64, 256, 96, 0), (64, 256, 128, 1), (64, 256, 32, 2)):
        assert L.psispec_w4_packed_bytes(*bad) == 0, bad


def test_workspace_query(L):
    for bad in ((0, 64, 256, 1), (4, 0, 256, 1), (4, 64, 0, 1), (4, 64, 256, 0), (4, 64, 256, 3), (1 << 24, 64, 256, 1)):
        assert L.psispec_w4_workspace(*bad) == 0
    assert L.psispec_w4_workspace(64, 1 << 16, 4096, 2) == 0  # few rows need none
    assert L.psispec_w4_workspace(576, 12288, 4096, 2) > 0
    w = _weight(n=12288, k=4096)
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(wsn=L.psispec_w4_workspace(576, 12288, 4096, 1) - 1)):
        assert _linear(L, w, xs=4096, os_=12288, rows=576, x=1 << 35, out=1 << 36, **kw) == -3, kw


def test_the_binding_needs_gpu_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_add_rmsnorm(x)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_w4_pack(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 1), dtype=torch.bfloat16))
    with pytest.raises(pkg.PsispecError):
        pkg.psispec_add_rmsnorm(x, quant="int8")


def test_references_agree_with_a_dense_form():
    """The references themselves: codes and scales by hand."""
    codes = torch.tensor([[0x10, 0x32, 0x7f] + [0x98] * 13], dtype=torch.uint8)
    w, _, _ = ref.weights(codes, torch.tensor([[0.5]], dtype=torch.bfloat16), "int", 32)
    assert w[0, :6].tolist() == [0, 0.5, 1.0, 1.5, -0.5, 3.5] and w[0, 6:8].tolist() == [-4.0, -3.5]
    w, _, _ = ref.weights(codes, torch.tensor([[128]], dtype=torch.uint8).view(torch.float8_e8m0fnu), "mx", 32)
    assert w[0, :6].tolist() == [0, 1.0, 2.0, 3.0, -12.0, 12.0] and w[0, 6:8].tolist() == [-0.0, -1.0]
    y, h = ref.norm(torch.tensor([[3.0, 4.0]]), None, torch.tensor([[0.0, 0.0]]), 0.0)
    assert torch.allclose(y, torch.tensor([[3.0, 4.0]]).double() / math.sqrt(12.5)) and h.tolist() == [[3.0, 4.0]]
