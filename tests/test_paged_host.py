"""Host-side checks of the paged-cache entry points (no GPU: every call here is refused, or is empty)
and the frequency tables of the rotation."""
import ctypes
import math

import pytest
import torch

import lossless_draft_verification_spec_amd as pkg

P = ctypes.c_void_p(256)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return pkg.lib()


def _cache(**kw):
    base = dict(k=256, v=256, k_scale=None, v_scale=None, table=256, page_stride=16 * 2 * 64,
                row_stride=128, head_stride=64, table_stride=4, num_pages=8, page_size=16, slots=4,
                heads=2, dim=64, dtype=pkg.PSISPEC_BF16)
    base.update(kw)
    return pkg.psispec_paged_cache(**base)


BAD_CACHES = [dict(num_pages=0), dict(page_size=0), dict(page_size=4097), dict(slots=0),
              dict(slots=5), dict(slots=1 << 27, table_stride=1 << 27), dict(heads=0),
              dict(dim=24), dict(dim=0), dict(dim=272), dict(row_stride=130), dict(page_stride=-16),
              dict(head_stride=4), dict(page_stride=1 << 62), dict(k_scale=256), dict(v_scale=256)]


FAR = ctypes.c_void_p(1 << 20)


def _attend(L, c, dtype=pkg.PSISPEC_BF16, batch=1, blk=2, hq=4, q=P, qs=256, out=FAR, ln=P, scale=1.0,
            ws=P, wsn=BIG):
    return L.psispec_paged_attention(ctypes.byref(c) if c is not None else None, q, qs, dtype, batch,
                                     blk, hq, None, ln, None, scale, out, 256, None, ws, wsn, None)


def test_attention_checks(L):
    for kw in BAD_CACHES:
        assert _attend(L, _cache(**kw)) == -1, kw
    assert _attend(L, None) == -1
    assert _attend(L, _cache(), dtype=pkg.PSISPEC_F32) == -2
    assert _attend(L, _cache(dtype=pkg.PSISPEC_F16)) == -2          # cache of another type
    assert _attend(L, _cache(dtype=7)) == -2
    for kw in (dict(hq=3), dict(hq=0), dict(blk=0), dict(blk=1025), dict(batch=-1), dict(qs=255),
               dict(qs=260), dict(q=None), dict(out=None), dict(ln=None), dict(scale=math.inf),
               dict(scale=math.nan), dict(scale=1e300), dict(q=ctypes.c_void_p(264))):
        assert _attend(L, _cache(), **kw) == -1, kw
    # out over q: the same rows, a part of them, rows of other strides
    for at in (256, 256 + 2 * 248, 256 - 2 * 128, 256 + 2 * 256):
        assert _attend(L, _cache(), out=ctypes.c_void_p(at)) == -1
    assert _attend(L, _cache(), qs=512, out=ctypes.c_void_p(256 + 2 * 512)) == -1
    for kw in (dict(k=None), dict(v=264), dict(table=None)):
        assert _attend(L, _cache(**kw)) == -1, kw
    assert _attend(L, _cache(), ws=None) == -3
    assert _attend(L, _cache(), wsn=16) == -3
    assert _attend(L, _cache(), ws=ctypes.c_void_p(264)) == -3
    assert _attend(L, _cache(k=None), batch=0, q=None, out=None, ln=None, ws=None) == 0
    assert L.psispec_paged_attention_workspace(2, 9, 8, 2, 128) > 0
    assert L.psispec_paged_attention_workspace(2, 9, 8, 3, 128) == 0
    assert L.psispec_paged_attention_workspace(2, 2000, 8, 2, 128) == 0
    assert L.psispec_paged_attention_workspace(2, 9, 8, 2, 100) == 0


def test_append_checks(L):
    def prep(**kw):
        return pkg.psispec_qkv_prep(**{**dict(q_weight=None, k_weight=None, inv_freq=256, eps=1e-6,
                                              rope_scale=1.0, rot=64, flags=0), **kw})

    def call(c=None, p=None, dtype=pkg.PSISPEC_BF16, batch=1, blk=2, hq=4, q=P, qs=512, ks=512, ln=P,
             qo=P):
        return L.psispec_qkv_append(ctypes.byref(c or _cache()), ctypes.byref(p or prep()), q, qs, P, ks,
                                    P, 512, dtype, batch, blk, hq, None, ln, None, qo, 512, None, None)

    for kw in BAD_CACHES + [dict(head_stride=48), dict(row_stride=0), dict(page_stride=0)]:
        assert call(c=_cache(**kw)) == -1, kw
    # heads, positions or pages inside one another
    for kw in (dict(row_stride=64), dict(head_stride=96, row_stride=64, page_size=2),
               dict(page_stride=128 * 16 - 64), dict(page_stride=128, row_stride=128),
               dict(head_stride=1 << 60, row_stride=1 << 59, page_stride=1 << 58)):
        assert call(c=_cache(**kw)) == -1, kw
    # q_out between the rows of q, over its end, and rows of other strides
    for qo in (256 + 2 * 8, 256 + 2 * 248, 256 + 2 * 512):
        assert call(qo=ctypes.c_void_p(qo)) == -1
    assert call(qs=520) == -1
    for kw in (dict(rot=24), dict(rot=80), dict(rot=-16), dict(inv_freq=None), dict(eps=-1.0),
               dict(eps=math.nan), dict(rope_scale=math.inf), dict(flags=2), dict(q_weight=264)):
        assert call(p=prep(**kw)) == -1, kw
    for kw in (dict(blk=0), dict(blk=(1 << 20) + 1), dict(hq=0), dict(qs=128), dict(qs=516), dict(ks=64),
               dict(ln=None), dict(qo=None), dict(q=ctypes.c_void_p(260)), dict(batch=1 << 24)):
        assert call(**kw) == -1, kw
    assert call(dtype=pkg.PSISPEC_F16) == -2 and call(dtype=pkg.PSISPEC_F8E4M3) == -2
    assert call(batch=0, q=None, ln=None, qo=None) == 0


def test_page_calls_checks(L):
    def pool(**kw):
        return pkg.psispec_page_pool(**{**dict(base=256, plane_stride=1 << 20, page_stride=16 * 64,
                                               row_bytes=64, planes=2, num_pages=8, page_size=16,
                                               reserved=0), **kw})

    def commit(p=None, slots=4, stride=4, batch=1, blk=4, keep=P, ks=4, tab=P):
        return L.psispec_paged_commit(ctypes.byref(p or pool()), tab, stride, slots, batch, blk, keep,
                                      ks, P, P, P, None, None)

    def reserve(p=None, slots=4, stride=4, batch=1, blk=4, ws=P, wsn=BIG, refs=P):
        return L.psispec_pages_reserve(ctypes.byref(p or pool()), P, stride, slots, refs, P, None, blk,
                                       None, batch, ws, wsn, None)

    def assign(slots=4, stride=4, pages=8, ps=16, batch=1, ws=P, wsn=BIG, src=P):
        return L.psispec_pages_assign(P, stride, slots, P, pages, ps, P, src, P, None, batch, ws, wsn,
                                      None)

    for kw in (dict(row_bytes=8), dict(row_bytes=40), dict(page_stride=1000), dict(page_stride=16 * 60),
               dict(plane_stride=8), dict(planes=0), dict(num_pages=0), dict(page_size=0),
               dict(reserved=1), dict(page_size=5000, page_stride=1 << 20), dict(base=264),
               dict(base=None), dict(planes=2**31 - 1, row_bytes=1 << 20, page_stride=1 << 24)):
        assert commit(pool(**kw)) == -1, kw
        assert reserve(pool(**kw)) == -1, kw
    for kw in (dict(slots=0), dict(stride=3), dict(batch=-1), dict(blk=0), dict(slots=1 << 27,
                                                                               stride=1 << 27)):
        assert commit(**kw) == -1, kw
        assert reserve(**kw) == -1, kw
    for kw in (dict(blk=1025), dict(blk=65), dict(ks=0), dict(tab=None)):
        assert commit(**kw) == -1, kw
    assert reserve(refs=None) == -1 and reserve(blk=(1 << 20) + 1) == -1
    for kw in (dict(slots=0), dict(stride=3), dict(pages=0), dict(ps=0), dict(ps=4097), dict(batch=-1),
               dict(src=None)):
        assert assign(**kw) == -1, kw
    for f in (reserve, assign):
        assert f(ws=None) == -3 and f(wsn=100) == -3 and f(ws=ctypes.c_void_p(264)) == -3
        assert f(batch=0) == 0
    assert commit(batch=0) == 0
    for at, n in ((256, 2), (260, 2), (256 + 4 * 7, 8), (256 - 4 * 7, 8)):  # partly over the old lengths
        bad = L.psispec_paged_commit(ctypes.byref(pool()), P, 4, 4, n, 4, P, 4, P, ctypes.c_void_p(at + 4),
                                     ctypes.c_void_p(at), None, None)
        assert bad == -1
    assert L.psispec_pages_workspace(4, 10, 100, 9, 16) > 0
    assert L.psispec_pages_workspace((1 << 23) + 1, 10, 100, 9, 16) == 0
    assert L.psispec_pages_workspace(4, 10, 1 << 28, 9, 16) == 0
    assert L.psispec_pages_workspace(4, 0, 100, 9, 16) == 0


def test_binding_takes_gpu_tensors_only():
    q = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_paged_attention(q, c, c, i, n)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_qkv_append(q, q, q, c, c, i, n)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_paged_commit(c[None], i, n, 1, n)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_pages_reserve(c[None], i, n, n, 1)
    with pytest.raises(pkg.PsispecError, match="GPU"):
        pkg.psispec_pages_assign(i, n, n, n, n, 16)


def test_rope_frequencies():
    f, m = pkg.rope_frequencies(64, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and m == 1.0
    assert f[0] == 1.0 and math.isclose(f[16], 0.01, rel_tol=1e-12)
    lin, m = pkg.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.allclose(lin, f / 4, rtol=1e-14) and m == 1.0
    ntk, _ = pkg.rope_frequencies(64, 10000.0, "base", 4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], f[-1] / 4, rel_tol=1e-12)
    part, m = pkg.rope_frequencies(64, 10000.0, "by_parts", 4.0, 4096)
    turns = 4096 * f / (2 * math.pi)
    # the borders are rounded outwards, so pairs beyond them are untouched or fully divided
    assert torch.equal(part[turns > 32 * 1.4], f[turns > 32 * 1.4])
    assert torch.allclose(part[turns < 1 / 1.4], f[turns < 1 / 1.4] / 4, rtol=1e-14)
    assert ((part <= f) & (part >= f / 4 * (1 - 1e-14))).all()
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    for bad in (dict(rot=3), dict(rot=0), dict(base=0.0), dict(factor=0.0), dict(scaling="x"),
                dict(scaling="by_parts"), dict(rot=2, scaling="base")):
        with pytest.raises(pkg.PsispecError):
            pkg.rope_frequencies(**{**dict(rot=64), **bad})
