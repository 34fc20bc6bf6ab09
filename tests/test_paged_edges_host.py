"""Host side of the paged-cache calls at the borders of what they take (no GPU: every call here is refused
or empty), and the frequency tables for long and short original lengths."""
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


@pytest.mark.parametrize("rot,base", [(128, 10000.0), (64, 10000.0), (128, 500000.0)])
@pytest.mark.parametrize("original", [4, 64, 200, 4096, 65536, 131072, 10**7])
@pytest.mark.parametrize("factor", [4.0, 40.0])
def test_by_parts_borders(rot, base, original, factor):
    """Pairs on either side of the borders, and the ramp between them, also where a border lies before the
    first pair or behind the last."""
    f, _ = pkg.rope_frequencies(rot, base)
    got, _ = pkg.rope_frequencies(rot, base, "by_parts", factor, original)
    j_of = lambda turns: rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
    lo, hi = math.floor(j_of(32.0)), math.ceil(j_of(1.0))
    for j in range(rot // 2):
        turns = original * float(f[j]) / (2 * math.pi)
        part = min(max((j - lo) / (hi - lo), 0.0), 1.0)  # of the divided frequency
        want = float(f[j]) * ((1 - part) + part / factor)
        assert math.isclose(float(got[j]), want, rel_tol=1e-12), j
        if turns >= 1.0 and j < hi:
            assert got[j] > f[j] / factor * (1 + 1e-9), "turns more than `slow` times, divided in full"
        if turns < 32.0 and j > lo:
            assert got[j] < f[j], "turns less than `fast` times, as it was"


def test_by_parts_last_pair():
    """rot 128, base 10000: the last pair turns 1.2 times in 65536 positions, so it is mixed."""
    f, _ = pkg.rope_frequencies(128, 10000.0)
    assert 1.1 < 65536 * float(f[-1]) / (2 * math.pi) < 1.3
    got, _ = pkg.rope_frequencies(128, 10000.0, "by_parts", 4.0, 65536)
    assert f[-1] / 4 * 1.01 < got[-1] < f[-1]


def test_by_parts_base_below_one():
    """Later pairs would turn faster: the borders would stand the wrong way round."""
    for base in (0.5, 1.0):
        with pytest.raises(pkg.PsispecError, match="base above 1"):
            pkg.rope_frequencies(64, base, "by_parts", 4.0, 4096)


def _cache(**kw):
    """8 pages of 16 positions of 2 heads of 64 at 2^30 (K) and 2^31 (V)."""
    return pkg.psispec_paged_cache(**{**dict(
        k=1 << 30, v=1 << 31, k_scale=None, v_scale=None, table=256, page_stride=16 * 2 * 64,
        row_stride=128, head_stride=64, table_stride=4, num_pages=8, page_size=16, slots=4, heads=2, dim=64,
        dtype=pkg.PSISPEC_BF16), **kw})


def _append(L, c=None, batch=1, blk=2, hq=4, q=1 << 20, qs=512, k=2 << 20, ks=512, v=3 << 20, vs=512, qo=4 << 20,
            os=512, ln=256, nn=None, pos=None, st=None):
    """One row of q is 256 elements, one of k or v 128."""
    p = pkg.psispec_qkv_prep(q_weight=None, k_weight=None, inv_freq=256, eps=1e-6, rope_scale=1.0, rot=64,
                             flags=0)
    return L.psispec_qkv_append(ctypes.byref(c or _cache()), ctypes.byref(p), q, qs, k, ks, v, vs,
                                pkg.PSISPEC_BF16, batch, blk, hq, pos, ln, nn, qo, os, st, None)


@pytest.mark.parametrize("which", ["k", "v"])
def test_append_output_over_keys_or_values(L, which):
    """q_out over the rows of k or v: from the same place, ends that meet, other strides."""
    at = 4 << 20  # q_out: rows of 512 bytes at 4 MiB, 1024 bytes apart
    for off in (0, 256, -240, 496, 1024, 1024 - 240, 1024 + 496):
        assert _append(L, **{which: at + off}) == -1, off
    for off, s in ((0, 136), (-272, 136), (512, 264)):
        assert _append(L, **{which: at + off, which + "s": s}) == -1, off
    assert _append(L, **{which: 1 << 20, "qo": 1 << 20}) == -1  # in place, with k or v over q


def _attend(L, c, out, os=256, batch=1, blk=2, hq=4, **kw):
    a = dict(parent=None, ln=256, nn=None, st=None, scale=1.0, ws=None, dtype=pkg.PSISPEC_BF16)
    a.update(kw)
    return L.psispec_paged_attention(ctypes.byref(c), 1 << 20, 512, a["dtype"], batch, blk, hq, a["parent"],
                                     a["ln"], a["nn"], a["scale"], out, os, a["st"], a["ws"], BIG, None)


def test_outputs_over_the_cache(L):
    """Rows of 256 elements over places of K and V, at their ends, and in the gaps between places: only
    the missing workspace is then left to refuse."""
    K, V = 1 << 30, 1 << 31
    page = 16 * 2 * 64 * 2  # bytes
    for base in (K, V):
        for at in (base, base - 1024, base - 496, base + 8 * page - 16, base + page + 32, base - 512):
            meets = at + 1024 > base  # two rows of 512 bytes
            assert _attend(L, _cache(), at) == (-1 if meets else -3), at - base
            if meets:
                assert _append(L, qo=at, os=256) == -1
        assert _attend(L, _cache(), base + 8 * page) == -3
        assert _attend(L, _cache(), base - 512, os=1 << 20) == -3  # the second row far behind the cache
        assert _attend(L, _cache(), base - page, os=page // 2) == -1
    # pages with a gap of their size behind each; heads with gaps
    wide = _cache(page_stride=2 * 16 * 2 * 64)
    for at, rc in ((0, -1), (page, -3), (2 * page - 1024, -3), (2 * page - 512, -1), (2 * page, -1),
                   (page - 16, -1), (15 * page, -3)):
        assert _attend(L, wide, K + at) == rc, at
    heads = _cache(head_stride=1024, row_stride=2048, page_stride=16 * 2048)
    for at, rc in ((0, -1), (128, -3), (2048 - 512, -3), (2048 - 496, -1)):
        assert _attend(L, heads, K + at, blk=1) == rc, at
    # positions before pages before heads (any order), and 8-bit places of half the bytes
    mixed = _cache(page_stride=64, row_stride=8 * 64, head_stride=1 << 16)
    assert _attend(L, mixed, K + 16 * 8 * 128) == -3 and _attend(L, mixed, K + (1 << 17)) == -1
    f8 = _cache(dtype=pkg.PSISPEC_F8E4M3)
    assert _attend(L, f8, K + 4 * page) == -3 and _attend(L, f8, K + 4 * page - 16) == -1
    # a cache whose pages are one page: read-only, its whole range counts
    assert _attend(L, _cache(page_stride=0), K + page) == -3
    assert _attend(L, _cache(page_stride=0), K + page - 16) == -1
    far = _cache(page_stride=1 << 59, num_pages=1 << 30)
    assert _attend(L, far, K + page) == -3 and _attend(L, far, K) == -1


def test_append_keys_over_values(L):
    """K and V in one place, and parts of a head, a head, some positions or pages apart."""
    K, head, row, page = 1 << 30, 128, 256, 4096
    wide = dict(row_stride=256, page_stride=16 * 256)  # rows with room for V's beside K's
    turns = dict(page_stride=2 * 16 * 128)             # pages with room for V's behind each
    mixed = dict(page_stride=64, row_stride=512, head_stride=1 << 14)
    for kw, shift in [({}, 0), ({}, head), ({}, -3 * row), ({}, 5 * page), ({}, -16), ({}, 8 * page - 16),
                      (wide, row - 16), (wide, 512 * 3 - head), (turns, page + 16), (mixed, 1 << 15),
                      (mixed, 128), (mixed, -1024 * 15)]:
        assert _append(L, _cache(k=K, v=K + shift, **kw)) == -1, (kw, shift)


def _commit(L, batch=8, blk=4, tab=1 << 12, keep=2 << 12, n_keep=3 << 12, ln=4 << 12, new=5 << 12, st=None):
    pool = pkg.psispec_page_pool(base=1 << 30, plane_stride=1 << 20, page_stride=16 * 64, row_bytes=64, planes=2,
                                 num_pages=8, page_size=16, reserved=0)
    return L.psispec_paged_commit(ctypes.byref(pool), tab, 6, 4, batch, blk, keep, 5, n_keep, ln, new, st, None)


def test_commit_lengths_over_inputs(L):
    """New lengths over the counts, the kept rows or the table: tiles of a line still read those when the
    first writes its new length."""
    for at in (3 << 12, (3 << 12) + 28, (3 << 12) - 28, 2 << 12, (2 << 12) + 4 * 39, 1 << 12, (1 << 12) + 4 * 45):
        assert _commit(L, new=at) == -1, at
        assert _commit(L, new=at, ln=at) == -1, at
    assert _commit(L, new=(4 << 12) + 4) == -1


def test_status_over_inputs(L):
    """A status over the lengths, counts, positions, parents, kept rows or table that the call reads."""
    A, B, C, T = 1 << 14, 2 << 14, 3 << 14, 4 << 14
    c = _cache(table=T)
    for st in (A, A + 28, A - 28, B, C, C + 4 * 15, T, T + 4 * 31):
        assert _append(L, c, batch=8, ln=A, nn=B, pos=C, st=st) == -1, st
        assert _attend(L, c, 1 << 26, batch=8, ln=A, nn=B, parent=C, st=st) == -1, st
    assert _attend(L, c, 1 << 26, batch=8, ln=A, nn=B, parent=C, st=5 << 14) == -3
    for st in (3 << 12, 4 << 12, 5 << 12, (2 << 12) + 4 * 39, (1 << 12) + 4 * 45):
        assert _commit(L, st=st) == -1, st
    pool = pkg.psispec_page_pool(base=1 << 30, plane_stride=1 << 20, page_stride=16 * 64, row_bytes=64, planes=2,
                                 num_pages=50, page_size=16, reserved=0)
    R = 5 << 14
    for st, rc in ((A, -1), (B, -1), (C, -1), (T, -1), (T + 4 * 45, -1), (R + 4 * 49, -1), (6 << 14, -3)):
        assert L.psispec_pages_assign(T, 6, 4, R, 50, 16, A, B, C, st, 8, None, BIG, None) == rc, st
        if st != C:
            assert L.psispec_pages_reserve(ctypes.byref(pool), T, 6, 4, R, A, B, 4, st, 8, None, BIG, None) == rc


def test_attention_sizes(L):
    """Batch, block and heads each at their limits, and several of them large at once."""
    size = L.psispec_paged_attention_workspace
    for a in ((256, 1024, 64, 8, 128), (64, 1024, 1024, 1, 256), (1 << 20, 1, 64, 8, 128), ((1 << 24) - 1, 1, 1, 1, 16)):
        assert size(*a) > 0, a
    for a in ((1 << 24, 1, 1, 1, 16), (1, 1025, 1, 1, 16), (1, 1, 1025, 1, 16), (1, 1, 1088, 17, 16)):
        assert size(*a) == 0, a
    assert _attend(L, _cache(), 1 << 40, batch=256, blk=1024, hq=2) == -3
    # more work than the shares can be cut from: 2^23 lines of 2^30 positions
    c = _cache(page_size=4096, slots=1 << 18, table_stride=1 << 18, page_stride=4096 * 128)
    assert _attend(L, c, 1 << 40, batch=1 << 23, blk=1) == -1


def test_numbers_that_32_bits_do_not_hold(L):
    for scale in (3e38, -3e38, 1e39):
        assert _attend(L, _cache(), 1 << 26, scale=scale) == -1, scale
    for scale in (2e38, -2e38, 0.0, 1e-40):
        assert _attend(L, _cache(), 1 << 26, scale=scale) == -3, scale
    for kw in (dict(eps=1e39), dict(rope_scale=1e39), dict(rope_scale=-1e300)):
        p = pkg.psispec_qkv_prep(**{**dict(q_weight=None, k_weight=None, inv_freq=256, eps=1e-6, rope_scale=1.0,
                                           rot=64, flags=0), **kw})
        assert L.psispec_qkv_append(ctypes.byref(_cache()), ctypes.byref(p), 1 << 20, 512, 2 << 20, 512, 3 << 20, 512,
                                    pkg.PSISPEC_BF16, 1, 2, 4, None, 256, None, 4 << 20, 512, None, None) == -1, kw
