"""The paged-cache operators of the HIP library (through the binding) against 64-bit references:
attention of a block over pages, the append that writes them, the commit, forks and reservations, and
a run of all of them together."""
import itertools

import numpy as np
import pytest
import torch

import paged_ref as ref
from lossless_draft_verification_spec_amd import (
    PsispecError, paged_attention_workspace_bytes, pages_workspace_bytes, psispec_paged_attention,
    psispec_paged_commit, psispec_pages_assign, psispec_pages_reserve, psispec_qkv_append,
    psispec_verify_tree, rope_frequencies, workloads)

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FH, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _make_table(lens, blk, ps, g, extra_slots=0):
    per = [-(-(L + blk) // ps) for L in lens]
    pages = sum(per) + 1
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    tab = torch.full((len(lens), max(max(per), 1) + extra_slots), -1, dtype=torch.int32)
    at = 0
    for r, p in enumerate(per):
        tab[r, :p] = perm[at:at + p]
        at += p
    return tab, pages


def _case(lens, blk, hq, hkv, dim, ps, dtype, cache, seed, live=None, tree=False, layout="nhd",
          spread=2.0):
    g = _gen(seed)
    tab, pages = _make_table(lens, blk, ps, g)
    c = dict(lens=torch.tensor(lens, dtype=torch.int32), table=tab, scale=dim ** -0.5)
    c["live"] = None if live is None else torch.tensor(live, dtype=torch.int32)
    shape = (pages, ps, hkv, dim)
    kv = [torch.randn(shape, generator=g).to(cache) for _ in range(2)]
    c["ks"] = c["vs"] = None
    if cache == F8:
        c["ks"], c["vs"] = (0.5 + torch.rand(hkv, generator=g) for _ in range(2))
    c["k"], c["v"] = kv
    c["q"] = (torch.randn((len(lens), blk, hq, dim), generator=g) * spread).to(dtype)
    c["parent"] = None
    if tree:
        par = torch.full((len(lens), blk), -1, dtype=torch.int32)
        for j in range(1, blk):
            par[:, j] = torch.randint(-1, j, (len(lens),), generator=g).to(torch.int32)
        c["parent"] = par
    c["layout"] = layout
    return c


def _cache_dev(t, layout):
    """The cache on the GPU: contiguous, heads before positions, or inside a wider pool."""
    t = t.to(DEV)
    if layout == "hnd":
        return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    if layout == "planes":  # [pages][layers][page_size][heads][dim + 16]: a strided view
        p, ps, h, d = t.shape
        raw = torch.zeros((p, 3, ps, h, d + 16), dtype=torch.uint8 if t.element_size() == 1 else t.dtype,
                          device=DEV).view(t.dtype)
        v = raw[:, 1, :, :, :d]
        v.copy_(t)
        return v
    return t


def _gpu(t):
    return None if t is None else t.to(DEV)


def _attend(c, **kw):
    return psispec_paged_attention(
        _gpu(c["q"]), _cache_dev(c["k"], c["layout"]), _cache_dev(c["v"], c["layout"]),
        _gpu(c["table"]), _gpu(c["lens"]), n_new=_gpu(c["live"]), parent=_gpu(c["parent"]),
        scale=c["scale"], k_scale=_gpu(c["ks"]), v_scale=_gpu(c["vs"]), **kw)


def _check_attend(c):
    b, blk = c["q"].shape[:2]
    live = c["live"] if c["live"] is not None else torch.full((b,), blk)
    want, bound = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], live, c["parent"],
                                c["scale"], c["ks"], c["vs"])
    out = torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device=DEV)
    st = torch.full((b,), -1, dtype=torch.int32, device=DEV)
    got = _attend(c, out=out, status=st).cpu().double()
    assert (st.cpu() == 0).all()
    for r in range(b):
        n = int(live[r])
        assert (got[r, n:] == 7.0).all(), "rows behind the line's last were written"
        err = (got[r, :n] - want[r, :n]).abs()
        assert (err <= bound[r, :n]).all(), (r, (err / bound[r, :n]).max())


@pytest.mark.parametrize("lens", [[0], [1], [15], [31], [32], [33], [127, 128, 129], [0, 700, 5, 0, 1],
                                  [2500], [1, 1023, 64]])
@pytest.mark.parametrize("blk", [1, 9])
def test_attend_lengths(lens, blk):
    _check_attend(_case(lens, blk, 8, 2, 128, 16, BF, BF, seed=len(lens) * 7 + lens[0] + blk))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 1), (7, 1), (10, 2), (16, 2), (24, 3), (40, 8),
                                    (17, 1), (96, 2)])
def test_attend_heads(hq, hkv):
    _check_attend(_case([70, 300, 9], 3, hq, hkv, 64, 16, FH, FH, seed=hq))


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("cache", ["same", "f8"])
def test_attend_dims(dim, cache):
    _check_attend(_case([77, 260], 5, 6, 2, dim, 16, BF, BF if cache == "same" else F8, seed=dim))


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, F8), (FH, F8)])
@pytest.mark.parametrize("ps", [1, 3, 8, 16, 24, 32, 100, 256, 4096])
def test_attend_page_sizes(dtype, cache, ps):
    _check_attend(_case([333, 95], 4, 8, 2, 64, ps, dtype, cache, seed=ps))


@pytest.mark.parametrize("layout", ["nhd", "hnd", "planes"])
@pytest.mark.parametrize("cache", [BF, F8])
def test_attend_layouts(layout, cache):
    _check_attend(_case([333, 95, 40], 2, 8, 4, 128, 16, BF, cache, seed=3, layout=layout))


@pytest.mark.parametrize("blk,hq,hkv", [(2, 4, 2), (16, 4, 1), (33, 8, 2), (33, 28, 4), (64, 8, 8),
                                        (65, 4, 1), (130, 2, 1), (257, 2, 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_blocks(blk, hq, hkv, tree):
    _check_attend(_case([50, 0, 201], blk, hq, hkv, 64, 16, BF, BF, seed=blk, tree=tree,
                        live=[blk, blk // 2 + 1, 1]))


def test_attend_large_block():
    _check_attend(_case([40], 1024, 2, 1, 32, 16, BF, BF, seed=1, tree=True, live=[1000]))


def test_attend_idle_lines_and_short_blocks():
    _check_attend(_case([100, 30, 0, 64, 7, 500], 9, 8, 2, 128, 16, BF, BF, seed=5,
                        live=[0, 9, 4, 1, 0, 8]))
    c = _case([10, 20], 3, 4, 2, 64, 16, BF, BF, seed=6, live=[0, 0])
    out = torch.full(c["q"].shape, 3.0, dtype=BF, device=DEV)
    assert (_attend(c, out=out) == 3.0).all()


def test_attend_many_ragged_lines():
    """More lines than a workgroup has threads; shares end inside lines."""
    g = _gen(9)
    lens = torch.randint(0, 120, (300,), generator=g).tolist()
    lens[7], lens[200] = 3000, 1500
    live = torch.randint(0, 3, (300,), generator=g).tolist()
    _check_attend(_case(lens, 2, 4, 2, 64, 16, BF, BF, seed=9, live=live))


def test_attend_batch_of_one_long_line():
    _check_attend(_case([20011], 1, 8, 1, 128, 16, BF, BF, seed=12))
    _check_attend(_case([20011], 1, 8, 1, 128, 64, BF, F8, seed=12))


@pytest.mark.parametrize("dim,dtype,cache,L", [(64, FH, FH, 67400), (128, BF, F8, 68600), (192, BF, BF, 33200)])
def test_attend_about_one_unit_of_work_per_share(dim, dtype, cache, L):
    """One job over a few more units than there are workgroups: a share without any would leave a part
    that nothing wrote to the join."""
    c = _case([L], 1, 2, 1, dim, 64, dtype, cache, seed=dim)
    ws = torch.full((paged_attention_workspace_bytes(1, 1, 2, 1, dim),), 255, dtype=torch.uint8, device=DEV)
    for cut in (0, 500, 1700, 2047):
        c["lens"] = torch.tensor([L - cut], dtype=torch.int32)
        _check_attend(c)
        ws.fill_(255)
        want = _attend(c)
        assert torch.equal(_attend(c, workspace=ws), want)


@pytest.mark.parametrize("dim,rows", [(64, 16), (64, 30), (64, 50), (64, 90), (128, 8), (128, 32), (128, 42),
                                      (128, 60), (256, 16), (256, 26), (256, 50)])
@pytest.mark.parametrize("hkv", [3, 4])
@pytest.mark.parametrize("dtype,cache", [(BF, BF), (FH, FH), (BF, F8), (FH, F8)])
def test_attend_row_groups(dim, rows, hkv, dtype, cache):
    """Every number of row tiles at lines of many tiles per wave, heads alone and in fours; twice the same
    bits."""
    c = _case([1555, 40, 777], rows // 2, 2 * hkv, hkv, dim, 16, dtype, cache, seed=rows + hkv)
    _check_attend(c)
    assert torch.equal(_attend(c), _attend(c))


@pytest.mark.parametrize("slots", [15, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("blk,hkv", [(1, 4), (9, 4), (9, 1)])
def test_attend_short_tables(slots, blk, hkv):
    """Full lines of tables about as wide as those that are not cut, with and without a status."""
    L = slots * 16 - blk
    c = _case([L, 0, L - 200], blk, 4 * hkv, hkv, 128, 16, BF, BF, seed=slots)
    assert c["table"].shape[1] == slots
    _check_attend(c)
    st = torch.full((3,), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(_attend(c), _attend(c, status=st)) and (st == 0).all()


@pytest.mark.parametrize("batch,blk,hq,hkv,dim,dtype,cache,longest", [
    (400, 1, 6, 3, 64, BF, BF, 100), (301, 9, 12, 3, 128, BF, BF, 100), (257, 3, 4, 2, 256, BF, F8, 60),
    (521, 1, 8, 4, 128, FH, FH, 480), (1100, 2, 1, 1, 80, FH, F8, 30), (103, 20, 20, 5, 128, BF, BF, 40)])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_many_short_lines(batch, blk, hq, hkv, dim, dtype, cache, longest, tree):
    """Enough short jobs for a wave each, idle and empty lines among them."""
    g = _gen(batch)
    lens = torch.randint(0, longest + 1, (batch,), generator=g).tolist()
    live = torch.randint(0, blk + 1, (batch,), generator=g).tolist()
    lens[3], live[3], live[7] = longest, blk, 0
    _check_attend(_case(lens, blk, hq, hkv, dim, 16, dtype, cache, seed=batch, live=live, tree=tree))


@pytest.mark.parametrize("hkv", [3, 4])
def test_attend_values_that_are_not_finite_in_cut_lines(hkv):
    """NaN and infinities in block rows of lines that several workgroups share."""
    c = _case([3000, 2000], 3, 2 * hkv, hkv, 128, 16, BF, BF, seed=hkv, live=[3, 2])
    want = _attend(c).cpu()
    for r, L in ((0, 3000), (1, 2000)):
        for j, bad in ((1, float("inf")), (2, float("nan"))):
            at = c["table"][r, (L + j) // 16].long(), (L + j) % 16
            c["v"][at][..., :hkv, 7] = bad
    got = _attend(c).cpu()
    assert torch.equal(got[0, 0], want[0, 0]) and torch.equal(got[1, 0], want[1, 0])
    other = [d for d in range(128) if d != 7]
    assert torch.equal(got[0, :, :, other], want[0, :, :, other])
    assert torch.isinf(got[0, 1, :, 7]).all() and torch.isinf(got[1, 1, :, 7]).all()
    assert torch.isnan(got[0, 2, :, 7]).all()


@pytest.mark.parametrize("dtype", [BF, FH])
def test_attend_peaked_and_flat_scores(dtype):
    """Scores of +-hundreds (one position takes all the weight, the maximum rises late) and all 0."""
    c = _case([600, 90], 2, 8, 2, 64, 16, dtype, dtype, seed=4, spread=60.0)
    _check_attend(c)
    c["q"].zero_()
    _check_attend(c)
    # the running maximum rises with every position
    c = _case([600], 1, 4, 1, 64, 16, dtype, dtype, seed=4)
    t = torch.arange(601)
    slot = c["table"][0][t // 16].long()
    c["k"][slot, t % 16, 0] = (t[:, None] / 64.0).to(dtype).expand(601, 64)
    c["q"].fill_(1.0)
    _check_attend(c)
    c["scale"] = -c["scale"]
    _check_attend(c)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("tree", [False, True])
def test_attend_ignores_what_a_row_does_not_see(bad, tree):
    """NaN and infinities behind the line's rows (in its last page), in free pages, and in block rows
    that a row does not see, have no effect on it."""
    c = _case([75, 0, 33], 9, 8, 2, 128, 16, BF, BF, seed=21, live=[9, 5, 7], tree=tree)
    lens, live = c["lens"], c["live"]
    used = torch.zeros(c["k"].shape[:2], dtype=torch.bool)
    for r in range(3):
        t = torch.arange(int(lens[r] + live[r]))
        used[c["table"][r][t // 16].long(), t % 16] = True
    for x in (c["k"], c["v"]):
        x[~used] = bad
    _check_attend(c)
    # block rows 3 and 6 of line 0 hold it too: rows that do not see them stay as they were
    want = _attend(c).cpu()
    sees = ref.seen_rows(9, 9, None if not tree else c["parent"][0])
    for j in (3, 6):
        p = 75 + j
        c["k"][c["table"][0, p // 16], p % 16] = bad
        c["v"][c["table"][0, p // 16], p % 16] = bad
    got = _attend(c).cpu()
    clean = [i for i in range(9) if not sees[i, 3] and not sees[i, 6]]
    assert len(clean) >= 3
    assert torch.equal(got[0, clean].view(torch.int16), want[0, clean].view(torch.int16))
    for r, n in ((1, 5), (2, 7)):
        assert torch.equal(got[r, :n].view(torch.int16), want[r, :n].view(torch.int16))
    for i in set(range(9)) - set(clean):
        assert not torch.isfinite(got[0, i].float()).all()


def test_attend_value_infinity_that_is_seen():
    """An infinite value of a block row reaches exactly the rows that see it."""
    c = _case([40], 6, 4, 2, 64, 16, BF, BF, seed=8)
    c["v"][c["table"][0, 42 // 16], 42 % 16, 1, 5] = float("inf")
    got = _attend(c).cpu().float()[0]
    inf = torch.isinf(got)
    assert inf[2:, 2:, 5].all() and int(inf.sum()) == 4 * 2
    want, bound = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], torch.tensor([6]), None,
                                c["scale"])
    ok = ~torch.isinf(want[0])
    assert (((got.double() - want[0]).abs() <= bound[0]) | ~ok).all()


def test_attend_status_and_other_lines():
    c = _case([75, 40, 33, 20], 4, 4, 2, 64, 16, BF, BF, seed=30, tree=True)
    good = _attend(c).cpu()
    pages = c["k"].shape[0]
    c["table"][0, 2] = pages            # a page outside the pool
    c["parent"][1, 2] = 2               # its own parent
    c["lens"][2] = -5
    st = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    got = _attend(c, status=st).cpu()
    assert st.cpu().tolist() == [ref.BAD_PAGE, ref.BAD_PARENT, ref.BAD_PAGE, 0]
    assert torch.equal(got[3], good[3])
    c["live"] = torch.tensor([4, 5, -1, 4], dtype=torch.int32)
    c["lens"][2] = 33
    _attend(c, status=st)
    assert st.cpu().tolist()[1:3] == [ref.BAD_PAGE, ref.BAD_PAGE]


def test_attend_strided_rows_streams_and_reruns():
    """q as a view of a packed projection, out as a view, a stream that is not current, a workspace
    full of NaN: the same bits."""
    c = _case([900, 64, 300], 3, 8, 2, 128, 16, BF, BF, seed=31)
    want = _attend(c).cpu()
    q = torch.zeros((3, 3, 12, 128), dtype=BF, device=DEV)
    q[:, :, :8] = _gpu(c["q"])
    outs = torch.zeros((3, 3, 10, 128), dtype=BF, device=DEV)
    k, v, tab, ln = _gpu(c["k"]), _gpu(c["v"]), _gpu(c["table"]), _gpu(c["lens"])
    wide = torch.full((3, tab.shape[1] + 5), 2**30, dtype=torch.int32, device=DEV)
    wide[:, :tab.shape[1]] = tab
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.full((paged_attention_workspace_bytes(3, 3, 8, 2, 128),), 255, dtype=torch.uint8,
                    device=DEV)
    torch.cuda.synchronize()
    for _ in range(3):
        o = psispec_paged_attention(q[:, :, :8], k, v, wide[:, :tab.shape[1]], ln,
                                    scale=c["scale"], out=outs[:, :, 1:9], workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(o.cpu(), want)
        assert (outs[:, :, 0] == 0).all() and (outs[:, :, 9] == 0).all()
        outs.zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("ps", [16, 24])
def test_pages_far_apart(ps):
    """A page stride of 2^31 elements (2^32 bytes), append and attention."""
    raw = torch.empty(3 * 2**31, dtype=BF, device=DEV)
    k, v = (torch.as_strided(raw, (3, ps, 2, 64), (2**31, 256, 64, 1), at) for at in (0, 128))
    c = _append_case([ps + 3], 4, 4, 2, 64, ps, BF, BF, seed=ps, rot=64, norm=False)
    tab = torch.tensor([[2, 0]], dtype=torch.int32)
    args = [_gpu(x) for x in (tab, c["lens"])]
    near = [torch.empty((3, ps, 2, 64), dtype=BF, device=DEV) for _ in range(2)]
    for kc, vc in ((k, v), near):
        kc.copy_(torch.randn((3, ps, 2, 64), generator=_gen(1)).to(BF))
        vc.copy_(torch.randn((3, ps, 2, 64), generator=_gen(2)).to(BF))
    outs = []
    for kc, vc in ((k, v), near):
        q = psispec_qkv_append(*_gpu(c["qkv"]).split([4, 2, 2], 2), kc, vc, *args, inv_freq=_gpu(c["f"]))
        outs.append(psispec_paged_attention(q, kc, vc, *args))
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(k, near[0]) and torch.equal(v, near[1])


def test_attend_pool_beyond_32_bits():
    """Pages past 2^31 elements of the pool."""
    ps, hkv, d = 16, 8, 128
    pages = (2**31) // (ps * hkv * d) + 64
    k = torch.zeros((pages, ps, hkv, d), dtype=F8, device=DEV)
    v = torch.zeros((pages, ps, hkv, d), dtype=F8, device=DEV)
    c = _case([700], 1, 8, 8, 128, 16, BF, F8, seed=77)
    n = c["k"].shape[0]
    k[pages - n:] = c["k"].to(DEV)
    v[pages - n:] = c["v"].to(DEV)
    want = _attend(c).cpu()
    got = psispec_paged_attention(_gpu(c["q"]), k, v, _gpu(c["table"] + (pages - n)), _gpu(c["lens"]),
                                  scale=c["scale"], k_scale=_gpu(c["ks"]), v_scale=_gpu(c["vs"])).cpu()
    assert torch.equal(got, want)


def _guarded(n):
    """A workspace of n bytes inside a buffer of 165s, and the buffer."""
    raw = torch.full((n + 8192,), 165, dtype=torch.uint8, device=DEV)
    return raw[4096:4096 + n], raw


def _guards_whole(raw):
    return bool((raw[:4096] == 165).all() and (raw[-4096:] == 165).all())


@pytest.mark.parametrize("batch,blk,hq,hkv,dim,cache,longest,tree", [
    (1, 1, 8, 8, 128, BF, 4000, False), (5, 9, 16, 4, 128, BF, 3000, True), (3, 50, 8, 4, 64, F8, 900, False),
    (200, 2, 8, 8, 256, BF, 600, True), (900, 1, 4, 4, 64, BF, 700, False), (700, 3, 4, 2, 128, F8, 60, True),
    (2, 1024, 2, 1, 64, BF, 100, True)])
def test_attend_workspace_bounds(batch, blk, hq, hkv, dim, cache, longest, tree):
    """Nothing outside the workspace and the outputs is written, however the work is cut."""
    g = _gen(batch + blk)
    lens = torch.randint(0, longest + 1, (batch,), generator=g).tolist()
    c = _case(lens, blk, hq, hkv, dim, 16, BF, cache, seed=blk, tree=tree)
    want = _attend(c)
    ws, raw = _guarded(paged_attention_workspace_bytes(batch, blk, hq, hkv, dim))
    rows = torch.full((batch + 2, blk, hq, dim), 5.0, dtype=BF, device=DEV)
    got = _attend(c, workspace=ws, out=rows[1:-1])
    assert torch.equal(got, want) and _guards_whole(raw)
    assert (rows[0] == 5.0).all() and (rows[-1] == 5.0).all()


@pytest.mark.parametrize("batch,slots,pages,blk", [(5, 9, 100, 7), (16, 256, 5000, 33), (700, 5, 9000, 1),
                                                   (1025, 7, 33000, 20), (40, 200, 8200, 900)])
def test_pages_workspace_bounds(batch, slots, pages, blk):
    """Calls with guards around the workspace, the table, the counts and the lengths."""
    ps = 4
    ws, raw = _guarded(pages_workspace_bytes(batch, slots, pages, blk, ps))
    held = [torch.full((n + 2048,), 0x25A5A5A5, dtype=torch.int32, device=DEV) for n in
            (batch * slots, pages, batch, batch)]
    tab, refs, ln, st = (x[1024:-1024] for x in held)
    tab.fill_(-1)
    refs.zero_()
    ln.zero_()
    tab = tab.view(batch, slots)
    pool = torch.zeros((2, pages, ps, 4), dtype=torch.int32, device=DEV)
    n = torch.full((batch,), min(blk, slots * ps // 2), dtype=torch.int32, device=DEV)
    psispec_pages_reserve(pool, tab, refs, ln, blk, n_new=n, status=st, workspace=ws)
    ln.copy_(torch.where(st == 0, n, 0))
    src = torch.arange(batch, dtype=torch.int32, device=DEV).flip(0).contiguous()
    psispec_pages_assign(tab, refs, ln, src, ln.flip(0).contiguous(), ps, status=st, workspace=ws)
    assert (st == 0).all()
    psispec_pages_reserve(pool, tab, refs, ln, blk, n_new=torch.ones_like(n), status=st, workspace=ws)
    assert _guards_whole(raw)
    for x in held:
        assert (x[:1024] == 0x25A5A5A5).all() and (x[-1024:] == 0x25A5A5A5).all()
    used = tab[tab >= 0].long()
    assert torch.equal(torch.bincount(used, minlength=pages).to(torch.int32), refs)


# ------------------------------------------------------------------------------------- append

def _append_case(lens, blk, hq, hkv, dim, ps, dtype, cache, seed, rot, inter=False, norm=True,
                 live=None, positions=None, rope_scale=1.0, packed=True):
    g = _gen(seed)
    tab, pages = _make_table(lens, blk, ps, g)
    c = dict(lens=torch.tensor(lens, dtype=torch.int32), table=tab, inter=inter, rs=rope_scale,
             packed=packed, pos=positions)
    c["live"] = None if live is None else torch.tensor(live, dtype=torch.int32)
    c["qkv"] = (torch.randn((len(lens), blk, hq + 2 * hkv, dim), generator=g) * 1.5).to(dtype)
    c["hq"], c["hkv"] = hq, hkv
    c["kc"] = torch.randn((pages, ps, hkv, dim), generator=g).to(cache)
    c["vc"] = torch.randn((pages, ps, hkv, dim), generator=g).to(cache)
    c["ks"] = c["vs"] = None
    if cache == F8:
        c["ks"], c["vs"] = (0.02 + 0.02 * torch.rand(hkv, generator=g) for _ in range(2))
        c["vs"][0] = 1e-3  # values beyond 448 scales are clamped
    c["qw"], c["kw"] = ((1 + 0.3 * torch.randn(dim, generator=g)).to(dtype) if norm else None
                        for _ in range(2))
    c["f"] = rope_frequencies(rot, 500000.0)[0] if rot else None
    return c


def _check_append(c, **kw):
    hq, hkv = c["hq"], c["hkv"]
    b, blk, _, dim = c["qkv"].shape
    dt, ct = c["qkv"].dtype, c["kc"].dtype
    live = c["live"] if c["live"] is not None else torch.full((b,), blk)
    ps = c["kc"].shape[1]
    parts = _gpu(c["qkv"]).split([hq, hkv, hkv], 2)
    if not c["packed"]:
        parts = [x.contiguous() for x in parts]
    kc, vc = _gpu(c["kc"]), _gpu(c["vc"])
    q_out = torch.full((b, blk, hq, dim), 7.0, dtype=dt, device=DEV)
    st = torch.full((b,), -1, dtype=torch.int32, device=DEV)
    got = psispec_qkv_append(*parts, kc, vc, _gpu(c["table"]), _gpu(c["lens"]), n_new=_gpu(c["live"]),
                             positions=_gpu(c["pos"]), q_weight=_gpu(c["qw"]), k_weight=_gpu(c["kw"]),
                             eps=1e-5, inv_freq=_gpu(c["f"]), interleaved=c["inter"],
                             rope_scale=c["rs"], k_scale=_gpu(c["ks"]), v_scale=_gpu(c["vs"]),
                             q_out=q_out, status=st, **kw).cpu()
    assert (st.cpu() == 0).all()
    kc, vc = kc.cpu(), vc.cpu()
    wrote = torch.zeros(c["kc"].shape[:2], dtype=torch.bool)
    for r in range(b):
        n, L = int(live[r]), int(c["lens"][r])
        assert (got[r, n:] == 7.0).all()
        if n == 0:
            continue
        pos = c["pos"][r, :n] if c["pos"] is not None else torch.arange(L, L + n)
        x = c["qkv"][r, :n]
        yq, eq = ref.prepared(x[:, :hq], c["qw"], 1e-5, pos, c["f"], c["inter"], c["rs"])
        yk, ek = ref.prepared(x[:, hq:hq + hkv], c["kw"], 1e-5, pos, c["f"], c["inter"], c["rs"])
        yv = x[:, hq + hkv:].double()
        ev = torch.zeros_like(yv)
        assert ((got[r, :n].double() - yq).abs() <= ref.stored_bound(yq, eq, dt)).all()
        t = torch.arange(L, L + n)
        page, off = c["table"][r][t // ps].long(), t % ps
        wrote[page, off] = True
        for cache, y, e, s in ((kc, yk, ek, c["ks"]), (vc, yv, ev, c["vs"])):
            if s is not None:
                y, e = y / s.double()[:, None], e / s.double()[:, None]
                e = e + 2.0**-23 * y.abs()  # the division's rounding
                y = y.clamp(-448, 448)
            err = (cache[page, off].double() - y).abs()
            assert (err <= ref.stored_bound(y, e, ct)).all()
        if ct != F8:
            assert torch.equal(vc[page, off], x[:, hq + hkv:])
    for new, old in ((kc, c["kc"]), (vc, c["vc"])):
        raw = torch.uint8 if ct == F8 else torch.int16
        assert torch.equal(new.view(raw)[~wrote], old.view(raw)[~wrote])


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 64), (80, 32), (96, 96), (112, 48),
                                     (256, 256), (16, 16), (48, 16), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("cache", ["same", "f8"])
def test_append_dims_and_layouts(dim, rot, inter, cache):
    dt = BF if dim % 32 else FH
    _check_append(_append_case([5, 0, 37], 3, 6, 2, dim, 16, dt, dt if cache == "same" else F8,
                               seed=dim + rot, rot=rot, inter=inter))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 8), (7, 7), (40, 8), (64, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_append_heads(hq, hkv, norm):
    _check_append(_append_case([100, 31], 9, hq, hkv, 128, 16, BF, BF, seed=hq, rot=128, norm=norm,
                               packed=norm))


@pytest.mark.parametrize("ps", [1, 7, 16, 64, 4096])
def test_append_pages_padding_positions(ps):
    g = _gen(ps)
    pos = torch.randint(-50, 2**30, (4, 5), generator=g).to(torch.int32)
    _check_append(_append_case([0, 13, 200, 63], 5, 4, 2, 64, ps, FH, FH, seed=ps, rot=64,
                               live=[5, 0, 3, 1], positions=pos, rope_scale=1.21))


def test_append_far_positions_and_long_blocks():
    _check_append(_append_case([1000003], 3, 2, 1, 64, 4096, BF, BF, seed=2, rot=64))
    _check_append(_append_case([17, 900], 700, 4, 2, 64, 16, BF, F8, seed=3, rot=64, live=[700, 650]))


def test_append_in_place_and_status():
    c = _append_case([40, 20, 10], 4, 4, 2, 128, 16, BF, BF, seed=11, rot=128)
    q, k, v = _gpu(c["qkv"]).split([4, 2, 2], 2)
    kw = dict(q_weight=_gpu(c["qw"]), k_weight=_gpu(c["kw"]), inv_freq=_gpu(c["f"]))
    kc, vc = _gpu(c["kc"]), _gpu(c["vc"])
    want = psispec_qkv_append(q, k, v, kc, vc, _gpu(c["table"]), _gpu(c["lens"]), **kw).clone()
    qq = q.clone(memory_format=torch.contiguous_format)
    psispec_qkv_append(qq, k, v, kc, vc, _gpu(c["table"]), _gpu(c["lens"]), q_out=qq, **kw)
    assert torch.equal(qq, want)
    packed = _gpu(c["qkv"])
    qp, kp, vp = packed.split([4, 2, 2], 2)
    psispec_qkv_append(qp, kp, vp, kc, vc, _gpu(c["table"]), _gpu(c["lens"]), q_out=qp, **kw)
    assert torch.equal(qp, want)
    # line 0: one of its two pages missing (rows 40..43 lie in slot 2); line 1: too long
    tab, ln = c["table"].clone(), c["lens"].clone()
    tab[0, 2] = -1
    ln[1] = tab.shape[1] * 16 - 3
    st = torch.full((3,), -1, dtype=torch.int32, device=DEV)
    kc2, vc2 = _gpu(c["kc"]), _gpu(c["vc"])
    out = torch.full((3, 4, 4, 128), 7.0, dtype=BF, device=DEV)
    psispec_qkv_append(q, k, v, kc2, vc2, _gpu(tab), _gpu(ln), q_out=out, status=st, **kw)
    assert st.cpu().tolist() == [ref.BAD_PAGE, ref.BAD_PAGE, 0]
    assert (out[:2] == 7.0).all() and torch.equal(out[2], want[2])
    t = torch.arange(10, 14)
    page, off = c["table"][2][t // 16].long(), t % 16
    keep = torch.ones(kc2.shape[:2], dtype=torch.bool)
    keep[page, off] = False
    assert torch.equal(kc2.cpu()[keep], c["kc"][keep]) and torch.equal(vc2.cpu()[keep], c["vc"][keep])
    assert torch.equal(kc2.cpu()[page, off], kc.cpu()[page, off])


def test_append_keeps_nan_and_infinity():
    c = _append_case([0], 2, 1, 1, 64, 16, BF, F8, seed=1, rot=0, norm=False)
    c["qkv"][0, 0, 2, 3], c["qkv"][0, 0, 2, 4] = float("nan"), float("inf")
    kc, vc = _gpu(c["kc"]), _gpu(c["vc"])
    psispec_qkv_append(*_gpu(c["qkv"]).split([1, 1, 1], 2), kc, vc, _gpu(c["table"]), _gpu(c["lens"]))
    got = vc.cpu().float()[int(c["table"][0, 0]), 0, 0]
    assert torch.isnan(got[3]) and got[4] == 448.0 and torch.isfinite(got[5:]).all()


# ------------------------------------------------------------------------------------- pages

def _np_pool(planes, pages, ps, words, seed):
    return np.random.default_rng(seed).integers(-2**31, 2**31 - 1, (planes, pages, ps, words),
                                                dtype=np.int64).astype(np.int32)


def _run_commit(pool, tab, ln, blk, n, keep):
    pg, lg = torch.from_numpy(pool).to(DEV), torch.from_numpy(ln).to(DEV)
    nl = torch.full_like(lg, -9)
    st = torch.full_like(lg, -1)
    psispec_paged_commit(pg, torch.from_numpy(tab).to(DEV), lg, blk, torch.from_numpy(n).to(DEV),
                         keep=None if keep is None else torch.from_numpy(keep).to(DEV), new_length=nl,
                         status=st)
    po = pool.copy()
    want, sto = ref.commit(po, tab, ln, blk, n, keep, pool.shape[2])
    assert st.cpu().numpy().tolist() == sto.tolist()
    assert nl.cpu().numpy().tolist() == want.tolist()
    assert np.array_equal(lg.cpu().numpy(), ln)
    assert np.array_equal(pg.cpu().numpy(), po)
    return sto


@pytest.mark.parametrize("planes,words,ps,blk,batch,maxk", [
    (1, 4, 1, 8, 3, 8), (2, 8, 16, 32, 9, 8), (3, 260, 5, 33, 4, 33), (56, 512, 16, 32, 5, 8),
    (2, 1028, 64, 17, 6, 17), (1, 4, 256, 1024, 2, 700)])
def test_commit_random_paths(planes, words, ps, blk, batch, maxk):
    rng = np.random.default_rng(planes * 31 + ps)
    lens = rng.integers(0, 3 * ps + 40, batch).astype(np.int32)
    tab, pages = _make_table(lens.tolist(), blk, ps, _gen(ps), extra_slots=blk)
    tab = tab.numpy()
    for seed in range(2):
        n = rng.integers(0, min(maxk, blk) + 1, batch).astype(np.int32)
        keep = np.full((batch, maxk), -1, np.int32)
        for r in range(batch):
            keep[r, :n[r]] = np.sort(rng.choice(blk, n[r], replace=False))
        pool = _np_pool(planes, pages, ps, words, seed)
        assert (_run_commit(pool, tab, lens, blk, n, keep) == 0).all()
        assert (_run_commit(pool, tab, lens, blk, n, None) == 0).all()


def test_commit_invalid_lines():
    lens = np.array([5, 20, 9, 30, 40, 3, 11], np.int32)
    tab, pages = _make_table(lens.tolist(), 6, 8, _gen(1))
    tab = tab.numpy()
    tab[6, 1] = pages + 3                   # the page of a row that moves
    pool = _np_pool(2, pages, 8, 4, 1)
    n = np.array([7, 2, 1, 1, 2, 2, 2], np.int32)
    keep = np.array([[0, 1, 2, 3, 4, 5, 5], [3, 3] + [-1] * 5, [6] + [-1] * 6, [5] + [-1] * 6,
                     [1, 4] + [-1] * 5, [-1, 2] + [-1] * 5, [1, 5] + [-1] * 5], np.int32)
    lens[3] = tab.shape[1] * 8 - 5
    st = _run_commit(pool, tab, lens, 6, n, keep)
    assert st.tolist() == [32, 32, 32, 32, 0, 32, 64]


def test_commit_in_place_length_and_tree_verify():
    """accept_len and accept_nodes of the tree verify go straight in; length advances in place."""
    tin = workloads.make_tree("c4b", device=DEV, batch=6, V=2000)
    N, D = tin.preset.N, tin.preset.depth
    lens = np.array([0, 7, 30, 16, 15, 90], np.int32)
    tab, pages = _make_table(lens.tolist(), N, 16, _gen(5))
    pool = _np_pool(4, pages, 16, 8, 3)
    o = psispec_verify_tree(tin.p, tin.parent, tin.node_tokens, D, seed=tin.seed, step=1)
    pg, lg = torch.from_numpy(pool).to(DEV), torch.from_numpy(lens).to(DEV)
    psispec_paged_commit(pg, tab.to(DEV), lg, N, o["accept_len"], keep=o["accept_nodes"])
    want, st = ref.commit(pool, tab.numpy(), lens, N, o["accept_len"].cpu().numpy(),
                          o["accept_nodes"].cpu().numpy(), 16)
    assert (st == 0).all() and np.array_equal(pg.cpu().numpy(), pool)
    assert lg.cpu().numpy().tolist() == want.tolist()


class _Pages:
    """One cache on the GPU and its reference, kept in step."""

    def __init__(self, planes, pages, ps, words, batch, slots, seed):
        self.ps = ps
        self.pool = _np_pool(planes, pages, ps, words, seed)
        self.tab = np.full((batch, slots), -1, np.int32)
        self.refs = np.zeros(pages, np.int32)
        self.len = np.zeros(batch, np.int32)
        self.g = [torch.from_numpy(x.copy()).to(DEV) for x in (self.pool, self.tab, self.refs, self.len)]

    def assign(self, src, new):
        src, new = np.asarray(src, np.int32), np.asarray(new, np.int32)
        st = torch.full((len(src),), -1, dtype=torch.int32, device=DEV)
        _, tab, refs, ln = self.g
        psispec_pages_assign(tab, refs, ln, torch.from_numpy(src).to(DEV),
                             torch.from_numpy(new).to(DEV), self.ps, status=st)
        want = ref.assign(self.tab, self.refs, self.len, src, new, self.ps)
        assert st.cpu().numpy().tolist() == want.tolist()
        self.same()
        return want

    def reserve(self, blk, n=None):
        pool, tab, refs, ln = self.g
        st = torch.full_like(ln, -1)
        nn = None if n is None else torch.tensor(n, dtype=torch.int32, device=DEV)
        psispec_pages_reserve(pool, tab, refs, ln, blk, n_new=nn, status=st)
        want = ref.reserve(self.pool, self.tab, self.refs, self.len, blk,
                           [blk] * len(self.len) if n is None else n, self.ps)
        assert st.cpu().numpy().tolist() == want.tolist()
        self.same()
        return want

    def grow(self, n):
        self.len += np.asarray(n, np.int32)
        self.g[3].copy_(torch.from_numpy(self.len))

    def same(self):
        for x, y in zip(self.g, (self.pool, self.tab, self.refs, self.len)):
            assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("ps", [1, 5, 16, 64])
@pytest.mark.parametrize("batch", [1, 7, 300])
def test_pages_random_life(ps, batch):
    """Random reservations, growth, forks, cuts, frees and reorders, with a pool
    that may run short."""
    rng = np.random.default_rng(ps * 1000 + batch)
    slots = 200 // ps + 4
    pages = max(6, int(batch * 60 / ps * 0.8))
    c = _Pages(2, pages, ps, 4, batch, slots, 1)
    for step in range(12):
        n = rng.integers(0, 25, batch)
        n = np.minimum(n, np.maximum(slots * ps - c.len, 0))
        st = c.reserve(24, n.tolist())
        c.grow(np.where(st == 0, rng.integers(0, n + 1), 0))
        src = np.arange(batch)
        new = c.len.copy()
        kind = rng.random(batch)
        other = rng.integers(0, batch, batch)
        src = np.where(kind < 0.3, other, np.where(kind > 0.85, -1, src))
        new = np.where(src >= 0, c.len[np.maximum(src, 0)], 0)
        new = np.where(rng.random(batch) < 0.3, rng.integers(0, new + 1), new)
        assert (c.assign(src, new) == 0).all()
        assert (np.bincount(c.tab[c.tab >= 0], minlength=pages) == c.refs).all()


def test_pages_beam_reorder_and_shared_tail():
    c = _Pages(3, 40, 16, 8, 4, 8, 2)
    assert (c.reserve(50) == 0).all()
    c.grow([37, 0, 0, 0])
    c.assign([0, -1, -1, -1], [37, 0, 0, 0])       # the empty lines give their pages back
    assert c.refs.sum() == 3
    c.assign([0, 0, 0, 0], [37, 37, 32, 5])         # fork, fork at a page's end, fork a prefix
    assert sorted(c.refs[c.refs > 0].tolist()) == [2, 3, 4]
    assert (c.reserve(9) == 0).all()                # tails copied, none shared any more
    c.grow([9, 9, 9, 9])
    c.assign([2, 1, 1, 0], [41, 46, 46, 46])        # reorder
    c.assign([-1] * 4, [0] * 4)
    assert (c.refs == 0).all() and (c.tab == -1).all()


def test_pages_invalid_lines():
    c = _Pages(1, 12, 4, 4, 5, 6, 3)
    c.reserve(7, [7, 7, 3, 0, 0])
    c.grow([6, 7, 3, 0, 0])
    st = c.assign([0, 9, 2, 1, -2], [7, 0, -1, 7, 0])
    assert st.tolist() == [64, 64, 64, 0, 64]
    st = c.reserve(7, [8, -1, 7, 7, 7])
    assert st.tolist() == [64, 64, 0, 0, 0]
    c.tab[0, 0] = 99
    c.g[1].copy_(torch.from_numpy(c.tab))
    assert c.assign([0, 0, 2, 3, 4], [6, 2, 3, 7, 0]).tolist() == [64, 64, 0, 0, 0]


def test_pages_many_chunks_of_pages():
    """More pages than one workgroup scans; the free ones scattered."""
    c = _Pages(1, 20000, 1, 4, 3, 64, 4)
    c.refs[:] = 1
    free = np.sort(np.random.default_rng(1).choice(20000, 100, replace=False))
    c.refs[free] = 0
    c.g[2].copy_(torch.from_numpy(c.refs))
    assert c.reserve(40, [40, 30, 40]).tolist() == [0, 0, ref.NO_PAGE]
    assert c.tab[0, :40].tolist() == free[:40].tolist()


@pytest.mark.parametrize("batch,slots,ps,pages", [(1, 4096, 1, 4096), (1, 4097, 1, 4097), (64, 64, 4, 32768),
                                                  (64, 65, 4, 32769), (1024, 4, 16, 9000), (1025, 4, 16, 9000),
                                                  (17, 40, 8, 5000)])
def test_pages_sizes_about_one_workgroup(batch, slots, ps, pages):
    """Tables and pools just within and just beyond what one workgroup does alone."""
    rng = np.random.default_rng(batch + slots)
    c = _Pages(1, pages, ps, 4, batch, slots, 5)
    blk = min(2 * ps + 1, slots * ps - 1)
    for step in range(3):
        n = np.minimum(rng.integers(0, blk + 1, batch), slots * ps - c.len)
        st = c.reserve(blk, n.tolist())
        c.grow(np.where(st == 0, n, 0))
        src = np.where(rng.random(batch) < 0.4, rng.integers(0, batch, batch), np.arange(batch))
        src = np.where(rng.random(batch) < 0.1, batch, src)  # refused
        new = np.where(src < batch, c.len[np.minimum(src, batch - 1)], 0)
        st = c.assign(src, np.maximum(new - (rng.random(batch) < 0.3), 0))
        assert (st == np.where(src < batch, 0, ref.BAD_PAGE)).all()
    c.reserve(max(min(300, slots * ps - int(c.len.max())), 1))  # the lines that this does not fit are refused


# ------------------------------------------------------------------------------------- together

def test_reserve_append_attend_verify_commit_loop():
    """Rounds of the verify path over one paged cache: reserve, append, attention, tree verify, commit,
    with a fork of a line and the freeing of another between them.  Every attention is checked against
    the rows that the line should hold by then."""
    g = _gen(40)
    batch, N, hq, hkv, dim, ps = 4, 15, 8, 2, 64, 16
    tin = workloads.make_tree("c4b", device=DEV, batch=batch, V=512, N=N)
    D = tin.preset.depth
    pages, slots = 60, 12
    pool = torch.zeros((2, pages, ps, hkv, dim), dtype=BF, device=DEV)
    tab = torch.full((batch, slots), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ln = torch.zeros(batch, dtype=torch.int32, device=DEV)
    inv = rope_frequencies(dim, 10000.0, "by_parts", 4.0, 64)
    depth = torch.zeros((batch, N), dtype=torch.int32)
    par = tin.parent.cpu()
    for j in range(N):
        for r in range(batch):
            depth[r, j] = 0 if par[r, j] < 0 else depth[r, par[r, j]] + 1
    lines = [[] for _ in range(batch)]  # the rows (k, v) that each line should hold
    kept = 0
    for step in range(5):
        st = torch.empty(batch, dtype=torch.int32, device=DEV)
        psispec_pages_reserve(pool, tab, refs, ln, N, status=st)
        assert (st == 0).all()
        qkv = torch.randn((batch, N, hq + 2 * hkv, dim), generator=g).to(BF)
        q, k, v = _gpu(qkv).split([hq, hkv, hkv], 2)
        pos = ln.cpu()[:, None] + depth
        qo = psispec_qkv_append(q, k, v, pool[0], pool[1], tab, ln, positions=_gpu(pos),
                                inv_freq=_gpu(inv[0]), rope_scale=inv[1], status=st)
        assert (st == 0).all()
        out = psispec_paged_attention(qo, pool[0], pool[1], tab, ln, parent=tin.parent, status=st)
        assert (st == 0).all()
        o = psispec_verify_tree(tin.p, tin.parent, tin.node_tokens, D, seed=3, step=step)
        # the reference keeps each line's rows as a plain list
        kc, vc = pool[0].cpu(), pool[1].cpu()
        tabc, lnc = tab.cpu(), ln.cpu()
        for r in range(batch):
            L = int(lnc[r])
            assert L == len(lines[r])
            t = torch.arange(L, L + N)
            page, off = tabc[r][t // ps].long(), t % ps
            new = list(zip(kc[page, off], vc[page, off]))
            dense = [torch.stack([x[w] for x in lines[r] + new])[None] for w in range(2)]
            want, bound = ref.attention(qo[r:r + 1].cpu(), *dense, torch.zeros((1, 1), dtype=torch.int32),
                                        [L], [N], par[r:r + 1], dim ** -0.5)
            assert ((out[r].cpu().double() - want[0]).abs() <= bound[0]).all()
            n = int(o["accept_len"][r])
            kept += n
            lines[r] += [new[int(j)] for j in o["accept_nodes"][r, :n]]
        psispec_paged_commit(pool, tab, ln, N, o["accept_len"], keep=o["accept_nodes"], status=st)
        assert (st == 0).all()
        if step == 2:  # line 3 becomes a copy of line 1, line 0 starts anew
            src = torch.tensor([-1, 1, 2, 1], dtype=torch.int32, device=DEV)
            psispec_pages_assign(tab, refs, ln, src, ln[[0, 1, 2, 1]].contiguous(), ps, status=st)
            assert (st == 0).all()
            lines[0], lines[3] = [], list(lines[1])
        torch.cuda.synchronize()
    assert kept > 0


def test_graph_replays():
    """Reserve, append, attention and commit recorded into one HIP graph and replayed with other
    inputs, lengths and tables between the replays, against the eager calls."""
    g = _gen(41)
    batch, blk, hq, hkv, dim, ps = 5, 9, 8, 2, 128, 16
    pages, slots = 80, 12

    def state(seed):
        gg = _gen(seed)
        s = dict(pool=torch.randn((2, pages, ps, hkv, dim), generator=gg).to(BF),
                 tab=torch.full((batch, slots), -1, dtype=torch.int32),
                 refs=torch.zeros(pages, dtype=torch.int32),
                 ln=torch.randint(0, 90, (batch,), generator=gg).to(torch.int32),
                 qkv=torch.randn((batch, blk, hq + 2 * hkv, dim), generator=gg).to(BF),
                 nk=torch.randint(0, blk + 1, (batch,), generator=gg).to(torch.int32),
                 live=torch.tensor([9, 9, 9, 0, 9], dtype=torch.int32))
        at = 0
        for r in range(batch):
            n = -(-int(s["ln"][r]) // ps)
            s["tab"][r, :n] = torch.arange(at, at + n)
            s["refs"][at:at + n] = 1
            at += n
        s["nk"] = torch.minimum(s["nk"], s["live"])
        return {k: v.to(DEV) for k, v in s.items()}

    inv = _gpu(rope_frequencies(dim, 500000.0)[0])

    def step(s, out, ws):
        psispec_pages_reserve(s["pool"], s["tab"], s["refs"], s["ln"], blk, n_new=s["live"], workspace=ws[0])
        q, k, v = s["qkv"].split([hq, hkv, hkv], 2)
        qo = psispec_qkv_append(q, k, v, s["pool"][0], s["pool"][1], s["tab"], s["ln"], n_new=s["live"],
                                inv_freq=inv)
        psispec_paged_attention(qo, s["pool"][0], s["pool"][1], s["tab"], s["ln"], n_new=s["live"],
                                out=out, workspace=ws[1])
        psispec_paged_commit(s["pool"], s["tab"], s["ln"], blk, s["nk"])

    def work():
        sizes = (pages_workspace_bytes(batch, slots, pages, blk, ps),
                 paged_attention_workspace_bytes(batch, blk, hq, hkv, dim))
        return [torch.empty(n, dtype=torch.uint8, device=DEV) for n in sizes]

    cap = state(0)
    out = torch.zeros((batch, blk, hq, dim), dtype=BF, device=DEV)
    ws = work()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cap, out, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap, out, ws)
    ws2 = work()
    for seed in range(1, 5):
        fresh = state(seed)
        for k in cap:
            cap[k].copy_(fresh[k])
        out.zero_()
        want = torch.zeros_like(out)
        step(fresh, want, ws2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for k in cap:
            assert torch.equal(cap[k], fresh[k]), k


# ------------------------------------------------------------------------------------- refusals

def test_binding_refusals():
    c = _case([20], 2, 4, 2, 64, 16, BF, BF, seed=1)
    q, k, v, tab, ln = (_gpu(c[x]) for x in ("q", "k", "v", "table", "lens"))
    ok = dict(q=q, k_cache=k, v_cache=v, table=tab, length=ln)
    psispec_paged_attention(**ok)
    f8 = k.float().to(F8)
    for change, word in [
            (dict(q=q.float()), "bfloat16"), (dict(q=q.cpu()), "GPU"), (dict(k_cache=k.to(FH)), "k_cache"),
            (dict(v_cache=v[:, :8]), "k_cache"), (dict(table=tab.long()), "table"),
            (dict(table=tab[:, ::2] if tab.shape[1] > 2 else tab.t()), "table"),
            (dict(length=ln.long()), "length"), (dict(length=ln[:0]), "length"),
            (dict(q=q.transpose(2, 3)), "rows"), (dict(k_scale=torch.ones(2, device=DEV)), "float8"),
            (dict(k_cache=f8, v_cache=f8, k_scale=torch.ones(3, device=DEV)), "k_scale"),
            (dict(q=q[:, :, :3]), "unsupported"), (dict(parent=ln), "parent"),
            (dict(scale=float("inf")), "invalid argument"), (dict(out=q.float()), "out"), (dict(out=q), "invalid argument"),
            (dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV)), "workspace"),
            (dict(q=torch.zeros((1, 1025, 4, 64), dtype=BF, device=DEV)), "unsupported"),
            (dict(n_new=ln.to(torch.int64)), "n_new"), (dict(status=ln.float()), "status"),
            (dict(v_cache=v.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)), "strides")]:
        with pytest.raises(PsispecError, match=word):
            psispec_paged_attention(**{**ok, **change})
    kk = torch.zeros((1, 2, 2, 64), dtype=BF, device=DEV)
    oka = dict(q=q, k=kk, v=kk, k_cache=k, v_cache=v, table=tab, length=ln)
    psispec_qkv_append(**oka)
    for change, word in [
            (dict(k=kk[:, :1]), "k and v"), (dict(k=kk.to(FH)), "k must"),
            (dict(inv_freq=torch.ones(32, device=DEV)), "float64"),
            (dict(inv_freq=torch.ones(4, dtype=torch.float64, device=DEV)), "invalid argument"),
            (dict(inv_freq=torch.ones(40, dtype=torch.float64, device=DEV)), "invalid argument"),
            (dict(eps=-1.0), "invalid argument"), (dict(rope_scale=float("nan")), "invalid argument"),
            (dict(q_weight=torch.ones(64, device=DEV)), "q_weight"),
            (dict(q_out=q[:, :1]), "q_out"), (dict(positions=ln), "positions"),
            (dict(k_cache=k[:1].expand(4, -1, -1, -1), v_cache=v[:1].expand(4, -1, -1, -1)), "invalid argument")]:
        with pytest.raises(PsispecError, match=word):
            psispec_qkv_append(**{**oka, **change})
    pool = torch.zeros((2, 8, 16, 8), dtype=torch.int32, device=DEV)
    refs = torch.zeros(8, dtype=torch.int32, device=DEV)
    for change, word in [(dict(pool=pool[..., :3].contiguous()), "invalid argument"), (dict(pool=pool[..., :4]), "row"),
                         (dict(blk=0), "unsupported"), (dict(refs=refs[:4]), "refs")]:
        with pytest.raises(PsispecError, match=word):
            psispec_pages_reserve(**{**dict(pool=pool, table=tab, refs=refs, length=ln, blk=4), **change})
    for change, word in [(dict(blk=0), "invalid argument"), (dict(blk=1025), "invalid argument"), (dict(keep=ln), "keep"),
                         (dict(keep=ln[:, None][:, :0]), "keep")]:
        with pytest.raises(PsispecError, match=word):
            psispec_paged_commit(**{**dict(pool=pool, table=tab, length=ln, blk=4, n_keep=ln), **change})
    with pytest.raises(PsispecError, match="unsupported"):
        psispec_pages_assign(tab, refs, ln, ln, ln.clone(), 5000)
