"""The paged-cache calls at the borders of their numbers and sizes: small softmax weights under a large
one, values that are not finite, and the largest sizes."""
import pytest
import torch

import paged_ref as ref
from lossless_draft_verification_spec_amd import (
    PsispecError, psispec_paged_attention, psispec_paged_commit, psispec_pages_reserve, psispec_qkv_append)
from test_gpu_paged import (BF, DEV, F8, FH, _append_case, _attend, _case, _check_attend, _gen, _gpu,
                            _make_table)

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (FH, FH), (BF, F8), (FH, F8)]


# ------------------------------------------------------------------ small weights under a large one

def _sink(c, r, at, depth, mag):
    """Position at[r] of line r scores `depth` above what it scored and has the value 0; every other
    value is between mag / 2 and 3 mag / 2, so that nothing cancels in the sums.  (Dimension 0 of the
    queries is 8 and the scale 1 / 8: dimension 0 of a key is added to its scores.)"""
    page, off = int(c["table"][r, at // 16]), at % 16
    c["k"][page, off, :, 0] = torch.tensor(float(depth)).to(c["k"].dtype)
    c["v"][page, off] = torch.zeros(()).to(c["v"].dtype)


def _sink_case(lens, ats, blk, hq, hkv, dim, dtype, cache, depth, spread, mag=1.0, seed=1, **kw):
    c = _case(lens, blk, hq, hkv, dim, 16, dtype, cache, seed=seed, spread=1.0, **kw)
    g = _gen(seed + 1)
    shape = c["k"].shape
    k = torch.randn(shape, generator=g) * (spread * 8 / (dim - 1) ** 0.5)
    k[..., 0] = 0.0
    c["k"] = k.to(cache)
    c["v"] = (mag * (0.5 + torch.rand(shape, generator=g))).to(cache)
    c["q"][..., 0] = 8.0
    c["scale"] = 0.125
    if cache == F8:
        c["ks"] = torch.ones(hkv)
    for r, at in enumerate(ats):
        if at is not None:
            _sink(c, r, at, depth, mag)
    return c


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("L,at", [(8000, 0), (300, 0), (300, 299), (37, 5)])
@pytest.mark.parametrize("depth", [8, 14, 16, 18, 26, 40])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_attend_small_weights_under_one_large(dtype, cache, L, at, depth, spread):
    """One position `depth` nats above all others, with the value 0: the output is what the small
    weights give."""
    _check_attend(_sink_case([L], [at], 1, 4, 1, 64, dtype, cache, depth, spread, seed=L + depth))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim,blk,hq,hkv,tree", [(64, 9, 8, 2, False), (64, 15, 8, 2, False),
                                                 (128, 9, 8, 4, True), (128, 3, 12, 4, False),
                                                 (256, 9, 4, 1, False), (80, 5, 6, 3, True)])
def test_attend_small_weights_in_row_tiles(dtype, cache, dim, blk, hq, hkv, tree):
    """The same for every number of row tiles, in cut and uncut lines; values of some hundreds."""
    lens = [2500, 700, 90, 3, 0]
    live = [blk, 1, blk, blk // 2, blk]
    _check_attend(_sink_case(lens, [1, 699, 88, 0, 0], blk, hq, hkv, dim, dtype, cache, 18, 1.0, mag=200.0,
                             live=live, tree=tree, seed=dim + blk))


@pytest.mark.parametrize("dtype,cache", [(FH, FH), (FH, F8)])
def test_attend_small_weights_in_many_short_lines(dtype, cache):
    """The same with a wave per line and head."""
    lens = torch.randint(30, 200, (300,), generator=_gen(3)).tolist()
    ats = [L // 2 if r % 3 else None for r, L in enumerate(lens)]
    _check_attend(_sink_case(lens, ats, 1, 4, 4, 128, dtype, cache, 16, 1.0))


@pytest.mark.parametrize("dtype,cache", [(FH, FH), (FH, F8)])
@pytest.mark.parametrize("steps", [[0.0, -12.0, -24.0, -12.0, 0.0], [0.0, -20.0, 6.0, -26.0, 12.0],
                                   [-30.0, 0.0, -30.0, 30.0, -30.0], [0.0, -44.0, -60.0, -30.0, -50.0]])
def test_attend_scores_in_steps(dtype, cache, steps):
    """Runs of positions whose scores lie apart by more than f16's range, up and down; all values of the
    highest run are 0, so the next one gives the output."""
    L = 640
    c = _sink_case([L], [None], 2, 4, 1, 64, dtype, cache, 0, 0.5)
    for i, s in enumerate(steps):
        t = torch.arange(i * 128, (i + 1) * 128)
        page, off = c["table"][0][t // 16].long(), t % 16
        c["k"][page, off, :, 0] = torch.tensor(s).to(cache)
        if s == max(steps):
            c["v"][page, off] = torch.zeros(()).to(cache)
    # the block's rows as low as the lowest run
    t = torch.arange(L, L + 2)
    c["k"][c["table"][0][t // 16].long(), t % 16, :, 0] = torch.tensor(min(steps)).to(cache)
    _check_attend(c)


@pytest.mark.parametrize("cache", [FH, F8])
def test_attend_tail_of_131072_equal_scores(cache):
    """A position of value 1 with 131,072 others 18 nats below it, whose sum is 0.2% of its weight."""
    c = _sink_case([131072], [7], 1, 2, 1, 64, FH, cache, 18, 0.0)
    page, off = int(c["table"][0, 0]), 7
    c["v"][page, off] = torch.ones(()).to(cache)
    _check_attend(c)


# ------------------------------------------------------------------ the end of a table

def test_short_blocks_at_the_end_of_the_table():
    """Lines whose short block ends with the last slot, and a full idle line, through reserve, append,
    attention and commit."""
    ps, slots, blk, hq, hkv, dim = 16, 3, 9, 4, 2, 64
    lens, live, kept = [44, 48, 40, 46, 10], [4, 0, 8, 2, 9], [4, 0, 3, 2, 5]
    g, batch = _gen(5), 5
    pages = batch * slots
    pool = torch.randn((2, pages, ps, hkv, dim), generator=g).to(BF).to(DEV)
    tab = torch.full((batch, slots), -1, dtype=torch.int32)
    for r, L in enumerate(lens):
        tab[r, :-(-L // ps)] = torch.arange(r * slots, r * slots - (-L // ps))
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[tab[tab >= 0].long()] = 1
    tab, refs = tab.to(DEV), refs.to(DEV)
    ln, n = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, live))
    st = torch.full((batch,), -1, dtype=torch.int32, device=DEV)

    def fine():
        ok = (st == 0).all()
        st.fill_(-1)
        return ok

    psispec_pages_reserve(pool, tab, refs, ln, blk, n_new=n, status=st)
    assert fine()
    qkv = torch.randn((batch, blk, hq + 2 * hkv, dim), generator=g).to(BF).to(DEV)
    q = psispec_qkv_append(*qkv.split([hq, hkv, hkv], 2), pool[0], pool[1], tab, ln, n_new=n, status=st)
    assert fine()
    out = psispec_paged_attention(q, pool[0], pool[1], tab, ln, n_new=n, status=st)
    assert fine()
    want, bound = ref.attention(q.cpu(), pool[0].cpu(), pool[1].cpu(), tab.cpu(), lens, live, None, dim**-0.5)
    for r in range(batch):
        assert ((out.cpu().double() - want)[r, :live[r]].abs() <= bound[r, :live[r]]).all()
    nk = torch.tensor(kept, dtype=torch.int32, device=DEV)
    new = torch.full_like(ln, -9)
    psispec_paged_commit(pool, tab, ln, blk, nk, new_length=new, status=st)  # a prefix
    assert fine() and torch.equal(new, ln + nk)
    keep = torch.full((batch, 5), -1, dtype=torch.int32)
    for r, rows in enumerate([[0, 1, 2, 3], [], [1, 6, 7], [0, 1], [0, 2, 3, 5, 8]]):
        keep[r, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
    before, tabc = pool.cpu(), tab.cpu()
    psispec_paged_commit(pool, tab, ln, blk, nk, keep=keep.to(DEV), status=st)  # a path, lengths in place
    assert fine() and ln.cpu().tolist() == [L + k for L, k in zip(lens, kept)]
    after = pool.cpu()
    for r, L in enumerate(lens):
        for i in range(kept[r]):
            s, d = L + int(keep[r, i]), L + i
            assert torch.equal(after[:, tabc[r, d // ps], d % ps], before[:, tabc[r, s // ps], s % ps])


def test_commit_rows_behind_the_table():
    """A kept row, or a kept count, that the table has no position for."""
    pool = torch.zeros((1, 8, 4, 4), dtype=torch.int32, device=DEV)
    tab = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    ln = torch.tensor([4, 5, 8, 2**31 - 1], dtype=torch.int32, device=DEV)
    st = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    nk = torch.tensor([1, 4, 0, 1], dtype=torch.int32, device=DEV)
    new = torch.zeros_like(ln)
    psispec_paged_commit(pool, tab, ln, 6, nk, new_length=new, status=st)
    assert st.tolist() == [0, ref.BAD_KEEP, 0, ref.BAD_KEEP] and new.tolist() == [5, 5, 8, 2**31 - 1]
    keep = torch.tensor([[4], [3], [0], [0]], dtype=torch.int32, device=DEV)
    nk.fill_(1)
    psispec_paged_commit(pool, tab, ln, 6, nk, keep=keep, new_length=new, status=st)
    assert st.tolist() == [ref.BAD_KEEP] * 4 and torch.equal(new, ln)
    keep[:2, 0] = torch.tensor([3, 2])
    psispec_paged_commit(pool, tab, ln, 6, nk, keep=keep, new_length=new, status=st)
    assert st.tolist() == [0, 0, ref.BAD_KEEP, ref.BAD_KEEP] and new.tolist() == [5, 6, 8, 2**31 - 1]


# ------------------------------------------------------------------ where outputs may lie

def test_append_output_beside_its_inputs():
    """q, k, v and q_out as parts of one packed buffer, q_out within the gaps of other rows, and refused
    over k and v."""
    c = _append_case([40, 20], 3, 4, 2, 64, 16, BF, BF, seed=3, rot=64)
    kw = dict(q_weight=_gpu(c["qw"]), k_weight=_gpu(c["kw"]), inv_freq=_gpu(c["f"]))

    def run(q, k, v, out):
        kc, vc = _gpu(c["kc"]), _gpu(c["vc"])
        psispec_qkv_append(q, k, v, kc, vc, _gpu(c["table"]), _gpu(c["lens"]), q_out=out, **kw)
        return out, kc, vc

    qkv = _gpu(c["qkv"])
    want = run(*qkv.split([4, 2, 2], 2), torch.empty((2, 3, 4, 64), dtype=BF, device=DEV))
    raw = torch.zeros((2, 3, 12, 64), dtype=BF, device=DEV)
    raw[:, :, :8] = qkv
    q, k, v, out = raw.split([4, 2, 2, 4], 2)
    for got, x in zip(run(q, k, v, out), want):
        assert torch.equal(got, x)
    raw[:, :, :8] = qkv
    for got, x in zip(run(q, k, v, q), want):  # in place
        assert torch.equal(got, x)
    # k's six rows with gaps, all rows of q_out in the first of them
    raw = torch.zeros((2, 3, 2 + 6 * 4, 64), dtype=BF, device=DEV)
    k = raw[:, :, :2]
    k.copy_(qkv[:, :, 4:6])
    out = raw[0, 0, 2:].view(2, 3, 4, 64)
    for got, x in zip(run(qkv[:, :, :4], k, qkv[:, :, 6:], out), want):
        assert torch.equal(got, x)
    raw = qkv.clone()
    q, k, v = raw.split([4, 2, 2], 2)
    for out in (raw[:, :, 2:6], raw[:, :, 4:8]):
        with pytest.raises(PsispecError, match="invalid argument"):
            run(qkv[:, :, :4].clone(), k, v, out)
    assert torch.equal(raw, qkv)


def test_outputs_in_the_gaps_of_a_cache():
    """Pages with a gap behind each: outputs there are taken, over a page they are refused."""
    c = _append_case([40, 20], 3, 4, 2, 64, 16, BF, BF, seed=4, rot=64)
    tab, ln = _gpu(c["table"]), _gpu(c["lens"])
    q, k, v = _gpu(c["qkv"]).split([4, 2, 2], 2)
    kw = dict(inv_freq=_gpu(c["f"]))
    near = [_gpu(c["kc"]), _gpu(c["vc"])]
    want_q = psispec_qkv_append(q, k, v, *near, tab, ln, **kw)
    want = psispec_paged_attention(want_q, *near, tab, ln)
    pages = near[0].shape[0]
    raw = torch.zeros((2, pages, 46, 2, 64), dtype=BF, device=DEV)  # 16 positions and a gap of 30
    far = [raw[0, :, :16], raw[1, :, :16]]
    for x, y in zip(far, (c["kc"], c["vc"])):
        x.copy_(y)
    gap = raw[0, 1, 16:].flatten()
    q_out, out = (x.view(2, 3, 4, 64) for x in gap[:2 * 1536].chunk(2))
    psispec_qkv_append(q, k, v, *far, tab, ln, q_out=q_out, **kw)
    psispec_paged_attention(q_out, *far, tab, ln, out=out)
    assert torch.equal(q_out, want_q) and torch.equal(out, want)
    assert torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    page = raw[0, 0].numel()
    over = raw.flatten()[page - 8:page + 1536 - 8].view(2, 3, 4, 64)  # from the gap into the next page
    for call in (lambda: psispec_qkv_append(q, k, v, *far, tab, ln, q_out=over, **kw),
                 lambda: psispec_paged_attention(want_q, *far, tab, ln, out=over)):
        with pytest.raises(PsispecError, match="invalid argument"):
            call()


@pytest.mark.parametrize("order", ["rows", "halves", "turns", "heads"])
def test_append_keys_beside_values(order):
    """K and V side by side in each position, in halves of a page, in pages in turn, and in heads in turn; one
    over the other is refused."""
    c = _append_case([40, 20], 3, 4, 2, 64, 16, BF, BF, seed=5, rot=64)
    tab, ln = _gpu(c["table"]), _gpu(c["lens"])
    q, k, v = _gpu(c["qkv"]).split([4, 2, 2], 2)
    near = [_gpu(c["kc"]), _gpu(c["vc"])]
    want = psispec_qkv_append(q, k, v, *near, tab, ln, inv_freq=_gpu(c["f"]))
    n = near[0].shape[0]
    if order == "rows":
        raw = torch.zeros((n, 16, 2, 2, 64), dtype=BF, device=DEV)
        far = [raw[:, :, 0], raw[:, :, 1]]
    elif order == "halves":
        raw = torch.zeros((n, 2, 2, 16, 64), dtype=BF, device=DEV)
        far = [raw[:, 0].transpose(1, 2), raw[:, 1].transpose(1, 2)]
    elif order == "turns":
        raw = torch.zeros((n, 2, 16, 2, 64), dtype=BF, device=DEV)
        far = [raw[:, 0], raw[:, 1]]
    else:
        raw = torch.zeros((n, 16, 2, 2, 64), dtype=BF, device=DEV)
        far = [raw[:, :, :, 0], raw[:, :, :, 1]]
    for x, y in zip(far, (c["kc"], c["vc"])):
        x.copy_(y)
    got = psispec_qkv_append(q, k, v, *far, tab, ln, inv_freq=_gpu(c["f"]))
    assert torch.equal(got, want) and torch.equal(far[0], near[0]) and torch.equal(far[1], near[1])
    with pytest.raises(PsispecError, match="invalid argument"):
        psispec_qkv_append(q, k, v, far[0], far[0], tab, ln, inv_freq=_gpu(c["f"]))


def test_append_rows_in_their_places():
    """Keys and values that a projection left in the cache itself are prepared there."""
    c = _append_case([0], 40, 4, 2, 128, 16, BF, BF, seed=6, rot=64)
    tab = torch.arange(3, dtype=torch.int32, device=DEV)[None]
    ln, f, kw = _gpu(c["lens"]), _gpu(c["f"]), _gpu(c["kw"])
    q, k, v = _gpu(c["qkv"]).split([4, 2, 2], 2)
    want = [torch.zeros((3, 16, 2, 128), dtype=BF, device=DEV) for _ in range(2)]
    want_q = psispec_qkv_append(q, k, v, *want, tab, ln, k_weight=kw, inv_freq=f)
    got = [torch.zeros_like(x) for x in want]
    rows = [x.view(1, 48, 2, 128)[:, :40] for x in got]
    rows[0].copy_(k)
    rows[1].copy_(v)
    got_q = psispec_qkv_append(q, *rows, *got, tab, ln, k_weight=kw, inv_freq=f)
    assert torch.equal(got_q, want_q) and all(torch.equal(x, y) for x, y in zip(got, want))


def test_commit_refuses_lengths_over_its_inputs():
    pool = torch.zeros((1, 8, 4, 4), dtype=torch.int32, device=DEV)
    raw = torch.zeros(24, dtype=torch.int32, device=DEV)
    tab = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    ln, nk, keep = raw[:4], raw[4:8], raw[8:16].view(4, 2)
    for new in (nk, keep[:2].flatten(), raw[5:9], tab[:2].flatten()):
        with pytest.raises(PsispecError, match="invalid argument"):
            psispec_paged_commit(pool, tab, ln, 6, nk, keep=keep, new_length=new)
    st = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    nk.fill_(1)
    psispec_paged_commit(pool, tab, ln, 6, nk, keep=keep, new_length=raw[16:20], status=st)
    assert (st == 0).all() and raw[16:20].tolist() == [1] * 4 and (raw[20:] == 0).all()


# ------------------------------------------------------------------ sizes

def test_attend_large_batch_of_large_blocks():
    """256 lines of 1024 rows and 64 query heads (2^24 rows): rows of a few lines against the reference, and
    against calls of those lines alone."""
    batch, blk, hq, hkv, dim, ps = 256, 1024, 64, 8, 16, 16
    g = torch.Generator(device=DEV).manual_seed(7)
    lens = [0 if r % 7 == 3 else (r * 37) % 150 for r in range(batch)]
    live = [0 if r % 11 == 5 else 5 if r in (0, 128, 255) else blk for r in range(batch)]
    tab, pages = _make_table(lens, blk, ps, _gen(7))
    k, v = (torch.randn((pages, ps, hkv, dim), generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.randn((batch, blk, hq, dim), generator=g, device=DEV, dtype=BF)
    tab, ln, n = tab.to(DEV), *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, live))
    st = torch.full((batch,), -1, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 7.0)
    psispec_paged_attention(q, k, v, tab, ln, n_new=n, out=out, status=st)
    assert (st == 0).all()
    for r in (0, 128, 255, 5):
        assert (out[r, live[r]:] == 7.0).all()
    few = [0, 128, 255]
    want, bound = ref.attention(q[few, :5].cpu(), k.cpu(), v.cpu(), tab[few].cpu(), ln[few].cpu(), [5] * 3, None,
                                dim**-0.5)
    assert ((out[few, :5].cpu().double() - want).abs() <= bound).all()
    for r in (1, 77, 254):
        alone = psispec_paged_attention(q[r:r + 1], k, v, tab[r:r + 1], ln[r:r + 1], n_new=n[r:r + 1])[0].float()
        both = out[r].float()
        # each within half a step of its own rounding, 2^-8, and the arithmetic's 2^-13 of values up to 6
        assert ((both - alone).abs() <= 2.0**-7 * alone.abs() + 2 * 6 * 2.0**-13).all()


# ------------------------------------------------------------------ values that are not finite

def _odd_case(kind, dtype, cache, tree):
    if kind == "cut":          # a workgroup per share, lines cut and joined
        return _case([1500, 0, 733], 9, 8, 4, 128, 16, dtype, cache, seed=50, live=[9, 5, 7], tree=tree)
    if kind == "rows":         # three row tiles, the queries in LDS
        return _case([600, 0, 333], 20, 8, 4, 128, 16, dtype, cache, seed=51, live=[20, 5, 7], tree=tree)
    if kind == "padded":       # heads and pages of no round size
        return _case([75, 0, 33], 9, 6, 3, 80, 24, dtype, cache, seed=52, live=[9, 5, 7], tree=tree)
    if kind == "wide":
        return _case([75, 0, 333], 9, 4, 2, 208, 8, dtype, cache, seed=53, live=[9, 5, 7], tree=tree)
    lens = [75, 0, 33] + torch.randint(0, 40, (260,), generator=_gen(4)).tolist()  # a wave per job
    live = [9, 5, 7] + torch.randint(0, 3, (260,), generator=_gen(5)).tolist()
    return _case(lens, 9, 4, 4, 64, 16, dtype, cache, seed=54, live=live, tree=tree)


@pytest.mark.parametrize("kind", ["cut", "rows", "padded", "wide", "short"])
@pytest.mark.parametrize("dtype,cache,bad", [(d, c, b) for d, c in TYPES for b in ("nan", "inf", "-inf")
                                             if c != F8 or b == "nan"])  # 8 bits have no infinities
@pytest.mark.parametrize("tree", [False, True])
def test_attend_unseen_values_of_every_type(kind, dtype, cache, bad, tree):
    """What a row does not see (free pages, the rest of a line's last page, block rows of other branches) has
    no effect on it, whatever it holds; values that are not finite reach exactly the rows that see them."""
    c = _odd_case(kind, dtype, cache, tree)
    lens, live, ps = c["lens"], c["live"], c["k"].shape[1]
    n0, dim = int(live[0]), c["q"].shape[3]

    def place(r, pos):
        return int(c["table"][r, pos // ps]), pos % ps

    fill = torch.tensor(float(bad)).to(cache)
    used = torch.zeros(c["k"].shape[:2], dtype=torch.bool)
    for r in range(len(lens)):
        t = torch.arange(int(lens[r] + live[r]))
        used[c["table"][r][t // ps].long(), t % ps] = True
    raw = torch.uint8 if cache == F8 else torch.int16
    for x in (c["k"], c["v"]):
        x.view(raw)[~used] = fill.view(raw)
    _check_attend(c)
    want = _attend(c).cpu()
    sees = ref.seen_rows(n0, n0, c["parent"][0] if tree else None)

    def clean_rows_kept(got, rows):
        clean = [i for i in range(n0) if not any(sees[i, j] for j in rows)]
        assert clean
        assert torch.equal(got[0, clean].view(torch.int16), want[0, clean].view(torch.int16))
        for r in range(1, len(lens)):
            assert torch.equal(got[r, :live[r]].view(torch.int16), want[r, :live[r]].view(torch.int16))
        return [i for i in range(n0) if i not in clean]

    # one dimension of two values
    spot = (3, dim - 5)
    old = {}
    for j in spot[:1] + (6,):
        at = place(0, int(lens[0]) + j)
        old[at] = c["v"][at].clone()
        c["v"].view(raw)[at[0], at[1], :, spot[1]] = fill.view(raw)
    got = _attend(c).cpu()
    for i in clean_rows_kept(got, (3, 6)):
        x = got[0, i].float()
        assert (torch.isnan(x[:, spot[1]]) | torch.isinf(x[:, spot[1]])).all()
        others = [d for d in range(dim) if d != spot[1]]
        assert torch.equal(got[0, i][:, others].view(torch.int16), want[0, i][:, others].view(torch.int16))
    # whole keys and values of the same rows
    for at in old:
        c["k"].view(raw)[at] = fill.view(raw)
        c["v"].view(raw)[at] = fill.view(raw)
    got = _attend(c).cpu()
    for i in clean_rows_kept(got, (3, 6)):
        assert not torch.isfinite(got[0, i].float()).any()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("power", [12, 18, 21, 22, 23, 24, 25, 26])
def test_attend_very_large_scores(dtype, cache, power):
    """Scores of about +-2^power, which 32 bits hold in steps of up to 8 and more: one position with all the
    weight, runs of equal scores, and rows that see only the lowest."""
    L = 300
    c = _case([L], 3, 2, 1, 64, 16, dtype, cache, seed=power)
    page, off = (c["table"][0][torch.arange(L + 3) // 16].long(), torch.arange(L + 3) % 16)
    if cache == F8:
        c["ks"], c["vs"] = torch.ones(1), torch.ones(1)
    c["scale"] = 1.0
    k = torch.zeros(L + 3)
    k[10:20], k[130], k[200:232] = -1.0, 0.875, -0.75
    c["k"][page, off, 0] = (k[:, None] * 2.0 ** 7).to(cache).expand(L + 3, 64)
    c["q"].copy_(torch.tensor([1.0, -1.0, 0.8125]).view(3, 1, 1) * 2.0 ** (power - 13))
    got = _attend(c).cpu().double()
    v = c["v"].double()[page, off, 0]
    top = (v[130], v[10:20].mean(0), v[130])
    for i in range(3):
        err = (got[0, i] - top[i]).abs()
        assert (err <= (ref.half_step(dtype) + 2.0**-14) * top[i].abs() + 2.0**-14).all(), (i, err.max())
