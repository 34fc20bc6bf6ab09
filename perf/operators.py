"""The paged-cache operators of the verify step as measured cases: the plain torch form of each
operator and the framework's call for it, on the same inputs.

Operators (key "op" of a case):
  attend  psispec_paged_attention: attention of a block of new tokens (one token in plain decoding,
          the drafted block or tree in a verify forward) over a paged key-value cache
  append  psispec_qkv_append: per-head norms of q and k, the position rotation, K and V into pages
  commit  psispec_paged_commit: the kept rows of a verified block moved down inside a line's pages
  fork    psispec_pages_assign and psispec_pages_reserve: lines forked from others by sharing their
          pages, then given pages of their own for the next block (the shared tail page is copied)
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f8": 1}
DEV = "cuda"


def listed():
    # 32 query heads and 8 key/value heads of 128 (hidden size 4096; cache rows of 8 x 128 in 28
    # layers), blocks of 8 drafts (9 rows with the token before them), trees of 32 nodes
    a = dict(op="attend", hq=32, hkv=8, dim=128, ps=16, type="bf16", cache="bf16", tree=False, pad=0)
    q = dict(op="append", hq=32, hkv=8, dim=128, ps=16, type="bf16", cache="bf16", rot=128,
             inter=False, norm=True, pad=0)
    c = dict(op="commit", planes=56, row=1024, ps=16, depth=8)
    f = dict(op="fork", planes=56, row=1024, ps=16)
    return [
        # one user, one token, a short conversation: latency
        dict(a, name="attend-one", batch=1, blk=1, lo=500, hi=500),
        # plain decoding of a serving batch, lengths uneven
        dict(a, name="attend-decode", batch=64, blk=1, lo=1000, hi=8000),
        # the verify forward of 8 drafts for a serving batch, 3 of the slots idle
        dict(a, name="attend-verify", batch=64, blk=9, lo=300, hi=4200, pad=3),
        # the verify forward of a 32-node tree for a few users
        dict(a, name="attend-tree", batch=8, blk=33, lo=3500, hi=4500, tree=True, type="f16",
             cache="f16"),
        # few users with very long contexts, cache in 8 bits
        dict(a, name="attend-long-f8", batch=4, blk=1, lo=120000, hi=131000, ps=64, cache="f8"),
        # one user's block of 8 drafts: latency
        dict(q, name="append-one", batch=1, blk=9, lo=700, hi=700),
        # a serving batch's blocks, half of each head rotated, neighbouring pairs, cache in 8 bits
        dict(q, name="append-verify-f8", batch=256, blk=9, lo=100, hi=8000, cache="f8", rot=64,
             inter=True, pad=5),
        # chunks of prompts being read in
        dict(q, name="append-prompt", batch=8, blk=1000, lo=0, hi=6000, type="f16", cache="f16"),
        # after the tree verify of a few users / of a large serving batch
        dict(c, name="commit-8", batch=8, blk=32, lo=40, hi=90),
        dict(c, name="commit-256", batch=256, blk=32, lo=40, hi=90),
        # one prompt forked into 4 samples / 16 prompts forked into 8 samples each
        dict(f, name="fork-4", batch=4, width=4, blk=9, lo=500, hi=500),
        dict(f, name="fork-128", batch=128, width=8, blk=9, lo=300, hi=900),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "commit", "fork"])
    ty = rng.choice(["bf16", "bf16", "f16"])
    ca = rng.choice([ty, ty, "f8"])
    hkv = rng.choice([1, 2, 4, 5, 8, 16])
    hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    ps = rng.choice([1, 8, 16, 16, 24, 32, 64, 100, 256])
    if op == "attend":
        blk = rng.choice([1, 1, _span(rng, 2, 64)])
        batch = _span(rng, 1, 128)
        # at most about 2^18 cached positions of 8 x 128 over the batch, and 16 GFLOP
        most = max(16, min(130000, (1 << 28) // (batch * hkv * dim),
                           (1 << 32) // (batch * hq * dim * blk)))
        hi = _span(rng, 1, most)
        return dict(op=op, batch=batch, blk=blk, hq=hq, hkv=hkv, dim=dim, ps=ps, type=ty, cache=ca,
                    lo=rng.randint(0, hi), hi=hi, tree=blk > 1 and rng.random() < 0.4,
                    pad=rng.randint(0, batch // 4))
    if op == "append":
        batch = _span(rng, 1, 256)
        blk = _span(rng, 1, max(1, min(1024, (1 << 25) // ((hq + hkv) * dim) // batch)))
        hi = _span(rng, 1, 100000 // max(1, batch // 16))
        return dict(op=op, batch=batch, blk=blk, hq=hq, hkv=hkv, dim=dim, ps=ps, type=ty, cache=ca,
                    lo=rng.randint(0, hi), hi=hi, rot=rng.choice([dim, dim, 32, 48, 64]),
                    inter=rng.random() < 0.4, norm=rng.random() < 0.7, pad=rng.randint(0, batch // 4))
    planes = rng.choice([2, 16, 56])
    row = rng.choice([64, 128, 256, 512, 1024, 1000])
    if op == "commit":
        hi = _span(rng, 8, 400)
        blk = _span(rng, 4, 64)
        batch = _span(rng, 1, max(1, min(256, 20000 // (hi + blk))))
        return dict(op=op, batch=batch, blk=blk, planes=planes, row=row, ps=ps, lo=rng.randint(0, hi),
                    hi=hi, depth=min(8, blk // 2))
    width = rng.choice([2, 3, 4, 8])
    batch = width * _span(rng, 1, max(1, min(128, (1 << 28) // (ps * planes * row)) // width))
    hi = _span(rng, 1, 900)
    return dict(op=op, batch=batch, width=width, blk=_span(rng, 1, 64), planes=planes, row=row, ps=ps,
                lo=rng.randint(0, hi), hi=hi)


def _lengths(case):
    """The lines' lengths, spread evenly over [lo, hi] in a mixed order (the same for every seed)."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    return [lo + int((hi - lo) * ((r * 0.6180339887498949 + 0.5) % 1.0) + 0.5) for r in range(n)]


def _live(case):
    """New rows of each line: blk, 0 for the padded slots at the end, and with padding shorter
    blocks on every fifth line."""
    n, blk, pad = case["batch"], case["blk"], case["pad"]
    return [0 if r >= n - pad else (blk + 1) // 2 if pad and r % 5 == 2 else blk for r in range(n)]


def _keys(case):
    return [(L + n) if n else 0 for L, n in zip(_lengths(case), _live(case))]


def _kept(case):
    """The kept count of each line: 0 to depth."""
    return [(r * 5 + 3) % (case["depth"] + 1) for r in range(case["batch"])]


def work(case):
    if case["op"] == "attend":
        es, d = BYTES[case["cache"]], case["dim"]
        keys, live = _keys(case), _live(case)
        rows = sum(live) * case["hq"]
        return {"bytes": 2 * sum(keys) * case["hkv"] * d * es + 2 * rows * d * BYTES[case["type"]],
                "flops": 4 * d * case["hq"] * sum(k * n for k, n in zip(keys, live))}
    if case["op"] == "append":
        d, t = case["dim"], sum(_live(case))
        es, ec = BYTES[case["type"]], BYTES[case["cache"]]
        return {"bytes": t * d * ((2 * case["hq"] + 2 * case["hkv"]) * es + 2 * case["hkv"] * ec),
                "flops": 10 * t * d * (case["hq"] + case["hkv"])}
    rb = case["planes"] * case["row"] * 2
    if case["op"] == "commit":
        moved = sum(n - _in_place(n) for n in _kept(case))
        return {"bytes": 2 * moved * rb + 8 * case["batch"] * (case["depth"] + 2), "flops": 0}
    copied = sum(L % case["ps"] for r, L in enumerate(_fork_lengths(case)) if r % case["width"])
    slots = sum(-(-L // case["ps"]) for L in _fork_lengths(case))
    return {"bytes": 2 * copied * rb + 8 * slots, "flops": 0}


def _in_place(n):
    return n // 3  # the leading kept rows that are already in place


def _fork_lengths(case):
    """Every line of a group has its leader's length."""
    lens, w = _lengths(case), case["width"]
    return [lens[r - r % w] for r in range(case["batch"])]


# ------------------------------------------------------------------------------------- inputs

def _table(batch, slots, per_line, pages, g):
    """A page table [batch][slots] whose line r holds per_line[r] pages, from a shuffled pool;
    -1 behind them."""
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(per_line, device=DEV)
    start = torch.cumsum(n, 0) - n
    s = torch.arange(slots, device=DEV)
    idx = (start[:, None] + s[None]).clamp(max=pages - 1)
    return torch.where(s[None] < n[:, None], perm[idx], torch.full_like(perm[idx], -1))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn(shape, g, dtype, scale=1.0):
    """Normal values of any type, made in slices of the first dimension."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        out[i:i + n] = (torch.randn((n, *shape[1:]), generator=g, device=DEV) * scale).to(dtype)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case, "op": case["op"]}
    return {"attend": _prep_attend, "append": _prep_append, "commit": _prep_commit,
            "fork": _prep_fork}[case["op"]](case, st, g)


def _prep_attend(case, st, g):
    b, blk, ps, d = case["batch"], case["blk"], case["ps"], case["dim"]
    lens, live = _lengths(case), _live(case)
    order = torch.randperm(b, generator=g, device=DEV).tolist()
    lens, live = [lens[r] for r in order], [live[r] for r in order]
    per = [-(-(L + blk) // ps) for L in lens]
    pages = sum(per)
    st["table"] = _table(b, max(per), per, pages, g)
    st["len"], st["n_new"] = _ints(lens), _ints(live) if case["pad"] else None
    ct = DTYPES[case["cache"]]
    st["k"] = _randn((pages, ps, case["hkv"], d), g, ct)
    st["v"] = _randn((pages, ps, case["hkv"], d), g, ct)
    st["k_scale"] = st["v_scale"] = None
    if case["cache"] == "f8":
        st["k_scale"] = 0.5 + torch.rand(case["hkv"], generator=g, device=DEV)
        st["v_scale"] = 0.5 + torch.rand(case["hkv"], generator=g, device=DEV)
    st["q"] = _randn((b, blk, case["hq"], d), g, DTYPES[case["type"]], 2.0)
    st["parent"] = None
    if case["tree"]:  # row 0 is the token before the tree; each node under one of the rows before it
        j = torch.arange(1, blk, device=DEV)
        u = torch.rand((b, blk - 1), generator=g, device=DEV)
        par = torch.minimum(((j - 1) // 4 + (u * (j - (j - 1) // 4)).long()), j - 1)
        st["parent"] = torch.cat([torch.full((b, 1), -1, device=DEV), par], 1).to(torch.int32)
    st["scale"] = d ** -0.5
    st["out"] = torch.zeros_like(st["q"])
    if own:
        import lossless_draft_verification_spec_amd as pkg
        st["ws"] = torch.empty(pkg.paged_attention_workspace_bytes(b, blk, case["hq"], case["hkv"], d),
                               dtype=torch.uint8, device=DEV)
    return st


def _prep_append(case, st, g):
    b, blk, ps, d, hq, hkv = (case[k] for k in ("batch", "blk", "ps", "dim", "hq", "hkv"))
    lens, live = _lengths(case), _live(case)
    order = torch.randperm(b, generator=g, device=DEV).tolist()
    lens, live = [lens[r] for r in order], [live[r] for r in order]
    # the pages of the new rows are the line's own; those before them are a prefix page that all
    # lines share (the operator does not touch them)
    slots = max(-(-(L + blk) // ps) for L in lens)
    first, last = [L // ps for L in lens], [(L + blk - 1) // ps for L in lens]
    per = [z - a + 1 for a, z in zip(first, last)]
    pages = sum(per) + 1
    perm = (torch.randperm(pages - 1, generator=g, device=DEV) + 1).to(torch.int32)
    s = torch.arange(slots, device=DEV)[None]
    f, n = torch.tensor(first, device=DEV)[:, None], torch.tensor(per, device=DEV)
    start = (torch.cumsum(n, 0) - n)[:, None]
    idx = (start + s - f).clamp(0, pages - 2)
    tab = torch.where((s >= f) & (s < f + n[:, None]), perm[idx], torch.full_like(perm[idx], -1))
    st["table"] = torch.where(s < f, torch.zeros_like(tab), tab)
    st["len"], st["n_new"] = _ints(lens), _ints(live) if case["pad"] else None
    dt, ct = DTYPES[case["type"]], DTYPES[case["cache"]]
    st["kc"] = _randn((pages, ps, hkv, d), g, ct)
    st["vc"] = _randn((pages, ps, hkv, d), g, ct)
    st["k_scale"] = st["v_scale"] = None
    if case["cache"] == "f8":
        st["k_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device=DEV)
        st["v_scale"] = 0.01 + 0.02 * torch.rand(hkv, generator=g, device=DEV)
    # the qkv projection's output: one row per token, [hq + 2 hkv][dim]
    st["qkv"] = _randn((b, blk, hq + 2 * hkv, d), g, dt)
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["kw"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(dt)
    j = torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64)
    st["inv_freq"] = 500000.0 ** (-2.0 * j / case["rot"])
    st["q_out"] = torch.zeros((b, blk, hq, d), dtype=dt, device=DEV)
    return st


def _prep_commit(case, st, g):
    b, blk, ps = case["batch"], case["blk"], case["ps"]
    lens, kept = _lengths(case), _kept(case)
    order = torch.randperm(b, generator=g, device=DEV).tolist()
    lens, kept = [lens[r] for r in order], [kept[r] for r in order]
    per = [-(-(L + blk) // ps) for L in lens]
    pages = sum(per)
    st["table"] = _table(b, max(per), per, pages, g)
    st["len"], st["n_keep"] = _ints(lens), _ints(kept)
    # a kept path: the first third of its rows already in place, the others from behind the kept
    # rows, in increasing order (so that the commit gives the same when it is repeated)
    D = case["depth"]
    u = torch.rand((b, blk), generator=g, device=DEV)
    n = st["n_keep"][:, None].long()
    j = torch.arange(blk, device=DEV)[None]
    pick = torch.where(j < n // 3, 0.0, torch.where(j < n, 3.0, 1.0 + u))
    chosen = torch.argsort(pick, dim=1, stable=True)[:, :D]
    i = torch.arange(D, device=DEV)[None]
    chosen = torch.sort(torch.where(i < n, chosen, blk), dim=1).values
    st["keep"] = torch.where(i < n, chosen, -1).to(torch.int32)
    st["pool"] = torch.randint(-32768, 32767, (case["planes"], pages, ps, case["row"]), generator=g,
                               device=DEV, dtype=torch.int16)
    st["new_len"] = torch.zeros_like(st["len"])
    return st


def _prep_fork(case, st, g):
    b, w, blk, ps = case["batch"], case["width"], case["blk"], case["ps"]
    lens = _fork_lengths(case)
    lead = [r - r % w for r in range(b)]
    per = [-(-L // ps) if r % w == 0 else 0 for r, L in enumerate(lens)]
    most = blk // ps + 2  # pages that one line's reservation can take
    pages = sum(per) + b * most
    slots = -(-(max(lens) + blk) // ps)
    st["table"] = _table(b, slots, per, pages, g)
    st["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    st["refs"][st["table"][st["table"] >= 0].long()] = 1
    st["len"] = _ints([L if r % w == 0 else 0 for r, L in enumerate(lens)])
    st["src"] = _ints(lead)
    st["want"] = _ints(lens)
    st["n_new"] = _ints([0 if r % w == 0 else blk for r in range(b)])
    st["pool"] = torch.randint(-32768, 32767, (case["planes"], pages, ps, case["row"]), generator=g,
                               device=DEV, dtype=torch.int16)
    st["status"] = torch.zeros(b, dtype=torch.int32, device=DEV)
    if own:
        import lossless_draft_verification_spec_amd as pkg
        st["ws"] = torch.empty(pkg.pages_workspace_bytes(b, slots, pages, blk, ps), dtype=torch.uint8,
                               device=DEV)
    return st


# ------------------------------------------------------------------------------------- one pass

def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


def _own_attend(st):
    import lossless_draft_verification_spec_amd as pkg
    return pkg.psispec_paged_attention(st["q"], st["k"], st["v"], st["table"], st["len"],
                                       n_new=st["n_new"], parent=st["parent"], scale=st["scale"],
                                       k_scale=st["k_scale"], v_scale=st["v_scale"], out=st["out"],
                                       workspace=st["ws"])


def _own_append(st):
    import lossless_draft_verification_spec_amd as pkg
    c = st["case"]
    q, k, v = st["qkv"].split([c["hq"], c["hkv"], c["hkv"]], dim=2)
    pkg.psispec_qkv_append(q, k, v, st["kc"], st["vc"], st["table"], st["len"], n_new=st["n_new"],
                           q_weight=st["qw"], k_weight=st["kw"], eps=1e-6, inv_freq=st["inv_freq"],
                           interleaved=c["inter"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                           q_out=st["q_out"])
    return st["q_out"], st["kc"], st["vc"]


def _own_commit(st):
    import lossless_draft_verification_spec_amd as pkg
    pkg.psispec_paged_commit(st["pool"], st["table"], st["len"], st["case"]["blk"], st["n_keep"],
                             keep=st["keep"], new_length=st["new_len"])
    return st["pool"], st["new_len"]


def _own_fork(st):
    import lossless_draft_verification_spec_amd as pkg
    pkg.psispec_pages_assign(st["table"], st["refs"], st["len"], st["src"], st["want"],
                             page_size=st["case"]["ps"], workspace=st["ws"])
    pkg.psispec_pages_reserve(st["pool"], st["table"], st["refs"], st["len"], st["case"]["blk"],
                              n_new=st["n_new"], status=st["status"], workspace=st["ws"])
    return st["pool"], st["table"], st["refs"], st["len"], st["status"]


def _plain_attend(st):
    c, q = st["case"], st["q"]
    b, blk, hkv, d, ps = c["batch"], c["blk"], c["hkv"], c["dim"], c["ps"]
    G = c["hq"] // hkv
    n = st["n_new"].long() if st["n_new"] is not None else torch.full((b,), blk, device=DEV)
    ln = st["len"].long()
    L = st["table"].shape[1] * ps
    page = st["table"].long().clamp(min=0)
    k = st["k"][page].reshape(b, L, hkv, d).transpose(1, 2).float()
    v = st["v"][page].reshape(b, L, hkv, d).transpose(1, 2).float()
    qs = q.float().reshape(b, blk, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, blk * G, d)
    s = torch.matmul(qs, k.transpose(2, 3).contiguous()) * st["scale"]
    if st["k_scale"] is not None:
        s = s * st["k_scale"][None, :, None, None]
    pos = torch.arange(L, device=DEV)
    j = pos[None] - ln[:, None]                              # block row of a cached position
    if st["parent"] is None:
        sees = torch.ones((blk, blk), device=DEV).tril()[None].expand(b, blk, blk) > 0
    else:  # row i sees row j where (I + A)^blk has a path, A[i][parent[i]] = 1
        par = st["parent"].long()
        A = (par[:, :, None] == torch.arange(blk, device=DEV)).float()
        sees = torch.matrix_power(torch.eye(blk, device=DEV) + A, blk) > 0
    inblk = (j >= 0) & (j < n[:, None])
    seen = torch.gather(sees, 2, j.clamp(0, blk - 1)[:, None].expand(b, blk, L)) & inblk[:, None]
    seen = (seen | (j < 0)[:, None]).repeat_interleave(G, dim=1)[:, None]
    s = s.masked_fill(~seen, float("-inf"))
    s = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(s, v.masked_fill(~(inblk | (j < 0))[:, None, :, None], 0.0))
    o = o / s.sum(-1, keepdim=True)
    if st["v_scale"] is not None:
        o = o * st["v_scale"][None, :, None, None]
    o = o.reshape(b, hkv, blk, G, d).permute(0, 2, 1, 3, 4).reshape(b, blk, c["hq"], d).to(q.dtype)
    live = torch.arange(blk, device=DEV)[None] < n[:, None]
    return torch.where(live[:, :, None, None], o, st["out"])


def _rotate(x, cos, sin, inter):
    if inter:
        a, z = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - z * sin, z * cos + a * sin], -1).flatten(-2)
    a, z = x.chunk(2, -1)
    return torch.cat([a * cos - z * sin, z * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    b, blk, ps, rot = c["batch"], c["blk"], c["ps"], c["rot"]
    i = torch.arange(blk, device=DEV)
    pos = st["len"].long()[:, None] + i[None]                # [b][blk]
    ang = pos.double()[..., None] * st["inv_freq"]
    cos, sin = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    q, k, v = st["qkv"].float().split([c["hq"], c["hkv"], c["hkv"]], dim=2)
    if st["qw"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * st["qw"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * st["kw"].float()
    q = torch.cat([_rotate(q[..., :rot], cos, sin, c["inter"]), q[..., rot:]], -1)
    k = torch.cat([_rotate(k[..., :rot], cos, sin, c["inter"]), k[..., rot:]], -1)
    live = i[None] < (st["n_new"].long()[:, None] if st["n_new"] is not None else blk)
    live = live.expand(b, blk)
    at = torch.gather(st["table"].long(), 1, pos // ps) * ps + pos % ps
    st["q_out"].copy_(torch.where(live[:, :, None, None], q.to(st["q_out"].dtype), st["q_out"]))
    for cache, x, scale in ((st["kc"], k, st["k_scale"]), (st["vc"], v, st["v_scale"])):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        raw = cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16).flatten(0, 1)
        x = x.to(cache.dtype).view(raw.dtype)
        raw[at] = torch.where(live[:, :, None, None], x, raw[at])
    return st["q_out"], st["kc"], st["vc"]


def _plain_commit(st):
    c = st["case"]
    ps, D = c["ps"], c["depth"]
    i = torch.arange(D, device=DEV)[None]
    kept = i < st["n_keep"].long()[:, None]
    ln = st["len"].long()[:, None]
    src, dst = ln + torch.where(kept, st["keep"].long(), i), ln + i
    tab = st["table"].long()
    src = torch.gather(tab, 1, src // ps) * ps + src % ps
    dst = torch.gather(tab, 1, dst // ps) * ps + dst % ps
    rows = st["pool"].flatten(1, 2)
    rows[:, dst] = rows[:, src]
    torch.add(st["len"], st["n_keep"], out=st["new_len"])
    return st["pool"], st["new_len"]


def _plain_fork(st):
    c, tab, refs = st["case"], st["table"], st["refs"]
    b, slots = tab.shape
    ps, blk = c["ps"], c["blk"]
    s = torch.arange(slots, device=DEV)[None]
    # every line becomes the first `want` positions of the line it is forked from
    new = torch.where(s < ((st["want"].long() + ps - 1) // ps)[:, None], tab[st["src"].long()], -1)
    pad = torch.zeros(1, dtype=torch.int32, device=DEV)
    cnt = torch.cat([refs, pad])                              # entry behind the last: no page
    one = torch.ones_like(new).flatten()
    none = refs.numel()
    cnt.index_add_(0, torch.where(tab >= 0, tab.long(), none).flatten(), -one)
    cnt.index_add_(0, torch.where(new >= 0, new.long(), none).flatten(), one)
    # then pages of its own for the next block
    n, ln = st["n_new"].long(), st["want"].long()
    first, last = ln // ps, (ln + n - 1) // ps
    j = torch.arange(blk // ps + 2, device=DEV)[None]
    at = first[:, None] + j
    act = (n > 0)[:, None] & (at <= last[:, None])
    at = at.clamp(max=slots - 1)
    old = torch.gather(new, 1, at).long()
    need = act & ((old < 0) | (cnt[old.clamp(min=0)] > 1))
    rank = torch.cumsum(need.flatten().long(), 0).reshape(need.shape)
    ids = torch.arange(none, device=DEV)
    free = torch.where(cnt[:none] == 0, ids, none)
    held = torch.argmax((cnt[:none] > 0).int())              # a page that nothing is written to
    served = rank[:, -1:] <= (free < none).sum()
    free = torch.sort(free).values
    take = need & served
    got = free[(rank - 1).clamp(0, none - 1)]
    cnt.index_add_(0, torch.where(take, got, none).flatten(), torch.ones_like(got, dtype=torch.int32).flatten())
    lost = take & (old >= 0)
    cnt.index_add_(0, torch.where(lost, old, none).flatten(), -torch.ones_like(old, dtype=torch.int32).flatten())
    wide = torch.cat([new, new[:, :1]], 1)
    wide.scatter_(1, torch.where(take, at, slots), got.to(torch.int32))
    # the rows of a tail page that was shared
    o = torch.arange(ps, device=DEV)[None]
    cow = (lost[:, :1] & (o < (ln % ps)[:, None]))
    src = torch.where(cow, old[:, :1], held) * ps + o
    dst = torch.where(cow, got[:, :1] * ps + o, src)
    rows = st["pool"].flatten(1, 2)
    rows[:, dst] = rows[:, src]
    tab.copy_(wide[:, :slots])
    refs.copy_(cnt[:none])
    st["len"].copy_(st["want"])
    st["status"].copy_(torch.where(served[:, 0], 0, 128))
    return st["pool"], tab, refs, st["len"], st["status"]


_OWN = {"attend": _own_attend, "append": _own_append, "commit": _own_commit, "fork": _own_fork}
_PLAIN = {"attend": _plain_attend, "append": _plain_append, "commit": _plain_commit,
          "fork": _plain_fork}


# ------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "attend":
        return _exact_attend(prepare(case, seed))
    if case["op"] == "append":
        return _exact_append(prepare(case, seed))
    return None  # rows and tables are moved, not computed


def _exact_attend(st):
    """Line by line and key/value head by head, from the definition."""
    c = st["case"]
    G, blk = c["hq"] // c["hkv"], c["blk"]
    out = st["out"].double()
    lens = st["len"].tolist()
    live = st["n_new"].tolist() if st["n_new"] is not None else [blk] * c["batch"]
    par = st["parent"].tolist() if st["parent"] is not None else None
    for r, (L, n) in enumerate(zip(lens, live)):
        if n == 0:
            continue
        t = torch.arange(L + n, device=DEV)
        page, off = st["table"][r][t // c["ps"]].long(), t % c["ps"]
        hidden = torch.zeros((n, L + n), dtype=torch.bool)
        for i in range(n):
            seen, a = set(range(i + 1)), i
            if par is not None:
                seen = set()
                while a >= 0:
                    seen.add(a)
                    a = par[r][a]
            for a in set(range(n)) - seen:
                hidden[i, L + a] = True
        hidden = hidden.to(DEV)
        for h in range(c["hkv"]):
            k, v = st["k"][page, off, h].double(), st["v"][page, off, h].double()
            if st["k_scale"] is not None:
                k, v = k * st["k_scale"][h].double(), v * st["v_scale"][h].double()
            q = st["q"][r, :n, h * G:(h + 1) * G].double()
            w = torch.softmax((torch.tensordot(q, k, ([2], [1])) * st["scale"]).masked_fill(
                hidden[:, None], -math.inf), -1)
            out[r, :n, h * G:(h + 1) * G] = torch.tensordot(w, v, ([2], [0]))
    return out


def _exact_append(st):
    c = st["case"]
    rot, half = c["rot"], c["rot"] // 2
    live = st["n_new"].tolist() if st["n_new"] is not None else [c["blk"]] * c["batch"]
    res = [st["q_out"].double(), st["kc"].double(), st["vc"].double()]
    d = torch.arange(half, device=DEV)
    lo, hi = (2 * d, 2 * d + 1) if c["inter"] else (d, d + half)
    for r, (L, n) in enumerate(zip(st["len"].tolist(), live)):
        if n == 0:
            continue
        t = torch.arange(L, L + n, device=DEV)
        turn = torch.exp(1j * (t.double()[:, None, None] * st["inv_freq"]))
        x = st["qkv"][r, :n].double()
        y = x.clone()
        for a, z, wt in ((0, c["hq"], st["qw"]), (c["hq"], c["hq"] + c["hkv"], st["kw"])):
            p = x[:, a:z]
            if wt is not None:
                p = p / torch.sqrt((p * p).mean(-1, keepdim=True) + 1e-6) * wt.double()
            cx = torch.complex(p[..., lo], p[..., hi]) * turn
            p = p.clone()
            p[..., lo], p[..., hi] = cx.real, cx.imag
            y[:, a:z] = p
        res[0][r, :n] = y[:, :c["hq"]]
        page, off = st["table"][r][t // c["ps"]].long(), t % c["ps"]
        k, v = y[:, c["hq"]:c["hq"] + c["hkv"]], y[:, c["hq"] + c["hkv"]:]
        if st["k_scale"] is not None:
            k = (k / st["k_scale"].double()[:, None]).clamp(-448.0, 448.0)
            v = (v / st["v_scale"].double()[:, None]).clamp(-448.0, 448.0)
        res[1][page, off], res[2][page, off] = k, v
    return tuple(res)
