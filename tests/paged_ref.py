"""Plain 64-bit references of the paged-cache operators, line by line from their definitions, and the
error bounds that the GPU tests allow against them."""
import numpy as np
import torch

BAD_PARENT, BAD_KEEP, BAD_PAGE, NO_PAGE = 16, 32, 64, 128


def half_step(dtype):
    """Largest relative rounding error of a type."""
    return torch.finfo(dtype).eps / 2


def gather_line(cache, table_row, page_size, n):
    """Positions 0..n-1 of a line: [n][heads][dim] in float64 (CPU tensors)."""
    t = torch.arange(n)
    return cache.double()[table_row[t // page_size].long(), t % page_size]


def seen_rows(blk, n, parent=None):
    """bool [n][n]: block row i sees block row j."""
    m = np.zeros((n, n), bool)
    for i in range(n):
        if parent is None:
            m[i, :i + 1] = True
        else:
            j = i
            while j >= 0:
                m[i, j] = True
                j = int(parent[j])
    return m


def attention(q, k_cache, v_cache, table, length, n_new, parent, scale, k_scale=None, v_scale=None):
    """(out, bound) for CPU tensors: out [batch][blk][hq][dim] float64 (NaN in rows that are not
    computed) and bound, what each element of the 16-bit result may be off by.

    The bound, per output element: half a step of the output type, and delta * sum w|v| / sum w for
    the arithmetic in 32 bits, where delta adds up
      2 ds   a weight's relative error from its score's error, in numerator and denominator;
             ds = (dim + 8) 2^-24 scale sum_d |q_d k_d| (dim fp32 additions, 8 more roundings)
      2^-15  the weight as a pair of 16-bit numbers (2^-16) and the hardware's exp2 (2^-22), twice
      (L / 16 + 256) 2^-24   sums over the positions: at least 16 are summed apart, joined later."""
    b, blk, hq, dim = q.shape
    ps, hkv = k_cache.shape[1], k_cache.shape[2]
    G = hq // hkv
    out = torch.full((b, blk, hq, dim), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for r in range(b):
        L, n = int(length[r]), int(n_new[r])
        if n == 0:
            continue
        k = gather_line(k_cache, table[r], ps, L + n)
        v = gather_line(v_cache, table[r], ps, L + n)
        if k_scale is not None:
            k = k * k_scale.double()[:, None]
        if v_scale is not None:
            v = v * v_scale.double()[:, None]
        block = torch.from_numpy(seen_rows(blk, n, None if parent is None else parent[r]))
        seen = torch.cat([torch.ones(n, L, dtype=torch.bool), block], 1)
        for i in range(n):
            at = seen[i].nonzero()[:, 0]
            for h in range(hkv):
                qq = q[r, i, h * G:(h + 1) * G].double()
                kk, vv = k[at, h], v[at, h]
                s = qq @ kk.T * scale
                w = torch.softmax(s, -1)
                o = w @ vv
                ds = (dim + 8) * 2.0**-24 * abs(scale) * (qq.abs() @ kk.abs().T).amax(-1)
                delta = 2 * ds + 2.0**-15 + (len(at) / 16 + 256) * 2.0**-24
                out[r, i, h * G:(h + 1) * G] = o
                # an infinite value makes the result infinite or NaN and has no bound
                bound[r, i, h * G:(h + 1) * G] = torch.nan_to_num(
                    half_step(q.dtype) * o.abs() + delta[:, None] * (w @ vv.abs())
                    + torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps)
    return out, bound


def prepared(x, weight, eps, pos, inv_freq, interleaved, rope_scale):
    """(y, bound) of heads x [n][heads][dim] at positions pos: norm, then rotation, in float64.  The
    bound is that of the 32-bit arithmetic alone: 2^-20 of the pair's magnitude (about 12 roundings of
    2^-24 in the norm, the sine's and cosine's absolute error of 2^-22 each)."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, mag = x.clone(), x.abs()
    if inv_freq is not None and inv_freq.numel():
        half = inv_freq.numel()
        j = torch.arange(half)
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        t = pos.double()[:, None] * inv_freq.double()
        cs, sn = torch.cos(t)[:, None], torch.sin(t)[:, None]
        a, z = x[..., lo], x[..., hi]
        y[..., lo] = rope_scale * (a * cs - z * sn)
        y[..., hi] = rope_scale * (z * cs + a * sn)
        m = abs(rope_scale) * (a.abs() + z.abs())
        mag = mag.clone()
        mag[..., lo] = m
        mag[..., hi] = m
    return y, 2.0**-20 * mag


def stored_bound(y, err, dtype):
    """What the stored number may be off by: the arithmetic's bound, half a step of the type, and half
    its smallest number."""
    fi = torch.finfo(dtype)
    return err * (1 + fi.eps) + half_step(dtype) * y.abs() + fi.smallest_normal * fi.eps / 2


def commit(pool, table, length, blk, n_keep, keep, page_size):
    """In place on numpy pool [planes][pages][page_size][row]; returns (new_len, status)."""
    b, slots = table.shape
    new, st = length.copy(), np.zeros(b, np.int32)
    for r in range(b):
        L, n = int(length[r]), int(n_keep[r])
        kp = [] if keep is None else [int(x) for x in keep[r]]
        if n < 0 or n > blk or L < 0 or L + blk > slots * page_size or (
                keep is not None and n > len(kp)):
            st[r] = BAD_KEEP
            continue
        rows = list(range(n)) if keep is None else kp[:n]
        if any(x < 0 or x >= blk for x in rows) or any(y <= x for x, y in zip(rows, rows[1:])):
            st[r] = BAD_KEEP
            continue
        moves = [(L + k, L + i) for i, k in enumerate(rows) if i != k]
        pages = [int(table[r, p // page_size]) for m in moves for p in m]
        if any(p < 0 or p >= pool.shape[1] for p in pages):
            st[r] = BAD_PAGE
            continue
        for s, d in moves:
            pool[:, table[r, d // page_size], d % page_size] = \
                pool[:, table[r, s // page_size], s % page_size]
        new[r] = L + n
    return new, st


def assign(table, refs, length, src, new_length, page_size):
    """In place on numpy arrays; returns status."""
    b, slots = table.shape
    old, oldlen = table.copy(), length.copy()
    st = np.zeros(b, np.int32)
    for r in range(b):
        s, n = int(src[r]), int(new_length[r])
        if s == -1:
            s, n = r, 0
        elif s < -1 or s >= b or n < 0 or n > oldlen[s] or n > slots * page_size:
            st[r] = BAD_PAGE
            continue
        cut = -(-n // page_size)
        if any(p < 0 or p >= len(refs) for p in old[s, :cut]):
            st[r] = BAD_PAGE
            continue
        new = np.full(slots, -1, np.int32)
        new[:cut] = old[s, :cut]
        for p in old[r]:
            if 0 <= p < len(refs):
                refs[p] -= 1
        for p in new[:cut]:
            refs[p] += 1
        table[r], length[r] = new, n
    return st


def reserve(pool, table, refs, length, blk, n_new, page_size):
    """In place on numpy arrays; returns status."""
    b, slots = table.shape
    free = [p for p in range(len(refs)) if refs[p] == 0]
    before = refs.copy()
    st, out = np.zeros(b, np.int32), False
    plan = []
    for r in range(b):
        L, n = int(length[r]), int(n_new[r])
        if L < 0 or n < 0 or n > blk or L + n > slots * page_size:
            st[r] = BAD_PAGE
            continue
        need, bad = [], False
        for s in range(L // page_size, (L + n - 1) // page_size + 1 if n else 0):
            p = int(table[r, s])
            bad |= p >= len(refs) or (p < 0 and s * page_size < L)
            if p < 0 or (p < len(refs) and before[p] > 1):
                need.append((s, p))
        if bad:
            st[r] = BAD_PAGE
            continue
        if not need:
            continue
        if out or len(need) > len(free):
            out = True
            st[r] = NO_PAGE
            continue
        for s, p in need:
            plan.append((r, s, p, free.pop(0)))
    for r, s, p, q in plan:
        table[r, s] = q
        refs[q] += 1
        if p >= 0:
            refs[p] -= 1
            k = int(length[r]) - s * page_size
            if k > 0:
                pool[:, q, :k] = pool[:, p, :k]
    return st
