"""The layers around the paged attention (through the binding) against 64-bit references: the norm with the
residual's addition, linear layers with weights of 4 bits, the gated projections, and a run of them together
with the cache."""
import math

import pytest
import torch

import layers_ref as ref
from layers_ref import BF, E8, F8, FH
from lossless_draft_verification_spec_amd import (
    PsispecError, W4Weight, psispec_add_rmsnorm, psispec_paged_attention, psispec_qkv_append, psispec_w4_gated,
    psispec_w4_linear, psispec_w4_pack, rope_frequencies, w4_workspace_bytes)

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32 = torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _gpu(t):
    return None if t is None else t.to(DEV)


def _inside(t, pad, fill=7.0):
    """t on the GPU as columns of wider rows whose other columns hold `fill` (7 in 8 bits too)."""
    raw = torch.full((t.shape[0], t.shape[1] + 2 * pad), fill, device=DEV).to(t.dtype)
    v = raw[:, pad:pad + t.shape[1]]
    v.copy_(t)
    return raw, v


def _untouched(raw, pad, width):
    side = torch.cat([raw[:, :pad], raw[:, pad + width:]], 1).float()
    assert (side == 7.0).all(), "columns beside the rows were written"


def _within(got, want, bound, what=""):
    err = (got.cpu().double() - want).abs()
    assert torch.isfinite(got.cpu().double()).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))


# ------------------------------------------------------------------------------------- norm

def _norm_case(rows, dim, dtype, residual, quant, pad, seed, weighted=True, eps=1e-6):
    g = _gen(seed)
    x = torch.randn((rows, dim), generator=g).to(dtype)
    w = (1 + 0.3 * torch.randn(dim, generator=g)).to(dtype) if weighted else None
    r = None if residual is None else (3 * torch.randn((rows, dim), generator=g)).to(residual)
    y, h = ref.norm(x, w, r, eps)
    _, xg = _inside(x, pad)
    rg = None if r is None else _inside(r, pad)[1]
    ro_raw, ro = (None, None) if r is None else _inside(torch.zeros_like(r), pad)
    ot = dtype if quant is None else F8
    o_raw, o = _inside(torch.zeros((rows, dim)).to(ot), pad)
    sc = None
    if quant == "row":
        sc = torch.full((rows,), -1.0, device=DEV)
    elif quant == "mx":
        sc = torch.zeros((rows, dim // 32 + pad), dtype=torch.uint8, device=DEV).view(E8)[:, :dim // 32]
    got, gro, gsc = psispec_add_rmsnorm(xg, _gpu(w), residual=rg, residual_out=ro, eps=eps, quant=quant,
                                        out=o, scale=sc)
    assert got is o and gro is ro and gsc is sc
    _untouched(o_raw, pad, dim)
    if r is not None:
        _untouched(ro_raw, pad, dim)
        # both terms are exact in 32 bits, their sum is rounded there and once more in residual's type
        _within(ro, h, ref.half_step(h, residual) + 2.0 ** -24 * h.abs(), "residual")
    rel = ref.NORM_REL * y.abs()
    if quant is None:
        _within(o, y, (rel + ref.half_step(y, dtype)) * (1 + 2.0 ** -8))
        return
    top = y.abs()
    if quant == "row":
        s = sc.cpu().double()[:, None]
        want = top.amax(1, keepdim=True) / 448
        assert ((s - want).abs() <= 2.0 ** -17 * want).all()
    else:
        s = ref.powers(sc.cpu())
        m = top.unflatten(1, (-1, 32)).amax(-1)
        # the smallest power of two that keeps the block within 448, but for what 32 bits may move it
        assert (m * (1 - 2.0 ** -17) <= 448 * s).all()
        assert ((m * (1 + 2.0 ** -17) > 224 * s) | (s == 2.0 ** -127)).all()
        s = s.repeat_interleave(32, 1)
    _within(o.float() * s.to(DEV, F32), y, (rel * 2 + s * ref.half_step(y / s.clamp(min=1e-300), F8)) * (1 + 2.0 ** -8))


@pytest.mark.parametrize("dim", [1, 7, 8, 31, 32, 64, 100, 500, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096,
                                 4104, 5120, 8192, 8200, 16384, 16392, 32768])
@pytest.mark.parametrize("quant", [None, "row", "mx"])
def test_norm_dims(dim, quant):
    if quant == "mx":
        dim = -(-dim // 32) * 32
    _norm_case(5, dim, BF, BF, quant, 0, seed=dim)


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("residual", ["none", "same", "f32"])
@pytest.mark.parametrize("quant", [None, "row", "mx"])
@pytest.mark.parametrize("pad", [0, 1, 16])
def test_norm_types_and_strides(dtype, residual, quant, pad):
    r = {"none": None, "same": dtype, "f32": F32}[residual]
    _norm_case(37, 288, dtype, r, quant, pad, seed=pad + 1)
    _norm_case(1, 1056, dtype, r, quant, pad, seed=pad + 2, weighted=False, eps=0.0)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 257, 1000])
def test_norm_rows(rows):
    _norm_case(rows, 96, FH, FH, "mx", 0, seed=rows)
    _norm_case(rows, 640, BF, F32, "row", 0, seed=rows)


def test_norm_in_place_and_defaults():
    g = _gen(5)
    x, r = torch.randn((9, 200), generator=g).to(BF), torch.randn((9, 200), generator=g).to(BF)
    w = torch.randn(200, generator=g).to(BF)
    a = psispec_add_rmsnorm(_gpu(x), _gpu(w), residual=_gpu(r))
    xi, ri = _gpu(x), _gpu(r)
    out, ro, sc = psispec_add_rmsnorm(xi, _gpu(w), residual=ri, out=xi)  # residual_out: residual itself
    assert out is xi and ro is ri and sc is None
    assert torch.equal(out, a[0]) and torch.equal(ro, a[1])
    # outputs swapped: out over the residual's rows, the new residual over x's
    xi, ri = _gpu(x), _gpu(r)
    out, ro, _ = psispec_add_rmsnorm(xi, _gpu(w), residual=ri, residual_out=xi, out=ri)
    assert torch.equal(out, a[0]) and torch.equal(ro, a[1])
    # three-dimensional rows; no residual, but the sum wanted in 32 bits
    x3 = _gpu(x).view(3, 3, 200)
    h = torch.zeros((3, 3, 200), device=DEV)
    out, ro, _ = psispec_add_rmsnorm(x3, residual_out=h)
    assert out.shape == x3.shape and torch.equal(ro, x3.float())
    q, _, s = psispec_add_rmsnorm(x3[..., :192], quant="mx")
    assert q.shape == (3, 3, 192) and s.shape == (3, 3, 6) and s.dtype == E8


def test_norm_of_a_single_row():
    x = torch.randn(96, generator=_gen(5)).to(BF).to(DEV)
    y, _, s = psispec_add_rmsnorm(x, quant="row")
    y2, _, s2 = psispec_add_rmsnorm(x[None], quant="row")
    assert s.shape == () and s == s2[0] and torch.equal(y.view(torch.uint8), y2[0].view(torch.uint8))
    assert psispec_add_rmsnorm(x, quant="mx")[2].shape == (3,)
    for bad in (torch.zeros(()), torch.zeros(2, device=DEV), torch.zeros(0, device=DEV)):
        with pytest.raises(PsispecError):
            psispec_add_rmsnorm(x, quant="row", scale=bad)


def test_norm_zeros_and_extremes():
    x = torch.zeros((4, 128), dtype=BF)
    x[1, 3] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1.0
    x[3, 64:] = 0.0
    for quant in ("row", "mx"):
        q, _, s = psispec_add_rmsnorm(_gpu(x), quant=quant)
        q, s = q.cpu().float(), s.cpu().float() if quant == "row" else ref.powers(s.cpu())
        assert (q[0] == 0).all() and (q[3, 64:] == 0).all()
        assert not torch.isfinite(s[1]).all() and not torch.isfinite(s[2]).all()
        assert torch.isfinite(s[0]).all() and torch.isfinite(s[3]).all()
    # tiny values: scales near the smallest numbers, eps 0 keeps the norm itself ordinary
    t = (torch.randn((3, 256), generator=_gen(1)) * 1e-3).to(BF)
    w = torch.full((256,), 2.0 ** -120, dtype=BF)
    y, _ = ref.norm(t, w, None, 0.0)
    q, _, s = psispec_add_rmsnorm(_gpu(t), _gpu(w), eps=0.0, quant="mx")
    s = ref.powers(s.cpu()).repeat_interleave(32, 1)
    err = (q.cpu().double() * s - y).abs()
    assert (err <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * s).all()
    q, _, s = psispec_add_rmsnorm(_gpu(t), _gpu(w), eps=0.0, quant="row")
    # y near 2^-120 is 448 times a scale near 2^-127, a number of 32 bits with 2^-149 as its step
    s = s.cpu().double()[:, None]
    err = (q.cpu().double() * s - y).abs()
    assert (err <= (2.0 ** -4 + 2.0 ** -16) * y.abs() + 2.0 ** -10 * s + 448 * 2.0 ** -149).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e25, 3e37])
@pytest.mark.parametrize("quant", [None, "row", "mx"])
@pytest.mark.parametrize("dim", [512, 3104, 9024])
def test_norm_of_numbers_whose_squares_32_bits_do_not_hold(scale, quant, dim):
    g = _gen(3)
    x = torch.zeros((5, dim), dtype=BF)
    r = torch.randn((5, dim), generator=g).clamp(-4, 4)
    r[[0, 1, 3, 4]] *= scale  # one ordinary row among them
    y, h = ref.norm(x, None, r, 0.0)
    out, ro, s = psispec_add_rmsnorm(_gpu(x), residual=_gpu(r), eps=0.0, quant=quant)
    assert torch.equal(ro.cpu(), r)
    s = 1.0 if s is None else s.cpu().double()[:, None] if quant == "row" else ref.powers(s.cpu()).repeat_interleave(32, 1)
    step = ref.half_step(y / s, BF if quant is None else F8) * s
    _within(out.cpu().double() * s, y, (2 * ref.NORM_REL * y.abs() + step) * (1 + 2.0 ** -8))


@pytest.mark.parametrize("dim,quant", [(8, None), (8, "row"), (32, "mx")])
def test_norm_of_more_rows_than_a_launch_takes(dim, quant):
    g = _gen(4)
    some, many = 4096, (1 << 21) + 4096 + 3
    x = torch.randn((some, dim), generator=g).to(BF).to(DEV)
    r = torch.randn((some, dim), generator=g).to(DEV)
    idx = torch.arange(many, device=DEV) % some
    first = psispec_add_rmsnorm(x, residual=r.clone(), quant=quant)
    for a, b in zip(psispec_add_rmsnorm(x[idx], residual=r[idx], quant=quant), first):
        if b is not None:
            assert torch.equal(a.view(torch.uint8), b[idx].view(torch.uint8))


# ------------------------------------------------------------------------------------- products

def _product(rows, n, k, dtype, fmt, group, seed, pad=0, bias=False, act=None, scale_dtype=BF, spread=4,
             out_dtype=None):
    g = _gen(seed)
    x, xs = ref.make_rows(rows, k, dtype, g)
    mats = [ref.make_weight(n, k, fmt, group, g, scale_dtype, spread) for _ in range(2 if act else 1)]
    ot = out_dtype or (BF if dtype == F8 else dtype)
    b = (torch.randn(n, generator=g)).to(ot) if bias else None
    packed = [psispec_w4_pack(_gpu(c), _gpu(s), fmt, group) for c, s in mats]
    _, xg = _inside(x, pad)
    xsg = None if xs is None else _inside(xs.view(torch.uint8), pad // 16)[1].view(E8)
    raw, out = _inside(torch.zeros((rows, n), dtype=ot), pad)
    if act:
        want, bound = ref.gated(x, xs, *mats, fmt, group, act, ot)
        got = psispec_w4_gated(xg, *packed, activation=act, x_scale=xsg, out=out)
    else:
        want, bound = ref.linear(x, xs, *mats[0], fmt, group, b, ot)
        got = psispec_w4_linear(xg, packed[0], x_scale=xsg, bias=_gpu(b), out=out)
    assert got is out
    _untouched(raw, pad, n)
    _within(out, want, bound, (rows, n, k))
    return x, xs, packed, out


KINDS = [(BF, "int", 128), (BF, "int", 64), (BF, "int", 32), (FH, "int", 128), (FH, "int", 64), (FH, "int", 32),
         (BF, "mx", 32), (FH, "mx", 32), (F8, "mx", 32)]


@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("k", [32, 64, 96, 128, 160, 256, 416, 1024, 1056, 4096])
def test_linear_inputs(dtype, fmt, group, k):
    _product(3, 40, k, dtype, fmt, group, seed=k)


@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 256, 300])
def test_linear_rows(dtype, fmt, group, rows):
    _product(rows, 72, 416, dtype, fmt, group, seed=rows)


@pytest.mark.parametrize("dtype,fmt,group", [(BF, "int", 128), (FH, "mx", 32), (F8, "mx", 32)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 129, 255, 257, 1003])
@pytest.mark.parametrize("rows", [1, 20, 40, 130])
def test_linear_outputs(dtype, fmt, group, n, rows):
    _product(rows, n, 288, dtype, fmt, group, seed=n)


@pytest.mark.parametrize("rows", [1, 20, 50, 140])
@pytest.mark.parametrize("dtype,fmt,group", KINDS)
def test_linear_bias_and_strides(dtype, fmt, group, rows):
    _product(rows, 50, 224, dtype, fmt, group, seed=rows, pad=16, bias=True)


@pytest.mark.parametrize("group", [128, 256, 384, 1024])
@pytest.mark.parametrize("scale_dtype", [BF, FH])
def test_linear_large_groups_and_scale_types(group, scale_dtype):
    _product(5, 24, 1056, BF, "int", group, seed=group, scale_dtype=scale_dtype)
    _product(70, 24, 1056, FH, "int", group, seed=group, scale_dtype=scale_dtype)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("rows", [1, 18, 40, 150])
def test_gated(act, dtype, fmt, group, rows):
    _product(rows, 90, 288, dtype, fmt, group, seed=rows, act=act, pad=16)


@pytest.mark.parametrize("rows,n,k", [(1, 6144, 4096), (9, 4096, 2048), (64, 1024, 4096), (576, 512, 4096),
                                      (130, 2048, 8192), (2000, 300, 1024)])
@pytest.mark.parametrize("dtype,fmt,group", [(BF, "int", 128), (FH, "int", 32), (BF, "mx", 32), (F8, "mx", 32)])
def test_linear_large(rows, n, k, dtype, fmt, group):
    _product(rows, n, k, dtype, fmt, group, seed=3, spread=8)


@pytest.mark.parametrize("rows,n,k", [(1601, 2039, 32), (1601, 2039, 160), (3137, 2047, 288), (801, 2033, 8224),
                                      (900, 2048, 16384)])
@pytest.mark.parametrize("dtype,fmt,group", KINDS)
def test_linear_many(rows, n, k, dtype, fmt, group):
    """Sizes that are cut into tiles of 64 rows x 256 and 128 outputs, and into parts of the inputs."""
    _product(rows, n, k, dtype, fmt, group, seed=k, pad=16 * (k < 1000), bias=k == 160, spread=8)


@pytest.mark.parametrize("rows,n,k", [(801, 2039, 160), (1600, 2047, 416), (449, 2035, 8224)])
@pytest.mark.parametrize("dtype,fmt,group", KINDS)
def test_gated_many(rows, n, k, dtype, fmt, group):
    _product(rows, n, k, dtype, fmt, group, seed=k, act="silu", pad=16 * (k < 1000), scale_dtype=FH)


def test_8bit_rows_to_f16():
    _product(20, 33, 256, F8, "mx", 32, seed=1, out_dtype=FH)
    _product(90, 33, 256, F8, "mx", 32, seed=1, out_dtype=FH, act="silu")


@pytest.mark.parametrize("rows,n", [(4, 48), (80, 48), (1601, 2039)])
def test_f16_rows_take_far_apart_mx_scales(rows, n):
    """Scales over 2^-30 of the largest are exact for F16 rows; an output whose scales are all small, or all
    large, is scaled back as a whole."""
    g = _gen(2)
    k = 512
    codes, s = ref.make_weight(n, k, "mx", 32, g, spread=30)
    e = s.view(torch.uint8).clone()
    e[1] = 60   # an output of tiny weights, one of large ones
    e[2] = 127 + 6
    e[3, :] = 97
    e[3, 5] = 127
    s = e.view(E8)
    x, _ = ref.make_rows(rows, k, FH, g)
    want, bound = ref.linear(x, None, codes, s, "mx", 32, None, FH)
    got = psispec_w4_linear(_gpu(x), psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32))
    _within(got, want, bound)
    # only the inputs of the small blocks: nothing of them is lost under the large one
    x[:, 160:192] = 0
    want, bound = ref.linear(x, None, codes, s, "mx", 32, None, FH)
    got = psispec_w4_linear(_gpu(x), psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32))
    _within(got, want, bound)


@pytest.mark.parametrize("rows,n", [(3, 40), (80, 40), (1601, 2039)])
@pytest.mark.parametrize("dtype", [BF, FH, F8])
def test_nan_scales_and_bad_rows_stay_where_they_are(rows, n, dtype):
    g = _gen(9)
    k = 288
    codes, s = ref.make_weight(n, k, "mx", 32, g)
    e = s.view(torch.uint8).clone()
    e[7, 3] = 255
    x, xs = ref.make_rows(rows, k, dtype, g)
    clean = psispec_w4_linear(_gpu(x), psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32), x_scale=_gpu(xs))
    w = psispec_w4_pack(_gpu(codes), _gpu(e.view(E8)), "mx", 32)
    out = psispec_w4_linear(_gpu(x), w, x_scale=_gpu(xs))
    assert torch.isnan(out[:, 7]).all()
    keep = [i for i in range(n) if i != 7]
    assert torch.equal(out[:, keep], clean[:, keep])
    if xs is not None:  # a NaN among the rows' scales
        e = xs.view(torch.uint8).clone()
        e[2, 4] = 255
        out = psispec_w4_linear(_gpu(x), psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32), x_scale=_gpu(e.view(E8)))
        rest = [i for i in range(rows) if i != 2]
        assert torch.isnan(out[2]).all() and torch.equal(out[rest], clean[rest])
    x2 = x.clone()
    x2[1, 10] = float("nan")
    out = psispec_w4_linear(_gpu(x2), psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32), x_scale=_gpu(xs))
    assert torch.isnan(out[1]).all()
    rest = [i for i in range(rows) if i != 1]
    assert torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("rows,n", [(3, 33), (80, 33), (1601, 2039)])
@pytest.mark.parametrize("dtype,fmt,group", KINDS)
def test_inputs_behind_the_last_are_not_read(rows, n, dtype, fmt, group):
    """NaN right behind each row's inputs, in the columns that a tile of 128 still covers, and behind the last row."""
    g = _gen(4)
    k = 160
    x, xs = ref.make_rows(rows, k, dtype, g)
    codes, s = ref.make_weight(n, k, fmt, group, g)
    raw = torch.full((rows + 40, k + 128), float("nan"), device=DEV).to(dtype)
    raw[:rows, :k] = _gpu(x)
    sraw = None
    if xs is not None:
        sraw = torch.full((rows + 40, 16), 255, dtype=torch.uint8, device=DEV)
        sraw[:rows, :k // 32] = _gpu(xs.view(torch.uint8))
        sraw = sraw.view(E8)[:rows, :k // 32]
    want, bound = ref.linear(x, xs, codes, s, fmt, group, None, BF if dtype == F8 else dtype)
    got = psispec_w4_linear(raw[:rows, :k], psispec_w4_pack(_gpu(codes), _gpu(s), fmt, group), x_scale=sraw)
    _within(got, want, bound)


def test_packing_takes_views():
    g = _gen(6)
    n, k = 37, 224
    codes, s = ref.make_weight(n, k, "int", 64, g)
    wide = torch.randint(0, 255, (n, 131), generator=g).to(torch.uint8).to(DEV)
    wide[:, 5:5 + k // 2] = _gpu(codes)
    sw = torch.zeros((n, 9), dtype=BF, device=DEV)
    sw[:, 3:7] = _gpu(s)
    a = psispec_w4_pack(_gpu(codes), _gpu(s), "int", 64)
    buf = torch.full((a.packed.numel() + 512,), 9, dtype=torch.uint8, device=DEV)
    b = psispec_w4_pack(wide[:, 5:5 + k // 2], sw[:, 3:7], "int", 64, packed=buf)
    used = 1024 * 3 * 2 + 64 * 3 * 2
    assert torch.equal(a.packed[:used], buf[:used]) and (buf[a.packed.numel():] == 9).all()
    x = torch.randn((4, k), generator=g).to(BF).to(DEV)
    assert torch.equal(psispec_w4_linear(x, a), psispec_w4_linear(x, b))


def test_rows_beyond_32_bit_offsets():
    """Rows more than 2^31 elements from the first, and more sums of groups than one launch has threads for."""
    g = _gen(31)
    some, many, n, k = 128, (1 << 17) + 70, 40, 16512
    codes, s = ref.make_weight(n, k, "int", 128, g)
    w = psispec_w4_pack(_gpu(codes), _gpu(s))
    x = _gpu(ref.make_rows(some, k, BF, g)[0])
    idx = torch.arange(many, device=DEV) % some
    y = psispec_w4_linear(x[idx], w)
    want, bound = ref.linear(x.cpu(), None, codes, s, "int", 128, None, BF)
    _within(y[-some:].roll(many % some, 0), want, bound)
    assert torch.equal(y, y[:some][idx])


def test_packed_bytes_again():
    g = _gen(32)
    codes, s = ref.make_weight(48, 160, "mx", 32, g)
    w = psispec_w4_pack(_gpu(codes), _gpu(s), "mx", 32)
    x = _gpu(ref.make_rows(3, 160, BF, g)[0])
    assert torch.equal(psispec_w4_linear(x, W4Weight(w.packed.clone(), 48, 160, 32, "mx", E8)), psispec_w4_linear(x, w))
    for bad in ((w.packed[:-1], 48, 160, 32, "mx", E8), (w.packed.cpu(), 48, 160, 32, "mx", E8),
                (w.packed, 64, 320, 32, "mx", E8), (w.packed, 48, 160, 32, "mx", BF), (w.packed, 48, 160, 32, "int", E8),
                (w.packed, 48, 150, 32, "mx", E8), (w.packed, 48, 160, 32, "nf4", BF), (w.packed.float(), 48, 160, 32, "mx", E8)):
        with pytest.raises(PsispecError):
            W4Weight(*bad)
    with pytest.raises(AttributeError):
        w.packed = w.packed.clone()


def test_gated_far_from_zero():
    """A gate of large negative and positive sums: what the activations leave is still right to the last bit but one."""
    codes = torch.full((16, 16), 0x22, dtype=torch.uint8)  # w = 1 and 1: MX code 2
    w = psispec_w4_pack(_gpu(codes), _gpu(torch.full((16, 1), 127, dtype=torch.uint8).view(E8)), "mx", 32)
    a = torch.tensor([-60.0, -12.0, -9.0, -6.5, -5.0, -4.0, -2.0, -0.5, 0.0, 0.5, 5.0, 60.0, 3e4, -3e4, 1e30, -1e30])
    x = torch.zeros((16, 32))
    x[:, 0] = a
    x = x.to(BF)
    a = x[:, 0].double()
    for act, f in ref.ACT.items():
        y = psispec_w4_gated(_gpu(x), w, w, activation=act).cpu().double()[:, 0]
        if act == "gelu":
            want = a * torch.special.log_ndtr(a).exp()
        else:
            u = a if act == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
            want = a * torch.where(u < -700, 0.0, torch.sigmoid(u))
        want = want * a
        # the exponent u is off by a few 2^-24 |u| in 32 bits, and the exponential by that much of itself; beyond
        # 2^11 a negative side is 0
        u = a.abs() if act == "silu" else (a * a / 2 if act == "gelu" else 2 * 0.8 * (a.abs() + 0.045 * a.abs() ** 3))
        big = want.abs() > 2.0 ** 120
        rel = 2.0 ** -8 + 2.0 ** -21 * (u.clamp(max=2048) + 8)
        err = (y - want).abs()
        assert (err[~big] <= (rel * want.abs() + 2.0 ** -126 * (1 + a.abs()))[~big]).all(), (act, y, want)
        assert torch.isfinite(y[a < 0][:8]).all()


def test_empty_and_batched_rows():
    g = _gen(8)
    codes, s = ref.make_weight(48, 128, "int", 128, g)
    w = psispec_w4_pack(_gpu(codes), _gpu(s))
    assert psispec_w4_linear(torch.empty((0, 128), dtype=BF, device=DEV), w).shape == (0, 48)
    x = torch.randn((5, 9, 128), generator=g).to(BF).to(DEV)
    y = psispec_w4_linear(x, w)
    assert y.shape == (5, 9, 48) and torch.equal(y.view(45, 48), psispec_w4_linear(x.view(45, 128), w))
    assert psispec_w4_gated(x, w, w).shape == (5, 9, 48)
    assert psispec_add_rmsnorm(x[:0])[0].shape == (0, 9, 128)


@pytest.mark.parametrize("rows,n", [(1, 520), (30, 520), (64, 520), (300, 520), (1601, 2039)])
def test_runs_are_bitwise_equal(rows, n):
    g = _gen(rows)
    codes, s = ref.make_weight(n, 2080, "int", 128, g)
    w = psispec_w4_pack(_gpu(codes), _gpu(s))
    x = _gpu(ref.make_rows(rows, 2080, BF, g)[0])
    first = psispec_w4_linear(x, w)
    for _ in range(5):
        assert torch.equal(first, psispec_w4_linear(x, w))


def test_two_streams_with_workspaces_of_their_own():
    g = _gen(12)
    codes, s = ref.make_weight(4096, 8192, "int", 128, g)
    w = psispec_w4_pack(_gpu(codes), _gpu(s))
    xs = [_gpu(ref.make_rows(r, 8192, BF, g)[0]) for r in (500, 440)]  # inputs in parts
    assert all(w4_workspace_bytes(x.shape[0], 4096, 8192) > x.shape[0] * 4096 * 4 for x in xs)
    want = [psispec_w4_linear(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(4):
        for i, (x, st) in enumerate(zip(xs, streams)):
            got[i].append(psispec_w4_linear(x, w, stream=st))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a, y) for y in b)


@pytest.mark.parametrize("fmt,rows,h,f", [("mx", 9, 256, 640), ("mx", 160, 256, 640), ("int", 1601, 1024, 2048),
                                          ("mx", 801, 2048, 8192)])
def test_layer_in_a_graph(fmt, rows, h, f):
    """Norm, gated projections and the projection back, captured once and replayed on new rows."""
    g = _gen(13)
    mats = [psispec_w4_pack(*map(_gpu, ref.make_weight(*nk, fmt, 32, g)), fmt, 32) for nk in
            ((f, h), (f, h), (h, f))]
    wt = _gpu((1 + 0.1 * torch.randn(h, generator=g)).to(BF))
    x = torch.zeros((rows, h), dtype=BF, device=DEV)
    res = torch.zeros((rows, h), device=DEV)
    ro = torch.zeros_like(res)

    def layer():
        q, _, s = psispec_add_rmsnorm(x, wt, residual=res, residual_out=ro, quant="mx" if fmt == "mx" else None)
        a = psispec_w4_gated(q, mats[0], mats[1], x_scale=s)
        return psispec_w4_linear(a, mats[2])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for i in range(4):
        x.copy_(_gpu(torch.randn((rows, h), generator=g).to(BF)))
        res.copy_(_gpu(torch.randn((rows, h), generator=g)))
        graph.replay()
        torch.cuda.synchronize()
        replayed, kept = y.clone(), ro.clone()
        assert torch.equal(replayed, layer()) and torch.equal(kept, ro)


def test_two_graphs_share_a_workspace():
    """Captured apart, replayed in turn on one stream with eager calls of the same workspace between them."""
    g = _gen(14)
    n, k = 4096, 8192
    w = psispec_w4_pack(*map(_gpu, ref.make_weight(n, k, "int", 128, g)))
    xs = [torch.zeros((r, k), dtype=BF, device=DEV) for r in (500, 440)]  # inputs in parts
    ws = torch.empty(max(w4_workspace_bytes(x.shape[0], n, k) for x in xs), dtype=torch.uint8, device=DEV)
    outs = [psispec_w4_linear(x, w, workspace=ws) for x in xs]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in xs]
    for x, o, gr in zip(xs, outs, graphs):
        with torch.cuda.graph(gr):
            psispec_w4_linear(x, w, out=o, workspace=ws)
    for i in range(4):
        for x in xs:
            x.copy_(_gpu(torch.randn(x.shape, generator=g).to(BF)))
        for gr in graphs:
            gr.replay()
        got = [o.clone() for o in outs]
        want = [psispec_w4_linear(x, w, workspace=ws) for x in xs]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_a_whole_layer_of_a_verify_forward():
    """Norm, projection, append, attention, projection back, norm, gated block: each step against its 64-bit form
    on the inputs that it was given."""
    g = _gen(21)
    b, blk, hq, hkv, d, f, ps = 3, 5, 4, 2, 64, 384, 16
    h = hq * d
    qkv_n = (hq + 2 * hkv) * d
    shapes = {"qkv": (qkv_n, h), "o": (h, h), "gate": (f, h), "up": (f, h), "down": (h, f)}
    raw = {k: ref.make_weight(*s, "int", 64, g) for k, s in shapes.items()}
    w = {k: psispec_w4_pack(_gpu(c), _gpu(s), "int", 64) for k, (c, s) in raw.items()}
    n1, n2 = ((1 + 0.1 * torch.randn(h, generator=g)).to(BF) for _ in range(2))
    stream = torch.randn((b, blk, h), generator=g).to(BF)
    lens = torch.tensor([3, 20, 0], dtype=torch.int32)
    tab = torch.arange(6, dtype=torch.int32).view(3, 2)
    kc = torch.randn((6, ps, hkv, d), generator=g).to(BF).to(DEV)
    vc = torch.randn((6, ps, hkv, d), generator=g).to(BF).to(DEV)
    inv, _ = rope_frequencies(d, device=DEV)

    def flat(t):
        return t.reshape(-1, t.shape[-1]).cpu()

    def check(y, x, key):
        want, bound = ref.linear(flat(x), None, *raw[key], "int", 64, None, BF)
        _within(flat(y), want, bound, key)

    x, _, _ = psispec_add_rmsnorm(_gpu(stream), _gpu(n1))
    p = psispec_w4_linear(x, w["qkv"])
    check(p, x, "qkv")
    q, k, v = p.view(b, blk, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=2)
    qo = psispec_qkv_append(q, k, v, kc, vc, _gpu(tab), _gpu(lens), inv_freq=inv)
    at = psispec_paged_attention(qo, kc, vc, _gpu(tab), _gpu(lens)).view(b, blk, h)
    o = psispec_w4_linear(at, w["o"])
    check(o, at, "o")
    res = _gpu(stream)
    y, res2, _ = psispec_add_rmsnorm(o, _gpu(n2), residual=res)
    wy, wh = ref.norm(flat(o), n2, flat(stream), 1e-6)
    _within(flat(y), wy, (ref.NORM_REL * wy.abs() + ref.half_step(wy, BF)) * (1 + 2.0 ** -8))
    _within(flat(res2), wh, ref.half_step(wh, BF) + 2.0 ** -24 * wh.abs())
    a = psispec_w4_gated(y, w["gate"], w["up"])
    want, bound = ref.gated(flat(y), None, raw["gate"], raw["up"], "int", 64, "silu", BF)
    _within(flat(a), want, bound)
    check(psispec_w4_linear(a, w["down"]), a, "down")


def test_refusals_of_the_binding():
    g = _gen(30)
    codes, s = (t.to(DEV) for t in ref.make_weight(32, 128, "int", 128, g))
    w = psispec_w4_pack(codes, s)
    x = torch.zeros((4, 128), dtype=BF, device=DEV)
    for bad in (x.float(), x[:, :64], x.cpu(), x.t().contiguous().t(), x.to(F8)):
        with pytest.raises(PsispecError):
            psispec_w4_linear(bad, w)
    odd = torch.zeros((4, 129), dtype=BF, device=DEV)
    for bad in (odd[:, :128], odd.view(-1)[1:513].view(4, 128)):  # rows that are not 16-byte aligned
        with pytest.raises(PsispecError, match="code -1"):
            psispec_w4_linear(bad, w)
    with pytest.raises(PsispecError):
        psispec_w4_linear(x, w, bias=torch.zeros(32, device=DEV))
    with pytest.raises(PsispecError):
        psispec_w4_linear(x, w, out=torch.zeros((4, 31), dtype=BF, device=DEV))
    with pytest.raises(PsispecError):
        psispec_w4_linear(x, w, out_dtype=FH)
    with pytest.raises(PsispecError):
        psispec_w4_linear(x, w, x_scale=torch.zeros((4, 4), dtype=torch.uint8, device=DEV).view(E8))
    with pytest.raises(PsispecError, match="code -1"):
        psispec_w4_linear(x, w, out=x[:, 64:96])
    with pytest.raises(PsispecError):
        psispec_w4_gated(x, w, w, activation="relu")
    other = psispec_w4_pack(codes, torch.ones((32, 4), dtype=BF, device=DEV), group=32)
    with pytest.raises(PsispecError):
        psispec_w4_gated(x, w, other)
    for kw in (dict(group=48), dict(group=96), dict(group=16), dict(format="nf4"), dict(format="mx", group=32)):
        with pytest.raises(PsispecError):
            psispec_w4_pack(codes, torch.ones((32, -(-128 // kw.get("group", 128))), dtype=BF, device=DEV), **kw)
    with pytest.raises(PsispecError):
        psispec_w4_pack(codes[:, :40], s)  # 80 inputs
    with pytest.raises(PsispecError):
        psispec_w4_pack(codes, s, packed=torch.zeros(100, dtype=torch.uint8, device=DEV))
    with pytest.raises(PsispecError):
        psispec_add_rmsnorm(x, out=x[:, :64])
    with pytest.raises(PsispecError, match="code -1"):
        psispec_add_rmsnorm(x[:3], out=x[1:])
    with pytest.raises(PsispecError):
        psispec_add_rmsnorm(x[:, :100], quant="mx")
    with pytest.raises(PsispecError):
        psispec_add_rmsnorm(x, eps=-1.0)
    with pytest.raises(PsispecError):
        psispec_add_rmsnorm(x, scale=torch.zeros(4, device=DEV))
    with pytest.raises(PsispecError):
        psispec_add_rmsnorm(x, residual=x.half())


def test_workspace_is_what_the_query_says():
    for rows, n, k in ((1, 64, 128), (100, 500, 512), (1601, 2039, 416), (801, 2033, 8224)):
        g = _gen(rows)
        codes, s = ref.make_weight(n, k, "int", 128, g)
        w = psispec_w4_pack(_gpu(codes), _gpu(s))
        x = _gpu(ref.make_rows(rows, k, BF, g)[0])
        need = w4_workspace_bytes(rows, n, k)
        ws = torch.full((need + 512,), 9, dtype=torch.uint8, device=DEV)
        y = psispec_w4_linear(x, w, workspace=ws[:need] if need else None)
        assert (ws[need:] == 9).all()
        assert torch.equal(y, psispec_w4_linear(x, w))
