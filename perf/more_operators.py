"""The layers around the paged attention of a verify or draft forward as measured cases: the plain torch
form of each operator and the framework's call for it, on the same inputs.

Operators (key "op" of a case):
  norm    psispec_add_rmsnorm: the residual's addition and the root-mean-square norm, the output in
          16 bits or in 8 bits with scales (one 32-bit number per row, or a power of two per 32 columns)
  linear  psispec_w4_linear: a linear layer with weights of 4 bits and a scale per group of inputs
  gated   psispec_w4_gated: the two projections of a gated feed-forward block, the activation and the
          product, weights of 4 bits
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "f8": 1}
DEV = "cuda"
EPS = 1e-6


def listed():
    # hidden size 4096, 32 query and 8 key/value heads of 128 (6144 rows in their projection), a
    # feed-forward width of three times the hidden size; 64 lines with 9 rows each in a verify forward
    r = dict(op="norm", dim=4096, type="bf16", residual="bf16", quant="none", pad=0)
    w = dict(op="linear", type="bf16", fmt="int", group=128, bias=False, pad=0)
    g = dict(op="gated", n=12288, k=4096, type="bf16", fmt="int", group=128, act="silu", pad=0)
    return [
        # one user's token: latency
        dict(r, name="norm-one", rows=1),
        # the verify forward of a serving batch, rows for the 8-bit products
        dict(r, name="norm-verify-mx", rows=576, quant="mx"),
        # chunks of prompts, a residual stream in 32 bits, 8 bits with a scale per row
        dict(r, name="norm-prompt-row", rows=8000, dim=5120, type="f16", residual="f32", quant="row"),
        # the query, key and value projection of one user's token
        dict(w, name="linear-one", rows=1, n=6144, k=4096),
        # one user's block of 8 drafts through the projection back from the feed-forward width
        dict(w, name="linear-block-mx", rows=9, n=4096, k=12288, fmt="mx", group=32),
        # a serving batch in plain decoding, the projection behind the attention
        dict(w, name="linear-decode-f16", rows=64, n=4096, k=4096, type="f16", group=64),
        # odd sizes: a small head with a bias, rows inside wider rows
        dict(w, name="linear-ragged", rows=37, n=1003, k=2720, group=32, bias=True, pad=24),
        # the verify forward of a serving batch, rows in 8 bits
        dict(w, name="linear-verify-mx8", rows=576, n=6144, k=4096, type="f8", fmt="mx", group=32),
        # chunks of prompts
        dict(w, name="linear-prompt", rows=2048, n=4096, k=12288),
        # one user's token through the wide layers of the feed-forward block
        dict(g, name="gated-one-mx", rows=1, fmt="mx", group=32),
        # a serving batch in plain decoding, rows in 8 bits
        dict(g, name="gated-decode-mx8", rows=64, type="f8", fmt="mx", group=32),
        # the verify forward of a serving batch
        dict(g, name="gated-verify", rows=576),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "gated"])
    ty = rng.choice(["bf16", "bf16", "f16"])
    if op == "norm":
        quant = rng.choice(["none", "row", "mx"])
        rows = _span(rng, 1, 8000)
        dim = _span(rng, 16, min(16384, 40000000 // rows))
        if quant == "mx" or rng.random() < 0.5:
            dim = max(1, dim // 32) * 32
        return dict(op=op, rows=rows, dim=dim, type=ty, residual=rng.choice(["none", ty, ty, "f32"]),
                    quant=quant, pad=rng.choice([0, 0, 32, 5]))
    fmt = rng.choice(["int", "int", "mx"])
    if fmt == "mx":
        ty = rng.choice([ty, "f8"])
    n = _span(rng, 16, 12288)
    k = 32 * _span(rng, 2, 384)
    most = (1 << 36) // (n * k * (2 if op == "gated" else 1))
    rows = _span(rng, 1, min(2048, max(1, most)))
    if rng.random() < 0.5:
        n = max(1, n // 16) * 16
    if rng.random() < 0.5:
        k = max(128, k // 128 * 128)
    c = dict(op=op, rows=rows, n=n, k=k, type=ty, fmt=fmt,
             group=32 if fmt == "mx" else rng.choice([32, 64, 128, 128]), pad=rng.choice([0, 0, 16, 48]))
    if op == "gated":
        return dict(c, act=rng.choice(["silu", "silu", "gelu"]))
    return dict(c, bias=rng.random() < 0.3)


def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        d, es = case["dim"], BYTES[case["type"]]
        stream = 0 if case["residual"] == "none" else 2 * BYTES[case["residual"]]
        quant = {"none": es, "row": 1, "mx": 1 + 1 / 32}[case["quant"]]
        return {"bytes": int(rows * d * (es + stream + quant)) + d * es + (4 * rows if case["quant"] == "row" else 0),
                "flops": 8 * rows * d}
    n, k = case["n"], case["k"]
    mats = 2 if case["op"] == "gated" else 1
    weight = n * k // 2 + n * -(-k // case["group"]) * (1 if case["fmt"] == "mx" else 2)
    xs = rows * k * BYTES[case["type"]] + (rows * k // 32 if case["type"] == "f8" else 0)
    return {"bytes": mats * weight + xs + 2 * rows * n, "flops": 2 * mats * rows * n * k}


# ------------------------------------------------------------------------------------- inputs

def _e2m1():
    """The values of the 16 codes of a 4-bit float: sign, two bits of exponent, one of mantissa."""
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.cat([v, -v])


def _nibbles(code):
    """Codes 0..15 [n][k] as bytes [n][k/2], the even column's in the low four bits."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)


def _quantised(n, k, fmt, group, g):
    """(bytes of codes, scales) of a layer's weights, drawn as a trained layer's are spread."""
    groups = -(-k // group)
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((n, groups), dtype=torch.uint8 if fmt == "mx" else torch.bfloat16, device=DEV)
    step = max(1, (1 << 24) // k)
    for i in range(0, n, step):
        m = min(step, n - i)
        w = torch.randn((m, groups * group), generator=g, device=DEV) * 0.02
        w = w * (1.0 + torch.rand((m, 1), generator=g, device=DEV))
        w[:, k:] = 0.0
        w = w.view(m, groups, group)
        top = w.abs().amax(-1)
        if fmt == "mx":
            e = torch.floor(torch.log2(top)) - 2.0  # 6 is the largest code
            v = (w * torch.exp2(-e)[..., None]).abs()
            edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
            code = torch.bucketize(v, edge) + 8 * (w < 0)
            scales[i:i + m] = (e + 127.0).to(torch.uint8)
        else:
            s = (top / 7.5).to(torch.bfloat16)
            code = torch.round(w / s.float()[..., None]).clamp(-8, 7).to(torch.int64) & 15
            scales[i:i + m] = s
        codes[i:i + m] = _nibbles(code.reshape(m, -1)[:, :k])
    return codes, scales.view(torch.float8_e8m0fnu) if fmt == "mx" else scales


def _rows(rows, width, pad, dtype):
    """Rows of `width` that lie inside rows of width + pad."""
    return torch.zeros((rows, width + pad), dtype=dtype, device=DEV)[:, :width]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    rows, pad = case["rows"], case["pad"]
    dt = DTYPES[case["type"]]
    if case["op"] == "norm":
        d = case["dim"]
        st["x"] = _rows(rows, d, pad, dt)
        st["x"].copy_(torch.randn((rows, d), generator=g, device=DEV))
        st["weight"] = (1.0 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["residual"] = st["residual_out"] = None
        if case["residual"] != "none":
            rt = DTYPES[case["residual"]]
            st["residual"], st["residual_out"] = _rows(rows, d, pad, rt), _rows(rows, d, pad, rt)
            # a few columns of a residual stream are far larger than the others
            big = 1.0 + 30.0 * (torch.rand(d, generator=g, device=DEV) < 0.004)
            st["residual"].copy_(torch.randn((rows, d), generator=g, device=DEV) * 3.0 * big)
        st["out"] = _rows(rows, d, pad if case["quant"] == "none" else 32 * (pad > 0),
                          dt if case["quant"] == "none" else DTYPES["f8"])
        st["scale"] = None
        if case["quant"] == "row":
            st["scale"] = torch.zeros(rows, device=DEV)
        elif case["quant"] == "mx":
            st["scale"] = torch.zeros((rows, d // 32), dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        return st
    n, k = case["n"], case["k"]
    st["w"] = [_quantised(n, k, case["fmt"], case["group"], g)
               for _ in range(2 if case["op"] == "gated" else 1)]
    x = torch.randn((rows, k), generator=g, device=DEV)
    x = x * (1.0 + 10.0 * (torch.rand(k, generator=g, device=DEV) < 0.01))
    st["x"], st["x_scale"] = _rows(rows, k, pad, dt), None
    if case["type"] == "f8":
        v = x.view(rows, k // 32, 32)
        e = torch.ceil(torch.log2(v.abs().amax(-1) / 448.0))
        st["x_scale"] = (e + 127.0).to(torch.uint8).view(torch.float8_e8m0fnu)
        x = (v * torch.exp2(-e)[..., None]).view(rows, k)
    st["x"].copy_(x.to(dt))
    st["out_type"] = torch.bfloat16 if case["type"] == "f8" else dt
    st["out"] = _rows(rows, n, (-n) % 8, st["out_type"])
    st["bias"] = None
    if case.get("bias"):
        st["bias"] = (0.5 * torch.randn(n, generator=g, device=DEV)).to(st["out_type"])
    if own:
        import lossless_draft_verification_spec_amd as pkg
        st["packed"] = [pkg.psispec_w4_pack(c, s, case["fmt"], group=case["group"]) for c, s in st["w"]]
        st["ws"] = torch.empty(max(1, pkg.w4_workspace_bytes(rows, n, k, len(st["w"]))), dtype=torch.uint8,
                               device=DEV)
    return st


# ------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "gated": _own_gated}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "gated": _plain_gated}[op](state)


def _own_norm(st):
    import lossless_draft_verification_spec_amd as pkg
    q = st["case"]["quant"]
    return pkg.psispec_add_rmsnorm(st["x"], st["weight"], residual=st["residual"],
                                   residual_out=st["residual_out"], eps=EPS,
                                   quant=None if q == "none" else q, out=st["out"], scale=st["scale"])


def _own_linear(st):
    import lossless_draft_verification_spec_amd as pkg
    return pkg.psispec_w4_linear(st["x"], st["packed"][0], x_scale=st["x_scale"], bias=st["bias"],
                                 out=st["out"], workspace=st["ws"])


def _own_gated(st):
    import lossless_draft_verification_spec_amd as pkg
    return pkg.psispec_w4_gated(st["x"], st["packed"][0], st["packed"][1],
                                activation=st["case"]["act"], x_scale=st["x_scale"], out=st["out"],
                                workspace=st["ws"])


def _powers(scale):
    """The 32-bit values of a tensor of powers of two stored as their exponents."""
    return torch.exp2(scale.view(torch.uint8).float() - 127.0)


def _plain_norm(st):
    c, x = st["case"], st["x"]
    h = x.float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
        st["residual_out"].copy_(h)
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * st["weight"].float()
    if c["quant"] == "row":
        s = y.abs().amax(-1) / 448.0
        st["scale"].copy_(s)
        y = torch.where(s[:, None] > 0, y / s[:, None], torch.zeros_like(y)).clamp(-448.0, 448.0)
    elif c["quant"] == "mx":
        v = y.view(c["rows"], -1, 32)
        top = v.abs().amax(-1)
        e = torch.ceil(torch.log2(top.double() / 448.0)).clamp(-127.0, 127.0)
        st["scale"].view(torch.uint8).copy_(e + 127.0)
        y = (v * torch.exp2(-e)[..., None]).float().view(y.shape)
    st["out"].copy_(y)
    return st["out"], st["residual_out"], st["scale"]


def _plain_weight(case, codes, scales):
    """The layer's weights [n][k] in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(1)
    if case["fmt"] == "mx":
        w, s = _e2m1()[code.int()], _powers(scales)
    else:
        w, s = ((code ^ 8).float() - 8.0), scales.float()
    return w * s.repeat_interleave(case["group"], 1)[:, :case["k"]]


def _plain_rows(st):
    x = st["x"].float()
    if st["x_scale"] is not None:
        x = x * _powers(st["x_scale"]).repeat_interleave(32, 1)
    return x


def _plain_linear(st):
    y = torch.matmul(_plain_rows(st), _plain_weight(st["case"], *st["w"][0]).t())
    if st["bias"] is not None:
        y = y + st["bias"].float()
    st["out"].copy_(y)
    return st["out"]


def _plain_gated(st):
    x = _plain_rows(st)
    a = torch.matmul(x, _plain_weight(st["case"], *st["w"][0]).t())
    u = torch.matmul(x, _plain_weight(st["case"], *st["w"][1]).t())
    if st["case"]["act"] == "silu":
        a = a / (1.0 + torch.exp(-a))
    else:
        a = a * 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
    st["out"].copy_(a * u)
    return st["out"]


# ------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, st)
    x = st["x"].double()
    if st["x_scale"] is not None:
        e = st["x_scale"].view(torch.uint8).int() - 127
        x = torch.ldexp(x.unflatten(1, (-1, 32)), e[..., None]).flatten(1)
    y = [_exact_product(case, x, *w) for w in st["w"]]
    if case["op"] == "linear":
        return y[0] if st["bias"] is None else y[0] + st["bias"].double()
    a = y[0]
    return y[1] * (a * torch.sigmoid(a) if case["act"] == "silu" else a * torch.special.ndtr(a))


def _exact_norm(case, st):
    h = st["x"].double()
    if st["residual"] is not None:
        h = h + st["residual"].double()
    size = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / case["dim"] + EPS)
    y, s = h / size * st["weight"].double(), None
    if case["quant"] == "row":
        s = torch.linalg.vector_norm(y, ord=math.inf, dim=1) / 448
        y = y / s[:, None]
    elif case["quant"] == "mx":
        b = y.unflatten(1, (-1, 32))
        frac, e = torch.frexp(torch.linalg.vector_norm(b, ord=math.inf, dim=2))  # frac in [1/2, 1)
        e = e - 9 + (frac > 0.875).int()  # 448 = 0.875 * 2^9
        s = torch.ldexp(torch.ones_like(frac), e)
        y = (b / s[..., None]).flatten(1)
    return y, None if st["residual"] is None else h, s


def _exact_product(case, x, codes, scales):
    """A slice of outputs at a time: values by a table of the 256 bytes, groups scaled one by one."""
    k, group = case["k"], case["group"]
    byte = torch.arange(256, device=DEV)
    pair = torch.stack([byte % 16, torch.div(byte, 16, rounding_mode="floor")], 1)
    if case["fmt"] == "mx":
        mant, ex = pair % 2, torch.div(pair % 8, 2, rounding_mode="floor")
        size = torch.where(ex > 0, (2 + mant) * 2.0 ** (ex - 2), mant * 0.5)
        value = torch.where(pair >= 8, -size, size).double()
        s = 2.0 ** (scales.view(torch.uint8).double() - 127)
    else:
        value = torch.where(pair >= 8, pair - 16, pair).double()
        s = scales.double()
    out = torch.empty((x.shape[0], codes.shape[0]), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // k)
    for i in range(0, codes.shape[0], step):
        w = value[codes[i:i + step].long()].flatten(1)
        for j in range(s.shape[1]):
            w[:, j * group:(j + 1) * group] *= s[i:i + step, j, None]
        out[:, i:i + step] = torch.mm(x, w.t())
    return out
