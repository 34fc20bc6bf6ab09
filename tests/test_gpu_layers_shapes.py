"""Every kernel of the 4-bit products (layers_shapes.py) against the 64-bit references, for every kind of rows and
weights, and run again: bitwise the same."""
import pytest
import torch

import layers_ref as ref
from layers_ref import BF, F8, FH
from layers_shapes import GATED, LINEAR
from lossless_draft_verification_spec_amd import psispec_w4_gated, psispec_w4_linear, psispec_w4_pack
from test_gpu_layers import KINDS, _gen, _gpu, _product

pytestmark = pytest.mark.gpu


def _name(key):
    return "-".join(map(str, key))


@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("kernel", LINEAR, ids=_name)
def test_linear_kernels(kernel, dtype, fmt, group):
    rows, n, k = LINEAR[kernel]
    _product(rows, n, k, dtype, fmt, group, seed=n, pad=16, bias=True, spread=8)


@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("kernel", GATED, ids=_name)
def test_gated_kernels(kernel, dtype, fmt, group):
    rows, n, k = GATED[kernel]
    _product(rows, n, k, dtype, fmt, group, seed=n, pad=16, act="silu", scale_dtype=FH)


@pytest.mark.parametrize("dtype,fmt,group", KINDS)
@pytest.mark.parametrize("table", [LINEAR, GATED], ids=["linear", "gated"])
def test_runs_are_bitwise_equal(table, dtype, fmt, group):
    """On new rows in the same buffers, and among calls of other kernels."""
    for kernel, (rows, n, k) in table.items():
        g = _gen(n)
        x, xs = (_gpu(t) for t in ref.make_rows(rows, k, dtype, g))
        w = [psispec_w4_pack(*map(_gpu, ref.make_weight(n, k, fmt, group, g, spread=4)), fmt, group)
             for _ in range(2 if table is GATED else 1)]
        out = torch.empty((rows, n), dtype=BF if dtype == F8 else dtype, device=x.device)

        def run(x):
            if table is GATED:
                return psispec_w4_gated(x, *w, x_scale=xs, out=out).clone()
            return psispec_w4_linear(x, w[0], x_scale=xs, out=out).clone()

        first, other = run(x), run(x.flip(0).contiguous())
        for _ in range(3):
            assert torch.equal(first, run(x)), kernel
            assert torch.equal(other, run(x.flip(0).contiguous())), kernel
