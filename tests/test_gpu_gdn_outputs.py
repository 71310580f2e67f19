"""Every element of the one-decay rule's bf16 outputs, not their 2-norm alone.

The chunked prefill forms bf16 outputs from the operands of its fp32 ones and
rounds once, so
  - they are the fp32 outputs' bits after that rounding, and
  - each lies within one bf16 step of the rounded 64-bit value plus 1e-3 of the
    outputs' RMS (the rule the per-key-dim kernels' outputs are held to).  In
    front of the rounding an output is off by about 2^-18 of the RMS, on nearly
    equal keys by 2^-16: the first allows the other side of a rounding border,
    the second outputs near zero, whose steps are smaller than that.
"""
import numpy as np
import pytest
import torch

from tests import parity
from tests.test_gpu_gdn import Case

pytestmark = pytest.mark.gpu

SHAPES = [  # lens, Hk, Hv, dk, dv
    ([512], 1, 1, 128, 128),
    ([300, 1, 85], 2, 4, 64, 128),
    ([200, 64], 2, 2, 32, 64),
    ([130, 70], 2, 6, 128, 32),
    ([1100, 64, 65, 900], 4, 16, 128, 128),  # chains beside prep
    ([2600], 4, 8, 64, 64),
]


def _case(out, shape, correlated):
    lens, Hk, Hv, dk, dv = shape
    kw = dict(gate=-10.0, beta=3.0) if correlated else {}
    c = Case(lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, out=out, seed=13 + dk + dv, **kw)
    if correlated:  # nearly equal keys: I + A is far from the identity, and outputs are small differences
        c.k[:] = c.k[:1] + 0.05 * c.k
    return c


@pytest.mark.parametrize("correlated", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bf16_outputs_are_the_fp32_ones_rounded(cuda_lib, shape, correlated):
    narrow, wide = _case("bf16", shape, correlated), _case("f32", shape, correlated)
    for c in (narrow, wide):
        c.prefill(cuda_lib)
        assert int(c.status.item()) == 0 and c.g_out.intact() and c.g_state.intact()
    assert torch.equal(narrow.g_out.tensor, wide.g_out.tensor.to(torch.bfloat16))
    assert torch.equal(narrow.g_state.tensor, wide.g_state.tensor)


@pytest.mark.parametrize("correlated", [False, True])
@pytest.mark.parametrize("shape", SHAPES[:5], ids=str)
def test_every_bf16_output(cuda_lib, shape, correlated):
    c = _case("bf16", shape, correlated)
    c.prefill(cuda_lib)
    out, _ = c.want()
    got = c.g_out.tensor[:c.T].double().cpu().numpy()
    assert np.isfinite(got).all()
    parity.assert_bf16_within_one_ulp(got, out)
