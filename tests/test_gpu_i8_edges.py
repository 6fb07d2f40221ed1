"""The 8-bit linear path where its arithmetic, its sizes and its streams come to their ends, against 64 bits."""
import pytest
import torch

import diffusion_transformer_text_block_b200 as moss
from tests.test_gpu_i8 import check_rows_of, no_device_error, randn, swiglu_reference  # noqa: F401 (a fixture among them)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ rows to 8 bits
GATES = [-86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -93.0, -104.0, -120.0, -150.0, -174.0]


@pytest.mark.parametrize("dim", [16, 1024, 8192])
def test_swiglu_gates_far_below_zero(dim):
    """Rows of one gate each, for which e^-g leaves FP32's range, times u from 1e37 to 3e38: SiLU(g) u is a number.
    __expf(g/2) twice is within 2 (2 + 1.173 |g| / 2) ulp (2 u each), the three products add 3 u: below the
    reference's bound; 2^-140 is far above what a subnormal intermediate could add and far below every h."""
    gu = torch.empty(len(GATES), 2 * dim, device="cuda", dtype=torch.bfloat16)
    gu[:, :dim] = torch.tensor(GATES, device="cuda")[:, None]
    gu[:, dim:] = (1e37 * 30 ** torch.rand(len(GATES), dim, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
                   * torch.sign(randn(2, len(GATES), dim))).bfloat16()
    q, scale = moss.op_swiglu_i8(gu)
    h, err = swiglu_reference(gu)
    assert (h.abs().amax(dim=1) > 2.0 ** -126).all()
    check_rows_of(q, scale, h, err + 2.0 ** -140)
    assert (q.abs().amax(dim=1) == 127).all()


def test_swiglu_far_gates_beside_others():
    """A far gate changes none of its neighbours, and gives a tiny value or 0 beside them as it should."""
    gu = randn(3, 6, 2 * 704, scale=2.0).bfloat16()
    gu[:, 5] = 0
    want = moss.op_swiglu_i8(gu)
    gu[:, 5], gu[:, 704 + 5] = -88.0, 1.0
    q, scale = moss.op_swiglu_i8(gu)
    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])
    gu[0, 9], gu[0, 704 + 9] = float("-inf"), 1.0
    gu[1, 9], gu[1, 704 + 9] = -200.0, float("inf")
    gu[2, 9], gu[2, 704 + 9] = -1e30, 3e38
    q, scale = moss.op_swiglu_i8(gu)
    assert torch.isnan(scale[:2]).all() and (q[:2] == 0).all()
    assert torch.isfinite(scale[2:]).all() and q[2, 9] == 0
