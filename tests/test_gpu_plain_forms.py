"""The plain torch forms that perf/operators.py measures the kernels against
follow the same definitions as the kernels."""
import pytest
import torch

from perf import operators

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_plain_8_bit_form_quantises_as_the_package(dt):
    """With the identity as the weights and scales of one, the product is q s,
    rounded once to fp32 on both sides: equality."""
    from bit_packed_index_b200 import vq
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((20000, 64), generator=g, device="cuda").to(dt)
    q, s = vq.quant_i8(x)
    eye, one = torch.eye(64, dtype=torch.int8, device="cuda"), torch.ones(64, device="cuda")
    assert torch.equal(operators._linear_plain(x, eye, one, None, torch.float32), q.float() * s[:, None])
