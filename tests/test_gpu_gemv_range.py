"""vq_gemv on rows whose sum passes fp32's range while their products do not."""
import pytest
import torch

import synth
from synth import LayerSpec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 2, 5, 8, 16])
@pytest.mark.parametrize("layout", ["rows", "tile4"])
@pytest.mark.parametrize("books,d", [((16,), 8), ((12, 8), 8), ((8, 8), 8), ((12, 4), 6), ((10,), 5), ((16, 8), 8)])
def test_finite_rows_have_finite_products(books, d, layout, batch):
    """Without a bias, rows of 1e35 give 1e35 times what rows of ones give (a
    power of two apart from it: 2^116): sum x = 2^128 is infinite in fp32."""
    from bit_packed_index_b200 import vq
    spec = LayerSpec(300, 4096 // d * d, d, books, (0.02, 0.005)[: len(books)], (0.5, 1.5), None)
    layer = vq.Layer.from_synth(synth.make_layer(spec, seed=batch), layout=layout)
    one = torch.ones((batch, spec.in_features), device="cuda").bfloat16()
    one[:, ::3] = 1.5                             # sum x = 1.17 * Kin
    y = vq.gemv(layer, one, out_dtype=torch.float32)
    z = vq.gemv(layer, one * 2.0 ** 116, out_dtype=torch.float32)
    assert torch.equal(z * 2.0 ** -116, y)
