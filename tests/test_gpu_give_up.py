"""Products whose waits give up (VQ_WAIT_BUDGET): whatever a block had in flight
has landed before the next call's blocks take its place."""
import pytest
import torch

import synth
from synth import LayerSpec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget", ["0", "1500", "6000"])
@pytest.mark.parametrize("call,books,kin,rows", [
    ("fused", (16,), 128, 300), ("fused", (12, 8), 1024, 300), ("staged", (16,), 128, 300), ("staged", (12, 8), 2048, 300),
    ("gemv", (16,), 128, 8), ("gemv", (16,), 16000, 8), ("gemv", (12, 8), 128, 8), ("gemv", (12, 8), 8000, 8)])
def test_calls_after_ones_that_gave_up(monkeypatch, call, books, kin, rows, budget):
    """Waits run out early (with every load of a short row already under way), in
    the middle or not at all; a call launched right behind is right every time."""
    from bit_packed_index_b200 import vq
    layer = vq.Layer.from_synth(synth.make_layer(LayerSpec(2000, kin, 8, books, (0.02, 0.005)[: len(books)]), seed=kin))
    if call != "gemv":
        monkeypatch.setenv("VQ_GEMM_MODE", call)
    x = torch.randn((rows, kin), device="cuda").bfloat16()
    run = vq.gemv if call == "gemv" else vq.gemm
    want = run(layer, x, out_dtype=torch.float32)
    plain = x.float() @ vq.dequant(layer).float().t()
    # the weights round to fp16 twice on either side (two books' sum, W_hat): at most 4 x 2^-11 of the magnitudes
    size = x.float().abs() @ vq.dequant(layer).float().abs().t()
    assert ((want - plain).abs() <= 2.0 ** -9 * size + 1e-6).all()
    spoilt, ys = torch.empty_like(want), []
    for _ in range(20):
        monkeypatch.setenv("VQ_WAIT_BUDGET", budget)
        run(layer, x, out=spoilt)
        monkeypatch.delenv("VQ_WAIT_BUDGET")
        ys.append(run(layer, x, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)
