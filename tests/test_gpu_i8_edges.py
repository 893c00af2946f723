"""8-bit layers at their edges.  Bounds and helpers: tests/test_gpu_i8.py."""
import pytest
import torch

from tests.test_gpu_i8 import _check, _vq, _weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget", ["0", "1500", "6000"])
@pytest.mark.parametrize("m,n,k", [(40, 300, 512), (3, 1024, 8192), (1, 5000, 128), (200, 1000, 300), (600, 3000, 2000)])
def test_calls_after_ones_that_gave_up(monkeypatch, m, n, k, budget):
    """Waits run out early, in the middle or not at all; whatever a block had in
    flight has landed before the next call's blocks take its place: that call,
    launched right behind, is right every time."""
    vq = _vq()
    w, ws, b = _weights(n, k, 2, True)
    layer = vq.Int8Layer(w, ws, b)
    q = torch.randint(-127, 128, (m, -(-k // 16) * 16), device="cuda", dtype=torch.int8)[:, :k]
    one = torch.ones(m, device="cuda")
    want = vq.gemm_i8(layer, q, one, out_dtype=torch.float32)
    _check(want, q, one, w, ws, b)
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    spoilt, ys = torch.empty_like(want), []
    for _ in range(20):
        monkeypatch.setenv("VQ_WAIT_BUDGET", budget)
        vq.gemm_i8(layer, q, one, out=spoilt, workspace=work)
        monkeypatch.delenv("VQ_WAIT_BUDGET")
        ys.append(vq.gemm_i8(layer, q, one, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32)) in (vq.VQ_OK, vq.VQ_ERR_TIMEOUT)
    assert all(torch.equal(y, want) for y in ys)
