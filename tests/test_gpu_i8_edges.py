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


@pytest.mark.parametrize("m,n,k", [(1, 1024, 16384), (3, 1000, 4200), (40, 700, 2049)])
def test_rows_in_turn_through_a_product_split_along_k(m, n, k):
    """linear_i8's product starts under the quantisation of its own rows: with
    rows of very different sizes in turn, each call takes its own scales."""
    vq = _vq()
    w, ws, b = _weights(n, k, 6, False)
    layer = vq.Int8Layer(w, ws, b)
    xs = [(torch.randn((m, k), device="cuda") * s).bfloat16() for s in (1.0, 1e-6, 1e6)]
    want = []
    for x in xs:
        q, s = vq.quant_i8(x)
        want.append(vq.gemm_i8(layer, q, s, out_dtype=torch.float32))
    work = torch.zeros(vq.linear_i8_workspace_size(layer, m), dtype=torch.uint8, device="cuda")
    got = [vq.linear_i8(layer, xs[i % 3], out_dtype=torch.float32, workspace=work) for i in range(60)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i % 3]) for i in range(60))


@pytest.mark.parametrize("steps", [8, 9, 15, 16, 17, 31, 32, 33, 49, 57, 64])
@pytest.mark.parametrize("m", [1, 33])
def test_runs_of_k_of_every_length(m, steps):
    """Steps of 128 values that two, four and eight CTAs share, evenly or not."""
    vq = _vq()
    k = 128 * steps - 5
    w, ws, b = _weights(300, k, steps, True)
    q = torch.empty((m, 128 * steps), dtype=torch.int8, device="cuda").fill_(-55)[:, :k]
    q.copy_(torch.randint(-128, 128, (m, k), device="cuda", dtype=torch.int8))
    s = torch.rand(m, device="cuda")
    _check(vq.gemm_i8(vq.Int8Layer(w, ws, b), q, s, out_dtype=torch.float32), q, s, w, ws, b)


def test_quant_of_the_longest_row():
    """2^31 - 1 values: positions pass 31 bits.  The row's largest is 127 times a
    power of two, so the quotients of the sixteen other values are exact."""
    vq = _vq()
    n = 2 ** 31 - 1
    x = torch.zeros((1, n), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 7, 1023, 65536, 2 ** 20 + 3, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1100, 2 ** 31 - 1024, 2 ** 31 - 1023,
                       2 ** 31 - 1000, 2 ** 31 - 9, 2 ** 31 - 8, 2 ** 31 - 3], device="cuda")
    x[0, at] = torch.arange(1, 16, device="cuda").bfloat16() / 4
    x[0, -1] = -127 / 4
    q, s = vq.quant_i8(x)
    assert float(s) == 0.25 and q.shape == (1, n)
    assert q[0, at].tolist() == list(range(1, 16)) and int(q[0, -1]) == -127
    q[0, at], q[0, -1] = 0, 0
    assert not any(bool(p.any()) for p in q[0].split(1 << 28))


def test_layers_that_no_call_accepts():
    """Refused when the layer is made: rows that do not start on 16 bytes, rows too long."""
    vq = _vq()
    base, ws = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    vq.Int8Layer(base[:, 16:48], ws)
    for w in (base[:, 8:48], torch.zeros((4, 50), dtype=torch.int8, device="cuda"),
              torch.zeros((4, 131072), dtype=torch.int8, device="cuda")):
        with pytest.raises(ValueError):
            vq.Int8Layer(w, ws)
    vq.Int8Layer(base.new_zeros((4, 0)), ws)                     # without inputs nothing is read
    vq.Int8Layer(base.new_zeros((1, 50)), ws[:1])                # one row has no stride
