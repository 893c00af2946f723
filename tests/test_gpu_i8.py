"""vq_quant_i8, vq_gemm_i8 and vq_linear_i8 against their definition in 64 bits.

The integers and scales of the quantisation are held to equality.  In the
product the sum is exact; turning it into fp32, two multiplications and the
addition of the bias round once each, and the output once more:
|y - r| <= 4 * 2^-24 * (|r - b| + |b|) (1 + 2^-20) + u |r| + the output type's
half subnormal step, u its unit roundoff."""
import numpy as np
import pytest
import torch

from tests._util import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

SUBNORMAL = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def _vq():
    from bit_packed_index_b200 import vq
    return vq


def _name(t):
    return str(t).split(".")[-1]


def _quant64(x):
    """q and s of the definition (x: any 16-bit tensor), in numpy fp64."""
    x = x.double().cpu().numpy()
    top = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0])
    s = (top.astype(np.float32) / np.float32(127)).astype(np.float64)
    with np.errstate(all="ignore"):
        q = np.rint(x / np.where(s > 0, s, 1)[:, None])
    q = np.clip(np.where((s > 0)[:, None], q, 0), -127, 127)
    bad = ~np.isfinite(x).all(axis=1)
    q[bad], s[bad] = 0, np.nan
    return q, s


def _product64(q, s, w, ws, b):
    p = (q.double() @ w.double().t()) * s.double()[:, None] * ws.double()[None, :]
    return p, (0.0 if b is None else b.double()[None, :])


def _check(y, q, s, w, ws, b):
    p, bias = _product64(q, s, w, ws, b)
    r = p + bias
    bound = 4 * 2.0 ** -24 * (p.abs() + abs(bias)) * (1 + 2.0 ** -20) + UNIT_ROUNDOFF[_name(y.dtype)] * r.abs() \
        + SUBNORMAL[y.dtype]
    bad = (y.double() - r).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: {float((y.double() - r).abs().max()):.3e}"


def _weights(n, k, seed, bias):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.empty((n, -(-k // 16) * 16), dtype=torch.int8, device="cuda").fill_(77)[:, :k]
    w.copy_(torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8))
    ws = (0.5 + torch.rand(n, generator=g, device="cuda")) * 1e-3
    return w, ws, torch.randn(n, generator=g, device="cuda").half() if bias else None


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n", [(1, 1), (3, 7), (2, 8), (5, 64), (4, 513), (3, 1000), (2, 4104), (7, 16384),
                                 (2, 53248), (2, 65536), (2, 70001), (300, 96)])
def test_quant_matches_the_definition(dt, m, n):
    g = torch.Generator(device="cuda").manual_seed(m * 7919 + n)
    x = torch.randn((m, n), generator=g, device="cuda")
    x[:, :: max(1, n // 7)] *= 20
    x = x.to(dt)
    q, s = _vq().quant_i8(x)
    q64, s64 = _quant64(x)
    assert np.array_equal(s.double().cpu().numpy(), s64)
    assert np.array_equal(q.cpu().numpy().astype(np.float64), q64)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_quant_ties_and_tiny_rows(dt):
    """Rows whose quotients are exact halves (the largest value is 127 times a
    power of two), rows near the type's smallest values, zeros, and rows with
    an infinity or a NaN."""
    half = torch.arange(-127, 128, device="cuda").float() / 2
    rows = [torch.cat([half, torch.tensor([127.0], device="cuda")]) * 2.0 ** e for e in (-6, 0, 7)]
    tiny = torch.finfo(dt).smallest_normal * 2.0 ** (-7 if dt == torch.bfloat16 else -10)
    rows += [torch.arange(256, device="cuda").float() * tiny, torch.ones(256, device="cuda") * tiny]
    if dt == torch.bfloat16:
        rows += [torch.linspace(-1, 1, 256, device="cuda") * 2.0 ** e for e in (-130, -94, -93, -92, 127)]
    zero = torch.zeros(256, device="cuda")
    inf, nan = zero.clone() + 1, zero.clone() + 1
    inf[9], nan[200] = float("-inf"), float("nan")
    x = torch.stack(rows + [zero, -zero, inf, nan]).to(dt)
    q, s = _vq().quant_i8(x)
    q64, s64 = _quant64(x)
    assert np.array_equal(s.double().cpu().numpy(), s64, equal_nan=True)
    assert np.array_equal(q.cpu().numpy().astype(np.float64), q64)


def test_quant_strides_and_alignment():
    """Odd starts and strides of x and q, and columns of q past n left alone."""
    vq = _vq()
    base = torch.randn((9, 200), device="cuda").bfloat16()
    for x in (base[:, 1:100], base[:, 8:100], base[1:, 3:4], base[::2, :64]):
        for q0 in (0, 1, 8):
            out = torch.full((x.shape[0], 220), 99, dtype=torch.int8, device="cuda")
            view = out[:, q0: q0 + x.shape[1]]
            _, s = vq.quant_i8(x, out=view)
            q64, s64 = _quant64(x)
            assert np.array_equal(view.cpu().numpy().astype(np.float64), q64)
            assert np.array_equal(s.double().cpu().numpy(), s64)
            assert (out[:, :q0] == 99).all() and (out[:, q0 + x.shape[1]:] == 99).all()


SHAPES = [(1, 1, 1), (1, 128, 64), (1, 1024, 16384), (2, 7, 33), (3, 1000, 500), (8, 300, 4104), (16, 512, 512),
          (17, 130, 256), (24, 640, 1000), (33, 257, 129), (64, 1024, 2048), (65, 96, 8191), (128, 128, 128),
          (129, 260, 300), (200, 1030, 777), (256, 512, 640), (300, 2000, 1024), (513, 385, 260), (1000, 1000, 96),
          (2100, 1100, 144)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("od", [torch.bfloat16, torch.float32])
def test_product(m, n, k, od):
    vq = _vq()
    w, ws, b = _weights(n, k, m + n + k, (m + n) % 2 == 0)
    g = torch.Generator(device="cuda").manual_seed(k)
    q = torch.empty((m, -(-k // 16) * 16), dtype=torch.int8, device="cuda").fill_(-55)[:, :k]
    q.copy_(torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8))
    qs = torch.rand(m, generator=g, device="cuda") * 0.05
    layer = vq.Int8Layer(w, ws, b)
    ws_ = torch.zeros(max(256, vq.gemm_i8_workspace_size(layer, m)), dtype=torch.uint8, device="cuda")
    y = vq.gemm_i8(layer, q, qs, out_dtype=od, workspace=ws_)
    _check(y, q, qs, w, ws, b)
    assert int(ws_[:4].view(torch.int32)) == 0
    ws_[4:].fill_(0xAB)                                   # what a workspace holds does not matter
    assert torch.equal(y, vq.gemm_i8(layer, q, qs, out_dtype=od, workspace=ws_))


def test_product_extremes():
    """Every product of -128 and -128 at the longest row: the sum is 2^31 - 2^14
    short of nothing (131071 * 16384), and the largest negative one."""
    vq = _vq()
    k = 131071
    w = torch.full((130, 131072), 1, dtype=torch.int8, device="cuda")[:, :k]
    w.fill_(-128)
    w[1].fill_(127)
    q = torch.full((3, 131072), 1, dtype=torch.int8, device="cuda")[:, :k]
    q.fill_(-128)
    one = torch.ones(130, device="cuda")
    y = vq.gemm_i8(vq.Int8Layer(w, one), q, one[:3], out_dtype=torch.float32)
    assert float(y[0, 0]) == float(np.float32(131071 * 16384)) and float(y[2, 1]) == float(np.float32(-131071 * 16256))
    assert float(y[2, 129]) == float(y[0, 0])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m,n,k", [(1, 300, 515), (5, 128, 1024), (40, 500, 999), (260, 700, 333)])
def test_linear_is_quantisation_and_product(m, n, k, dt):
    vq = _vq()
    w, ws, b = _weights(n, k, 3 * m + n, True)
    layer = vq.Int8Layer(w, ws, b)
    x = torch.randn((m, k + 5), device="cuda").to(dt)[:, 2: 2 + k]          # rows not on 16 bytes
    y = vq.linear_i8(layer, x, out_dtype=torch.float16)
    q, s = vq.quant_i8(x)
    assert torch.equal(y, vq.gemm_i8(layer, q, s, out_dtype=torch.float16))
    q64, s64 = _quant64(x)
    _check(y, torch.from_numpy(q64).cuda(), torch.from_numpy(s64).cuda(), w, ws, b)


def test_layer_from_a_matrix():
    """Weights quantised by the same call: y stays within the two roundings of
    the exact product, (|x|_max sum|w| + |w|_max sum|x|) / 254 and their product."""
    vq = _vq()
    x, w = torch.randn((20, 600), device="cuda").half(), torch.randn((90, 600), device="cuda").half()
    y = vq.linear_i8(vq.Int8Layer.quantise(w), x, out_dtype=torch.float32).double()
    xd, wd = x.double(), w.double()
    hx, hw = xd.abs().amax(1) / 254, wd.abs().amax(1) / 254
    bound = hx[:, None] * wd.abs().sum(1) + hw[None, :] * xd.abs().sum(1)[:, None] + 600 * hx[:, None] * hw[None, :]
    assert ((y - xd @ wd.t()).abs() <= bound * (1 + 1e-6)).all()


def test_nonfinite_rows_stay_apart():
    vq = _vq()
    w, ws, _ = _weights(64, 96, 5, False)
    x = torch.randn((6, 96), device="cuda").bfloat16()
    clean = vq.linear_i8(vq.Int8Layer(w, ws), x, out_dtype=torch.float32)
    x[1, 3], x[4, 95] = float("inf"), float("nan")
    y = vq.linear_i8(vq.Int8Layer(w, ws), x, out_dtype=torch.float32)
    assert y[[1, 4]].isnan().all() and torch.equal(y[[0, 2, 3, 5]], clean[[0, 2, 3, 5]])


@pytest.mark.parametrize("m", [1, 40, 300])
def test_output_strides_empty_inputs_and_untouched_columns(m):
    vq = _vq()
    w, ws, b = _weights(200, 64, m, True)
    layer = vq.Int8Layer(w, ws, b)
    x = torch.randn((m, 64), device="cuda").half()
    full = torch.full((m, 211), 7.0, dtype=torch.bfloat16, device="cuda")
    vq.linear_i8(layer, x, out=full[:, 3:203])
    assert torch.equal(full[:, 3:203], vq.linear_i8(layer, x)) and (full[:, :3] == 7).all() and (full[:, 203:] == 7).all()
    assert vq.linear_i8(layer, x[:0]).shape == (0, 200)
    empty = vq.Int8Layer(torch.empty((200, 0), dtype=torch.int8, device="cuda"), ws, b)
    y = vq.linear_i8(empty, x[:, :0], out_dtype=torch.float16)
    assert torch.equal(y, b.expand(m, 200))


def test_streams_and_graphs():
    """A captured call replays on new inputs; two streams with their own
    workspaces do not disturb each other."""
    vq = _vq()
    w, ws, b = _weights(1500, 700, 9, True)
    layer = vq.Int8Layer(w, ws, b)
    xs = [torch.randn((m, 700), device="cuda").bfloat16() for m in (1, 70)]
    for x in xs:
        work = torch.zeros(vq.linear_i8_workspace_size(layer, x.shape[0]), dtype=torch.uint8, device="cuda")
        y = torch.empty((x.shape[0], 1500), dtype=torch.bfloat16, device="cuda")
        vq.linear_i8(layer, x, out=y, workspace=work)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            vq.linear_i8(layer, x, out=y, workspace=work)
        x.copy_(torch.randn_like(x))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, vq.linear_i8(layer, x))
        del g
    want = [vq.linear_i8(layer, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, (st, x) in enumerate(zip(streams, xs)):
            with torch.cuda.stream(st):
                got[i] = vq.linear_i8(layer, x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("m,n,k", [(3, 1024, 8192), (40, 300, 512), (200, 1000, 3000)])
def test_device_waits_give_up_with_a_status(monkeypatch, m, n, k):
    """A wait whose budget is zero gives up: the call ends, the status word
    says so and stays set until it is cleared, and the next call is right."""
    vq = _vq()
    w, ws, b = _weights(n, k, 2, True)
    layer = vq.Int8Layer(w, ws, b)
    q = torch.randint(-127, 128, (m, -(-k // 16) * 16), device="cuda", dtype=torch.int8)[:, :k]
    one = torch.ones(m, device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("VQ_WAIT_BUDGET", "0")
    vq.gemm_i8(layer, q, one, workspace=work)
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32)) == vq.VQ_ERR_TIMEOUT
    monkeypatch.delenv("VQ_WAIT_BUDGET")
    y = vq.gemm_i8(layer, q, one, out_dtype=torch.float32, workspace=work)
    _check(y, q, one, w, ws, b)
    assert int(work[:4].view(torch.int32)) == vq.VQ_ERR_TIMEOUT


def test_binding_checks():
    vq = _vq()
    w, ws, b = _weights(64, 48, 1, True)
    layer = vq.Int8Layer(w, ws, b)
    x = torch.randn((4, 48), device="cuda").bfloat16()
    for bad in (x.float(), x[:, :40], x[0], x.t()[:48, :4].contiguous().t()[:, :48], x.cpu()):
        with pytest.raises(ValueError):
            vq.linear_i8(layer, bad)
    with pytest.raises(ValueError):
        vq.linear_i8(layer, x, out=torch.empty((4, 63), device="cuda"))
    with pytest.raises(ValueError):
        vq.linear_i8(layer, x, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        vq.Int8Layer(w, ws.double())
    with pytest.raises(ValueError):
        vq.Int8Layer(w, ws, b.float())
    with pytest.raises(vq.VQError):                              # rows not on 16 bytes
        vq.gemm_i8(layer, torch.zeros((4, 50), dtype=torch.int8, device="cuda")[:, :48], torch.ones(4, device="cuda"))
    with pytest.raises(vq.VQError):
        vq.linear_i8(layer, x, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
