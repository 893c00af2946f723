"""vq_group_rows, vq_gemm_experts and vq_combine_rows against plain
implementations in 64 bits.

Bound of the product for grouped row r and output o, A = s sum_k |x_k (c1 +
c2)_k| + |t| sum_k |x_k|:
  * the fp32 sums over Kin terms (whatever their order or splitting), the
    handful of operations of the epilogue and up to 64 joined parts:
    (Kin + 128) 2^-23 A -- twice the unit roundoff per addition, since the
    tensor cores may truncate;
  * two books: c1 + c2 rounded to fp16, half a step of 2^-11 |c1 + c2| or
    2^-25 where the sum is subnormal, times |x| s;
  * the output's rounding, u |r| and half a subnormal step.
x itself is exact as an fp16 multiple of a power of two (values within 2^-28
of the row's largest; these rows hold no smaller non-zero ones that count:
below it they lose at most 2^-40 of the largest, counted as 2^-38 max|x|
sum|c|)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from synth import LayerSpec
from tests._util import UNIT_ROUNDOFF

pytestmark = pytest.mark.gpu

SUBNORMAL = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def _vq():
    from bit_packed_index_b200 import vq
    return vq


# ---- grouping ----------------------------------------------------------------
def _group_plain(ids, e):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < e)
    order = np.argsort(np.where(ok, flat, e), kind="stable")
    count = np.bincount(flat[ok], minlength=e)
    offsets = np.concatenate([[0], np.cumsum(count)])
    rows = np.full(flat.size, -1)
    pos = np.full(flat.size, -1)
    n = int(offsets[-1])
    rows[:n] = order[:n] // ids.shape[1]
    pos[order[:n]] = np.arange(n)
    return offsets, rows, pos.reshape(ids.shape)


@pytest.mark.parametrize("t,k,e", [(0, 1, 1), (1, 1, 1), (1, 8, 8), (5, 2, 3), (16, 8, 64), (33, 3, 100), (257, 1, 7),
                                   (1000, 2, 1024), (1024, 2, 16), (1025, 2, 16), (3000, 5, 33), (8191, 8, 128),
                                   (40000, 4, 256), (50, 64, 1000)])
def test_group_rows(t, k, e):
    rng = np.random.default_rng(t + k)
    full = rng.integers(-2, e + 2, size=(t, k + 3)).astype(np.int32)       # some ids name no expert
    ids = torch.from_numpy(full).cuda()[:, 1: 1 + k]
    out = _vq().group_rows(ids, e)
    again = _vq().group_rows(ids, e)
    for got, twice, want in zip(out, again, _group_plain(full[:, 1: 1 + k], e)):
        assert np.array_equal(got.cpu().numpy(), want) and torch.equal(got, twice)


@pytest.mark.parametrize("fill", [0, 6, -1, 7, 2 ** 31 - 1, -2 ** 31])
def test_group_rows_one_expert_or_none(fill):
    ids = torch.full((700, 3), fill, dtype=torch.int32, device="cuda")
    for got, want in zip(_vq().group_rows(ids, 7), _group_plain(ids.cpu().numpy(), 7)):
        assert np.array_equal(got.cpu().numpy(), want)


# ---- products ------------------------------------------------------------------
def _experts(spec, e, layout, seed, shared=False):
    vq = _vq()
    data = [synth.make_layer(spec, seed=seed + i, pad_garbage=True) for i in range(e)]
    if shared:
        for d in data[1:]:
            d.codebooks = data[0].codebooks
    ex = vq.Experts.from_layers([vq.Layer.from_synth(d, layout=layout) for d in data])
    if shared:
        ex = vq.Experts(ex.out_features, ex.in_features, ex.vec_dim, ex.log2k, ex.idx, [c[:1] for c in ex.codebooks],
                        ex.scale, ex.bias, layout, ex.out_bias)
    return data, ex


def _weights64(data):
    """C1[i1] + C2[i2], s, t, b of one expert in fp64."""
    s = data.spec
    c = 0.0
    for words, book, b in zip(data.idx_words, data.codebooks, s.log2k):
        c = c + oracle.f16_to_f32(book).astype(np.float64).reshape(1 << b, s.d)[oracle.unpack(words, b, s.nvec)]
    vec = lambda v, none: np.full(s.out_features, none) if v is None else oracle.f16_to_f32(v).astype(np.float64)
    return (c.reshape(s.out_features, -1)[:, : s.in_features], vec(data.scale, 1.0), vec(data.bias, 0.0),
            vec(data.out_bias, 0.0))


def _check(y, x, data, offsets, rows, fill):
    """y against the definition, rows behind the last group against `fill`."""
    xd, kin = x.double(), x.shape[1]
    for e, d in enumerate(data):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r0 == r1:
            continue
        c, s, t, b = (torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in _weights64(d))
        if rows is None:
            xr = xd[r0:r1]
        else:
            at = rows[r0:r1].long()
            ok = (at >= 0) & (at < x.shape[0])
            xr = torch.where(ok[:, None], xd[at.clamp(0, x.shape[0] - 1)], torch.zeros_like(xd[:1]))
        ref = (xr @ c.t()) * s + xr.sum(1)[:, None] * t + b
        xa = xr.abs()
        a = (xa @ c.abs().t()) * s + xa.sum(1)[:, None] * t.abs()
        bound = (kin + 128) * 2.0 ** -23 * (a + b.abs()) + 2.0 ** -38 * xa.amax(1)[:, None] * c.abs().sum(1) * s
        if d.spec.n_books == 2:
            step = torch.maximum(c.abs() * 2.0 ** -11, torch.full_like(c, 2.0 ** -25))
            bound = bound + (xa @ step.t()) * s
        bound = bound + UNIT_ROUNDOFF[str(y.dtype).split(".")[-1]] * ref.abs() + SUBNORMAL[y.dtype]
        err = (y[r0:r1].double() - ref).abs()
        bad = ~(err <= bound)
        assert not bad.any(), f"expert {e}: {int(bad.sum())} of {bad.numel()}, worst {float((err / bound).max()):.3g} bounds"
    last = int(offsets[-1])
    assert (y[last:] == fill).all()


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _run(ex, x, offsets, rows=None, od=torch.float32, m=None, fill=-3.0):
    vq = _vq()
    m = (rows.shape[0] if rows is not None else x.shape[0]) if m is None else m
    y = torch.full((m, ex.out_features), fill, dtype=od, device="cuda")
    ws = torch.full((max(256, vq.gemm_experts_workspace_size(ex, m)),), 0x7F, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    vq.gemm_experts(ex, x, offsets, rows=rows, out=y, workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    return y


SPECS = [
    LayerSpec(256, 64, 8, (16,), (0.02,)),
    LayerSpec(300, 1000, 8, (12, 8), (0.02, 0.005), out_bias_std=1.0),
    LayerSpec(129, 800, 8, (16, 8), (0.02, 0.005)),
    LayerSpec(600, 520, 8, (16,), (0.02,), None, None),
    LayerSpec(257, 6 * 100 + 4, 6, (12, 4), (0.02, 0.005)),
    LayerSpec(100, 5 * 40 + 3, 5, (7, 3), (0.02, 0.005), out_bias_std=0.5),
    LayerSpec(64, 512, 8, (8, 8), (0.02, 0.005), (0.5, 1.5), None),
    LayerSpec(1, 8, 8, (4,), (0.02,)),
    LayerSpec(130, 3 * 64, 4, (9, 2), (0.02, 0.005), None, 1e-3),
    LayerSpec(70, 16 * 9 + 5, 16, (10, 6), (0.02, 0.005)),
    LayerSpec(200, 12 * 30, 12, (11,), (0.02,)),
    LayerSpec(140, 77, 1, (5, 1), (0.02, 0.005)),
    LayerSpec(150, 700, 7, (13, 13), (0.02, 0.005)),
    LayerSpec(90, 640, 8, (12, 12), (0.02, 0.02)),
    LayerSpec(90, 333, 3, (16, 16), (0.02, 0.02)),
]
COUNTS = [[1], [0, 3, 0], [5, 0, 17, 1], [16, 15], [40, 0, 33], [2, 130, 7], [300, 1, 64, 0]]


@pytest.mark.parametrize("layout", ["rows", "tile4"])
@pytest.mark.parametrize("i", range(len(SPECS)))
def test_products_of_every_kind_of_layer(i, layout):
    spec = SPECS[i]
    for counts in COUNTS[i % 3::3] + [[33, 2]]:
        data, ex = _experts(spec, len(counts), layout, 40 * i)
        offsets = _offsets(counts)
        m = sum(counts) + 5
        x = torch.randn((m, spec.in_features), device="cuda") * 2
        for dt, od in ((torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16)):
            y = _run(ex, x.to(dt), offsets, od=od)
            _check(y, x.to(dt), data, offsets, None, -3.0)


@pytest.mark.parametrize("layout,books", [("tile4", (12, 8)), ("rows", (16,)), ("rows", (12, 4))])
@pytest.mark.parametrize("tokens", [1, 7, 200, 1300])
def test_gathered_rows_and_padding(layout, books, tokens):
    """Rows gathered from the tokens, some of them named by several experts, some by none."""
    vq = _vq()
    spec = LayerSpec(390, 1040, 6 if books == (12, 4) else 8, books, (0.02, 0.005)[: len(books)])
    data, ex = _experts(spec, 6, layout, 7, shared=tokens == 7)
    ids = torch.randint(-1, 6, (tokens, 3), device="cuda", dtype=torch.int32)
    offsets, rows, _ = vq.group_rows(ids, 6)
    x = torch.randn((tokens, 1040), device="cuda").bfloat16()
    x[:, 5] *= 3000
    y = _run(ex, x, offsets, rows=rows)
    _check(y, x, data, offsets, rows, -3.0)
    assert torch.equal(y, _run(ex, x, offsets, rows=rows))               # bit for bit


@pytest.mark.parametrize("counts", [[0, 0, 0], [600, 0, 700], [1024], [512, 513, 1]])
def test_long_and_empty_groups(counts):
    spec = LayerSpec(260, 200, 8, (12, 8), (0.02, 0.005))
    data, ex = _experts(spec, len(counts), "tile4", 3)
    offsets = _offsets(counts)
    x = torch.randn((sum(counts) + 1, 200), device="cuda").half()
    _check(_run(ex, x, offsets), x, data, offsets, None, -3.0)


@pytest.mark.parametrize("books,layout", [((12, 8), "rows"), ((16,), "tile4"), ((16, 8), "rows"), ((9, 9), "tile4")])
@pytest.mark.parametrize("counts", [[1, 2000, 0, 7, 130, 0, 385, 193], [600, 520]])
def test_uneven_groups(books, layout, counts):
    """One expert with most of the rows: token tiles of one and two halves, and
    shares that end inside tiles, in both places that W's tiles can lie."""
    spec = LayerSpec(400, 328, 8, books, (0.02, 0.005)[: len(books)])
    data, ex = _experts(spec, len(counts), layout, 13)
    x = torch.randn((sum(counts) + 3, 328), device="cuda").bfloat16()
    y = _run(ex, x, _offsets(counts), od=torch.bfloat16)
    _check(y, x, data, _offsets(counts), None, -3.0)


def test_many_experts_many_rows():
    """1024 experts, the most, each with its own small books."""
    spec = LayerSpec(130, 48, 8, (5, 3), (0.02, 0.005))
    data, ex = _experts(spec, 1024, "tile4", 100)
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 6, size=1024)
    counts[500] = 100
    x = torch.randn((int(counts.sum()), 48), device="cuda").half()
    _check(_run(ex, x, _offsets(counts)), x, data, _offsets(counts), None, -3.0)


def test_one_workspace_for_two_graphs():
    """Two captured calls that share a workspace, replayed one after the other."""
    vq = _vq()
    data, ex = _experts(LayerSpec(700, 500, 8, (12, 8), (0.02, 0.005)), 3, "tile4", 41)
    xs = [torch.randn((m, 500), device="cuda").bfloat16() for m in (5, 300)]
    offs = [_offsets([2, 0, 3]), _offsets([100, 150, 50])]
    ys = [torch.empty((x.shape[0], 700), dtype=torch.float32, device="cuda") for x in xs]
    work = torch.zeros(max(vq.gemm_experts_workspace_size(ex, x.shape[0]) for x in xs), dtype=torch.uint8, device="cuda")
    graphs = []
    for x, o, y in zip(xs, offs, ys):
        vq.gemm_experts(ex, x, o, out=y, workspace=work)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            vq.gemm_experts(ex, x, o, out=y, workspace=work)
    for _ in range(3):
        for x in xs:
            x.copy_(torch.randn_like(x))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, o, y in zip(xs, offs, ys):
            _check(y, x, data, o, None, -3.0)


def test_many_experts_few_rows():
    spec = LayerSpec(128, 96, 8, (6, 4), (0.02, 0.005))
    data, ex = _experts(spec, 200, "rows", 11)
    counts = np.zeros(200, int)
    counts[[0, 3, 77, 78, 199]] = [1, 2, 1, 40, 3]
    x = torch.randn((50, 96), device="cuda").bfloat16()
    _check(_run(ex, x, _offsets(counts)), x, data, _offsets(counts), None, -3.0)


def test_rows_of_any_size_and_non_finite_rows():
    """Rows from 1e-30 to 1e30 (bf16) are scaled one by one; a row with an
    infinity or a NaN is non-finite and leaves the others as they were."""
    spec = LayerSpec(130, 264, 8, (12, 8), (0.02, 0.005))
    data, ex = _experts(spec, 2, "rows", 5)
    x = torch.randn((40, 264), device="cuda") * torch.logspace(-30, 30, 40, device="cuda")[:, None]
    x[7] = 0
    x = x.bfloat16()
    offsets = _offsets([17, 23])
    y = _run(ex, x, offsets)
    _check(y, x, data, offsets, None, -3.0)
    x[3, 9], x[20, 263] = float("inf"), float("nan")
    z = _run(ex, x, offsets)
    keep = [i for i in range(40) if i not in (3, 20)]
    assert torch.equal(z[keep], y[keep]) and not z[3].isfinite().any() and not z[20].isfinite().any()


def test_offsets_and_rows_out_of_range():
    """Offsets past m and descending ones are clamped, row numbers outside x
    count as zeros: nothing outside the buffers is read or written."""
    spec = LayerSpec(64, 72, 8, (8,), (0.02,), out_bias_std=1.0)
    data, ex = _experts(spec, 4, "rows", 9)
    x = torch.randn((20, 72), device="cuda").bfloat16()
    big = torch.tensor([0, 5, 1000, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    y = _run(ex, x, big)
    _check(y, x, data, torch.tensor([0, 5, 20, 20, 20]), None, -3.0)
    down = torch.tensor([-9, 6, 3, 12, 12], dtype=torch.int32, device="cuda")
    y = _run(ex, x, down)
    _check(y, x, data, torch.tensor([0, 6, 6, 12, 12]), None, -3.0)
    rows = torch.tensor([3, -1, 19, 20, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    offsets = _offsets([2, 0, 4, 1])
    _check(_run(ex, x, offsets, rows=rows), x, data, offsets, rows, -3.0)


def test_strided_input_and_output():
    spec = LayerSpec(96, 100, 6, (12, 4), (0.02, 0.005))
    data, ex = _experts(spec, 3, "tile4", 2)
    x = torch.randn((30, 131), device="cuda").half()[:, 3:103]
    offsets = _offsets([9, 20, 1])
    full = torch.full((30, 133), 5.0, dtype=torch.float16, device="cuda")
    _vq().gemm_experts(ex, x, offsets, out=full[:, 7:103])
    _check(full[:, 7:103], x, data, offsets, None, 5.0)
    assert (full[:, :7] == 5).all() and (full[:, 103:] == 5).all()


def test_empty_layers():
    vq = _vq()
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    book = torch.zeros((2, 16, 8), dtype=torch.float16, device="cuda")
    ob = torch.randn((2, 5), device="cuda").half()
    ex = vq.Experts(5, 0, 8, [4], [z(2, 5, 0)], [book], out_bias=ob)
    y = _run(ex, torch.empty((6, 0), dtype=torch.float16, device="cuda"), _offsets([2, 3]), od=torch.float16)
    assert torch.equal(y[:2], ob[:1].expand(2, 5)) and torch.equal(y[2:5], ob[1:].expand(3, 5)) and (y[5:] == -3).all()
    ex = vq.Experts(0, 64, 8, [4], [z(2, 0, 4)], [book])
    assert _run(ex, torch.empty((6, 64), dtype=torch.float16, device="cuda"), _offsets([2, 3])).shape == (6, 0)


# ---- combining ------------------------------------------------------------------
@pytest.mark.parametrize("t,k,n", [(1, 1, 1), (3, 2, 7), (5, 8, 64), (33, 4, 2050), (7, 13, 100), (300, 8, 1024)])
@pytest.mark.parametrize("zt,yt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                   (torch.float32, torch.float16)])
def test_combine(t, k, n, zt, yt):
    """k products and sums in fp32: |y - r| <= (k + 1) 2^-24 sum |w z| + u |r| + a subnormal's half step."""
    g = torch.Generator(device="cuda").manual_seed(t * k + n)
    z = torch.randn((2 * t + 1, n), generator=g, device="cuda").to(zt)
    pos = torch.randint(-1, 2 * t + 3, (t, k), generator=g, device="cuda", dtype=torch.int32)
    w = torch.rand((t, k + 1), generator=g, device="cuda")[:, :k]
    ok = (pos >= 0) & (pos < z.shape[0])
    v = z.double()[pos.clamp(0, z.shape[0] - 1).long()] * (w.double() * ok)[:, :, None]
    y = _vq().combine_rows(z, pos, w, out_dtype=yt)
    ref = v.sum(1)
    bound = (k + 1) * 2.0 ** -24 * v.abs().sum(1) + UNIT_ROUNDOFF[str(yt).split(".")[-1]] * ref.abs() + SUBNORMAL[yt]
    assert ((y.double() - ref).abs() <= bound).all()


def test_combine_skips_what_is_not_there():
    """Tokens without picks give zeros, whatever their weights and z hold; odd starts and strides."""
    z = torch.full((4, 40), float("nan"), device="cuda").half()
    z[2] = 2
    pos = torch.tensor([[-1, -1], [2, -7], [4, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan"), 1.0], [0.5, float("inf")], [1.0, 1.0]], device="cuda")
    full = torch.full((3, 50), 9.0, device="cuda")
    _vq().combine_rows(z[:, 1:34], pos, w, out=full[:, 5:38])
    assert (full[0, 5:38] == 0).all() and (full[1, 5:38] == 1).all() and (full[2, 5:38] == 0).all()
    assert (full[:, :5] == 9).all() and (full[:, 38:] == 9).all()
    assert _vq().combine_rows(z[:0], pos, w).eq(0).all()
    assert _vq().combine_rows(z, pos[:0], w[:0]).shape == (0, 40)


# ---- together ---------------------------------------------------------------------
def _block(vq, proj, gate_up, down, x, router):
    """Attention's output projection in 8-bit integers, then a mixture of experts, as a model runs them."""
    h = vq.linear_i8(proj, x)
    score, ids = (h.float() @ router).topk(2, dim=1)
    offsets, rows, pos = vq.group_rows(ids.int(), gate_up.n_experts)
    g = vq.gemm_experts(gate_up, h, offsets, rows=rows)
    n = g.shape[1] // 2
    a = torch.nn.functional.silu(g[:, :n].float()) * g[:, n:].float()
    z = vq.gemm_experts(down, a.bfloat16(), offsets, out_dtype=torch.float32)
    return h, ids, a, z, vq.combine_rows(z, pos, torch.softmax(score, dim=1))


@pytest.mark.parametrize("tokens", [1, 150])
def test_a_block_eager_and_captured(tokens):
    """The whole block against the per-layer calls of vq.h on each expert's
    rows, and the same block captured once and replayed on another input."""
    vq = _vq()
    dim, inner, e = 256, 192, 5
    up_data, gate_up = _experts(LayerSpec(2 * inner, dim, 8, (12, 8), (0.05, 0.01)), e, "tile4", 60)
    down_data, down = _experts(LayerSpec(dim, inner, 8, (12, 8), (0.05, 0.01)), e, "tile4", 80)
    proj = vq.Int8Layer.quantise((torch.randn((dim, dim), device="cuda") / 16).half())
    router = torch.randn((dim, e), device="cuda")
    x = torch.randn((tokens, dim), device="cuda").bfloat16()
    h, ids, a, z, y = _block(vq, proj, gate_up, down, x, router)
    offsets, rows, pos = vq.group_rows(ids.int(), e)
    _check(vq.gemm_experts(gate_up, h, offsets, rows=rows), h, up_data, offsets, rows, -3.0)
    _check(z, a.bfloat16(), down_data, offsets, None, -3.0)
    for k in range(e):
        at = (ids == k).any(1).nonzero()[:, 0]
        if len(at) and tokens > 1:
            one = vq.gemm(gate_up.layer(k), h[at].contiguous())
            mine = vq.gemm_experts(gate_up, h, offsets, rows=rows)[int(offsets[k]): int(offsets[k + 1])]
            assert (one.float() - mine.float()).abs().max() <= 2.0 ** -6 * one.float().abs().max()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = _block(vq, proj, gate_up, down, x, router)[-1]
    for _ in range(2):
        x.copy_(torch.randn_like(x))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _block(vq, proj, gate_up, down, x, router)[-1])


def test_two_streams_at_once():
    vq = _vq()
    data, ex = _experts(LayerSpec(512, 512, 8, (12, 8), (0.02, 0.005)), 4, "rows", 21)
    cases = []
    for counts in ([3, 0, 9, 1], [90, 200, 3, 60]):
        x = torch.randn((sum(counts), 512), device="cuda").bfloat16()
        cases.append((x, _offsets(counts), torch.cuda.Stream()))
    want = [vq.gemm_experts(ex, x, o) for x, o, _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i, (x, o, s) in enumerate(cases):
            with torch.cuda.stream(s):
                got[i] = vq.gemm_experts(ex, x, o)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("counts", [[3, 0, 2], [300, 40, 700]])
def test_device_waits_give_up_with_a_status(monkeypatch, counts):
    """A wait whose budget is zero gives up: the call ends, the status word
    says so and stays set, and the next call is right."""
    vq = _vq()
    data, ex = _experts(LayerSpec(900, 1000, 8, (12, 8), (0.02, 0.005)), 3, "tile4", 31)
    x, offsets = torch.randn((sum(counts), 1000), device="cuda").bfloat16(), _offsets(counts)
    work = torch.zeros(vq.gemm_experts_workspace_size(ex, sum(counts)), dtype=torch.uint8, device="cuda")
    monkeypatch.setenv("VQ_WAIT_BUDGET", "0")
    vq.gemm_experts(ex, x, offsets, workspace=work)
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32)) == vq.VQ_ERR_TIMEOUT
    monkeypatch.delenv("VQ_WAIT_BUDGET")
    y = vq.gemm_experts(ex, x, offsets, out_dtype=torch.float32, workspace=work)
    _check(y, x, data, offsets, None, 0)
    assert int(work[:4].view(torch.int32)) == vq.VQ_ERR_TIMEOUT


def test_binding_checks():
    vq = _vq()
    data, ex = _experts(LayerSpec(32, 64, 8, (8,), (0.02,)), 2, "rows", 1)
    x, o = torch.randn((4, 64), device="cuda").half(), _offsets([2, 2])
    for bad in (dict(x=x.float()), dict(x=x[:, :60]), dict(offsets=o[:2]), dict(offsets=o.long()),
                dict(rows=torch.zeros(4, device="cuda")), dict(out=torch.empty((3, 32), device="cuda")),
                dict(out_dtype=torch.int32), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            vq.gemm_experts(ex, **{**dict(x=x, offsets=o), **bad})
    with pytest.raises(vq.VQError):
        vq.gemm_experts(ex, x, o, workspace=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        vq.Experts(32, 64, 8, [8], [t[:, :, :1] for t in ex.idx], ex.codebooks)       # rows too short
    with pytest.raises(ValueError):
        vq.Experts(32, 64, 8, [9], ex.idx, ex.codebooks)
    with pytest.raises(ValueError):
        vq.Experts.from_layers([ex.layer(0), vq.repack_tile4(ex.layer(1))])


@pytest.mark.parametrize("n,kin,books,d", [(161, 66, (16, 8), 8), (112, 96, (8,), 4), (40, 9, (12, 4), 6)])
def test_many_rows_of_short_weights(n, kin, books, d):
    """Few steps per tile: a tile per CTA and more, none of them cut."""
    spec = LayerSpec(n, kin, d, books, (0.02, 0.005)[: len(books)], out_bias_std=1.0)
    counts = [900, 0, 333, 1500]
    data, ex = _experts(spec, 4, "rows", 17)
    x = torch.randn((sum(counts), kin), device="cuda").bfloat16()
    _check(_run(ex, x, _offsets(counts)), x, data, _offsets(counts), None, -3.0)
