"""vq_gemm_experts at its edges.  Bounds and helpers: tests/test_gpu_experts.py."""
import numpy as np
import pytest
import torch

import oracle
import synth
from synth import LayerSpec
from tests.test_gpu_experts import _check, _experts, _offsets, _run, _vq

pytestmark = pytest.mark.gpu


# ---- index streams that are columns of a wider array --------------------------
def _column_experts(spec, e, after, seed):
    """Row-order experts whose index words are columns 4 .. of a wider array,
    `after` words of ones behind them.  A field of ones names the last entry of
    its book, an infinity that no vector uses: a read past a row's own words
    shows as NaN (the fields behind the last vector meet zeros of x)."""
    vq = _vq()
    data = [synth.make_layer(spec, seed=seed + i) for i in range(e)]
    idx, books = [], []
    for m, b in enumerate(spec.log2k):
        words = []
        for d in data:
            fields = oracle.unpack(d.idx_words[m], b, spec.nvec)
            d.idx_words[m] = oracle.pack(np.minimum(fields, (1 << b) - 2).astype(np.uint32), b, d.idx_words[m].shape[1])
            words.append(d.idx_words[m])
        words = np.stack(words)
        wide = np.full((e, spec.out_features, 4 + words.shape[2] + after), 0xFFFFFFFF, np.uint32)
        wide[:, :, 4: 4 + words.shape[2]] = words
        idx.append(torch.from_numpy(wide.view(np.int32)).cuda()[:, :, 4: 4 + words.shape[2]])
        book = torch.from_numpy(np.stack([d.codebooks[m] for d in data]).view(np.int16)).cuda().view(torch.float16)
        book = book.reshape(e, 1 << b, spec.d).clone()
        book[:, -1] = float("inf")
        books.append(book)
    half = lambda name: torch.from_numpy(np.stack([getattr(d, name) for d in data]).view(np.int16)).cuda().view(torch.float16)
    return data, vq.Experts(spec.out_features, spec.in_features, spec.d, list(spec.log2k), idx, books, half("scale"),
                            half("bias"))


@pytest.mark.parametrize("after", [4, 0], ids=["inside", "at_the_end"])
@pytest.mark.parametrize("books", [(12, 8), (12, 4), (12,), (16,), (8, 8)])
@pytest.mark.parametrize("nvec", [9, 10, 17, 21, 41, 50])
def test_index_words_in_columns_of_a_wider_array(nvec, books, after):
    """`inside`: words follow each row; `at_the_end`: the last row of the last
    expert ends with the storage."""
    spec = LayerSpec(130, 8 * nvec - 3, 8, books, (0.02, 0.005)[: len(books)])
    data, ex = _column_experts(spec, 2, after, 3 * nvec)
    x = torch.randn((21, spec.in_features), device="cuda").bfloat16()
    _check(_run(ex, x, _offsets([2, 17])), x, data, _offsets([2, 17]), None, -3.0)


@pytest.mark.parametrize("n", [130, 1])
def test_one_of_those_experts_as_a_layer(n):
    """A layer's arrays own the distance between rows behind the last row too."""
    spec = LayerSpec(n, 8 * 17, 8, (12, 8), (0.02, 0.005))
    data, ex = _column_experts(spec, 2, 0, 5)
    x = torch.randn((3, spec.in_features), device="cuda").bfloat16()
    for e in range(2):
        layer = ex.layer(e)
        for t in layer.idx:
            assert t.storage_offset() + t.shape[0] * t.stride(0) <= t.untyped_storage().nbytes() // 4
        _check(_vq().gemv(layer, x, out_dtype=torch.float32), x, [data[e]], _offsets([3]), None, -3.0)


# ---- blocks that give up -------------------------------------------------------
@pytest.mark.parametrize("budget", ["0", "1500", "6000"])
@pytest.mark.parametrize("kin,counts", [(200, [3, 0, 2]), (1000, [300, 40, 700]), (1000, [1, 0, 0])])
def test_calls_after_ones_that_gave_up(monkeypatch, kin, counts, budget):
    """Waits run out early, in the middle or not at all; whatever a block had in
    flight has landed before the next call's blocks take its place: that call,
    launched right behind, is right every time."""
    vq = _vq()
    data, ex = _experts(LayerSpec(900, kin, 8, (12, 8), (0.02, 0.005)), 3, "tile4", 31)
    x, offsets = torch.randn((sum(counts), kin), device="cuda").bfloat16(), _offsets(counts)
    want = _run(ex, x, offsets)
    _check(want, x, data, offsets, None, -3.0)
    work = torch.zeros(vq.gemm_experts_workspace_size(ex, sum(counts)), dtype=torch.uint8, device="cuda")
    spoilt, ys = torch.empty_like(want), []
    for _ in range(20):
        monkeypatch.setenv("VQ_WAIT_BUDGET", budget)
        vq.gemm_experts(ex, x, offsets, out=spoilt, workspace=work)
        monkeypatch.delenv("VQ_WAIT_BUDGET")
        ys.append(vq.gemm_experts(ex, x, offsets, out_dtype=torch.float32))
    torch.cuda.synchronize()
    assert int(work[:4].view(torch.int32)) in (vq.VQ_OK, vq.VQ_ERR_TIMEOUT)
    assert all(torch.equal(y, want) for y in ys)


# ---- rows near the end of bf16's range ------------------------------------------
@pytest.mark.parametrize("od", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bias", [None, 1e-3])
@pytest.mark.parametrize("books,layout", [((12, 8), "tile4"), ((16,), "rows"), ((9, 4), "rows")])
def test_finite_rows_have_finite_products(books, layout, bias, od):
    """Rows whose sums pass fp32's range while y does not; the rows beside them
    keep every bit."""
    spec = LayerSpec(300, 4096, 8, books, (0.02, 0.005)[: len(books)], (0.5, 1.5), bias, out_bias_std=1.0)
    data, ex = _experts(spec, 2, layout, 12)
    x = torch.randn((40, 4096), device="cuda").bfloat16()
    offsets = _offsets([17, 20])
    plain = _run(ex, x, offsets, od=od)
    big = [1, 2, 5, 16, 20, 36]
    x[1] = 1e35                                     # 4096 of them: sum x = 4.1e38
    x[2] = -1e35
    x[5] = torch.where(torch.arange(4096, device="cuda") % 2 == 0, 3e38, -3e38).bfloat16() * 2.0 ** -6
    x[16] = 2.0 ** 64                               # the first that counts as big
    x[20, :7], x[20, 7:] = 3e38, 0
    x[36] = 1e36 * torch.randn(4096, device="cuda")
    y = _run(ex, x, offsets, od=od)
    _check(y, x, data, offsets, None, -3.0)
    keep = [i for i in range(40) if i not in big]
    assert torch.equal(y[keep], plain[keep])


@pytest.mark.parametrize("value", [3.3e38, 1e-30])
def test_the_largest_scales(value):
    """Scales up to fp16's largest on rows of one value, centroids so small that
    y stays in range."""
    spec = LayerSpec(150, 64, 8, (8,), (1e-6,), (30000.0, 65000.0), None)
    data, ex = _experts(spec, 1, "rows", 4)
    x = torch.zeros((3, 64), device="cuda")
    x[0, 5], x[2, 63] = value, -value
    x = x.bfloat16()
    y = _run(ex, x, _offsets([3]))
    _check(y, x, data, _offsets([3]), None, -3.0)
    assert y.isfinite().all()


# ---- the longest rows -----------------------------------------------------------
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 8])
def test_combining_the_longest_rows(n):
    """One token of 2^31 - 1 columns (value by value) and of 2^31 - 8 (by words)."""
    vq = _vq()
    z = torch.zeros((1, n), dtype=torch.bfloat16, device="cuda")
    at = [0, 9, 2 ** 30, n - 1025, n - 8, n - 1]
    z[0, at] = torch.arange(1, 7, device="cuda").bfloat16()
    y = vq.combine_rows(z, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1, 1), 0.5, device="cuda"))
    assert y[0, at].tolist() == [0.5, 1, 1.5, 2, 2.5, 3]
    y[0, at] = 0
    assert not any(bool(p.any()) for p in y[0].split(1 << 28))


# ---- descriptions that no call accepts ------------------------------------------
def test_experts_that_no_call_accepts():
    vq = _vq()
    words = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    book = torch.zeros((2, 16, 8), dtype=torch.float16, device="cuda")
    make = lambda idx, books=book, n=6, k=64: vq.Experts(n, k, 8, [4], [idx], [books])
    make(words(2, 6, 12)[:, :, 4:8])
    flat = torch.zeros(2 * 16 * 8 + 8, dtype=torch.float16, device="cuda")
    for bad in (lambda: make(words(2, 6, 6)[:, :, :4]),                     # rows 6 words apart
                lambda: make(words(2, 6, 8)[:, :, 2:6]),                    # starts on 8 bytes
                lambda: make(words(2, 6, 4), flat[1:257].view(2, 16, 8)),   # a book that starts on 2
                lambda: make(words(2, 6, 4), flat.as_strided((2, 16, 8), (132, 8, 1))),
                lambda: make(words(1025, 6, 4), book[:1]),
                lambda: make(words(0, 6, 4), book[:0]),
                lambda: vq.Experts.from_layers([])):
        with pytest.raises(ValueError):
            bad()
