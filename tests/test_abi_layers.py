"""include/vq_i8.h and include/vq_experts.h: every declared symbol is exported,
and malformed arguments are refused on the host before any CUDA call."""
import ctypes as C

import pytest
import torch

from bit_packed_index_b200 import build, vq

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = (vq.VQ_OK, vq.VQ_ERR_INVALID_ARG, vq.VQ_ERR_UNSUPPORTED,
                                              vq.VQ_ERR_ALIGNMENT, vq.VQ_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vq.lib()


def test_every_declared_symbol_is_exported(lib):
    names = vq.exported_names(vq.HEADER_I8) + vq.exported_names(vq.HEADER_EXPERTS)
    assert set(names) == {"vq_quant_i8", "vq_gemm_i8_workspace_size", "vq_gemm_i8", "vq_linear_i8_workspace_size",
                          "vq_linear_i8", "vq_group_rows", "vq_gemm_experts_workspace_size", "vq_gemm_experts",
                          "vq_combine_rows"}
    for n in names:
        assert hasattr(lib, n), n


def _i8(n=64, k=100, ldw=112):
    d = vq._I8Desc()
    d.out_features, d.in_features, d.w, d.ldw, d.scale = n, k, 0x10000, ldw, 0x20000
    return d


def test_quant_i8_refusals(lib):
    def call(x=0x1000, t=vq.VQ_BF16, rows=3, n=10, ldx=16, q=0x2000, ldq=16, s=0x3000):
        return lib.vq_quant_i8(x, t, rows, n, ldx, q, ldq, s, None)
    for bad in (dict(rows=-1), dict(n=-1), dict(ldx=9), dict(ldq=9), dict(t=vq.VQ_FP32), dict(t=7), dict(x=None),
                dict(q=None), dict(s=None)):
        assert call(**bad) == INVALID, bad
    assert call(x=0x1001) == ALIGN
    assert call(s=0x3002) == ALIGN
    assert call(rows=0, x=None, q=None, s=None) == OK


def test_gemm_i8_refusals(lib):
    def call(d=None, q=0x4000, ldq=112, s=0x5000, m=4, y=0x6000, t=vq.VQ_BF16, ldy=64, ws=0x7000, nws=1 << 40):
        d = _i8() if d is None else d
        return lib.vq_gemm_i8(C.byref(d), q, ldq, s, m, y, t, ldy, ws, nws, None)
    for bad in (dict(m=-1), dict(ldq=99), dict(ldy=63), dict(t=5), dict(q=None), dict(s=None), dict(y=None),
                dict(d=_i8(n=-1)), dict(d=_i8(k=-1)), dict(d=_i8(ldw=96))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q=0x4008), dict(ldq=104), dict(s=0x5002), dict(y=0x6001), dict(y=0x6002, t=vq.VQ_FP32),
                dict(ws=0x7080), dict(d=_i8(ldw=104))):
        assert call(**bad) == ALIGN, bad
    assert call(m=(1 << 30) + 1) == UNSUPPORTED
    assert call(d=_i8(k=131072, ldw=131072), ldq=131072) == UNSUPPORTED
    assert call(ws=None) == WORKSPACE
    assert call(nws=16) == WORKSPACE
    assert call(m=0, q=None, s=None, y=None, ws=None) == OK
    assert call(d=_i8(n=0), ldy=0, ws=None) == OK
    d = _i8()
    d.w = None
    assert call(d=d) == INVALID
    d = _i8()
    d.out_bias = 0x8001
    assert call(d=d) == ALIGN
    assert lib.vq_gemm_i8(None, 0x4000, 112, 0x5000, 4, 0x6000, 0, 64, 0x7000, 1 << 40, None) == INVALID


def test_linear_i8_refusals_and_sizes(lib):
    def call(x=0x4000, xt=vq.VQ_FP16, m=4, ldx=100, y=0x6000, t=vq.VQ_FP32, ldy=64, ws=0x7000, nws=1 << 40):
        return lib.vq_linear_i8(C.byref(_i8()), x, xt, m, ldx, y, t, ldy, ws, nws, None)
    for bad in (dict(m=-1), dict(ldx=99), dict(xt=vq.VQ_FP32), dict(ldy=60), dict(x=None), dict(y=None)):
        assert call(**bad) == INVALID, bad
    assert call(x=0x4001) == ALIGN
    n = C.c_size_t(0)
    assert lib.vq_linear_i8_workspace_size(C.byref(_i8()), 4, C.byref(n)) == OK
    assert n.value >= 256 + 4 * 4 + 4 * 112 and n.value % 256 == 0
    assert call(nws=n.value - 1) == WORKSPACE
    assert lib.vq_linear_i8_workspace_size(C.byref(_i8()), 0, C.byref(n)) == OK and n.value == 0
    assert lib.vq_linear_i8_workspace_size(C.byref(_i8()), -1, C.byref(n)) == INVALID
    assert lib.vq_gemm_i8_workspace_size(C.byref(_i8()), 4, None) == INVALID


def test_group_rows_refusals(lib):
    def call(ids=0x1000, t=5, k=2, ld=2, e=8, off=0x2000, rows=0x3000, pos=0x4000):
        return lib.vq_group_rows(ids, t, k, ld, e, off, rows, pos, None)
    for bad in (dict(t=-1), dict(k=0), dict(ld=1), dict(e=0), dict(ids=None), dict(off=None), dict(rows=None),
                dict(pos=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(e=1025), dict(k=65, ld=65), dict(t=1 << 30)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(ids=0x1002), dict(off=0x2001), dict(rows=0x3002), dict(pos=0x4002)):
        assert call(**bad) == ALIGN, bad


def _ex(n=32, k=64, e=4, b=8, d=8, layout=vq.VQ_IDX_ROWS):
    D = vq._ExpertsDesc()
    L = D.layer
    L.out_features, L.in_features, L.vec_dim, L.n_books = n, k, d, 1
    L.log2k[0], L.idx[0], L.codebook[0], L.idx_layout = b, 0x10000, 0x20000, layout
    L.idx_row_words[0] = vq.row_words(k, max(d, 1), b) if layout == vq.VQ_IDX_ROWS else vq.tile4_words(n, b)
    D.n_experts = e
    D.idx_stride[0], D.codebook_stride[0] = 4096, (1 << b) * d
    return D


def test_gemm_experts_refusals(lib):
    def call(D=None, x=0x1000, xt=vq.VQ_BF16, xr=9, ldx=64, rows=0x2000, off=0x3000, m=12, y=0x4000, t=vq.VQ_BF16,
             ldy=32, ws=0x5000, nws=1 << 40):
        return lib.vq_gemm_experts(C.byref(_ex() if D is None else D), x, xt, xr, ldx, rows, off, m, y, t, ldy, ws,
                                   nws, None)
    for bad in (dict(m=-1), dict(xr=-1), dict(ldx=63), dict(ldy=31), dict(xt=vq.VQ_FP32), dict(t=3), dict(x=None),
                dict(off=None), dict(y=None), dict(rows=None), dict(D=_ex(e=0)), dict(D=_ex(d=0)), dict(D=_ex(b=17))):
        assert call(**bad) == INVALID, bad
    for field, value, want in (("reserved", 1, INVALID), ("scale_stride", -1, INVALID), ("bias_stride", -2, INVALID),
                               ("out_bias_stride", -1, INVALID), ("n_experts", 1025, UNSUPPORTED)):
        D = _ex()
        setattr(D, field, value)
        assert call(D=D) == want, field
    for field, value, want in (("idx_stride", -4, INVALID), ("idx_stride", 4098, ALIGN),
                               ("codebook_stride", -8, INVALID), ("codebook_stride", 4, ALIGN)):
        D = _ex()
        getattr(D, field)[0] = value
        assert call(D=D) == want, field
    for bad in (dict(x=0x1001), dict(rows=0x2002), dict(off=0x3002), dict(y=0x4001), dict(ws=0x5010)):
        assert call(**bad) == ALIGN, bad
    assert call(m=(1 << 24) + 1) == UNSUPPORTED
    assert call(D=_ex(n=1 << 30), m=1 << 20, xr=1 << 20, ldy=1 << 30) == UNSUPPORTED      # tiles past 2^31
    assert call(ws=None) == WORKSPACE
    assert call(nws=128) == WORKSPACE
    assert call(m=0, x=None, y=None, ws=None) == OK
    assert call(D=_ex(n=0), ws=None) == OK
    n = C.c_size_t(0)
    assert lib.vq_gemm_experts_workspace_size(C.byref(_ex()), 12, C.byref(n)) == OK and n.value >= 256
    assert lib.vq_gemm_experts_workspace_size(C.byref(_ex()), -1, C.byref(n)) == INVALID
    assert lib.vq_gemm_experts_workspace_size(None, 12, C.byref(n)) == INVALID


def test_combine_rows_refusals(lib):
    def call(z=0x1000, zt=vq.VQ_BF16, zr=9, n=16, ldz=16, pos=0x2000, w=0x3000, ldw=2, t=5, k=2, y=0x4000,
             yt=vq.VQ_FP32, ldy=16):
        return lib.vq_combine_rows(z, zt, zr, n, ldz, pos, w, ldw, t, k, y, yt, ldy, None)
    for bad in (dict(zr=-1), dict(n=-1), dict(ldz=15), dict(ldw=1), dict(t=-1), dict(k=0), dict(ldy=15), dict(zt=4),
                dict(yt=-1), dict(z=None), dict(pos=None), dict(w=None), dict(y=None)):
        assert call(**bad) == INVALID, bad
    assert call(k=65, ldw=65) == UNSUPPORTED
    for bad in (dict(z=0x1001), dict(pos=0x2002), dict(w=0x3002), dict(y=0x4002)):
        assert call(**bad) == ALIGN, bad
    assert call(t=0, y=None) == OK and call(n=0, y=None) == OK


def test_binding_refuses_host_tensors():
    """The binding's own checks come before the library: wrong device, type,
    shape or stride raises ValueError."""
    i8, f32, bf = torch.zeros((4, 16), dtype=torch.int8), torch.zeros(4), torch.zeros((2, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vq.Int8Layer(i8, f32)                                    # not on a CUDA device
    with pytest.raises(ValueError):
        vq.quant_i8(bf)
    with pytest.raises(ValueError):
        vq.group_rows(torch.zeros((2, 2), dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        vq.combine_rows(bf, torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)))
    with pytest.raises(ValueError):
        vq.Experts(4, 16, 8, [8], [torch.zeros((2, 4, 4), dtype=torch.int32)], [torch.zeros((2, 256, 8)).half()])
    with pytest.raises(ValueError):
        vq.Experts(4, 16, 8, [8], [torch.zeros((2, 4, 4), dtype=torch.int32)], [], layout="tile4")
