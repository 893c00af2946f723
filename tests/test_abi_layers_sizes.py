"""Sizes of vq_experts.h's workspaces at the ends of their arguments' ranges."""
import ctypes as C

import pytest

from bit_packed_index_b200 import build, vq


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vq.lib()


@pytest.mark.parametrize("kin", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 9, 2 ** 30])
def test_workspace_of_the_longest_rows(lib, kin):
    """One row of x' takes 16 bytes per vector of one to eight values."""
    D = vq._ExpertsDesc()
    L = D.layer
    L.out_features, L.in_features, L.vec_dim, L.n_books = 8, kin, 1, 1
    L.log2k[0], L.idx[0], L.codebook[0] = 1, 0x10000, 0x20000
    L.idx_row_words[0] = vq.row_words(kin, 1, 1)
    D.n_experts = 1
    n = C.c_size_t(0)
    assert lib.vq_gemm_experts_workspace_size(C.byref(D), 1, C.byref(n)) == vq.VQ_OK
    row = 128 * -(-kin // 8)
    assert row <= n.value <= row + (64 << 20)
