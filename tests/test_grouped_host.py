"""Host side of the row-grouped operators: sizes, refusals, bindings (no GPU)."""

import ctypes

import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from fp8_fine_grained_nt_b200 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


P, MIS, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), None
BF16, FP16, F32 = 1, 2, 0


@pytest.mark.parametrize("name", ["m_grouped_gemm_nt_ragged", "m_grouped_gemm_nn_ragged"])
def test_ragged_rows_refusals(lib, name):
    f = getattr(lib, name)  # fake pointers, never dereferenced: refused before any launch
    assert f(P, P, P, P, BF16, 0, 64, 64, 64, None) == 1       # no groups
    assert f(P, P, P, P, F32, 2, 64, 64, 64, None) == 1        # FP32 operands
    assert f(P, P, P, P, 7, 2, 64, 64, 64, None) == 1
    assert f(P, P, P, P, BF16, 2, -1, 64, 64, None) == 1
    assert f(P, P, P, P, BF16, 1025, 64, 64, 64, None) == 3    # groups
    assert f(P, P, P, P, BF16, 2, 64, 60, 64, None) == 3       # N % 8
    assert f(P, P, P, P, BF16, 2, 64, 64, 4, None) == 3        # K % 8
    assert f(P, P, P, P, BF16, 2, 64, 0, 64, None) == 3
    assert f(P, P, P, P, BF16, 1024, 64, 1 << 20, 1 << 20, None) == 3   # a group's weights over 2^40 bytes
    assert f(P, P, P, P, BF16, 1024, 2 ** 30, 1 << 18, 64, None) == 3      # tiles over 2^31
    assert f(P, P, P, P, BF16, 4, 2 ** 31 - 1, 64, 64, None) == 3          # rows
    assert f(P, P, P, P, BF16, 1, 16, 2 ** 31 - 8, 8, None) == 3           # columns
    assert f(P, P, P, P, BF16, 1, 16, 8, 2 ** 31 - 8, None) == 3
    for bad in range(4):
        args = [P] * 4
        args[bad] = NULL
        assert f(*args, BF16, 2, 64, 64, 64, None) == 1
    for bad in range(3):
        args = [P] * 4
        args[bad] = MIS
        assert f(*args, FP16, 2, 64, 64, 64, None) == 2
    assert f(P, P, P, ctypes.c_void_p(0x10002), BF16, 2, 64, 64, 64, None) == 2
    assert f(NULL, P, NULL, P, BF16, 2, 0, 64, 64, None) == 0   # no rows: nothing to do


def test_ragged_weight_gradient_refusals(lib):
    f = lib.k_grouped_gemm_tn_ragged
    assert f(P, P, P, P, BF16, FP16, 0, 2, 64, 64, 64, None) == 1   # result of another 16-bit type
    assert f(P, P, P, P, BF16, BF16, 1, 2, 64, 64, 64, None) == 1   # adding in 16 bits
    assert f(P, P, P, P, BF16, 9, 0, 2, 64, 64, 64, None) == 1
    assert f(P, P, P, P, BF16, F32, 0, 2, 64, 12, 64, None) == 3
    assert f(P, P, NULL, P, BF16, F32, 0, 2, 0, 64, 64, None) == 1  # no rows still write zeros


def test_group_sizes_and_refusals(lib):
    assert fp8.get_row_groups_capacity(10, 4) == 10
    assert fp8.get_row_groups_capacity(10, 4, 128) == 10 + 4 * 127 + (-(10 + 4 * 127)) % 128
    assert fp8.get_row_groups_capacity(2, 400, 128) == 256     # at most two groups have rows
    assert fp8.get_row_groups_capacity(0, 4, 128) == 0
    assert fp8.get_group_rows_workspace_size(100, 16) == 0
    assert fp8.get_group_rows_workspace_size(100000, 16) > 0
    for call in (lambda: fp8.get_row_groups_capacity(-1, 4), lambda: fp8.get_row_groups_capacity(4, 0),
                 lambda: fp8.get_row_groups_capacity(4, 4, 0), lambda: fp8.get_row_groups_capacity(1 << 30, 4, 128),
                 lambda: fp8.get_group_rows_workspace_size(4, 1025)):
        with pytest.raises(fp8.Fp8NtError):
            call()
    f = lib.group_rows_by_index
    assert f(P, 5, P, P, P, P, 8, 4, 1, P, 0, None) == 1
    assert f(P, 0, P, P, P, P, 8, 4, 0, P, 0, None) == 1
    assert f(P, 0, P, P, P, P, 8, 2000, 1, P, 1 << 20, None) == 3
    assert f(P, 0, NULL, P, P, P, 8, 4, 1, P, 0, None) == 1
    assert f(NULL, 0, P, P, P, P, 8, 4, 1, P, 0, None) == 1
    assert f(P, 0, P, P, P, P, 100000, 4, 1, P, 8, None) == 1       # workspace too small
    assert f(P, 0, P, P, P, P, 100000, 4, 1, NULL, 1 << 20, None) == 1
    assert f(ctypes.c_void_p(0x10004), 1, P, P, P, P, 8, 4, 1, P, 0, None) == 2  # int64 at 4 bytes
    assert f(P, 0, P, ctypes.c_void_p(0x10002), P, P, 8, 4, 1, P, 0, None) == 2


def test_lora_sizes_and_refusals(lib):
    assert fp8.get_lora_workspace_size(0, 2, 16, 64, 64) == 0
    assert fp8.get_lora_workspace_size(64, 2, 16, 64, 7168) >= 64 * 16 * 4
    assert fp8.get_lora_workspace_size(4096, 8, 16, 64, 7168) == 0   # long batches need none
    for args in ((4, 2, 12, 64, 64), (4, 2, 264, 64, 64), (4, 2, 0, 64, 64), (4, 2, 16, 60, 64), (4, 2, 16, 64, 4),
                 (-1, 2, 16, 64, 64), (4, 0, 16, 64, 64)):
        with pytest.raises(fp8.Fp8NtError):
            fp8.get_lora_workspace_size(*args)

    def call(x=P, ld_x=64, a=P, b=P, s=P, c=P, ld_c=64, d=P, ld_d=64, m=P, o=P, dtype=BF16, slots=4, rows=4,
             adapters=2, rank=16, N=64, K=64, ws=P, size=1 << 30):
        return lib.m_grouped_lora_add(x, ld_x, a, b, s, c, ld_c, d, ld_d, m, o, dtype, slots, rows, adapters, rank,
                                      N, K, ws, size, None)

    assert call(dtype=F32) == 1 and call(rows=-1) == 1 and call(adapters=0) == 1 and call(slots=-1) == 1
    assert call(rank=12) == 3 and call(rank=512) == 3 and call(N=60) == 3 and call(K=60) == 3
    assert call(ld_x=56) == 1 and call(ld_c=56) == 1 and call(ld_d=0) == 1
    assert call(ld_x=68) == 3 and call(ld_c=68) == 3 and call(ld_d=68) == 3
    assert call(slots=0) == 0 and call(rows=0) == 0
    assert call(size=0) == 1 and call(ws=NULL) == 1 and call(m=NULL) == 1 and call(s=NULL) == 1 and call(d=NULL) == 1
    assert call(x=MIS) == 2 and call(a=MIS) == 2 and call(b=MIS) == 2 and call(c=MIS) == 2 and call(ws=MIS) == 2
    assert call(m=ctypes.c_void_p(0x10002)) == 2


def test_lora_columns_near_2_to_31(lib):
    assert lib.get_lora_workspace_size(1, 1, 8, 2 ** 31 - 8, 64) == -3
    assert lib.get_lora_workspace_size(1, 1, 8, 64, 2 ** 31 - 8) == -3
    assert lib.get_lora_workspace_size(1, 1, 8, 0x7fff0000, 64) > 0


@pytest.mark.parametrize("slots", [1, 24, 512, 768])
@pytest.mark.parametrize("rank", [8, 64, 256])
def test_lora_workspace_near_2_to_31(lib, slots, rank):
    """The largest N and K are cut into ranges like any other: between one and
    32 ranges of k, FP32 sums of each."""
    for N, K in ((64, 0x7fff0000), (0x7fff0000, 64), (64, 2080000000), (64, 0x7fff0000 - 8)):
        size = lib.get_lora_workspace_size(slots, 1000, rank, N, K)
        splits = size // (slots * rank * 4)
        assert size == splits * slots * rank * 4 and 1 <= splits <= 32


def test_force_ragged(lib):
    try:
        for form in ((1, 0, 16, 8), (1, 0, 64, 4), (1, 0, 16), (1, 0, 32), (1, 0, 64), (1, 0, 128), (0, 1, 256), (0, 0, 256), (0, 0, 128), (0, 0, 0)):
            fp8.force_ragged(*form)
        for form in ((1, 1, 256), (1, 0, 48), (0, 1, 128), (1, 0, 128, 2), (1, 0, 16, 3), (0, 1, 256, 2)):
            with pytest.raises(fp8.Fp8NtError):
                fp8.force_ragged(*form)
    finally:
        fp8.force_ragged(0, 0, 0)


def test_bindings_refuse_before_the_library(lib):
    a, b, d = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 64, dtype=torch.bfloat16), None
    off = torch.zeros(3, dtype=torch.int32)
    d = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (fp8.m_grouped_gemm_nt_ragged, fp8.m_grouped_gemm_nn_ragged):
        with pytest.raises(ValueError, match="CUDA"):
            call(a, b, d, off)
        with pytest.raises(ValueError, match="shape"):
            call(a, b, d, off[:2])
        with pytest.raises(ValueError, match="shape"):
            call(a[:, :8], b, d, off)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.k_grouped_gemm_tn_ragged(a, a, b, off)
    with pytest.raises(ValueError, match="shape"):
        fp8.k_grouped_gemm_tn_ragged(a, a[:3], b, off)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.group_rows_by_index(off, 4, off, off)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.m_grouped_lora_add(a, torch.zeros(2, 8, 64), torch.zeros(2, 64, 8), torch.zeros(2), d, d, off)
    with pytest.raises(ValueError, match="slots"):
        fp8.m_grouped_lora_add(a, torch.zeros(2, 8, 64), torch.zeros(2, 64, 8), torch.zeros(2), d, d,
                               torch.zeros(5, dtype=torch.int32))
