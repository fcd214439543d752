"""Low-rank adapters at the ends of the sizes that they accept."""

import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from tests.test_grouping_lora_gpu import gen, lora_check

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
MOST = 0x7fff0000


@pytest.mark.parametrize("slots", [1, 24])
def test_columns_near_2_to_31(slots):
    """The last of the column ranges ends near 2^31 (B: 34 GB, zero but for both ends)."""
    R, N, K, T = 8, MOST, 64, 2048
    x, A = gen(1, K, seed=1, dtype=BF16), gen(1, R, K, seed=2, dtype=BF16, scale=K ** -0.5)
    B, d = torch.zeros(1, N, R, dtype=BF16, device="cuda"), torch.zeros(1, N, dtype=BF16, device="cuda")
    ends = [slice(0, T), slice(N - T, N)]
    for i, e in enumerate(ends):
        B[0, e] = gen(T, R, seed=3 + i, dtype=BF16)
        d[0, e] = gen(T, seed=5 + i, dtype=BF16)
    before = [d[:, e].clone() for e in ends]
    ids = torch.zeros(slots, dtype=torch.int32, device="cuda")
    order = torch.tensor([0] + [-1] * (slots - 1), dtype=torch.int32, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(1, device="cuda"), d, d, ids, order)
    assert fp8.get_device_status() == 0
    for e, c in zip(ends, before):
        lora_check(d[:, e], x, A[0], B[0, e], 1.0, c)
    assert not d[0, T:N - T].any()


@pytest.mark.parametrize("named_stream", [False, True])
def test_no_memory_for_the_workspace(named_stream):
    """torch's own error whichever way the call goes, and the next call works."""
    T, L, R, N, K = 40960, 4, 256, 8, 64
    need = fp8.get_lora_workspace_size(T, L, R, N, K)
    assert need > 32 << 20   # a block of its own, not a part of one that is there
    x, A = gen(T, K, seed=1, dtype=BF16), gen(L, R, K, seed=2, dtype=BF16, scale=K ** -0.5)
    B, c = gen(L, N, R, seed=3, dtype=BF16), gen(T, N, seed=4, dtype=BF16)
    ids, d = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, N, dtype=BF16, device="cuda")
    args = (x, A, B, torch.ones(L, device="cuda"), c, d, ids)
    stream = dict(stream=torch.cuda.current_stream()) if named_stream else {}
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            fp8.m_grouped_lora_add(*args, **stream)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not d.any()
    fp8.m_grouped_lora_add(*args, **stream)
    lora_check(d, x, A[0], B[0], 1.0, c)


def test_long_sums_near_2_to_31():
    """The last of the ranges of k ends near 2^31 (A: 34 GB, zero but for both ends)."""
    R, N, K, T = 8, 64, MOST, 2048
    x, A = torch.zeros(1, K, dtype=BF16, device="cuda"), torch.zeros(1, R, K, dtype=BF16, device="cuda")
    for i, e in enumerate((slice(0, T), slice(K - T, K))):
        x[:, e] = gen(1, T, seed=1 + i, dtype=BF16)
        A[0, :, e] = gen(R, T, seed=3 + i, dtype=BF16, scale=T ** -0.5)
    B, c = gen(1, N, R, seed=5, dtype=BF16), gen(1, N, seed=6, dtype=BF16)
    d = torch.zeros(1, N, dtype=BF16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(1, device="cuda"), c, d, torch.zeros(1, dtype=torch.int32).cuda())
    assert fp8.get_device_status() == 0
    both = lambda t: torch.cat([t[..., :T], t[..., K - T:]], -1)  # noqa: E731
    lora_check(d, both(x), both(A[0]), B[0], 1.0, c)
