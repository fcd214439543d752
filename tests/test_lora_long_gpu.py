"""Low-rank adapters in their long form (one kernel over blocks of 128 slots).

Which form a call takes follows from its sizes; the long one needs no
workspace, and every test here asserts the form that it is about.  Bounds are
those of tests/test_grouping_lora_gpu.py (lora_check).
"""

import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from tests.test_grouping_lora_gpu import gen, lora_case, lora_check, sorted_order

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def is_long(slots, adapters, rank, N, K):
    return fp8.get_lora_workspace_size(slots, adapters, rank, N, K) == 0


@pytest.mark.parametrize("slots", [768, 769])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_both_sides_of_the_form_boundary(slots, dtype):
    assert is_long(slots, 4, 24, 264, 520) == (slots == 769)
    lora_case(slots, 4, 24, 264, 520, dtype, [t * 4 // slots for t in range(slots)], seed=slots)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("R", [8, 16, 24, 40, 64, 72, 104, 128])
def test_every_rank(R, dtype):
    """Blocks of one adapter, of several (more passes above rank 64), rows without one."""
    T, L, N, K = 900, 5, 200, 328
    assert is_long(T, L, R, N, K)
    lora_case(T, L, R, N, K, dtype, [t // 50 % 6 - 1 for t in range(T)], seed=R)
    ids = [t * L // T for t in range(T)]
    lora_case(T, L, R, N, K, dtype, ids, seed=R + 1, order=sorted_order(ids)[::-1], inplace=True)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("R", [16, 128])
@pytest.mark.parametrize("N,K", [(8, 8), (8, 2112), (2112, 8), (72, 1032), (4096, 7168)])
def test_every_size(N, K, R, dtype):
    T = 800
    assert is_long(T, 3, R, N, K)
    lora_case(T, 3, R, N, K, dtype, [(t // 100) % 4 - 1 for t in range(T)], seed=N + K)


@pytest.mark.parametrize("R", [64, 128])
@pytest.mark.parametrize("T", [1900, 2000, 4224, 4300, 9472, 9500])
def test_long_sums_in_every_cluster_size(T, R):
    """Clusters of 8, 4, 2 and 1 CTAs (up to 15, 33, 74 and more blocks of 128
    slots), K long enough for each CTA to go round its ring many times."""
    assert is_long(T, 6, R, 264, 7168)
    lora_case(T, 6, R, 264, 7168, BF16, [t * 6 // T for t in range(T)], seed=T)


@pytest.mark.parametrize("R", [72, 128])
def test_fp16_middle_result_beyond_its_range(R):
    """x . A^T is about 2e6, beyond FP16; B brings the result back into it, all but
    its tail: the deviation is 100 * 1000 * 512 ** 0.5 * 1e-3 * R ** 0.5, 19200 at
    rank 72 and 25600 at rank 128, so 3.4 and 2.6 of it reach 65520, from where
    rounding to nearest gives infinity."""
    T, N, K = 900, 136, 512
    assert is_long(T, 1, R, N, K)
    x, A = gen(T, K, seed=1, dtype=FP16, scale=100.0), gen(1, R, K, seed=2, dtype=FP16, scale=1000.0)
    B, c = gen(1, N, R, seed=3, dtype=FP16, scale=1e-3), gen(T, N, seed=4, dtype=FP16)
    d = torch.zeros(T, N, dtype=FP16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(1, device="cuda"), c, d, torch.zeros(T, dtype=torch.int32).cuda())
    x, A, B, c = x.double(), A[0].double(), B[0].double(), c.double()
    ref, mid = c + (x @ A.T) @ B.T, (x @ A.T).abs() @ B.abs().T
    mag = (x.abs() @ A.abs().T) @ B.abs().T
    bound = (2.0 ** -11 * ref.abs() + 2.0 ** -25 + (K / 16 + R / 8 + 96) * 2.0 ** -23 * mag + 2.0 ** -16 * mid
             + 2.0 ** -23 * c.abs())   # lora_check's
    over, inside = ref.abs() - bound > 65520, ref.abs() + bound < 65520
    assert torch.equal(d[over].double(), ref[over].sign() * float("inf"))
    assert 0 < over.sum() < 0.02 * ref.numel() and torch.isfinite(d[inside]).all()
    assert ((d.double() - ref).abs()[inside] <= bound[inside]).all()


@pytest.mark.parametrize("R", [40, 64, 128])
def test_special_values_stay_in_their_rows(R):
    """NaN in a row, Inf in an adapter, where a block of 128 slots has several."""
    T, L, N, K = 900, 3, 136, 264
    assert is_long(T, L, R, N, K)
    x, c = gen(T, K, seed=1, dtype=BF16), gen(T, N, seed=2, dtype=BF16)
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    x[3, 5] = float("nan")
    A[1, 2, 7] = float("inf")
    B[2, 11, 0] = float("inf")
    ids = [0] * 100 + [1] * 60 + [2] * (T - 160)
    d = torch.zeros(T, N, dtype=BF16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), c, d, torch.tensor(ids, dtype=torch.int32).cuda())
    want = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    want[3] = True
    want[100:160] = True
    want[160:, 11] = True
    assert torch.equal(~torch.isfinite(d), want)


def test_column_ranges_of_wider_tensors():
    T, L, R, N, K = 900, 3, 72, 136, 264
    assert is_long(T, L, R, N, K)
    wide_x, wide_c, wide_d = (gen(T, 2 * K, seed=1, dtype=BF16), gen(T, 3 * N, seed=2, dtype=BF16),
                              torch.full((T, 2 * N), 7.0, dtype=BF16, device="cuda"))
    x, c, d = wide_x[:, K:], wide_c[:, N:2 * N], wide_d[:, :N]
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), c, d,
                           torch.tensor([t // 300 for t in range(T)], dtype=torch.int32).cuda())
    for g in range(L):
        rows = slice(300 * g, 300 * g + 300)
        lora_check(d[rows], x[rows], A[g], B[g], 1.0, c[rows])
    assert (wide_d[:, N:] == 7).all()


def test_graph_and_concurrent_streams():
    T, L, R, N, K = 1500, 4, 128, 520, 1032
    assert is_long(T, L, R, N, K)
    x, A = gen(T, K, seed=1, dtype=BF16), gen(L, R, K, seed=2, dtype=BF16, scale=K ** -0.5)
    B, c = gen(L, N, R, seed=3, dtype=BF16), gen(T, N, seed=4, dtype=BF16)
    scales, ids = torch.ones(L, device="cuda"), torch.tensor([t * L // T for t in range(T)], dtype=torch.int32).cuda()
    want = torch.empty_like(c)
    fp8.m_grouped_lora_add(x, A, B, scales, c, want, ids)
    graphs, outs = [], []
    for _ in range(2):
        d, graph = torch.zeros_like(c), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fp8.m_grouped_lora_add(x, A, B, scales, c, d, ids)
        graphs.append(graph)
        outs.append(d)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    eager = [torch.zeros_like(c) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, s in zip(eager, streams):
            fp8.m_grouped_lora_add(x, A, B, scales, c, d, ids, stream=s)
    torch.cuda.synchronize()
    for d in outs + eager:
        assert torch.equal(d, want)
    assert fp8.get_device_status() == 0
