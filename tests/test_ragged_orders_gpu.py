"""Ragged grouped products where CTAs of a cluster hand memory to one another:
shared reductions over many tiles, and segment ends of CTA pairs.  Results are
compared with their definition in 64 bits, and repeated calls bit by bit: a
buffer written again before it was read would show in either.  Bounds are
those of tests/test_ragged_gpu.py (check)."""

import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from tests.test_ragged_gpu import check, form, gen, layout, run_rows, run_tn  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("split", [2, 4, 8])
@pytest.mark.parametrize("bn", [16, 32, 64])
@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_shared_reductions_of_many_tiles(direction, bn, split, form):  # noqa: F811
    """FP16, many segments, a hundred tiles or so for each cluster."""
    form((1, 0, bn, split))
    call = fp8.m_grouped_gemm_nt_ragged if direction == "nt" else fp8.m_grouped_gemm_nn_ragged
    counts = [(7 * i) % 41 for i in range(48)]
    a, b, d, offsets = run_rows(direction, counts, 2112, 1160, FP16, seed=bn + split)
    for _ in range(20):
        again = torch.full_like(d, 7.0)
        call(a, b, again, offsets)
        assert torch.equal(again, d)
    assert fp8.get_device_status() == 0


@pytest.mark.parametrize("out,accumulate", [(FP32, False), (FP32, True), (FP16, False)])
def test_segment_ends_of_pairs(out, accumulate, form):  # noqa: F811
    """Weight gradients by CTA pairs of segments that end within a block; the
    rows behind hold NaN or the next segment."""
    form((0, 1, 256))
    counts = [1, 127, 129, 0, 17, 255, 63, 2, 640, 31, 300, 5]
    a, b, d, offsets = run_tn(counts, 520, 776, FP16, out, accumulate, seed=3)
    if not accumulate:
        for _ in range(20):
            again = torch.full_like(d, 7.0)
            fp8.k_grouped_gemm_tn_ragged(a, b, again, offsets)
            assert torch.equal(again, d)


def test_adding_to_a_gradient_from_a_graph():
    """Each replay of a captured step adds once more, with the segments of the replay."""
    counts, N, K = [40, 0, 90, 600], 264, 136
    offsets, ends, T = layout(counts)
    gy, x = gen(T, N, seed=1, dtype=BF16), gen(T, K, seed=2, dtype=BF16)
    gw = gen(4, N, K, seed=3, dtype=FP32)
    start = gw.double()
    graph = torch.cuda.CUDAGraph()
    fp8.k_grouped_gemm_tn_ragged(gy, x, torch.empty_like(gw), offsets)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fp8.k_grouped_gemm_tn_ragged(gy, x, gw, offsets, accumulate=True)
    assert torch.equal(gw.double(), start)
    segments = [(0, 40, 40, 130, 730), (0, 0, 300, 301, 700), (0, 40, 40, 130, 730)]
    for ends in segments:
        offsets.copy_(torch.tensor(ends, dtype=torch.int32))
        graph.replay()
    for g in range(4):
        ref, mag, rows = start[g].clone(), start[g].abs(), 0
        for ends in segments:
            r = slice(ends[g], ends[g + 1])
            ref += gy[r].double().T @ x[r].double()
            mag += gy[r].double().abs().T @ x[r].double().abs()
            rows += ends[g + 1] - ends[g]
        check(gw[g], ref, mag, rows)   # (three roundings of the sum more: of the 32 steps allowed)
    assert fp8.get_device_status() == 0
