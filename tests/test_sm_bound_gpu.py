"""set_num_sms bounds the CTAs of every launch of the grouping and the adapters.

The launches of a call are read from a captured graph (their grids, one CTA or
more per SM); the results under a bound are checked as those without one.
"""

import ctypes

import numpy as np
import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from tests.test_grouping_lora_gpu import gen, group_call, group_reference, lora_case, sorted_order

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
BOUNDS = [1, 2, 3, 20, 147]


@pytest.fixture(params=BOUNDS)
def bound(request):
    fp8.set_num_sms(request.param)
    yield request.param
    fp8.set_num_sms(0)


class KernelNode(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def ctas_of(call):
    """CTAs of each kernel that `call` launches."""
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu, raw = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph())
    n = ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    ctas = []
    for node in nodes:
        kind, k = ctypes.c_int(-1), KernelNode()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)) == 0
            ctas.append(k.grid[0] * k.grid[1] * k.grid[2])
    return ctas


def bounded(call, bound):
    """`call` launches more CTAs without the bound, and no more than it under it."""
    inside = ctas_of(call)
    assert inside and max(inside) <= bound, inside
    fp8.set_num_sms(0)
    try:
        return max(ctas_of(call)) > bound
    finally:
        fp8.set_num_sms(bound)


@pytest.mark.parametrize("R,G", [(700, 7), (4097, 1024), (131075, 64), (600000, 5)])
def test_grouping(bound, R, G):
    rng = np.random.default_rng(R)
    index = rng.integers(-1, G, R)
    for got, ref in zip(group_call(index, G, 5, torch.int64), group_reference(index, G, 5)):
        assert np.array_equal(got, ref)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx = torch.as_tensor(index, device="cuda")
    out = torch.empty(G + 1, **i32), torch.empty(R, **i32), torch.empty(R, **i32), torch.empty(R, **i32)
    more = bounded(lambda: fp8.group_rows_by_index(idx, G, *out), bound)
    assert more or R < 2048 * bound


def adapters(T, L, R, N, K, dtype, ids, order, bound):
    lora_case(T, L, R, N, K, dtype, ids, seed=T + R, order=order)
    x, A = gen(T, K, seed=1, dtype=dtype), gen(L, R, K, seed=2, dtype=dtype)
    B, c = gen(L, N, R, seed=3, dtype=dtype), gen(T, N, seed=4, dtype=dtype)
    m, s = torch.tensor(ids, dtype=torch.int32, device="cuda"), torch.ones(L, device="cuda")
    return bounded(lambda: fp8.m_grouped_lora_add(x, A, B, s, c, c, m), bound)


@pytest.mark.parametrize("T,R,N,K", [(1, 16, 2112, 2048), (40, 24, 520, 1032), (300, 16, 264, 520), (700, 256, 264, 520),
                                     (100, 136, 2112, 264)])
def test_adapters_of_short_batches(bound, T, R, N, K):
    ids = [(t // 3) % 6 - 1 for t in range(T)]
    assert adapters(T, 5, R, N, K, BF16, ids, sorted_order(ids), bound) or bound == 147
    lora_case(T, 5, R, N, K, FP16, ids, seed=1)                  # slot i is row i
    lora_case(T, 5, R, N, K, FP16, ids, seed=2, inplace=True)


def test_adapters_of_long_batches_in_short_form(bound):
    """More adapters than a block of slots can share: many pieces."""
    T, L = 3000, 200
    assert fp8.get_lora_workspace_size(T, L, 24, 264, 136) > 0
    ids = [t * 7 // T for t in range(T)]
    assert adapters(T, L, 24, 264, 136, BF16, ids, None, bound)


@pytest.mark.parametrize("T", [900, 4300, 20000])
@pytest.mark.parametrize("R", [16, 128])
def test_adapters_of_long_batches(bound, T, R):
    assert fp8.get_lora_workspace_size(T, 5, R, 136, 264) == 0
    ids = [(t * 6 // T) - 1 for t in range(T)]
    more = adapters(T, 5, R, 136, 264, FP16, ids, None, bound)
    assert more or T < 128 * bound
    if T == 4300:
        lora_case(T, 5, R, 136, 264, BF16, ids, seed=2, order=sorted_order(ids)[::-1], inplace=True)
