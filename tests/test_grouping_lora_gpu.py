"""Rows grouped by index, low-rank adapters, and a run of the grouped operators
together, against plain implementations in 64 bits (integers: exactly)."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from fp8_fine_grained_nt_b200 import inputs
from tests import helpers as H

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ rows grouped by index


def group_reference(index, G, alignment):
    index = np.asarray(index)
    R = len(index)
    capacity = (R + min(R, G) * (alignment - 1) + alignment - 1) // alignment * alignment
    offsets, order, m_indices = [0], np.full(capacity, -1), np.full(capacity, -1)
    slots = np.full(R, -1)
    rows_of = [[] for _ in range(G)]
    for r, g in enumerate(index.tolist()):
        if 0 <= g < G:
            rows_of[g].append(r)
    for g in range(G):
        rows, at = rows_of[g], offsets[-1]
        order[at:at + len(rows)] = rows
        m_indices[at:at + len(rows)] = g
        slots[rows] = np.arange(at, at + len(rows))
        offsets.append(at + -(-len(rows) // alignment) * alignment)
    return np.array(offsets), order, slots, m_indices


def group_call(index, G, alignment, dtype, **kw):
    idx = torch.as_tensor(np.asarray(index), dtype=dtype, device="cuda")
    cap = fp8.get_row_groups_capacity(len(index), G, alignment)
    new = lambda n: torch.full((n,), 12345, dtype=torch.int32, device="cuda")  # noqa: E731
    out = fp8.group_rows_by_index(idx, G, new(G + 1), new(cap), new(len(index)), new(cap),
                                  alignment=alignment, **kw)
    return [t.cpu().numpy() for t in out]


@pytest.mark.parametrize("R", [0, 1, 31, 33, 512, 4095, 4096, 4097, 20000, 131075])
@pytest.mark.parametrize("G", [1, 7, 256, 1024])
@pytest.mark.parametrize("alignment", [1, 5, 128])
def test_grouping(R, G, alignment):
    rng = np.random.default_rng(R * 31 + G)
    index = np.minimum((rng.random(R) ** 2 * G).astype(np.int64), G - 1)
    index[rng.random(R) < 0.2] = -1
    want = group_reference(index, G, alignment)
    for dtype in (torch.int32, torch.int64):
        for got, ref in zip(group_call(index, G, alignment, dtype), want):
            assert np.array_equal(got, ref)
    assert fp8.get_device_status() == 0


@pytest.mark.parametrize("index", [[3] * 9000, [-1] * 9000, [0, 3] * 3000, [-1], [3]])
def test_grouping_one_sided(index):
    for got, ref in zip(group_call(index, 4, 128, torch.int32), group_reference(index, 4, 128)):
        assert np.array_equal(got, ref)


def test_grouping_bad_index_is_flagged_and_left_out():
    for bad, dtype in ((4, torch.int32), (-2, torch.int32), (1 << 40, torch.int64), ((1 << 32) + 1, torch.int64)):
        index = [0, 1, bad, 3, 1]
        for got, ref in zip(group_call(index, 4, 1, dtype), group_reference(index, 4, 1)):
            assert np.array_equal(got, ref)
        assert fp8.get_device_status() == 7
    assert fp8.get_device_status() == 0


def test_grouping_optional_results_workspace_and_graph():
    rng = np.random.default_rng(5)
    index = rng.integers(-1, 64, 30000)
    want = group_reference(index, 64, 1)
    idx = torch.as_tensor(index, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, order = torch.empty(65, **i32), torch.empty(30000, **i32)
    ws = torch.empty(fp8.get_group_rows_workspace_size(30000, 64), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0 and fp8.get_group_rows_workspace_size(64, 64) == 0
    out = fp8.group_rows_by_index(idx, 64, offsets, order, workspace=ws)
    assert out[2] is None and out[3] is None
    assert np.array_equal(offsets.cpu(), want[0]) and np.array_equal(order.cpu(), want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8.group_rows_by_index(idx, 64, offsets, order)
    index = np.ascontiguousarray(index[::-1])
    idx.copy_(torch.as_tensor(index))
    graph.replay()
    want = group_reference(index, 64, 1)
    assert np.array_equal(offsets.cpu(), want[0]) and np.array_equal(order.cpu(), want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    order.zero_()
    side.wait_stream(torch.cuda.current_stream())
    fp8.group_rows_by_index(idx, 64, offsets, order, stream=side)
    side.synchronize()
    assert np.array_equal(order.cpu(), want[1])


# ------------------------------------------------------------------ low-rank adapters


def gen(*shape, seed, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def lora_check(got, x, A, B, scale, c):
    """Rounding of the result (eps / 2), the FP32 sums (steps of 16 products,
    plus 64 for the joins of k ranges, each off by 2^-23 of the sum of
    magnitudes) and the middle result as two 16-bit terms (2^-16 of it)."""
    (K, R), eps = (A.shape[1], A.shape[0]), torch.finfo(got.dtype).eps
    x, A, B, c = x.double(), A.double(), B.double(), c.double()
    v = x @ A.T
    ref = c + scale * (v @ B.T)
    mag = abs(scale) * ((x.abs() @ A.abs().T) @ B.abs().T)
    mid = abs(scale) * (v.abs() @ B.abs().T)
    tiny = 2.0 ** -25 if got.dtype == FP16 else 0.0
    bound = (eps / 2 * ref.abs() + tiny + (K / 16 + R / 8 + 96) * 2.0 ** -23 * mag + 2.0 ** -16 * mid
             + 2.0 ** -23 * c.abs())
    diff = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (diff <= bound).all(), f"worst {(diff / bound).max().item()} of the bound"
    if ref.numel() >= 64:
        assert diff.norm() <= eps / 2 * ref.norm()


def lora_case(T, L, R, N, K, dtype, ids, seed=0, order=None, inplace=False):
    x, A = gen(T, K, seed=seed, dtype=dtype), gen(L, R, K, seed=seed + 1, dtype=dtype, scale=K ** -0.5)
    B, c = gen(L, N, R, seed=seed + 2, dtype=dtype, scale=R ** -0.5), gen(T, N, seed=seed + 3, dtype=dtype)
    scales = torch.rand(L, device="cuda") + 0.5
    before = c.clone()
    d = c if inplace else torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    m_indices = torch.tensor(ids if order is None else [ids[t] if t >= 0 else 0 for t in order],
                             dtype=torch.int32, device="cuda")
    o = None if order is None else torch.tensor(order, dtype=torch.int32, device="cuda")
    assert fp8.m_grouped_lora_add(x, A, B, scales, c, d, m_indices, o) is d
    assert fp8.get_device_status() == 0
    covered = set(range(T)) if order is None else set(order)
    for g in range(L):
        rows = torch.tensor([t for t in range(T) if ids[t] == g and t in covered], dtype=torch.long, device="cuda")
        if len(rows):
            lora_check(d[rows], x[rows], A[g], B[g], float(scales[g]), before[rows])
    rest = torch.tensor([t for t in range(T) if ids[t] < 0 or t not in covered], dtype=torch.long, device="cuda")
    assert torch.equal(d[rest], before[rest] if inplace else torch.full_like(d[rest], 7.0))


def sorted_order(ids):
    return sorted((t for t in range(len(ids)) if ids[t] >= 0), key=lambda t: (ids[t], t))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 256, 257, 300, 700, 769, 1000])
@pytest.mark.parametrize("R", [8, 16, 40, 64, 136, 256])
def test_lora_rows_and_ranks(T, R):
    rng = np.random.default_rng(T * 100 + R)
    ids = rng.integers(-1, 5, T).tolist()
    lora_case(T, 5, R, 264, 520, BF16, ids, seed=T, order=sorted_order(ids))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N,K", [(8, 8), (8, 2112), (2112, 8), (72, 1032), (4096, 7168)])
@pytest.mark.parametrize("T", [3, 400, 800])
def test_lora_sizes(dtype, N, K, T):
    ids = [(t // 3) % 4 - 1 for t in range(T)]
    lora_case(T, 3, 16, N, K, dtype, ids, seed=N + K, order=sorted_order(ids))


@pytest.mark.parametrize("T", [5, 100, 900])
@pytest.mark.parametrize("R", [24, 64, 128])
def test_lora_fp16_ranks(T, R):
    ids = [(t // 7) % 4 - 1 for t in range(T)]
    lora_case(T, 3, R, 200, 328, FP16, ids, seed=T + R, order=sorted_order(ids))


@pytest.mark.parametrize("T", [2100, 4400, 9600])
@pytest.mark.parametrize("R", [64, 72])
def test_lora_long_batches(T, R):
    ids = [t * 5 // T for t in range(T)]
    lora_case(T, 5, R, 264, 520, BF16, ids, seed=T)


@pytest.mark.parametrize("T", [40, 300, 900])
@pytest.mark.parametrize("kind", ["unsorted", "all_different", "none", "one", "runs"])
def test_lora_orders(T, kind):
    L = T if kind == "all_different" else 6
    ids = {"unsorted": [t * 7 % 6 for t in range(T)], "all_different": list(range(T)), "none": [-1] * T,
           "one": [3] * T, "runs": [t // 50 % 6 for t in range(T)]}[kind]
    lora_case(T, L, 24, 136, 264, BF16, ids, seed=T)                          # slot i is row i
    lora_case(T, L, 24, 136, 264, BF16, ids, seed=T, inplace=True)
    lora_case(T, L, 24, 136, 264, BF16, ids, seed=T, order=sorted_order(ids) + [-1, -1, -1])  # padded slots
    lora_case(T, L, 24, 136, 264, BF16, ids, seed=T, order=list(range(T))[::-2], inplace=True)


def test_lora_column_ranges_of_wider_tensors():
    T, L, R, N, K = 50, 3, 16, 136, 264
    wide_x, wide_c, wide_d = (gen(T, 2 * K, seed=1, dtype=BF16), gen(T, 3 * N, seed=2, dtype=BF16),
                              torch.full((T, 2 * N), 7.0, dtype=BF16, device="cuda"))
    x, c, d = wide_x[:, K:], wide_c[:, N:2 * N], wide_d[:, :N]
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    scales = torch.ones(L, device="cuda")
    ids = torch.tensor([t % 3 for t in range(T)], dtype=torch.int32, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, scales, c, d, ids)
    for g in range(L):
        lora_check(d[g::3], x[g::3], A[g], B[g], 1.0, c[g::3])
    assert (wide_d[:, N:] == 7).all()


@pytest.mark.parametrize("R", [16, 40])
def test_lora_special_values_stay_in_their_rows(R):
    """NaN in a row, Inf in an adapter: other rows of the same 16 are clean."""
    T, L, N, K = 20, 3, 136, 264
    x, c = gen(T, K, seed=1, dtype=BF16), gen(T, N, seed=2, dtype=BF16)
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    x[3, 5] = float("nan")
    A[1, 2, 7] = float("inf")
    B[2, 11, 0] = float("inf")
    ids = [0] * 6 + [1] * 5 + [2] * 9
    d = torch.zeros(T, N, dtype=BF16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), c, d, torch.tensor(ids, dtype=torch.int32).cuda())
    bad = ~torch.isfinite(d)
    want = torch.zeros_like(bad)
    want[3] = True
    want[6:11] = True
    want[11:, 11] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T", [300, 900])
def test_lora_special_values_in_long_batches(T):
    """The same where 128 slots of up to three adapters are computed together."""
    L, R, N, K = 3, 16, 136, 264
    x, c = gen(T, K, seed=1, dtype=BF16), gen(T, N, seed=2, dtype=BF16)
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    x[3, 5] = float("nan")
    A[1, 2, 7] = float("inf")
    B[2, 11, 0] = float("inf")
    ids = [0] * 100 + [1] * 60 + [2] * (T - 160)
    d = torch.zeros(T, N, dtype=BF16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), c, d, torch.tensor(ids, dtype=torch.int32).cuda())
    bad = ~torch.isfinite(d)
    want = torch.zeros_like(bad)
    want[3] = True
    want[100:160] = True
    want[160:, 11] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("T,R", [(20, 16), (20, 40), (900, 16), (900, 40)])
def test_lora_fp16_middle_result_beyond_its_range(T, R):
    """x . A^T is about 2e6, beyond FP16; B brings the result back into it."""
    L, N, K = 1, 136, 512
    x, A = gen(T, K, seed=1, dtype=FP16, scale=100.0), gen(L, R, K, seed=2, dtype=FP16, scale=1000.0)
    B, c = gen(L, N, R, seed=3, dtype=FP16, scale=1e-3), gen(T, N, seed=4, dtype=FP16)
    d = torch.zeros(T, N, dtype=FP16, device="cuda")
    fp8.m_grouped_lora_add(x, A, B, torch.ones(1, device="cuda"), c, d, torch.zeros(T, dtype=torch.int32).cuda())
    lora_check(d, x, A[0], B[0], 1.0, c)


def test_lora_bad_slots_are_flagged_and_skipped():
    T, L, R, N, K = 4, 2, 16, 64, 64
    x, c = gen(T, K, seed=1, dtype=BF16), gen(T, N, seed=2, dtype=BF16)
    A, B = gen(L, R, K, seed=3, dtype=BF16), gen(L, N, R, seed=4, dtype=BF16)
    i32 = dict(dtype=torch.int32, device="cuda")
    for ids, order in (([0, 2, 1], [0, 1, 2]), ([0, 1, 1], [0, 4, 2])):
        d = torch.full((T, N), 7.0, dtype=BF16, device="cuda")
        fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), c, d, torch.tensor(ids, **i32),
                               torch.tensor(order, **i32))
        assert fp8.get_device_status() == 7
        assert (d[1] == 7).all() and (d[3] == 7).all()
        lora_check(d[2:3], x[2:3], A[1], B[1], 1.0, c[2:3])


@pytest.mark.parametrize("T", [5, 400, 900])
def test_lora_negative_slots(T):
    x, A, B = gen(T, 64, seed=1, dtype=BF16), gen(2, 8, 64, seed=2, dtype=BF16), gen(2, 64, 8, seed=3, dtype=BF16)
    scale, c = torch.ones(2, device="cuda"), gen(T, 64, seed=4, dtype=BF16)
    ids = torch.ones(T, dtype=torch.int32, device="cuda")
    order = torch.arange(T, dtype=torch.int32, device="cuda")
    for bad_ids, bad_order, status in ((-1, 3, 0), (-2, 3, 7), (1, -1, 0), (1, -2, 7)):
        ids[3], order[3] = bad_ids, bad_order
        d = torch.full_like(c, 9.0)
        fp8.m_grouped_lora_add(x, A, B, scale, c, d, ids, order)
        assert fp8.get_device_status() == status
        assert (d[3] == 9).all() and not (d[4] == 9).all()


def test_lora_no_slots():
    x, c = gen(4, 64, seed=1, dtype=BF16), gen(4, 64, seed=2, dtype=BF16)
    A, B = gen(2, 8, 64, seed=3, dtype=BF16), gen(2, 64, 8, seed=4, dtype=BF16)
    d = torch.full_like(c, 7.0)
    fp8.m_grouped_lora_add(x, A, B, torch.ones(2, device="cuda"), c, d, torch.empty(0, dtype=torch.int32).cuda(),
                           torch.empty(0, dtype=torch.int32).cuda())
    assert (d == 7).all()


def test_lora_graph_and_concurrent_streams():
    """Two captured calls and two streams at once, each with a workspace of its own."""
    T, L, R, N, K = 40, 4, 16, 520, 1032
    x, A = gen(T, K, seed=1, dtype=BF16), gen(L, R, K, seed=2, dtype=BF16, scale=K ** -0.5)
    B, c = gen(L, N, R, seed=3, dtype=BF16), gen(T, N, seed=4, dtype=BF16)
    scales, ids = torch.ones(L, device="cuda"), torch.tensor([t % 4 for t in range(T)], dtype=torch.int32).cuda()
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
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    eager = [torch.zeros_like(c) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, s in zip(eager, streams):
            fp8.m_grouped_lora_add(x, A, B, scales, c, d, ids, stream=s)
    torch.cuda.synchronize()
    for d in outs + eager:
        assert torch.equal(d, want)


def test_lora_rows_beyond_2_to_31_elements():
    T, L, R, N, K = 70001, 2, 8, 32768, 64
    x, A = gen(T, K, seed=1, dtype=BF16), gen(L, R, K, seed=2, dtype=BF16, scale=K ** -0.5)
    B, d = gen(L, N, R, seed=3, dtype=BF16), torch.zeros(T, N, dtype=BF16, device="cuda")
    ids = (torch.arange(T, device="cuda") >= 35000).to(torch.int32)
    zero = torch.zeros(40, N, dtype=BF16, device="cuda")
    for slots in (T, 40):   # a long batch, and a few rows at the end
        d.zero_()
        order = torch.arange(T - slots, T, dtype=torch.int32, device="cuda")
        fp8.m_grouped_lora_add(x, A, B, torch.ones(L, device="cuda"), d, d, ids[T - slots:], order)
        lora_check(d[T - 40:], x[T - 40:], A[1], B[1], 1.0, zero)
        if slots == T:
            lora_check(d[34960:35000], x[34960:35000], A[0], B[0], 1.0, zero)


def test_lora_many_adapters_and_long_batches():
    """The forms for few and for many slots on the same rows agree to rounding."""
    T, R, N, K = 1000, 16, 264, 520
    ids = [t * 7 // T for t in range(T)]
    lora_case(T, 7, R, N, K, FP16, ids, seed=3)              # about 143 rows each: the long form
    lora_case(T, 200, R, N, K, FP16, ids, seed=3)            # 200 adapters loaded, 7 in use: the short one
    lora_case(T, 31, 64, N, K, BF16, [t % 31 for t in range(T)], seed=4)   # unsorted: 128 segments a block


def test_refusals_of_device_tensors():
    x, A, B, c = (gen(4, 64, seed=1, dtype=BF16), gen(2, 8, 64, seed=2, dtype=BF16), gen(2, 64, 8, seed=3, dtype=BF16),
                  gen(4, 64, seed=4, dtype=BF16))
    s, m = torch.ones(2, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((x.float(), A, B, s, c, c, m), (x, A.half(), B, s, c, c, m), (x, A, B, s.double(), c, c, m),
                (x, A, B, s, c.half(), c, m), (x, A, B, s, c, c, m.long())):
        with pytest.raises(TypeError):
            fp8.m_grouped_lora_add(*bad)
    for bad in ((x, A.transpose(1, 2), B, s, c, c, m), (x, A, B, s, c.t().contiguous().t(), c, m),
                (x, A, B, s, c[:3], c, m), (x, A, B, s, c, c, torch.zeros(5, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fp8.m_grouped_lora_add(*bad)
    with pytest.raises(ValueError):
        fp8.m_grouped_lora_add(x, A, B, s, c, c, m, workspace=torch.empty(64, dtype=torch.uint8))
    with pytest.raises(fp8.Fp8NtError) as e:
        fp8.m_grouped_lora_add(x, A, B, s, c, c, m, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 1
    wide = gen(4, 68, seed=5, dtype=BF16)
    with pytest.raises(fp8.Fp8NtError) as e:   # rows 136 bytes apart
        fp8.m_grouped_lora_add(wide[:, :64], A, B, s, c, c, m)
    assert e.value.status == 3
    i32 = dict(dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        fp8.group_rows_by_index(s, 4, torch.empty(5, **i32), torch.empty(2, **i32))
    with pytest.raises(ValueError):
        fp8.group_rows_by_index(m, 4, torch.empty(5, **i32), torch.empty(3, **i32))
    with pytest.raises(fp8.Fp8NtError):
        fp8.group_rows_by_index(m, 0, torch.empty(1, **i32), torch.empty(4, **i32))
    with pytest.raises(fp8.Fp8NtError):
        fp8.group_rows_by_index(torch.zeros(9000, **i32), 4, torch.empty(5, **i32), torch.empty(9000, **i32),
                                workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert fp8.get_device_status() == 0


# ------------------------------------------------------------------ together


def test_moe_layer_forward_and_backward():
    """A router's choices -> layout -> experts' products -> both gradients."""
    T, top, G, N, K = 200, 3, 6, 264, 136
    g = torch.Generator().manual_seed(0)
    choice = torch.stack([torch.randperm(G, generator=g)[:top] for _ in range(T)]).flatten().cuda()
    choice[::7] = -1  # experts of another rank
    R = T * top
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, order, slots, _ = fp8.group_rows_by_index(
        choice, G, torch.empty(G + 1, **i32), torch.empty(R, **i32), torch.empty(R, **i32))
    x, w = gen(T, K, seed=1, dtype=BF16), gen(G, N, K, seed=2, dtype=BF16, scale=K ** -0.5)
    rows = order.clamp(min=0).long() // top
    xs = x[rows]
    y = torch.full((R, N), 7.0, dtype=BF16, device="cuda")
    fp8.m_grouped_gemm_nt_ragged(xs, w, y, offsets)
    gy = gen(R, N, seed=3, dtype=BF16)
    gx = torch.zeros(R, K, dtype=BF16, device="cuda")
    gw = torch.zeros(G, N, K, dtype=FP32, device="cuda")
    fp8.m_grouped_gemm_nn_ragged(gy, w, gx, offsets)
    fp8.k_grouped_gemm_tn_ragged(gy, xs, gw, offsets, accumulate=True)
    assert fp8.get_device_status() == 0
    wd, gwd = w.double(), torch.zeros(G, N, K, dtype=torch.float64, device="cuda")
    for r in range(R):
        s, e = int(slots[r]), int(choice[r])
        if e < 0:
            assert s == -1
            continue
        xr = x[r // top].double()
        ref, mag = wd[e] @ xr, wd[e].abs() @ xr.abs()
        assert ((y[s].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 48 * 2.0 ** -23 * mag).all()
        ref, mag = gy[s].double() @ wd[e], gy[s].double().abs() @ wd[e].abs()
        assert ((gx[s].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 64 * 2.0 ** -23 * mag).all()
        gwd[e] += torch.outer(gy[s].double(), xr)
    assert (gw.double() - gwd).norm() <= 2.0 ** -18 * gwd.norm()
    assert (y[int(offsets[-1]):] == 7).all()


def test_layout_feeds_the_contiguous_fp8_gemm():
    """alignment = 128: order and m_indices are what the contiguous FP8 form reads."""
    G, N, K, R = 5, 264, 256, 700
    idx = torch.randint(-1, G, (R,), generator=torch.Generator().manual_seed(1)).cuda()
    al = fp8.get_m_alignment_for_contiguous_layout()
    cap = fp8.get_row_groups_capacity(R, G, al)
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, order, slots, m_indices = fp8.group_rows_by_index(
        idx, G, torch.empty(G + 1, **i32), torch.empty(cap, **i32), torch.empty(R, **i32), torch.empty(cap, **i32),
        alignment=al)
    x = gen(R, K, seed=2, dtype=BF16)
    q, sa = torch.empty(cap, K, dtype=torch.uint8, device="cuda"), torch.empty(K // 128, cap, device="cuda")
    fp8.quantize_fp8_1x128(x[order.clamp(min=0).long()], q, sa)
    bs = [inputs.quantize_rhs(torch.randn(N, K, generator=torch.Generator().manual_seed(g))) for g in range(G)]
    b, sb = torch.stack([t[0] for t in bs]).cuda(), torch.stack([t[1] for t in bs]).cuda()
    d = H.sentinel_like((cap, N))
    fp8.m_grouped_gemm_fp8_fp8_bf16_nt_contiguous(q, sa, b, sb, d, m_indices)
    assert fp8.get_device_status() == 0
    dec = lambda t: t.view(torch.float8_e4m3fn).double()  # noqa: E731
    for g in range(G):
        s = torch.nonzero(m_indices == g).flatten()
        a64 = dec(q[s]) * sa[:, s].t().double().repeat_interleave(128, 1)
        b64 = dec(b[g]) * sb[g].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        H.assert_close(H.bf16_bits_to_f64(d[s]), (a64 @ b64.T).cpu().numpy())
    assert H.untouched(d)[(m_indices < 0).cpu().numpy()].all()


def test_adapters_beside_the_fp8_projection():
    """Shared FP8 projection, requests sorted by adapter, adapters added in place."""
    T, L, R, N, K = 70, 6, 16, 264, 512
    prob = inputs.make_dense(T, N, K, seed=4)
    c = H.run_dense(prob)
    base = c.clone()
    ids = torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    _, order, _, m_indices = fp8.group_rows_by_index(ids, L, torch.empty(L + 1, **i32), torch.empty(T, **i32),
                                                     None, torch.empty(T, **i32))
    x = gen(T, K, seed=5, dtype=BF16)
    A, B = gen(L, R, K, seed=6, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=7, dtype=BF16)
    scales = torch.rand(L, device="cuda") + 0.5
    fp8.m_grouped_lora_add(x, A, B, scales, c, c, m_indices, order)
    assert fp8.get_device_status() == 0
    for g in range(L):
        rows = torch.nonzero(ids == g).flatten()
        if len(rows):
            lora_check(c[rows], x[rows], A[g], B[g], float(scales[g]), base[rows])
    none = torch.nonzero(ids < 0).flatten()
    assert torch.equal(c[none], base[none])


def test_adapter_gradients_from_ragged_products():
    """A fine-tuning step's adapter gradients are three ragged products:
    gv = gy B, gA = gv^T x, gB = gy^T v (scales folded into gy)."""
    counts, R, N, K = [40, 0, 33], 16, 136, 72
    T, L = sum(counts), len(counts)
    ends = np.cumsum([0] + counts)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, gy = gen(T, K, seed=1, dtype=BF16), gen(T, N, seed=2, dtype=BF16)
    A, B = gen(L, R, K, seed=3, dtype=BF16, scale=K ** -0.5), gen(L, N, R, seed=4, dtype=BF16)
    v, gv = torch.empty(T, R, dtype=BF16, device="cuda"), torch.empty(T, R, dtype=BF16, device="cuda")
    gA, gB = torch.empty(L, R, K, device="cuda"), torch.empty(L, N, R, device="cuda")
    fp8.m_grouped_gemm_nt_ragged(x, A, v, offsets)
    fp8.m_grouped_gemm_nn_ragged(gy, B, gv, offsets)
    fp8.k_grouped_gemm_tn_ragged(gv, x, gA, offsets)
    fp8.k_grouped_gemm_tn_ragged(gy, v, gB, offsets)
    for g in range(L):
        r = slice(ends[g], ends[g + 1])
        xd, gd, Ad, Bd = x[r].double(), gy[r].double(), A[g].double(), B[g].double()
        # one BF16 rounding of the middle result: at most 2^-8 of it per term
        for got, ref, mag in ((gA[g], (gd @ Bd).T @ xd, (gd @ Bd).abs().T @ xd.abs()),
                              (gB[g], gd.T @ (xd @ Ad.T), gd.abs().T @ (xd @ Ad.T).abs())):
            assert ((got.double() - ref).abs() <= 2.0 ** -8 * 1.01 * mag + 1e-6 * mag.max().clamp_min(1)).all()
