"""Ragged grouped products against their definition in 64 bits.

Tolerance of one element, derived from the arithmetic: the result is rounded
once (half a step: eps / 2 relative, or half the smallest subnormal), and the
FP32 sum of R products is made of R / 16 tensor-core steps, each off by at most
one step of 2^-23 relative to the sum of magnitudes S, plus the adds inside a
step (counted as 32 more): |gpu - ref| <= eps/2 |ref| + tiny + (R/16 + 32) 2^-23 S.
Over all elements the rounding errors average out below half a step, so the
2-norm of the difference is at most eps / 2 of the result's (FP32 results:
2^-18 of it, the rounding of the sums).
"""

import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8

pytestmark = pytest.mark.gpu

FORMS = {"auto": (0, 0, 0), "swap16": (1, 0, 16), "swap32": (1, 0, 32), "swap64": (1, 0, 64),
         "swap16_by_8": (1, 0, 16, 8), "swap32_by_2": (1, 0, 32, 2), "swap64_by_4": (1, 0, 64, 4), "swap128": (1, 0, 128),
         "single": (0, 0, 256), "pair": (0, 1, 256)}
TN_FORMS = {"auto": (0, 0, 0), "single128": (0, 0, 128), "single256": (0, 0, 256), "pair": (0, 1, 256)}
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32

# rows per group: empty, one, tile edges and beyond
COUNTS = {
    "edges": [0, 1, 31, 32, 33, 0, 127, 128, 129, 255, 256, 257, 64, 65, 0],
    "one_row": [1],
    "all_empty": [0, 0, 0],
    "skewed": [700, 0, 3, 1],
}
TINY = {BF16: 0.0, FP16: 2.0 ** -25, FP32: 0.0}


def gen(*shape, seed, dtype, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def layout(counts, head=0, tail=0):
    """offsets on the device, segment bounds, total rows."""
    ends = [head]
    for c in counts:
        ends.append(ends[-1] + c)
    return torch.tensor(ends, dtype=torch.int32, device="cuda"), ends, ends[-1] + tail


def check(got, ref, mag, reduction):
    eps = torch.finfo(got.dtype).eps
    bound = eps / 2 * ref.abs() + TINY[got.dtype] + (reduction / 16 + 32) * 2.0 ** -23 * mag
    diff = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (diff <= bound).all(), f"worst {(diff / bound.clamp_min(1e-300)).max().item()} of the bound"
    norm = ref.norm()
    if norm > 0 and ref.numel() >= 64:
        assert (got.double() - ref).norm() <= (eps / 2 if got.dtype != FP32 else 2.0 ** -18) * norm


@pytest.fixture
def form():
    yield lambda f: fp8.force_ragged(*f)
    fp8.force_ragged()


def run_rows(direction, counts, N, K, dtype, seed=0, head=3, tail=5):
    """One forward / input-gradient call; rows outside the segments hold NaN."""
    offsets, ends, T = layout(counts, head, tail)
    G = len(counts)
    red, out = (K, N) if direction == "nt" else (N, K)
    a = gen(T, red, seed=seed, dtype=dtype)
    a[:ends[0]] = float("nan")
    a[ends[-1]:] = float("inf")
    b = gen(G, N, K, seed=seed + 1, dtype=dtype, scale=red ** -0.5)
    d = torch.full((T, out), 7.0, dtype=dtype, device="cuda")
    call = fp8.m_grouped_gemm_nt_ragged if direction == "nt" else fp8.m_grouped_gemm_nn_ragged
    assert call(a, b, d, offsets) is d
    for g in range(G):
        rows = slice(ends[g], ends[g + 1])
        if ends[g] == ends[g + 1]:
            continue
        w = b[g].double().T if direction == "nt" else b[g].double()
        check(d[rows], a[rows].double() @ w, a[rows].double().abs() @ w.abs(), red)
    assert (d[:ends[0]] == 7).all() and (d[ends[-1]:] == 7).all()
    assert fp8.get_device_status() == 0
    return a, b, d, offsets


@pytest.mark.parametrize("name", list(FORMS))
@pytest.mark.parametrize("direction", ["nt", "nn"])
@pytest.mark.parametrize("counts", list(COUNTS))
def test_rows_every_form(direction, name, counts, form):
    form(FORMS[name])
    run_rows(direction, COUNTS[counts], 264, 136, BF16)


@pytest.mark.parametrize("split", [1, 2, 4, 8])
@pytest.mark.parametrize("bn", [16, 32, 64])
@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_rows_shared_reductions(direction, bn, split, form):
    """Tiles whose reduction a cluster shares, many tiles per cluster."""
    form((1, 0, bn, split))
    run_rows(direction, [5, 0, 70, 1, 33, 16], 1032, 1160, BF16, seed=split)
    run_rows(direction, [1], 264, 2112, FP16, seed=split)


@pytest.mark.parametrize("direction", ["nt", "nn"])
@pytest.mark.parametrize("N,K", [(8, 8), (8, 520), (520, 8), (72, 64), (2112, 1032), (256, 512)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_rows_sizes(direction, N, K, dtype):
    run_rows(direction, [5, 0, 300, 40], N, K, dtype, seed=N + K)
    run_rows(direction, [2, 1, 0, 9], N, K, dtype, seed=N - K)


@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_rows_many_groups(direction):
    counts = [(i * 7) % 5 for i in range(1024)]
    run_rows(direction, counts, 64, 72, BF16, head=0, tail=0)


@pytest.mark.parametrize("direction", ["nt", "nn"])
def test_rows_model_sizes(direction):
    run_rows(direction, [37, 0, 211, 1, 90, 600, 13, 128], 4096, 7168, BF16, seed=11)


def run_tn(counts, N, K, dtype, out, accumulate=False, seed=0, head=2, tail=9):
    """One weight-gradient call; rows outside the segments hold NaN and Inf."""
    offsets, ends, T = layout(counts, head, tail)
    a, b = gen(T, N, seed=seed, dtype=dtype), gen(T, K, seed=seed + 1, dtype=dtype)
    for t in (a, b):
        t[:ends[0]] = float("inf")
        t[ends[-1]:] = float("nan")
    d = gen(len(counts), N, K, seed=seed + 2, dtype=out)
    start = d.double()
    assert fp8.k_grouped_gemm_tn_ragged(a, b, d, offsets, accumulate=accumulate) is d
    for g in range(len(counts)):
        rows = slice(ends[g], ends[g + 1])
        ref = a[rows].double().T @ b[rows].double()
        mag = a[rows].double().abs().T @ b[rows].double().abs()
        if accumulate:
            ref, mag = ref + start[g], mag + start[g].abs()
        check(d[g], ref, mag, counts[g])
        if counts[g] == 0 and not accumulate:
            assert (d[g] == 0).all()
    assert fp8.get_device_status() == 0
    return a, b, d, offsets


@pytest.mark.parametrize("name", list(TN_FORMS))
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("out,accumulate", [(FP32, False), (FP32, True), (BF16, False)])
def test_tn_every_form(name, counts, out, accumulate, form):
    form(TN_FORMS[name])
    run_tn(COUNTS[counts], 264, 392, BF16, out, accumulate)


@pytest.mark.parametrize("N,K", [(8, 8), (8, 520), (520, 8), (72, 264), (1032, 2112)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_tn_sizes(N, K, dtype):
    run_tn([5, 0, 300, 40], N, K, dtype, dtype, seed=N + K)
    run_tn([5, 0, 300, 40], N, K, dtype, FP32, seed=N - K)


@pytest.mark.parametrize("name", list(TN_FORMS))
@pytest.mark.parametrize("rows", [256, 2049, 20000])
def test_tn_long_sums_in_fp32(name, rows, form):
    """FP32 results hold their accuracy over long segments: a partial sum of 512
    rows is 32 truncated steps, each off by half a step of 2^-23 of the sum so far
    on average (so 32 / 2 * 2/3 * 2^-23 of the whole, 1.3e-6 at the very most and
    half of that with the mantissas' spread), the errors of the partial sums add
    up as the sums themselves do: within 2^-20 of the result."""
    form(TN_FORMS[name])
    offsets, ends, T = layout([rows, 3])
    a, b = gen(T, 256, seed=1, dtype=BF16), gen(T, 264, seed=2, dtype=BF16)
    d = torch.empty(2, 256, 264, dtype=FP32, device="cuda")
    fp8.k_grouped_gemm_tn_ragged(a, b, d, offsets)
    ref = a[:rows].double().T @ b[:rows].double()
    assert (d[0].double() - ref).norm() <= 2.0 ** -20 * ref.norm()


def test_tn_neighbours_do_not_leak():
    """A segment's last block reads the next segment's rows: Inf there stays there."""
    counts = [17, 30, 1, 64, 63]
    offsets, ends, T = layout(counts)
    a, b = gen(T, 256, seed=1, dtype=BF16), gen(T, 256, seed=2, dtype=BF16)
    a[ends[1]:ends[2]] = float("inf")
    b[ends[1]:ends[2]] = float("nan")
    d = torch.empty(5, 256, 256, dtype=FP32, device="cuda")
    fp8.k_grouped_gemm_tn_ragged(a, b, d, offsets)
    assert not torch.isfinite(d[1]).any()
    for g in (0, 2, 3, 4):
        rows = slice(ends[g], ends[g + 1])
        check(d[g], a[rows].double().T @ b[rows].double(), a[rows].double().abs().T @ b[rows].double().abs(), counts[g])


def test_special_values_reach_their_rows_only():
    """Inf and NaN of a token or of a weight appear where the product has them."""
    offsets, ends, T = layout([40, 3, 70])
    a, b = gen(T, 128, seed=3, dtype=BF16), gen(3, 136, 128, seed=4, dtype=BF16)
    a[5, 7] = float("nan")
    a[41, 0] = float("inf")
    b[2, 9, 3] = float("inf")
    for f in (FORMS["swap64"], FORMS["pair"]):
        try:
            fp8.force_ragged(*f)
            d = torch.empty(T, 136, dtype=BF16, device="cuda")
            fp8.m_grouped_gemm_nt_ragged(a, b, d, offsets)
        finally:
            fp8.force_ragged(0, 0, 0)
        bad = ~torch.isfinite(d)
        want = torch.zeros_like(bad)
        want[5] = want[41] = True
        want[43:, 9] = True
        assert torch.equal(bad, want)


def test_bad_offsets_are_flagged_and_clamped():
    a, b = gen(64, 128, seed=5, dtype=BF16), gen(3, 128, 128, seed=6, dtype=BF16)
    d = torch.full((64, 128), 7.0, dtype=BF16, device="cuda")
    fp8.m_grouped_gemm_nt_ragged(a, b, d, torch.tensor([-4, 20, 10, 900], dtype=torch.int32, device="cuda"))
    assert fp8.get_device_status() == 7
    # group 0: rows 0..19; group 1: empty (its end lies before its start); group 2: rows 20..63
    ref = a[20:].double() @ b[2].double().T
    check(d[20:], ref, a[20:].double().abs() @ b[2].double().abs().T, 128)
    g = torch.full((3, 128, 128), 7.0, dtype=FP32, device="cuda")
    fp8.k_grouped_gemm_tn_ragged(a, a, g, torch.tensor([0, 30, 30, 65], dtype=torch.int32, device="cuda"))
    assert fp8.get_device_status() == 7
    check(g[2], a[30:].double().T @ a[30:].double(), a[30:].double().abs().T @ a[30:].double().abs(), 34)


def test_bad_offsets_do_not_overlap():
    a, b = gen(128, 64, seed=7, dtype=BF16), gen(4, 64, 64, seed=8, dtype=BF16)
    offsets = torch.tensor([0, 100, 40, 120, 90], dtype=torch.int32, device="cuda")
    d = torch.full((128, 64), 7.0, dtype=BF16, device="cuda")
    w = torch.full((4, 64, 64), 7.0, dtype=FP32, device="cuda")
    bounds = [(0, 100), (100, 100), (100, 120), (120, 120)]
    fp8.m_grouped_gemm_nt_ragged(a, b, d, offsets)
    assert fp8.get_device_status() == 7
    for g, (lo, hi) in enumerate(bounds):
        check(d[lo:hi], a[lo:hi].double() @ b[g].double().T, a[lo:hi].double().abs() @ b[g].double().abs().T, 64)
    assert (d[120:] == 7).all()
    fp8.k_grouped_gemm_tn_ragged(a, a, w, offsets)
    assert fp8.get_device_status() == 7
    for g, (lo, hi) in enumerate(bounds):
        x = a[lo:hi].double()
        check(w[g], x.T @ x, x.abs().T @ x.abs(), hi - lo)


def test_no_rows():
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    a, b, d = (torch.empty(0, 64, dtype=BF16, device="cuda"), gen(2, 64, 64, seed=1, dtype=BF16),
               torch.empty(0, 64, dtype=BF16, device="cuda"))
    fp8.m_grouped_gemm_nt_ragged(a, b, d, offsets)
    fp8.m_grouped_gemm_nn_ragged(a, b, d, offsets)
    w = torch.full((2, 64, 64), 7.0, dtype=FP32, device="cuda")
    fp8.k_grouped_gemm_tn_ragged(a, d, w, offsets, accumulate=True)
    assert (w == 7).all()
    fp8.k_grouped_gemm_tn_ragged(a, d, w, offsets)
    assert (w == 0).all()


def test_gradients_are_those_of_the_forward():
    """<gy, f(x + h u)> against the input and weight gradients, by differences.

    f is bilinear, so a central difference in 64 bits has no truncation error:
    it equals <gx, u> of the definition; the call's gx is off by its own
    rounding (eps / 2 of each element, so at most eps / 2 |gx| |u| in the sum).
    """
    counts = [33, 0, 70, 1]
    offsets, ends, T = layout(counts)
    N, K = 136, 72
    x, w = gen(T, K, seed=1, dtype=BF16), gen(4, N, K, seed=2, dtype=BF16)
    gy, u = gen(T, N, seed=3, dtype=BF16), gen(T, K, seed=4, dtype=torch.float64)
    uw = gen(4, N, K, seed=5, dtype=torch.float64)

    def f(xx, ww):
        y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for g in range(4):
            y[ends[g]:ends[g + 1]] = xx[ends[g]:ends[g + 1]] @ ww[g].T
        return (y * gy.double()).sum()

    gx, gw = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(4, N, K, dtype=FP32, device="cuda")
    fp8.m_grouped_gemm_nn_ragged(gy, w, gx, offsets)
    fp8.k_grouped_gemm_tn_ragged(gy, x, gw, offsets)
    h, xd, wd = 0.5, x.double(), w.double()
    num = (f(xd + h * u, wd) - f(xd - h * u, wd)) / (2 * h)
    assert (num - (gx.double() * u).sum()).abs() <= 2.0 ** -8 * (gx.double().abs() * u.abs()).sum()
    num = (f(xd, wd + h * uw) - f(xd, wd - h * uw)) / (2 * h)
    assert (num - (gw.double() * uw).sum()).abs() <= 2.0 ** -18 * (gw.double().abs() * uw.abs()).sum()


def test_graph_replay_and_other_stream():
    """A captured forward and backward read the segments at replay; a call on
    another stream than the current one runs there."""
    counts, N, K = [40, 0, 90, 20], 264, 136
    offsets, ends, T = layout(counts)
    x, w, gy = gen(T, K, seed=1, dtype=BF16), gen(4, N, K, seed=2, dtype=BF16), gen(T, N, seed=3, dtype=BF16)
    y, gx = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, K, dtype=BF16, device="cuda")
    gw = torch.zeros(4, N, K, dtype=FP32, device="cuda")

    def step():
        fp8.m_grouped_gemm_nt_ragged(x, w, y, offsets)
        fp8.m_grouped_gemm_nn_ragged(gy, w, gx, offsets)
        fp8.k_grouped_gemm_tn_ragged(gy, x, gw, offsets)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    offsets.copy_(torch.tensor([0, 0, 100, 101, 150], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (y, gx, gw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (y, gx, gw):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    fp8.m_grouped_gemm_nt_ragged(x, w, y, offsets, stream=side)
    fp8.m_grouped_gemm_nn_ragged(gy, w, gx, offsets, stream=side)
    fp8.k_grouped_gemm_tn_ragged(gy, x, gw, offsets, stream=side)
    side.synchronize()
    for a, b in zip(got, (y, gx, gw)):
        assert torch.equal(a, b)
    for g, (lo, hi) in enumerate([(0, 0), (0, 100), (100, 101), (101, 150)]):
        check(y[lo:hi], x[lo:hi].double() @ w[g].double().T, x[lo:hi].double().abs() @ w[g].double().abs().T, K)


def test_repeated_calls_are_bit_equal():
    counts = [300, 17, 0, 513]
    offsets, ends, T = layout(counts)
    a, b = gen(T, 520, seed=1, dtype=BF16), gen(T, 264, seed=2, dtype=BF16)
    first = None
    for _ in range(3):
        d = torch.zeros(4, 520, 264, dtype=FP32, device="cuda")
        fp8.k_grouped_gemm_tn_ragged(a, b, d, offsets, accumulate=True)
        first = d if first is None else first
        assert torch.equal(d, first)


@pytest.mark.parametrize("sms", [1, 2, 3])
def test_sm_bound(sms):
    try:
        fp8.set_num_sms(sms)
        run_rows("nt", [30, 400, 0, 200], 520, 136, BF16)
        run_tn([30, 400, 0, 200], 520, 264, BF16, FP32)
    finally:
        fp8.set_num_sms(0)


def test_results_beyond_2_to_31_elements():
    """Rows and groups whose offset in the result does not fit 32 bits."""
    T, N, K = 70001, 32768, 8
    a, b = gen(T, K, seed=1, dtype=BF16), gen(2, N, K, seed=2, dtype=BF16)
    offsets = torch.tensor([0, 35000, T - 1], dtype=torch.int32, device="cuda")
    d = torch.zeros(T, N, dtype=BF16, device="cuda")
    fp8.m_grouped_gemm_nt_ragged(a, b, d, offsets)
    for rows, g in ((slice(0, 40), 0), (slice(34990, 35000), 0), (slice(35000, 35010), 1), (slice(T - 30, T - 1), 1)):
        w = b[g].double().T
        check(d[rows], a[rows].double() @ w, a[rows].double().abs() @ w.abs(), K)
    assert (d[T - 1] == 0).all()
    del d
    G, N, K = 40, 8192, 8192
    offsets = torch.arange(G + 1, dtype=torch.int32, device="cuda") * 3
    a, b = gen(3 * G, N, seed=3, dtype=BF16), gen(3 * G, K, seed=4, dtype=BF16)
    d = torch.empty(G, N, K, dtype=BF16, device="cuda")
    fp8.k_grouped_gemm_tn_ragged(a, b, d, offsets)
    for g in (0, 31, 32, G - 1):
        x, y = a[3 * g:3 * g + 3].double(), b[3 * g:3 * g + 3].double()
        check(d[g, -64:], (x.T @ y)[-64:], (x.abs().T @ y.abs())[-64:], 3)


def test_refusals_of_device_tensors():
    a, b, d = gen(8, 64, seed=1, dtype=BF16), gen(2, 64, 64, seed=2, dtype=BF16), gen(8, 64, seed=3, dtype=BF16)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for bad in ((a.float(), b, d, off), (a, b.half(), d, off), (a, b, d.float(), off), (a, b, d, off.long())):
        with pytest.raises(TypeError):
            fp8.m_grouped_gemm_nt_ragged(*bad)
    for bad in ((a.t().contiguous().t(), b, d, off), (a, b.transpose(1, 2), d, off), (a, b, d, off.cpu()),
                (a, b, d, off[:2]), (a[:4], b, d, off), (a, b[0], d, off)):
        with pytest.raises(ValueError):
            fp8.m_grouped_gemm_nt_ragged(*bad)
    wide = gen(8 * 64 + 4, seed=4, dtype=BF16)
    with pytest.raises(fp8.Fp8NtError) as e:   # 8 bytes off a 16-byte boundary
        fp8.m_grouped_gemm_nt_ragged(wide[4:].view(8, 64), b, d, off)
    assert e.value.status == 2
    with pytest.raises(fp8.Fp8NtError) as e:
        fp8.m_grouped_gemm_nt_ragged(a[:, :4].contiguous(), b[:, :, :4].contiguous(), d, off)
    assert e.value.status == 3
    w = gen(2, 64, 64, seed=5, dtype=BF16)
    with pytest.raises(TypeError):
        fp8.k_grouped_gemm_tn_ragged(a, d, w, off, accumulate=True)
    with pytest.raises(TypeError):
        fp8.k_grouped_gemm_tn_ragged(a, d, w.half(), off)
    assert fp8.get_device_status() == 0


def test_error_of_an_argument_itself():
    a, w = gen(16, 64, seed=1, dtype=BF16), torch.zeros(1, 64, 64, device="cuda")
    offsets = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        fp8.k_grouped_gemm_tn_ragged(a, a, w, offsets, accumulate=torch.zeros(2))
