"""Workloads of the row-grouped operators, in plain torch and through the library.

Operators
---------
group      group_rows_by_index: rows sorted (stably) by the group each belongs
           to, with segment offsets, the permutation both ways, and the group
           of every slot; segments start at multiples of `align`.
nt         m_grouped_gemm_nt_ragged: d[t] = a[t] . b[g]^T for the rows t of
           group g's segment, segments of any length (experts' products).
nn         m_grouped_gemm_nn_ragged: d[t] = a[t] . b[g] (their input gradient).
tn         k_grouped_gemm_tn_ragged: d[g] = a[segment g]^T . b[segment g]
           (their weight gradient).
lora       m_grouped_lora_add: d[t] = c[t] + s_g (x[t] . A_g^T) . B_g^T, row t
           using its request's adapter g, beside a shared projection c.

`own` selects the library's calls; otherwise `run` is the plain form.  Sizes
(N, K) follow the library's own workloads: (4096, 7168), (7168, 2048) and
(2112, 7168), with odd and small ones beside them.
"""

import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # decode step: 64 tokens, 8 experts each of 256, exact segments
        dict(name="group_decode", op="group", rows=512, groups=256, align=1, bits=64, empty=0.0, mix=0),
        # prefill: 32768 tokens x 8 choices, half of the experts on this
        # rank (the others' rows have no group here), 128-aligned segments as
        # the contiguous grouped GEMM reads them
        dict(name="group_prefill", op="group", rows=262144, groups=64, align=128, bits=64, empty=0.5, mix=1),
        # decode: 128 rows over 16 experts, some of them empty
        dict(name="nt_decode", op="nt", T=128, G=16, N=4096, K=7168, dtype="bf16", dist="uniform", tail=0, mix=2),
        # odd sizes, FP16, skewed load, rows behind the last segment
        dict(name="nt_odd", op="nt", T=2999, G=64, N=2112, K=1032, dtype="fp16", dist="zipf", tail=37, mix=3),
        # prefill / training forward, 8 experts with U{1..8192} rows
        dict(name="nt_prefill", op="nt", T=32768, G=8, N=4096, K=7168, dtype="bf16", dist="uniform", tail=0, mix=4),
        # input gradient of a small batch with many experts
        dict(name="nn_small", op="nn", T=1000, G=64, N=2112, K=2048, dtype="fp16", dist="uniform", tail=5, mix=5),
        # input gradient of a training step
        dict(name="nn_train", op="nn", T=16384, G=8, N=7168, K=2048, dtype="bf16", dist="uniform", tail=0, mix=6),
        # weight gradient, small skewed batch with empty experts, 16-bit result
        dict(name="tn_small", op="tn", T=1999, G=64, N=2048, K=520, dtype="bf16", out="bf16", dist="zipf", tail=11, mix=7),
        # weight gradient of a training step into FP32
        dict(name="tn_train", op="tn", T=16384, G=8, N=7168, K=2048, dtype="bf16", out="fp32", dist="uniform", tail=0, mix=8),
        # one token of one request
        dict(name="lora_one", op="lora", T=1, L=4, R=16, N=2112, K=7168, dtype="bf16", none=0.0, mix=9),
        # decode batch: 64 rows of up to 32 adapters, some without one
        dict(name="lora_decode", op="lora", T=64, L=32, R=16, N=7168, K=2048, dtype="bf16", none=0.1, mix=10),
        # prefill of several requests
        dict(name="lora_prefill", op="lora", T=4096, L=8, R=64, N=4096, K=7168, dtype="bf16", none=0.0, mix=11),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["group", "nt", "nn", "tn", "lora"])
    mix = rng.randrange(1 << 20)
    if op == "group":
        return dict(op=op, rows=_log(rng, 1, 262144), groups=_log(rng, 1, 512), align=rng.choice([1, 128]),
                    bits=rng.choice([32, 64]), empty=rng.choice([0.0, 0.1, 0.7]), mix=mix)
    if op == "lora":
        return dict(op=op, T=_log(rng, 1, 4096), L=_log(rng, 1, 64), R=rng.choice([8, 16, 24, 32, 64]),
                    N=8 * _log(rng, 16, 512), K=8 * _log(rng, 16, 896),
                    dtype=rng.choice(["bf16", "bf16", "fp16"]), none=rng.choice([0.0, 0.2]), mix=mix)
    case = dict(op=op, T=_log(rng, 1, 16384), G=_log(rng, 1, 64), N=8 * _log(rng, 8, 896),
                K=8 * _log(rng, 8, 896), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                dist=rng.choice(["uniform", "zipf", "even"]), tail=rng.choice([0, 0, 1, 77]), mix=mix)
    if op == "tn":
        case["out"] = rng.choice(["fp32", case["dtype"]])
    while case["T"] * case["N"] * case["K"] > 16384 * 7168 * 2048 and case["T"] > 1:
        case["T"] = case["T"] * 2 // 3
    while case["G"] * case["N"] * case["K"] > 16 * 4096 * 7168:
        case["G"] = case["G"] * 2 // 3
    return case


def _counts(case):
    """Rows of each group: a property of the case, not of the seed."""
    T, G = case["T"], case["G"]
    rng = random.Random(case["mix"])
    if case["dist"] == "even":
        share = [1.0] * G
    elif case["dist"] == "zipf":
        share = [1.0 / (i + 1) ** 1.2 for i in range(G)]
        rng.shuffle(share)
    else:
        share = [rng.random() for _ in range(G)]
    total = sum(share)
    counts = [int(T * s / total) for s in share]
    counts[max(range(G), key=lambda g: share[g])] += T - sum(counts)
    return counts


def _adapters(case):
    """Adapter of each row (-1: none), prefill-like runs for long batches."""
    rng = random.Random(case["mix"])
    T, L = case["T"], case["L"]
    pick = lambda: -1 if rng.random() < case["none"] else rng.randrange(L)  # noqa: E731
    if T <= 256:
        return [pick() for _ in range(T)]
    cuts = sorted(rng.randrange(T) for _ in range(2 * L))
    ids, at = [], 0
    for end in cuts + [T]:
        ids += [pick()] * (end - at)
        at = end
    return ids


# ------------------------------------------------------------------ the state


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    st = dict(case=case, op=case["op"])
    if case["op"] == "group":
        R, G, al = case["rows"], case["groups"], case["align"]
        # a router's choices are uneven over the experts
        load = torch.rand(G, generator=gen, device="cuda") ** 2 + 1e-3
        idx = torch.multinomial(load, R, replacement=True, generator=gen)
        if case["empty"]:
            idx[torch.rand(R, generator=gen, device="cuda") < case["empty"]] = -1
        cap = R + min(R, G) * (al - 1)
        cap = (cap + al - 1) // al * al
        i32 = dict(dtype=torch.int32, device="cuda")
        st.update(index=idx.to(torch.int32 if case["bits"] == 32 else torch.int64), groups=G, align=al,
                  offsets=torch.empty(G + 1, **i32), order=torch.empty(cap, **i32),
                  slots=torch.empty(R, **i32), m_indices=torch.empty(cap, **i32))
        return st
    dt = DTYPES[case["dtype"]]
    N, K = case["N"], case["K"]
    if case["op"] == "lora":
        T, L, R = case["T"], case["L"], case["R"]
        ids = np.array(_adapters(case), dtype=np.int64)
        order = np.argsort(np.where(ids < 0, L, ids), kind="stable")
        order = order[: int((ids >= 0).sum())]
        st.update(x=rnd(T, K).to(dt), lora_a=(rnd(L, R, K) / K ** 0.5).to(dt), lora_b=(rnd(L, N, R) / R ** 0.5).to(dt),
                  scales=torch.rand(L, generator=gen, device="cuda") + 0.5, c=rnd(T, N).to(dt),
                  order=torch.from_numpy(order.astype(np.int32)).cuda(),
                  m_indices=torch.from_numpy(ids[order].astype(np.int32)).cuda())
        st["d"] = st["c"].clone()
        return st
    counts, T, G = _counts(case), case["T"] + case["tail"], case["G"]
    ends = np.cumsum([0] + counts)
    st.update(offsets=torch.from_numpy(ends.astype(np.int32)).cuda(), most=max(counts))
    weights = lambda: rnd(G, N, K).mul_(K ** -0.5).to(dt)  # noqa: E731
    if case["op"] == "nt":
        st.update(a=rnd(T, K).to(dt), b=weights(), d=torch.ones(T, N, dtype=dt, device="cuda"))
    elif case["op"] == "nn":
        st.update(a=rnd(T, N).to(dt), b=weights(), d=torch.ones(T, K, dtype=dt, device="cuda"))
    else:
        st.update(a=rnd(T, N).to(dt), b=rnd(T, K).to(dt),
                  d=torch.empty(G, N, K, dtype=DTYPES[case["out"]], device="cuda"))
    return st


# ------------------------------------------------------------------ one pass


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "group":
        return _plain_group(st)
    if op == "lora":
        return _plain_lora(st)
    return _plain_grouped(st, op)


def _run_own(st):
    import fp8_fine_grained_nt_b200 as fp8
    op = st["op"]
    if op == "group":
        return fp8.group_rows_by_index(st["index"], st["groups"], st["offsets"], st["order"], st["slots"],
                                       st["m_indices"], alignment=st["align"])
    if op == "nt":
        return fp8.m_grouped_gemm_nt_ragged(st["a"], st["b"], st["d"], st["offsets"])
    if op == "nn":
        return fp8.m_grouped_gemm_nn_ragged(st["a"], st["b"], st["d"], st["offsets"])
    if op == "tn":
        return fp8.k_grouped_gemm_tn_ragged(st["a"], st["b"], st["d"], st["offsets"])
    return fp8.m_grouped_lora_add(st["x"], st["lora_a"], st["lora_b"], st["scales"], st["c"], st["d"],
                                  st["m_indices"], st["order"])


def _plain_group(st):
    idx, G, al = st["index"], st["groups"], st["align"]
    R, cap = idx.numel(), st["order"].numel()
    groups = torch.arange(G, device=idx.device)
    ok = (idx >= 0) & (idx < G)
    key = torch.where(ok, idx, G)
    perm = torch.argsort(key, stable=True)
    key = key[perm]
    counts = torch.zeros(G + 1, dtype=torch.int64, device=idx.device).scatter_add_(0, key, torch.ones_like(key))
    first = counts.cumsum(0) - counts
    padded = (counts[:G] + al - 1) // al * al
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    at = torch.arange(R, device=idx.device) - first[key] + offsets[key]
    at = torch.where(key < G, at, cap)  # rows without a group: one place past the end
    order = torch.full((cap + 1,), -1, dtype=torch.int32, device=idx.device)
    order[at] = perm.to(torch.int32)
    m_indices = torch.full((cap + 1,), -1, dtype=torch.int32, device=idx.device)
    m_indices[at] = groups.to(torch.int32)[key.clamp(max=G - 1)]
    slots = torch.empty(R, dtype=torch.int32, device=idx.device)
    slots[perm] = torch.where(key < G, at, -1).to(torch.int32)
    return offsets.to(torch.int32), order[:cap], slots, m_indices[:cap]


def _segments(st):
    """Every group's rows, padded to the longest group: (row numbers, which are real)."""
    off = st["offsets"].long()
    row = off[:-1, None] + torch.arange(st["most"], device=off.device)
    real = row < off[1:, None]
    return torch.where(real, row, 0), real


def _plain_grouped(st, op):
    a, b, off = st["a"], st["b"], st["offsets"].long()
    row, real = _segments(st)
    a_pad = a.float()[row] * real[..., None]
    if op == "tn":
        return torch.bmm(a_pad.transpose(1, 2), b.float()[row] * real[..., None]).to(st["d"].dtype)
    w = b.float()
    prod = torch.bmm(a_pad, w.transpose(1, 2) if op == "nt" else w)
    t = torch.arange(a.shape[0], device=a.device)
    g = (torch.searchsorted(off, t, right=True) - 1).clamp(max=off.numel() - 2)
    inside = t < off[-1]
    mine = prod[g, torch.where(inside, t - off[g], 0)].to(st["d"].dtype)
    return torch.where(inside[:, None], mine, st["d"])


def _plain_lora(st):
    # every row with every adapter it could have, by one masked product per
    # factor: the down-projections of all adapters side by side, the ones a row
    # does not use set to zero, then all up-projections at once
    x, A, B, rows, g = st["x"], st["lora_a"], st["lora_b"], st["order"].long(), st["m_indices"].long()
    L, R, K = A.shape
    v = x[rows].float() @ A.float().reshape(L * R, K).t()
    mine = torch.arange(L, device=x.device) == g[:, None]
    v = torch.where(mine[..., None], v.view(-1, L, R), 0.0) * st["scales"][:, None]
    up = v.reshape(-1, L * R) @ B.float().transpose(1, 2).reshape(L * R, -1)
    d = st["d"]
    d[rows] = (st["c"][rows].float() + up).to(d.dtype)
    return d


# ------------------------------------------------------------------ what it takes


def work(case):
    if case["op"] == "group":
        R, G, al = case["rows"], case["groups"], case["align"]
        cap = -(-(R + min(R, G) * (al - 1)) // al) * al
        return {"bytes": R * case["bits"] // 8 + 4 * (G + 1 + 2 * cap + R), "flops": 0}
    N, K = case["N"], case["K"]
    if case["op"] == "lora":
        ids = [i for i in _adapters(case) if i >= 0]
        T, R, used = len(ids), case["R"], len(set(ids))
        return {"bytes": 2 * T * (K + 2 * N) + 2 * used * R * (K + N) + 8 * T + 4 * used,
                "flops": 2 * T * R * (K + N)}
    counts = _counts(case)
    T, used, G = sum(counts), sum(c > 0 for c in counts), case["G"]
    if case["op"] == "tn":
        size = 4 if case["out"] == "fp32" else 2
        moved = 2 * T * (N + K) + size * G * N * K
    else:
        moved = 2 * T * (N + K) + 2 * used * N * K
    return {"bytes": moved + 4 * (G + 1), "flops": 2 * T * N * K}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    if case["op"] == "group":
        return None  # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "lora":
        d = st["c"].double()
        rows, g = st["order"].cpu().numpy(), st["m_indices"].cpu().numpy()
        for adapter in np.unique(g):
            r = torch.from_numpy(rows[g == adapter].astype(np.int64)).cuda()
            low = st["x"][r].double() @ st["lora_a"][adapter].double().T
            d[r] += float(st["scales"][adapter]) * (low @ st["lora_b"][adapter].double().T)
        return d
    ends = st["offsets"].tolist()
    d = st["d"].double() if case["op"] != "tn" else torch.zeros(st["d"].shape, dtype=torch.float64, device="cuda")
    for g in range(case["G"]):
        rows = slice(ends[g], ends[g + 1])
        if rows.start == rows.stop:
            continue
        left = st["a"][rows].double()
        if case["op"] == "tn":
            d[g] = left.T @ st["b"][rows].double()
        else:
            w = st["b"][g].double()
            d[rows] = left @ (w.T if case["op"] == "nt" else w)
    return d
