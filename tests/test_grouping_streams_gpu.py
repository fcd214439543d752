"""Calls of group_rows_by_index that run at the same time, from streams and from
captured graphs, each with a workspace of its own; and one whose index is
written just before it."""

import numpy as np
import pytest
import torch

import fp8_fine_grained_nt_b200 as fp8
from tests.test_grouping_lora_gpu import group_reference

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def results(R, G):
    return (torch.full((G + 1,), 9, **I32), torch.full((R,), 9, **I32), torch.full((R,), 9, **I32),
            torch.full((R,), 9, **I32))


def same(out, want):
    return all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(out, want))


@pytest.mark.parametrize("R,G", [(1000, 64), (100000, 1024)])
def test_streams_and_graphs_at_the_same_time(R, G):
    rng = np.random.default_rng(R)
    index = [rng.integers(-1, G, R) for _ in range(4)]
    want = [group_reference(i, G, 1) for i in index]
    idx = [torch.as_tensor(i, device="cuda") for i in index]
    out = [results(R, G) for _ in index]
    graphs = []
    for i in range(2):
        fp8.group_rows_by_index(idx[i], G, *out[i])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fp8.group_rows_by_index(idx[i], G, *out[i])
        graphs.append(graph)
    for o in out:
        for t in o:
            t.fill_(9)
    streams = [torch.cuda.Stream() for _ in index]
    torch.cuda.synchronize()
    for _ in range(30):
        for i, s in enumerate(streams):
            if i < 2:
                with torch.cuda.stream(s):
                    graphs[i].replay()
            else:
                fp8.group_rows_by_index(idx[i], G, *out[i], stream=s)
    torch.cuda.synchronize()
    assert all(same(o, w) for o, w in zip(out, want))
    assert fp8.get_device_status() == 0


@pytest.mark.parametrize("R,G", [(1000, 64), (100000, 64)])
def test_index_written_right_before(R, G):
    """The index comes from the kernel before, again and again."""
    rng = np.random.default_rng(R)
    index = [rng.integers(-1, G, R) for _ in range(6)]
    src = [torch.as_tensor(i, device="cuda") for i in index]
    idx, outs = torch.empty_like(src[0]), []
    for s in src * 3:
        idx.copy_(s)
        outs.append(results(R, G))
        fp8.group_rows_by_index(idx, G, *outs[-1])
    for o, i in zip(outs, index * 3):
        assert same(o, group_reference(i, G, 1))
    slot = torch.empty(R, **I32)   # the slots of one call are the index of the next
    for i in range(len(src)):
        fp8.group_rows_by_index(src[i], G, *results(R, G)[:2], slot)
        part = slot // (R // G + 1)
        out = results(R, G)
        fp8.group_rows_by_index(part, G, *out)
        assert same(out, group_reference(part.cpu().numpy(), G, 1))
