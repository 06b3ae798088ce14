"""Counts that a kernel has just written are the next call's lengths, read before that call waits: eager, through the
moves of rows, and in a graph, with other lengths in the same memory each time."""
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_score_mod import cache_of
from test_gpu_tree import cumulative, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("move", [False, True])
@pytest.mark.parametrize("rows", [3, 40])
def test_counts_of_a_selection(rows, move):
    pk = require_gpu()
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(1, 700, (rows,), generator=g).tolist()
    kc, vc, tables, _ = cache_of(lens, 2, 64, 16, torch.bfloat16, 1)
    kc.nan_to_num_(), vc.nan_to_num_()
    q = torch.randn(rows, 8, 64, generator=g).to(torch.bfloat16).to(DEV)
    ctx, w = ints(lens), torch.rand(rows, 2, max(lens), generator=g).to(DEV)
    k2, v2 = kc.clone(), vc.clone()
    ws = torch.empty(pk.decode_workspace_bytes(rows, 8, 64, 700), dtype=torch.uint8, device=DEV)
    keeps = [int(x) for x in torch.randint(1, 700, (60,), generator=g)]

    def step(keep, wait):
        pos, counts = pk.evict_select(w, ctx, keep, sink=1 if keep > 1 else 0)
        if move:
            pk.compact_cache(k2, v2, tables, pos, counts)
        if wait:
            torch.cuda.synchronize()
        return pk.paged_decode_attention(q, k2, v2, tables, counts, 700, 0.1, workspace=ws)

    outs = []
    for wait in (True, False):
        got = []
        for keep in keeps:
            k2.copy_(kc), v2.copy_(vc)
            got.append(step(keep, wait))
        outs.append(got)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert len({tuple(x.flatten()[:4].tolist()) for x in outs[0]}) > 10

    keep = 77
    graph = torch.cuda.CUDAGraph()
    step(keep, False)
    with torch.cuda.graph(graph):
        out = step(keep, False)
    for seed in range(10):                                   # other lengths, so other counts, in the graph's memory
        g.manual_seed(seed)
        now = torch.tensor([int(torch.randint(0, n + 1, (1,), generator=g)) for n in lens], dtype=torch.int32)
        ctx.copy_(now)
        k2.copy_(kc), v2.copy_(vc)
        graph.replay()
        got = out.clone()
        k2.copy_(kc), v2.copy_(vc)
        assert torch.equal(got, step(keep, True))


def test_counts_of_accepted_paths():
    """Paths of 0 to 31 nodes as lengths of a decode call."""
    pk = require_gpu()
    g = torch.Generator().manual_seed(5)
    n, most = 64, 31
    kc, vc, tables, _ = cache_of([32] * n, 2, 64, 16, torch.float32, 2)
    q = torch.randn(n, 4, 64, generator=g).to(DEV)
    chain = ints(list(range(-1, most - 1)) * n)
    cu = cumulative([most] * n)
    ws = torch.empty(pk.decode_workspace_bytes(n, 4, 64, 32), dtype=torch.uint8, device=DEV)
    cases = []
    for seed in range(40):
        g.manual_seed(seed)
        drafted = torch.randint(0, 9, (n, most), generator=g, dtype=torch.int32)
        target = torch.cat((drafted[:, 1:], drafted[:, :1]), 1)
        target[torch.rand(n, most, generator=g) < 0.1] = 99
        cases.append((drafted.flatten().to(DEV), target.flatten().to(DEV)))
    outs = []
    for wait in (True, False):
        got = []
        for drafted, target in cases:
            _, _, counts, _ = pk.tree_accept(drafted, chain, target, cu, cu, most)
            if wait:
                torch.cuda.synchronize()
            got.append(pk.paged_decode_attention(q, kc, vc, tables, counts, 32, 0.1, workspace=ws))
        outs.append(got)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert not torch.equal(outs[0][0], outs[0][1])
