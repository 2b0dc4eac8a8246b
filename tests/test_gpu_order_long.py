"""The expert order above 1.2 million entries, where a warp's part no longer fits in registers and
is read again, and the order on another stream and in a graph."""
import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


def entries(N, E, k, dropped, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    topk = torch.randint(0, E, (N, k), generator=g, device="cuda", dtype=torch.int32)
    topk[N // 3: N // 2] %= 3  # a stretch that crowds on few experts
    topk[torch.rand(N, k, generator=g, device="cuda") < dropped] = -1
    if dropped:
        topk[5, 0], topk[N - 1, k - 1] = E, -(2 ** 31)
    return topk


def blank(N, E, k):
    return [torch.full(s, -9, dtype=torch.int32, device="cuda") for s in ((E,), (E + 1,), (N, k), (N * k,))]


def matches(out, topk, E):
    return all(np.array_equal(got.cpu().numpy(), want)
               for got, want in zip(out, ref.order(topk.cpu().numpy(), E)))


@pytest.mark.parametrize("dropped", [0.0, 0.2])
@pytest.mark.parametrize("N,E,k", [(400001, 32, 6), (400001, 1024, 6), (524288, 256, 6),
                                   (1300000, 96, 1), (207520, 256, 6), (207600, 256, 6)])
def test_order_of_long_parts(qb, N, E, k, dropped):
    topk = entries(N, E, k, dropped, N + E)
    out, ws = blank(N, E, k), qb.order_workspace(N, E, k).fill_(255)
    qb.qb_expert_order(topk, E, *out, ws)
    assert matches(out, topk, E)


def test_order_on_another_stream_and_in_a_graph(qb):
    N, E, k = 60000, 256, 6
    topk, other = entries(N, E, k, 0.1, 1), entries(N, E, k, 0.3, 2)
    ws = qb.order_workspace(N, E, k)
    out, s = blank(N, E, k), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    qb.qb_expert_order(topk, E, *out, ws, stream=s)
    s.synchronize()
    assert matches(out, topk, E)
    # in a graph with a call before and behind it that use the same memory
    held, chained = topk.clone(), [blank(N, E, k) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.qb_expert_order(held, E, *chained[0], ws)
        held.copy_(other)
        qb.qb_expert_order(held, E, *chained[1], ws)
        held.copy_(topk)
    for _ in range(3):
        for t in chained[0] + chained[1]:
            t.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert matches(chained[0], topk, E) and matches(chained[1], other, E)
