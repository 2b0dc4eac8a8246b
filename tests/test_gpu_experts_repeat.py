"""The experts' products call after call: the pairs' CTAs pass tiles, scales and accumulators to each
other through rings of buffers, and a stale one shows as other bits.  Every K block of every row has
a scale of its own here, the shapes take many rounds of each ring, and the calls overlap with others
that fill the memory system; all must give the bits of the first, which is held against 64 bits."""
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


def operand(rows, K, seed, scale_rows=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = (torch.randn(rows, K, generator=g, device="cuda") * 60).clamp(-448, 448)
    s = torch.randint(112, 130, (-(-rows // scale_rows), ref.pitch(K)), generator=g, device="cuda",
                      dtype=torch.uint8)
    return v.to(torch.float8_e4m3fn), s


def host(q, s, rows=1):
    return ref.value(q.double().cpu().numpy(), s.cpu().numpy(), rows)


def close(got, want, size, K):
    # (S + 24) units of 2^-23 of sum |A| |B|: S additions in the accumulator (64 at most), one for
    # each further 2048 values
    tol = (min(-(-K // 32), 64) + -(-K // 2048) + 24) * 2.0 ** -23 * size
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def repeat(call, out, times):
    call()
    first = out.clone()
    side, big = torch.cuda.Stream(), torch.zeros(1 << 28, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(times // 10):
            big.add_(1.0)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(times):
        out.fill_(float("nan"))
        call()
        same &= (out == first).all()
    side.synchronize()
    assert bool(same)
    return first


@pytest.mark.parametrize("M,G,N,K", [(900, 7, 1032, 4112), (40, 96, 520, 2064), (6000, 3, 2056, 656)])
def test_product_repeats(qb, M, G, N, K):
    a, sa = operand(M, K, 1)
    bs = [operand(N, K, 10 + g, 128) for g in range(G)]
    b, sb = torch.stack([q for q, _ in bs]), torch.stack([s for _, s in bs])
    off = (torch.arange(G + 1, device="cuda") * M // G).to(torch.int32)
    y = torch.empty(M, N, device="cuda")
    first = repeat(lambda: qb.qb_fp8_expert_gemm(a, sa, b, sb, y, offsets=off), y, 100)
    A, o = host(a, sa), off.tolist()
    for g in (0, G - 1):
        B, r = host(b[g], sb[g], 128), slice(o[g], o[g + 1])
        close(first[r], A[r] @ B.T, np.abs(A[r]) @ np.abs(B).T, K)
    assert qb.device_status() == 0


@pytest.mark.parametrize("M,G,N,K", [(20000, 5, 300, 520), (6000, 40, 264, 1032), (9000, 1, 512, 2056)])
def test_weight_gradient_repeats(qb, M, G, N, K):
    n = M // G // 128 * 128  # whole blocks, so that every column is a token
    M = n * G
    a, sa = operand(N, M, 1)
    b, sb = operand(K, M, 2)
    off = (torch.arange(G + 1, device="cuda") * n).to(torch.int32)
    dw = torch.empty(G, N, K, device="cuda")
    first = repeat(lambda: qb.qb_fp8_expert_wgrad(a, sa, b, sb, dw, offsets=off), dw, 100)
    A, B = host(a, sa), host(b, sb)
    for g in (0, G - 1):
        c = slice(g * n, g * n + n)
        close(first[g], A[:, c] @ B[:, c].T, np.abs(A[:, c]) @ np.abs(B[:, c]).T, n)
    assert qb.device_status() == 0
