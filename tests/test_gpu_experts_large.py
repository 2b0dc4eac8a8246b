"""The quantisers and the weight gradient on another stream, in a graph, and past 2^31 elements."""
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


def source(T, K, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(T, K, generator=g, device="cuda")
    return (x * torch.exp(2.0 * torch.randn(T, 1, generator=g, device="cuda"))).to(torch.bfloat16)


def blank(*shape):
    return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")


def codes_equal(q, want):
    return np.array_equal(q.view(torch.float8_e4m3fn).double().cpu().numpy(), want, equal_nan=True)


def test_quantisers_and_weight_gradient_on_another_stream_and_in_a_graph(qb):
    M, G, N, K = 900, 5, 208, 336
    a, b = source(M, N, 1), source(M, K, 2)
    w = source(G * N, K, 3).view(G, N, K)
    off = torch.tensor([0, 100, 100, 333, 700, M], dtype=torch.int32, device="cuda")
    width = qb.fp8_cols_width(M, G)
    out = dict(r=blank(M, K), rs=blank(M, ref.pitch(K)), at=blank(N, width), bt=blank(K, width),
               ats=blank(N, ref.pitch(width)), bts=blank(K, ref.pitch(width)), q=blank(G, N, K),
               qs=blank(G, 2, ref.pitch(K)), qt=blank(G, K, N), qts=blank(G, 3, ref.pitch(N)),
               dw=torch.full((G, N, K), float("nan"), device="cuda"))

    def step(stream=None):
        qb.qb_fp8_quantize_rows(b, out["r"], out["rs"], stream=stream)
        qb.qb_fp8_quantize_blocks(w, out["q"], out["qs"], out["qt"], out["qts"], stream=stream)
        qb.qb_fp8_quantize_cols(a, out["at"], out["ats"], offsets=off, stream=stream)
        qb.qb_fp8_quantize_cols(b, out["bt"], out["bts"], offsets=off, stream=stream)
        qb.qb_fp8_expert_wgrad(out["at"], out["ats"], out["bt"], out["bts"], out["dw"], offsets=off,
                               stream=stream)
    step()
    want = {n: t.clone() for n, t in out.items()}
    assert torch.isfinite(want["dw"]).all() and not want["dw"][1].any()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(out[n], want[n]) for n in out)

    def wipe():
        for t in out.values():
            t.zero_() if t.dtype == torch.uint8 else t.fill_(float("nan"))
        torch.cuda.synchronize()
    wipe()
    s = torch.cuda.Stream()
    step(s)
    s.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        wipe()
        g.replay()
        assert same()
    assert qb.device_status() == 0


def test_token_major_codes_past_32_bits(qb):
    # 2.2e9 codes; the last features' columns, and all groups, against the statement
    T, M, K, G = 8, 131200, 16400, 3
    x = source(T, K, 4)
    index = (torch.arange(M, device="cuda") % T).to(torch.int32)
    off = torch.tensor([0, 1000, 70001, M], dtype=torch.int32, device="cuda")
    width = qb.fp8_cols_width(M, G)
    assert K * width > 1 << 31
    q = torch.empty(K, width, dtype=torch.uint8, device="cuda")
    s = torch.empty(K, ref.pitch(width), dtype=torch.uint8, device="cuda")
    qb.qb_fp8_quantize_cols(x, q, s, offsets=off, row_idx=index)
    tail = x[:, -4:].double().cpu().numpy()[index.cpu().numpy()]
    want, scale = ref.quantize(ref.grouped_columns(tail, off.tolist(), width), 1)
    assert codes_equal(q[-4:], want) and np.array_equal(s[-4:].cpu().numpy(), scale)


def test_weights_past_32_bits(qb):
    G, N, K = 17, 8208, 16400
    assert G * N * K > 1 << 31
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    w[-1] = source(N, K, 5)
    q = torch.empty(G, N, K, dtype=torch.uint8, device="cuda")
    qt = torch.empty(G, K, N, dtype=torch.uint8, device="cuda")
    s, st = blank(G, 65, ref.pitch(K)), blank(G, 129, ref.pitch(N))
    qb.qb_fp8_quantize_blocks(w, q, s, qt, st)
    h = w[-1, -16:, :].double().cpu().numpy()  # the last, short block row (8208 = 64 * 128 + 16)
    want, scale = ref.quantize(h, 128)
    assert codes_equal(q[-1, -16:], want) and np.array_equal(s[-1, -1:].cpu().numpy(), scale)
    assert codes_equal(qt[-1, :, -16:].contiguous(), want.T)
    assert torch.equal(q[-1].t(), qt[-1])
    assert not q[-2].any() and not qt[-2].any()


def test_weight_gradient_past_32_bits(qb):
    G, N, K, width = 3, 27000, 27008, 512
    assert G * N * K > 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(6)

    def operand(rows):
        v = (torch.randn(rows, width, generator=g, device="cuda") * 60).clamp(-448, 448)
        return v.to(torch.float8_e4m3fn), torch.randint(117, 124, (rows, 4), generator=g,
                                                        device="cuda", dtype=torch.uint8)
    (a, sa), (b, sb) = operand(N), operand(K)
    off = torch.tensor([0, 128, 128, 512], dtype=torch.int32, device="cuda")
    dw = torch.full((G, N, K), float("nan"), dtype=torch.float32, device="cuda")
    qb.qb_fp8_expert_wgrad(a, sa, b, sb, dw, offsets=off)
    A = ref.value(a[-40:].double().cpu().numpy(), sa[-40:].cpu().numpy())[:, 128:]
    B = ref.value(b[-300:].double().cpu().numpy(), sb[-300:].cpu().numpy())[:, 128:]
    # (12 steps of the accumulator + 25) units of 2^-23 of sum |A| |B|
    got = dw[-1, -40:, -300:].double().cpu().numpy()
    assert np.all(np.abs(got - A @ B.T) <= 37 * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T))
    assert not dw[1].any()
    assert bool(torch.isfinite(dw[0]).all()) and bool(torch.isfinite(dw[2]).all())
    total = dw.clone()
    qb.qb_fp8_expert_wgrad(a, sa, b, sb, total, offsets=off, accumulate=True)
    assert torch.equal(total[-1, -40:], 2 * dw[-1, -40:]) and torch.equal(total[0], 2 * dw[0])
    assert qb.device_status() == 0
