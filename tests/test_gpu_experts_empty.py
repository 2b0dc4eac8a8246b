"""One expert without tokens in a call of its own: every operator of its path takes it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


def empty_cols(qb, K, dtype):
    width = qb.fp8_cols_width(0, 1)
    assert width == 0
    q = torch.empty(K, width, dtype=torch.uint8, device="cuda")
    s = torch.empty(K, qb.fp8_scale_pitch(width), dtype=torch.uint8, device="cuda")
    qb.qb_fp8_quantize_cols(torch.empty(0, K, dtype=dtype, device="cuda"), q, s)
    return q, s


@pytest.mark.parametrize("offsets", [False, True])
@pytest.mark.parametrize("N,K", [(16, 16), (144, 80), (1024, 2048)])
def test_weight_gradient_of_no_tokens(qb, N, K, offsets):
    a, b = empty_cols(qb, N, torch.bfloat16), empty_cols(qb, K, torch.float32)
    off = torch.zeros(2, dtype=torch.int32, device="cuda") if offsets else None
    for dtype in (torch.float32, torch.bfloat16):
        dw = torch.full((1, N, K), float("nan"), dtype=dtype, device="cuda")
        qb.qb_fp8_expert_wgrad(*a, *b, dw, offsets=off)
        assert not dw.any()
    kept = torch.randn(1, N, K, device="cuda")
    total = kept.clone()
    qb.qb_fp8_expert_wgrad(*a, *b, total, offsets=off, accumulate=True)
    assert torch.equal(total, kept)
    # nothing but the result is written
    field = torch.full((3, N, K), 7.0, device="cuda")
    qb.qb_fp8_expert_wgrad(*a, *b, field[1:2], offsets=off)
    assert bool((field[0] == 7).all()) and not field[1].any() and bool((field[2] == 7).all())


def test_weight_gradient_of_no_tokens_in_its_stream(qb):
    a = empty_cols(qb, 64, torch.float32)
    s = torch.cuda.Stream()
    dw = torch.full((1, 64, 64), 3.0, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    qb.qb_fp8_expert_wgrad(*a, *a, dw, stream=s)
    s.synchronize()
    assert not dw.any()
    dw.fill_(3.0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qb.qb_fp8_expert_wgrad(*a, *a, dw)
    g.replay()
    torch.cuda.synchronize()
    assert not dw.any()
    with pytest.raises(qb.QBError):  # only fp32 accumulates, without tokens too
        qb.qb_fp8_expert_wgrad(*a, *a, dw.to(torch.bfloat16), accumulate=True)
    assert qb.device_status() == 0
