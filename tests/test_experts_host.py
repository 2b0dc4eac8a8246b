"""Argument checks of the balance loss, the expert order, the 8-bit quantisers and the experts'
products: refused before any CUDA work (CPU only), and the 64-bit statements the GPU tests use,
pinned on small cases."""
import ctypes

import numpy as np
import pytest
import torch

import experts_ref as ref


@pytest.fixture(scope="module")
def qb():
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


F, ODD, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None


def swap(args, i, v):
    return [v if j == i else a for j, a in enumerate(args)]


def refusals(fn, ok, bad):
    for i, v, want in bad:
        assert fn(*swap(ok, i, v)) == want, (fn.__name__, i, v)


def test_balance_refusals(qb):
    L = qb.lib
    ok = [F, 0, F, NUL, 0, 256, 6, 0, 0, 0.01, F, F, F, F, F, 1 << 30, NUL]
    assert L.qb_balance_loss(*ok) == qb.QB_OK  # no tokens: nothing to do
    ok[4] = 100000
    refusals(L.qb_balance_loss, ok, [
        (0, NUL, qb.QB_EINVAL), (0, ODD, qb.QB_EINVAL), (1, 3, qb.QB_EINVAL), (2, NUL, qb.QB_EINVAL),
        (4, -1, qb.QB_EINVAL), (4, 1 << 31, qb.QB_EOVERFLOW), (5, 48, qb.QB_EUNSUPPORTED),
        (5, 2048, qb.QB_EUNSUPPORTED), (6, 0, qb.QB_EINVAL), (6, 16, qb.QB_EUNSUPPORTED),
        (7, -1, qb.QB_EINVAL), (8, 2, qb.QB_EINVAL), (10, NUL, qb.QB_EINVAL), (11, NUL, qb.QB_EINVAL),
        (12, NUL, qb.QB_EINVAL), (13, NUL, qb.QB_EINVAL), (14, NUL, qb.QB_EINVAL),
        (15, 16, qb.QB_EINVAL)])
    ok = [F, 1, NUL, F, F, F, 0, 256, 6, 0, 1, 0.01, F, 0, NUL]
    assert L.qb_balance_grad(*ok) == qb.QB_OK
    ok[6] = 1000
    refusals(L.qb_balance_grad, ok, [
        (0, ODD, qb.QB_EINVAL), (1, -1, qb.QB_EINVAL), (3, NUL, qb.QB_EINVAL), (4, NUL, qb.QB_EINVAL),
        (5, NUL, qb.QB_EINVAL), (6, -5, qb.QB_EINVAL), (7, 31, qb.QB_EUNSUPPORTED),
        (8, 256, qb.QB_EINVAL), (10, 9, qb.QB_EINVAL), (12, ODD, qb.QB_EINVAL), (12, NUL, qb.QB_EINVAL)])
    assert L.qb_balance_workspace(-1, 256, 0) == qb.QB_EINVAL
    assert L.qb_balance_workspace(10, 100, 0) == qb.QB_EUNSUPPORTED


def test_order_refusals(qb):
    L = qb.lib
    ok = [F, 100, 256, 6, F, F, F, F, F, 1 << 30, NUL]
    refusals(L.qb_expert_order, ok, [
        (0, NUL, qb.QB_EINVAL), (1, -1, qb.QB_EINVAL), (1, 1 << 30, qb.QB_EOVERFLOW),
        (2, 40, qb.QB_EUNSUPPORTED), (3, 0, qb.QB_EINVAL), (4, NUL, qb.QB_EINVAL),
        (5, NUL, qb.QB_EINVAL), (6, NUL, qb.QB_EINVAL), (7, NUL, qb.QB_EINVAL), (8, NUL, qb.QB_EINVAL), (9, 16, qb.QB_EINVAL),
        (0, ctypes.c_void_p(0x10002), qb.QB_EINVAL)])
    assert L.qb_order_workspace(1 << 30, 256, 6) == qb.QB_EOVERFLOW
    assert L.qb_order_workspace(5, 33, 6) == qb.QB_EUNSUPPORTED


def test_fp8_sizes(qb):
    assert [qb.fp8_scale_pitch(n) for n in (1, 128, 129, 512, 513, 2048)] == [4, 4, 4, 4, 8, 16]
    for n in (0, 1, 127, 128, 511, 512, 513, 5000):
        assert qb.fp8_scale_pitch(n) == qb.lib.qb_fp8_scale_pitch(n)
        assert qb.fp8_cols_width(n, 7) == qb.lib.qb_fp8_cols_width(n, 7)
    assert qb.fp8_cols_width(0, 1) == 0 and qb.fp8_cols_width(1, 1) == 128
    assert qb.fp8_cols_width(129, 2) == 256 and qb.fp8_cols_width(130, 2) == 384
    # never less than any split of M into G groups takes
    rng = np.random.default_rng(0)
    for _ in range(200):
        G, M = int(rng.integers(1, 9)), int(rng.integers(0, 700))
        cut = np.sort(rng.integers(0, M + 1, G - 1))
        n = np.diff(np.concatenate([[0], cut, [M]]))
        assert (-(-n // 128) * 128).sum() <= qb.fp8_cols_width(M, G)


def test_fp8_refusals(qb):
    L = qb.lib
    ok = [F, 1, 100, 256, NUL, 100, 256, F, F, NUL]
    refusals(L.qb_fp8_quantize_rows, ok, [
        (0, NUL, qb.QB_EINVAL), (0, ODD, qb.QB_EINVAL), (1, 2, qb.QB_EINVAL), (2, 99, qb.QB_EINVAL),
        (3, 240, qb.QB_EINVAL), (3, 264, qb.QB_EINVAL), (4, ctypes.c_void_p(0x10001), qb.QB_EINVAL),
        (5, -1, qb.QB_EINVAL), (6, 250, qb.QB_EINVAL), (6, 0, qb.QB_EINVAL), (7, ODD, qb.QB_EINVAL),
        (8, NUL, qb.QB_EINVAL)])
    assert L.qb_fp8_quantize_rows(*swap(ok, 5, 0)) == qb.QB_OK
    ok = [F, 1, 100, 256, NUL, F, 3, 100, 256, 384, F, F, NUL]
    refusals(L.qb_fp8_quantize_cols, ok, [
        (5, NUL, qb.QB_EINVAL), (6, 0, qb.QB_EINVAL), (6, 1025, qb.QB_EUNSUPPORTED),
        (9, 256, qb.QB_EINVAL), (9, 400, qb.QB_EINVAL), (10, ODD, qb.QB_EINVAL), (11, NUL, qb.QB_EINVAL)])
    ok = [F, 0, 4, 64, 64, F, F, F, F, NUL]
    refusals(L.qb_fp8_quantize_blocks, ok, [
        (0, NUL, qb.QB_EINVAL), (2, 0, qb.QB_EINVAL), (3, 40, qb.QB_EINVAL), (4, 40, qb.QB_EINVAL),
        (7, NUL, qb.QB_EINVAL), (8, NUL, qb.QB_EINVAL), (8, ODD, qb.QB_EINVAL)])
    ok = [F, F, F, F, F, 4, 100, 64, 64, F, 1, NUL]
    refusals(L.qb_fp8_expert_gemm, ok, [
        (0, NUL, qb.QB_EINVAL), (1, ODD, qb.QB_EINVAL), (2, ODD, qb.QB_EINVAL), (3, NUL, qb.QB_EINVAL),
        (4, NUL, qb.QB_EINVAL), (5, 2000, qb.QB_EUNSUPPORTED), (6, -1, qb.QB_EINVAL),
        (6, 1 << 31, qb.QB_EOVERFLOW), (7, 0, qb.QB_EINVAL), (8, 72, qb.QB_EINVAL),
        (9, ODD, qb.QB_EINVAL), (10, 5, qb.QB_EINVAL)])
    assert L.qb_fp8_expert_gemm(*swap(ok, 6, 0)) == qb.QB_OK
    ok = [F, F, F, F, F, 4, 512, 64, 64, F, 0, 0, NUL]
    refusals(L.qb_fp8_expert_wgrad, ok, [
        (0, ODD, qb.QB_EINVAL), (4, NUL, qb.QB_EINVAL), (5, 0, qb.QB_EINVAL), (6, 500, qb.QB_EINVAL),
        (6, 0, qb.QB_EINVAL), (7, 0, qb.QB_EINVAL), (8, 0, qb.QB_EINVAL), (9, ODD, qb.QB_EINVAL),
        (10, 4, qb.QB_EINVAL)])
    assert L.qb_fp8_expert_wgrad(*swap(swap(ok, 10, 1), 11, 1)) == qb.QB_EINVAL


def test_the_statements_agree_with_torch():
    rng = np.random.default_rng(3)
    v = rng.standard_normal(20000) * np.exp(rng.standard_normal(20000) * 3)
    v = np.clip(v, -448, 448).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(v.astype(np.float64)), want)
    assert list(ref.exponent(np.array([448.0, 448.1, 224.0, 0.0, 1e-45]))) == [0, 1, -1, -127, -127]
    x = rng.standard_normal((12, 32))
    topk = np.argsort(-x, 1)[:, :3]
    t = torch.from_numpy(x).requires_grad_()
    s = torch.sigmoid(t)
    p = s / (s.sum(1, keepdim=True) + ref.EPS)
    c = torch.bincount(torch.from_numpy(topk.reshape(-1)), minlength=32).double()
    loss = 0.5 * 32 / (3 * 12 * 12) * (c * p.sum(0)).sum()
    loss.backward()
    out, grad, _ = ref.balance(x, topk, None, 0.5, 0, "sigmoid", np.ones(1))
    assert abs(out["loss"][0] - float(loss.detach())) < 1e-12
    assert np.allclose(grad, t.grad.numpy(), rtol=1e-10, atol=1e-16)
    # uniform loads and shares: the loss is the coefficient
    eye = np.arange(32).repeat(2).reshape(-1, 1)
    even = ref.balance(np.zeros((64, 32)), eye, None, 0.5, 0, "softmax")[0]["loss"][0]
    assert abs(even - 0.5) < 1e-12


def test_the_binding_refuses_tensors_of_the_host(qb):
    x, q = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8)
    s = torch.zeros(4, 4, dtype=torch.uint8)
    topk = torch.zeros(4, 2, dtype=torch.int32)
    i64 = torch.zeros(64, dtype=torch.int32)
    f = torch.zeros(1, 64)
    with pytest.raises(ValueError):
        qb.qb_fp8_quantize_rows(x, q, s, stream=0)
    with pytest.raises(ValueError):
        qb.qb_expert_order(topk, 64, i64, torch.zeros(65, dtype=torch.int32), topk,
                           topk.reshape(-1), s, stream=0)
    with pytest.raises(ValueError):
        qb.qb_balance_loss(x, topk, 0.01, i64.view(1, 64), i64[:1], f, f[0, :1], s, stream=0)
    with pytest.raises(ValueError):
        qb.qb_fp8_expert_gemm(q, s, q.view(1, 4, 64), s[:1].view(1, 1, 4), torch.zeros(4, 4), stream=0)
