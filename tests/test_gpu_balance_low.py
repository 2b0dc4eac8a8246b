"""The sigmoid balance loss and its gradient in rows whose logits are all very negative, where the
scores' sum comes near the 1e-20 beside it, against the 64-bit statement.

Tolerance, from the arithmetic (u = 2^-24, inputs down to -80): exp by ex2.approx(x * log2 e) is
within 2^-22 of the instruction and 80 u of each of the two roundings of the argument, 164 u; a
score adds its sum and reciprocal (4 u), a row's sum 16 at most.  A gradient element is
s * (s e) / S (s e is near 1 here; s, S and the products within 350 u) times a difference of terms
within 350 u of their sizes: within 700 u of the sum of the terms' sizes.  There is no absolute
slack.  A share is within 350 u and the sums over the rows add under 200."""
import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu
TOL = 700 * 2.0 ** -24


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


LEVELS = [-40.0, -44.0, -46.0, -48.0, -50.0, -52.0, -54.0, -56.0, -60.0, -65.0, -72.0, -79.0]


def rows(E, dtype, closed, seed):
    """Four rows at each level, spread over one unit; in the last two of a level every third column
    is closed (-inf) where asked, and in the last one column is an ordinary logit."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.tensor(LEVELS, device="cuda").repeat_interleave(4)[:, None]
    x = x + torch.rand(x.shape[0], E, generator=g, device="cuda")
    if closed:
        x[2::4, ::3] = float("-inf")
        x[3::4, ::3] = float("-inf")
    x[3::4, 1] = 0.5
    topk = torch.topk(x + torch.rand(x.shape, generator=g, device="cuda"), 6, dim=1).indices
    return x.to(dtype), topk.to(torch.int32).contiguous()


def run(qb, x, topk, coeff):
    N, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, tokens = torch.empty(1, E, **i32), torch.empty(1, **i32)
    prob_sum, loss = torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    qb.qb_balance_loss(x, topk, coeff, counts, tokens, prob_sum, loss, qb.balance_workspace(N, E))
    grad = torch.full((N, E), float("nan"), device="cuda")
    qb.qb_balance_grad(x, counts, tokens, torch.ones(1, device="cuda"), coeff, topk.shape[1], grad)
    return prob_sum[0].double().cpu().numpy(), float(loss), grad.double().cpu().numpy()


def statement(x, topk, coeff):
    """The 64-bit result, its gradient, and the sum of the sizes of each element's terms."""
    x, t = x.double().cpu().numpy(), topk.cpu().numpy()
    out, grad, _ = ref.balance(x, t, None, coeff, 0, "sigmoid", np.ones(1))
    p, s, total = ref.shares(x, "sigmoid")
    w = coeff * x.shape[1] / (t.shape[1] * float(x.shape[0]) ** 2) * out["counts"][0]
    return out, grad, s * (1.0 - s) / total * (w + (p @ w)[:, None] + w.mean())


@pytest.mark.parametrize("closed", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [32, 64, 192, 256, 384, 512, 1024])
def test_rows_of_very_negative_logits(qb, E, dtype, closed):
    x, topk = rows(E, dtype, closed, E)
    coeff = 0.05
    prob_sum, loss, grad = run(qb, x, topk, coeff)
    out, want, size = statement(x, topk, coeff)
    assert np.all(np.abs(grad - want) <= TOL * size)
    assert np.all(np.abs(prob_sum - out["prob_sum"][0]) <= TOL * out["prob_sum"][0])
    assert abs(loss - out["loss"][0]) <= TOL * out["loss"][0]
    # the rows are no dust: their gradients are of an ordinary row's size down to about -50
    norm = np.linalg.norm(want, axis=1)
    assert norm[4 * LEVELS.index(-50.0)] > 0.5 * norm[0]


def test_a_closed_row_has_no_gradient(qb):
    x, topk = rows(64, torch.float32, True, 3)
    x[5] = float("-inf")
    _, _, grad = run(qb, x, topk, 0.05)
    assert not grad[5].any()
    closed = torch.isneginf(x).cpu().numpy()
    assert not grad[closed].any() and np.isfinite(grad).all()


def test_nan_stays_nan(qb):
    x, topk = rows(64, torch.float32, False, 4)
    x[9, 3] = float("nan")
    _, loss, grad = run(qb, x, topk, 0.05)
    assert np.isnan(loss) and np.isnan(grad[9]).all()
    assert np.isfinite(np.delete(grad, 9, 0)).all()


def test_gradient_agrees_with_the_loss(qb):
    # differences of the 64-bit loss along directions that move one row, at levels where the
    # gradient's front factor is far below the smallest fp32 square
    E, coeff, h = 64, 1.0, 1e-4
    x, topk = rows(E, torch.float32, False, 7)
    _, _, grad = run(qb, x, topk, coeff)
    _, _, size = statement(x, topk, coeff)
    x64, t = x.double().cpu().numpy(), topk.cpu().numpy()
    rng = np.random.default_rng(2)
    for level in (-46.0, -50.0, -54.0):
        r = 4 * LEVELS.index(level)
        v = np.zeros_like(x64)
        v[r] = rng.standard_normal(E)
        up, down = (ref.balance(x64 + d * h * v, t, None, coeff, 0, "sigmoid")[0]["loss"][0]
                    for d in (1, -1))
        # off by h^2 (third derivatives of the terms' size) and by the 64-bit losses' rounding,
        # under 2^-50 of them over h
        terms = (size[r] * np.abs(v[r])).sum()
        assert abs((up - down) / (2 * h) - (grad[r] * v[r]).sum()) <= (
            (1e-6 + TOL) * terms + 2.0 ** -50 * abs(up) / h), level
