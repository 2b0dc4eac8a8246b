"""Balance loss, its gradient and the expert order against the 64-bit statements.

Tolerances, from the arithmetic (u = 2^-24, inputs |x| <= 16):
 exp by ex2.approx(x * log2 e): 2^-22 of the instruction and |x| u of each of the two roundings of
 the argument, together under 40 u; a score adds its sum and reciprocal (4 u), a row's sum at most
 16 more, so a share is within 110 u.  A CTA's sums of shares add at most one u per row of a lane
 (under 150 rows here) and 20 for the joins: prob_sum within 280 u < 2e-5, as is the loss.
 A gradient element is a front factor (within 120 u) times the difference of two terms, each within
 150 u of its size: within 300 u < 2e-5 of the sum of the terms' sizes, both relative to the counts'
 mean."""
import ctypes

import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu
TOL = 2e-5


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import qb as _qb
    return _qb


def inputs(N, E, k, dtype, seed=0, masked=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(N, E, generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda")
    topk = torch.topk(x, k, dim=1).indices.to(torch.int32).contiguous()
    mask = torch.rand(N, generator=g, device="cuda") >= masked if masked else None
    return x.to(dtype), topk, mask


def run(qb, x, topk, mask=None, batch=0, score="sigmoid", coeff=0.01, loss_grad=None, ws=None,
        grad=None, accumulate=False, stream=None):
    N, E = x.shape
    nb = -(-N // batch) if batch else 1
    out = dict(counts=torch.full((nb, E), -7, dtype=torch.int32, device="cuda"),
               tokens=torch.full((nb,), -7, dtype=torch.int32, device="cuda"),
               prob_sum=torch.full((nb, E), float("nan"), device="cuda"),
               loss=torch.full((nb,), float("nan"), device="cuda"))
    ws = qb.balance_workspace(N, E, batch) if ws is None else ws
    qb.qb_balance_loss(x, topk, coeff, out["counts"], out["tokens"], out["prob_sum"], out["loss"],
                       ws, token_mask=mask, batch_tokens=batch, score=score, stream=stream)
    if loss_grad is not None:
        grad = torch.full((N, E), float("nan"), device="cuda") if grad is None else grad
        qb.qb_balance_grad(x, out["counts"], out["tokens"], loss_grad, coeff, topk.shape[1], grad,
                           token_mask=mask, batch_tokens=batch, score=score, accumulate=accumulate,
                           stream=stream)
        out["grad"] = grad
    return out


def check(out, x, topk, mask, batch, score, coeff=0.01, loss_grad=None, before=None):
    lg = None if loss_grad is None else loss_grad.cpu().numpy()
    want, grad, size = ref.balance(x.float().cpu().numpy(), topk.cpu().numpy(),
                                   None if mask is None else mask.cpu().numpy(), coeff, batch,
                                   score, lg)
    assert np.array_equal(out["counts"].cpu().numpy(), want["counts"])
    assert np.array_equal(out["tokens"].cpu().numpy(), want["tokens"])
    for n in ("prob_sum", "loss"):
        got = out[n].double().cpu().numpy()
        assert np.all(np.abs(got - want[n]) <= TOL * np.abs(want[n])), n
    if loss_grad is not None:
        got = out["grad"].double().cpu().numpy()
        slack = 0.0
        if before is not None:
            b = before.double().cpu().numpy()
            grad, slack = grad + b, 2.0 ** -23 * (np.abs(b) + size)
        assert np.all(np.abs(got - grad) <= TOL * size + slack)


SHAPES = [(1, 32, 1, 0), (1, 256, 15, 0), (3, 64, 6, 1), (130, 96, 4, 0), (257, 160, 7, 100),
          (1000, 256, 6, 333), (4099, 256, 8, 0), (700, 384, 2, 0), (515, 512, 15, 64),
          (300, 992, 3, 0), (130, 1024, 15, 129), (20000, 64, 6, 0)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,k,batch", SHAPES)
def test_loss_and_gradient(qb, N, E, k, batch, dtype, score):
    x, topk, mask = inputs(N, E, k, dtype, seed=N + E, masked=0.2 if N % 2 else 0.0)
    nb = -(-N // batch) if batch else 1
    lg = torch.linspace(0.5, -1.5, nb, device="cuda")
    out = run(qb, x, topk, mask, batch, score, loss_grad=lg)
    check(out, x, topk, mask, batch, score, loss_grad=lg)
    again = run(qb, x, topk, mask, batch, score, loss_grad=lg)
    for n in out:
        assert torch.equal(out[n], again[n]), n  # the same bits every time
    assert qb.device_status() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_against_differences(qb, score):
    N, E, k, batch = 96, 64, 6, 40
    x, topk, mask = inputs(N, E, k, torch.float32, seed=5, masked=0.1)
    lg = torch.tensor([1.0, -2.0, 0.5], device="cuda")
    got = run(qb, x, topk, mask, batch, score, coeff=1.0, loss_grad=lg)["grad"].double().cpu().numpy()
    x0, t, m = x.double().cpu().numpy(), topk.cpu().numpy(), mask.cpu().numpy()
    rng = np.random.default_rng(1)
    h = 1e-4  # the differences are off by h^2 (third derivatives of size one) and 1e-16 / h
    for _ in range(8):
        v = rng.standard_normal((N, E))

        def total(s):
            return float((ref.balance(x0 + s * h * v, t, m, 1.0, batch, score)[0]["loss"] * lg.cpu().numpy()).sum())
        num = (total(1) - total(-1)) / (2 * h)
        scale = np.sqrt(((got * v) ** 2).sum()) + np.abs(got * v).sum() * TOL
        assert abs((got * v).sum() - num) <= 1e-5 * np.abs(got * v).sum() + 1e-6 * scale


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_rows_do_not_reach_the_result(qb, score):
    x, topk, _ = inputs(300, 96, 6, torch.float32, seed=3)
    mask = torch.ones(300, dtype=torch.uint8, device="cuda")
    mask[::3] = 0
    mask[200:] = 0  # a batch with nothing live
    lg = torch.ones(3, device="cuda")
    clean = run(qb, x, topk, mask, 100, score, loss_grad=lg)
    dirty, t2 = x.clone(), topk.clone()
    dirty[mask == 0] = float("nan")
    dirty[0, 1], dirty[3, 2] = float("inf"), float("-inf")
    t2[mask == 0] = 2 ** 30
    out = run(qb, dirty, t2, mask, 100, score, loss_grad=lg)
    for n in clean:
        assert torch.equal(clean[n], out[n]), n
    assert out["loss"][2] == 0 and out["tokens"][2] == 0 and not out["grad"][200:].any()
    check(out, x, topk, mask, 100, score, loss_grad=lg)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_closed_experts_dropped_entries_and_extremes(qb, score):
    x, topk, _ = inputs(64, 64, 6, torch.float32, seed=4)
    x[:, 5] = float("-inf")
    x[7] = -1000.0            # a row whose sigmoid scores all vanish
    x[8] = 1000.0
    x[9, ::2] = 1000.0
    if score == "softmax":
        x[10] = float("-inf")  # nothing to choose from
    topk[::4, 2] = -1
    topk[1, 0] = 64
    lg = torch.ones(1, device="cuda")
    out = run(qb, x, topk, None, 0, score, loss_grad=lg)
    assert torch.isfinite(out["grad"]).all()
    want, grad, size = ref.balance(x.double().cpu().numpy(), topk.cpu().numpy(), None, 0.01, 0,
                                   score, np.ones(1))
    assert np.array_equal(out["counts"].cpu().numpy(), want["counts"])
    assert np.allclose(out["prob_sum"].cpu().numpy(), want["prob_sum"], rtol=TOL, atol=1e-12)
    assert np.allclose(out["loss"].cpu().numpy(), want["loss"], rtol=TOL)
    assert np.all(np.abs(out["grad"].double().cpu().numpy() - grad) <= TOL * size + 1e-18)


def test_nan_shows_in_its_batch_only(qb):
    x, topk, _ = inputs(200, 64, 6, torch.float32, seed=6)
    x[150, 3] = float("nan")
    out = run(qb, x, topk, None, 100, "sigmoid")
    assert torch.isfinite(out["loss"][0]) and torch.isnan(out["loss"][1])


def test_accumulates_into_a_gradient(qb):
    x, topk, mask = inputs(500, 256, 6, torch.bfloat16, seed=8, masked=0.3)
    lg = torch.tensor([2.0, -1.0], device="cuda")
    g0 = torch.randn(500, 256, device="cuda") * 1e-6
    out = run(qb, x, topk, mask, 300, "sigmoid", loss_grad=lg, grad=g0.clone(), accumulate=True)
    check(out, x, topk, mask, 300, "sigmoid", loss_grad=lg, before=g0)
    assert torch.equal(out["grad"][~mask], g0[~mask])


def test_one_workspace_for_calls_of_several_sizes(qb):
    ws = qb.balance_workspace(40000, 512, 0)
    for N, E, batch in ((40000, 512, 0), (40000, 64, 700), (300, 32, 0), (30000, 512, 10000),
                        (40000, 512, 0)):
        x, topk, _ = inputs(N, E, 4, torch.float32, seed=N + E)
        out = run(qb, x, topk, None, batch, "sigmoid", ws=ws)
        check(out, x, topk, None, batch, "sigmoid")


def test_on_another_stream_and_in_a_graph(qb):
    x, topk, _ = inputs(30000, 256, 6, torch.float32, seed=9)
    lg = torch.ones(1, device="cuda")
    ws = qb.balance_workspace(30000, 256, 0)
    want = run(qb, x, topk, loss_grad=lg, ws=ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    grad = torch.empty(30000, 256, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = run(qb, x, topk, loss_grad=lg, ws=ws, grad=grad)
    s.synchronize()
    for n in want:
        assert torch.equal(want[n], out[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(qb, x, topk, loss_grad=lg, ws=ws, grad=grad)
    for _ in range(2):
        grad.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(want[n], out[n]), n


def test_gradient_past_32_bit_offsets(qb):
    N, E, k = (1 << 31) // 1024 + 70, 1024, 2
    x = torch.zeros(N, E, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    tail = torch.randn(128, E, generator=g, device="cuda").to(torch.bfloat16)
    x[-128:] = tail
    topk = torch.zeros(N, k, dtype=torch.int32, device="cuda")
    topk[:, 1] = 1
    topk[-128:] = torch.topk(tail.float(), k, dim=1).indices.to(torch.int32)
    batch = N - 128  # the last batch is the tail
    lg = torch.ones(2, device="cuda")
    out = run(qb, x, topk, None, batch, "sigmoid", loss_grad=lg)
    last = {n: out[n][1:] for n in ("counts", "tokens", "prob_sum", "loss")}
    last["grad"] = out["grad"][-128:]
    check(last, tail, topk[-128:], None, 0, "sigmoid", loss_grad=lg[1:])
    assert int(out["counts"][0, 0]) == batch
    # equal logits: uniform shares, so expert 0's gradient is c (1 - 2/E) of the formula
    c = 0.01 * E / (k * float(batch) ** 2) * batch
    want = 0.25 / (0.5 * E) * c * (1 - 2 / E)
    assert abs(float(out["grad"][12345, 0]) - want) <= TOL * abs(want) * 2


# ------------------------------------------------------------------ order

ORDER = [(1, 32, 1), (7, 256, 6), (1, 1024, 15), (33, 64, 6), (1500, 96, 3), (2049, 256, 4),
         (5000, 256, 6), (9001, 1024, 8), (50000, 32, 2), (131, 992, 31)]


@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("N,E,k", ORDER)
def test_order(qb, N, E, k, dropped):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + k)
    # half of the tokens crowd on few experts
    topk = torch.randint(0, E, (N, k), generator=g, device="cuda", dtype=torch.int32)
    topk[: N // 2] %= 3
    topk[torch.rand(N, k, generator=g, device="cuda") < dropped] = -1
    if dropped and N > 3:
        topk[3, 0], topk[2, 0] = E, 2 ** 31 - 1
    out = [torch.full((E,), -9, dtype=torch.int32, device="cuda"),
           torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
           torch.full((N, k), -9, dtype=torch.int32, device="cuda"),
           torch.full((N * k,), -9, dtype=torch.int32, device="cuda")]
    ws = torch.full((max(4, qb.lib.qb_order_workspace(N, E, k)),), 255, dtype=torch.uint8, device="cuda")
    qb.qb_expert_order(topk, E, *out, ws)
    for got, want in zip(out, ref.order(topk.cpu().numpy(), E)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_loss_of_no_tokens(qb):
    x, none = torch.empty(0, 64, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda")
    i, f = torch.full((1, 64), 3, dtype=torch.int32, device="cuda"), torch.full((1, 64), 3.0, device="cuda")
    ws = qb.balance_workspace(0, 64)
    qb.qb_balance_loss(x, none, 0.01, i, i[0, :1], f, f[0, :1], ws)
    qb.qb_balance_grad(x, i, i[0, :1], f[0, :1], 0.01, 4, x)
    assert bool((i == 3).all()) and bool((f == 3).all())  # nothing to do, nothing written


def test_order_of_no_tokens(qb):
    counts = torch.full((64,), 5, dtype=torch.int32, device="cuda")
    offsets = torch.full((65,), 5, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    qb.qb_expert_order(e, 64, counts, offsets, e, e.reshape(0), qb.order_workspace(0, 64, 4))
    assert not counts.any() and not offsets.any()


# ------------------------------------------------------------------ refusals

def test_the_binding_refuses(qb):
    x, topk, _ = inputs(40, 64, 6, torch.float32)
    ok = dict(counts=torch.empty(1, 64, dtype=torch.int32, device="cuda"),
              tokens=torch.empty(1, dtype=torch.int32, device="cuda"),
              prob_sum=torch.empty(1, 64, device="cuda"), loss=torch.empty(1, device="cuda"),
              workspace=qb.balance_workspace(40, 64))

    def loss(x=x, topk=topk, **kw):
        a = {**ok, **{n: v for n, v in kw.items() if n in ok}}
        rest = {n: v for n, v in kw.items() if n not in ok}
        qb.qb_balance_loss(x, topk, 0.01, a["counts"], a["tokens"], a["prob_sum"], a["loss"],
                           a["workspace"], **rest)
    loss()
    with pytest.raises(TypeError):
        loss(x=x.half())
    with pytest.raises(TypeError):
        loss(topk=topk.long())
    with pytest.raises(ValueError):
        loss(x=x.t().contiguous().t())
    with pytest.raises(ValueError):
        loss(batch_tokens=20)  # outputs of one batch
    with pytest.raises(ValueError):
        loss(token_mask=torch.ones(39, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        loss(score="relu")
    with pytest.raises(qb.QBError):  # a workspace that is too small
        big, t, _ = inputs(4000, 64, 6, torch.float32)
        loss(x=big, topk=t, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qb.QBError) as e:
        loss(x=torch.empty(40 * 64 + 1, device="cuda")[1:].view(40, 64))
    assert e.value.status == qb.QB_EINVAL
    with pytest.raises(ValueError):
        qb.qb_expert_order(topk, 64, ok["counts"][0], torch.empty(64, dtype=torch.int32, device="cuda"),
                           topk, topk.reshape(-1), ok["workspace"])
    torch.cuda.synchronize()
    assert ctypes.c_int(qb.device_status()).value == 0
