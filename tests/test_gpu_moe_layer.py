"""The operators together: one step of the mixture-of-experts layer against the same layer in
64-bit torch autograd on the same weights, inputs and top-k sets.

Tolerance (norm of the difference over the norm): a code is within 2^-4 of its value, 0.026 of it
in the mean square (uniform over the spacing's 2^-3..2^-4), so a product of two coded operands is
off by 0.037 of its norm; the layer chains two products forward (0.053), three back to x and w1
(0.065), and bf16 rounds in between (under 0.01): 0.1 for each.  The router's gradient through the
gates follows y (0.053) and differences of it; 0.15."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer_mod():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import moe_layer, qb
    return moe_layer, qb


def make(moe, E, k, H, F, N, eta=0.0, batch=0, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    w1 = randn(E, F, H) * H ** -0.5
    w2 = randn(E, H, F) * F ** -0.5
    router = (randn(E, H) * H ** -0.5).to(torch.bfloat16)
    layer = moe.MoELayer(w1, w2, router, k, N, coeff=0.05, eta=eta, batch_tokens=batch)
    layer.bias.copy_(randn(E) * 0.05)
    x = randn(N, H).to(torch.bfloat16)
    dout = randn(N, H).to(torch.bfloat16)
    return layer, x, dout


def reference(layer, x, dout, loss_grad):
    x, dout = x.double().requires_grad_(), dout.double()
    w1, w2 = layer.w1.w.double().requires_grad_(), layer.w2.w.double().requires_grad_()
    r = layer.router.double().requires_grad_()
    topk, N, E, k = layer.topk.long(), layer.N, layer.E, layer.k
    logits = x @ r.t()
    s = torch.sigmoid(logits)
    picked = s.gather(1, topk)
    gates = picked / picked.sum(1, keepdim=True)
    out = torch.zeros(N, layer.H, dtype=torch.float64, device="cuda")
    for e in range(E):
        i, t = (topk == e).nonzero(as_tuple=True)
        if len(i):
            y = torch.nn.functional.silu(x[i] @ w1[e].t()) @ w2[e].t()
            out = out.index_add(0, i, gates[i, t][:, None] * y)
    p = s / (s.sum(1, keepdim=True) + 1e-20)
    losses = []
    for lo in range(0, N, layer.batch or N):
        hi = min(N, lo + (layer.batch or N))
        c = torch.bincount(topk[lo:hi].reshape(-1), minlength=E).double()
        losses.append(layer.coeff * E / (k * (hi - lo) ** 2) * (c * p[lo:hi].sum(0)).sum())
    losses = torch.stack(losses)
    ((out * dout).sum() + (losses * loss_grad.double()).sum()).backward()
    return out, losses, {"x": x.grad, "w1": w1.grad, "w2": w2.grad, "router": r.grad}


def off(a, b):
    return float(((a.double() - b).norm() / b.norm()).detach())


@pytest.mark.parametrize("E,k,H,F,N,batch", [(32, 4, 128, 96, 300, 0), (64, 6, 256, 144, 515, 200),
                                             (32, 2, 64, 16, 5, 0)])
def test_layer_step(layer_mod, E, k, H, F, N, batch):
    moe, qb = layer_mod
    layer, x, dout = make(moe, E, k, H, F, N, batch=batch)
    out = layer.forward(x)
    loss_grad = torch.full((layer.loss.numel(),), 100.0, device="cuda")
    grads = layer.backward(dout, loss_grad)
    want, losses, wgrads = reference(layer, x, dout, loss_grad)
    assert off(out, want) < 0.1
    assert torch.allclose(layer.loss.double(), losses, rtol=1e-4)  # logits of a bf16 product
    for n, tol in (("x", 0.1), ("w1", 0.1), ("w2", 0.1), ("router", 0.15)):
        assert off(grads[n], wgrads[n]) < tol, n
    assert qb.device_status() == 0


def test_load_error_injection_reaches_the_logits(layer_mod):
    moe, qb = layer_mod
    plain, x, dout = make(moe, 64, 6, 128, 64, 400, batch=100)
    shifted, _, _ = make(moe, 64, 6, 128, 64, 400, eta=0.5, batch=100)
    g = torch.zeros(4, device="cuda")
    a = (plain.forward(x), plain.backward(dout, g))[1]
    b = (shifted.forward(x), shifted.backward(dout, g))[1]
    rho = torch.zeros(400, 64, device="cuda")
    ws = torch.empty(4, 64, device="cuda")
    qb.lei_inject(rho, plain.topk, 0.5, ws, batch_tokens=100)
    s = torch.sigmoid(plain.logits)
    assert torch.allclose(b["logits"] - a["logits"], rho * s * (1 - s), atol=1e-5)


def test_bias_update_balances_the_loads(layer_mod):
    moe, _ = layer_mod
    layer, x, _ = make(moe, 64, 6, 256, 32, 4096)
    layer.bias.zero_()
    offset = torch.randn(64, device="cuda") * 0.03
    layer.router.add_((offset[:, None] * torch.ones(256, device="cuda")).to(torch.bfloat16))
    x = (x + 0.5).to(torch.bfloat16)
    layer.forward(x)
    first = int(layer.load.max())
    layer.update_bias()
    layer.forward(x)
    assert int(layer.load.max()) < first
    assert int(layer.load.sum()) == 4096 * 6
