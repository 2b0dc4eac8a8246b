"""The mixture-of-experts layer over a global batch of several forward calls, and the balance
loss's part of its gradient alone."""
import numpy as np
import pytest
import torch

import experts_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from exact_distributed_quantiles_gb300 import build
    build.build()
    from exact_distributed_quantiles_gb300 import moe_layer
    return moe_layer


def make(moe, E, k, H, F, N, batch=0, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")
    router = (randn(E, H) * H ** -0.5).to(torch.bfloat16)
    layer = moe.MoELayer(randn(E, F, H) * H ** -0.5, randn(E, H, F) * F ** -0.5, router, k, N,
                         coeff=0.05, batch_tokens=batch)
    layer.bias.copy_(randn(E) * 0.05)
    return layer, [randn(N, H).to(torch.bfloat16) for _ in range(4)]


def oracle_bias(orc, logits, bias, k):
    return orc.eqb_global_batch([x.cpu().numpy() for x in logits], bias.cpu().numpy(), k)["bias_out"]


@pytest.mark.parametrize("E,k,N,calls", [(64, 6, 500, 1), (64, 6, 500, 2), (256, 8, 333, 3),
                                         (32, 2, 5, 2)])
def test_bias_of_several_forwards(moe, orc, E, k, N, calls):
    layer, xs = make(moe, E, k, 128, 32, N)
    for _ in range(2):  # the second global batch starts afresh
        start, logits = layer.bias.clone(), []
        for x in xs[:calls]:
            layer.forward(x)
            logits.append(layer.logits.clone())
        layer.update_bias()
        want = oracle_bias(orc, logits, start, k)
        assert np.array_equal(layer.bias.cpu().numpy().view(np.uint32), want.view(np.uint32))


def test_forward_outside_the_batch(moe, orc):
    # an evaluation, or a forward computed anew for its backward pass, leaves the bias alone
    layer, xs = make(moe, 64, 6, 128, 32, 300)
    start = layer.bias.clone()
    layer.forward(xs[0])
    logits = [layer.logits.clone()]
    counted = layer.forward(xs[1])
    logits.append(layer.logits.clone())
    layer.forward(xs[2], count=False)
    assert torch.equal(layer.forward(xs[1], count=False), counted)
    layer.backward(counted, torch.ones(1, device="cuda"))
    layer.update_bias()
    want = oracle_bias(orc, logits, start, 6)
    assert np.array_equal(layer.bias.cpu().numpy().view(np.uint32), want.view(np.uint32))


def test_no_batch_no_bias(moe):
    layer, xs = make(moe, 64, 6, 128, 32, 100)
    with pytest.raises(RuntimeError):
        layer.update_bias()
    layer.forward(xs[0], count=False)
    with pytest.raises(RuntimeError):
        layer.update_bias()
    layer.forward(xs[0])
    layer.update_bias()
    with pytest.raises(RuntimeError):
        layer.update_bias()


@pytest.mark.parametrize("E,k,N,batch", [(32, 4, 300, 0), (64, 6, 515, 200), (256, 8, 700, 128),
                                         (32, 2, 5, 2)])
def test_balance_part_of_the_logits_gradient(moe, E, k, N, batch):
    """The difference that loss_grad makes, a weight of its own for each batch.  The balance part is
    within 2e-5 of its terms' sizes (300 roundings of 32 bits); adding it to the task's part rounds
    once, as does taking the difference here: 2^-23 of the sum's size."""
    layer, xs = make(moe, E, k, 64, 16, N, batch)
    x, dout = xs[0], xs[1]
    layer.forward(x)
    nb = layer.loss.numel()
    weight = 100.0 * torch.linspace(1.0, -0.7, nb, device="cuda")
    none = layer.backward(dout, torch.zeros(nb, device="cuda"))["logits"]
    both = layer.backward(dout, weight)["logits"]
    _, want, size = ref.balance(layer.logits.double().cpu().numpy(), layer.topk.cpu().numpy(), None,
                                0.05, batch, "sigmoid", weight.double().cpu().numpy())
    none, both = none.double().cpu().numpy(), both.double().cpu().numpy()
    slack = 2.0 ** -23 * (np.abs(none) + size)
    assert np.all(np.abs(both - none - want) <= 2e-5 * size + slack)
    assert np.linalg.norm(want) > 100 * np.linalg.norm(slack)
