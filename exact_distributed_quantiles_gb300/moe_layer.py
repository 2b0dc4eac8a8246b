"""A mixture-of-experts layer from the library's operators, forward and backward.

One training step of the layer around the router:

  route        qb_router_gemm, qb_route_hist_hi (top-k sets and the quantile histogram),
               qb_balance_loss (per local batch), qb_expert_order (rows by expert)
  experts      qb_fp8_quantize_rows (gathered into expert order), qb_fp8_expert_gemm, SiLU,
               the same again, and the gate-weighted sum over a token's experts
  backward     qb_fp8_expert_gemm with the transposed weights, qb_fp8_quantize_cols and
               qb_fp8_expert_wgrad for the weights, lei_inject on the score gradient,
               qb_balance_grad added to the logits' gradient
  bias         qb_select_hi, qb_keys_hist_lo, qb_finalize once per global batch, over the keys of
               every forward call of it

Each expert e computes W2[e] silu(W1[e] x).  The gates are a token's sigmoid scores of its k
experts, normalised ("[Dev] Add global-batch quantile balancing", "Quantile estimator": the bias
selects, the scores weigh).  Everything between the library's calls is plain torch; no call waits
for the device.
"""
from __future__ import annotations

import torch

from . import qb


def _fp8(*shape, device):
    return torch.empty(*shape, dtype=torch.float8_e4m3fn, device=device)


def _bytes(*shape, device):
    return torch.empty(*shape, dtype=torch.uint8, device=device)


class Weights:
    """Experts' weights w [E, N, K] with their codes in both orientations."""

    def __init__(self, w: torch.Tensor):
        E, N, K = w.shape
        d = w.device
        self.w = w
        self.q, self.q_t = _fp8(E, N, K, device=d), _fp8(E, K, N, device=d)
        self.scale = _bytes(E, -(-N // 128), qb.fp8_scale_pitch(K), device=d)
        self.scale_t = _bytes(E, -(-K // 128), qb.fp8_scale_pitch(N), device=d)
        self.encode()

    def encode(self):
        """Codes the weights anew; call it after an optimizer step."""
        qb.qb_fp8_quantize_blocks(self.w, self.q, self.scale, self.q_t, self.scale_t)


class MoELayer:
    """w1 [E, F, H], w2 [E, H, F] (fp32 or bf16; H and F multiples of 16), router [E, H] bf16
    (H a multiple of 64, E a multiple of 32 up to 256).  `tokens`: rows of x in every call.

    A global batch is the forward calls between two bias updates, one for each microbatch; each
    keeps its keys (2 E bytes a token) until the update, in buffers that later batches take again."""

    def __init__(self, w1, w2, router, k, tokens, coeff=1e-2, eta=0.0, batch_tokens=0):
        self.E, self.F, self.H = w1.shape
        self.k, self.N, self.coeff, self.eta, self.batch = k, tokens, coeff, eta, batch_tokens
        self.w1, self.w2, self.router = Weights(w1), Weights(w2), router
        d, E, N = w1.device, self.E, tokens
        self.device = d
        self.bias = torch.zeros(E, device=d)
        self.state = qb.EQBState(E, d)
        # a buffer of keys for each forward call of a global batch, and the current one's calls
        self.keys, self.counted = [torch.empty(N, E, dtype=torch.int16, device=d)], 0
        self.uncounted = torch.zeros_like(self.state.hist_hi)  # of the calls outside any
        nb = -(-N // batch_tokens) if batch_tokens else 1
        self.logits = torch.empty(N, E, device=d)
        self.topk = torch.empty(N, k, dtype=torch.int32, device=d)
        self.counts = torch.empty(nb, E, dtype=torch.int32, device=d)
        self.live = torch.empty(nb, dtype=torch.int32, device=d)
        self.prob_sum = torch.empty(nb, E, device=d)
        self.loss = torch.empty(nb, device=d)
        self.load = torch.empty(E, dtype=torch.int32, device=d)
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=d)
        self.slot_of = torch.empty(N, k, dtype=torch.int32, device=d)
        self.token_of = torch.empty(N * k, dtype=torch.int32, device=d)
        self.loss_ws = qb.balance_workspace(N, E, batch_tokens, d)
        self.order_ws = qb.order_workspace(N, E, k, d)
        self.lei_ws = torch.empty(nb, E, device=d)

    # ---- pieces

    def _rows(self, x, index=None):
        """Codes of x's rows (or of the rows that index names)."""
        M = x.shape[0] if index is None else index.numel()
        q = _fp8(M, x.shape[1], device=self.device)
        s = _bytes(M, qb.fp8_scale_pitch(x.shape[1]), device=self.device)
        qb.qb_fp8_quantize_rows(x, q, s, row_idx=index)
        return q, s

    def _cols(self, x, index=None):
        """Codes of x's rows with the scales along the tokens of each expert."""
        width = qb.fp8_cols_width(self.N * self.k, self.E)
        q = _fp8(x.shape[1], width, device=self.device)
        s = _bytes(x.shape[1], qb.fp8_scale_pitch(width), device=self.device)
        qb.qb_fp8_quantize_cols(x, q, s, offsets=self.offsets, row_idx=index)
        return q, s

    def _product(self, rows, q, scale):
        out = torch.empty(rows[0].shape[0], q.shape[1], dtype=torch.bfloat16, device=self.device)
        qb.qb_fp8_expert_gemm(*rows, q, scale, out, offsets=self.offsets)
        return out

    def _wgrad(self, a, b):
        out = torch.empty(self.E, a[0].shape[0], b[0].shape[0], device=self.device)
        qb.qb_fp8_expert_wgrad(*a, *b, out, offsets=self.offsets)
        return out

    # ---- one step

    def forward(self, x, count=True):
        """x [N, H] bf16 -> [N, H] bf16; the balance losses are in self.loss.  The call adds its
        tokens to the global batch of the next update_bias; with count=False it does not (an
        evaluation, or a forward computed again for its backward pass)."""
        qb.qb_router_gemm(x, self.router, self.logits)
        hist, keys = self.uncounted, None
        if count:
            if self.counted == len(self.keys):
                self.keys.append(torch.empty(self.N, self.E, dtype=torch.int16, device=self.device))
            hist, keys = self.state.hist_hi, self.keys[self.counted]
        qb.qb_route_hist_hi(self.logits, self.bias, self.k, hist, keys_out=keys, topk_out=self.topk)
        self.counted += bool(count)
        qb.qb_balance_loss(self.logits, self.topk, self.coeff, self.counts, self.live,
                           self.prob_sum, self.loss, self.loss_ws, batch_tokens=self.batch)
        qb.qb_expert_order(self.topk, self.E, self.load, self.offsets, self.slot_of, self.token_of,
                           self.order_ws)
        self.x = x
        self.scores = torch.sigmoid(self.logits.gather(1, self.topk.long()))
        self.gates = self.scores / self.scores.sum(1, keepdim=True)
        self.h = self._product(self._rows(x, self.token_of), self.w1.q, self.w1.scale)
        self.act = torch.nn.functional.silu(self.h.float()).to(torch.bfloat16)
        self.y = self._product(self._rows(self.act), self.w2.q, self.w2.scale)
        y = self.y[self.slot_of.long()].float()  # [N, k, H]
        return (self.gates[..., None] * y).sum(1).to(torch.bfloat16)

    def backward(self, dout, loss_grad):
        """Gradients of <out, dout> + <self.loss, loss_grad>: a dict with x, w1, w2, router."""
        k, token, slot = self.k, self.token_of.long(), self.slot_of.long()
        # each row's token and gate, in expert order
        gate = torch.empty(self.N * k, device=self.device)
        gate[slot.reshape(-1)] = self.gates.reshape(-1)
        dy = (gate[:, None] * dout[token].float()).to(torch.bfloat16)
        dact = self._product(self._rows(dy), self.w2.q_t, self.w2.scale_t).float()
        dw2 = self._wgrad(self._cols(dy), self._cols(self.act))
        h = self.h.float()
        sig = torch.sigmoid(h)
        dh = (dact * sig * (1.0 + h * (1.0 - sig))).to(torch.bfloat16)
        dxs = self._product(self._rows(dh), self.w1.q_t, self.w1.scale_t)
        dw1 = self._wgrad(self._cols(dh), self._cols(self.x, self.token_of))
        dx = dxs[slot].float().sum(1)
        # gates -> scores (with the load-error injection) -> logits, and the balance loss
        dgate = (self.y[slot].float() * dout[:, None, :].float()).sum(-1)
        total = self.scores.sum(1, keepdim=True)
        dscore = torch.zeros(self.N, self.E, device=self.device)
        dscore.scatter_(1, self.topk.long(),
                        (dgate - (dgate * self.gates).sum(1, keepdim=True)) / total)
        if self.eta:
            qb.lei_inject(dscore, self.topk, self.eta, self.lei_ws, batch_tokens=self.batch)
        s = torch.sigmoid(self.logits)
        dlogits = dscore * s * (1.0 - s)
        qb.qb_balance_grad(self.logits, self.counts, self.live, loss_grad, self.coeff, k, dlogits,
                           batch_tokens=self.batch, accumulate=True)
        dx += dlogits @ self.router.float()
        return {"x": dx, "w1": dw1, "w2": dw2, "router": dlogits.t() @ self.x.float(),
                "logits": dlogits}

    def update_bias(self):
        """The quantile bias of the global batch: all tokens of the forward calls since the last
        update."""
        if self.counted == 0:
            raise RuntimeError("update_bias: no forward call since the last update")
        qb.qb_select_hi(self.state.hist_hi, qb.rank(self.counted * self.N, self.E, self.k),
                        self.state.sel, self.state.r_lo)
        for keys in self.keys[:self.counted]:
            qb.qb_keys_hist_lo(keys, self.state.sel, self.state.hist_lo)
        qb.qb_finalize(self.state.hist_hi, self.state.hist_lo, self.state.sel, self.state.r_lo,
                       self.bias, qkey_out=self.state.qkey, reset=True)
        self.counted = 0


def main():
    """A few steps at one layer's sizes: the loss, the loads and the time of a step."""
    torch.manual_seed(0)
    E, k, H, F, N = 256, 6, 2048, 1024, 16384
    d = "cuda"
    w1 = (torch.randn(E, F, H, device=d) * H ** -0.5).to(torch.bfloat16)
    w2 = (torch.randn(E, H, F, device=d) * F ** -0.5).to(torch.bfloat16)
    router = (torch.randn(E, H, device=d) * H ** -0.5).to(torch.bfloat16)
    layer = MoELayer(w1, w2, router, k, N, eta=8e-5, batch_tokens=4096)
    loss_grad = torch.ones(N // 4096, device=d)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for step in range(5):
        x = torch.randn(N, H, device=d).to(torch.bfloat16)
        begin.record()
        out = layer.forward(x)
        layer.backward(out, loss_grad)
        layer.update_bias()
        end.record()
        torch.cuda.synchronize()
        busiest = int(layer.load.max()) * E / (N * k)
        print(f"step {step}: balance loss {float(layer.loss.mean()):.5f}, busiest expert "
              f"{busiest:.2f} x uniform, {begin.elapsed_time(end):.2f} ms")


if __name__ == "__main__":
    main()
