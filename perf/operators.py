"""The operators next to the router, as measurable cases.

Six operators share one path, a mixture-of-experts layer around the router:
the load-balance loss and its gradient, the order of rows by expert, the
quantisers to 8-bit floating point with one power-of-two scale for each 128
values, the experts' products on such operands, and the weight gradient of
those products.  `run` computes a case in plain torch operations (`own` false)
or by this package's entry points (`own` true); `exact` states the same from
the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

FP8_MAX = 448.0  # the largest finite e4m3 value
EPS = 1e-20      # keeps a row of vanished sigmoid scores from dividing by zero


def listed():
    return [
        # one optimizer step's tokens of one router: 16 local batches of 32768 tokens
        dict(name="balance_loss_step", op="balance", N=524288, E=256, k=6, batch=32768,
             dtype="f32", score="sigmoid", masked=0.0, grad=False),
        # loss and gradient of a bf16 router's batch of 4 x 65536 tokens
        dict(name="balance_train_bf16", op="balance", N=262144, E=256, k=8, batch=65536,
             dtype="bf16", score="sigmoid", masked=0.0, grad=True),
        # a small router with padded sequences of 1000 tokens, the last one all padding
        dict(name="balance_train_padded", op="balance", N=4096, E=64, k=6, batch=1000,
             dtype="f32", score="softmax", masked=0.1, grad=True),
        # the dispatch of four microbatches
        dict(name="order_step", op="order", N=131072, E=256, k=6, dropped=0.0),
        # the dispatch of a few decoded tokens: latency
        dict(name="order_tokens", op="order", N=7, E=256, k=6, dropped=0.0),
        # a microbatch's hidden states gathered into expert order as they are quantised
        dict(name="quant_rows_gather", op="quant_rows", T=32768, M=196608, K=2048, dtype="bf16",
             gather=True),
        # the same values laid out for the weight gradient: scales along the tokens
        dict(name="quant_cols_step", op="quant_cols", T=16384, M=65536, K=2048, G=64,
             dtype="bf16", gather=True),
        # the experts' weights after an optimizer step, in both orientations
        dict(name="quant_weights", op="quant_blocks", G=64, N=1024, K=2048, dtype="bf16",
             both=True),
        # the experts' product of 16384 tokens routed to 6 of 256 experts
        dict(name="product_prompt", op="gemm", M=98304, G=256, N=1024, K=2048, out="bf16"),
        # the same layer for 8 decoded tokens
        dict(name="product_tokens", op="gemm", M=48, G=256, N=1024, K=2048, out="bf16"),
        # few experts, ragged rows, no size a multiple of a tile
        dict(name="product_odd", op="gemm", M=1003, G=5, N=333, K=1136, out="f32"),
        # the weight gradient of 64 experts
        dict(name="wgrad_step", op="wgrad", M=65536, G=64, N=1024, K=2048, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, unit, lo, hi):
    """A power of two or an odd multiple of unit, between lo and hi units."""
    n = _log(rng, lo, hi)
    return unit * (1 << n.bit_length() - 1 if rng.random() < 0.4 else n | 1)


def draw(rng):
    """One more case of the listed ones' ranges, at most the largest one's work."""
    case = _draw(rng)
    while work(case)["bytes"] > 900e6:
        rows = "M" if "M" in case else "G" if "G" in case else "N"
        case[rows] = case[rows] * 2 // 3
        if "T" in case:
            case["T"] = min(case["T"], case[rows])
    return case


def _draw(rng):
    op = rng.choice(["balance", "balance", "order", "quant_rows", "quant_cols", "quant_blocks",
                     "gemm", "gemm", "wgrad"])
    if op == "balance":
        E = 32 * rng.choice([1, 2, 3, 5, 8, 8, 12, 16, 32])
        grad = rng.random() < 0.6
        N = _log(rng, 1, (262144 if grad else 524288) * 256 // max(E, 256))
        return dict(op=op, N=N, E=E, k=rng.randint(1, min(15, E - 1)),
                    batch=rng.choice([0, _log(rng, max(1, N // 64), N)]),
                    dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["sigmoid", "softmax"]),
                    masked=rng.choice([0.0, 0.0, 0.1, 0.5]), grad=grad)
    if op == "order":
        E = 32 * rng.choice([1, 2, 3, 8, 8, 12, 32])
        return dict(op=op, N=_log(rng, 1, 131072), E=E, k=rng.randint(1, 8),
                    dropped=rng.choice([0.0, 0.0, 0.05]))
    if op == "quant_rows":
        K = _size(rng, 16, 1, 510)
        M = _log(rng, 1, 196608 * 2048 // max(K, 2048))
        return dict(op=op, T=max(1, M // rng.randint(1, 8)), M=M, K=K,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), gather=rng.random() < 0.6)
    if op == "quant_cols":
        K = _size(rng, 16, 1, 255)
        M = _log(rng, 1, 65536 * 2048 // max(K, 2048))
        return dict(op=op, T=max(1, M // rng.randint(1, 8)), M=M, K=K,
                    G=rng.choice([1, 3, 8, 64, 200]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    gather=rng.random() < 0.6)
    if op == "quant_blocks":
        N, K = _size(rng, 16, 1, 128), _size(rng, 16, 1, 128)
        return dict(op=op, G=_log(rng, 1, max(1, min(256, 64 * 1024 * 2048 // (N * K)))), N=N, K=K,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), both=rng.random() < 0.5)
    if op == "gemm":
        K = _size(rng, 16, 4, 256)
        N = rng.choice([_size(rng, 8, 5, 500), _size(rng, 1, 40, 4000)])
        G = min(rng.choice([1, 1, 6, 32, 256]), max(1, 256 * 1024 * 2048 // (N * K)))
        M = _log(rng, 1, max(2, min(98304, 98304 * 1024 * 2048 // (N * K))))
        return dict(op=op, M=M, G=G, N=N, K=K, out=rng.choice(["bf16", "bf16", "f32"]))
    K, N = _size(rng, 8, 8, 512), _size(rng, 8, 8, 512)
    G = min(rng.choice([1, 3, 16, 64]), max(1, 64 * 1024 * 2048 // (N * K)))
    M = _log(rng, 1, max(2, min(65536, 65536 * 1024 * 2048 // (N * K))))
    return dict(op="wgrad", M=M, G=G, N=N, K=K, out=rng.choice(["f32", "f32", "bf16"]))


# ------------------------------------------------------------------ inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _blocks(n):
    return -(-n // 128)


def _pitch(n):
    """Bytes of one row of scales: one for each 128 values, padded to whole 32-bit words."""
    return -(-_blocks(n) // 4) * 4


def _width(M, G):
    """Columns that M tokens in G groups need when every group starts at a multiple of 128."""
    return (M + 127 * G) // 128 * 128


def _offsets(g, M, G):
    """Row offsets of G experts with uneven loads, M rows in all."""
    load = torch.softmax(0.5 * _randn(g, G), 0)
    of = torch.multinomial(load, M, replacement=True, generator=g)
    sizes = torch.bincount(of, minlength=G)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    off[1:] = sizes.cumsum(0)
    return off, sizes.cpu()


def _activations(g, T, K, dtype):
    """Hidden states: unit rows with a few channels much larger than the rest."""
    channel = torch.exp(0.8 * _randn(g, K))
    return (_randn(g, T, K) * channel).to(_DT[dtype])


def _codes(g, rows, K, width=None):
    """8-bit operands [rows, K] with their scales, as a program keeps them."""
    q = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 27) // max(K, 1))
    for r in range(0, rows, step):
        n = min(step, rows - r)
        q[r:r + n] = (_randn(g, n, K) * 100.0).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    s = torch.randint(115, 122, (rows, _pitch(K)), generator=g, device="cuda", dtype=torch.uint8)
    return q, s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "balance":
        N, E, k = case["N"], case["E"], case["k"]
        nb = -(-N // case["batch"]) if case["batch"] else 1
        x = _randn(g, N, E) + 0.5 * _randn(g, E)
        bias = 0.1 * _randn(g, E)
        s["logits"] = x.to(_DT[case["dtype"]])
        s["topk"] = torch.topk(x + bias, k, dim=1).indices.to(torch.int32).sort(1).values
        s["mask"] = None
        if case["masked"]:
            m = torch.rand(N, generator=g, device="cuda") >= case["masked"]
            if nb > 1:
                m[(nb - 1) * case["batch"]:] = False
            s["mask"] = m
        s["coeff"] = 1e-2
        s["loss_grad"] = torch.rand(nb, generator=g, device="cuda") + 0.5
        s["counts"] = torch.empty(nb, E, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(nb, dtype=torch.int32, device="cuda")
        s["prob_sum"] = torch.empty(nb, E, device="cuda")
        s["loss"] = torch.empty(nb, device="cuda")
        s["dlogits"] = torch.empty(N, E, device="cuda") if case["grad"] else None
    elif op == "order":
        N, E, k = case["N"], case["E"], case["k"]
        x = _randn(g, N, E) + 0.7 * _randn(g, E)
        s["topk"] = torch.topk(x, k, dim=1).indices.to(torch.int32).sort(1).values
        if case["dropped"]:
            s["topk"][torch.rand(N, k, generator=g, device="cuda") < case["dropped"]] = -1
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["slot_of"] = torch.empty(N, k, dtype=torch.int32, device="cuda")
        s["token_of"] = torch.empty(N * k, dtype=torch.int32, device="cuda")
    elif op in ("quant_rows", "quant_cols"):
        T, M, K = case["T"] if case["gather"] else case["M"], case["M"], case["K"]
        s["x"] = _activations(g, T, K, case["dtype"])
        s["index"] = None
        if case["gather"]:
            s["index"] = torch.randint(0, T, (M,), generator=g, device="cuda", dtype=torch.int32)
        if op == "quant_rows":
            s["q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
            s["scale"] = torch.empty(M, _pitch(K), dtype=torch.uint8, device="cuda")
        else:
            W = _width(M, case["G"])
            s["offsets"] = _offsets(g, M, case["G"])[0]
            s["q"] = torch.empty(K, W, dtype=torch.float8_e4m3fn, device="cuda")
            s["scale"] = torch.empty(K, _pitch(W), dtype=torch.uint8, device="cuda")
    elif op == "quant_blocks":
        G, N, K = case["G"], case["N"], case["K"]
        s["w"] = (0.02 * _randn(g, G, N, K)).to(_DT[case["dtype"]])
        s["q"] = torch.empty(G, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty(G, _blocks(N), _pitch(K), dtype=torch.uint8, device="cuda")
        s["q_t"] = s["scale_t"] = None
        if case["both"]:
            s["q_t"] = torch.empty(G, K, N, dtype=torch.float8_e4m3fn, device="cuda")
            s["scale_t"] = torch.empty(G, _blocks(K), _pitch(N), dtype=torch.uint8, device="cuda")
    elif op == "gemm":
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        s["offsets"], sizes = _offsets(g, M, G)
        s["longest"] = int(sizes.max())
        s["a"], s["a_scale"] = _codes(g, M, K)
        q, _ = _codes(g, G * N, K)
        s["b"] = q.view(G, N, K)
        s["b_scale"] = torch.randint(112, 116, (G, _blocks(N), _pitch(K)), generator=g,
                                     device="cuda", dtype=torch.uint8)
        s["y"] = torch.empty(M, N, dtype=_DT[case["out"]], device="cuda")
    else:
        M, G, N, K = case["M"], case["G"], case["N"], case["K"]
        W = _width(M, G)
        s["offsets"], sizes = _offsets(g, M, G)
        s["longest"] = int(sizes.max())
        s["a"], s["a_scale"] = _codes(g, N, W)
        s["b"], s["b_scale"] = _codes(g, K, W)
        # past a group's last token the operands hold zeros, as the quantiser leaves them
        used = _column_source(s["offsets"], W) >= 0
        s["a"].view(torch.uint8).mul_(used)
        s["b"].view(torch.uint8).mul_(used)
        s["dw"] = torch.empty(G, N, K, dtype=_DT[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from exact_distributed_quantiles_gb300 import qb
    op = s["op"]
    if op == "balance":
        if "ws" not in s:
            s["ws"] = qb.balance_workspace(s["N"], s["E"], s["batch"])
        qb.qb_balance_loss(s["logits"], s["topk"], s["coeff"], s["counts"], s["tokens"],
                           s["prob_sum"], s["loss"], s["ws"], token_mask=s["mask"],
                           batch_tokens=s["batch"], score=s["score"])
        out = {n: s[n] for n in ("counts", "tokens", "prob_sum", "loss")}
        if s["grad"]:
            qb.qb_balance_grad(s["logits"], s["counts"], s["tokens"], s["loss_grad"], s["coeff"],
                               s["k"], s["dlogits"], token_mask=s["mask"],
                               batch_tokens=s["batch"], score=s["score"])
            out["dlogits"] = s["dlogits"]
        return out
    if op == "order":
        if "ws" not in s:
            s["ws"] = qb.order_workspace(s["N"], s["E"], s["k"])
        qb.qb_expert_order(s["topk"], s["E"], s["counts"], s["offsets"], s["slot_of"],
                           s["token_of"], s["ws"])
        return {n: s[n] for n in ("counts", "offsets", "slot_of", "token_of")}
    if op == "quant_rows":
        qb.qb_fp8_quantize_rows(s["x"], s["q"], s["scale"], row_idx=s["index"])
        return {"q": s["q"], "scale": s["scale"]}
    if op == "quant_cols":
        qb.qb_fp8_quantize_cols(s["x"], s["q"], s["scale"], offsets=s["offsets"],
                                row_idx=s["index"])
        return {"q": s["q"], "scale": s["scale"]}
    if op == "quant_blocks":
        qb.qb_fp8_quantize_blocks(s["w"], s["q"], s["scale"], q_t=s["q_t"], scale_t=s["scale_t"])
        out = {"q": s["q"], "scale": s["scale"]}
        return {**out, "q_t": s["q_t"], "scale_t": s["scale_t"]} if s["both"] else out
    if op == "gemm":
        qb.qb_fp8_expert_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"], s["y"],
                              offsets=s["offsets"])
        return s["y"]
    qb.qb_fp8_expert_wgrad(s["a"], s["a_scale"], s["b"], s["b_scale"], s["dw"],
                           offsets=s["offsets"])
    return s["dw"]


def _batched(s):
    """(number of local batches, each token's batch)."""
    N, bt = s["N"], s["batch"] or s["N"]
    nb = -(-N // bt)
    return nb, bt, torch.arange(N, device="cuda") // bt


def _per_batch(v, nb, bt):
    """Sums the rows of v over each batch."""
    pad = nb * bt - v.shape[0]
    if pad:
        v = torch.cat([v, v.new_zeros(pad, v.shape[1])])
    return v.view(nb, bt, v.shape[1]).sum(1)


def _plain_balance(s):
    nb, bt, batch = _batched(s)
    N, E, k = s["N"], s["E"], s["k"]
    live = s["mask"] if s["mask"] is not None else torch.ones(N, dtype=torch.bool, device="cuda")
    x = s["logits"].float()
    if s["score"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-x))
        total = sc.sum(1, keepdim=True) + EPS
    else:
        sc = torch.exp(x - x.amax(1, keepdim=True))
        total = sc.sum(1, keepdim=True)
    p = torch.where(live[:, None], sc / total, 0.0)
    flat = (batch[:, None] * E + s["topk"]).reshape(-1)
    ones = live.to(torch.int32)[:, None].expand(N, k).reshape(-1)
    counts = torch.zeros(nb * E, dtype=torch.int32, device="cuda").index_add_(0, flat, ones).view(nb, E)
    n = torch.zeros(nb, dtype=torch.int32, device="cuda").index_add_(0, batch, live.to(torch.int32))
    psum = _per_batch(p, nb, bt)
    nf = n.clamp(min=1).float()
    weight = s["coeff"] * E / (k * nf * nf)
    loss = weight * (counts.float() * psum).sum(1)
    out = {"counts": counts, "tokens": n, "prob_sum": psum, "loss": loss}
    if s["grad"]:
        w = ((s["loss_grad"] * weight)[:, None] * counts.float())[batch]
        d = w - (w * p).sum(1, keepdim=True)
        if s["score"] == "sigmoid":
            d = d / total * sc * (1.0 - sc)
        else:
            d = d * p
        out["dlogits"] = torch.where(live[:, None], d, 0.0)
    return out


def _plain_order(s):
    N, E, k = s["N"], s["E"], s["k"]
    flat = s["topk"].reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int32, device="cuda").index_add_(
        0, key, torch.ones_like(key, dtype=torch.int32))[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    place = torch.arange(N * k, dtype=torch.int32, device="cuda")
    slot = torch.empty_like(place)
    slot[order] = place
    slot = torch.where(flat < 0, -1, slot).to(torch.int32)
    token = torch.where(place < offsets[E], (order // k).to(torch.int32), -1)
    return {"counts": counts, "offsets": offsets, "slot_of": slot.view(N, k),
            "token_of": token.to(torch.int32)}


def _power(e):
    """2^e as fp32 for whole e in [-127, 127]."""
    return torch.where(e > -127, ((e + 127) << 23), 1 << 22).to(torch.int32).view(torch.float32)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, from -127 up."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e.clamp(-127, 127), -127).to(torch.int32)


def _plain_quant(x, rows, cols, pitch):
    """x [..., R, C] in blocks of rows x cols -> codes [..., R, C], exponent bytes [..., R / rows, pitch]."""
    R, C = x.shape[-2:]
    x = x.float()
    rb, cb = -(-R // rows), -(-C // cols)
    if (rb * rows, cb * cols) != (R, C):
        full = x.new_zeros(*x.shape[:-2], rb * rows, cb * cols)
        full[..., :R, :C] = x
        x = full
    v = x.view(*x.shape[:-2], rb, rows, cb, cols)
    a = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(-1).amax(-2)
    e = _exponent(a)
    q = (v * _power(-e)[..., :, None, :, None]).to(torch.float8_e4m3fn)
    q = q.view(*x.shape)[..., :R, :C].contiguous()
    scale = torch.zeros(*e.shape[:-1], pitch, dtype=torch.uint8, device=x.device)
    scale[..., :cb] = (e + 127).to(torch.uint8)
    return q, scale


def _column_source(offsets, width):
    """For each of `width` columns, groups starting at multiples of 128: its row, or -1."""
    off = offsets.long()
    size = off[1:] - off[:-1]
    end = ((size + 127) // 128 * 128).cumsum(0)
    j = torch.arange(width, device="cuda")
    g = torch.searchsorted(end, j, right=True)
    at = g.clamp(max=size.numel() - 1)
    r = j - (end - (size + 127) // 128 * 128)[at]
    return torch.where((g < size.numel()) & (r < size[at]), off[:-1][at] + r, -1)


def _dequant(q, scale, rows):
    """codes [..., R, C] times their scales, fp32; each row of scales serves `rows` rows."""
    R, C = q.shape[-2:]
    e = scale.to(torch.int32) - 127
    f = _power(e).repeat_interleave(rows, -2)[..., :R, :] if rows > 1 else _power(e)
    return q.float() * f.repeat_interleave(128, -1)[..., :C]


def _run_plain(s):
    op = s["op"]
    if op == "balance":
        return _plain_balance(s)
    if op == "order":
        return _plain_order(s)
    if op == "quant_rows":
        x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        q, scale = _plain_quant(x, 1, 128, _pitch(s["K"]))
        return {"q": q, "scale": scale}
    if op == "quant_cols":
        src = _column_source(s["offsets"], s["q"].shape[1])
        row = src.clamp(min=0) if s["index"] is None else s["index"].long()[src.clamp(min=0)]
        x = torch.where((src >= 0)[:, None], s["x"][row], 0.0)
        q, scale = _plain_quant(x.t(), 1, 128, _pitch(x.shape[0]))
        return {"q": q, "scale": scale}
    if op == "quant_blocks":
        q, scale = _plain_quant(s["w"], 128, 128, _pitch(s["K"]))
        out = {"q": q, "scale": scale}
        if s["both"]:
            out["q_t"], out["scale_t"] = _plain_quant(s["w"].transpose(1, 2), 128, 128, _pitch(s["N"]))
        return out
    off = s["offsets"].long()
    size = off[1:] - off[:-1]
    if op == "gemm":
        # every expert's rows padded to the longest expert's, one batched product
        j = torch.arange(s["longest"], device="cuda")
        at = (off[:-1, None] + j).clamp(max=s["M"] - 1)
        a = _dequant(s["a"], s["a_scale"], 1)[at]
        y = torch.bmm(a, _dequant(s["b"], s["b_scale"], 128).transpose(1, 2))
        row = torch.arange(s["M"], device="cuda")
        g = torch.searchsorted(off[1:], row, right=True)
        return y[g, row - off[:-1][g]].to(_DT[s["out"]])
    first = ((size + 127) // 128 * 128).cumsum(0) - (size + 127) // 128 * 128
    j = torch.arange(s["longest"], device="cuda")
    at = (first[:, None] + j).clamp(max=s["a"].shape[1] - 1)
    live = j < size[:, None]
    a = _dequant(s["a"], s["a_scale"], 1).t()[at] * live[..., None]
    b = _dequant(s["b"], s["b_scale"], 1).t()[at]
    return torch.bmm(a.transpose(1, 2), b).to(_DT[s["out"]])


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_balance(s):
    N, E, k, bt = s["N"], s["E"], s["k"], s["batch"] or s["N"]
    out = {"counts": [], "tokens": [], "prob_sum": [], "loss": []}
    grads = []
    for b, i in enumerate(range(0, N, bt)):
        x = s["logits"][i:i + bt].double()
        live = torch.ones(len(x), dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][i:i + bt]
        if s["score"] == "sigmoid":
            sc = torch.sigmoid(x)
            total = sc.sum(1, keepdim=True) + EPS
            p = sc / total
        else:
            p = torch.softmax(x, 1)
        p = p * live[:, None]
        c = torch.bincount(s["topk"][i:i + bt][live].reshape(-1).long(), minlength=E)
        n = int(live.sum())
        f = s["coeff"] * E / (k * n * n) if n else 0.0
        out["counts"].append(c.to(torch.int32))
        out["tokens"].append(torch.tensor(n, dtype=torch.int32))
        out["prob_sum"].append(p.sum(0))
        out["loss"].append(f * (c.double() * p.sum(0)).sum())
        if s["grad"]:
            w = float(s["loss_grad"][b].double()) * f * c.double()
            d = w - (p @ w)[:, None]
            d = d / total * sc * (1 - sc) if s["score"] == "sigmoid" else d * p
            grads.append(d * live[:, None])
    got = {n: torch.stack(v) for n, v in out.items()}
    if s["grad"]:
        got["dlogits"] = torch.cat(grads)
    return got


def _exact_order(s):
    key = s["topk"].reshape(-1).cpu().numpy()
    N, E, k = s["N"], s["E"], s["k"]
    kept = np.flatnonzero(key >= 0)
    order = kept[np.argsort(key[kept], kind="stable")]
    counts = np.bincount(key[kept], minlength=E)
    slot = np.full(N * k, -1, np.int32)
    slot[order] = np.arange(len(order))
    token = np.full(N * k, -1, np.int32)
    token[:len(order)] = order // k
    return {"counts": counts.astype(np.int32),
            "offsets": np.concatenate([[0], np.cumsum(counts)]).astype(np.int32),
            "slot_of": slot.reshape(N, k), "token_of": token}


def _exact_codes(x, rows):
    """Codes' values (fp64) and exponent bytes of x [R, C] in blocks of rows x 128, one block row at a time."""
    q = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    scale = torch.zeros(-(-x.shape[0] // rows), _pitch(x.shape[1]), dtype=torch.uint8, device="cuda")
    for c in range(0, x.shape[1], 128):
        v = x[:, c:c + 128].double()
        a = v.abs().amax(1)
        if rows > 1:
            a = torch.stack([t.max() for t in a.split(rows)])
        e = torch.ceil(torch.log2(a / FP8_MAX))
        e = torch.where(a > FP8_MAX * torch.exp2(e), e + 1, e)
        e = torch.where(a <= FP8_MAX * torch.exp2(e - 1), e - 1, e).clamp(-127, 127)
        scale[:, c // 128] = (e + 127).to(torch.uint8)
        v = v * torch.exp2(-e).repeat_interleave(rows)[:len(x), None]
        low = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(low - 3)
        q[:, c:c + 128] = torch.round(v / step) * step
    return q, scale


def _value(q, scale, rows):
    """What codes [R, C] and their scales stand for, fp64."""
    f = torch.exp2(scale.double() - 127.0).repeat_interleave(rows, 0)[:q.shape[0]]
    return q.double() * f.repeat_interleave(128, 1)[:, :q.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "balance":
        return _exact_balance(s)
    if op == "order":
        return _exact_order(s)
    if op == "quant_rows":
        x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        q, scale = _exact_codes(x, 1)
        return {"q": q, "scale": scale}
    off = s["offsets"].tolist() if "offsets" in s else []
    if op == "quant_cols":
        x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        full = torch.zeros(s["q"].shape[1], s["K"], dtype=x.dtype, device="cuda")
        at = 0
        for lo, hi in zip(off, off[1:]):
            full[at:at + hi - lo] = x[lo:hi]
            at += _blocks(hi - lo) * 128
        q, scale = _exact_codes(full.t(), 1)
        return {"q": q, "scale": scale}
    if op == "quant_blocks":
        got = [_exact_codes(w, 128) for w in s["w"]]
        out = {"q": torch.stack([q for q, _ in got]), "scale": torch.stack([e for _, e in got])}
        if s["both"]:
            got = [_exact_codes(w.t(), 128) for w in s["w"]]
            out["q_t"] = torch.stack([q for q, _ in got])
            out["scale_t"] = torch.stack([e for _, e in got])
        return out
    if op == "gemm":
        y = torch.empty(s["M"], s["N"], dtype=torch.float64, device="cuda")
        for i, (lo, hi) in enumerate(zip(off, off[1:])):
            if hi > lo:
                y[lo:hi] = _value(s["a"][lo:hi], s["a_scale"][lo:hi], 1) @ _value(s["b"][i], s["b_scale"][i], 128).t()
        return y
    dw = torch.zeros(s["G"], s["N"], s["K"], dtype=torch.float64, device="cuda")
    at = 0
    for i, (lo, hi) in enumerate(zip(off, off[1:])):
        c = slice(at // 128, at // 128 + _blocks(hi - lo))
        cols = slice(at, at + hi - lo)
        if hi > lo:
            dw[i] = (_value(s["a"][:, cols], s["a_scale"][:, c], 1)
                     @ _value(s["b"][:, cols], s["b_scale"][:, c], 1).t())
        at += _blocks(hi - lo) * 128
    return dw


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "balance":
        N, E, k = case["N"], case["E"], case["k"]
        nb = -(-N // case["batch"]) if case["batch"] else 1
        b = N * E * size + N * k * 4 + (N if case["masked"] else 0) + nb * (8 * E + 8)
        f = 5 * N * E
        if case["grad"]:
            b += N * E * 4
            f += 10 * N * E
        return {"bytes": b, "flops": f}
    if op == "order":
        return {"bytes": 12 * case["N"] * case["k"] + 8 * case["E"], "flops": case["N"] * case["k"]}
    if op in ("quant_rows", "quant_cols"):
        M, K = case["M"], case["K"]
        rows = min(case["T"], M) if case["gather"] else M
        out = M * K + M * _pitch(K)
        if op == "quant_cols":
            W = _width(M, case["G"])
            out = K * W + K * _pitch(W)
        return {"bytes": rows * K * size + out + (4 * M if case["gather"] else 0), "flops": 2 * M * K}
    if op == "quant_blocks":
        n = case["G"] * case["N"] * case["K"]
        return {"bytes": n * (size + (2 if case["both"] else 1)), "flops": 2 * n}
    M, G, N, K = case["M"], case["G"], case["N"], case["K"]
    out = 4 if case["out"] == "f32" else 2
    if op == "gemm":
        # with few rows not every expert's weights are needed: the rows fall on this many
        hit = G * (1 - (1 - 1 / G) ** M)
        return {"bytes": M * K + hit * N * K + M * N * out, "flops": 2 * M * N * K}
    return {"bytes": M * (N + K) + G * N * K * out, "flops": 2 * M * N * K}
