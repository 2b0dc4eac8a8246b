"""Plain 64-bit statements of the balance loss, the expert order, the 8-bit
operands and the experts' products, which the tests compare the kernels with."""
import numpy as np

EPS = 1e-20


def batches(N, batch):
    step = batch or N
    return [(i, min(N, i + step)) for i in range(0, N, step)]


def shares(x, score):
    x = np.asarray(x, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-x))
        total = s.sum(1, keepdims=True) + EPS
        return s / total, s, total
    m = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(m), 0.0, m))
    total = e.sum(1, keepdims=True)
    return e / np.where(total == 0, 1.0, total), e, total


def balance(x, topk, mask, coeff, batch, score, loss_grad=None):
    """counts, tokens, prob_sum, loss and, per element, the gradient and the size of the terms whose
    difference it is."""
    N, E = x.shape
    k = topk.shape[1]
    out = {n: [] for n in ("counts", "tokens", "prob_sum", "loss")}
    grad, size = np.zeros((N, E)), np.zeros((N, E))
    for b, (lo, hi) in enumerate(batches(N, batch)):
        live = np.ones(hi - lo, bool) if mask is None else np.asarray(mask[lo:hi], bool)
        t = topk[lo:hi][live].reshape(-1)
        c = np.bincount(t[(t >= 0) & (t < E)], minlength=E)
        n = int(live.sum())
        p, s, total = shares(x[lo:hi][live], score)
        f = coeff * E / (k * n * n) if n else 0.0
        P = p.sum(0) if n else np.zeros(E)
        out["counts"].append(c)
        out["tokens"].append(n)
        out["prob_sum"].append(P)
        out["loss"].append(f * float((c * P).sum()))
        if loss_grad is not None and n:
            w = float(loss_grad[b]) * f * c
            d = w - (p @ w)[:, None]
            front = s * (1.0 - s) / total if score == "sigmoid" else p
            spread = np.abs(w - w.mean())
            grad[lo:hi][live] = front * d
            size[lo:hi][live] = front * (spread + (p @ spread)[:, None])
    return {n: np.array(v) for n, v in out.items()}, grad, size


def order(topk, E):
    flat = topk.reshape(-1)
    k = topk.shape[1]
    kept = np.flatnonzero((flat >= 0) & (flat < E))
    by = kept[np.argsort(flat[kept], kind="stable")]
    counts = np.bincount(flat[kept], minlength=E)
    slot = np.full(flat.size, -1, np.int64)
    slot[by] = np.arange(by.size)
    token = np.full(flat.size, -1, np.int64)
    token[:by.size] = by // k
    return counts, np.concatenate([[0], np.cumsum(counts)]), slot.reshape(topk.shape), token


def e4m3(v):
    """Nearest e4m3 value, ties to even, of finite v with |v| <= 448."""
    low = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = np.exp2(low - 3)
    return np.rint(v / step) * step


def exponent(amax):
    with np.errstate(divide="ignore"):
        e = np.ceil(np.log2(amax / 448.0))
    e = np.where(amax > 448.0 * np.exp2(e), e + 1, e)
    e = np.where((amax > 0) & (amax <= 448.0 * np.exp2(e - 1)), e - 1, e)
    return np.clip(e, -127, 127)


def pitch(n):
    return -(-(-(-n // 128)) // 4) * 4


def quantize(x, rows):
    """Codes' values and scale bytes of x [R, C] in blocks of rows x 128."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    q = np.empty((R, C))
    scale = np.zeros((-(-R // rows), pitch(C)), np.uint8)
    for i in range(0, R, rows):
        for j in range(0, C, 128):
            v = x[i:i + rows, j:j + 128]
            fin = np.isfinite(v)
            e = exponent(np.abs(np.where(fin, v, 0.0)).max())
            q[i:i + rows, j:j + 128] = np.where(fin, e4m3(np.where(fin, v, 0.0) * 2.0 ** -e), np.nan)
            scale[i // rows, j // 128] = int(e) + 127
    return q, scale


def grouped_columns(x, offsets, width):
    """x [M, K] -> [K, width], every group at a multiple of 128, zeros between."""
    out = np.zeros((x.shape[1], width))
    at = 0
    for lo, hi in zip(offsets, offsets[1:]):
        out[:, at:at + hi - lo] = x[lo:hi].T
        at += -(-(hi - lo) // 128) * 128
    return out


def value(q, scale, rows=1):
    f = np.exp2(scale.astype(np.float64) - 127.0).repeat(rows, 0)[:q.shape[0]]
    return q * f.repeat(128, 1)[:, :q.shape[1]]
