"""The 8-bit quantisers and the experts' products against the 64-bit statements.

Codes and scales are defined exactly (one rounding), so they are compared bit for bit as values.
A product of fp32 output is within (S + 24) * 2^-23 of sum |A| |B|: S MMA steps of 32 values whose
additions may truncate (one unit each; S <= 64, longer sums go on in registers, one rounding for
each further 2048 values), and 24 for the additions within a step and the joins.  bf16 output is
the fp32 output rounded once, bit for bit."""
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


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def source(T, K, dtype, seed):
    g = gen(seed)
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.exp(2.0 * torch.randn(T, 1, generator=g, device="cuda"))
    x *= torch.exp(torch.randn(K, generator=g, device="cuda"))
    return x.to(dtype)


def codes_equal(q, want):
    got = q.view(torch.float8_e4m3fn).double().cpu().numpy()
    return np.array_equal(got, want, equal_nan=True)


def blank(*shape):
    return torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")


def split(M, G, seed):
    """Ascending offsets of G groups with M rows, some empty."""
    cut = torch.sort(torch.randint(0, M + 1, (G - 1,), generator=gen(seed), device="cuda")).values
    ends = torch.tensor([M], device="cuda")
    return torch.cat([torch.zeros(1, device="cuda", dtype=torch.long), cut, ends]).to(torch.int32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,gather", [(1, 16, False), (1, 2048, True), (5, 128, False),
                                        (33, 144, True), (130, 528, False), (77, 4112, True)])
def test_quantize_rows(qb, M, K, gather, dtype):
    T = M if not gather else M // 2 + 1
    x = source(T, K, dtype, M + K)
    index = None
    if gather:
        index = torch.randint(0, T, (M,), generator=gen(K), device="cuda", dtype=torch.int32)
        index[M // 2] = -1
        if M > 3:
            index[3] = T  # outside: zeros
    q, s = blank(M, K), blank(M, ref.pitch(K))
    qb.qb_fp8_quantize_rows(x, q, s, row_idx=index)
    h = x.double().cpu().numpy()
    if gather:
        i = index.cpu().numpy()
        h = np.where(((i >= 0) & (i < T))[:, None], h[np.clip(i, 0, T - 1)], 0.0)
    want, scale = ref.quantize(h, 1)
    assert codes_equal(q, want) and np.array_equal(s.cpu().numpy(), scale)


def test_quantize_values_at_the_edges(qb):
    x = torch.zeros(12, 256, device="cuda")
    x[0, 5] = 448.0            # exactly the largest code
    x[1, 5] = 448.0 * (1 + 2 ** -23)
    x[2, 5], x[2, 6] = float("inf"), 3.0
    x[3, 5], x[3, 6] = float("nan"), -3.0
    x[4, 5] = 3.4e38
    x[5, 5], x[5, 6] = 1e-40, 2e-45  # subnormal inputs
    x[6, 5] = 1.17e-38
    x[7, 5], x[7, 200] = float("-inf"), 1e-30
    x[8, :128] = torch.arange(128, device="cuda") * 0.5 - 30.0
    x[9, 0], x[9, 1] = 0.875 * 2.0 ** -20, 2.0 ** -40
    x[10] = -0.0
    x[11, 0], x[11, 1], x[11, 2] = 448.0, 2.0 ** -10, 3 * 2.0 ** -10  # ties at the smallest codes
    q, s = blank(12, 256), blank(12, 4)
    qb.qb_fp8_quantize_rows(x, q, s)
    want, scale = ref.quantize(x.double().cpu().numpy(), 1)
    assert codes_equal(q, want) and np.array_equal(s.cpu().numpy(), scale)
    q3, s3, qt, st = blank(1, 12, 256), blank(1, 1, 4), blank(1, 256, 16), blank(1, 2, 4)
    w = torch.zeros(1, 16, 256, device="cuda")
    w[0, :12] = x
    q3, s3 = blank(1, 16, 256), blank(1, 1, 4)
    qb.qb_fp8_quantize_blocks(w, q3, s3, q_t=qt, scale_t=st)
    want, scale = ref.quantize(w[0].double().cpu().numpy(), 128)
    assert codes_equal(q3[0], want) and np.array_equal(s3[0].cpu().numpy(), scale)
    assert codes_equal(qt[0], want.T)
    wt, scale_t = ref.quantize(w[0].double().cpu().numpy().T, 128)
    assert np.array_equal(st[0].cpu().numpy(), scale_t)
    qc, sc = blank(256, 128), blank(256, 4)
    qb.qb_fp8_quantize_cols(x, qc, sc)
    want, scale = ref.quantize(ref.grouped_columns(x.double().cpu().numpy(), [0, 12], 128), 1)
    assert codes_equal(qc, want) and np.array_equal(sc.cpu().numpy(), scale)


def test_quantize_strided_rows(qb):
    big = source(40, 512, torch.bfloat16, 1)
    x = big[3:30:2, 64:64 + 160]
    q, s = blank(14, 160), blank(14, 4)
    qb.qb_fp8_quantize_rows(x, q, s)
    want, scale = ref.quantize(x.double().cpu().numpy(), 1)
    assert codes_equal(q, want) and np.array_equal(s.cpu().numpy(), scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,K,G,gather", [(1, 16, 1, False), (5, 16, 3, True), (300, 144, 7, True),
                                          (128, 256, 1, False), (1000, 80, 40, False),
                                          (700, 400, 1, True), (900, 48, 1024, False)])
def test_quantize_cols(qb, M, K, G, gather, dtype):
    T = M // 3 + 1 if gather else M
    x = source(T, K, dtype, M + K)
    index = torch.randint(0, T, (M,), generator=gen(K), device="cuda", dtype=torch.int32) if gather else None
    off = split(M, G, M)
    width = qb.fp8_cols_width(M, G)
    q, s = blank(K, width), blank(K, ref.pitch(width))
    qb.qb_fp8_quantize_cols(x, q, s, offsets=off if G > 1 else None, row_idx=index)
    h = x.double().cpu().numpy()
    h = h[index.cpu().numpy()] if gather else h
    want, scale = ref.quantize(ref.grouped_columns(h, off.tolist(), width), 1)
    assert codes_equal(q, want) and np.array_equal(s.cpu().numpy(), scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G,N,K,both", [(1, 1, 16, False), (3, 16, 16, True), (2, 130, 272, False),
                                        (5, 144, 400, True), (1, 256, 128, True)])
def test_quantize_blocks(qb, G, N, K, both, dtype):
    w = source(G * N, K, dtype, N + K).view(G, N, K)
    q, s = blank(G, N, K), blank(G, -(-N // 128), ref.pitch(K))
    qt = blank(G, K, N) if both else None
    st = blank(G, -(-K // 128), ref.pitch(N)) if both else None
    qb.qb_fp8_quantize_blocks(w, q, s, q_t=qt, scale_t=st)
    for g in range(G):
        h = w[g].double().cpu().numpy()
        want, scale = ref.quantize(h, 128)
        assert codes_equal(q[g], want) and np.array_equal(s[g].cpu().numpy(), scale)
        if both:
            want, scale = ref.quantize(h.T, 128)
            assert codes_equal(qt[g], want) and np.array_equal(st[g].cpu().numpy(), scale)


# ------------------------------------------------------------------ products

def operand(rows, K, seed, scale_rows=1):
    g = gen(seed)
    v = (torch.randn(rows, K, generator=g, device="cuda") * 60).clamp(-448, 448)
    q = v.to(torch.float8_e4m3fn)
    s = torch.randint(117, 124, (-(-rows // scale_rows), ref.pitch(K)), generator=g, device="cuda",
                      dtype=torch.uint8)
    return q, s


def host(q, s, rows=1):
    return ref.value(q.double().cpu().numpy(), s.cpu().numpy(), rows)


def close(got, want, size, K):
    tol = (min(-(-K // 32), 64) + -(-K // 2048) + 24) * 2.0 ** -23 * size
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


GEMM = [(1, 1, 1, 16), (1, 3, 64, 128), (7, 1, 40, 80), (128, 1, 128, 512), (129, 2, 333, 144),
        (300, 5, 260, 1136), (40, 200, 96, 272), (513, 3, 1024, 2064), (1000, 64, 72, 48),
        (5000, 2, 520, 256), (64, 1, 256, 6160), (700, 1024, 40, 48)]


@pytest.mark.parametrize("M,G,N,K", GEMM)
def test_expert_gemm(qb, M, G, N, K):
    a, sa = operand(M, K, M + 1)
    b, sb = [], []
    for g in range(G):
        q, s = operand(N, K, 1000 + g, 128)
        b.append(q)
        sb.append(s)
    b, sb = torch.stack(b), torch.stack(sb)
    off = split(M, G, M + N)
    y = torch.full((M, N), float("nan"), device="cuda")
    y16 = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16)
    for out in (y, y16):
        qb.qb_fp8_expert_gemm(a, sa, b, sb, out, offsets=off if G > 1 else None)
    torch.cuda.synchronize()
    assert torch.equal(y16, y.to(torch.bfloat16))
    assert qb.device_status() == 0
    A, o = host(a, sa), off.tolist()
    for g in range(G):
        if o[g + 1] > o[g]:
            B, r = host(b[g], sb[g], 128), slice(o[g], o[g + 1])
            close(y[r], A[r] @ B.T, np.abs(A[r]) @ np.abs(B).T, K)


def test_rows_outside_the_groups_stay(qb):
    M, N, K = 300, 72, 144
    a, sa = operand(M, K, 1)
    b, sb = operand(2 * N, K, 2)[0].view(2, N, K), blank(2, 1, 4).fill_(120)
    off = torch.tensor([5, 5, 200], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), 7.0, device="cuda")
    qb.qb_fp8_expert_gemm(a, sa, b, sb, y, offsets=off)
    assert bool((y[:5] == 7).all()) and bool((y[200:] == 7).all())
    A, B = host(a, sa)[5:200], host(b[1], sb[1], 128)
    close(y[5:200], A @ B.T, np.abs(A) @ np.abs(B).T, K)


def test_nan_codes_stay_in_their_row_and_column(qb):
    M, N, K = 150, 200, 256
    a, sa = operand(M, K, 1)
    b, sb = operand(N, K, 2, 128)
    a.view(torch.uint8)[17, 30] = 0x7F
    b.view(torch.uint8)[140, 200] = 0xFF
    y = torch.empty(M, N, device="cuda")
    qb.qb_fp8_expert_gemm(a, sa, b.view(1, N, K), sb.view(1, -1, sb.shape[1]), y)
    bad = torch.isnan(y).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[17], want[:, 140] = True, True
    assert np.array_equal(bad, want)


WGRAD = [(1, 1, 1, 1), (5, 3, 16, 16), (300, 7, 200, 136), (129, 1, 128, 256), (1000, 40, 72, 33),
         (9000, 2, 130, 264), (400, 3, 640, 1032)]


@pytest.mark.parametrize("M,G,N,K", WGRAD)
def test_expert_wgrad(qb, M, G, N, K):
    width = qb.fp8_cols_width(M, G)
    off = split(M, G, M + N)
    a, sa = operand(N, width, 1)
    b, sb = operand(K, width, 2)
    o, at, cols = off.tolist(), 0, np.zeros(width, bool)
    where = []
    for g in range(G):
        n = o[g + 1] - o[g]
        where.append((at, at + n))
        cols[at:at + n] = True
        at += -(-n // 128) * 128
    live = torch.from_numpy(cols).cuda()
    a.view(torch.uint8).mul_(live)
    b.view(torch.uint8).mul_(live)
    dw = torch.full((G, N, K), float("nan"), device="cuda")
    dw16 = torch.full((G, N, K), float("nan"), device="cuda", dtype=torch.bfloat16)
    for out in (dw, dw16):
        qb.qb_fp8_expert_wgrad(a, sa, b, sb, out, offsets=off if G > 1 else None)
    torch.cuda.synchronize()
    assert torch.equal(dw16, dw.to(torch.bfloat16))
    assert qb.device_status() == 0
    A, B = host(a, sa), host(b, sb)
    for g, (lo, hi) in enumerate(where):
        close(dw[g], A[:, lo:hi] @ B[:, lo:hi].T, np.abs(A[:, lo:hi]) @ np.abs(B[:, lo:hi]).T,
              max(32, hi - lo + 127))
    before = torch.randn(G, N, K, device="cuda")
    total = before.clone()
    qb.qb_fp8_expert_wgrad(a, sa, b, sb, total, offsets=off if G > 1 else None, accumulate=True)
    assert torch.equal(total, before + dw)


def test_groups_without_any_row(qb):
    # offsets of nothing: a product writes nothing, a weight gradient is zeros
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, sa = operand(50, 64, 1)
    b, sb = operand(3 * 32, 64, 2)[0].view(3, 32, 64), blank(3, 1, 4).fill_(120)
    y = torch.full((50, 32), 7.0, device="cuda")
    qb.qb_fp8_expert_gemm(a, sa, b, sb, y, offsets=off)
    assert bool((y == 7).all())
    at, st = operand(24, 384, 3)
    dw = torch.full((3, 24, 24), float("nan"), device="cuda")
    qb.qb_fp8_expert_wgrad(at, st, at, st, dw, offsets=off)
    assert not dw.any()
    kept = torch.randn(3, 24, 24, device="cuda")
    total = kept.clone()
    qb.qb_fp8_expert_wgrad(at, st, at, st, total, offsets=off, accumulate=True)
    assert torch.equal(total, kept)
    q, s = blank(64, qb.fp8_cols_width(50, 3)), blank(64, ref.pitch(qb.fp8_cols_width(50, 3)))
    qb.qb_fp8_quantize_cols(source(50, 64, torch.float32, 1), q, s, offsets=off)
    assert not q.any() and not s.any()
    empty = torch.empty(0, 64, device="cuda")
    qb.qb_fp8_quantize_rows(source(5, 64, torch.float32, 1), empty.to(torch.uint8),
                            torch.empty(0, 4, dtype=torch.uint8, device="cuda"),
                            row_idx=torch.empty(0, dtype=torch.int32, device="cuda"))
    qb.qb_fp8_expert_gemm(empty.to(torch.uint8), torch.empty(0, 4, dtype=torch.uint8, device="cuda"),
                          b, sb, empty[:, :32].contiguous(), offsets=off)
    torch.cuda.synchronize()
    assert qb.device_status() == 0


def test_products_repeat_bit_for_bit_on_another_stream_and_in_a_graph(qb):
    M, G, N, K = 700, 6, 264, 528
    a, sa = operand(M, K, 1)
    b, sb = operand(G * N, K, 2)[0].view(G, N, K), torch.full((G, 3, 8), 119, dtype=torch.uint8, device="cuda")
    off = split(M, G, 3)
    y = torch.empty(M, N, device="cuda")
    qb.qb_fp8_expert_gemm(a, sa, b, sb, y, offsets=off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    z = torch.empty_like(y)
    qb.qb_fp8_expert_gemm(a, sa, b, sb, z, offsets=off, stream=s)
    s.synchronize()
    assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qb.qb_fp8_expert_gemm(a, sa, b, sb, z, offsets=off)
    z.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, z)


def test_offsets_past_32_bits(qb):
    # codes of 2.2e9 values, every row a copy of one of 8
    T, M, K = 8, 140000, 16384
    x = source(T, K, torch.bfloat16, 1)
    index = (torch.arange(M, device="cuda") % T).to(torch.int32)
    q = torch.empty(M, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(M, K // 128, dtype=torch.uint8, device="cuda")
    qb.qb_fp8_quantize_rows(x, q, s, row_idx=index)
    want, scale = ref.quantize(x.double().cpu().numpy(), 1)
    assert codes_equal(q[-T:], want) and np.array_equal(s[-T:].cpu().numpy(), scale)
    assert torch.equal(q[-T:], q[:T])
    del x
    # a product of 2.2e9 outputs from those rows
    N, Kn = 16400, 64
    a, sa = q[:, :Kn].contiguous(), s[:, :4].contiguous()
    b, sb = operand(N, Kn, 3, 128)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    qb.qb_fp8_expert_gemm(a, sa, b.view(1, N, Kn), sb.view(1, -1, 4), y)
    A, B = host(a[-T:].view(torch.float8_e4m3fn), sa[-T:]), host(b, sb, 128)
    few = torch.empty(T, N, device="cuda")
    qb.qb_fp8_expert_gemm(a[-T:], sa[-T:], b.view(1, N, Kn), sb.view(1, -1, 4), few)
    close(few, A @ B.T, np.abs(A) @ np.abs(B).T, Kn)
    assert torch.equal(y[-T:], few.to(torch.bfloat16)) and torch.equal(y[:T], y[-T:])


# ------------------------------------------------------------------ refusals

def test_the_binding_refuses(qb):
    x = source(32, 64, torch.float32, 1)
    q, s = blank(32, 64), blank(32, 4)
    qb.qb_fp8_quantize_rows(x, q, s)
    with pytest.raises(TypeError):
        qb.qb_fp8_quantize_rows(x.double(), q, s)
    with pytest.raises(ValueError):
        qb.qb_fp8_quantize_rows(x, q, blank(32, 1))
    with pytest.raises(ValueError):
        qb.qb_fp8_quantize_rows(x.t(), blank(64, 32), blank(64, 4))
    with pytest.raises(TypeError):
        qb.qb_fp8_quantize_rows(x, q, s, row_idx=torch.zeros(32, dtype=torch.int64, device="cuda"))
    with pytest.raises(qb.QBError):  # K not a multiple of 16
        qb.qb_fp8_quantize_rows(x[:, :24].contiguous(), blank(32, 24), s)
    with pytest.raises(qb.QBError):  # codes not on 16 bytes
        qb.qb_fp8_quantize_rows(x, blank(32 * 64 + 8)[8:].view(32, 64), s)
    with pytest.raises(qb.QBError):  # narrower than the groups need
        qb.qb_fp8_quantize_cols(x, blank(64, 128), blank(64, 4), offsets=split(32, 3, 1))
    with pytest.raises(TypeError):   # both or neither of the transposed pair
        qb.qb_fp8_quantize_blocks(x.view(1, 32, 64), q.view(1, 32, 64), blank(1, 1, 4),
                                  q_t=blank(1, 64, 32))
    b, sb, y = blank(2, 16, 64), blank(2, 1, 4), torch.empty(32, 16, device="cuda")
    with pytest.raises(TypeError):   # two groups want offsets
        qb.qb_fp8_expert_gemm(q, s, b, sb, y)
    with pytest.raises(ValueError):
        qb.qb_fp8_expert_gemm(q, s, b, sb, y, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        qb.qb_fp8_expert_gemm(q, s, b, sb, y.half(), offsets=split(32, 2, 1))
    at, st = blank(16, 128), blank(16, 4)
    with pytest.raises(qb.QBError):  # only fp32 accumulates
        qb.qb_fp8_expert_wgrad(at, st, at, st, torch.empty(1, 16, 16, dtype=torch.bfloat16, device="cuda"),
                               accumulate=True)
    torch.cuda.synchronize()
    assert qb.device_status() == 0
