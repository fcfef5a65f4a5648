"""The calls of lp_moe.h past 2^32 bytes and elements, on inputs drawn on the
device, against whole-tensor identities and sampled rows (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def sample(n):
    return torch.tensor(sorted({0, 1, *range(0, n, n // 9), n - 2, n - 1}), device="cuda")


def randn_bf16(shape, g):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def test_rows_past_2_to_32_elements(lp):
    T, k, H = (1 << 18) + 5, 2, 8208                     # 2^32 + 8.6e6 elements of rows
    g = gen(1)
    x = randn_bf16((T, H), g)
    e = torch.randint(0, 7, (T, k), generator=g, device="cuda").int()
    off, rows, order = lp.lp_moe_sort(e, 7)
    y = lp.lp_moe_gather(x, rows)
    r = sample(T * k)
    assert torch.equal(y[r], x[order[r].long() // k])
    # quantized: what the gathered rows give, all of it
    q = [(a.codes, a.scales) for a in lp.lp_moe_gather_quant(x, order, off, k)]
    want = [(a.codes, a.scales) for a in lp.lp_r128_quant_dual(y, off)]
    ends = [0, *off.tolist()]
    for (a, b), (c, d) in zip(q, want):
        assert torch.equal(a, c)
        if b.shape[2] == T * k:
            assert torch.equal(b, d)
        for i in range(7):
            at = slice(ends[i] // 128 + i, ends[i] // 128 + i + (ends[i + 1] - ends[i] + 127) // 128)
            assert b.shape[2] == T * k or torch.equal(b[:, at], d[:, at])
    del q, want, a, b, c, d
    # back: distinct values by row
    y.mul_(torch.rand(T * k, 1, generator=g, device="cuda").bfloat16())
    w = torch.rand(T, k, generator=g, device="cuda")
    out = lp.lp_moe_combine(y, rows, w)
    t = sample(T)
    terms = y[rows[t].long()].double() * w[t].double()[:, :, None]
    size = terms.abs().sum(1)
    assert ((out[t].double() - terms.sum(1)).abs() <= U16 * terms.sum(1).abs() + 4 * U32 * size + 2.0 ** -133).all()
    gy, gw = lp.lp_moe_combine_bwd(x, y, rows, w)
    dots = (x[t].double()[:, None] * y[rows[t].long()].double())
    assert ((gw[t].double() - dots.sum(2)).abs() <= H * U32 * dots.abs().sum(2)).all()
    want = (x[t].float()[:, None] * w[t][:, :, None]).bfloat16()
    assert torch.equal(gy[rows[t].long()], want)


@pytest.mark.parametrize("T,k,H", [(1 << 18, 4, 64), ((1 << 18) + 1, 1, 264), (17000, 4, 1024), (900, 8, 7168), (511, 9, 8200), (5000, 3, 4096)])
def test_gradients_of_rows_past_the_caches(lp, T, k, H):
    """More than 64 MB of rows, by every number of threads a token can have: each result alone and both."""
    g = gen(7)
    x, y = randn_bf16((T, H), g), randn_bf16((T * k, H), g)
    e = torch.randint(-1, 9, (T, k), generator=g, device="cuda").int()
    _, rows, _ = lp.lp_moe_sort(e, 9)
    w = torch.rand(T, k, generator=g, device="cuda")
    gy, gw = lp.lp_moe_combine_bwd(x, y, rows, w)
    assert torch.equal(gw, lp.lp_moe_combine_bwd(x, y, rows, w, need_dy=False)[1])
    live = rows.reshape(-1) >= 0
    r = rows.reshape(-1)[live].long()
    assert torch.equal(gy[r], lp.lp_moe_combine_bwd(x, None, rows, w, need_dw=False)[0][r])
    t = sample(T)
    dots = x[t].double()[:, None] * y[rows[t].clamp(min=0).long()].double() * (rows[t] >= 0)[:, :, None]
    assert ((gw[t].double() - dots.sum(2)).abs() <= H * U32 * dots.abs().sum(2)).all()
    pair = sample(T * k)
    pair = pair[live[pair]]
    want = (x[pair // k].float() * w.reshape(-1)[pair][:, None]).bfloat16()
    assert torch.equal(gy[rows.reshape(-1)[pair].long()], want)


def test_gate_past_2_to_32_elements(lp):
    T, E, k = (1 << 22) + 3, 1024, 2
    l = randn_bf16((T, E), gen(2))
    w, e = lp.lp_moe_gate(l, k)
    gw = torch.rand(T, k, generator=gen(3), device="cuda")
    gl = lp.lp_moe_gate_bwd(gw, l, w, e)
    t = sample(T)
    part = l[t].contiguous()
    pw, pe = lp.lp_moe_gate(part, k)
    assert torch.equal(w[t], pw) and torch.equal(e[t], pe)
    assert torch.equal(gl[t], lp.lp_moe_gate_bwd(gw[t].contiguous(), part, pw, pe))
    assert torch.equal(l[t].max(1).values, l[t].gather(1, e[t].long())[:, 0])


def test_the_most_pairs(lp):
    n, E = (1 << 30) - 1, 1024
    e = torch.randint(-1, E, (n,), generator=gen(4), device="cuda", dtype=torch.int32)
    off, rows, order = lp.lp_moe_sort(e, E)
    live = int(off[-1])
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    for part in e.split(1 << 27):
        counts += torch.bincount(part + 1, minlength=E + 1)
    assert torch.equal(off.long(), counts[1:].cumsum(0)) and live == n - int(counts[0])
    for a in range(0, live - 1, 1 << 26):                # by expert, then by pair; each pair at its row
        o = order[a:min(a + (1 << 26) + 1, live)].long()
        x = e[o]
        assert ((x[1:] > x[:-1]) | ((x[1:] == x[:-1]) & (o[1:] > o[:-1]))).all()
        assert torch.equal(rows[o], torch.arange(a, a + o.numel(), dtype=torch.int32, device="cuda"))
    for a in range(0, n, 1 << 27):
        assert torch.equal(rows[a:a + (1 << 27)] < 0, e[a:a + (1 << 27)] < 0)


def close(y, x, w):
    """y against x w^T in fp64, w the weight's bf16 values: sums of K terms and one rounding (nvfp4's values may be rounded
    to bf16 before the product or not)."""
    want, size = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    assert ((y.double() - want).abs() <= U16 * want.abs() + (U16 + x.shape[1] * U32) * size).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_w4_weights_past_2_to_32_bytes(lp, fmt):
    G, N, K = 40, 16400, 14336
    g = gen(5)
    run = 32 if fmt == "mxfp4" else 16
    codes = torch.randint(0, 256, (G, N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(*((118, 126) if fmt == "mxfp4" else (0x20, 0x40)), (G, N, K // run), generator=g, dtype=torch.uint8, device="cuda")
    ts = torch.tensor([0.03], device="cuda") if fmt == "nvfp4" else None
    q = lp.QTensor(fmt, codes, scales, ts, shape=(G, N, K))
    for M, at in ((3, 1), (40, 17)):
        x = randn_bf16((M, K), g)
        off = torch.full((G,), M - at, dtype=torch.int32, device="cuda")
        off[-1] = M
        y = lp.lp_grouped_fwd_w4(x, q, off)
        for e, r in ((0, slice(0, M - at)), (G - 1, slice(M - at, M))):
            one = lp.QTensor(fmt, codes[e:e + 1], scales[e:e + 1], ts, shape=(1, N, K))
            close(y[r], x[r], lp.lp_dequant(one)[0])


def test_w4_results_past_2_to_32_bytes(lp):
    M, N, K = (1 << 17) + 5, 16400, 64
    g = gen(6)
    q = lp.lp_mx_quant(randn_bf16((N, K), g), -1, "mxfp4")
    x = randn_bf16((M, K), g)
    y = lp.lp_linear_fwd_w4(x, q)
    t = sample(M)
    close(y[t], x[t], lp.lp_dequant(q)[0])
