"""8-bit experts: row codes, dispatch and the grouped product against integers and 64-bit arithmetic, and the
layer that runs on them."""
from fractions import Fraction

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ref as ref  # noqa: E402

if torch.cuda.is_available():
    import sparse_moe_layer_joint_b200 as moe


def quantize(x):
    rows, K = x.shape
    q = torch.full((rows + 1, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 1,), -3.0, device="cuda")
    moe.moe_int8_quantize_rows(x.cuda(), rows, K, q, s)
    torch.cuda.synchronize()
    assert (q[rows] == 99).all() and s[rows] == -3.0  # nothing behind the last row
    return q[:rows].cpu(), s[:rows].cpu()


@pytest.mark.parametrize("rows,K", [(1, 8), (3, 64), (37, 200), (130, 256), (5, 1024), (19, 1032), (7, 2048), (3, 4104),
                                    (2, 7168), (2, 8192), (3, 8200), (1, 40000), (5000, 72)])
def test_codes_are_exact(rows, K):
    g = torch.Generator().manual_seed(rows * 10007 + K)
    x = (torch.randn(rows, K, generator=g) * torch.exp(torch.randn(rows, 1, generator=g) * 3)).bfloat16()
    if rows > 2:
        x[rows // 2] = 0.0
    q, s = quantize(x)
    want, scale = ref.codes64(x)
    assert torch.equal(q.double(), want)
    assert torch.equal(s, (x.float().abs().amax(1) / 127.0))
    assert ((s.double() - scale).abs() <= ref.U32 * scale).all()


def test_ties_and_extremes():
    """Every quotient that is exactly a half-integer, by exact rationals, at the ends of the exponent range too."""
    rows = []
    for e in (-133 + 8, -70, -60, 0, 100, 120):
        for top in (127.0, 254.0, 255.0, 129.0, 192.0, 128.0):
            vals = [top] + [v for v in range(1, 255) if v <= top] + [top / 2, top / 4]
            rows.append([v * 2.0 ** (e - 7) for v in vals] + [0.0] * (264 - len(vals)))
    x = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    x = torch.cat([x, -x])
    q, _ = quantize(x)
    for r in range(x.shape[0]):
        vals = [Fraction(float(v)) for v in x[r]]
        a = max(abs(v) for v in vals)
        want = [int(round(127 * v / a)) if a else 0 for v in vals]  # round(): ties to even
        assert q[r].tolist() == want, r


def test_rows_with_nan_or_infinity():
    x = torch.randn(6, 96).bfloat16()
    x[1, 5] = float("nan")
    x[2, 95] = float("inf")
    x[3, 0] = float("-inf")
    x[4] = 0.0
    q, s = quantize(x)
    assert torch.isnan(s[1:4]).all() and (q[1:5] == 0).all() and s[4] == 0.0
    want, _ = ref.codes64(x[[0, 5]])
    assert torch.equal(q[[0, 5]].double(), want)


@pytest.mark.parametrize("T,d,k,shared", [(1, 64, 1, True), (33, 328, 6, True), (300, 1048, 8, False), (7, 8192, 3, True),
                                          (5, 9000, 2, True)])
def test_dispatch(T, d, k, shared):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g).bfloat16()
    n_rows = T * k
    rows = torch.randperm(n_rows, generator=g).to(torch.int32).view(T, k)
    rows.view(-1)[::5] = -1            # dropped by a capacity
    rows.view(-1)[2::11] = n_rows      # out of range: skipped
    xq = torch.full((n_rows, d), 99, dtype=torch.int8, device="cuda")
    xs = torch.full((n_rows,), -3.0, device="cuda")
    tq = torch.full((T, d), 99, dtype=torch.int8, device="cuda") if shared else None
    ts = torch.full((T,), -3.0, device="cuda") if shared else None
    moe.moe_int8_dispatch(x.cuda(), rows.cuda(), T, d, k, n_rows, xq, xs, tq, ts)
    torch.cuda.synchronize()
    q, _ = ref.codes64(x)
    s = x.float().abs().amax(1) / 127.0
    want = torch.full((n_rows, d), 99.0, dtype=torch.float64)
    wants = torch.full((n_rows,), -3.0)
    for t in range(T):
        for j in range(k):
            r = int(rows[t, j])
            if 0 <= r < n_rows:
                want[r], wants[r] = q[t], s[t]
    assert torch.equal(xq.cpu().double(), want) and torch.equal(xs.cpu(), wants)
    if shared:
        assert torch.equal(tq.cpu().double(), q) and torch.equal(ts.cpu(), s)


def gemm(aq, a_s, off, wq, w_s, N, epi, base=0, groups=None, stream=None):
    n_rows, K = aq.shape
    G = groups if groups is not None else len(off) - 1
    out = torch.full((n_rows if off is not None else G * n_rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    o = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    moe.moe_int8_grouped_gemm(aq.cuda(), a_s.cuda(), o, G, n_rows, base, wq.cuda(), w_s.cuda(), N, K, epi, out,
                              stream=stream)
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    return out.cpu().double()


def gemm64(aq, a_s, wq, w_s, epi):
    """Result in 64 bits (the integer sums are exact) and the bound: fp32's two products and the sum's
    conversion (3 half steps), the activation, and the rounding to bf16."""
    u = (aq.double() @ wq.double().T) * a_s.double()[:, None] * w_s.double()
    du = 3.01 * ref.U32 * u.abs()
    kind = {0: "none", 1: "gelu", 2: "swiglu"}[epi]
    out = ref.act64(u, kind)
    err = ref.act_error(u, du, kind)
    return out, err + ref.BF16 * (out.abs() + err) + 1e-38


def operands(rows, K, G, wn, seed):
    g = torch.Generator().manual_seed(seed)
    aq = torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (G, wn, K), generator=g, dtype=torch.int8)
    a_s = torch.rand(rows, generator=g) * 0.02 + 0.01
    w_s = (torch.rand(G, wn, generator=g) + 0.5) * 0.02 / K ** 0.5
    return aq, a_s, wq, w_s


SIZES = [
    # rows per group, N, K
    ([1], 32, 16),
    ([3, 0, 1], 96, 48),                    # K shorter than a stage, an empty group, a ragged last column tile
    ([5, 130, 0, 128, 17], 288, 144),       # ragged rows around a tile's 128, K past one stage
    ([0, 0, 200, 1], 64, 2048),
    ([300, 257, 511, 40], 544, 272),        # pair tiles with half tiles
    ([1100, 1500], 512, 640),
    ([700, 1, 900, 0, 512], 160, 7168),     # many stages
    ([256], 1056, 128),
    ([32, 33, 31, 160, 161], 352, 400),     # around the 32 rows of a load of a group's last tile
    ([64, 65, 96, 97, 224, 225], 288, 272),
]


@pytest.mark.parametrize("epi", [0, 1, 2], ids=["none", "gelu", "swiglu"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{sum(s[0])}rows{len(s[0])}g{s[1]}x{s[2]}")
def test_grouped_product(size, epi):
    counts, N, K = size
    rows = sum(counts) + 9  # rows behind the last group stay as they were
    wn = 2 * N if epi == 2 else N
    aq, a_s, wq, w_s = operands(rows, K, len(counts) + 1, wn, seed=sum(counts) + N + K)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    out = gemm(aq, a_s, off, wq, w_s, N, epi, base=1)
    for g in range(len(counts)):
        lo, hi = off[g], off[g + 1]
        want, tol = gemm64(aq[lo:hi], a_s[lo:hi], wq[g + 1], w_s[g + 1], epi)
        bad = (out[lo:hi] - want).abs() > tol
        assert not bad.any(), (g, int(bad.sum()))
    assert (out[off[-1]:] == 7.0).all()


@pytest.mark.parametrize("epi", [0, 2], ids=["none", "swiglu"])
@pytest.mark.parametrize("rows,G", [(1, 2), (70, 3), (600, 2)])
def test_groups_that_see_all_rows(rows, G, epi):
    N, K = 128, 320
    aq, a_s, wq, w_s = operands(rows, K, G, 2 * N if epi == 2 else N, seed=rows)
    out = gemm(aq, a_s, None, wq, w_s, N, epi, groups=G).view(G, rows, N)
    for g in range(G):
        want, tol = gemm64(aq, a_s, wq[g], w_s[g], epi)
        assert ((out[g] - want).abs() <= tol).all()


def test_largest_sums_and_nan_scales():
    """All codes at -127 and 127 with K = 16384: the sums pass 2^24 and stay exact; a NaN row scale stays in
    its row."""
    K, N = 16384, 64
    aq = torch.full((130, K), 127, dtype=torch.int8)
    aq[1] = -127
    wq = torch.full((1, N, K), 127, dtype=torch.int8)
    wq[0, 1] = -127
    a_s = torch.full((130,), 2.0 ** -20)
    a_s[5] = float("nan")
    w_s = torch.ones(1, N)
    out = gemm(aq, a_s, [0, 130], wq, w_s, N, 0)
    want, tol = gemm64(aq, torch.nan_to_num(a_s), wq[0], w_s[0], 0)
    keep = torch.arange(130) != 5
    assert torch.isnan(out[5]).all()
    assert ((out - want).abs() <= tol)[keep].all()


@pytest.mark.parametrize("rows", ["0", "1", "2", "64"])
@pytest.mark.parametrize("epi", [0, 1, 2], ids=["none", "gelu", "swiglu"])
def test_tile_order_does_not_change_the_bits(monkeypatch, rows, epi):
    """The sums are exact, so the tiles' order cannot change a result."""
    counts, N, K = [300, 90, 0, 700], 320, 400
    aq, a_s, wq, w_s = operands(sum(counts), K, 4, 2 * N if epi == 2 else N, seed=8)
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    a = gemm(aq, a_s, off, wq, w_s, N, epi)
    monkeypatch.setenv("MOE_GEMM_NMAJOR", rows)
    assert torch.equal(a, gemm(aq, a_s, off, wq, w_s, N, epi))


@pytest.mark.parametrize("act,capacity", [("gelu_tanh", None), ("swiglu", None), ("gelu_tanh", 1.0)])
def test_layer(act, capacity):
    """MoELayer(precision="int8") end to end: its stages recomputed in 64 bits from its own routing, and the
    distance from the bf16 layer, which is the format's (8-bit steps of rows whose largest value is about 3.5
    deviations: 1% a matrix and operand) and only bounded loosely."""
    T, d, f, n, ns, k = 150, 256, 192, 24, 2, 4
    g = torch.Generator().manual_seed(4)
    f1 = 2 * f if act == "swiglu" else f
    x = torch.randn(T, d, generator=g).bfloat16()
    w_r = (torch.randn(n + ns, d, generator=g) / d ** 0.5).bfloat16()
    w1 = (torch.randn(n + ns, f1, d, generator=g) / d ** 0.5).bfloat16()
    w2 = (torch.randn(n + ns, d, f, generator=g) / f ** 0.5).bfloat16()
    bias = torch.zeros(n)
    shape = moe.LayerShape(T, d, f, n, ns, k)
    dev = [t.cuda() for t in (x, w_r, w1, w2, bias)]
    layer = moe.MoELayer(shape, activation=act, precision="int8", capacity_factor=capacity)
    layer.set_int8_weights(dev[2], dev[3])
    out = layer.forward(dev[0], dev[1], None, None, dev[4]).cpu().double()
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    plain = moe.MoELayer(shape, activation=act, capacity_factor=capacity)
    other = plain.forward(dev[0], dev[1], dev[2], dev[3], dev[4]).cpu().double()
    assert torch.equal(layer.topk_idx, plain.topk_idx) and torch.equal(layer.token_row, plain.token_row)
    assert ((out - other).norm() / other.norm()).item() < 0.05

    q1, s1 = ref.codes64(w1)
    q2, s2 = ref.codes64(w2)
    assert torch.equal(layer.w1q.cpu().double(), q1) and torch.equal(layer.w2q.cpu().double(), q2)
    # y rows from the layer's own (bf16) hidden rows: exact codes, exact sums, two fp32 products, bf16
    off = layer.offsets.cpu().tolist()
    rt = layer.row_token.cpu().long()
    h, y = layer.h.cpu(), layer.y_perm.cpu().double()
    kind = 2 if act == "swiglu" else 1
    served = 0
    for e in range(n):
        lo, hi = off[e], off[e + 1]
        served += hi - lo
        if lo == hi:
            continue
        aq, a_s = ref.codes64(x[rt[lo:hi]])
        want, tol = gemm64(aq, a_s.float(), q1[e], s1[e].float(), kind)
        assert ((h[lo:hi].double() - want).abs() <= tol).all()
        hq, hs = ref.codes64(h[lo:hi])
        want, tol = gemm64(hq, hs.float(), q2[e], s2[e].float(), 0)
        assert ((y[lo:hi] - want).abs() <= tol).all()
    assert served == off[n] and (capacity is not None or served == T * k)
    aq, a_s = ref.codes64(x)
    for s in range(ns):
        want, tol = gemm64(aq, a_s.float(), q1[n + s], s1[n + s].float(), kind)
        hh = layer.h_shared[s].cpu()
        assert ((hh.double() - want).abs() <= tol).all()
        hq, hs = ref.codes64(hh)
        want, tol = gemm64(hq, hs.float(), q2[n + s], s2[n + s].float(), 0)
        assert ((layer.y_shared[s].cpu().double() - want).abs() <= tol).all()


def test_captured_layer_with_new_tokens():
    T, d, f, n, ns, k = 70, 128, 64, 16, 1, 3
    g = torch.Generator().manual_seed(6)
    w_r, w1, w2 = ((torch.randn(*s, generator=g) / s[-1] ** 0.5).bfloat16().cuda()
                   for s in ((n + ns, d), (n + ns, f, d), (n + ns, d, f)))
    bias = torch.zeros(n, device="cuda")
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    layer = moe.MoELayer(moe.LayerShape(T, d, f, n, ns, k), precision="int8")
    layer.set_int8_weights(w1, w2)
    layer.forward(x, w_r, None, None, bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, w_r, None, None, bias)
    x.copy_(torch.randn(T, d, generator=g).bfloat16())
    graph.replay()
    replayed = layer.out.clone()
    assert torch.equal(replayed, layer.forward(x, w_r, None, None, bias))


def test_a_tensor_elsewhere_is_refused():
    x = torch.randn(4, 64, device="cuda").bfloat16()
    q, s = torch.empty(4, 64, dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    for bad in (dict(x=x.cpu()), dict(x=x.float()), dict(q=q[:2]), dict(s=s.double()), dict(x=x.t())):
        a = dict(x=x, q=q, s=s)
        a.update(bad)
        with pytest.raises(ValueError):
            moe.moe_int8_quantize_rows(a["x"], 4, 64, a["q"], a["s"])
