"""A wait limit that few waits keep, for the kernels whose copies and products are in flight when a wait runs out: a call
is whole or reports that it ran out, and the next call with the usual limit is whole."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sparse_moe_layer_joint_b200 as moe
    from test_gpu_nvfp4 import _gemm_inputs


def run_short(call, outputs, times=10):
    """Calls with a limit of 1 ns; outputs() names what a whole call fills with one set of bits."""
    call()
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    want = [t.clone() for t in outputs()]
    whole = lambda: all(torch.equal(a, b) for a, b in zip(want, outputs()))
    moe.moe_set_wait_timeout_ns(1)
    try:
        for _ in range(times):
            for t in outputs():
                t.zero_()
            call()
            torch.cuda.synchronize()
            status = moe.moe_get_status()
            assert status in (0, moe.MOE_STATUS_TIMEOUT)
            assert status != 0 or whole()
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    call()
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0 and whole()


def test_router(monkeypatch):
    monkeypatch.setenv("MOE_ROUTER_SMALL", "0")
    T, d, n, ns, k = 1500, 2048, 64, 2, 4
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, d, generator=g).bfloat16().cuda()
    w = (torch.randn(n + ns, d, generator=g) / d ** 0.5).bfloat16().cuda()
    bias = torch.zeros(n, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gates = torch.empty(T, k + ns, device="cuda")
    counts = torch.empty(n, dtype=torch.int32, device="cuda")
    run_short(lambda: moe.moe_router_topk(x, w, bias, None, T, d, n, ns, k, 1.0, idx, gates, counts),
              lambda: (idx, gates, counts))


@pytest.mark.parametrize("pair", ["0", "1"])
def test_nvfp4_product(monkeypatch, pair):
    monkeypatch.setenv("MOE_FP4_PAIR", pair)
    sizes, N, K = [130, 0, 64, 300], 512, 1024
    _, _, _, _, rows_cap, dev = _gemm_inputs(sizes, N, K, 3)
    n = sum(sizes)
    off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")
    out = torch.empty(n, N, dtype=torch.bfloat16, device="cuda")
    run_short(lambda: moe.moe_nvfp4_grouped_gemm(dev["aq"], dev["asf"], dev["off_pad"], 4, rows_cap, dev["wq"], dev["wsf"],
                                                 dev["g"], N, K, moe.MOE_NVFP4_EPI_BF16, None, None, out, off, n),
              lambda: (out,), 3 if pair == "1" else 10)  # a pair's loaders give up after a second


@pytest.mark.parametrize("act", ["MOE_ACT_GELU_TANH", "MOE_ACT_SWIGLU"])
@pytest.mark.parametrize("cta", ["1", "2"])
def test_bf16_products(monkeypatch, cta, act):
    monkeypatch.setenv("MOE_GEMM_CTA", cta)
    counts, d, f = [130, 0, 64, 700], 1024, 512
    n, f1 = sum(counts), 1024 if act == "MOE_ACT_SWIGLU" else 512
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, d, generator=g).bfloat16().cuda()
    w1 = (torch.randn(4, f1, d, generator=g) / d ** 0.5).bfloat16().cuda()
    w2 = (torch.randn(4, d, f, generator=g) / f ** 0.5).bfloat16().cuda()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    h = torch.empty(n, f, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    run_short(lambda: moe.moe_grouped_ffn(x, off, 4, n, 0, w1, w2, d, f, getattr(moe, act), h, y), lambda: (h, y),
              3 if cta == "2" else 10)


def test_int8_product():
    counts, N, K = [130, 0, 64, 300], 512, 1024
    n = sum(counts)
    g = torch.Generator().manual_seed(2)
    aq = torch.randint(-127, 128, (n, K), generator=g, dtype=torch.int8).cuda()
    wq = torch.randint(-127, 128, (4, N, K), generator=g, dtype=torch.int8).cuda()
    a_s, w_s = torch.rand(n, generator=g).cuda(), torch.rand(4, N, generator=g).cuda()
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    out = torch.empty(n, N, dtype=torch.bfloat16, device="cuda")
    run_short(lambda: moe.moe_int8_grouped_gemm(aq, a_s, off, 4, n, 0, wq, w_s, N, K, moe.MOE_INT8_EPI_BF16, out),
              lambda: (out,))
