"""The 8-bit and few-token entry points without a GPU: argument checks (nothing is launched), sizes, and the
binding's refusals."""
import pytest

import sparse_moe_layer_joint_b200 as moe

A16, MIS, NULL = 0x10000, 0x10004, None
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
L = moe.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(x=NULL), INV), (dict(q=NULL), INV), (dict(s=NULL), INV), (dict(x=MIS), INV), (dict(q=MIS), INV),
    (dict(s=0x10002), INV), (dict(rows=-1), INV), (dict(K=0), INV), (dict(K=12), UNS), (dict(rows=0), moe.MOE_OK)])
def test_quantize_rows_checks(kw, code):
    a = dict(x=A16, rows=4, K=64, q=A16, s=A16)
    a.update(kw)
    assert L.moe_int8_quantize_rows(a["x"], a["rows"], a["K"], a["q"], a["s"], NULL) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=NULL), INV), (dict(tr=NULL), INV), (dict(xq=MIS), INV), (dict(xs=0x10002), INV), (dict(k=0), INV),
    (dict(k=9), INV), (dict(T=-1), INV), (dict(n=-1), INV), (dict(d=20), UNS), (dict(tq=A16), INV), (dict(ts=A16), INV),
    (dict(T=0), moe.MOE_OK)])
def test_dispatch_checks(kw, code):
    a = dict(x=A16, tr=A16, T=4, d=64, k=2, n=8, xq=A16, xs=A16, tq=NULL, ts=NULL)
    a.update(kw)
    assert L.moe_int8_dispatch(a["x"], a["tr"], a["T"], a["d"], a["k"], a["n"], a["xq"], a["xs"], a["tq"], a["ts"],
                               NULL) == code


@pytest.mark.parametrize("kw,code", [
    (dict(a=NULL), INV), (dict(sa=NULL), INV), (dict(w=MIS), INV), (dict(sw=MIS), INV), (dict(out=NULL), INV),
    (dict(off=0x10002), INV), (dict(G=-1), INV), (dict(rows=-1), INV), (dict(base=-1), INV), (dict(epi=3), INV),
    (dict(epi=-1), INV), (dict(N=0), INV), (dict(N=40), UNS), (dict(K=24), UNS), (dict(K=131088), UNS),
    (dict(G=5000), UNS), (dict(off=NULL, G=1024, rows=1 << 30), UNS), (dict(rows=0), moe.MOE_OK),
    (dict(G=0), moe.MOE_OK)])
def test_grouped_gemm_checks(kw, code):
    a = dict(a=A16, sa=A16, off=A16, G=4, rows=16, base=0, w=A16, sw=A16, N=64, K=64, epi=0, out=A16)
    a.update(kw)
    assert L.moe_int8_grouped_gemm(a["a"], a["sa"], a["off"], a["G"], a["rows"], a["base"], a["w"], a["sw"], a["N"],
                                   a["K"], a["epi"], a["out"], NULL) == code


FEW = [
    (dict(x=NULL), INV), (dict(wr=MIS), INV), (dict(b=NULL), INV), (dict(off=0x10002), INV), (dict(w1=NULL), INV),
    (dict(w2=MIS), INV), (dict(idx=NULL), INV), (dict(g=0x10001), INV), (dict(c=NULL), INV), (dict(out=MIS), INV),
    (dict(scr=NULL), INV), (dict(scr=MIS), INV), (dict(T=-1), INV), (dict(d=0), INV), (dict(f=0), INV),
    (dict(n=0), INV), (dict(ns=-1), INV), (dict(k=0), INV), (dict(k=9), INV), (dict(n=3, k=4), INV),
    (dict(act=2), INV), (dict(rs=0.0), INV), (dict(rs=float("nan")), INV), (dict(rs=float("inf")), INV),
    (dict(T=65), UNS), (dict(n=257), UNS), (dict(ns=9), UNS), (dict(d=96), UNS), (dict(f=72), UNS),
    (dict(d=32832), UNS), (dict(sb=1000), moe.MOE_ERR_SCRATCH)]


def few(int8, **kw):
    a = dict(x=A16, wr=A16, b=A16, off=NULL, w1=A16, s1=A16, w2=A16, s2=A16, T=4, d=64, f=64, n=16, ns=2, k=4, rs=1.0,
             act=0, idx=A16, g=A16, c=A16, out=A16, scr=A16, sb=1 << 40)
    a.update(kw)
    w = [a["w1"], a["s1"], a["w2"], a["s2"]] if int8 else [a["w1"], a["w2"]]
    fn = L.moe_few_tokens_int8 if int8 else L.moe_few_tokens
    return fn(a["x"], a["wr"], a["b"], a["off"], *w, a["T"], a["d"], a["f"], a["n"], a["ns"], a["k"], a["rs"], a["act"],
              a["idx"], a["g"], a["c"], a["out"], a["scr"], a["sb"], NULL)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kw,code", FEW)
def test_few_tokens_checks(kw, code, int8):
    assert few(int8, **kw) == code


def test_few_tokens_int8_needs_scales():
    assert few(True, s1=NULL) == INV and few(True, s2=NULL) == INV and few(True, s2=0x10002) == INV


def test_few_tokens_scratch_grows_with_every_size():
    base = moe.moe_few_tokens_scratch_bytes(8, 256, 128, 64, 2, 4)
    assert base % 16 == 0
    for other in ((16, 256, 128, 64, 2, 4), (8, 512, 128, 64, 2, 4), (8, 256, 512, 64, 2, 4), (8, 256, 128, 64, 4, 4),
                  (8, 256, 128, 64, 2, 8)):
        assert moe.moe_few_tokens_scratch_bytes(*other) > base
    # rows of h (fp32), y (fp32) and codes alone
    assert base >= 8 * 6 * (128 * 5 + 256 * 4)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe.moe_int8_quantize_rows(x, 4, 64, q, s, stream=0)
    with pytest.raises(ValueError, match="aq is on cpu"):
        moe.moe_int8_grouped_gemm(q, s, None, 1, 4, 0, q, s, 32, 64, moe.MOE_INT8_EPI_BF16, x, stream=0)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe.moe_int8_dispatch(x, None, 4, 64, 1, 4, q, s, stream=0)
    with pytest.raises(ValueError, match="x is on cpu"):
        moe.moe_few_tokens(x, x, s, None, x, x, 4, 64, 64, 4, 0, 1, 1.0, 0, None, None, None, x, None, 0, stream=0)
