"""Calls without tokens or rows: the tensors that then have no elements may have no address (torch gives them none)."""
import pytest

import sparse_moe_layer_joint_b200 as moe

L = moe.lib()
A16, NULL = 0x10000, None


def test_quantize_no_rows():
    assert L.moe_int8_quantize_rows(NULL, 0, 64, NULL, NULL, NULL) == moe.MOE_OK
    assert L.moe_int8_quantize_rows(NULL, 0, 12, NULL, NULL, NULL) == moe.MOE_ERR_UNSUPPORTED


def test_dispatch_no_tokens():
    assert L.moe_int8_dispatch(NULL, NULL, 0, 64, 2, 8, A16, A16, NULL, NULL, NULL) == moe.MOE_OK
    assert L.moe_int8_dispatch(NULL, NULL, 0, 64, 2, 0, NULL, NULL, NULL, NULL, NULL) == moe.MOE_OK
    assert L.moe_int8_dispatch(NULL, NULL, 0, 20, 2, 8, A16, A16, NULL, NULL, NULL) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("groups,rows", [(4, 0), (0, 16), (0, 0)])
def test_product_no_rows_or_groups(groups, rows):
    assert L.moe_int8_grouped_gemm(NULL, NULL, A16, groups, rows, 0, NULL, NULL, 64, 64, 0, NULL, NULL) == moe.MOE_OK
    assert L.moe_int8_grouped_gemm(NULL, NULL, A16, groups, rows, 0, NULL, NULL, 64, 24, 0, NULL, NULL) == \
        moe.MOE_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("precision", ["bf16", "int8"])
def test_layer_for_no_tokens(precision):
    torch = pytest.importorskip("torch")
    d, f, n, ns, k = 128, 64, 8, 1, 2
    w_r = torch.randn(n + ns, d, device="cuda").bfloat16()
    w1, w2 = torch.randn(n + ns, f, d, device="cuda").bfloat16(), torch.randn(n + ns, d, f, device="cuda").bfloat16()
    layer = moe.MoELayer(moe.LayerShape(0, d, f, n, ns, k), precision=precision, few_tokens=True)
    if precision == "int8":
        layer.set_int8_weights(w1, w2)
    layer.counts.fill_(7)
    out = layer.forward(torch.empty(0, d, dtype=torch.bfloat16, device="cuda"), w_r, w1, w2, torch.zeros(n, device="cuda"))
    torch.cuda.synchronize()
    assert out.shape == (0, d) and (layer.counts == 0).all() and moe.moe_get_status() == 0
