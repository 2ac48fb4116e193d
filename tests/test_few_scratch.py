"""moe_few_tokens_scratch_bytes: a buffer sized for the most tokens serves every smaller call."""
import pytest

import sparse_moe_layer_joint_b200 as moe


@pytest.mark.parametrize("layer", [(7168, 2048, 256, 2, 6), (256, 128, 256, 2, 6), (2048, 768, 160, 1, 8),
                                   (4096, 1024, 256, 2, 6), (64, 32768, 2, 1, 1), (32768, 64, 3, 0, 2)])
def test_size_for_many_tokens_serves_fewer(layer):
    sizes = [moe.moe_few_tokens_scratch_bytes(T, *layer) for T in range(moe.MOE_FEW_MAX_T + 1)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), sizes
