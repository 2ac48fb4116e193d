"""8-bit products at the ends of what they take: the longest K, whose sums nearly fill 32 bits, at every row count around
a load and a tile."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_int8 import gemm, gemm64  # noqa: E402


@pytest.mark.parametrize("epi", [0, 1, 2], ids=["none", "gelu", "swiglu"])
@pytest.mark.parametrize("counts", [[1, 0, 32], [33, 129]], ids=str)
def test_longest_k(counts, epi):
    """K = 131072: rows and channels of 127 and -127 sum to 131072 * 127^2 = 2114060288, 1.5% below 2^31; the scale brings
    the largest u to 2^11 * 1.06, so that no activation overflows."""
    K, N = 131072, 32
    rows, wn = sum(counts), 64 if epi == 2 else 32
    g = torch.Generator().manual_seed(rows + epi)
    aq = torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (len(counts), wn, K), generator=g, dtype=torch.int8)
    aq[0], wq[:, 0], wq[:, 1] = 127, 127, -127
    aq[-1] = -127
    a_s = torch.rand(rows, generator=g) * 2.0 ** -20 + 2.0 ** -20
    w_s = torch.rand(len(counts), wn, generator=g) * 0.5 + 0.5
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    out = gemm(aq, a_s, off, wq, w_s, N, epi)
    for e in range(len(counts)):
        lo, hi = off[e], off[e + 1]
        want, tol = gemm64(aq[lo:hi], a_s[lo:hi], wq[e], w_s[e], epi)
        assert ((out[lo:hi] - want).abs() <= tol).all(), e
