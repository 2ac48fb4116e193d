"""moe_few_tokens and moe_few_tokens_int8 at the ends of what they take: wait limits that run out, and calls that reuse one
scratch buffer."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_few_tokens import Call, make, to_int8  # noqa: E402

if torch.cuda.is_available():
    import sparse_moe_layer_joint_b200 as moe


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("case", [(4, 1024, 512, 24, 1, 4, "gelu"), (24, 512, 256, 16, 2, 4, "swiglu")],
                         ids=lambda c: "T{}d{}f{}n{}s{}k{}{}".format(*c))
def test_a_limit_that_no_barrier_keeps_is_reported(case, int8):
    """A block that has to wait at a grid barrier looks at the clock after its first poll, a microsecond's round trip: of
    twenty calls with a limit of 1 ns at least one reports that it ran out.  The next call is whole."""
    p = make(*case, seed=8)
    c = Call(to_int8(p) if int8 else p)
    c().check()
    seen = []
    moe.moe_set_wait_timeout_ns(1)
    try:
        for _ in range(20):
            c()
            torch.cuda.synchronize()
            seen.append(moe.moe_get_status())
            if seen[-1] == 0:
                c.check()
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    assert set(seen) <= {0, moe.MOE_STATUS_TIMEOUT} and moe.MOE_STATUS_TIMEOUT in seen, seen
    c.out.fill_(float("nan"))
    c().check()


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_one_scratch_buffer_serves_every_smaller_call(int8):
    """A buffer sized once for the most tokens, as a serving program has it; 6 tokens need more of it than 7."""
    layer = (2048, 768, 64, 2, 4, "gelu")
    d, f, n, ns, k, _ = layer
    nb = moe.moe_few_tokens_scratch_bytes(64, d, f, n, ns, k)
    scratch = torch.full((nb,), 0xff, dtype=torch.uint8, device="cuda")
    for T in (7, 1, 6, 20, 3):
        p = make(T, *layer, seed=T)
        c = Call(to_int8(p) if int8 else p)
        c.scratch, c.nb = scratch, nb
        c().check()
