"""moe_few_tokens and moe_few_tokens_int8 (the whole layer for a few tokens, one kernel) against the layer
in 64 bits, over shapes, expert types and token counts where a split, a tile or a tail could go wrong."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ref as ref  # noqa: E402

if torch.cuda.is_available():
    import sparse_moe_layer_joint_b200 as moe


def make(T, d, f, n, ns, k, act, seed=0, offset=False):
    g = torch.Generator().manual_seed(seed)
    f1 = 2 * f if act == "swiglu" else f
    rnd = lambda *s: torch.randn(*s, generator=g)
    p = dict(T=T, d=d, f=f, n=n, ns=ns, k=k, act=act, scale=2.5)
    p["x"] = rnd(T, d).bfloat16()
    p["w_r"] = (rnd(n + ns, d) / d ** 0.5).bfloat16()
    p["bias"] = (torch.rand(n, generator=g) - 0.5) * 0.2
    p["offset"] = rnd(n) * 0.5 if offset else None
    p["w1"] = (rnd(n + ns, f1, d) / d ** 0.5).bfloat16()
    p["w2"] = (rnd(n + ns, d, f) / f ** 0.5).bfloat16()
    return p


def to_int8(p):
    q1, s1 = ref.codes64(p["w1"])
    q2, s2 = ref.codes64(p["w2"])
    return dict(p, w1=q1.to(torch.int8), w1s=s1.float(), w2=q2.to(torch.int8), w2s=s2.float())


class Call:
    """Device copies of a problem, poisoned outputs and scratch, and the call."""

    def __init__(self, p):
        self.p = p
        self.t = {k: v.cuda() for k, v in p.items() if isinstance(v, torch.Tensor)}
        T, n, ns, k = p["T"], p["n"], p["ns"], p["k"]
        self.out = torch.full((T, p["d"]), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        self.gates = torch.full((T, k + ns), float("nan"), device="cuda")
        self.counts = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        self.nb = moe.moe_few_tokens_scratch_bytes(T, p["d"], p["f"], n, ns, k)
        self.scratch = torch.full((self.nb,), 0xff, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None):
        p, t = self.p, self.t
        a = (p["T"], p["d"], p["f"], p["n"], p["ns"], p["k"], p["scale"],
             moe.MOE_ACT_SWIGLU if p["act"] == "swiglu" else moe.MOE_ACT_GELU_TANH, self.idx, self.gates,
             self.counts, self.out, self.scratch, self.nb)
        if "w1s" in t:
            moe.moe_few_tokens_int8(t["x"], t["w_r"], t["bias"], t.get("offset"), t["w1"], t["w1s"], t["w2"],
                                    t["w2s"], *a, stream=stream)
        else:
            moe.moe_few_tokens(t["x"], t["w_r"], t["bias"], t.get("offset"), t["w1"], t["w2"], *a, stream=stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        assert moe.moe_get_status() == 0
        p = self.p
        out, gates, idx, gap, tol = ref.few64(p["x"], p["w_r"], p["bias"], p["offset"], p["w1"], p["w2"], p["n"],
                                              p["k"], p["scale"], p["act"], p.get("w1s"), p.get("w2s"))
        assert gap > 1e-6, "the case's scores are too close to compare a selection"
        assert torch.equal(self.idx.cpu().long(), idx)
        assert torch.equal(self.counts.cpu().long(), torch.bincount(idx.reshape(-1), minlength=p["n"]))
        assert ((self.gates.cpu().double() - gates).abs() <= 2.0 ** -18 * gates).all()
        bad = (self.out.cpu().double() - out).abs() > tol
        assert not bad.any(), (int(bad.sum()), ((self.out.cpu().double() - out).abs() / tol).max().item())


CASES = [
    # T, d, f, n, ns, k, activation
    (1, 64, 64, 8, 0, 1, "gelu"),         # half a chunk of K for 8-bit experts, no shared experts
    (2, 256, 128, 256, 2, 6, "gelu"),
    (1, 192, 320, 60, 1, 4, "swiglu"),    # odd numbers of 64-byte halves
    (7, 448, 192, 16, 2, 8, "swiglu"),
    (8, 128, 64, 9, 8, 3, "gelu"),        # a full tile of tokens, most shared experts
    (9, 128, 64, 9, 0, 8, "gelu"),        # one past a tile
    (17, 576, 128, 24, 1, 2, "swiglu"),   # past two tiles for the shared expert
    (33, 320, 192, 8, 2, 8, "gelu"),      # every token picks every expert: 33 tokens an expert
    (64, 256, 64, 40, 2, 6, "swiglu"),    # the largest T
    (3, 2048, 768, 12, 2, 3, "gelu"),     # rows split over several warps
    (2, 4096, 2048, 6, 1, 2, "swiglu"),   # over all warps
    (1, 64, 4096, 4, 1, 4, "gelu"),       # wide hidden rows, narrow model
    (1, 32768, 64, 3, 0, 2, "gelu"),      # the largest widths
    (2, 64, 32768, 2, 1, 1, "swiglu"),
    (16, 1408, 704, 30, 3, 5, "swiglu"),  # two full tiles, odd slices of K
    (1, 64, 1024, 4, 1, 1, "gelu"),       # around the hidden values that every CTA forms for itself
    (1, 64, 1088, 4, 1, 1, "swiglu"),
    (8, 128, 64, 9, 2, 2, "swiglu"),
    (4, 1024, 128, 24, 0, 4, "gelu"),
]


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "T{}d{}f{}n{}s{}k{}{}".format(*c))
def test_matches_the_layer_in_64_bits(case, int8):
    p = make(*case, seed=sum(case[:6]), offset=case[0] % 2 == 1)
    Call(to_int8(p) if int8 else p)().check()


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
@pytest.mark.parametrize("case", [(13, 1024, 512, 48, 2, 6, "swiglu"), (2, 4096, 2048, 6, 1, 2, "swiglu"),
                                  (1, 2048, 1024, 16, 2, 4, "gelu"), (40, 512, 256, 20, 2, 5, "gelu")],
                         ids=lambda c: "T{}d{}f{}n{}s{}k{}{}".format(*c))
def test_equal_inputs_give_equal_bits(case, int8):
    """Hundreds of launches, each of whose items land on other warps: a race on a ring stage or a counter would show."""
    p = make(*case, seed=5)
    p = to_int8(p) if int8 else p
    a, b = Call(p)(), Call(p)
    b.scratch.fill_(0x3c)
    different = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        b.out.fill_(float("nan"))
        b()
        for u, v in ((a.out, b.out), (a.gates, b.gates), (a.idx, b.idx), (a.counts, b.counts)):
            different += (u != v).sum()
    a.check()
    assert int(different) == 0


def test_two_calls_at_once_on_two_streams():
    ps = [make(4, 512, 256, 16, 2, 4, "gelu", seed=s) for s in (1, 2)]
    calls = [Call(ps[0]), Call(to_int8(ps[1]))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(calls, streams):
            c(stream=s)
    for c in calls:
        c.check()


def test_captured_and_replayed_on_new_tokens():
    p = make(5, 256, 128, 32, 2, 6, "gelu", seed=3)
    c = Call(p)
    c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c()
    for seed in (11, 12):
        q = make(5, 256, 128, 32, 2, 6, "gelu", seed=seed)
        p["x"] = q["x"]
        c.t["x"].copy_(q["x"])
        c.out.fill_(float("nan"))
        graph.replay()
        c.check()


@pytest.mark.parametrize("int8", [False, True], ids=["bf16", "int8"])
def test_a_bad_token_spoils_only_its_own_row(int8):
    p = make(6, 256, 128, 16, 1, 4, "gelu", seed=9)
    p["x"][1] = 0.0
    good = Call(to_int8(p) if int8 else p)()
    q = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in p.items()}
    q["x"][3, 17] = float("nan")
    q["x"][4, 0] = float("inf")
    bad = Call(to_int8(q) if int8 else q)()
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    idx = bad.idx.cpu()
    assert ((idx >= 0) & (idx < 16)).all() and all(len(set(r.tolist())) == 4 for r in idx)
    assert torch.isnan(bad.out[3]).all() and not torch.isfinite(bad.out[4]).any()
    for t in (0, 1, 2, 5):
        assert torch.equal(bad.out[t], good.out[t]) and torch.equal(bad.idx[t], good.idx[t])
    good.check()


def test_equal_scores_go_to_the_lower_index():
    p = make(3, 128, 64, 12, 1, 5, "gelu", seed=2)
    p["w_r"][:12] = p["w_r"][0]
    p["bias"].zero_()
    p["bias"][7] = 0.25
    c = Call(p)()
    torch.cuda.synchronize()
    assert c.idx.cpu().tolist() == [[7, 0, 1, 2, 3]] * 3


def test_no_tokens_only_zeroes_the_counts():
    p = make(1, 128, 64, 12, 1, 5, "gelu")
    c = Call(p)
    c.p = dict(p, T=0)
    c()
    torch.cuda.synchronize()
    assert (c.counts == 0).all() and torch.isnan(c.out).all() and (c.idx == -7).all()


def test_a_tensor_elsewhere_is_refused():
    c = Call(make(2, 128, 64, 12, 1, 5, "gelu"))
    for name, t in (("x", c.t["x"].cpu()), ("w1", c.t["w1"].float()), ("w2", c.t["w2"].transpose(1, 2)),
                    ("bias", c.t["bias"][:3])):
        keep = c.t[name]
        c.t[name] = t
        with pytest.raises(ValueError, match=name):
            c()
        c.t[name] = keep


@pytest.mark.parametrize("precision", ["bf16", "int8"])
@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_layer_few_tokens_against_its_many_token_form(precision, act):
    """MoELayer(few_tokens=True) beside MoELayer: the same routing, and outputs within what rounding h and y
    to bf16 on the way (2^-8 each, before a sum of 8 contributors) and 8-bit codes that fall to the other
    side of a step do to the many-token form."""
    import numpy as np

    T, d, f = 24, 512, 256
    p = make(T, d, f, 64, 2, 6, "swiglu" if act == "swiglu" else "gelu", seed=21)
    t = {k: v.cuda() for k, v in p.items() if isinstance(v, torch.Tensor)}
    shape = moe.LayerShape(T, d, f, 64, 2, 6)
    outs = []
    for few in (False, True):
        layer = moe.MoELayer(shape, activation=act, route_scale=2.5, precision=precision, few_tokens=few)
        w1, w2 = t["w1"], t["w2"]
        if precision == "int8":
            layer.set_int8_weights(w1, w2)
            w1 = w2 = None
        bias = t["bias"].clone()
        layer.forward(t["x"], t["w_r"], w1, w2, bias)
        layer.bias_update(bias, 1e-3)
        bal = layer.balance()
        torch.cuda.synchronize()
        assert moe.moe_get_status() == 0
        outs.append((layer.out.float(), layer.topk_idx.clone(), layer.counts.clone(), bias, bal))
    (a, ia, ca, ba, la), (b, ib, cb, bb, lb) = outs
    assert torch.equal(ia, ib) and torch.equal(ca, cb) and torch.equal(ba, bb) and la == lb
    rel = ((a - b).norm() / b.norm()).item()
    # h and y are each off by at most 2^-8 of their values (uniform: 2^-8 / sqrt 3 in the norm), out by 2^-8
    # on both sides; 8-bit codes of the rounded h differ where bf16 moved them over a step: at most 2^-8 again
    assert rel <= 2.0 ** -8 * np.sqrt(5), rel


def test_prefill_and_decode_layers_share_their_weights():
    """The many-token layer of a prompt and the few-token layer of the next tokens, on one copy of 8-bit weights, with
    the balancing bias running through both."""
    T, d, f, n, ns, k = 200, 256, 128, 32, 2, 4
    p = make(T, d, f, n, ns, k, "swiglu", seed=31)
    t = {key: v.cuda() for key, v in p.items() if isinstance(v, torch.Tensor)}
    prompt = moe.MoELayer(moe.LayerShape(T, d, f, n, ns, k), activation="swiglu", precision="int8")
    step = moe.MoELayer(moe.LayerShape(5, d, f, n, ns, k), activation="swiglu", precision="int8", few_tokens=True)
    with pytest.raises(ValueError):
        step.share_int8_weights(prompt)  # it has none yet
    prompt.set_int8_weights(t["w1"], t["w2"])
    step.share_int8_weights(prompt)
    assert step.w1q.data_ptr() == prompt.w1q.data_ptr()
    bias = t["bias"].clone()
    whole = prompt.forward(t["x"], t["w_r"], None, None, bias).float()
    few = step.forward(t["x"][40:45].contiguous(), t["w_r"], None, None, bias).float()
    assert torch.equal(step.topk_idx, prompt.topk_idx[40:45])
    rel = ((few - whole[40:45]).norm() / few.norm()).item()
    assert rel <= 2.0 ** -8 * 5 ** 0.5, rel  # h and y rounded to bf16 on the way of one of them, and both outputs
    prompt.bias_update(bias, 1e-3)
    b0 = bias.clone()
    step.bias_update(bias, 1e-3)
    torch.cuda.synchronize()
    assert moe.moe_get_status() == 0
    load = torch.bincount(step.topk_idx.flatten().long(), minlength=n)
    want = b0 + torch.tensor(1e-3, device="cuda") * torch.sign((5 * k - n * load).float())
    assert torch.equal(bias, want)
    other = moe.MoELayer(moe.LayerShape(5, d, f, n, ns, k), precision="int8", few_tokens=True)
    with pytest.raises(ValueError):
        other.share_int8_weights(prompt)  # another activation


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_whole():
    """With a limit that few waits can keep (they look at the clock only now and then) a call ends in order: it is
    whole or the status bit is set.  Nothing is left behind for the next call."""
    c = Call(make(4, 1024, 512, 24, 1, 4, "gelu", seed=8))
    moe.moe_set_wait_timeout_ns(1)
    try:
        for _ in range(3):
            c()
            torch.cuda.synchronize()
            status = moe.moe_get_status()
            assert status in (0, moe.MOE_STATUS_TIMEOUT)
            if status == 0:
                c.check()
    finally:
        moe.moe_set_wait_timeout_ns(2_000_000_000)
    c().check()


def test_layer_refuses_what_the_kernel_does_not_do():
    s = moe.LayerShape(65, 128, 64, 16, 1, 4)
    with pytest.raises(ValueError):
        moe.MoELayer(s, few_tokens=True)
    s = moe.LayerShape(8, 128, 64, 16, 1, 4)
    with pytest.raises(ValueError):
        moe.MoELayer(s, few_tokens=True, capacity_factor=1.25)
    with pytest.raises(ValueError):
        moe.MoELayer(s, few_tokens=True, precision="nvfp4")
    layer = moe.MoELayer(s, precision="int8", few_tokens=True)
    with pytest.raises(RuntimeError):
        layer.forward(None, None, None, None, None)
