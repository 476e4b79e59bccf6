"""The gated delta rule on the GPU against its definition in float64.

Tolerance: |got - ref| <= h |ref| + c max|ref of the same head|.  h is the
rounding of the output's type (half a step: bf16 2^-8, float32 2^-24).  c
covers the arithmetic: float32 sums over dstate, headdim or a chunk (at most
128 terms: 128 2^-24 = 2^-17 of the sum of the terms' sizes), operands split
into two bf16 terms (2^-16 of it), and sums of sizes up to 2^4 above the
head's largest value where terms cancel: c = 2^-11 for outputs rounded to
bf16, whose inner operands may take one more rounding, and 2^-13 for float32
results of float32 or of two-term arithmetic.
"""
import pytest
import torch

from tests import delta_testlib as R

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from selective_state_space_36_b200 import binding
    return binding


def near(got, ref, what, heads_axis):
    assert got.shape == ref.shape, what
    half = torch.finfo(got.dtype).eps / 2
    c = 2.0 ** -11 if got.dtype == torch.bfloat16 else 2.0 ** -13
    got, ref = got.detach().double().cpu(), ref.double()
    if not got.numel():
        return
    assert torch.isfinite(got).all(), what
    axes = [i for i in range(ref.ndim) if i not in (0, heads_axis)]
    big = ref.abs().amax(axes, keepdim=True) if axes else ref.abs()
    over = (got - ref).abs() - half * ref.abs() - c * big
    assert over.max() <= 0, f"{what}: {over.max():.3e} over the bound, largest value {ref.abs().max():.3e}"


def dev(x):
    return {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in x.items()}


# batch, seqlen, heads, groups, headdim, dstate, io, decay, state
SHAPES = [
    (1, 1, 1, 1, 1, 1, "f32", "mixed", True),
    (1, 1, 2, 1, 64, 128, "bf16", "mixed", False),
    (2, 2, 4, 2, 64, 64, "bf16", "mixed", True),
    (1, 37, 8, 4, 64, 64, "bf16", "mixed", True),
    (3, 63, 3, 1, 40, 48, "f32", "mixed", True),
    (1, 64, 2, 2, 128, 128, "bf16", "mixed", True),
    (2, 65, 2, 1, 128, 128, "bf16", "slow", True),
    (1, 130, 6, 3, 33, 77, "bf16", "mixed", True),
    (1, 200, 1, 1, 128, 64, "bf16", "none", False),
    (2, 257, 4, 2, 64, 128, "bf16", "mixed", True),
    (1, 300, 2, 1, 96, 112, "bf16", "mixed", True),
    (1, 129, 2, 1, 16, 16, "bf16", "slow", True),
    (1, 150, 2, 2, 200, 128, "bf16", "mixed", True),
    (1, 193, 2, 1, 130, 100, "f32", "mixed", True),
    (2, 640, 2, 1, 64, 128, "bf16", "slow", True),
]


@gpu
@pytest.mark.parametrize("batch,seqlen,heads,groups,headdim,dstate,io,decay,state", SHAPES)
def test_forward(lib, batch, seqlen, heads, groups, headdim, dstate, io, decay, state):
    x = R.delta_inputs(batch, seqlen, heads, groups, headdim, dstate, io, 7, decay, state)
    d = dev(x)
    end = d["h0"].clone() if state else None
    scale = 0.37
    out = lib.delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=scale, last_state=end)
    ro, rs = R.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], scale, x["h0"])
    near(out, ro, "out", 2)
    if state:
        near(end, rs, "last_state", 1)


@gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_resume_and_tokens_equal_one_pass(lib, io):
    x = R.delta_inputs(2, 150, 4, 2, 64, 64, io, 3)
    d = dev(x)
    ro, rs = R.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.125, x["h0"])
    state, outs = d["h0"].clone(), []
    for lo, hi in ((0, 70), (70, 71), (71, 140)):
        cut = {n: d[n][:, lo:hi].contiguous() for n in ("q", "k", "v", "g", "beta")}
        outs.append(lib.delta_rule_fwd(cut["q"], cut["k"], cut["v"], cut["g"], cut["beta"], scale=0.125,
                                       last_state=state))
    for t in range(140, 150):
        cut = {n: d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")}
        outs.append(lib.delta_rule_update(state, cut["q"], cut["k"], cut["v"], cut["g"], cut["beta"],
                                          scale=0.125)[:, None])
    near(torch.cat(outs, 1), ro, "out", 2)
    near(state, rs, "state", 1)


@gpu
@pytest.mark.parametrize("batch,heads,groups,headdim,dstate,io", [
    (1, 1, 1, 1, 1, "f32"), (3, 4, 2, 64, 128, "bf16"), (2, 6, 6, 128, 128, "bf16"), (5, 3, 1, 33, 20, "f32"),
    (2, 2, 1, 17, 127, "bf16"), (1, 16, 16, 64, 128, "bf16"), (7, 2, 1, 256, 64, "bf16"), (2, 1, 1, 8, 33, "bf16")])
def test_update(lib, batch, heads, groups, headdim, dstate, io):
    x = R.delta_inputs(batch, 1, heads, groups, headdim, dstate, io, 5)
    d = {n: v[:, 0].contiguous() if n not in ("h0", "dend") else v for n, v in dev(x).items()}
    ro, rs = R.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], dstate ** -0.5, x["h0"])
    out = lib.delta_rule_update(d["h0"], d["q"], d["k"], d["v"], d["g"], d["beta"])
    near(out, ro[:, 0], "out", 1)
    near(d["h0"], rs, "state", 1)


@gpu
@pytest.mark.parametrize("seqlen", [5, 200])
def test_padding_forgetting_and_written_range(lib, seqlen):
    """Tokens with beta = 0, g = 0 keep the state; g = -inf forgets it; nothing
    beside the outputs is written."""
    x = R.delta_inputs(2, seqlen, 2, 1, 64, 64, "bf16", 11)
    half = seqlen // 2
    x["beta"][1, half:] = 0
    x["g"][1, half:] = 0
    x["g"][0, half] = -float("inf")
    x["g"][0, half + 1] = -1e30
    d = dev(x)
    big = torch.full((seqlen * 2 * 2 * 64 + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[128:-128].view(2, seqlen, 2, 64)
    held = torch.full((2 * 2 * 64 * 64 + 256,), 7.0, device="cuda")
    state = held[128:-128].view(2, 2, 64, 64)
    state.copy_(d["h0"])
    lib.delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.1, out=out, last_state=state)
    ro, rs = R.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.1, x["h0"])
    near(out, ro, "out", 2)
    near(state, rs, "state", 1)
    short = {n: d[n][1:, :half].contiguous() for n in ("q", "k", "v", "g", "beta")}
    s2 = d["h0"][1:].clone()
    lib.delta_rule_fwd(short["q"], short["k"], short["v"], short["g"], short["beta"], scale=0.1, last_state=s2)
    near(state[1:], s2.double().cpu(), "state of the padded row", 1)
    for t in (big, held):
        assert (t[:128] == 7).all() and (t[-128:] == 7).all()


@gpu
def test_unaligned_tensors(lib):
    """Tensors one element off any vector alignment give the same results."""
    x = R.delta_inputs(1, 130, 2, 1, 64, 64, "bf16", 13)
    d = dev(x)

    def off(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        room[1:] = t.reshape(-1)
        return room[1:].view(t.shape)

    y = {n: off(v) for n, v in d.items()}
    out = lib.delta_rule_fwd(y["q"], y["k"], y["v"], y["g"], y["beta"], scale=0.3, out=off(d["v"]),
                             last_state=y["h0"])
    ro, rs = R.delta_ref(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.3, x["h0"])
    near(out, ro, "out", 2)
    near(y["h0"], rs, "state", 1)


@gpu
def test_two_streams_and_a_captured_graph(lib):
    """Calls on two streams at once, and a replayed graph, give what one call gives."""
    xs = [R.delta_inputs(2, 260, 4, 2, 64, 128, "bf16", s) for s in (21, 22)]
    ds = [dev(x) for x in xs]
    call = lambda d, st: lib.delta_rule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale=0.1, last_state=st)
    alone = []
    for d in ds:
        st = d["h0"].clone()
        alone.append((call(d, st), st))
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                st = d["h0"].clone()
                got.append((call(d, st), st))
        torch.cuda.synchronize()
        for (o, s), (ro, rs) in zip(got, alone):
            assert torch.equal(o, ro) and torch.equal(s, rs)
    graphs = []
    for d in ds:
        st = d["h0"].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.copy_(d["h0"])
            o = call(d, st)
        graphs.append((g, o, st))
    for _ in range(3):
        for (g, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, o, st), (ro, rs) in zip(graphs, alone):
            assert torch.equal(o, ro) and torch.equal(st, rs)


def test_empty_and_refused(request):
    """Host-side checks (no GPU): empty sizes are no-ops, bad arguments are named."""
    from selective_state_space_36_b200 import binding as b
    f = b.lib.ssm_delta_rule_fwd

    def call(dims, io=1, **kw):
        p = dict(q=0x10000, k=0x20000, v=0x30000, g=0x40000, beta=0x50000, out=0x60000, state=None)
        p.update(kw)
        return f(b.SSMSsdDims(*dims), io, p["q"], p["k"], p["v"], p["g"], p["beta"], 1.0, p["out"], p["state"], None)

    ok = (2, 16, 4, 64, 2, 64)  # batch, seqlen, heads, headdim, groups, dstate
    assert call(ok, io=9) == b.SSM_ERR_INVALID_ARG
    assert call((2, -1, 4, 64, 2, 64)) == b.SSM_ERR_INVALID_ARG
    assert call((2, 16, 4, 64, 3, 64)) == b.SSM_ERR_INVALID_ARG
    assert call((2, 16, 4, 64, 0, 64)) == b.SSM_ERR_INVALID_ARG
    assert call((2, 16, 4, 64, 2, 0)) == b.SSM_ERR_INVALID_ARG
    assert call((2, 16, 4, 64, 2, 129)) == b.SSM_ERR_UNSUPPORTED
    assert call((1 << 40, 1 << 30, 4, 64, 2, 64)) == b.SSM_ERR_INVALID_ARG
    assert call((1 << 31, 1, 4, 64, 2, 64)) == b.SSM_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "g", "beta", "out"):
        assert call(ok, **{name: None}) == b.SSM_ERR_INVALID_ARG
    for name, bad in (("q", 0x10001), ("v", 0x30001), ("out", 0x60001), ("g", 0x40002), ("beta", 0x50002),
                      ("state", 0x70002)):
        assert call(ok, **{name: bad}) == b.SSM_ERR_INVALID_ARG
        assert b"aligned" in b.lib.ssm_last_error()
    for dims in [(0, 16, 4, 64, 2, 64), (2, 0, 4, 64, 2, 64), (2, 16, 0, 64, 2, 64), (2, 16, 4, 0, 2, 64)]:
        assert call(dims, q=None, out=None) == b.SSM_OK
    none = b.lib.ssm_delta_rule_update(b.SSMSsdDims(2, 0, 4, 64, 2, 64), 1, None, 0x10000, 0x20000, 0x30000, 0x40000,
                                       0x50000, 1.0, 0x60000, None)
    assert none == b.SSM_ERR_INVALID_ARG
    x = R.delta_inputs(1, 4, 2, 1, 8, 8, "f32", 1)
    with pytest.raises(TypeError):
        b.delta_rule_fwd(x["q"], x["k"], x["v"].double(), x["g"], x["beta"])
    with pytest.raises(ValueError):
        b.delta_rule_fwd(x["q"], x["k"][:, :2], x["v"], x["g"], x["beta"])
    with pytest.raises(ValueError):
        b.delta_rule_fwd(x["q"].transpose(1, 3).contiguous().transpose(1, 3), x["k"], x["v"], x["g"], x["beta"])


def test_reference_gradients_match_differences():
    """The float64 form's autograd gradients against central differences."""
    x = R.delta_inputs(1, 5, 2, 1, 3, 4, "f32", 2)
    got = R.delta_grads(x, 0.6)

    def loss(y):
        o, s = R.delta_ref(y["q"], y["k"], y["v"], y["g"], y["beta"], 0.6, y["h0"])
        return ((o * x["dout"].double()).sum() + (s * x["dend"].double()).sum()).item()

    for name, grad in got.items():
        base = x[name].double()
        for i in range(0, base.numel(), max(1, base.numel() // 7)):
            step = torch.zeros(base.numel(), dtype=torch.float64)
            step[i] = 1e-6
            step = step.view(base.shape)
            d = (loss({**x, name: base + step}) - loss({**x, name: base - step})) / 2e-6
            assert abs(d - grad.reshape(-1)[i].item()) <= 1e-7 * (1 + abs(d)), name
