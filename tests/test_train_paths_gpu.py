"""The training calls as a training loop makes them, on a B200: captured and replayed, on other streams, at once, twice,
on padded and on inconsistent batches, with nothing to do and with much.

Runs of one call on the same inputs are compared bit by bit: no kernel uses an atomic on its results.
"""
import pytest
import torch

from tests import grad_utils as G
from tests.test_bwd_gpu import NAMES, make

pytestmark = pytest.mark.gpu

IO = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def gdn(cuda_device):
    import gated_deltanet_chunk_b200 as g
    g.lib()
    return g


def cu_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()


def cuda(x):
    return {k: (t.cuda() if t is not None else None) for k, t in x.items()}


def rule(gdn, d, cu, **kw):
    return gdn.chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu,
                         output_d_initial_state=True, **kw)


def same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        if x is None:
            assert y is None, i
        else:
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i


class Layer:
    """Every training call of one layer, on buffers that stay where they are."""

    def __init__(self, gdn, io, lens, seed, nqk=1, nv=2, d=64, k=4):
        r = torch.Generator().manual_seed(seed)
        n = lambda *s, io=torch.float32, by=1.0: (by * torch.randn(*s, generator=r)).to(io).cuda()  # noqa: E731
        t, c = sum(lens), 2 * nqk * d + nv * d
        self.gdn, self.io, self.cu = gdn, io, cu_of(lens)
        self.x = dict(X=n(t, c, io=io), W=n(c, k, by=0.5), B=n(c, by=0.1), a=n(t, nv), b=n(t, nv), A=n(nv) - 2, dt=n(nv), z=n(t, nv, d, io=io),
                      nw=n(d) + 1, dy=n(t, nv, d, io=io), o=n(t, nv, d, io=io), q=n(t, nqk, d, io=io), k=n(t, nqk, d, io=io),
                      v=n(t, nv, d, io=io))
        self.ws = torch.empty(gdn.chunk_bwd_workspace(self.x["q"], self.x["v"], self.cu), dtype=torch.uint8, device="cuda")

    def run(self):
        g, x = self.gdn, self.x
        kx, kz = g.act_quantize(x["X"]), g.act_quantize(x["z"])
        do, dz, dnw = g.gated_rmsnorm_bwd(x["dy"], x["o"], kz, x["nw"])
        dq, dk, dv, dg, dbeta, _ = g.chunk_bwd(x["q"], x["k"], x["v"], x["a"], x["b"], do, A_log=x["A"], dt_bias=x["dt"], cu_seqlens=self.cu,
                                               workspace=self.ws)
        gate = g.gate_bwd(dg, dbeta, x["a"], x["b"], x["A"], x["dt"])
        conv = g.qkv_conv_bwd(dq, dk, dv, kx, x["W"], bias=x["B"], cu_seqlens=self.cu)
        return [do, dz, dnw, dq, dk, dv, dg, dbeta, *gate, *conv[:3], g.act_dequantize(*kx, self.io), kx[0], kx[1]]


LENS = (150, 0, 3, 64, 90, 1)


@pytest.mark.parametrize("io", IO)
def test_captured_and_replayed(gdn, io):
    """The replay reads its inputs when it runs, and its bits are those of the eager calls."""
    one, two = Layer(gdn, io, LENS, 1), Layer(gdn, io, LENS, 2)
    want1, want2 = one.run(), two.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = one.run()
    graph.replay()
    torch.cuda.synchronize()
    same(got, want1)
    for name, t in one.x.items():
        t.copy_(two.x[name])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        same(got, want2)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("io", IO)
def test_two_captured_graphs_at_once(gdn, io):
    """Each has its own workspace: replayed on two streams, neither disturbs the other."""
    layers = [Layer(gdn, io, LENS, s) for s in (3, 4)]
    wants = [y.run() for y in layers]
    torch.cuda.synchronize()
    graphs, gots = [], []
    for y in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gots.append(y.run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(gots, wants):
        same(got, want)


@pytest.mark.parametrize("io", IO)
def test_another_stream(gdn, io):
    """stream= gives what a call under torch.cuda.stream gives, workspace included, behind work of that stream."""
    d, cu = cuda(make((200, 31), 1, 2, 64, 64, io, s0=True, ds=True)), cu_of((200, 31))
    want = rule(gdn, d, cu)
    s = torch.cuda.Stream()
    late = {k: torch.zeros_like(t) for k, t in d.items()}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        for k in late:
            late[k].copy_(d[k])
    gots = [rule(gdn, late, cu, stream=s) for _ in range(2)]
    s.synchronize()
    for got in gots:
        same(got, want)


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")])
def test_dirty_workspace_and_twice(gdn, io, kernel):
    """What the workspace held does not matter, NaN included; a second run gives the same bits."""
    lens = (129, 64, 0, 2)
    d, cu = cuda(make(lens, 2, 6, 128, 64, io, s0=True, ds=True)), cu_of(lens)
    need = gdn.chunk_bwd_workspace(d["q"], d["v"], cu, kernel=kernel)
    want = rule(gdn, d, cu, kernel=kernel)
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        same(rule(gdn, d, cu, kernel=kernel, workspace=ws), want)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("dv", [64, 128])
def test_outputs_are_written_where_given(gdn, io, dv):
    """Into slices of larger tensors, whose other rows stay as they were."""
    lens = (65, 30)
    d, cu = cuda(make(lens, 1, 2, 64, dv, io, s0=True, ds=True)), cu_of(lens)
    want = rule(gdn, d, cu)
    big = [torch.full((t.shape[0] + 16, *t.shape[1:]), 7.0, dtype=t.dtype, device="cuda") for t in want]
    out = [b[8:8 + t.shape[0]] for b, t in zip(big, want)]
    got = rule(gdn, d, cu, dq=out[0], dk=out[1], dv=out[2], dg=out[3], dbeta=out[4], d_initial_state=out[5])
    for b, o, g, w in zip(big, out, got, want):
        assert g.data_ptr() == o.data_ptr() and torch.equal(o, w)
        assert (b[:8] == 7).all() and (b[8 + w.shape[0]:] == 7).all()


@pytest.mark.parametrize("io", IO)
def test_empty_sequences_pass_the_state_on(gdn, io):
    """Padding: empty sequences in front, between and behind."""
    lens = (0, 0, 70, 0, 5, 0)
    x = make(lens, 1, 2, 64, 128, io, s0=True, ds=True)
    got = rule(gdn, cuda(x), cu_of(lens))
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens)
    for name, a, b in zip(NAMES, got, want):
        G.assert_close(a, b, io if name != "ds0" else (torch.float32 if io == torch.float32 else torch.bfloat16), name)
    for n, length in enumerate(lens):
        if length == 0:
            assert torch.equal(got[5][n].cpu(), x["ds"][n])


@pytest.mark.parametrize("io", IO)
def test_no_tokens(gdn, io):
    lens = (0, 0)
    d = cuda(make(lens, 1, 2, 64, 64, io, s0=True, ds=True))
    got = rule(gdn, d, cu_of(lens))
    assert got[0].shape == (0, 1, 64) and torch.equal(got[5], d["ds"])
    d["ds"] = None
    assert not rule(gdn, d, cu_of(lens))[5].any()


@pytest.mark.parametrize("io", IO)
def test_many_short_sequences(gdn, io):
    lens = tuple(1 + (7 * i) % 5 for i in range(300))
    x = make(lens, 1, 1, 64, 64, io)
    got = rule(gdn, cuda(x), cu_of(lens))
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["dout"], None, lens)
    for name, a, b in zip(NAMES, got, want):
        G.assert_close(a, b, io, name)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("cu", [[0, 40, 90, 100], [0, 60, 40, 128], [0, 40, 90, 200], [8, 40, 90, 128], [-64, 40, 90, 128], [0, 300, 90, 128]])
def test_inconsistent_offsets_are_reported(gdn, io, cu):
    """Every offset is clamped to the tokens there are; the status says that the results are not to be used."""
    d = cuda(make((128, 0, 0), 1, 2, 64, 64, io, s0=True, ds=True))
    rule(gdn, d, torch.tensor(cu, dtype=torch.int32).cuda())
    assert gdn.device_status() == -8
    x, w, z = torch.randn(128, 256).cuda().to(io), torch.ones(256, 4).cuda(), d["q"]
    gdn.qkv_conv_bwd(z, d["k"], d["v"], x, w, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), output_d_state=True)
    assert gdn.device_status() == -8
    assert gdn.device_status() == 0


@pytest.mark.parametrize("io", IO)
def test_tokens_behind_the_last_sequence_are_left(gdn, io):
    """Also where the offsets end early, which is reported, nothing is written behind them."""
    lens = (70, 20)
    x = make((100,), 1, 2, 64, 64, io)
    d = cuda(x)
    out = [torch.full(s, 7.0, dtype=io, device="cuda") for s in ((100, 1, 64), (100, 1, 64), (100, 2, 64), (100, 2), (100, 2))]
    got = gdn.chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], cu_seqlens=cu_of(lens), dq=out[0], dk=out[1], dv=out[2],
                        dg=out[3], dbeta=out[4])
    assert gdn.device_status() == -8
    assert all((t[90:] == 7).all() for t in got[:5])
    dx = torch.full((100, 256), 7.0, dtype=io, device="cuda")
    gdn.qkv_conv_bwd(d["q"], d["k"], d["v"], torch.randn(100, 256).to(io).cuda(), torch.ones(256, 4, device="cuda"), cu_seqlens=cu_of(lens), dx=dx)
    assert gdn.device_status() == -8
    assert (dx[90:] == 7).all() and not (dx[:90] == 7).all()


@pytest.mark.parametrize("name,value", [("g", 0.5), ("g", float("nan")), ("beta", -0.1), ("beta", 2.5), ("beta", float("nan"))])
def test_a_gate_out_of_range_is_reported(gdn, name, value):
    lens = (100,)
    d = cuda(make(lens, 1, 2, 64, 64, torch.bfloat16))
    d[name][57, 1] = value
    rule(gdn, d, cu_of(lens))
    assert gdn.device_status() == -9


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "simt")])
def test_growing_states(gdn, io, kernel):
    """The other path takes any finite gate: here g > 0, and beta beyond 2 and below 0."""
    lens = (80, 7)
    x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
    x["g"] = -0.02 + 0.04 * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(5))
    x["beta"][3], x["beta"][50] = 2.5, -0.5
    got = rule(gdn, cuda(x), cu_of(lens), kernel=kernel)
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens)
    for n, a, b in zip(NAMES, got, want):
        G.assert_close(a, b, io, n)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("io", IO)
def test_scales_far_from_one(gdn, io):
    """Activations and gradients of 2^-40 and 2^40: every factor of two is the tensors' own.  The tolerances are
    relative to each result's largest element, and powers of two leave the inputs' digits as they are."""
    lens = (130,)
    for pv, po in ((-40, 40), (40, -40)):
        x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
        x["v"], x["dout"] = x["v"] * 2.0 ** pv, x["dout"] * 2.0 ** po
        x["s0"], x["ds"] = x["s0"] * 2.0 ** pv, x["ds"] * 2.0 ** po
        got = rule(gdn, cuda(x), cu_of(lens))
        want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens)
        for n, a, b in zip(NAMES, got, want):
            G.assert_close(a, b, io, n)


@pytest.mark.parametrize("io", IO)
def test_rows_of_zeros(gdn, io):
    """Padding inside a sequence: q, k, v and dout of zero, beta and g of zero; and a head that has no gradient at all."""
    lens = (100,)
    x = make(lens, 1, 2, 64, 64, io)
    for n in ("q", "k", "v", "dout", "g", "beta"):
        x[n][20:50] = 0
    x["dout"][:, 1] = 0
    got = rule(gdn, cuda(x), cu_of(lens))
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], None, x["dout"], None, lens)
    for n, a, b in zip(NAMES, got, want):
        G.assert_close(a, b, io, n)


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")])
def test_nan_stays_in_its_head_and_sequence(gdn, io, kernel):
    lens = (70, 70)
    x = make(lens, 2, 4, 64, 64, io)
    want = rule(gdn, cuda(x), cu_of(lens), kernel=kernel)
    x["v"][30, 3, 5] = float("nan")
    got = rule(gdn, cuda(x), cu_of(lens), kernel=kernel)
    assert torch.isnan(got[4][30, 3])                     # dbeta of that token
    for n, a, b in zip(NAMES[:5], got, want):
        heads = 1 if n in ("dq", "dk") else 3             # v-head 3 shares qk-head 1
        assert torch.equal(a[:, :heads], b[:, :heads]) and torch.equal(a[70:], b[70:]), n


def test_quantize_beyond_32_bits(gdn):
    """More than 2^32 values: the last groups are as those of a short tensor."""
    n = 2 ** 32 + 96
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(160, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    x[-160:] = tail
    codes, scales = gdn.act_quantize(x)
    c, s = gdn.act_quantize(tail)
    assert torch.equal(codes[-160:].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[-5:], s)
    assert not codes[:1 << 20].view(torch.uint8).any() and not codes[2 ** 32 - 192:2 ** 32 - 64].view(torch.uint8).any()
    out = gdn.act_dequantize(codes, scales, torch.bfloat16, out=x)
    assert torch.equal(out[-160:], gdn.act_dequantize(c, s, torch.bfloat16)) and not out[:-160].any()


@pytest.mark.parametrize("io", IO)
def test_large_offsets(gdn, io):
    """32 v-heads over 70,000 tokens: 287 million values a tensor, 1.1 GB in fp32.  Sequences are cut off at both ends
    and must be as when they are alone."""
    lens = (130, 69740, 130)
    t, nv, d = sum(lens), 32, 128
    r = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, io=io: torch.randn(*s, generator=r, device="cuda").to(io)  # noqa: E731
    q, k, v, do = n(t, 1, d), n(t, 1, d), n(t, nv, d), n(t, nv, d)
    g, beta = -0.05 * torch.rand(t, nv, generator=r, device="cuda"), torch.rand(t, nv, generator=r, device="cuda")
    whole = gdn.chunk_bwd(q, k, v, g, beta, do, cu_seqlens=cu_of(lens))
    for at in (0, lens[0] + lens[1]):
        cut = [y[at:at + 130].contiguous() for y in (q, k, v, g, beta, do)]
        alone = gdn.chunk_bwd(*cut, cu_seqlens=cu_of((130,)))
        for name, a, b in zip(NAMES[:5], whole, alone):
            assert torch.equal(a[at:at + 130], b), name
    assert gdn.device_status() == 0
