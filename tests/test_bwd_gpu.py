"""Gradients of the chunked forward on a B200 (gdn_chunk_bwd) against 64-bit autograd of the token recurrence."""
import pytest
import torch

from tests import grad_utils as G

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "ds0")


@pytest.fixture(scope="module")
def gdn(cuda_device):
    import gated_deltanet_chunk_b200 as g
    g.lib()
    return g


def make(lens, nqk, nv, dk, dv, io, seed=0, s0=False, ds=False, decay="mild"):
    """Inputs on the CPU, drawn in a fixed order."""
    r = torch.Generator().manual_seed(seed)
    t, n = sum(lens), len(lens)
    q, k = (torch.randn(t, nqk, dk, generator=r).to(io) for _ in range(2))
    v, do = (torch.randn(t, nv, dv, generator=r).to(io) for _ in range(2))
    rate = {"mild": 0.05, "strong": 6.0, "none": 0.0}[decay]
    g = -rate * torch.rand(t, nv, generator=r)
    beta = torch.rand(t, nv, generator=r)
    st = 0.3 * torch.randn(n, nv, dk, dv, generator=r) if s0 else None
    dst = 0.3 * torch.randn(n, nv, dk, dv, generator=r) if ds else None
    return dict(q=q, k=k, v=v, g=g, beta=beta, dout=do, s0=st, ds=dst)


def run(gdn, x, lens, use_cu=True, **kw):
    d = {k: (t.cuda() if t is not None else None) for k, t in x.items()}
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda() if use_cu else None
    return gdn.chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["dout"], initial_state=d["s0"], d_final_state=d["ds"],
                         cu_seqlens=cu, num_seqs=None if use_cu else len(lens), output_d_initial_state=True, **kw)


def check(gdn, x, lens, io, use_cu=True, kernel="auto", **kw):
    got = run(gdn, x, lens, use_cu, kernel=kernel, **kw)
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens, **kw)
    for name, a, b in zip(NAMES, got, want):
        G.assert_close(a, b, io, name)
    assert gdn.device_status() == 0
    return got


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("lens,nqk,nv,s0", [((130,), 1, 1, False), ((64, 1, 63, 65), 2, 4, True), ((17, 0, 100, 2), 1, 3, True)])
def test_gradients(gdn, io, kernel, dk, dv, lens, nqk, nv, s0):
    check(gdn, make(lens, nqk, nv, dk, dv, io, s0=s0, ds=s0), lens, io, kernel=kernel)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("decay", ["strong", "none"])
def test_decays(gdn, io, decay):
    """Decays whose exp(-gcum) would overflow, and none at all."""
    lens = (200, 77)
    check(gdn, make(lens, 1, 2, 128, 128, io, s0=True, ds=True, decay=decay), lens, io)


def test_single_tokens_carry_the_state(gdn):
    lens = (1, 1, 1)
    check(gdn, make(lens, 1, 2, 128, 128, torch.float32, s0=True, ds=True), lens, torch.float32)


def test_equal_lengths_without_cu(gdn):
    lens = (70, 70)
    check(gdn, make(lens, 2, 2, 64, 64, torch.float32, s0=True), lens, torch.float32, use_cu=False)


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_without_l2norm_and_with_a_scale(gdn, io):
    lens = (90, 31)
    x = make(lens, 1, 2, 64, 64, io)
    x["k"] = (x["k"].float() / x["k"].float().norm(dim=-1, keepdim=True)).to(io)
    check(gdn, x, lens, io, qk_l2norm=False, scale=0.3)


def test_beta_zero_and_one(gdn):
    lens = (100,)
    x = make(lens, 1, 1, 64, 64, torch.float32, s0=True, ds=True)
    x["beta"][::3] = 0.0
    x["beta"][1::3] = 1.0
    check(gdn, x, lens, torch.float32)


def test_repeated_keys(gdn):
    """The same key at every token: A is full, and its inverse alternates."""
    lens = (128,)
    x = make(lens, 1, 1, 64, 64, torch.float32, decay="none")
    x["k"] = x["k"][:1].expand_as(x["k"]).contiguous()
    check(gdn, x, lens, torch.float32)
