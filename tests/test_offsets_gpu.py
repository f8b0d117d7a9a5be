"""Training calls on a B200 whose offsets end before the tokens do: this is reported, and what belongs to the sequences is as
if the tokens behind them were not there."""
import pytest
import torch

from tests.test_bwd_gpu import gdn, make  # noqa: F401 (gdn: the fixture)

pytestmark = pytest.mark.gpu

IO = [torch.float32, torch.bfloat16]
LENS, ALL = (70, 20), 100


def cu():
    return torch.tensor([0, 70, 90], dtype=torch.int32).cuda()


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("k", [1, 2, 3, 4])
def test_conv(gdn, io, bits8, k):
    r = torch.Generator().manual_seed(k)
    n = lambda *s, io=io: torch.randn(*s, generator=r).to(io).cuda()  # noqa: E731
    x, w, b = n(ALL, 256), n(256, k, io=torch.float32), n(256, io=torch.float32)
    dq, dk, dv, state, dstate = n(ALL, 1, 64), n(ALL, 1, 64), n(ALL, 2, 64), n(2, 256, k), n(2, 256, k)
    keep = (lambda t: gdn.act_quantize(t)) if bits8 else (lambda t: t)
    kw = dict(bias=b, conv_state=state, cu_seqlens=cu(), d_state_out=dstate)
    want = gdn.qkv_conv_bwd(dq[:90], dk[:90], dv[:90], keep(x[:90].contiguous()), w, **kw)
    assert gdn.device_status() == 0
    dx = torch.full((ALL, 256), 7.0, dtype=io, device="cuda")
    got = gdn.qkv_conv_bwd(dq, dk, dv, keep(x), w, dx=dx, **kw)
    assert gdn.device_status() == -8
    assert torch.equal(dx[:90], want[0]) and (dx[90:] == 7).all()
    for a, e in zip(got[1:], want[1:]):
        assert torch.equal(a, e)


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")])
def test_rule(gdn, io, kernel):
    d = {n: (t.cuda() if t is not None else None) for n, t in make((ALL, 0), 1, 2, 64, 64, io, s0=True, ds=True).items()}
    names = ("q", "k", "v", "g", "beta", "dout")
    kw = dict(initial_state=d["s0"], d_final_state=d["ds"], cu_seqlens=cu(), kernel=kernel)
    want = gdn.chunk_bwd(*[d[n][:90] for n in names], **kw)
    assert gdn.device_status() == 0
    out = {n: torch.full_like(d[m], 7.0) for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"))}
    out.update({n: torch.full((ALL, 2), 7.0, dtype=io, device="cuda") for n in ("dg", "dbeta")})
    got = gdn.chunk_bwd(*[d[n] for n in names], **out, **kw)
    assert gdn.device_status() == -8
    for a, e in zip(got[:5], want):
        assert torch.equal(a[:90], e) and (a[90:] == 7).all()
    assert torch.equal(got[5], want[5])
