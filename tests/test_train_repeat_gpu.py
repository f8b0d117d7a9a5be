"""The rule's gradients on a B200 call after call, other inputs between and nothing waited for: the bits are those of each
input's first call, whatever the calls before left in the memory that they share."""
import pytest
import torch

from tests import grad_utils as G
from tests.test_bwd_gpu import gdn, make, run  # noqa: F401 (gdn: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")])
@pytest.mark.parametrize("lens", [(1, 172, 127, 5, 39), (700, 900)])
def test_calls_in_turn(gdn, io, kernel, lens):
    x = [{k: t.cuda() for k, t in make(lens, 2, 4, 128, 128, io, seed=s, s0=True, ds=True).items()} for s in (1, 2)]
    want = []
    for y in x:
        want.append(run(gdn, y, lens, kernel=kernel))
        torch.cuda.synchronize()
    for _ in range(8):
        got = [run(gdn, y, lens, kernel=kernel) for y in x]
        for a, b in zip(got, want):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


@pytest.mark.parametrize("io,kernel", [(torch.float32, "auto"), (torch.bfloat16, "auto")])
def test_as_many_sequences_as_there_may_be(gdn, io, kernel):
    """65,535 sequences of one token, but for an empty one and one of two chunks: more chunks than a grid's second and
    third dimensions hold.  Of one token from no state, o = scale (q . k) beta v, whose gradients need no recurrence."""
    n, d, io64 = 65535, 64, torch.float64
    lens = torch.ones(n, dtype=torch.int64)
    lens[100], lens[-1] = 0, 100
    t = int(lens.sum())
    r = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(t, 1, d, generator=r, device="cuda").to(io) for _ in range(4))
    g, beta = -torch.rand(t, 1, generator=r, device="cuda"), torch.rand(t, 1, generator=r, device="cuda")
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32).cuda()
    got = gdn.chunk_bwd(q, k, v, g, beta, do, cu_seqlens=cu, kernel=kernel)
    assert gdn.device_status() == 0
    ones = t - 100
    x = [y[:ones].to(io64).requires_grad_() for y in (q, k, v, beta)]
    qh, kh = (y / torch.sqrt((y * y).sum(-1, keepdim=True) + 1e-6) for y in x[:2])
    o = (qh * kh).sum(-1, keepdim=True) * d ** -0.5 * x[3][..., None] * x[2]
    want = torch.autograd.grad(o, x, do[:ones].to(io64))
    for name, a, e in zip(("dq", "dk", "dv", "dbeta"), (got[0], got[1], got[2], got[4]), want):
        G.assert_close(a[:ones], e, io, name)
    assert not got[3][:ones].any()
    alone = gdn.chunk_bwd(*[y[ones:].clone() for y in (q, k, v, g, beta, do)], kernel=kernel)
    for a, e in zip(got[:5], alone):
        assert torch.equal(a[ones:], e)
