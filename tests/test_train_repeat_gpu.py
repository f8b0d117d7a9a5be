"""The rule's gradients on a B200 call after call, other inputs between and nothing waited for: the bits are those of each
input's first call, whatever the calls before left in the memory that they share."""
import pytest
import torch

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
