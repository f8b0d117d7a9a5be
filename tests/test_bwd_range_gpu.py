"""Gradients of the chunked forward on a B200 where factors of a chunk lie many binades apart: strong gates, tokens without a
value or a gradient, small or large beta, keys that repeat.  Every head is held to its own largest element, against 64-bit
autograd of the token recurrence.

Tolerances.  bf16 tensors: a path from the inputs to a gradient takes at most eleven operands that are rounded to fp16 (five
to V', six to dX), by half a step, 2^-11 of the value, each.  The roundings are independent: sqrt(11) * 2^-11 < 2^-9 of the
largest element, and the rounding of a bf16 output, 2^-8 of the element.  fp32, and bf16 with kernel="simt": operands within 2^-22, sums of at most 128 terms in fp32 (2^-24 sqrt(128) < 2^-20),
at most about 16 such products: 16 * 2^-20 = 2^-16 of the largest element.
"""
import pytest
import torch

from tests import grad_utils as G
from tests.test_bwd_gpu import NAMES, gdn, make, run  # noqa: F401 (gdn: the fixture)

pytestmark = pytest.mark.gpu

PATHS = [(torch.float32, "auto"), (torch.bfloat16, "auto"), (torch.bfloat16, "simt")]


def close(name, got, want, io, kernel, by=1.0):
    """Head by head (axis 1); ds0 also sequence by sequence.  `by`: how often the tolerance of the operands is allowed."""
    got, want = got.detach().cpu().double(), want.detach().cpu().double()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    operands = by * (2.0 ** -9 if io == torch.bfloat16 and kernel == "auto" else 2.0 ** -16)
    own = 0.0 if io == torch.float32 or name == "ds0" else 2.0 ** -8
    for n in range(want.shape[0]) if name == "ds0" else [slice(None)]:
        for h in range(want.shape[1]):
            a, b = got[n, h] if name == "ds0" else got[:, h], want[n, h] if name == "ds0" else want[:, h]
            top = b.abs().max().item()
            over = ((a - b).abs() - own * b.abs()).max().item()
            assert over <= operands * top, "%s of head %d: off by %.2e of its largest element %.2e" % (name, h, over / max(top, 1e-300), top)


def check(gdn, x, lens, io, kernel, names, by=1.0, **kw):
    got = run(gdn, x, lens, kernel=kernel, **kw)
    assert gdn.device_status() == 0
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens)
    for name, a, b in zip(NAMES, got, want):
        if name in names:
            close(name, a, b, io, kernel, by)


def starts(lens):
    """The first token of every chunk."""
    at, out = 0, []
    for length in lens:
        out += list(range(at, at + length, 64))
        at += length
    return out


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("lens", [(1,), (40,), (64, 3)])
@pytest.mark.parametrize("first", [-8.0, -12.0, -16.0, -30.0])
def test_output_gradients_reach_the_state_behind_a_strong_gate(gdn, io, kernel, lens, first):
    """d_initial_state is then what dout leaves of it: with beta = 0 nothing else adds to it."""
    x = make(lens, 1, 2, 128, 64, io, s0=True)
    x["g"][starts(lens)] = first
    x["beta"].zero_()
    check(gdn, x, lens, io, kernel, ("ds0",))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("lens", [(1,), (40,), (64, 3)])
@pytest.mark.parametrize("first", [-8.0, -12.0, -16.0, -30.0])
def test_state_gradient_behind_a_strong_gate(gdn, io, kernel, lens, first):
    x = make(lens, 1, 2, 128, 64, io, s0=True, ds=True)
    x["g"][starts(lens)] = first
    check(gdn, x, lens, io, kernel, ("dq", "dk", "dv", "dbeta", "ds0"))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("length,gate", [(64, -0.1), (64, -0.25), (64, -0.4), (64, -0.8), (130, -0.25), (130, -0.4)])
def test_state_gradient_through_tokens_without_one(gdn, io, kernel, dk, dv, length, gate):
    """dout = 0, as where a loss is masked: what comes from behind still has to pass all these tokens.  Their shares of it
    are of one size, while the decays up to them differ by exp(gate * length)."""
    lens = (length,)
    x = make(lens, 1, 2, dk, dv, io, s0=True, ds=True)
    x["g"][:] = gate
    x["dout"].zero_()
    check(gdn, x, lens, io, kernel, ("ds0",), by=-(-length // 64))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
@pytest.mark.parametrize("length,gate", [(64, -0.1), (64, -0.25), (64, -0.4), (64, -0.8), (128, -0.25), (128, -0.4)])
def test_state_through_tokens_without_a_value(gdn, io, kernel, dk, dv, length, gate):
    """The same forwards: v = 0, and the first token with a gradient reads what is left of the initial state."""
    lens = (length + 6,)
    x = make(lens, 1, 2, dk, dv, io, s0=True)
    x["g"][:] = gate
    x["v"].zero_()
    x["dout"][:length] = 0
    check(gdn, x, lens, io, kernel, ("dq",), by=-(-length // 64))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("last", [-8.0, -16.0, -30.0])
def test_state_behind_a_strong_last_gate(gdn, io, kernel, last):
    """What a chunk writes, decayed at its last token, which writes nothing itself; read by the next chunk's first."""
    lens = (65,)
    x = make(lens, 1, 2, 128, 128, io)
    x["g"][63] = last
    x["beta"][63:] = 0
    x["dout"][:64] = 0
    check(gdn, x, lens, io, kernel, ("dq",))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("beta", [1e-4, 1e-8, 1e-16])
def test_small_beta(gdn, io, kernel, beta):
    """All writes small: what they leave in the outputs' gradients is as small, and as exact."""
    lens = (100,)
    x = make(lens, 1, 2, 128, 64, io)
    x["beta"] = beta * (0.5 + 0.5 * x["beta"])
    check(gdn, x, lens, io, kernel, ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("gate", [-100.0, -1e3, -1e4, -1e6, -3.4e38, -float("inf")])
def test_gates_that_reset_the_state(gdn, io, kernel, gate):
    """The tokens behind a reset keep their decays among themselves, whatever the gate that did it."""
    lens = (100,)
    x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
    for t in (5, 20, 21, 60):
        x["g"][t] = gate
    check(gdn, x, lens, io, kernel, ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("gate", [-1e3, -1e6, -3.4e38, -float("inf")])
def test_gates_that_all_reset_the_state(gdn, io, kernel, gate):
    """Every token by itself."""
    lens = (70,)
    x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
    x["g"][:] = gate
    check(gdn, x, lens, io, kernel, ("dq", "dk", "dv", "dbeta"))


@pytest.mark.parametrize("io,kernel", [PATHS[0], PATHS[2]])
def test_resets_among_growing_gates(gdn, io, kernel):
    """Gates of both signs: what grows behind a reset does not bring back what it took."""
    lens = (60,)
    x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
    x["g"] = 0.5 * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(3))
    x["beta"] = 1 + 0.0 * x["beta"]
    x["g"][20], x["g"][40] = -300.0, -1e5
    check(gdn, x, lens, io, kernel, ("dq", "dk", "dv", "dg", "dbeta"))


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("gate", [-1.0, -8.0, -16.0, -30.0])
@pytest.mark.parametrize("length", [1, 2])
def test_gate_gradients_of_short_sequences_behind_strong_gates(gdn, io, kernel, gate, length):
    """dg is what passes through the gate, exp(gate) of what the token itself does.  The last tokens of the sequences, each
    behind one gate, are held to the largest of theirs."""
    lens = (length,) * 5
    x = make(lens, 1, 2, 64, 64, io, s0=True, ds=True)
    x["g"][:] = gate
    got = run(gdn, x, lens, kernel=kernel)[3]
    want = G.rule_grads(x["q"], x["k"], x["v"], x["g"], x["beta"], x["s0"], x["dout"], x["ds"], lens)[3]
    close("dg", got[length - 1::length], want[length - 1::length], io, kernel)


def near(kind, lo, hi, dk, io):
    """Keys that repeat through the sequence, or all but, and beta in [lo, hi]; nothing decays."""
    x = make((128,), 8, 8, dk, dk, io, s0=True, ds=True, decay="none", seed=11)
    k = x["k"][:1].expand_as(x["k"])
    x["k"] = (k if kind == "repeated" else (k.float() + 0.1 * x["k"].float()).to(io)).contiguous()
    x["beta"] = lo + (hi - lo) * x["beta"]
    return x


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("kind", ["repeated", "near"])
@pytest.mark.parametrize("lo,hi,by", [(0.0, 1.0, 2), (0.9, 1.0, 2), (1.0, 2.0, 5), (1.8, 2.0, 16), (2.0, 2.0, 16)])
def test_keys_that_repeat(gdn, io, kernel, dk, kind, lo, hi, by):
    """T_ri = -beta_r prod (1 - beta_m) between them, so what a product with T takes shows as often as its rows' magnitudes
    sum to: 1 + 1 where beta <= 1; 1 + 2 (1 + 1/2 + 1/4 + ...) = 5 for beta evenly in [1, 2]; and where nothing falls off,
    64 independent roundings of entries of 2: 2 sqrt(64)."""
    check(gdn, near(kind, lo, hi, dk, io), (128,), io, kernel, ("dq", "dk", "dv", "ds0"), by=by)


@pytest.mark.parametrize("io,kernel", PATHS)
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("kind", ["repeated", "near"])
@pytest.mark.parametrize("lo,hi", [(0.0, 1.0), (0.9, 1.0)])
def test_beta_gradients_where_keys_repeat(gdn, io, kernel, dk, kind, lo, hi):
    """dbeta_r is the product of what the token writes and of the gradient of that, V' and dX: each may show its roundings
    twice (see above), and the largest element need not be where the terms are large, so the eleven are taken one by one:
    2 * 11 * 2^-11, 5.5 times the tolerance of independent ones."""
    check(gdn, near(kind, lo, hi, dk, io), (128,), io, kernel, ("dbeta",), by=5.5)


@pytest.mark.parametrize("io,kernel", PATHS)
def test_beta_gradients_at_and_near_zero(gdn, io, kernel):
    """Of tokens that write nothing, or next to nothing, beside tokens that do."""
    x = make((100,), 1, 2, 128, 64, io, s0=True, ds=True)
    x["beta"][::3] = 0.0
    x["beta"][1::3] = 10.0 ** -torch.linspace(1, 12, x["beta"][1::3].shape[0])[:, None]
    check(gdn, x, (100,), io, kernel, ("dbeta",))


@pytest.mark.parametrize("io,kernel", PATHS)
def test_raw_gates_of_every_rate(gdn, io, kernel):
    """a and b in the places of g and beta: rates up to 16, so that heads forget in one token or in thousands."""
    lens = (70, 129, 1)
    x = make(lens, 4, 8, 128, 128, io, s0=True, ds=True)
    r = torch.Generator().manual_seed(9)
    a, b, dt = torch.randn(200, 8, generator=r), torch.randn(200, 8, generator=r), torch.randn(8, generator=r) - 1
    A_log = torch.log(torch.tensor([0.001, 0.01, 0.1, 0.5, 1.0, 4.0, 10.0, 16.0]))
    x["g"], x["beta"] = a, b
    got = run(gdn, x, lens, kernel=kernel, A_log=A_log.cuda(), dt_bias=dt.cuda())
    assert gdn.device_status() == 0
    g, beta = G.gate(a.double(), b.double(), A_log.double(), dt.double())
    want = G.rule_grads(x["q"], x["k"], x["v"], g, beta, x["s0"], x["dout"], x["ds"], lens)
    for name, y, z in zip(NAMES[:5], got, want):
        close(name, y, z, io, kernel)
