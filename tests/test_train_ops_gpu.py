"""Gradients of the gate, the gated RMSNorm and the conv, and activations in 8 bits, on a B200, against 64-bit autograd
of the definitions in tests/grad_utils.py."""
import pytest
import torch

from tests import grad_utils as G

pytestmark = pytest.mark.gpu

IO = [torch.float32, torch.bfloat16]


@pytest.fixture(scope="module")
def gdn(cuda_device):
    import gated_deltanet_chunk_b200 as g
    g.lib()
    return g


def draws(seed):
    r = torch.Generator().manual_seed(seed)
    return lambda *shape, io=torch.float32, by=1.0: (by * torch.randn(*shape, generator=r)).to(io)


def read_back(codes, scales):
    """The values that codes and scales stand for, by the format's definition, in 64 bits."""
    c = codes.cpu().view(torch.uint8).to(torch.int64)
    sign, ex, man = 1 - 2 * (c >> 7), (c >> 3) & 15, c & 7
    v = torch.where(ex == 0, man.double() * 2.0 ** -9, (1 + man.double() / 8) * torch.exp2(ex.double() - 7))
    v = torch.where((ex == 15) & (man == 7), torch.nan, sign * v)
    return v * torch.exp2(scales.cpu().double() - 127).repeat_interleave(32, -1)


def kept(gdn, x, bits8):
    """(what the call gets, the 64-bit values it stands for)"""
    if not bits8:
        return x.cuda(), x.double()
    pair = gdn.act_quantize(x.cuda())
    return pair, read_back(*pair)


# ---------------------------------------------------------------- 8 bits

@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("shape", [(32,), (1, 64), (3, 96), (1031, 1024), (7, 5, 128)])
def test_quantize(gdn, io, shape):
    x = draws(1)(*shape, io=io) * torch.exp2(draws(2)(*shape, by=6.0)).to(io)
    codes, scales = gdn.act_quantize(x.cuda())
    want = x.double().unflatten(-1, (-1, 32))
    top = want.abs().amax(-1)
    e = scales.cpu().double() - 127
    assert (top <= 448 * torch.exp2(e)).all() and (top > 448 * torch.exp2(e - 1)).all()  # the least power of two
    got = read_back(codes, scales)
    unit = torch.exp2(e).repeat_interleave(32, -1)
    # half a step: 2^-4 of the value, or of the least value with full precision, 2^-6
    assert ((got - x.double()).abs() <= 2.0 ** -4 * torch.maximum(x.double().abs(), 2.0 ** -6 * unit)).all()
    for dtype in IO:
        assert torch.equal(gdn.act_dequantize(codes, scales, dtype).cpu().double(), got)  # bf16 holds them too


def test_quantize_ties_and_borders(gdn):
    base = torch.tensor([448.0, 464.0 - 2 ** -15, 1.0625, 1.1875, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -0.0, -448.0])
    x = torch.zeros(3, 32)
    x[0, :12] = base.clamp(max=448.0)                 # scale 1: ties go to even
    x[1, 0] = 448.0 * (1 + 2.0 ** -22)                # just beyond 448: the next power of two
    x[2, :4] = torch.tensor([3.0e38, 1.0, -3.4e38, 2.0 ** -126])
    codes, scales = gdn.act_quantize(x.cuda())
    assert scales.flatten().tolist()[:2] == [127, 128]
    got = read_back(codes, scales)
    assert got[0, :12].tolist() == [448.0, 448.0, 1.0, 1.25, 16.0, 20.0, 2.0 ** -9, 0.0, 2.0 ** -8, 0.0, 0.0, -448.0]
    assert got[1, 0].item() == 448.0
    assert torch.isfinite(gdn.act_dequantize(codes, scales, torch.float32)).all()  # the largest finite values stay finite


def test_quantize_keeps_bad_values_to_themselves(gdn):
    x = draws(3)(2, 64)
    x[0, 3], x[0, 40], x[1, 5] = torch.inf, torch.nan, -torch.inf
    good = torch.isfinite(x)
    y = gdn.act_dequantize(*gdn.act_quantize(x.cuda()), torch.float32).cpu()
    z = gdn.act_dequantize(*gdn.act_quantize(torch.where(good, x, 0.0).cuda()), torch.float32).cpu()
    assert torch.isnan(y[~good]).all() and torch.equal(y[good], z[good])


def test_quantize_zeros_and_smallest(gdn):
    x = torch.zeros(2, 32)
    x[1] = 1e-45
    y = gdn.act_dequantize(*gdn.act_quantize(x.cuda()), torch.float32).cpu()
    assert torch.equal(y, torch.zeros(2, 32))


# ---------------------------------------------------------------- gated RMSNorm

@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows", [1, 7, 1000, 20011])
@pytest.mark.parametrize("o8,z8", [(False, False), (True, True)])
def test_norm_gradients(gdn, io, dim, rows, o8, z8):
    n = draws(rows + dim)
    o, z, dy, w = n(rows, dim, io=io, by=0.3), n(rows, dim, io=io, by=2.0), n(rows, dim, io=io), n(dim) + 1
    check_norm(gdn, o, z, dy, w, io, o8, z8)


@pytest.mark.parametrize("o8,z8", [(False, True), (True, False)])
def test_norm_gradients_with_one_in_8_bits(gdn, o8, z8):
    n = draws(5)
    check_norm(gdn, n(300, 128, io=torch.bfloat16), n(300, 128, io=torch.bfloat16), n(300, 128, io=torch.bfloat16), n(128),
               torch.bfloat16, o8, z8)


def check_norm(gdn, o, z, dy, w, io, o8=False, z8=False, eps=1e-6):
    (oin, o64), (zin, z64) = kept(gdn, o, o8), kept(gdn, z, z8)
    got = gdn.gated_rmsnorm_bwd(dy.cuda(), oin, zin, w.cuda(), eps)
    leaves = [t.double().requires_grad_() for t in (o64, z64, w)]
    want = torch.autograd.grad(G.norm(*leaves, eps), leaves, dy.double())
    for name, a, b, t in zip(("do", "dz", "dw"), got, want, (io, io, torch.float32)):
        G.assert_close(a, b, t, name)


def test_norm_gradients_at_extremes(gdn):
    """Rows of zeros, gates far out on both sides, an eps of zero."""
    n = draws(6)
    o, z, dy, w = n(64, 64), n(64, 64), n(64, 64), n(64)
    z[0], z[1], z[2, ::2] = 200.0, -200.0, 0.0
    check_norm(gdn, o, z, dy, w, torch.float32, eps=0.0)
    o[3] = 0.0
    dy[3] *= 1e-3  # do of a row of zeros is dy w silu(z) / sqrt(eps)
    check_norm(gdn, o, z, dy, w, torch.float32)


def test_norm_gradients_of_no_rows(gdn):
    e = torch.empty(0, 64, device="cuda")
    do, dz, dw = gdn.gated_rmsnorm_bwd(e, e, e, torch.ones(64, device="cuda"))
    assert do.shape == dz.shape == (0, 64) and torch.equal(dw.cpu(), torch.zeros(64))


# ---------------------------------------------------------------- conv

def check_conv(gdn, lens, nqk, nv, dk, dv, k, io, bias=True, window=True, dstate=False, bits8=False, use_cu=True, seed=0):
    n = draws(seed + sum(lens) + 7 * k)
    t, c = sum(lens), 2 * nqk * dk + nv * dv
    x, w = n(t, c, io=io), n(c, k, by=0.5)
    b = n(c, by=0.5) if bias else None
    st = n(len(lens), c, k, io=io) if window else None
    dso = n(len(lens), c, k, io=io) if dstate else None
    dq, dk_, dv_ = n(t, nqk, dk, io=io), n(t, nqk, dk, io=io), n(t, nv, dv, io=io)
    xin, x64 = kept(gdn, x, bits8)
    cuda = lambda y: None if y is None else y.cuda()  # noqa: E731
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda() if use_cu else None
    got = gdn.qkv_conv_bwd(dq.cuda(), dk_.cuda(), dv_.cuda(), xin, w.cuda(), bias=cuda(b), conv_state=cuda(st), cu_seqlens=cu,
                           num_seqs=None if use_cu else len(lens), d_state_out=cuda(dso), output_d_state=True)
    zero = torch.zeros(len(lens), c, k).double()
    leaves = [x64.clone().requires_grad_(), w.double().requires_grad_(), (b if b is not None else torch.zeros(c)).double().requires_grad_(),
              (st.double() if st is not None else zero.clone()).requires_grad_()]
    y, new = G.conv(*leaves, lens)
    dy = torch.cat([dq.flatten(1), dk_.flatten(1), dv_.flatten(1)], 1).double()
    want = torch.autograd.grad([y, new], leaves, [dy, dso.double() if dso is not None else torch.zeros_like(new)], allow_unused=True)
    for name, a, e, ty in zip(("dx", "dw", "db", "dstate"), got, want, (io, torch.float32, torch.float32, io)):
        if name == "db" and not bias:
            assert a is None
            continue
        G.assert_close(a, e if e is not None else zero, ty, name)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("k", [1, 2, 3, 4])
@pytest.mark.parametrize("lens", [(1,), (33, 1, 2, 3, 0, 61), (200,)])
def test_conv_gradients(gdn, io, k, lens):
    check_conv(gdn, lens, 1, 2, 64, 64, k, io, dstate=True)


@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("bias,window", [(False, False), (True, True)])
def test_conv_gradients_of_long_runs(gdn, io, bits8, bias, window):
    """Several channel blocks, runs that cross sequences, sequences that cross runs."""
    check_conv(gdn, (511, 7, 2, 1000, 300), 4, 8, 128, 64, 4, io, bias=bias, window=window, bits8=bits8)


def test_conv_gradients_of_equal_lengths(gdn):
    check_conv(gdn, (40, 40, 40), 1, 1, 64, 128, 4, torch.bfloat16, use_cu=False, dstate=True)


def test_conv_gradients_of_no_tokens(gdn):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    dso = torch.randn(2, 192, 4, device="cuda")
    dx, dw, db, ds = gdn.qkv_conv_bwd(e(0, 1, 64), e(0, 1, 64), e(0, 1, 64), e(0, 192), torch.ones(192, 4, device="cuda"),
                                      bias=torch.ones(192, device="cuda"), cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda"),
                                      d_state_out=dso, output_d_state=True)
    assert dx.shape == (0, 192) and not dw.any() and not db.any() and torch.equal(ds, dso)


# ---------------------------------------------------------------- gate

@pytest.mark.parametrize("io", IO)
@pytest.mark.parametrize("tokens,nv", [(1, 1), (3, 300), (257, 8), (20000, 32), (4099, 33)])
def test_gate_gradients(gdn, io, tokens, nv):
    n = draws(tokens)
    a, b, al, dt = n(tokens, nv, by=3.0), n(tokens, nv, by=3.0), n(nv), n(nv)
    a[0], b[0] = 60.0, -60.0
    if tokens > 1:
        a[1], b[1] = -60.0, 60.0
    dg, dbeta = n(tokens, nv, io=io), n(tokens, nv, io=io)
    got = gdn.gate_bwd(*(t.cuda() for t in (dg, dbeta, a, b, al, dt)))
    leaves = [t.double().requires_grad_() for t in (a, b, al, dt)]
    want = torch.autograd.grad(list(G.gate(*leaves)), leaves, [dg.double(), dbeta.double()])
    for name, x, y, t in zip(("da", "db", "dA_log", "ddt"), got, want, (io, io, torch.float32, torch.float32)):
        G.assert_close(x, y, t, name, floor=1e-3)


def test_gate_gradients_of_no_tokens(gdn):
    e, h = torch.empty(0, 5, device="cuda"), torch.zeros(5, device="cuda")
    da, db, dA, ddt = gdn.gate_bwd(e, e, e, e, h, h)
    assert da.shape == db.shape == (0, 5) and not dA.any() and not ddt.any()


# ---------------------------------------------------------------- the layer

@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("io", IO)
def test_the_layer_and_back(gdn, io, bits8):
    """conv -> gated rule -> gated RMSNorm, and its gradients from what a training step keeps."""
    lens, nqk, nv, d, k = (150, 3, 64, 90), 1, 2, 64, 4
    n = draws(11)
    t, c = sum(lens), 2 * nqk * d + nv * d
    x, w, b = n(t, c, io=io), n(c, k, by=0.5), n(c, by=0.1)
    a, bb, al, dt = n(t, nv), n(t, nv), n(nv) - 2, n(nv)
    z, nw, dy = n(t, nv, d, io=io), n(d) + 1, n(t, nv, d, io=io)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    dev = [y.cuda() for y in (x, w, b, a, bb, al, dt, z, nw, dy)]
    X, W_, B_, A, BB, AL, DT, Z, NW, DY = dev
    keep = gdn.act_quantize if bits8 else (lambda y: y)
    back = (lambda y: gdn.act_dequantize(*y, io)) if bits8 else (lambda y: y)
    # forward
    q, kk, v, _ = gdn.qkv_conv_fwd(X, W_, nqk, nv, d, d, bias=B_, cu_seqlens=cu)
    o, _ = gdn.chunk_fwd_gated(q, kk, v, A, BB, AL, DT, cu_seqlens=cu)
    gdn.gated_rmsnorm(o, Z, NW)
    kx, ko, kz = keep(X), keep(o), keep(Z)
    # backward
    do, dz, dnw = gdn.gated_rmsnorm_bwd(DY, ko, kz, NW)
    q2, k2, v2, _ = gdn.qkv_conv_fwd(back(kx), W_, nqk, nv, d, d, bias=B_, cu_seqlens=cu)
    dq, dk, dv, dg, dbeta, _ = gdn.chunk_bwd(q2, k2, v2, A, BB, do, A_log=AL, dt_bias=DT, cu_seqlens=cu)
    da, db, dal, ddt = gdn.gate_bwd(dg, dbeta, A, BB, AL, DT)
    dx, dw, dbias, _ = gdn.qkv_conv_bwd(dq, dk, dv, kx, W_, bias=B_, cu_seqlens=cu)
    assert gdn.device_status() == 0
    # each stage's gradients in 64 bits from the inputs that the stage had
    o64, z64 = (read_back(*y) if bits8 else y.cpu().double() for y in (ko, kz))
    leaves = [o64.requires_grad_(), z64.requires_grad_(), nw.double().requires_grad_()]
    want = torch.autograd.grad(G.norm(*leaves, 1e-6), leaves, dy.double())
    for name, g, e, ty in zip(("do", "dz", "dnw"), (do, dz, dnw), want, (io, io, torch.float32)):
        G.assert_close(g, e, ty, name)
    gate = [y.double().requires_grad_() for y in (a, bb, al, dt)]
    g64, b64 = G.gate(*gate)
    want = G.rule_grads(q2, k2, v2, g64, b64, None, do, None, lens)
    for name, g, e in zip(("dq", "dk", "dv", "dg", "dbeta"), (dq, dk, dv, dg, dbeta), want):
        G.assert_close(g, e, io, name)
    want = torch.autograd.grad([g64, b64], gate, [dg.cpu().double(), dbeta.cpu().double()])
    for name, g, e, ty in zip(("da", "db", "dA_log", "ddt"), (da, db, dal, ddt), want, (io, io, torch.float32, torch.float32)):
        G.assert_close(g, e, ty, name)
    x64 = read_back(*kx) if bits8 else x.double()
    leaves = [x64.requires_grad_(), w.double().requires_grad_(), b.double().requires_grad_()]
    want = torch.autograd.grad(G.conv(*leaves, None, lens)[0], leaves, torch.cat([y.cpu().flatten(1) for y in (dq, dk, dv)], 1).double())
    for name, g, e, ty in zip(("dx", "dw", "dbias"), (dx, dw, dbias), want, (io, torch.float32, torch.float32)):
        G.assert_close(g, e, ty, name)


# ---------------------------------------------------------------- 8 bits, every bf16 number

def test_quantize_every_bf16_number(gdn):
    """All 65,536 bit patterns, 32 neighbours a group: subnormal groups, the last binade, infinities and NaN."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(2048, 32)
    x64 = x.double()
    fin = torch.isfinite(x64)
    top = torch.where(fin, x64.abs(), 0.0).amax(1, keepdim=True)
    m, ex = torch.frexp(top)                                   # top = m 2^ex, m in [1/2, 1): 448 = 7/8 2^9
    e = torch.where(top > 0, ex - 9 + (m > 0.875).int(), torch.tensor(-126)).clamp(min=-126)
    lim = torch.where(e >= 120, 240.0, 448.0)
    y = torch.where(fin, x64, 0.0) * torch.exp2(-e.double())
    step = torch.exp2(torch.frexp(y)[1].clamp(min=-5).double() - 4)   # three bits behind the first, 2^-9 at least
    want = torch.minimum(torch.maximum(torch.round(y / step) * step, -lim), lim) * torch.exp2(e.double())
    codes, scales = gdn.act_quantize(x.cuda())
    assert torch.equal(scales.cpu().int() - 127, e.int())
    got = read_back(codes, scales)
    assert torch.isnan(got[~fin]).all() and torch.equal(got[fin], want[fin])
    codes32, scales32 = gdn.act_quantize(x.float().cuda())
    assert torch.equal(scales32, scales) and torch.equal(codes32.view(torch.uint8)[fin.cuda()], codes.view(torch.uint8)[fin.cuda()])
