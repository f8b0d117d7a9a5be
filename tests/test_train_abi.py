"""Refusals of the training calls, on the host: the C ABI with fake addresses, and the binding's checks of its tensors."""
import ctypes

import pytest
import torch

A = 0x100000          # fake, never dereferenced; tensors 16 MB apart
S = 0x1000000
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_chunk_b200 import build
    build.build()
    import gated_deltanet_chunk_b200 as g
    return g.lib()


def valid(rc):
    """Past every check of the arguments: on a machine without a GPU the device check is what is left."""
    assert torch.cuda.is_available() or rc in (-5, -6), rc


def params(nqk=2, nv=4, dk=128, dv=128, bf16=True, l2=True, scale=0.0, kernel="auto"):
    import gated_deltanet_chunk_b200 as g
    return g.make_params(nqk, nv, dk, dv, bf16, l2, scale, kernel)


RULE = ["q", "k", "v", "g", "beta", "A_log", "dt", "s0", "dout", "ds", "cu", "dq", "dk", "dv", "dg", "dbeta", "ds0", "ws"]
AT = {n: A + i * S for i, n in enumerate(RULE)}


def rule(L, p=None, n=2, T=256, size=BIG, **kw):
    x = dict(AT, A_log=None, dt=None, s0=None, ds=None, cu=None, ds0=None)
    x.update(kw)
    p = params() if p is None else p
    return L.gdn_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["beta"], x["A_log"], x["dt"], x["s0"], x["dout"], x["ds"], x["cu"], n, T,
                           x["dq"], x["dk"], x["dv"], x["dg"], x["dbeta"], x["ds0"], x["ws"], size, ctypes.byref(p), None)


def test_chunk_bwd_refusals(L):
    for name in ("q", "k", "v", "g", "beta", "dout", "dq", "dk", "dv", "dg", "dbeta", "ws"):
        assert rule(L, **{name: None}) == -1, name
    assert L.gdn_chunk_bwd(*[None] * 11, 1, 0, *[None] * 7, 0, None, None) == -1
    assert rule(L, A_log=AT["A_log"]) == -1 and rule(L, dt=AT["dt"]) == -1      # both or neither
    for p in (params(nqk=3), params(dk=96), params(dv=32)):
        assert rule(L, p) == -2
    assert rule(L, n=0) == -2 and rule(L, n=65536) == -2 and rule(L, T=-64) == -2 and rule(L, T=1 << 31) == -2
    assert rule(L, T=255) == -2                                                 # uneven without cu_seqlens
    for p in (params(bf16=False, kernel="tc"), params(l2=False, kernel="tc")):
        assert rule(L, p) == -2                                                 # no tensor-core path for them
    need = L.gdn_chunk_bwd_workspace(2, 256, ctypes.byref(params()))
    assert need > 0 and rule(L, size=need - 1) == -2
    for name in ("q", "dout", "g", "cu", "ds0", "ws", "dbeta"):
        assert rule(L, **{name: AT[name] + 8}) == -3, name
    assert rule(L, A_log=AT["A_log"] + 2, dt=AT["dt"]) == -3
    for name, over in (("dq", "q"), ("dv", "dout"), ("dk", "dq"), ("dbeta", "dg"), ("ws", "v"), ("ws", "dk"), ("dg", "g")):
        assert rule(L, **{name: AT[over]}) == -4, name
    assert rule(L, ds=AT["ds"], ds0=AT["ds"]) == -4 and rule(L, s0=AT["s0"], ds0=AT["s0"] + 64) == -4
    assert rule(L, ds0=AT["dv"] + 1024) == -4
    valid(rule(L))
    valid(rule(L, size=need))
    valid(rule(L, s0=AT["s0"], ds=AT["ds"], ds0=AT["ds0"], cu=AT["cu"], A_log=AT["A_log"] + 4, dt=AT["dt"] + 4))
    valid(rule(L, params(bf16=False, l2=False)))
    nothing = {k: None for k in RULE}
    valid(rule(L, T=0, size=0, **nothing))                                      # no tokens: nothing is needed


def test_chunk_bwd_workspace(L):
    def need(n, t, **kw):
        return L.gdn_chunk_bwd_workspace(n, t, ctypes.byref(params(**kw)))
    assert need(1, 0) == 0 and need(0, 64) == -2 and need(1, -1) == -2 and need(1, 64, dk=32) == -2
    assert need(1, 64) % 16 == 0 and need(1, 64) < need(2, 64) <= need(2, 128)   # a slot for every sequence's ragged end
    assert need(1, 1 << 30, nv=64, nqk=64) > 1 << 40                             # beyond 32 bits
    assert need(1, 4096, kernel="simt") != need(1, 4096)


ACT = dict(x=A, codes=A + S, scales=A + 2 * S, n=4096, io=1)


def test_act_refusals(L):
    for f, order in ((L.gdn_act_quantize, ("x", "codes", "scales")), (L.gdn_act_dequantize, ("codes", "scales", "x"))):
        def call(**kw):
            y = dict(ACT, **kw)
            return f(*[y[k] for k in order], y["n"], y["io"], None)
        for name in order:
            assert call(**{name: None}) == -1
        assert call(n=33) == -2 and call(n=-32) == -2 and call(io=2) == -2
        assert call(x=A + 8) == -3 and call(codes=A + S + 8) == -3
        assert call(codes=A + 4096) == -4 and call(scales=A + S + 32) == -4
        assert call(n=0, x=None, codes=None, scales=None) == 0
        valid(call(scales=A + 2 * S + 1))
        valid(call())


def test_norm_refusals(L):
    need = L.gdn_gated_rmsnorm_bwd_workspace(100, 128, 1)
    assert need > 0 and L.gdn_gated_rmsnorm_bwd_workspace(-1, 128, 1) == -2 and L.gdn_gated_rmsnorm_bwd_workspace(1, 96, 1) == -2
    base = dict(dy=A, o=A + S, os=None, z=A + 2 * S, zs=None, w=A + 3 * S, eps=1e-6, do=A + 4 * S, dz=A + 5 * S, dw=A + 6 * S,
                rows=100, dim=128, io=1, ws=A + 7 * S, size=need)

    def call(**kw):
        return L.gdn_gated_rmsnorm_bwd(*dict(base, **kw).values(), None)
    for name in ("dy", "o", "z", "w", "do", "dz", "dw", "ws"):
        assert call(**{name: None}) == -1, name
    assert call(dim=32) == -2 and call(rows=1 << 31) == -2 and call(io=5) == -2 and call(size=need - 1) == -2
    assert call(eps=-1.0) == -2 and call(eps=float("nan")) == -2 and call(eps=float("inf")) == -2
    assert call(dy=A + 4) == -3 and call(w=A + 3 * S + 4) == -3 and call(dw=A + 6 * S + 2) == -3
    assert call(do=A) == -4 and call(dz=A + 2 * S + 256) == -4 and call(dz=A + 4 * S) == -4 and call(ws=A + 6 * S) == -4
    assert call(os=A + 4 * S) == -4                                             # the scales are an input too
    valid(call())
    valid(call(os=A + 8 * S + 1, zs=A + 9 * S + 3))
    valid(call(rows=0, dy=None, o=None, z=None, w=None, do=None, dz=None, ws=None, size=0))


def test_conv_refusals(L):
    p = params()
    need = L.gdn_qkv_conv_bwd_workspace(256, 4, ctypes.byref(p))
    assert need > 0 and L.gdn_qkv_conv_bwd_workspace(256, 5, ctypes.byref(p)) == -2
    base = dict(dq=A, dk=A + S, dv=A + 2 * S, x=A + 3 * S, xs=None, w=A + 4 * S, b=None, st=None, dso=None, cu=None, n=2, T=256, k=4,
                dx=A + 5 * S, dw=A + 6 * S, db=None, ds=None, ws=A + 7 * S, size=need)

    def call(pp=p, **kw):
        return L.gdn_qkv_conv_bwd(*dict(base, **kw).values(), ctypes.byref(pp), None)
    for name in ("dq", "dk", "dv", "x", "w", "dx", "dw", "ws"):
        assert call(**{name: None}) == -1, name
    assert call(k=0) == -2 and call(k=5) == -2 and call(n=0) == -2 and call(T=255) == -2 and call(size=need - 1) == -2
    assert call(params(nqk=3)) == -2
    assert call(x=A + 3 * S + 8) == -3 and call(w=A + 4 * S + 4) == -3 and call(xs=A + 8 * S + 1) == -3 and call(cu=A + 8 * S + 4) == -3
    assert call(dx=A + 3 * S) == -4 and call(dw=A + 4 * S) == -4 and call(db=A + 6 * S) == -4
    assert call(dso=A + 8 * S, ds=A + 8 * S) == -4 and call(ws=A + 5 * S + 4096) == -4
    valid(call())
    valid(call(xs=A + 8 * S + 2, b=A + 9 * S + 4, db=A + 10 * S + 4, st=A + 11 * S, dso=A + 12 * S, ds=A + 13 * S))


def test_gate_refusals(L):
    need = L.gdn_gate_bwd_workspace(65536, 32)
    assert need > 0 and L.gdn_gate_bwd_workspace(1, 8) == 0                     # few tokens: one block
    assert L.gdn_gate_bwd_workspace(-1, 8) == -2 and L.gdn_gate_bwd_workspace(1, 0) == -2 and L.gdn_gate_bwd_workspace(1, 65536) == -2
    base = dict(dg=A, dbeta=A + S, a=A + 2 * S, b=A + 4 * S, A_log=A + 6 * S, dt=A + 7 * S, da=A + 8 * S, db=A + 9 * S, dA=A + 10 * S,
                ddt=A + 11 * S, T=65536, nv=32, io=1, ws=A + 12 * S, size=need)

    def call(**kw):
        return L.gdn_gate_bwd(*dict(base, **kw).values(), None)
    for name in ("dg", "dbeta", "a", "b", "A_log", "dt", "da", "db", "dA", "ddt", "ws"):
        assert call(**{name: None}) == -1, name
    assert call(T=-1) == -2 and call(nv=0) == -2 and call(io=3) == -2 and call(size=need - 1) == -2
    assert call(dg=A + 2) == -3 and call(A_log=A + 6 * S + 2) == -3
    assert call(da=A) == -4 and call(db=A + 8 * S) == -4 and call(dA=A + 6 * S) == -4 and call(ddt=A + 10 * S + 64) == -4
    valid(call())
    valid(call(T=0, dg=None, dbeta=None, a=None, b=None, da=None, db=None, ws=None, size=0))


# ---------------------------------------------------------------- the binding

def gdn():
    import gated_deltanet_chunk_b200 as g
    return g


def tokens(t=8, nqk=1, nv=2, d=64, io=torch.float32):
    e = torch.zeros
    return dict(q=e(t, nqk, d, dtype=io), k=e(t, nqk, d, dtype=io), v=e(t, nv, d, dtype=io), g=e(t, nv), beta=e(t, nv), dout=e(t, nv, d, dtype=io))


def refuses(word, f, *args, **kw):
    with pytest.raises(gdn().GdnError, match=word) as e:
        f(*args, **kw)
    assert e.value.status == -2


def test_binding_checks_the_rules_tensors(L):
    f, x = gdn().chunk_bwd, tokens()
    refuses("tensors on cpu", f, **x, workspace=torch.zeros(1 << 22, dtype=torch.uint8))
    refuses("dout", f, **dict(x, dout=x["dout"][:1].expand(8, 2, 64)))                  # an expanded gradient
    refuses("dout", f, **dict(x, dout=x["dout"].transpose(0, 1).contiguous().transpose(0, 1)))
    refuses("dout", f, **dict(x, dout=x["dout"].bfloat16()))
    refuses("dout", f, **dict(x, dout=x["dout"][1:]))
    refuses("q ", f, **dict(x, q=x["q"].half()))
    refuses("k ", f, **dict(x, k=x["k"].bfloat16()))
    refuses("g ", f, **dict(x, g=x["g"].double()))
    refuses("cu_seqlens", f, **x, cu_seqlens=torch.tensor([0, 8]))                     # 64-bit offsets
    refuses("initial_state", f, **x, initial_state=torch.zeros(2, 2, 64, 64))
    refuses("dq", f, **x, dq=torch.zeros(8, 64))
    refuses("workspace", f, **x, workspace=torch.zeros(64, 64).t())
    refuses("gdn_chunk_bwd", f, **tokens(d=96))


def test_binding_checks_the_other_calls_tensors(L):
    g, z = gdn(), torch.zeros
    f8 = torch.float8_e4m3fn
    refuses("gdn_act_quantize", g.act_quantize, z(4, 40))
    refuses("x ", g.act_quantize, z(64, 32).t())
    refuses("x ", g.act_quantize, z(4, 32, dtype=torch.float16))
    refuses("codes", g.act_quantize, z(4, 32), codes=z(4, 32, dtype=torch.uint8))
    refuses("scales", g.act_dequantize, z(4, 32, dtype=f8), z(4, 2, dtype=torch.uint8), torch.float32)
    refuses("gdn_act_dequantize", g.act_dequantize, z(4, 32, dtype=f8), z(4, 1, dtype=torch.uint8), torch.float16)
    y = z(4, 64)
    refuses("dy", g.gated_rmsnorm_bwd, z(64, 4).t(), y, y, z(64))
    refuses("o ", g.gated_rmsnorm_bwd, y, y.bfloat16(), y, z(64))
    refuses("o ", g.gated_rmsnorm_bwd, y, z(4, 64, dtype=f8), y, z(64))                 # codes without their scales
    refuses("z codes", g.gated_rmsnorm_bwd, y, y, (y, z(4, 2, dtype=torch.uint8)), z(64))
    refuses("weight", g.gated_rmsnorm_bwd, y, y, y, z(64).bfloat16())
    q, v = z(5, 1, 64), z(5, 2, 64)
    refuses("mixed_qkv", g.qkv_conv_bwd, q, q, v, z(5, 512)[:, ::2], z(256, 4))
    refuses("weight", g.qkv_conv_bwd, q, q, v, z(5, 256), z(4, 256).t())
    refuses("dk", g.qkv_conv_bwd, q, z(6, 1, 64), v, z(5, 256), z(256, 4))
    refuses("gdn_qkv_conv_bwd", g.qkv_conv_bwd, q, q, v, z(5, 320), z(320, 4))
    refuses("d_state_out", g.qkv_conv_bwd, q, q, v, z(5, 256), z(256, 4), d_state_out=z(1, 256, 3))
    a, h = z(5, 3), z(3)
    refuses("dbeta", g.gate_bwd, a, a.bfloat16(), a, a, h, h)
    refuses("A_log", g.gate_bwd, a, a, a, a, z(1).expand(3), h)
    refuses("ddt_bias", g.gate_bwd, a, a, a, a, h, h, ddt_bias=z(4))
