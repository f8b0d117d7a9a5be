"""The training operators of the Gated DeltaNet layer, as they are measured: cases, inputs, plain forms and 64-bit values.

Five operators, each the backward half of something the library runs forward, or what the backward reads:

  rule      gradients of the chunked gated delta rule (chunk_bwd)
  save      activations kept in 8 bits (e4m3, a power-of-two scale per 32 values) and read back
            (act_quantize, act_dequantize)
  norm      gradients of the gated RMSNorm epilogue (gated_rmsnorm_bwd), its saved o and z in 16 or 32
            bits, or in 8
  conv      gradients of the causal conv1d + SiLU (qkv_conv_bwd), its saved input in 16 or 32 bits, or in 8
  gate      gradients of the layer's gate (gate_bwd)

A plain form loops only where the definition recurs: over the chunks of a sequence, and over the six
doublings of a triangular inverse.
"""
import math

import torch

own = False

_CHUNK = 64   # tokens per chunk of the plain form
_GROUP = 32   # values that share a scale in 8 bits
_EPS = 1e-6   # of the L2 norm and of the gated RMSNorm


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short sequence of a small fp32 model: nothing but latency
        dict(name="rule f32 1x256 d64", op="rule", io="f32", lens="256", nqk=1, nv=1, dk=64, dv=64, s0=False),
        # a batch of an fp32 model that carries states between segments
        dict(name="rule f32 4x4096 d128", op="rule", io="f32", lens="4096,4096,4096,4096", nqk=4, nv=8, dk=128, dv=128, s0=True),
        # packed documents of very different lengths, one of them a single token
        dict(name="rule bf16 packed d128", op="rule", io="bf16", lens="4033,100,1,2757,640,65,3391,1500,64,2049,977,351",
             nqk=16, nv=32, dk=128, dv=128, s0=False),
        # two long documents
        dict(name="rule bf16 2x32768 d128", op="rule", io="bf16", lens="32768,32768", nqk=16, nv=32, dk=128, dv=128, s0=False),
        # the gate z of a short fp32 batch
        dict(name="save f32 1031x1024", op="save", io="f32", rows=1031, cols=1024),
        # the packed projection of a long batch
        dict(name="save bf16 65536x8192", op="save", io="bf16", rows=65536, cols=8192),
        # the epilogue of the fp32 batch
        dict(name="norm f32 16384x8 d128", op="norm", io="f32", tokens=16384, nv=8, dv=128, bits8=False),
        # the epilogue of the long batch, from what was kept in 8 bits
        dict(name="norm bf16 65536x32 d128 8bit", op="norm", io="bf16", tokens=65536, nv=32, dv=128, bits8=True),
        # packed documents that continue others: windows before every sequence, a bias
        dict(name="conv bf16 packed k4", op="conv", io="bf16", lens="4033,100,1,2757,640,65,3391,1500,2,2049,977,351",
             nqk=16, nv=32, dk=128, dv=128, k=4, bias=True, window=True, bits8=False),
        # the long batch, from what was kept in 8 bits
        dict(name="conv bf16 2x32768 k4 8bit", op="conv", io="bf16", lens="32768,32768", nqk=16, nv=32, dk=128, dv=128,
             k=4, bias=False, window=False, bits8=True),
        # the gate of one short fp32 sequence
        dict(name="gate f32 256x8", op="gate", io="f32", tokens=256, nv=8),
        # the gate of the long batch
        dict(name="gate bf16 65536x32", op="gate", io="bf16", tokens=65536, nv=32),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of the range."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(rng, most):
    total = _between(rng, 65, most)
    n = min(total, rng.choice([1, 1, 2, 3, 5, 9]))
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["rule", "rule", "save", "norm", "conv", "gate"])
    io = rng.choice(["f32", "bf16"])
    nqk = rng.choice([1, 2, 4, 8, 16])
    nv = nqk * rng.choice([1, 2, 2, 3, 4]) if nqk < 16 else nqk * rng.choice([1, 2])
    if op == "rule":
        # the state is kept in 32 bits; where the tokens are bf16 the sequences start from zeros
        return dict(op=op, io=io, lens=_lens(rng, 16384), nqk=nqk, nv=nv, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    s0=io == "f32" and rng.random() < 0.5)
    if op == "save":
        return dict(op=op, io=io, rows=_between(rng, 1, 32768), cols=64 * _between(rng, 1, 128))
    if op == "norm":
        return dict(op=op, io=io, tokens=_between(rng, 1, 32768), nv=nv, dv=rng.choice([64, 128]), bits8=rng.random() < 0.5)
    if op == "conv":
        return dict(op=op, io=io, lens=_lens(rng, 16384), nqk=nqk, nv=nv, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    k=rng.choice([1, 2, 3, 4, 4]), bias=rng.random() < 0.5, window=rng.random() < 0.5, bits8=rng.random() < 0.5)
    return dict(op=op, io=io, tokens=_between(rng, 1, 65536), nv=nv)


def work(case):
    e = 4 if case["io"] == "f32" else 2
    op = case["op"]
    if op == "rule":
        lens = [int(x) for x in case["lens"].split(",")]
        t, nqk, nv, dk, dv = sum(lens), case["nqk"], case["nv"], case["dk"], case["dv"]
        states = len(lens) * nv * dk * dv * 4 * (2 if case["s0"] else 0)
        # q, k, v, dout, g, beta in; dq, dk, dv, dg, dbeta out
        bytes_ = t * (4 * nqk * dk * e + 3 * nv * dv * e + nv * (8 + 2 * e)) + states
        # per chunk and v-head: eight products with the state or its gradient, the triangular products
        # within the chunk (five over Dk, six over Dv, half of each) and the inverse
        c = _CHUNK
        macs = 8 * c * dk * dv + c * c * (6 * dk + 5 * dv) / 2 + c ** 3 / 6
        return {"bytes": bytes_, "flops": 2 * macs * t / c * nv}
    if op == "save":
        n = case["rows"] * case["cols"]
        # in, the codes and scales out and in again, out
        return {"bytes": n * (2 * e + 2 + 2 / _GROUP), "flops": 4 * n}
    if op == "norm":
        n = case["tokens"] * case["nv"] * case["dv"]
        kept = (1 + 1 / _GROUP) if case["bits8"] else e
        return {"bytes": n * (3 * e + 2 * kept) + 8 * case["dv"], "flops": 24 * n}
    if op == "conv":
        lens = [int(x) for x in case["lens"].split(",")]
        c = 2 * case["nqk"] * case["dk"] + case["nv"] * case["dv"]
        n = sum(lens) * c
        kept = (1 + 1 / _GROUP) if case["bits8"] else e
        rest = c * case["k"] * 8 + (len(lens) * c * case["k"] * e * 2 if case["window"] else 0)
        return {"bytes": n * (2 * e + kept) + rest, "flops": n * (6 * case["k"] + 8)}
    n = case["tokens"] * case["nv"]
    return {"bytes": n * (8 + 4 * e) + 16 * case["nv"], "flops": 20 * n}


# ---------------------------------------------------------------------------------------- inputs

def _conv_plan(lens, k):
    """For every token and tap the row of [x; windows] it meets, and the tokens that meet a row: what a program that packs
    sequences knows from their lengths."""
    total, meets = sum(lens), []
    start = torch.repeat_interleave(torch.tensor([sum(lens[:i]) for i in range(len(lens))]), torch.tensor(lens))
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens))
    t = torch.arange(total)
    for i in range(k):
        p = t - (k - 1) + i
        meets.append(torch.where(p >= start, p, total + seq * k + (k + p - start)))
    return torch.stack(meets)


def prepare(case, seed):
    d = torch.device("cuda")
    r = torch.Generator(device=d)
    r.manual_seed(seed)
    io = torch.float32 if case["io"] == "f32" else torch.bfloat16
    op = case["op"]

    def normal(*shape, dtype=io, by=1.0):
        return (torch.randn(*shape, generator=r, device=d) * by).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=r, device=d) * (hi - lo) + lo

    s = {"case": dict(case), "io": io}
    if op in ("rule", "conv"):
        lens = [int(x) for x in case["lens"].split(",")]
        t, n = sum(lens), len(lens)
        s["lens"] = lens
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=d)
    if op == "rule":
        nqk, nv, dk, dv = case["nqk"], case["nv"], case["dk"], case["dv"]
        # q, k and v leave the conv through SiLU; the gate by the layer's own parametrisation, its rates log-uniform
        silu = torch.nn.functional.silu
        s["q"], s["k"], s["v"] = (silu(normal(t, h, w, dtype=torch.float32)).to(io) for h, w in ((nqk, dk), (nqk, dk), (nv, dv)))
        rate = uniform(0.0, 16.0, nv) * torch.exp(uniform(math.log(1e-3), math.log(1e-1), nv))
        s["g"] = -rate * torch.exp(0.5 * normal(t, nv, dtype=torch.float32))
        s["beta"] = torch.sigmoid(normal(t, nv, dtype=torch.float32))
        s["dout"] = normal(t, nv, dv, by=1e-3)
        s["s0"] = normal(n, nv, dk, dv, dtype=torch.float32, by=0.1) if case["s0"] else None
        s["ds"] = normal(n, nv, dk, dv, dtype=torch.float32, by=1e-3) if case["s0"] else None
        # where each token stands in [sequence, chunk, place], for the plain form
        chunks = -(-max(lens) // _CHUNK)
        s["chunks"] = chunks
        at = [torch.arange(x, device=d) + i * chunks * _CHUNK for i, x in enumerate(lens)]
        s["at"] = torch.cat(at) if len(set(lens)) > 1 or lens[0] % _CHUNK else None
    elif op == "save":
        s["x"] = normal(case["rows"], case["cols"])
    elif op == "norm":
        t, nv, dv = case["tokens"], case["nv"], case["dv"]
        s["o"], s["z"] = normal(t, nv, dv, by=0.3), normal(t, nv, dv)
        s["dy"] = normal(t, nv, dv, by=1e-3)
        s["w"] = uniform(0.5, 1.5, dv)
        if case["bits8"]:
            s["o"], s["z"] = _kept(s["o"]), _kept(s["z"])
    elif op == "conv":
        nqk, nv, dk, dv, k = case["nqk"], case["nv"], case["dk"], case["dv"], case["k"]
        c = 2 * nqk * dk + nv * dv
        s["x"] = normal(t, c)
        s["w"] = uniform(-1 / math.sqrt(k), 1 / math.sqrt(k), c, k)
        s["b"] = uniform(-1 / math.sqrt(k), 1 / math.sqrt(k), c) if case["bias"] else None
        s["state"] = normal(n, c, k) if case["window"] else None
        s["dq"], s["dk"], s["dv"] = (normal(t, h, w, by=1e-3) for h, w in ((nqk, dk), (nqk, dk), (nv, dv)))
        s["plan"] = _conv_plan(lens, k).to(d)
        if case["bits8"]:
            s["x"] = _kept(s["x"])
    else:
        t, nv = case["tokens"], case["nv"]
        s["a"], s["b"] = normal(t, nv, dtype=torch.float32), normal(t, nv, dtype=torch.float32)
        s["A_log"] = torch.log(uniform(0.01, 16.0, nv))
        s["dt"] = uniform(-7.0, 1.0, nv)
        s["dg"], s["dbeta"] = normal(t, nv, by=1e-3), normal(t, nv, by=1e-3)
    return s


# ---------------------------------------------------------------------------------------- 8 bits

def _scale_exponent(x):
    """The least e for which every |value| of a group of 32 is at most 448 * 2^e; x [..., groups, 32]."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True))
    return torch.clamp(e - torch.where(m <= 0.875, 9, 8), min=-126)


def _kept(x):
    """(codes, scale bytes) of x [..., D]: e4m3 codes, and e + 127 for every 32 values."""
    y = x.float().unflatten(-1, (-1, _GROUP))
    e = _scale_exponent(y)
    return torch.ldexp(y, -e).to(torch.float8_e4m3fn).flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _read(kept):
    """The values that (codes, scale bytes) stand for, in 32 bits."""
    codes, scale = kept
    y = codes.float().unflatten(-1, (-1, _GROUP))
    return torch.ldexp(y, scale.to(torch.int32).unsqueeze(-1) - 127).flatten(-2)


def _values(x):
    return _read(x) if isinstance(x, tuple) else x.float()


# ---------------------------------------------------------------------------------------- plain forms

def _plain_rule(s):
    c = s["case"]
    n, nc, cs = len(s["lens"]), s["chunks"], _CHUNK
    nqk, nv, dk, dv = c["nqk"], c["nv"], c["dk"], c["dv"]
    group = nv // nqk

    def chunked(x, heads):  # [T, heads, ...] -> [N, chunk, heads, place, ...] in 32 bits, zeros behind a sequence
        x = x.float()
        if s["at"] is not None:
            y = torch.zeros(n * nc * cs, *x.shape[1:], device=x.device)
            y[s["at"]] = x
            x = y
        x = x.reshape(n, nc, cs, *x.shape[1:]).transpose(2, 3)
        return x.repeat_interleave(group, 2) if heads == nqk and group > 1 else x

    def packed(x):  # the reverse, without the group: [N, chunk, heads, place, ...] -> [T, heads, ...]
        x = x.transpose(2, 3).flatten(0, 2)
        return x[s["at"]] if s["at"] is not None else x

    q, k, v, do = chunked(s["q"], nqk), chunked(s["k"], nqk), chunked(s["v"], nv), chunked(s["dout"], nv)
    g, beta = chunked(s["g"], nv), chunked(s["beta"], nv)
    rq = torch.rsqrt((q * q).sum(-1, keepdim=True) + _EPS)
    rk = torch.rsqrt((k * k).sum(-1, keepdim=True) + _EPS)
    scale = 1.0 / math.sqrt(dk)
    q, k = q * rq, k * rk
    # within the chunks, all at once
    gc = torch.cumsum(g, -1)
    last = gc[..., -1:]
    i = torch.arange(cs, device=q.device)
    low, strict = i[:, None] >= i[None, :], i[:, None] > i[None, :]
    decay = torch.exp(torch.where(low, gc[..., :, None] - gc[..., None, :], -math.inf))
    eg, el = torch.exp(gc)[..., None], torch.exp(last - gc)[..., None]
    kd = (k @ k.mT) * decay * strict          # decayed key products, below the diagonal
    p = (q @ k.mT) * decay * scale            # decayed query products, with the diagonal
    a = -beta[..., None] * kd
    t = _unit_inverse(a)
    w = t @ (k * eg * beta[..., None])
    u = t @ (v * beta[..., None])
    qe, kl = q * eg * scale, k * el
    gl = torch.exp(last)[..., None]
    # the states before every chunk, and the writes of every chunk
    state = s["s0"] if s["s0"] is not None else torch.zeros(n, nv, dk, dv, device=q.device)
    states, writes = [], []
    for j in range(nc):
        states.append(state)
        writes.append(u[:, j] - w[:, j] @ state)
        state = gl[:, j] * state + kl[:, j].mT @ writes[-1]
    # the gradient of the state behind every chunk, and of the writes
    y = p.mT @ do
    dstate = s["ds"] if s["ds"] is not None else torch.zeros(n, nv, dk, dv, device=q.device)
    dstates, dwrites = [None] * nc, [None] * nc
    for j in reversed(range(nc)):
        dstates[j] = dstate
        dwrites[j] = y[:, j] + kl[:, j] @ dstate
        dstate = gl[:, j] * dstate + qe[:, j].mT @ do[:, j] - w[:, j].mT @ dwrites[j]
    st, wr, dst, dwr = (torch.stack(x, 1) for x in (states, writes, dstates, dwrites))
    del states, writes, dstates, dwrites, y, w, u
    # everything else, all chunks at once
    dx = t.mT @ dwr
    da = (dx @ wr.mT) * strict
    dp = (do @ wr.mT) * low
    dqe, dkl, ks = do @ st.mT, wr @ dst.mT, k @ st
    dke = -(beta[..., None] * eg) * (dx @ st.mT)
    pair = -(beta[..., None]) * da * decay
    dot = dp * decay * scale
    dq = dqe * eg * scale + dot @ k
    dk = dkl * el + dot.mT @ q + dke + pair @ k + pair.mT @ k
    dval = beta[..., None] * dx
    dbeta = (dx * (v - eg * ks)).sum(-1) - (da * kd).sum(-1)
    both = dp * p * strict + da * a
    through = (dkl * kl).sum(-1)
    dgc = both.sum(-1) - both.sum(-2) + (dqe * qe).sum(-1) - (beta * eg[..., 0]) * (dx * ks).sum(-1) - through
    dgc[..., -1] += through.sum(-1) + gl[..., 0, 0] * (st * dst).sum((-1, -2))
    dg = torch.flip(torch.cumsum(torch.flip(dgc, (-1,)), -1), (-1,))
    # the heads of a group share q and k; then the norms
    dq, dk = (x.unflatten(2, (nqk, group)).sum(3) for x in (dq, dk))
    q, k, rq, rk = (x.unflatten(2, (nqk, group))[:, :, :, 0] for x in (q, k, rq, rk))
    dq = rq * (dq - q * (q * dq).sum(-1, keepdim=True))
    dk = rk * (dk - k * (k * dk).sum(-1, keepdim=True))
    io = s["io"]
    return {"dq": packed(dq).to(io), "dk": packed(dk).to(io), "dv": packed(dval).to(io), "dg": packed(dg[..., None])[..., 0].to(io),
            "dbeta": packed(dbeta[..., None])[..., 0].to(io), "ds0": dstate if s["s0"] is not None else None}


def _unit_inverse(a):
    """(I - A)^-1 of strictly lower triangular A [..., 64, 64]: [[T0, 0], [T1 A10 T0, T1]], doubling from single rows."""
    size = a.shape[-1]
    t = torch.eye(size, device=a.device).expand_as(a).clone()
    half = 1
    while half < size:
        at = torch.arange(0, size, 2 * half, device=a.device)
        i = at[:, None] + torch.arange(half, device=a.device)
        rows, cols = (i + half)[:, :, None], i[:, None, :]
        t0, t1 = t[..., i[:, :, None], cols], t[..., rows, rows.mT]
        t[..., rows, cols] = t1 @ a[..., rows, cols] @ t0
        half *= 2
    return t


def _plain_norm(s):
    o, z, dy, w = _values(s["o"]), _values(s["z"]), s["dy"].float(), s["w"]
    r = torch.rsqrt((o * o).mean(-1, keepdim=True) + _EPS)
    n, sig = o * r, torch.sigmoid(z)
    dn = dy * w * (z * sig)
    do = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dz = dy * n * w * (sig * (1 + z * (1 - sig)))
    return {"do": do.to(s["io"]), "dz": dz.to(s["io"]), "dw": (dy * n * (z * sig)).flatten(0, -2).sum(0)}


def _plain_conv(s):
    c, x, w, plan = s["case"], _values(s["x"]), s["w"], s["plan"]
    t, ch = x.shape
    k, n = c["k"], len(s["lens"])
    if s["state"] is not None:
        rows = torch.cat([x, s["state"].float().transpose(1, 2).reshape(n * k, ch)])
    else:
        rows = torch.cat([x, torch.zeros(n * k, ch, device=x.device)])
    pre = torch.zeros_like(x) if s["b"] is None else s["b"].expand_as(x).clone()
    for i in range(k):
        pre += w[:, i] * rows[plan[i]]
    sig = torch.sigmoid(pre)
    dy = torch.cat([s["dq"].flatten(1), s["dk"].flatten(1), s["dv"].flatten(1)], 1).float()
    dpre = dy * (sig * (1 + pre * (1 - sig)))
    del pre, sig, dy
    drows, dw = torch.zeros_like(rows), []
    for i in range(k):
        drows[plan[i]] += w[:, i] * dpre  # a tap meets every row at most once
        dw.append((dpre * rows[plan[i]]).sum(0))
    dstate = drows[t:].reshape(n, k, ch).transpose(1, 2).to(s["io"]) if s["state"] is not None else None
    return {"dx": drows[:t].to(s["io"]), "dw": torch.stack(dw, 1), "db": dpre.sum(0) if s["b"] is not None else None, "dstate": dstate}


def _plain_gate(s):
    u = s["a"] + s["dt"]
    rate, beta = torch.exp(s["A_log"]), torch.sigmoid(s["b"])
    g = -rate * (torch.clamp(u, min=0) + torch.log1p(torch.exp(-u.abs())))
    dg, dbeta = s["dg"].float(), s["dbeta"].float()
    da = -dg * rate * torch.sigmoid(u)
    db = dbeta * beta * (1 - beta)
    return {"da": da.to(s["io"]), "db": db.to(s["io"]), "dA_log": (dg * g).sum(0), "ddt": da.sum(0)}


# ---------------------------------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "save":
            return _read(_kept(s["x"])).to(s["io"])
        return {"rule": _plain_rule, "norm": _plain_norm, "conv": _plain_conv, "gate": _plain_gate}[op](s)
    import gated_deltanet_chunk_b200 as gdn
    if op == "rule":
        r = gdn.chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"], initial_state=s["s0"], d_final_state=s["ds"], cu_seqlens=s["cu"])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), r))
    if op == "save":
        codes, scales = gdn.act_quantize(s["x"])
        return gdn.act_dequantize(codes, scales, s["io"])
    if op == "norm":
        return dict(zip(("do", "dz", "dw"), gdn.gated_rmsnorm_bwd(s["dy"], s["o"], s["z"], s["w"], _EPS)))
    if op == "conv":
        r = gdn.qkv_conv_bwd(s["dq"], s["dk"], s["dv"], s["x"], s["w"], bias=s["b"], conv_state=s["state"], cu_seqlens=s["cu"])
        return dict(zip(("dx", "dw", "db", "dstate"), r))
    return dict(zip(("da", "db", "dA_log", "ddt"), gdn.gate_bwd(s["dg"], s["dbeta"], s["a"], s["b"], s["A_log"], s["dt"])))


# ---------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def double(x):
        """The 64-bit values of a tensor, or of what is kept in 8 bits."""
        if isinstance(x, tuple):
            return x[0].double() * torch.exp2(x[1].double() - 127).repeat_interleave(_GROUP, -1)
        return x.double()

    if op == "save":
        y = double(s["x"]).unflatten(-1, (-1, _GROUP))
        top = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(top / 448).clamp(min=-200))
        e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, torch.where(top > 448 * torch.exp2(e), e + 1, e)).clamp(min=-126)
        y = y * torch.exp2(-e)
        # the numbers with three bits behind the first one, none finer than 2^-9
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(y / step) * step * torch.exp2(e)).flatten(-2)  # round() takes ties to even

    if op in ("norm", "gate", "conv"):  # the definition of the forward pass, differentiated
        if op == "norm":
            o, z, w = (double(s[x]).requires_grad_() for x in ("o", "z", "w"))
            y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + _EPS) * w * (z / (1 + torch.exp(-z)))
            got = torch.autograd.grad(y, [o, z, w], double(s["dy"]))
            return dict(zip(("do", "dz", "dw"), got))
        if op == "gate":
            a, b, al, dt = (double(s[x]).requires_grad_() for x in ("a", "b", "A_log", "dt"))
            g, beta = -torch.exp(al) * torch.log(1 + torch.exp(a + dt)), 1 / (1 + torch.exp(-b))
            got = torch.autograd.grad([g, beta], [a, b, al, dt], [double(s["dg"]), double(s["dbeta"])])
            return dict(zip(("da", "db", "dA_log", "ddt"), got))
        x, w, k = double(s["x"]), double(s["w"]), case["k"]
        dy = torch.cat([s["dq"].flatten(1), s["dk"].flatten(1), s["dv"].flatten(1)], 1)
        n, ch = len(s["lens"]), x.shape[1]
        dx, dw, db, dstate = torch.empty_like(x), torch.empty_like(w), torch.empty(ch, device=x.device).double(), torch.empty(n, ch, k, device=x.device).double()
        for lo in range(0, ch, 512):
            cut = slice(lo, min(lo + 512, ch))
            xs, ws = x[:, cut].clone().requires_grad_(), w[cut].clone().requires_grad_()
            bs = (double(s["b"])[cut] if s["b"] is not None else torch.zeros_like(ws[:, 0])).detach().requires_grad_()
            st = (double(s["state"])[:, cut] if s["state"] is not None else torch.zeros(n, ws.shape[0], k, device=x.device).double()).detach().clone().requires_grad_()
            rows, at = [], 0
            for j, length in enumerate(s["lens"]):
                line = torch.cat([st[j].t(), xs[at:at + length]])  # the window's k inputs, then the sequence
                pre = bs + sum(ws[:, i] * line[1 + i:1 + i + length] for i in range(k))
                rows.append(pre / (1 + torch.exp(-pre)))
                at += length
            got = torch.autograd.grad(torch.cat(rows), [xs, ws, bs, st], double(dy[:, cut]))
            dx[:, cut], dw[cut], db[cut], dstate[:, cut] = got
        return {"dx": dx, "dw": dw, "db": db if s["b"] is not None else None, "dstate": dstate if s["state"] is not None else None}

    # the rule, token by token, and back: the states of a stretch are formed again from the one before it
    lens, nqk, nv, dk, dv = s["lens"], case["nqk"], case["nv"], case["dk"], case["dv"]
    longest, stretch = max(lens), 64
    if longest * len(lens) * nv * dk * dv > 6e10 or longest > 20000:
        return None  # over about 20 seconds
    n, group = len(lens), nv // nqk

    def padded(x, heads):  # [T, heads, ...] -> [place, N, heads, ...]
        y = torch.zeros(longest, n, *x.shape[1:], device=x.device, dtype=torch.float64)
        at = 0
        for j, length in enumerate(lens):
            y[:length, j] = x[at:at + length].double()
            at += length
        return y.repeat_interleave(group, 2) if heads != nv else y

    q0, k0 = padded(s["q"], nqk), padded(s["k"], nqk)
    rq, rk = ((x * x).sum(-1, keepdim=True).add(_EPS).pow(-0.5) for x in (q0, k0))
    q, k = q0 * rq / math.sqrt(dk), k0 * rk
    v, do, g, beta = padded(s["v"], nv), padded(s["dout"], nv), padded(s["g"], nv), padded(s["beta"], nv)
    alpha = torch.exp(g)
    zero = torch.zeros(n, nv, dk, dv, device=q.device, dtype=torch.float64)

    def step(state, j):  # the state of token j, its decayed predecessor, and what the key did not find
        kept = alpha[j, ..., None, None] * state
        miss = v[j] - (kept * k[j, ..., None]).sum(-2)
        return kept + k[j, ..., None] * (beta[j, ..., None] * miss)[..., None, :], kept, miss

    state, marks = s["s0"].double() if s["s0"] is not None else zero, []
    for j in range(longest):
        if j % stretch == 0:
            marks.append(state)
        state = step(state, j)[0]
    dq, dkey, dval, dg, dbeta = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(g)
    ds = s["ds"].double() if s["ds"] is not None else zero.clone()
    for m in reversed(range(len(marks))):
        state, seen = marks[m], []
        for j in range(m * stretch, min(longest, (m + 1) * stretch)):
            state, kept, miss = step(state, j)
            seen.append((j, state, kept, miss))
        for j, after, kept, miss in reversed(seen):
            dq[j] = (after * do[j, ..., None, :]).sum(-1)
            ds = ds + q[j, ..., None] * do[j, ..., None, :]
            ddelta = (ds * k[j, ..., None]).sum(-2)
            dmiss = beta[j, ..., None] * ddelta
            dval[j], dbeta[j] = dmiss, (ddelta * miss).sum(-1)
            dkey[j] = (ds * (beta[j, ..., None] * miss)[..., None, :]).sum(-1) - (kept * dmiss[..., None, :]).sum(-1)
            ds = ds - k[j, ..., None] * dmiss[..., None, :]
            dg[j] = (ds * kept).sum((-1, -2))
            ds = alpha[j, ..., None, None] * ds
    dq, dkey = (x.unflatten(2, (nqk, group)).sum(3) for x in (dq / math.sqrt(dk), dkey))
    q0, k0, rq, rk = (x[:, :, ::group] for x in (q0, k0, rq, rk))
    dq = rq * dq - rq ** 3 * q0 * (q0 * dq).sum(-1, keepdim=True)
    dkey = rk * dkey - rk ** 3 * k0 * (k0 * dkey).sum(-1, keepdim=True)

    def packed(x):
        return torch.cat([x[:length, j] for j, length in enumerate(lens)])

    return {"dq": packed(dq), "dk": packed(dkey), "dv": packed(dval), "dg": packed(dg), "dbeta": packed(dbeta),
            "ds0": ds if s["s0"] is not None else None}
