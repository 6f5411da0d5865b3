"""Cases of the layers around the sparse memory, for timing and for comparing outputs.

Three operators, each for prompts, for single tokens and for training:

- the short causal convolution over the tokens of a packed projection,
- the selective state space scan that reads its output,
- the block norm that joins a layer's output to the residual stream and normalises it for the
  next layer.

With ``own`` false :func:`run` computes them from elementary torch operations in float32 (float64
for the cumulated log-decays and the sums over them); with ``own`` true it calls the library.
:func:`exact` computes the same values in float64, token by token where the operator is a
recurrence.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_DEVICE = "cuda"
_CHUNK = 256  # tokens per block of the plain scan
_EPS = 1e-5


# --------------------------------------------------------------------------------------- cases
def _conv(name, op, B, T, C, K, dtype, ragged=False, state=False, bias=True, act="silu", gap=0):
    return dict(name=name, op=op, B=B, T=T, C=C, K=K, dtype=dtype, ragged=ragged, state=state, bias=bias, act=act,
                gap=gap)


def _scan(name, op, B, T, H, G, d_k, d_v, dtype, ragged=False, state=False):
    return dict(name=name, op=op, B=B, T=T, H=H, G=G, d_k=d_k, d_v=d_v, dtype=dtype, ragged=ragged, state=state)


def _norm(name, op, M, D, y, r, x, gate, gate_rows, act, scale=1.0):
    return dict(name=name, op=op, M=M, D=D, y=y, r=r, x=x, gate=gate, gate_rows=gate_rows, act=act, scale=scale)


def listed():
    return [
        # a batch of prompts of the 1.4B-scale layer: x | B | C of 16 heads, read out of the wider
        # projection that also holds the output gate
        _conv("conv prompts", "conv", 8, 4096, 16 * 64 + 2 * 128, 4, "bf16", gap=1024),
        # one new token of 64 sequences
        _conv("conv tokens", "conv_step", 64, 1, 16 * 128 + 2 * 128, 4, "bf16"),
        # a training step on sequences of different lengths that continue from a state
        _conv("conv training", "conv_backward", 4, 2048, 8 * 128 + 4 * 128, 4, "bf16", ragged=True, state=True),
        # the same prompts through the scan: 128 units fill half the chip
        _scan("scan prompts", "scan", 8, 4096, 16, 1, 128, 64, "bf16"),
        # one long document of the 8B-scale layer: few units, many tokens
        _scan("scan long", "scan", 1, 131072, 8, 2, 128, 128, "bf16"),
        # three short float32 sequences of different lengths, odd widths, continued from a state
        _scan("scan ragged", "scan", 3, 777, 6, 3, 40, 24, "f32", ragged=True, state=True),
        # one new token of 64 sequences
        _scan("scan tokens", "scan_step", 64, 1, 16, 1, 128, 128, "bf16"),
        # one new token of one sequence: latency alone
        _scan("scan one token", "scan_step", 1, 1, 8, 1, 64, 64, "bf16"),
        # a training step of the small layer
        _scan("scan training", "scan_backward", 4, 2048, 8, 1, 128, 128, "bf16"),
        # the residual stream of those prompts, with a gate of every token
        _norm("norm prompts", "norm", 8 * 4096, 2048, "f32", "bf16", "bf16", "bf16", 8 * 4096, "sigmoid"),
        # one new token of 64 sequences, with a learned scale of each channel
        _norm("norm tokens", "norm", 64, 1024, "f32", "f32", "bf16", "f32", 1, "none", 0.5),
        # a training step, with a gate of each sequence
        _norm("norm training", "norm_backward", 8192, 1536, "bf16", "f32", "f32", "bf16", 4, "silu", 0.7),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
        return max(lo, min(hi, int(v) // step * step))

    op = rng.choice(["conv", "conv_step", "conv_backward", "scan", "scan_step", "scan_backward", "norm",
                     "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("conv"):
        C, K = log(8, 4096, 8), rng.randint(2, 8)
        bias, act = rng.random() < 0.5, rng.choice(["silu", "none"])
        if op == "conv_step":
            return _case(_conv(None, op, log(1, 256), 1, C, K, dtype, bias=bias, act=act))
        T = log(1, 8192)
        B = log(1, max(1, (12 if op == "conv_backward" else 40) * 2**20 // (T * C)))
        return _case(_conv(None, op, min(B, 64), T, C, K, dtype, rng.random() < 0.5, rng.random() < 0.5, bias, act,
                           rng.choice([0, 8, 512])))
    if op.startswith("scan"):
        G = log(1, 8)
        H = G * log(1, 16 // G)
        d_k, d_v = rng.choice([16, 24, 40, 64, 64, 128, 128]), rng.choice([8, 24, 32, 64, 64, 128, 128, 200])
        if op == "scan_step":
            return _case(_scan(None, op, log(1, 128), 1, H, G, d_k, d_v, dtype))
        T = log(1, 2500 if op == "scan_backward" else 20000)
        most = 2**29 if op == "scan_backward" else 2**33  # states of every token are kept by the check
        B = log(1, max(1, min(most // (T * H * d_k * d_v), 2**19 // (T * H))))
        return _case(_scan(None, op, min(B, 32), T, H, G, d_k, d_v, dtype, rng.random() < 0.5, rng.random() < 0.5))
    D = log(64, 8192, 8)
    B = log(1, 16)
    M = B * log(1, max(1, (12 if op == "norm_backward" else 50) * 2**20 // (B * D)))
    y, r, x, g = (rng.choice(["f32", "bf16"]) for _ in range(4))
    return _case(_norm(None, op, M, D, y, r, x, g, rng.choice([0, 1, B, M]), rng.choice(["none", "sigmoid", "silu"]),
                       rng.choice([1.0, 0.25])))


def _case(c):
    del c["name"]
    return c


# -------------------------------------------------------------------------------------- inputs
def _lengths(c, g):
    """Lengths of a ragged batch: spread over [0, T], one sequence full, one (of several) empty."""
    n = torch.randint(0, c["T"] + 1, (c["B"],), generator=g, device=_DEVICE, dtype=torch.int32)
    n[0] = c["T"]
    if c["B"] > 2:
        n[1] = 0
    return n


def prepare(case, seed):
    c = case
    g = torch.Generator(device=_DEVICE).manual_seed(seed)

    def normal(*shape, dtype="f32", scale=1.0):
        return (torch.randn(*shape, generator=g, device=_DEVICE) * scale).to(_DTYPES[dtype])

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=_DEVICE) * (hi - lo) + lo

    def empty(*shape, dtype="f32"):
        return torch.empty(*shape, device=_DEVICE, dtype=_DTYPES[dtype])

    s = {"case": c}
    if c["op"].startswith("conv"):
        B, T, C, K, dt = c["B"], c["T"], c["C"], c["K"], c["dtype"]
        wide = normal(B, T, C + c["gap"], dtype=dt)
        s.update(x=wide[..., :C], w=normal(C, K, scale=K ** -0.5), b=normal(C, scale=0.2) if c["bias"] else None,
                 lengths=_lengths(c, g) if c["ragged"] else None, y=empty(B, T, C, dtype=dt),
                 s_in=normal(B, K - 1, C, dtype=dt) if c["state"] or c["op"] == "conv_step" else None,
                 s_out=empty(B, K - 1, C, dtype=dt))
        if c["op"] == "conv_backward":
            s.update(dy=normal(B, T, C), ds_out=normal(B, K - 1, C) if c["state"] else None, dx=empty(B, T, C + c["gap"])[..., :C],
                     dw=empty(C, K), db=empty(C) if c["bias"] else None, ds_in=empty(B, K - 1, C) if c["state"] else None)
        return s
    if c["op"].startswith("scan"):
        B, T, H, G, N, P, dt = c["B"], c["T"], c["H"], c["G"], c["d_k"], c["d_v"], c["dtype"]
        xbc = normal(B, T, H * P + 2 * G * N, dtype=dt)
        step = torch.exp(uniform(math.log(1e-3), math.log(0.1), H))  # time steps before the input's share
        s.update(xbc=xbc, dt=normal(B, T, H), A_log=torch.log(uniform(1.0, 16.0, H)),
                 dt_bias=step + torch.log(-torch.expm1(-step)), D=uniform(0.5, 1.5, H),
                 lengths=_lengths(c, g) if c["ragged"] else None,
                 s_in=normal(B, H, P, N, scale=0.1) if c["state"] or c["op"] == "scan_step" else None,
                 s_out=empty(B, H, P, N), o=empty(B, H, T, P))
        if c["op"] == "scan_backward":
            s.update(go=normal(B, H, T, P), ds_out=normal(B, H, P, N, scale=0.1) if c["state"] else None,
                     dxbc=empty(B, T, H * P + 2 * G * N), ddt=empty(B, T, H), dA_log=empty(H), ddt_bias=empty(H),
                     dD=empty(H), ds_in=empty(B, H, P, N) if c["state"] else None)
        return s
    M, D, gr = c["M"], c["D"], c["gate_rows"]
    s.update(y=normal(M, D, dtype=c["y"]), r=normal(M, D, dtype=c["r"], scale=2.0),
             gate=normal(gr, D, dtype=c["gate"]) if gr else None, w_post=uniform(0.5, 1.5, D), w_pre=uniform(0.5, 1.5, D),
             r_out=empty(M, D, dtype=c["r"]), x=empty(M, D, dtype=c["x"]))
    if c["op"] == "norm_backward":
        s.update(dr_out=normal(M, D), dx=normal(M, D), dy=empty(M, D), dr=empty(M, D),
                 dgate=empty(gr, D) if gr else None, dw_post=empty(D), dw_pre=empty(D))
    return s


# ----------------------------------------------------------------------------- the plain forms
def _live(lengths, T):
    """[B, T] truth values: the token lies inside its sequence (None: all do)."""
    return None if lengths is None else torch.arange(T, device=lengths.device)[None] < lengths[:, None]


def _silu_slope(v):
    q = torch.sigmoid(v)
    return q * (1 + v * (1 - q))


def _conv_windows(s):
    """The inputs behind the state, float32 [B, K-1+T, C], and the K of them that each token sees."""
    c, x = s["case"], s["x"].float()
    live = _live(s["lengths"], c["T"])
    if live is not None:
        x = torch.where(live[..., None], x, x.new_zeros(()))
    past = s["s_in"].float() if s["s_in"] is not None else x.new_zeros(c["B"], c["K"] - 1, c["C"])
    xp = torch.cat([past, x], 1)
    return xp, xp.unfold(1, c["K"], 1), live


def _conv_last(s, xp):
    c = s["case"]
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), c["T"], device=xp.device)
    return n[:, None] + torch.arange(c["K"] - 1, device=xp.device)


def _plain_conv(s):
    c = s["case"]
    xp, win, live = _conv_windows(s)
    pre = (win * s["w"]).sum(-1)
    if s["b"] is not None:
        pre = pre + s["b"]
    y = pre * torch.sigmoid(pre) if c["act"] == "silu" else pre
    if live is not None:
        y = torch.where(live[..., None], y, y.new_zeros(()))
    last = xp.gather(1, _conv_last(s, xp)[..., None].expand(-1, -1, c["C"])).to(_DTYPES[c["dtype"]])
    y = y.to(_DTYPES[c["dtype"]])
    if c["op"] == "conv_step":
        s["s_in"].copy_(last)
        return {"y": y, "state": s["s_in"]}
    return {"y": y, "state": last}


def _plain_conv_backward(s):
    c = s["case"]
    K = c["K"]
    xp, win, live = _conv_windows(s)
    pre = (win * s["w"]).sum(-1)
    if s["b"] is not None:
        pre = pre + s["b"]
    g = s["dy"] * _silu_slope(pre) if c["act"] == "silu" else s["dy"]
    if live is not None:
        g = torch.where(live[..., None], g, g.new_zeros(()))
    around = torch.nn.functional.pad(g, (0, 0, K - 1, K - 1)).unfold(1, K, 1)
    dxp = (around * s["w"].flip(1)).sum(-1)
    if s["ds_out"] is not None:
        dxp = dxp.scatter_add(1, _conv_last(s, xp)[..., None].expand(-1, -1, c["C"]), s["ds_out"])
    out = {"dx": dxp[:, K - 1:], "dw": (win * g[..., None]).sum((0, 1))}
    if s["b"] is not None:
        out["db"] = g.sum((0, 1))
    if s["ds_in"] is not None:
        out["ds_in"] = dxp[:, :K - 1]
    return out


def _parts(s, x):
    """x [B,H,T,d_v], B and C [B,H,T,d_k] of a packed [B, T, H d_v + 2 G d_k] tensor, in float32."""
    c = s["case"]
    H, G, N, P = c["H"], c["G"], c["d_k"], c["d_v"]
    b, t = x.shape[:2]
    x = x.float()
    u, bm, cm = x.split([H * P, G * N, G * N], -1)
    bm, cm = (v.reshape(b, t, G, N).repeat_interleave(H // G, 2).transpose(1, 2) for v in (bm, cm))
    return u.reshape(b, t, H, P).transpose(1, 2), bm, cm


def _steps(s):
    """Time step and log-decay of every token, [B,H,T]: zero behind the end of a sequence."""
    raw = s["dt"].float().transpose(1, 2) + s["dt_bias"][:, None]
    dtv = torch.where(raw > 20, raw, torch.log1p(torch.exp(torch.clamp(raw, max=20.0))))
    live = _live(s["lengths"], s["case"]["T"])
    if live is not None:
        dtv = torch.where(live[:, None], dtv, dtv.new_zeros(()))
    return raw, dtv, -torch.exp(s["A_log"])[:, None].double() * dtv.double()


def _blocks(t, Q):
    """[B,H,T,...] -> [B,H,blocks,Q,...], zeros behind the end."""
    pad = -t.shape[2] % Q
    if pad:
        t = torch.cat([t, t.new_zeros(*t.shape[:2], pad, *t.shape[3:])], 2)
    return t.reshape(*t.shape[:2], -1, Q, *t.shape[3:])


def _carried(total, local, first):
    """States before every block, and after the last: the earlier blocks' own contributions `local`
    [B,H,n,P,N] and the `first` state, decayed by the blocks between (log-decays `total` [B,H,n])."""
    b, h, n, p, k = local.shape
    upto = torch.cat([total.new_zeros(b, h, 1), total.cumsum(-1)], -1)  # [B,H,n+1]
    gap = upto[..., :, None] - upto[..., None, 1:]                       # before block i, after block j
    seen = torch.ones(n + 1, n, device=local.device, dtype=torch.bool).tril(-1)
    m = torch.exp(torch.where(seen, gap, gap.new_full((), -math.inf))).float()
    got = torch.matmul(m, local.reshape(b, h, n, p * k)).reshape(b, h, n + 1, p, k)
    if first is not None:
        got = got + torch.exp(upto).float()[..., None, None] * first[:, :, None]
    return got


def _plain_scan(s):
    c = s["case"]
    T, Q = c["T"], min(_CHUNK, c["T"])
    x, bm, cm = _parts(s, s["xbc"])
    live = _live(s["lengths"], T)
    if live is not None:
        x, bm, cm = (torch.where(live[:, None, :, None], v, v.new_zeros(())) for v in (x, bm, cm))
    _, dtv, la = _steps(s)
    xc, bc, cc, dc = (_blocks(v, Q) for v in (x, bm, cm, dtv))
    L = _blocks(la, Q).cumsum(-1)
    tri = torch.ones(Q, Q, device=x.device, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(tri, L[..., :, None] - L[..., None, :], L.new_full((), -math.inf))).float()
    total = L[..., -1]
    left = (torch.exp(total[..., None] - L).float() * dc)[..., None]
    states = _carried(total, torch.matmul((xc * left).transpose(-1, -2), bc), s["s_in"])
    o = torch.matmul(torch.matmul(cc, bc.transpose(-1, -2)) * decay * dc[..., None, :], xc)
    o = o + torch.exp(L).float()[..., None] * torch.matmul(cc, states[:, :, :-1].transpose(-1, -2))
    o = o.reshape(*x.shape[:2], -1, c["d_v"])[:, :, :T] + s["D"][:, None, None] * x
    return {"o": o, "state": states[:, :, -1]}


def _plain_scan_step(s):
    c = s["case"]
    x, bm, cm = (v[:, :, 0] for v in _parts(s, s["xbc"]))
    _, dtv, la = _steps(s)
    S = torch.exp(la).float()[..., None] * s["s_in"] + (dtv * x)[..., None] * bm[:, :, None]
    o = (S * cm[:, :, None]).sum(-1) + s["D"][:, None] * x
    s["s_in"].copy_(S)
    return {"o": o[:, :, None], "state": s["s_in"]}


def _plain_scan_backward(s):
    c = s["case"]
    B, T, H, G, N, P = c["B"], c["T"], c["H"], c["G"], c["d_k"], c["d_v"]
    Q = min(_CHUNK, T)
    x, bm, cm = _parts(s, s["xbc"])
    go = s["go"]
    live = _live(s["lengths"], T)
    if live is not None:
        x, bm, cm, go = (torch.where(live[:, None, :, None], v, v.new_zeros(())) for v in (x, bm, cm, go))
    raw, dtv, la = _steps(s)
    xc, bc, cc, gc, dc = (_blocks(v, Q) for v in (x, bm, cm, go, dtv))
    L = _blocks(la, Q).cumsum(-1)
    total = L[..., -1]
    tri = torch.ones(Q, Q, device=x.device, dtype=torch.bool).tril()
    decay = torch.exp(torch.where(tri, L[..., :, None] - L[..., None, :], L.new_full((), -math.inf))).float()
    since, left = torch.exp(L).float()[..., None], torch.exp(total[..., None] - L).float()[..., None]
    states = _carried(total, torch.matmul((xc * left * dc[..., None]).transpose(-1, -2), bc), s["s_in"])
    back = _carried(total.flip(2), torch.matmul((gc * since).transpose(-1, -2), cc).flip(2), s["ds_out"]).flip(2)
    ends = back[:, :, 1:]  # gradient of the state after each block
    plain, pair = torch.matmul(cc, bc.transpose(-1, -2)), torch.matmul(gc, xc.transpose(-1, -2)) * decay
    score = plain * decay
    dx = torch.matmul(score.transpose(-1, -2), gc) + left * torch.matmul(bc, ends.transpose(-1, -2))
    db = torch.matmul(pair.transpose(-1, -2), cc) + left * torch.matmul(xc, ends)
    dcm = torch.matmul(pair * dc[..., None, :], bc) + since * torch.matmul(gc, states[:, :, :-1])
    q = (db * bc).sum(-1)  # gradient of the time step through the written outer product
    # log-decay of token t: what tokens before t (or the block's first state) give to tokens from t on
    # (or to the state after the block); pairs of one side cancel exactly in the float64 sums
    both = (plain * pair * dc[..., None, :]).tril(-1).double()
    read = since[..., 0] * (torch.matmul(gc, states[:, :, :-1]) * cc).sum(-1)
    put = left[..., 0] * dc * (torch.matmul(xc, ends) * bc).sum(-1)
    ahead = (both.sum(-1) - both.sum(-2) + read).flip(-1).cumsum(-1).flip(-1)
    behind = put.double().cumsum(-1) - put
    dla = ahead + behind + (torch.exp(total) * (ends * states[:, :, :-1]).double().sum((-1, -2)))[..., None]
    flat = lambda v: v.reshape(B, H, -1, *v.shape[4:])[:, :, :T]  # noqa: E731
    dx = flat(dx * dc[..., None]) + s["D"][:, None, None] * go
    heads = lambda v: flat(v).reshape(B, G, H // G, T, N).sum(2).permute(0, 2, 1, 3).reshape(B, T, G * N)  # noqa: E731
    dla, q = flat(dla), flat(q)
    rate = -torch.exp(s["A_log"].double())[:, None]
    ddt = (q.double() + dla * rate) * torch.sigmoid(raw.double())
    if live is not None:
        dla = torch.where(live[:, None], dla, dla.new_zeros(()))
        ddt = torch.where(live[:, None], ddt, ddt.new_zeros(()))
    out = {"dxbc": torch.cat([dx.transpose(1, 2).reshape(B, T, H * P), heads(db * dc[..., None]), heads(dcm)], -1),
           "ddt": ddt.transpose(1, 2).float(), "ddt_bias": ddt.sum((0, 2)).float(),
           "dA_log": (dla * rate * dtv.double()).sum((0, 2)).float(),
           "dD": (go * x).double().sum((0, 2, 3)).float()}
    if s["ds_in"] is not None:
        out["ds_in"] = back[:, :, 0]
    return out


def _gate(c, v):
    """Value and slope of the gate's activation."""
    if c["act"] == "none":
        return v, torch.ones_like(v)
    q = torch.sigmoid(v)
    return (q, q * (1 - q)) if c["act"] == "sigmoid" else (v * q, _silu_slope(v))


def _spread(c, g):
    """A gate of gate_rows rows, over the M rows."""
    return g.repeat_interleave(c["M"] // c["gate_rows"], 0)


def _plain_norm(s):
    c = s["case"]
    y, r = s["y"].float(), s["r"].float()
    u = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * s["w_post"]
    if s["gate"] is not None:
        u = u * _spread(c, _gate(c, s["gate"].float())[0])
    r = r + c["scale"] * u
    x = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS) * s["w_pre"]
    return {"r_out": r.to(_DTYPES[c["r"]]), "x": x.to(_DTYPES[c["x"]])}


def _plain_norm_backward(s):
    c = s["case"]
    y, r = s["y"].float(), s["r"].float()
    ry = torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS)
    yn = y * ry
    u = yn * s["w_post"]
    a = 1.0
    if s["gate"] is not None:
        a, slope = (_spread(c, v) for v in _gate(c, s["gate"].float()))
    r = r + c["scale"] * a * u
    rr = torch.rsqrt(r.square().mean(-1, keepdim=True) + _EPS)
    h = r * rr
    t = s["dx"] * s["w_pre"]
    dr = s["dr_out"] + rr * (t - h * (t * h).mean(-1, keepdim=True))
    du = c["scale"] * a * dr
    t = du * s["w_post"]
    out = {"dy": ry * (t - yn * (t * yn).mean(-1, keepdim=True)), "dr": dr, "dw_post": (du * yn).sum(0),
           "dw_pre": (s["dx"] * h).sum(0)}
    if s["gate"] is not None:
        out["dgate"] = (c["scale"] * dr * u * slope).reshape(c["gate_rows"], -1, c["D"]).sum(1)
    return out


# -------------------------------------------------------------------------- the library's calls
def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(max(1, size), dtype=torch.uint8, device=_DEVICE)
    return s["ws"]


def _own(s):
    import sparse_memory_linear_amd as S
    c = s["case"]
    op = c["op"]
    if op.startswith("conv"):
        if "shape" not in s:
            s["shape"] = S.make_conv_shape(c["B"], c["T"], c["C"], c["K"], c["dtype"], c["act"], ld_x=c["C"] + c["gap"])
        sh = s["shape"]
        if op == "conv":
            S.short_conv(sh, s["x"], s["w"], s["y"], bias=s["b"], lengths=s["lengths"], s_in=s["s_in"], s_out=s["s_out"])
            return {"y": s["y"], "state": s["s_out"]}
        if op == "conv_step":
            S.short_conv_step(sh, s["x"], s["w"], s["s_in"], s["y"], bias=s["b"])
            return {"y": s["y"], "state": s["s_in"]}
        S.short_conv_backward(sh, s["x"], s["w"], s["dy"], s["dx"], s["dw"],
                              _workspace(s, S.short_conv_backward_workspace_bytes(sh)), bias=s["b"], dbias=s["db"],
                              lengths=s["lengths"], s_in=s["s_in"], ds_out=s["ds_out"], ds_in=s["ds_in"])
        return {k: s[k] for k in ("dx", "dw", "db", "ds_in") if s[k] is not None}
    if op.startswith("scan"):
        B, T, H, G, N, P = c["B"], c["T"], c["H"], c["G"], c["d_k"], c["d_v"]
        if "shape" not in s:
            ld = H * P + 2 * G * N
            s["shape"] = S.make_scan_shape(B, T, H, G, N, P, c["dtype"], ld_x=ld, ld_b=ld, ld_c=ld)
            s["parts"] = s["xbc"].split([H * P, G * N, G * N], -1)
        sh = s["shape"]
        x, bm, cm = s["parts"]
        if op == "scan":
            S.selective_scan(sh, x, bm, cm, s["dt"], s["A_log"], s["dt_bias"], s["o"],
                             _workspace(s, S.selective_scan_workspace_bytes(sh)), D=s["D"], lengths=s["lengths"],
                             s_in=s["s_in"], s_out=s["s_out"])
            return {"o": s["o"], "state": s["s_out"]}
        if op == "scan_step":
            S.selective_scan_step(sh, x, bm, cm, s["dt"], s["A_log"], s["dt_bias"], s["s_in"], s["o"], D=s["D"])
            return {"o": s["o"], "state": s["s_in"]}
        if "dparts" not in s:
            s["dparts"] = s["dxbc"].split([H * P, G * N, G * N], -1)
        S.selective_scan_backward(sh, x, bm, cm, s["dt"], s["A_log"], s["dt_bias"], s["go"], *s["dparts"], s["ddt"],
                                  s["dA_log"], s["ddt_bias"],
                                  _workspace(s, S.selective_scan_backward_workspace_bytes(sh)), D=s["D"], dD=s["dD"],
                                  lengths=s["lengths"], s_in=s["s_in"], ds_out=s["ds_out"], ds_in=s["ds_in"])
        return {k: s[k] for k in ("dxbc", "ddt", "ddt_bias", "dA_log", "dD", "ds_in") if s[k] is not None}
    if "shape" not in s:
        s["shape"] = S.make_norm_shape(c["M"], c["D"], y_dtype=c["y"], r_dtype=c["r"], x_dtype=c["x"],
                                       gate_dtype=c["gate"], gate_rows=c["gate_rows"], gate_act=c["act"], eps=_EPS,
                                       scale=c["scale"])
    sh = s["shape"]
    if op == "norm":
        S.block_norm(sh, s["y"], s["r"], s["r_out"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], x=s["x"])
        return {"r_out": s["r_out"], "x": s["x"]}
    S.block_norm_backward(sh, s["y"], s["r"], s["dy"], s["dr"], _workspace(s, S.block_norm_backward_workspace_bytes(sh)),
                          gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], dr_out=s["dr_out"], dx=s["dx"],
                          dgate=s["dgate"], dw_post=s["dw_post"], dw_pre=s["dw_pre"])
    return {k: s[k] for k in ("dy", "dr", "dw_post", "dw_pre", "dgate") if s[k] is not None}


_PLAIN = {"conv": _plain_conv, "conv_step": _plain_conv, "conv_backward": _plain_conv_backward, "scan": _plain_scan,
          "scan_step": _plain_scan_step, "scan_backward": _plain_scan_backward, "norm": _plain_norm,
          "norm_backward": _plain_norm_backward}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------ work of one pass
def work(case):
    c = case
    size = lambda dt: 4 if dt == "f32" else 2  # noqa: E731
    if c["op"].startswith("conv"):
        e, n = size(c["dtype"]), c["B"] * c["T"] * c["C"]
        held = c["B"] * (c["K"] - 1) * c["C"] * e
        past = held if c["state"] or c["op"] == "conv_step" else 0
        if c["op"] == "conv_backward":
            return {"bytes": n * (e + 8) + c["C"] * (c["K"] * 8 + 8) + past + (2 * held * 4 // e if c["state"] else 0),
                    "flops": n * (6 * c["K"] + 10)}
        return {"bytes": 2 * n * e + c["C"] * (c["K"] + 1) * 4 + past + held, "flops": n * (2 * c["K"] + 5)}
    if c["op"].startswith("scan"):
        e, tok, H = size(c["dtype"]), c["B"] * c["T"], c["H"]
        held = c["B"] * H * c["d_k"] * c["d_v"] * 4
        past = held if c["state"] or c["op"] == "scan_step" else 0
        into = tok * ((H * c["d_v"] + 2 * c["G"] * c["d_k"]) * e + H * 4)
        outer = tok * H * c["d_k"] * c["d_v"]
        if c["op"] == "scan_backward":
            return {"bytes": into + tok * (H * c["d_v"] * 8 + 8 * c["G"] * c["d_k"] + H * 4)
                    + (3 * held if c["state"] else 0), "flops": 14 * outer}
        return {"bytes": into + tok * H * c["d_v"] * 4 + past + held, "flops": 5 * outer}
    n = c["M"] * c["D"]
    gate = c["gate_rows"] * c["D"]
    into = n * (size(c["y"]) + size(c["r"])) + gate * size(c["gate"]) + 8 * c["D"]
    if c["op"] == "norm_backward":
        return {"bytes": into + 16 * n + 4 * gate + 8 * c["D"], "flops": 40 * n}
    return {"bytes": into + n * (size(c["r"]) + size(c["x"])), "flops": 12 * n}


# ---------------------------------------------------------------------------- values in 64 bits
def _exact_conv(s):
    c = s["case"]
    B, T, C, K = c["B"], c["T"], c["C"], c["K"]
    ext = torch.zeros(B, K - 1 + T, C, dtype=torch.float64, device=_DEVICE)
    if s["s_in"] is not None:
        ext[:, :K - 1] = s["s_in"]
    ext[:, K - 1:] = s["x"]
    ends = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    for b, n in enumerate(ends):
        ext[b, K - 1 + n:] = 0
    w = s["w"].double()
    z = torch.zeros(B, T, C, dtype=torch.float64, device=_DEVICE)
    if s["b"] is not None:
        z += s["b"]
    for j in range(K):
        z += ext[:, j:j + T] * w[:, j]
    sig = 1 / (1 + torch.exp(-z))
    last = torch.stack([ext[b, n:n + K - 1] for b, n in enumerate(ends)])
    if c["op"] != "conv_backward":
        y = z * sig if c["act"] == "silu" else z
        for b, n in enumerate(ends):
            y[b, n:] = 0
        return {"y": y, "state": last}
    dz = s["dy"].double()
    if c["act"] == "silu":
        dz = dz * (sig + z * sig * (1 - sig))
    for b, n in enumerate(ends):
        dz[b, n:] = 0
    dext, dw = torch.zeros_like(ext), torch.zeros_like(w)
    for j in range(K):
        dext[:, j:j + T] += dz * w[:, j]
        dw[:, j] = (dz * ext[:, j:j + T]).sum((0, 1))
    if s["ds_out"] is not None:
        for b, n in enumerate(ends):
            dext[b, n:n + K - 1] += s["ds_out"][b]
    out = {"dx": dext[:, K - 1:], "dw": dw}
    if s["b"] is not None:
        out["db"] = dz.sum((0, 1))
    if s["ds_in"] is not None:
        out["ds_in"] = dext[:, :K - 1]
    return out


def _exact_scan(s):
    c = s["case"]
    B, T, H, G, N, P = c["B"], c["T"], c["H"], c["G"], c["d_k"], c["d_v"]
    v = s["xbc"].double().transpose(0, 1).contiguous()  # token first
    x = v[..., :H * P].reshape(T, B, H, P)
    of = torch.arange(H, device=_DEVICE) // (H // G)
    bm = v[..., H * P:H * P + G * N].reshape(T, B, G, N)
    cm = v[..., H * P + G * N:].reshape(T, B, G, N)
    raw = s["dt"].double().transpose(0, 1) + s["dt_bias"].double()
    dtv = torch.logaddexp(raw, torch.zeros_like(raw))
    inside = torch.ones(T, B, dtype=torch.bool, device=_DEVICE)
    if s["lengths"] is not None:
        inside = torch.arange(T, device=_DEVICE)[:, None] < s["lengths"][None]
    dtv = dtv * inside[..., None]
    rate = -torch.exp(s["A_log"].double())
    a = torch.exp(rate * dtv)[..., None, None]
    D = s["D"].double()
    S = torch.zeros(B, H, P, N, dtype=torch.float64, device=_DEVICE)
    if s["s_in"] is not None:
        S += s["s_in"]
    if c["op"] != "scan_backward":
        o = torch.empty(T, B, H, P, dtype=torch.float64, device=_DEVICE)
        put = (dtv[..., None] * x)[..., None]
        bh, ch = bm[:, :, of, None], cm[:, :, of, :, None]
        for t in range(T):
            S = torch.addcmul(a[t] * S, put[t], bh[t])
            torch.matmul(S, ch[t], out=o[t].unsqueeze(-1))
        o = (o + D[:, None] * x) * inside[..., None, None]
        return {"o": o.permute(1, 2, 0, 3), "state": S}
    go = s["go"].double().permute(2, 0, 1, 3) * inside[..., None, None]
    kept = [S]
    for t in range(T):
        kept.append(a[t] * kept[-1] + (dtv[t][..., None] * x[t])[..., None] * bm[t][:, of][:, :, None])
    U = torch.zeros_like(S)
    if s["ds_out"] is not None:
        U += s["ds_out"]
    dx, dbm, dcm = torch.empty_like(x), torch.zeros_like(bm), torch.zeros_like(cm)
    dla, dwrite = torch.empty_like(dtv), torch.empty_like(dtv)
    for t in reversed(range(T)):
        U = U + go[t][..., None] * cm[t][:, of][:, :, None]
        dcm[t].index_add_(1, of, (kept[t + 1] * go[t][..., None]).sum(2))
        ub = (U * bm[t][:, of][:, :, None]).sum(-1)
        dx[t] = dtv[t][..., None] * ub
        dbm[t].index_add_(1, of, dtv[t][..., None] * (U * x[t][..., None]).sum(2))
        dwrite[t] = (ub * x[t]).sum(-1)
        dla[t] = (a[t] * U * kept[t]).sum((-1, -2))
        U = a[t] * U
    dx += D[:, None] * go
    dla = dla * inside[..., None]
    ddt = (dwrite + dla * rate) * torch.sigmoid(raw) * inside[..., None]
    row = lambda t, n: t.transpose(0, 1).reshape(B, T, n)  # noqa: E731
    out = {"dxbc": torch.cat([row(dx, H * P), row(dbm, G * N), row(dcm, G * N)], -1), "ddt": ddt.transpose(0, 1),
           "ddt_bias": ddt.sum((0, 1)), "dA_log": (dla * rate * dtv).sum((0, 1)), "dD": (go * x).sum((0, 1, 3))}
    if s["ds_in"] is not None:
        out["ds_in"] = U
    return out


def _exact_norm(s):
    c = s["case"]
    M, D, k = c["M"], c["D"], c["scale"]
    y, r, wp, wn = s["y"].double(), s["r"].double(), s["w_post"].double(), s["w_pre"].double()
    ny = torch.sqrt((y * y).sum(1, keepdim=True) / D + _EPS)
    if s["gate"] is None:
        a, slope = torch.ones(1, 1, D, dtype=torch.float64, device=_DEVICE), None
    else:
        g = s["gate"].double()[:, None]
        sig = 1 / (1 + torch.exp(-g))
        a = {"none": g, "sigmoid": sig, "silu": g * sig}[c["act"]]
        slope = {"none": torch.ones_like(g), "sigmoid": sig - sig * sig, "silu": sig + g * (sig - sig * sig)}[c["act"]]
    grouped = lambda v: v.reshape(a.shape[0], -1, D)  # noqa: E731
    r = r + k * (a * grouped(y / ny * wp)).reshape(M, D)
    nr = torch.sqrt((r * r).sum(1, keepdim=True) / D + _EPS)
    if c["op"] == "norm":
        return {"r_out": r, "x": r / nr * wn}
    gx = s["dx"].double()
    gr = s["dr_out"].double() + gx * wn / nr - r * (gx * wn * r).sum(1, keepdim=True) / (D * nr ** 3)
    gu = k * (a * grouped(gr)).reshape(M, D)
    out = {"dy": gu * wp / ny - y * (gu * wp * y).sum(1, keepdim=True) / (D * ny ** 3), "dr": gr,
           "dw_post": (gu * y / ny).sum(0), "dw_pre": (gx * r / nr).sum(0)}
    if s["gate"] is not None:
        out["dgate"] = (k * grouped(gr * y / ny * wp)).sum(1) * slope[:, 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_conv if case["op"].startswith("conv") else _exact_scan if case["op"].startswith("scan") else
            _exact_norm)(s)
