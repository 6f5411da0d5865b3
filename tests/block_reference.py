"""Float64 references of the short convolution, the selective scan and the block norm, token by
token and row by row, with their gradients by torch's autograd, and the sums of absolute terms that
float32 error bounds are stated against.

A float32 sum of n terms is off by at most about n 2^-24 times the sum of the terms' absolute
values. Running a multilinear operator on the absolute values of its inputs gives that sum, for the
outputs and for the gradients alike.
"""
import torch

EPS32 = 2.0 ** -24  # half a step of float32, relative
EPS16 = 2.0 ** -8   # half a step of bfloat16


def f64(t):
    return None if t is None else t.detach().double()


def absolute(t):
    return None if t is None else t.abs()


def silu(v):
    return v * torch.sigmoid(v)


# --------------------------------------------------------------------------------- convolution
def conv(x, w, bias, s_in, lengths, act):
    """x [B,T,C], w [C,K], s_in [B,K-1,C] -> y [B,T,C], state [B,K-1,C]."""
    B, T, C = x.shape
    K = w.shape[1]
    ys, states = [], []
    for b in range(B):
        n = T if lengths is None else max(0, min(T, int(lengths[b])))
        past = s_in[b] if s_in is not None else x.new_zeros(K - 1, C)
        seq = torch.cat([past, x[b, :n]], 0)
        z = x.new_zeros(n, C) + (bias if bias is not None else 0.0)
        for j in range(K):
            z = z + seq[j:j + n] * w[:, j]
        y = silu(z) if act == "silu" else z
        ys.append(torch.cat([y, x.new_zeros(T - n, C)], 0))
        states.append(seq[n:n + K - 1])
    return torch.stack(ys), torch.stack(states)


# ------------------------------------------------------------------------------- selective scan
def scan_gates(dt, A_log, dt_bias, lengths):
    """Time step and log-decay [B,T,H] of every token (0 behind the end of a sequence)."""
    raw = dt + dt_bias
    dtv = torch.logaddexp(raw, torch.zeros_like(raw))
    la = -torch.exp(A_log) * dtv
    if lengths is not None:
        live = (torch.arange(dt.shape[1], device=dt.device)[None] < lengths.clamp(0, dt.shape[1])[:, None])[..., None]
        dtv, la = dtv * live, la * live
    return raw, dtv, la


def scan(x, Bm, Cm, dtv, la, D, s_in, lengths):
    """x [B,T,H,P], Bm, Cm [B,T,G,N], dtv, la [B,T,H] -> o [B,H,T,P], state [B,H,P,N]."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    of = torch.arange(H, device=x.device) // (H // G)
    live = torch.ones(B, T, dtype=torch.bool, device=x.device)
    if lengths is not None:
        live = torch.arange(T, device=x.device)[None] < lengths.clamp(0, T)[:, None]
    zero = x.new_zeros(())
    x, Bm, Cm = (torch.where(live[..., None, None], v, zero) for v in (x, Bm, Cm))
    S = s_in if s_in is not None else x.new_zeros(B, H, P, N)
    out = []
    for t in range(T):
        S = torch.exp(la[:, t])[..., None, None] * S + (dtv[:, t][..., None] * x[:, t])[..., None] * Bm[:, t, of][:, :, None]
        o = (S * Cm[:, t, of][:, :, None]).sum(-1)
        if D is not None:
            o = o + D[:, None] * x[:, t]
        out.append(torch.where(live[:, t, None, None], o, zero))
    o = torch.stack(out, 2) if T else x.new_zeros(B, H, 0, P)
    return o, S


def scan_gradients(x, Bm, Cm, dt, A_log, dt_bias, D, s_in, lengths, go, ds_out):
    """Every gradient of <go, o> + <ds_out, s_out>, and the sums of absolute terms of each."""
    raw, dtv, la = scan_gates(dt, A_log, dt_bias, lengths)
    rate = -torch.exp(A_log)
    results = []
    for take in (lambda t: t, absolute):
        leaf = {k: None if v is None else take(v).clone().requires_grad_(True)
                for k, v in dict(x=x, Bm=Bm, Cm=Cm, dtv=dtv, D=D, s_in=s_in).items()}
        decay = la.clone().requires_grad_(True)
        o, S = scan(leaf["x"], leaf["Bm"], leaf["Cm"], leaf["dtv"], decay, leaf["D"], leaf["s_in"], lengths)
        loss = (take(go) * o).sum()
        if ds_out is not None:
            loss = loss + (take(ds_out) * S).sum()
        # a graph that does not reach a leaf gives no gradient: zeros
        given = [v for v in list(leaf.values()) + [decay] if v is not None]
        grads = torch.autograd.grad(loss, given, allow_unused=True) if loss.requires_grad else [None] * len(given)
        got = {id(v): torch.zeros_like(v) if g is None else g for v, g in zip(given, grads)}
        g = {k: None if v is None else got[id(v)] for k, v in leaf.items()}
        dl, sign = got[id(decay)], (rate if take is not absolute else rate.abs())
        slope = torch.sigmoid(raw)
        if lengths is not None:
            slope = slope * (torch.arange(dt.shape[1], device=dt.device)[None] < lengths.clamp(0, dt.shape[1])[:, None])[..., None]
        ddt = (g["dtv"] + sign * dl) * slope
        results.append(dict(dx=g["x"], dBm=g["Bm"], dCm=g["Cm"], ddt=ddt, ddt_bias=ddt.sum((0, 1)),
                            dA_log=(dl * sign * dtv).sum((0, 1)), dD=g["D"], ds_in=g["s_in"]))
    return results


# ----------------------------------------------------------------------------------- block norm
def act_of(name, g):
    return {"none": lambda v: v, "sigmoid": torch.sigmoid, "silu": silu}[name](g)


def norm(y, r, gate, w_post, w_pre, act, eps, scale):
    """-> r_out, x (None without w_pre)."""
    u = y
    if w_post is not None:
        u = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        u = u * act_of(act, gate).repeat_interleave(y.shape[0] // gate.shape[0], 0)
    r = r + scale * u
    if w_pre is None:
        return r, None
    return r, r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps) * w_pre
