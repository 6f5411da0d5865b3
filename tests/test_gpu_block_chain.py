"""A layer of the convolution, the scan, the library's output projection and the block norm, run
together as a program runs them: prompts and then single tokens against the whole sequence at once, the
captured token step, the gradient through the three operators, and calls on several streams."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

B, H, G, N, P, K, DM, TP = 2, 4, 2, 32, 64, 4, 136, 77
C = H * P + 2 * G * N


@pytest.fixture(scope="module")
def sdm():
    import sparse_memory_linear_amd as S
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    S.lib()
    return S


class Layer:
    def __init__(self, sdm, seed=0):
        self.S = sdm
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.w, self.b = rnd(C, K) * 0.5, rnd(C) * 0.1
        self.A_log, self.dt_bias, self.D = torch.log(torch.rand(H, generator=g, device="cuda") * 15 + 1), rnd(H) - 3, rnd(H)
        self.wn = torch.rand(P, generator=g, device="cuda") + 0.5
        self.Wo = (rnd(DM, H * P) * (H * P) ** -0.5).bfloat16()
        self.w_post, self.w_pre = torch.rand(DM, generator=g, device="cuda") + 0.5, torch.rand(DM, generator=g, device="cuda") + 0.5
        self.gate = rnd(1, DM)

    def shapes(self, T):
        S = self.S
        return (S.make_conv_shape(B, T, C, K, "bf16", "silu"),
                S.make_scan_shape(B, T, H, G, N, P, "bf16", ld_x=C, ld_b=C, ld_c=C),
                S.make_shape(B, H, T, 16, 16, P, 2, 2, 2, "bf16", "f32"),
                S.make_norm_shape(B * T, DM, "f32", "f32", "bf16", "f32", 1, "silu"))

    def buffers(self, T):
        e = lambda *s, dtype=torch.float32: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
        sh = self.shapes(T)
        return dict(y=e(B, T, C, dtype=torch.bfloat16), o=e(B, H, T, P), m=e(B * T, DM), r_out=e(B * T, DM),
                    x=e(B * T, DM, dtype=torch.bfloat16),
                    ws=torch.empty(self.S.selective_scan_workspace_bytes(sh[1]), dtype=torch.uint8, device="cuda"))

    def run(self, xbc, dt, z, r, conv_state, state, f, stream=None):
        """The layer on T tokens: r_out and the next layer's x; both states go on in place."""
        S, T = self.S, xbc.shape[1]
        cs, ss, hs, ns = self.shapes(T)
        if T == 1:
            S.short_conv_step(cs, xbc, self.w, conv_state, f["y"], bias=self.b, stream=stream)
        else:
            S.short_conv(cs, xbc, self.w, f["y"], bias=self.b, s_in=conv_state, s_out=conv_state, stream=stream)
        x, bm, cm = f["y"].split([H * P, G * N, G * N], -1)
        if T == 1:
            S.selective_scan_step(ss, x, bm, cm, dt, self.A_log, self.dt_bias, state, f["o"], D=self.D, stream=stream)
        else:
            S.selective_scan(ss, x, bm, cm, dt, self.A_log, self.dt_bias, f["o"], f["ws"], D=self.D, s_in=state, s_out=state,
                             stream=stream)
        S.output_project(hs, f["o"], z, self.wn, 1e-5, self.Wo, DM, f["m"], stream=stream)
        S.block_norm(ns, f["m"], r, f["r_out"], gate=self.gate, w_post=self.w_post, w_pre=self.w_pre, x=f["x"], stream=stream)
        return f["r_out"].view(B, T, DM), f["x"].view(B, T, DM)

    def states(self):
        return torch.zeros(B, K - 1, C, device="cuda", dtype=torch.bfloat16), torch.zeros(B, H, P, N, device="cuda")


def inputs(T, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return rnd(B, T, C).bfloat16(), rnd(B, T, H), rnd(B, T, H, P).bfloat16(), rnd(B, T, DM)


def part(t, a, b):
    return t[:, a:b].contiguous()


def close(a, b, steps):
    """Two orders of the same float32 sums, one rounding of x and o's bf16 operand in between: a value of
    the projection's operand that falls on the other side of a bf16 step moves the sums by 2^-8 of one of
    its 256 terms; so the two differ by a few such steps of the terms' size, not of the sum's."""
    d = (a.float() - b.float()).abs()
    return (d <= steps * R.EPS16 * (b.float().abs() + b.float().square().mean().sqrt())).all()


def test_prompt_and_tokens_equal_the_whole(sdm):
    L = Layer(sdm)
    xbc, dt, z, r = inputs(TP)
    cs, st = L.states()
    ra, xa = L.run(xbc, dt, z, r.view(B * TP, DM), cs, st, L.buffers(TP))
    cs2, st2 = L.states()
    n = 70
    rb, xb = L.run(part(xbc, 0, n), part(dt, 0, n), part(z, 0, n), part(r, 0, n).view(-1, DM), cs2, st2, L.buffers(n))
    assert close(rb, ra[:, :n], 1) and close(xb, xa[:, :n], 2)
    f = L.buffers(1)
    for t in range(n, TP):
        rt, xt = L.run(part(xbc, t, t + 1), part(dt, t, t + 1), part(z, t, t + 1), part(r, t, t + 1).view(-1, DM), cs2, st2, f)
        assert close(rt, ra[:, t:t + 1], 1) and close(xt, xa[:, t:t + 1], 2)
    assert torch.equal(cs, cs2)
    assert ((st - st2).abs() <= 1e-5 * (st.abs() + st.square().mean().sqrt())).all()


@pytest.mark.parametrize("T", [1, 40])
def test_captured_and_replayed(sdm, T):
    """A captured call replays on new inputs and goes on from its states, like the eager calls beside it."""
    L = Layer(sdm)
    feeds = [inputs(T, seed=s) for s in range(5)]
    hold = [t.clone() for t in feeds[0]]
    cs, st = L.states()
    f = L.buffers(T)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        L.run(hold[0], hold[1], hold[2], hold[3].view(B * T, DM), cs.clone(), st.clone(), f)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.run(hold[0], hold[1], hold[2], hold[3].view(B * T, DM), cs, st, f)
    cs.zero_()
    st.zero_()
    ce, se = L.states()
    fe = L.buffers(T)
    for feed in feeds:
        for h, t in zip(hold, feed):
            h.copy_(t)
        graph.replay()
        r, x = L.run(*feed[:3], feed[3].view(B * T, DM), ce, se, fe)
        torch.cuda.synchronize()
        assert torch.equal(f["r_out"], fe["r_out"]) and torch.equal(f["x"], fe["x"])
        assert torch.equal(cs, ce) and torch.equal(st, se)


def test_captured_gradients(sdm):
    """The three gradients captured in one graph, replayed on other inputs, against the eager calls."""
    T, M = 70, 2 * 70
    L = Layer(sdm)
    S = sdm
    cs, ss, _, _ = L.shapes(T)
    ns = S.make_norm_shape(M, DM, "f32", "f32", "f32", "f32", B, "silu")
    e = lambda *s, dtype=torch.float32: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        return dict(xbc=rnd(B, T, C).bfloat16(), y=rnd(B, T, C).bfloat16(), dt=rnd(B, T, H), go=rnd(B, H, T, P), m=rnd(M, DM),
                    r=rnd(M, DM), gate=rnd(B, DM), dr=rnd(M, DM), dx=rnd(M, DM))

    def buffers():
        return dict(dy=e(B, T, C), dxbc=e(B, T, C), dw=e(C, K), db=e(C), ddt=e(B, T, H), dA=e(H), dbias=e(H), dD=e(H), dm=e(M, DM),
                    dres=e(M, DM), dg=e(B, DM), dwp=e(DM), dwn=e(DM),
                    w1=e(S.short_conv_backward_workspace_bytes(cs), dtype=torch.uint8),
                    w2=e(S.selective_scan_backward_workspace_bytes(ss), dtype=torch.uint8),
                    w3=e(S.block_norm_backward_workspace_bytes(ns), dtype=torch.uint8))

    def run(i, o):
        S.block_norm_backward(ns, i["m"], i["r"], o["dm"], o["dres"], o["w3"], gate=i["gate"], w_post=L.w_post, w_pre=L.w_pre,
                              dr_out=i["dr"], dx=i["dx"], dgate=o["dg"], dw_post=o["dwp"], dw_pre=o["dwn"])
        parts = [H * P, G * N, G * N]
        S.selective_scan_backward(ss, *i["y"].split(parts, -1), i["dt"], L.A_log, L.dt_bias, i["go"], *o["dy"].split(parts, -1),
                                  o["ddt"], o["dA"], o["dbias"], o["w2"], D=L.D, dD=o["dD"])
        S.short_conv_backward(cs, i["xbc"], L.w, o["dy"], o["dxbc"], o["dw"], o["w1"], bias=L.b, dbias=o["db"])

    feeds = [make(s) for s in range(4)]
    hold, o, oe = {k: v.clone() for k, v in feeds[0].items()}, buffers(), buffers()
    run(hold, o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(hold, o)
    for feed in feeds:
        for k in hold:
            hold[k].copy_(feed[k])
        graph.replay()
        run(feed, oe)
        torch.cuda.synchronize()
        for k in o:
            assert k.startswith("w") or torch.equal(o[k], oe[k]), k


def test_gradient_through_convolution_and_scan(sdm):
    """The scan's gradients of its packed input, fed to the convolution's gradient, against autograd
    through both in float64. The convolution's bf16 output is what both scans read."""
    T = 66
    L = Layer(sdm, seed=3)
    S = sdm
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    xbc, dt, go = rnd(B, T, C), rnd(B, T, H), rnd(B, H, T, P)
    lengths = torch.tensor([T, 41], dtype=torch.int32, device="cuda")
    cs = S.make_conv_shape(B, T, C, K, "f32", "silu")
    ss = S.make_scan_shape(B, T, H, G, N, P, "f32", ld_x=C, ld_b=C, ld_c=C)
    y, o = torch.empty(B, T, C, device="cuda"), torch.empty(B, H, T, P, device="cuda")
    S.short_conv(cs, xbc, L.w, y, bias=L.b, lengths=lengths)
    parts = [H * P, G * N, G * N]
    ws = torch.empty(S.selective_scan_workspace_bytes(ss), dtype=torch.uint8, device="cuda")
    S.selective_scan(ss, *y.split(parts, -1), dt, L.A_log, L.dt_bias, o, ws, D=L.D, lengths=lengths)
    dy, dx, dw, db = torch.empty_like(y), torch.empty_like(y), torch.empty_like(L.w), torch.empty_like(L.b)
    ddt, dA, dbias, dD = torch.empty_like(dt), torch.empty(H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws2 = torch.empty(S.selective_scan_backward_workspace_bytes(ss), dtype=torch.uint8, device="cuda")
    S.selective_scan_backward(ss, *y.split(parts, -1), dt, L.A_log, L.dt_bias, go, *dy.split(parts, -1), ddt, dA, dbias, ws2, D=L.D,
                              dD=dD, lengths=lengths)
    ws3 = torch.empty(S.short_conv_backward_workspace_bytes(cs), dtype=torch.uint8, device="cuda")
    S.short_conv_backward(cs, xbc, L.w, dy, dx, dw, ws3, bias=L.b, dbias=db, lengths=lengths)
    leaf = {k: v.double().requires_grad_(True) for k, v in dict(x=xbc, w=L.w, b=L.b, dt=dt, A=L.A_log, bias=L.dt_bias, D=L.D).items()}
    ry, _ = R.conv(leaf["x"], leaf["w"], leaf["b"], None, lengths, "silu")
    x, bm, cm = ry.split(parts, -1)
    _, dtv, la = R.scan_gates(leaf["dt"], leaf["A"], leaf["bias"], lengths)
    ro, _ = R.scan(x.reshape(B, T, H, P), bm.reshape(B, T, G, N), cm.reshape(B, T, G, N), dtv, la, leaf["D"], None, lengths)
    grads = dict(zip(leaf, torch.autograd.grad((go.double() * ro).sum(), list(leaf.values()))))
    # float32 throughout: the norms' relative difference is a few times the root of the roundings on the way
    for got, k in ((dx, "x"), (dw, "w"), (db, "b"), (ddt, "dt"), (dA, "A"), (dbias, "bias"), (dD, "D")):
        want = grads[k]
        assert (got.double() - want).norm() <= 64 * R.EPS32 * want.norm(), k
    assert ((o.double() - ro.detach()).norm() <= 32 * R.EPS32 * ro.detach().norm())


def test_streams_of_their_own(sdm):
    """Two layers on two streams at once give what each gives alone."""
    L = [Layer(sdm, seed=s) for s in (1, 2)]
    feeds = [inputs(TP, seed=s) for s in (3, 4)]
    alone, together = [], []
    for l, i in zip(L, feeds):
        cs, st = l.states()
        r, x = l.run(*i[:3], i[3].view(B * TP, DM), cs, st, l.buffers(TP))
        alone.append((r.clone(), x.clone(), st.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in L]
    held = [(l.states(), l.buffers(TP)) for l in L]
    torch.cuda.synchronize()
    for _ in range(3):
        together = []
        for l, i, s, ((cs, st), f) in zip(L, feeds, streams, held):
            with torch.cuda.stream(s):
                cs.zero_()
                st.zero_()
            r, x = l.run(*i[:3], i[3].view(B * TP, DM), cs, st, f, stream=s)
            together.append((r, x, st))
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_refusals_of_the_binding(sdm):
    S = sdm
    cs = S.make_conv_shape(2, 3, 16, 4, "f32")
    x, w, y = torch.zeros(2, 3, 16, device="cuda"), torch.zeros(16, 4, device="cuda"), torch.zeros(2, 3, 16, device="cuda")
    with pytest.raises(ValueError, match="strides"):
        S.short_conv(cs, x.transpose(0, 1), w, y)
    with pytest.raises(ValueError, match="shape"):
        S.short_conv(cs, x, w[:8], y)
    with pytest.raises(ValueError, match="not torch.float32"):
        S.short_conv(cs, x.bfloat16(), w, y)
    with pytest.raises(ValueError, match="not on a GPU"):
        S.short_conv(cs, x, w.cpu(), y)
    with pytest.raises(ValueError, match="int32"):
        S.short_conv(cs, x, w, y, lengths=torch.tensor([1, 2], device="cuda"))
    with pytest.raises(S.SdmError):
        S.short_conv(cs, x, w, x)  # y in the place of x
    ss = S.make_scan_shape(1, 4, 2, 1, 16, 16, "f32")
    v = [torch.zeros(1, 4, n, device="cuda") for n in (32, 16, 16, 2)]
    h, o = torch.zeros(2, device="cuda"), torch.zeros(1, 2, 4, 16, device="cuda")
    with pytest.raises(S.SdmError, match="WORKSPACE"):
        S.selective_scan(ss, *v, h, h, o, torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(S.SdmError, match="WORKSPACE"):
        S.selective_scan(ss, *v, h, h, o, None)
    with pytest.raises(ValueError, match="token stride"):
        S.selective_scan(S.make_scan_shape(1, 4, 2, 1, 16, 16, "f32", ld_x=40), *v, h, h, o, None)
    ns = S.make_norm_shape(4, 16, "f32", "f32", "f32")
    m = [torch.zeros(4, 16, device="cuda") for _ in range(3)]
    with pytest.raises(S.SdmError):
        S.block_norm(ns, *m, x=torch.zeros(4, 16, device="cuda"))  # x without its weights
