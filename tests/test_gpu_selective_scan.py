"""The selective scan on the GPU: prompts, single tokens, continued and split sequences and gradients
against the float64 reference, with float32 error bounds stated against the sums of absolute terms."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sdm():
    import sparse_memory_linear_amd as S
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    S.lib()
    return S


class Case:
    """Inputs as slices of one packed tensor, lengths, states; padding holds NaN."""

    def __init__(self, B, T, H, G, N, P, dtype, lengths=None, state=True, D=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.dims = (B, T, H, G, N, P)
        self.width = H * P + 2 * G * N
        self.xbc = rnd(B, T, self.width).to(DT[dtype])
        self.dt = rnd(B, T, H + 3)[..., :H]
        self.A_log = torch.log(torch.rand(H, generator=g, device="cuda") * 15 + 1)
        self.dt_bias = rnd(H) - 3.0
        self.D = rnd(H) if D else None
        self.s_in = rnd(B, H, P, N) if state else None
        self.go, self.ds_out = rnd(B, H, T, P), rnd(B, H, P, N) if state else None
        self.lengths = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
        if lengths is not None:
            for b, n in enumerate(lengths):
                n = max(0, min(n, T))
                self.xbc[b, n:], self.dt[b, n:], self.go[b, :, n:] = float("nan"), float("inf"), float("nan")
        self.dtype = dtype

    def shape(self, sdm):
        return sdm.make_scan_shape(*self.dims, self.dtype, ld_x=self.width, ld_b=self.width, ld_c=self.width, ld_dt=self.dims[2] + 3)

    def split(self, t):
        B, T, H, G, N, P = self.dims
        return t.split([H * P, G * N, G * N], -1)

    def wide(self, clean=False):
        """x [B,T,H,P], B, C [B,T,G,N], dt in float64 (padding as 0 if `clean`)."""
        B, T, H, G, N, P = self.dims
        x, b, c = self.split(self.xbc.double().nan_to_num() if clean else self.xbc.double())
        dt = self.dt.double()
        return x.reshape(B, T, H, P), b.reshape(B, T, G, N), c.reshape(B, T, G, N), dt.nan_to_num(posinf=0.0) if clean else dt

    def forward(self, sdm, s_out=True):
        B, T, H, G, N, P = self.dims
        sh = self.shape(sdm)
        o = torch.full((B, H, T, P), 7.0, device="cuda")
        end = torch.full((B, H, P, N), 7.0, device="cuda") if s_out else None
        ws = torch.empty(sdm.selective_scan_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        sdm.selective_scan(sh, *self.split(self.xbc), self.dt, self.A_log, self.dt_bias, o, ws, D=self.D,
                           lengths=self.lengths, s_in=self.s_in, s_out=end)
        return o, end

    def reference(self):
        x, b, c, dt = self.wide(clean=True)
        _, dtv, la = R.scan_gates(dt, R.f64(self.A_log), R.f64(self.dt_bias), self.lengths)
        D, s = R.f64(self.D), R.f64(self.s_in)
        o, S = R.scan(x, b, c, dtv, la, D, s, self.lengths)
        oa, Sa = R.scan(x.abs(), b.abs(), c.abs(), dtv, la, R.absolute(D), R.absolute(s), self.lengths)
        return o, S, oa, Sa

    def roundings(self):
        """Roundings on the way of a term, each at most 2^-24 of the sum of absolute terms: the sums over
        d_k or d_v and over the tokens (a term that is carried far has decayed), and the factors
        themselves: the time step, its log-decay and exp of it, whose error is |l| exp(l) < 1/2 steps
        for each step of l's own relative error."""
        B, T, H, G, N, P = self.dims
        return min(T, 128) + max(N, P) + 40


CASES = [
    # B, T, H, G, d_k, d_v, lengths, state, D
    (1, 1, 1, 1, 8, 8, None, False, False),
    (2, 1, 3, 1, 64, 64, None, True, True),
    (1, 63, 2, 2, 16, 24, None, True, True),
    (1, 64, 2, 1, 128, 64, None, False, True),
    (2, 65, 4, 2, 40, 72, None, True, False),
    (4, 130, 2, 1, 128, 128, [130, 0, 1, 65], True, True),
    (3, 200, 6, 3, 32, 16, [64, 128, 63], True, True),
    (1, 192, 1, 1, 72, 200, None, True, True),
    (2, 257, 2, 2, 96, 256, [300, -4], False, True),
    (3, 0, 2, 1, 16, 16, None, True, True),
    (70, 200, 8, 2, 16, 16, None, True, True),          # as many units as fill the chip: one segment
    (20, 300, 8, 1, 24, 16, [300, 150] * 10, True, True),  # segments of several blocks
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,G,N,P,lengths,state,D", CASES)
def test_prompts(sdm, dtype, B, T, H, G, N, P, lengths, state, D):
    c = Case(B, T, H, G, N, P, dtype, lengths, state, D, seed=T)
    o, end = c.forward(sdm)
    ro, rS, oa, Sa = c.reference()
    k = c.roundings() * R.EPS32
    assert ((o.double() - ro).abs() <= k * oa + 1e-30).all()
    assert ((end.double() - rS).abs() <= k * Sa + 1e-30).all()
    if state:  # in place
        sh, held, o2 = c.shape(sdm), c.s_in.clone(), torch.empty_like(o)
        ws = torch.empty(sdm.selective_scan_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
        sdm.selective_scan(sh, *c.split(c.xbc), c.dt, c.A_log, c.dt_bias, o2, ws, D=c.D, lengths=c.lengths, s_in=held, s_out=held)
        assert torch.equal(held, end) and torch.equal(o2, o)
    o3, _ = c.forward(sdm, s_out=False)
    assert torch.equal(o3, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,G,N,P,lengths", [
    (1, 3000, 2, 1, 64, 32, None),          # few heads: the tokens are split into segments
    (2, 2500, 1, 1, 128, 72, [2500, 1111]),
    (1, 4161, 3, 3, 16, 128, None),
])
def test_long_sequences(sdm, dtype, B, T, H, G, N, P, lengths):
    c = Case(B, T, H, G, N, P, dtype, lengths, seed=T)
    o, end = c.forward(sdm)
    ro, rS, oa, Sa = c.reference()
    k = c.roundings() * R.EPS32
    assert ((o.double() - ro).abs() <= k * oa + 1e-30).all()
    assert ((end.double() - rS).abs() <= k * Sa + 1e-30).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cuts", [[1, 129], [64, 66], [100, 1, 1, 28], [0, 130]])
def test_calls_continue_from_the_state(sdm, dtype, cuts):
    c = Case(2, 130, 4, 2, 40, 24, dtype, seed=9)
    B, T, H, G, N, P = c.dims
    ro, rS, oa, Sa = c.reference()
    state, at, got = c.s_in.clone(), 0, []
    for n in cuts:
        o = torch.empty(B, H, n, P, device="cuda")
        x, b, cm = (v[:, at:at + n].contiguous() for v in c.split(c.xbc))
        dt, sh = c.dt[:, at:at + n].contiguous(), sdm.make_scan_shape(B, n, H, G, N, P, dtype)
        if n == 1:
            sdm.selective_scan_step(sh, x, b, cm, dt, c.A_log, c.dt_bias, state, o, D=c.D)
        else:
            ws = torch.empty(sdm.selective_scan_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
            sdm.selective_scan(sh, x, b, cm, dt, c.A_log, c.dt_bias, o, ws, D=c.D, s_in=state, s_out=state)
        got.append(o)
        at += n
    k = (c.roundings() + 8) * R.EPS32
    assert ((torch.cat(got, 2).double() - ro).abs() <= k * oa).all()
    assert ((state.double() - rS).abs() <= k * Sa).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,G,N,P,D", [(1, 1, 1, 8, 8, False), (5, 4, 2, 40, 24, True), (3, 8, 1, 128, 128, True),
                                          (2, 6, 6, 64, 200, True), (2, 2, 1, 120, 256, True)])
def test_single_tokens(sdm, dtype, B, H, G, N, P, D):
    c = Case(B, 1, H, G, N, P, dtype, None, True, D, seed=N)
    ro, rS, oa, Sa = c.reference()
    state, o = c.s_in.clone(), torch.empty(B, H, 1, P, device="cuda")
    sdm.selective_scan_step(c.shape(sdm), *c.split(c.xbc), c.dt, c.A_log, c.dt_bias, state, o, D=c.D)
    k = c.roundings() * R.EPS32
    assert ((o.double() - ro).abs() <= k * oa).all() and ((state.double() - rS).abs() <= k * Sa).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["x", "B", "C"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_later_values_reach_no_earlier_output(sdm, dtype, what, bad):
    """A NaN or an infinity at token 77 leaves the outputs before it as they were."""
    c = Case(2, 140, 2, 1, 32, 24, dtype, seed=4)
    before, _ = c.forward(sdm)
    B, T, H, G, N, P = c.dims
    c.split(c.xbc)[{"x": 0, "B": 1, "C": 2}[what]][0, 77, 5] = bad
    after, end = c.forward(sdm)
    ro, rS, oa, Sa = Case(2, 140, 2, 1, 32, 24, dtype, seed=4).reference()
    assert ((after[0, :, :77].double() - ro[0, :, :77]).abs() <= c.roundings() * R.EPS32 * oa[0, :, :77]).all()
    assert torch.equal(after[1], before[1])
    assert not torch.isfinite(after[0, 0, 77]).all()
    if what == "C":  # a read alone: the state and the later outputs stay
        assert torch.equal(after[0, :, 78:], before[0, :, 78:]) and torch.isfinite(end).all()


def test_extreme_time_steps(sdm):
    """Steps that forget everything and steps that forget nothing, side by side."""
    c = Case(1, 150, 2, 1, 16, 16, "f32", seed=6)
    c.dt[0, 10:20] = 400.0
    c.dt[0, 20:40] = -80.0
    c.dt[0, 100] = 3000.0
    c.dt[0, 101:] = -200.0
    o, end = c.forward(sdm)
    ro, rS, oa, Sa = c.reference()
    k = c.roundings() * R.EPS32
    assert torch.isfinite(o).all()
    assert ((o.double() - ro).abs() <= k * oa + 1e-30).all() and ((end.double() - rS).abs() <= k * Sa + 1e-30).all()


GRAD = [
    (1, 1, 1, 1, 8, 8, None, False, False),
    (2, 1, 3, 1, 64, 64, None, True, True),
    (1, 63, 2, 2, 16, 24, None, True, True),
    (1, 64, 2, 1, 128, 64, None, False, True),
    (2, 65, 4, 2, 40, 72, None, True, False),
    (4, 130, 2, 1, 128, 128, [130, 0, 1, 65], True, True),
    (3, 200, 6, 3, 32, 16, [64, 128, 63], True, True),
    (1, 130, 1, 1, 72, 200, None, True, True),
    (2, 129, 2, 2, 96, 256, [300, -4], False, True),
    (1, 70, 8, 1, 24, 40, None, True, True),
    (3, 0, 2, 1, 16, 16, None, True, True),
    (40, 200, 8, 2, 16, 16, None, True, True),             # one segment of several blocks
    (10, 300, 8, 1, 40, 72, [300, 150, 0, 63, 64] * 2, True, True),  # segments of several blocks
    (64, 100, 8, 1, 24, 136, None, False, True),           # several heads and channel blocks a workgroup
]


def backward(sdm, c, **kw):
    B, T, H, G, N, P = c.dims
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = dict(dxbc=new(B, T, c.width), ddt=new(B, T, H + 3), dA_log=new(H), ddt_bias=new(H), dD=new(H) if c.D is not None else None,
               ds_in=new(B, H, P, N) if c.s_in is not None else None)
    sh = c.shape(sdm)
    ws = torch.full((sdm.selective_scan_backward_workspace_bytes(sh),), 255, dtype=torch.uint8, device="cuda")
    sdm.selective_scan_backward(sh, *c.split(c.xbc), c.dt, c.A_log, c.dt_bias, c.go, *c.split(out["dxbc"]), out["ddt"][..., :H],
                                out["dA_log"], out["ddt_bias"], ws, D=c.D, dD=out["dD"], lengths=c.lengths, s_in=c.s_in,
                                ds_out=c.ds_out, ds_in=out["ds_in"])
    return out


def check_gradients(sdm, c):
    B, T, H, G, N, P = c.dims
    out = backward(sdm, c)
    x, b, cm, dt = c.wide(clean=True)
    go = c.go.double().nan_to_num()
    ref, most = R.scan_gradients(x, b, cm, dt, R.f64(c.A_log), R.f64(c.dt_bias), R.f64(c.D), R.f64(c.s_in), c.lengths, go,
                                 R.f64(c.ds_out))
    dx, db, dc = c.split(out["dxbc"])
    got = dict(dx=dx.reshape(B, T, H, P), dBm=db.reshape(B, T, G, N), dCm=dc.reshape(B, T, G, N), ddt=out["ddt"][..., :H],
               ddt_bias=out["ddt_bias"], dA_log=out["dA_log"], dD=out["dD"], ds_in=out["ds_in"])
    assert (out["ddt"][..., H:] == 7.0).all()
    k = (2 * c.roundings() + P + H // G) * R.EPS32
    for name, g in got.items():
        if g is not None:
            assert ((g.double() - ref[name]).abs() <= k * most[name] + 1e-30).all(), name
    again = backward(sdm, c)
    for name, g in out.items():
        assert g is None or torch.equal(g, again[name]), f"{name} differs from run to run"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H,G,N,P,lengths,state,D", GRAD)
def test_gradients(sdm, dtype, B, T, H, G, N, P, lengths, state, D):
    check_gradients(sdm, Case(B, T, H, G, N, P, dtype, lengths, state, D, seed=T))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_long_sequences(sdm, dtype):
    check_gradients(sdm, Case(2, 1500, 2, 1, 16, 24, dtype, [1500, 777], seed=2))


def test_gradient_of_differences(sdm):
    """The directional difference of the float32 forward is the gradient's inner product (step 2^-7: a
    third-order term of about 2^-14 of the terms, and 2^-24 / 2^-7 of rounding, over sums of them)."""
    c = Case(1, 100, 2, 1, 16, 16, "f32", seed=8)
    B, T, H, G, N, P = c.dims
    g = torch.Generator(device="cuda").manual_seed(11)
    dirs = [torch.randn(t.shape, generator=g, device="cuda") for t in (c.xbc, c.dt, c.A_log, c.D)]
    grad = backward(sdm, c)
    total = []
    for s in (1, -1):
        m = Case(1, 100, 2, 1, 16, 16, "f32", seed=8)
        for t, v in zip((m.xbc, m.dt, m.A_log, m.D), dirs):
            t += s * 2.0 ** -7 * v
        o, end = m.forward(sdm)
        total.append((o.double() * c.go.double(), end.double() * c.ds_out.double()))
    slope = [(a - b) * 2.0 ** 6 for a, b in zip(*total)]
    got = sum((v.double() * w.double()).sum() for v, w in zip(dirs, (grad["dxbc"], grad["ddt"][..., :H], grad["dA_log"], grad["dD"])))
    most = sum(s.abs().sum() for s in slope)
    assert abs(sum(s.sum() for s in slope) - got) <= 2e-3 * most


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", [(1, 200, 2), (40, 130, 8), (2, 0, 2), (1, 20, 1)])
def test_gradient_without_states(sdm, dtype, B, T, H):
    """States that are left out are zeros; a first state's gradient that is not wanted changes nothing."""
    c = Case(B, T, H, 1, 24, 40, dtype, state=True, seed=3)
    c.s_in.zero_()
    c.ds_out.zero_()
    want = backward(sdm, c)
    s_in, ds_out = c.s_in, c.ds_out
    c.ds_out = None
    got = backward(sdm, c)
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    c.s_in, c.ds_out = None, ds_out  # (and so no ds_in)
    got = backward(sdm, c)
    for k, v in want.items():
        assert k == "ds_in" or torch.equal(got[k], v), k
    # ds_in alone
    c.ds_out = None
    end = torch.full_like(s_in, 7.0)
    o = {k: torch.full_like(v, 7.0) for k, v in want.items()}
    sh = c.shape(sdm)
    ws = torch.empty(sdm.selective_scan_backward_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    sdm.selective_scan_backward(sh, *c.split(c.xbc), c.dt, c.A_log, c.dt_bias, c.go, *c.split(o["dxbc"]), o["ddt"][..., :H],
                                o["dA_log"], o["ddt_bias"], ws, D=c.D, dD=o["dD"], ds_in=end)
    assert torch.equal(end, want["ds_in"]) and torch.equal(o["dxbc"], want["dxbc"]) and torch.equal(o["ddt"], want["ddt"])
