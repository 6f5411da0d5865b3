"""The short causal convolution on the GPU: prompts, single tokens and gradients against the float64
reference, with the float32 error bounds of the sums of absolute terms."""
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


def make(B, T, C, K, dtype, gap=0, bias=True, state=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rnd(B, T, C + gap).to(DT[dtype])[..., gap:] if gap else rnd(B, T, C).to(DT[dtype])
    return dict(x=x, w=rnd(C, K), bias=rnd(C) if bias else None, s_in=rnd(B, K - 1, C).to(DT[dtype]) if state else None)


def value_bound(d, K, act, dtype, y, lengths):
    """K+1 roundings of the sum of absolute terms; silu's slope is below 1.1, its own error a few
    steps; one rounding to the output type."""
    za, _ = R.conv(*(R.absolute(R.f64(d[k])) for k in ("x", "w", "bias", "s_in")), lengths, "none")
    b = (2 * K + 8) * R.EPS32 * (1.1 * za + y.abs())
    return b + (R.EPS16 * y.abs() * 1.01 if dtype == "bf16" else 0) + 1e-30


LENGTHS = {1: None, 2: [5, 0], 3: [0, 1, 2], 4: [37, 2, 0, 16]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,K,act,gap,ragged,bias,state", [
    (1, 1, 8, 4, "silu", 0, False, True, True),
    (2, 5, 24, 2, "none", 8, True, False, True),
    (3, 17, 40, 8, "silu", 0, True, True, False),
    (4, 37, 520, 4, "silu", 16, True, True, True),
    (1, 300, 1288, 3, "silu", 0, False, False, False),
    (2, 129, 256, 5, "none", 0, False, True, True),
])
def test_prompts(sdm, dtype, B, T, C, K, act, gap, ragged, bias, state):
    d = make(B, T, C, K, dtype, gap, bias, state, seed=T + C)
    lengths = torch.tensor(LENGTHS[B], dtype=torch.int32, device="cuda") if ragged else None
    if ragged:  # what padding holds has no effect
        for b, n in enumerate(LENGTHS[B]):
            d["x"][b, n:] = float("nan")
    sh = sdm.make_conv_shape(B, T, C, K, dtype, act, ld_x=C + gap, ld_y=C + 8)
    wide = torch.full((B, T, C + 8), 7.0, device="cuda", dtype=DT[dtype])
    y, s_out = wide[..., :C], torch.empty(B, K - 1, C, device="cuda", dtype=DT[dtype])
    sdm.short_conv(sh, d["x"], d["w"], y, bias=d["bias"], lengths=lengths, s_in=d["s_in"], s_out=s_out)
    ry, rs = R.conv(*(R.f64(d[k]) for k in ("x", "w", "bias", "s_in")), lengths, act)
    clean = dict(d, x=torch.nan_to_num(d["x"]))
    assert torch.equal(s_out.double(), rs)
    assert ((y.double() - ry).abs() <= value_bound(clean, K, act, dtype, ry, lengths)).all()
    assert (wide[..., C:] == 7.0).all()  # columns beside the output stay
    # the same with the state in place
    if state:
        held, y2 = d["s_in"].clone(), torch.empty(B, T, C, device="cuda", dtype=DT[dtype])
        sdm.short_conv(sdm.make_conv_shape(B, T, C, K, dtype, act, ld_x=C + gap), d["x"], d["w"], y2, bias=d["bias"],
                       lengths=lengths, s_in=held, s_out=held)
        assert torch.equal(held, s_out) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cuts", [[40], [1, 39], [16, 24], [2, 1, 1, 20, 16], [0, 40]])
def test_calls_continue_from_the_state(sdm, dtype, cuts):
    B, C, K = 2, 72, 4
    d = make(B, 40, C, K, dtype, state=False)
    whole, end = torch.empty(B, 40, C, device="cuda", dtype=DT[dtype]), torch.empty(B, K - 1, C, device="cuda", dtype=DT[dtype])
    sdm.short_conv(sdm.make_conv_shape(B, 40, C, K, dtype), d["x"], d["w"], whole, bias=d["bias"], s_out=end)
    state, at, got = torch.zeros(B, K - 1, C, device="cuda", dtype=DT[dtype]), 0, []
    for n in cuts:
        y = torch.empty(B, n, C, device="cuda", dtype=DT[dtype])
        part = d["x"][:, at:at + n].contiguous()
        if n == 1:
            sdm.short_conv_step(sdm.make_conv_shape(B, 1, C, K, dtype), part, d["w"], state, y, bias=d["bias"])
        else:
            sdm.short_conv(sdm.make_conv_shape(B, n, C, K, dtype), part, d["w"], y, bias=d["bias"], s_in=state, s_out=state)
        got.append(y)
        at += n
    assert torch.equal(torch.cat(got, 1), whole) and torch.equal(state, end)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,K,act,gap,ragged,bias,state", [
    (1, 1, 8, 4, "silu", 0, False, True, True),
    (2, 5, 24, 2, "none", 8, True, False, True),
    (3, 17, 40, 8, "silu", 0, True, True, False),
    (4, 37, 264, 4, "silu", 16, True, True, True),
    (1, 300, 72, 3, "silu", 0, False, False, True),
    (2, 0, 16, 4, "silu", 0, False, True, True),
    (3, 1200, 8, 2, "none", 8, False, True, True),     # several workgroups of few channels
    (2, 1100, 128, 8, "silu", 0, True, True, True),
    (9, 3900, 136, 3, "silu", 0, False, True, True),   # many rows of few sums
])
def test_gradients(sdm, dtype, B, T, C, K, act, gap, ragged, bias, state):
    d = make(B, T, C, K, dtype, gap, bias, state, seed=T)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy, ds_out = torch.randn(B, T, C, generator=g, device="cuda"), None
    if state:
        ds_out = torch.randn(B, K - 1, C, generator=g, device="cuda")
    lengths = torch.tensor(LENGTHS[B], dtype=torch.int32, device="cuda") if ragged else None
    if ragged:
        for b, n in enumerate(LENGTHS[B]):
            d["x"][b, n:] = float("nan")
            dy[b, n:] = float("inf")
    sh = sdm.make_conv_shape(B, T, C, K, dtype, act, ld_x=C + gap)
    wide = torch.full((B, T, C + gap), 7.0, device="cuda")
    out = dict(dx=wide[..., gap:], dw=torch.full((C, K), 7.0, device="cuda"), dbias=torch.full((C,), 7.0, device="cuda") if bias else None,
               ds_in=torch.full((B, K - 1, C), 7.0, device="cuda") if state else None)
    ws = torch.empty(sdm.short_conv_backward_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    sdm.short_conv_backward(sh, d["x"], d["w"], dy, out["dx"], out["dw"], ws, bias=d["bias"], dbias=out["dbias"],
                            lengths=lengths, s_in=d["s_in"], ds_out=ds_out, ds_in=out["ds_in"])
    names = [k for k in ("x", "w", "bias", "s_in") if d[k] is not None]
    leaf = {k: R.f64(d[k]).nan_to_num().requires_grad_(True) for k in names}
    args = [leaf.get(k) for k in ("x", "w", "bias", "s_in")]
    y, s = R.conv(*args, lengths, act)
    live = torch.isfinite(dy)
    loss = (torch.where(live, dy, dy.new_zeros(())).double() * y).sum() + ((ds_out.double() * s).sum() if state else 0)
    ref = dict(zip(names, torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True))) if loss.requires_grad else {}
    # sums of absolute terms: the convolution without activation on absolute values, the upstream
    # gradient scaled by the largest slope of silu (1.1) and its change under z's own error
    al = {k: v.detach().abs().requires_grad_(True) for k, v in leaf.items()}
    ya, sa = R.conv(*[al.get(k) for k in ("x", "w", "bias", "s_in")], lengths, "none")
    za = ya.detach()
    up = torch.where(live, dy, dy.new_zeros(())).double().abs() * (1.1 + 0.6 * za)
    la = (up * ya).sum() + ((ds_out.double().abs() * sa).sum() if state else 0)
    ab = dict(zip(names, torch.autograd.grad(la, [al[k] for k in names], allow_unused=True))) if la.requires_grad else {}
    tokens = B * T
    for k, o in (("x", out["dx"]), ("w", out["dw"]), ("bias", out["dbias"]), ("s_in", out["ds_in"])):
        if o is None:
            continue
        want = ref.get(k) if ref.get(k) is not None else torch.zeros_like(o, dtype=torch.float64)
        most = ab.get(k) if ab.get(k) is not None else torch.zeros_like(want)
        adds = 2 * K + 12 + (min(tokens, 32) if k in ("w", "bias") else 0)
        assert ((o.double() - want).abs() <= adds * R.EPS32 * most + 1e-30).all(), k
    assert gap == 0 or (wide[..., :gap] == 7.0).all()


def test_gradient_of_differences(sdm):
    """The directional difference of the float32 forward is the gradient's inner product: the step of
    2^-6 leaves a third-order term of about 2^-12 of the terms, the float32 outputs 2^-24 / 2^-6."""
    B, T, C, K = 2, 33, 16, 4
    d = make(B, T, C, K, "f32")
    g = torch.Generator(device="cuda").manual_seed(3)
    v, dy = torch.randn(B, T, C, generator=g, device="cuda"), torch.randn(B, T, C, generator=g, device="cuda")
    sh = sdm.make_conv_shape(B, T, C, K, "f32")
    ys = []
    for s in (1, -1):
        y = torch.empty(B, T, C, device="cuda")
        sdm.short_conv(sh, d["x"] + s * 2.0 ** -6 * v, d["w"], y, bias=d["bias"], s_in=d["s_in"])
        ys.append(y.double())
    dx, dw, db = torch.empty(B, T, C, device="cuda"), torch.empty(C, K, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(sdm.short_conv_backward_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    sdm.short_conv_backward(sh, d["x"], d["w"], dy, dx, dw, ws, bias=d["bias"], dbias=db, s_in=d["s_in"])
    slope = (ys[0] - ys[1]) * 2.0 ** 5
    most = (dy.double() * slope).abs().sum()
    assert abs((dy.double() * slope).sum() - (dx.double() * v.double()).sum()) <= 2e-3 * most
