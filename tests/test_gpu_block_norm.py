"""The block norm on the GPU against the float64 reference: types, gates of every extent, optional
parts, gradients."""
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


def make(M, D, types, gate_rows, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    y, r, gd = types
    return dict(y=rnd(M, D).to(DT[y]), r=(2 * rnd(M, D)).to(DT[r]), gate=rnd(gate_rows, D).to(DT[gd]) if gate_rows else None,
                w_post=torch.rand(D, generator=g, device="cuda") + 0.5, w_pre=torch.rand(D, generator=g, device="cuda") + 0.5)


CASES = [
    # M, D, (y, r, gate) types, x type, gate rows, activation, post, pre
    (1, 8, ("f32", "f32", "f32"), "f32", 1, "none", True, True),
    (5, 64, ("bf16", "bf16", "bf16"), "bf16", 5, "silu", True, True),
    (12, 520, ("f32", "bf16", "bf16"), "bf16", 3, "sigmoid", True, True),
    (12, 1000, ("f32", "bf16", "f32"), "f32", 0, "none", True, True),
    (7, 2056, ("bf16", "f32", "f32"), "bf16", 1, "silu", False, True),
    (9, 4104, ("f32", "f32", "bf16"), "bf16", 3, "silu", True, False),
    (3, 8192, ("bf16", "f32", "bf16"), "f32", 1, "sigmoid", False, False),
    (4, 16384, ("f32", "f32", "f32"), "f32", 2, "silu", True, True),
    (1100, 24, ("f32", "f32", "f32"), "f32", 2, "silu", True, True),
    (1026, 72, ("f32", "bf16", "f32"), "f32", 513, "silu", True, True),
    (600, 136, ("bf16", "bf16", "bf16"), "bf16", 200, "none", True, True),
    (2000, 40, ("f32", "f32", "f32"), "f32", 1000, "silu", True, True),       # more groups than workgroups
    (3000, 24, ("bf16", "f32", "bf16"), "bf16", 1000, "sigmoid", True, True),  # that begin and end anywhere in their rows
    (2310, 1032, ("f32", "f32", "bf16"), "f32", 33, "silu", True, True),
    (5000, 64, ("f32", "f32", "f32"), "f32", 8, "silu", True, True),           # several rows a wave
    (901, 128, ("bf16", "f32", "f32"), "bf16", 901, "sigmoid", True, True),
    (2049, 256, ("f32", "bf16", "bf16"), "f32", 0, "none", True, True),
]


def adds(D):
    """Roundings on the way of a value: a tree of sums over D values in threads, waves and workgroup
    (D/512 + 16 or fewer), and the elementwise steps, twice for the two norms."""
    return 2 * (D // 512 + 40)


@pytest.mark.parametrize("M,D,types,xt,gate_rows,act,post,pre", CASES)
def test_forward(sdm, M, D, types, xt, gate_rows, act, post, pre):
    d = make(M, D, types, gate_rows)
    if not post:
        d["w_post"] = None
    if not pre:
        d["w_pre"] = None
    sh = sdm.make_norm_shape(M, D, types[0], types[1], xt, types[2], gate_rows, act, 1e-5, 0.7)
    r_out, x = torch.empty_like(d["r"]), torch.empty(M, D, device="cuda", dtype=DT[xt]) if pre else None
    sdm.block_norm(sh, d["y"], d["r"], r_out, gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"], x=x)
    a = {k: R.f64(v) for k, v in d.items()}
    rr, rx = R.norm(a["y"], a["r"], a["gate"], a["w_post"], a["w_pre"], act, 1e-5, 0.7)
    most = a["r"].abs() + (rr - a["r"]).abs()
    half = R.EPS16 * 1.01 if types[1] == "bf16" else 0
    assert ((r_out.double() - rr).abs() <= adds(D) * R.EPS32 * most + half * rr.abs()).all()
    if pre:
        rms = torch.sqrt(rr.square().mean(-1, keepdim=True) + 1e-5)
        half = R.EPS16 * 1.01 if xt == "bf16" else 0
        assert ((x.double() - rx).abs() <= adds(D) * R.EPS32 * (most / rms * a["w_pre"] + rx.abs()) + half * rx.abs()).all()
    # in place
    held, x2 = d["r"].clone(), torch.empty_like(x) if pre else None
    sdm.block_norm(sh, d["y"], held, held, gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"], x=x2)
    assert torch.equal(held, r_out) and (not pre or torch.equal(x2, x))


@pytest.mark.parametrize("M,D,types,xt,gate_rows,act,post,pre", CASES)
@pytest.mark.parametrize("with_dr", [True, False])
def test_gradients(sdm, M, D, types, xt, gate_rows, act, post, pre, with_dr):
    d = make(M, D, types, gate_rows)
    if not post:
        d["w_post"] = None
    if not pre:
        d["w_pre"] = None
    g = torch.Generator(device="cuda").manual_seed(5)
    dr_out = torch.randn(M, D, generator=g, device="cuda") if with_dr else None
    dx = torch.randn(M, D, generator=g, device="cuda") if pre else None
    sh = sdm.make_norm_shape(M, D, types[0], types[1], xt, types[2], gate_rows, act, 1e-5, 0.7)
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    out = dict(y=new(M, D), r=new(M, D), gate=new(gate_rows, D) if gate_rows else None, w_post=new(D) if post else None,
               w_pre=new(D) if pre else None)
    nws = sdm.block_norm_backward_workspace_bytes(sh)
    run = lambda o, up: sdm.block_norm_backward(  # noqa: E731
        sh, d["y"], d["r"], o["y"], o["r"], torch.empty(nws, dtype=torch.uint8, device="cuda"), gate=d["gate"],
        w_post=d["w_post"], w_pre=d["w_pre"], dr_out=up, dx=dx, dgate=o["gate"], dw_post=o["w_post"], dw_pre=o["w_pre"])
    run(out, dr_out)
    leaf = {k: None if v is None else R.f64(v).requires_grad_(True) for k, v in d.items()}
    rr, rx = R.norm(leaf["y"], leaf["r"], leaf["gate"], leaf["w_post"], leaf["w_pre"], act, 1e-5, 0.7)
    loss = torch.zeros((), device="cuda", dtype=torch.float64, requires_grad=True)
    if with_dr:
        loss = loss + (dr_out.double() * rr).sum()
    if pre:
        loss = loss + (dx.double() * rx).sum()
    names = [k for k, v in leaf.items() if v is not None]
    got = torch.autograd.grad(loss, [leaf[k] for k in names], allow_unused=True)
    ref = {k: torch.zeros_like(leaf[k]) if v is None else v for k, v in zip(names, got)}
    # each gradient is a difference of two terms no larger than about the row's largest values:
    # bounded by the rms of the row (or, for the column sums, of the column) times a few
    for k in names:
        want = ref[k]
        if k in ("y", "r"):
            size = want.square().mean(-1, keepdim=True).sqrt() + want.abs()
            spread = 6.0  # |t - h mean(t h)| against its rms: the terms before the difference
        else:
            size = want.abs() + want.square().mean().sqrt()
            spread = 6.0
        n = adds(D) + (min(M, 64) if k not in ("y", "r") else 0)
        assert ((out[k].double() - want).abs() <= spread * n * R.EPS32 * size + 1e-30).all(), k
    if with_dr:  # dr in the place of dr_out
        held = dr_out.clone()
        again = {k: None if v is None else torch.empty_like(v) for k, v in out.items()}
        again["r"] = held
        run(again, held)
        for k in names:
            assert torch.equal(again[k], out[k]), k


def test_row_of_zeros(sdm):
    """With eps = 0 a row of zeros normalises to zeros, and its gradients are finite."""
    D = 64
    sh = sdm.make_norm_shape(2, D, "f32", "f32", "f32", eps=0.0)
    y, r, w = torch.zeros(2, D, device="cuda"), torch.zeros(2, D, device="cuda"), torch.ones(D, device="cuda")
    y[1] = 1.0
    r_out, x = torch.empty_like(r), torch.empty_like(r)
    sdm.block_norm(sh, y, r, r_out, w_post=w, w_pre=w, x=x)
    assert (r_out[0] == 0).all() and (x[0] == 0).all()
    assert (x[1] - 1).abs().max() < 1e-6
    dy, dr, dwp, dwn = torch.empty_like(y), torch.empty_like(y), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(sdm.block_norm_backward_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    sdm.block_norm_backward(sh, y, r, dy, dr, ws, w_post=w, w_pre=w, dr_out=torch.ones_like(y), dx=torch.ones_like(y),
                            dw_post=dwp, dw_pre=dwn)
    for v in (dy, dr, dwp, dwn):
        assert torch.isfinite(v).all()


def test_no_rows(sdm):
    D = 64
    sh = sdm.make_norm_shape(0, D, "f32", "f32", "f32", gate_rows=2)
    e, w, g = torch.empty(0, D, device="cuda"), torch.ones(D, device="cuda"), torch.ones(2, D, device="cuda")
    sdm.block_norm(sh, e, e, e.clone(), gate=g, w_post=w, w_pre=w, x=e.clone())
    dg, dwp, dwn = torch.ones_like(g), torch.ones_like(w), torch.ones_like(w)
    ws = torch.empty(sdm.block_norm_backward_workspace_bytes(sh), dtype=torch.uint8, device="cuda")
    sdm.block_norm_backward(sh, e, e, e.clone(), e.clone(), ws, gate=g, w_post=w, w_pre=w, dr_out=e, dx=e, dgate=dg, dw_post=dwp,
                            dw_pre=dwn)
    assert not dg.any() and not dwp.any() and not dwn.any()


def test_other_rows_do_not_matter(sdm):
    """A NaN row stays in its row."""
    M, D = 6, 136
    d = make(M, D, ("f32", "f32", "f32"), M)
    sh = sdm.make_norm_shape(M, D, "f32", "f32", "f32", gate_rows=M, gate_act="silu")
    r1, x1, r2, x2 = (torch.empty(M, D, device="cuda") for _ in range(4))
    sdm.block_norm(sh, d["y"], d["r"], r1, gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"], x=x1)
    d["y"][2, 5] = float("nan")
    sdm.block_norm(sh, d["y"], d["r"], r2, gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"], x=x2)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(r1[keep], r2[keep]) and torch.equal(x1[keep], x2[keep]) and torch.isnan(x2[2]).all()
