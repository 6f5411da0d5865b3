"""The convolution, scan and norm calls on the host: shape limits, workspace sizes, and bad arguments
refused before any HIP call (no GPU needed); and the float64 references the GPU tests use, against
differences and against other forms."""
import ctypes

import pytest
import torch

import block_reference as R

FAKE = 1 << 40  # 16-byte aligned fake device addresses, never dereferenced
GAP = 1 << 36


@pytest.fixture(scope="module")
def sdm():
    import os

    import sparse_memory_linear_amd as S
    if not os.path.exists(S.lib_path):
        from sparse_memory_linear_amd import build
        build.build(verbose=False)
    return S


@pytest.fixture(scope="module")
def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("fake-pointer validation tests run only where no GPU is visible")


def conv(S, **kw):
    return S.make_conv_shape(**{**dict(B=2, T=64, C=64, K=4, in_dtype="bf16", act="silu"), **kw})


def scan(S, **kw):
    return S.make_scan_shape(**{**dict(B=2, T=64, H=4, G=2, d_k=64, d_v=64, in_dtype="bf16"), **kw})


def norm(S, **kw):
    return S.make_norm_shape(**{**dict(M=8, D=64, gate_rows=2), **kw})


@pytest.mark.parametrize("kw,code", [
    ({}, 0), ({"T": 0}, 0), ({"B": 0}, -1), ({"T": -1}, -1), ({"C": 0}, -1), ({"K": 0}, -1), ({"K": 1}, -2), ({"K": 9}, -2),
    ({"C": 60}, -2), ({"in_dtype": 2}, -1), ({"act": "sigmoid"}, -1), ({"act": 9}, -1), ({"ld_x": 56}, -1), ({"ld_x": 68}, -2),
    ({"ld_y": 100}, -2), ({"ld_y": 1 << 25}, -2), ({"B": 1 << 16, "T": 1 << 16}, -2), ({"B": 1 << 20, "T": 64, "C": 1 << 18}, -2),
])
def test_check_conv_shape(sdm, kw, code):
    assert sdm.check_conv_shape(conv(sdm, **kw)) == code
    assert (sdm.short_conv_backward_workspace_bytes(conv(sdm, **kw)) > 0) == (code == 0)


@pytest.mark.parametrize("kw,code", [
    ({}, 0), ({"T": 0}, 0), ({"B": 0}, -1), ({"H": 0}, -1), ({"G": 0}, -1), ({"G": 3}, -1), ({"d_k": 0}, -1), ({"d_v": 0}, -1),
    ({"d_k": 12}, -2), ({"d_k": 136}, -2), ({"d_v": 264}, -2), ({"d_v": 20}, -2), ({"in_dtype": 5}, -1), ({"ld_x": 128}, -1),
    ({"ld_b": 64}, -1), ({"ld_c": 132}, -2), ({"ld_dt": 3}, -1), ({"ld_dt": 5}, 0), ({"ld_x": (1 << 22) + 8}, -2),
    ({"B": 1 << 15, "T": 1 << 15}, -2), ({"B": 1 << 14, "H": 8}, -2), ({"H": 8192, "G": 1}, -2),
])
def test_check_scan_shape(sdm, kw, code):
    s = scan(sdm, **kw)
    assert sdm.check_scan_shape(s) == code
    if code:
        assert sdm.selective_scan_workspace_bytes(s) == 0 and sdm.selective_scan_backward_workspace_bytes(s) == 0
    elif s.T:
        assert sdm.selective_scan_workspace_bytes(s) >= 20 * s.B * s.H * s.T


def test_scan_gradient_size_limit(sdm):
    s = scan(sdm, B=64, T=1 << 20, H=4)
    assert sdm.check_scan_shape(s) == 0
    assert sdm.selective_scan_workspace_bytes(s) > 0 and sdm.selective_scan_backward_workspace_bytes(s) == 0


@pytest.mark.parametrize("kw,code", [
    ({}, 0), ({"M": 0}, 0), ({"M": -1}, -1), ({"D": 0}, -1), ({"D": 60}, -2), ({"D": 16392}, -2), ({"gate_rows": 3}, -1),
    ({"gate_rows": -1}, -1), ({"gate_rows": 0}, 0), ({"y_dtype": 3}, -1), ({"r_dtype": -1}, -1), ({"x_dtype": 2}, -1),
    ({"gate_dtype": 2}, -1), ({"gate_act": 3}, -1), ({"eps": -1.0}, -1), ({"eps": 2.0}, -1), ({"eps": float("nan")}, -1),
    ({"scale": float("inf")}, -1), ({"M": 1 << 31, "gate_rows": 0}, -2),
])
def test_check_norm_shape(sdm, kw, code):
    assert sdm.check_norm_shape(norm(sdm, **kw)) == code
    assert (sdm.block_norm_backward_workspace_bytes(norm(sdm, **kw)) > 0) == (code == 0)


def every_bad_pointer(call, args, required, optional=()):
    """Each pointer null (if it may not be) and misaligned."""
    for i in required:
        bad = list(args)
        bad[i] = None
        assert call(*bad) == -1, f"null argument {i}"
    for i in list(required) + list(optional):
        bad = list(args)
        bad[i] = bad[i] + 4
        assert call(*bad) == -1, f"misaligned argument {i}"


def ptrs(n):
    return [FAKE + i * GAP for i in range(n)]


def test_conv_pointers(sdm, no_gpu):
    L, s = sdm.lib(), conv(sdm)
    p = ptrs(12)
    call = lambda *a: L.sdm_short_conv(ctypes.byref(s), *a, None)  # noqa: E731  x w bias lengths s_in s_out y
    every_bad_pointer(call, p[:7], (0, 1, 6), (2, 3, 4, 5))
    overlap = list(p[:7])
    overlap[6] = p[0] + 4096  # y inside x
    assert call(*overlap) == -1
    overlap = list(p[:7])
    overlap[5] = p[4] + 64    # s_out shifted against s_in
    assert call(*overlap) == -1
    s1 = conv(sdm, T=1)
    step = lambda *a: L.sdm_short_conv_step(ctypes.byref(s1), *a, None)  # noqa: E731  x w bias state y
    every_bad_pointer(step, p[:5], (0, 1, 3, 4), (2,))
    assert L.sdm_short_conv_step(ctypes.byref(s), *p[:5], None) == -1  # T = 64
    need = sdm.short_conv_backward_workspace_bytes(s)
    # x w bias lengths s_in dy ds_out dx dw dbias ds_in ws
    back = lambda *a: L.sdm_short_conv_backward(ctypes.byref(s), *a, need, None)  # noqa: E731
    every_bad_pointer(back, p, (0, 1, 5, 7, 8), (3, 4, 6, 10, 11))
    assert back(*p[:2], None, *p[3:]) == -1      # dbias without bias
    assert back(*p[:9], None, *p[10:]) == -1     # bias without dbias
    assert L.sdm_short_conv_backward(ctypes.byref(s), *p, need - 1, None) == -3
    assert back(*p[:11], None) == -3
    assert back(*p[:7], p[5], *p[8:]) == -1      # dx in the place of dy


def test_scan_pointers(sdm, no_gpu):
    L, s = sdm.lib(), scan(sdm)
    p = ptrs(20)
    need = sdm.selective_scan_workspace_bytes(s)
    # x B C dt A_log dt_bias D lengths s_in s_out o ws
    call = lambda *a: L.sdm_selective_scan(ctypes.byref(s), *a, need, None)  # noqa: E731
    every_bad_pointer(call, p[:12], (0, 1, 2, 3, 4, 5, 10), (6, 7, 8, 9, 11))
    assert L.sdm_selective_scan(ctypes.byref(s), *p[:12], need - 1, None) == -3
    assert call(*p[:11], None) == -3
    assert call(*p[:10], p[0] + 128, p[11]) == -1           # o inside x
    assert call(*p[:9], p[8] + 1024, *p[10:12]) == -1       # s_out shifted against s_in
    s1 = scan(sdm, T=1)
    # x B C dt A_log dt_bias D state o
    step = lambda *a: L.sdm_selective_scan_step(ctypes.byref(s1), *a, None)  # noqa: E731
    every_bad_pointer(step, p[:9], (0, 1, 2, 3, 4, 5, 7, 8), (6,))
    assert L.sdm_selective_scan_step(ctypes.byref(s), *p[:9], None) == -1
    nb = sdm.selective_scan_backward_workspace_bytes(s)
    # x B C dt A_log dt_bias D lengths s_in go ds_out dx dB dC ddt dA_log ddt_bias dD ds_in ws
    back = lambda *a: L.sdm_selective_scan_backward(ctypes.byref(s), *a, nb, None)  # noqa: E731
    every_bad_pointer(back, p, (0, 1, 2, 3, 4, 5, 9, 11, 12, 13, 14, 15, 16), (7, 8, 10, 18, 19))
    assert back(*p[:6], None, *p[7:]) == -1       # dD without D
    assert back(*p[:17], None, *p[18:]) == -1     # D without dD
    assert L.sdm_selective_scan_backward(ctypes.byref(s), *p, nb - 1, None) == -3
    assert back(*p[:12], p[11] + 64, *p[13:]) == -1  # dB inside dx


def test_slices_of_one_buffer(sdm, no_gpu):
    """Column slices of one wide buffer may hold outputs side by side, but not on top of each other."""
    L = sdm.lib()
    wide = 4 * 64 + 2 * 2 * 64
    s = scan(sdm, ld_x=wide, ld_b=wide, ld_c=wide)
    p = ptrs(20)
    nb = sdm.selective_scan_backward_workspace_bytes(s)
    dx, db, dc = p[11], p[11] + 256 * 4, p[11] + (256 + 128) * 4
    args = p[:11] + [dx, db, dc] + p[14:]
    args[11 + 2] = db + 64 * 4  # dC over the end of dB
    assert L.sdm_selective_scan_backward(ctypes.byref(s), *args, nb, None) == -1
    args[11 + 2], args[11 + 1] = dc, dx + 192 * 4  # dB over the end of dx
    assert L.sdm_selective_scan_backward(ctypes.byref(s), *args, nb, None) == -1
    s2 = scan(sdm, ld_x=wide, ld_b=wide, ld_c=wide + 8)  # another distance between rows
    args[11 + 1] = db
    assert L.sdm_selective_scan_backward(ctypes.byref(s2), *args, nb, None) == -1


def test_norm_pointers(sdm, no_gpu):
    L, s = sdm.lib(), norm(sdm)
    p = ptrs(13)
    # y r gate w_post w_pre r_out x
    call = lambda *a: L.sdm_block_norm(ctypes.byref(s), *a, None)  # noqa: E731
    every_bad_pointer(call, p[:7], (0, 1, 2, 4, 5, 6), (3,))
    assert L.sdm_block_norm(ctypes.byref(norm(sdm, gate_rows=0)), *p[:7], None) == -1  # a gate without rows
    assert call(*p[:5], p[1] + 32, p[6]) == -1    # r_out shifted against r
    assert call(*p[:6], p[0]) == -1               # x in the place of y
    nb = sdm.block_norm_backward_workspace_bytes(s)
    # y r gate w_post w_pre dr_out dx dy dr dgate dw_post dw_pre ws
    back = lambda *a: L.sdm_block_norm_backward(ctypes.byref(s), *a, nb, None)  # noqa: E731
    every_bad_pointer(back, p, (0, 1, 2, 3, 4, 6, 7, 8, 9, 10, 11), (5, 12))
    assert L.sdm_block_norm_backward(ctypes.byref(s), *p, nb - 1, None) == -3
    assert back(*p[:7], p[6], *p[8:]) == -1       # dy in the place of dx


def test_binding_refuses_tensors_on_the_host(sdm):
    s = conv(sdm, B=1, T=2, C=8)
    x, w = torch.zeros(1, 2, 8, dtype=torch.bfloat16), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="not on a GPU"):
        sdm.short_conv(s, x, w, torch.empty_like(x))
    with pytest.raises(ValueError, match="x is torch.float32"):
        sdm.short_conv(s, x.float(), w, torch.empty_like(x))
    with pytest.raises(ValueError, match="missing"):
        sdm.short_conv(s, None, w, x)


# ------------------------------------------------------------------- the references themselves
def differences(f, x, v, step=1e-6):
    return (f(x + step * v) - f(x - step * v)) / (2 * step)


def test_reference_gradients_against_differences():
    torch.manual_seed(0)
    B, T, H, G, N, P = 2, 9, 4, 2, 3, 5
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    a = dict(x=rnd(B, T, H, P), Bm=rnd(B, T, G, N), Cm=rnd(B, T, G, N), dt=rnd(B, T, H), A_log=rnd(H), dt_bias=rnd(H), D=rnd(H),
             s_in=rnd(B, H, P, N))
    lengths = torch.tensor([9, 4])
    go, ds = rnd(B, H, T, P), rnd(B, H, P, N)

    def loss(**kw):
        v = {**a, **kw}
        _, dtv, la = R.scan_gates(v["dt"], v["A_log"], v["dt_bias"], lengths)
        o, s = R.scan(v["x"], v["Bm"], v["Cm"], dtv, la, v["D"], v["s_in"], lengths)
        return (go * o).sum() + (ds * s).sum()

    g = R.scan_gradients(*[a[k] for k in ("x", "Bm", "Cm", "dt", "A_log", "dt_bias", "D", "s_in")], lengths, go, ds)[0]
    for k, name in (("x", "dx"), ("Bm", "dBm"), ("Cm", "dCm"), ("dt", "ddt"), ("A_log", "dA_log"), ("dt_bias", "ddt_bias"), ("D", "dD"),
                    ("s_in", "ds_in")):
        v = torch.randn_like(a[k])
        want = differences(lambda t: loss(**{k: t}), a[k], v)
        # a step of 1e-6 in float64: its square, and 2^-53 / 1e-6 of the terms
        assert abs((g[name] * v).sum() - want) < 1e-7 * (1 + abs(want)), name


def test_reference_scan_against_its_closed_form():
    """o_i = sum_{j<=i} exp(l_i - l_j) step_j (C_i . B_j) x_j + exp(l_i) S C_i + D x_i."""
    torch.manual_seed(1)
    B, T, H, N, P = 1, 12, 2, 4, 3
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    x, b, c, dt, al, bias, D, s = rnd(B, T, H, P), rnd(B, T, 1, N), rnd(B, T, 1, N), rnd(B, T, H), rnd(H), rnd(H), rnd(H), rnd(B, H, P, N)
    _, dtv, la = R.scan_gates(dt, al, bias, None)
    o, _ = R.scan(x, b, c, dtv, la, D, s, None)
    l = la.cumsum(1)
    for h in range(H):
        E = torch.exp(l[0, :, None, h] - l[0, None, :, h]).tril()
        M = (c[0, :, 0] @ b[0, :, 0].T) * E * dtv[0, None, :, h]
        want = M @ x[0, :, h] + torch.exp(l[0, :, h, None]) * (c[0, :, 0] @ s[0, h].T) + D[h] * x[0, :, h]
        assert (o[0, h] - want).abs().max() < 1e-12


def test_reference_convolution_against_torch():
    torch.manual_seed(2)
    B, T, C, K = 2, 11, 5, 4
    x, w, bias = (torch.randn(*s, dtype=torch.float64) for s in ((B, T, C), (C, K), (C,)))
    y, s = R.conv(x, w, bias, None, None, "none")
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (K - 1, 0)), w[:, None], bias, groups=C)
    assert (y - want.transpose(1, 2)).abs().max() < 1e-12 and torch.equal(s, x[:, T - K + 1:])
