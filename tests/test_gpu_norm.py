"""RMS norm with the residual's addition, its E4M3 form and its gradient, against
the formulas in float64.

Tolerances. u = 2^-24 is half a step of fp32. s = x + residual is rounded once;
the sum of its squares goes through at most 8 + 4 additions in a thread and 5 + 5
in the reductions, each off by u of a sum of positive numbers, and one rounding a
square: with the division by d and eps's addition at most 26 u, half of it in the
square root, and three more roundings: 16 u of rstd, 20 u of y. SLACK = 32 u covers
both. An output of type t adds half a step of t, eps(t) / 2.

Codes: the nearest E4M3 number of y / scale, off by half a step of E4M3 (a step is
2^(e - 3), at least 2^-9) plus what y, the scale and its reciprocal are off, 40 u.

Gradient. dx = d_sum + rstd (a - n m), m = mean(a n): a, n are off by 2 u of
themselves, m by at most (8 + 4 + 10 + 4) u of mean |a n|, the last three operations by
u of what they add: 8 u (|d_sum| + rstd (|a| + |n m|)) + 30 u rstd |n| mean |a n|.
dw = sum of dy n over the tokens: a group's rows one after another (152 groups or more,
or a row each), the 8 groups of a CTA, then at most 608 CTAs in 32 chains of 19, and the
32: at most N = rows of a group + 8 + 19 + 32 additions in a row, each off by u of the
sum of the magnitudes, and 3 u a term.
"""
import pytest
import torch

from mixture_experts_layer_router_gb300 import capi
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SLACK = 32 * U
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def rand(shape, seed, dtype, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def half_step(t):
    return torch.finfo(t).eps / 2


def near(got, want, dtype, slack=SLACK):
    tol = (half_step(dtype) if dtype != torch.float64 else 0.0) + slack
    d = (got.double() - want).abs()
    assert bool((d <= tol * want.abs() * (1 + 1e-3) + 1e-37).all()), float((d / want.abs().clamp(min=1e-30)).max())


def formula(x, weight, residual, eps=EPS):
    s = x.double() if residual is None else x.double() + residual.double()
    rstd = (s.square().mean(1) + eps).rsqrt()
    return s, rstd, s * rstd[:, None] * weight.double()


def check_codes(got, y, block):
    T, d = y.shape
    width = block or d
    n = -(-d // width)
    assert got["codes"].shape == (T, d) and got["codes"].dtype == torch.uint8
    assert got["scales"].shape == (T, n)
    top = torch.stack([y[:, i * width:(i + 1) * width].abs().amax(1) for i in range(n)], 1)
    want = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    near(got["scales"], want, F32)
    scale = want.repeat_interleave(width, 1)[:, :d]
    q = y / scale
    c = got["codes"].view(torch.float8_e4m3fn).double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))) / 8
    assert bool(((c - q).abs() <= step / 2 * (1 + 1e-6) + 40 * U * q.abs()).all())


# one row and several; widths of one element, a warp's row and its neighbours, the
# borders of one, two and four pieces a thread, odd ones, the widest
SIZES = [(1, 1), (3, 7), (5, 128), (128, 256), (33, 257), (4, 1000), (7, 1024), (6, 1025), (9, 2048),
         (2, 4096), (3, 4097), (5, 6656), (1, 8704), (2, 8705), (2, 16383), (2, 16384), (700, 96)]


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, F32)])
def test_norm(T, d, xt, rt):
    gh.lib()
    x = rand((T, d), 3 * T + d, xt)
    r = None if rt is None else rand((T, d), 5 * T + d, rt, 3.0)
    for wt in (BF16, F32):
        w = 1 + rand((d,), d, F32, 0.3)
        w = w.to(wt)
        s, rstd, y = formula(x, w, r)
        got = capi.rms_norm(x, w, eps=EPS, residual=r)
        assert set(got) == ({"y", "rstd"} if r is None else {"y", "rstd", "sum"})
        assert got["y"].dtype == xt
        near(got["y"], y, xt)
        near(got["rstd"], rstd, F32)
        if r is not None:
            assert torch.equal(got["sum"], (x.float() + r.float()).to(rt))
        other = F32 if xt == BF16 else BF16
        near(capi.rms_norm(x, w, eps=EPS, residual=r, y_dtype=other)["y"], y, other)
        again = capi.rms_norm(x, w, eps=EPS, residual=r)
        assert torch.equal(again["y"], got["y"]) and torch.equal(again["rstd"], got["rstd"])


@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("kind", ["token", "block"])
def test_codes(T, d, kind):
    gh.lib()
    x, w = rand((T, d), T + d, BF16), (1 + rand((d,), d, F32, 0.3)).to(BF16)
    r = rand((T, d), 7 * T + d, F32, 2.0)
    for residual in (None, r):
        _, rstd, y = formula(x, w, residual)
        got = capi.rms_norm(x, w, eps=EPS, residual=residual, quantize=kind)
        assert "y" not in got
        check_codes(got, y, 128 if kind == "block" else 0)
        near(got["rstd"], rstd, F32)
        both = capi.rms_norm(x, w, eps=EPS, residual=residual, quantize=kind, keep_y=True)
        assert torch.equal(both["codes"], got["codes"]) and torch.equal(both["scales"], got["scales"])
        near(both["y"], y, BF16)


def test_codes_of_zeros_and_nan():
    """A block of zeros has scale 1; a NaN in the weight is the NaN code and leaves the
    scale of the others alone; a row of zeros is zeros."""
    gh.lib()
    x = rand((4, 512), 1, BF16)
    x[1] = 0
    x[2, 128:256] = 0
    w = torch.ones(512, device="cuda")
    w[300] = float("nan")
    got = capi.rms_norm(x, w, quantize="block", keep_y=True)
    c = got["codes"].view(torch.float8_e4m3fn).float()
    assert torch.equal(got["scales"][1, [0, 1, 3]], torch.ones(3, device="cuda"))
    assert got["scales"][2, 1] == 1 and bool((c[2, 128:256] == 0).all())
    assert bool(c[:, 300].isnan().all()) and int(c.isnan().sum()) == 4
    _, _, y = formula(x, torch.nan_to_num(w, nan=0.0), None)
    near(got["scales"][0, 2], y[0, 256:384].abs().amax() / 448, F32)


@pytest.mark.parametrize("d", [256, 1000, 6656, 8705])
def test_magnitudes(d):
    """Squares beyond fp32 (1e25, near its end) and below it, with the rows between
    them as ever."""
    gh.lib()
    x = rand((6, d), d, F32)
    for row, f in ((0, 1e25), (2, 1e-25), (3, 1e30), (5, 1e-38)):
        x[row] *= f
    w = 1 + rand((d,), d, F32, 0.3)
    for eps in (1e-6, 1e-30):
        s, rstd, y = formula(x, w, None, eps)
        got = capi.rms_norm(x, w, eps=eps)
        near(got["rstd"], rstd, F32)
        # subnormal results have fewer bits than a relative bound asks for
        keep = y.abs() > 1e-30
        near(got["y"][keep], y[keep], F32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [200, 2048, 8704])
def test_bad_rows_stay_their_own(bad, d):
    gh.lib()
    x, w = rand((9, d), d, BF16), torch.ones(d, device="cuda")
    clean = capi.rms_norm(x, w)["y"]
    y = x.clone()
    y[4, d // 2] = bad
    got = capi.rms_norm(y, w)["y"]
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(got[keep], clean[keep])
    assert bool(got[4, d // 2].isnan())


@pytest.mark.parametrize("d", [64, 768, 2040])
def test_strides_and_places(d):
    """Rows of wider tensors, at 16-byte boundaries and off them; the sum written over
    the residual; what lies between the rows stays."""
    gh.lib()
    T = 11
    for shift, pad in ((0, 8), (8, 24), (1, 3)):
        wide = rand((T, d + shift + pad), d, BF16)
        x = wide[:, shift:shift + d]
        rw = rand((T, d + shift + pad), d + 1, F32)
        r = rw[:, shift:shift + d]
        w = (1 + rand((d,), d, F32, 0.3)).to(BF16)
        s, rstd, y = formula(x, w, r)
        before = rw.clone()
        want = capi.rms_norm(x, w, residual=r)
        assert torch.equal(rw, before)
        near(want["y"], y, BF16)
        got = capi.rms_norm(x, w, residual=r, out_sum=r, quantize="block", keep_y=True)
        assert torch.equal(got["y"], want["y"]) and torch.equal(r, want["sum"])
        before[:, shift:shift + d] = want["sum"]
        assert torch.equal(rw, before)
        check_codes(got, y, 128)


def test_stream_and_graph():
    gh.lib()
    T, d = 300, 1536
    x, r, w = rand((T, d), 1, BF16), rand((T, d), 2, F32), rand((d,), 3, F32)
    dy = rand((T, d), 4, BF16)
    want = capi.rms_norm(x, w, residual=r)
    grad = capi.rms_norm_backward(dy, want["sum"], w, want["rstd"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = capi.rms_norm(x, w, residual=r, stream=side)
    back = capi.rms_norm_backward(dy, got["sum"], w, got["rstd"], stream=side)
    side.synchronize()
    assert torch.equal(got["y"], want["y"])
    assert torch.equal(back["dx"], grad["dx"]) and torch.equal(back["dw"], grad["dw"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = capi.rms_norm(x, w, residual=r)
        held_back = capi.rms_norm_backward(dy, held["sum"], w, held["rstd"], d_sum=r)
    for seed in (5, 6):
        x.copy_(rand((T, d), seed, BF16))
        dy.copy_(rand((T, d), seed + 10, BF16))
        g.replay()
        now = capi.rms_norm(x, w, residual=r)
        now_back = capi.rms_norm_backward(dy, now["sum"], w, now["rstd"], d_sum=r)
        assert torch.equal(held["y"], now["y"]) and torch.equal(held["sum"], now["sum"])
        assert torch.equal(held_back["dx"], now_back["dx"]) and torch.equal(held_back["dw"], now_back["dw"])


def gradient(dy, s, w, rstd, d_sum):
    a, n = dy.double() * w.double(), s.double() * rstd.double()[:, None]
    m = (a * n).mean(1, keepdim=True)
    r = rstd.double()[:, None]
    dx = r * (a - n * m) + (0 if d_sum is None else d_sum.double())
    size = r * (a.abs() + (n * m).abs()) + (0 if d_sum is None else d_sum.double().abs())
    tol = 8 * U * size + 30 * U * r * n.abs() * (a * n).abs().mean(1, keepdim=True)
    return dx, tol, (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)


@pytest.mark.parametrize("T,d", SIZES + [(5000, 64), (1300, 2048), (999, 777), (640, 6656)])
@pytest.mark.parametrize("yt,st", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
def test_backward(T, d, yt, st):
    gh.lib()
    s, dy = rand((T, d), T + d, st, 2.0), rand((T, d), 2 * T + d, yt, 1e-2)
    d_sum = rand((T, d), 3 * T + d, st, 1e-2)
    rstd = (s.double().square().mean(1) + EPS).rsqrt().float()
    for wt, ds in ((BF16, None), (F32, d_sum)):
        w = (1 + rand((d,), d, F32, 0.3)).to(wt)
        dx, tol, dw, size = gradient(dy, s, w, rstd, ds)
        got = capi.rms_norm_backward(dy, s, w, rstd, d_sum=ds, dx_bf16=st == F32)
        assert got["dx"].dtype == st and got["dw"].dtype == F32
        assert bool(((got["dx"].double() - dx).abs() <= tol * (1 + half_step(st)) + half_step(st) * dx.abs()).all())
        if st == F32:
            assert torch.equal(got["dx16"], got["dx"].to(BF16))
        rows = 8 if d <= 256 else 1
        groups = max(1, min(-(-T // rows) * rows, 152))
        n = -(-T // groups) + 8 + 19 + 32 + 3
        assert bool(((got["dw"].double() - dw).abs() <= n * U * size).all())
        again = capi.rms_norm_backward(dy, s, w, rstd, d_sum=ds)
        assert torch.equal(again["dx"], got["dx"]) and torch.equal(again["dw"], got["dw"])
        alone = capi.rms_norm_backward(dy, s, w, rstd, d_sum=ds, dw=False)
        assert "dw" not in alone and torch.equal(alone["dx"], got["dx"])


def test_backward_rows_of_wider_tensors():
    gh.lib()
    T, d = 37, 520
    for shift, pad in ((8, 16), (3, 2)):
        cut = lambda seed, t: rand((T, d + shift + pad), seed, t)[:, shift:shift + d]  # noqa: E731
        s, dy, d_sum, w = cut(1, F32), cut(2, BF16), cut(3, F32), rand((d,), 4, F32)
        rstd = rand((T,), 5, F32).abs()
        got = capi.rms_norm_backward(dy, s, w, rstd, d_sum=d_sum)
        want = capi.rms_norm_backward(dy.contiguous(), s.contiguous(), w, rstd, d_sum=d_sum.contiguous())
        dx, tol, dw, size = gradient(dy, s, w, rstd, d_sum)
        assert bool(((got["dx"].double() - dx).abs() <= tol + U * dx.abs()).all())
        assert bool(((want["dw"] - got["dw"]).double().abs() <= 2 * (T + 40) * U * size).all())


def test_backward_against_differences():
    """The forward's own values (fp32 in and out) as x moves by h: central differences of
    sum(dy y) + sum(d_sum s). Truncation h^2 / 6 times a third derivative (of order
    rstd^3 |dy|, 1e-6 with h = 1e-2 and |dy| 1), rounding 2 * 32 u * sum |dy y| / h = 5e-3
    at 16 channels."""
    gh.lib()
    T, d, h = 4, 16, 1e-2
    x, w = rand((T, d), 1, F32), 1 + rand((d,), 2, F32, 0.3)
    r, dy, ds = rand((T, d), 3, F32), rand((T, d), 4, F32), rand((T, d), 5, F32)
    f = capi.rms_norm(x, w, residual=r)
    got = capi.rms_norm_backward(dy, f["sum"], w, f["rstd"], d_sum=ds)
    for c in range(d):
        up, dn = x.clone(), x.clone()
        up[:, c] += h
        dn[:, c] -= h
        diff = 0.0
        for sign, v in ((1, up), (-1, dn)):
            o = capi.rms_norm(v, w, residual=r)
            diff = diff + sign * ((dy.double() * o["y"].double()).sum(1) + (ds.double() * o["sum"].double()).sum(1))
        diff = diff / (up[:, c].double() - dn[:, c].double())
        assert bool(((got["dx"][:, c].double() - diff).abs() <= 1e-2).all())
    for c in range(d):
        up, dn = w.clone(), w.clone()
        up[c] += h
        dn[c] -= h
        diff = (dy.double() * (capi.rms_norm(x, up, residual=r)["y"].double()
                               - capi.rms_norm(x, dn, residual=r)["y"].double())).sum()
        diff = diff / (up[c].double() - dn[c].double())
        assert abs(float(got["dw"][c]) - float(diff)) <= 1e-2


def test_backward_in_place():
    """dx over d_sum or over s, through the C entry."""
    import ctypes
    lib = gh.lib()
    T, d = 50, 1280
    s, dy, d_sum, w = rand((T, d), 1, F32), rand((T, d), 2, BF16), rand((T, d), 3, F32), rand((d,), 4, F32)
    rstd = rand((T,), 5, F32).abs()
    want = capi.rms_norm_backward(dy, s, w, rstd, d_sum=d_sum)
    for over in ("s", "d_sum"):
        held = {"s": s.clone(), "d_sum": d_sum.clone()}
        dw = torch.empty(d, device="cuda")
        ws = torch.empty(lib.latentmoe_rms_norm_backward_workspace(T, d), dtype=torch.uint8, device="cuda")
        a = capi.latentmoe_norm_grad(dy=dy.data_ptr(), s=held["s"].data_ptr(), weight=w.data_ptr(),
                                     rstd=rstd.data_ptr(), d_sum=held["d_sum"].data_ptr(),
                                     dx=held[over].data_ptr(), dw=dw.data_ptr(), dy_dtype=capi.BF16,
                                     s_dtype=capi.FP32, weight_dtype=capi.FP32)
        assert lib.latentmoe_rms_norm_backward(ctypes.byref(a), T, d, ws.data_ptr(), ws.numel(),
                                               torch.cuda.current_stream().cuda_stream) == capi.OK
        assert torch.equal(held[over], want["dx"]) and torch.equal(dw, want["dw"])
