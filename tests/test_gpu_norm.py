"""The root-mean-square norm and its gradients against their formulas in float64.

Tolerances, element by element, with h the float32 step 2^-24:
 - half a step of the type for each rounding to it, and half the smallest subnormal;
 - rstd: a row's squares are all positive, so their float32 sum is off by at most h for each addition on the way to an
   element, 32 in a lane (128 in rows past 16384 columns of the sizes here), 6 in a wave, 16 between waves; the root
   halves that, and the mean, eps, root and quotient add 4: under 96 h of rstd, and n = h rstd and y under 100 h;
 - mean(dn n): its sum's additions and its factors' errors, under 300 h of mean |dn n|; so dx is off by at most
   512 h (|dh| + rstd (|dn| + |n| mean |dn n|));
 - dweight: a group of lanes adds its rows one by one (at most N / 256 of them, in rows past 16384 columns N / 64), a
   workgroup up to 32 groups' sums, a column's thread up to 64 workgroups' and then 16 threads': under
   (N / 256 + 256) h of sum |dy n|.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
STEP = 2.0 ** -24


def half(t, dt):
    return t.abs() * (torch.finfo(dt).eps / 2) + TINY[dt]


def close(got, ref, tol, what):
    assert got is not None and tuple(got.shape) == tuple(ref.shape), what
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err.max()), float((err / tol.clamp_min(1e-300)).max()))


def randn(*shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def check(N, H, dt, residual=True, weight=True, dh=True, eps=1e-6, scale=1.0, seed=0):
    x = randn(N, H, dt=dt, seed=seed, scale=scale)
    res = randn(N, H, dt=dt, seed=seed + 1, scale=scale) if residual else None
    w = (1 + randn(H, dt=torch.float32, seed=seed + 2, scale=0.2)).to(dt) if weight else None
    y, h, rstd = L.flce_rms_norm_forward(x, w, res, eps=eps, keep=True)
    h64 = x.double() + (res.double() if residual else 0)
    r64 = (h64.square().mean(1, keepdim=True) + eps).rsqrt()
    w64 = w.double() if weight else torch.ones(H, dtype=torch.float64, device="cuda")
    y64 = h64 * r64 * w64
    # the sum of two 16-bit numbers is rounded to float32 on its way
    close(h, h64, half(h64, dt) + STEP * h64.abs(), "h")
    close(y, y64, half(y64, dt) + 101 * STEP * y64.abs(), "y")
    close(rstd, r64[:, 0], 96 * STEP * r64[:, 0], "rstd")
    if not residual:
        assert h is x
    # gradients: of the rounded h that the backward is given
    dy = randn(N, H, dt=dt, seed=seed + 3, scale=0.1)
    g = randn(N, H, dt=dt, seed=seed + 4, scale=0.1) if dh else None
    dx, dw = L.flce_rms_norm_backward(h, w, rstd, dy, g)
    # rstd is that of h before its rounding: taken as it is given
    hh, rr = h.double(), rstd.double()[:, None]
    n, dn = hh * rr, dy.double() * w64
    dot = (dn * n).mean(1, keepdim=True)
    dx64 = rr * (dn - n * dot) + (g.double() if dh else 0)
    mag = rr * (dn.abs() + n.abs() * (dn * n).abs().mean(1, keepdim=True)) + (g.double().abs() if dh else 0)
    close(dx, dx64, half(dx64, dt) + 512 * STEP * mag, "dx")
    dw64 = (dy.double() * n).sum(0)
    rows = math.ceil(N / 64) if H > 16384 else math.ceil(N / 256)
    close(dw, dw64, half(dw64, dt) + (rows + 256) * STEP * (dy.double() * n).abs().sum(0), "dweight")
    return x, res, w, y, h, rstd, dy, g, dx, dw


# one column; less than, exactly and just past each number of lanes and runs
SHAPES = [(1, 1), (3, 7), (1, 64), (70, 64), (5, 65), (9, 511), (4, 512), (6, 513), (130, 1000), (2, 1024), (3, 1025),
          (17, 2047), (2, 2048), (2, 2056), (33, 4096), (5, 4099), (2, 8192), (3, 8200), (2, 16383), (3, 16384),
          (2, 16392), (3, 20001), (600, 40), (2100, 264), (1, 4096)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    check(*shape, DT[dtype])
    check(*shape, DT[dtype], residual=False, weight=False, dh=False, seed=9)


@pytest.mark.parametrize("dtype", list(DT))
def test_scales_of_the_inputs(dtype):
    for scale in (1e-3, 30.0):
        check(40, 300, DT[dtype], scale=scale)
    check(8, 128, DT[dtype], eps=0.0)


def test_many_rows_in_every_group():
    # more rows than a launch has groups: dweight's groups and the forward's workgroups walk several
    check(20_011, 72, torch.float32)
    check(9001, 1500, torch.bfloat16)


def test_zero_rows_and_infinite_ones():
    x = torch.zeros(4, 100, device="cuda")
    y, _, rstd = L.flce_rms_norm_forward(x, eps=1e-6, keep=True)
    assert not bool(y.any()) and torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)
    dx, dw = L.flce_rms_norm_backward(x, None, rstd, torch.ones_like(x))
    assert torch.allclose(dx, torch.full_like(dx, 1e3), rtol=1e-6) and not bool(dw.any())
    # as the formula has it: infinity times 0
    x[1, 5] = math.inf
    x[2, 7] = math.nan
    y, _, _ = L.flce_rms_norm_forward(x, eps=1e-6)
    assert bool(y[1, 5].isnan()) and not bool(y[1, :5].any()) and bool(y[2].isnan().all()) and not bool(y[3].any())


@pytest.mark.parametrize("dtype", list(DT))
def test_no_rows(dtype):
    x = torch.empty(0, 48, dtype=DT[dtype], device="cuda")
    y, h, rstd = L.flce_rms_norm_forward(x, keep=True)
    assert y.shape == (0, 48) and rstd.shape == (0,)
    dx, dw = L.flce_rms_norm_backward(h, None, rstd, x)
    assert dx.shape == (0, 48) and dw.shape == (48,) and not bool(dw.any())
    q, _ = L.flce_rms_norm_mx_forward(x)
    assert q.codes.shape == (0, 128)


def test_no_long_rows_have_a_weight_gradient_of_zero():
    x = torch.empty(0, 20000, device="cuda")
    dx, dw = L.flce_rms_norm_backward(x, None, torch.empty(0, device="cuda"), x)
    assert dx.shape == (0, 20000) and dw.shape == (20000,) and not bool(dw.any())


def test_strided_and_unaligned_inputs():
    dt, N, H = torch.bfloat16, 37, 200
    base = randn(N, 3 * H + 1, dt=dt, seed=1)
    x, res = base[:, 1:H + 1], base[:, H + 1:2 * H + 1]
    w = randn(2 * H, dt=dt, seed=2)[1::2]
    a = L.flce_rms_norm_forward(x, w, res, keep=True)
    b = L.flce_rms_norm_forward(x.clone(), w.clone(), res.clone(), keep=True)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    dy = randn(H, N, dt=dt, seed=3).T
    p = L.flce_rms_norm_backward(a[1], w, a[2], dy, x)
    q = L.flce_rms_norm_backward(a[1], w.clone(), a[2], dy.contiguous(), x.clone())
    assert all(torch.equal(s, t) for s, t in zip(p, q))


def test_weight_at_any_element():
    w = randn(4099, dt=torch.bfloat16, seed=2)
    x = randn(5, 4096, dt=torch.bfloat16, seed=1)
    for o in (1, 3):
        a, b = L.flce_rms_norm_forward(x, w[o:o + 4096])[0], L.flce_rms_norm_forward(x, w[o:o + 4096].clone())[0]
        assert torch.equal(a, b)


@pytest.mark.parametrize("H", [72, 4096, 16400])
def test_in_place(H):
    from lm_head_cross_flce_amd import _lib
    N = 50
    x, r, dy, g = (randn(N, H, dt=torch.bfloat16, seed=i) for i in range(4))
    y, h, rstd = L.flce_rms_norm_forward(x, None, r, keep=True)
    stream = torch.cuda.current_stream().cuda_stream
    for into in (0, 1):
        a, b, out = x.clone(), r.clone(), torch.empty_like(x)
        _lib.flce_rms_norm_forward(a.data_ptr(), b.data_ptr(), None, N, H, 1, 1e-6, out.data_ptr(),
                                   (a, b)[into].data_ptr(), None, stream)
        assert torch.equal((a, b)[into], h) and torch.equal(out, y)
    dx, dw = L.flce_rms_norm_backward(h, None, rstd, dy, g)
    ws = torch.empty(L.flce_rms_norm_workspace_size(N, H, x.dtype), dtype=torch.uint8, device="cuda")
    for into in (0, 1):
        a, b, dw2 = dy.clone(), g.clone(), torch.empty_like(dw)
        last = None if into == 0 and H > 16384 else dw2.data_ptr()
        _lib.flce_rms_norm_backward(h.data_ptr(), None, rstd.data_ptr(), a.data_ptr(), b.data_ptr(), N, H, 1,
                                    (a, b)[into].data_ptr(), last, ws.data_ptr(), ws.numel(), stream)
        assert torch.equal((a, b)[into], dx) and (last is None or torch.equal(dw2, dw))
    # x and the residual are one tensor
    _lib.flce_rms_norm_forward(x.data_ptr(), x.data_ptr(), None, N, H, 1, 1e-6, out.data_ptr(), x.data_ptr(), None, stream)
    assert x.isfinite().all()


@pytest.mark.parametrize("N,H", [(5, 33), (3, 4096), (2, 20001)])
@pytest.mark.parametrize("dtype", list(DT))
def test_nothing_is_written_outside_the_outputs(N, H, dtype):
    from lm_head_cross_flce_amd import _lib
    dt = DT[dtype]
    x, r, dy = (randn(N, H, dt=dt, seed=i) for i in range(3))
    code = _lib.FLCE_BF16 if dtype == "bf16" else _lib.FLCE_F16 if dtype == "f16" else _lib.FLCE_F32
    pad = 64
    bufs = [torch.full((N * H + 2 * pad,), 7.0, dtype=dt, device="cuda") for _ in range(3)]
    y, h, dx = (b[pad:pad + N * H] for b in bufs)
    rb = torch.full((N + 2 * pad,), 7.0, device="cuda")
    wb = torch.full((H + 2 * pad,), 7.0, dtype=dt, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    _lib.flce_rms_norm_forward(x.data_ptr(), r.data_ptr(), None, N, H, code, 1e-6, y.data_ptr(), h.data_ptr(),
                               rb[pad:].data_ptr(), stream)
    ws = torch.empty(_lib.flce_rms_norm_workspace_size(N, H, code) + 256, dtype=torch.uint8, device="cuda").fill_(7)
    _lib.flce_rms_norm_backward(h.data_ptr(), None, rb[pad:].data_ptr(), dy.data_ptr(), None, N, H, code, dx.data_ptr(),
                                wb[pad:].data_ptr(), ws.data_ptr(), ws.numel() - 256, stream)
    for b, n in [(b, N * H) for b in bufs] + [(rb, N), (wb, H)]:
        assert bool((b[:pad] == 7).all()) and bool((b[pad + n:] == 7).all())
    assert bool((ws[-256:] == 7).all())
    padded = (H + 127) // 128 * 128
    for fmt, per in (("e4m3", 1), ("e2m1", 2)):
        codes = torch.full((N * padded // per + 2 * pad,), 7, dtype=torch.uint8, device="cuda")
        scales = torch.full((N * padded // 32 + 2 * pad,), 7, dtype=torch.uint8, device="cuda")
        _lib.flce_rms_norm_mx_forward(x.data_ptr(), r.data_ptr(), None, N, H, code, 1e-6, _lib.MX_FORMATS[fmt],
                                      codes[pad:].data_ptr(), scales[pad:].data_ptr(), h.data_ptr(), None, stream)
        for b, n in ((codes, N * padded // per), (scales, N * padded // 32)):
            assert bool((b[:pad] == 7).all()) and bool((b[pad + n:] == 7).all())


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("N,H", [(1, 1), (7, 100), (3, 512), (9, 1000), (5, 4096), (4, 9000), (2, 20001)])
@pytest.mark.parametrize("dtype", list(DT))
def test_microscaled_output(N, H, dtype, fmt):
    # The same rows as a float32 y, quantised: that y is within 101 steps of the formula's, so an element or a scale
    # may fall to either side of a border it is that near to; all others are equal.
    dt = DT[dtype]
    x, r = randn(N, H, dt=dt, seed=1), randn(N, H, dt=dt, seed=2)
    w = (1 + randn(H, dt=torch.float32, seed=3, scale=0.2)).to(dt)
    q, h = L.flce_rms_norm_mx_forward(x, w, r, format=fmt)
    y, _, _ = L.flce_rms_norm_forward(x.float(), w.float(), r.float())
    ref = L.flce_mx_quantize(y, fmt)
    assert torch.equal(h, L.flce_rms_norm_forward(x, w, r)[1])
    a, b = L.flce_mx_dequantize(q, torch.float32), L.flce_mx_dequantize(ref, torch.float32)
    step = {"e4m3": 2.0 ** -3, "e2m1": 0.5}[fmt]
    assert torch.equal(q.scales, ref.scales) or int((q.scales != ref.scales).sum()) <= 1 + q.scales.numel() // 10_000
    assert bool(((a - b).abs() <= step * b.abs().amax().clamp_min(1e-30)).all())
    assert int((a != b).sum()) <= 1 + a.numel() // 1000
    if H % 128:   # zeros past the columns
        per = 2 if fmt == "e2m1" else 1
        assert not bool(q.codes[:, (H + per - 1) // per:].any())
        assert not bool(q.scales[:, (H + 31) // 32:].any())


def test_rows_a_mask_left_empty_are_zeros_in_8_bits():
    x = torch.zeros(3, 200, device="cuda", dtype=torch.bfloat16)
    x[1] = 1
    for eps in (1e-6, 0.0):
        q, _ = L.flce_rms_norm_mx_forward(x, eps=eps)
        v = L.flce_mx_dequantize(q)
        # 1 / sqrt(1 + 1e-6) = 0.9999995 lies under 1, so its block's scale is 2^(-1 - 8), and 0.9999995 2^9 = 511.9997 is
        # held to 448, which stands for 0.875
        assert bool((v[1] == (0.875 if eps else 1.0)).all())
        if eps:
            assert not bool(v[0].any()) and not bool(q.scales[0].any())
        else:
            assert bool(v[0].isnan().all())   # 0 times the reciprocal of 0, as the formula has it
            assert not bool(q.codes[:, 200:].any())


def test_requested_gradients_only():
    x, dy = randn(30, 100, dt=torch.float32, seed=1), randn(30, 100, dt=torch.float32, seed=2)
    _, h, rstd = L.flce_rms_norm_forward(x, keep=True)
    dx, dw = L.flce_rms_norm_backward(h, None, rstd, dy)
    a, none = L.flce_rms_norm_backward(h, None, rstd, dy, need_dweight=False)
    assert none is None and torch.equal(a, dx)
    none, b = L.flce_rms_norm_backward(h, None, rstd, dy, need_dx=False)
    assert none is None and torch.equal(b, dw)
    assert L.flce_rms_norm_backward(h, None, rstd, dy, need_dx=False, need_dweight=False) == (None, None)


def test_results_repeat_bit_for_bit():
    args = [randn(3000, 1000, dt=torch.bfloat16, seed=i) for i in range(4)]
    w = randn(1000, dt=torch.bfloat16, seed=9)

    def call():
        y, h, rstd = L.flce_rms_norm_forward(args[0], w, args[1], keep=True)
        return (y, h, rstd, *L.flce_rms_norm_backward(h, w, rstd, args[2], args[3]))

    ref = call()
    for _ in range(3):
        assert all(torch.equal(s, t) for s, t in zip(ref, call()))


def test_autograd_against_differences():
    # the directional derivative of a weighted sum of both outputs, against central differences of the formula in float64
    N, H = 6, 50
    x, r, cy, ch = (randn(N, H, dt=torch.float32, seed=i) for i in range(4))
    w = randn(H, dt=torch.float32, seed=5)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, r)]
    y, h = L.fused_rms_norm(leaves[0], leaves[1], leaves[2])
    ((y * cy).sum() + (h * ch).sum()).backward()
    assert torch.equal(leaves[0].grad, leaves[2].grad)

    def f(x, w, r):
        h = x + r
        return float(((h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w * cy.double()) + h * ch.double()).sum())

    for i, leaf in enumerate(leaves):
        d = torch.randn(leaf.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(i)).cuda()
        at = [t.double() for t in (x, w, r)]
        e = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + e * d, at[i] - e * d
        diff = (f(*up) - f(*down)) / (2 * e)
        got = float((leaf.grad.double() * d).sum())
        # float32 gradients: 512 steps of the terms' sizes, over 300 terms; differences: e^2 and 2^-53 / e
        assert abs(got - diff) <= 1e-3 * max(1.0, abs(diff)), (i, got, diff)


def test_autograd_keeps_what_is_needed():
    x = randn(2, 3, 64, dt=torch.bfloat16, seed=1).requires_grad_(True)
    norm = L.RMSNorm(64, device="cuda", dtype=torch.bfloat16)
    y = norm(x)
    assert y.shape == x.shape
    y.sum().backward()
    assert x.grad is not None and norm.weight.grad is not None
    # only the residual sum goes on
    x.grad = norm.weight.grad = None
    r = randn(2, 3, 64, dt=torch.bfloat16, seed=2).requires_grad_(True)
    y, h = norm(x, r)
    h.sum().backward()
    assert bool((x.grad == 1).all()) and bool((r.grad == 1).all()) and not bool(norm.weight.grad.any())
    # frozen weight, and no gradients at all
    x.grad = None
    norm.weight.requires_grad_(False)
    norm(x).sum().backward()
    assert x.grad is not None
    with torch.no_grad():
        assert norm(x).grad_fn is None
    with torch.inference_mode():
        norm(x)


@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64)])
def test_gradients_of_x_and_the_residual_share_no_memory(shape):
    x, r = (randn(*shape, dt=torch.float32, seed=i).requires_grad_(True) for i in (1, 2))
    y, h = L.fused_rms_norm(x, None, r)
    (y.sum() + h.sum()).backward()
    assert torch.equal(x.grad, r.grad) and x.grad.data_ptr() != r.grad.data_ptr()
    x.grad.zero_()
    assert bool(r.grad.any())


def test_on_another_stream_and_two_at_once():
    args = [(randn(300 + 37 * i, 1024, dt=torch.bfloat16, seed=i), randn(1024, dt=torch.bfloat16, seed=9),
             randn(300 + 37 * i, 1024, dt=torch.bfloat16, seed=20 + i)) for i in range(4)]

    def call(x, w, dy):
        y, h, rstd = L.flce_rms_norm_forward(x, w, x, keep=True)
        return (y, h, *L.flce_rms_norm_backward(h, w, rstd, dy, x))

    ref = [call(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(call(*a))
        torch.cuda.synchronize()
        for r, g in zip(ref, got):
            assert all(torch.equal(p, q) for p, q in zip(r, g))


def test_graph_replays():
    x, r, dy = (randn(200, 520, dt=torch.bfloat16, seed=i) for i in range(3))
    w = randn(520, dt=torch.bfloat16, seed=4)

    def call():
        y, h, rstd = L.flce_rms_norm_forward(x, w, r, keep=True)
        return (y, h, *L.flce_rms_norm_backward(h, w, rstd, dy, r))

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in range(4):
        for t in (x, r, dy):
            t.copy_(randn(200, 520, dt=torch.bfloat16, seed=50 + 3 * i))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call()))


def test_offsets_past_32_bits():
    # 2.2e9 elements, 4.4 GB a tensor
    N, H = 2_200_003, 1000
    x = torch.zeros(N, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, 1_073_741, 1_073_742, 2_147_483, 2_147_484, 2_147_485, N - 1], device="cuda")
    x[rows] = randn(len(rows), H, dt=torch.bfloat16, seed=1)
    y, h, rstd = L.flce_rms_norm_forward(x, keep=True)
    ref, _, r2 = L.flce_rms_norm_forward(x[rows], keep=True)
    assert torch.equal(y[rows], ref) and torch.equal(rstd[rows], r2)
    del y
    dy = torch.zeros_like(x)
    dy[rows] = randn(len(rows), H, dt=torch.bfloat16, seed=2)
    dx, dw = L.flce_rms_norm_backward(h, None, rstd, dy)
    rx, _ = L.flce_rms_norm_backward(x[rows], None, r2, dy[rows])
    assert torch.equal(dx[rows], rx)
    dw64 = (dy[rows].double() * x[rows].double() * r2.double()[:, None]).sum(0)
    close(dw, dw64, half(dw64, torch.bfloat16) + 512 * STEP * (dy[rows].double() * x[rows].double()).abs().sum(0), "dweight")
    q, _ = L.flce_rms_norm_mx_forward(x)
    assert torch.equal(q.codes[rows], L.flce_rms_norm_mx_forward(x[rows])[0].codes)
