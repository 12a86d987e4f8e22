"""The linear layer and the gated product against their formulas in float64.

Tolerances, element by element, from the number formats:
 - eps/2 of the type (bf16 2^-8 / 2 .. = finfo.eps / 2) for each rounding to it,
   plus half the smallest subnormal;
 - a sum of K products in fp32: at most 8 sqrt(K) 2^-24 sum |a b| (each of the
   K additions rounds by at most 2^-24 of a partial sum no larger than
   sum |a b|, independently: 8 standard deviations are far beyond what a test
   of this size meets);
 - the activation: relative 1e-5 (16-bit: hardware exp2 and reciprocal, the
   normal distribution function to 8.7e-6) or 2e-6 (fp32);
 - act' and act'' are at most 1.13 and 1 for every activation here, ReLU's jump
   at 0 apart, which moves dz by dy where |z| is within z's own error.
Rounded intermediates (dz) enter a product as
independent errors e_k, so the product is off by at most 6 sqrt(sum (e_k w_k)^2).
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = tuple(_lib.ACTIVATIONS)
# smallest subnormal's half: what a rounding may lose near zero
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def act64(name):
    fn = torch.nn.functional
    return {"none": lambda z: z, "relu": torch.relu, "gelu": fn.gelu, "gelu_tanh": lambda z: fn.gelu(z, approximate="tanh"),
            "silu": fn.silu, "sigmoid": torch.sigmoid}[name]


def dact64(name, z):
    z = z.detach().clone().requires_grad_(True)
    act64(name)(z).sum().backward()
    return z.grad


def half(t, dt):
    """Half a step of dt at t's values."""
    return t.abs() * (torch.finfo(dt).eps / 2) + TINY[dt]


def act_err(dt):
    return 2e-6 if dt == torch.float32 else 1e-5


def sum_err(a, b):
    """Rounding of a @ b summed in fp32."""
    return 8 * math.sqrt(max(a.shape[1], 1)) * 2.0 ** -24 * (a.abs() @ b.abs())


def close(got, ref, tol, what):
    assert got is not None and tuple(got.shape) == tuple(ref.shape), what
    if ref.numel() == 0:
        return
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err.max()),
                                 float((err / tol.clamp_min(1e-300)).max()))


def randn(*shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


def z_with_err(x, W, b):
    """x W^T + b in float64 and the bound on its fp32 value."""
    x, W = x.double(), W.double()
    z, e = x @ W.T, sum_err(x, W.T)
    if b is not None:
        z = z + b.double()
        e = e + z.abs() * 2.0 ** -24
    return z, e


def product_tol(a, ea, b, ref, dt):
    """a @ b with a's entries off by ea, rounded to dt."""
    return 6 * ((ea ** 2) @ (b ** 2)).sqrt() + sum_err(a, b) + half(ref, dt)


def relu_flip(act, z, ez, mag):
    return torch.where(z.abs() <= ez, mag, torch.zeros_like(mag)) if act == "relu" else 0.0


def check_linear(N, H, F, dt, act, bias, residual, seed=0):
    x, W = randn(N, H, dt=dt, seed=seed), randn(F, H, dt=dt, seed=seed + 1, scale=H ** -0.5)
    b = randn(F, dt=dt, seed=seed + 2) if bias else None
    r = randn(N, F, dt=dt, seed=seed + 3) if residual else None
    dy = randn(N, F, dt=dt, seed=seed + 4)
    y, z = L.flce_linear_forward(x, W, b, r, act, keep=True)
    z64, ez = z_with_err(x, W, b)
    a64 = act64(act)(z64)
    y64 = a64 + r.double() if residual else a64
    ea = 1.13 * ez + act_err(dt) * a64.abs() * (act != "none") + 2.0 ** -24 * y64.abs()
    close(y, y64, ea + half(y64, dt), "y")
    assert (z is None) == (act == "none")
    ez_kept = ez
    if z is not None:
        assert z.dtype == torch.float32
        close(z, z64, ez + half(z64, torch.float32), "z")
        ez_kept = ez + half(z64, torch.float32)
    y2, z2 = L.flce_linear_forward(x, W, b, r, act)
    assert z2 is None and torch.equal(y, y2)
    dx, dW, db = L.flce_linear_backward(x, W, dy, z, act, need_db=True)
    d64 = dy.double()
    dz64 = d64 * dact64(act, z64)
    edz = torch.zeros_like(dz64) if act == "none" else (
        d64.abs() * ez_kept + 4 * act_err(dt) * d64.abs() + half(dz64, dt) + relu_flip(act, z64, ez_kept, d64.abs()))
    x64, W64 = x.double(), W.double()
    dx64, dW64, db64 = dz64 @ W64, dz64.T @ x64, dz64.sum(0)
    close(dx, dx64, product_tol(dz64, edz, W64, dx64, dt), "dx")
    close(dW, dW64, product_tol(dz64.T, edz.T, x64, dW64, dt), "dW")
    ones = torch.ones(N, 1, dtype=torch.float64, device="cuda")
    close(db, db64, product_tol(dz64.T, edz.T, ones, db64[:, None], dt)[:, 0], "db")


def check_glu(N, H, F, dt, act, bias, seed=0):
    x = randn(N, H, dt=dt, seed=seed)
    Wg, Wu = (randn(F, H, dt=dt, seed=seed + 1 + i, scale=H ** -0.5) for i in range(2))
    bg, bu = (randn(F, dt=dt, seed=seed + 3 + i) if bias else None for i in range(2))
    dh = randn(N, F, dt=dt, seed=seed + 5)
    h, g, u = L.flce_glu_forward(x, Wg, Wu, bg, bu, act, keep=True)
    g64, eg = z_with_err(x, Wg, bg)
    u64, eu = z_with_err(x, Wu, bu)
    a64 = act64(act)(g64)
    h64 = a64 * u64
    e_a = 1.13 * eg + act_err(dt) * a64.abs()
    close(h, h64, e_a * (u64.abs() + eu) + a64.abs() * eu + 2.0 ** -24 * h64.abs() + half(h64, dt), "h")
    close(g, g64, eg + half(g64, torch.float32), "g")
    close(u, u64, eu + half(u64, torch.float32), "u")
    h2, g2, u2 = L.flce_glu_forward(x, Wg, Wu, bg, bu, act)
    assert g2 is None and u2 is None and torch.equal(h, h2)
    dx, dWg, dWu, dbg, dbu = L.flce_glu_backward(x, Wg, Wu, g, u, dh, act, need_db=True)
    eg, eu = eg + half(g64, torch.float32), eu + half(u64, torch.float32)
    d64, da64 = dh.double(), dact64(act, g64)
    dg64, du64 = d64 * u64 * da64, d64 * a64
    edg = d64.abs() * (eu * 1.13 + (u64.abs() + eu) * (eg + 4 * act_err(dt))) + half(dg64, dt) + relu_flip(
        act, g64, eg, d64.abs() * (u64.abs() + eu))
    edu = d64.abs() * (1.13 * eg + act_err(dt) * a64.abs()) + half(du64, dt)
    x64 = x.double()
    Wgu = torch.cat([Wg.double(), Wu.double()])
    dz64, edz = torch.cat([dg64, du64], 1), torch.cat([edg, edu], 1)
    dx64 = dz64 @ Wgu
    close(dx, dx64, product_tol(dz64, edz, Wgu, dx64, dt), "dx")
    ones = torch.ones(N, 1, dtype=torch.float64, device="cuda")
    for name, dW, db, d, e in (("g", dWg, dbg, dg64, edg), ("u", dWu, dbu, du64, edu)):
        ref, refb = d.T @ x64, d.sum(0)
        close(dW, ref, product_tol(d.T, e.T, x64, ref, dt), "dW" + name)
        close(db, refb, product_tol(d.T, e.T, ones, refb[:, None], dt)[:, 0], "db" + name)


# N on both sides of every tile and of the few-token kernels; F odd, under one
# 16-byte piece, across tiles; H down to one piece; long K that is split
# (forward: H; dx: F; dW: N).
SHAPES = [
    (1, 8, 1), (1, 64, 16), (2, 4096, 37), (15, 72, 40), (16, 136, 17), (17, 264, 24), (32, 40, 129), (33, 512, 50),
    (63, 264, 100), (64, 520, 15), (65, 520, 100), (128, 200, 72), (129, 64, 257), (255, 128, 128), (256, 256, 256),
    (257, 264, 300), (300, 1032, 515), (700, 72, 1000), (70, 4096, 256), (100, 64, 4104), (5000, 64, 72),
    (1030, 512, 640),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(shape, dtype):
    i = SHAPES.index(shape)
    check_linear(*shape, DT[dtype], ACTS[i % 6], bias=i % 2 == 0, residual=i % 3 == 0, seed=i)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_glu_shapes(shape, dtype):
    i = SHAPES.index(shape)
    check_glu(*shape, DT[dtype], ACTS[(i + 4) % 6], bias=i % 2 == 1, seed=i)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [5, 300])
def test_every_activation(act, dtype, N):
    # tiles that need no split (their own epilogue) as well as few tokens
    check_linear(N, 72, 2600, DT[dtype], act, True, True, seed=7)
    check_glu(N, 72, 1400, DT[dtype], act, True, seed=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_whole_grid_of_tiles(dtype):
    # more output tiles than workgroups: each takes several
    check_linear(1100, 64, 16400, DT[dtype], "silu", True, True, seed=9)
    check_glu(2100, 64, 4200, DT[dtype], "silu", False, seed=10)


TILED = [(65, 72, 40), (70, 4096, 256), (257, 264, 300), (300, 1032, 515), (700, 72, 1000), (100, 64, 4104),
         (5000, 64, 72), (1030, 512, 640)]


@pytest.mark.parametrize("tile", [8, 4, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", TILED, ids=str)
def test_every_tile(monkeypatch, shape, dtype, tile):
    # each size of output tile on shapes that the library may give another
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", str(tile))
    i = TILED.index(shape)
    check_linear(*shape, DT[dtype], ACTS[(i + 2) % 6], bias=i % 2 == 0, residual=i % 3 == 0, seed=i)
    check_glu(*shape, DT[dtype], ACTS[(i + 3) % 6], bias=i % 2 == 1, seed=i)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8, 1), (3, 4096, 37), (9, 1032, 100), (16, 72, 515), (5, 12288, 16)], ids=str)
def test_few_tokens(monkeypatch, shape, dtype):
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", "1")
    i = shape[0]
    check_linear(*shape, DT[dtype], ACTS[i % 6], bias=i % 2 == 0, residual=True, seed=i)
    check_glu(*shape, DT[dtype], ACTS[(i + 3) % 6], bias=i % 2 == 1, seed=i)


def extreme(dt):
    big = float(torch.finfo(dt).max)
    return [0.0, -0.0, 1e-6, -1e-6, 1.0, -1.0, 20.0, -20.0, 21.0, -21.0, 90.0, -90.0, 3e4, -3e4, big, -big, math.inf,
            -math.inf, math.nan]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [4, 300])
def test_values_at_the_ends_of_the_range(act, dtype, N):
    # x W^T + b with x = 0: z is the bias, so the activation sees the listed values themselves
    dt = DT[dtype]
    vals = extreme(dt)
    b = torch.tensor(vals, dtype=dt, device="cuda")
    F = len(vals)
    x, W = torch.zeros(N, 8, dtype=dt, device="cuda"), torch.zeros(F, 8, dtype=dt, device="cuda")
    y, z = L.flce_linear_forward(x, W, b, None, act, keep=True)
    ref = act64(act)(b.float()).to(dt)   # float32's own limits: silu(-inf) is NaN there too
    assert torch.equal(torch.isnan(y[0]), torch.isnan(ref)), (y[0], ref)
    ok = torch.isfinite(ref)
    # 0.01 absolute: silu(-90) and the like, whose fp16 and bf16 neighbours are 0
    assert bool(((y[0].double() - ref.double()).abs()[ok] <= 1e-5 + ref.double().abs()[ok] * 2.0 ** -7).all())
    assert torch.equal(y, y[:1].expand_as(y)) or bool(torch.isnan(ref).any())
    if z is not None:
        assert torch.equal(z[0].nan_to_num(7.0), b.float().nan_to_num(7.0))
        fin = torch.isfinite(b)
        dy = torch.ones(N, F, dtype=dt, device="cuda")
        _, _, db = L.flce_linear_backward(x, W, dy, z, act, need_db=True)
        d64 = dact64(act, b[fin].float()).double() * N
        # gelu's and silu's own derivative is 0 * inf = NaN in float32 at the ends of the range, its limit here
        d64 = torch.where(torch.isnan(d64), (b[fin] > 0).double() * N, d64)
        # 0.01: an absolute allowance for the tails of the derivatives
        assert bool(((db[fin].double() - d64).abs() <= 0.01 * N * 2.0 ** -7 + d64.abs() * 2.0 ** -7).all()), (db[fin], d64)


def test_relu_keeps_infinite_gradients_apart():
    x = torch.zeros(3, 8, device="cuda")
    W = torch.zeros(2, 8, device="cuda")
    b = torch.tensor([-1.0, 1.0], device="cuda")
    _, z = L.flce_linear_forward(x, W, b, None, "relu", keep=True)
    _, _, db = L.flce_linear_backward(x, W, torch.full((3, 2), math.inf, device="cuda"), z, "relu", need_db=True)
    assert db[0].item() == 0.0 and db[1].item() == math.inf


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    dt = DT[dtype]
    x, W = torch.zeros(0, 24, dtype=dt, device="cuda"), torch.ones(10, 24, dtype=dt, device="cuda")
    y, z = L.flce_linear_forward(x, W, W[:, 0].contiguous(), None, "silu", keep=True)
    assert y.shape == (0, 10) and z.shape == (0, 10)
    dx, dW, db = L.flce_linear_backward(x, W, y, z, "silu", need_db=True)
    assert dx.shape == (0, 24) and not dW.any() and not db.any()
    h, g, u = L.flce_glu_forward(x, W, W, keep=True)
    assert h.shape == (0, 10)
    out = L.flce_glu_backward(x, W, W, g, u, h, need_db=True)
    assert out[0].shape == (0, 24) and not any(bool(t.any()) for t in out[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 13, 21), (16, 1001, 8), (300, 75, 333), (130, 2049, 70), (600, 7, 900)],
                         ids=str)
def test_hidden_sizes_that_are_no_whole_pieces(shape, dtype):
    check_linear(*shape, DT[dtype], "gelu", True, True)
    check_glu(*shape, DT[dtype], "silu", True)


@pytest.mark.parametrize("tile", [8, 4, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_odd_hidden_size_in_every_tile(monkeypatch, dtype, tile):
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", str(tile))
    check_linear(270, 301, 275, DT[dtype], "silu", True, True)
    check_glu(270, 301, 275, DT[dtype], "silu", True)


@pytest.mark.parametrize("N", [9, 200, 600])
def test_strided_and_unaligned_inputs(N):
    H, F = 64, 48
    x, W, r = randn(N, H, dt=torch.bfloat16, seed=1), randn(F, H, dt=torch.bfloat16, seed=2), randn(
        N, F, dt=torch.bfloat16, seed=3)
    ref, _ = L.flce_linear_forward(x, W, None, r, "silu")

    def odd(t):   # the same values, transposed in memory and off a 16-byte boundary
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
        v = buf[1:].view(t.shape[1], t.shape[0]).T
        v.copy_(t)
        return v

    y, _ = L.flce_linear_forward(odd(x), odd(W), None, odd(r), "silu")
    assert torch.equal(y, ref)
    flat = torch.empty(N * H + 1, dtype=x.dtype, device="cuda")[1:].view(N, H).copy_(x)
    assert flat.data_ptr() % 16 != 0
    assert torch.equal(L.flce_linear_forward(flat, W, None, r, "silu")[0], ref)
    big = torch.empty(2 * N, 3 * H, dtype=x.dtype, device="cuda")
    big[::2, H:2 * H] = x
    assert torch.equal(L.flce_linear_forward(big[::2, H:2 * H], W, None, r, "silu")[0], ref)
    bias = torch.empty(F + 1, dtype=x.dtype, device="cuda").normal_()[1:]   # biases need no more than their element's
    assert torch.equal(L.flce_linear_forward(x, W, bias, r, "silu")[0],
                       L.flce_linear_forward(x, W, bias.clone(), r, "silu")[0])
    dy = torch.ones((), dtype=x.dtype, device="cuda").expand(N, F)   # as a sum's backward gives it
    a = L.flce_linear_backward(x, W, dy, need_db=True)
    b = L.flce_linear_backward(x, W, dy.contiguous(), need_db=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("N", [9, 200, 2000])
def test_residual_in_place(N):
    x, W, r = randn(N, 512, dt=torch.bfloat16, seed=1), randn(72, 512, dt=torch.bfloat16, seed=2), randn(
        N, 72, dt=torch.bfloat16, seed=3)
    ref, _ = L.flce_linear_forward(x, W, None, r)
    y, _ = L.flce_linear_forward(x, W, None, r, out=r)
    assert y is r and torch.equal(r, ref)
    with pytest.raises(ValueError):
        L.flce_linear_forward(x, W, None, None, out=torch.empty(72, N, dtype=r.dtype, device="cuda").T)


@pytest.mark.parametrize("N,H,F", [(7, 64, 33), (70, 1024, 72), (300, 64, 333), (7, 61, 33), (300, 1027, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_is_written_outside_the_outputs(N, H, F, dtype):
    # outputs and workspaces inside larger buffers of a known pattern
    dt = DT[dtype]
    x, W, b = randn(N, H, dt=dt, seed=1), randn(F, H, dt=dt, seed=2), randn(F, dt=dt, seed=3)
    dy = randn(N, F, dt=dt, seed=4)
    bufs = []

    def guarded(nbytes):
        t = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        bufs.append((t, nbytes))
        return t.data_ptr() + 4096

    es = x.element_size()
    code = {"bf16": 1, "f32": 0}[dtype]
    st = torch.cuda.current_stream().cuda_stream
    fb, bb = _lib.flce_linear_workspace_size(N, H, F, code, 4)
    z = guarded(N * F * 4)
    _lib.flce_linear_forward(x.data_ptr(), W.data_ptr(), b.data_ptr(), 0, N, H, F, code, 4, guarded(N * F * es), z,
                             guarded(fb), fb, st)
    _lib.flce_linear_backward(x.data_ptr(), W.data_ptr(), z, dy.data_ptr(), N, H, F, code, 4, guarded(N * H * es),
                              guarded(F * H * es), guarded(F * es), guarded(bb), bb, st)
    fb, bb = _lib.flce_glu_workspace_size(N, H, F, code)
    g, u = guarded(N * F * 4), guarded(N * F * 4)
    _lib.flce_glu_forward(x.data_ptr(), W.data_ptr(), W.data_ptr(), b.data_ptr(), 0, N, H, F, code, 4,
                          guarded(N * F * es), g, u, guarded(fb), fb, st)
    _lib.flce_glu_backward(x.data_ptr(), W.data_ptr(), W.data_ptr(), g, u, dy.data_ptr(), N, H, F, code, 4,
                           guarded(N * H * es), guarded(F * H * es), guarded(F * H * es), guarded(F * es),
                           guarded(F * es), guarded(bb), bb, st)
    torch.cuda.synchronize()
    for i, (t, n) in enumerate(bufs):
        assert bool((t[:4096] == 0xA5).all()) and bool((t[4096 + n:] == 0xA5).all()), i


@pytest.mark.parametrize("N", [3, 90, 520])
def test_requested_gradients_only(N):
    H, F = 72, 200
    x, W, V = (randn(n, H, dt=torch.bfloat16, seed=s) for n, s in ((N, 1), (F, 2), (F, 3)))
    dy = randn(N, F, dt=torch.bfloat16, seed=4)
    h, g, u = L.flce_glu_forward(x, W, V, keep=True)
    full = L.flce_glu_backward(x, W, V, g, u, dy, need_db=True)
    for need in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        part = L.flce_glu_backward(x, W, V, g, u, dy, need_dx=need[0], need_dWg=need[1], need_dWu=need[2])
        for want, p, f in zip(need, part, full):
            assert (p is not None) == want and (p is None or torch.equal(p, f))
    dx, dW, db = L.flce_linear_backward(x, W, dy, None, need_dx=False, need_dW=False, need_db=True)
    assert dx is None and dW is None and torch.equal(db, L.flce_linear_backward(x, W, dy, None, need_db=True)[2])


@pytest.mark.parametrize("N", [1, 40, 150, 600])
def test_results_repeat_bit_for_bit(N):
    x, W, V = (randn(n, 1024, dt=torch.bfloat16, seed=s) for n, s in ((N, 1), (136, 2), (136, 3)))
    dy = randn(N, 136, dt=torch.bfloat16, seed=4)

    def call():
        h, g, u = L.flce_glu_forward(x, W, V, keep=True)
        return (h, g, u, *L.flce_glu_backward(x, W, V, g, u, dy, need_db=True))

    first = call()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, call()))


def test_directional_differences():
    # fp32 central differences of the operators themselves along random
    # directions; h = 1e-2 leaves h^2 / 6 of the third derivative and the
    # outputs' rounding over h, both under 1e-3 of the derivative's size
    # |grad| |v|, which the directions' random signs do not cancel below.
    N, H, F = 40, 64, 48
    x, Wg, Wu = (randn(n, H, dt=torch.float32, seed=s, scale=sc) for n, s, sc in ((N, 1, 1.0), (F, 2, 0.125), (F, 3, 0.125)))
    dy = randn(N, F, dt=torch.float32, seed=4)
    for act in ("silu", "gelu", "gelu_tanh", "sigmoid"):
        _, g, u = L.flce_glu_forward(x, Wg, Wu, activation=act, keep=True)
        grads = L.flce_glu_backward(x, Wg, Wu, g, u, dy, activation=act)[:3]
        _, z = L.flce_linear_forward(x, Wg, activation=act, keep=True)
        lgrads = L.flce_linear_backward(x, Wg, dy, z, activation=act)[:2]
        for i, p in enumerate((x, Wg, Wu)):
            v = torch.sign(randn(*p.shape, dt=torch.float32, seed=10 + i)) * torch.sign(grads[i])   # partly aligned
            v = torch.where(randn(*p.shape, dt=torch.float32, seed=20 + i) > 0, torch.sign(grads[i]), v)
            e = 1e-2 / math.sqrt(p.numel())
            args = [x, Wg, Wu]

            def at(s):
                args[i] = p + s * e * v
                return float((L.flce_glu_forward(*args, activation=act)[0].double() * dy.double()).sum())

            num, ana = (at(1) - at(-1)) / (2 * e), float((grads[i].double() * v.double()).sum())
            assert abs(num - ana) <= 2e-3 * float(grads[i].norm() * v.norm()), (act, i, num, ana)
            if i < 2:
                def at1(s):
                    a = [x, Wg]
                    a[i] = p + s * e * v
                    return float((L.flce_linear_forward(*a, activation=act)[0].double() * dy.double()).sum())

                num, ana = (at1(1) - at1(-1)) / (2 * e), float((lgrads[i].double() * v.double()).sum())
                assert abs(num - ana) <= 2e-3 * float(lgrads[i].norm() * v.norm()), (act, i, num, ana)


def test_on_another_stream():
    x, W = randn(300, 512, dt=torch.bfloat16, seed=1), randn(136, 512, dt=torch.bfloat16, seed=2)
    ref, _ = L.flce_linear_forward(x, W, activation="gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = L.flce_linear_forward(x, W, activation="gelu")
    s.synchronize()
    assert torch.equal(y, ref)


@pytest.mark.parametrize("N", [4, 100, 520])
def test_graph_replays(N):
    H, F = 1024, 136
    x, Wg, Wu, Wd = (randn(*s, dt=torch.bfloat16, seed=i) for i, s in enumerate(((N, H), (F, H), (F, H), (H, F))))
    dy = randn(N, H, dt=torch.bfloat16, seed=9)

    def step():
        h, g, u = L.flce_glu_forward(x, Wg, Wu, keep=True)
        y, _ = L.flce_linear_forward(h, Wd, None, x)
        dh, dWd, _ = L.flce_linear_backward(h, Wd, dy)
        dx, dWg, dWu, dbg, _ = L.flce_glu_backward(x, Wg, Wu, g, u, dh, need_db=True)
        return y, dWd, dx, dWg, dWu, dbg

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        x.copy_(randn(N, H, dt=torch.bfloat16, seed=100 + i))
        ref = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref)), i


@pytest.mark.parametrize("lead", [(6,), (2, 70), (3, 5, 30)], ids=str)
def test_block_and_loss_as_used(lead):
    # feed-forward block on the residual stream, the head's loss, its backward, clipping: the gradients in
    # float64 autograd, each tensor's relative norm of the error within 2^-7 (a chain of four
    # bf16 roundings of independent elements, 2^-9 each, doubled)
    torch.manual_seed(0)
    H, F, V = 64, 176, 500
    block = L.GatedFeedForward(H, F, "silu", bias=True, device="cuda", dtype=torch.bfloat16)
    head = torch.nn.Linear(H, V, bias=False, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(*lead, H, device="cuda").to(torch.bfloat16).requires_grad_(True)
    tgt = torch.randint(0, V, lead, device="cuda")
    params = [*block.parameters(), head.weight]
    y = block(x, x)
    loss = L.FusedLinearCrossEntropyLoss()(y, tgt, head.weight)
    loss.backward()
    p64 = [p.detach().double().requires_grad_(True) for p in (x, *params)]
    x64, gw, gb, uw, ub, dw, db, hw = p64
    fn = torch.nn.functional
    y64 = x64 + fn.linear(fn.silu(fn.linear(x64, gw, gb)) * fn.linear(x64, uw, ub), dw, db)
    l64 = fn.cross_entropy(fn.linear(y64, hw).reshape(-1, V), tgt.reshape(-1))
    l64.backward()
    assert abs(float(loss) - float(l64)) <= 1e-2 * float(l64)
    for p, q in zip((x, *params), p64):
        assert float((p.grad.double() - q.grad).norm()) <= 2.0 ** -7 * float(q.grad.norm())
    raw = [p.grad.clone() for p in params]
    norm = L.clip_grad_norm_(params, 0.01)
    n64 = math.sqrt(sum(float(g.double().square().sum()) for g in raw))
    assert norm.shape == () and abs(float(norm) - n64) <= 1e-6 * n64 and n64 > 0.01
    for p, g in zip(params, raw):
        ref = g.double() * (0.01 / (n64 + 1e-6))
        assert bool(((p.grad.double() - ref).abs() <= half(ref, torch.bfloat16) * 1.001).all())


def test_gradients_only_where_needed_in_autograd():
    torch.manual_seed(0)
    x = torch.randn(5, 24, device="cuda")
    w, v = torch.randn(16, 24, device="cuda"), torch.randn(16, 24, device="cuda", requires_grad=True)
    b = torch.randn(16, device="cuda", requires_grad=True)
    h = L.fused_glu(x, w, v, None, b)
    h.sum().backward()
    assert w.grad is None and v.grad is not None and b.grad is not None
    ref = (torch.nn.functional.silu(x @ w.T)).sum(0)
    assert torch.allclose(b.grad, ref, rtol=1e-4, atol=1e-5)
    r = torch.randn(5, 16, device="cuda", requires_grad=True)
    y = L.fused_linear(x, w, None, r)
    y.backward(torch.ones_like(y))
    assert torch.equal(r.grad, torch.ones_like(r))
    with torch.no_grad():
        assert not L.fused_linear(x, w, b).requires_grad
    with pytest.raises(RuntimeError):
        (gx,) = torch.autograd.grad(L.fused_glu(x, w, v).sum(), v, create_graph=True)
        gx.sum().backward()
    with pytest.raises(ValueError):
        L.fused_linear(x, w, None, r[:4])
    with pytest.raises(TypeError):
        L.fused_linear(x, w.bfloat16())
    with pytest.raises(ValueError):
        L.fused_linear(x, w[:, :8])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    # 2.5e9 outputs: elements and bytes past 2^31 and 2^32 in y, z, dy and dz; sampled rows and all of dW
    dt = DT[dtype]
    N, H, F = 300_003, 16, 8200
    x, W = randn(N, H, dt=dt, seed=1), randn(F, H, dt=dt, seed=2, scale=0.25)
    y, z = L.flce_linear_forward(x, W, None, None, "gelu_tanh", keep=True)
    rows = torch.tensor([0, 1, 131_072, 261_900, 261_901, 262_143, N - 2, N - 1], device="cuda")
    z64, ez = z_with_err(x[rows], W, None)
    y64 = act64("gelu_tanh")(z64)
    close(y[rows], y64, 1.13 * ez + act_err(dt) * y64.abs() + half(y64, dt), "y")
    close(z[rows], z64, ez + half(z64, torch.float32), "z")
    del y
    dy = torch.zeros(N, F, dtype=dt, device="cuda")   # zero but for the sampled rows: dW is theirs alone
    dy[rows] = randn(len(rows), F, dt=dt, seed=3)
    dx, dW, db = L.flce_linear_backward(x, W, dy, z, "gelu_tanh", need_db=True)
    d64 = dy[rows].double()
    dz64 = d64 * dact64("gelu_tanh", z64)
    edz = d64.abs() * (ez + half(z64, torch.float32)) + 4 * act_err(dt) * d64.abs() + half(dz64, dt)
    x64, W64 = x[rows].double(), W.double()
    dx64, dW64, db64 = dz64 @ W64, dz64.T @ x64, dz64.sum(0)
    close(dx[rows], dx64, product_tol(dz64, edz, W64, dx64, dt), "dx")
    close(dW, dW64, product_tol(dz64.T, edz.T, x64, dW64, dt), "dW")
    ones = torch.ones(len(rows), 1, dtype=torch.float64, device="cuda")
    close(db, db64, product_tol(dz64.T, edz.T, ones, db64[:, None], dt)[:, 0], "db")
    dx[rows] = 0
    assert not bool(dx.any())


def test_two_streams_at_once():
    # calls in flight together, each with its own workspace
    args = [(randn(300 + 37 * i, 1024, dt=torch.bfloat16, seed=i), randn(136, 1024, dt=torch.bfloat16, seed=9),
             randn(300 + 37 * i, 136, dt=torch.bfloat16, seed=20 + i)) for i in range(4)]

    def call(x, W, dy):
        h, g, u = L.flce_glu_forward(x, W, W, keep=True)
        return (h, *L.flce_glu_backward(x, W, W, g, u, dy, need_db=True))

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
