"""Microscaled tensors and the linear layer over them, against their definitions in float64.

Quantisation and its inverse are exact: codes and scales are equal to those of a search among the format's values.
The product's tolerances, element by element: half a step of the type; 8 sqrt(K) 2^-24 sum |x w| for float32 sums (each
of K additions is off by at most 2^-24 of a partial sum no larger than that, independently: 8 standard deviations); with
an e4m3 x and 16-bit results, of each of a piece's 128 products what lies under 2^-16 of the piece's largest, so 2^-9 of
the largest product of each piece at most; an activation's slope is at most 1.13, its own error relative 1e-5 (2e-6 for
float32).
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
FORMATS = ("e4m3", "e2m1")
EMAX = {"e4m3": 8, "e2m1": 2}


def grid(fmt):
    """The format's magnitudes by code, in order."""
    bits, bias, n = (3, 7, 127) if fmt == "e4m3" else (1, 1, 8)
    out = []
    for code in range(n):
        e, m = code >> bits, code & ((1 << bits) - 1)
        out.append((m / (1 << bits)) * 2.0 ** (1 - bias) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias))
    return torch.tensor(out, dtype=torch.float64)


def unpack(q):
    """(code magnitudes, signs, scale bytes) on the CPU, [R, C']."""
    codes = q.codes.cpu()
    if q.format == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1)
        return (codes & 7).long(), (codes >> 3).bool(), q.scales.cpu().long()
    return (codes & 127).long(), (codes >> 7).bool(), q.scales.cpu().long()


def values(q):
    """float64 values [R, C'] of a microscaled matrix without NaN, on the GPU."""
    mag, neg, s = unpack(q)
    v = grid(q.format)[mag] * torch.where(neg, -1.0, 1.0)
    return (v * torch.exp2(s.double() - 127).repeat_interleave(32, 1)).cuda()


def define(x, fmt):
    """(code magnitudes, scale bytes) of x [R, C] by search among the format's values."""
    g = grid(fmt)
    R, C = x.shape
    v = torch.zeros(R, (C + 127) // 128 * 128, dtype=torch.float64)
    v[:, :C] = x.cpu().double()
    blocks = v.reshape(R, -1, 32)
    top = blocks.abs().amax(2)
    s = torch.zeros(top.shape, dtype=torch.long)
    for i, t in enumerate(top.flatten().tolist()):
        if not math.isfinite(t):
            s.view(-1)[i] = 255
        elif t > 0:
            s.view(-1)[i] = max(math.frexp(t)[1] - 1 - EMAX[fmt], -127) + 127
    mag = (blocks.abs() * torch.exp2(127.0 - s.double())[:, :, None]).nan_to_num(0.0, 0.0)
    hi = torch.searchsorted(g, mag).clamp(1, len(g) - 1)
    lo = hi - 1
    a, b = mag - g[lo], g[hi] - mag
    code = torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    code[s == 255] = 0
    return code.reshape(R, -1), s


def exact(x, fmt):
    q = L.flce_mx_quantize(x, fmt)
    code, s = define(x, fmt)
    mag, neg, scales = unpack(q)
    assert torch.equal(scales, s)
    assert torch.equal(mag, code)
    C = x.shape[1]
    keep = (code[:, :C] > 0)
    assert torch.equal(neg[:, :C][keep], (x.cpu() < 0)[keep])
    assert not bool(mag[:, C:].any()) and not bool(neg[:, C:].any())
    for dt in DT.values():
        y = L.flce_mx_dequantize(q, dt)
        finite = (s < 255).repeat_interleave(32, 1)[:, :C].cuda()
        v = values(q._replace(scales=q.scales.clamp(max=254)))[:, :C]
        assert torch.equal(y[finite], v[finite].to(dt)), dt
        assert bool(y[~finite].isnan().all())
    return q


def randn(*shape, dt=torch.float32, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 32), (5, 33), (4, 127), (3, 128), (2, 129), (77, 1000), (1, 4096)],
                         ids=str)
def test_quantize_shapes(shape, dtype, fmt):
    exact(randn(*shape, dt=DT[dtype], seed=sum(shape)), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_every_scale(dtype, fmt):
    # each power of two that the type has, its neighbours and everything between, subnormals included
    fi = torch.finfo(DT[dtype])
    lo, hi = (-149, 127) if dtype == "f32" else (-133, 127) if dtype == "bf16" else (-24, 15)
    e = torch.arange(lo, hi + 1, dtype=torch.float64, device="cuda")
    x = torch.exp2(e)[:, None] * (1 + torch.rand(len(e), 64, dtype=torch.float64, device="cuda",
                                                generator=torch.Generator(device="cuda").manual_seed(1)))
    x[:, 0] = torch.exp2(e)
    x[:, 1::2] *= -torch.rand(len(e), 32, dtype=torch.float64, device="cuda",
                              generator=torch.Generator(device="cuda").manual_seed(2))
    exact(x.clamp(-fi.max, fi.max).to(DT[dtype]), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_ties_and_saturation(fmt):
    # every midpoint between neighbours of the grid, and values past the largest, under a scale of 1
    g = grid(fmt)
    mid = torch.cat([(g[1:] + g[:-1]) / 2, g, torch.tensor([g[-1] * 1.05, 2.0 ** (EMAX[fmt] + 1) * 0.999])])
    mid = torch.cat([mid, -mid])
    n = -(-len(mid) // 31)
    x = torch.zeros(n, 32, dtype=torch.float64)
    x[:, 0] = g[-1]
    flat = torch.zeros(n * 31, dtype=torch.float64)
    flat[:len(mid)] = mid
    x[:, 1:] = flat.view(n, 31)
    for k in (0, 40, -100):
        exact((x * 2.0 ** k).float().cuda(), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_infinities_and_nan(dtype, fmt):
    x = randn(6, 160, dt=DT[dtype], seed=3)
    x[0, 5], x[1, 40], x[2, 159] = math.inf, math.nan, -math.inf
    x[3, :32] = math.nan
    x[4] = 0
    x[5, 64:96] = -0.0
    q = exact(x, fmt)
    assert q.scales[0].tolist().count(255) == 1 and q.scales[3, 0] == 255 and not bool(q.scales[4].any())


def test_strided_inputs_and_no_rows():
    x = randn(50, 301, dt=torch.bfloat16, seed=4)
    for fmt in FORMATS:
        a, b = L.flce_mx_quantize(x[:, 1:], fmt), L.flce_mx_quantize(x[:, 1:].clone(), fmt)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        t = L.flce_mx_quantize(x.T, fmt)
        assert torch.equal(t.codes, L.flce_mx_quantize(x.T.contiguous(), fmt).codes)
        every = a._replace(codes=torch.stack((a.codes, a.codes), 2)[:, :, 0], scales=a.scales.T.contiguous().T)
        assert torch.equal(L.flce_mx_dequantize(every), L.flce_mx_dequantize(a))
        e = L.flce_mx_quantize(x[:0], fmt)
        assert e.codes.shape[0] == 0 and L.flce_mx_dequantize(e).shape == (0, 301)


def test_quantize_past_32_bits():
    R, C = 1_100_000, 4096   # 4.5e9 elements
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 524_287, 524_288, 1_048_575, 1_048_576, R - 1], device="cuda")
    x[rows] = randn(len(rows), C, dt=torch.bfloat16, seed=1)
    for fmt in FORMATS:
        q, ref = L.flce_mx_quantize(x, fmt), L.flce_mx_quantize(x[rows], fmt)
        assert torch.equal(q.codes[rows], ref.codes) and torch.equal(q.scales[rows], ref.scales)
        if fmt == "e2m1":
            x.fill_(1)
            del x
            y = L.flce_mx_dequantize(q)
            assert torch.equal(y[rows], L.flce_mx_dequantize(ref))


# ---------------------------------------------------------------------------
# The product
# ---------------------------------------------------------------------------

def act64(name):
    fn = torch.nn.functional
    return {"none": lambda z: z, "relu": torch.relu, "gelu": fn.gelu, "gelu_tanh": lambda z: fn.gelu(z, approximate="tanh"),
            "silu": fn.silu, "sigmoid": torch.sigmoid}[name]


def operands(N, K, F, fmt, seed=0):
    gain = torch.exp(randn(K, seed=seed + 5))
    x = L.flce_mx_quantize(randn(N, K, seed=seed) * gain, fmt)
    return x, L.flce_mx_quantize(randn(F, K, seed=seed + 1, scale=K ** -0.5), "e2m1")


def tolerance(x64, W64, y64, fmt, dt):
    K = x64.shape[1]
    tol = 8 * math.sqrt(K) * 2.0 ** -24 * (x64.abs() @ W64.abs().T)
    if fmt == "e4m3" and dt != torch.float32:
        for k in range(0, K, 128):   # the piece's largest product, by a bound on it
            tol = tol + 2.0 ** -9 * x64[:, k:k + 128].abs().amax(1)[:, None] * W64[:, k:k + 128].abs().amax(1)
    return 1.13 * tol


def check(N, K, F, fmt, dt, act="none", bias=False, residual=False, seed=0):
    x, W = operands(N, K, F, fmt, seed)
    b = randn(F, dt=dt, seed=seed + 2) if bias else None
    r = randn(N, F, dt=dt, seed=seed + 3) if residual else None
    y = L.flce_mx_linear(x, W, b, r, activation=act, dtype=dt)
    x64, W64 = values(x), values(W)
    z = x64 @ W64.T + (b.double() if bias else 0)
    a = act64(act)(z)
    ref = a + (r.double() if residual else 0)
    tol = (tolerance(x64, W64, ref, fmt, dt) + (2e-6 if dt == torch.float32 else 1e-5) * a.abs()
           + 2.0 ** -23 * (z.abs() + ref.abs()) + ref.abs() * (torch.finfo(dt).eps / 2) + TINY[dt])
    assert y.shape == (N, F) and y.dtype == dt
    err = (y.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float(err.max()), float((err / tol).max()))
    return x, W, y


SHAPES = [(1, 1, 1), (1, 128, 16), (1, 4096, 300), (3, 129, 17), (4, 1000, 64), (16, 300, 33), (16, 8192, 5), (17, 128, 64),
          (17, 256, 65), (33, 384, 70), (64, 640, 129), (65, 1000, 64), (100, 4096, 256), (129, 2304, 300),
          (517, 520, 260), (1000, 128, 1100)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_shapes(shape, dtype, fmt):
    check(*shape, fmt, DT[dtype])
    check(*shape, fmt, DT[dtype], "silu", True, True, seed=20)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_linear_large_tiles(dtype, fmt):
    check(2100, 640, 4200, fmt, DT[dtype], "gelu", True, True)


@pytest.mark.parametrize("tile", [2, 4, 8])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_every_tile(monkeypatch, dtype, fmt, tile):
    # whole and partial tiles, K of every remainder by the tiles' steps and runs, K split or not, whole and ragged features
    monkeypatch.setenv("FLCE_DEBUG_MX_TILE", str(tile))
    for N, K, F in ((1, 512, 8), (300, 640, 700), (257, 1152, 264), (60, 1300, 513), (256, 1408, 256), (130, 1700, 96),
                    (513, 2048, 320), (20, 2300, 40), (270, 4600, 260), (520, 5000, 1000)):
        check(N, K, F, fmt, DT[dtype])
        check(N, K, F, fmt, DT[dtype], "gelu", True, True, seed=11)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_few_tokens_many_features(dtype, fmt):
    for N, K, F in ((1, 512, 49_152), (16, 700, 49_170), (3, 1100, 50_001), (7, 130, 49_200)):
        check(N, K, F, fmt, DT[dtype])
        check(N, K, F, fmt, DT[dtype], "silu", True, True, seed=5)


@pytest.mark.parametrize("dtype", list(DT))
def test_large_tiles_in_several_rounds(monkeypatch, dtype):
    # more tiles of 256 x 256 than CUs: each workgroup's stores run on under its next tile
    for fmt in FORMATS:
        for F in (8200, 8193):
            check(2300, 1024, F, fmt, DT[dtype], "none", False, F == 8200)


@pytest.mark.parametrize("act", tuple(_lib.ACTIVATIONS))
@pytest.mark.parametrize("N", [5, 40, 400])
def test_every_activation(act, N):
    for dt in DT.values():
        check(N, 512, 200, "e4m3", dt, act, True, True)


@pytest.mark.parametrize("N", [2, 150])
def test_normal_operands_error(N):
    # the 2-norm of the error beside the results' rounding: float32 2e-6, and half steps of the others
    for fmt in FORMATS:
        x, W = operands(N, 4096, 512, fmt, 7)
        ref = values(x) @ values(W).T
        for dt, most in ((torch.float32, 2e-6), (torch.float16, 2.0 ** -11), (torch.bfloat16, 2.0 ** -8)):
            y = L.flce_mx_linear(x, W, dtype=dt)
            assert float((y.double() - ref).norm() / ref.norm()) <= most


@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_scales_far_apart(fmt, N, dtype):
    # x's blocks span 2^60 and W's undo it: each block weighs the same
    K, F = 512, 50
    e = torch.arange(16, device="cuda").repeat_interleave(32) * 4 - 30
    x = L.flce_mx_quantize(randn(N, K, seed=1) * torch.exp2(e.float()), fmt)
    W = L.flce_mx_quantize(randn(F, K, seed=2) * torch.exp2(-e.float()), "e2m1")
    y = L.flce_mx_linear(x, W, dtype=DT[dtype])
    x64, W64 = values(x), values(W)
    ref = x64 @ W64.T
    tol = 2.0 ** -9 * 16 * 64 if fmt == "e4m3" and dtype != "f32" else 0
    tol = tol + 8 * math.sqrt(K) * 2.0 ** -24 * (x64.abs() @ W64.abs().T) + ref.abs() * torch.finfo(DT[dtype]).eps / 2
    assert bool(((y.double() - ref).abs() <= tol + TINY[DT[dtype]]).all())


@pytest.mark.parametrize("N,K,F", [(3, 300, 90), (40, 300, 90), (600, 300, 90), (2, 600, 49_200), (300, 1664, 8200)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", list(DT))
def test_nan_scales_stay_in_their_rows(N, K, F, fmt, dtype):
    x, W = operands(N, K, F, fmt)
    xs, ws = x.scales.clone(), W.scales.clone()
    xs[1, 3] = 255
    ws[70, 0] = 255
    clean = L.flce_mx_linear(x, W, dtype=DT[dtype])
    y = L.flce_mx_linear(x._replace(scales=xs), W._replace(scales=ws), dtype=DT[dtype])
    nan = torch.zeros_like(y, dtype=torch.bool)
    nan[1], nan[:, 70] = True, True
    assert torch.equal(y.isnan(), nan) and torch.equal(y[~nan], clean[~nan])


def test_no_rows_and_strided_operands():
    x, W = operands(0, 200, 30, "e4m3")
    assert L.flce_mx_linear(x, W).shape == (0, 30)
    x, W = operands(20, 200, 30, "e4m3")
    b, r = randn(60, dt=torch.bfloat16, seed=1), randn(30, 20, dt=torch.bfloat16, seed=2)
    a = L.flce_mx_linear(x, W, b[::2], r.T)
    wide = torch.empty(20, 300, dtype=torch.uint8, device="cuda")
    wide[:, 3:259] = x.codes
    y = L.flce_mx_linear(x._replace(codes=wide[:, 3:259]), W, b[::2].clone(), r.T.contiguous())
    assert torch.equal(a, y)


@pytest.mark.parametrize("K,F", [(512, 66_000), (512, 66_001), (128, 66_000)])   # 256-row tiles, their ragged rows, small tiles
def test_linear_past_32_bits(K, F):
    N = 33_000
    x, W = operands(N, K, F, "e2m1")
    y = L.flce_mx_linear(x, W)
    rows = torch.tensor([0, 32_500, 32_511, 32_512, 32_767, 32_768, N - 1], device="cuda")
    x64, W64 = values(L.MXTensor(x.codes[rows], x.scales[rows], K, "e2m1")), values(W)
    ref = x64 @ W64.T
    tol = tolerance(x64, W64, ref, "e2m1", torch.bfloat16) + ref.abs() * 2.0 ** -8 + TINY[torch.bfloat16]
    assert bool(((y[rows].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("N", [4, 100, 700])
def test_residual_in_place(N):
    x, W = operands(N, 512, 256, "e4m3")
    r = randn(N, 256, dt=torch.bfloat16, seed=3)
    ref = L.flce_mx_linear(x, W, None, r)
    version = r._version
    out = L.flce_mx_linear(x, W, None, r, out=r)
    assert out is r and torch.equal(r, ref) and r._version > version


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("N,K,F", [(3, 200, 17), (40, 4096, 33), (300, 200, 1001)])
@pytest.mark.parametrize("dtype", list(DT))
def test_nothing_is_written_outside_the_output(N, K, F, dtype, fmt):
    x, W = operands(N, K, F, fmt)
    dt, code = DT[dtype], L._DTYPES[DT[dtype]]
    buf = torch.full((N * F + 128,), 7.0, dtype=dt, device="cuda")
    need = L.flce_mx_linear_workspace_size(N, K, F, fmt, dt)
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    _lib.flce_mx_linear(x.codes.data_ptr(), x.scales.data_ptr(), _lib.MX_FORMATS[fmt], W.codes.data_ptr(),
                        W.scales.data_ptr(), None, None, N, K, F, code, 0, buf[64:].data_ptr(), ws.data_ptr(), need,
                        torch.cuda.current_stream().cuda_stream)
    assert torch.equal(buf[64:64 + N * F].view(N, F), L.flce_mx_linear(x, W, dtype=dt))
    assert bool((buf[:64] == 7).all()) and bool((buf[64 + N * F:] == 7).all()) and bool((ws[need:] == 7).all())


def test_repeats_streams_and_graphs():
    args = [operands(n, 1024, 400, fmt, n) for n in (1, 90, 700) for fmt in FORMATS]
    ref = [L.flce_mx_linear(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                got.append(L.flce_mx_linear(*a))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(ref, got))
    x = randn(90, 1024, dt=torch.bfloat16, seed=5)
    W = args[0][1]

    def call():
        q = L.flce_mx_quantize(x, "e4m3")
        return L.flce_mx_linear(q, W), L.flce_mx_dequantize(q)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for i in range(4):
        x.copy_(randn(90, 1024, dt=torch.bfloat16, seed=60 + i))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, call()))


def test_binding_refusals_on_the_gpu():
    x, W = operands(4, 200, 30, "e4m3")
    with pytest.raises(ValueError):
        L.flce_mx_linear(x, x)                      # W in e4m3
    with pytest.raises(ValueError):
        L.flce_mx_linear(x, operands(4, 100, 30, "e4m3")[1])
    with pytest.raises(TypeError):
        L.flce_mx_linear(x, W, torch.zeros(30, device="cuda"))
    with pytest.raises(ValueError):
        L.flce_mx_linear(x, W, torch.zeros(31, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        L.flce_mx_linear(x, W, out=torch.zeros(30, 4, device="cuda", dtype=torch.bfloat16).T)
    with pytest.raises(ValueError):
        L.flce_mx_linear(x, W, torch.zeros(30, dtype=torch.bfloat16))


def test_module_follows_its_linear_layer():
    lin = torch.nn.Linear(300, 70, device="cuda", dtype=torch.bfloat16)
    mx = L.MXLinear(lin, activation="relu")
    x = randn(2, 5, 300, dt=torch.bfloat16, seed=1)
    r = randn(2, 5, 70, dt=torch.bfloat16, seed=2)
    y = mx(x, r)
    q = L.flce_mx_quantize(x.view(10, 300), "e4m3")
    ref = L.flce_mx_linear(q, L.flce_mx_quantize(lin.weight.detach()), lin.bias, r.view(10, 70), "relu")
    assert torch.equal(y.view(10, 70), ref) and torch.equal(mx(q).shape == (10, 70) and mx(q, r.view(10, 70)), ref)
    again = L.MXLinear(torch.nn.Linear(300, 70, device="cuda", dtype=torch.bfloat16), activation="relu")
    again.load_state_dict(mx.state_dict())
    assert torch.equal(again(x, r), y)
