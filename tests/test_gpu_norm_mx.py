"""The norm's microscaled output against the formula in float64, element by element, and the rstd beside it.

The library's float32 y is within 101 steps of 2^-24 of the formula's (the sums' additions and the last products, as the
norm's other tests count them), so a block's largest magnitude is too, and a scale or a code may be that of any value
within that distance: where both ends of it round to the same code, as for all but a few elements, that code.  rstd is
within 96 such steps.  h is the sum rounded once.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
STEP = 2.0 ** -24
EMAX = {"e4m3": 8, "e2m1": 2}


def grid(fmt):
    bits, bias, n = (3, 7, 127) if fmt == "e4m3" else (1, 1, 8)
    out = []
    for code in range(n):
        e, m = code >> bits, code & ((1 << bits) - 1)
        out.append((m / (1 << bits)) * 2.0 ** (1 - bias) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (e - bias))
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def scale_of(top, fmt):
    """The scale byte of a block of this largest magnitude (over 0)."""
    return (torch.frexp(top)[1] - 1 - EMAX[fmt]).clamp_min(-127) + 127


def code_of(mag, fmt):
    """The code of a magnitude over its scale: nearest, ties to even, held to the largest."""
    g = grid(fmt)
    hi = torch.searchsorted(g, mag.contiguous()).clamp(1, len(g) - 1)
    lo = hi - 1
    a, b = mag - g[lo], g[hi] - mag
    return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def unpack(codes, fmt):
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), 2).flatten(1)
        return (codes & 7).long(), (codes >> 3).bool()
    return (codes & 127).long(), (codes >> 7).bool()


def check(codes, scales, y64, fmt):
    """How many scales and codes had a choice."""
    N, H = y64.shape
    padded = (H + 127) // 128 * 128
    y = torch.zeros(N, padded, dtype=torch.float64, device="cuda")
    y[:, :H] = y64
    tol = 101 * STEP
    top = y.abs().unflatten(1, (-1, 32)).amax(2)
    some = top > 0
    s = scales.long()
    lo, hi = scale_of(top * (1 - tol), fmt), scale_of(top * (1 + tol), fmt)
    assert bool((s[~some] == 0).all())
    assert bool(((s >= lo) & (s <= hi))[some].all())
    per = torch.exp2(127.0 - s.double()).repeat_interleave(32, 1)
    mag, neg = unpack(codes, fmt)
    a, b = code_of(y.abs() * (1 - tol) * per, fmt), code_of(y.abs() * (1 + tol) * per, fmt)
    assert bool(((mag >= a) & (mag <= b)).all()), int(((mag < a) | (mag > b)).sum())
    assert bool((b - a <= 1).all())
    sure = mag > 0
    assert torch.equal(neg[sure], (y < 0)[sure])
    assert not bool(mag[:, H:].any()) and not bool(neg[:, H:].any())
    return int((lo != hi)[some].sum()), int((a != b).sum())


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("N,H", [(1, 1), (64, 1), (7, 100), (3, 512), (9, 1000), (5, 4096), (130, 4096), (4, 9000), (3, 16_384),
                                 (2, 20_001)])
@pytest.mark.parametrize("dtype", list(DT))
def test_every_code_and_scale(N, H, dtype, fmt):
    dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(N + H)
    x, r = (torch.randn(N, H, generator=g, device="cuda").to(dt) for _ in range(2))
    # columns of very different size: in most blocks small elements stand beside a large one
    w = (torch.exp(1.5 * torch.randn(H, generator=g, device="cuda"))).to(dt)
    padded = (H + 127) // 128 * 128
    for res in (r, None):
        codes = torch.full((N, padded // (2 if fmt == "e2m1" else 1)), 85, dtype=torch.uint8, device="cuda")
        scales = torch.full((N, padded // 32), 85, dtype=torch.uint8, device="cuda")
        h = torch.full_like(x, 7.0) if res is not None else None
        rstd = torch.full((N + 2,), 7.0, device="cuda")
        _lib.flce_rms_norm_mx_forward(x.data_ptr(), None if res is None else res.data_ptr(), w.data_ptr(), N, H, L._DTYPES[dt],
                                      1e-6, _lib.MX_FORMATS[fmt], codes.data_ptr(), scales.data_ptr(),
                                      None if h is None else h.data_ptr(), rstd[1:].data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
        h64 = x.double() + (0 if res is None else res.double())
        r64 = (h64.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        scale_choice, code_choice = check(codes, scales, h64 * r64 * w.double(), fmt)
        # a border within 101 steps: at 2 x 101 x 2^-24 x some ten borders to a binade, 2^-12 of the elements at most (one
        # column: all elements are the weight)
        if H > 1:
            assert scale_choice <= 1 + scales.numel() // 1000 and code_choice <= 1 + N * H // 1000
        assert bool(((rstd[1:-1].double() - r64[:, 0]).abs() <= 96 * STEP * r64[:, 0]).all())
        assert float(rstd[0]) == 7.0 and float(rstd[-1]) == 7.0
        q, h2 = L.flce_rms_norm_mx_forward(x, w, res, format=fmt)
        assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)
        y, h3, rstd3 = L.flce_rms_norm_forward(x, w, res, keep=True)
        assert torch.equal(rstd3, rstd[1:-1]) and torch.equal(h2, h3)
        if h is not None:
            tol = h64.abs() * (torch.finfo(dt).eps / 2 + STEP) + 2.0 ** -25
            assert torch.equal(h, h2) and bool(((h.double() - h64).abs() <= tol).all())


def test_scale_borders_are_met_exactly():
    # rows of equal magnitudes with rstd 1 / magnitude: |y| is the weight, here powers of two and their neighbours
    H = 128
    x = torch.full((1, H), 4.0, device="cuda")
    for e in range(-20, 21, 5):
        for w in (2.0 ** e, 2.0 ** e * (1 + 2.0 ** -7), 2.0 ** e * (2 - 2.0 ** -7)):
            wt = torch.full((H,), w, device="cuda")
            for fmt in ("e4m3", "e2m1"):
                q, _ = L.flce_rms_norm_mx_forward(x, wt, eps=0.0, format=fmt)
                want = math.frexp(w)[1] - 1 - EMAX[fmt] + 127
                assert bool((q.scales == want).all()), (w, fmt)
