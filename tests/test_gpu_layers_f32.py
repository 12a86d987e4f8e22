"""float32 products: infinite operands, and how near a product comes to the exact one.

Tolerances.  A float32 operand x is multiplied as three bfloat16 parts h + m + l of 8 bits each, h rounded to
nearest, m and l cut off what it leaves: |m| <= 2^-8 |x| and |l| < 2^-15 |x|.  The products left out,
ml + lm + ll, are at most (2 * 2^-23 + 2^-30) |x y|.  The six that are added up come to x y in float32 with the
small ones first: their own additions round at 2^-23 (an adder that cuts off) of values under 2^-7 |x y|, and the last,
of hh, at 2^-23 |x y|.  So one product is within
    2^-22 (left out) + 2^-23 (the last addition) + 5 * 2^-23 * 2^-7 (the others) < 3.1 * 2^-23
of x y.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * scale


def same(got, ref):
    """Equal infinities and NaN; elsewhere float32 sums of products (8 sqrt(K) steps of terms of size one)."""
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(torch.isinf(got), torch.isinf(ref)) and torch.equal(got[torch.isinf(got)] > 0, ref[torch.isinf(ref)] > 0)
    fin = torch.isfinite(ref)
    assert bool(((got.double() - ref)[fin].abs() <= 1e-3).all())


# one row, the few-token kernel's last, the tiles' first, both tiles, a split K
SHAPES = [(1, 72, 40), (16, 72, 40), (17, 72, 40), (70, 4096, 72), (300, 264, 300), (900, 136, 1300)]


@pytest.mark.parametrize("tile", ["0", "4", "2"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_an_infinite_token(monkeypatch, shape, tile):
    # a row of x with an infinity: +-inf by its weights' signs, NaN where the weight is 0, and no other row changes
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    N, H, F = shape
    x, W = randn(N, H, seed=1), randn(F, H, seed=2, scale=H ** -0.5)
    clean, _ = L.flce_linear_forward(x, W)
    n = N * 2 // 3
    x[n, H - 3] = math.inf
    W[0, H - 3] = 0.0
    y, _ = L.flce_linear_forward(x, W)
    same(y, x.double() @ W.double().T)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[n] = False
    # the rows of other tiles are the same bits; those beside it may add up in another order
    assert bool(((y - clean)[keep][:, 1:].abs() <= 1e-3).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_an_infinite_weight_and_both(shape):
    N, H, F = shape
    x, W = randn(N, H, seed=1), randn(F, H, seed=2, scale=H ** -0.5)
    W[F // 2, 1] = -math.inf
    x[N // 2, 5] = math.inf
    same(L.flce_linear_forward(x, W)[0], x.double() @ W.double().T)
    V = randn(F, H, seed=3, scale=H ** -0.5)
    h, g, u = L.flce_glu_forward(x, W, V, activation="none", keep=True)
    g64, u64 = x.double() @ W.double().T, x.double() @ V.double().T
    same(g, g64)
    same(u, u64)
    x[N // 2, 5] = math.nan
    y, _ = L.flce_linear_forward(x, W)
    same(y, x.double() @ W.double().T)


@pytest.mark.parametrize("tile", ["0", "4", "2"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_infinite_gradients(monkeypatch, shape, tile):
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    N, H, F = shape
    x, W, dy = randn(N, H, seed=1, scale=0.1), randn(F, H, seed=2, scale=0.1), randn(N, F, seed=3, scale=0.1)
    dy[N // 2, F // 3] = math.inf
    dx, dW, db = L.flce_linear_backward(x, W, dy, need_db=True)
    d64 = dy.double()
    same(dx, d64 @ W.double())
    same(dW, d64.T @ x.double())
    same(db, d64.sum(0))


def test_the_largest_floats():
    # past bfloat16's largest finite value, where a rounded part is infinite though the operand is not
    big = torch.finfo(torch.float32).max
    N, H, F = 40, 8, 24
    x, W = torch.zeros(N, H, device="cuda"), torch.zeros(F, H, device="cuda")
    x[:, 0] = torch.tensor([big, -big, big * (1 - 2.0 ** -9)], device="cuda").repeat(14)[:N]
    W[:, 0] = torch.tensor([1.0, 0.5, -0.25, 2.0], device="cuda").repeat(6)
    y, _ = L.flce_linear_forward(x, W)
    ref = x[:, :1].double() * W[:, 0].double()
    over = ref.abs() > big
    assert bool(torch.isinf(y[over]).all()) and torch.equal(y[over] > 0, ref[over] > 0)
    assert bool(((y.double() - ref).abs()[~over] <= 3.1 * 2.0 ** -23 * ref.abs()[~over]).all())


@pytest.mark.parametrize("tile", ["4", "2"])
def test_one_product(monkeypatch, tile):
    # rows and weights with one element that is not zero: each output is one product
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    N, H, F = 400, 40, 300
    x, W = torch.zeros(N, H, device="cuda"), torch.zeros(F, H, device="cuda")
    x[:, 7], W[:, 7] = randn(N, seed=1), randn(F, seed=2)
    x[0, 7] = W[0, 7] = 1 + 2.0 ** -7 - 2.0 ** -23   # a long run of ones behind the first part
    y, _ = L.flce_linear_forward(x, W)
    ref = x[:, 7:8].double() * W[:, 7].double()
    rel = (y.double() - ref) / ref
    assert float(rel.abs().max()) <= 3.1 * 2.0 ** -23
    # the parts' errors have either sign: the mean over 400 x 300 products, of at least 300 independent ones, lies
    # within 6 standard errors of 0
    assert abs(float(rel.mean())) <= 6 * float(rel.square().mean().sqrt()) / math.sqrt(300)


@pytest.mark.parametrize("tile", ["4", "2"])
def test_long_sums_have_no_bias(monkeypatch, tile):
    # sums of K products that are all positive: independent errors of at most 3.1 * 2^-23 of each product (root mean
    # square at most that) grow with sqrt(K); a one-sided error of the parts would grow with K.  The float32
    # accumulation rounds K / 4 times or more at up to 2^-24 of the sum so far, of either sign: 8 standard deviations.
    monkeypatch.setenv("FLCE_DEBUG_LAYER_TILE", tile)
    N, H, F = 130, 4096, 96
    x, W = randn(N, H, seed=1).abs() + 0.5, randn(F, H, seed=2).abs() + 0.5
    y, _ = L.flce_linear_forward(x, W)
    ref = x.double() @ W.double().T
    tol = 8 * math.sqrt(H) * (3.1 * 2.0 ** -23 / H * 2 + 2.0 ** -24)
    assert float(((y.double() - ref) / ref).abs().max()) <= tol
