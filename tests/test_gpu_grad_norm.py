"""The global gradient norm and clipping against float64.

The norm is summed in float64 and rounded once to float32: relative 2^-24, plus
float64's own roundings (2^-53 each, nothing here).  A scaled gradient is a
float32 product rounded to its type: half a step, plus 2^-23 for the factor's and
the product's roundings.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import _lib
from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def rand(n, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dt)


def norm64(grads, p):
    if math.isinf(p):
        return max([float(g.double().abs().max()) for g in grads if g.numel()], default=0.0)
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(grads, ratio, p=2.0, out=False):
    n = norm64(grads, p)
    max_norm = ratio * n
    raw = [g.clone() for g in grads]
    outs = [torch.full_like(g, 7.0) for g in grads] if out else None
    assert abs(float(L.flce_grad_norm(grads, p)) - n) <= 2.0 ** -23 * n
    norm = L.flce_clip_grad_norm(grads, max_norm, p, out=outs)
    assert norm.shape == (1,) and norm.dtype == FP and abs(float(norm) - n) <= 2.0 ** -23 * n
    c = min(1.0, max_norm / (n + 1e-6))
    for g, r, o in zip(grads, raw, outs or grads):
        ref = r.double() * c
        tol = ref.abs() * (torch.finfo(r.dtype).eps / 2 + 2.0 ** -22) + TINY[r.dtype]
        assert bool(((o.double() - ref).abs() <= tol).all())
        if out:
            assert torch.equal(g, r)


# one chunk of work is 32 KB: both sides of it, of the 16-byte pieces, and empty tensors
SIZES = [1, 3, 7, 8, 9, 255, 256, 257, 0, 4095, 8192, 8193, 16383, 16384, 16385, 16392, 70001, 1]


@pytest.mark.parametrize("dt", [BF, HF, FP], ids=str)
@pytest.mark.parametrize("p", [2.0, math.inf])
@pytest.mark.parametrize("out", [False, True])
def test_sizes(dt, p, out):
    for ratio in (0.3, 2.0):
        check([rand(n, dt, i, 10.0 ** (i % 5 - 3)) for i, n in enumerate(SIZES)], ratio, p, out)
    for n in SIZES:
        check([rand(n, dt, 1)], 0.5, p, out) if n else None


@pytest.mark.parametrize("count", [1, 95, 96, 97, 300, 1000])
def test_many_tensors_of_mixed_types(count):
    # more tensors than one launch's table holds
    check([rand(1 + 37 * i % 1500, (BF, HF, FP)[i % 3], i) for i in range(count)], 0.1)


@pytest.mark.parametrize("out", [False, True])
def test_large(out):
    check([rand(30_000_001, BF, 1), rand(5_000_003, FP, 2), rand(100, FP, 3)], 0.2, out=out)


@pytest.mark.parametrize("dt", [BF, FP], ids=str)
@pytest.mark.parametrize("shift", range(0, 9))
def test_any_alignment(dt, shift):
    buf = rand(40_100, dt, 5)
    keep = buf.clone()
    n = 40_001
    g = buf[shift:shift + n]
    check([g, rand(5, FP, 6)], 0.5)
    assert torch.equal(buf[:shift], keep[:shift]) and torch.equal(buf[shift + n:], keep[shift + n:])
    # the output off the gradient's alignment
    g = rand(n, dt, 7)
    out = torch.full((n + 16,), 3.0, dtype=dt, device="cuda")
    L.flce_clip_grad_norm([g], 1e-3, out=[out[shift:shift + n]])
    ref = torch.empty_like(g)
    L.flce_clip_grad_norm([g], 1e-3, out=[ref])
    assert torch.equal(out[shift:shift + n], ref) and bool((out[:shift] == 3).all()) and bool((out[shift + n:] == 3).all())


def test_shapes_and_strides():
    a = rand(6000, BF, 1).view(20, 300)
    t = rand(6000, BF, 2).view(300, 20).T              # dense, transposed
    s = rand(12000, BF, 3).view(20, 600)[:, ::2]       # every second element
    hole = s._base if s._base is not None else s
    grads = [a, t, s, rand(1, FP, 4).reshape(())]
    before = hole.clone()
    check(grads, 0.4)
    assert torch.equal(hole.view(20, 600)[:, 1::2], before.view(20, 600)[:, 1::2])
    outs = [torch.empty(20, 300, dtype=BF, device="cuda").T.contiguous().T]
    raw = a.clone()
    L.flce_clip_grad_norm([a], 1e-2, out=outs)          # out transposed in memory
    ref = torch.empty_like(raw)
    L.flce_clip_grad_norm([raw], 1e-2, out=[ref])
    assert torch.equal(outs[0], ref)
    e = torch.ones(1, device="cuda").expand(10)
    assert abs(float(L.flce_grad_norm([e])) - math.sqrt(10)) < 1e-6
    with pytest.raises(ValueError):
        L.flce_clip_grad_norm([e], 1.0)


def test_refusals():
    g = rand(100, FP, 1)
    with pytest.raises(_lib.FlceError):
        L.flce_clip_grad_norm([g, g], 1.0)
    with pytest.raises(_lib.FlceError):
        L.flce_clip_grad_norm([g[:60], g[50:]], 1.0)
    with pytest.raises(_lib.FlceError):
        L.flce_clip_grad_norm([g], -1.0)
    with pytest.raises(_lib.FlceError):
        L.flce_grad_norm([g], 1.0)
    with pytest.raises(TypeError):
        L.flce_grad_norm([g.double()])
    with pytest.raises(ValueError):
        L.flce_clip_grad_norm([g], 1.0, out=[])
    with pytest.raises(ValueError):
        L.flce_clip_grad_norm([g], 1.0, out=[g.bfloat16()])
    assert abs(float(L.flce_grad_norm([g, g])) - math.sqrt(2) * norm64([g], 2)) < 1e-4   # reading twice is fine


def test_values_beyond_float32_squares():
    for dt, v in ((FP, 1e30), (BF, 1e30), (FP, 1e-30), (BF, 1e-30)):
        check([torch.full((5000,), v, dtype=dt, device="cuda")], 0.5 if v > 1 else 2.0)


def test_nan_and_infinity():
    for p in (2.0, math.inf):
        g = [rand(5000, BF, 1), rand(5000, FP, 2)]
        g[0][77] = math.nan
        n = L.flce_clip_grad_norm(g, 1.0, p)
        assert math.isnan(float(n)) and all(bool(torch.isnan(t).all()) for t in g)
        g = [rand(5000, BF, 1), rand(5000, FP, 2)]
        g[1][4999] = -math.inf
        n = L.flce_clip_grad_norm(g, 1.0, p)
        assert float(n) == math.inf and bool((g[0] == 0).all()) and bool((g[1][:-1] == 0).all()) and bool(
            torch.isnan(g[1][-1]))
    z = [torch.zeros(300, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(L.flce_clip_grad_norm(z, 0.0)) == 0.0 and not bool(z[0].any())
    g = [rand(300, FP, 1)]
    L.flce_clip_grad_norm(g, 0.0)
    assert not bool(g[0].any())
    g = [rand(300, FP, 1)]
    r = g[0].clone()
    L.flce_clip_grad_norm(g, math.inf)
    assert torch.equal(g[0], r)


def test_a_given_norm():
    g = [rand(5000, BF, 1), rand(70000, FP, 2)]
    ref = [t.clone() for t in g]
    n = L.flce_grad_norm(g)
    L.flce_clip_grads_with_norm(g, 0.5, n)
    L.flce_clip_grad_norm(ref, 0.5)
    # the factor from the norm rounded to float32: 2^-24 more
    for a, b in zip(g, ref):
        assert bool(((a.double() - b.double()).abs() <= b.double().abs() * torch.finfo(a.dtype).eps).all())
    out = [torch.empty_like(t) for t in g]
    L.flce_clip_grads_with_norm(g, 1.0, torch.full((1,), 2.0, device="cuda"), out=out)
    for o, t in zip(out, g):   # the factor is 1 / (2 + 1e-6), not 1 / 2
        v = t.double() / (2 + 1e-6)
        assert bool(((o.double() - v).abs() <= v.abs() * (torch.finfo(t.dtype).eps / 2 + 2.0 ** -22) + TINY[t.dtype]).all())
    with pytest.raises(ValueError):
        L.flce_clip_grads_with_norm(g, 1.0, torch.ones(2, device="cuda"))


def test_parameters():
    m = torch.nn.Sequential(torch.nn.Linear(33, 65), torch.nn.Linear(65, 7)).cuda()
    ref = [p.detach().clone().requires_grad_(True) for p in m.parameters()]
    for i, (p, q) in enumerate(zip(m.parameters(), ref)):
        p.grad = rand(p.numel(), FP, i).view_as(p)
        q.grad = p.grad.clone()
    n = L.clip_grad_norm_(m.parameters(), 1.0)
    nr = torch.nn.utils.clip_grad_norm_(ref, 1.0)
    assert torch.allclose(n, nr, rtol=1e-6)
    for p, q in zip(m.parameters(), ref):
        assert torch.allclose(p.grad, q.grad, rtol=1e-6)
    assert float(L.clip_grad_norm_([torch.nn.Parameter(torch.ones(3, device="cuda"))], 1.0)) == 0.0
    assert float(L.clip_grad_norm_(ref[0], 1e9)) > 0


def test_repeats_bit_for_bit_and_on_another_stream():
    g = [rand(1_000_003, BF, 1), rand(77, FP, 2)]
    a = L.flce_grad_norm(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = L.flce_grad_norm(g)
    s.synchronize()
    assert torch.equal(a, b) and all(torch.equal(a, L.flce_grad_norm(g)) for _ in range(3))


def test_graph_replays():
    g = [rand(50_001, BF, 1), rand(777, FP, 2)]
    out = [torch.empty_like(t) for t in g]

    def step():
        return L.flce_clip_grad_norm(g, 1.0, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for i in range(3):
        for k, t in enumerate(g):
            t.copy_(rand(t.numel(), t.dtype, 10 * i + k))
        want = step().clone()
        ref = [o.clone() for o in out]
        for o in out:
            o.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, ref)), i


@pytest.mark.parametrize("dt", [BF, FP], ids=str)
def test_a_tensor_past_32_bits(dt):
    n = 2 ** 31 + 12_345
    g = torch.full((n,), 0.5, dtype=dt, device="cuda")
    g[n - 7:] = 3.0
    ref = math.sqrt(0.25 * (n - 7) + 9.0 * 7)
    norm = L.flce_clip_grad_norm([g, torch.full((3,), 0.5, device="cuda")], ref / 4)
    assert abs(float(norm) - math.sqrt(ref * ref + 0.75)) <= 2.0 ** -23 * ref
    c = (ref / 4) / (math.sqrt(ref * ref + 0.75) + 1e-6)
    for i, v in ((0, 0.5), (2 ** 30, 0.5), (2 ** 31 - 1, 0.5), (2 ** 31, 0.5), (n - 8, 0.5), (n - 7, 3.0), (n - 1, 3.0)):
        assert abs(float(g[i]) - v * c) <= v * c * (torch.finfo(dt).eps / 2 + 2.0 ** -22), i
    assert int((g > 0.2).sum()) == 7
