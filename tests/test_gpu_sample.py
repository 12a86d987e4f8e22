"""Sampling against its definition.

Tokens are whole numbers and have to be equal.  The reference ranks in Python and adds float64 weights with math.fsum;
the library adds whole numbers of 2^-s (s = 46 at 128256 tokens).  Both are within 2^-40 of the true sums relative to the
row's, so a draw differs only where u or top_p lies within that of a border: for one of R rows of V tokens with chance
under R V 2^-39, 1e-5 for all rows here.  Where borders are met on purpose, every weight is a power of two and both are
exact.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def define(z, u, T=1.0, k=0, p=1.0, m=0.0):
    """The token of one row, z a list of Python floats."""
    T, p, m, u = f32(T), f32(p), f32(m), f32(u)
    if any(math.isnan(v) for v in z) or max(z) == -math.inf:
        return -1
    top = max(z)
    order = sorted(range(len(z)), key=lambda j: (-z[j], j))
    if not T > 0:
        return order[0]

    def weight(v):
        if v == top:
            return 1.0
        return 0.0 if v == -math.inf or top == math.inf else math.exp((v - top) / T)

    w = {j: weight(z[j]) for j in order}
    kept = order[:k] if 0 < k < len(z) else order
    if p < 1:
        whole, before, some = math.fsum(w[j] for j in kept), 0.0, []
        for i, j in enumerate(kept):
            if i and not before < p * whole:
                break
            some.append(j)
            before = before + w[j]
        kept = some
    if m > 0:
        kept = [j for j in kept if w[j] >= min(m, 1.0)]
    kept = sorted(kept)
    spot = max(u, 0.0) if u == u else 0.0
    whole, cum, last = math.fsum(w[j] for j in kept), 0.0, None
    for j in kept:
        cum += w[j]
        if w[j] > 0:
            last = j
        if cum > spot * whole:
            return j
    return last


def check(z, u, **kw):
    got = L.flce_sample(z, u, **{k: v for k, v in kw.items()})
    assert got.dtype == torch.int64 and got.shape == (z.shape[0],)
    rows, us = z.float().cpu().tolist(), u.cpu().tolist()
    at = lambda v, i, d: d if v is None else (v[i].item() if isinstance(v, torch.Tensor) else v)   # noqa: E731
    want = [define(rows[i], us[i], at(kw.get("temperature"), i, 1.0), at(kw.get("top_k"), i, 0),
                   at(kw.get("top_p"), i, 1.0), at(kw.get("min_p"), i, 0.0)) for i in range(len(rows))]
    assert got.tolist() == want, [(i, a, b) for i, (a, b) in enumerate(zip(got.tolist(), want)) if a != b][:10]
    return got


def draw(N, V, dt=torch.float32, seed=0, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.randn(N, V, generator=g, device="cuda") * scale).to(dt), torch.rand(N, generator=g, device="cuda"))


PARAMS = [{}, dict(temperature=0.7), dict(temperature=0.0), dict(top_k=1), dict(top_k=5), dict(top_k=40),
          dict(top_p=0.9), dict(top_p=0.1, temperature=2.0), dict(min_p=0.05), dict(min_p=1.0),
          dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02), dict(temperature=30.0, top_p=0.99),
          dict(temperature=1.5, top_k=700, top_p=0.8)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [1, 2, 3, 8, 63, 64, 65, 511, 512, 513, 1000, 8191, 8192, 8193, 40_001])
def test_sizes_and_parameters(V, dtype):
    z, u = draw(7, V, DT[dtype], seed=V)
    for kw in PARAMS:
        check(z, u, **kw)


@pytest.mark.parametrize("dtype", list(DT))
def test_large_vocabularies(dtype):
    for V in (128_256, 256_000):
        z, u = draw(3, V, DT[dtype], seed=V)
        for kw in (dict(temperature=0.8, top_k=50, top_p=0.95), dict(top_p=0.999), dict(temperature=1.3),
                   dict(top_k=30_000, top_p=0.5, temperature=4.0)):
            check(z, u, **kw)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [9000, 50_001])
def test_wide_nuclei(V, dtype):
    # nuclei of thousands of tokens: ends inside a bin, among ties, cut off by min-p, in a row partly masked
    N = 6
    z, u = draw(N, V, DT[dtype], seed=V + 1, scale=1.5)
    z[1, ::3] = -math.inf
    z[2] = (z[2] * 2).round() / 2
    z[3, V // 3:] = -math.inf
    u[4], u[5] = 0.0, 1 - 2.0 ** -24
    for kw in (dict(top_p=0.5, temperature=3.0), dict(top_p=0.9, temperature=1.5), dict(top_p=0.99, temperature=1e3),
               dict(top_p=0.999), dict(top_p=0.95, temperature=2.0, min_p=0.05), dict(top_p=0.3, temperature=2.0, min_p=1e-4),
               dict(min_p=0.01, temperature=4.0), dict(top_p=0.9, temperature=1e-3), dict(top_p=0.9, temperature=2e-4),
               dict(top_p=1 - 2.0 ** -24), dict(top_p=2.0 ** -20, temperature=5.0), dict(top_p=0.7, top_k=V // 2, temperature=2.0)):
        check(z, u, **kw)
    check(z - 500, u, top_p=0.9, temperature=0.2)      # z / T far from 0
    check(z.float() * 1e-3 - 41, u, top_p=0.9, temperature=0.01)


@pytest.mark.parametrize("dtype", list(DT))
def test_parameters_of_each_row(dtype):
    N, V = 60, 3000
    z, u = draw(N, V, DT[dtype], seed=5)
    pick = lambda v, dt: torch.tensor(v, dtype=dt, device="cuda")[torch.arange(N, device="cuda") % len(v)]   # noqa: E731
    check(z, u, temperature=pick([0.0, 0.5, 1.0, 2.5], torch.float32), top_k=pick([0, 1, 7, 100, 5000], torch.int64),
          top_p=pick([1.0, 0.3, 0.9], torch.float32), min_p=pick([0.0, 0.1], torch.float32))


@pytest.mark.parametrize("dtype", list(DT))
def test_ties(dtype):
    # whole-numbered logits: many equal ones at every border
    N, V = 40, 2000
    g = torch.Generator(device="cuda").manual_seed(8)
    z = torch.randint(-3, 4, (N, V), generator=g, device="cuda").to(DT[dtype])
    u = torch.rand(N, generator=g, device="cuda")
    for kw in PARAMS + [dict(top_k=k) for k in (283, 286, 290, 600, 1999, 2000, 2001)]:
        check(z, u, **kw)


@pytest.mark.parametrize("dtype", list(DT))
def test_equal_logits_and_exact_borders(dtype):
    # all weights 1: u V and top_p V fall on whole numbers exactly
    V = 1024
    z = torch.full((V + 1, V), -1.5, dtype=DT[dtype], device="cuda")
    u = torch.arange(V + 1, device="cuda") / V
    got = check(z, u)
    assert got.tolist() == [min(i, V - 1) for i in range(V + 1)]
    for p in (0.0, 2.0 ** -10, 0.25, 0.5, 1 - 2.0 ** -10):
        kept = max(1, int(p * V))
        got = L.flce_sample(z, u, top_p=p)
        assert got.tolist() == [min(i * kept // V, kept - 1) for i in range(V + 1)]
    got = L.flce_sample(z, u, top_k=512, top_p=0.5)
    assert got.tolist() == [min(i * 256 // V, 255) for i in range(V + 1)]


def test_zeros_of_either_sign_are_equal():
    z = torch.tensor([[-1.0, -0.0, 0.0, -0.0, -2.0]], device="cuda").repeat(3, 1)
    u = torch.tensor([0.0, 0.5, 0.99], device="cuda")
    assert L.flce_sample(z, u, temperature=0.0).tolist() == [1, 1, 1]
    assert L.flce_sample(z, u, top_k=2).tolist() == [1, 2, 2]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [5, 700, 9000])
def test_masks(V, dtype):
    z, u = draw(12, V, DT[dtype], seed=3)
    z[0] = -math.inf                         # nothing left
    z[1, :] = -math.inf
    z[1, V - 1] = -5.0                       # one token left
    z[2, ::2] = -math.inf
    z[3, 1] = math.nan
    z[4, 2] = -math.nan
    z[5, 3] = math.inf
    z[6, 1], z[6, 4] = math.inf, math.inf    # two share the weight
    z[7] = torch.finfo(DT[dtype]).min        # all at the type's lowest: as likely as each other
    z[8, 1:] = torch.finfo(DT[dtype]).min
    z[9, V // 2:] = -math.inf
    u[9] = 1 - 2.0 ** -24
    z[10] = torch.finfo(DT[dtype]).max
    z[11, 0] = -math.inf
    for kw in PARAMS + [dict(temperature=math.inf), dict(temperature=1e-30), dict(temperature=1e30)]:
        got = check(z, u, **kw)
        assert got[0] == -1 and got[1] == V - 1 and got[3] == -1 and got[4] == -1 and got[5] == 3


def test_parameters_out_of_their_range():
    z, u = draw(6, 500, seed=1)
    plain, first = check(z, u), L.flce_sample(z, u, temperature=0.0)
    nan = math.nan
    for kw in (dict(top_k=0), dict(top_k=-3), dict(top_k=500), dict(top_k=1 << 40), dict(top_p=1.0), dict(top_p=7.0),
               dict(top_p=nan), dict(min_p=0.0), dict(min_p=-1.0), dict(min_p=nan)):
        assert torch.equal(L.flce_sample(z, u, **kw), plain), kw
    for kw in (dict(temperature=-1.0), dict(temperature=nan), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.0),
               dict(min_p=9.0)):
        assert torch.equal(L.flce_sample(z, u, **kw), first), kw
    # u outside [0, 1)
    zeros = L.flce_sample(z, torch.zeros_like(u))
    for bad in (-1.0, nan, -math.inf):
        assert torch.equal(L.flce_sample(z, torch.full_like(u, bad)), zeros)
    for bad in (1.0, 5.0, math.inf):
        assert L.flce_sample(z, torch.full_like(u, bad)).tolist() == [499] * 6
    z[:, 400:] = -math.inf
    assert L.flce_sample(z, torch.full_like(u, 1.0)).tolist() == [399] * 6


@pytest.mark.parametrize("V", [500, 9000])
def test_an_infinite_temperature_makes_tokens_equally_likely(V):
    z, u = draw(6, V, seed=2)
    z[1, ::3] = -math.inf
    for kw in ({}, dict(top_k=40), dict(top_p=0.3), dict(top_p=0.95), dict(min_p=0.5), dict(min_p=1.0, top_p=0.9)):
        check(z, u, temperature=math.inf, **kw)


def test_more_slices_than_a_histogram_walk_takes():
    V = 1024 * 8192 + 77
    z, u = draw(2, V, torch.float16, seed=3)
    for p, T in ((1.0, 1.0), (0.9, 1.0), (0.02, 0.5)):
        got = L.flce_sample(z, u, temperature=T, top_p=p)
        for i in range(2):
            v, order = torch.sort(z[i].double(), descending=True, stable=True)
            w = torch.exp((v - v[0]) / T)
            cum = w.cumsum(0)
            keep = (cum - w < f32(p) * cum[-1]) if p < 1 else torch.ones_like(w, dtype=torch.bool)
            kept = torch.zeros(V, dtype=torch.float64, device="cuda").index_put_((order[keep],), w[keep]).cumsum(0)
            assert int(got[i]) == int(torch.searchsorted(kept, float(u[i]) * kept[-1], right=True)), (p, T, i)


def test_frequencies():
    # 200000 draws of one row of 6 tokens: each frequency within 6 standard deviations
    z = torch.log(torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], device="cuda")).repeat(200_000, 1)
    u = torch.rand(200_000, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    count = torch.bincount(L.flce_sample(z, u), minlength=6).cpu().double() / 200_000
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], dtype=torch.float64)
    assert bool(((count - p).abs() <= 6 * (p * (1 - p) / 200_000).sqrt()).all())


def test_strided_rows_none_and_streams():
    z, u = draw(8, 777, torch.bfloat16, seed=2)
    wide = torch.empty(8, 900, dtype=torch.bfloat16, device="cuda")
    wide[:, 5:782] = z
    ref = L.flce_sample(z, u, top_p=0.9)
    uu = torch.stack((u, u), 1)[:, 0]
    assert torch.equal(L.flce_sample(wide[:, 5:782], uu, top_p=0.9), ref)
    assert torch.equal(L.flce_sample(z.T.contiguous().T, u, top_p=0.9), ref)
    assert L.flce_sample(z[:0], u[:0]).shape == (0,)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(L.flce_sample(z, u, top_p=0.9))
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref) for g in got)
    for bad in (dict(u=u[:4]), dict(u=u.double()), dict(temperature=u.double()), dict(top_k=u), dict(top_p=u[:1]),
                dict(min_p=u.cpu())):
        with pytest.raises(ValueError):
            L.flce_sample(z, **{"u": u, **bad})


@pytest.mark.parametrize("N,V", [(1, 128_256), (40, 3001)])
def test_graph_replays(N, V):
    z, u = draw(N, V, torch.bfloat16, seed=4)
    kw = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    L.flce_sample(z, u, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = L.flce_sample(z, u, **kw)
    for i in range(4):
        a, b = draw(N, V, torch.bfloat16, seed=40 + i)
        z.copy_(a)
        u.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.flce_sample(z, u, **kw))


def test_offsets_past_32_bits():
    N, V = 17_000, 128_256    # 2.2e9 logits, 4.4 GB
    z = torch.full((N, V), -30.0, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 8_371, 16_742, 16_743, 16_744, N - 1], device="cuda")
    a, b = draw(len(rows), V, torch.bfloat16, seed=1)
    z[rows] = a
    u = torch.zeros(N, device="cuda")
    u[rows] = b
    assert torch.equal(L.flce_sample(z, u, top_p=0.9)[rows], L.flce_sample(a, b, top_p=0.9))
