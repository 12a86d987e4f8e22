"""Sampling from large vocabularies against the definition in float64.

Past 262144 tokens the row's workgroup looks at groups of 64 tokens and more, and tokens are found through the groups'
numbers; past 8.4 million (1024 slices) a nucleus has no histograms.

The library adds weights as whole numbers of 2^-s of the largest.  Up to V = 2^18 tokens s = 62 - ceil(log2 V); each is
then off by 2^-(s + 1) at most, all by V 2^-(s + 1), 2^-27 of the row's sum at most.  In longer rows a list of up to 4096
tokens has s = 44 (2^-33 in all), and a row that is walked whole s by a bound on its sum: a token's rounding is 2^-57 of the
sum, n kept tokens have n / V of it at least, so all roundings V 2^-57 of what is kept (2^-34 at 8.4 million tokens).
Histograms hold each weight to 2^-39 of itself.  float64 sums of these rows are within 2^-38.  Tokens have to be equal:
a random draw lies that near to one of n borders with chance under n 2^-32, 1e-5 for all rows here where n is under 4096,
and for wider rows, whose roundings are as often up as down and hardly add up, less than that too.
"""

import math

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def define(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row [V] on the GPU."""
    T, p, m = f32(temperature), f32(top_p), f32(min_p)
    v, order = torch.sort(z.double(), descending=True, stable=True)
    if not T > 0:
        return int(order[0])
    w = torch.where(v > -math.inf, torch.exp((v - v[0]) / T), 0.0)
    if 0 < top_k < len(w):
        w[top_k:] = 0.0
    if p < 1:
        cum = w.cumsum(0)
        keep = cum - w < p * cum[-1]
        keep[0] = True
        w = torch.where(keep, w, 0.0)
    if m > 0:
        w = torch.where(w >= min(m, 1.0), w, 0.0)
    kept = torch.zeros_like(w).index_put_((order,), w).cumsum(0)
    return int(torch.searchsorted(kept, float(u) * kept[-1], right=True))


PARAMS = [dict(temperature=0.0), dict(top_k=50), dict(top_k=1), dict(min_p=0.05), dict(top_p=0.1, temperature=0.5),
          dict(top_p=0.95, temperature=1.5), dict(top_p=0.9, temperature=1e3), dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02),
          dict(top_k=30_000, top_p=0.5, temperature=4.0), dict(top_p=0.999, min_p=1e-3), {}]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [262_144, 262_145, 600_001, 5_000_011])
def test_merged_groups(V, dtype):
    size = 32
    while -(-V // size) > 8192:
        size *= 2
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(6, V, generator=g, device="cuda") * 3
    u = torch.rand(6, generator=g, device="cuda")
    z[1, V - 1], z[1, V - 2], z[1, V - V % size - 1] = 30.0, 29.5, 29.0           # in the last group, a partial one if V is odd
    for i in (1, 2, 700, 4095, V // size - 1):                                    # on both sides of the groups' borders
        z[2, i * size - 1], z[2, i * size] = 25.0, 25.0
    z[3, torch.rand(V, generator=g, device="cuda") < 0.67] = -math.inf
    z[4] = (z[4] * 2).round() / 2                                                 # ties at every border
    z[5, : V // 2] = -math.inf
    z = z.to(DT[dtype])
    for kw in PARAMS:
        got = L.flce_sample(z, u, **kw).tolist()
        want = [define(z[i], u[i], **kw) for i in range(6)]
        assert got == want, kw
