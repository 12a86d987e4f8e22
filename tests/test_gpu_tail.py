"""The norm, the microscaled product and the sampler as a serving step uses them, and the norm in a training step."""

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def randn(*shape, seed, scale=1.0, dt=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dt)


@pytest.mark.parametrize("N", [1, 33])
def test_from_the_residual_stream_to_a_token(N):
    H, F, V = 512, 1024, 5000
    up = L.MXLinear(torch.nn.Linear(H, F, device="cuda", dtype=torch.bfloat16), activation="silu")
    down = L.MXLinear(torch.nn.Linear(F, H, device="cuda", dtype=torch.bfloat16), x_format="e2m1")
    head = L.MXLinear(torch.nn.Linear(H, V, bias=False, device="cuda", dtype=torch.bfloat16))
    w1, w2 = (1 + randn(H, seed=i, scale=0.1) for i in (1, 2))
    x, stream = randn(N, H, seed=3), randn(N, H, seed=4)
    u = torch.rand(N, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    kw = dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.01)

    def step():
        q, h = L.flce_rms_norm_mx_forward(x, w1, stream)
        y = down(up(q), h)
        q2, h2 = L.flce_rms_norm_mx_forward(y, w2)
        logits = head(q2)
        return logits, L.flce_sample(logits, u, **kw), y

    logits, token, y = step()
    # the same by hand, each operand as the values it stands for, in float64: MXLinear rounds at its outputs only
    def val(q):
        return L.flce_mx_dequantize(q, torch.float32).double()

    q, h = L.flce_rms_norm_mx_forward(x, w1, stream)
    W = lambda m: val(L.MXTensor(m.codes, m.scales, m.cols, "e2m1"))   # noqa: E731
    a = torch.nn.functional.silu(val(q) @ W(up).T + up.bias.double())
    mid = up(q)
    assert float((mid.double() - a).norm() / a.norm()) <= 2.0 ** -8
    b = val(L.flce_mx_quantize(mid, "e2m1")) @ W(down).T + down.bias.double() + h.double()
    assert float((y.double() - b).norm() / b.norm()) <= 2.0 ** -8
    q2, _ = L.flce_rms_norm_mx_forward(y, w2)
    ref = val(q2) @ W(head).T
    assert float((logits.double() - ref).norm() / ref.norm()) <= 2.0 ** -8
    assert torch.equal(token, L.flce_sample(logits, u, **kw)) and bool((token >= 0).all()) and bool((token < V).all())

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(3):
        x.copy_(randn(N, H, seed=30 + i))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))


def test_norm_block_head_and_loss_in_training():
    # gradients of a pre-norm block, the final norm and the loss, in float32 against float64 autograd of the formulas:
    # products of float32 operands are right to 2^-22, sums of at most 300 terms: 1e-4 of each gradient's norm is ample
    H, F, V, N = 64, 96, 300, 50
    torch.manual_seed(0)
    n1, n2 = L.RMSNorm(H, device="cuda"), L.RMSNorm(H, device="cuda")
    block = L.GatedFeedForward(H, F, device="cuda")
    head = torch.nn.Linear(H, V, bias=False, device="cuda")
    x = torch.randn(N, H, device="cuda").requires_grad_(True)
    r = torch.randn(N, H, device="cuda").requires_grad_(True)
    t = torch.randint(0, V, (N,), device="cuda")
    y, h = n1(x, r)
    out = block(y, h)
    loss = L.FusedLinearCrossEntropyLoss()(n2(out), t, head.weight)
    loss.backward()
    mods = torch.nn.ModuleList([n1, n2, block, head])
    leaves = [x, r, *mods.parameters()]
    got = [p.grad.double() for p in leaves]
    d = {id(p): p.detach().double().requires_grad_(True) for p in leaves}

    def norm(v, w):
        return v * (v.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w

    h64 = d[id(x)] + d[id(r)]
    y64 = norm(h64, d[id(n1.weight)])
    lin = torch.nn.functional.linear
    g64 = torch.nn.functional.silu(lin(y64, d[id(block.gate_proj.weight)])) * lin(y64, d[id(block.up_proj.weight)])
    o64 = lin(g64, d[id(block.down_proj.weight)]) + h64
    l64 = torch.nn.functional.cross_entropy(lin(norm(o64, d[id(n2.weight)]), d[id(head.weight)]), t)
    assert abs(float(loss) - float(l64)) <= 1e-5 * float(l64)
    ref = torch.autograd.grad(l64, [d[id(p)] for p in leaves])
    for a, b in zip(got, ref):
        assert float((a - b).norm()) <= 1e-4 * float(b.norm())
    norm_before = L.clip_grad_norm_(leaves, 0.1)
    assert float(norm_before) > 0
