"""The cases on which the feed-forward and gradient-clipping operators are timed and checked.

Three operators around the fused linear cross entropy: the gated product of a feed-forward block
(``flce_glu_forward`` / ``flce_glu_backward``), a linear layer with bias, activation and residual
(``flce_linear_forward`` / ``flce_linear_backward``), and the global gradient norm with clipping
(``flce_grad_norm`` / ``flce_clip_grad_norm``).

``own`` selects what ``run`` computes: False, the operators' formulas in elementary float32 torch operations,
rounded once to the outputs' type; True, the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _glu(name, N, H, F, act, dtype, train=False, bias=False):
    return {"name": name, "op": "glu", "N": N, "H": H, "F": F, "act": act, "dtype": dtype, "train": train,
            "bias": bias}


def _linear(name, N, H, F, act, dtype, train=False, bias=False, residual=False):
    return {"name": name, "op": "linear", "N": N, "H": H, "F": F, "act": act, "dtype": dtype, "train": train,
            "bias": bias, "residual": residual}


def _clip(name, sizes, dtype, small_dtype, ratio, in_place, norm):
    # sizes: "a x b" or "a" per tensor, joined by commas; ratio: max_norm over the norm the gradients have.
    return {"name": name, "op": "clip", "sizes": sizes, "dtype": dtype, "small_dtype": small_dtype, "ratio": ratio,
            "in_place": in_place, "norm": norm}


def listed():
    return [
        # One token of one sequence being generated: both projections' weights stream past a single row.
        _glu("glu_one_token", 1, 4096, 12288, "silu", "bf16"),
        # 48 sequences generated together, a GELU gate.
        _glu("glu_48_tokens", 48, 2048, 8192, "gelu", "f16"),
        # A prompt of odd length being read.
        _glu("glu_prompt", 517, 4096, 10240, "silu", "bf16"),
        # One training step's tokens at the benchmark's N and H: forward and backward.
        _glu("glu_train", 8192, 4096, 12288, "silu", "bf16", train=True),
        # A small model with biases, every size odd, half precision: forward and backward.
        _glu("glu_train_odd", 1037, 1000, 2731, "gelu_tanh", "f16", train=True, bias=True),
        # The block's output projection onto the residual stream for one generated token.
        _linear("linear_one_token", 1, 12288, 4096, "none", "bf16", residual=True),
        # The first layer of a plain feed-forward block for 200 rows.
        _linear("linear_200_rows", 200, 2048, 8192, "gelu", "bf16", bias=True),
        # The block's output projection in training, residual added: forward and backward.
        _linear("linear_train", 8192, 12288, 4096, "none", "bf16", train=True, residual=True),
        # A plain feed-forward layer trained in single precision.
        _linear("linear_train_f32", 2048, 1024, 4096, "gelu", "f32", train=True, bias=True),
        # Norm weights, biases and adapters: many small tensors, where launches and latency count.
        _clip("clip_small", ",".join(["4096"] * 8 + ["1024"] * 8 + ["16x1024"] * 4 + ["4096x16"] * 4 + ["1"]),
              "bf16", "f32", 0.3, False, 2.0),
        # An ordinary healthy step of a small model: odd sizes, single precision, the norm below the limit.
        _clip("clip_below_limit", "32000x2048,8191x2048,2048x8191,2048,2048,777x1023,333", "f32", "f32", 1.5, True, 2.0),
        # The head and one block of a large model, clipped.
        _clip("clip_head_and_block", "128256x4096,12288x4096,12288x4096,4096x12288," +
              ",".join(["4096x4096"] * 4 + ["4096"] * 2), "bf16", "f32", 0.25, False, 2.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("glu", "linear", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "clip":
        sizes = []
        for _ in range(_log_int(rng, 1, 300)):
            if rng.random() < 0.4:
                sizes.append(str(_log_int(rng, 1, 16384)))
            else:
                sizes.append(f"{_log_int(rng, 1, 4096)}x{_log_int(rng, 1, 2048)}")
        return {"op": "clip", "sizes": ",".join(sizes), "dtype": dtype, "small_dtype": rng.choice((dtype, "f32")),
                "ratio": rng.choice((0.01, 0.5, 2.0)), "in_place": False,
                "norm": rng.choice((2.0, 2.0, math.inf))}
    train = rng.random() < 0.5
    case = {"op": op, "N": _log_int(rng, 1, 4096 if train else 8192), "H": 8 * _log_int(rng, 8, 512),
            "F": _log_int(rng, 64, 8192), "act": rng.choice(ACTS), "dtype": dtype, "train": train,
            "bias": rng.random() < 0.5}
    if rng.random() < 0.5:
        case["F"] = (case["F"] + 63) // 64 * 64
    if rng.random() < 0.2:
        case["H"] -= rng.randrange(1, 8)
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


def _shapes(case):
    return [tuple(int(d) for d in s.split("x")) for s in case["sizes"].split(",")]


def work(case):
    if case["op"] == "clip":
        n = 0
        for s in _shapes(case):
            e = math.prod(s)
            n += e * DTYPES[case["dtype"] if len(s) > 1 else case["small_dtype"]].itemsize
        # Below the limit, in place, nothing needs to be written.
        writes = 0 if case["in_place"] and case["ratio"] >= 1 else n
        return {"bytes": n + writes, "flops": 3 * sum(math.prod(s) for s in _shapes(case))}
    N, H, F, es = case["N"], case["H"], case["F"], DTYPES[case["dtype"]].itemsize
    mats = 2 if case["op"] == "glu" else 1
    elems = N * H + mats * F * H + N * F                       # x, weights in; the output
    if case["bias"]:
        elems += mats * F
    if case.get("residual"):
        elems += N * F
    flops = 2 * mats * N * H * F
    if case["train"]:
        elems += N * F + N * H + mats * F * H                  # the output's gradient in; dx, dW
        if case["bias"]:
            elems += mats * F
        flops *= 3
    return {"bytes": elems * es, "flops": flops}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(shape, scale, dtype):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    state = {"case": case}
    if case["op"] == "clip":
        grads = []
        for s in _shapes(case):
            dt = DTYPES[case["dtype"] if len(s) > 1 else case["small_dtype"]]
            # each layer's gradients have a scale of their own
            grads.append(normal(s, 10.0 ** float(torch.rand((), generator=gen, device=dev) * 2 - 4), dt))
        if math.isinf(case["norm"]):
            norm = max(float(g.abs().max()) for g in grads)
        else:
            norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
        state["grads"] = grads
        state["max_norm"] = norm * case["ratio"]
        # The clipped gradients' own buffers; an in-place call has none.
        state["out"] = None if case["in_place"] else [torch.empty_like(g) for g in grads]
        return state
    N, H, F, dt = case["N"], case["H"], case["F"], DTYPES[case["dtype"]]
    # hidden states after a norm: unit scale, some channels larger than others
    gain = torch.exp(0.3 * torch.randn(H, generator=gen, device=dev))
    state["x"] = torch.randn((N, H), generator=gen, device=dev).mul_(gain).to(dt)
    names = ("Wg", "Wu") if case["op"] == "glu" else ("W",)
    for w in names:
        state[w] = normal((F, H), H ** -0.5, dt)
    for b in ("bg", "bu") if case["op"] == "glu" else ("b",):
        state[b] = normal((F,), 0.1, dt) if case["bias"] else None
    if case["op"] == "linear":
        state["residual"] = normal((N, F), 1.0, dt) if case["residual"] else None
    if case["train"]:
        state["dy"] = normal((N, F), 0.02, dt)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _act(z, act):
    """act(z) and its derivative, elementwise."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if act == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s, s * (1.0 - s)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(z * (0.5 ** 0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "clip":
        if math.isinf(case["norm"]):
            norm = torch.stack([g.float().abs().max() for g in state["grads"]]).max()
        else:
            # long sums of squares: 64 bits
            norm = torch.sqrt(torch.stack([g.double().square().sum() for g in state["grads"]]).sum()).float()
        coef = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
        outs = []
        for i, g in enumerate(state["grads"]):
            out = g if case["in_place"] else state["out"][i]
            out.copy_(g.float() * coef)
            outs.append(out)
        return [norm.reshape(1)] + outs
    dt = state["x"].dtype
    x = state["x"].float()
    if case["op"] == "glu":
        Wg, Wu = state["Wg"].float(), state["Wu"].float()
        g, u = x @ Wg.T, x @ Wu.T
        if case["bias"]:
            g, u = g + state["bg"].float(), u + state["bu"].float()
        a, da = _act(g, case["act"])
        h = a * u
        if not case["train"]:
            return [h.to(dt)]
        dh = state["dy"].float()
        dg, du = dh * u * da, dh * a
        out = [h, dg @ Wg + du @ Wu, dg.T @ x, du.T @ x]
        if case["bias"]:
            out += [dg.sum(0), du.sum(0)]
        return [t.to(dt) for t in out]
    W = state["W"].float()
    z = x @ W.T
    if case["bias"]:
        z = z + state["b"].float()
    a, da = _act(z, case["act"])
    y = a + state["residual"].float() if case["residual"] else a
    if not case["train"]:
        return [y.to(dt)]
    dz = state["dy"].float() * da
    out = [y, dz @ W, dz.T @ x]
    if case["bias"]:
        out.append(dz.sum(0))
    return [t.to(dt) for t in out]


def _run_own(state):
    from lm_head_cross_flce_amd import functional as L

    case = state["case"]
    if case["op"] == "clip":
        norm = L.flce_clip_grad_norm(state["grads"], state["max_norm"], norm_type=case["norm"], out=state["out"])
        return [norm] + (state["grads"] if case["in_place"] else state["out"])
    act, train, bias = case["act"], case["train"], case["bias"]
    if case["op"] == "glu":
        h, g, u = L.flce_glu_forward(state["x"], state["Wg"], state["Wu"], state["bg"], state["bu"], activation=act,
                                     keep=train)
        if not train:
            return [h]
        dx, dWg, dWu, dbg, dbu = L.flce_glu_backward(state["x"], state["Wg"], state["Wu"], g, u, state["dy"],
                                                     activation=act, need_db=bias)
        return [h, dx, dWg, dWu] + ([dbg, dbu] if bias else [])
    y, z = L.flce_linear_forward(state["x"], state["W"], state["b"], residual=state["residual"], activation=act,
                                 keep=train)
    if not train:
        return [y]
    dx, dW, db = L.flce_linear_backward(state["x"], state["W"], state["dy"], z, activation=act, need_db=bias)
    return [y, dx, dW] + ([db] if bias else [])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """The operators' definitions in float64, the gradients from automatic differentiation of the forward."""
    state = prepare(case, seed)
    if case["op"] == "clip":
        flat = [g.double() for g in state["grads"]]
        if math.isinf(case["norm"]):
            norm = max(float(torch.linalg.vector_norm(f, math.inf)) for f in flat)
        else:
            norm = math.hypot(*[float(torch.linalg.vector_norm(f)) for f in flat])
        c = min(1.0, state["max_norm"] / (norm + 1e-6))
        return [torch.tensor([norm], dtype=torch.float64, device="cuda")] + [f.mul_(c) for f in flat]
    fn = torch.nn.functional
    acts = {"none": lambda v: v, "relu": torch.relu, "gelu": fn.gelu,
            "gelu_tanh": lambda v: fn.gelu(v, approximate="tanh"), "silu": fn.silu, "sigmoid": torch.sigmoid}
    act = acts[case["act"]]
    keys = (("x", "Wg", "Wu", "bg", "bu") if case["op"] == "glu" else ("x", "W", "b"))
    leaves = {k: state[k].double().requires_grad_(case["train"]) for k in keys if state[k] is not None}
    with torch.set_grad_enabled(case["train"]):
        if case["op"] == "glu":
            y = act(fn.linear(leaves["x"], leaves["Wg"], leaves.get("bg"))) * fn.linear(leaves["x"], leaves["Wu"],
                                                                                       leaves.get("bu"))
        else:
            y = act(fn.linear(leaves["x"], leaves["W"], leaves.get("b")))
            if state["residual"] is not None:
                y = y + state["residual"].double()
    if not case["train"]:
        return [y]
    grads = torch.autograd.grad(y, list(leaves.values()), state["dy"].double())
    return [y.detach()] + list(grads)
