"""The cases on which the norm, the microscaled product and the sampler are timed and checked.

Four operators on the way from the residual stream to a token: the root-mean-square norm with the residual's addition,
its gradients and its output in 8 or 4 bits (``flce_rms_norm_forward`` / ``flce_rms_norm_mx_forward`` /
``flce_rms_norm_backward``), microscaled quantisation (``flce_mx_quantize`` / ``flce_mx_dequantize``), the linear layer
over microscaled operands (``flce_mx_linear``), and sampling from the head's logits (``flce_sample``).

Microscaled tensors: 32 consecutive columns share a scale 2^(s - 127), s a byte; their elements are e4m3 (a byte) or
e2m1 (half a byte, the even column in the low half).  Rows are padded with zeros to a multiple of 128 columns.

``own`` selects what ``run`` computes: False, the operators' formulas in elementary torch operations, in 32 bits (64 for
the sampler's sums and next to the quantisation's borders), rounded once to the outputs' type; True, the library's entry
points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "gelu", "silu")
FORMATS = ("e4m3", "e2m1")
# (exponent of the largest element, largest element, explicit mantissa bits, least exponent)
FORMAT = {"e4m3": (8, 448.0, 3, -6), "e2m1": (2, 6.0, 1, 0)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _norm(name, N, H, dtype, out, residual):
    # out: "train" (forward and backward), "same" (the tensors' type), or a microscaled format
    return {"name": name, "op": "norm", "N": N, "H": H, "dtype": dtype, "out": out, "residual": residual}


def _quantize(name, N, H, dtype, fmt):
    return {"name": name, "op": "quantize", "N": N, "H": H, "dtype": dtype, "format": fmt}


def _linear(name, N, H, F, fmt, dtype, act="none", bias=False, residual=False):
    return {"name": name, "op": "linear", "N": N, "H": H, "F": F, "format": fmt, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual}


def _sample(name, N, V, dtype, mode, masked):
    # mode: "greedy", "plain", "top_k", "top_p", "min_p", "all" (the three together), "mixed" (each row its own)
    return {"name": name, "op": "sample", "N": N, "V": V, "dtype": dtype, "mode": mode, "masked": masked}


def listed():
    return [
        # One generated token: the block's output joins the residual stream and leaves as the next product's operand.
        _norm("norm_one_token_8bit", 1, 4096, "bf16", "e4m3", True),
        # A prompt's tokens, the same.
        _norm("norm_prompt_8bit", 2048, 4096, "f16", "e4m3", True),
        # One training step's tokens at the benchmark's N and H: forward and backward.
        _norm("norm_train", 8192, 4096, "bf16", "train", True),
        # A small model in single precision, every size odd: forward and backward.
        _norm("norm_train_odd_f32", 1037, 2731, "f32", "train", False),
        # One of a block's weights going into 4 bits, and what it stands for from then on.
        _quantize("quantize_weight", 12288, 4096, "bf16", "e2m1"),
        # A short prompt's activations of odd sizes in single precision.
        _quantize("quantize_rows_odd", 517, 1000, "f32", "e4m3"),
        # One token's logits: the benchmark's head in 4 bits.
        _linear("mx_one_token_head", 1, 4096, 128256, "e4m3", "bf16"),
        # 48 sequences generated together, the first layer of a plain feed-forward block.
        _linear("mx_48_rows", 48, 2048, 8192, "e2m1", "f16", act="gelu", bias=True),
        # A prompt of odd length onto a ragged number of features.
        _linear("mx_prompt_odd", 517, 4000, 10241, "e4m3", "bf16", residual=True),
        # A batch of prompts, both operands in 4 bits.
        _linear("mx_many_rows", 8192, 4096, 12288, "e2m1", "bf16"),
        # One sequence's next token.
        _sample("sample_one_row", 1, 128256, "bf16", "all", False),
        # Requests of a serving batch, each with its own parameters, some held to part of the vocabulary.
        _sample("sample_batch", 256, 128256, "f32", "mixed", True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "quantize", "linear", "sample"))
    dtype = rng.choice(("bf16", "f16", "f32"))
    if op == "norm":
        H = _log_int(rng, 1, 20000)
        return {"op": op, "N": _log_int(rng, 1, min(16384, max(2, 33554432 // H))), "H": H, "dtype": dtype,
                "out": rng.choice(("train", "train", "same", "e4m3", "e2m1")), "residual": rng.random() < 0.6}
    if op == "quantize":
        H = _log_int(rng, 1, 16384)
        return {"op": op, "N": _log_int(rng, 1, min(16384, max(2, 50331648 // H))), "H": H, "dtype": dtype,
                "format": rng.choice(FORMATS)}
    if op == "linear":
        case = {"op": op, "N": _log_int(rng, 1, 4096), "H": _log_int(rng, 32, 8192), "F": _log_int(rng, 16, 12288),
                "format": rng.choice(FORMATS), "dtype": dtype, "act": rng.choice(ACTS), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.4}
        if rng.random() < 0.5:
            case["H"] = (case["H"] + 127) // 128 * 128
            case["F"] = (case["F"] + 15) // 16 * 16
        return case
    V = _log_int(rng, 2, 256000)
    return {"op": op, "N": _log_int(rng, 1, min(512, max(2, 32833536 // V))), "V": V, "dtype": dtype,
            "mode": rng.choice(("greedy", "plain", "top_k", "top_p", "min_p", "all", "mixed")),
            "masked": rng.random() < 0.3}


def _padded(n):
    return (n + 127) // 128 * 128


def _mx_bytes(fmt, rows, cols):
    p = _padded(cols)
    return rows * (p // (2 if fmt == "e2m1" else 1) + p // 32)


def work(case):
    N, es = case["N"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "norm":
        H = case["H"]
        n = N * H * es
        byte = n + H * es + (2 * n if case["residual"] else 0)               # x, weight; the residual and the sum
        if case["out"] in FORMATS:
            byte += _mx_bytes(case["out"], N, H)
        else:
            byte += n
        if case["out"] == "train":
            byte += 2 * n + H * es + (n if case["residual"] else 0)          # dy, the sum's gradient; dx, dweight
        return {"bytes": byte, "flops": N * H * (16 if case["out"] == "train" else 5)}
    if case["op"] == "quantize":
        n = N * case["H"]
        return {"bytes": n * es + _mx_bytes(case["format"], N, case["H"]) + 2 * n, "flops": 4 * n}
    if case["op"] == "linear":
        H, F = case["H"], case["F"]
        byte = _mx_bytes(case["format"], N, H) + _mx_bytes("e2m1", F, H) + N * F * es
        byte += (F * es if case["bias"] else 0) + (N * F * es if case["residual"] else 0)
        return {"bytes": byte, "flops": 2 * N * H * F}
    return {"bytes": N * case["V"] * es + N * 36, "flops": 4 * N * case["V"]}


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
    N, dt = case["N"], DTYPES[case["dtype"]]
    if case["op"] == "sample":
        V, mode = case["V"], case["mode"]
        # a head's logits: most tokens far below a few likely ones
        z = torch.randn((N, V), generator=gen, device=dev).mul_(2.5)
        likely = torch.rand((N, V), generator=gen, device=dev) < 16 / V
        z.add_(torch.rand((N, V), generator=gen, device=dev).mul_(12).mul_(likely))
        if case["masked"]:
            # a grammar's tokens: about a third of the vocabulary, in every second row
            off = torch.rand((N, V), generator=gen, device=dev) < 0.67
            off[::2] = False
            z.masked_fill_(off, -math.inf)
        state["logits"] = z.to(dt)
        state["u"] = torch.rand(N, generator=gen, device=dev)

        def per_row(values, dtype):
            pick = torch.randint(0, len(values), (N,), generator=gen, device=dev)
            return torch.tensor(values, dtype=dtype, device=dev)[pick]

        mixed = mode == "mixed"
        state["temperature"] = (0.0 if mode == "greedy" else 0.8) if not mixed else per_row(
            [0.0, 0.3, 0.7, 1.0, 1.5], torch.float32)
        state["top_k"] = per_row([0, 1, 20, 50, 1000], torch.int64) if mixed else 50 if mode in ("top_k", "all") else None
        state["top_p"] = (per_row([1.0, 0.5, 0.9, 0.95], torch.float32) if mixed
                          else 0.95 if mode in ("top_p", "all") else None)
        state["min_p"] = (per_row([0.0, 0.02, 0.1], torch.float32) if mixed
                          else 0.02 if mode in ("min_p", "all") else None)
        return state
    H = case["H"]
    # activations: unit scale, some channels larger than others
    gain = torch.exp(0.3 * torch.randn(H, generator=gen, device=dev))
    x = torch.randn((N, H), generator=gen, device=dev).mul_(gain)
    if case["op"] == "norm":
        state["x"] = x.to(dt)
        state["weight"] = normal((H,), 0.1, torch.float32).add_(1.0).to(dt)
        state["residual"] = normal((N, H), 2.0, dt) if case["residual"] else None
        if case["out"] == "train":
            state["dy"] = normal((N, H), 0.02, dt)
            # the residual stream's own gradient
            state["dh"] = normal((N, H), 0.02, dt) if case["residual"] else None
    elif case["op"] == "quantize":
        state["x"] = x.to(dt)
    else:
        F = case["F"]
        state["x"] = _pack(x, case["format"])
        state["W"] = _pack(normal((F, H), H ** -0.5, torch.float32), "e2m1")
        state["b"] = normal((F,), 0.1, dt) if case["bias"] else None
        state["residual"] = normal((N, F), 1.0, dt) if case["residual"] else None
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _quantized(x, fmt):
    """Elements (float64) and scale exponents of x [R, C], rows padded to 128 columns: the scale is
    2^(floor(log2(largest)) - the format's largest exponent), elements are rounded to nearest even and held to the
    format's largest."""
    emax, most, bits, least = FORMAT[fmt]
    R, C = x.shape
    v = torch.zeros((R, _padded(C)), dtype=torch.float64, device=x.device)
    v[:, :C] = x
    v = v.reshape(R, -1, 32)
    top = v.abs().amax(2)
    s = torch.frexp(top)[1] - 1 - emax
    s = torch.where(top > 0, s, torch.full_like(s, -127)).clamp_(-127, 127)
    v = v * torch.exp2(-s.double())[:, :, None]
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp_min_(least).double() - bits)
    return (torch.round(v / step) * step).clamp_(-most, most), s


def _pack(x, fmt):
    """(codes, scales): microscaled x as the library stores it."""
    v, s = _quantized(x, fmt)
    v = v.reshape(x.shape[0], -1)
    scales = (s + 127).to(torch.uint8)
    if fmt == "e4m3":
        return v.float().to(torch.float8_e4m3fn).view(torch.uint8), scales
    table = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    code = torch.bucketize(v.abs(), table).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def _unpacked(packed, fmt, cols):
    """float32 values of (codes, scales)."""
    codes, scales = packed
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), 2).reshape(codes.shape[0], -1).int()]
    scale = scales.view(torch.float8_e8m0fnu).float()
    return (v.reshape(v.shape[0], -1, 32) * scale[:, :, None]).reshape(v.shape[0], -1)[:, :cols]


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return z * 0.5 * (1.0 + torch.erf(z * (0.5 ** 0.5)))
    return z


def _column(p, like):
    """A parameter per row as the operator has it: a float32 number (or a whole one)."""
    if isinstance(p, torch.Tensor):
        return p[:, None].double()
    return torch.full_like(like[:, :1], p).float().double()


def _run_plain(state):
    case = state["case"]
    if case["op"] == "norm":
        dt = state["x"].dtype
        h, w = state["x"].float(), state["weight"].float()
        if state["residual"] is not None:
            h = h + state["residual"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        n = h * r
        y = n * w
        out = [h.to(dt)] if state["residual"] is not None else []
        if case["out"] in FORMATS:
            v, s = _quantized(y, case["out"])
            if case["out"] == "e4m3":
                return out + [v.reshape(case["N"], -1).float().to(torch.float8_e4m3fn),
                              (s + 127).to(torch.uint8).view(torch.float8_e8m0fnu)]
            v = v * torch.exp2(s.double())[:, :, None]
            return out + [v.reshape(case["N"], -1)[:, :case["H"]].to(torch.bfloat16)]
        out.append(y.to(dt))
        if case["out"] == "same":
            return out
        dy = state["dy"].float()
        dn = dy * w
        dx = (dn - n * (dn * n).mean(1, keepdim=True)) * r
        if state["dh"] is not None:
            dx = dx + state["dh"].float()
        return out + [dx.to(dt), (dy * n).sum(0).to(dt)]
    if case["op"] == "quantize":
        v, s = _quantized(state["x"], case["format"])
        return [(v * torch.exp2(s.double())[:, :, None]).reshape(case["N"], -1)[:, :case["H"]].to(torch.bfloat16)]
    if case["op"] == "linear":
        z = _unpacked(state["x"], case["format"], case["H"]) @ _unpacked(state["W"], "e2m1", case["H"]).T
        if state["b"] is not None:
            z = z + state["b"].float()
        y = _act(z, case["act"])
        if state["residual"] is not None:
            y = y + state["residual"].float()
        return [y.to(DTYPES[case["dtype"]])]
    z = state["logits"].double()
    V = z.shape[1]
    best = z.amax(1, keepdim=True)
    T = _column(state["temperature"], z)
    # by value from the largest, equal ones by index; weights relative to the largest
    ranked, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.where(ranked > -math.inf, torch.exp((ranked - best) / T), 0.0)
    rank = torch.arange(V, device=z.device)
    if state["top_k"] is not None:
        k = _column(state["top_k"], z)
        w = torch.where((rank < k) | (k <= 0), w, 0.0)
    if state["top_p"] is not None:
        p = _column(state["top_p"], z)
        before = torch.cumsum(w, 1) - w
        w = torch.where((before < p * w.sum(1, keepdim=True)) | (rank == 0) | (p >= 1), w, 0.0)
    if state["min_p"] is not None:
        w = torch.where(w >= _column(state["min_p"], z), w, 0.0)
    # the kept weights in the vocabulary's order; the first at which their sum passes u times the whole
    cum = torch.cumsum(torch.zeros_like(w).scatter_(1, order, w), 1)
    token = (cum <= state["u"].double()[:, None] * cum[:, -1:]).sum(1)
    token = torch.where(T[:, 0] > 0, token, order[:, 0])
    return [torch.where(best[:, 0] > -math.inf, token, -1)]   # a row that the mask left empty


def _run_own(state):
    from lm_head_cross_flce_amd import functional as L

    case = state["case"]
    if case["op"] == "norm":
        x, w, res, fmt = state["x"], state["weight"], state["residual"], case["out"]
        if fmt in FORMATS:
            q, h = L.flce_rms_norm_mx_forward(x, w, res, eps=EPS, format=fmt)
            out = [h] if res is not None else []
            if fmt == "e4m3":
                return out + [q.codes.view(torch.float8_e4m3fn), q.scales.view(torch.float8_e8m0fnu)]
            return out + [L.flce_mx_dequantize(q, torch.bfloat16)]
        y, h, rstd = L.flce_rms_norm_forward(x, w, res, eps=EPS, keep=fmt == "train")
        out = [h, y] if res is not None else [y]
        if fmt == "same":
            return out
        dx, dw = L.flce_rms_norm_backward(h, w, rstd, state["dy"], state["dh"])
        return out + [dx, dw]
    if case["op"] == "quantize":
        return [L.flce_mx_dequantize(L.flce_mx_quantize(state["x"], case["format"]), torch.bfloat16)]
    if case["op"] == "linear":
        x = L.MXTensor(*state["x"], case["H"], case["format"])
        W = L.MXTensor(*state["W"], case["H"], "e2m1")
        return [L.flce_mx_linear(x, W, state["b"], state["residual"], activation=case["act"],
                                 dtype=DTYPES[case["dtype"]])]
    return [L.flce_sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                          top_p=state["top_p"], min_p=state["min_p"])]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _nearest(x, fmt):
    """(elements, scales) of x [R, C] float64, by search among the format's values; ties go to the even code."""
    emax, most, bits, least = FORMAT[fmt]
    n = 2 ** bits
    grid = [m * 2.0 ** (least - bits) for m in range(n)]
    e = least
    while grid[-1] < most:
        grid += [(n + m) * 2.0 ** (e - bits) for m in range(n)]
        e += 1
    grid = torch.tensor([g for g in grid if g <= most], dtype=torch.float64, device=x.device)
    blocks = torch.nn.functional.pad(x, (0, _padded(x.shape[1]) - x.shape[1])).unflatten(1, (-1, 32))
    top = torch.linalg.vector_norm(blocks, math.inf, dim=2)
    e = torch.floor(torch.log2(top))
    e = torch.where(torch.ldexp(torch.ones_like(e), e) > top, e - 1, e)     # a logarithm rounded up to a whole number
    e = torch.where(torch.ldexp(torch.ones_like(e), e + 1) <= top, e + 1, e)
    scale = torch.ldexp(torch.ones_like(e), torch.clamp(e - emax, -127, 127))
    mag = (blocks / scale[:, :, None]).abs()
    hi = torch.searchsorted(grid, mag.contiguous()).clamp_(1, len(grid) - 1)
    lo = hi - 1
    a, b = mag - grid[lo], grid[hi] - mag
    pick = torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)
    return (torch.copysign(grid[pick], blocks)).flatten(1), scale


def exact(case, seed):
    """The operators' definitions in float64, the norm's gradients from automatic differentiation."""
    if case["op"] == "sample":
        return None
    state = prepare(case, seed)
    if case["op"] == "quantize":
        v, s = _nearest(state["x"].double(), case["format"])
        return [(v * s.repeat_interleave(32, 1))[:, :case["H"]]]
    if case["op"] == "linear":
        def values(packed, fmt):
            codes, scales = packed
            if fmt == "e2m1":
                codes = torch.stack((codes % 16, codes // 16), -1).flatten(1)
                bits, bias = 1, 1
            else:
                bits, bias = 3, 7
            codes = codes.double()
            top = 2 ** (3 if fmt == "e2m1" else 7)
            sign = 1 - 2 * torch.floor(codes / top)
            mag = codes % top
            e, m = torch.floor(mag / 2 ** bits), mag % 2 ** bits
            v = torch.where(e > 0, torch.exp2(e - bias) * (1 + m / 2 ** bits), 2.0 ** (1 - bias) * m / 2 ** bits)
            return sign * v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
        fn = torch.nn.functional
        acts = {"none": lambda t: t, "relu": torch.relu, "gelu": fn.gelu, "silu": fn.silu}
        z = fn.linear(values(state["x"], case["format"]), values(state["W"], "e2m1"),
                      None if state["b"] is None else state["b"].double())
        y = acts[case["act"]](z)
        return [y if state["residual"] is None else y + state["residual"].double()]
    train = case["out"] == "train"
    x = state["x"].double().requires_grad_(train)
    w = state["weight"].double().requires_grad_(train)
    with torch.set_grad_enabled(train):
        h = x if state["residual"] is None else x + state["residual"].double()
        y = w * h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    out = [h.detach()] if state["residual"] is not None else []
    if case["out"] in FORMATS:
        v, s = _nearest(y, case["out"])
        if case["out"] == "e4m3":
            return out + [v, s]
        return out + [(v * s.repeat_interleave(32, 1))[:, :case["H"]]]
    out.append(y.detach())
    if not train:
        return out
    loss = (y * state["dy"].double()).sum()
    if state["dh"] is not None:
        loss = loss + (h * state["dh"].double()).sum()
    return out + list(torch.autograd.grad(loss, (x, w)))
