"""MXLinear under changes of type, and its state."""

import pytest
import torch

from lm_head_cross_flce_amd import functional as L

pytestmark = pytest.mark.gpu


def made(K, F, dtype, bias=True):
    torch.manual_seed(K + F)
    return torch.nn.Linear(K, F, bias=bias, device="cuda", dtype=dtype)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("to", [torch.float16, torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("start", [torch.bfloat16, torch.float32], ids=str)
def test_a_change_of_type_reaches_the_output(start, to, bias):
    lin = made(300, 70, start, bias)
    mx = L.MXLinear(lin, activation="silu")
    W = L.MXTensor(mx.codes.clone(), mx.scales.clone(), 300, "e2m1")
    x = torch.randn(2, 5, 300, device="cuda").to(to)
    r = torch.randn(2, 5, 70, device="cuda").to(to)
    q = L.flce_mx_quantize(x.view(10, 300), "e4m3")
    b = lin.bias.detach().to(to) if bias else None
    for changed in (mx.to(to), torch.nn.Sequential(mx).to("cuda", to)[0]):
        y = changed(x, r)
        assert y.dtype == to and changed.dtype == to
        assert torch.equal(y.view(10, 70), L.flce_mx_linear(q, W, b, r.view(10, 70), "silu", to))
    assert torch.equal(mx.codes, W.codes) and torch.equal(mx.scales, W.scales)


def test_half_float_and_bfloat16():
    mx = L.MXLinear(made(256, 40, torch.bfloat16))
    x = torch.randn(3, 256, device="cuda")
    for change, dt in ((mx.half, torch.float16), (mx.float, torch.float32), (mx.bfloat16, torch.bfloat16)):
        assert change()(x).dtype == dt
    assert mx.cuda()(x).dtype == torch.bfloat16 and mx.to("cuda:0")(x).dtype == torch.bfloat16
    with pytest.raises(TypeError):   # no kernel for it: refused, not computed in another type
        mx.double()(x)
    assert mx.float()(x).dtype == torch.float32


@pytest.mark.parametrize("to", [torch.float16, torch.bfloat16, torch.float32, torch.float64], ids=str)
def test_type_leaves_the_weight_whole_numbers(to):
    # .type() converts every buffer, also those of whole numbers; 0 to 255 are exact in each of these
    mx = L.MXLinear(made(256, 400, torch.bfloat16))
    codes, scales = mx.codes.clone(), mx.scales.clone()
    x = torch.randn(3, 256, device="cuda")
    mx.type(to)
    assert torch.equal(mx.codes, codes) and torch.equal(mx.scales, scales) and mx.dtype == to
    if to != torch.float64:
        assert mx(x).dtype == to


def test_a_state_of_another_width_is_refused():
    # 300 and 310 columns are padded to the same 384
    a, b = L.MXLinear(made(300, 70, torch.bfloat16)), L.MXLinear(made(310, 70, torch.bfloat16))
    assert a.codes.shape == b.codes.shape and a.scales.shape == b.scales.shape
    codes, bias = b.codes.clone(), b.bias.clone()
    for strict in (True, False):
        with pytest.raises(RuntimeError, match="columns"):
            b.load_state_dict(a.state_dict(), strict=strict)
        with pytest.raises(RuntimeError, match="columns"):
            torch.nn.ModuleDict({"head": b}).load_state_dict(torch.nn.ModuleDict({"head": a}).state_dict(), strict=strict)
    assert torch.equal(b.codes, codes) and torch.equal(b.bias, bias)


def test_states_load_from_files_and_without_columns(tmp_path):
    a, b = L.MXLinear(made(300, 70, torch.bfloat16)), L.MXLinear(made(300, 70, torch.bfloat16, False))
    x = torch.randn(4, 300, device="cuda", dtype=torch.bfloat16)
    net = torch.nn.ModuleDict({"a": a, "b": b})
    torch.save(net.state_dict(), tmp_path / "net.pt")
    state = torch.load(tmp_path / "net.pt", weights_only=True)
    assert all(isinstance(v, torch.Tensor) for v in state.values())
    other = torch.nn.ModuleDict({"a": L.MXLinear(made(300, 70, torch.float32)), "b": L.MXLinear(made(300, 70, torch.float32, False))})
    for m in other.values():
        m.codes.zero_()
    other.load_state_dict(state)
    assert other["a"].dtype == torch.float32   # the module's, as a torch.nn.Linear keeps its own
    other.bfloat16()
    assert all(torch.equal(other[k](x), net[k](x)) for k in net)
    # a state from before it held the columns
    old = {k: v for k, v in state.items() if not k.endswith("_extra_state")}
    assert len(old) == len(state) - 2
    for m in other.values():
        m.codes.zero_()
    other.load_state_dict(old)
    assert all(torch.equal(other[k](x), net[k](x)) for k in net)
