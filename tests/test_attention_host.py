"""The host side of the 8-bit operators: streams, devices and the binding's own refusals, with stand-ins for torch and the library."""
import pytest

import bit_quantized_tensor_gb300 as qg
from tests.test_block_host import Library, Nothing, Stream, Tensor, Torch


class Heads(Tensor):
    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def stand_ins(monkeypatch):
    import torch as real
    torch, lib = Torch(), Library()
    torch.int8, torch.int32, torch.Tensor = real.int8, real.int32, Tensor
    torch.empty = lambda shape, dtype, device, base=torch.empty: Heads(base(shape, dtype, device).shape, dtype, device.index)
    monkeypatch.setattr(qg, "_torch_module", torch)
    monkeypatch.setattr(qg, "lib", lambda: lib)
    monkeypatch.setattr(qg, "_ordinary", Nothing)
    monkeypatch.setattr(qg, "_dtype_ids", None)
    return torch, lib


def calls(torch, index=0, **change):
    """Every call, operands on cuda:index; `change` replaces an operand by name."""
    def t(name, shape, dtype):
        return change.get(name) or Heads(shape, dtype, index)
    b, f, i, c = torch.bfloat16, torch.float32, torch.int32, torch.int8
    X, codes, scales = t("X", (40, 64), b), t("codes", (40, 64), c), t("scales", (40,), f)
    Q, K, r = t("Q", (40, 4, 64), b), t("K", (40, 2, 64), b), t("rq", (40, 4), f)
    rk, g, pos, table = t("rk", (40, 2), f), t("g", (64,), b), t("pos", (40,), i), t("angles", (9, 64), f)
    cache = (t("kq", (8, 2, 16, 64), c), t("vq", (8, 2, 16, 64), c), t("ks", (8, 2), f), t("vs", (8, 2), f))
    batch = (t("table", (3, 5), i), t("starts", (4,), i), t("lengths", (3,), i))
    return {
        "s8_quantize": lambda **kw: qg.s8_quantize(X, **kw),
        "s8_gemm": lambda **kw: qg.s8_gemm(codes, scales, codes, scales, 64, **kw),
        "s8_linear": lambda **kw: qg.s8_linear(X, codes, scales, **kw),
        "qk_norm_rope": lambda **kw: qg.qk_norm_rope(Q, K, g, g, pos, table, **kw),
        "qk_norm_rope_backward": lambda **kw: qg.qk_norm_rope_backward(Q, K, Q, K, g, g, pos, table, r, rk, **kw),
        "kv8_append": lambda **kw: qg.kv8_append(K, K, cache, *batch, **kw),
        "kv8_gather": lambda **kw: qg.kv8_gather(cache, *batch, 40, **kw),
        "kv8_attention": lambda **kw: qg.kv8_attention(Q, cache, *batch, **kw),
    }


CALLS = ["s8_quantize", "s8_gemm", "s8_linear", "qk_norm_rope", "qk_norm_rope_backward", "kv8_append", "kv8_gather",
         "kv8_attention"]


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_allocates_belongs_to_its_stream(stand_ins, name):
    torch, lib = stand_ins
    calls(torch)[name]()
    assert lib.launched == [(name, 1)] and set(torch.allocated_on) <= {1}
    lib.launched.clear(), torch.allocated_on.clear()
    calls(torch)[name](stream=Stream(2))
    assert lib.launched == [(name, 2)] and set(torch.allocated_on) <= {2}
    assert torch.current.cuda_stream == 1


@pytest.mark.parametrize("name", CALLS)
def test_operands_on_another_device_are_refused(stand_ins, name):
    torch, lib = stand_ins
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        calls(torch, index=1)[name]()
    with pytest.raises(ValueError, match="is on cuda:0, the current device is cuda:1"):
        calls(torch)[name](stream=Stream(2, index=1))
    assert not lib.launched
    calls(torch, index=1)[name](stream=Stream(2, index=1))
    assert lib.launched == [(name, 2)]


WRONG = {
    "s8_gemm": [("codes", (40, 80), "int8"), ("codes", (40, 64), "bfloat16"), ("scales", (39,), "float32")],
    "s8_linear": [("X", (40, 65), "bfloat16"), ("scales", (40,), "bfloat16"), ("X", (40, 2, 32), "bfloat16")],
    "qk_norm_rope": [("K", (39, 2, 64), "bfloat16"), ("K", (40, 2, 32), "bfloat16"), ("K", (40, 2, 64), "float32"),
                     ("g", (63,), "bfloat16"), ("g", (64,), "float16"), ("pos", (39,), "int32"), ("pos", (40,), "float32"),
                     ("angles", (9, 64), "bfloat16"), ("Q", (40, 256), "bfloat16")],
    "qk_norm_rope_backward": [("rq", (40, 3), "float32"), ("rk", (40, 2), "bfloat16")],
    "kv8_append": [("K", (40, 3, 64), "bfloat16"), ("kq", (8, 2, 16, 64), "bfloat16"), ("vq", (8, 2, 32, 64), "int8"),
                   ("ks", (8, 3), "float32"), ("table", (3, 5), "float32"), ("starts", (3,), "int32"), ("lengths", (4,), "int32")],
    "kv8_attention": [("Q", (40, 3, 64), "bfloat16"), ("Q", (40, 4, 32), "bfloat16"), ("Q", (40, 4, 64), "float32"),
                      ("vs", (8, 2), "bfloat16")],
}


@pytest.mark.parametrize("name,wrong", [(n, w) for n in WRONG for w in WRONG[n]])
def test_operands_that_do_not_fit_are_refused(stand_ins, name, wrong):
    import torch as real
    torch, lib = stand_ins
    operand, shape, dtype = wrong
    with pytest.raises((TypeError, ValueError)):
        calls(torch, **{operand: Heads(shape, getattr(real, dtype))})[name]()
    assert not lib.launched


def test_names_are_checked(stand_ins):
    torch, lib = stand_ins
    with pytest.raises(ValueError, match="style"):
        calls(torch)["qk_norm_rope"](style="other")
    assert not lib.launched
