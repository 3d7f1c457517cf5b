"""Every tensor that a helper makes for a call on a given stream (outputs, scratch,
status words) comes from that stream's memory, on the host with a torch whose CUDA
side is recorded instead of run: the caching allocator may give the current stream's
blocks to a call on another one while work there still uses them."""

import contextlib
import types

import pytest
import torch

from fp8_fine_grained_permute_b200 import fg8

u8, f32, i32, bf16 = torch.uint8, torch.float32, torch.int32, torch.bfloat16


class Tensor:
    def __init__(self, shape, dtype, made_on=None):
        self.shape = torch.Size(shape if isinstance(shape, (tuple, list)) else (shape,))
        self.dtype, self.device, self.is_cuda, self.made_on, self.users = dtype, torch.device("cuda", 0), True, made_on, []

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def get_device(self):
        return 0

    def numel(self):
        return self.shape.numel()

    def view(self, dtype):
        return Tensor(self.shape, dtype)

    def record_stream(self, s):
        self.users.append(s)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return isinstance(other, Stream) and other.cuda_stream == self.cuda_stream


MAIN, SIDE = 0x1000, 0x2000


@pytest.fixture
def recorded(monkeypatch):
    """Replaces fg8's torch and library; -> list of the tensors made."""
    made, current = [], [Stream(MAIN)]

    def make(*shape, dtype=None, device=None):
        t = Tensor(shape[0] if len(shape) == 1 else shape, dtype, current[-1])
        made.append(t)
        return t

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    fake = types.SimpleNamespace(
        empty=make, zeros=make, uint8=u8, float32=f32, int32=i32, bfloat16=bf16, int16=torch.int16,
        uint16=torch.uint16, device=torch.device, Tensor=Tensor,
        _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda d: current[-1].cuda_stream, _cuda_getDevice=lambda: 0),
        cuda=types.SimpleNamespace(Stream=Stream, ExternalStream=Stream, stream=on, current_stream=lambda d=None: current[-1]))

    class Lib:
        def __getattr__(self, name):
            sizes = name.endswith(("workspace", "capacity"))
            return lambda *a: 1024 if sizes else calls.append((name, a[-1])) or 0

    calls = []
    monkeypatch.setattr(fg8, "torch", fake)
    monkeypatch.setattr(fg8, "lib", Lib)
    monkeypatch.setattr(fg8, "_device", lambda: 0)
    return made, calls


T, E, k, C, I, P = 4, 2, 2, 256, 128, 1024
R = T * k


def t(*shape, dt=u8):
    return Tensor(shape, dt)


HELPERS = {
    "quantize_act": lambda s: fg8.quantize_act(t(T, C, dt=bf16), t(T, k, dt=i32), E, stream=s),
    "route_quantize_act": lambda s: fg8.route_quantize_act(t(T, E, dt=f32), t(E, dt=f32), t(T, C, dt=bf16), k, stream=s),
    "quantize_act_rows": lambda s: fg8.quantize_act_rows(t(R, C, dt=bf16), stream=s),
    "quantize_act_colwise": lambda s: fg8.quantize_act_colwise(t(R, C, dt=bf16), t(E + 1, dt=i32), stream=s),
    "quantize_weight": lambda s: fg8.quantize_weight(t(E, C, C, dt=bf16), stream=s),
    "quantize_weight_transposed": lambda s: fg8.quantize_weight_transposed(t(E, C, C, dt=bf16), stream=s),
    "transpose_blockq": lambda s: fg8.transpose_blockq(t(E, C, C), t(E, 2, 2, dt=f32), stream=s),
    "grouped_gemm": lambda s: fg8.grouped_gemm(t(R, C), t(2, R, dt=f32), t(E, C, C), t(E, 2, 2, dt=f32),
                                               t(E + 1, dt=i32), stream=s),
    "grouped_gemm_by_k": lambda s: fg8.grouped_gemm(t(C, P), t(8, C, dt=f32), t(C, P), t(8, C, dt=f32), t(E + 1, dt=i32),
                                                    group_mode=fg8.FG8_GROUP_K, stream=s),
    "grouped_gemm_swiglu_quant": lambda s: fg8.grouped_gemm_swiglu_quant(
        t(R, C), t(2, R, dt=f32), t(E, 2 * I, C), t(E, 2, 2, dt=f32), t(E + 1, dt=i32), stream=s),
    "grouped_gemm_swiglu_quant_save": lambda s: fg8.grouped_gemm_swiglu_quant_save(
        t(R, C), t(2, R, dt=f32), t(E, 2 * I, C), t(E, 2, 2, dt=f32), t(E + 1, dt=i32), stream=s),
    "swiglu_backward_quant": lambda s: fg8.swiglu_backward_quant(
        t(R, I, dt=bf16), t(R, 2 * I), t(2, R, dt=f32), t(E + 1, dt=i32), stream=s),
    "requantize_colwise": lambda s: fg8.requantize_colwise(t(R, C), t(2, R, dt=f32), t(E + 1, dt=i32), stream=s),
    "gate_weights": lambda s: fg8.gate_weights(t(R, dt=i32), t(T, k, dt=f32), R, stream=s),
    "gate_backward": lambda s: fg8.gate_backward(t(1, R, dt=f32), t(R, dt=i32), t(T, k, dt=i32), t(T, k, dt=f32), E, stream=s),
    "grouped_gemm_combine": lambda s: fg8.grouped_gemm_combine(
        t(R, C), t(2, R, dt=f32), t(E, C, C), t(E, 2, 2, dt=f32), t(E + 1, dt=i32), t(R, dt=i32), t(R, dt=i32),
        t(T, k, dt=f32), stream=s),
    "moe_decode": lambda s: fg8.moe_decode(
        t(T, C, dt=bf16), t(E, 2 * I, C), t(E, 2, 2, dt=f32), t(E, C, I), t(E, 2, 1, dt=f32), k,
        logits=t(T, E, dt=f32), bias=t(E, dt=f32), stream=s),
    "unpermute_combine": lambda s: fg8.unpermute_combine(t(R, C, dt=bf16), t(R, dt=i32), t(T, k, dt=f32), stream=s),
    "route_topk": lambda s: fg8.route_topk(t(T, E, dt=f32), t(E, dt=f32), k, stream=s),
}


def outputs(result):
    if isinstance(result, dict):
        result = list(result.values())
    return [x for x in (result if isinstance(result, (list, tuple)) else [result]) if isinstance(x, Tensor)]


@pytest.mark.parametrize("name", HELPERS)
@pytest.mark.parametrize("form", ["stream", "handle", "none"])
def test_made_on_the_calls_stream(recorded, name, form):
    made, calls = recorded
    stream = {"stream": Stream(SIDE), "handle": SIDE, "none": None}[form]
    want = MAIN if form == "none" else SIDE
    out = outputs(HELPERS[name](stream))
    assert made and [m.made_on.cuda_stream for m in made] == [want] * len(made)
    assert calls and calls[-1][1] == want
    # an output is usually read on the current stream: it must not go to another
    # call there before that is done
    fresh = [o for o in out if any(o is m for m in made)]
    assert fresh
    if form != "none":
        assert all(Stream(MAIN) in o.users for o in fresh)


def test_legacy_handle_is_the_default_stream(recorded):
    """1 is the runtime's name for the legacy default stream; torch's is 0."""
    made, _ = recorded
    fg8.gate_weights(t(R, dt=i32), t(T, k, dt=f32), R, stream=1)
    assert [m.made_on.cuda_stream for m in made] == [0]
