"""Helpers called with a stream while the current stream is held up: their outputs lie
in memory that nothing still pending on the current stream writes, and an output that
is dropped while the current stream has yet to read it is not handed to the next call
on the other stream."""

import pytest
import torch

from fp8_fine_grained_permute_b200 import build as fbuild
from fp8_fine_grained_permute_b200 import fg8

pytestmark = pytest.mark.gpu

T, E, k, C, I = 96, 4, 2, 512, 256
R = T * k


@pytest.fixture(scope="module")
def data():
    fbuild.build()
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
    d = dict(x=n(T, C).to(torch.bfloat16), logits=n(T, E), bias=torch.zeros(E, device="cuda"))
    d["wu"], d["su"] = fg8.quantize_weight((n(E, 2 * I, C) * 0.06).to(torch.bfloat16))
    d["wd"], d["sd"] = fg8.quantize_weight((n(E, C, I) * 0.06).to(torch.bfloat16))
    d["act"] = fg8.route_quantize_act(d["logits"], d["bias"], d["x"], k)
    d["dh"] = n(R, I).to(torch.bfloat16)
    d["save"] = fg8.grouped_gemm_swiglu_quant_save(d["act"]["xq"], d["act"]["sa"], d["wu"], d["su"], d["act"]["offsets"])
    d["dot"], d["y"] = n(2, R), n(R, C).to(torch.bfloat16)
    torch.cuda.synchronize()
    return d


CALLS = {
    "quantize_act": lambda d, s: fg8.quantize_act(d["x"], d["act"]["ids"], E, stream=s)["xq"],
    "up_save": lambda d, s: fg8.grouped_gemm_swiglu_quant_save(
        d["act"]["xq"], d["act"]["sa"], d["wu"], d["su"], d["act"]["offsets"], stream=s)[2],
    "act_backward": lambda d, s: fg8.swiglu_backward_quant(
        d["dh"], d["save"][2], d["save"][3], d["act"]["offsets"], stream=s)["dq"],
    "requantize": lambda d, s: fg8.requantize_colwise(d["act"]["xq"], d["act"]["sa"], d["act"]["offsets"], stream=s)[0],
    "gates": lambda d, s: fg8.gate_backward(d["dot"], d["act"]["token_row"], d["act"]["ids"], d["act"]["affinity"], E,
                                            stream=s)[1],
    "moe_decode": lambda d, s: fg8.moe_decode(d["x"][:64], d["wu"], d["su"], d["wd"], d["sd"], k, logits=d["logits"][:64],
                                              bias=d["bias"], stream=s)[0],
    "grouped_gemm": lambda d, s: fg8.grouped_gemm(d["save"][0], d["save"][1], d["wd"], d["sd"], d["act"]["offsets"], stream=s),
    "combine": lambda d, s: fg8.unpermute_combine(d["y"], d["act"]["token_row"], d["act"]["affinity"], stream=s),
}


def bits(t, n):
    """The written part, as bytes (column-wise operands: the columns of rows)."""
    t = t[:, :n] if n is not None else t
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_output_is_not_in_memory_that_the_current_stream_still_uses(data, name, handle):
    call = CALLS[name]
    n = 128 if name == "requantize" else None     # the first expert's first tile is written
    first = call(data, None)
    torch.cuda.synchronize()
    want, shape, dtype = bits(first, n).clone(), first.shape, first.dtype
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    # blocks of the output's size, freed here while writes to them are yet to run
    held = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del first
    torch.cuda._sleep(60_000_000)   # about 30 ms
    for h in held:
        h.view(torch.uint8).fill_(0x5A)
    del held, h
    got = call(data, s)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(bits(got, n), want)

    # the current stream reads it late; it is dropped, and the next call may not take it
    torch.cuda._sleep(60_000_000)
    late = bits(got, n).clone()
    del got
    outs = []
    for _ in range(4):
        with torch.cuda.stream(side):
            outs.append(torch.empty(shape, dtype=dtype, device="cuda"))
            outs[-1].view(torch.uint8).fill_(0xA5)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(late, want)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_stream_named_inside_a_capture(data, name, handle):
    """A capture whose calls name its own stream: what they allocate belongs to the graph."""
    call = CALLS[name]
    n = 128 if name == "requantize" else None
    want = bits(call(data, None), n).clone()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out = call(data, s.cuda_stream if handle else s)
    for _ in range(2):
        out.view(torch.uint8).fill_(0x5A)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out, n), want)
