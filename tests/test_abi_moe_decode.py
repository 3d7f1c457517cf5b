"""Refusals and sizes of the few-token layer's entry point, on the host (no GPU)."""

import pytest
import torch

from fp8_fine_grained_permute_b200 import build as fbuild
from fp8_fine_grained_permute_b200 import fg8

INV, UNS, OK = fg8.FG8_ERR_INVALID_ARG, fg8.FG8_ERR_UNSUPPORTED, fg8.FG8_OK


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fg8.lib()


def test_refusals(L):
    need = fg8.fg8_moe_decode_workspace(4, 2, 256, 128)
    good = dict(x=16, T=4, C=256, logits=16, bias=16, ids=16, aff=16, k=2, E=8, wu=16, su=16, I=128, wd=16, sd=16,
                norm=1, dt=0, out=16, ws=16, n=need, st=None, stream=None)
    call = lambda **c: L.fg8_moe_decode(*[c.get(key, v) for key, v in good.items()])   # noqa: E731
    for c in [{key: None} for key in ("x", "bias", "ids", "aff", "wu", "su", "wd", "sd", "out", "ws")]:
        assert call(**c) == INV, c
    for c in [{key: 24} for key in ("x", "wu", "wd", "out", "ws")] + \
             [{key: 18} for key in ("logits", "bias", "ids", "aff", "su", "sd")]:
        assert call(**c) == INV, c
    for c in [dict(T=-1), dict(C=0), dict(C=200), dict(I=64), dict(I=130), dict(k=0), dict(k=9), dict(E=0),
              dict(norm=2), dict(dt=2), dict(n=need - 1)]:
        assert call(**c) == INV, c
    for c in [dict(T=65), dict(E=1025), dict(k=17, E=64), dict(E=1024, I=1 << 21), dict(E=1024, C=1 << 22)]:
        assert call(**c) == UNS, c
    assert call(T=0, x=None, out=None) == OK


def test_workspace_sizes(L):
    f = fg8.fg8_moe_decode_workspace
    assert f(0, 2, 256, 128) == 0 and f(65, 2, 256, 128) == 0 and f(4, 17, 256, 128) == 0 and f(4, 2, 256, 0) == 0
    assert f(1, 1, 256, 128) > fg8.FG8_MOE_DECODE_HEAD
    # growing with each size, so one made for the largest call serves the smaller ones
    sizes = [f(t, k, 2048, i) for t, k, i in ((1, 1, 128), (1, 8, 768), (8, 8, 768), (64, 8, 768), (64, 16, 2048))]
    assert sizes == sorted(sizes)


def test_helper_refuses(L):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)   # noqa: E731
    f32, bf16 = torch.float32, torch.bfloat16
    w = (z(2, 256, 128), z(2, 2, 1, dt=f32), z(2, 128, 128), z(2, 1, 1, dt=f32))
    x = z(3, 128, dt=bf16)
    with pytest.raises(ValueError, match="logits"):
        fg8.moe_decode(x, *w, 1)
    with pytest.raises(ValueError, match="logits of shape"):
        fg8.moe_decode(x, *w, 1, logits=z(3, 3, dt=f32), bias=z(2, dt=f32))
    with pytest.raises(ValueError, match="wq_dn"):
        fg8.moe_decode(x, w[0], w[1], z(2, 256, 128), w[3], 1, logits=z(3, 2, dt=f32), bias=z(2, dt=f32))
    with pytest.raises(ValueError, match="expected"):
        fg8.moe_decode(x, *w, 1, ids=z(3, 2, dt=torch.int32), affinity=z(3, 1, dt=f32))
    with pytest.raises(TypeError):
        fg8.moe_decode(x.float(), *w, 1, ids=z(3, 1, dt=torch.int32), affinity=z(3, 1, dt=f32),
                       workspace=z(1), out=z(3, 128, dt=bf16))
    with pytest.raises(ValueError, match="CUDA"):
        fg8.moe_decode(x, *w, 1, ids=z(3, 1, dt=torch.int32), affinity=z(3, 1, dt=f32), workspace=z(1))
    with pytest.raises(ValueError, match="64 tokens"):
        fg8.moe_decode_workspace(65, 1, 128, 128)


def test_helper_refuses_in_a_torch_without_cuda(L, monkeypatch):
    """Such a torch lacks the private functions that look the device and stream up."""
    import importlib.util
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("fp8_fine_grained_permute_b200.fg8_without_cuda", fg8.__file__)
    bare = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bare)
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)   # noqa: E731
    f32, i32 = torch.float32, torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        bare.moe_decode(z(3, 128, dt=torch.bfloat16), z(2, 256, 128), z(2, 2, 1, dt=f32), z(2, 128, 128),
                        z(2, 1, 1, dt=f32), 1, ids=z(3, 1, dt=i32), affinity=z(3, 1, dt=f32), workspace=z(1))
    with pytest.raises(ValueError, match="CUDA"):
        bare.requantize_colwise(z(128, 128), z(1, 128, dt=f32), z(2, dt=i32))
    with pytest.raises(ValueError, match="CUDA"):
        bare.gate_weights(z(6, dt=i32), z(3, 2, dt=f32), 6)
    with pytest.raises(ValueError, match="CUDA"):
        bare.route_topk(z(3, 4, dt=f32), z(4, dt=f32), 2)
