"""Refusals of the checkpointed backward's entry points: found on the host,
before anything is launched (no GPU)."""

import pytest
import torch

from fp8_fine_grained_permute_b200 import build as fbuild
from fp8_fine_grained_permute_b200 import fg8

INV, UNS, OK = fg8.FG8_ERR_INVALID_ARG, fg8.FG8_ERR_UNSUPPORTED, fg8.FG8_OK
MAX32 = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    fbuild.build()
    return fg8.lib()


def _call(f, good, **changed):
    return f(*[changed.get(k, v) for k, v in good.items()])


def _refused(f, good, table):
    for status, changes in table:
        for c in changes:
            assert _call(f, good, **c) == status, (f.__name__, c)


def test_swiglu_backward_quant_refusals(L):
    good = dict(dh=16, guq=16, sgu=16, row_w=16, offsets=16, R=128, I=128, E=1, dq=16, sd=16, dqT=16, sdT=16,
                hqT=16, shT=16, dot=16, off=16, st=None, stream=None)
    _refused(L.fg8_swiglu_backward_quant, good, [
        (INV, [{k: None} for k in ("dh", "guq", "sgu", "offsets", "dq", "sd", "dqT", "sdT", "hqT", "shT", "off")]),
        (INV, [{k: 24} for k in ("dh", "guq", "dq", "dqT", "hqT")]),
        (INV, [{k: 18} for k in ("sgu", "row_w", "offsets", "sd", "sdT", "shT", "dot", "off")]),
        (INV, [dict(R=-1), dict(I=0), dict(I=64), dict(I=200), dict(E=0)]),
        (UNS, [dict(E=1025), dict(R=MAX32 + 1), dict(I=2 ** 30)])])


def test_requantize_colwise_refusals(L):
    good = dict(xq=16, sx=16, T=128, K=128, rt=16, offsets=16, R=128, E=1, xqT=16, saT=16, off=16, st=None,
                stream=None)
    _refused(L.fg8_requantize_colwise, good, [
        (INV, [{k: None} for k in ("xq", "sx", "offsets", "xqT", "saT", "off")]),
        (INV, [dict(xq=24), dict(xqT=8)] + [{k: 18} for k in ("sx", "rt", "offsets", "saT", "off")]),
        (INV, [dict(T=-1), dict(R=-1), dict(K=0), dict(K=100), dict(E=0), dict(T=0), dict(rt=None, R=127)]),
        (UNS, [dict(E=1025), dict(R=MAX32 + 1), dict(T=MAX32 + 1)])])


def test_gate_refusals(L):
    good = dict(tr=16, aff=16, T=4, k=2, norm=1, R=8, w=16, stream=None)
    _refused(L.fg8_gate_weights, good, [
        (INV, [dict(tr=None), dict(aff=None), dict(w=None), dict(tr=18), dict(aff=18), dict(w=18)]),
        (INV, [dict(T=-1), dict(k=0), dict(k=17), dict(norm=2), dict(R=-1)]),
        (UNS, [dict(R=MAX32 + 1), dict(T=MAX32)]),
        (OK, [dict(T=0, tr=None), dict(R=0, w=None)])])
    good = dict(dot=16, nb=2, R=8, tr=16, ids=16, aff=16, T=4, k=2, E=4, norm=1, da=16, dl=16, stream=None)
    _refused(L.fg8_gate_backward, good, [
        (INV, [{k: None} for k in ("dot", "tr", "ids", "aff", "da")]),
        (INV, [{k: 18} for k in ("dot", "tr", "ids", "aff", "da", "dl")]),
        (INV, [dict(T=-1), dict(k=0), dict(k=17), dict(norm=-1), dict(R=-1), dict(nb=0), dict(E=0)]),
        (UNS, [dict(R=MAX32 + 1), dict(T=MAX32)]),
        (OK, [dict(T=0, da=None)])])


def test_up_save_refusals(L):
    good = dict(a=16, sa=16, b=16, sb=16, offsets=16, M=128, I=128, K=128, E=1, hq=16, sh=16, guq=16, sgu=16,
                st=None, stream=None)
    _refused(L.fg8_grouped_gemm_swiglu_quant_save, good, [
        (INV, [{k: None} for k in ("a", "sa", "b", "sb", "offsets", "hq", "sh", "guq", "sgu")]),
        (INV, [{k: 24} for k in ("a", "b", "hq", "guq")] + [dict(sgu=18), dict(sh=18)]),
        (INV, [dict(I=96), dict(K=100), dict(E=0), dict(M=-1)]),
        (UNS, [dict(E=2000), dict(M=MAX32 + 1)]),
        (OK, [dict(M=0)])])


def test_helpers_refuse_cpu_tensors_and_wrong_outputs(L):
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)   # noqa: E731
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fg8.swiglu_backward_quant(z(4, 128, dt=torch.bfloat16), z(4, 256), z(2, 4, dt=torch.float32), off)
    with pytest.raises(TypeError):
        fg8.swiglu_backward_quant(z(4, 128, dt=torch.float32), z(4, 256), z(2, 4, dt=torch.float32), off)
    with pytest.raises(ValueError, match="expected"):
        fg8.swiglu_backward_quant(z(4, 128, dt=torch.bfloat16), z(4, 256), z(2, 4, dt=torch.float32), off,
                                  dq=z(4, 128))
    with pytest.raises(ValueError, match="expected"):
        fg8.requantize_colwise(z(4, 128), z(1, 4, dt=torch.float32), off, xqT=z(128, 128))
    with pytest.raises(ValueError, match="sgu"):
        fg8.swiglu_backward_quant(z(4, 128, dt=torch.bfloat16), z(4, 256), z(4, 2, dt=torch.float32), off)
    with pytest.raises(ValueError, match="row_token"):
        fg8.requantize_colwise(z(4, 128), z(1, 4, dt=torch.float32), off, row_token=z(4, dt=torch.int64))
    with pytest.raises(ValueError, match="affinity"):
        fg8.gate_weights(z(4, dt=torch.int32), z(2, 2, dt=torch.float64), 4)
    with pytest.raises(ValueError, match="topk_ids"):
        fg8.gate_backward(z(1, 4, dt=torch.float32), z(4, dt=torch.int32), z(4, dt=torch.int64),
                          z(2, 2, dt=torch.float32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        fg8.gate_weights(z(4, dt=torch.int32), z(2, 2, dt=torch.float32), 4)


class _Elsewhere:
    """A tensor of another device, as far as the binding looks at it."""
    shape, dtype = (4,), torch.float32

    def __init__(self, d, contiguous=True):
        self.d, self.c = d, contiguous

    def get_device(self):
        return self.d

    def is_contiguous(self):
        return self.c

    def numel(self):
        return 4

    def data_ptr(self):
        return 4096


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(fg8, "_device", lambda: 1)
    for take in (fg8._raw, lambda t: fg8._arg("x", t, (4,), torch.float32),
                 lambda t: fg8._arg_n("x", t, 4, torch.float32)):
        assert take(_Elsewhere(1)) == 4096
        with pytest.raises(ValueError, match="cuda:0, current device cuda:1"):
            take(_Elsewhere(0))
    assert fg8._raw(None) is None


def test_left_out_dots_and_logits(L):
    """What may be left out is refused with the rest of the arguments, not for its absence."""
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)   # noqa: E731
    f32, i32 = torch.float32, torch.int32
    with pytest.raises(ValueError, match="topk_ids"):
        fg8.gate_backward(z(1, 6, dt=f32), z(6, dt=i32), None, z(3, 2, dt=f32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        fg8.gate_backward(z(1, 6, dt=f32), z(6, dt=i32), None, z(3, 2, dt=f32), 4, want_dlogits=False)
    with pytest.raises(ValueError, match="CUDA"):
        fg8.swiglu_backward_quant(z(6, 128, dt=torch.bfloat16), z(6, 256), z(2, 6, dt=f32), z(2, dt=i32), want_dots=False)
    with pytest.raises(ValueError, match="gate_dot"):
        fg8.swiglu_backward_quant(z(6, 128, dt=torch.bfloat16), z(6, 256), z(2, 6, dt=f32), z(2, dt=i32),
                                  gate_dot=z(2, 6, dt=f32), want_dots=False)


def test_gemms_of_no_rows_take_no_row_buffers(L):
    """An empty batch's buffers have no address; the weights and offsets are still looked at."""
    swiglu = dict(a=None, sa=None, b=16, sb=16, offsets=16, M=0, I=128, K=128, E=1, hq=None, sh=None)
    save = dict(swiglu, guq=None, sgu=None, st=None, stream=None)
    swiglu.update(st=None, stream=None)
    gemm = dict(a=None, sa=None, b=16, sb=16, offsets=16, M=0, N=128, K=128, E=1, mode=fg8.FG8_GROUP_M,
                bmode=fg8.FG8_BSCALE_BLOCK128, dt=fg8.FG8_OUT_BF16, out=None, ws=None, n=0, st=None, stream=None)
    combine = dict(a=None, sa=None, b=16, sb=16, offsets=16, M=0, N=128, K=128, E=1, rt=None, tr=None, aff=None, T=0,
                   k=2, norm=1, out=None, ws=None, n=0, st=None, stream=None)
    for f, good in ((L.fg8_grouped_gemm_swiglu_quant, swiglu), (L.fg8_grouped_gemm_swiglu_quant_save, save),
                    (L.fg8_grouped_gemm, gemm), (L.fg8_grouped_gemm_combine, combine)):
        _refused(f, good, [(OK, [{}]), (INV, [dict(b=None), dict(sb=None), dict(offsets=None), dict(E=0), dict(K=100)]),
                           (INV, [dict(M=1), dict(M=-1)])])
    _refused(L.fg8_grouped_gemm_combine, combine, [(INV, [dict(T=1), dict(T=1, tr=16, aff=16), dict(M=1, a=16, sa=16)])])
