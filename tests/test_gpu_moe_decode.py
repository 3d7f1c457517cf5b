"""The few-token expert layer in one kernel against the layer in 64 bits and
against the chain of kernels that computes it for many tokens.

The input's codes are the quantizer's own (bit-equal, so they carry no error
here).  Reference: [G; U] in 64 bits from the dequantized operands; h = silu(G) U
quantized to E4M3 in 1x128 tiles; out = sum_j w_j Wdn hq.

Tolerance, per output element.  A GEMM value (tensor-core partial of 128 products,
fp32 promotion over the blocks) is off by at most D = (128 + blocks) 2^-24 of
sum |a b|; through silu(G) U (slope of silu at most 1.1, fast exponential and
division 2^-20) h is off by dh, and h / scale by dz.  A code of h then equals the
reference's unless h / scale lies within 2 dz of a rounding midpoint, where it may
be one step away.  So out is off by at most
    sum_j w_j sum_i |Wdn_i| (step_i [midpoint in reach] + scale's own error)
    + D2 sum_j w_j sum_i |Wdn_i hq_i|,  D2 = (128 + 2 blocks + k + 8) 2^-24,
and half a step of the output's type."""

import numpy as np
import pytest
import torch

from fp8_fine_grained_permute_b200 import build as fbuild
from fp8_fine_grained_permute_b200 import fg8
from fp8_fine_grained_permute_b200 import workloads as W

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbuild.build()
    fg8.lib()
    torch.cuda.init()


class Layer:
    def __init__(self, E, C, I, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")   # noqa: E731
        self.E, self.C, self.I = E, C, I
        self.wq_up, self.sw_up = fg8.quantize_weight((n(E, 2 * I, C) * (1.5 / C ** 0.5)).to(torch.bfloat16))
        self.wq_dn, self.sw_dn = fg8.quantize_weight((n(E, C, I) * (1.0 / I ** 0.5)).to(torch.bfloat16))
        self.g = g

    def weights(self):
        return self.wq_up, self.sw_up, self.wq_dn, self.sw_dn

    def x(self, T):
        return torch.randn(T, self.C, generator=self.g, device="cuda").to(torch.bfloat16)

    def routing(self, T):
        return (torch.randn(T, self.E, generator=self.g, device="cuda"),
                0.2 * torch.rand(self.E, generator=self.g, device="cuda") - 0.1)


def _deq_block(q, s):
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _half_step(z):
    a = z.abs().clamp(min=2.0 ** -6)
    return 0.5 * torch.exp2(torch.floor(torch.log2(a)) - 3)


def _e4m3(z):
    """Nearest E4M3 value in 64 bits (ties to even)."""
    st = 2 * _half_step(z)
    return (torch.round(z / st) * st).clamp(-448, 448)


def reference(L, x, ids, aff, normalize=True):
    """-> (out, bound without the output's own rounding), fp64 [T, C]."""
    T, k = ids.shape
    xq, sx = fg8.quantize_act_rows(x)
    xd = xq.view(torch.float8_e4m3fn).double() * sx.double().t().repeat_interleave(128, 1)
    kept = (ids >= 0) & (ids < L.E)
    a = torch.where(kept, aff.double(), 0.0)
    s = a.sum(1, keepdim=True)
    w = torch.where(s != 0, a / s, 0.0) if normalize else a
    out = torch.zeros(T, L.C, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    I = L.I
    D, D2 = (128 + L.C // 128) * EPS, (128 + 2 * I // 128 + k + 8) * EPS
    for e in torch.unique(ids[kept]).tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        Wu, Wd = _deq_block(L.wq_up[e], L.sw_up[e]), _deq_block(L.wq_dn[e], L.sw_dn[e])
        gu, mag = xd[t] @ Wu.t(), xd[t].abs() @ Wu.abs().t()
        g, u = gu[:, :I], gu[:, I:]
        sig = torch.sigmoid(g)
        h = g * sig * u
        # silu' <= 1.1; fast exp and division: 2^-20 relative
        dh = 1.1 * u.abs() * D * mag[:, :I] + (g * sig).abs() * D * mag[:, I:] + 2.0 ** -20 * h.abs()
        amax = h.abs().view(-1, I // 128, 128).amax(2)
        sc = torch.where(amax > 0, amax / 448, 1.0).repeat_interleave(128, 1)
        dmax = dh.view(-1, I // 128, 128).amax(2).repeat_interleave(128, 1)
        z = h / sc
        q = _e4m3(z)
        # a scale off by dmax / 448 moves z by |z| dmax / amax
        dz = dh / sc + z.abs() * (dmax / (448 * sc) + 2 * EPS)
        reach = _half_step(z) - (z - q).abs() <= 2 * dz
        dq = torch.where(reach, 2 * _half_step(z), 0.0) * sc + q.abs() * (dmax / 448 + 2 * EPS * sc)
        hq = q * sc
        wt = w[t, j][:, None]
        out.index_add_(0, t, wt * (hq @ Wd.t()))
        bound.index_add_(0, t, wt * (dq @ Wd.abs().t() + D2 * (hq.abs() @ Wd.abs().t())))
    return out, bound


def check(L, x, ids, aff, out, normalize=True):
    ref, bound = reference(L, x, ids, aff, normalize)
    err = (out.double() - ref).abs()
    half = 2.0 ** -8 if out.dtype == torch.bfloat16 else EPS
    lim = bound + half * (ref.abs() + bound) + 1e-30
    assert torch.all(err <= lim), f"{(err / lim).max().item()} of the limit"


def run(L, x, k, ws=None, **kw):
    st = fg8.new_status()
    out, ids, aff = fg8.moe_decode(x, *L.weights(), k, workspace=ws, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert st.item() == 0, st.item()
    return out, ids, aff


CASES = [  # T, E, k, C, I
    (1, 4, 1, 128, 128), (1, 64, 6, 2048, 768), (2, 3, 3, 256, 384), (5, 8, 2, 640, 128),
    (16, 4, 4, 384, 256), (17, 4, 2, 256, 256), (33, 5, 1, 512, 640), (64, 8, 8, 256, 256),
    (64, 1, 1, 384, 128), (40, 100, 7, 128, 384), (3, 1000, 16, 256, 128), (11, 64, 6, 1024, 512)]


@pytest.mark.parametrize("T,E,k,C,I", CASES)
@pytest.mark.parametrize("f32", [False, True])
def test_layer_matches_formula(T, E, k, C, I, f32):
    L = Layer(E, C, I, seed=T * 7 + E)
    x = L.x(T)
    logits, bias = L.routing(T)
    out, ids, aff = run(L, x, k, logits=logits, bias=bias, out_dtype=fg8.FG8_OUT_F32 if f32 else fg8.FG8_OUT_BF16)
    rid, raff = fg8.route_topk(logits, bias, k)
    assert torch.equal(ids, rid) and torch.equal(aff, raff)
    check(L, x, ids, aff, out)


def test_given_routing_bad_ids_repeated_experts_and_no_normalization():
    L = Layer(6, 384, 256, seed=2)
    T, k = 20, 4
    x = L.x(T)
    ids = torch.randint(0, 6, (T, k), device="cuda", dtype=torch.int32)   # repeats happen
    ids[3] = 2                                  # one expert in every slot
    aff = torch.rand(T, k, device="cuda") + 0.01
    aff[5] = 0                                  # affinities that sum to 0: zeros when normalized
    for normalize in (True, False):
        out, _, _ = run(L, x, k, ids=ids, affinity=aff, normalize=normalize, out_dtype=fg8.FG8_OUT_F32)
        check(L, x, ids, aff, out, normalize)
    bad = ids.clone()
    bad[0, 1], bad[7], bad[9, 0] = -1, 6, 1 << 20
    st = fg8.new_status()
    out, _, _ = fg8.moe_decode(x, *L.weights(), k, ids=bad, affinity=aff, dev_status=st, out_dtype=fg8.FG8_OUT_F32)
    torch.cuda.synchronize()
    assert st.item() == fg8.FG8_ERR_BAD_EXPERT_ID
    assert torch.all(out[7] == 0) and torch.all(out[5] == 0)
    check(L, x, bad, aff, out)


def test_no_valid_expert_and_no_tokens():
    L = Layer(2, 256, 128, seed=3)
    x = L.x(3)
    ids = torch.full((3, 2), -1, device="cuda", dtype=torch.int32)
    st = fg8.new_status()
    out, _, _ = fg8.moe_decode(x, *L.weights(), 2, ids=ids, affinity=torch.ones(3, 2, device="cuda"), dev_status=st,
                               out=torch.full((3, 256), 7.0, device="cuda", dtype=torch.bfloat16))
    torch.cuda.synchronize()
    assert st.item() == fg8.FG8_ERR_BAD_EXPERT_ID and torch.all(out == 0)
    out, ids, _ = fg8.moe_decode(x[:0], *L.weights(), 2, ids=ids[:0], affinity=torch.ones(0, 2, device="cuda"))
    assert out.shape == (0, 256)


def test_all_tokens_on_one_expert():
    """More tokens than a group holds, every one of them on the same experts."""
    L = Layer(4, 512, 256, seed=4)
    x = L.x(64)
    ids = torch.tensor([[3, 1]], device="cuda", dtype=torch.int32).repeat(64, 1)
    aff = torch.rand(64, 2, device="cuda") + 0.1
    out, _, _ = run(L, x, 2, ids=ids, affinity=aff, out_dtype=fg8.FG8_OUT_F32)
    check(L, x, ids, aff, out)


def test_equal_calls_equal_bits_on_one_workspace_of_many_sizes():
    """One workspace, zeroed once, through calls of different sizes; results repeat."""
    ws = fg8.moe_decode_workspace(64, 8, 2048, 768)
    La, Lb = Layer(16, 1024, 768, seed=5), Layer(5, 256, 128, seed=6)
    xa, xb = La.x(50), Lb.x(3)
    ra, rb = La.routing(50), Lb.routing(3)
    first = None
    for _ in range(4):
        oa, _, _ = run(La, xa, 8, ws=ws, logits=ra[0], bias=ra[1], out_dtype=fg8.FG8_OUT_F32)
        ob, _, _ = run(Lb, xb, 2, ws=ws, logits=rb[0], bias=rb[1], out_dtype=fg8.FG8_OUT_F32)
        if first is None:
            first = oa.clone(), ob.clone()
        assert torch.equal(oa, first[0]) and torch.equal(ob, first[1])


def test_close_to_the_chain_of_kernels():
    """The same layer through the many-token kernels: they differ by the chain's
    bf16 rows between the down-projection and the combine (2^-8 each at most)
    and by codes of h at rounding midpoints."""
    L = Layer(64, 2048, 768, seed=7)
    T, k = 24, 6
    x = L.x(T)
    logits, bias = L.routing(T)
    out, ids, aff = run(L, x, k, logits=logits, bias=bias, out_dtype=fg8.FG8_OUT_F32)
    act = fg8.route_quantize_act(logits, bias, x, k)
    hq, sh = fg8.grouped_gemm_swiglu_quant(act["xq"], act["sa"], L.wq_up, L.sw_up, act["offsets"])
    y = fg8.grouped_gemm(hq, sh, L.wq_dn, L.sw_dn, act["offsets"])
    want = fg8.unpermute_combine(y, act["token_row"], act["affinity"], out_dtype=fg8.FG8_OUT_F32)
    assert torch.equal(ids, act["ids"])
    assert ((out - want).norm() / want.norm()).item() <= 2.0 ** -8


def test_captured_graphs_share_a_workspace_and_a_side_stream():
    L = Layer(8, 512, 256, seed=8)
    ws = fg8.moe_decode_workspace(32, 4, 512, 256)
    st = fg8.new_status()
    s = torch.cuda.Stream()
    graphs = []
    for T in (1, 20):
        x, (logits, bias) = L.x(T), L.routing(T)
        bufs = dict(out=torch.empty(T, 512, device="cuda"), ids=torch.empty(T, 4, device="cuda", dtype=torch.int32),
                    affinity=torch.empty(T, 4, device="cuda"))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fg8.moe_decode(x, *L.weights(), 4, logits=logits, bias=bias, out_dtype=fg8.FG8_OUT_F32, workspace=ws,
                           dev_status=st, **bufs)
        graphs.append((g, x, logits, bias, bufs))
    for rep in range(3):
        for g, x, logits, bias, bufs in graphs:
            x.copy_(L.x(x.shape[0]))
            logits.copy_(L.routing(x.shape[0])[0])
            g.replay()
            torch.cuda.synchronize()
            assert st.item() == 0
            check(L, x, bufs["ids"], bufs["affinity"], bufs["out"])


def test_two_calls_at_once_on_their_own_workspaces():
    L = Layer(32, 1024, 512, seed=9)
    T, k = 30, 4
    streams = [torch.cuda.Stream() for _ in range(2)]
    xs = [L.x(T) for _ in streams]
    rs = [L.routing(T) for _ in streams]
    ws = [fg8.moe_decode_workspace(T, k, 1024, 512) for _ in streams]
    st = [fg8.new_status() for _ in streams]
    want = [run(L, x, k, logits=r[0], bias=r[1])[0].clone() for x, r in zip(xs, rs)]
    torch.cuda.synchronize()
    outs = [torch.empty(T, 1024, device="cuda", dtype=torch.bfloat16) for _ in streams]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                fg8.moe_decode(xs[i], *L.weights(), k, logits=rs[i][0], bias=rs[i][1], out=outs[i], workspace=ws[i],
                               dev_status=st[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert st[i].item() == 0 and torch.equal(outs[i], want[i])


def test_saturating_inputs():
    """Tokens of very different sizes in one batch, zeros among them."""
    L = Layer(4, 256, 256, seed=10)
    x = L.x(6)
    x[0] *= 300.0
    x[1] *= 1e-6
    x[2] = 0
    ids = torch.tensor([[0, 1]] * 6, device="cuda", dtype=torch.int32)
    aff = torch.rand(6, 2, device="cuda") + 0.1
    out, _, _ = run(L, x, 2, ids=ids, affinity=aff, out_dtype=fg8.FG8_OUT_F32)
    assert torch.all(out[2] == 0)
    for t in range(6):
        check(L, x[t:t + 1], ids[t:t + 1], aff[t:t + 1], out[t:t + 1])


@pytest.mark.parametrize("calls", [2 ** 29 - 1, 2 ** 30 - 2, 2 ** 31 - 2, 2 ** 32 - 2])
def test_call_numbers_that_come_round(calls):
    """The workspace counts calls in 32 bits and tags partial sums with them.  The
    counters are set as after `calls` calls, and (at a multiple of 2^29, where old
    words are cleared) every partial to a word that a call 2^30 before left."""
    L = Layer(8, 1024, 512, 77)
    x, (lg, bi) = L.x(5), L.routing(5)
    want = run(L, x, 2, logits=lg, bias=bi)[0]
    ws = fg8.moe_decode_workspace(5, 2, L.C, L.I)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    i32 = lambda v: (v + 2 ** 31) % 2 ** 32 - 2 ** 31   # noqa: E731
    head = ws[:4096].view(torch.int32)
    head[:2] = i32(calls * ctas)
    head[2:2 + ctas] = i32(calls)
    if (calls + 1) % 2 ** 29 == 0:
        words = ws[4096:4096 + 2 * 160 * 64 * 128 * 8].view(torch.int32).view(2, 160, 64 * 128, 2)
        words[..., 0] = 0x41200000   # 10.0
        words[0, ..., 1] = i32(4 * (calls + 2) + 1)
        words[1, ..., 1] = i32(4 * (calls + 2) + 2)
    for _ in range(5):
        assert torch.equal(run(L, x, 2, ws=ws, logits=lg, bias=bi)[0], want)


@pytest.mark.parametrize("handle", [False, True])
def test_default_workspace_is_zeroed_on_the_given_stream(handle):
    """The current stream is held up: what the call needs zeroed may not wait in it."""
    L = Layer(8, 1024, 512, 78)
    x, (lg, bi) = L.x(4), L.routing(4)
    want = run(L, x, 2, logits=lg, bias=bi)[0]
    tr = torch.arange(8, dtype=torch.int32, device="cuda")
    aff = torch.rand(4, 2, device="cuda")
    side = torch.cuda.Stream()
    dirty = torch.full((40 << 20,), 0x5A, dtype=torch.uint8, device="cuda")
    st = fg8.new_status()
    torch.cuda.synchronize()
    del dirty                          # the allocator hands this memory out again
    torch.cuda._sleep(100_000_000)     # about 50 ms
    s = side.cuda_stream if handle else side
    got, _, _ = fg8.moe_decode(x, *L.weights(), 2, logits=lg, bias=bi, dev_status=st, stream=s)
    w = fg8.gate_weights(tr, aff, 8, normalize=False, stream=s)
    side.synchronize()
    torch.cuda.synchronize()
    assert st.item() == 0 and torch.equal(got, want)
    assert torch.equal(w, aff.flatten())


def test_largest_routing():
    """64 tokens in 16 slots of 1024 experts, and all their slots on the last expert."""
    L = Layer(1024, 128, 128, 79)
    x, (lg, bi) = L.x(64), L.routing(64)
    out, ids, aff = run(L, x, 16, logits=lg, bias=bi)
    check(L, x, ids, aff, out)
    ids = torch.full((64, 16), 1023, dtype=torch.int32, device="cuda")
    out, _, _ = run(L, x, 16, ids=ids, affinity=aff, out_dtype=fg8.FG8_OUT_F32)
    check(L, x, ids, aff, out)


def test_a_tokens_nan_stays_its_own():
    L = Layer(6, 384, 256, 80)
    x, (lg, bi) = L.x(20), L.routing(20)
    want = run(L, x, 3, logits=lg, bias=bi)[0]
    x[7, 100] = float("nan")
    x[13, 3] = float("inf")
    got = run(L, x, 3, logits=lg, bias=bi)[0]
    rest = [t for t in range(20) if t not in (7, 13)]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[7]).all() and torch.isnan(got[13]).all()


@pytest.mark.parametrize("E", [3, 64, 65, 256, 1000])
def test_routing_is_the_routing_kernels_with_ties_and_masked_experts(E):
    """Equal scores, experts masked by a bias of -inf, saturated logits: the ids and
    affinities of the routing kernel, bit for bit."""
    k = min(E, 7)
    L = Layer(E, 128, 128, 81)
    for T in (1, 5, 64):
        x, (lg, bi) = L.x(T), L.routing(T)
        lg = (2 * lg).round() / 2      # ties
        lg[0, 0], lg[-1, -1] = 200.0, -200.0
        bi = torch.zeros_like(bi)
        bi[::3] = float("-inf")        # E = 3: fewer finite experts than slots
        out, ids, aff = run(L, x, k, logits=lg, bias=bi)
        want = fg8.route_topk(lg, bi, k)
        assert torch.equal(ids, want[0]) and torch.equal(aff, want[1])
        check(L, x, ids, aff, out)


def test_default_workspace_on_the_default_stream_by_handle():
    L = Layer(4, 256, 128, 82)
    x, (lg, bi) = L.x(2), L.routing(2)
    want = run(L, x, 2, logits=lg, bias=bi)[0]
    got = run(L, x, 2, logits=lg, bias=bi, stream=torch.cuda.default_stream().cuda_stream)[0]
    assert torch.equal(got, want)


def test_input_codes_are_the_quantizers_bit_for_bit():
    """x's codes and scales, in a kept workspace, are those of quantize_act_rows: for
    tiles of every mantissa of the maximum, values on exact midpoints between two
    codes, subnormal scales and tiles of zeros."""
    T, C = 64, 1024
    L = Layer(2, C, 128, 83)
    x = L.x(T).float()
    tiles = x.view(T, C // 128, 128)
    m = torch.arange(128, device="cuda").float() / 128 + 1          # every bf16 mantissa
    tiles[:16] *= 0.1
    tiles[:16, :, 5] = 8.0 * m.view(16, 8)                          # as the tile's maximum, random values below
    tiles[16:32, :, :] = (m.flip(0) * torch.exp2(-(torch.arange(128, device="cuda") % 17).float()))[None, None]
    tiles[16:32, :, 0] = 2 * m.view(16, 8)                          # every mantissa over every maximum
    # scales that are powers of two: all values midpoints (5 significant bits, or halves of the smallest code)
    mid = (2 * torch.randint(0, 8, (16, 8, 128), generator=L.g, device="cuda") + 17).float()
    mid *= torch.exp2(torch.randint(-9, 4, (16, 8, 128), generator=L.g, device="cuda").float())
    low = (torch.randint(0, 8, (16, 8, 128), generator=L.g, device="cuda").float() + 0.5) * 2.0 ** -9
    tiles[32:48] = torch.where(torch.rand((16, 8, 128), generator=L.g, device="cuda") < 0.8, mid, low)
    tiles[32:48, :, 77] = 448.0
    tiles[32:48] *= torch.exp2(torch.randint(-30, 30, (16, 8, 1), generator=L.g, device="cuda").float())
    tiles[48:56] *= torch.exp2(-110 - 2.0 * torch.arange(8, device="cuda").float())[:, None, None]
    tiles[56:58] = 0
    tiles[58] *= 1e30
    x *= torch.where(torch.rand(x.shape, generator=L.g, device="cuda") < 0.5, -1.0, 1.0)
    x = x.to(torch.bfloat16)
    ws = fg8.moe_decode_workspace(T, 2, C, 128)
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device="cuda")
    run(L, x, 2, ws=ws, ids=ids, affinity=torch.ones(T, 2, device="cuda"))
    want_q, want_s = fg8.quantize_act_rows(x)
    at = fg8.FG8_MOE_DECODE_HEAD
    got_q = ws[at:at + T * C].view(T, C)
    at += (T * C + 255) // 256 * 256
    got_s = ws[at:at + 4 * T * (C // 128)].view(torch.float32).view(T, C // 128)
    assert torch.equal(got_s.t(), want_s)
    assert torch.equal(got_q, want_q)


def _winds_down(L, x, k, routing, head, status, limit, T):
    """A call whose counters are set to `head` (int32 words of the workspace's first
    4096 bytes) gives up with `status`; the context stays usable, and with the
    workspace zeroed again the next call is right."""
    import time
    ws = fg8.moe_decode_workspace(T, k, L.C, L.I)
    want = run(L, x, k, logits=routing[0], bias=routing[1])[0]
    words = ws[:4096].view(torch.int32)
    words[:len(head)] = torch.tensor(head, dtype=torch.int32, device="cuda")
    before = words.clone()
    st = fg8.new_status()
    torch.cuda.synchronize()
    t0 = time.monotonic()
    fg8.moe_decode(x, *L.weights(), k, logits=routing[0], bias=routing[1], workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < limit
    assert st.item() == status
    after = words.clone()
    ws.zero_()
    for _ in range(2):
        assert torch.equal(run(L, x, k, ws=ws, logits=routing[0], bias=routing[1])[0], want)
    return before, after


@pytest.mark.parametrize("T,E,k,C,I", [(1, 64, 6, 2048, 768), (20, 8, 4, 512, 256), (2, 3, 2, 256, 128)])
def test_codes_that_never_come_time_out(T, E, k, C, I):
    """The counter of CTAs that have written x's codes starts so far behind that the
    wait runs out, with weight copies in flight and few or many steps a CTA: the call
    reports it, lands its copies and ends; no CTA goes on to the next meeting."""
    L = Layer(E, C, I, seed=84)
    before, after = _winds_down(L, L.x(T), k, L.routing(T), [-10_000_000], fg8.FG8_ERR_TIMEOUT, 30.0, T)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    assert after[0].item() == before[0].item() + ctas      # every CTA wrote its codes
    assert (after[2:2 + ctas] == 0).any()                  # CTAs with a share of the up-projection did not finish


@pytest.mark.parametrize("T,E,k,C,I", [(1, 64, 6, 2048, 768), (20, 8, 4, 512, 256), (2, 3, 2, 256, 128)])
@pytest.mark.parametrize("meeting", [0, 1])
def test_a_workspace_that_another_call_uses_stops_the_call(T, E, k, C, I, meeting):
    """A meeting's counter holds the arrivals of another call's CTAs, as two calls at
    once on one workspace leave it: the call reports it and ends without going on to
    what it could not wait for, and says so again until the workspace is zeroed."""
    L = Layer(E, C, I, seed=85)
    x, routing = L.x(T), L.routing(T)
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    head = [2 * ctas] if meeting == 0 else [0, 2 * ctas]
    before, after = _winds_down(L, x, k, routing, head, fg8.FG8_ERR_WORKSPACE_SHARED, 10.0, T)
    assert after[0].item() == before[0].item() + ctas
    if meeting == 0:
        assert (after[2:2 + ctas] == 0).any()    # CTAs with a share of the up-projection did not finish
    # a workspace with both counters ahead, as after such a call
    ws = fg8.moe_decode_workspace(T, k, C, I)
    ws[:4096].view(torch.int32)[:2] = ctas
    for _ in range(2):
        st = fg8.new_status()
        fg8.moe_decode(x, *L.weights(), k, logits=routing[0], bias=routing[1], workspace=ws, dev_status=st)
        torch.cuda.synchronize()
        assert st.item() == fg8.FG8_ERR_WORKSPACE_SHARED
