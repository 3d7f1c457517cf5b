"""The 8-bit checkpointed backward of the expert layer against its formulas in
64 bits: the up-projection that saves gate and up, the gated activation's
backward with its three quantizations, the column-wise operand from saved rows,
the gate weights and the router's gradient, and all of them together with the
GEMMs.

Tolerances (derived, with eps = 2^-24 the fp32 half step):
  * g = code * scale: eps relative.  exp(-g): the argument's two roundings and
    the hardware's 2^-22 give (2 |g| + 4) eps relative, and the reciprocal 2 eps
    more, so sig is within SIG(g) = (2 |g| + 8) eps relative.
  * h = g sig u: SIG + 5 eps; dU = d g sig: the same.
  * dG = d u sig (1 + g - g sig): the last factor is a sum of terms up to
    1 + |g|, so it is off by (1 + |g|) (SIG + 4 eps) absolutely; the product adds
    SIG + 5 eps of itself.
  * a tile's scale is off by its largest value's error / 448 and eps; a code is
    the nearest one to within half a step (E4M3 step: 2^-3 of the binade), plus
    the value's own error and that of the scale, taken as twice the value's error.
"""

import numpy as np
import pytest
import torch

from fp8_fine_grained_permute_b200 import build as fbuild
from fp8_fine_grained_permute_b200 import fg8
from fp8_fine_grained_permute_b200 import workloads as W

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
CANARY = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fbuild.build()
    fg8.lib()
    torch.cuda.init()


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def padded(counts):
    return np.concatenate([[0], np.cumsum((np.asarray(counts) + 127) // 128 * 128)]).astype(np.int32)


def deq_rows(oracle, q, s):
    """codes [R, C], scales [C/128, R] -> fp64."""
    return oracle.e4m3_decode_table()[q].astype(np.float64) * np.repeat(s.T.astype(np.float64), 128, axis=1)


def half_step(x):
    ax = np.maximum(np.abs(x), 2.0 ** -6)
    return 0.5 * 2.0 ** (np.floor(np.log2(ax)) - 3)


def check_tiles(oracle, q, s, v, tol, what):
    """q [n, C] codes and s [n, C/128] scales of v (fp64, off by at most tol),
    one tile per row and 128 columns."""
    n, C = v.shape
    vt, tt = v.reshape(n, C // 128, 128), tol.reshape(n, C // 128, 128)
    amax, tmax = np.abs(vt).max(2), tt.max(2)
    s64 = s.astype(np.float64)
    zero = amax == 0
    assert np.all(s64[zero] == 1.0), what
    err = np.abs(448.0 * s64 - amax)
    lim = tmax + 4 * EPS * amax + 448 * 2.0 ** -149
    assert np.all(err[~zero] <= lim[~zero]), f"{what}: scale off by {np.max((err / lim)[~zero])} of its limit"
    se = np.repeat(s64, 128, axis=1)
    deq = oracle.e4m3_decode_table()[q].astype(np.float64) * se
    x = np.maximum(np.abs(v), np.abs(deq)) / se
    lim = half_step(x) * se * (1 + 2.0 ** -20) + 2 * tol + 2.0 ** -140
    bad = np.abs(deq - v) > lim
    assert not bad.any(), f"{what}: {bad.sum()} codes out of bounds"


def check_columns(oracle, qT, sT, v, tol, counts, what):
    """qT [C, P], sT [P/128, C]: v's rows per expert in tiles of 128, padded; the
    columns behind the last expert keep the canary."""
    C, P = qT.shape
    off, pad = offsets_of(counts), padded(counts)
    used = pad[-1]
    vp, tp = np.zeros((used, C)), np.zeros((used, C))
    real = np.zeros(used, bool)
    for e, c in enumerate(counts):
        vp[pad[e]:pad[e] + c] = v[off[e]:off[e + 1]]
        tp[pad[e]:pad[e] + c] = tol[off[e]:off[e + 1]]
        real[pad[e]:pad[e] + c] = True
    assert np.all(qT[:, used:] == CANARY), what
    assert np.all(qT[:, :used][:, ~real] == 0), f"{what}: padding codes"
    if used:
        check_tiles(oracle, qT[:, :used], sT[:used // 128].T, vp.T, tp.T, what)


# ---------------------------------------------------------------------------
# the activation's backward
# ---------------------------------------------------------------------------

def act_case(counts, I, seed, extra_rows=0, gscale=2.0 ** -7, weights=True):
    rng = np.random.default_rng(seed)
    R = int(sum(counts)) + extra_rows
    guq = W.gen_e4m3_codes((R, 2 * I), seed, 1).numpy()
    sgu = (gscale * np.exp2(rng.uniform(-3, 1, (2 * I // 128, R)))).astype(np.float32)
    dh = (rng.standard_t(3, (R, I)) * np.exp(rng.standard_normal((R, 1)))).astype(np.float32)
    dh = torch.from_numpy(dh).to(torch.bfloat16)
    w = rng.uniform(0.01, 1.0, R).astype(np.float32) if weights else None
    return dict(counts=counts, I=I, R=R, guq=guq, sgu=sgu, dh=dh, w=w)


def act_run(c, stream=None):
    E, I, R = len(c["counts"]), c["I"], c["R"]
    P = fg8.fg8_colwise_capacity(R, E)
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    u8 = lambda *s: torch.full(s, CANARY, dtype=torch.uint8, device="cuda")   # noqa: E731
    o = dict(dq=u8(R, 2 * I), dqT=u8(2 * I, P), hqT=u8(I, P),
             sd=torch.full((2 * I // 128, R), -7.0, device="cuda"),
             gate_dot=torch.full((I // 128, R), -7.0, device="cuda"))
    st = fg8.new_status()
    out = fg8.swiglu_backward_quant(c["dh"].cuda(), g(c["guq"]), g(c["sgu"]), g(offsets_of(c["counts"])),
                                    row_w=None if c["w"] is None else g(c["w"]), dev_status=st,
                                    stream=stream, **o)
    torch.cuda.synchronize()
    assert st.item() == 0
    return {k: v.cpu().numpy() for k, v in out.items()}


def act_formula(oracle, c):
    I, R = c["I"], c["R"]
    gu = deq_rows(oracle, c["guq"], c["sgu"])
    g, u = gu[:, :I], gu[:, I:]
    dh = c["dh"].double().numpy()
    w = np.ones((R, 1)) if c["w"] is None else c["w"].astype(np.float64)[:, None]
    sig = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    h, d = g * sig * u, dh * w
    SIG = (2 * np.abs(g) + 8) * EPS
    # below exp(-125 ln 2) the kernel holds sig at 2^-125: that much absolutely
    # (or lets it go to 0 below 2^-126, as it does now: within the same)
    floor = 2.0 ** -124
    dG, dU = d * u * sig * (1 + g * (1 - sig)), d * g * sig
    tG = (np.abs(d * u * sig) * ((1 + np.abs(g)) * (SIG + 4 * EPS)) + np.abs(dG) * (SIG + 5 * EPS)
          + np.abs(d * u) * (1 + np.abs(g)) * floor)
    tU = np.abs(dU) * (SIG + 5 * EPS) + np.abs(d * g) * floor
    tH = np.abs(h) * (SIG + 5 * EPS) + np.abs(g * u) * floor
    return dict(dG=dG, dU=dU, wh=w * h, h=h, tG=tG, tU=tU, twh=w * tH + EPS * np.abs(w * h), th=tH, dh=dh)


def act_check(oracle, c, out):
    I, n = c["I"], int(sum(c["counts"]))
    f = act_formula(oracle, c)
    v = np.concatenate([f["dG"], f["dU"]], 1)
    t = np.concatenate([f["tG"], f["tU"]], 1)
    check_tiles(oracle, out["dq"][:n], out["sd"][:, :n].T, v[:n], t[:n], "rows")
    assert np.all(out["dq"][n:] == CANARY) and np.all(out["sd"][:, n:] == -7.0)
    assert np.array_equal(out["offsets_out"], padded(c["counts"]))
    check_columns(oracle, out["dqT"], out["sdT"], v[:n], t[:n], c["counts"], "columns of dG, dU")
    check_columns(oracle, out["hqT"], out["shT"], f["wh"][:n], f["twh"][:n], c["counts"], "columns of w h")
    dot = (f["dh"] * f["h"]).reshape(c["R"], I // 128, 128).sum(2).T
    mag = np.abs(f["dh"] * f["h"]).reshape(c["R"], I // 128, 128).sum(2).T
    tol = (np.abs(f["dh"]) * f["th"]).reshape(c["R"], I // 128, 128).sum(2).T + 16 * EPS * mag + 1e-30
    assert np.all(np.abs(out["gate_dot"] - dot)[:, :n] <= tol[:, :n])
    assert np.all(out["gate_dot"][:, n:] == -7.0)


@pytest.mark.parametrize("counts,I,extra", [
    ([1], 128, 0), ([127, 1, 0, 130], 256, 0), ([0, 0, 5], 384, 3), ([128, 256, 64], 128, 0),
    ([300, 0, 17, 129, 1, 1, 640], 640, 7), ([0, 0], 128, 4), ([3] * 200, 256, 0)])
def test_act_backward_matches_formula(oracle, counts, I, extra):
    c = act_case(counts, I, seed=sum(counts) + I, extra_rows=extra)
    act_check(oracle, c, act_run(c))


def test_act_backward_saturated_gates_zero_rows_and_no_weights(oracle):
    c = act_case([200, 60], 256, seed=5, gscale=1.0, weights=False)   # gates up to +-900
    c["dh"][7] = 0                                      # an all-zero row: scale 1
    c["dh"][:, 3] = 0                                   # an all-zero column
    c["guq"][:, 256 + 9] = 0                            # up = 0: dG and h vanish there
    c["guq"][11] = 0                                    # gate and up 0: silu(0) = 0
    act_check(oracle, c, act_run(c))


def test_act_backward_tiny_scales(oracle):
    """Gradients whose tiles have subnormal scales take the division."""
    c = act_case([140], 128, seed=6)
    c["dh"] = (c["dh"].float() * 2.0 ** -124).to(torch.bfloat16)
    out = act_run(c)
    f = act_formula(oracle, c)
    v = np.concatenate([f["dG"], f["dU"]], 1)
    # products may round into the subnormal range: 2^-149 absolutely, a few times
    t = np.concatenate([f["tG"], f["tU"]], 1) + 2.0 ** -146 * (1 + np.abs(np.tile(deq_rows(oracle, c["guq"], c["sgu"])[:, 128:], 2)))
    s = out["sd"].T.astype(np.float64)
    assert np.all(s > 0) and np.any(s < 2.0 ** -126)
    check_tiles(oracle, out["dq"], out["sd"].T, v, t, "rows")


def test_act_backward_garbage_outside_the_experts_rows(oracle):
    """Rows of the buffers that no expert owns, and the next expert's rows in a
    tile, take no part: NaN codes there change nothing."""
    counts = [70, 133]
    c = act_case(counts, 256, seed=8, extra_rows=40)
    ref = act_run(c)
    d = {k: (v.copy() if isinstance(v, np.ndarray) else v.clone() if torch.is_tensor(v) else v) for k, v in c.items()}
    d["guq"][sum(counts):] = 0x7F
    d["dh"][sum(counts):] = float("nan")
    out = act_run(d)
    for k in ref:
        a, b = ref[k], out[k]
        if k in ("sdT", "shT"):
            used = padded(counts)[-1] // 128
            a, b = a[:used], b[:used]
        assert np.array_equal(a, b), k


def test_act_backward_nonfinite_values_of_the_next_expert(oracle):
    """A tile's rows behind an expert's last belong to the next one: infinities and
    NaN there change nothing of the first expert's."""
    counts = [70, 133, 3]
    c = act_case(counts, 256, seed=18)
    ref = act_run(c)
    d = {k: (v.copy() if isinstance(v, np.ndarray) else v.clone() if torch.is_tensor(v) else v) for k, v in c.items()}
    d["dh"][70:203:2] = float("inf")
    d["dh"][71:203:3] = float("nan")
    d["guq"][70:203:5] = 0x7F
    d["sgu"][:, 72:203] = np.inf
    d["w"][75:203:4] = np.nan
    out = act_run(d)
    for e, (r0, r1) in ((0, (0, 70)), (2, (203, 206))):
        for k in ("dq", "sd", "gate_dot"):
            a, b = (ref[k], out[k]) if k == "dq" else (ref[k].T, out[k].T)
            assert np.array_equal(a[r0:r1], b[r0:r1]), (e, k)
        p0, p1 = padded(counts)[e], padded(counts)[e + 1]
        for k in ("dqT", "hqT"):
            assert np.array_equal(ref[k][:, p0:p1], out[k][:, p0:p1]), (e, k)
        for k in ("sdT", "shT"):
            assert np.array_equal(ref[k][p0 // 128:p1 // 128], out[k][p0 // 128:p1 // 128]), (e, k)


def test_act_backward_gradient_against_differences(oracle):
    """A central difference of L = sum w dh h along a random direction."""
    c = act_case([150, 20], 128, seed=9)
    out = act_run(c)
    I = c["I"]
    gu = deq_rows(oracle, c["guq"], c["sgu"])
    v = np.random.default_rng(1).standard_normal(gu.shape) * np.maximum(np.abs(gu), 1e-3)
    dh, w = c["dh"].double().numpy(), c["w"].astype(np.float64)[:, None]
    L = lambda x: np.sum(w * dh * x[:, I:] * x[:, :I] / (1 + np.exp(-x[:, :I])))   # noqa: E731
    step = 1e-5
    want = (L(gu + step * v) - L(gu - step * v)) / (2 * step)
    got = deq_rows(oracle, out["dq"], out["sd"])
    se = np.repeat(out["sd"].T.astype(np.float64), 128, axis=1)
    # every element is off by at most half a step; the difference by ~step^2
    bound = np.sum(half_step(got / se) * se * 1.01 * np.abs(v)) + 1e-6 * np.sum(np.abs(got * v))
    assert abs(np.sum(got * v) - want) <= bound
    # and the weights' gradient: L is linear in w
    dw = out["gate_dot"].sum(0).astype(np.float64)
    assert abs(np.sum(dw * w[:, 0]) - L(gu)) <= 1e-5 * np.sum(np.abs(w * dh * gu[:, I:] * gu[:, :I]))


# ---------------------------------------------------------------------------
# column-wise operand from saved rows
# ---------------------------------------------------------------------------

def requant_reference(oracle, q, s, row_token, counts):
    """fp32 arithmetic of the definition, value by value, with codes by the oracle's table."""
    x = oracle.e4m3_decode_table()[q].astype(np.float32) * np.repeat(s.T, 128, axis=1)
    rows = x if row_token is None else np.where((row_token >= 0)[:, None] & (row_token < len(x))[:, None],
                                                x[np.clip(row_token, 0, len(x) - 1)], np.float32(0))
    off, pad = offsets_of(counts), padded(counts)
    C = q.shape[1]
    v = np.zeros((pad[-1], C), np.float32)
    for e, c in enumerate(counts):
        v[pad[e]:pad[e] + c] = rows[off[e]:off[e + 1]]
    t = v.reshape(-1, 128, C)
    amax = np.abs(t).max(1)
    sT = np.where(amax == 0, np.float32(1), amax / np.float32(448))
    sT = np.where(sT == 0, np.float32(2.0 ** -149), sT)     # the quotient rounded to 0
    z = torch.from_numpy(t / sT[:, None, :]).clamp(-448, 448)   # the cast alone does not saturate
    codes = z.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes.reshape(-1, C).T, sT, pad


@pytest.mark.parametrize("counts,K,gather,extra", [
    ([1], 128, False, 0), ([200, 0, 129, 1], 256, True, 0), ([5, 5, 5], 640, True, 2),
    ([128, 128], 128, False, 0), ([1000, 3, 0, 270], 384, True, 0)])
def test_requantize_matches_definition_bit_for_bit(oracle, counts, K, gather, extra):
    rng = np.random.default_rng(K + sum(counts))
    R = int(sum(counts)) + extra
    T = 97 if gather else R
    q = W.gen_e4m3_codes((T, K), 3, K).numpy()
    s = np.exp2(rng.uniform(-12, 4, (K // 128, T))).astype(np.float32)
    row_token = rng.integers(0, T, R).astype(np.int32) if gather else None
    if gather:
        row_token[:3] = row_token[0]           # the same token more than once
    g = lambda x: torch.from_numpy(x).cuda()   # noqa: E731
    P = fg8.fg8_colwise_capacity(R, len(counts))
    buf = torch.full((K, P), CANARY, dtype=torch.uint8, device="cuda")
    st = fg8.new_status()
    xqT, sT, pad = fg8.requantize_colwise(g(q), g(s), g(offsets_of(counts)), None if row_token is None else g(row_token),
                                          xqT=buf, dev_status=st)
    torch.cuda.synchronize()
    codes, ref_s, ref_pad = requant_reference(oracle, q, s, row_token, counts)
    used = ref_pad[-1]
    assert st.item() == 0 and np.array_equal(pad.cpu().numpy(), ref_pad)
    assert np.array_equal(sT.cpu().numpy()[:used // 128], ref_s)
    got = xqT.cpu().numpy()
    assert np.array_equal(got[:, :used], codes)
    assert np.all(got[:, used:] == CANARY)


def test_requantize_equal_scales_ties_tiny_scales_and_bad_rows(oracle):
    """Equal row scales (every quotient a code or an exact midpoint), scales that
    make the column scale subnormal, and a row index out of range."""
    K, counts = 256, [130]
    q = W.gen_e4m3_codes((130, K), 4, 4).numpy()
    s = np.full((2, 130), 0.5, np.float32)
    s[0, ::3] = 0.25                    # quotients halve: midpoints among the subnormal codes
    s[1] = np.float32(2.0 ** -140)      # values and column scales below the normal range
    rt = np.arange(130, dtype=np.int32)
    rt[17], rt[40] = -1, 5000
    g = lambda x: torch.from_numpy(x).cuda()   # noqa: E731
    st = fg8.new_status()
    xqT, sT, _ = fg8.requantize_colwise(g(q), g(s), g(offsets_of(counts)), g(rt), dev_status=st)
    torch.cuda.synchronize()
    codes, ref_s, pad = requant_reference(oracle, q, s, rt, counts)
    assert st.item() == fg8.FG8_ERR_INVALID_ARG
    assert np.array_equal(sT.cpu().numpy()[:2], ref_s)
    assert np.array_equal(xqT.cpu().numpy()[:, :256], codes)


# ---------------------------------------------------------------------------
# gate weights and the router's gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k,nb,normalize", [(1, 4, 1, 1, True), (37, 64, 6, 6, True), (300, 5, 3, 9, False),
                                                (129, 1000, 16, 16, True), (65, 7, 2, 1, True), (513, 256, 8, 16, True)])
def test_gates_match_formula(T, E, k, nb, normalize):
    rng = np.random.default_rng(T + E)
    R = T * k
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    aff = rng.uniform(0.01, 0.99, (T, k)).astype(np.float32)
    tr = rng.permutation(R).astype(np.int32).reshape(T, k)
    dot = rng.standard_normal((nb, R)).astype(np.float32)
    if T > 10:
        tr[3, 0] = -1                  # a slot without a row
        tr[5] = -1                     # a token without rows
        tr[6, k - 1] = R + 3
        aff[7] = 0.0                   # affinities that sum to 0
        ids[8] = ids[8, 0]             # one expert in every slot
        ids[9, 0] = E                  # a bad id: no logit to give its gradient to
    g = lambda x: torch.from_numpy(x).cuda()   # noqa: E731
    row_w = torch.full((R,), -7.0, device="cuda")
    fg8.gate_weights(g(tr.ravel()), g(aff), R, normalize=normalize, row_w=row_w)
    daff, dlog = fg8.gate_backward(g(dot), g(tr.ravel()), g(ids), g(aff), E, normalize=normalize,
                                   dlogits=torch.full((T, E), 3.0, device="cuda"))
    daff2, _ = fg8.gate_backward(g(dot), g(tr.ravel()), g(ids), g(aff), E, normalize=normalize)
    torch.cuda.synchronize()
    assert torch.equal(daff, daff2)
    kept = (tr >= 0) & (tr < R)
    # weights: the combine's own arithmetic, bit for bit
    want = np.full(R, -7.0, np.float32)
    for t in range(T):
        s = np.float32(0)
        for j in range(k):
            if kept[t, j]:
                s = np.float32(s + aff[t, j])
        for j in range(k):
            if kept[t, j]:
                want[tr[t, j]] = aff[t, j] if not normalize else (aff[t, j] / s if s != 0 else 0.0)
    assert np.array_equal(row_w.cpu().numpy(), want)
    # gradients
    a = np.where(kept, aff.astype(np.float64), 0)
    D = np.where(kept, dot.astype(np.float64).sum(0)[np.clip(tr, 0, R - 1)], 0)
    M = np.where(kept, np.abs(dot.astype(np.float64)).sum(0)[np.clip(tr, 0, R - 1)], 0)
    S = a.sum(1, keepdims=True)
    if normalize:
        ok = S != 0
        w = a / np.where(ok, S, 1)
        da = np.where(ok & kept, (D - (w * D).sum(1, keepdims=True)) / np.where(ok, S, 1), 0)
        # sums of nb terms, then k products and adds, a subtraction and a division
        tol = (nb + 2 * k + 8) * EPS * 2 * (M + (w * M).sum(1, keepdims=True)) / np.where(ok, S, 1) + 1e-38
    else:
        da, tol = D, (nb + 2) * EPS * M + 1e-38
    got = daff.cpu().numpy()
    assert np.all(np.abs(got - da) <= tol)
    assert np.all(got[~kept] == 0)
    dl, tl = np.zeros((T, E)), np.full((T, E), 1e-38)
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                v = aff[t, j] * (1 - aff[t, j].astype(np.float64))
                dl[t, ids[t, j]] += da[t, j] * v
                tl[t, ids[t, j]] += tol[t, j] * v + (k + 6) * EPS * abs(da[t, j]) * v
    got = dlog.cpu().numpy()
    assert np.all(np.abs(got - dl) <= tl)
    hit = np.zeros((T, E), bool)
    for t in range(T):
        hit[t, ids[t][(ids[t] >= 0) & (ids[t] < E)]] = True
    assert np.all(got[~hit] == 0)


@pytest.mark.parametrize("normalize", [True, False])
def test_gate_backward_dropped_slots_affinity_may_be_anything(normalize):
    T, E, k = 5, 7, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    aff = torch.rand(T, k, device="cuda", generator=g)
    ids = torch.tensor([[0, 1, 2], [3, 4, 5], [6, 0, 1], [2, 3, 4], [5, 6, 0]], dtype=torch.int32, device="cuda")
    tr = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    dot = torch.randn(2, T * k, device="cuda", generator=g)
    tr[1, 2] = tr[3, 0] = -1
    aff[1, 2], aff[3, 0] = 0.5, 0.5
    want = fg8.gate_backward(dot, tr, ids, aff, E, normalize=normalize)
    aff[1, 2], aff[3, 0] = float("nan"), float("inf")
    got = fg8.gate_backward(dot, tr, ids, aff, E, normalize=normalize)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.isfinite(got[1]).all()


def test_gate_gradient_against_differences():
    """d/dlogits of L = sum_j w_j D_j with w from the logits, by central differences in 64 bits."""
    rng = np.random.default_rng(2)
    T, E, k = 20, 12, 4
    u = rng.standard_normal((T, E))
    ids = np.argsort(-u, 1)[:, :k].astype(np.int32)
    D = rng.standard_normal((T, k))
    aff = (1 / (1 + np.exp(-np.take_along_axis(u, ids, 1)))).astype(np.float32)
    rows = np.arange(T * k, dtype=np.int32)
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    _, dl = fg8.gate_backward(g(D.astype(np.float32).reshape(1, -1)), g(rows), g(ids), g(aff), E)
    L = lambda x: (lambda a: np.sum(a / a.sum(1, keepdims=True) * D))(1 / (1 + np.exp(-np.take_along_axis(x, ids, 1))))  # noqa: E731
    for _ in range(5):
        v = rng.standard_normal((T, E))
        want = (L(u + 1e-5 * v) - L(u - 1e-5 * v)) / 2e-5
        got = np.sum(dl.double().cpu().numpy() * v)
        # fp32 inputs and arithmetic: a few tens of eps of the terms' sizes
        assert abs(got - want) <= 200 * EPS * np.sum(np.abs(v)) * np.abs(D).max() + 1e-8


# ---------------------------------------------------------------------------
# the saving up-projection
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("counts,I,K,extra", [([1], 128, 128, 0), ([127, 0, 130, 1], 256, 384, 5), ([300, 20], 384, 640, 0)])
def test_up_save_keeps_the_gemms_own_values(oracle, counts, I, K, extra):
    """h as from the kernel that saves nothing; the checkpoint is the 1x128
    quantization (IEEE division) of the plain GEMM's fp32 output, bit for bit:
    the same partial products in the same order."""
    R, E = int(sum(counts)) + extra, len(counts)
    a = W.gen_e4m3_codes((R, K), 1, 1).cuda()
    sa = torch.exp2(torch.empty((K // 128, R)).uniform_(-11, -7, generator=torch.Generator().manual_seed(1))).cuda()
    b = W.gen_e4m3_codes((E, 2 * I, K), 1, 3).cuda()
    sb = torch.exp2(torch.empty((E, 2 * I // 128, K // 128)).uniform_(-11, -7, generator=torch.Generator().manual_seed(2))).cuda()
    off = torch.from_numpy(offsets_of(counts)).cuda()
    bufs = dict(guq=torch.full((R, 2 * I), CANARY, dtype=torch.uint8, device="cuda"),
                sgu=torch.full((2 * I // 128, R), -7.0, device="cuda"),
                hq=torch.full((R, I), CANARY, dtype=torch.uint8, device="cuda"))
    st = fg8.new_status()
    hq, sh, guq, sgu = fg8.grouped_gemm_swiglu_quant_save(a, sa, b, sb, off, dev_status=st, **bufs)
    hq0, sh0 = fg8.grouped_gemm_swiglu_quant(a, sa, b, sb, off, dev_status=st)
    gu = fg8.grouped_gemm(a, sa, b, sb, off, out_dtype=fg8.FG8_OUT_F32, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    n = sum(counts)
    assert torch.equal(hq[:n], hq0[:n]) and torch.equal(sh[:, :n], sh0[:, :n])
    v = gu[:n].cpu().numpy().reshape(n, -1, 128)
    amax = np.abs(v).max(2)
    s = np.where(amax == 0, np.float32(1), amax / np.float32(448))
    codes = torch.from_numpy(v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(n, -1)
    assert np.array_equal(sgu[:, :n].cpu().numpy().T, s)
    assert np.array_equal(guq[:n].cpu().numpy(), codes)
    assert torch.all(guq[n:] == CANARY) and torch.all(sgu[:, n:] == -7.0) and torch.all(hq[n:] == CANARY)


@pytest.mark.parametrize("lo,hi", [(-64, -58), (-74, -66), (-52, -46)])
def test_up_save_tiny_and_zero_tiles(lo, hi):
    """Scales around 2^-100 and below the normal range (the codes' division) and
    rows of zeros: still the IEEE quotients of the plain GEMM's output."""
    R, E, K, I = 140, 2, 256, 256
    gen = torch.Generator().manual_seed(hi)
    a = W.gen_e4m3_codes((R, K), 1, 5).cuda()
    a[7] = 0
    a[139] = 0
    sa = torch.exp2(torch.empty((K // 128, R)).uniform_(lo, hi, generator=gen)).cuda()
    b = W.gen_e4m3_codes((E, 2 * I, K), 1, 6).cuda()
    b[0, :128] = 0
    sb = torch.exp2(torch.empty((E, 2 * I // 128, K // 128)).uniform_(lo, hi, generator=gen)).cuda()
    off = torch.from_numpy(offsets_of([100, 40])).cuda()
    hq, sh, guq, sgu = fg8.grouped_gemm_swiglu_quant_save(a, sa, b, sb, off)
    hq0, sh0 = fg8.grouped_gemm_swiglu_quant(a, sa, b, sb, off)
    gu = fg8.grouped_gemm(a, sa, b, sb, off, out_dtype=fg8.FG8_OUT_F32)
    torch.cuda.synchronize()
    assert torch.equal(hq, hq0) and torch.equal(sh, sh0)
    v = gu.cpu().numpy().reshape(R, -1, 128)
    amax = np.abs(v).max(2)
    s = np.where(amax == 0, np.float32(1), amax / np.float32(448))
    s = np.where(s == 0, np.float32(2.0 ** -149), s)
    z = torch.from_numpy(v / s[..., None]).clamp(-448, 448)
    assert np.array_equal(sgu.cpu().numpy().T, s)
    assert np.array_equal(guq.cpu().numpy(), z.to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(R, -1))


# ---------------------------------------------------------------------------
# together: one training step of the layer
# ---------------------------------------------------------------------------

def _step(x, logits, bias, wu, wd, dout, k):
    """Forward and backward of the expert layer through the library."""
    E, C, I = wd.shape
    T = x.shape[0]
    wuq, swu = fg8.quantize_weight(wu)
    wdq, swd = fg8.quantize_weight(wd)
    wuT, swuT = fg8.transpose_blockq(wuq, swu)
    wdT, swdT = fg8.transpose_blockq(wdq, swd)
    act = fg8.route_quantize_act(logits, bias, x, k)
    R, off = T * k, act["offsets"]
    x8, sx8 = fg8.quantize_act_rows(x)                      # what is kept of the input
    hq, sh, guq, sgu = fg8.grouped_gemm_swiglu_quant_save(act["xq"], act["sa"], wuq, swu, off)
    y = fg8.grouped_gemm(hq, sh, wdq, swd, off)
    out = fg8.unpermute_combine(y, act["token_row"], act["affinity"], out_dtype=fg8.FG8_OUT_F32)
    # backward
    ids = act["ids"]
    row_w = fg8.gate_weights(act["token_row"], act["affinity"], R)
    dact = fg8.quantize_act(dout, ids, E)
    dh = fg8.grouped_gemm(dact["xq"], dact["sa"], wdT, swdT, off)
    b = fg8.swiglu_backward_quant(dh, guq, sgu, off, row_w=row_w)
    dx_rows = fg8.grouped_gemm(b["dq"], b["sd"], wuT, swuT, off)
    dx = fg8.unpermute_combine(dx_rows, act["token_row"], torch.ones_like(act["affinity"]), normalize=False,
                               out_dtype=fg8.FG8_OUT_F32)
    xT, sxT, pad = fg8.requantize_colwise(x8, sx8, off, act["row_token"])
    doT, sdoT, _ = fg8.quantize_act_colwise(dout, off, k=k, row_token=act["row_token"])
    dwu = fg8.grouped_gemm(b["dqT"], b["sdT"], xT, sxT, pad, out_dtype=fg8.FG8_OUT_F32, group_mode=fg8.FG8_GROUP_K)
    dwd = fg8.grouped_gemm(doT, sdoT, b["hqT"], b["shT"], pad, out_dtype=fg8.FG8_OUT_F32, group_mode=fg8.FG8_GROUP_K)
    daff, dlogits = fg8.gate_backward(b["gate_dot"], act["token_row"], ids, act["affinity"], E)
    torch.cuda.synchronize()
    return dict(out=out, dx=dx, dwu=dwu, dwd=dwd, dlogits=dlogits, ids=ids)


def test_training_step_gradients_against_autograd_in_64_bits():
    """The whole layer's output and every gradient against autograd of the
    unquantized layer in 64 bits.  Every tensor that enters a GEMM carries E4M3's
    rounding: at most 2^-4 relative for a value, uniform inside its step, so an
    rms of at most 2^-4 / sqrt(3) = 0.036 of the tensor's own norm (independent
    over elements: it does not add up coherently in the contractions).  The
    longest chain, a weight gradient, multiplies operands that come from at most
    8 rounded tensors (x, Wu, h, gate and up, dout, Wd, the operand itself twice):
    sqrt(8) * 0.036 = 0.102 of the norm."""
    torch.manual_seed(3)
    T, E, k, C, I = 300, 6, 2, 256, 256
    x = torch.randn(T, C, device="cuda").to(torch.bfloat16)
    logits, bias = torch.randn(T, E, device="cuda"), 0.1 * torch.randn(E, device="cuda")
    wu = (torch.randn(E, 2 * I, C, device="cuda") * 0.08).to(torch.bfloat16)
    wd = (torch.randn(E, C, I, device="cuda") * 0.08).to(torch.bfloat16)
    dout = torch.randn(T, C, device="cuda").to(torch.bfloat16)
    r = _step(x, logits, bias, wu, wd, dout, k)
    P = [t.double().requires_grad_() for t in (x, logits, wu, wd)]
    X, L, WU, WD = P
    a = torch.sigmoid(L).gather(1, r["ids"].long())
    w = a / a.sum(1, keepdim=True)
    out = torch.zeros(T, C, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (r["ids"] == e).nonzero(as_tuple=True)
        gu = X[t] @ WU[e].t()
        h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
        out = out.index_add(0, t, (h @ WD[e].t()) * w[t, j][:, None])
    g = torch.autograd.grad(out, P, dout.double())
    for name, got, want in [("out", r["out"], out), ("dx", r["dx"], g[0]), ("dlogits", r["dlogits"], g[1]),
                            ("dwu", r["dwu"], g[2]), ("dwd", r["dwd"], g[3])]:
        rel = ((got.double() - want).norm() / want.norm()).item()
        assert rel <= 0.102, (name, rel)


def test_backward_kernels_in_a_captured_graph_on_a_side_stream(oracle):
    """Captured on another stream and replayed on new inputs in the same buffers."""
    c1, c2 = act_case([100, 40], 256, seed=21), act_case([100, 40], 256, seed=22)
    ref = act_run(c2)
    s = torch.cuda.Stream()
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    off = g(offsets_of(c1["counts"]))
    guq, sgu, w, dh = g(c1["guq"]), g(c1["sgu"]), g(c1["w"]), c1["dh"].cuda()
    st = fg8.new_status()
    bufs = fg8.swiglu_backward_quant(dh, guq, sgu, off, row_w=w, dev_status=st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fg8.swiglu_backward_quant(dh, guq, sgu, off, row_w=w, dev_status=st, **bufs)
    guq.copy_(g(c2["guq"])), sgu.copy_(g(c2["sgu"])), w.copy_(g(c2["w"])), dh.copy_(c2["dh"].cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert st.item() == 0
    used = padded(c1["counts"])[-1]
    for k in ("dq", "sd", "gate_dot"):
        assert np.array_equal(bufs[k].cpu().numpy(), ref[k]), k
    for k in ("dqT", "hqT"):
        assert np.array_equal(bufs[k].cpu().numpy()[:, :used], ref[k][:, :used]), k


# ---------------------------------------------------------------------------
# very large gates
# ---------------------------------------------------------------------------

def test_act_backward_gates_beyond_the_integers_of_fp32(oracle):
    """Gates from 2^12 to 2^31 of both signs.  exp(-g) is 0 or infinite there, so sig
    is 1 or 0 exactly and the last factor of dG, 1 + g (1 - sig), is 1 or meets a sig
    of 0: nothing grows with g.  For g > 0: dG = d u is off by the roundings of u, d
    and the three products (5 eps; 8 with the reciprocal of 1), dU = d g and h = g u
    by those of g, d, u and three products (the same); for g < 0 all are 0."""
    counts, I = [130, 40], 256
    c = act_case(counts, I, seed=31)
    R = c["R"]
    rng = np.random.default_rng(32)
    c["guq"][:, :I][(c["guq"][:, :I] & 0x7F) == 0] = 0x01          # no gate of 0
    c["sgu"][:I // 128] = np.exp2(21 + rng.uniform(0, 1, (I // 128, R))).astype(np.float32)
    # single values: where g + 1 rounds up, and where it is g
    c["guq"][:6, :I] = 0x38                                           # code 1.0
    c["sgu"][:I // 128, :6] = np.float32([2 ** 24, 2 ** 24 + 2, 2 ** 25, 2 ** 23 + 1, 3e9, 2 ** 26 + 8])
    out = act_run(c)
    f = act_formula(oracle, c)
    gu = deq_rows(oracle, c["guq"], c["sgu"])
    g, u = gu[:, :I], gu[:, I:]
    assert np.all(np.abs(g) >= 2.0 ** 12) and np.abs(g).max() > 2.0 ** 30
    # sig < exp(-2^12) < 2^-5900 there (the formula's clip at -700 is not that small):
    # every product is 0 in fp32, and a tile of zeros has scale 1
    for key in ("dG", "dU", "wh"):
        f[key][g < 0] = 0.0
    tol = lambda v: 8 * EPS * np.abs(v)   # noqa: E731
    v = np.concatenate([f["dG"], f["dU"]], 1)
    check_tiles(oracle, out["dq"], out["sd"].T, v, tol(v), "rows")
    check_columns(oracle, out["dqT"], out["sdT"], v, tol(v), counts, "columns of dG, dU")
    check_columns(oracle, out["hqT"], out["shT"], f["wh"], tol(f["wh"]), counts, "columns of w h")
    # the first rows' dG is d u, not 0 and not twice that
    d = f["dh"] * c["w"].astype(np.float64)[:, None]
    got = deq_rows(oracle, out["dq"], out["sd"])[:6, :I]
    du = (d * u)[:6]
    big = np.abs(du) > 0.1 * np.abs(du).max(1, keepdims=True)
    assert np.all((np.abs(got - du) <= 2.0 ** -4 * 1.01 * np.abs(du))[big])


# ---------------------------------------------------------------------------
# without the router's gradient
# ---------------------------------------------------------------------------

def test_act_backward_without_dots_is_the_same():
    counts = [130, 0, 61]
    c = act_case(counts, 256, seed=41, extra_rows=3)
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()   # noqa: E731
    args = c["dh"].cuda(), g(c["guq"]), g(c["sgu"]), g(offsets_of(counts))
    n, used = sum(counts), int(padded(counts)[-1])
    st = fg8.new_status()
    want = fg8.swiglu_backward_quant(*args, row_w=g(c["w"]), dev_status=st)
    got = fg8.swiglu_backward_quant(*args, row_w=g(c["w"]), want_dots=False, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and got["gate_dot"] is None and want["gate_dot"] is not None
    for k, cut in (("dq", lambda t: t[:n]), ("sd", lambda t: t[:, :n]), ("dqT", lambda t: t[:, :used]),
                   ("sdT", lambda t: t[:used // 128]), ("hqT", lambda t: t[:, :used]),
                   ("shT", lambda t: t[:used // 128]), ("offsets_out", lambda t: t)):
        assert torch.equal(cut(got[k]), cut(want[k])), k


@pytest.mark.parametrize("normalize", [True, False])
def test_gate_backward_without_logits_is_the_same(normalize):
    T, E, k, nb = 77, 9, 3, 5
    gen = torch.Generator(device="cuda").manual_seed(4)
    aff = torch.rand(T, k, device="cuda", generator=gen)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=gen, dtype=torch.int32)
    tr = torch.randperm(T * k, device="cuda", generator=gen).to(torch.int32)
    tr[7] = -1
    dot = torch.randn(nb, T * k, device="cuda", generator=gen)
    want, dlogits = fg8.gate_backward(dot, tr, ids, aff, E, normalize=normalize)
    got, none = fg8.gate_backward(dot, tr, None, aff, E, normalize=normalize, want_dlogits=False)
    torch.cuda.synchronize()
    assert none is None and dlogits is not None and torch.equal(got, want)


def test_training_step_of_no_tokens():
    """A rank whose batch is empty: every call of the step takes it, outputs of no rows
    are empty and the weights' gradients are zeros."""
    E, k, C, I = 3, 2, 256, 128
    z = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)   # noqa: E731
    r = _step(z(0, C), torch.randn(0, E, device="cuda"), torch.zeros(E, device="cuda"), z(E, 2 * I, C), z(E, C, I),
              z(0, C), k)
    assert r["out"].shape == (0, C) and r["dx"].shape == (0, C) and r["dlogits"].shape == (0, E)
    assert r["dwu"].shape == (E, 2 * I, C) and not r["dwu"].any()
    assert r["dwd"].shape == (E, C, I) and not r["dwd"].any()
