"""Norms in front of and behind the block against the float64 oracle.

Tolerances, from the float32 arithmetic (u = 2^-24).  A sum over a row has at most
16 sequential terms a thread, 6 shuffle steps and 8 waves: 30 roundings, and a
mean and a reciprocal square root add 4, so a statistic is within S = 40 u of itself (sums
of magnitudes).  With M = sum_j |g_j| |row_j| >= |y| and kappa = |M| / |y| (row norms),
y is within (k + 1) u M, r within (k + 1) u kappa + S of itself, n = y r within N =
((k + 1) (1 + kappa) u + 2 S) r M.  Products of a few factors add 4 u each.  An
output is then rounded once: 2^-8 (bf16) or 2^-24 (float32) of its value."""
import numpy as np
import pytest
import torch

from _gpu import host, log
from oracle import block_oracle as bo
from oracle import moe_oracle as om
from top_routing_expert_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 40 * U
ROUND = {True: 2.0 ** -8, False: 2.0 ** -24}
EPS = 1e-5


def _make(rng, shape, bf, std=1.0):
    a = (rng.standard_normal(shape) * std).astype(np.float32)
    return om.round_bf16(a) if bf else a


def _dev(a):
    return None if a is None else B.to_device(a)


def _new(*shape, bf=None):
    dt = torch.float32 if bf is None else torch.bfloat16 if bf else torch.float32
    return torch.full(shape, 7.0, dtype=dt, device="cuda")


def _f(t):
    return om._f64(host(t))


def _close(got, want, bound, name):
    bad = np.abs(got - want) - bound
    assert (bad <= 0).all(), (name, float(bad.max()), float(np.abs(got - want).max()))


def _cfg(T, d, bf, k=1):
    return B.config(T=T, d=d, E=max(k, 1), k=k, f=64, dtype=B.MOE_BF16 if bf else B.MOE_F32)


SIZES = [(1, 64, True), (3, 7168, True), (1000, 320, True), (1500, 1024, True), (5, 8192, True),
         (4, 8256, True), (3, 16384, True), (1, 4, False), (777, 1028, False), (6, 4096, False),
         (5, 4100, False), (2, 8192, False)]


@pytest.mark.parametrize("T,d,bf", SIZES)
@pytest.mark.parametrize("given", [True, False])
def test_norm_forward_and_backward(T, d, bf, given):
    log(f"[norm] T={T} d={d} bf16={bf} weight={given}")
    rng = np.random.default_rng(T + d)
    x = _make(rng, (T, d), bf)
    if T > 3:
        x[1] = 0                                # a row of zeros: r = 1 / sqrt(eps)
        x[2] = _make(rng, (d,), bf, 1e-4)       # eps of the row's own size
        x[3] = _make(rng, (d,), bf, 300.0)
    w = _make(rng, (d,), bf) if given else None
    g, dr = _make(rng, (T, d), bf), _make(rng, (T, d), bf) if given else None
    cfg = _cfg(T, d, bf)
    xd, wd, gd, drd = _dev(x), _dev(w), _dev(g), _dev(dr)
    xn, rstd = _new(T + 1, d, bf=bf), _new(T)
    B.moe_norm(cfg, xd, wd, EPS, xn, rstd)
    want, r = bo.rms_norm(x, w, EPS)
    assert (xn[T:] == 7.0).all()
    _close(_f(rstd), r, 2 * S * r, "rstd")
    _close(_f(xn[:T]), want, (ROUND[bf] + 2 * S + 4 * U) * np.abs(want) * (1 + 1e-6) + 1e-40, "xn")
    only = _new(T, d, bf=bf)
    B.moe_norm(cfg, xd, wd, EPS, only)  # without rstd
    assert torch.equal(only, xn[:T])

    d_x, d_w = _new(T + 1, d, bf=bf), _new(d)
    ws = B.workspace(cfg, "norm_backward")
    ws.fill_(0xFF)
    B.moe_norm_backward(cfg, gd, xd, wd, rstd, drd, d_x, d_w, ws)
    want_x, want_w = bo.rms_norm_backward(g, x, w, EPS, dr)
    assert (d_x[T:] == 7.0).all()
    xf, gf, wf = om._f64(x), om._f64(g), np.ones(d) if w is None else om._f64(w)
    n = np.abs(xf) * r[:, None]
    gw = np.abs(gf * wf)
    size = r[:, None] * (gw + n * (gw * n).mean(-1, keepdims=True))
    _close(_f(d_x[:T]), want_x, ROUND[bf] * np.abs(want_x) * (1 + 1e-6) + 10 * S * size
           + 4 * U * (0 if dr is None else np.abs(om._f64(dr))), "d_x")
    terms = (np.abs(gf) * n).sum(0)
    _close(_f(d_w), want_w, (3 * S + (T + 64) * U) * terms, "d_weight")
    # without a weight gradient no workspace is needed; d_x may be d_residual
    if dr is not None:
        B.moe_norm_backward(cfg, gd, xd, wd, rstd, drd, drd, None)
        assert torch.equal(drd, d_x[:T])


COMBINE = [  # T, d, k, bf, n_gate, with weight and residual
    (1, 64, 1, True, 0, True), (1, 7168, 8, True, 1, True), (6, 320, 2, True, 2, True),
    (6, 320, 2, True, 6, False), (1400, 256, 3, True, 7, True), (1400, 128, 2, True, 1400, True),
    (1400, 128, 2, True, 1, False), (90, 1024, 16, True, 15, True), (90, 1024, 5, True, 30, True),
    (3, 8256, 8, True, 3, True), (2, 16384, 16, True, 1, True), (2, 16384, 4, True, 0, False),
    (777, 1028, 2, False, 7, True), (40, 4096, 8, False, 20, True), (4, 4100, 8, False, 2, True),
    (3, 8192, 16, False, 0, True), (5, 4, 1, False, 5, True), (2100, 132, 4, False, 35, True),
]


def _combine_case(T, d, k, bf, n_gate, given, token_order=False):
    rng = np.random.default_rng(T + d + k)
    rows = T if token_order else T * k
    c = dict(y=_make(rng, (rows, d), bf, 0.3), res=_make(rng, (T, d), bf) if given else None,
             w=_make(rng, (d,), bf) if given else None,
             gate=_make(rng, (n_gate, d), bf) if n_gate else None, up=_make(rng, (T, d), bf))
    if token_order:
        c |= dict(slot=None, tw=None)
    else:
        c |= dict(slot=rng.permutation(rows).astype(np.int32),
                  tw=(rng.random((T, k)) + 0.05).astype(np.float32))
    return c


def _check_combine(T, d, k, bf, n_gate, given, token_order=False):
    c = _combine_case(T, d, k, bf, n_gate, given, token_order)
    kk = 1 if token_order else k
    cfg = _cfg(T, d, bf, k)
    dev = {n: _dev(v) for n, v in c.items()}
    out, rstd = _new(T + 1, d, bf=bf), _new(T)
    scale = 0.7
    B.moe_combine_norm(cfg, dev["y"], dev["slot"], dev["tw"], dev["res"], dev["w"], dev["gate"],
                       n_gate, EPS, scale, out, rstd)
    sc = float(np.float32(scale))
    want, r = bo.combine_norm(c["y"], c["slot"], c["tw"], c["res"], c["w"], c["gate"], EPS, sc)
    rows, g = bo._rows_of(c["y"], c["slot"], c["tw"], T)
    M = (np.abs(rows) * np.abs(g)[..., None]).sum(1)
    y = (rows * g[..., None]).sum(1)
    kappa = np.linalg.norm(M, axis=1) / np.linalg.norm(y, axis=1)
    rel_r = ((kk + 1) * U * kappa + S)[:, None]
    N = ((kk + 1) * U + 2 * rel_r) * r[:, None] * M   # error of n
    nM = r[:, None] * M
    wf = np.ones(d) if c["w"] is None else np.abs(om._f64(c["w"]))
    gate = om._f64(c["gate"]) if n_gate else np.ones((1, d))
    gf = np.repeat(gate, T // gate.shape[0], 0)
    gw = np.abs(gf) * wf
    assert (out[T:] == 7.0).all()
    _close(_f(rstd), r, 2 * rel_r[:, 0] * r, "rstd")
    size = gw * nM + (0 if c["res"] is None else sc * np.abs(om._f64(c["res"])))
    _close(_f(out[:T]), want, ROUND[bf] * np.abs(want) * (1 + 1e-6) + gw * N + 6 * U * size, "out")
    if c["res"] is not None:  # in place
        res = dev["res"].clone()
        B.moe_combine_norm(cfg, dev["y"], dev["slot"], dev["tw"], res, dev["w"], dev["gate"],
                           n_gate, EPS, scale, res)
        assert torch.equal(res, out[:T])

    d_y, d_tw = _new(len(c["y"]) + 1, d, bf=bf), None if token_order else _new(T, k)
    d_res, d_w, d_gate = _new(T, d, bf=bf), _new(d), _new(n_gate, d) if n_gate else None
    ws = B.combine_norm_workspace(cfg, n_gate)
    ws.fill_(0xFF)
    args = (cfg, dev["up"], dev["y"], dev["slot"], dev["tw"], dev["w"], dev["gate"], n_gate, scale,
            rstd)
    B.moe_combine_norm_backward(*args, d_y, d_tw, d_res, d_w, d_gate, ws)
    ref = bo.combine_norm_backward(c["up"], c["y"], c["slot"], c["tw"], c["w"], c["gate"], EPS, sc)
    up = np.abs(om._f64(c["up"]))
    dn = gw * up
    cM = (dn * nM).mean(-1, keepdims=True)
    rr = r[:, None]
    # dy: the factor r, n twice, the mean's sum
    dy_size = rr * (dn + nM * cM)
    dy_err = (2 * rel_r + S + 8 * U) * dy_size + rr * (N * cM + nM * (dn * N).mean(-1, keepdims=True))
    ag = np.abs(g)
    row_err = ag[..., None] * dy_err[:, None]
    if c["slot"] is not None:
        t = np.zeros((T * k, d))
        t[c["slot"]] = row_err.reshape(-1, d)
        row_err = t
    else:
        row_err = row_err[:, 0]
    assert (d_y[-1] == 7.0).all()
    _close(_f(d_y[:-1]), ref["d_y"], ROUND[bf] * np.abs(ref["d_y"]) * (1 + 1e-6) + row_err
           + 2 * U * np.abs(ref["d_y"]) + 1e-40, "d_y")
    if d_tw is not None:
        b = (np.abs(rows) * (dy_err + S * dy_size)[:, None]).sum(-1)
        _close(_f(d_tw), ref["d_topk_w"], b, "d_topk_w")
    _close(_f(d_res), ref["d_residual"], (ROUND[bf] + 2 * U) * np.abs(ref["d_residual"]) + 1e-40,
           "d_residual")
    adds = (T + 64) * U
    _close(_f(d_w), ref["d_weight"], (np.abs(gf) * up * (N + (adds + 4 * U) * nM)).sum(0), "d_weight")
    if n_gate:
        e = (wf * up * (N + (adds + 4 * U) * nM)).reshape(n_gate, -1, d).sum(1)
        _close(_f(d_gate), ref["d_gate"], e, "d_gate")
    # the optional outputs left out, one by one, leave the others as they were
    d_y2 = _new(len(c["y"]) + 1, d, bf=bf)
    B.moe_combine_norm_backward(*args, d_y2, None, None, None, None)
    assert torch.equal(d_y2, d_y)
    d_w2 = _new(d)
    B.moe_combine_norm_backward(*args, d_y2, d_tw, None, d_w2, None, ws)
    assert torch.equal(d_w2, d_w)


@pytest.mark.parametrize("T,d,k,bf,n_gate,given", COMBINE)
def test_combine_norm(T, d, k, bf, n_gate, given):
    log(f"[norm] combine T={T} d={d} k={k} bf16={bf} n_gate={n_gate} given={given}")
    _check_combine(T, d, k, bf, n_gate, given)


@pytest.mark.parametrize("T,d,bf,n_gate", [(1, 64, True, 1), (13, 7168, True, 13), (50, 516, False, 2),
                                           (3, 16384, True, 0)])
def test_token_order(T, d, bf, n_gate):
    log(f"[norm] token order T={T} d={d} bf16={bf}")
    _check_combine(T, d, 4 if d < 600 else 2, bf, n_gate, True, token_order=True)


def test_empty_batch():
    cfg = _cfg(0, 128, True, 2)
    d_w, d_gate = _new(128), _new(3, 128)
    gate = torch.ones((3, 128), dtype=torch.bfloat16, device="cuda")
    B.moe_norm(cfg, None, None, EPS, None)
    B.moe_norm_backward(cfg, None, None, None, None, None, None, d_w)
    assert (d_w == 0).all()
    d_w.fill_(1.0)
    B.moe_combine_norm(cfg, None, None, None, None, None, gate, 3, EPS, 1.0, None)
    B.moe_combine_norm_backward(cfg, None, None, None, None, None, gate, 3, 1.0, None, None, None,
                                None, d_w, d_gate)
    assert (d_w == 0).all() and (d_gate == 0).all()


def test_malformed_slots_stay_in_bounds():
    T, d, k = 9, 256, 2
    cfg = _cfg(T, d, True, k)
    y = torch.randn((T * k, d), device="cuda").bfloat16()
    slot = torch.arange(T * k, dtype=torch.int32, device="cuda")
    slot[0], slot[5] = -7, 10 ** 9
    tw = torch.rand((T, k), device="cuda")
    out, rstd = _new(T, d, bf=True), _new(T)
    B.moe_combine_norm(cfg, y, slot, tw, None, None, None, 0, EPS, 1.0, out, rstd)
    ref, _ = bo.combine_norm(host(y), np.clip(host(slot), 0, T * k - 1), host(tw), None, eps=EPS)
    assert np.abs(_f(out) - ref).max() <= 2.0 ** -8 * np.abs(ref).max() * 1.01


def test_captured_backward_next_to_eager():
    """Forward and backward captured, replayed between eager calls on other inputs."""
    T, d, k, n = 300, 512, 2, 3
    cfg = _cfg(T, d, True, k)
    bf = lambda *s: torch.randn(s, device="cuda").bfloat16()  # noqa: E731
    y, res, w, gate, up = bf(T * k, d), bf(T, d), bf(d), bf(n, d), bf(T, d)
    slot = torch.randperm(T * k, device="cuda").int()
    tw = torch.rand((T, k), device="cuda")
    o = [_new(T, d, bf=True), _new(T), _new(T * k, d, bf=True), _new(T, k), _new(T, d, bf=True), _new(d), _new(n, d)]
    ws = B.combine_norm_workspace(cfg, n)

    def step():
        B.moe_combine_norm(cfg, y, slot, tw, res, w, gate, n, EPS, 0.5, o[0], o[1])
        B.moe_combine_norm_backward(cfg, up, y, slot, tw, w, gate, n, 0.5, o[1], o[2], o[3], o[4],
                                    o[5], o[6], ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        y.copy_(torch.randn_like(y))
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in o]
        for v in o:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(o, want):
            assert torch.equal(a, b), i


def test_stores_past_the_cache_write_the_same():
    """Calls large enough to store past the cache, against the same tokens in four
    calls that are not: every token's row is its own, so the bits are the same."""
    T, d, k, parts = 5120, 7168, 8, 4
    n = T // parts
    log(f"[norm] combine T={T} d={d} k={k} in one call and in {parts}")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    y, res, up, w, gate = bf(T * k, d), bf(T, d), bf(T, d), bf(d), bf(parts, d)
    local = torch.cat([torch.randperm(n * k, device="cuda", generator=g) for _ in range(parts)]).int()
    slot = (local.view(parts, -1) + torch.arange(parts, device="cuda").int()[:, None] * n * k).flatten()
    tw = torch.rand((T, k), device="cuda", generator=g)

    def run(cfg, y, slot, tw, res, gate, up):
        t, q = res.shape[0], gate.shape[0]
        o = [_new(t, d, bf=True), _new(t), _new(t * k, d, bf=True), _new(t, k), _new(t, d, bf=True)]
        B.moe_combine_norm(cfg, y, slot, tw, res, w, gate, q, EPS, 0.5, o[0], o[1])
        B.moe_combine_norm_backward(cfg, up, y, slot, tw, w, gate, q, 0.5, o[1], o[2], o[3], o[4],
                                    None, None)
        return o

    whole = run(_cfg(T, d, True, k), y, slot, tw, res, gate, up)
    for i in range(parts):
        r, rk = slice(i * n, (i + 1) * n), slice(i * n * k, (i + 1) * n * k)
        part = run(_cfg(n, d, True, k), y[rk], local[rk], tw[r], res[r], gate[i:i + 1], up[r])
        for j, p in enumerate(part):
            assert torch.equal(p, whole[j][rk if j == 2 else r]), (i, j)
