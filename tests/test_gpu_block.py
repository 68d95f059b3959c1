"""The operators around the block as they are used together: a decode step, a prefill
on 4-bit operands, and a training step forward and back, against float64.

Tolerances.  Where a stage is checked on the bits that the stage before it wrote, its
own: 2^-8 of a value rounded to bf16, and for the norms the float32 terms of a row's sums
(u = 2^-24, S = 40 u a statistic, N = ((k + 1) (1 + kappa) u + 2 S) r M of a combined
row, M = sum_j |g_j| |row_j|, kappa = |M| / |y|).  The training step is checked from end
to end: on its way from d_out to a gradient a value meets at most nine roundings to bf16
(xn, a and u kept from the forward pass, h, y, d_y, da or du, d_xn, the output), each at
most 2^-8 of its array's norm, so 9 * 2^-8 norm-wise."""
import numpy as np
import pytest
import torch

from _gpu import TOL_LAYER, TOL_STAGE, alloc, f64, host, log, rel_err, routing_kwargs, upload
from oracle import block_oracle as bo
from oracle import moe_oracle as om
from top_routing_expert_amd import binding as B
from top_routing_expert_amd import configs as C
from top_routing_expert_amd import inputs as I

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
S = 40 * U
EPS = 1e-5
SCALE = 0.75
TOL_TRAIN = 9 * 2.0 ** -8

DECODE = C.MoEShape("decode", T=1, d=384, E=16, k=2, f=256)


def _params(shape, n_gate, seed):
    """Weights of the two norms and the gate rows, near one."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *s: (1 + 0.2 * torch.randn(s, device="cuda", generator=g)).bfloat16()  # noqa: E731
    return new(shape.d), new(shape.d), new(n_gate, shape.d)


def _like(*size, dtype=torch.bfloat16):
    return torch.full(size, 7.0, dtype=dtype, device="cuda")


def _check_norm(xn, x, w):
    want, _ = bo.rms_norm(host(x), host(w), EPS)
    assert (np.abs(f64(host(xn)) - want) <= (2.0 ** -8 + 2 * S + 4 * U) * np.abs(want) + 1e-40).all()


def _check_combine(out, y, slot, tw, res, w, gate):
    """out on the bits of y."""
    h = lambda t: None if t is None else host(t)  # noqa: E731
    T = out.shape[0]
    want, r = bo.combine_norm(host(y), h(slot), h(tw), host(res), host(w), host(gate), EPS, SCALE)
    rows, g = bo._rows_of(host(y), h(slot), h(tw), T)
    M = (np.abs(rows) * np.abs(g)[..., None]).sum(1)
    yy = (rows * g[..., None]).sum(1)
    k = g.shape[1]
    kappa = (np.sqrt((M * M).sum(-1)) / np.sqrt((yy * yy).sum(-1)))[:, None]
    gate_rows = np.repeat(np.abs(f64(host(gate))), T // gate.shape[0], 0)
    size = r[:, None] * M * np.abs(f64(host(w))) * gate_rows
    bound = (2.0 ** -8 * np.abs(want) + ((k + 1) * (1 + kappa) * U + 2 * S + 8 * U) * size
             + 4 * U * np.abs(SCALE * f64(host(res))))
    assert (np.abs(f64(host(out)) - want) <= 1.01 * bound).all()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 6, 32])
def test_decode_step(T, mx):
    """norm -> layer for a few tokens -> norm, gate and residual, eager and replayed
    from a graph between eager steps on other tokens."""
    shape = DECODE.replace(T=T)
    log(f"[block] decode T={T} mx={mx}")
    inp = I.make_inputs(shape, 3 + T)
    dev = upload(inp)
    cfg = B.config(shape)
    w1, w2, gate = _params(shape, T if T < 32 else 2, T)
    if mx:
        q = {n: B.quantize_mxfp4(dev[n]) for n in ("w_gate", "w_up", "w_down")}
        images = B.pack_weights_mxfp4(cfg, q["w_gate"], q["w_up"], q["w_down"])
        vals = {n: bo.mxfp4_decode(host(c), host(s)) for n, (c, s) in q.items()}
    else:
        images = B.pack_weights(cfg, dev["w_gate"], dev["w_up"], dev["w_down"])
        vals = {n: inp[n] for n in ("w_gate", "w_up", "w_down")}
    x = dev["x"]
    xn, y, out = (_like(T, shape.d) for _ in range(3))
    logits = _like(T, shape.E, dtype=torch.float32)
    ws = B.workspace(cfg, "layer_few")

    def step():
        B.moe_norm(cfg, x, w1, EPS, xn)
        B.moe_layer_fwd_few(cfg, xn, dev["w_router"], dev["bias"], *images, int(mx), y,
                            dict(logits=logits), ws)
        B.moe_combine_norm(cfg, y, None, None, x, w2, gate, gate.shape[0], EPS, SCALE, out)

    step()
    torch.cuda.synchronize()
    _check_norm(xn, x, w1)
    ref = om.layer(host(xn), inp["w_router"], inp["bias"], vals["w_gate"], vals["w_up"],
                   vals["w_down"], logits32=host(logits), **routing_kwargs(shape))
    assert rel_err(host(y), ref["out"]) <= TOL_LAYER["bf16"]
    _check_combine(out, y, None, None, x, w2, gate)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn_like(x))
        step()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


@pytest.mark.parametrize("key", ["e8", "e64", "e16"])
def test_prefill_on_mxfp4_operands(key):
    """norm -> routing -> quantise -> gate/up -> quantise -> down -> combine and norm."""
    shape = C.SMALL[key].replace(d=384, f=256)
    log(f"[block] prefill {shape.name}")
    T, d, k, f = shape.T, shape.d, shape.k, shape.f
    inp = I.make_inputs(shape, 5)
    dev, buf, cfg = upload(inp), alloc(shape), B.config(shape)
    w1, w2, gate = _params(shape, 4, 9)
    q = {n: B.quantize_mxfp4(dev[n]) for n in ("w_gate", "w_up", "w_down")}
    wg, wu, wd = (bo.mxfp4_decode(host(c), host(s)) for c, s in q.values())
    images = B.pack_weights_mxfp4(cfg, q["w_gate"], q["w_up"], q["w_down"])
    xn, out = _like(T, d), _like(T, d)
    B.moe_norm(cfg, dev["x"], w1, EPS, xn)
    B.moe_route(cfg, xn, dev["w_router"], dev["bias"], buf["logits"], buf["topk_idx"],
                buf["topk_w"], B.workspace(cfg, "route"))
    B.moe_permute(cfg, xn, buf["topk_idx"], buf["expert_offsets"], buf["rank_offsets"],
                  buf["slot_of"], buf["src_of"], buf["x_perm"], B.workspace(cfg, "permute"))
    xc, xs = B.quantize_mxfp4(xn)
    B.moe_ffn_gate_up_mxfp4_gather(cfg, xc, xs, buf["src_of"], buf["expert_offsets"], images[0],
                                   buf["h"])
    hc, hs = B.quantize_mxfp4(buf["h"])
    B.moe_ffn_down_mxfp4(cfg, hc, hs, buf["expert_offsets"], images[1], buf["y_perm"])
    B.moe_combine_norm(cfg, buf["y_perm"], buf["slot_of"], buf["topk_w"], dev["x"], w2, gate, 4,
                       EPS, SCALE, out)
    torch.cuda.synchronize()
    _check_norm(xn, dev["x"], w1)
    for got, src in ((xc, xs), xn), ((hc, hs), buf["h"]):
        codes, scales = bo.mxfp4_quantize(host(src))
        assert np.array_equal(host(got[0]), codes) and np.array_equal(host(got[1]), scales)
    offs, src = host(buf["expert_offsets"]), host(buf["src_of"])
    rows, hv = bo.mxfp4_decode(host(xc), host(xs))[src // k], bo.mxfp4_decode(host(hc), host(hs))
    want_h, want_y = np.zeros((T * k, f)), np.zeros((T * k, d))
    for e in range(shape.E):
        r = slice(offs[e], offs[e + 1])
        want_h[r] = om.silu(rows[r] @ wg[e].T) * (rows[r] @ wu[e].T)
        want_y[r] = hv[r] @ wd[e].T
    assert rel_err(host(buf["h"]), want_h) <= TOL_STAGE["bf16"]
    assert rel_err(host(buf["y_perm"]), want_y) <= TOL_STAGE["bf16"]
    _check_combine(out, buf["y_perm"], buf["slot_of"], buf["topk_w"], dev["x"], w2, gate)


def _norm_err(got, want, by_row=False):
    got, want = f64(host(got)), np.asarray(want, np.float64)
    ax = -1 if by_row else None
    num, den = np.sqrt(((got - want) ** 2).sum(ax)), np.sqrt((want ** 2).sum(ax))
    assert (np.asarray(num)[den == 0] == 0).all()
    return float(np.max(num[den > 0] / den[den > 0])) if np.ndim(den) else float(num / den)


@pytest.mark.parametrize("key", ["e8", "e16", "e256"])
def test_training_step(key):
    """out = SCALE x + gate norm(MoE(norm(x) w1)) w2, and every gradient of it."""
    shape = C.SMALL[key]
    log(f"[block] train {shape.name}")
    T, d, E, k, f = shape.T, shape.d, shape.E, shape.k, shape.f
    inp, dout = I.make_inputs(shape, 7), I.make_grad_out(shape, 7)
    dev, buf, cfg = upload(inp), alloc(shape), B.config(shape)
    n_gate = 4
    w1, w2, gate = _params(shape, n_gate, 1)
    x, d_out = dev["x"], B.to_device(dout)
    new, f32 = lambda *s: _like(*s), torch.float32  # noqa: E731
    new32 = lambda *s: _like(*s, dtype=f32)  # noqa: E731
    xn, r1, out, r2 = new(T, d), new32(T), new(T, d), new32(T)
    a, u = new(T * k, f), new(T * k, f)
    gu, dn = B.pack_weights(cfg, dev["w_gate"], dev["w_up"], dev["w_down"])
    # forward
    B.moe_norm(cfg, x, w1, EPS, xn, r1)
    B.moe_route(cfg, xn, dev["w_router"], dev["bias"], buf["logits"], buf["topk_idx"],
                buf["topk_w"], B.workspace(cfg, "route"))
    B.moe_permute(cfg, xn, buf["topk_idx"], buf["expert_offsets"], buf["rank_offsets"],
                  buf["slot_of"], buf["src_of"], buf["x_perm"], B.workspace(cfg, "permute"))
    B.moe_ffn_gate_up_packed_train(cfg, buf["x_perm"], None, buf["expert_offsets"], gu, buf["h"], a, u)
    B.moe_ffn_down_packed(cfg, buf["h"], buf["expert_offsets"], dn, buf["y_perm"])
    B.moe_combine_norm(cfg, buf["y_perm"], buf["slot_of"], buf["topk_w"], x, w2, gate, n_gate, EPS,
                       SCALE, out, r2)
    # and back
    g = dict(d_y=new(T * k, d), d_topk_w=new32(T, k), d_res=new(T, d), d_w2=new32(d),
             d_gate=new32(n_gate, d), d_x_perm=new(T * k, d), d_w_gate=new(E, f, d),
             d_w_up=new(E, f, d), d_w_down=new(E, d, f), d_logits=new32(T, E),
             d_x_router=new(T, d), d_w_router=new(E, d), d_bias=new32(E), d_xn=new(T, d),
             d_x=new(T, d), d_w1=new32(d))
    B.moe_combine_norm_backward(cfg, d_out, buf["y_perm"], buf["slot_of"], buf["topk_w"], w2, gate,
                                n_gate, SCALE, r2, g["d_y"], g["d_topk_w"], g["d_res"], g["d_w2"],
                                g["d_gate"], B.combine_norm_workspace(cfg, n_gate))
    B.moe_ffn_backward(cfg, buf["x_perm"], buf["expert_offsets"], dev["w_gate"], dev["w_up"],
                       dev["w_down"], g["d_y"], g["d_x_perm"], g["d_w_gate"], g["d_w_up"],
                       g["d_w_down"], B.workspace(cfg, "ffn_backward"), a=a, u=u)
    B.moe_route_backward(cfg, xn, dev["w_router"], buf["logits"], dev["bias"], buf["topk_idx"],
                         g["d_topk_w"], g["d_logits"], g["d_x_router"], g["d_w_router"],
                         g["d_bias"], B.workspace(cfg, "route_backward"))
    B.moe_unpermute_backward(cfg, g["d_x_perm"], buf["slot_of"], g["d_x_router"], g["d_xn"])
    B.moe_norm_backward(cfg, g["d_xn"], x, w1, r1, g["d_res"], g["d_x"], g["d_w1"],
                        B.workspace(cfg, "norm_backward"))
    torch.cuda.synchronize()

    kw = routing_kwargs(shape)
    args = (host(xn), inp["w_router"], inp["bias"], inp["w_gate"], inp["w_up"], inp["w_down"])
    fwd = om.layer(*args, ep_ranks=shape.ep_ranks, logits32=host(buf["logits"]), **kw)
    assert np.array_equal(host(buf["topk_idx"]), fwd["topk_idx"])
    hb = lambda t: f64(host(t))  # noqa: E731
    want_out, _ = bo.combine_norm(fwd["out"], None, None, host(x), hb(w2), hb(gate), EPS, SCALE)
    b = bo.combine_norm_backward(dout, fwd["out"], None, None, hb(w2), hb(gate), EPS, SCALE)
    ref = om.layer_backward(*args, b["d_y"], fwd=fwd, ep_ranks=shape.ep_ranks, **kw)
    d_x, d_w1 = bo.rms_norm_backward(ref["dx"], host(x), hb(w1), EPS, b["d_residual"])
    _check_norm(xn, x, w1)
    errs = dict(out=_norm_err(out, want_out, True), d_x=_norm_err(g["d_x"], d_x, True),
                d_xn=_norm_err(g["d_xn"], ref["dx"], True),
                d_y=_norm_err(g["d_y"], ref["dy_perm"], True))
    for name, want in dict(d_w1=d_w1, d_w2=b["d_weight"], d_gate=b["d_gate"],
                           d_topk_w=ref["d_topk_w"], d_w_gate=ref["dw_gate"],
                           d_w_up=ref["dw_up"], d_w_down=ref["dw_down"],
                           d_w_router=ref["dw_router"], d_bias=ref["d_bias"]).items():
        errs[name] = _norm_err(g[name], want)
    log("  norm-wise errors " + " ".join(f"{n}={e:.1e}" for n, e in errs.items()))
    assert max(errs.values()) <= TOL_TRAIN, errs
