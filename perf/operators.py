"""Measured cases of the few-token layer, the MXFP4 payload and expert products, and the norms around the MoE block.

Five operators, each in a plain form of elementary torch operations and as the calls a user makes of
`top_routing_expert_amd.binding`:

  few      the whole MoE layer for 1..32 tokens (decode, speculative decode), on bf16 or MXFP4 expert weights
  payload  per-block 4-bit dispatch payload: quantise the token rows, decode them into expert order
  product  expert products on MXFP4 operands: gate/up with SiLU, or down
  norm     RMS norm in front of the block, forward and (train) backward
  combine  combine + RMS norm + gate + scaled residual behind the block, forward and (train) backward

MXFP4: 32 consecutive elements share the scale 2^(floor(log2 max|x|) - 2), held as its exponent plus 127 in one byte;
elements are 0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives, to nearest with ties to the even code, saturating at 6.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


# ------------------------------------------------------------------------------------------------------------ cases
def _few(name, T, d, E, k, f, weights, n_group=1, topk_group=1, presel=0, renorm=1, bias=0.0):
    return dict(name=name, op="few", T=T, d=d, E=E, k=k, f=f, weights=weights, n_group=n_group, topk_group=topk_group,
                presel=presel, renorm=renorm, bias=bias)


def _payload(name, T, d, E, k, skew):
    return dict(name=name, op="payload", T=T, d=d, E=E, k=k, skew=skew)


def _product(name, which, T, d, E, k, f, skew):
    return dict(name=name, op="product", which=which, T=T, d=d, E=E, k=k, f=f, skew=skew)


def _norm(name, T, d, dtype, train):
    return dict(name=name, op="norm", T=T, d=d, dtype=dtype, train=train)


def _combine(name, T, d, k, dtype, n_gate, train):
    return dict(name=name, op="combine", T=T, d=d, k=k, dtype=dtype, n_gate=n_gate, train=train)


def listed():
    return [
        # one decoded token of a layer of few experts: the smallest weight stream, where launches and latency count
        _few("few-T1-d5120-E16-top2-f1536-bf16", 1, 5120, 16, 2, 1536, "bf16"),
        # one decoded token of a layer of many experts with group-limited top-8: a stream of eight experts' weights
        _few("few-T1-d7168-E256-g8x4-top8-f2048-bf16", 1, 7168, 256, 8, 2048, "bf16", n_group=8, topk_group=4),
        # a draft of 29 tokens checked at once, 4-bit experts, gates over a pre-selection
        _few("few-T29-d2048-E64-presel8-top2-f1408-mxfp4", 29, 2048, 64, 2, 1408, "mxfp4", presel=8, renorm=0, bias=0.1),
        # the payload of five tokens of a decode batch
        _payload("payload-T5-d2048-E64-top2", 5, 2048, 64, 2, 0.0),
        # the payload of a long prefill, experts of uneven load
        _payload("payload-T16384-d5120-E16-top2", 16384, 5120, 16, 2, 1.1),
        # a short ragged batch: experts of a few rows each, some of none
        _product("gate_up-T37-d5120-E16-top2-f1536", "gate_up", 37, 5120, 16, 2, 1536, 1.1),
        # a rank's prefill share, a thousand rows an expert: bound by the matrix units
        _product("gate_up-T8192-d7168-E64-top8-f2048", "gate_up", 8192, 7168, 64, 8, 2048, 0.0),
        # few wide experts: the down product of one prefill chunk
        _product("down-T1024-d4096-E8-top2-f11008", "down", 1024, 4096, 8, 2, 11008, 0.0),
        # the norm in front of a decode step of three tokens
        _norm("norm-T3-d7168-bf16", 3, 7168, "bf16", False),
        # the same in a training step, forward and backward, with a last token missing from the batch
        _norm("norm-train-T16383-d5120-bf16", 16383, 5120, "bf16", True),
        # behind the block in a training step of four sequences, a gate row each
        _combine("combine-train-T8192-d7168-k8-bf16", 8192, 7168, 8, "bf16", 4, True),
        # a small float32 model: seven sequences of 111 tokens, odd width
        _combine("combine-train-T777-d1028-k2-f32", 777, 1028, 2, "f32", 7, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("few", "few", "payload", "product", "product", "norm", "combine", "combine"))
    if op == "few":
        E, k, n_group, topk_group = rng.choice(((8, 2, 1, 1), (16, 2, 1, 1), (64, 2, 1, 1), (64, 6, 8, 3), (256, 8, 8, 4), (96, 4, 1, 1)))
        presel = rng.choice((0, 0, 8)) if n_group == 1 else 0
        weights, unit = rng.choice((("bf16", 64), ("mxfp4", 128)))  # 4-bit products take whole 128-wide steps
        return _few("", _log(rng, 1, 32), unit * _log(rng, 512 // unit, 4096 // unit), E, k, unit * _log(rng, 256 // unit, 2048 // unit), weights,
                    n_group, topk_group, presel, rng.choice((0, 1)), rng.choice((0.0, 0.1)))
    if op == "payload":
        return _payload("", _log(rng, 1, 8192), 64 * _log(rng, 4, 112), rng.choice((8, 16, 64)), rng.choice((1, 2, 4)), rng.choice((0.0, 1.1)))
    if op == "product":
        return _product("", rng.choice(("gate_up", "down")), _log(rng, 1, 6000), 128 * _log(rng, 4, 48), rng.choice((4, 8, 16, 33)), rng.choice((1, 2, 4)),
                        128 * _log(rng, 2, 24), rng.choice((0.0, 1.1)))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    d = 64 * _log(rng, 2, 112) if dtype == "bf16" else 4 * _log(rng, 16, 1200)
    if op == "norm":
        return _norm("", _log(rng, 1, 10000), d, dtype, rng.choice((False, True)))
    L, n_gate = _log(rng, 1, 500), _log(rng, 1, 12)
    return _combine("", L * n_gate, d, rng.choice((1, 2, 3, 6, 8)), dtype, rng.choice((0, 1, n_gate, L * n_gate)), rng.choice((False, True)))


def work(case):
    T, d = case["T"], case["d"]
    op = case["op"]
    if op == "few":
        E, k, f = case["E"], case["k"], case["f"]
        experts = E * (1 - (1 - k / E) ** T)  # distinct experts that T tokens of even load call
        per = 2.0 if case["weights"] == "bf16" else 17 / 32
        return {"bytes": experts * 3 * d * f * per + E * d * 2 + T * d * 4, "flops": 6 * T * k * d * f + 2 * T * d * E}
    if op == "payload":
        return {"bytes": T * d * 2 + T * case["k"] * (d * 2 + 4), "flops": 4 * T * d}
    if op == "product":
        E, k, f = case["E"], case["k"], case["f"]
        rows = T * k
        experts = min(E, rows)
        if case["which"] == "gate_up":
            return {"bytes": experts * 2 * f * d * 17 / 32 + T * d * 2 + rows * (f * 2 + 4), "flops": 4 * rows * d * f}
        return {"bytes": experts * f * d * 17 / 32 + rows * (f + d) * 2, "flops": 2 * rows * d * f}
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        n = T * d
        # forward: x in, xn out; backward: d_xn, x, d_residual in, d_x out
        return {"bytes": n * es * (2 + (4 if case["train"] else 0)) + d * es, "flops": n * (4 + (12 if case["train"] else 0))}
    n, k = T * d, case["k"]
    # forward: k rows and the residual in, out out; backward: k rows and d_out in, k rows and d_residual out
    return {"bytes": n * es * (k + 2 + ((2 * k + 2) if case["train"] else 0)) + case["n_gate"] * d * es,
            "flops": n * (2 * k + 6 + ((6 * k + 14) if case["train"] else 0))}


# ----------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1_000_003 * (seed + 1))
    return g


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g)


def _values(codes):
    """E2M1 codes, two a byte with the lower nibble first -> float32 values."""
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), dtype=torch.float32, device=codes.device)
    both = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return lut.index_select(0, both.flatten().int()).view(both.shape)


def _decode(codes, scales):
    """MXFP4 codes [..., n / 2] and scales [..., n / 32] -> float32 [..., n]."""
    v = _values(codes).unflatten(-1, (-1, 32))
    v *= torch.pow(2.0, scales.double() - 127).float().unsqueeze(-1)
    return v.flatten(-2)


def _encode(x):
    """[..., n] -> MXFP4 codes [..., n / 2] and scales [..., n / 32]."""
    v = x.float().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp_(-127, 127)
    v = v * torch.pow(2.0, -e.double()).float().unsqueeze(-1)
    a = v.abs()
    q = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp_(max=6)
    code = torch.where(q < 2, 2 * q, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mx_weights(g, E, rows, cols, std=0.02):
    codes = torch.empty((E, rows, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, rows, cols // 32), dtype=torch.uint8, device=DEV)
    for e in range(E):
        codes[e], scales[e] = _encode(_normal(g, (rows, cols), std, torch.float32))
    return codes, scales


def _few_inputs(c, seed):
    g = _gen(seed)
    T, d, E, f = c["T"], c["d"], c["E"], c["f"]
    s = dict(x=_normal(g, (T, d)), w_router=_normal(g, (E, d), 0.02),
             bias=_normal(g, (E,), c["bias"], torch.float32) if c["bias"] else None)
    shapes = (("gate", (f, d)), ("up", (f, d)), ("down", (d, f)))
    for n, (rows, cols) in shapes:
        s[n] = _normal(g, (E, rows, cols), 0.02) if c["weights"] == "bf16" else _mx_weights(g, E, rows, cols)
    return s


def _dispatch(c, g):
    """A routing as the dispatch leaves it: expert-ordered rows, stable within an expert."""
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.rand((T, E), device=DEV, generator=g).log_().neg_().log_().neg_()
    score -= c["skew"] * torch.log(torch.arange(E, device=DEV) + 1.0)
    idx = score.topk(k, -1).indices.flatten()
    order = torch.sort(idx, stable=True).indices
    counts = torch.bincount(idx, minlength=E)
    offs = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offs[1:] = counts.cumsum(0)
    return order.int(), offs, counts


def _product_inputs(c, seed):
    g = _gen(seed)
    T, d, E, k, f = c["T"], c["d"], c["E"], c["k"], c["f"]
    src, offs, counts = _dispatch(c, g)
    s = dict(src_of=src, offsets=offs, counts=counts)
    if c["which"] == "gate_up":
        s["act"] = _normal(g, (T, d))
        s["gate"], s["up"] = _mx_weights(g, E, f, d), _mx_weights(g, E, f, d)
    else:  # what SiLU(a) u leaves: a product of two nearly normal values
        s["act"] = _normal(g, (T * k, f)) * _normal(g, (T * k, f), 0.5)
        s["down"] = _mx_weights(g, E, d, f)
    return s


def _norm_inputs(c, seed):
    g = _gen(seed)
    T, d = c["T"], c["d"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    size = 0.25 + 3 * torch.rand((T, 1), device=DEV, generator=g)  # tokens differ in size, as residual streams do
    s = dict(x=(_normal(g, (T, d), 1.0, torch.float32) * size).to(dt), weight=(1 + _normal(g, (d,), 0.1, torch.float32)).to(dt))
    if c["train"]:
        s["d_xn"], s["d_residual"] = _normal(g, (T, d), 1.0, dt), _normal(g, (T, d), 1.0, dt)
    return s


def _combine_inputs(c, seed):
    g = _gen(seed)
    T, d, k = c["T"], c["d"], c["k"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    s = dict(y=_normal(g, (T * k, d), 0.3, dt), residual=_normal(g, (T, d), 1.0, dt), weight=(1 + _normal(g, (d,), 0.1, torch.float32)).to(dt),
             topk_w=torch.softmax(_normal(g, (T, k), 1.0, torch.float32), -1),
             slot_of=torch.randperm(T * k, device=DEV, generator=g).int(),
             gate=_normal(g, (c["n_gate"], d), 0.5, dt) if c["n_gate"] else None)
    if c["train"]:
        s["d_out"] = _normal(g, (T, d), 1.0, dt)
    return s


RES_SCALE = 0.75


def prepare(case, seed):
    c = dict(case)
    make = dict(few=_few_inputs, payload=lambda c, s: dict(zip(("src_of", "x"), (_dispatch(c, _gen(s))[0], _normal(_gen(s + 17), (c["T"], c["d"]))))),
                product=_product_inputs, norm=_norm_inputs, combine=_combine_inputs)[c["op"]]
    s = make(c, seed)
    s["case"] = c
    if own:
        _prepare_own(c, s)
    elif c["op"] == "product":  # where each expert's rows stand in a batch padded to the longest expert
        counts, rows = s.pop("counts"), c["T"] * c["k"]
        longest = max(1, int(counts.max()))
        at = torch.arange(longest, device=DEV)
        s["rows"] = torch.where(at < counts[:, None], s["offsets"][:-1, None].long() + at, rows)
        s["expert"] = torch.repeat_interleave(torch.arange(c["E"], device=DEV), counts)
        s["place"] = torch.arange(rows, device=DEV) - s["offsets"].long()[s["expert"]]
    return s


def _prepare_own(c, s):
    """The handle of a user's program: config, weight images, workspaces and output buffers."""
    from top_routing_expert_amd import binding as B

    T, d, k, E, f = c["T"], c["d"], c.get("k", 1), c.get("E", 1), c.get("f", 64)
    if "dtype" in c and c["dtype"] == "f32":
        dt, tag = torch.float32, B.MOE_F32
    else:
        dt, tag = torch.bfloat16, B.MOE_BF16
    new = lambda *shape, t=dt: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
    u8, f32 = torch.uint8, torch.float32
    s["B"] = B
    if c["op"] == "few":
        cfg = s["cfg"] = B.config(T=T, d=d, E=E, k=k, f=f, n_group=c["n_group"], topk_group=c["topk_group"], presel=c["presel"], renorm=c["renorm"])
        if c["weights"] == "bf16":
            s["images"] = B.pack_weights(cfg, s.pop("gate"), s.pop("up"), s.pop("down"))
            s["format"] = B.MOE_WEIGHTS_BF16
        else:
            s["images"] = B.pack_weights_mxfp4(cfg, s.pop("gate"), s.pop("up"), s.pop("down"))
            s["format"] = B.MOE_WEIGHTS_MXFP4
        s["ws"], s["out"] = B.workspace(cfg, "layer_few"), new(T, d)
    elif c["op"] == "payload":
        s["cfg"] = B.config(T=T, d=d, E=E, k=k, f=f)
        s["codes"], s["scales"], s["x_perm"] = new(T, d // 2, t=u8), new(T, d // 32, t=u8), new(T * k, d)
    elif c["op"] == "product":
        cfg = s["cfg"] = B.config(T=T, d=d, E=E, k=k, f=f)
        if c["which"] == "gate_up":
            s["image"] = B.pack_weights_mxfp4(cfg, s.pop("gate"), s.pop("up"), None)[0]
            s["q_cfg"], s["out"] = cfg, new(T * k, f)
        else:
            s["image"] = B.pack_weights_mxfp4(cfg, None, None, s.pop("down"))[1]
            s["q_cfg"], s["out"] = B.config(T=T * k, d=f, E=1, k=1, f=64), new(T * k, d)
        rows, cols = s["act"].shape
        s["codes"], s["scales"] = new(rows, cols // 2, t=u8), new(rows, cols // 32, t=u8)
    elif c["op"] == "norm":
        cfg = s["cfg"] = B.config(T=T, d=d, E=1, k=1, f=64, dtype=tag)
        s["xn"], s["rstd"] = new(T, d), new(T, t=f32)
        if c["train"]:
            s["d_x"], s["d_weight"], s["ws"] = new(T, d), new(d, t=f32), B.workspace(cfg, "norm_backward")
    else:
        cfg = s["cfg"] = B.config(T=T, d=d, E=k, k=k, f=64, dtype=tag)
        s["out"], s["rstd"] = new(T, d), new(T, t=f32)
        if c["train"]:
            n = c["n_gate"]
            s["d_y"], s["d_topk_w"], s["d_res"], s["d_weight"] = new(T * k, d), new(T, k, t=f32), new(T, d), new(d, t=f32)
            s["d_gate"] = new(n, d, t=f32) if n else None
            s["ws"] = B.combine_norm_workspace(cfg, n)


# -------------------------------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if own:
        return dict(few=_own_few, payload=_own_payload, product=_own_product, norm=_own_norm, combine=_own_combine)[op](state)
    return dict(few=_plain_few, payload=_plain_payload, product=_plain_product, norm=_plain_norm, combine=_plain_combine)[op](state)


def _own_few(s):
    gu, dn = s["images"]
    s["B"].moe_layer_fwd_few(s["cfg"], s["x"], s["w_router"], s["bias"], gu, dn, s["format"], s["out"], None, s["ws"])
    return s["out"]


def _own_payload(s):
    s["B"].moe_quantize_mxfp4(s["cfg"], s["x"], s["codes"], s["scales"])
    s["B"].moe_dequantize_mxfp4(s["cfg"], s["codes"], s["src_of"], s["scales"], s["x_perm"])
    return s["x_perm"]


def _own_product(s):
    B = s["B"]
    B.moe_quantize_mxfp4(s["q_cfg"], s["act"], s["codes"], s["scales"])
    if s["case"]["which"] == "gate_up":
        B.moe_ffn_gate_up_mxfp4_gather(s["cfg"], s["codes"], s["scales"], s["src_of"], s["offsets"], s["image"], s["out"])
    else:
        B.moe_ffn_down_mxfp4(s["cfg"], s["codes"], s["scales"], s["offsets"], s["image"], s["out"])
    return s["out"]


def _own_norm(s):
    B, cfg = s["B"], s["cfg"]
    B.moe_norm(cfg, s["x"], s["weight"], EPS, s["xn"], s["rstd"])
    if not s["case"]["train"]:
        return s["xn"]
    B.moe_norm_backward(cfg, s["d_xn"], s["x"], s["weight"], s["rstd"], s["d_residual"], s["d_x"], s["d_weight"], s["ws"])
    return dict(xn=s["xn"], d_x=s["d_x"], d_weight=s["d_weight"])


def _own_combine(s):
    B, cfg, n = s["B"], s["cfg"], s["case"]["n_gate"]
    B.moe_combine_norm(cfg, s["y"], s["slot_of"], s["topk_w"], s["residual"], s["weight"], s["gate"], n, EPS, RES_SCALE, s["out"], s["rstd"])
    if not s["case"]["train"]:
        return s["out"]
    B.moe_combine_norm_backward(cfg, s["d_out"], s["y"], s["slot_of"], s["topk_w"], s["weight"], s["gate"], n, RES_SCALE, s["rstd"], s["d_y"],
                                s["d_topk_w"], s["d_res"], s["d_weight"], s["d_gate"], s["ws"])
    r = dict(out=s["out"], d_y=s["d_y"], d_topk_w=s["d_topk_w"], d_residual=s["d_res"], d_weight=s["d_weight"])
    return r | (dict(d_gate=s["d_gate"]) if n else {})


def _route(c, z, bias):
    """Logits -> chosen experts [T, k] (best first, ties to the lowest index) and gates, in the logits' type."""
    score = z if bias is None else z + bias.to(z.dtype)
    T, E = score.shape
    open_ = score
    if c["n_group"] > 1:
        best = score.view(T, c["n_group"], -1).amax(-1)
        keep = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        open_ = score.masked_fill(~mask.repeat_interleave(E // c["n_group"], 1), -math.inf)
    val, idx = torch.sort(open_, dim=-1, descending=True, stable=True)
    k = c["k"]
    over = val[:, :k] if c["renorm"] else val[:, :c["presel"]] if c["presel"] else score
    return idx[:, :k], torch.exp(val[:, :k] - val[:, :1]) / torch.exp(over - val[:, :1]).sum(-1, keepdim=True)


def _plain_few(s):
    c = s["case"]
    x = s["x"].float()
    # logits in 64 bits: two experts next to the border of the selection must not change places
    idx, gates = _route(c, s["x"].double() @ s["w_router"].double().T, s["bias"])
    pairs = idx.flatten()
    take = lambda w: w[pairs].float() if torch.is_tensor(w) else _decode(w[0][pairs], w[1][pairs])  # noqa: E731
    rows = x.repeat_interleave(c["k"], 0).unsqueeze(-1)
    a = torch.matmul(take(s["gate"]), rows).squeeze(-1)
    h = a / (1 + torch.exp(-a)) * torch.matmul(take(s["up"]), rows).squeeze(-1)
    y = torch.matmul(take(s["down"]), h.unsqueeze(-1)).squeeze(-1)
    return (y.view(c["T"], c["k"], -1) * gates.float().unsqueeze(-1)).sum(1).to(s["x"].dtype)


def _plain_payload(s):
    token = s["src_of"].long() // s["case"]["k"]
    codes, scales = _encode(s["x"])
    return _decode(codes[token], scales[token]).to(s["x"].dtype)


def _experts(s, act, weight):
    """act [rows, K] in expert order times each row's expert's weight [E, N, K] -> [rows, N], in float32."""
    padded = torch.cat((act, act.new_zeros(1, act.shape[1])))[s["rows"]]  # [E, longest, K]
    out = torch.bmm(_decode(*weight), padded.transpose(1, 2).contiguous())  # [E, N, longest]
    return out[s["expert"], :, s["place"]]


def _plain_product(s):
    act = _decode(*_encode(s["act"]))
    if s["case"]["which"] == "down":
        return _experts(s, act, s["down"]).to(s["act"].dtype)
    act = act[s["src_of"].long() // s["case"]["k"]]
    a = _experts(s, act, s["gate"])
    return (a / (1 + torch.exp(-a)) * _experts(s, act, s["up"])).to(s["act"].dtype)


def _plain_norm(s):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["weight"].float()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    xn = (n * w).to(dt)
    if not s["case"]["train"]:
        return xn
    g = s["d_xn"].float()
    gw = g * w
    d_x = s["d_residual"].float() + r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dict(xn=xn, d_x=d_x.to(dt), d_weight=(g * n).sum(0))


def _plain_combine(s):
    c = s["case"]
    dt, (T, d), k, n_gate = s["residual"].dtype, s["residual"].shape, c["k"], c["n_gate"]
    w, slot = s["weight"].float(), s["slot_of"].long()
    rows = s["y"][slot].float().view(T, k, d)
    y = (rows * s["topk_w"].unsqueeze(-1)).sum(1)
    r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
    n = y * r
    gate = s["gate"].float().repeat_interleave(T // n_gate, 0) if n_gate else 1.0
    out = (RES_SCALE * s["residual"].float() + gate * w * n).to(dt)
    if not c["train"]:
        return out
    g = s["d_out"].float()
    dn = gate * w * g
    dy = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    d_y = torch.empty_like(s["y"])
    d_y[slot] = (s["topk_w"].unsqueeze(-1) * dy.unsqueeze(1)).to(dt).view(T * k, d)
    grads = dict(out=out, d_y=d_y, d_topk_w=(rows * dy.unsqueeze(1)).sum(-1), d_residual=(RES_SCALE * g).to(dt), d_weight=(gate * g * n).sum(0))
    return grads | (dict(d_gate=(w * g * n).view(n_gate, T // n_gate, d).sum(1)) if n_gate else {})


# ------------------------------------------------------------------------------------- the definitions, in 64 bits
def _exact_values(codes, scales):
    """MXFP4 -> float64 by the bits of the code: sign, two exponent bits of bias 1, one mantissa bit."""
    flat = torch.empty(codes.shape + (2,), dtype=torch.uint8, device=codes.device)
    flat[..., 0], flat[..., 1] = codes % 16, codes // 16
    flat = flat.flatten(-2)
    e, m = (flat // 2 % 4).double(), (flat % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2 ** (e - 1)) * (1 - 2 * (flat // 8).double())
    return v * torch.repeat_interleave(2 ** (scales.double() - 127), 32, -1)


def _exact_mx(x):
    """The float64 values that MXFP4 holds of x."""
    v = x.double().view(*x.shape[:-1], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(2 ** e > top, e - 1, torch.where(2 ** (e + 1) <= top, e + 1, e))
    scale = 2 ** torch.where(top > 0, torch.clamp(e - 2, -127, 127), -127.0)
    a = v.abs() / scale
    # a tie goes to the even code: midpoints above an even code stay, above an odd one move up
    code = sum((a > m).long() for m in (0.25, 1.25, 2.5, 5.0)) + sum((a >= m).long() for m in (0.75, 1.75, 3.5))
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)[code]
    return (torch.copysign(level, v) * scale).view(x.shape)


def _exact_few(c, seed):
    s = _few_inputs(c, seed)
    k = c["k"]
    x = s["x"].double()
    z = (x[:, None] * s["w_router"].double()).sum(-1)
    if s["bias"] is not None:
        z = z + s["bias"].double()
    out = torch.zeros_like(x)
    size = c["E"] // c["n_group"]
    for t, row in enumerate(z.cpu().numpy()):
        groups = sorted(range(c["n_group"]), key=lambda q: (-row[q * size:(q + 1) * size].max(), q))[:c["topk_group"]]
        order = sorted((e for q in groups for e in range(q * size, (q + 1) * size)), key=lambda e: (-row[e], e))
        over = order[:k] if c["renorm"] else order[:c["presel"]] if c["presel"] else range(c["E"])
        total = np.exp(row[list(over)] - row[order[0]]).sum()
        for e in order[:k]:
            g, u, dn = (w[e].double() if torch.is_tensor(w) else _exact_values(w[0][e], w[1][e]) for w in (s["gate"], s["up"], s["down"]))
            a = g @ x[t]
            out[t] += float(np.exp(row[e] - row[order[0]]) / total) * (dn @ (a * torch.sigmoid(a) * (u @ x[t])))
    return out


def _exact_product(c, seed):
    s = _product_inputs(c, seed)
    act = _exact_mx(s["act"])
    if c["which"] == "gate_up":
        act = act[s["src_of"].long() // c["k"]]
    at = s["offsets"].tolist()
    parts = []
    for e in range(c["E"]):
        rows = act[at[e]:at[e + 1]]
        if c["which"] == "down":
            parts.append(rows @ _exact_values(s["down"][0][e], s["down"][1][e]).T.contiguous())
        else:
            a, u = (rows @ _exact_values(w[0][e], w[1][e]).T.contiguous() for w in (s["gate"], s["up"]))
            parts.append(a * torch.sigmoid(a) * u)
    return torch.cat(parts)


def _exact_norm(c, seed):
    s = {n: v.double() for n, v in _norm_inputs(c, seed).items()}
    x, w = s["x"], s["weight"]
    rms = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn = x / rms * w
    if not c["train"]:
        return xn
    # y = x w / rms(x): dy/dx = diag(w) / rms - x (x w)^T / (d rms^3)
    along = (s["d_xn"] * w * x).sum(-1, keepdim=True)
    d_x = s["d_residual"] + s["d_xn"] * w / rms - x * along / (c["d"] * rms ** 3)
    return dict(xn=xn, d_x=d_x, d_weight=(s["d_xn"] * x / rms).sum(0))


def _exact_combine(c, seed):
    s = _combine_inputs(c, seed)
    T, d, k, n = c["T"], c["d"], c["k"], c["n_gate"]
    slot = s["slot_of"].long().view(T, k)
    f = {m: v.double() for m, v in s.items() if v is not None and m != "slot_of"}
    y = torch.zeros((T, d), dtype=torch.float64, device=DEV)
    for j in range(k):
        y += f["topk_w"][:, j:j + 1] * f["y"][slot[:, j]]
    rms = torch.sqrt(y.square().mean(-1, keepdim=True) + EPS)
    gate = f["gate"][torch.arange(T, device=DEV) // (T // n)] if n else torch.ones((1, d), dtype=torch.float64, device=DEV)
    out = RES_SCALE * f["residual"] + gate * f["weight"] * (y / rms)
    if not c["train"]:
        return out
    up = f["d_out"] * gate * f["weight"]
    dy = up / rms - y * (up * y).sum(-1, keepdim=True) / (d * rms ** 3)
    d_y = torch.empty((T * k, d), dtype=torch.float64, device=DEV)
    d_topk_w = torch.empty((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        d_y[slot[:, j]] = f["topk_w"][:, j:j + 1] * dy
        d_topk_w[:, j] = (f["y"][slot[:, j]] * dy).sum(-1)
    each = f["d_out"] * y / rms
    r = dict(out=out, d_y=d_y, d_topk_w=d_topk_w, d_residual=RES_SCALE * f["d_out"], d_weight=(gate * each).sum(0))
    if n:
        r["d_gate"] = torch.stack([(f["weight"] * part).sum(0) for part in each.split(T // n)])
    return r


def exact(case, seed):
    c = dict(case)
    if c["op"] == "payload":
        x = _normal(_gen(seed + 17), (c["T"], c["d"]))
        return _exact_mx(x)[_dispatch(c, _gen(seed))[0].long() // c["k"]]
    return dict(few=_exact_few, product=_exact_product, norm=_exact_norm, combine=_exact_combine)[c["op"]](c, seed)
