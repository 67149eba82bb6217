"""Cases of the operators around and beside the MoE-FFN layer: what each is given, its plain form,
its definition in 64 bits, and the work it cannot do without.

Three operators of a transformer block whose FFN is a mixture of experts:

* residual_norm: r' = a r + g * rmsnorm(f) w_post, n = rmsnorm(r') w_pre, and its gradients;
* router: top-k selection over expert logits with its weights and statistics, and its gradient;
* moe_decode: the whole MoE layer (router product, selection, experts, weighted sum) for a few
  tokens, with bf16 expert weights or e4m3 ones that carry a scale per 128 x 128 block.

`own` chooses between the plain forms (elementary torch operations in 32 bits, rounded once at the
end) and the library's calls.
"""
import math

import torch

own = False

BLOCK = 128  # rows and columns of an e4m3 weight that share one scale
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4, "fp8": 1}
EPS = 1e-6
#: elements of the largest listed residual_norm case, rows x experts of the largest router case
MOST_NORM, MOST_ROUTER = 16384 * 2048, 16384 * 128


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # the step between two blocks for one token of a decoder: launch and row latency count
        _norm("norm_fwd_1x2048", "norm_fwd", 1, 2048, "bf16", "bf16", groups=1),
        # a prompt of the wide layer: 8 sequences of 512 tokens, each with a gate of its own
        _norm("norm_fwd_4096x7168", "norm_fwd", 4096, 7168, "bf16", "bf16", groups=8),
        # a training batch of the 2048-wide layer, a learned gate per channel
        _norm("norm_bwd_16384x2048", "norm_bwd", 16384, 2048, "bf16", "bf16", groups=1),
        # an odd width (rows that end off a 16-byte boundary), 32-bit tensors, 8 ragged groups
        _norm("norm_bwd_1000x2047_fp32", "norm_bwd", 1000, 2047, "fp32", "fp32", groups=8),
        # a decoding batch's selection, sigmoid scores
        _router("router_fwd_64x256", "router_fwd", 64, 256, 8, "fp32", "sigmoid", False, False),
        # a training batch's selection with a balancing bias and the loss statistics; bf16
        # logits tie often
        _router("router_fwd_16384x128", "router_fwd", 16384, 128, 8, "bf16", "softmax", True, True),
        # the gradient of a training batch through weights and loss statistics
        _router("router_bwd_8192x256", "router_bwd", 8192, 256, 8, "fp32", "softmax", False, True),
        # one token through the 128-expert layer: eight experts' weights, latency
        _decode("decode_1_e128", 1, 2048, 768, 128, 8, "bf16"),
        # a few concurrent requests, 8-bit weights
        _decode("decode_8_e128_fp8", 8, 2048, 768, 128, 8, "fp8"),
        # a full decoding batch: nearly every expert is hit
        _decode("decode_64_e128", 64, 2048, 768, 128, 8, "bf16"),
        # skewed ids from a router of the caller's, an odd batch, a shared expert
        _decode("decode_33_e32_zipf", 33, 2048, 768, 32, 6, "bf16", ids="zipf", shared=1536),
        # the wide layer: 16 requests, 8-bit weights, about 100 of 256 experts
        _decode("decode_16_e256_fp8", 16, 7168, 2048, 256, 8, "fp8", score="sigmoid"),
    ]


def _norm(name, op, T, H, stream, block, groups):
    return {"name": name, "op": op, "T": T, "H": H, "stream": stream, "block": block,
            "groups": groups, "post": True, "pre": True, "scale": 0.75}


def _router(name, op, T, E, K, dtype, score, bias, stats):
    return {"name": name, "op": op, "T": T, "E": E, "K": K, "dtype": dtype, "score": score,
            "normalize": True, "bias": bias, "stats": stats, "scale": 1.0}


def _decode(name, T, H, I, E, K, dtype, ids="router", shared=0, score="softmax"):
    return {"name": name, "op": "decode", "T": T, "H": H, "I": I, "E": E, "K": K, "dtype": dtype,
            "ids": ids, "shared": shared, "score": score}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "router_fwd", "router_bwd", "decode", "decode"])
    if op.startswith("norm"):
        # widths of 512 to 7168: mostly multiples of 8, some odd; 1 to 16384 tokens
        H = _log_int(rng, 512, 7168)
        H = H if rng.random() < 0.25 else max(512, H // 8 * 8)
        T = _log_int(rng, 1, min(16384, MOST_NORM // H))
        groups = rng.choice([0, 1, 1, 2, 5, T])
        T = max(1, T // max(1, groups)) * max(1, groups)
        while T * H > MOST_NORM:
            T, groups = max(1, T // 2), min(groups, 1)
        stream, block = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "bf16"),
                                    ("fp32", "fp32")])
        if stream == "fp32" and T * H > MOST_NORM // 2:
            stream, block = "bf16", "bf16"
        c = _norm("", op, T, H, stream, block, groups)
        c["post"], c["pre"] = rng.choice([(True, True), (True, True), (False, True), (True, False)])
        c["scale"] = rng.choice([1.0, 0.75])
    elif op.startswith("router"):
        E = rng.choice([4, 8, 16, 32, 60, 64, 100, 128, 160, 256, 384, 512, 1024])
        K = min(E, rng.choice([1, 2, 4, 6, 8, 8, 10, 16]))
        T = _log_int(rng, 1, min(16384, MOST_ROUTER // E))
        # a bias adds to the logits under softmax; under sigmoid it would add to scores
        # that differ by a last bit from one exponential to another, and so would ties
        score = rng.choice(["softmax", "softmax", "sigmoid"])
        c = _router("", op, T, E, K, rng.choice(["bf16", "fp32"]), score,
                    score == "softmax" and rng.random() < 0.5, rng.random() < 0.5)
        c["normalize"] = rng.random() < 0.7
        c["scale"] = rng.choice([1.0, 2.5])
    else:
        H, I, E, K = rng.choice([(512, 128, 4, 2), (1024, 512, 16, 4), (2048, 768, 32, 6),
                                 (2048, 768, 128, 8), (2048, 768, 128, 8), (7168, 2048, 64, 8)])
        if rng.random() < 0.3:  # odd widths
            H, I = H - 8 * rng.randrange(1, 12), I - 16 * rng.randrange(1, 6)
        T = _log_int(rng, 1, 64)
        c = _decode("", T, H, I, E, K, rng.choice(["bf16", "fp8"]),
                    ids=rng.choice(["router", "router", "zipf"]),
                    shared=rng.choice([0, 0, I]), score=rng.choice(["softmax", "sigmoid"]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op.startswith("norm"):
        return _prepare_norm(case, g)
    if op.startswith("router"):
        return _prepare_router(case, g)
    return _prepare_decode(case, g)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _prepare_norm(case, g):
    T, H, G = case["T"], case["H"], case["groups"]
    st, bt = TYPES[case["stream"]], TYPES[case["block"]]
    s = {"case": case, "scale": case["scale"]}
    # a residual stream that has grown over some layers, with a few channels far above the rest
    hot = 1.0 + 15.0 * (torch.rand(H, generator=g, device="cuda") < 0.004)
    s["residual"] = (3.0 * hot * _randn(g, T, H)).to(st)
    s["branch"] = (0.5 * _randn(g, T, H)).to(bt)
    s["post_weight"] = (0.3 + 0.1 * _randn(g, H)).to(st) if case["post"] else None
    s["pre_weight"] = (1.0 + 0.2 * _randn(g, H)).to(st) if case["pre"] else None
    s["gate"] = (0.6 + 0.3 * _randn(g, G, H)).to(st) if G else None
    if case["op"] == "norm_bwd":  # the forward's residual output, and the gradients of both outputs
        s["d_residual_out"] = (0.02 * _randn(g, T, H)).to(st)
        s["d_normed"] = (0.02 * _randn(g, T, H)).to(bt) if case["pre"] else None
    return s


def _prepare_router(case, g):
    T, E, K = case["T"], case["E"], case["K"]
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    # some experts are liked more than others, by all tokens
    s["logits"] = (1.2 * _randn(g, T, E) + 0.5 * _randn(g, E)).to(dt)
    s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
    if case["op"] == "router_bwd":
        ids, _ = _plain_select(s["logits"].float() + (s["bias"] if case["bias"] else 0.0), K)
        s["ids"] = ids.to(torch.int32)
        s["d_weights"] = _randn(g, T, K)
        s["d_prob_sum"] = _randn(g, E) * (0.01 * E / T) if case["stats"] else None
        s["d_lse"] = _randn(g, T) * 1e-3 if case["stats"] else None
    return s


def _quantized(w):
    """[R, C] in 32 bits -> e4m3 of the same shape and the scales of its 128 x 128 blocks."""
    R, C = w.shape
    br, bc = -(-R // BLOCK), -(-C // BLOCK)
    pad = torch.nn.functional.pad(w, (0, bc * BLOCK - C, 0, br * BLOCK - R))
    pad = pad.view(br, BLOCK, bc, BLOCK)
    scale = (pad.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(1e-12)
    q = (pad / scale[:, None, :, None]).view(br * BLOCK, bc * BLOCK)[:R, :C]
    return q.to(torch.float8_e4m3fn), scale


def _weights(g, n, R, C, dtype):
    """n matrices [R, C] ~ N(0, 1 / R): bf16, or e4m3 with scales."""
    if dtype == "bf16":
        w = torch.empty(n, R, C, dtype=torch.bfloat16, device="cuda")
        w.normal_(0.0, 1.0 / math.sqrt(R), generator=g)
        return w, None
    q = torch.empty(n, R, C, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(n, -(-R // BLOCK), -(-C // BLOCK), device="cuda")
    for e in range(n):
        q[e], sc[e] = _quantized(_randn(g, R, C) * (1.0 / math.sqrt(R)))
    return q, sc


def _prepare_decode(case, g):
    T, H, I, E, K = (case[k] for k in "THIEK")
    s = {"case": case}
    s["x"] = _randn(g, T, H).to(torch.bfloat16)
    s["up"], s["up_scale"] = _weights(g, E, H, 2 * I, case["dtype"])
    s["down"], s["down_scale"] = _weights(g, E, I, H, case["dtype"])
    s["shared"] = None
    if case["shared"]:
        Is = case["shared"]
        su, sus = _weights(g, 1, H, 2 * Is, case["dtype"])
        sd, sds = _weights(g, 1, Is, H, case["dtype"])
        s["shared"] = [None if t is None else t[0] for t in (su, sd, sus, sds)]
    s["router"] = s["ids"] = s["weights"] = None
    if case["ids"] == "router":
        s["router"] = (_randn(g, E, H) * (1.2 / math.sqrt(H))).to(torch.bfloat16)
    else:  # drawn without replacement, expert e as popular as (e + 1)^-1.2
        p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-1.2).expand(T, E)
        s["ids"] = torch.multinomial(p, K, generator=g).to(torch.int32)
        s["weights"] = torch.softmax(_randn(g, T, K), dim=1)
    return s


# ------------------------------------------------------------------------------------ the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


_ops = None


def _api():
    global _ops
    if _ops is None:
        from moe_ffn_expert_gb300 import block_ops
        _ops = block_ops
    return _ops


def _own_norm_fwd(s):
    out, normed = _api().residual_norm_forward(
        s["residual"], s["branch"], post_weight=s["post_weight"], pre_weight=s["pre_weight"],
        gate=s["gate"], residual_scale=s["scale"], eps=EPS)
    return {"residual_out": out, "normed": normed}


def _own_norm_bwd(s):
    names = ("d_residual", "d_branch", "d_post_weight", "d_pre_weight", "d_gate")
    return dict(zip(names, _api().residual_norm_backward(
        s["residual"], s["branch"], s["d_residual_out"], s["d_normed"],
        post_weight=s["post_weight"], pre_weight=s["pre_weight"], gate=s["gate"],
        residual_scale=s["scale"], eps=EPS)))


def _own_router_fwd(s):
    c = s["case"]
    names = ("ids", "weights", "prob_sum", "lse")
    return dict(zip(names, _api().router_forward(
        s["logits"], c["K"], bias=s["bias"], score=c["score"], normalize=c["normalize"],
        scale=c["scale"], stats=c["stats"])))


def _own_router_bwd(s):
    c = s["case"]
    return {"d_logits": _api().router_backward(
        s["logits"], s["ids"], s["d_weights"], s["d_prob_sum"], s["d_lse"], score=c["score"],
        normalize=c["normalize"], scale=c["scale"])}


def _own_decode(s):
    layer = s.get("layer")
    if layer is None:  # a serving program makes one for its weights and keeps it
        c = s["case"]
        layer = s["layer"] = _api().MoEDecoder(
            s["up"], s["down"], up_scale=s["up_scale"], down_scale=s["down_scale"], k=c["K"],
            router_weight=s["router"], score=c["score"], shared=s["shared"], max_tokens=c["T"])
    return {"y": layer(s["x"], s["ids"], s["weights"])}


# ------------------------------------------------------------------------------------ plain forms

def _plain_rms(v, eps):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps)


def _spread(gate, T):
    """[G, H] -> [T, H]: row t belongs to group t / (T / G)."""
    return gate.float().repeat_interleave(T // gate.shape[0], dim=0)


def _plain_norm_fwd(s):
    r, f = s["residual"].float(), s["branch"].float()
    if s["post_weight"] is not None:
        f = f * _plain_rms(f, EPS) * s["post_weight"].float()
    if s["gate"] is not None:
        f = f * _spread(s["gate"], r.shape[0])
    out = s["scale"] * r + f
    normed = None
    if s["pre_weight"] is not None:
        normed = (out * _plain_rms(out, EPS) * s["pre_weight"].float()).to(s["branch"].dtype)
    return {"residual_out": out.to(s["residual"].dtype), "normed": normed}


def _plain_norm_bwd(s):
    r, f = s["residual"].float(), s["branch"].float()  # r: the forward's residual output
    T, H = r.shape
    st, bt = s["residual"].dtype, s["branch"].dtype
    d = s["d_residual_out"].float()
    d_pre = d_post = d_gate = None
    if s["pre_weight"] is not None:
        dn, w = s["d_normed"].float(), s["pre_weight"].float()
        q = _plain_rms(r, EPS)
        d_pre = (dn * r * q).sum(dim=0).to(st)
        wd = dn * w
        d = d + q * wd - r * (q ** 3 / H) * (wd * r).sum(dim=1, keepdim=True)
    p = f
    if s["post_weight"] is not None:
        q = _plain_rms(f, EPS)
        p = f * q * s["post_weight"].float()
    dp = d
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        d_gate = (d * p).view(G, T // G, H).sum(dim=1).to(st)
        dp = d * _spread(s["gate"], T)
    df = dp
    if s["post_weight"] is not None:
        d_post = (dp * f * q).sum(dim=0).to(st)
        wd = dp * s["post_weight"].float()
        df = q * wd - f * (q ** 3 / H) * (wd * f).sum(dim=1, keepdim=True)
    return {"d_residual": (s["scale"] * d).to(st), "d_branch": df.to(bt), "d_post_weight": d_post,
            "d_pre_weight": d_pre, "d_gate": d_gate}


def _plain_select(key, K):
    """The K largest of each row, equal ones from the lowest index."""
    v, i = torch.sort(key, dim=1, descending=True, stable=True)
    return i[:, :K], v[:, :K]


def _plain_scores(logits, score):
    """a: what softmax or sigmoid gives each expert before any division, and its row sum."""
    if score == "softmax":
        a = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    else:
        a = 1.0 / (1.0 + torch.exp(-logits))
    return a, a.sum(dim=1, keepdim=True)


def _plain_weights(a, total, ids, score, normalize, scale):
    sel = torch.gather(a, 1, ids)
    if normalize:
        return scale * sel / sel.sum(dim=1, keepdim=True)
    return scale * sel / total if score == "softmax" else scale * sel


def _plain_router_fwd(s):
    c = s["case"]
    z = s["logits"].float()
    ids, _ = _plain_select(z + s["bias"] if s["bias"] is not None else z, c["K"])
    a, total = _plain_scores(z, c["score"])
    w = _plain_weights(a, total, ids, c["score"], c["normalize"], c["scale"])
    out = {"ids": ids.to(torch.int32), "weights": w}
    if c["stats"]:
        out["prob_sum"] = (a / total).sum(dim=0)
        out["lse"] = torch.log(torch.exp(z - z.amax(1, keepdim=True)).sum(1)) + z.amax(1)
    return out


def _plain_router_bwd(s):
    c = s["case"]
    z = s["logits"].float()
    ids, dw = s["ids"].long(), s["d_weights"]
    a, total = _plain_scores(z, c["score"])
    sel = torch.gather(a, 1, ids)
    da = torch.zeros_like(a)
    if c["normalize"]:
        n = sel.sum(dim=1, keepdim=True)
        u = c["scale"] * (dw - (dw * sel).sum(dim=1, keepdim=True) / n) / n
    elif c["score"] == "softmax":
        u = c["scale"] * dw / total
        da = da - c["scale"] * (dw * sel).sum(dim=1, keepdim=True) / (total * total)
    else:
        u = c["scale"] * dw
    da = da.scatter_add(1, ids, u)
    if s["d_prob_sum"] is not None:
        dp = s["d_prob_sum"]
        da = da + (dp - (dp * a).sum(dim=1, keepdim=True) / total) / total
    dz = da * (a if c["score"] == "softmax" else a * (1.0 - a))
    if s["d_lse"] is not None:
        e = torch.exp(z - z.amax(dim=1, keepdim=True))
        dz = dz + s["d_lse"][:, None] * e / e.sum(dim=1, keepdim=True)
    return {"d_logits": dz.to(s["logits"].dtype)}


def _plain_dequantized(q, scale):
    """[n, R, C] in 32 bits."""
    if scale is None:
        return q.float()
    n, R, C = q.shape
    sc = scale.repeat_interleave(BLOCK, dim=1)[:, :R].repeat_interleave(BLOCK, dim=2)[:, :, :C]
    return q.float() * sc


def _plain_pick(q, hit):
    """q[hit] (8-bit types have no indexing of their own)."""
    return q.view(torch.uint8)[hit].view(q.dtype) if q.dtype == torch.float8_e4m3fn else q[hit]


def _plain_ffn(x, up, down):
    """x [T, H], up [n, H, 2I], down [n, I, H] -> [n, T, H]."""
    gu = torch.matmul(x, up)
    gate, lin = gu.chunk(2, dim=2)
    return torch.matmul(gate / (1.0 + torch.exp(-gate)) * lin, down)


def _plain_decode(s):
    c = s["case"]
    x = s["x"].float()
    if s["router"] is not None:
        z = torch.matmul(x, s["router"].float().t())
        ids, _ = _plain_select(z, c["K"])
        a, total = _plain_scores(z, c["score"])
        w = _plain_weights(a, total, ids, c["score"], True, 1.0)
    else:
        ids, w = s["ids"].long(), s["weights"]
    hit, at = torch.unique(ids, return_inverse=True)
    scales = [None if t is None else t[hit] for t in (s["up_scale"], s["down_scale"])]
    o = _plain_ffn(x, _plain_dequantized(_plain_pick(s["up"], hit), scales[0]),
                   _plain_dequantized(_plain_pick(s["down"], hit), scales[1]))
    share = torch.zeros(c["T"], hit.numel(), device="cuda").scatter_add(1, at, w)
    y = (share.t()[:, :, None] * o).sum(dim=0)
    if s["shared"] is not None:
        su, sd, sus, sds = s["shared"]
        y = y + _plain_ffn(x, _plain_dequantized(su[None], None if sus is None else sus[None]),
                           _plain_dequantized(sd[None], None if sds is None else sds[None]))[0]
    return {"y": y.to(torch.bfloat16)}


_PLAIN = {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "decode": _plain_decode,
          "router_fwd": _plain_router_fwd, "router_bwd": _plain_router_bwd}
_OWN = {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "decode": _own_decode,
        "router_fwd": _own_router_fwd, "router_bwd": _own_router_bwd}


# ------------------------------------------------------------------------------------ the work

def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        H, st, bt = case["H"], SIZE[case["stream"]], SIZE[case["block"]]
        vectors = (case["post"] + case["pre"] + case["groups"]) * H * st
        if op == "norm_fwd":  # residual and branch in, residual out and its norm out
            return {"bytes": T * H * (2 * st + bt + case["pre"] * bt) + vectors, "flops": 12 * T * H}
        # residual, branch and both gradients in, two gradients out
        return {"bytes": T * H * (3 * st + 2 * bt + case["pre"] * bt) + 2 * vectors,
                "flops": 30 * T * H}
    if op.startswith("router"):
        E, K, b = case["E"], case["K"], SIZE[case["dtype"]]
        stats = case["stats"] * (4 * T + 4 * E)
        if op == "router_fwd":
            return {"bytes": T * E * b + 8 * T * K + 4 * E * case["bias"] + stats,
                    "flops": 8 * T * E}
        return {"bytes": 2 * T * E * b + 8 * T * K + stats, "flops": 12 * T * E}
    H, I, E, K, b = case["H"], case["I"], case["E"], case["K"], SIZE[case["dtype"]]
    if case["ids"] == "router":  # distinct experts over T tokens of K each, uniform choice
        hit = E * (1.0 - (1.0 - K / E) ** T)
    else:  # a token of popularity p_e has expert e with probability of about 1 - (1 - p_e)^K
        total = sum((e + 1) ** -1.2 for e in range(E))
        hit = sum(1.0 - (1.0 - (e + 1) ** -1.2 / total) ** (K * T) for e in range(E))
    scale = 4.0 / (BLOCK * BLOCK) if case["dtype"] == "fp8" else 0.0
    weights = (hit * I + case["shared"]) * 3 * H * (b + scale)
    router = 2 * E * H if case["ids"] == "router" else 8 * T * K
    return {"bytes": weights + router + 4 * T * H, "flops": 6 * H * T * (K * I + case["shared"])}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        return _exact_norm_fwd(s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    if op == "router_fwd":
        return _exact_router_fwd(s)
    if op == "router_bwd":
        return _exact_router_bwd(s)
    return {"y": _exact_decode(s)}


def _group_of(s):
    """The gate's row of each token."""
    T = s["residual"].shape[0]
    return torch.div(torch.arange(T, device="cuda") * s["gate"].shape[0], T, rounding_mode="floor")


def _unit(v):
    """v over the root of its rows' mean square (with eps), and that root."""
    root = torch.sqrt(torch.einsum("th,th->t", v, v) / v.shape[1] + EPS)[:, None]
    return v / root, root


def _exact_norm_fwd(s):
    y = s["branch"].double()
    if s["post_weight"] is not None:
        y = _unit(y)[0].mul_(s["post_weight"].double())
    if s["gate"] is not None:
        y = y * s["gate"].double()[_group_of(s)]
    y = y + s["residual"].double() * s["scale"]
    n = None if s["pre_weight"] is None else _unit(y)[0] * s["pre_weight"].double()
    return {"residual_out": y, "normed": n}


def _unit_gradient(unit, root, d):
    """Through v -> unit(v): the part of d along the unit row drops out, the rest is divided."""
    along = torch.einsum("th,th->t", unit, d)[:, None] / unit.shape[1]
    return (d - unit * along) / root


def _exact_norm_bwd(s):
    out = dict.fromkeys(("d_residual", "d_branch", "d_post_weight", "d_pre_weight", "d_gate"))
    d = s["d_residual_out"].double()
    if s["pre_weight"] is not None:
        unit, root = _unit(s["residual"].double())
        dn = s["d_normed"].double()
        out["d_pre_weight"] = torch.einsum("th,th->h", unit, dn)
        d = d + _unit_gradient(unit, root, dn * s["pre_weight"].double())
    out["d_residual"] = d * s["scale"]
    y = unit = s["branch"].double()
    root = None
    if s["post_weight"] is not None:
        unit, root = _unit(y)
        y = unit * s["post_weight"].double()
    if s["gate"] is not None:
        of = _group_of(s)
        out["d_gate"] = torch.zeros(s["gate"].shape, dtype=torch.float64,
                                    device="cuda").index_add_(0, of, d * y)
        d = d * s["gate"].double()[of]
    if root is not None:
        out["d_post_weight"] = torch.einsum("th,th->h", unit, d)
        d = _unit_gradient(unit, root, d * s["post_weight"].double())
    out["d_branch"] = d
    return out


def _exact_choice(key32, K):
    """Expert by expert: the largest left, the first of equals. The key is a number in 32 bits."""
    key = key32.clone()
    picked = []
    for _ in range(K):
        top = key == key.amax(dim=1, keepdim=True)
        first = top.to(torch.int32).argmax(dim=1)
        picked.append(first)
        key[torch.arange(key.shape[0], device="cuda"), first] = -math.inf
    return torch.stack(picked, dim=1)


def _exact_probabilities(z, score):
    if score == "softmax":
        return torch.softmax(z, dim=1)
    v = torch.sigmoid(z)
    return v / v.sum(dim=1, keepdim=True)


def _exact_share(z, ids, score, normalize, scale):
    at = torch.gather(z, 1, ids)
    if score == "softmax":
        w = torch.softmax(at, 1) if normalize else torch.exp(at - torch.logsumexp(z, 1)[:, None])
    else:
        w = torch.sigmoid(at)
        w = w / w.sum(dim=1, keepdim=True) if normalize else w
    return w * scale


def _exact_router_fwd(s):
    c, z32 = s["case"], s["logits"].float()
    z = z32.double()
    ids = _exact_choice(z32 if s["bias"] is None else z32 + s["bias"], c["K"])
    out = {"ids": ids.to(torch.int32),
           "weights": _exact_share(z, ids, c["score"], c["normalize"], c["scale"])}
    if c["stats"]:
        out["prob_sum"] = _exact_probabilities(z, c["score"]).sum(dim=0)
        out["lse"] = torch.logsumexp(z, dim=1)
    return out


def _exact_router_bwd(s):
    """The definition's derivative, by torch's own differentiation in 64 bits."""
    c = s["case"]
    z = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        loss = (_exact_share(z, s["ids"].long(), c["score"], c["normalize"], c["scale"])
                * s["d_weights"].double()).sum()
        if c["stats"]:
            loss = loss + (_exact_probabilities(z, c["score"]) * s["d_prob_sum"].double()).sum()
            loss = loss + (torch.logsumexp(z, dim=1) * s["d_lse"].double()).sum()
        return {"d_logits": torch.autograd.grad(loss, z)[0]}


def _exact_matrix(q, scale):
    w = q.float().double()
    if scale is None:
        return w
    rows = torch.arange(w.shape[0], device="cuda") // BLOCK
    cols = torch.arange(w.shape[1], device="cuda") // BLOCK
    return w * scale.double()[rows][:, cols]


def _exact_expert(x, up, down):
    gate, lin = torch.tensor_split(x @ up, 2, dim=1)
    return (gate * torch.sigmoid(gate) * lin) @ down


def _exact_decode(s):
    c = s["case"]
    x = s["x"].double()
    if s["router"] is not None:
        z = x @ s["router"].double().t()
        ids = _exact_choice(z, c["K"])
        w = _exact_share(z, ids, c["score"], True, 1.0)
    else:
        ids, w = s["ids"].long(), s["weights"].double()
    y = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, k = (ids == e).nonzero(as_tuple=True)
        us, ds = (None, None) if s["up_scale"] is None else (s["up_scale"][e], s["down_scale"][e])
        o = _exact_expert(x[t], _exact_matrix(s["up"][e], us), _exact_matrix(s["down"][e], ds))
        y.index_add_(0, t, o * w[t, k][:, None])
    if s["shared"] is not None:
        su, sd, sus, sds = s["shared"]
        y = y + _exact_expert(x, _exact_matrix(su, sus), _exact_matrix(sd, sds))
    return y
