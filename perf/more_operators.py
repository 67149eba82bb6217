"""Cases of the operators for experts of a caller's own form: what each is given, its plain form, its
definition in 64 bits, and the work it cannot do without.

* dispatch: the stable order of a selection's slots by expert (offsets, rows of slots, slots of rows)
  and the tokens' rows in that order; ids outside [0, E) are slots that no expert gets.
* grouped: the product of each expert's rows with its matrix, ragged sizes, and its gradients.
* combine: a token's weighted sum of its slots' rows, and its gradients.
* clip: the norm of all gradients together, and the gradients scaled down to a largest norm.

`own` chooses between the plain forms (elementary torch operations in 32 bits, rounded once at the
end) and the library's calls.
"""
import math
import random

import numpy
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-6
#: the largest listed cases: elements of dispatched rows, flops of a product, elements of gradients
MOST_ROWS, MOST_FLOPS, MOST_GRADS = 16384 * 8 * 2048, 2 * 131072 * 2048 * 1536, 128 * 2048 * 768 * 3
#: elements of the experts' matrices of the largest listed case
MOST_WEIGHTS = 128 * 2048 * 1536


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a decoding batch of 64 requests, 8 of 128 experts each: launches count
        _rows("dispatch_64x8", "dispatch", 64, 2048, 128, 8, "bf16"),
        # a training batch of the 128-expert layer
        _rows("dispatch_16384x8", "dispatch", 16384, 2048, 128, 8, "bf16"),
        # a prompt of the wide layer back in token order
        _rows("combine_fwd_4096x8", "combine_fwd", 4096, 7168, 256, 8, "bf16"),
        # an odd width, 32-bit rows, an odd batch of which every seventh slot has no expert
        _rows("combine_bwd_1001x6_fp32", "combine_bwd", 1001, 2047, 60, 6, "fp32", dropped=7),
        # one token of the 128-expert layer: eight experts' matrices, latency
        _grouped("grouped_fwd_8_e128", "grouped_fwd", 8, 2048, 1536, 128),
        # a decoding batch's second product, matrices [N, K] as a linear layer keeps them, 32-bit results
        _grouped("grouped_fwd_512_e128_t", "grouped_fwd", 512, 768, 2048, 128, out="fp32", transposed=True),
        # skewed sizes, odd widths, rows behind the last expert's (a buffer of fixed size)
        _grouped("grouped_fwd_6007_e32_zipf", "grouped_fwd", 6007, 2040, 1528, 32, zipf=True, tail=137),
        # a training batch of the 128-expert layer, first product
        _grouped("grouped_fwd_131072_e128", "grouped_fwd", 131072, 2048, 1536, 128),
        # the gradients of a skewed batch, some experts without rows
        _grouped("grouped_bwd_32768_e128_zipf", "grouped_bwd", 32768, 768, 2048, 128, zipf=True),
        # few wide experts, weight gradients in 32 bits
        _grouped("grouped_bwd_8192_e8_fp32", "grouped_bwd", 8192, 7168, 2048, 8, out="fp32"),
        # the small parameters of some blocks, mixed types, odd sizes, an empty tensor: latency
        _clip("clip_48_small", 48, 60000, "mixed"),
        # the experts' and other gradients of one 128-expert layer
        _clip("clip_24_layer", 24, MOST_GRADS, "bf16"),
    ]


def _rows(name, op, T, H, E, K, dtype, dropped=0):
    """dropped: every how many slots one has no expert (0: none)."""
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "K": K, "dtype": dtype, "dropped": dropped}


def _grouped(name, op, R, D, N, E, out="bf16", transposed=False, zipf=False, tail=0):
    """R rows of D in the groups and `tail` behind them, matrices D x N; out: the type of the results,
    of the weight gradients backward."""
    return {"name": name, "op": op, "R": R, "D": D, "N": N, "E": E, "out": out,
            "transposed": transposed, "zipf": zipf, "tail": tail}


def _clip(name, count, total, dtype, clips=True, sizes=1):
    """count tensors with about `total` elements together; sizes: which way they share them."""
    return {"name": name, "op": "clip", "count": count, "total": total, "dtype": dtype,
            "clips": clips, "sizes": sizes}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "combine_fwd", "combine_bwd", "grouped_fwd", "grouped_fwd",
                     "grouped_bwd", "grouped_bwd", "clip"])
    if op == "clip":
        total = _log_int(rng, 1000, MOST_GRADS)
        c = _clip("", _log_int(rng, 1, 400), total, rng.choice(["bf16", "fp32", "mixed"]),
                  rng.random() < 0.7, rng.randrange(1, 1000000))
        if c["dtype"] != "bf16":
            c["total"] = min(c["total"], MOST_GRADS // 2)
    elif op.startswith("grouped"):
        # widths of 64 to 7168, mostly multiples of 8, some odd; 1 to 131072 rows of 1 to 256 experts
        E = rng.choice([1, 2, 8, 16, 32, 60, 64, 128, 128, 256])
        D, N = _log_int(rng, 64, 7168), _log_int(rng, 64, 4096)
        if rng.random() < 0.75:
            D, N = D // 8 * 8, N // 8 * 8
        while E * D * N > MOST_WEIGHTS:
            E = max(1, E // 2)
        flops = 2 if op == "grouped_fwd" else 4
        R = _log_int(rng, 1, max(1, min(131072, MOST_FLOPS // (flops * D * N))))
        c = _grouped("", op, R, D, N, E, rng.choice(["bf16", "bf16", "fp32"]), rng.random() < 0.4,
                     rng.random() < 0.4, rng.choice([0, 0, 1, 77]))
    else:
        H = _log_int(rng, 64, 7168)
        H = H if rng.random() < 0.25 else H // 8 * 8
        E = rng.choice([2, 8, 16, 60, 64, 128, 256, 1024])
        K = min(E, rng.choice([1, 2, 4, 6, 8, 8, 16]))
        c = _rows("", op, _log_int(rng, 1, min(16384, MOST_ROWS // (2 * K * H))), H, E, K,
                  rng.choice(["bf16", "bf16", "fp32"]), rng.choice([0, 0, 3, 11]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "clip":
        return _prepare_clip(case, g)
    return _prepare_grouped(case, g) if op.startswith("grouped") else _prepare_rows(case, g)


def _normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _prepare_rows(case, g):
    T, H, E, K, dt = case["T"], case["H"], case["E"], case["K"], TYPES[case["dtype"]]
    s = {"case": case}
    # distinct experts per token, some liked more than others by all tokens
    liking = torch.randn(T, E, generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(liking, K, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        n = torch.arange(T * K, device="cuda").view(T, K)
        ids = torch.where(n % case["dropped"] == 1, torch.full_like(ids, -1), ids)
    s["ids"] = ids.contiguous()
    if case["op"] == "dispatch":
        s["x"] = _normal(g, (T, H), dt)
        return s
    # the order is in hand from the dispatch, as three arrays
    s["order"] = _plain_order(s["ids"], E)
    s["weights"] = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), dim=1)
    s["rows"] = _normal(g, (T * K, H), dt)
    if case["op"] == "combine_bwd":
        s["dy"] = _normal(g, (T, H), dt, 0.02)
    return s


def _prepare_grouped(case, g):
    R, D, N, E = (case[k] for k in ("R", "D", "N", "E"))
    s = {"case": case}
    p = torch.ones(E, device="cuda")
    if case["zipf"]:  # expert of rank i as popular as i^-1.2, ranks in any order
        p = (1.0 + torch.randperm(E, generator=g, device="cuda").float()).pow(-1.2)
    of = torch.multinomial(p, R, replacement=True, generator=g)
    counts = torch.bincount(of, minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["rows"] = _normal(g, (R + case["tail"], D), torch.bfloat16)
    shape = (E, N, D) if case["transposed"] else (E, D, N)
    w = _normal(g, shape, torch.bfloat16, 1.0 / math.sqrt(D))
    s["weight"] = w.transpose(1, 2) if case["transposed"] else w
    if case["op"] == "grouped_bwd":
        s["d_out"] = _normal(g, (R + case["tail"], N), torch.bfloat16, 0.02)
    return s


def _sizes(case):
    """Element counts: shares of very different size, one tensor without elements among many."""
    rng = random.Random(case["sizes"])
    n = case["count"]
    share = [math.exp(rng.uniform(0.0, 6.0)) for _ in range(n)]
    total = sum(share)
    sizes = [max(1, int(case["total"] * v / total)) for v in share]
    if n > 20:
        sizes[n // 2] = 0
    return sizes


def _prepare_clip(case, g):
    s = {"case": case, "grads": []}
    for i, n in enumerate(_sizes(case)):
        dt = TYPES[case["dtype"]] if case["dtype"] != "mixed" else (torch.bfloat16, torch.float32)[i % 2]
        s["grads"].append(_normal(g, (n,), dt, 0.02))
    s["max_norm"] = 1e-3 * math.sqrt(case["total"]) if case["clips"] else 1e6
    # where the optimizer wants them: the accumulated gradients stay as they are
    s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


# ------------------------------------------------------------------------------------ the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _expert_ops():
    from moe_ffn_expert_gb300 import expert_ops
    return expert_ops


def _order(s):
    """The order that the dispatch gave."""
    c = s["case"]
    return _expert_ops().ExpertTable(*s["order"], c["T"], c["K"], c["E"])


def _own_dispatch(s):
    ops = _expert_ops()
    table = ops.expert_table(s["ids"], s["case"]["E"])
    return {"offsets": table.offsets, "row_of_slot": table.row_of_slot,
            "slot_of_row": table.slot_of_row, "rows": ops.dispatch_forward(s["x"], table)}


def _own_combine_fwd(s):
    return {"y": _expert_ops().combine_forward(s["rows"], _order(s), s["weights"])}


def _own_combine_bwd(s):
    d_rows, d_weights = _expert_ops().combine_backward(s["dy"], s["rows"], _order(s), s["weights"])
    return {"d_rows": d_rows, "d_weights": d_weights}


def _own_grouped_fwd(s):
    return {"out": _expert_ops().grouped_mm_forward(s["rows"], s["weight"], s["offsets"],
                                                    out_dtype=TYPES[s["case"]["out"]])}


def _own_grouped_bwd(s):
    d_rows, d_weight = _expert_ops().grouped_mm_backward(
        s["d_out"], s["rows"], s["weight"], s["offsets"], weight_grad_dtype=TYPES[s["case"]["out"]])
    return {"d_rows": d_rows, "d_weight": d_weight}


def _own_clip(s):
    from moe_ffn_expert_gb300 import grad_ops
    norm = grad_ops.clip_grad_norm(s["grads"], s["max_norm"], eps=EPS, out=s["out"])
    return {"norm": norm, "grads": s["out"]}


# ------------------------------------------------------------------------------------ plain forms

def _plain_order(ids, E):
    """offsets [E+1], row_of_slot [T, K], slot_of_row [T K], int32."""
    flat = ids.reshape(-1).long()
    S = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    slots = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(S, device=ids.device)
    row = torch.empty_like(place)
    row[slots] = place
    row = torch.where(key < E, row, torch.full_like(row, -1))
    slots = torch.where(place < offsets[E], slots, torch.full_like(slots, -1))
    return offsets.to(torch.int32), row.view(ids.shape).to(torch.int32), slots.to(torch.int32)


def _plain_dispatch(s):
    offsets, row, slot = _plain_order(s["ids"], s["case"]["E"])
    taken = (slot >= 0)[:, None]
    rows = s["x"][slot.clamp_min(0).long() // s["case"]["K"]]
    rows = torch.where(taken, rows, torch.zeros_like(rows))
    return {"offsets": offsets, "row_of_slot": row, "slot_of_row": slot, "rows": rows}


def _plain_combine_fwd(s):
    T, H, K = (s["case"][k] for k in "THK")
    row = s["order"][1].long()
    y = torch.zeros(T, H, device="cuda")
    for k in range(K):
        at = row[:, k]
        o = s["rows"][at.clamp_min(0)].float() * s["weights"][:, k, None]
        y = y + torch.where((at >= 0)[:, None], o, torch.zeros_like(o))
    return {"y": y.to(s["rows"].dtype)}


def _plain_combine_bwd(s):
    T, H, K = (s["case"][k] for k in "THK")
    row, slot = s["order"][1].long(), s["order"][2].long()
    dy = s["dy"].float()
    at, taken = slot.clamp_min(0), (slot >= 0)[:, None]
    d_rows = dy[at // K] * s["weights"].reshape(-1)[at][:, None]
    d_rows = torch.where(taken, d_rows, torch.zeros_like(d_rows)).to(s["rows"].dtype)
    d_weights = torch.zeros(T, K, device="cuda")
    for k in range(K):
        dot = (dy * s["rows"][row[:, k].clamp_min(0)].float()).sum(dim=1)
        d_weights[:, k] = torch.where(row[:, k] >= 0, dot, torch.zeros_like(dot))
    return {"d_rows": d_rows, "d_weights": d_weights}


def _plain_grouped_fwd(s):
    c = s["case"]
    out = torch.zeros(s["rows"].shape[0], c["N"], dtype=TYPES[c["out"]], device="cuda")
    at = s["offsets"].tolist()
    for e in range(c["E"]):
        if at[e] < at[e + 1]:
            rows = slice(at[e], at[e + 1])
            out[rows] = torch.matmul(s["rows"][rows].float(), s["weight"][e].float()).to(out.dtype)
    return {"out": out}


def _plain_grouped_bwd(s):
    c = s["case"]
    d_rows = torch.zeros_like(s["rows"])
    d_weight = torch.zeros(s["weight"].shape, dtype=TYPES[c["out"]], device="cuda")
    at = s["offsets"].tolist()
    for e in range(c["E"]):
        if at[e] < at[e + 1]:
            rows = slice(at[e], at[e + 1])
            d = s["d_out"][rows].float()
            d_rows[rows] = torch.matmul(d, s["weight"][e].float().t()).to(d_rows.dtype)
            d_weight[e] = torch.matmul(s["rows"][rows].float().t(), d).to(d_weight.dtype)
    return {"d_rows": d_rows, "d_weight": d_weight}


def _plain_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")  # a long sum
    for t in s["grads"]:
        v = t.float()
        total = total + (v * v).sum(dtype=torch.float64)
    norm = total.sqrt()
    scale = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0).float()
    return {"norm": norm.float(), "grads": [(t.float() * scale).to(t.dtype) for t in s["grads"]]}


_PLAIN = {"dispatch": _plain_dispatch, "combine_fwd": _plain_combine_fwd,
          "combine_bwd": _plain_combine_bwd, "grouped_fwd": _plain_grouped_fwd,
          "grouped_bwd": _plain_grouped_bwd, "clip": _plain_clip}
_OWN = {"dispatch": _own_dispatch, "combine_fwd": _own_combine_fwd, "combine_bwd": _own_combine_bwd,
        "grouped_fwd": _own_grouped_fwd, "grouped_bwd": _own_grouped_bwd, "clip": _own_clip}


# ------------------------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    if op == "clip":
        sizes = _sizes(case)
        b = sum(n * (SIZE[case["dtype"]] if case["dtype"] != "mixed" else (2, 4)[i % 2])
                for i, n in enumerate(sizes))
        return {"bytes": 2 * b, "flops": 3 * sum(sizes)}
    if op.startswith("grouped"):
        R, D, N, E = (case[k] for k in ("R", "D", "N", "E"))
        weights = [(e + 1) ** -1.2 if case["zipf"] else 1.0 for e in range(E)]
        total = sum(weights)
        hit = sum(1.0 - (1.0 - w / total) ** R for w in weights)  # experts with a row, on average
        out = SIZE[case["out"]]
        tail = case["tail"]
        if op == "grouped_fwd":
            return {"bytes": 2 * R * D + 2 * hit * D * N + out * (R + tail) * N + 4 * (E + 1),
                    "flops": 2 * R * D * N}
        return {"bytes": 2 * R * (D + N) + 2 * hit * D * N + 2 * (R + tail) * D + out * E * D * N + 4 * (E + 1),
                "flops": 4 * R * D * N}
    T, H, E, K, b = case["T"], case["H"], case["E"], case["K"], SIZE[case["dtype"]]
    S = T * K
    lost = len(range(1, S, case["dropped"])) if case["dropped"] else 0  # slots without an expert
    if op == "dispatch":
        return {"bytes": b * H * (T + S) + 12 * S + 4 * (E + 1), "flops": 4 * S}
    if op == "combine_fwd":
        return {"bytes": b * H * (S - lost + T) + 8 * S, "flops": 2 * S * H}
    return {"bytes": b * H * (S - lost + T + S) + 16 * S, "flops": 3 * S * H}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        return _exact_clip(s)
    if op.startswith("grouped"):
        return _exact_grouped(s)
    if op == "dispatch":
        return _exact_dispatch(s)
    return _exact_combine(s)


def _exact_dispatch(s):
    """Slot lists expert by expert, on the host."""
    T, H, E, K = (s["case"][k] for k in "THEK")
    ids = s["ids"].cpu().numpy().reshape(-1)
    order = numpy.argsort(ids, kind="stable")
    order = order[(ids[order] >= 0) & (ids[order] < E)]
    starts = numpy.searchsorted(ids[order], numpy.arange(E + 1))
    slot = numpy.full(T * K, -1, dtype=numpy.int32)
    slot[:order.size] = order
    row = numpy.full(T * K, -1, dtype=numpy.int32)
    row[order] = numpy.arange(order.size)
    rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    token = torch.from_numpy(order // K).cuda()
    rows[:order.size] = s["x"].double().index_select(0, token)
    return {"offsets": torch.from_numpy(starts.astype(numpy.int32)).cuda(),
            "row_of_slot": torch.from_numpy(row.reshape(T, K)).cuda(),
            "slot_of_row": torch.from_numpy(slot).cuda(), "rows": rows}


def _exact_combine(s):
    """By pairs (token, row) of the slots that have an expert."""
    T, H, K = (s["case"][k] for k in "THK")
    row = s["order"][1].reshape(-1).long()
    slot = (row >= 0).nonzero()[:, 0]
    row, token = row[slot], torch.div(slot, K, rounding_mode="floor")
    w = s["weights"].double().reshape(-1)
    if s["case"]["op"] == "combine_fwd":
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for part in torch.arange(slot.numel(), device="cuda").split(1 << 14):
            y.index_add_(0, token[part], w[slot[part], None] * s["rows"][row[part]].double())
        return {"y": y}
    d_rows = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    d_w = torch.zeros(T * K, dtype=torch.float64, device="cuda")
    dy = s["dy"].double()
    for part in torch.arange(slot.numel(), device="cuda").split(1 << 14):
        d = dy[token[part]]
        d_rows[row[part]] = d * w[slot[part], None]
        d_w[slot[part]] = torch.einsum("sh,sh->s", d, s["rows"][row[part]].double())
    return {"d_rows": d_rows, "d_weights": d_w.view(T, K)}


def _exact_grouped(s):
    c = s["case"]
    x, n = s["rows"], s["rows"].shape[0]
    bounds = list(zip(s["offsets"][:-1].tolist(), s["offsets"][1:].tolist()))
    if c["op"] == "grouped_fwd":
        parts = [x[a:b].double() @ s["weight"][e].double() for e, (a, b) in enumerate(bounds)]
        parts.append(torch.zeros(n - bounds[-1][1], c["N"], dtype=torch.float64, device="cuda"))
        return {"out": torch.cat(parts)}
    d_rows = torch.zeros(n, c["D"], dtype=torch.float64, device="cuda")
    d_weight = torch.empty(c["E"], c["D"], c["N"], dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(bounds):
        d = s["d_out"][a:b].double()
        d_rows[a:b] = torch.einsum("rn,dn->rd", d, s["weight"][e].double())
        d_weight[e] = torch.einsum("rd,rn->dn", x[a:b].double(), d)
    return {"d_rows": d_rows, "d_weight": d_weight}


def _exact_clip(s):
    parts = [torch.linalg.vector_norm(t.double()) for t in s["grads"] if t.numel()]
    norm = torch.linalg.vector_norm(torch.stack(parts))
    share = min(1.0, s["max_norm"] / (norm.item() + EPS))
    return {"norm": norm, "grads": [t.double() * share for t in s["grads"]]}
