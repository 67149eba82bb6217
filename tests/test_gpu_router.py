"""The router against its definition in 64 bits. The selection's key is a 32-bit number (logit, or
logit plus bias), so the ids have to be equal. Weights and statistics: exponentials within 2 units
in the last place, sums of at most 1024 terms in a tree and one division, so 4e-6 of the value; a
sum over T tokens in 32-bit partial sums stays within 1e-5. A gradient is a difference of terms:
1e-5 of the sum of their magnitudes, and 2^-8 of the value more for a bf16 one."""
import math

import pytest
import torch

from moe_ffn_expert_gb300 import _abi, block_ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def choose(key, K):
    """K largest per row, first of equals; NaN last."""
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key) + 0.0
    nan_last = torch.sort(key, dim=1, descending=True, stable=True).indices
    return nan_last[:, :K]


def shares(z, ids, score, normalize, scale):
    at = torch.gather(z, 1, ids)
    if score == "sigmoid":
        w = torch.sigmoid(at)
        if normalize:
            s = w.sum(1, keepdim=True)
            w = torch.where(s > 0, w / s, torch.zeros_like(w))
        return scale * w
    ref = at if normalize else z
    m = ref.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s = torch.exp(ref - m).sum(1, keepdim=True)
    return scale * torch.where(s > 0, torch.exp(at - m) / s, torch.zeros_like(at))


def probs(z, score):
    a = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    return a if score == "softmax" else a / a.sum(1, keepdim=True)


def logits(T, E, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1.5 * torch.randn(T, E, generator=g, device="cuda")).to(dt)


def check_forward(z, K, score, normalize, bias=None, scale=1.0, key=None):
    ids, w, ps, lse = block_ops.router_forward(z, K, bias=bias, score=score, normalize=normalize,
                                               scale=scale, stats=True)
    z32 = z.float()
    want = choose(z32 if bias is None else z32 + bias, K) if key is None else choose(key, K)
    assert torch.equal(ids.long(), want)
    z64 = z32.double()
    ref = shares(z64, want, score, normalize, scale)
    assert ((w.double() - ref).abs() <= 4e-6 * ref.abs() + 1e-37).all()
    ref = probs(z64, score).sum(0)
    assert ((ps.double() - ref).abs() <= 1e-5 * ref + 1e-37).all()
    ref = torch.logsumexp(z64, 1)
    assert ((lse.double() - ref).abs() <= 4e-6 * (1 + ref.abs())).all()
    ids2, w2, none, _ = block_ops.router_forward(z, K, bias=bias, score=score, normalize=normalize, scale=scale)
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and none is None


def gradient(z, ids, dw, dP, dL, score, normalize, scale):
    """In 64 bits, by the formulas; and the sums of the terms' magnitudes."""
    z = z.double()
    at = torch.gather(z, 1, ids)
    dz, mag = torch.zeros_like(z), torch.zeros_like(z)
    w = shares(z, ids, score, normalize, 1.0)
    one = 1.0 - torch.sigmoid(at) if score == "sigmoid" else torch.ones_like(at)
    if normalize:
        dot = (dw * w).sum(1, keepdim=True)
        t, m = scale * w * (dw - dot) * one, scale * w * (dw.abs() + (dw * w).abs().sum(1, keepdim=True)) * one
    else:
        t = scale * dw * w * one
        m = t.abs()
    if not normalize and score == "softmax":
        p = torch.softmax(z, 1)
        dz = dz - p * t.sum(1, keepdim=True)
        mag = mag + p * t.abs().sum(1, keepdim=True)
    dz, mag = dz.scatter_add(1, ids, t), mag.scatter_add(1, ids, m)
    if dP is not None:
        p = probs(z, score)
        f = p * (1 - torch.sigmoid(z)) if score == "sigmoid" else p
        dz = dz + f * (dP - (dP * p).sum(1, keepdim=True))
        mag = mag + f * (dP.abs() + (dP * p).abs().sum(1, keepdim=True))
    if dL is not None:
        dz = dz + dL[:, None] * torch.softmax(z, 1)
        mag = mag + dL.abs()[:, None] * torch.softmax(z, 1)
    return dz, mag


def check_backward(z, K, score, normalize, stats, scale=1.0, seed=3):
    T, E = z.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = choose(z.float(), K)
    dw = torch.randn(T, K, generator=g, device="cuda")
    dP = torch.randn(E, generator=g, device="cuda") if stats else None
    dL = torch.randn(T, generator=g, device="cuda") if stats else None
    got = block_ops.router_backward(z, ids.to(torch.int32), dw, dP, dL, score=score,
                                    normalize=normalize, scale=scale)
    d64 = [None if t is None else t.double() for t in (dw, dP, dL)]
    ref, mag = gradient(z, ids, *d64, score, normalize, scale)
    tol = 1e-5 * mag + (2.0 ** -8 * ref.abs() if z.dtype == BF else 0) + 1e-37
    assert got.dtype == z.dtype and ((got.double() - ref).abs() <= tol).all()


SHAPES = [(1, 1, 1), (1, 128, 8), (5, 7, 3), (64, 256, 8), (33, 60, 6), (130, 32, 16), (9, 1024, 16),
          (17, 500, 10), (2, 16, 16), (3000, 128, 8)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dt", [BF, F32])
def test_forward_and_backward(T, E, K, score, normalize, dt):
    z = logits(T, E, dt, seed=T + E)
    check_forward(z, K, score, normalize, scale=1.0 if normalize else 2.5)
    for stats in (False, True):
        check_backward(z, K, score, normalize, stats, scale=1.0 if normalize else 2.5)


@pytest.mark.parametrize("dt", [BF, F32])
def test_bias_takes_part_in_the_selection_only(dt):
    z = logits(300, 96, dt)
    b = torch.randn(96, device="cuda")
    check_forward(z, 8, "softmax", True, bias=b)
    check_forward(z, 8, "softmax", False, bias=b)
    check_forward(z, 8, "softmax", True, bias=40.0 * b)  # selected logits far below the row's largest


def test_sigmoid_bias_adds_to_the_score():
    """Keys on a coarse grid of biases (steps of 2 against scores in (0, 1)): the bias decides
    between groups, the score within one, and neither is near a tie."""
    z = (torch.arange(64, device="cuda").float() * 0.05 - 1.6).expand(7, 64)[:, torch.randperm(64, device="cuda")].contiguous()
    b = 2.0 * (torch.arange(64, device="cuda") % 5).float()
    check_forward(z, 6, "sigmoid", True, bias=b, key=torch.sigmoid(z.double()).float() + b)


def test_ties_go_to_the_lowest_expert():
    z = torch.zeros(40, 200, device="cuda")
    ids = block_ops.router_forward(z, 16)[0]
    assert torch.equal(ids, torch.arange(16, device="cuda", dtype=torch.int32).expand(40, 16))
    z[:, 150] = -0.0
    z[:, 3] = -0.0  # -0 equals 0
    assert torch.equal(block_ops.router_forward(z, 16)[0], ids)
    q = logits(500, 64, F32).mul(2).round().to(BF)  # a dozen values over 64 experts
    check_forward(q, 8, "softmax", True)


def test_masked_rows():
    inf = math.inf
    z = logits(6, 40, F32)
    z[0] = -inf                 # nothing left
    z[1, 3:] = -inf             # fewer than K left
    z[2, :20] = -inf
    z[3, 7] = inf
    z[4, 11] = math.nan
    z[5] = math.nan
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            ids, w, ps, lse = block_ops.router_forward(z, 8, score=score, normalize=normalize, stats=True)
            assert ((ids >= 0) & (ids < 40)).all()
            assert all(len(set(r)) == 8 for r in ids.tolist())
            assert torch.equal(ids[0], torch.arange(8, device="cuda", dtype=torch.int32))
            assert not w[0].any()
            assert set(ids[1].tolist()) == set(range(8)) and not w[1, 3:].any() and (w[1, :3] > 0).all()
            assert (ids[2] >= 20).all() and torch.isfinite(w[2]).all()
            assert ids[3, 0] == 7 and 11 not in ids[4].tolist()
            assert torch.isnan(w[5]).all()
            assert lse[0] == -inf and torch.isfinite(lse[1:3]).all()
            ref = shares(z[1:3].double(), ids[1:3].long(), score, normalize, 1.0)
            assert ((w[1:3].double() - ref).abs() <= 4e-6 * ref).all()
    ps = block_ops.router_forward(z[:3], 8, stats=True)[2].double()
    ref = torch.softmax(z[1:3].double(), 1).sum(0)  # the row of -inf adds nothing
    assert ((ps - ref).abs() <= 1e-5 * ref + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_masked_logits_get_no_gradient(score, normalize):
    z = logits(4, 50, F32)
    z[0] = -math.inf
    z[1, 5:] = -math.inf
    z[2, ::2] = -math.inf
    ids = choose(z, 8).to(torch.int32)
    g = block_ops.router_backward(z, ids, torch.randn(4, 8, device="cuda"), torch.randn(50, device="cuda"),
                                  torch.randn(4, device="cuda"), score=score, normalize=normalize)
    assert torch.isfinite(g).all() and not g[torch.isinf(z)].any() and g[3].any()


def test_ids_out_of_range_are_ignored():
    z = logits(3, 20, F32)
    ids = choose(z, 4).to(torch.int32)
    dw = torch.randn(3, 4, device="cuda")
    bad = ids.clone()
    bad[1, 2], bad[2, 0] = 20, -5
    got = block_ops.router_backward(z, bad, dw, score="sigmoid", normalize=False)
    ref = block_ops.router_backward(z, ids, dw, score="sigmoid", normalize=False)
    ref[1, ids[1, 2]] = 0
    ref[2, ids[2, 0]] = 0
    assert torch.equal(got, ref)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(score, normalize):
    """Along random directions; the step h = 2e-3 moves no logit past another (gaps of 0.05 at
    least), its third-order term is ~h^2 and the 32-bit noise ~1e-6 / h: 1 % of the gradient's norm
    is above both."""
    T, E, K = 6, 48, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.stack([torch.randperm(E, generator=g, device="cuda") for _ in range(T)]).float() * 0.05 - 1.2
    cw, cp, cl = (torch.randn(s, generator=g, device="cuda") for s in ((T, K), (E,), (T,)))
    kw = dict(score=score, normalize=normalize, scale=1.5, stats=True)

    def loss(v):
        _, w, p, l = block_ops.router_forward(v, K, **kw)
        return float((w.double() * cw).sum() + (p.double() * cp).sum() + (l.double() * cl).sum())

    leaf = z.clone().requires_grad_(True)
    _, w, p, l = block_ops.moe_router(leaf, K, **kw)
    torch.autograd.backward([w, p, l], [cw, cp, cl])
    for _ in range(6):
        d = torch.randn(T, E, generator=g, device="cuda").clamp(-3, 3)
        h = 2e-3
        num = (loss(z + h * d) - loss(z - h * d)) / (2 * h)
        assert abs(num - float((leaf.grad * d).sum())) <= 1e-2 * float(leaf.grad.norm())


def test_the_layer_takes_the_selection():
    """ids and weights go into the fused layer as they are, and the gradient comes back."""
    from moe_ffn_expert_gb300.torch_api import hyper_mega_moe
    T, H, I, E, K = 300, 256, 128, 8, 2
    z = logits(T, E, F32).requires_grad_(True)
    x = torch.randn(T, H, device="cuda").to(BF)
    up = (torch.randn(E, H, 2 * I, device="cuda") / 16).to(BF)
    down = (torch.randn(E, I, H, device="cuda") / 11).to(BF)
    ids, w, ps, lse = block_ops.moe_router(z, K, stats=True)
    y = hyper_mega_moe(x, ids, w, up, down)
    (y.float().square().mean() + 1e-2 * (ps / T).square().sum() + 1e-3 * lse.square().mean()).backward()
    assert torch.isfinite(z.grad).all() and z.grad.abs().sum() > 0


def test_no_tokens_strides_and_repeats():
    z = torch.empty(0, 16, device="cuda")
    ids, w, ps, lse = block_ops.router_forward(z, 4, stats=True)
    assert ids.shape == w.shape == (0, 4) and not ps.any() and lse.shape == (0,)
    assert block_ops.router_backward(z, ids, w).shape == (0, 16)
    a = logits(1000, 128, BF)
    wide = torch.stack([a, a], -1)[..., 0]
    r1, r2 = (block_ops.router_forward(t, 8, stats=True) for t in (a, wide))
    assert all(torch.equal(p, q) for p, q in zip(r1, r2))
    odd = torch.empty(a.numel() + 1, dtype=BF, device="cuda")[1:].view(a.shape).copy_(a)
    assert all(torch.equal(p, q) for p, q in zip(r1, block_ops.router_forward(odd, 8, stats=True)))


def test_refusals():
    z = logits(4, 16, F32)
    f = block_ops.router_forward
    for bad, err in ((lambda: f(z.cpu(), 2), ValueError), (lambda: f(z, 0), ValueError),
                     (lambda: f(z, 17), ValueError), (lambda: f(z.half(), 2), TypeError),
                     (lambda: f(z, 2, score="tanh"), ValueError), (lambda: f(z[0], 2), ValueError),
                     (lambda: f(z, 2, bias=torch.zeros(15, device="cuda")), ValueError),
                     (lambda: f(torch.zeros(2, 1025, device="cuda"), 2), _abi.MMError),
                     (lambda: f(torch.zeros(2, 64, device="cuda"), 17), _abi.MMError),
                     (lambda: block_ops.router_backward(z, torch.zeros(4, 2, device="cuda"), z[:, :2]), ValueError)):
        with pytest.raises(err):
            bad()


@pytest.mark.parametrize("T,E,K", [(20000, 128, 8), (9000, 100, 6), (20000, 16, 2), (9801, 64, 16), (6000, 256, 8),
                                   (6000, 512, 10), (5001, 1024, 16), (20000, 4, 1), (12345, 160, 8)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_many_rows(T, E, K, dt):
    z = logits(T, E, dt, seed=E)
    check_forward(z, K, "softmax", True)
    check_forward(z, K, "softmax", False, bias=torch.randn(E, device="cuda"))
    check_backward(z, K, "softmax", False, True)
    check_backward(z, K, "sigmoid", True, True)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("E", [32, 64, 128, 256, 512, 1024])
def test_logits_off_a_16_byte_boundary(dt, E):
    z = logits(300, E, dt)
    buf = torch.empty(z.numel() + 1, dtype=dt, device="cuda")
    odd = buf[1:].view(z.shape).copy_(z)
    K = 8
    a = block_ops.router_forward(z, K, stats=True)
    b = block_ops.router_forward(odd, K, stats=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    dw = torch.randn(300, K, device="cuda")
    g = block_ops.router_backward(z, a[0], dw, normalize=False)
    assert torch.equal(g, block_ops.router_backward(odd, a[0], dw, normalize=False))


@pytest.mark.parametrize("E", [3, 64, 128, 200, 1024])
def test_rows_of_equal_logits(E):
    """Every key alike, in every lane: the experts come in order."""
    K = min(E, 16)
    for v in (0.0, -0.0, -math.inf):
        ids, w, _, _ = block_ops.router_forward(torch.full((40, E), v, device="cuda"), K)
        assert torch.equal(ids, torch.arange(K, device="cuda", dtype=torch.int32).expand(40, K))
    z = torch.zeros(40, E, device="cuda", dtype=BF)
    z[:, E // 2:] = 1.0  # two values only
    assert torch.equal(block_ops.router_forward(z, K)[0].long(), choose(z.float(), K))


def test_more_than_2_31_logits():
    T, E = 2 ** 21 + 40, 1024
    z = logits(64, E, BF).repeat(T // 64 + 1, 1)[:T].contiguous()
    ids, w, ps, lse = block_ops.router_forward(z, 4, stats=True)
    assert torch.equal(ids[-64:].long(), choose(z[-64:].float(), 4))
    assert torch.allclose(lse[-64:].double(), torch.logsumexp(z[-64:].double(), 1), rtol=4e-6, atol=4e-6)
    dz = block_ops.router_backward(z, ids, torch.ones_like(w), None, torch.ones_like(lse), normalize=False)
    ref, mag = gradient(z[-64:], ids[-64:].long(), torch.ones(64, 4, device="cuda", dtype=torch.float64), None,
                        torch.ones(64, device="cuda", dtype=torch.float64), "softmax", False, 1.0)
    assert ((dz[-64:].double() - ref).abs() <= 1e-5 * mag + 2.0 ** -8 * ref.abs() + 1e-37).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_normalized_expert_has_a_constant_weight(score):
    """K = 1, normalised: the weight is `scale` whatever the logits, so their gradient is zero, without
    rounding noise (dw - dw w / w)."""
    z = logits(400, 16, F32)
    ids, w, _, _ = block_ops.router_forward(z, 1, score=score, scale=2.5)
    assert (w == 2.5).all()
    dw = torch.randn(400, 1, device="cuda")
    assert not block_ops.router_backward(z, ids, dw, score=score, scale=2.5).any()


@pytest.mark.parametrize("shift", [60.0, 88.0, 100.0, 200.0, 600.0])
@pytest.mark.parametrize("E,K", [(20, 3), (128, 8), (256, 8), (1000, 16)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sigmoid_scores_far_below_zero(shift, E, K, dt):
    """Scores whose sigmoids 32 bits cannot hold still have ratios: normalised weights, probabilities
    and their gradients, as defined. Rows of ordinary logits stand between."""
    z = logits(40, E, F32, seed=E)
    z[::2] -= shift
    z[5, 3:] = -math.inf
    z[6, 3:] = -math.inf
    z = z.to(dt)
    check_forward(z, K, "sigmoid", True, scale=1.5)
    check_backward(z[7:].contiguous(), K, "sigmoid", True, True, scale=1.5)


def test_log_sum_of_infinite_logits():
    """log sum exp of a row with +inf is +inf, unless a NaN stands beside it."""
    z = logits(4, 40, F32)
    z[0, 7] = math.inf
    z[1, 7], z[1, 9] = math.inf, -math.inf
    z[2, 7], z[2, 30] = math.inf, math.nan
    for score in ("softmax", "sigmoid"):
        lse = block_ops.router_forward(z, 4, score=score, stats=True)[3]
        assert torch.equal(lse.isnan(), torch.logsumexp(z, 1).isnan()) and (lse[:2] == math.inf).all()
        assert torch.isfinite(lse[3])
