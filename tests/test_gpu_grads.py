"""The norm of many tensors and clipping against their definitions in 64 bits.

A thread sums at most 64 squares in 32 bits, four chains of 16, each step off by 2^-24 of the chain, the
rest in 64 bits: the sum of squares is off by at most 19 2^-24 of itself, the norm by half of that and
its own rounding, below 11 2^-24 = 7e-7. A scaled element is off by the scale's error (that and two
roundings) and by half a step of its type."""
import math

import pytest
import torch

from moe_ffn_expert_gb300 import grad_ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NORM = 7e-7
SETS = {"one": [1], "tiny": [1, 2, 3, 7, 8, 9], "empty": [0, 5, 0], "nothing": [0], "edges": [16383, 16384, 16385, 32768],
        "odd": [100003], "many": [(37 * i) % 101 for i in range(300)], "most": [5] * 2500, "large": [3_000_001, 70_000]}


def tensors(sizes, kind, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"bf16": [BF], "fp32": [F32], "mixed": [BF, F32]}[kind]
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(dt[i % len(dt)]) for i, n in enumerate(sizes)]


def norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def check_scaled(got, given, norm, max_norm, eps=1e-6):
    share = min(1.0, max_norm / (norm + eps))
    for d, s in zip(got, given):
        ref = s.double() * share
        assert d.shape == s.shape
        assert ((d.double() - ref).abs() <= (torch.finfo(d.dtype).eps / 2 + NORM + 2.0 ** -22) * ref.abs() + 1e-44).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", SETS.values(), ids=SETS)
def test_norm_and_clipping(sizes, kind):
    given = tensors(sizes, kind)
    norm = norm64(given)
    got = grad_ops.grad_norm(given)
    assert got.shape == () and got.dtype == F32 and abs(float(got) - norm) <= NORM * norm
    assert torch.equal(got, grad_ops.grad_norm(given))
    for max_norm in (0.5 * norm, 0.0):
        kept = [t.clone() for t in given]
        assert torch.equal(grad_ops.clip_grad_norm(kept, max_norm), got)
        check_scaled(kept, given, norm, max_norm)
    kept = [t.clone() for t in given]
    grad_ops.clip_grad_norm(kept, 2 * norm + 1)
    assert all(torch.equal(a, b) for a, b in zip(kept, given))


@pytest.mark.parametrize("sizes", SETS.values(), ids=SETS)
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("to", [BF, F32])
def test_into_other_tensors(sizes, kind, to):
    given = tensors(sizes, kind)
    before = [t.clone() for t in given]
    norm = norm64(given)
    for max_norm in (0.5 * norm, 2 * norm + 1):
        out = [torch.full_like(t, float("nan"), dtype=to) for t in given]
        grad_ops.clip_grad_norm(given, max_norm, out=out)
        check_scaled(out, given, norm, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(given, before))


def test_elements_of_any_size():
    """Squares beyond 32 bits: sums as in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.randn(70001, generator=g, device="cuda")
    for power in (-140, -130, -75, -60, -45, 50, 60, 70, 100, 110):
        t = (base.double() * 2.0 ** power).to(F32)
        norm = norm64([t])
        got = float(grad_ops.grad_norm([t]))
        assert abs(got - norm) <= NORM * norm + 2.0 ** -149
        if power < -130:
            continue  # (eps and the scaled elements are below 32 bits)
        kept = t.clone()
        grad_ops.clip_grad_norm([kept], 0.25 * norm, eps=0.0)
        check_scaled([kept], [t], norm, 0.25 * norm, eps=0.0)
    mixed = [base, base * 2.0 ** 100, base * 2.0 ** -100, torch.zeros(50000, device="cuda")]
    assert abs(float(grad_ops.grad_norm(mixed)) - norm64(mixed)) <= NORM * norm64(mixed)
    huge = torch.full((1000,), 3e38, device="cuda")  # a norm above 32 bits
    kept = huge.clone()
    assert math.isinf(float(grad_ops.clip_grad_norm([kept], 1.0)))
    check_scaled([kept], [huge], norm64([huge]), 1.0)


def test_infinities_and_nan_as_the_formula_has_them():
    for bad in (float("inf"), -float("inf"), float("nan")):
        for dt in (BF, F32):
            a, b = torch.ones(100, dtype=dt, device="cuda"), torch.ones(40000, dtype=dt, device="cuda")
            b[31234] = bad
            norm = grad_ops.clip_grad_norm([a, b], 1.0)
            if bad != bad:
                assert norm.isnan() and a.isnan().all() and b.isnan().all()
            else:
                assert norm.isinf() and (a == 0).all() and b[31234].isnan() and (b[:31234] == 0).all()
            assert not grad_ops.grad_norm(torch.ones(10, device="cuda")).isnan()


def test_strides_and_alignment():
    g = torch.Generator(device="cuda").manual_seed(2)
    for dt in (BF, F32):
        flat = torch.randn(5001, generator=g, device="cuda").to(dt)
        views = [flat[1:1001], flat[1001:1003], flat[1005:5001].view(4, 999).t(), flat[:0]]
        gaps = torch.randn(60, 70, generator=g, device="cuda").to(dt)
        views += [gaps[:, 3:20], torch.randn(3, 4, 5, generator=g, device="cuda").to(dt).permute(2, 0, 1)]
        before, rest = [v.clone() for v in views], gaps.clone()
        norm = norm64(before)
        assert abs(float(grad_ops.grad_norm(views)) - norm) <= NORM * norm
        out = [torch.empty_like(v.contiguous()).t().contiguous().t() if v.dim() == 2 else torch.empty_like(v)
               for v in views]
        grad_ops.clip_grad_norm(views, 0.1 * norm, out=out)
        check_scaled(out, before, norm, 0.1 * norm)
        strided = [torch.zeros(v.shape + (2,), dtype=v.dtype, device="cuda")[..., 0] for v in views]
        grad_ops.clip_grad_norm(views, 0.1 * norm, out=strided)
        check_scaled(strided, before, norm, 0.1 * norm)
        assert all(torch.equal(a, b) for a, b in zip(views, before))
        versions = [v._version for v in views]
        grad_ops.clip_grad_norm(views, 0.1 * norm)
        check_scaled(views, before, norm, 0.1 * norm)
        assert all(v._version > n for v, n in zip(views, versions))
        assert torch.equal(gaps[:, :3], rest[:, :3]) and torch.equal(gaps[:, 20:], rest[:, 20:])
        assert flat[0] == flat.clone()[0] and torch.equal(flat[1003:1005], flat[1003:1005].clone())


def test_a_model_with_parameters_that_have_no_gradient():
    p = [torch.nn.Parameter(torch.ones(50, device="cuda")) for _ in range(3)]
    (3 * p[0].sum() + 4 * p[2].sum()).backward()
    norm = grad_ops.clip_grad_norm([q.grad for q in p], 1.0)
    assert abs(float(norm) - 5 * math.sqrt(50)) <= NORM * 40
    assert abs(float(torch.cat([p[0].grad, p[2].grad]).norm()) - 1.0) < 1e-5 and p[1].grad is None
    assert float(grad_ops.grad_norm([None])) == 0 and float(grad_ops.clip_grad_norm([], 1.0)) == 0


def test_a_captured_call_replays_with_new_values():
    given = tensors([5000, 3, 70000], "mixed")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        grad_ops.grad_norm(given)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    norms = []
    for graph in graphs:
        with torch.cuda.graph(graph, stream=stream):
            norms.append(grad_ops.clip_grad_norm(given, 2.0))
    for seed in range(4):
        new = tensors([5000, 3, 70000], "mixed", seed=seed, scale=3.0 + seed)
        for t, v in zip(given, new):
            t.copy_(v)
        graphs[seed % 2].replay()
        torch.cuda.synchronize()
        norm = norm64(new)
        assert abs(float(norms[seed % 2]) - norm) <= NORM * norm
        check_scaled(given, new, norm, 2.0)


def test_offsets_past_32_bits():
    n = 2 ** 31 + 12345
    t = torch.full((n,), 0.5, dtype=BF, device="cuda")
    t[-3] = 3.0
    norm = math.sqrt((n - 1) * 0.25 + 9.0)
    assert abs(float(grad_ops.clip_grad_norm([t], norm / 2, eps=0.0)) - norm) <= NORM * norm
    assert float(t[0]) == 0.25 and float(t[-3]) == 1.5 and float(t[-1]) == 0.25 and float(t[2 ** 31 + 1]) == 0.25


def test_refusals():
    a, b = torch.ones(10, device="cuda"), torch.ones(10, device="cuda")
    for call in (lambda: grad_ops.grad_norm([a.cpu()]), lambda: grad_ops.grad_norm([a, b.cpu()]),
                 lambda: grad_ops.clip_grad_norm([a], -1.0), lambda: grad_ops.clip_grad_norm([a], float("nan")),
                 lambda: grad_ops.clip_grad_norm([a], 1.0, eps=-1.0), lambda: grad_ops.clip_grad_norm([a, a], 1.0),
                 lambda: grad_ops.clip_grad_norm([a, b], 1.0, out=[a]), lambda: grad_ops.clip_grad_norm([a], 1.0, out=[a[:5]]),
                 lambda: grad_ops.clip_grad_norm([a, b], 1.0, out=[b, torch.ones(10, device="cuda")]),
                 lambda: grad_ops.clip_grad_norm([a], 1.0, out=[None]), lambda: grad_ops.clip_grad_norm([a], 1.0, out=[a.cpu()])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: grad_ops.grad_norm([a.half()]), lambda: grad_ops.clip_grad_norm([a], 1.0, out=[a.double()])):
        with pytest.raises(TypeError):
            call()
    assert torch.equal(a, torch.ones(10, device="cuda"))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("to", [None, BF, F32])
def test_what_lies_around_the_tensors_stays_as_it_was(dt, to):
    """Views of one buffer at any place, elements between them and behind the last."""
    g = torch.Generator(device="cuda").manual_seed(4)
    flat = torch.randn(60000, generator=g, device="cuda").to(dt)
    given, at, inside = flat.clone(), 1, torch.zeros(60000, dtype=torch.bool, device="cuda")
    places = []
    for i, n in enumerate([1, 2, 7, 8, 9, 1003, 16383, 16385, 3, 20000, 5]):
        places.append((at, at + n))
        inside[at:at + n] = True
        at += n + 1 + i % 3
    target = flat if to is None else torch.full((60000,), 7.0, dtype=to, device="cuda")
    rest = target[~inside].clone()
    cut = lambda t: [t[a:b] for a, b in places]
    norm = norm64(cut(given))
    grad_ops.clip_grad_norm(cut(flat), 0.5 * norm, out=None if to is None else cut(target))
    check_scaled(cut(target), cut(given), norm, 0.5 * norm)
    assert torch.equal(target[~inside], rest)
    assert to is None or torch.equal(flat, given)
