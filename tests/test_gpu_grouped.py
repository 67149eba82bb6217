"""Products grouped by expert against their definition in 64 bits.

Tolerances: products of bf16 numbers are exact in 32 bits. An instruction of the tensor cores adds 16 of
them to the accumulator; the sum of its 17 numbers is off by at most 2^-22 of the sum of magnitudes so
far (each number is cut at the 24 bits of the largest). Over a sum of n terms that is
(n / 16 + 1) 2^-22 of the magnitudes' sum, and the result's rounding is half a step of its type."""
import random

import pytest
import torch

from moe_ffn_expert_gb300 import _abi, expert_ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SINGLE, PAIRS = _abi.MM_GROUPED_SINGLE_CTA, _abi.MM_GROUPED_CTA_PAIRS
NAN = float("nan")


def offsets_of(sizes, before=0):
    at = [before]
    for n in sizes:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def inputs(sizes, K, N, transposed=False, before=0, behind=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, E = before + sum(sizes) + behind, len(sizes)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").to(BF)

    w = randn(E, N, K).transpose(1, 2) if transposed else randn(E, K, N)
    return randn(R, K), w, offsets_of(sizes, before), randn(R, N)


def spans(offsets):
    at = offsets.tolist()
    return list(enumerate(zip(at[:-1], at[1:])))


def close(got, ref, mag, terms):
    assert got.shape == ref.shape
    tol = torch.finfo(got.dtype).eps / 2 * ref.abs() + (terms / 16 + 1) * 2.0 ** -22 * mag
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def check_forward(rows, weight, offsets, **how):
    got = expert_ops.grouped_mm_forward(rows, weight, offsets, **how)
    ref = torch.zeros(got.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for e, (a, b) in spans(offsets):
        x, w = rows[a:b].double(), weight[e].double()
        ref[a:b], mag[a:b] = x @ w, x.abs() @ w.abs()
    assert got.dtype == (how.get("out_dtype") or BF) and got.is_contiguous()
    close(got, ref, mag, rows.shape[1])
    return got


def check_weight_grad(rows, d_out, offsets, weight, **how):
    got = expert_ops.grouped_mm_weight_grad(rows, d_out, offsets, weight, **how)
    ref = torch.zeros(weight.shape, dtype=torch.float64, device="cuda")
    mag, terms = torch.zeros_like(ref), 0
    for e, (a, b) in spans(offsets):
        x, d = rows[a:b].double(), d_out[a:b].double()
        ref[e], mag[e], terms = x.t() @ d, x.abs().t() @ d.abs(), max(terms, b - a)
    assert got.dtype == (how.get("dtype") or BF)
    close(got, ref, mag, terms)
    return got


SIZES = {"one": [1], "two": [1, 1], "ragged": [16, 17, 255, 256, 257, 0, 513, 3], "empty": [0, 0, 0],
         "last": [0, 0, 31], "even": [64, 128], "many": [5] * 40, "wide": [1025, 700]}


@pytest.mark.parametrize("form", [SINGLE, PAIRS, 0])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (200, 520), (1024, 264)])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES)
def test_forward(sizes, K, N, form):
    for transposed in (False, True):
        for out in (BF, F32):
            x, w, at, _ = inputs(sizes, K, N, transposed)
            check_forward(x, w, at, out_dtype=out, flags=form)


@pytest.mark.parametrize("form", [SINGLE, PAIRS, 0])
@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (520, 200), (264, 1024)])
@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES)
def test_weight_grad(sizes, K, N, form):
    for transposed in (False, True):
        for out in (BF, F32):
            x, w, at, d = inputs(sizes, K, N, transposed)
            got = check_weight_grad(x, d, at, w, dtype=out, flags=form)
            assert got.transpose(1, 2).is_contiguous() if transposed else got.is_contiguous()


@pytest.mark.parametrize("K,N", [(33, 70), (7, 8), (64, 1), (1, 1), (130, 96)])
def test_odd_widths(K, N):
    x, w, at, d = inputs([3, 0, 40, 1], K, N, transposed=True, behind=2)
    check_forward(x, w, at)
    got = check_weight_grad(x, d, at, w, dtype=F32)
    assert got.transpose(1, 2).is_contiguous()
    into = torch.ones(w.shape, device="cuda")
    expert_ops.grouped_mm_weight_grad(x, d, at, w, into=into)
    assert torch.allclose(into - 1, check_weight_grad(x, d, at, w, dtype=F32), atol=1e-5, rtol=1e-6)


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
def test_both_forms_give_the_same_bits(form):
    x, w, at, d = inputs([300, 1, 0, 77, 900], 776, 392, behind=9)
    assert torch.equal(expert_ops.grouped_mm_forward(x, w, at, flags=form), expert_ops.grouped_mm_forward(x, w, at))
    assert torch.equal(expert_ops.grouped_mm_weight_grad(x, d, at, w, flags=form),
                       expert_ops.grouped_mm_weight_grad(x, d, at, w))


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_rows_of_others_have_no_part(form, value):
    """An expert's results do not depend on what its neighbours' rows and the rows of nobody hold."""
    sizes = [21, 5, 40, 0, 130, 1]
    x, w, at, d = inputs(sizes, 136, 264, before=3, behind=50)
    clean_out = check_forward(x, w, at, flags=form)
    clean_dw = check_weight_grad(x, d, at, w, flags=form)
    assert (clean_out[:3] == 0).all() and (clean_out[-50:] == 0).all()
    for e, (a, b) in spans(at):
        x2, d2 = torch.full_like(x, value), torch.full_like(d, value)
        x2[a:b], d2[a:b] = x[a:b], d[a:b]
        assert torch.equal(expert_ops.grouped_mm_forward(x2, w, at, flags=form)[a:b], clean_out[a:b])
        assert torch.equal(expert_ops.grouped_mm_weight_grad(x2, d2, at, w, flags=form)[e], clean_dw[e])
    w2 = torch.full_like(w, value)
    w2[4] = w[4]
    a, b = at[4].item(), at[5].item()
    got = expert_ops.grouped_mm_forward(x, w2, at, flags=form)
    assert torch.equal(got[a:b], clean_out[a:b]) and (got[:3] == 0).all() and (got[-50:] == 0).all()


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("bad", [[-1, 5, 9], [0, 9, 5], [0, 5, 41], [0, 2 ** 31 - 1, 3], [7, 3, 40],
                                 [-(2 ** 31), 0, 40]])
def test_offsets_that_are_none(bad, form):
    x, w, _, d = inputs([20, 20], 64, 72)
    at = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for out in (BF, F32):
        assert expert_ops.grouped_mm_forward(x, w, at, out_dtype=out, flags=form).isnan().all()
        assert expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=out, flags=form).isnan().all()
    x, w, at, _ = inputs([20, 20], 64, 72)
    check_forward(x, w, at, flags=form)  # the next call is none the worse
    big = at.long().clone()
    big[2] = 2 ** 32 + 40  # 40 in the low half
    assert expert_ops.grouped_mm_forward(x, w, big).isnan().all()
    assert torch.equal(expert_ops.grouped_mm_forward(x, w, at.long()), expert_ops.grouped_mm_forward(x, w, at))


def test_many_experts_and_none_of_the_rows():
    x, w, at, d = inputs([(7 * e) % 5 for e in range(1024)], 64, 40)
    check_forward(x, w, at)
    check_weight_grad(x, d, at, w)
    x, w, at, d = inputs([0, 0], 64, 40)
    assert expert_ops.grouped_mm_forward(x, w, at).shape == (0, 40)
    assert (check_weight_grad(x, d, at, w) == 0).all()
    x, w, at, d = inputs([0, 0], 64, 40, behind=7)
    assert (check_forward(x, w, at) == 0).all() and (check_weight_grad(x, d, at, w) == 0).all()


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
def test_sums_into_a_kept_gradient(form, transposed, dt):
    x, w, at, d = inputs([70, 0, 9], 136, 72, transposed)
    own = expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=F32)
    into = torch.full((3, 72, 136) if transposed else (3, 136, 72), 0.5, dtype=dt, device="cuda")
    into = into.transpose(1, 2) if transposed else into
    before = into.clone()
    got = expert_ops.grouped_mm_weight_grad(x, d, at, w, into=into, flags=form)
    assert got.data_ptr() == into.data_ptr() and got.stride() == into.stride()
    assert torch.equal(into, (before.float() + own).to(dt))
    assert torch.equal(into[1], before[1])


def test_strides_alignment_and_other_layouts():
    x, w, at, d = inputs([30, 11], 64, 72)
    ref, dw = expert_ops.grouped_mm_forward(x, w, at), expert_ops.grouped_mm_weight_grad(x, d, at, w)
    wide = torch.zeros(41, 100, dtype=BF, device="cuda")
    wide[:, 3:67] = x
    for rows in (wide[:, 3:67], x.t().contiguous().t(), torch.cat([x.flatten()[:1], x.flatten()])[1:].view(41, 64)):
        assert torch.equal(expert_ops.grouped_mm_forward(rows, w, at), ref)
        assert torch.equal(expert_ops.grouped_mm_weight_grad(rows, d, at, w), dw)
    for weight in (w.permute(1, 0, 2).contiguous().permute(1, 0, 2), torch.cat([w.flatten()[:1], w.flatten()])[1:].view(2, 64, 72),
                   w.transpose(1, 2).contiguous().transpose(1, 2)):
        assert torch.equal(expert_ops.grouped_mm_forward(x, weight, at), ref)
        assert torch.equal(expert_ops.grouped_mm_weight_grad(x, d, at, weight), dw)
    one = w[:1].expand(2, 64, 72)  # the experts share one matrix
    assert torch.equal(expert_ops.grouped_mm_forward(x, one, at)[:30], ref[:30])


def test_gradients_by_the_formula_and_by_differences():
    x, w, at, d = inputs([50, 0, 33], 72, 136, transposed=True, behind=4)
    x.requires_grad_(True)
    w = w.detach().requires_grad_(True)
    out = expert_ops.grouped_mm(x, w, at)
    out.backward(d)
    assert torch.equal(x.grad, check_forward(d, w.detach().transpose(1, 2), at))
    assert torch.equal(w.grad, check_weight_grad(x.detach(), d, at, w.detach()))
    assert (x.grad[-4:] == 0).all() and (w.grad[1] == 0).all()
    # out is linear in each: the difference over a step of bf16 numbers, 32-bit results
    g = torch.Generator(device="cuda").manual_seed(9)
    for t, other in ((x, lambda s: (s, w.detach())), (w, lambda s: (x.detach(), s))):
        step = torch.randint(-2, 3, t.shape, generator=g, device="cuda").to(BF)
        moved = expert_ops.grouped_mm_forward(*other(step), at, out_dtype=F32)
        by_difference, by_gradient = (moved * d).double().sum(), (t.grad.double() * step.double()).sum()
        # the gradient's rounding: 2^-8 of each element, random signs; 8 deviations of their sum
        tol = 8 * 2.0 ** -8 * (t.grad.double() * step.double()).square().sum().sqrt() + 1e-5 * moved.abs().sum()
        assert abs(by_difference - by_gradient) <= tol
    out = expert_ops.grouped_mm(x, w, at, out_dtype=F32)
    assert out.dtype == F32
    x.grad = w.grad = None
    out.sum().backward()  # an expanded gradient
    ones = torch.ones_like(d)
    assert torch.equal(x.grad, expert_ops.grouped_mm_forward(ones, w.detach().transpose(1, 2), at))
    only = expert_ops.grouped_mm(x.detach(), w, at)
    w.grad = None
    only.backward(d)
    assert w.grad is not None
    with pytest.raises(RuntimeError, match="differentiable once"):
        (gx,) = torch.autograd.grad((expert_ops.grouped_mm(x, w, at) * d).sum(), x, create_graph=True)
        gx.square().sum().backward()


def test_a_captured_step_replays_with_other_sizes():
    K, N, R = 136, 264, 400
    x, w, at, d = inputs([100, 0, 200, 90], K, N, behind=10)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        expert_ops.grouped_mm_backward(d, x, w, at)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = expert_ops.grouped_mm_forward(x, w, at)
        dx, dw = expert_ops.grouped_mm_backward(d, x, w, at)
    for sizes in ([0, 0, 0, 400], [1, 2, 3, 4], [400, 0, 0, 0], [0, 0, 0, 0], [133, 133, 133, 1]):
        x2, w2, at2, d2 = inputs(sizes, K, N, behind=R - sum(sizes), seed=3)
        for t, v in ((x, x2), (w, w2), (at, at2), (d, d2)):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expert_ops.grouped_mm_forward(x2, w2, at2))
        want = expert_ops.grouped_mm_backward(d2, x2, w2, at2)
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_calls_on_two_streams_at_once():
    cases = [inputs([90, 300, 1], 200, 136, seed=s) for s in range(2)]
    want = [expert_ops.grouped_mm_backward(d, x, w, at) for x, w, at, d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (x, w, at, d) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(expert_ops.grouped_mm_backward(d, x, w, at))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want[i]))


def test_refusals():
    x, w, at, d = inputs([3, 4], 64, 72)
    call = expert_ops.grouped_mm_forward
    for args in ((x[:, :32], w, at), (x[0], w, at), (x, w[0], at), (x, w, at[:2]), (x, w, at.float()), (x.cpu(), w, at),
                 (x, w, at.cpu())):
        with pytest.raises(ValueError):
            call(*args)
    with pytest.raises(ValueError):
        call(x, w, at, flags=3)
    for args in ((x.float(), w, at), (x, w.float(), at)):
        with pytest.raises(TypeError):
            call(*args)
    with pytest.raises(TypeError):
        call(x, w, at, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        expert_ops.grouped_mm_weight_grad(x, d[:, :8], at, w)
    with pytest.raises(ValueError):
        expert_ops.grouped_mm_weight_grad(x, d, at, w, into=torch.zeros(2, 64, 80, device="cuda")[:, :, :72])
    with pytest.raises(ValueError):
        expert_ops.grouped_mm_weight_grad(x, d, at, w, into=torch.zeros(2, 72, 64, device="cuda"))
    with pytest.raises(TypeError):
        expert_ops.grouped_mm_weight_grad(x, d, at, w, into=torch.zeros(2, 64, 72, device="cuda"), dtype=BF)


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
def test_a_sum_that_never_arrives_is_nan(form):
    """The failure path: the first CTA withholds its first accumulator, and its waits run out."""
    x, w, at, d = inputs([300, 5, 70], 136, 264)
    got = expert_ops.grouped_mm_forward(x, w, at, flags=form | _abi.MM_GROUPED_TEST_STALL)
    assert got[:128, :128].isnan().all()
    good = expert_ops.grouped_mm_forward(x, w, at, flags=form)
    assert torch.equal(torch.where(got.isnan(), good, got), good)
    got = expert_ops.grouped_mm_weight_grad(x, d, at, w, flags=form | _abi.MM_GROUPED_TEST_STALL)
    assert got[0, :128, :128].isnan().all()  # (the largest expert's is the first)
    check_forward(x, w, at, flags=form)
    check_weight_grad(x, d, at, w, flags=form)


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("sizes,K,N", [([1], 7168, 128), ([3], 2056, 264), ([0, 2, 0], 4096, 72), ([2], 4104, 1000)])
def test_few_tiles_of_long_sums(sizes, K, N, form):
    """Sums cut over k, with slices that a launch behind adds up."""
    for transposed in (False, True):
        for out in (BF, F32):
            x, w, at, _ = inputs(sizes, K, N, transposed, before=2, behind=3)
            got = check_forward(x, w, at, out_dtype=out, flags=form)
            assert (got[:2] == 0).all() and (got[-3:] == 0).all()
            assert torch.equal(got, expert_ops.grouped_mm_forward(x, w, at, out_dtype=out))
            at2 = at.clone()
            at2[-1] = x.shape[0] + 1
            assert expert_ops.grouped_mm_forward(x, w, at2, out_dtype=out, flags=form).isnan().all()
    stalled = expert_ops.grouped_mm_forward(x, w, at, flags=form | _abi.MM_GROUPED_TEST_STALL)
    assert stalled.isnan().any() and torch.equal(torch.where(stalled.isnan(), got.to(BF), stalled), got.to(BF))


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("sizes,K,N", [([9000], 136, 72), ([0, 5000, 33, 0, 4000, 1, 700], 264, 40), ([3001, 64, 2999], 64, 520),
                                       ([513] * 5 + [20000], 24, 24), ([1024, 1024, 1025], 72, 64)])
def test_experts_with_most_rows(sizes, K, N, form):
    """Sums over rows cut into parts, for the experts that have many."""
    for transposed in (False, True):
        x, w, at, d = inputs(sizes, K, N, transposed, before=1, behind=5)
        for out in (BF, F32):
            got = check_weight_grad(x, d, at, w, dtype=out, flags=form)
            assert torch.equal(got, expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=out))
            shape = (len(sizes), N, K) if transposed else (len(sizes), K, N)
            into = torch.full(shape, 0.5, dtype=out, device="cuda")
            into = into.transpose(1, 2) if transposed else into
            expert_ops.grouped_mm_weight_grad(x, d, at, w, into=into, flags=form)
            own = expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=F32)
            assert torch.equal(into, (0.5 + own).to(out))
        bad = at.clone()
        bad[-1] = x.shape[0] + 1
        assert expert_ops.grouped_mm_weight_grad(x, d, bad, w, flags=form).isnan().all()
    stalled = expert_ops.grouped_mm_weight_grad(x, d, at, w, flags=form | _abi.MM_GROUPED_TEST_STALL)
    assert stalled.isnan().any()


def test_long_sums_of_32_bits_keep_their_bits():
    """Runs of 512 terms, added up in 32 bits: 32 additions of a run each lose at most 2^-23 of the sum so
    far, always towards zero, so below 32 / 2 2^-23 = 2e-6 of a result that grows evenly, and the runs'
    sum next to nothing. All terms of one sign, where this bias shows most."""
    x, w, at, d = (t.abs() if t.is_floating_point() else t for t in inputs([9000, 70], 7168, 136))
    for form in (SINGLE, PAIRS):
        got = expert_ops.grouped_mm_forward(x, w, at, out_dtype=F32, flags=form).double()
        ref = torch.cat([x[a:b].double() @ w[e].double() for e, (a, b) in spans(at)])
        assert ((got - ref).norm() / ref.norm()) <= 2e-6
        got = expert_ops.grouped_mm_weight_grad(x[:, :264], d, at, w[:, :264], dtype=F32, flags=form).double()
        ref = torch.stack([x[a:b, :264].double().t() @ d[a:b].double() for _, (a, b) in spans(at)])
        assert ((got - ref).norm() / ref.norm()) <= 2e-6


@pytest.mark.parametrize("seed", range(24))
def test_random_sizes(seed):
    rng = random.Random(seed)
    E = rng.choice([1, 2, 3, 7, 16, 40, 200])
    K, N = (8 * rng.randint(1, rng.choice([8, 40, 150])) for _ in range(2))
    most = rng.choice([3, 40, 300, 1500]) if E < 40 else rng.choice([3, 40, 300])
    sizes = [0 if rng.random() < 0.2 else rng.randint(0, most) for _ in range(E)]
    if rng.random() < 0.3:
        sizes[rng.randrange(E)] += 4000
    before, behind = rng.choice([0, 0, 5]), rng.choice([0, 0, 1, 300])
    if before + sum(sizes) + behind == 0:
        behind = 1
    x, w, at, d = inputs(sizes, K, N, rng.random() < 0.5, before, behind, seed)
    form = rng.choice([SINGLE, PAIRS, 0])
    for out in (BF, F32):
        got = check_forward(x, w, at, out_dtype=out, flags=form)
        assert (got[:before] == 0).all() and (got[before + sum(sizes):] == 0).all()
        assert torch.equal(got, expert_ops.grouped_mm_forward(x, w, at, out_dtype=out))
        got = check_weight_grad(x, d, at, w, dtype=out, flags=form)
        assert torch.equal(got, expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=out))


def test_offsets_past_32_bits():
    """Results of more than 2^31 elements, and rows behind as many elements of inputs."""
    R, K, N = 300_001, 8, 7200
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(R, K, generator=g, device="cuda").to(BF)
    w = torch.randn(2, K, N, generator=g, device="cuda").to(BF)
    at = torch.tensor([0, 5, R], dtype=torch.int32, device="cuda")
    out = expert_ops.grouped_mm_forward(x, w, at)
    pick = torch.tensor([0, 4, 5, 150_000, 298_262, 298_263, R - 2, R - 1], device="cuda")
    ref = torch.stack([x[r].double() @ w[int(r >= 5)].double() for r in pick])
    close(out[pick], ref, torch.full_like(ref, 8 * 16.0), K)
    dx = expert_ops.grouped_mm_forward(out, w.transpose(1, 2), at)  # reads them again
    ref = torch.stack([out[r].double() @ w[int(r >= 5)].double().t() for r in pick])
    mag = torch.stack([out[r].double().abs() @ w[int(r >= 5)].double().abs().t() for r in pick])
    close(dx[pick], ref, mag, N)
    one = torch.zeros_like(x)
    one[R - 1] = 1.0  # the last row alone
    dw = expert_ops.grouped_mm_weight_grad(one, out, at, w)
    assert torch.equal(dw[1], out[R - 1].expand(K, N)) and (dw[0] == 0).all()


def test_forms_and_types_in_turn_without_a_pause():
    """Launches of one and of two CTAs a tile, of bf16 and 32-bit results, each of which takes tensor memory
    that the one before has held: the same bits every time."""
    x, w, at, d = inputs([300, 0, 65, 513], 264, 392, behind=3)
    calls = [lambda how=how: (expert_ops.grouped_mm_forward(x, w, at, **how),
                              expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=how["out_dtype"], flags=how["flags"]))
             for how in (dict(out_dtype=dt, flags=form) for dt in (BF, F32) for form in (PAIRS, SINGLE, 0))]
    want = [call() for call in calls]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(120):
        c = (5 * i + i // 6) % len(calls)
        for got, ref in zip(calls[c](), want[c]):
            wrong += (got != ref).sum()
    assert int(wrong) == 0


@pytest.mark.parametrize("form", [SINGLE, PAIRS, 0])
@pytest.mark.parametrize("R,K,N", [(1, 2048, 8), (1, 2400, 8), (1, 2048, 1), (1, 7168, 8), (2, 4096, 8), (1, 2304, 16)])
def test_sums_in_parts_of_few_results(R, K, N, form):
    """Slices that are smaller than the smallest workspace there is otherwise (a token through an adapter of
    rank 8), also as the gradient of the rows of an N -> K product."""
    for transposed in (False, True):
        for out in (BF, F32):
            x, w, at, d = inputs([R], K, N, transposed)
            check_forward(x, w, at, out_dtype=out, flags=form)
    x, w, at, d = inputs([R], N, K)
    dx, _ = expert_ops.grouped_mm_backward(d, x, w, at, flags=form)
    assert torch.equal(dx, check_forward(d, w.transpose(1, 2), at, flags=form))


def test_a_workspace_of_256_bytes_means_none():
    """As the header says: for the library's own sizes, called as a C program calls it."""
    import ctypes
    lib = _abi._lib()
    for R, K, N in ((1, 2048, 8), (1, 2400, 8), (1, 64, 8), (1, 4096, 72), (3, 2056, 264)):
        x, w, at, _ = inputs([R], K, N)
        d = _abi.mm_grouped_desc(R, K, N, 1, 0, 0, 0)
        n = lib.mm_grouped_mm_workspace_size(ctypes.addressof(d))
        ws = None if n == 256 else torch.empty(n, dtype=torch.uint8, device="cuda")
        out = torch.empty(R, N, dtype=BF, device="cuda")
        _abi.check(lib.mm_grouped_mm(ctypes.addressof(d), x.data_ptr(), w.data_ptr(), at.data_ptr(), out.data_ptr(),
                                     None if ws is None else ws.data_ptr(), n if ws is not None else 0,
                                     torch.cuda.current_stream().cuda_stream), "mm_grouped_mm")
        assert torch.equal(out, expert_ops.grouped_mm_forward(x, w, at))


STALL = _abi.MM_GROUPED_TEST_STALL


def stalled_calls():
    x, w, at, d = inputs([300, 5, 70], 136, 264)
    long = inputs([2], 4104, 264)
    into = lambda dt: torch.zeros(w.shape, dtype=dt, device="cuda")
    return {"rows": lambda dt, **how: expert_ops.grouped_mm_forward(x, w, at, out_dtype=dt, **how),
            "parts": lambda dt, **how: expert_ops.grouped_mm_forward(*long[:3], out_dtype=dt, **how),
            "weights": lambda dt, **how: expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=dt, **how),
            "into": lambda dt, **how: expert_ops.grouped_mm_weight_grad(x, d, at, w, into=into(dt), **how)}


@pytest.mark.parametrize("form", [SINGLE, PAIRS])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("name", ["rows", "parts", "weights", "into"])
def test_a_wait_that_runs_out_is_told(name, dt, form):
    call = stalled_calls()[name]
    status = expert_ops.grouped_status()
    good = call(dt, flags=form, status=status)
    expert_ops.check_grouped_status(status)
    got = call(dt, flags=form | STALL, status=status)
    with pytest.raises(_abi.MMError, match="MM_ERR_TIMEOUT") as error:
        expert_ops.check_grouped_status(status)
    assert error.value.status == _abi.MM_ERR_TIMEOUT
    code, where = status.tolist()
    assert where >> 8 in (0, 1) and 1 <= where & 255 <= 6  # (the first CTA's, or its pair's other one)
    assert got.isnan().any() and torch.equal(torch.where(got.isnan(), good, got), good)
    assert torch.equal(call(dt, flags=form, status=status), good)  # the next call is none the worse,
    assert status.tolist() == [code, where]                       # and what happened stays told
    status.zero_()
    call(dt, flags=form, status=status)
    expert_ops.check_grouped_status(status)


def test_a_loop_ends_at_the_first_wait_that_ran_out():
    call, status, done = stalled_calls()["weights"], expert_ops.grouped_status(), 0
    with pytest.raises(_abi.MMError):
        for i in range(10):
            call(F32, flags=STALL if i == 3 else 0, status=status)
            expert_ops.check_grouped_status(status)
            done += 1
    assert done == 3


def test_a_status_of_all_calls_together():
    x, w, at, d = inputs([50, 0, 33], 72, 136, transposed=True, behind=4)
    status = expert_ops.grouped_status()
    want = expert_ops.grouped_mm_backward(d, x, w, at)
    x.requires_grad_(True)
    w = w.detach().requires_grad_(True)
    expert_ops.grouped_mm(x, w, at, status=status).backward(d)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
    x, w, at, d = inputs([3, 0, 40, 1], 33, 70)  # padded
    for a, b in zip(expert_ops.grouped_mm_backward(d, x, w, at, status=status), expert_ops.grouped_mm_backward(d, x, w, at)):
        assert torch.equal(a, b)
    expert_ops.check_grouped_status(status)
    for bad in (status[:1], status.long(), status.cpu(), torch.zeros(4, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError, match="status"):
            expert_ops.grouped_mm_forward(x, w, at, status=bad)
        with pytest.raises(ValueError, match="status"):
            expert_ops.grouped_mm_weight_grad(x, d, at, w, status=bad)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("K,N", [(136, 72), (33, 70)])
@pytest.mark.parametrize("transposed", [False, True])
def test_sums_into_a_kept_gradient_off_a_16_byte_boundary(transposed, K, N, dt):
    """Of any widths; what lies around it stays as it was."""
    x, w, at, d = inputs([70, 0, 9], K, N, transposed)
    own = expert_ops.grouped_mm_weight_grad(x, d, at, w, dtype=F32)
    for start in (1, 3):
        flat = torch.full((start + w.numel() + 5,), 0.5, dtype=dt, device="cuda")
        into = flat[start:start + w.numel()].view(3, *((N, K) if transposed else (K, N)))
        into = into.transpose(1, 2) if transposed else into
        got = expert_ops.grouped_mm_weight_grad(x, d, at, w, into=into)
        assert into.data_ptr() % 16 and got.data_ptr() == into.data_ptr()
        assert torch.equal(into, (0.5 + own).to(dt))
        assert (flat[:start] == 0.5).all() and (flat[-5:] == 0.5).all()
