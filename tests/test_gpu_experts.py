"""The order of a selection, the rows in that order and their weighted sums, against their definitions.

The order and the dispatched rows are equal bit for bit. A sum of K terms in 32 bits is off by at most
K 2^-23 of the sum of magnitudes, and its rounding by half a step; a dot product of H terms (partial
sums of a thread, then a tree) by at most (H / 32 + 16) 2^-24 of the magnitudes' sum, for H <= 7168 less
than 2^-16 of it."""
import pytest
import torch

from moe_ffn_expert_gb300 import block_ops, expert_ops
from moe_ffn_expert_gb300.torch_api import hyper_mega_moe

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def selection(T, K, E, seed=0, dropped=0, skew=False):
    g = torch.Generator().manual_seed(seed)
    if skew:
        ids = torch.randint(0, E, (T, K), generator=g) ** 2 // max(1, E)
    else:
        ids = torch.randint(0, E, (T, K), generator=g)
    if dropped:
        ids.view(-1)[torch.rand(T * K, generator=g) < dropped] = -1
    return ids.to(torch.int32)


def order(ids, E):
    """offsets, row_of_slot, slot_of_row by lists."""
    flat = ids.flatten().tolist()
    slots = sorted((e, s) for s, e in enumerate(flat) if 0 <= e < E)
    offsets = [0] * (E + 1)
    for e, _ in slots:
        offsets[e + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    row, slot = [-1] * len(flat), [-1] * len(flat)
    for r, (_, s) in enumerate(slots):
        row[s], slot[r] = r, s
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    return t(offsets), t(row).view(ids.shape), t(slot)


@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (1, 8, 128), (3, 2, 1024), (64, 8, 128), (255, 8, 60), (256, 8, 64),
                                   (257, 8, 2), (4001, 16, 1024), (9000, 6, 7), (40000, 8, 128)])
@pytest.mark.parametrize("dropped", [0, 0.2, 1.0])
def test_table(T, K, E, dropped):
    ids = selection(T, K, E, dropped=dropped, skew=T % 2 == 1)
    table = expert_ops.expert_table(ids.cuda(), E)
    for got, want in zip(table, order(ids, E)):
        assert torch.equal(got, want)
    assert table[3:] == (T, K, E)


def test_table_of_any_ids():
    ids = torch.tensor([[5, -1, 2 ** 31 - 1], [-(2 ** 31), 4, 0], [5, 5, 5]], dtype=torch.int32)
    wide = ids.long()
    wide[1, 2] = 2 ** 32  # 0 in the low half
    wide[2, 0] = -(2 ** 32) + 5
    for t in (ids, wide):
        for got, want in zip(expert_ops.expert_table(t.cuda(), 5), order(t, 5)):
            assert torch.equal(got, want)
    strided = torch.stack([ids, ids], 2)[:, :, 0].cuda()
    assert torch.equal(expert_ops.expert_table(strided, 6).row_of_slot, order(ids, 6)[1])
    none = expert_ops.expert_table(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 3)
    assert none.offsets.tolist() == [0, 0, 0, 0] and none.row_of_slot.shape == (0, 4)


def test_table_of_one_expert_many_blocks():
    """More blocks than add up each other's counts (a launch between), all slots in one expert."""
    T, K, E = 70000, 8, 33
    ids = torch.full((T, K), 32, dtype=torch.int32, device="cuda")
    table = expert_ops.expert_table(ids, E)
    every = torch.arange(T * K, dtype=torch.int32, device="cuda")
    assert torch.equal(table.row_of_slot.flatten(), every) and torch.equal(table.slot_of_row, every)
    assert table.offsets.tolist() == [0] * 33 + [T * K]
    ids = torch.randint(-1, E, (T, K), dtype=torch.int32, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    table = expert_ops.expert_table(ids, E)
    flat = ids.flatten().long()
    key = torch.where(flat < 0, E, flat)
    slots = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    assert torch.equal(table.slot_of_row[:n].long(), slots[:n]) and (table.slot_of_row[n:] == -1).all()
    assert torch.equal(table.row_of_slot.flatten()[slots[:n]], every[:n])
    assert (table.row_of_slot.flatten()[flat < 0] == -1).all()


def rows_case(T, K, E, H, dt, dropped=0.0, seed=0):
    ids = selection(T, K, E, seed, dropped).cuda()
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    table = expert_ops.expert_table(ids, E)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return table, randn(T, H).to(dt), randn(T * K, H).to(dt), randn(T, K)


ROWS = [(1, 1, 1, 1), (1, 8, 16, 64), (5, 2, 4, 7), (33, 6, 60, 2047), (64, 8, 128, 2048), (17, 16, 32, 136),
        (3, 9, 9, 7168), (100, 3, 5, 4098)]


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("dropped", [0, 0.3, 1.0])
@pytest.mark.parametrize("T,K,E,H", ROWS)
def test_dispatch(T, K, E, H, dt, dropped):
    table, x, _, _ = rows_case(T, K, E, H, dt, dropped)
    got = expert_ops.dispatch_forward(x, table)
    slot = table.slot_of_row.long()
    want = torch.where((slot >= 0)[:, None], x[slot.clamp_min(0) // K], torch.zeros_like(x[:1]))
    assert got.dtype == dt and torch.equal(got, want)


def combined(rows, table, weights):
    """y and the sum of its terms' magnitudes in 64 bits."""
    row = table.row_of_slot.long()
    o = rows.double()[row.clamp_min(0)] * (row >= 0)[:, :, None]
    o = torch.where((row >= 0)[:, :, None], o, torch.zeros_like(o))
    o = o if weights is None else o * weights.double()[:, :, None]
    return o.sum(1), o.abs().sum(1)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("dropped", [0, 0.3, 1.0])
@pytest.mark.parametrize("T,K,E,H", ROWS)
def test_combine(T, K, E, H, dt, dropped):
    table, _, rows, w = rows_case(T, K, E, H, dt, dropped)
    for weights in (w, None):
        got = expert_ops.combine_forward(rows, table, weights)
        ref, mag = combined(rows, table, weights)
        assert got.dtype == dt
        assert ((got.double() - ref).abs() <= torch.finfo(dt).eps / 2 * ref.abs() + K * 2.0 ** -23 * mag).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("dropped", [0, 0.3, 1.0])
@pytest.mark.parametrize("T,K,E,H", ROWS)
def test_combine_backward(T, K, E, H, dt, dropped):
    table, dy, rows, w = rows_case(T, K, E, H, dt, dropped)
    slot, row = table.slot_of_row.long(), table.row_of_slot.long()
    for weights in (w, None):
        d_rows, d_w = expert_ops.combine_backward(dy, rows, table, weights)
        at = slot.clamp_min(0)
        want = dy[at // K].float() * (1 if weights is None else weights.flatten()[at][:, None])
        want = torch.where((slot >= 0)[:, None], want, torch.zeros_like(want)).to(dt)
        assert torch.equal(d_rows, want)  # one product, one rounding
        terms = dy.double()[:, None, :] * rows.double()[row.clamp_min(0)] * (row >= 0)[:, :, None]
        assert ((d_w.double() - terms.sum(2)).abs() <= 2.0 ** -16 * terms.abs().sum(2)).all()
        again, none = expert_ops.combine_backward(dy, None, table, weights, weight_grad=False)
        assert torch.equal(again, d_rows) and none is None


def test_rows_nobody_uses_have_no_part():
    table, dy, rows, w = rows_case(20, 4, 6, 72, F32, dropped=0.4)
    n = int(table.offsets[-1])
    assert 0 < n < 80
    y, d = expert_ops.combine_forward(rows, table, w), expert_ops.combine_backward(dy, rows, table, w)
    rows2, w2 = rows.clone(), w.clone()
    rows2[n:] = float("nan")
    w2[table.row_of_slot < 0] = float("nan")
    assert torch.equal(expert_ops.combine_forward(rows2, table, w2), y)
    again = expert_ops.combine_backward(dy, rows2, table, w2)
    assert torch.equal(again[0], d[0]) and torch.equal(again[1], d[1])
    assert (d[0][n:] == 0).all() and (d[1][table.row_of_slot < 0] == 0).all()


def test_strides_and_alignment():
    table, x, rows, w = rows_case(20, 4, 6, 72, BF)
    want = (expert_ops.dispatch_forward(x, table), expert_ops.combine_forward(rows, table, w),
            *expert_ops.combine_backward(x, rows, table, w))

    def other(t):
        if t.dim() != 2:
            return [t]
        wide = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device="cuda")
        wide[:, 1:-2] = t
        off = torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)
        return [wide[:, 1:-2], t.t().contiguous().t(), off]

    for x2, rows2, w2 in zip(other(x), other(rows), other(w)):
        got = (expert_ops.dispatch_forward(x2, table), expert_ops.combine_forward(rows2, table, w2),
               *expert_ops.combine_backward(x2, rows2, table, w2))
        for a, b in zip(got, want):
            # (the dot products of unaligned rows are summed in another order)
            assert torch.equal(a, b) or (a.dtype == F32 and torch.allclose(a, b, rtol=0, atol=2.0 ** -16 * 72 * 4))


def test_offsets_past_32_bits():
    T, K, H = 40000, 8, 7168  # 2.3e9 elements of dispatched rows
    ids = torch.randint(0, 16, (T, K), dtype=torch.int32, device="cuda")
    table = expert_ops.expert_table(ids, 16)
    x = torch.arange(T, device="cuda", dtype=F32)[:, None].expand(T, H).to(BF).contiguous()
    rows = expert_ops.dispatch_forward(x, table)
    pick = torch.tensor([0, 1, 160000, T * K - 2, T * K - 1], device="cuda")
    assert torch.equal(rows[pick], x[table.slot_of_row[pick].long() // K])
    y = expert_ops.combine_forward(rows, table, torch.full((T, K), 0.125, device="cuda"))
    assert torch.equal(y, x)
    d_rows, d_w = expert_ops.combine_backward(x, rows, table, torch.ones(T, K, device="cuda"))
    assert torch.equal(d_rows[pick], rows[pick])
    assert torch.allclose(d_w[-1].double(), x[-1].double().square().sum().expand(K), rtol=1e-4)


def test_gradients_by_the_formula_and_by_differences():
    table, x, rows, w = rows_case(13, 3, 5, 40, F32, dropped=0.2)
    for t in (x, rows, w):
        t.requires_grad_(True)
    g = torch.Generator(device="cuda").manual_seed(5)
    d_rows = torch.randn(39, 40, generator=g, device="cuda")
    expert_ops.expert_dispatch(x, table).backward(d_rows)
    assert torch.equal(x.grad, expert_ops.combine_forward(d_rows, table))
    dy = torch.randn(13, 40, generator=g, device="cuda")
    expert_ops.expert_combine(rows, table, w).backward(dy)
    want = expert_ops.combine_backward(dy, rows.detach(), table, w.detach())
    assert torch.equal(rows.grad, want[0]) and torch.equal(w.grad, want[1])
    # all three are linear: the difference over a step is the step's own result
    s = torch.randn(13, 40, generator=g, device="cuda")
    by_difference = (expert_ops.dispatch_forward(s, table).double() * d_rows).sum()
    assert torch.isclose(by_difference, (x.grad.double() * s).sum(), rtol=1e-5)
    s = torch.randn(39, 40, generator=g, device="cuda")
    by_difference = (expert_ops.combine_forward(s, table, w.detach()).double() * dy).sum()
    assert torch.isclose(by_difference, (rows.grad.double() * s).sum(), rtol=1e-5)
    s = torch.randn(13, 3, generator=g, device="cuda")
    by_difference = (expert_ops.combine_forward(rows.detach(), table, s).double() * dy).sum()
    assert torch.isclose(by_difference, (w.grad.double() * s).sum(), rtol=1e-5)
    half = w.detach().to(BF).requires_grad_(True)
    expert_ops.expert_combine(rows.detach(), table, half).sum().backward()
    assert half.grad.dtype == BF
    for out, at in ((lambda: expert_ops.expert_dispatch(x, table).square(), x),
                    (lambda: expert_ops.expert_combine(rows, table, w).square(), w)):
        (first,) = torch.autograd.grad(out().sum(), at, create_graph=True)
        with pytest.raises(RuntimeError, match="differentiable once"):
            first.square().sum().backward()


def test_a_captured_run_of_all_replays():
    T, K, E, H = 70, 4, 12, 72
    ids, x, w, wt = (selection(T, K, E).cuda(), torch.randn(T, H, device="cuda").to(BF), torch.rand(T, K, device="cuda"),
                     torch.randn(E, H, 64, device="cuda").to(BF))

    def step(ids, x, w, wt):
        table = expert_ops.expert_table(ids, E)
        rows = expert_ops.dispatch_forward(x, table)
        out = expert_ops.grouped_mm_forward(rows, wt, table.offsets)
        return (*table[:3], rows, out, expert_ops.combine_forward(out, table, w))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(ids, x, w, wt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step(ids, x, w, wt)
    for seed in (1, 2):
        ids.copy_(selection(T, K, E, seed, dropped=0.1))
        x.copy_(torch.randn(T, H, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(ids, x, w, wt)):
            assert torch.equal(a, b)


def test_the_parts_together_are_the_layer():
    """SwiGLU experts from the parts, forward and backward, against the fused layer and 64 bits. bf16
    rounding between the parts: each of rows, gate|up, h and the experts' outputs and their gradients
    is off by up to 2^-8 of its value with random signs, well below 2 % of a result's norm."""
    T, H, I, E, K = 300, 256, 128, 8, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, up, down = randn(T, H).to(BF), (randn(E, H, 2 * I) / 16).to(BF), (randn(E, I, H) / 11).to(BF)
    ids, weights, *_ = block_ops.moe_router(randn(T, E), K)
    dy = randn(T, H).to(BF)
    leaves = [t.requires_grad_(True) for t in (x, up, down, weights.detach())]

    def parts(x, up, down, w):
        table = expert_ops.expert_table(ids, E)
        gate, lin = expert_ops.grouped_mm(expert_ops.expert_dispatch(x, table), up, table.offsets).chunk(2, 1)
        h = torch.nn.functional.silu(gate) * lin
        return expert_ops.expert_combine(expert_ops.grouped_mm(h, down, table.offsets), table, w)

    def plain(x, up, down, w):
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for e in range(E):
            t, k = (ids == e).nonzero(as_tuple=True)
            a, b = (x[t] @ up[e]).chunk(2, 1)
            y = y.index_add(0, t, w[t, k][:, None] * ((a * torch.sigmoid(a) * b) @ down[e]))
        return y

    y = parts(*leaves)
    got = (y, *torch.autograd.grad(y, leaves, dy))
    z = hyper_mega_moe(leaves[0], ids, leaves[3], leaves[1], leaves[2])
    fused = (z, *torch.autograd.grad(z, (leaves[0], leaves[1], leaves[2], leaves[3]), dy))
    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    r = plain(*wide)
    ref = (r, *torch.autograd.grad(r, wide, dy.double()))
    for a, b, c in zip(got, fused, ref):
        assert (a.double() - c).norm() <= 0.02 * c.norm()
        assert (a.double() - b.double()).norm() <= 0.02 * c.norm()


def test_refusals():
    table, x, rows, w = rows_case(6, 2, 4, 16, BF)
    for bad in (torch.zeros(4, device="cuda", dtype=torch.int32), torch.zeros(4, 2, device="cuda"),
                torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 17, device="cuda", dtype=torch.int32)):
        with pytest.raises(ValueError):
            expert_ops.expert_table(bad, 4)
    for E in (0, 1025):
        with pytest.raises(ValueError):
            expert_ops.expert_table(table.row_of_slot, E)
    for call in (lambda: expert_ops.dispatch_forward(x[:5], table), lambda: expert_ops.combine_forward(rows[:5], table, w),
                 lambda: expert_ops.combine_forward(rows, table, w[:, :1]), lambda: expert_ops.combine_forward(rows, table, w.double()),
                 lambda: expert_ops.combine_backward(x, None, table, w), lambda: expert_ops.dispatch_forward(x.cpu(), table),
                 lambda: expert_ops.dispatch_forward(x, table._replace(offsets=table.offsets[:3])),
                 lambda: expert_ops.dispatch_forward(x, table._replace(offsets=table.offsets.cpu())),
                 lambda: expert_ops.dispatch_forward(x, table._replace(row_of_slot=table.row_of_slot.long())),
                 lambda: expert_ops.combine_backward(x[:, :8], rows, table, w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: expert_ops.dispatch_forward(x.half(), table), lambda: expert_ops.combine_backward(x.float(), rows, table, w),
                 lambda: expert_ops.expert_combine(rows, table, table.row_of_slot)):
        with pytest.raises(TypeError):
            call()


def test_tables_of_any_strides():
    """After a call with a contiguous table of the same shapes: strided and transposed copies of it give
    the same results, an expanded one those of the numbers that it shows."""
    T, K, H = 40, 4, 32
    table, x, rows, w = rows_case(T, K, 8, H, BF)

    def calls(t):
        return (expert_ops.dispatch_forward(x, t), expert_ops.combine_forward(rows, t, w),
                *expert_ops.combine_backward(x, rows, t, w))

    want = calls(table)
    two = lambda t: torch.stack([t, t + 1000], -1).flatten(-2)[..., ::2]
    for other in (table._replace(row_of_slot=two(table.row_of_slot), offsets=two(table.offsets)),
                  table._replace(row_of_slot=table.row_of_slot.t().contiguous().t())):
        assert not other.row_of_slot.is_contiguous() and torch.equal(other.row_of_slot, table.row_of_slot)
        for got, ref in zip(calls(other), want):
            assert torch.equal(got, ref)
    shown = table._replace(row_of_slot=table.row_of_slot[:1].expand(T, K))
    assert torch.equal(expert_ops.combine_forward(rows, shown, w),
                       expert_ops.combine_forward(rows, shown._replace(row_of_slot=shown.row_of_slot.contiguous()), w))
