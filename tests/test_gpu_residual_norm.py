"""residual_norm against its definition in 64 bits, forward and backward.

Tolerances, from the arithmetic: every value is a sum of a few products in 32 bits whose row
statistics come from sums of at most 16384 terms in a tree (relative error below 2e-6 of the sum of
magnitudes); 1e-5 times the sum of the magnitudes of a value's terms bounds that with room for the
reciprocal root. A bf16 output adds half a unit in the last place, 2^-9 of the value (2^-8 is
allowed: the rounding may sit on the other side of a 32-bit error)."""
import pytest
import torch

from moe_ffn_expert_gb300 import _abi, block_ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def make(T, H, st=BF, bt=BF, pt=BF, groups=1, post=True, pre=True, branch=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")

    i = dict(residual=(2 * r(T, H)).to(st), branch=(0.7 * r(T, H)).to(bt) if branch else None,
             post_weight=(0.5 + 0.2 * r(H)).to(pt) if post and branch else None,
             pre_weight=(1 + 0.2 * r(H)).to(pt) if pre else None,
             gate=(0.5 + 0.5 * r(groups, H)).to(pt) if groups and branch else None)
    up = dict(d_out=(0.1 * r(T, H)).to(st), d_normed=(0.1 * r(T, H)).to(bt) if pre else None)
    return i, up


def oracle_forward(i, scale, eps):
    """(r', n) and the sums of their terms' magnitudes."""
    x = i["residual"].double()
    T, H = x.shape
    y = torch.zeros_like(x) if i["branch"] is None else i["branch"].double()
    if i["post_weight"] is not None:
        y = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * i["post_weight"].double()
    if i["gate"] is not None:
        y = y * i["gate"].double().repeat_interleave(T // i["gate"].shape[0], 0)
    out, mag = scale * x + y, (scale * x).abs() + y.abs()
    if i["pre_weight"] is None:
        return out, None, mag, None
    inv = (out.square().mean(1, keepdim=True) + eps).rsqrt() * i["pre_weight"].double()
    return out, out * inv, mag, mag * inv.abs()


def oracle_backward(i, up, scale, eps):
    """Gradients at residual = r' and the sums of their terms' magnitudes."""
    x, u = i["residual"].double(), up["d_out"].double()
    T, H = x.shape
    res = {}
    d, dm = u, u.abs()
    if i["pre_weight"] is not None:
        v, w = up["d_normed"].double(), i["pre_weight"].double()
        q = (x.square().mean(1, keepdim=True) + eps).rsqrt()
        res["pre"] = ((v * x * q).sum(0), (v * x * q).abs().sum(0))
        c = q ** 3 / H
        d = d + q * w * v - c * x * (w * v * x).sum(1, keepdim=True)
        dm = dm + (q * w * v).abs() + (c * x).abs() * (w * v * x).abs().sum(1, keepdim=True)
    res["residual"] = (scale * d, abs(scale) * dm)
    if i["branch"] is None:
        return res
    f = i["branch"].double()
    p, e = f, torch.ones_like(f)
    if i["post_weight"] is not None:
        s = (f.square().mean(1, keepdim=True) + eps).rsqrt()
        e = i["post_weight"].double().expand_as(f)
        p = f * s * e
    g = torch.ones_like(f)
    if i["gate"] is not None:
        G = i["gate"].shape[0]
        g = i["gate"].double().repeat_interleave(T // G, 0)
        res["gate"] = ((d * p).view(G, -1, H).sum(1), (dm * p.abs()).view(G, -1, H).sum(1))
    if i["post_weight"] is not None:
        res["post"] = ((g * d * f * s).sum(0), (g * dm * f * s).abs().sum(0))
        df = s * e * g * d - f * s ** 3 / H * (e * g * d * f).sum(1, keepdim=True)
        m = (s * e * g).abs() * dm + (f * s ** 3 / H).abs() * ((e * g * f).abs() * dm).sum(1, keepdim=True)
        res["branch"] = (df, m)
    else:
        res["branch"] = (g * d, g.abs() * dm)
    return res


def close(name, got, ref, mag):
    tol = 1e-5 * mag + (2.0 ** -8 * ref.abs() if got.dtype == BF else 0)
    err = (got.double() - ref).abs()
    assert got.shape == ref.shape
    assert bool((err <= tol + 1e-30).all()), (name, float((err - tol).max()), float(err.max()))


def run_both(i, up, scale=0.75, eps=1e-6):
    kw = dict(post_weight=i["post_weight"], pre_weight=i["pre_weight"], gate=i["gate"],
              residual_scale=scale, eps=eps)
    ndt = up["d_normed"].dtype if up["d_normed"] is not None else None
    out, n = block_ops.residual_norm_forward(i["residual"], i["branch"], normed_dtype=ndt, **kw)
    grads = block_ops.residual_norm_backward(i["residual"], i["branch"], up["d_out"],
                                             up["d_normed"], **kw)
    return (out, n), dict(zip(("residual", "branch", "post", "pre", "gate"), grads))


def check(i, up, scale=0.75, eps=1e-6):
    (out, n), grads = run_both(i, up, scale, eps)
    ro, rn, mo, mn = oracle_forward(i, scale, eps)
    close("residual_out", out, ro, mo)
    assert (n is None) == (rn is None)
    if n is not None:
        close("normed", n, rn, mn)
    ref = oracle_backward(i, up, scale, eps)
    for k, got in grads.items():
        assert (got is None) == (k not in ref), k
        if got is not None:
            close("d_" + k, got, *ref[k])


TYPES = [(BF, BF, BF), (BF, BF, F32), (F32, BF, F32), (F32, BF, BF), (F32, F32, F32), (F32, F32, BF)]


@pytest.mark.parametrize("st,bt,pt", TYPES)
@pytest.mark.parametrize("T,H,groups", [(1, 2048, 1), (37, 512, 37), (96, 264, 3), (50, 1001, 5), (3, 1, 1)])
def test_types_and_sizes(T, H, groups, st, bt, pt):
    check(*make(T, H, st, bt, pt, groups))


@pytest.mark.parametrize("H", [2, 7, 8, 31, 33, 256, 1023, 2047, 4096, 4097, 7168, 8192, 8200, 9001, 16384])
@pytest.mark.parametrize("st", [BF, F32])
def test_widths(H, st):
    check(*make(5, H, st, st, st))


@pytest.mark.parametrize("T,groups", [(700, 1), (700, 7), (700, 350), (700, 700), (1300, 2), (2048, 4)])
def test_many_tokens_and_gate_groups(T, groups):
    check(*make(T, 136, groups=groups))
    check(*make(T, 135, F32, F32, F32, groups=groups))


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("groups", [0, 1])
@pytest.mark.parametrize("H", [640, 77])
def test_parts_left_out(post, pre, groups, H):
    check(*make(40, H, post=post, pre=pre, groups=groups))


@pytest.mark.parametrize("st,bt", [(BF, BF), (F32, BF), (F32, F32)])
def test_norm_before_the_first_block(st, bt):
    check(*make(33, 512, st, bt, st, branch=False), scale=1.0)


def test_only_one_upstream_gradient():
    i, up = make(64, 512)
    kw = dict(post_weight=i["post_weight"], pre_weight=i["pre_weight"], gate=i["gate"])
    got = block_ops.residual_norm_backward(i["residual"], i["branch"], None, up["d_normed"], **kw)
    ref = oracle_backward(i, dict(up, d_out=torch.zeros_like(up["d_out"])), 1.0, 1e-6)
    for g, k in zip(got, ("residual", "branch", "post", "pre", "gate")):
        close(k, g, *ref[k])


def test_strided_and_unaligned_inputs():
    i, up = make(48, 256)
    ref = run_both(i, up)
    wide = {k: None if t is None else torch.stack([t, t], -1)[..., 0] for k, t in {**i, **up}.items()}
    odd = {}
    for k, t in {**i, **up}.items():  # contiguous, two bytes off a 16-byte boundary
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        odd[k] = buf[1:].view(t.shape).copy_(t)
    for other in (wide, odd):
        got = run_both({k: other[k] for k in i}, {k: other[k] for k in up})
        for a, b in zip(got[0], ref[0]):
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-4)
        for k in ref[1]:
            assert torch.allclose(got[1][k].float(), ref[1][k].float(), rtol=2 ** -7, atol=1e-4), k


def test_repeat_gives_the_same_bits():
    i, up = make(3000, 1024, groups=4)
    a, b = run_both(i, up), run_both(i, up)
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(torch.equal(a[1][k], b[1][k]) for k in a[1])


def test_a_bad_row_stays_in_its_row():
    i, up = make(20, 512, groups=0)
    clean = run_both(i, up)
    for bad in (float("nan"), float("inf")):
        j = dict(i, residual=i["residual"].clone(), branch=i["branch"].clone())
        j["residual"][7, 3] = bad
        j["branch"][11, 500] = bad
        got = run_both(j, up)
        rows = [t for t in range(20) if t not in (7, 11)]
        for a, b in zip((*got[0], got[1]["residual"], got[1]["branch"]),
                        (*clean[0], clean[1]["residual"], clean[1]["branch"])):
            assert torch.equal(a[rows], b[rows])
        assert not torch.isfinite(got[0][1][7]).all()


def test_without_the_norm_before_the_residual_is_not_used():
    """No pre_weight: the gradients do not depend on r', not even on an infinite one."""
    i, up = make(6, 128, pre=False)
    a = run_both(i, up)[1]
    i["residual"][2, 5] = float("inf")
    b = run_both(i, up)[1]
    assert all(torch.equal(a[k], b[k]) for k in a if a[k] is not None)


def test_zero_rows_and_eps():
    i, up = make(4, 96, F32, F32, F32)
    i["residual"].zero_()
    i["branch"].zero_()
    (out, n), g = run_both(i, up, eps=1e-5)
    assert not out.any() and not n.any()
    assert all(torch.isfinite(t).all() for t in g.values())
    check(i, up, eps=1e-5)


@pytest.mark.parametrize("groups", [0, 1])
def test_no_tokens(groups):
    i, up = make(0, 64, groups=groups)
    (out, n), g = run_both(i, up)
    assert out.shape == n.shape == (0, 64) and g["residual"].shape == (0, 64)
    assert not g["post"].any() and not g["pre"].any()
    assert g["gate"] is None if groups == 0 else not g["gate"].any()


def test_gradient_against_differences():
    """(L(x + h d) - L(x - h d)) / 2h along random directions; L is in 64 bits over 32-bit outputs:
    its rounding noise is ~1e-7 sqrt(elements) / h and its third-order term ~h^2: 1 % of the
    directional derivative's own size (the norm of the gradient) is far above both at h = 1e-2."""
    i, up = make(9, 200, F32, F32, F32, groups=3)
    kw = dict(residual_scale=0.75)
    leaves = {k: t.clone().requires_grad_(True) for k, t in i.items()}
    co, cn = up["d_out"].double(), up["d_normed"].double()

    def loss(ins):
        out, n = block_ops.residual_norm_forward(ins["residual"], ins["branch"], **kw, **{
            k: ins[k] for k in ("post_weight", "pre_weight", "gate")})
        return float((out.double() * co).sum() + (n.double() * cn).sum())

    out, n = block_ops.residual_norm(leaves["residual"], leaves["branch"], **kw, **{
        k: leaves[k] for k in ("post_weight", "pre_weight", "gate")})
    torch.autograd.backward([out, n], [up["d_out"], up["d_normed"]])
    g = torch.Generator(device="cuda").manual_seed(5)
    for k, t in i.items():
        for _ in range(3):
            d = torch.randn(t.shape, generator=g, device="cuda")
            h = 1e-2
            num = (loss({**i, k: t + h * d}) - loss({**i, k: t - h * d})) / (2 * h)
            grad = leaves[k].grad
            assert abs(num - float((grad * d).sum())) <= 1e-2 * float(grad.norm()) + 1e-4, k


def test_in_place_through_the_c_abi():
    i, up = make(500, 512)
    (out, n), g = run_both(i, up, scale=1.0)
    d = _abi.mm_norm_desc(500, 512, 1, 0, 0, 0, 1.0, 1e-6)
    import ctypes
    lib, at = _abi._lib(), ctypes.addressof(d)
    st = torch.cuda.current_stream().cuda_stream
    p = {k: t.data_ptr() for k, t in {**i, **up}.items()}
    dr, r2, n2 = up["d_out"].clone(), i["residual"].clone(), torch.empty_like(n)
    nbytes = lib.mm_residual_norm_workspace_size(at)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    df, dpost, dpre, dg = (torch.empty_like(i[k]) for k in ("branch", "post_weight", "pre_weight", "gate"))
    assert lib.mm_residual_norm_forward(at, r2.data_ptr(), p["branch"], p["post_weight"], p["pre_weight"],
                                        p["gate"], r2.data_ptr(), n2.data_ptr(), st) == 0
    assert torch.equal(r2, out) and torch.equal(n2, n)
    assert lib.mm_residual_norm_backward(
        at, p["residual"], p["branch"], p["post_weight"], p["pre_weight"], p["gate"], dr.data_ptr(),
        p["d_normed"], dr.data_ptr(), df.data_ptr(), dpost.data_ptr(), dpre.data_ptr(), dg.data_ptr(),
        ws.data_ptr(), nbytes, st) == 0
    assert torch.equal(dr, g["residual"]) and torch.equal(df, g["branch"]) and torch.equal(dg, g["gate"])


def test_side_stream_and_graph():
    i, up = make(256, 512)
    ref = run_both(i, up)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_both(i, up)
    s.synchronize()
    assert all(torch.equal(got[1][k], ref[1][k]) for k in ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run_both(i, up)
    i["branch"].mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    ref = run_both(i, up)
    assert all(torch.equal(cap[1][k], ref[1][k]) for k in ref[1]) and torch.equal(cap[0][1], ref[0][1])


def test_refusals():
    i, _ = make(8, 64)
    r, f = i["residual"], i["branch"]
    fwd = block_ops.residual_norm_forward
    for bad, err in ((lambda: fwd(r.cpu(), f.cpu()), ValueError),
                     (lambda: fwd(r.half(), f.half()), TypeError),
                     (lambda: fwd(r, f.float()), TypeError),
                     (lambda: fwd(r, f[:, :32]), ValueError),
                     (lambda: fwd(r, None, gate=i["gate"]), ValueError),
                     (lambda: fwd(r, f, gate=i["gate"].expand(3, 64)), ValueError),
                     (lambda: fwd(r, f, pre_weight=i["pre_weight"][:32]), ValueError),
                     (lambda: fwd(r, f, pre_weight=i["pre_weight"], post_weight=i["post_weight"].float()), TypeError),
                     (lambda: fwd(r[0], f[0]), ValueError),
                     (lambda: fwd(r, f, eps=-1.0), _abi.MMError),
                     (lambda: fwd(torch.zeros(1, 16385, device="cuda"), None), _abi.MMError),
                     (lambda: block_ops.residual_norm_backward(r, f, r, None, pre_weight=i["pre_weight"]), ValueError)):
        with pytest.raises(err):
            bad()


# Rows by bulk copies take over the forward above two waves of blocks (a few hundred to a few
# thousand tokens, by width), and the backward wherever a few rows fit in shared memory.

@pytest.mark.parametrize("T,H,groups", [
    (1000, 2048, 1), (1000, 2048, 4), (999, 2048, 333), (1001, 2048, 1001), (310, 7168, 1),
    (310, 7680, 2), (310, 7688, 1), (2500, 512, 2500), (2500, 512, 250), (2501, 200, 0), (3000, 64, 1),
    # odd: rows start off 16-byte boundaries, the last one ends off one
    (1000, 2047, 1), (999, 2047, 333), (310, 3839, 310), (620, 3839, 2), (310, 3841, 1),
    (1601, 1023, 1601), (1100, 1999, 0), (2501, 77, 1), (2501, 65, 1), (2501, 63, 1)])
@pytest.mark.parametrize("st,bt,pt", [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32)])
def test_many_rows(T, H, groups, st, bt, pt):
    check(*make(T, H, st, bt, pt, groups))


@pytest.mark.parametrize("post,pre,groups", [(False, True, 1), (True, False, 1), (False, False, 1), (True, True, 0),
                                             (False, True, 0), (False, False, 1250), (True, False, 1250),
                                             (False, True, 1250)])
@pytest.mark.parametrize("H", [1024, 1021])
def test_parts_left_out_of_many_rows(post, pre, groups, H):
    check(*make(2500, H, post=post, pre=pre, groups=groups))


@pytest.mark.parametrize("H", [1024, 1021])
def test_many_rows_before_the_first_block(H):
    check(*make(3300, H, F32, BF, F32, branch=False), scale=1.0)


@pytest.mark.parametrize("H", [1024, 1021])
def test_many_rows_in_place_through_the_c_abi(H):
    import ctypes
    T = 3300
    i, up = make(T, H)
    (out, n), g = run_both(i, up, scale=1.0)
    d = _abi.mm_norm_desc(T, H, 1, 0, 0, 0, 1.0, 1e-6)
    lib, at, st = _abi._lib(), ctypes.addressof(d), torch.cuda.current_stream().cuda_stream
    r2, f2, dr = i["residual"].clone(), i["branch"].clone(), up["d_out"].clone()
    w = [i[k].data_ptr() for k in ("post_weight", "pre_weight", "gate")]
    assert lib.mm_residual_norm_forward(at, r2.data_ptr(), f2.data_ptr(), *w, r2.data_ptr(),
                                        f2.data_ptr(), st) == 0
    assert torch.equal(r2, out) and torch.equal(f2, n)
    nbytes = lib.mm_residual_norm_workspace_size(at)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    sums = [torch.empty_like(i[k]) for k in ("post_weight", "pre_weight", "gate")]
    df = torch.empty_like(f2)
    assert lib.mm_residual_norm_backward(
        at, i["residual"].data_ptr(), i["branch"].data_ptr(), *w, dr.data_ptr(), up["d_normed"].data_ptr(),
        dr.data_ptr(), df.data_ptr(), *[s.data_ptr() for s in sums], ws.data_ptr(), nbytes, st) == 0
    assert torch.equal(dr, g["residual"]) and torch.equal(df, g["branch"])
    assert torch.equal(sums[0], g["post"]) and torch.equal(sums[2], g["gate"])


def test_bad_rows_among_many_stay_in_their_rows():
    i, up = make(2500, 1021, groups=0)
    clean = run_both(i, up)
    j = dict(i, residual=i["residual"].clone(), branch=i["branch"].clone())
    j["residual"][1700, 1020] = float("nan")
    j["branch"][2499, 0] = float("inf")
    got = run_both(j, up)
    rows = [t for t in range(2500) if t not in (1700, 2499)]
    for a, b in zip((*got[0], got[1]["residual"], got[1]["branch"]),
                    (*clean[0], clean[1]["residual"], clean[1]["branch"])):
        assert torch.equal(a[rows], b[rows])


@pytest.mark.parametrize("H", [7168, 2047])
def test_more_than_2_31_elements(H):
    """The last rows of a tensor whose offsets pass 32 bits, against the oracle for those rows."""
    T = (2 ** 31 + 4096) // H + 8
    small, up = make(16, H)
    def tall(t):
        return t.repeat((T + 15) // 16, 1)[:T].contiguous()
    i = dict(small, residual=tall(small["residual"]), branch=tall(small["branch"]))
    u = {k: tall(t) for k, t in up.items()}
    (out, n), g = run_both(i, u)
    at = [t % 16 for t in range(T - 5, T)]
    part = dict(small, residual=small["residual"][at], branch=small["branch"][at])
    ro, rn, mo, mn = oracle_forward(part, 0.75, 1e-6)
    close("residual_out", out[-5:], ro, mo)
    close("normed", n[-5:], rn, mn)
    ref = oracle_backward(part, {k: t[at] for k, t in up.items()}, 0.75, 1e-6)
    close("d_residual", g["residual"][-5:], *ref["residual"])
    close("d_branch", g["branch"][-5:], *ref["branch"])


def test_scale_as_a_tensor_is_read_at_every_call():
    i, _ = make(4, 64)
    s = torch.tensor(1.0)
    a = block_ops.residual_norm_forward(i["residual"], None, residual_scale=s)[0]
    s.fill_(2.0)
    b = block_ops.residual_norm_forward(i["residual"], None, residual_scale=s)[0]
    assert torch.equal(a * 2, b)


@pytest.mark.parametrize("T,H,groups", [(400, 7168, 1), (400, 7680, 4), (330, 6144, 330)])
def test_rows_of_which_one_fits_in_shared_memory(T, H, groups):
    check(*make(T, H, F32, F32, F32, groups))


@pytest.mark.parametrize("T,H,groups", [
    # rows of bulk copies in blocks of 2 to 15 working warps, and of 2 to 15 with odd rows
    (3300, 1024, 0), (2500, 2048, 1), (1300, 5120, 1), (1300, 7680, 4), (2500, 1024, 2500),
    (3300, 513, 1), (2501, 1021, 0), (1300, 2047, 1), (1300, 3839, 2)])
def test_post_norm_alone_over_many_rows_repeats(T, H, groups):
    """After the last block there is one sum per row, whose buffer the next row's sum must not
    overwrite while a slower warp still reads it. An overwritten partial sum scales part of a row by
    another row's norm: rows of very different sizes next to each other make that visible."""
    i, up = make(T, H, pre=False, groups=groups)
    i["branch"].mul_(torch.exp2(4.0 * (torch.arange(T, device="cuda") % 3))[:, None].to(BF))
    kw = dict(post_weight=i["post_weight"], gate=i["gate"], residual_scale=0.75)
    ref, _, mag, _ = oracle_forward(i, 0.75, 1e-6)
    first, none = block_ops.residual_norm_forward(i["residual"], i["branch"], **kw)
    assert none is None
    close("residual_out", first, ref, mag)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        differ += (block_ops.residual_norm_forward(i["residual"], i["branch"], **kw)[0] != first).sum()
    assert int(differ) == 0


@pytest.mark.parametrize("H", [1024, 1021, 8192])
@pytest.mark.parametrize("groups", [0, 1, 2500])
@pytest.mark.parametrize("pre", [True, False])
def test_without_a_post_weight_the_branch_value_is_not_used(H, groups, pre):
    """d_branch = gate * d does not depend on the branch, not even on an infinite one, whether rows come
    by bulk copies or straight from memory."""
    T = 2500
    i, up = make(T, H, post=False, pre=pre, groups=groups)
    kw = dict(pre_weight=i["pre_weight"], gate=i["gate"])
    clean = block_ops.residual_norm_backward(i["residual"], i["branch"], up["d_out"], up["d_normed"], **kw)
    f = i["branch"].clone()
    f[3], f[2000, 5], f[T - 1, H - 1] = float("inf"), float("-inf"), float("nan")
    got = block_ops.residual_norm_backward(i["residual"], f, up["d_out"], up["d_normed"], **kw)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("H", [512, 511, 8192])
@pytest.mark.parametrize("stream,branch", [(2.0 ** 46, 1.0), (1.0, 2.0 ** 46), (2.0 ** 54, 2.0 ** 50),
                                           (2.0 ** -46, 1.0), (2.0 ** -46, 2.0 ** -50)])
def test_gradients_of_very_large_and_small_rows(H, stream, branch):
    """Rows whose 1 / rms has a cube beyond 32 bits; without an eps, which would hide small ones. The
    upstream gradient of r' is left out: it would cover what comes through the norm of a large row."""
    i, up = make(700, H, F32, F32, F32)
    i["residual"].mul_(stream)
    i["branch"].mul_(branch)
    kw = dict(post_weight=i["post_weight"], pre_weight=i["pre_weight"], gate=i["gate"], eps=0.0)
    got = block_ops.residual_norm_backward(i["residual"], i["branch"], None, up["d_normed"], **kw)
    ref = oracle_backward(i, dict(up, d_out=torch.zeros_like(up["d_out"])), 1.0, 0.0)
    for g, k in zip(got, ("residual", "branch", "post", "pre", "gate")):
        want, mag = ref[k]
        assert ((g.double() - want).abs() <= 1e-5 * mag + 1e-37).all(), k


@pytest.mark.parametrize("T,H,groups", [(2500, 1024, 1), (2500, 1021, 0), (1300, 7168, 4), (2500, 1024, 2500)])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_rows_that_never_come_are_nan(T, H, groups, post, pre):
    """One block's loads stop after its first row: its other rows and all parameter gradients that they
    belong to are NaN, every other row is what it is otherwise, and the next call is as ever."""
    i, up = make(T, H, groups=groups, post=post, pre=pre)
    ref = run_both(i, up)
    lib = _abi._lib()
    lib.mm_residual_norm_test_stall(1)
    try:
        got = run_both(i, up)
        torch.cuda.synchronize()
    finally:
        lib.mm_residual_norm_test_stall(0)

    def rows(a, b):
        lost = torch.isnan(a).all(1)
        assert 1 <= int(lost.sum()) < T // 2
        assert torch.equal(a[~lost], b[~lost])
        return lost

    lost = rows(got[0][0], ref[0][0])
    if pre:
        assert torch.equal(rows(got[0][1], ref[0][1]), lost)
    lost = rows(got[1]["residual"], ref[1]["residual"])
    assert torch.equal(rows(got[1]["branch"], ref[1]["branch"]), lost)
    for k in ("post", "pre"):
        assert got[1][k] is None or torch.isnan(got[1][k]).all()
    if groups:
        gates = torch.isnan(got[1]["gate"]).all(1)
        assert gates.any() and torch.equal(gates, lost.view(groups, -1).any(1))
        assert torch.equal(got[1]["gate"][~gates], ref[1]["gate"][~gates])
    again = run_both(i, up)
    assert all(torch.equal(again[1][k], ref[1][k]) for k in ref[1] if ref[1][k] is not None)
    assert torch.equal(again[0][0], ref[0][0])


def test_a_normed_dtype_that_is_not_the_branch_s_is_refused():
    i, _ = make(8, 64, F32, BF, F32)
    for op in (block_ops.residual_norm, block_ops.residual_norm_forward):
        with pytest.raises(TypeError):
            op(i["residual"], i["branch"], pre_weight=i["pre_weight"], normed_dtype=F32)
        assert op(i["residual"], i["branch"], pre_weight=i["pre_weight"], normed_dtype=BF)[1].dtype == BF
        assert op(i["residual"], None, pre_weight=i["pre_weight"], normed_dtype=F32)[1].dtype == F32
