"""The few-token MoE layer against its definition in 64 bits, and the quantiser of its weights.

Tolerance of y: the products w h are rounded to bf16 once (2^-9 of each, random), y once more
(2^-9 of itself). With terms c_i = (w h)_i Wd_i, the first error is a sum of independent terms of
standard deviation at most 2^-9 |c_i| / sqrt(3): six standard deviations are 3.5 * 2^-9 times the
root of the sum of c_i^2. 32-bit sums add less than 1e-5 of the sum of |c_i|."""
import ctypes
import math

import pytest
import torch

from moe_ffn_expert_gb300 import _abi, block_ops

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def matrix(g, n, R, C, fp8):
    w = (torch.randn(n, R, C, generator=g, device="cuda") / math.sqrt(R)).to(BF)
    return block_ops.quantize_expert_weights(w) if fp8 else (w, None)


def values(q, scale):
    """[n, R, C] in 64 bits."""
    w = q.float().double()
    if scale is None:
        return w
    r = torch.arange(w.shape[1], device="cuda") // 128
    c = torch.arange(w.shape[2], device="cuda") // 128
    return w * scale.double()[:, r][:, :, c]


def make(T, H, I, E, K, fp8=False, shared=0, ids=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    up, us = matrix(g, E, H, 2 * I, fp8)
    down, ds = matrix(g, E, I, H, fp8)
    m = dict(x=torch.randn(T, H, generator=g, device="cuda").to(BF), up=up, us=us, down=down, ds=ds, K=K,
             router=(1.5 * torch.randn(E, H, generator=g, device="cuda") / math.sqrt(H)).to(BF), shared=None)
    if shared:
        su, sus = matrix(g, 1, H, 2 * shared, fp8)
        sd, sds = matrix(g, 1, shared, H, fp8)
        m["shared"] = (su[0], sd[0], None if sus is None else sus[0], None if sds is None else sds[0])
    if ids is None:
        ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:K] for _ in range(T)]) \
            if T else torch.empty(0, K, device="cuda")
    m["ids"] = ids.to(torch.int32)
    m["w"] = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    return m


def decoder(m, route=False, **kw):
    return block_ops.MoEDecoder(m["up"], m["down"], k=m["K"], up_scale=m["us"], down_scale=m["ds"],
                                router_weight=m["router"] if route else None, shared=m["shared"],
                                max_tokens=kw.pop("max_tokens", max(1, m["x"].shape[0])), **kw)


def ffn(x, up, down):
    """o and the sums of its terms' squares and magnitudes (of h Wd)."""
    gate, lin = (x @ up).chunk(2, -1)
    h = gate * torch.sigmoid(gate) * lin
    return h @ down, h.square() @ down.square(), h.abs() @ down.abs()


def reference(m, ids=None, w=None):
    x, ids, w = m["x"].double(), (m["ids"] if ids is None else ids).long(), (m["w"] if w is None else w).double()
    y, sq, ab = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    for e in ids.unique().tolist():
        t, k = (ids == e).nonzero(as_tuple=True)
        up = values(m["up"][e:e + 1].view(m["up"].dtype), None if m["us"] is None else m["us"][e:e + 1])[0]
        down = values(m["down"][e:e + 1], None if m["ds"] is None else m["ds"][e:e + 1])[0]
        o, s, a = ffn(x[t], up, down)
        c = w[t, k][:, None]
        y.index_add_(0, t, c * o)
        sq.index_add_(0, t, c * c * s)
        ab.index_add_(0, t, c.abs() * a)
    if m["shared"] is not None:
        su, sd, sus, sds = m["shared"]
        o, s, a = ffn(x, values(su[None], None if sus is None else sus[None])[0],
                      values(sd[None], None if sds is None else sds[None])[0])
        y, sq, ab = y + o, sq + s, ab + a
    return y, 2.0 ** -8 * y.abs() + 3.5 * 2.0 ** -9 * sq.sqrt() + 1e-5 * ab


def close(y, ref):
    want, tol = ref
    err = (y.double() - want).abs()
    assert torch.isfinite(y).all()
    assert (err <= tol + 1e-30).all(), (float((err / (tol + 1e-30)).max()), float(err.max()))


def check(m, **kw):
    d = decoder(m, **kw)
    y = d(m["x"], m["ids"], m["w"])
    assert d.status() == _abi.MM_OK
    close(y, reference(m))
    return y


SIZES = [(1, 64, 64, 1, 1), (1, 2048, 768, 16, 8), (3, 512, 128, 4, 2), (7, 256, 64, 40, 5), (8, 1024, 512, 16, 4),
         (33, 512, 256, 32, 6), (64, 512, 128, 8, 2), (64, 256, 64, 130, 16), (17, 2048, 768, 32, 6)]


@pytest.mark.parametrize("T,H,I,E,K", SIZES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shared", [0, 96])
def test_sizes(T, H, I, E, K, fp8, shared):
    check(make(T, H, I, E, K, fp8, shared))


@pytest.mark.parametrize("H,I", [(8, 8), (16, 24), (72, 40), (136, 1032), (200, 120), (520, 72), (1000, 56), (4104, 8)])
def test_odd_widths_bf16(H, I):
    check(make(5, H, I, 6, 3, shared=I + 8))


@pytest.mark.parametrize("H,I", [(16, 16), (144, 48), (208, 112), (528, 80), (1008, 336), (4112, 16), (4096, 4240)])
def test_odd_widths_e4m3(H, I):
    check(make(5, H, I, 6, 3, True, shared=I + 16))


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 31, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_one_expert_takes_all(T, fp8):
    """Every token on the same expert (several chunks of rows), the others unused."""
    ids = torch.full((T, 1), 3, device="cuda")
    check(make(T, 256, 192, 5, 1, fp8, ids=ids))


def test_an_expert_twice_in_a_row():
    ids = torch.tensor([[1, 1, 2], [0, 0, 0], [2, 1, 2]], device="cuda")
    check(make(3, 256, 128, 3, 3, ids=ids))


def test_split_of_long_inner_sizes():
    check(make(1, 128, 4096, 2, 1))            # few column tiles: I is cut into parts
    check(make(1, 128, 4096, 2, 1, True, shared=2048))


def test_weights_of_any_size_and_sign():
    m = make(6, 256, 128, 8, 4)
    m["w"] = torch.randn(6, 4, device="cuda") * 10
    m["w"][2] = 0
    check(m)
    y = decoder(m)(m["x"], m["ids"], m["w"])
    assert not y[2].any()


@pytest.mark.parametrize("E,K", [(8, 2), (60, 4), (128, 8), (256, 8), (500, 10), (1024, 16)])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_routing(E, K, score, normalize):
    T, H = 19, 136
    m = make(T, H, 32, E, K)
    d = decoder(m, route=True, score=score, normalize=normalize, scale=1.5)
    y, ids, w = d.with_routing(m["x"])
    assert d.status() == _abi.MM_OK
    z = m["x"].double() @ m["router"].double().t()
    top = torch.sort(z, 1, descending=True).values
    for t in range(T):  # 32-bit logits may swap experts whose 64-bit logits are this close
        assert len(set(ids[t].tolist())) == K
        assert (z[t, ids[t].long()] - top[t, :K]).abs().max() < 1e-5
    at = torch.gather(z, 1, ids.long())
    if score == "sigmoid":
        ref = torch.sigmoid(at)
        ref = ref / ref.sum(1, keepdim=True) if normalize else ref
    else:
        ref = torch.softmax(at, 1) if normalize else torch.exp(at - torch.logsumexp(z, 1)[:, None])
    assert ((w.double() - 1.5 * ref).abs() <= 2e-5 * ref).all()
    close(y, reference(m, ids, w))
    assert torch.equal(d(m["x"]), y)


def test_routing_with_bias_and_32_bit_router():
    m = make(10, 256, 64, 40, 4)
    bias = torch.randn(40, device="cuda")
    d = block_ops.MoEDecoder(m["up"], m["down"], k=4, router_weight=m["router"].float() * 1.001, router_bias=bias)
    y, ids, w = d.with_routing(m["x"])
    z = m["x"].double() @ (m["router"].float() * 1.001).double().t()
    top = torch.sort(z + bias.double(), 1, descending=True).values[:, :4]
    assert (torch.gather(z + bias.double(), 1, ids.long()) - top).abs().max() < 1e-5
    ref = torch.softmax(torch.gather(z, 1, ids.long()), 1)
    assert ((w.double() - ref).abs() <= 2e-5 * ref).all()
    close(y, reference(m, ids, w))


def test_agrees_with_the_router_and_the_layer():
    """router_forward's selection and the fused layer's output on the same weights."""
    from moe_ffn_expert_gb300.torch_api import hyper_mega_moe
    m = make(40, 512, 256, 16, 4)
    d = decoder(m, route=True)
    y, ids, w = d.with_routing(m["x"])
    ids2, w2, _, _ = block_ops.router_forward(m["x"].float() @ m["router"].float().t(), 4)
    assert torch.equal(ids, ids2) and torch.allclose(w, w2, rtol=1e-4)
    with torch.no_grad():
        full = hyper_mega_moe(m["x"], ids, w, m["up"], m["down"])
    assert torch.allclose(y.float(), full.float(), rtol=2e-2, atol=2e-2)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_bad_token_stays_in_its_row(fp8):
    m = make(24, 256, 128, 4, 2, fp8, shared=64)
    d = decoder(m)
    clean = d(m["x"], m["ids"], m["w"])
    x = m["x"].clone()
    x[5, 17], x[11, 200] = float("nan"), float("inf")
    y = d(x, m["ids"], m["w"])
    rows = [t for t in range(24) if t not in (5, 11)]
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[5]).all() and not torch.isfinite(y[11]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_experts_that_are_not_selected_are_not_read(fp8):
    """NaN weights of unselected experts change nothing, and those of a selected one reach only the
    tokens that selected it."""
    m = make(12, 200 + 8 * (not fp8), 144, 6, 2, fp8)
    if fp8:
        m = make(12, 208, 144, 6, 2, True)
    m["ids"] = (m["ids"] % 4).to(torch.int32)
    clean = decoder(m)(m["x"], m["ids"], m["w"])
    for name in ("up", "down"):
        m[name] = m[name].clone()
        raw = m[name].view(torch.uint8) if fp8 else m[name]
        raw[4:] = 0x7F if fp8 else float("nan")
    assert torch.equal(decoder(m)(m["x"], m["ids"], m["w"]), clean)
    raw = m["down"].view(torch.uint8) if fp8 else m["down"]
    raw[1] = 0x7F if fp8 else float("nan")
    y = decoder(m)(m["x"], m["ids"], m["w"])
    hit = (m["ids"] == 1).any(1)
    assert torch.isnan(y[hit]).all() and torch.equal(y[~hit], clean[~hit])


def test_stale_shared_memory_and_workspace():
    """Narrow problems after wide ones full of infinities, in the same workspace."""
    big = make(8, 512, 256, 4, 2)
    d = decoder(big)
    big["x"].fill_(float("inf"))
    d(big["x"], big["ids"], big["w"])
    small = make(3, 72, 40, 4, 2)
    ds = decoder(small)
    ds._ws = d._ws  # larger than needed, dirty
    ds._ws.fill_(0xFF)
    close(ds(small["x"], small["ids"], small["w"]), reference(small))


def test_repeat_streams_and_graphs():
    m = make(9, 1024, 512, 16, 4, shared=128)
    d = decoder(m, route=True)
    y = d(m["x"])
    for _ in range(50):
        assert torch.equal(d(m["x"]), y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z = d(m["x"])
    s.synchronize()
    assert torch.equal(z, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = d(m["x"])
    m["x"].copy_(m["x"].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, d(m["x"])) and torch.equal(out, y.flip(0))


def test_two_decoders_on_two_streams():
    ms = [make(16, 1024, 512, 16, 4, seed=i) for i in range(2)]
    ds = [decoder(m) for m in ms]
    ref = [d(m["x"], m["ids"], m["w"]) for d, m in zip(ds, ms)]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(ds[i](ms[i]["x"], ms[i]["ids"], ms[i]["w"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert ds[i].status() == _abi.MM_OK and all(torch.equal(o, ref[i]) for o in outs[i])


def test_bad_expert_ids_are_reported():
    m = make(4, 128, 64, 8, 2)
    d = decoder(m)
    y = d(m["x"], m["ids"], m["w"])
    for bad in (8, -1, 2 ** 31 - 1):
        ids = m["ids"].clone()
        ids[2, 1] = bad
        d(m["x"], ids, m["w"])
        assert d.status() == _abi.MM_ERR_BAD_EXPERT_ID
    assert torch.equal(d(m["x"], m["ids"], m["w"]), y) and d.status() == _abi.MM_OK


def test_no_tokens_and_strides():
    m = make(0, 128, 64, 8, 2)
    assert decoder(m)(m["x"], m["ids"], m["w"]).shape == (0, 128)
    m = make(6, 128, 64, 8, 2)
    d = decoder(m)
    y = d(m["x"], m["ids"], m["w"])
    wide = torch.stack([m["x"], m["x"]], -1)[..., 0]
    assert torch.equal(d(wide, m["ids"].long(), m["w"].double()), y)
    assert torch.equal(d(m["x"][:4], m["ids"][:4], m["w"][:4]), y[:4])


def test_quantizer():
    g = torch.Generator(device="cuda").manual_seed(2)
    for n, R, C in ((1, 1, 8), (2, 128, 128), (3, 300, 264), (1, 1000, 2048)):
        w = (torch.randn(n, R, C, generator=g, device="cuda") * torch.exp(3 * torch.randn(n, R, 1, generator=g, device="cuda"))).to(BF)
        if R == 300:
            w[1, 128:256, :128] = 0
        q, s = block_ops.quantize_expert_weights(w)
        br, bc = -(-R // 128), -(-C // 128)
        pad = torch.nn.functional.pad(w.float(), (0, bc * 128 - C, 0, br * 128 - R)).view(n, br, 128, bc, 128)
        amax = pad.abs().amax((2, 4))
        want = torch.where(amax > 0, (amax.double() / 448.0).float(), torch.ones_like(amax))
        assert torch.equal(s, want)
        ref = (pad / want[:, :, None, :, None]).view(n, br * 128, bc * 128)[:, :R, :C].to(F8)
        assert torch.equal(q.view(torch.uint8), ref.view(torch.uint8))
    w = torch.ones(1, 256, 128, device="cuda", dtype=BF)
    w[0, 3, 3], w[0, 200, 0] = float("inf"), 2.0
    _, s = block_ops.quantize_expert_weights(w)
    assert torch.isnan(s[0, 0, 0]) and s[0, 1, 0] == 2.0 / 448.0


def test_refusals():
    m = make(4, 128, 64, 8, 2)
    D = block_ops.MoEDecoder
    up, down = m["up"], m["down"]
    d = decoder(m)
    q, s = block_ops.quantize_expert_weights(up)
    for bad, err in ((lambda: D(up.cpu(), down.cpu(), k=2), ValueError), (lambda: D(up.float(), down.float(), k=2), TypeError),
                     (lambda: D(up, down[:, :32], k=2), ValueError), (lambda: D(up, down, k=9), ValueError),
                     (lambda: D(up, down, k=2, up_scale=s), ValueError), (lambda: D(q, q, k=2), ValueError),
                     (lambda: D(up, down, k=2, max_tokens=65), ValueError),
                     (lambda: D(up, down, k=2, router_weight=m["router"][:4]), ValueError),
                     (lambda: D(up, down, k=2, router_bias=torch.zeros(8, device="cuda")), ValueError),
                     (lambda: D(up, down, k=2, shared=(up[0],)), ValueError),
                     (lambda: d(m["x"]), ValueError), (lambda: d(m["x"].float(), m["ids"], m["w"]), ValueError),
                     (lambda: d(m["x"], m["ids"][:, :1], m["w"]), ValueError),
                     (lambda: d(m["x"], m["ids"].float(), m["w"]), TypeError),
                     (lambda: d(torch.zeros(5, 128, device="cuda", dtype=BF), m["ids"], m["w"]), ValueError),
                     (lambda: decoder(m, route=True)(m["x"], m["ids"], m["w"]), ValueError)):
        with pytest.raises(err):
            bad()


@pytest.mark.parametrize("T", [15, 17, 18, 47, 49])
@pytest.mark.parametrize("fp8", [False, True])
def test_chunks_of_rows_begin_and_end(T, fp8):
    ids = torch.full((T, 1), 2, device="cuda")
    check(make(T, 256, 192, 4, 1, fp8, shared=64, ids=ids))


@pytest.mark.parametrize("T", [1, 11, 12, 13, 14, 31, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_routing_at_every_number_of_tokens(T, fp8, score, normalize):
    """Selected by the experts' kernel itself, or from 13 tokens on by a launch before it: what a
    decoder does with its own selection is what one without a router does with the same."""
    m = make(T, 272, 64, 48, 6, fp8, shared=32)
    y, ids, w = decoder(m, route=True, score=score, normalize=normalize, max_tokens=64).with_routing(m["x"])
    z = m["x"].float() @ m["router"].float().t()
    ids2, w2, _, _ = block_ops.router_forward(z, 6, score=score, normalize=normalize)
    assert torch.equal(ids, ids2) and torch.allclose(w, w2, rtol=1e-4)
    assert torch.equal(y, decoder(m, max_tokens=64)(m["x"], ids, w))
    close(y, reference(m, ids, w))


@pytest.mark.parametrize("fp8", [False, True])
def test_experts_whose_offsets_pass_32_bits(fp8):
    """Only the last experts hold numbers; the ones before are not read."""
    T, H, I, E, K = 3, 4096, 1024, 300, 2
    m = make(T, H, I, 2, K, fp8)
    dt = m["up"].dtype
    big = dict(m, up=torch.empty(E, H, 2 * I, dtype=dt, device="cuda"), down=torch.empty(E, I, H, dtype=dt, device="cuda"))
    for k in ("up", "down"):
        big[k][E - 2:] = m[k]
    if fp8:
        for k in ("us", "ds"):
            big[k] = torch.full((E, *m[k].shape[1:]), float("nan"), device="cuda")
            big[k][E - 2:] = m[k]
    assert big["up"].numel() > 2 ** 31
    y = decoder(m)(m["x"], m["ids"], m["w"])
    got = decoder(big)(m["x"], m["ids"] + (E - 2), m["w"])
    assert torch.equal(got, y)
    close(y, reference(m))


def test_ids_of_another_device_are_refused():
    m = make(2, 64, 32, 4, 2)
    d = decoder(m)
    with pytest.raises(ValueError):
        d(m["x"], m["ids"].cpu(), m["w"])
    with pytest.raises(ValueError):
        d(m["x"], m["ids"], m["w"].cpu())


@pytest.mark.parametrize("H,I,fp8", [(1016, 496, True), (1000, 32, True), (8, 16, True), (7160, 64, True), (120, 48, True),
                                     (1001, 40, False), (3, 8, False), (515, 512, False)])
@pytest.mark.parametrize("T,shared", [(1, 0), (21, 48)])
def test_widths_that_are_padded(H, I, fp8, T, shared):
    m = make(T, H, I, 16, 4, fp8, shared=shared)
    y = check(m)
    assert y.shape == (T, H) and y.is_contiguous()
    y, ids, w = decoder(m, route=True).with_routing(m["x"])
    close(y, reference(m, ids, w))


@pytest.mark.parametrize("fp8", [False, True])
def test_two_decoders_on_streams_of_different_priority(fp8):
    """A grid of higher priority takes SMs that free up while the other is partly dispatched: what a
    running CTA waits for must never belong to one that has no SM yet."""
    ms = [make(T, 1024, 512, 16, 4, fp8, seed=T) for T in (16, 40)]
    ds = [decoder(m) for m in ms]
    ref = [d(m["x"], m["ids"], m["w"]) for d, m in zip(ds, ms)]
    streams = [torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(40):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(ds[i](ms[i]["x"], ms[i]["ids"], ms[i]["w"]))
    torch.cuda.synchronize()
    for i in range(2):
        assert ds[i].status() == _abi.MM_OK and all(torch.equal(o, ref[i]) for o in outs[i])


def test_64_bit_ids_out_of_range_are_reported():
    """Also those whose low 32 bits are an expert's number."""
    m = make(4, 128, 64, 8, 2)
    d = decoder(m)
    y = d(m["x"], m["ids"].long(), m["w"])
    assert d.status() == _abi.MM_OK
    for bad in (2 ** 32 + 3, -2 ** 32, 8, -1):
        ids = m["ids"].long()
        ids[2, 1] = bad
        d(m["x"], ids, m["w"])
        assert d.status() == _abi.MM_ERR_BAD_EXPERT_ID, bad
    assert torch.equal(d(m["x"], m["ids"].long(), m["w"]), y)


@pytest.mark.parametrize("H,fp8", [(1000, True), (515, False), (512, False), (512, True)])
@pytest.mark.parametrize("strided", [False, True])
def test_updates_of_the_weights_take_effect(H, fp8, strided):
    """Whether the decoder reads the given weights themselves or copies of them (an H that is padded,
    non-contiguous tensors)."""
    def spread(t):  # the same values, non-contiguous
        raw = t.view(torch.uint8) if t.dtype == F8 else t
        return torch.stack([raw, raw], -1)[..., 0].view(t.dtype) if t.dtype != F8 else \
            raw.transpose(-1, -2).contiguous().transpose(-1, -2).view(t.dtype)

    m = make(9, H, 64, 8, 2, fp8, shared=32)
    new = make(9, H, 64, 8, 2, fp8, shared=32, seed=1)
    new["x"] = m["x"]
    if strided:
        m.update({k: spread(m[k]) for k in ("up", "down", "router")})
    d = decoder(m, route=True)
    graph = torch.cuda.CUDAGraph()
    before = d(m["x"])
    with torch.cuda.graph(graph):
        captured = d(m["x"])
    for k in ("up", "down", "us", "ds", "router"):
        if m[k] is not None:
            raw = [t.view(torch.uint8) if t.dtype == F8 else t for t in (m[k], new[k])]
            raw[0].copy_(raw[1])
    for given, value in zip(m["shared"], new["shared"]):
        if given is not None:
            given.view(torch.uint8).copy_(value.view(torch.uint8))
    want = decoder(new, route=True)(m["x"])
    assert not torch.equal(before, want)
    assert torch.equal(d(m["x"]), want)
    graph.replay()  # (the call before it has renewed what there are copies of)
    torch.cuda.synchronize()
    assert torch.equal(captured, want)
    for t in (m["down"], m["shared"][1]):
        (t.data.view(torch.uint8) if fp8 else t.data).zero_()  # not counted by autograd
    d.reload()
    assert not d(m["x"]).any()
    graph.replay()
    torch.cuda.synchronize()
    assert not captured.any()


def test_inference_weights_are_reloaded():
    with torch.inference_mode():
        m = make(3, 515, 64, 4, 2)
        d = decoder(m)
        d(m["x"], m["ids"], m["w"])
        m["down"].zero_()
        d.reload()
        assert not d(m["x"], m["ids"], m["w"]).any()


@pytest.mark.parametrize("H,E", [(136, 128), (2048, 128), (512, 500), (1024, 24)])
def test_a_token_is_routed_alike_among_any_number(H, E):
    """The router's product has a form for few outputs and one for many; both add in one order."""
    m = make(64, H, 16, E, 4)
    d = decoder(m, route=True)
    _, ids, w = d.with_routing(m["x"])
    for T in (1, 2, 7, 8, 12, 13, 33, 48):
        _, ids_t, w_t = d.with_routing(m["x"][:T].contiguous())
        assert torch.equal(ids_t, ids[:T]) and torch.equal(w_t, w[:T]), T


@pytest.mark.parametrize("T,H,I,E,K,shared", [(1, 512, 64, 4, 2, 0), (7, 264, 72, 6, 2, 40), (33, 256, 128, 2, 1, 64),
                                              (64, 512, 128, 8, 2, 0), (64, 136, 64, 1, 1, 0)])
def test_only_the_output_is_rounded_to_16_bits(T, H, I, E, K, shared):
    """w h goes into the second product in two bf16 parts, 2^-18 of it left out. With the sums of both
    products in 32 bits (below 1e-5 of their terms' magnitudes each), 3e-5 of the magnitudes and the
    rounding of y bound the error. A single bf16 w h leaves 2^-9 / sqrt(3) of the root of the sum of
    squares, some times that where y is small."""
    m = make(T, H, I, E, K, shared=shared)
    y = decoder(m)(m["x"], m["ids"], m["w"])
    x, ids, w = m["x"].double(), m["ids"].long(), m["w"].double()
    want, ab = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        o, _, a = ffn(x[t], m["up"][e].double(), m["down"][e].double())
        want.index_add_(0, t, w[t, k][:, None] * o)
        ab.index_add_(0, t, w[t, k][:, None] * a)
    if shared:
        o, _, a = ffn(x, m["shared"][0].double(), m["shared"][1].double())
        want, ab = want + o, ab + a
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 3e-5 * ab).all()


@pytest.mark.parametrize("T,H,I,E,K,shared", [(1, 512, 64, 4, 2, 0), (7, 272, 80, 6, 2, 48), (33, 256, 128, 2, 1, 64),
                                              (64, 512, 128, 8, 2, 0), (64, 144, 64, 1, 1, 0)])
def test_e4m3_weights_meet_more_than_eight_bits_of_h(T, H, I, E, K, shared):
    """w h goes into the second product in three e4m3 parts, each of which leaves at most 2^-4 of what it is
    a part of: 2^-12 of a value. Independent errors of that size add up to 2^-12 / sqrt(3) of the root of
    the terms' sum of squares, six times that is allowed; the sums and y's rounding as above."""
    m = make(T, H, I, E, K, True, shared=shared)
    y = decoder(m)(m["x"], m["ids"], m["w"])
    want, _ = reference(m)
    sq, ab = (torch.zeros_like(want) for _ in range(2))
    x, ids, w = m["x"].double(), m["ids"].long(), m["w"].double()
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        _, s, a = ffn(x[t], values(m["up"][e:e + 1], m["us"][e:e + 1])[0], values(m["down"][e:e + 1], m["ds"][e:e + 1])[0])
        sq.index_add_(0, t, w[t, k][:, None].square() * s)
        ab.index_add_(0, t, w[t, k][:, None] * a)
    if shared:
        su, sd, sus, sds = m["shared"]
        _, s, a = ffn(x, values(su[None], sus[None])[0], values(sd[None], sds[None])[0])
        sq, ab = sq + s, ab + a
    tol = 2.0 ** -8 * want.abs() + 3.5 * 2.0 ** -12 * sq.sqrt() + 3e-5 * ab
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("T", [1, 16, 40])
def test_rows_with_a_few_large_channels_and_e4m3_weights(T):
    """Values of x down to 2^-13 of their row's largest keep their 8 bits, smaller ones are off by 2^-21 of
    the largest at most, which the sums' 1e-5 of the magnitudes of the row's terms covers: the largest is
    one of them. Channels of 2^10 and 2^18 times the others, whose weights are as large as any."""
    for factor in (2.0 ** 10, 2.0 ** 18):
        m = make(T, 512, 128, 8, 2, True, shared=64)
        m["x"][:, 7::100] *= factor
        check(m)


@pytest.mark.parametrize("fp8", [False, True])
def test_tensors_off_a_16_byte_boundary(fp8):
    def odd(t):
        raw = t.view(torch.uint8) if t.dtype == F8 else t
        buf = torch.empty(raw.numel() + 1, dtype=raw.dtype, device="cuda")
        return buf[1:].view(raw.shape).copy_(raw).view(t.dtype)

    m = make(5, 256, 64, 8, 2, fp8)
    y = decoder(m)(m["x"], m["ids"], m["w"])
    n = {k: odd(v) if isinstance(v, torch.Tensor) else v for k, v in m.items()}
    assert n["x"].data_ptr() % 16 and n["up"].data_ptr() % 16
    d = decoder(n)
    assert torch.equal(d(n["x"], n["ids"], n["w"]), y)
    (n["down"].view(torch.uint8) if fp8 else n["down"]).zero_()
    assert not d(n["x"], n["ids"], n["w"]).any()
    w = torch.randn(2, 256, 128, device="cuda").to(BF)
    for a, b in zip(block_ops.quantize_expert_weights(odd(w)), block_ops.quantize_expert_weights(w)):
        assert torch.equal(a.float(), b.float())


def test_copies_made_in_inference_mode_are_renewed_outside():
    m = make(3, 515, 64, 4, 2)
    m["down"] = torch.nn.Parameter(m["down"])
    with torch.inference_mode():
        d = decoder(m)
        y = d(m["x"], m["ids"], m["w"])
    with torch.no_grad():
        m["down"].mul_(2)
    assert torch.equal(d(m["x"], m["ids"], m["w"]), 2 * y)
    assert not any(copy.requires_grad for _, copy in d._copies)
    assert torch.equal(decoder(m)(m["x"], m["ids"], m["w"]), 2 * y)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 4, 40, 64])
def test_bad_expert_ids_leave_no_result(T, fp8):
    """All of y is NaN, whichever way the tables are built, and the next call is as ever."""
    m = make(T, 528, 64, 20, 4, fp8, shared=32)
    d = decoder(m)
    y = d(m["x"], m["ids"], m["w"])
    for at, bad in (((0, 0), 20), ((T - 1, 3), -1)):
        ids = m["ids"].clone()
        ids[at] = bad
        assert torch.isnan(d(m["x"], ids, m["w"])).all() and d.status() == _abi.MM_ERR_BAD_EXPERT_ID
    assert torch.equal(d(m["x"], m["ids"], m["w"]), y) and d.status() == _abi.MM_OK
