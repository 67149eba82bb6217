"""include/mm_ops.h: the library exports every function it declares, and the host-side checks
return before any CUDA call."""
import ctypes
import os
import re

import pytest

from moe_ffn_expert_gb300 import _abi
from moe_ffn_expert_gb300 import build as mm_build


@pytest.fixture(scope="module", autouse=True)
def built():
    mm_build.build()


def ref(d):
    return ctypes.addressof(d)


def test_exports_every_header_symbol():
    names = _abi.header_symbols(_abi.OPS_HEADER_PATH)
    assert len(names) >= 7
    lib = _abi._lib()
    for n in names:
        assert getattr(lib, n).argtypes is not None, n
    assert lib.mm_ops_version() == 1


def test_constants_match_the_header():
    text = open(_abi.OPS_HEADER_PATH).read()
    found = re.findall(r"#define\s+(MM_\w+)\s+(\d+)", text) + re.findall(r"\b(MM_(?:BF16|FP32|E4M3))\s*=\s*(\d+)", text)
    assert len(found) >= 5
    for name, value in found:
        assert getattr(_abi, name) == int(value), name


def test_headers_compile_as_c(tmp_path):
    import subprocess
    src = tmp_path / "h.c"
    src.write_text('#include "mm_ops.h"\nint main(void) { return mm_ops_version() ? 0 : 1; }\n')
    inc = os.path.dirname(_abi.OPS_HEADER_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", inc, "-c", str(src), "-o",
                    str(tmp_path / "h.o")], check=True)


def norm(T=8, H=64, groups=1, st=0, bt=0, pt=0, scale=1.0, eps=1e-6):
    return _abi.mm_norm_desc(T, H, groups, st, bt, pt, scale, eps)


def test_residual_norm_host_checks():
    lib = _abi._lib()
    bad, unsup, ws = _abi.MM_ERR_INVALID_ARG, _abi.MM_ERR_UNSUPPORTED, _abi.MM_ERR_WORKSPACE

    def fwd(d, *p):
        return lib.mm_residual_norm_forward(ref(d), *p, None)

    full = (16, 16, 16, 16, 16, 16, 16)
    assert lib.mm_residual_norm_forward(None, *full, None) == bad
    for d in (norm(T=-1), norm(H=0), norm(groups=-1), norm(groups=3), norm(st=2), norm(st=0, bt=1),
              norm(pt=5), norm(eps=-1.0), norm(eps=float("nan")), norm(eps=float("inf"))):
        assert fwd(d, *full) == bad
        assert lib.mm_residual_norm_workspace_size(ref(d)) == 0
    assert fwd(norm(H=16385), *full) == unsup
    assert fwd(norm(T=2 ** 31), *full) == unsup
    assert fwd(norm(), None, 16, 16, 16, 16, 16, 16) == bad          # no residual
    assert fwd(norm(), 16, None, 16, 16, 16, 16, 16) == bad          # a post weight without a branch
    assert fwd(norm(), 16, 16, 16, 16, None, 16, 16) == bad          # groups without a gate
    assert fwd(norm(groups=0), 16, 16, 16, 16, 16, 16, 16) == bad    # a gate without groups
    assert fwd(norm(), 16, 16, 16, 16, 16, 16, None) == bad          # a pre weight without its output
    assert fwd(norm(), 17, 16, 16, 16, 16, 16, 16) == bad            # odd address
    assert fwd(norm(st=1), 18, 16, 16, 16, 16, 16, 16) == bad        # fp32 at 2 bytes
    assert fwd(norm(T=0), *([None] * 7)) == _abi.MM_OK
    d = norm()
    n = lib.mm_residual_norm_workspace_size(ref(d))
    assert n >= 256

    def bwd(d, *p, w=256, size=n):
        return lib.mm_residual_norm_backward(ref(d), *p, w, size, None)

    full = (16,) * 12
    assert bwd(d, *full, w=None) == ws and bwd(d, *full, w=128) == ws and bwd(d, *full, size=0) == ws
    assert bwd(d, None, *full[1:]) == bad
    assert bwd(d, *full[:11], None) == bad                            # no d_gate
    assert bwd(d, *full[:6], None, *full[7:]) == bad                  # no d_normed
    assert bwd(d, *full[:8], None, *full[9:]) == bad                  # no d_branch


def test_router_host_checks():
    lib = _abi._lib()

    def desc(T=8, E=16, K=2, lt=1, score=0, norm=1):
        return _abi.mm_router_desc(T, E, K, lt, score, norm, 1.0)

    def fwd(d, *p, w=256, size=1 << 20):
        return lib.mm_router_forward(ref(d), *p, w, size, None)

    full = (16, 16, 16, 16, 16, 16)
    for d in (desc(T=-1), desc(E=0), desc(K=0), desc(K=17), desc(lt=2), desc(score=2)):
        assert fwd(d, *full) == _abi.MM_ERR_INVALID_ARG
        assert lib.mm_router_workspace_size(ref(d)) == 0
    assert fwd(desc(E=1025), *full) == _abi.MM_ERR_UNSUPPORTED
    assert fwd(desc(E=32, K=17), *full) == _abi.MM_ERR_UNSUPPORTED
    d = desc()
    assert fwd(d, None, *full[1:]) == _abi.MM_ERR_INVALID_ARG
    assert fwd(d, 18, *full[1:]) == _abi.MM_ERR_INVALID_ARG
    assert fwd(d, *full, w=None) == _abi.MM_ERR_WORKSPACE
    assert fwd(d, *full, size=16) == _abi.MM_ERR_WORKSPACE
    assert lib.mm_router_workspace_size(ref(d)) >= 256
    assert lib.mm_router_backward(ref(d), 16, None, 16, None, None, 16, None) == _abi.MM_ERR_INVALID_ARG
    assert lib.mm_router_backward(ref(desc(T=0)), None, None, None, None, None, None, None) == _abi.MM_OK


def test_decode_host_checks():
    lib = _abi._lib()
    bad, unsup, wsz = _abi.MM_ERR_INVALID_ARG, _abi.MM_ERR_UNSUPPORTED, _abi.MM_ERR_WORKSPACE

    def desc(T=4, H=64, I=32, E=8, K=2, Is=0, wt=0, rt=0, score=0):
        return _abi.mm_decode_desc(_abi.dims(T, H, I, E, K), Is, wt, rt, score, 1, 1.0)

    def weights(up=16, down=16, us=0, ds=0, su=0, sd=0, sus=0, sds=0, r=16, b=0):
        return _abi.mm_decode_weights(*[p or None for p in (up, down, us, ds, su, sd, sus, sds, r, b)])

    def call(d, w, x=16, ids=16, tw=16, y=16, ws=256, size=1 << 30):
        return lib.mm_decode(ref(d), ref(w), x, ids, tw, y, ws, size, None)

    for d in (desc(T=-1), desc(H=0), desc(I=0), desc(E=0), desc(K=0), desc(Is=-8), desc(wt=1), desc(rt=2), desc(score=3)):
        assert call(d, weights()) == bad and lib.mm_decode_workspace_size(ref(d)) == 0
    for d in (desc(T=65), desc(K=17), desc(T=64, K=17), desc(E=1025), desc(H=60), desc(I=36), desc(Is=4), desc(H=65544),
              desc(wt=2, H=72), desc(wt=2, I=40)):
        assert call(d, weights()) == unsup and lib.mm_decode_workspace_size(ref(d)) == 0
    d = desc()
    n = lib.mm_decode_workspace_size(ref(d))
    assert n > 0
    assert call(d, weights(), size=n - 1) == wsz and call(d, weights(), ws=128) == wsz and call(d, weights(), ws=None) == wsz
    for w in (weights(up=0), weights(down=24), weights(us=16, ds=16), weights(su=16, sd=16), weights(r=8), weights(b=2),
              weights(r=0, b=16)):
        assert call(d, w) == bad
    assert call(d, weights(), x=None) == bad and call(d, weights(), y=24) == bad and call(d, weights(), ids=18) == bad
    assert call(d, weights(r=0), ids=None) == bad                      # no router: the ids are inputs
    assert call(desc(E=1, K=2), weights()) == bad                      # more experts wanted than there are
    assert call(desc(wt=2), weights()) == bad                          # 8-bit weights without scales
    assert call(desc(Is=32), weights()) == bad                         # a shared expert without weights
    assert lib.mm_quantize_blocks(-1, 8, 8, 16, 16, 16, None) == bad
    assert lib.mm_quantize_blocks(1, 8, 12, 16, 16, 16, None) == unsup
    assert lib.mm_quantize_blocks(1, 8, 8, 24, 16, 16, None) == bad
    assert lib.mm_quantize_blocks(0, 8, 8, None, None, None, None) == _abi.MM_OK
