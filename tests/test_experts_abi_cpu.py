"""include/mm_experts.h: the library exports every function it declares, and the host-side checks
return before any CUDA call."""
import ctypes
import os
import re
import subprocess

import pytest

from moe_ffn_expert_gb300 import _abi
from moe_ffn_expert_gb300 import build as mm_build

BAD, UNSUP, WS = _abi.MM_ERR_INVALID_ARG, _abi.MM_ERR_UNSUPPORTED, _abi.MM_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def built():
    mm_build.build()


def ref(d):
    return ctypes.addressof(d)


def test_exports_every_header_symbol():
    names = _abi.header_symbols(_abi.EXPERTS_HEADER_PATH)
    assert len(names) >= 4
    lib = _abi._lib()
    for n in names:
        assert getattr(lib, n).argtypes is not None, n
    assert lib.mm_experts_version() == 1


def test_constants_match_the_header():
    found = re.findall(r"#define\s+(MM_\w+)\s+(0x[0-9A-Fa-f]+|\d+)u?\b", open(_abi.EXPERTS_HEADER_PATH).read())
    assert len(found) >= 2
    for name, value in found:
        assert getattr(_abi, name) == int(value, 0), name


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "mm_experts.h"\nint main(void) { return mm_experts_version() ? 0 : 1; }\n')
    inc = os.path.dirname(_abi.EXPERTS_HEADER_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", inc, "-c", str(src), "-o",
                    str(tmp_path / "h.o")], check=True)


def grouped(R=8, K=64, N=72, E=4, transposed=0, out=0, flags=0):
    return _abi.mm_grouped_desc(R, K, N, E, transposed, out, flags)


def test_grouped_host_checks():
    lib = _abi._lib()

    def product(d, *p):
        return lib.mm_grouped_mm(ref(d), *p, 256, 1 << 40, None)

    def weight(d, *p, w=256, size=1 << 40):
        return lib.mm_grouped_mm_weight_grad(ref(d), *p, 0, w, size, None)

    full = (16, 16, 16, 16)
    assert lib.mm_grouped_mm(None, *full, 256, 1 << 40, None) == BAD
    sizes = (lib.mm_grouped_mm_workspace_size, lib.mm_grouped_weight_grad_workspace_size)
    assert [f(None) for f in sizes] == [0, 0]
    for call in (product, weight):
        for d in (grouped(R=-1), grouped(K=0), grouped(N=0), grouped(E=0), grouped(out=2), grouped(flags=3),
                  grouped(flags=4)):
            assert call(d, *full) == BAD and [f(ref(d)) for f in sizes] == [0, 0]
        for d in (grouped(K=60), grouped(N=4), grouped(K=65544), grouped(N=65544), grouped(E=1025),
                  grouped(R=2 ** 30)):
            assert call(d, *full) == UNSUP and [f(ref(d)) for f in sizes] == [0, 0]
        for i in range(4):
            for p in (None, 2 if i == 2 else 8):
                assert call(grouped(), *full[:i], p, *full[i + 1:]) == BAD
    d = grouped()
    n = sizes[1](ref(d))
    assert n >= 256 and sizes[0](ref(d)) >= 256
    assert weight(d, *full, w=None) == WS and weight(d, *full, w=128) == WS and weight(d, *full, size=n - 1) == WS
    assert product(grouped(R=0), None, None, None, None) == _abi.MM_OK
    assert weight(grouped(R=0), None, None, None, 16) == BAD  # zeros have to go somewhere


def test_expert_host_checks():
    lib = _abi._lib()

    def desc(T=8, H=64, E=4, K=2, type=0):
        return _abi.mm_expert_desc(T, H, E, K, type)

    def table(d, *p, w=256, size=1 << 30):
        return lib.mm_expert_table(ref(d), *p, w, size, None)

    def dispatch(d, *p):
        return lib.mm_expert_dispatch(ref(d), *p, None)

    def combine(d, *p):
        return lib.mm_expert_combine(ref(d), *p, None)

    def backward(d, *p):
        return lib.mm_expert_combine_backward(ref(d), *p, None)

    four, seven = (16,) * 4, (16,) * 7
    assert lib.mm_expert_table(None, *four, 256, 1 << 30, None) == BAD
    for d in (desc(T=-1), desc(E=0), desc(K=0)):
        assert table(d, *four) == BAD and lib.mm_expert_table_workspace_size(ref(d)) == 0
        assert dispatch(d, *four) == BAD and combine(d, *four) == BAD and backward(d, *seven) == BAD
    for d in (desc(E=1025), desc(K=17), desc(T=2 ** 31 - 1), desc(T=2 ** 40)):
        assert table(d, *four) == UNSUP and lib.mm_expert_table_workspace_size(ref(d)) == 0
        assert dispatch(d, *four) == UNSUP and combine(d, *four) == UNSUP and backward(d, *seven) == UNSUP
    for d in (desc(H=0), desc(type=2)):
        assert dispatch(d, *four) == BAD and combine(d, *four) == BAD and backward(d, *seven) == BAD
    big = desc(H=2 ** 20 + 1)
    assert dispatch(big, *four) == UNSUP and combine(big, *four) == UNSUP and backward(big, *seven) == UNSUP
    d, f = desc(), desc(type=1)
    n = lib.mm_expert_table_workspace_size(ref(d))
    assert n >= 256
    many = desc(T=2049)  # (up to 2048 slots need no workspace)
    n = lib.mm_expert_table_workspace_size(ref(many))
    assert table(many, *four, size=n - 1) == WS and table(many, *four, w=None) == WS and table(many, *four, w=64) == WS
    for i in range(4):
        for p in (None, 2):
            assert table(d, *four[:i], p, *four[i + 1:]) == BAD
        if i != 2:
            assert combine(d, *four[:i], None, *four[i + 1:]) == (BAD if i != 2 else 0)
        assert dispatch(f, *four[:i], 2, *four[i + 1:]) == BAD and combine(f, *four[:i], 2, *four[i + 1:]) == BAD
        assert dispatch(d, *four[:i], None, *four[i + 1:]) == BAD
    for i in range(7):
        assert backward(f, *seven[:i], 2, *seven[i + 1:]) == BAD
        if i not in (4, 6):  # no weights: 1; no d_weights: not wanted
            assert backward(d, *seven[:i], None, *seven[i + 1:]) == BAD
    empty = desc(T=0)
    assert dispatch(empty, *[None] * 4) == combine(empty, *[None] * 4) == backward(empty, *[None] * 7) == _abi.MM_OK


def test_grad_host_checks():
    lib = _abi._lib()

    def refs(*items):
        return (_abi.mm_tensor_ref * len(items))(*[_abi.mm_tensor_ref(*i) for i in items])

    def norm(t, n=None, out=16, w=256, size=1 << 30):
        return lib.mm_grad_norm(len(t) if n is None else n, ctypes.addressof(t) if t else None, out, w, size, None)

    def clip(t, max_norm=1.0, eps=1e-6, n=None, out=16, w=256, size=1 << 30):
        return lib.mm_grad_clip(len(t) if n is None else n, ctypes.addressof(t) if t else None, max_norm, eps, out, w,
                                size, None)

    good = refs((32, 32, 5, 0, 0))
    for call in (norm, clip):
        assert call(good, n=-1) == BAD and call(good, n=2 ** 20) == UNSUP and call(None, n=1) == BAD
        assert call(good, out=None) == BAD and call(good, out=2) == BAD
        assert call(good, w=None) == WS and call(good, w=64) == WS
        assert call(good, size=lib.mm_grad_workspace_size(1) - 1) == WS
        for t in ((32, 32, -1, 0, 0), (32, 32, 5, 2, 0), (None, 32, 5, 0, 0), (33, 33, 5, 0, 0), (34, 34, 5, 1, 1)):
            assert call(refs(t)) == BAD
        assert call(refs((32, 32, 1 << 44, 0, 0))) == UNSUP
    for t in ((32, None, 5, 0, 0), (32, 64, 5, 0, 2), (32, 66, 5, 0, 1), (32, 32, 5, 0, 1)):
        assert clip(refs(t)) == BAD
    for value in (-1.0, float("nan")):
        assert clip(good, max_norm=value) == BAD and clip(good, eps=value) == BAD
    assert clip(good, eps=float("inf")) == BAD
    assert lib.mm_grad_workspace_size(-1) == lib.mm_grad_workspace_size(2 ** 20) == 0
    assert lib.mm_grad_workspace_size(0) >= 256


def test_grouped_status_host_checks():
    lib = _abi._lib()
    d, full = grouped(), (16, 16, 16, 16)
    for status in (2, 18):
        assert lib.mm_grouped_mm_ex(ref(d), *full, 256, 1 << 40, status, None) == BAD
        assert lib.mm_grouped_mm_weight_grad_ex(ref(d), *full, 0, 256, 1 << 40, status, None) == BAD
    assert lib.mm_grouped_mm_ex(ref(grouped(R=0)), *[None] * 4, None, 0, 64, None) == _abi.MM_OK
    assert lib.mm_grouped_mm_weight_grad_ex(ref(d), *full, 0, None, 1 << 40, 64, None) == WS
