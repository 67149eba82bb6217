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
    found = re.findall(r"#define\s+(MM_\w+)\s+(0x\d+|\d+)u?\b", open(_abi.EXPERTS_HEADER_PATH).read())
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

    def product(d, *p, w=256, size=1 << 30):
        return lib.mm_grouped_mm(ref(d), *p, w, size, None)

    def weight(d, *p, w=256, size=1 << 30):
        return lib.mm_grouped_mm_weight_grad(ref(d), *p, 0, w, size, None)

    full = (16, 16, 16, 16)
    assert lib.mm_grouped_mm(None, *full, 256, 1 << 30, None) == BAD
    assert lib.mm_grouped_workspace_size(None) == 0
    for call in (product, weight):
        for d in (grouped(R=-1), grouped(K=0), grouped(N=0), grouped(E=0), grouped(out=2), grouped(flags=3),
                  grouped(flags=4)):
            assert call(d, *full) == BAD and lib.mm_grouped_workspace_size(ref(d)) == 0
        for d in (grouped(K=60), grouped(N=4), grouped(K=65544), grouped(N=65544), grouped(E=1025),
                  grouped(R=2 ** 31)):
            assert call(d, *full) == UNSUP and lib.mm_grouped_workspace_size(ref(d)) == 0
        d = grouped()
        n = lib.mm_grouped_workspace_size(ref(d))
        assert n >= 256
        assert call(grouped(), *full, w=None) == WS and call(grouped(), *full, w=128) == WS
        assert call(grouped(), *full, size=n - 1) == WS
        for i in range(4):
            for p in (None, 2 if i == 2 else 8):
                assert call(grouped(), *full[:i], p, *full[i + 1:]) == BAD
    assert product(grouped(R=0), None, None, None, None) == _abi.MM_OK
    assert weight(grouped(R=0), None, None, None, 16) == BAD  # zeros have to go somewhere
