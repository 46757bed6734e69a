"""Static checks on the gfx950 code of the norm, the 8-bit products and the convolution (CPU
only: hipcc cross-compiles; nothing runs on a GPU)."""
import re

import pytest

from test_glr_kernel_asm import scratch
from test_kernel_asm import _compile_asm, _hipcc

# kernels of the source, and for name patterns the scratch they may use: the norm's backward
# over rows of 24577 to 32768 channels holds 32 of two inputs in each of 1024 lanes
SOURCES = {
    "sscan_rms.hip": (84, {r"rms_bwd_kernel\w*Li1024ELi4E": 64}),
    "sscan_i8_matmul.hip": (14, {}),
    "sscan_dwconv.hip": (44, {}),
}


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
@pytest.mark.parametrize("src", list(SOURCES))
def test_no_calls_and_no_more_scratch_than_stated(tmp_path, src):
    asm = _compile_asm(src, str(tmp_path / (src + ".s")))
    assert "s_swappc" not in asm and not re.search(r"\bv_pk_(add|mul|fma)_f32\b", asm)
    kernels, allowed = scratch(asm), SOURCES[src][1]
    assert len(kernels) == SOURCES[src][0], sorted(kernels)
    for name, size in kernels.items():
        most = max([v for k, v in allowed.items() if re.search(k, name)], default=0)
        assert size <= most, (name, size)


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
def test_products_use_matrix_instructions_and_loads_into_lds(tmp_path):
    asm = _compile_asm("sscan_i8_matmul.hip", str(tmp_path / "i8.s"))
    assert "v_mfma_i32_16x16x64_i8" in asm and re.search(r"global_load_lds_dwordx4|buffer_load_dwordx4.* lds", asm)
