"""Static checks on the gfx950 code of the gated recurrence's and the 8-bit kernels (CPU only:
hipcc cross-compiles; nothing runs on a GPU)."""
import re

import pytest

from test_kernel_asm import _compile_asm, _hipcc


def scratch(asm):
    """{kernel: bytes of scratch a lane}."""
    return dict((k, int(v)) for k, v in re.findall(
        r"\.name:\s+(_ZN5sscan\w+)\n(?:.*\n)*?\s+\.private_segment_fixed_size:\s*(\d+)", asm))


# kernels of the source, and for name patterns the scratch they may use: a few registers of 16
# tokens spilled at the waves a SIMD that the kernels' comments give reasons for
SOURCES = {
    "sscan_act8.hip": (12, {}),
    "sscan_glr_step.hip": (4, {}),
    # gated and packed, two channels a lane
    "sscan_glr_fwd.hip": (49, {r"glr_fwd_kernelItLi2ELb\dELb1ELb1E": 8, r"glr_fwd_kernelIfLi2ELb\dELb1ELb1E": 36}),
    # bf16 dense without a gate, at four waves a SIMD; gated and packed
    "sscan_glr_bwd.hip": (33, {r"glr_bwd_kernelItLb\dELb0ELb0E": 16, r"glr_bwd_kernelItLb\dELb1ELb1E": 36,
                               r"glr_bwd_kernelIfLb\dELb1ELb1E": 32}),
}


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not found")
@pytest.mark.parametrize("src", list(SOURCES))
def test_no_calls_and_no_more_scratch_than_stated(tmp_path, src):
    asm = _compile_asm(src, str(tmp_path / (src + ".s")))
    assert "s_swappc" not in asm
    kernels, allowed = scratch(asm), SOURCES[src][1]
    assert len(kernels) == SOURCES[src][0], sorted(kernels)
    for name, size in kernels.items():
        most = max([v for k, v in allowed.items() if re.search(k, name)], default=0)
        assert size <= most, (name, size)
