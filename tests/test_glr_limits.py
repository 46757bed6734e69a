"""The largest sizes that the gated linear recurrence and the 8-bit activations accept, and the
first that they refuse: checked on the host, so none of this needs a GPU.  A call of a size
that is accepted goes on to the next check here, a missing pointer."""
import pytest

from test_glr_abi import INVALID, bwd, fwd, lib, step  # noqa: F401


@pytest.mark.parametrize("most", [dict(batch=2 ** 31 - 1, seqlen=1, dim=64), dict(batch=1, seqlen=2 ** 30, dim=64 * 127),
                                  dict(batch=1, seqlen=2 ** 30, dim=1), dict(batch=1, seqlen=64, dim=2 ** 28)])
def test_tiles(lib, most):  # noqa: F811
    for call, missing in ((fwd, "y"), (bwd, "dlam")):
        assert call(lib, **most, **{missing: None}) == INVALID and b"null" in lib.sscan_last_error()


@pytest.mark.parametrize("over", [dict(batch=2 ** 31, seqlen=1, dim=64), dict(batch=1, seqlen=2 ** 30, dim=64 * 128),
                                  dict(batch=2 ** 30, seqlen=65, dim=1), dict(batch=1, seqlen=1, dim=2 ** 28 + 1)])
def test_too_many_tiles(lib, over):  # noqa: F811
    for call in (fwd, bwd):
        assert call(lib, **over) == INVALID and b"too large" in lib.sscan_last_error()


def test_step_rows(lib):  # noqa: F811
    assert step(lib, batch=2 ** 31 - 1, slots_n=2 ** 31 - 1, y=None) == INVALID and b"null" in lib.sscan_last_error()
    assert step(lib, batch=2 ** 31, slots_n=2 ** 31) == INVALID and b"too large" in lib.sscan_last_error()


def test_packed_lanes(lib):  # noqa: F811
    most = 2 ** 39 - 257                         # 2^31 - 2 whole workgroups of 256 lanes, and 255
    for n, word in ((most, b"null"), (most + 1, b"too large")):
        assert lib.sscan_act8_pack(n, 1, 1, 0, None, 0, None, 0, None) == INVALID and word in lib.sscan_last_error()
        assert lib.sscan_act8_unpack(n, 1, 1, 0, None, 0, None, None) == INVALID and word in lib.sscan_last_error()


def test_binding_refuses_a_gate_without_z():
    import torch
    import selective_state_space_45_amd as ss

    class OnGpu(torch.Tensor):                    # as far as the host's checks see
        is_cuda = True

    x = torch.zeros(1, 4, 8).as_subclass(OnGpu)
    with pytest.raises(ValueError, match="z is required"):
        ss.sscan_glr_bwd(torch.zeros(8), x, torch.zeros(8), x=x, r=x, i=x, gated=True)
    with pytest.raises(ValueError, match="GPU"):
        ss.sscan_glr_bwd(torch.zeros(8), torch.zeros(1, 4, 8), torch.zeros(8), x=x, r=x, i=x, z=x, gated=True)
