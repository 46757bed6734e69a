"""The largest sizes that the norm, the 8-bit rows and products and the convolution accept, and
the first that they refuse: checked on the host, so none of this needs a GPU.  A call of a size
that is accepted goes on to the next check here, a missing pointer."""
import pytest

from test_layer_abi import INVALID, conv_bwd, conv_fwd, conv_step, lib, matmul, quant, rms_bwd, rms_fwd  # noqa: F401

MOST = 2 ** 31 - 1


def accepts(lib, call, **kw):  # noqa: F811
    assert call(lib, **kw) == INVALID and b"null" in lib.sscan_last_error(), lib.sscan_last_error()


def refuses(lib, call, **kw):  # noqa: F811
    assert call(lib, **kw) == INVALID and b"too large" in lib.sscan_last_error(), lib.sscan_last_error()


@pytest.mark.parametrize("call,missing", [(rms_fwd, "x"), (rms_bwd, "s"), (quant, "x")])
def test_rows(lib, call, missing):  # noqa: F811
    accepts(lib, call, rows=MOST, dim=32768, **{missing: None})
    refuses(lib, call, rows=MOST + 1, dim=1)


def test_products(lib):  # noqa: F811
    for size in (dict(m=MOST, n=1), dict(m=1, n=MOST), dict(m=2 ** 20, n=2 ** 19 - 16), dict(m=2 ** 20 - 16, n=2 ** 19)):
        accepts(lib, matmul, **size, k=131071, a=None)
    for size in (dict(m=MOST + 1, n=1), dict(m=1, n=MOST + 1), dict(m=2 ** 20, n=2 ** 19), dict(m=MOST, n=17 * 16)):
        refuses(lib, matmul, **size)


@pytest.mark.parametrize("most", [dict(batch=MOST, seqlen=1, dim=64), dict(batch=1, seqlen=2 ** 30, dim=64 * 127),
                                  dict(batch=1, seqlen=2 ** 30, dim=1), dict(batch=1, seqlen=64, dim=2 ** 28)])
def test_convolution(lib, most):  # noqa: F811
    for call in (conv_fwd, conv_bwd):
        accepts(lib, call, **most, w=None)


@pytest.mark.parametrize("over", [dict(batch=MOST + 1, seqlen=1, dim=64), dict(batch=1, seqlen=2 ** 30, dim=64 * 128),
                                  dict(batch=2 ** 30, seqlen=65, dim=1), dict(batch=1, seqlen=1, dim=2 ** 28 + 1)])
def test_convolution_over(lib, over):  # noqa: F811
    for call in (conv_fwd, conv_bwd):
        refuses(lib, call, **over)


def test_convolution_step(lib):  # noqa: F811
    accepts(lib, conv_step, batch=MOST, dim=64, pool=MOST, y=None)
    refuses(lib, conv_step, batch=MOST + 1, dim=64, pool=MOST + 1)
    refuses(lib, conv_step, batch=1, dim=2 ** 28, pool=2 ** 20)


def never_shrinks(size, fixed, values, at):
    """size(*fixed) with its argument `at` going through `values` in order."""
    last = 0
    for v in values:
        args = list(fixed)
        args[at] = v
        now = size(*args)
        assert now >= last, (args, now, last)
        last = now


COUNTS = sorted({1, 2, 3, 5, 7} | {2 ** k + d for k in range(4, 16) for d in (-1, 0, 1)})


def test_workspaces_serve_smaller_calls(lib):  # noqa: F811
    """A buffer for the longest batch serves every shorter one: sizes do not shrink as any count grows."""
    norm, conv = lib.sscan_rms_bwd_workspace_size, lib.sscan_dwconv_bwd_workspace_size
    for dim in (1, 64, 96, 512, 513, 1535, 2048, 2049, 2560, 8193, 32768):
        never_shrinks(norm, (0, dim), COUNTS, 0)
    for rows in (1, 511, 1023, 1024, 4096, 70000):
        never_shrinks(norm, (rows, 0), [d for d in COUNTS if d <= 32768], 1)
    for dim in (1, 3, 4, 130, 257, 1535, 2048, 2560, 10240):
        for batch in (1, 3, 8, 64):
            never_shrinks(conv, (batch, 0, dim, 4), COUNTS, 1)
        for seqlen in (1, 33, 65, 700, 4096):
            never_shrinks(conv, (0, seqlen, dim, 4), COUNTS, 0)
    for batch, seqlen in ((1, 1), (1, 4094), (1, 16411), (8, 4032), (8, 4096), (300, 64)):
        never_shrinks(conv, (batch, seqlen, 0, 4), COUNTS, 2)
        never_shrinks(conv, (batch, seqlen, 2048, 0), (1, 2, 3, 4), 3)
