"""Refusals of the gated linear recurrence and of the 8-bit activations: every argument is
checked on the host, so none of this needs a GPU."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "selective_state_space_45_amd", "libselscan.so")
P = ctypes.c_void_p
MB = 1 << 20
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from selective_state_space_45_amd import build as b
        b.build()
    import selective_state_space_45_amd as ss
    return ss.library()


def at(k):
    """An address that no call here reaches: each fails its checks first, or is empty."""
    return P((k + 1) * MB)


def strides(*v):
    return ctypes.cast((ctypes.c_int64 * 4)(*v), P)


def fwd(lib, **kw):
    a = dict(batch=2, seqlen=70, dim=4, dtype=0, x=at(0), r=at(1), i=at(2), z=None, strides=None, lam=at(4), rb=None,
             ib=None, scale=8.0, h0=None, off=None, nseq=0, y=at(8), last=None, ck=None, nck=0, sv=None, nsv=0,
             ws=at(12), nws=1 << 30, stream=None)
    assert set(kw) <= set(a)
    return lib.sscan_glr_fwd(*{**a, **kw}.values())


def bwd(lib, **kw):
    a = dict(batch=2, seqlen=70, dim=4, dtype=0, x=at(0), r=at(1), i=at(2), z=None, strides=None, sv=None, nsv=0,
             lam=at(4), rb=None, ib=None, scale=8.0, h0=None, off=None, nseq=0, ck=at(5), nck=1 << 20, dy=at(6),
             dlast=None, dx=at(8), dr=at(9), di=at(10), dz=None, gst=None, dlam=at(11), drb=None, dib=None, dh0=None,
             ws=at(20), nws=1 << 30, stream=None)
    assert set(kw) <= set(a)
    return lib.sscan_glr_bwd(*{**a, **kw}.values())


def step(lib, **kw):
    a = dict(batch=2, dim=4, dtype=0, state=at(0), slots_n=4, slots=None, out=None, x=at(1), r=at(2), i=at(3), z=None,
             strides=None, lam=at(5), rb=None, ib=None, scale=8.0, y=at(6), stream=None)
    assert set(kw) <= set(a)
    return lib.sscan_glr_step(*{**a, **kw}.values())


COMMON = [(dict(dtype=5), UNSUPPORTED, b"dtype"), (dict(batch=-1), INVALID, b"negative"),
          (dict(dim=-1), INVALID, b"negative"), (dict(x=None), INVALID, b"null"), (dict(r=None), INVALID, b"null"),
          (dict(i=None), INVALID, b"null"), (dict(lam=None), INVALID, b"null"), (dict(x=P(MB + 2)), INVALID, b"align"),
          (dict(lam=P(5 * MB + 1)), INVALID, b"align"), (dict(rb=P(5 * MB + 2)), INVALID, b"align"),
          (dict(ib=P(5 * MB + 2)), INVALID, b"align"), (dict(scale=0.0), INVALID, b"decay_scale"),
          (dict(scale=-1.0), INVALID, b"decay_scale"), (dict(scale=float("nan")), INVALID, b"decay_scale"),
          (dict(scale=float("inf")), INVALID, b"decay_scale"), (dict(strides=strides(4, 4, 3, 4)), INVALID, b"stride of i"),
          (dict(strides=strides(1 << 50, 4, 4, 4)), INVALID, b"too large")]
SEQ = [(dict(seqlen=-1), INVALID, b"negative"), (dict(seqlen=(1 << 30) + 1), INVALID, b"SSCAN_MAX_SEQLEN"),
       (dict(batch=1 << 40, dim=1 << 40), INVALID, b"too large"), (dict(off=at(30), nseq=3), INVALID, b"batch 1"),
       (dict(off=at(30), nseq=0, batch=1), INVALID, b"num_seqs"), (dict(off=P(2), nseq=1, batch=1), INVALID, b"align"),
       (dict(h0=P(31 * MB + 2)), INVALID, b"align")]


@pytest.mark.parametrize("kw,code,word", COMMON + SEQ + [
    (dict(y=None), INVALID, b"null"), (dict(y=P(MB + 16)), INVALID, b"overlap"), (dict(y=at(4)), INVALID, b"overlap"),
    (dict(last=P(9 * MB + 1)), INVALID, b"align"), (dict(last=at(8)), INVALID, b"overlap"),
    (dict(h0=at(30), last=P(31 * MB + 4)), INVALID, b"overlap"), (dict(ck=at(30), nck=63), INVALID, b"too small"),
    (dict(ck=at(8), nck=1 << 20), INVALID, b"overlap"), (dict(sv=P(31 * MB + 128), nsv=1 << 20), INVALID, b"align"),
    (dict(sv=at(30), nsv=100), INVALID, b"too small"), (dict(sv=at(0), nsv=1 << 20), INVALID, b"overlap")])
def test_forward_refuses(lib, kw, code, word):
    assert fwd(lib, **kw) == code
    assert word in lib.sscan_last_error()


@pytest.mark.parametrize("kw,code,word", COMMON + SEQ + [
    (dict(dy=None), INVALID, b"null"), (dict(dx=None), INVALID, b"null"), (dict(dr=None), INVALID, b"null"),
    (dict(di=None), INVALID, b"null"), (dict(dlam=None), INVALID, b"null"), (dict(ck=None), INVALID, b"checkpoints"),
    (dict(nck=63), INVALID, b"too small"), (dict(z=at(3)), INVALID, b"dz"), (dict(dz=at(13)), INVALID, b"dz"),
    (dict(sv=at(30), nsv=1 << 20), INVALID, b"must be null"),
    (dict(sv=at(30), nsv=100, x=None, r=None, i=None), INVALID, b"too small"), (dict(dx=at(0)), INVALID, b"overlap"),
    (dict(dr=at(8)), INVALID, b"overlap"), (dict(dlam=at(8)), INVALID, b"overlap"),
    (dict(gst=strides(3, 4, 4, 4)), INVALID, b"stride of dx"),
    # interleaved rows whose columns meet, and rows of unequal strides across one another
    (dict(dx=at(8), dr=P(9 * MB + 8), gst=strides(8, 8, 4, 4)), INVALID, b"overlap"),
    (dict(dx=at(8), dr=P(9 * MB + 16), gst=strides(8, 9, 4, 4)), INVALID, b"overlap")])
def test_backward_refuses(lib, kw, code, word):
    assert bwd(lib, **kw) == code
    assert word in lib.sscan_last_error()


@pytest.mark.parametrize("kw,code,word", COMMON + [
    (dict(y=None), INVALID, b"null"), (dict(state=None), INVALID, b"null"), (dict(batch=5), INVALID, b"num_slots"),
    (dict(slots_n=-1), INVALID, b"num_slots"), (dict(slots=P(2)), INVALID, b"align"), (dict(out=P(2)), INVALID, b"align"),
    (dict(y=at(0)), INVALID, b"overlap"), (dict(x=P(MB + 32)), INVALID, b"overlap"), (dict(y=at(1)), INVALID, b"overlap")])
def test_step_refuses(lib, kw, code, word):
    assert step(lib, **kw) == code
    assert word in lib.sscan_last_error()


def test_empty_calls_do_nothing(lib):
    assert fwd(lib, batch=0) == OK and fwd(lib, dim=0) == OK
    assert bwd(lib, dim=0) == OK
    assert step(lib, batch=0) == OK and step(lib, dim=0) == OK
    assert lib.sscan_act8_pack(0, 5, 5, 0, None, 0, None, 0, None) == OK
    assert lib.sscan_act8_unpack(1, 0, 5, 0, None, 0, None, None) == OK


def test_act8_refuses(lib):
    pack = lambda **kw: lib.sscan_act8_pack(*{**dict(b=1, l=20, d=4, t=0, x=at(0), s=0, p=at(1), n=1 << 20, q=None), **kw}.values())
    unpack = lambda **kw: lib.sscan_act8_unpack(*{**dict(b=1, l=20, d=4, t=0, p=at(1), n=1 << 20, x=at(0), q=None), **kw}.values())
    for call in (pack, unpack):
        for kw, code, word in ((dict(t=9), UNSUPPORTED, b"dtype"), (dict(l=-1), INVALID, b"negative"),
                               (dict(x=None), INVALID, b"null"), (dict(p=None), INVALID, b"null"),
                               (dict(p=P(MB * 2 + 64)), INVALID, b"align"), (dict(n=511), INVALID, b"too small"),
                               (dict(x=P(MB * 2 + 16)), INVALID, b"overlap"), (dict(x=P(MB + 1)), INVALID, b"align")):
            assert call(**kw) == code, kw
            assert word in lib.sscan_last_error()
    assert pack(s=3) == INVALID and b"stride" in lib.sscan_last_error()


def test_sizes(lib):
    up = lambda v, k: -(-v // k) * k
    for b, l, d in ((1, 1, 1), (2, 17, 5), (8, 4096, 2048), (1, 65, 1001)):
        one = up(b * l * d, 256) + up(b * (-(-l // 16)) * d, 256)
        assert lib.sscan_act8_bytes(b, l, d) == one
        assert lib.sscan_glr_saved_bytes(b, l, d, 0) == 3 * one and lib.sscan_glr_saved_bytes(b, l, d, 1) == 4 * one
        assert lib.sscan_glr_checkpoint_bytes(b, l, d) == 4 * b * (-(-l // 64)) * d
    for f in (lib.sscan_act8_bytes, lib.sscan_glr_checkpoint_bytes, lib.sscan_glr_fwd_workspace_size,
              lib.sscan_glr_bwd_workspace_size):
        assert f(-1, 5, 5) == 0 and f(1 << 40, 1 << 30, 1 << 40) == 0 and f(1, (1 << 30) + 1, 5) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    import selective_state_space_45_amd as ss
    x = torch.zeros(1, 4, 8)
    lam = torch.zeros(8)
    for call in (lambda: ss.sscan_glr_fwd(x, x, x, lam), lambda: ss.sscan_glr_bwd(lam, x, lam, x=x, r=x, i=x),
                 lambda: ss.sscan_act8_pack(x), lambda: ss.sscan_glr_step(x[0], x[0], x[0], x[0], lam)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="batch, seqlen, dim"):
        ss.sscan_glr_fwd(x[0], x, x, lam)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ss.sscan_act8_pack(x.double())
