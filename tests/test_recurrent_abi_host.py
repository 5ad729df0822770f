"""Host-side tests of the gated scan's and the state cache's C ABI (no GPU): sizes, and what is
refused before any CUDA call (fake device addresses are never dereferenced)."""
import ctypes

import pytest

import mamba_ssd_scan_mixer_b200 as m2

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A0 = 1 << 20


def _dims(**kw):
    d = m2.make_gated_scan_dims(2, 300, 64)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_DIMS = [(dict(batch=-1), INVALID), (dict(seqlen=-1), INVALID), (dict(width=0), INVALID),
            (dict(io_dtype=2), INVALID), (dict(decay_scale=0.0), INVALID),
            (dict(decay_scale=float("inf")), INVALID), (dict(decay_scale=float("nan")), INVALID),
            (dict(width=12), UNSUPPORTED), (dict(width=(1 << 20) + 8), UNSUPPORTED),
            (dict(seqlen=1 << 31), UNSUPPORTED), (dict(batch=1 << 30, seqlen=1 << 30), UNSUPPORTED)]


def _prefill(d, **kw):
    a = dict(lam=A0, x=A0 + 0x1000, lx=64, r=A0 + 0x2000, lr=64, g=A0 + 0x3000, lg=64, z=None, lz=0,
             cu=None, y=A0 + 0x4000, h=A0 + 0x5000, sin=0, ck=None, ws=A0 + 0x10000, bytes=1 << 30)
    a.update(kw)
    return m2.lib().mamba2_gated_scan_prefill(ctypes.byref(d) if d is not None else None,
                                              *list(a.values()), None)


def _backward(d, **kw):
    a = dict(lam=A0, x=A0 + 0x1000, lx=64, r=A0 + 0x2000, lr=64, g=A0 + 0x3000, lg=64, z=None, lz=0,
             cu=None, hin=None, dy=A0 + 0x4000, dh=None, ck=None, dx=A0 + 0x5000, dr=A0 + 0x6000,
             dg=A0 + 0x7000, dz=None, dlam=A0 + 0x8000, dhin=None, ws=A0 + 0x10000, bytes=1 << 30)
    a.update(kw)
    return m2.lib().mamba2_gated_scan_backward(ctypes.byref(d) if d is not None else None,
                                               *list(a.values()), None)


def _step(d, **kw):
    a = dict(lam=A0, x=A0 + 0x1000, lx=64, r=A0 + 0x2000, lr=64, g=A0 + 0x3000, lg=64, z=None, lz=0,
             y=A0 + 0x4000, h=A0 + 0x5000)
    a.update(kw)
    return m2.lib().mamba2_gated_scan_step(ctypes.byref(d) if d is not None else None,
                                           *list(a.values()), None)


@pytest.mark.parametrize("kw,want", BAD_DIMS)
def test_bad_dims(kw, want):
    d = _dims(**kw)
    assert _prefill(d) == want and _backward(d) == want
    if "seqlen" not in kw:
        assert _step(d) == want
    for packed in (0, 1):
        assert m2.mamba2_gated_scan_workspace_size(d, packed) == 0
        assert m2.mamba2_gated_scan_backward_workspace_size(d, packed) == 0
        assert m2.lib().mamba2_gated_scan_checkpoint_count(ctypes.byref(d), packed) == 0


def test_limits_count_rows_not_sequences():
    # 4096 sequences in a packed row of 131072 tokens are one row of tiles
    d = _dims(batch=4096, seqlen=131072, width=5120)
    sizes = (m2.mamba2_gated_scan_workspace_size, m2.mamba2_gated_scan_backward_workspace_size)
    for f in sizes:
        assert f(d, True) > 0 and f(d, False) == 0
    assert m2.lib().mamba2_gated_scan_checkpoint_count(ctypes.byref(d), 1) == 8192 * 5120
    ld = dict(lx=5120, lr=5120, lg=5120)
    assert _prefill(d, cu=A0 + 0x9000, bytes=0, **ld) == WORKSPACE
    assert _backward(d, cu=A0 + 0x9000, bytes=0, **ld) == WORKSPACE
    assert _prefill(d, **ld) == UNSUPPORTED and _backward(d, **ld) == UNSUPPORTED
    # the most tiles, and one more
    most = _dims(batch=(1 << 30) - 1, seqlen=1, width=32)
    assert sizes[0](most) == 0  # (sequences are fewer than 2^29)
    for batch, ok in (((1 << 29) - 1, True), (1 << 29, False)):
        assert (sizes[0](_dims(batch=batch, seqlen=64, width=64)) > 0) == ok
    for seqlen, ok in (((1 << 31) - 128, True), ((1 << 31) - 1, False)):
        assert (sizes[0](_dims(batch=1, seqlen=seqlen, width=1024)) > 0) == ok
    # products that pass 64 bits
    d = _dims(batch=1 << 28, seqlen=(1 << 31) - 64, width=1 << 20)
    assert sizes[0](d) == 0 and sizes[1](d) == 0
    assert _prefill(d, lx=1 << 20, lr=1 << 20, lg=1 << 20) == UNSUPPORTED


def test_sizes():
    assert m2.lib().mamba2_gated_scan_checkpoint_count(ctypes.byref(_dims()), 0) == 2 * 19 * 64
    assert m2.lib().mamba2_gated_scan_checkpoint_count(ctypes.byref(_dims()), 1) == 19 * 64
    assert m2.lib().mamba2_gated_scan_checkpoint_count(ctypes.byref(_dims(seqlen=0)), 0) == 0
    small, large = _dims(seqlen=4096), _dims(seqlen=32768)
    for f in (m2.mamba2_gated_scan_workspace_size, m2.mamba2_gated_scan_backward_workspace_size):
        assert 0 < f(small) < f(large)
    assert m2.gated_scan_checkpoints(_dims(), device="cpu").shape == (2, 19, 64)
    assert m2.gated_scan_checkpoints(_dims(), packed=True, device="cpu").shape == (1, 19, 64)


SHARED = [dict(lam=None), dict(lam=A0 + 2), dict(x=None), dict(r=None), dict(g=None),
          dict(x=A0 + 8), dict(lx=56), dict(lx=68), dict(lg=8), dict(z=A0 + 0x100, lz=32)]


@pytest.mark.parametrize("kw", SHARED + [dict(y=None), dict(y=A0 + 2), dict(h=A0 + 4), dict(sin=2),
                                         dict(h=None, sin=1), dict(ck=A0 + 4), dict(cu=A0 + 2)])
def test_prefill_refuses(kw):
    assert _prefill(_dims(), **kw) == INVALID


@pytest.mark.parametrize("kw", SHARED + [dict(dy=None), dict(dy=A0 + 2), dict(dx=None), dict(dr=A0 + 8),
                                         dict(dg=None), dict(dlam=None), dict(dlam=A0 + 1),
                                         dict(z=A0 + 0x100, lz=64), dict(dz=A0 + 0x100),
                                         dict(hin=A0 + 4), dict(dh=A0 + 4), dict(dhin=A0 + 8),
                                         dict(ck=A0 + 8), dict(cu=A0 + 2)])
def test_backward_refuses(kw):
    assert _backward(_dims(), **kw) == INVALID


@pytest.mark.parametrize("kw", SHARED + [dict(y=None), dict(y=A0 + 4), dict(h=None), dict(h=A0 + 8)])
def test_step_refuses(kw):
    assert _step(_dims(), **kw) == INVALID


def test_workspaces_and_empty_calls():
    d = _dims()
    for call, size in ((_prefill, m2.mamba2_gated_scan_workspace_size(d)),
                       (_backward, m2.mamba2_gated_scan_backward_workspace_size(d))):
        assert call(d, ws=None) == WORKSPACE
        assert call(d, ws=A0 + 0x10010) == WORKSPACE
        assert call(d, bytes=size - 1) == WORKSPACE
        assert call(None) == INVALID
    # packed rows need a sequence for their tokens
    assert _prefill(_dims(batch=0), cu=A0) == INVALID
    assert _backward(_dims(batch=0), cu=A0) == INVALID
    # nothing to do
    assert _prefill(_dims(batch=0), x=None, r=None, g=None, y=None, ws=None) == OK
    assert _prefill(_dims(seqlen=0), x=None, r=None, g=None, y=None, h=None, ws=None) == OK
    assert _step(_dims(batch=0), x=None, r=None, g=None, y=None, h=None) == OK


def _cache(load, **kw):
    a = dict(batch=3, row=100, nslots=4, block=64, format=0, state_dtype=0, state=A0, ld=100,
             slots=A0 + 0x1000, codes=A0 + 0x2000, scales=A0 + 0x3000)
    a.update(kw)
    d = m2.Mamba2StateCacheDims(*[a[k] for k in ("batch", "row", "nslots", "block", "format",
                                                  "state_dtype")])
    if load:
        return m2.lib().mamba2_state_cache_load(ctypes.byref(d), a["codes"], a["scales"],
                                                a["slots"], a["state"], a["ld"], None)
    return m2.lib().mamba2_state_cache_store(ctypes.byref(d), a["state"], a["ld"], a["slots"],
                                             a["codes"], a["scales"], None)


@pytest.mark.parametrize("load", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), INVALID), (dict(row=0), INVALID), (dict(nslots=-1), INVALID),
    (dict(format=2), INVALID), (dict(state_dtype=3), INVALID), (dict(block=16), UNSUPPORTED),
    (dict(block=0), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(state=None), INVALID),
    (dict(state=A0 + 2), INVALID), (dict(ld=99), INVALID), (dict(slots=None), INVALID),
    (dict(slots=A0 + 2), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID),
    (dict(batch=0, state=None, slots=None), OK),
])
def test_state_cache_refuses(load, kw, want):
    assert _cache(load, **kw) == want
