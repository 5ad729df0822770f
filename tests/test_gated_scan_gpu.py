"""GPU parity of the gated scan against its fp64 oracle (oracle/gated_scan.py).

Tolerances: an fp32 result may be off by the oracle's own running error bound (every
factor off by KAPPA half-steps of fp32, carried through the recurrence); a bf16 result by
that, plus half a step of bf16 (2^-8 of the value).
"""
import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_scan_mixer_b200 as m2
from oracle import gated_scan as GS

pytestmark = pytest.mark.gpu

C = 8.0
TINY = 1e-30  # a bound of zero still allows a flushed subnormal


def _inputs(rows, L, D, seed, dtype, gated, spread=1.0, lam=None):
    """rows None: [L, D]; else [rows, L, D].  x, r, g, z are columns of one buffer."""
    gen = torch.Generator().manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    lead = (L,) if rows is None else (rows, L)
    k = 4 if gated else 3
    proj = spread * torch.randn(*lead, k * D, generator=gen)
    proj = proj.clamp(-8, 8).to(dt).cuda()
    v = {n: proj[..., i * D:(i + 1) * D] for i, n in enumerate(("x", "r", "g", "z")[:k])}
    v.setdefault("z", None)
    v["dy"] = torch.randn(*lead, D, generator=gen).to(dt).cuda()
    if lam is None:
        u = 0.9 + 0.099 * torch.rand(D, generator=gen)
        lam = torch.log(torch.expm1(-torch.log(u) / C))
    v["lam"] = lam.float().cuda()
    return v


def _states(batch, D, seed):
    gen = torch.Generator().manual_seed(seed + 77)
    return torch.randn(batch, D, generator=gen).cuda(), torch.randn(batch, D, generator=gen).cuda()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _sequences(v, lens, packed):
    """The oracle's inputs of each sequence."""
    p = 0
    for i, n in enumerate(lens):
        at = (slice(p, p + n),) if packed else (i,)
        yield i, at, {k: (None if v[k] is None else _np(v[k][at])) for k in ("x", "r", "g", "z", "dy")}
        p += n


def _check(got, want, off, what, bf16=False):
    g = _np(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if not want.size:
        return
    allow = off + TINY + (np.abs(want) * 2.0 ** -8 * (1 + 2.0 ** -8) + off * 2.0 ** -8 if bf16 else 0.0)
    bad = ~(np.abs(g - want) <= allow)
    worst = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / allow, 0)), want.shape)
    assert not bad.any(), (what, int(bad.sum()), worst, g[worst], want[worst], allow[worst])


def _run(v, lens, D, dtype, packed, h0, dh, checkpoints=True):
    batch = len(lens)
    L = sum(lens) if packed else lens[0]
    dims = m2.make_gated_scan_dims(batch, L, D, io_dtype=dtype, decay_scale=C)
    cu = None
    if packed:
        cu = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32, device="cuda")
    h = torch.full((batch, D), 7.0, device="cuda") if h0 is None else h0.clone()
    ck = m2.gated_scan_checkpoints(dims, packed) if checkpoints else None
    y = m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], z=v["z"], h_state=h,
                              states_in=h0 is not None, cu_seqlens=cu, checkpoints=ck)
    gr = m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], z=v["z"],
                                h_state_in=h0, d_h_state_out=dh, cu_seqlens=cu, checkpoints=ck)
    torch.cuda.synchronize()
    assert m2.device_errors() == 0
    return y, h, gr


def _compare(v, lens, dtype, packed, h0, dh, y, h, gr):
    bf = dtype == "bf16"
    lam = _np(v["lam"])
    dlam, dlam_off = np.zeros_like(lam), np.zeros_like(lam)
    for i, at, o in _sequences(v, lens, packed):
        start = None if h0 is None else _np(h0[i])
        f = GS.forward(lam, o["x"], o["r"], o["g"], o["z"], start, C)
        _check(y[at], f["y"], f["y_off"], f"y of sequence {i}", bf)
        _check(h[i], f["h_end"], f["h_end_off"], f"final state {i}")
        b = GS.backward(lam, o["x"], o["r"], o["g"], o["dy"], o["z"], start,
                        None if dh is None else _np(dh[i]), C)
        for k in ("x", "r", "g") + (("z",) if o["z"] is not None else ()):
            _check(gr[k][at], b[k], b[k + "_off"], f"d{k} of sequence {i}", bf)
        if h0 is not None:
            _check(gr["h_state"][i], b["h0"], b["h0_off"], f"dh0 {i}")
        dlam += b["lam"]
        dlam_off += b["lam_off"]
    _check(gr["lam"], dlam, dlam_off, "dlam")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,D,states", [
    (1, 1, 8, True), (3, 2, 8, False), (2, 15, 64, True), (1, 16, 72, False), (2, 17, 136, True),
    (5, 31, 24, True), (1, 64, 64, False), (2, 127, 40, True), (1, 128, 200, True),
    (3, 129, 64, False), (2, 255, 128, True), (1, 257, 512, True), (2, 1000, 96, True),
    (1, 2049, 64, True), (1, 5000, 40, False),
])
def test_matches_oracle(batch, L, D, states, dtype, gated):
    v = _inputs(batch, L, D, 1000 * L + D, dtype, gated)
    h0, dh = _states(batch, D, L) if states else (None, None)
    y, h, gr = _run(v, [L] * batch, D, dtype, False, h0, dh)
    _compare(v, [L] * batch, dtype, False, h0, dh, y, h, gr)


PACKS = [
    [1], [5, 0, 3], [0, 0, 1, 0], [127, 1, 128, 0, 1, 1, 255], [128, 128, 128], [300, 1, 0, 700, 41],
    [1] * 150, [2, 3] * 70, [2047, 1, 2100], [0] * 40 + [9] + [0] * 300 + [200],
]


@pytest.mark.parametrize("dtype,gated", [("f32", True), ("bf16", False)])
@pytest.mark.parametrize("lens", PACKS, ids=lambda l: f"{len(l)}x{sum(l)}")
def test_packed_rows_match_oracle(lens, dtype, gated):
    D = 72
    v = _inputs(None, sum(lens), D, len(lens), dtype, gated)
    h0, dh = _states(len(lens), D, 5)
    y, h, gr = _run(v, lens, D, dtype, True, h0, dh)
    _compare(v, lens, dtype, True, h0, dh, y, h, gr)
    y, h, gr = _run(v, lens, D, dtype, True, None, None)
    _compare(v, lens, dtype, True, None, None, y, h, gr)


@pytest.mark.parametrize("packed", [False, True])
def test_backward_without_checkpoints_is_the_same(packed):
    lens = [700, 1, 0, 450] if packed else [700, 700]
    D = 136
    v = _inputs(None if packed else 2, sum(lens) if packed else 700, D, 3, "bf16", True)
    h0, dh = _states(len(lens), D, 9)
    _, _, a = _run(v, lens, D, "bf16", packed, h0, dh, checkpoints=True)
    _, _, b = _run(v, lens, D, "bf16", packed, h0, dh, checkpoints=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_gates_and_decays(dtype):
    # gates from nearly shut to wide open, decays from none to immediate
    D = 64
    lam = torch.linspace(-30, 12, D)
    v = _inputs(2, 200, D, 4, dtype, True, spread=4.0, lam=lam)
    h0, dh = _states(2, D, 6)
    y, h, gr = _run(v, [200, 200], D, dtype, False, h0, dh)
    _compare(v, [200, 200], dtype, False, h0, dh, y, h, gr)


@pytest.mark.parametrize("dtype,gated", [("f32", False), ("bf16", True)])
def test_wide_decays_in_packed_rows(dtype, gated):
    D, lens = 72, [3, 400, 1, 0, 130, 129, 16]
    lam = torch.linspace(-30, 12, D)
    v = _inputs(None, sum(lens), D, 50, dtype, gated, spread=4.0, lam=lam)
    h0, dh = _states(len(lens), D, 51)
    y, h, gr = _run(v, lens, D, dtype, True, h0, dh)
    _compare(v, lens, dtype, True, h0, dh, y, h, gr)


@pytest.mark.parametrize("dtype,gated,lo", [("f32", True, -5.0), ("bf16", False, -5.0),
                                            ("bf16", True, 3.0)])
@pytest.mark.parametrize("L", [17, 64])
def test_short_rows_of_a_large_batch(L, dtype, gated, lo):
    # enough threads for a row each; decays near one and far from it
    D, batch = 1096, 120
    lam = lo + torch.rand(D, generator=torch.Generator().manual_seed(1))
    v = _inputs(batch, L, D, 52, dtype, gated, lam=lam)
    h0, dh = _states(batch, D, 53)
    y, h, gr = _run(v, [L] * batch, D, dtype, False, h0, dh)
    _compare(v, [L] * batch, dtype, False, h0, dh, y, h, gr)


def test_shut_gates_keep_the_state_exactly():
    # r = -inf at padded tokens: the state passes through, nothing is NaN, forwards and back
    D, L = 40, 300
    v = _inputs(2, L, D, 5, "f32", False)
    r = v["r"].clone()
    r[:, 100:] = -float("inf")
    v["r"] = r
    h0, dh = _states(2, D, 7)
    v["dy"][:, 100:] = 0
    y, h, gr = _run(v, [L, L], D, "f32", False, h0, dh)
    # within the tile of 128 tokens in which the last live token lies, the state is put together
    # from parts (rounded, and compared below); from the next tile on it is the same number
    assert torch.equal(y[:, 128:], y[:, 128:129].expand(-1, L - 128, -1))
    assert torch.equal(h, y[:, 128])
    short = {k: (t if t is None or k == "lam" else t[:, :100].contiguous()) for k, t in v.items()}
    y2, h2, gr2 = _run(short, [100, 100], D, "f32", False, h0, dh)
    for k in ("x", "r", "g"):
        assert torch.count_nonzero(gr[k][:, 100:]) == 0, k
        assert torch.isfinite(gr[k]).all(), k
    _compare(v, [L, L], "f32", False, h0, dh, y, h, gr)


@pytest.mark.parametrize("far", [90.0, float("inf")])
def test_open_and_shut_extremes_stay_finite(far):
    D, L = 32, 140
    v = _inputs(1, L, D, 8, "f32", True)
    for k, sign in (("r", 1), ("g", -1)):
        t = v[k].clone()
        t[:, ::3] = sign * far
        t[:, 1::3] = -sign * far
        v[k] = t
    h0, dh = _states(1, D, 8)
    y, h, gr = _run(v, [L], D, "f32", False, h0, dh)
    for t in (y, h, *gr.values()):
        assert torch.isfinite(t).all()
    if far < 100:
        # gates of e^-90 and less: only their being finite and next to nothing is asked
        _check(y[0], *[GS.forward(_np(v["lam"]), *[_np(v[k][0]) for k in ("x", "r", "g", "z")],
                                  _np(h0[0]), C)[k] for k in ("y", "y_off")], "y")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_broken_sequence_stays_alone(bad):
    # packed rows: what one sequence holds never reaches another, not even through a zero
    D, lens = 24, [100, 60, 1, 200]
    v = _inputs(None, sum(lens), D, 11, "f32", False)
    x = v["x"].clone()
    x[150] = bad      # sequence 1
    v["x"] = x
    h0, dh = _states(4, D, 1)
    y, h, gr = _run(v, lens, D, "f32", True, h0, dh)
    assert not torch.isfinite(y[150:160]).any()
    clean = dict(v)
    clean["x"] = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    y2, h2, gr2 = _run(clean, lens, D, "f32", True, h0, dh)
    for sl in (slice(0, 100), slice(160, None)):
        assert torch.equal(y[sl], y2[sl])
        for k in ("x", "r", "g"):
            assert torch.equal(gr[k][sl], gr2[k][sl]), k
    for i in (0, 2, 3):
        assert torch.equal(h[i], h2[i])
        assert torch.equal(gr["h_state"][i], gr2["h_state"][i])


def test_nan_passes_on_within_its_sequence():
    D, L = 16, 400
    v = _inputs(2, L, D, 12, "f32", False)
    for k in ("x", "r", "g"):
        w = dict(v)
        w[k] = v[k].clone()
        w[k][0, 37, 3] = float("nan")
        y, h, _ = _run(w, [L, L], D, "f32", False, None, None)
        assert torch.isnan(y[0, 37:, 3]).all() and torch.isnan(h[0, 3]), k
        assert torch.isfinite(y[0, :37]).all() and torch.isfinite(y[1]).all(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,D,gated", [(1, 8, False), (1, 5120, True), (3, 72, True),
                                           (257, 264, False), (1000, 40, True)])
def test_step_matches_oracle(batch, D, gated, dtype):
    v = _inputs(None, batch, D, 13, dtype, gated)
    h0, _ = _states(batch, D, 2)
    h = h0.clone()
    dims = m2.make_gated_scan_dims(batch, 0, D, io_dtype=dtype, decay_scale=C)
    y = m2.gated_scan_step(dims, v["lam"], v["x"], v["r"], v["g"], h, z=v["z"])
    torch.cuda.synchronize()
    f = [GS.forward(_np(v["lam"]), *[None if v[k] is None else _np(v[k][i:i + 1])
                                     for k in ("x", "r", "g", "z")], _np(h0[i]), C)
         for i in range(batch)]
    cat = lambda k: np.concatenate([q[k] for q in f])  # noqa: E731
    _check(y, cat("y"), cat("y_off"), "y", dtype == "bf16")
    _check(h, cat("h"), cat("h_off"), "h")


def test_prefill_in_pieces_and_steps_go_on_from_the_state():
    # the serving run: a prompt in two pieces, then single tokens; against the oracle's one run
    D, L, n = 136, 333, 5
    v = _inputs(2, L + n, D, 14, "f32", True)
    sub = lambda p, q: [v[k][:, p:q].contiguous() for k in ("x", "r", "g", "z")]  # noqa: E731
    h = torch.empty(2, D, device="cuda")
    out, p = [], 0
    for q in (200, L):
        dims = m2.make_gated_scan_dims(2, q - p, D, io_dtype="f32", decay_scale=C)
        x, r, g, z = sub(p, q)
        out.append(m2.gated_scan_prefill(dims, v["lam"], x, r, g, z=z, h_state=h, states_in=p > 0))
        p = q
    dims = m2.make_gated_scan_dims(2, 1, D, io_dtype="f32", decay_scale=C)
    for t in range(L, L + n):
        # single tokens as views of the long buffer
        x, r, g, z = (v[k][:, t] for k in ("x", "r", "g", "z"))
        out.append(m2.gated_scan_step(dims, v["lam"], x, r, g, h, z=z)[:, None])
    y = torch.cat(out, 1)
    for i in range(2):
        f = GS.forward(_np(v["lam"]), *[_np(v[k][i]) for k in ("x", "r", "g", "z")], None, C)
        _check(y[i], f["y"], f["y_off"], "y")
        _check(h[i], f["h_end"], f["h_end_off"], "h")


def test_single_token_rows_of_any_batch_stride():
    D = 64
    v = _inputs(3, 6, D, 15, "bf16", False)
    one = [v[k][:, 2:3] for k in ("x", "r", "g")]  # [3, 1, D], batch stride six tokens
    dims = m2.make_gated_scan_dims(3, 1, D)
    a = m2.gated_scan_prefill(dims, v["lam"], *one)
    b = m2.gated_scan_prefill(dims, v["lam"], *[t.contiguous() for t in one])
    assert torch.equal(a, b)


def test_no_tokens():
    D = 16
    e = torch.empty(2, 0, D, device="cuda")
    lam = torch.zeros(D, device="cuda")
    dims = m2.make_gated_scan_dims(2, 0, D, io_dtype="f32")
    h = torch.full((2, D), 3.0, device="cuda")
    assert m2.gated_scan_prefill(dims, lam, e, e, e, h_state=h, states_in=True).shape == (2, 0, D)
    assert (h == 3).all()
    m2.gated_scan_prefill(dims, lam, e, e, e, h_state=h)
    assert (h == 0).all()
    dh = torch.randn(2, D, device="cuda")
    gr = m2.gated_scan_backward(dims, lam, e, e, e, e, h_state_in=h, d_h_state_out=dh)
    assert torch.equal(gr["h_state"], dh) and (gr["lam"] == 0).all()
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    e = e[0]
    gr = m2.gated_scan_backward(dims, lam, e, e, e, e, h_state_in=h, d_h_state_out=dh, cu_seqlens=cu)
    assert torch.equal(gr["h_state"], dh) and (gr["lam"] == 0).all()
    none = m2.make_gated_scan_dims(0, 5, D, io_dtype="f32")
    e = torch.empty(0, 5, D, device="cuda")
    assert m2.gated_scan_prefill(none, lam, e, e, e).shape == (0, 5, D)


@pytest.mark.parametrize("cu", [[0, 300, 200, 600], [1, 300, 500, 600], [0, 300, 500, 599],
                                [0, 300, 500, 601], [0, -5, 500, 600], [0, 300, 2 ** 31 - 1, 600]])
def test_bad_offsets_write_nothing(cu):
    D, L = 40, 600
    v = _inputs(None, L, D, 16, "f32", True)
    dims = m2.make_gated_scan_dims(3, L, D, io_dtype="f32")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h = torch.full((3, D), 5.0, device="cuda")
    y = torch.full((L, D), 6.0, device="cuda")
    m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], z=v["z"], h_state=h,
                          states_in=True, cu_seqlens=c, y=y)
    assert m2.device_errors() == 4
    assert (h == 5).all() and (y == 6).all()
    for ck in (None, m2.gated_scan_checkpoints(dims, True)):
        m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], z=v["z"],
                               h_state_in=h, cu_seqlens=c, checkpoints=ck)
        assert m2.device_errors() == 4
    # the next call is an ordinary one
    _compare(v, [100, 0, 500], "f32", True, h, None, *_run(v, [100, 0, 500], D, "f32", True, h, None))


def test_workspace_contents_and_repeats_do_not_matter():
    D, L = 264, 3000
    v = _inputs(1, L, D, 17, "bf16", True)
    h0, dh = _states(1, D, 3)
    dims = m2.make_gated_scan_dims(1, L, D)
    first = None
    for fill in (0, 1, 0x7f, 0xff):
        ws = torch.full((m2.mamba2_gated_scan_workspace_size(dims),), fill, dtype=torch.uint8,
                        device="cuda")
        wb = torch.full((m2.mamba2_gated_scan_backward_workspace_size(dims),), fill,
                        dtype=torch.uint8, device="cuda")
        for _ in range(3):
            h = h0.clone()
            y = m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], z=v["z"], h_state=h,
                                      states_in=True, workspace=ws)
            gr = m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], z=v["z"],
                                        h_state_in=h0, d_h_state_out=dh, workspace=wb)
            now = [y, h, *gr.values()]
            first = first or now
            assert all(torch.equal(a, b) for a, b in zip(first, now))
    assert m2.device_errors() == 0


def test_two_streams_and_graphs():
    D, L = 520, 2500
    dims = m2.make_gated_scan_dims(1, L, D)
    vs = [_inputs(1, L, D, 20 + i, "bf16", False) for i in range(2)]
    h0, dh = _states(1, D, 4)

    def call(v, stream=None):
        h = h0.clone()
        ck = m2.gated_scan_checkpoints(dims)
        y = m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], h_state=h,
                                  states_in=True, checkpoints=ck, stream=stream)
        gr = m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], h_state_in=h0,
                                    d_h_state_out=dh, checkpoints=ck, stream=stream)
        return [y, h, *gr.values()]

    want = [call(v) for v in vs]
    torch.cuda.synchronize()
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in vs]
    got = []
    for v, s in zip(vs, streams):
        with torch.cuda.stream(s):
            got.append([call(v, s) for _ in range(4)])
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))
    # captured, and replayed on new inputs
    live = {k: (t.clone() if t is not None else None) for k, t in vs[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(live)
    for v, w in ((vs[1], want[1]), (vs[0], want[0]), (vs[1], want[1])):
        for k, t in live.items():
            if t is not None:
                t.copy_(v[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(w, out))
    assert m2.device_errors() == 0


def test_a_named_stream_orders_what_the_call_allocates():
    D, L = 64, 700
    v = _inputs(1, L, D, 30, "f32", False)
    dims = m2.make_gated_scan_dims(1, L, D, io_dtype="f32")
    want = m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream, 0):
        got = m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], stream=st)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_offsets_beyond_32_bits():
    # rows far apart in one large buffer: 64 tokens, 2^26 elements between them
    D, L, stride = 64, 40, 1 << 26
    big = torch.empty(L * stride, dtype=torch.bfloat16, device="cuda")
    v = _inputs(None, L, D, 31, "bf16", False)
    far = {}
    for i, k in enumerate(("x", "r", "g")):
        far[k] = big[i * 4096:].as_strided((1, L, D), (L * stride, stride, 1))
        far[k].copy_(v[k][None])
    dims = m2.make_gated_scan_dims(1, L, D)
    got = m2.gated_scan_prefill(dims, v["lam"], far["x"], far["r"], far["g"])
    want = m2.gated_scan_prefill(dims, v["lam"], *[v[k][None].contiguous() for k in ("x", "r", "g")])
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_does_not_depend_on_its_batch(dtype):
    # the same numbers whatever else is in the call, forwards and back
    D, L = 72, 1500
    v = _inputs(5, L, D, 40, dtype, True)
    h0, dh = _states(5, D, 41)
    y, h, gr = _run(v, [L] * 5, D, dtype, False, h0, dh)
    for i in (0, 3):
        one = {k: (t if t is None or k == "lam" else t[i:i + 1].contiguous()) for k, t in v.items()}
        y1, h1, gr1 = _run(one, [L], D, dtype, False, h0[i:i + 1], dh[i:i + 1])
        assert torch.equal(y1[0], y[i]) and torch.equal(h1[0], h[i])
        for k in ("x", "r", "g", "z", "h_state"):
            assert torch.equal(gr1[k][0], gr[k][i]), k


def test_nan_of_any_payload():
    # blocks tell by a NaN pattern what has not been written yet: no input may look like it
    D, L = 40, 1000
    v = _inputs(1, L, D, 42, "f32", False)
    bad = torch.tensor([-1], dtype=torch.int32, device="cuda").view(torch.float32)[0]
    h0, dh = _states(1, D, 43)
    for k in ("x", "r", "g", "dy", "h0", "dh", "lam"):
        w, s, e = dict(v), h0.clone(), dh.clone()
        if k == "h0":
            s.fill_(bad)
        elif k == "dh":
            e.fill_(bad)
        else:
            w[k] = v[k].clone().fill_(bad)
        y, h, gr = _run(w, [L], D, "f32", False, s, e)  # (no wait ran out)
        assert torch.isnan(gr["h_state"]).all() if k in ("dh", "dy", "r", "lam") else True
        if k in ("x", "r", "g", "h0", "lam"):
            assert torch.isnan(y).all() and torch.isnan(h).all(), k


def test_sums_over_many_partial_ones():
    # lam's gradient over more tiles than one round of its sum takes
    D, batch = 8, 1500
    v = _inputs(batch, 20, D, 54, "f32", False)
    y, h, gr = _run(v, [20] * batch, D, "f32", False, None, None)
    _compare(v, [20] * batch, "f32", False, None, None, y, h, gr)


def test_a_long_row():
    D, L = 8, 70001
    v = _inputs(1, L, D, 44, "f32", False)
    h0, dh = _states(1, D, 45)
    y, h, gr = _run(v, [L], D, "f32", False, h0, dh)
    _compare(v, [L], "f32", False, h0, dh, y, h, gr)


def test_more_sequences_than_65535():
    D, n = 8, 70000
    v = _inputs(None, n, D, 46, "f32", False)
    h0, dh = _states(n, D, 47)
    y, h, gr = _run(v, [1] * n, D, "f32", True, h0, dh)
    # single tokens: the recurrence once, for all of them side by side
    lam = _np(v["lam"])
    R, G, la, a, m = GS._gates(lam, _np(v["r"]), _np(v["g"]), C)
    want = a * _np(h0) + m * G * _np(v["x"])
    off = 2 * GS.KAPPA * GS.U * (a * np.abs(_np(h0)) + m * G * np.abs(_np(v["x"])))
    _check(y, want, off, "y")
    _check(h, want, off, "h")
    d = _np(v["dy"]) + _np(dh)
    _check(gr["h_state"], a * d, 3 * GS.KAPPA * GS.U * a * (np.abs(_np(v["dy"])) + np.abs(_np(dh))),
           "dh0")


@pytest.mark.parametrize("dtype,gated", [("f32", False), ("bf16", True)])
def test_sequences_times_tokens_beyond_the_tiles(dtype, gated):
    # as one packed row they are few tiles, as rows of all tokens they would pass 2^30
    D, n = 64, 200000
    assert n * (n // 64) * (D // 32) >= 1 << 30
    v = _inputs(None, n, D, 48, dtype, gated)
    h0, dh = _states(n, D, 49)
    y, h, gr = _run(v, [1] * n, D, dtype, True, h0, dh)
    # single tokens: one token of n * D channels
    lam = np.tile(_np(v["lam"]), n)
    one = lambda t: None if t is None else _np(t).reshape(1, -1)
    ins = [one(v[k]) for k in ("x", "r", "g")]
    f = GS.forward(lam, *ins, one(v["z"]), one(h0)[0], C)
    bf = dtype == "bf16"
    _check(y.reshape(1, -1), f["y"], f["y_off"], "y", bf)
    _check(h.reshape(-1), f["h_end"], f["h_end_off"], "h")
    b = GS.backward(lam, *ins, one(v["dy"]), one(v["z"]), one(h0)[0], one(dh)[0], C)
    for k in ("x", "r", "g") + (("z",) if gated else ()):
        _check(gr[k].reshape(1, -1), b[k], b[k + "_off"], f"d{k}", bf)
    _check(gr["h_state"].reshape(-1), b["h0"], b["h0_off"], "dh0")
    _check(gr["lam"], b["lam"].reshape(n, D).sum(0), b["lam_off"].reshape(n, D).sum(0), "dlam")


def test_waits_that_run_out_are_reported():
    D, L = 200, 900
    v = _inputs(2, L, D, 48, "bf16", True)
    h0, dh = _states(2, D, 49)
    assert m2.device_errors() == 0
    dims = m2.make_gated_scan_dims(2, L, D)
    m2.debug_stall_waits(True)
    try:
        y = torch.full((2, L, D), 3.0, device="cuda", dtype=torch.bfloat16)
        m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], z=v["z"], y=y)
        assert m2.device_errors() & 1
        assert (y == 3).all()
        ck = m2.gated_scan_checkpoints(dims).zero_()
        m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], z=v["z"],
                               checkpoints=ck)
        assert m2.device_errors() & 1
    finally:
        m2.debug_stall_waits(False)
    assert m2.device_errors() == 0
    _compare(v, [L, L], "bf16", False, h0, dh, *_run(v, [L, L], D, "bf16", False, h0, dh))


def test_binding_refuses_what_does_not_fit():
    D, L = 32, 10
    v = _inputs(2, L, D, 32, "bf16", False)
    dims = m2.make_gated_scan_dims(2, L, D)
    ok = [v["lam"], v["x"], v["r"], v["g"]]

    def refused(match, *args, **kw):
        with pytest.raises(ValueError, match=match):
            m2.gated_scan_prefill(dims, *args, **kw)

    refused("lam", v["lam"].double(), *ok[1:])
    refused("lam", v["lam"].cpu(), *ok[1:])
    refused("x", ok[0], v["x"].float(), *ok[2:])
    refused("r", ok[0], ok[1], v["r"][:, :5], ok[3])
    refused("g", *ok[:3], v["g"].cpu())
    refused("g", *ok[:3], v["g"].transpose(1, 2).contiguous().transpose(1, 2))
    refused("batch stride", *ok[:3], _inputs(2, L + 1, D, 1, "bf16", False)["g"][:, :L])
    refused("z", *ok, z=v["x"][:1])
    refused("h_state", *ok, h_state=torch.zeros(2, D, device="cuda", dtype=torch.bfloat16))
    refused("h_state", *ok, h_state=torch.zeros(1, D, device="cuda"))
    refused("cu_seqlens", ok[0], *[t.reshape(-1, D)[:L] for t in (t.contiguous() for t in ok[1:])],
            cu_seqlens=torch.zeros(3, dtype=torch.int64, device="cuda"))
    refused("checkpoints", *ok, checkpoints=torch.zeros(2, 2, D, device="cuda"))
    refused("y", *ok, y=torch.zeros(2, L, D, device="cuda"))
    with pytest.raises(m2.Mamba2Error, match="invalid argument"):
        m2.gated_scan_prefill(dims, *ok, states_in=True)
    with pytest.raises(m2.Mamba2Error, match="workspace"):
        m2.gated_scan_prefill(dims, *ok, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(2 * L * D * 3 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, L, 3 * D)
    with pytest.raises(m2.Mamba2Error, match="invalid argument"):
        m2.gated_scan_prefill(dims, ok[0], odd[..., :D], *ok[2:])
    with pytest.raises(m2.Mamba2Error, match="unsupported"):
        w = 12
        m2.gated_scan_prefill(m2.make_gated_scan_dims(2, L, w), torch.zeros(w, device="cuda"),
                              *[torch.zeros(2, L, w, device="cuda", dtype=torch.bfloat16)] * 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
def test_many_tiles_a_step_match_oracle(dtype, gated):
    # 24 tiles of a step and more: states are put together from the one eight tiles back
    batch, L, D = 8, 3000, 136
    v = _inputs(batch, L, D, 60, dtype, gated)
    h0, dh = _states(batch, D, 61)
    y, h, gr = _run(v, [L] * batch, D, dtype, False, h0, dh)
    _compare(v, [L] * batch, dtype, False, h0, dh, y, h, gr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("lens", [[3000], [1300, 0, 1, 1500, 199]], ids=["one", "five"])
def test_many_tiles_a_step_of_packed_rows_match_oracle(lens, dtype, gated):
    D = 800
    v = _inputs(None, sum(lens), D, 62, dtype, gated)
    h0, dh = _states(len(lens), D, 63)
    y, h, gr = _run(v, lens, D, dtype, True, h0, dh)
    _compare(v, lens, dtype, True, h0, dh, y, h, gr)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gated", [False, True])
def test_the_same_bits_from_eight_tiles_back_and_from_further(dtype, gated):
    # nine rows look eight tiles back, one row of them 32: bit for bit the same
    D, L, batch = 72, 2600, 9
    v = _inputs(batch, L, D, 64, dtype, gated)
    h0, dh = _states(batch, D, 65)
    y, h, gr = _run(v, [L] * batch, D, dtype, False, h0, dh)
    for i in (0, 4, 8):
        one = {k: (t if t is None or k == "lam" else t[i:i + 1].contiguous()) for k, t in v.items()}
        y1, h1, gr1 = _run(one, [L], D, dtype, False, h0[i:i + 1], dh[i:i + 1])
        assert torch.equal(y1[0], y[i]) and torch.equal(h1[0], h[i])
        for k in ("x", "r", "g", "h_state") + (("z",) if gated else ()):
            assert torch.equal(gr1[k][0], gr[k][i]), k


@pytest.mark.parametrize("recompute", [False, True])
@pytest.mark.parametrize("cu", [[0, 0, 200, 100, 600], [0, 0, 300, 500, 599], [1, 1, 300, 500, 600]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bad_offsets_leave_every_output(cu, dtype, recompute):
    # (an empty sequence before the wrong offset: its state is written before any tile runs)
    D, L, n = 40, 600, 4
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    v = _inputs(None, L, D, 66, dtype, True)
    dims = m2.make_gated_scan_dims(n, L, D, io_dtype=dtype, decay_scale=C)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    h0, dh = _states(n, D, 67)
    for states_in in (False, True):
        h = torch.full((n, D), 5.0, device="cuda")
        y = torch.full((L, D), 6.0, device="cuda", dtype=dt)
        ck = m2.gated_scan_checkpoints(dims, True).fill_(7.0)
        m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], z=v["z"], h_state=h,
                              states_in=states_in, cu_seqlens=c, checkpoints=ck, y=y)
        assert m2.device_errors() == 4
        assert (h == 5).all() and (y == 6).all() and (ck == 7).all()
    outs = {k: torch.full((L, D), 8.0, device="cuda", dtype=dt) for k in ("x", "r", "g", "z")}
    outs["lam"] = torch.full((D,), 8.0, device="cuda")
    outs["h"] = torch.full((n, D), 8.0, device="cuda")
    size = m2.mamba2_gated_scan_backward_workspace_size(dims, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    rows = [a for k in ("x", "r", "g", "z") for a in (v[k].data_ptr(), v[k].stride(0))]
    st = m2.lib().mamba2_gated_scan_backward(
        ctypes.byref(dims), v["lam"].data_ptr(), *rows, c.data_ptr(), h0.data_ptr(),
        v["dy"].data_ptr(), dh.data_ptr(), None if recompute else ck.data_ptr(),
        *[outs[k].data_ptr() for k in ("x", "r", "g", "z", "lam", "h")], ws.data_ptr(), size,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0 and m2.device_errors() == 4
    for k, t in outs.items():
        assert (t == 8).all(), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,L,D,gated,h,d", [
    (2, 1, 72, False, True, True), (3, 16, 72, True, False, True), (2, 16, 40, False, True, False),
    (120, 64, 1096, True, True, False), (120, 33, 1096, False, False, False),
    (2, 700, 136, False, False, True), (2, 700, 136, True, False, False),
])
def test_backward_without_checkpoints(batch, L, D, gated, h, d, dtype):
    # the scan run again inside the call, short rows among them, with and without each state
    v = _inputs(batch, L, D, 68, dtype, gated)
    h0, dh = _states(batch, D, 69)
    h0, dh = h0 if h else None, dh if d else None
    y, h1, a = _run(v, [L] * batch, D, dtype, False, h0, dh, checkpoints=True)
    _, _, b = _run(v, [L] * batch, D, dtype, False, h0, dh, checkpoints=False)
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k
    _compare(v, [L] * batch, dtype, False, h0, dh, y, h1, b)


@pytest.mark.parametrize("h,d", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("dtype,gated", [("f32", True), ("bf16", False)])
def test_packed_backward_without_checkpoints(dtype, gated, h, d):
    lens, D = [5, 0, 300, 1, 130, 16], 72
    v = _inputs(None, sum(lens), D, 70, dtype, gated)
    h0, dh = _states(len(lens), D, 71)
    h0, dh = h0 if h else None, dh if d else None
    y, h1, a = _run(v, lens, D, dtype, True, h0, dh, checkpoints=True)
    _, _, b = _run(v, lens, D, dtype, True, h0, dh, checkpoints=False)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    _compare(v, lens, dtype, True, h0, dh, y, h1, b)


@pytest.mark.parametrize("lam", [-6.0, -1.0, 2.0], ids=["near", "wide", "wider"])
def test_gradients_of_saturated_gates(lam):
    """Gates from nearly shut to fully open: the gradients of r and g go with 1 - R and 1 - G, and
    are as exact, relative to themselves, as everything else.

    One token from a zero state, so that nothing cancels: dg = dy m x G (1 - G) and
    dr = -dy (a^2 / m) G x la (1 - R).  In half-steps of fp32, with KAPPA for a factor as in the
    oracle: m G x has KAPPA; 1 - G = e^-g G has twice |g| (the exponential's argument: the
    constant and the product) and 8 (the exponential, the sum, the reciprocal and the product), and
    KAPPA for G.  dr has b = m G x, a^2 by a KAPPA (1 + |la|) each, 1 / (1 - a^2) and la by a KAPPA
    each, and 1 - R as above.  |la| <= 8 * 2.2.  dx = dy m G has KAPPA."""
    D, n = 512, 40
    gen = torch.Generator().manual_seed(72)
    draw = lambda: (40 * torch.rand(n, 1, D, generator=gen) - 20).cuda()  # noqa: E731
    r, g = draw(), draw()
    x = torch.randn(n, 1, D, generator=gen).cuda()
    dy = torch.randn(n, 1, D, generator=gen).cuda()
    lam = torch.full((D,), lam).cuda()
    dims = m2.make_gated_scan_dims(n, 1, D, io_dtype="f32", decay_scale=C)
    gr = m2.gated_scan_backward(dims, lam, x, r, g, dy)
    rd, gd, ld, xd, dd = (_np(t) for t in (r, g, lam, x, dy))
    R, G, la, a, m = GS._gates(ld, rd, gd, C)
    shut_r, shut_g = 1 / (1 + np.exp(rd)), 1 / (1 + np.exp(gd))  # 1 - R, 1 - G
    want = {"x": dd * m * G, "g": dd * m * xd * G * shut_g,
            "r": -dd * a * a / m * G * xd * la * shut_r}
    K = GS.KAPPA
    off = {"x": K, "g": 2 * K + 2 * np.abs(gd) + 8,
           "r": (3 + 2 * (1 - la)) * K + K + 2 * np.abs(rd) + 8}
    for k, w in want.items():
        _check(gr[k], w, off[k] * GS.U * np.abs(w) + 1e-37, f"d{k}")


def test_equal_short_rows_are_equal_whatever_their_place():
    """Rows of 36 channel pairs share warps with their neighbours in the kernel of short rows; which
    arithmetic a decay takes must not depend on who else is in the warp.  Decays whose exponent is
    within steps of the border of -1/2 (lam a step of fp32 after the other), gates fully open, and
    eight channels far beyond it."""
    D, L, n = 72, 16, 64
    lam = np.full(D, 3.0, np.float32)
    at = np.float32(0.3)
    c = np.float32(0.5 / (np.log1p(np.exp(np.float64(at))) * np.log2(np.e)))
    for i in range(64):
        lam[i] = at + np.float32(2.0 ** -25 * (i - 32))
    gen = torch.Generator().manual_seed(73)
    row = lambda f: f(torch.randn(1, L, D, generator=gen)).expand(n, L, D).contiguous().cuda()  # noqa: E731
    x, g = row(lambda t: t), row(lambda t: t)
    r = row(lambda t: 20 + t)
    h0 = torch.randn(1, D, generator=gen).expand(n, D).contiguous().cuda()
    dims = m2.make_gated_scan_dims(n, L, D, io_dtype="f32", decay_scale=float(c))
    lam = torch.from_numpy(lam).cuda()
    h = h0.clone()
    y = m2.gated_scan_prefill(dims, lam, x, r, g, h_state=h, states_in=True)
    assert torch.equal(y, y[:1].expand_as(y))
    assert torch.equal(h, h[:1].expand_as(h))
    # and as single tokens
    s = h0.clone()
    one = m2.make_gated_scan_dims(n, 1, D, io_dtype="f32", decay_scale=float(c))
    for t in range(L):
        yt = m2.gated_scan_step(one, lam, *[v[:, t].contiguous() for v in (x, r, g)], s)
        assert torch.equal(yt, y[:, t]), t
    assert torch.equal(s, h)


@pytest.mark.parametrize("batch,L,D", [(1, 6000, 64), (8, 2500, 104)])
def test_long_memories(batch, L, D):
    # decays of 0.99 to 0.9995 and inputs of one sign, against bounds counted rounding by rounding
    gen = torch.Generator().manual_seed(74)
    pos = lambda *s: torch.randn(*s, generator=gen).abs().cuda()  # noqa: E731
    gate = lambda: (1 + 0.5 * torch.randn(batch, L, D, generator=gen)).clamp(-4, 4).cuda()  # noqa: E731
    v = {"x": pos(batch, L, D), "r": gate(), "g": gate(), "z": None, "dy": pos(batch, L, D)}
    u = torch.linspace(0.99, 0.9995, D, dtype=torch.float64)
    v["lam"] = torch.log(torch.expm1(-torch.log(u) / C)).float().cuda()
    h0, dh = pos(batch, D), pos(batch, D)
    y, h, gr = _run(v, [L] * batch, D, "f32", False, h0, dh)
    lam = _np(v["lam"])
    for i in range(batch):
        x, r, g, dy = (_np(v[k][i]) for k in ("x", "r", "g", "dy"))
        off = GS.memory_bounds(lam, x, r, g, _np(h0[i]), dy, _np(dh[i]), C)
        f = GS.forward(lam, x, r, g, None, _np(h0[i]), C)
        b = GS.backward(lam, x, r, g, dy, None, _np(h0[i]), _np(dh[i]), C)
        _check(y[i], f["h"], off["h_off"], f"y of row {i}")
        _check(h[i], f["h_end"], off["h_off"][-1], f"final state {i}")
        _check(gr["x"][i], b["x"], off["x_off"], f"dx of row {i}")
        _check(gr["h_state"][i], b["h0"], off["h0_off"], f"dh0 of row {i}")


@pytest.mark.parametrize("packed", [False, True])
def test_infinite_states_stay_in_their_channel(packed):
    # (a tile's decays multiply to zero, and zero times infinity is NaN: not finite is all that
    # holds for the channel itself)
    D, lens = 40, [500, 3, 397]
    lam = torch.linspace(-3, 6, D)
    v = _inputs(None, sum(lens), D, 75, "f32", False, lam=lam)
    if not packed:
        v = {k: (t if t is None or k == "lam" else t[None]) for k, t in v.items()}
        lens = [900]
    h0, dh = _states(len(lens), D, 76)
    y, h, gr = _run(v, lens, D, "f32", packed, h0, dh)
    bad = h0.clone()
    bad[0, ::4] = float("inf")
    y2, h2, gr2 = _run(v, lens, D, "f32", packed, bad, dh)
    own = torch.zeros(D, dtype=torch.bool, device="cuda")
    own[::4] = True
    one, two = (t.reshape(-1, D) for t in (y, y2))
    n = lens[0]
    assert not torch.isfinite(two[:n, own]).any() and not torch.isfinite(h2[0, own]).any()
    assert torch.equal(one[:n, ~own], two[:n, ~own]) and torch.equal(one[n:], two[n:])
    assert torch.equal(h[0, ~own], h2[0, ~own]) and torch.equal(h[1:], h2[1:])
    for k in ("x", "g", "r"):
        assert torch.equal(gr[k].reshape(-1, D)[:, ~own], gr2[k].reshape(-1, D)[:, ~own]), k
        assert torch.equal(gr[k].reshape(-1, D)[n:], gr2[k].reshape(-1, D)[n:]), k


def test_a_captured_fork_and_join():
    # two prompts on two streams of one capture, copies before them and a cache and a step behind
    # the join; replayed on other inputs, against the same calls made one by one
    D, L = 136, 900
    dims = m2.make_gated_scan_dims(1, L, D)
    one = m2.make_gated_scan_dims(2, 1, D)
    sets = [[_inputs(1, L, D, 80 + 2 * i + k, "bf16", False) for k in range(2)] for i in range(2)]
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def run(ins, fork):
        main = torch.cuda.current_stream()
        other = side if fork else main
        h, back = torch.zeros(2, D, device="cuda"), torch.zeros(2, D, device="cuda")
        codes, scales = m2.state_cache(2, D)
        other.wait_stream(main)
        ys = []
        for k, s in ((0, main), (1, other)):
            with torch.cuda.stream(s):
                v = {n: t.clone() for n, t in ins[k].items() if n in ("lam", "x", "r", "g")}
                ys.append(m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"],
                                                h_state=h[k:k + 1]))
        main.wait_stream(other)
        m2.state_cache_store(h, slots, codes, scales)
        m2.state_cache_load(codes, scales, slots, back)
        last = [torch.cat([ins[k][n][:, -1] for k in range(2)]) for n in ("x", "r", "g")]
        ys.append(m2.gated_scan_step(one, ins[0]["lam"], *last, back))
        return [*ys, h, back]

    want = [run(s, False) for s in sets]
    torch.cuda.synchronize()
    live = [{n: (None if t is None else t.clone()) for n, t in v.items()} for v in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(live, True)
    for i in (1, 0, 1):
        for a, b in zip(live, sets[i]):
            for n, t in a.items():
                if t is not None:
                    t.copy_(b[n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[i], out)), i
    assert m2.device_errors() == 0


@pytest.mark.parametrize("D", [8, 1000, 1024, 1032, 5120])
def test_empty_sequences_hand_their_states_on(D):
    # a copy of d_h_state_out in pieces of a row; with states_in false the state is zero
    lens = [0, 5, 0, 0, 70, 0]
    v = _inputs(None, sum(lens), D, 90, "f32", False)
    h0, dh = _states(len(lens), D, 91)
    y, h, gr = _run(v, lens, D, "f32", True, h0, dh)
    zero = _run(v, lens, D, "f32", True, None, None)[1]
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(h[i], h0[i]) and torch.equal(gr["h_state"][i], dh[i]), i
            assert torch.count_nonzero(zero[i]) == 0, i


def test_an_empty_sequence_costs_next_to_nothing():
    # (one warp that copied a row's state 32 channels after the other took 0.33 ms here)
    D, L = 65536, 64
    v = _inputs(None, L, D, 92, "bf16", False)
    dims = m2.make_gated_scan_dims(2, L, D)
    h0, dh = _states(2, D, 93)
    ck = m2.gated_scan_checkpoints(dims, True)

    def took(cu):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        best = float("inf")
        for _ in range(10):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(5):
                m2.gated_scan_backward(dims, v["lam"], v["x"], v["r"], v["g"], v["dy"], h_state_in=h0,
                                       d_h_state_out=dh, cu_seqlens=c, checkpoints=ck)
            e[1].record()
            torch.cuda.synchronize()
            best = min(best, e[0].elapsed_time(e[1]) / 5 * 1000)
        return best

    m2.gated_scan_prefill(dims, v["lam"], v["x"], v["r"], v["g"], h_state=h0.clone(), states_in=True,
                          cu_seqlens=torch.tensor([0, 30, L], dtype=torch.int32, device="cuda"),
                          checkpoints=ck)
    full, empty = took([0, 30, L]), took([0, 0, L])
    assert empty < full + 200, (empty, full)
