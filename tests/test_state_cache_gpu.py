"""GPU tests of the 8-bit state cache.  Its definition is exact (power-of-two scales), so the
codes, scales and values are compared bit for bit with a plain fp64 form."""
import math

import numpy as np
import pytest
import torch

import mamba_ssd_scan_mixer_b200 as m2

pytestmark = pytest.mark.gpu


def _round_e4m3(q):
    a = np.abs(q)
    e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    step = 2.0 ** (e - 3)
    return np.sign(q) * np.round(a / step) * step


def _plain(state, block, codes):
    """Values and scale bytes of one fp64 state, block by block."""
    top = 127.0 if codes == "int8" else 448.0
    vals, scales = np.empty_like(state), []
    for i in range(0, len(state), block):
        v = state[i:i + block]
        if not np.isfinite(v).all():
            vals[i:i + block] = np.nan
            scales.append(255)
            continue
        e = -127
        while np.max(np.abs(v)) > top * 2.0 ** e:
            e += 1
        q = v / 2.0 ** e
        q = np.round(q) if codes == "int8" else _round_e4m3(q)
        vals[i:i + block] = q * 2.0 ** e
        scales.append(e + 127)
    return vals, scales


def _states(b, n, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(6 * torch.randn(b, -(-n // 32), 1, generator=g))
    size[torch.rand(size.shape, generator=g) < 0.1] = 0
    v = (torch.randn(b, size.shape[1], 32, generator=g) * size).reshape(b, -1)[:, :n]
    return v.to(torch.float32 if dtype == "f32" else torch.bfloat16).contiguous()


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("b,n,block", [(1, 1, 32), (2, 31, 32), (3, 33, 64), (4, 4096, 64),
                                       (2, 1000, 128), (5, 1023, 32), (2, 4100, 128), (3, 6, 128),
                                       (7, 5248 * 4, 32), (2, 16400, 64)])
def test_round_trip_is_exact(b, n, block, dtype, codes):
    state = _states(b, n, n + b, dtype)
    slots = torch.randperm(b + 3, generator=torch.Generator().manual_seed(b))[:b].int()
    q, sc = m2.state_cache(b + 3, n, block, codes)
    q.view(torch.uint8).fill_(0x55)
    sc.fill_(0x66)
    m2.state_cache_store(state.cuda(), slots.cuda(), q, sc, block=block)
    out = torch.full((b, n), 9.0, dtype=state.dtype, device="cuda")
    m2.state_cache_load(q, sc, slots.cuda(), out, block=block)
    torch.cuda.synchronize()
    assert m2.device_errors() == 0
    for i in range(b):
        vals, scales = _plain(state[i].double().numpy(), block, codes)
        assert sc[slots[i]].tolist() == scales, i
        assert np.array_equal(out[i].double().cpu().numpy(), vals), i
    left = [s for s in range(b + 3) if s not in slots.tolist()]
    assert (q.view(torch.uint8)[left] == 0x55).all() and (sc[left] == 0x66).all()
    # written again: the same values.  (For e4m3 the scale may halve: an amax just over
    # 224 2^e rounds to 224 2^e = 448 2^(e-1); every code then doubles, which is exact.)
    q2, sc2 = m2.state_cache(b + 3, n, block, codes)
    m2.state_cache_store(out, slots.cuda(), q2, sc2, block=block)
    again = torch.empty_like(out)
    m2.state_cache_load(q2, sc2, slots.cuda(), again, block=block)
    assert torch.equal(again, out)
    if codes == "int8":
        used = slots.long().cuda()
        assert torch.equal(q2[used], q[used]) and torch.equal(sc2[used], sc[used])


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_extremes(codes):
    top = 127.0 if codes == "int8" else 448.0
    n, block = 32 * 9, 32
    v = torch.zeros(9, 32)
    v[0, 3], v[1, 4], v[2, 5] = math.inf, -math.inf, math.nan
    v[3, :3] = torch.tensor([top, -top / 2, 0.4])
    v[4, :2] = torch.tensor([math.nextafter(top, 1e9), 1.0])   # just past the codes' range
    v[5, :4] = torch.tensor([3e38, -1e38, 1.0, 0.0])
    v[6, :3] = torch.tensor([1e-40, -3e-42, 1e-45])            # subnormal: the least scale
    v[7, :3] = torch.tensor([top, 0.5, 1.5])                   # ties go to the even code
    v[8, 0] = -0.0
    q, sc = m2.state_cache(1, n, block, codes)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    m2.state_cache_store(v.reshape(1, -1).cuda(), zero, q, sc, block=block)
    out = torch.empty(1, n, device="cuda")
    m2.state_cache_load(q, sc, zero, out, block=block)
    vals, scales = _plain(v.reshape(-1).double().numpy(), block, codes)
    assert sc[0].tolist() == scales
    assert np.array_equal(out[0].double().cpu().numpy(), vals, equal_nan=True)


def test_slots_skipped_repeated_and_out_of_range():
    n = 200
    state = _states(6, n, 1, "f32").cuda()
    q, sc = m2.state_cache(4, n)
    slots = torch.tensor([2, -1, 2, 0, 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    m2.state_cache_store(state, slots, q, sc)
    assert m2.device_errors() == 8
    alone, alone_sc = m2.state_cache(4, n)
    m2.state_cache_store(state[[2, 5]], torch.tensor([2, 0], dtype=torch.int32, device="cuda"), alone,
                         alone_sc)
    assert torch.equal(q, alone) and torch.equal(sc, alone_sc)  # the last of each slot's rows
    out = torch.full((6, n), 4.0, device="cuda")
    take = torch.tensor([2, 2, -7, 4, 0, 2], dtype=torch.int32, device="cuda")
    m2.state_cache_load(q, sc, take, out)
    assert m2.device_errors() == 8
    assert (out[2:4] == 4).all()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[5])
    assert not torch.equal(out[0], out[4])
    assert m2.device_errors() == 0


def test_many_rows_of_one_slot_the_last_counts():
    n, b = 96, 3000
    state = torch.arange(b, device="cuda").float()[:, None].expand(b, n).contiguous()
    slots = (torch.arange(b, device="cuda") % 7).int()
    q, sc = m2.state_cache(7, n, 32)
    m2.state_cache_store(state, slots, q, sc, block=32)
    ref, ref_sc = m2.state_cache(7, n, 32)
    m2.state_cache_store(state[-7:], slots[-7:], ref, ref_sc, block=32)
    assert torch.equal(q, ref) and torch.equal(sc, ref_sc)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off,extra", [(0, 0), (1, 3), (4, 8), (3, 1)])
def test_strided_and_unaligned_states(off, extra, dtype):
    b, n = 3, 640
    src = _states(b, n, 2, dtype).cuda()
    buf = torch.full((off + b * (n + extra),), 5.0, dtype=src.dtype, device="cuda")
    view = buf[off:].as_strided((b, n), (n + extra, 1))
    view.copy_(src)
    slots = torch.tensor([1, 0, 2], dtype=torch.int32, device="cuda")
    q, sc = m2.state_cache(3, n, codes="e4m3")
    q2, sc2 = m2.state_cache(3, n, codes="e4m3")
    m2.state_cache_store(view, slots, q, sc)
    m2.state_cache_store(src, slots, q2, sc2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(sc, sc2)
    out = torch.empty(b, n, dtype=src.dtype, device="cuda")
    m2.state_cache_load(q, sc, slots, out)
    before = buf.clone()
    m2.state_cache_load(q, sc, slots, view)
    assert torch.equal(view, out)
    view.copy_(src)
    assert torch.equal(buf, before)  # nothing between the rows was touched


def test_a_cache_beyond_32_bits():
    n, nslots = 1 << 20, 2100
    q, sc = m2.state_cache(nslots, n, 128, "e4m3")
    state = torch.randn(1, n, device="cuda")
    slot = torch.tensor([nslots - 1], dtype=torch.int32, device="cuda")
    m2.state_cache_store(state, slot, q, sc, block=128)
    out = torch.empty(1, n, device="cuda")
    m2.state_cache_load(q, sc, slot, out, block=128)
    assert (out - state).norm() < 0.05 * state.norm()
    assert torch.count_nonzero(q[:-1].view(torch.uint8)) == 0
    assert torch.count_nonzero(sc[:-1]) == 0


def test_prefill_store_load_step():
    """The serving run: a prompt's states put aside in 8 bits, taken up by two sequences, which
    then decode; against the same run with the values that the codes stand for."""
    from mamba_ssd_scan_mixer_b200 import workloads as W
    from harness import case, dev_params
    cfg = case("zamba2_2p7b_prefill", batch=1, seqlen=300, nheads=4)
    params = W.make_params(cfg, 3)
    keep, pp = dev_params(params)
    v = W.split_packed(cfg, W.make_prefill_inputs(cfg, 3)["zxbcdt"].cuda())
    cs = torch.zeros(1, cfg.conv_dim, 4, dtype=torch.bfloat16, device="cuda")
    hs = torch.zeros(1, cfg.nheads, 64, 64, device="cuda")
    m2.prefill(m2.dims_from_config(cfg), pp, v["xBC"], v["z"], v["dt_raw"], cs, hs)
    D = 128
    gen = torch.Generator().manual_seed(5)
    lam = torch.randn(D, generator=gen).cuda() - 4
    x, r, g = (torch.randn(1, 300, D, generator=gen).bfloat16().cuda() for _ in range(3))
    h = torch.empty(1, D, device="cuda")
    m2.gated_scan_prefill(m2.make_gated_scan_dims(1, 300, D), lam, x, r, g, h_state=h)
    caches = [m2.state_cache(3, t[0].numel(), codes="int8") for t in (hs, cs, h)]
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    for t, c in zip((hs, cs, h), caches):
        m2.state_cache_store(t, slot, *c)
    both = [t.new_empty(2, *t.shape[1:]) for t in (hs, cs, h)]
    for t, c in zip(both, caches):
        m2.state_cache_load(*c, slot.expand(2).contiguous(), t)
    for t, back in zip((hs, cs, h), both):
        flat = t.reshape(-1).double().cpu().numpy()
        vals, _ = _plain(flat, 64, "int8")
        for row in back:
            assert np.array_equal(row.reshape(-1).double().cpu().numpy(), vals)
    two = cfg.with_(batch=2)
    sv = W.split_packed(two, W.make_step_inputs(two, 3, 0)["zxbcdt"].cuda())
    want = [t.clone() for t in both]
    dims = m2.dims_from_config(two)
    y1 = m2.step(dims, pp, sv["xBC"], sv["z"], sv["dt_raw"], both[1], both[0])
    y2 = m2.step(dims, pp, sv["xBC"], sv["z"], sv["dt_raw"], want[1], want[0])
    assert torch.equal(y1, y2) and torch.isfinite(y1).all()
    gd = m2.make_gated_scan_dims(2, 1, D)
    xs = [torch.randn(2, D, generator=gen).bfloat16().cuda() for _ in range(3)]
    y1 = m2.gated_scan_step(gd, lam, *xs, both[2])
    y2 = m2.gated_scan_step(gd, lam, *xs, want[2])
    assert torch.equal(y1, y2) and torch.equal(both[2], want[2])
    assert m2.device_errors() == 0


def test_graph_replay():
    n = 4096
    q, sc = m2.state_cache(5, n)
    state = torch.randn(2, n, device="cuda")
    out = torch.zeros(2, n, device="cuda")
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    m2.state_cache_store(state, slots, q, sc)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m2.state_cache_store(state, slots, q, sc)
        m2.state_cache_load(q, sc, slots, out)
    for s in ([3, 2], [4, -1]):
        state.normal_()
        slots.copy_(torch.tensor(s))
        out.fill_(2.0)
        graph.replay()
        for i, k in enumerate(s):
            if k < 0:
                assert (out[i] == 2).all()
            else:
                vals, _ = _plain(state[i].double().cpu().numpy(), 64, "int8")
                assert np.array_equal(out[i].double().cpu().numpy(), vals)


def test_binding_refuses_what_does_not_fit():
    n = 64
    q, sc = m2.state_cache(4, n)
    state = torch.zeros(2, n, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")

    def refused(match, *a, **kw):
        with pytest.raises(ValueError, match=match):
            m2.state_cache_store(*a, **kw)

    refused("state", state.cpu(), slots, q, sc)
    refused("state", state.half(), slots, q, sc)
    refused("state", state[:, :60], slots, q, sc)
    refused("contiguous", torch.zeros(n, 2, device="cuda").t(), slots, q, sc)
    refused("codes", state, slots, q.int(), sc)
    refused("slots", state, slots.long(), q, sc)
    refused("slots", state, slots[:1], q, sc)
    refused("scales", state, slots, q, sc, block=32)
    refused("block", state, slots, q, sc, block=16)
    with pytest.raises(ValueError, match="codes"):
        m2.state_cache(4, n, codes="int4")
    m2.state_cache_store(state[:0], slots[:0], q, sc)  # nothing to do
