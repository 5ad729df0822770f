"""What the gated linear recurrence and the 8-bit state cache are measured on.

The recurrence keeps one fp32 state per channel.  With s = softplus(lam),
R = sigmoid(r), G = sigmoid(g):

    a_t = exp(-c s R_t)      h_t = a_t h_{t-1} + sqrt(1 - a_t^2) G_t x_t      y_t = h_t [silu(z_t)]

The state cache holds recurrent states as 8-bit codes (int8 or e4m3) with a
power-of-two scale for each block of consecutive values.

Kinds of case: "prefill" (many tokens, y and the final state), "step" (one
token for each sequence, the state updated in place), "train" (forward and
backward), "write" (states into slots of the cache, and read back) and "read"
(slots into working states).
"""
import math

import torch

own = False

C = 8.0  # decay scale of every case


def listed():
    return [
        # one 4096-token prompt at the 2.7B mixer's inner width
        {"name": "prefill_2p7b", "kind": "prefill", "batch": 1, "seqlen": 4096, "width": 5120,
         "dtype": "bf16", "gated": False, "packed": False, "states_in": False},
        # a long document at the 7B width, continued from a carried state, with the output gate
        {"name": "prefill_7b_long", "kind": "prefill", "batch": 1, "seqlen": 32768, "width": 7168,
         "dtype": "bf16", "gated": True, "packed": False, "states_in": True},
        # requests of different lengths served together, empty and one-token ones among them
        {"name": "prefill_packed", "kind": "prefill", "batch": 13, "seqlen": 8191, "width": 4096,
         "dtype": "bf16", "gated": False, "packed": True, "states_in": True},
        # the smallest configuration: latency
        {"name": "prefill_tiny_f32", "kind": "prefill", "batch": 1, "seqlen": 256, "width": 64,
         "dtype": "f32", "gated": False, "packed": False, "states_in": True},
        # decode of 256 sequences, and of one (latency)
        {"name": "step_b256", "kind": "step", "batch": 256, "width": 5120, "dtype": "bf16",
         "gated": True},
        {"name": "step_b1", "kind": "step", "batch": 1, "width": 5120, "dtype": "bf16",
         "gated": False},
        # training steps: one long row, a batch with the output gate, an odd fp32 size in packed rows
        {"name": "train_2p7b", "kind": "train", "batch": 1, "seqlen": 4096, "width": 5120,
         "dtype": "bf16", "gated": False, "packed": False, "states_in": False},
        {"name": "train_1p2b_gated", "kind": "train", "batch": 8, "seqlen": 2048, "width": 4096,
         "dtype": "bf16", "gated": True, "packed": False, "states_in": False},
        {"name": "train_packed_f32", "kind": "train", "batch": 7, "seqlen": 1723, "width": 1000,
         "dtype": "f32", "gated": False, "packed": True, "states_in": True},
        # every SSM state of a 256-sequence decode batch put aside in 8 bits and taken back
        {"name": "write_2p7b_int8", "kind": "write", "batch": 256, "slots": 300, "row": 80 * 64 * 64,
         "block": 64, "codes": "int8", "dtype": "f32"},
        # conv states (bf16, 5248 channels of 4) of a few sequences
        {"name": "write_conv_e4m3", "kind": "write", "batch": 11, "slots": 64, "row": 5248 * 4,
         "block": 32, "codes": "e4m3", "dtype": "bf16"},
        # a shared prefix's state given to new sequences
        {"name": "read_7b_e4m3", "kind": "read", "batch": 40, "slots": 16, "row": 112 * 64 * 64,
         "block": 128, "codes": "e4m3", "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "step", "train", "train", "write", "read"])
    if kind in ("write", "read"):
        row = _log_int(rng, 500, 500_000)
        return {"kind": kind, "batch": min(_log_int(rng, 1, 512), max(1, 80_000_000 // row)),
                "slots": 520, "row": row, "block": rng.choice([32, 64, 128]),
                "codes": rng.choice(["int8", "e4m3"]), "dtype": rng.choice(["f32", "bf16"])}
    width = 8 * _log_int(rng, 8, 1024)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    gated = rng.random() < 0.4
    if kind == "step":
        return {"kind": kind, "batch": _log_int(rng, 1, 1024), "width": width, "dtype": dtype,
                "gated": gated}
    most = (120_000_000 if kind == "prefill" else 30_000_000) // width  # tokens
    seqlen = _log_int(rng, 1, min(32768, most))
    packed = rng.random() < 0.35
    batch = _log_int(rng, 1, 40) if packed else _log_int(rng, 1, max(1, min(64, most // seqlen)))
    return {"kind": kind, "batch": batch, "seqlen": seqlen, "width": width, "dtype": dtype,
            "gated": gated, "packed": packed, "states_in": rng.random() < 0.5}


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _type(case)
    randn = lambda *s, t=dt: torch.randn(*s, generator=gen, device="cuda", dtype=t)  # noqa: E731
    if case["kind"] in ("write", "read"):
        return _prepare_cache(case, gen, dt)
    b, D = case["batch"], case["width"]
    rows = (b,) if case["kind"] == "step" else ((1 if case["packed"] else b), case["seqlen"])
    k = 4 if case["gated"] else 3
    # x, r, g (and z) are columns of one projection's output, as a layer has them
    proj = randn(*rows, k * D)
    if case.get("packed"):
        proj = proj[0]
    s = {"kind": case["kind"], "case": case}
    for i, name in enumerate(("x", "r", "g", "z")[:k]):
        s[name] = proj[..., i * D:(i + 1) * D]
    s.setdefault("z", None)
    # decays a in [0.9, 0.999] at an open gate: the range such layers are initialised to
    u = 0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda")
    s["lam"] = torch.log(torch.expm1(-torch.log(u) / C))
    s["cu"] = None
    if case.get("packed"):
        cuts = torch.randint(0, case["seqlen"] + 1, (b - 1,), generator=gen, device="cuda")
        if b > 4:
            cuts[1] = cuts[0]                                   # an empty sequence
            cuts[3] = (cuts[2] + 1).clamp(max=case["seqlen"])   # and one of a single token
        ends = torch.tensor([0, case["seqlen"]], device="cuda")
        s["cu"] = torch.cat([cuts, ends]).sort().values.to(torch.int32)
    if case["kind"] == "train":
        s["dy"] = randn(*s["x"].shape)
        s["h0"] = randn(b, D, t=torch.float32) if case["states_in"] else None
        s["dh"] = randn(b, D, t=torch.float32) if case["states_in"] else None
    else:
        s["h"] = randn(b, D, t=torch.float32)
    return s


def _prepare_cache(case, gen, dt):
    b, n, blk = case["batch"], case["row"], case["block"]
    # values of a state differ in size from head to head; some rows of it are still zero
    blocks = -(-n // blk)
    size = torch.exp(torch.randn(b, blocks, 1, generator=gen, device="cuda") - 2)
    size *= torch.rand(b, blocks, 1, generator=gen, device="cuda") > 0.02
    state = torch.randn(b, blocks, blk, generator=gen, device="cuda") * size
    state = state.reshape(b, blocks * blk)[:, :n].to(dt).contiguous()
    s = {"kind": case["kind"], "case": case}
    slots = case["slots"]
    s["codes"] = torch.zeros(slots, n, device="cuda",
                             dtype=torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn)
    s["scales"] = torch.zeros(slots, blocks, device="cuda", dtype=torch.uint8)
    if case["kind"] == "write":
        s["slots"] = torch.randperm(slots, generator=gen, device="cuda")[:b].to(torch.int32)
        if b > 4:
            s["slots"][3] = -1  # a row of the batch that holds no sequence
        s["state"] = state
        s["out"] = torch.zeros(b, n, device="cuda", dtype=dt)
    else:
        q = torch.randn(slots, n, generator=gen, device="cuda") * 40
        s["codes"] = q.clamp(-127, 127).round().to(torch.int8) if case["codes"] == "int8" else q.to(
            torch.float8_e4m3fn)
        s["scales"] = torch.randint(110, 125, (slots, blocks), generator=gen, device="cuda",
                                    dtype=torch.uint8)
        s["slots"] = torch.randint(0, slots, (b,), generator=gen, device="cuda", dtype=torch.int32)
        s["out"] = torch.zeros(b, n, device="cuda", dtype=dt)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return {"prefill": _prefill, "step": _step, "train": _train, "write": _write,
            "read": _read}[s["kind"]](s)


def _dims(m2, s):
    c = s["case"]
    return m2.make_gated_scan_dims(c["batch"], c.get("seqlen", 1), c["width"],
                                   io_dtype=c["dtype"], decay_scale=C)


def _prefill(s):
    c = s["case"]
    if own:
        import mamba_ssd_scan_mixer_b200 as m2
        y = m2.gated_scan_prefill(_dims(m2, s), s["lam"], s["x"], s["r"], s["g"], z=s["z"],
                                  h_state=s["h"], states_in=c["states_in"], cu_seqlens=s["cu"])
    else:
        y, h_end = _forward(s, s["h"] if c["states_in"] else None)[:2]
        s["h"].copy_(h_end)
    return {"y": y, "h": s["h"]}


def _step(s):
    if own:
        import mamba_ssd_scan_mixer_b200 as m2
        y = m2.gated_scan_step(_dims(m2, s), s["lam"], s["x"], s["r"], s["g"], s["h"], z=s["z"])
    else:
        a, m, _, _, G = _gates(s)
        h = a * s["h"] + m * G * s["x"].float()
        y = (h if s["z"] is None else h * _silu(s["z"].float())).to(s["x"].dtype)
        s["h"].copy_(h)
    return {"y": y, "h": s["h"]}


def _train(s):
    """Forward, then the gradients for the dy that the loss gave back."""
    if own:
        import mamba_ssd_scan_mixer_b200 as m2
        dims = _dims(m2, s)
        ck = m2.gated_scan_checkpoints(dims, packed=s["cu"] is not None, device=s["x"].device)
        h = None if s["h0"] is None else s["h0"].clone()
        y = m2.gated_scan_prefill(dims, s["lam"], s["x"], s["r"], s["g"], z=s["z"], h_state=h,
                                  states_in=h is not None, cu_seqlens=s["cu"], checkpoints=ck)
        grads = m2.gated_scan_backward(dims, s["lam"], s["x"], s["r"], s["g"], s["dy"], z=s["z"],
                                       h_state_in=s["h0"], d_h_state_out=s["dh"],
                                       cu_seqlens=s["cu"], checkpoints=ck)
        if s["cu"] is not None and s["z"] is not None:
            grads["z"] = grads["z"][None]  # laid out as the plain form gives it: one row
        return {"y": y, **{"d_" + k: v for k, v in grads.items()}}
    y, _, h, h_prev, first, last = _forward(s, s["h0"])
    a, m, la, R, G = _gates(s)
    x, dy, dt = s["x"].float(), s["dy"].float(), s["x"].dtype
    out = {"y": y}
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        out["d_z"] = (dy * h * sig * (1 + z * (1 - sig))).to(dt)
        dy = dy * z * sig
    dy = dy.reshape(h.shape).clone()
    if s["dh"] is not None:
        dy[last[0], last[1]] += s["dh"][last[2]]
    # d_t = dy_t + a_{t+1} d_{t+1}; nothing comes back across a sequence's first token
    back = torch.zeros_like(h)
    back[:, :-1] = a.reshape(h.shape)[:, 1:]
    if s["cu"] is not None:
        inner = first[1] > 0
        back[first[0][inner], first[1][inner] - 1] = 0
    d = _scan(back.flip(1), dy.flip(1)).flip(1)
    if s["h0"] is not None:
        dh0 = s["dh"].clone()
        dh0[first[2]] = (a.reshape(h.shape) * d)[first[0], first[1]]
        out["d_h_state"] = dh0
    d = d.reshape(x.shape)
    out["d_x"] = (d * m * G).to(dt)
    out["d_g"] = (d * m * x * G * (1 - G)).to(dt)
    per_m = torch.where(m > 0, 1 / m, torch.zeros_like(m))
    d_la = d * (a * h_prev.reshape(x.shape) - a * a * per_m * G * x)
    out["d_r"] = (d_la * la * (1 - R)).to(dt)
    dl = (d_la * R).reshape(-1, x.shape[-1]).sum(0, dtype=torch.float64)
    out["d_lam"] = (-C * torch.sigmoid(s["lam"].double()) * dl).float()
    return out


def _write(s):
    """States into their slots, and back: what 8 bits hold is returned as the values it stands for."""
    blk = s["case"]["block"]
    if own:
        import mamba_ssd_scan_mixer_b200 as m2
        m2.state_cache_store(s["state"], s["slots"], s["codes"], s["scales"], block=blk)
        m2.state_cache_load(s["codes"], s["scales"], s["slots"], s["out"], block=blk)
    else:
        used = s["slots"] >= 0
        codes, scales = _quantise(s["state"][used].float(), blk, s["codes"].dtype)
        at = s["slots"][used].long()
        s["codes"].view(torch.uint8)[at] = codes.view(torch.uint8)
        s["scales"][at] = scales
        _take(s, at, used)
    return {"state": s["out"], "scales": s["scales"]}


def _read(s):
    if own:
        import mamba_ssd_scan_mixer_b200 as m2
        m2.state_cache_load(s["codes"], s["scales"], s["slots"], s["out"], block=s["case"]["block"])
    else:
        used = s["slots"] >= 0
        _take(s, s["slots"][used].long(), used)
    return {"state": s["out"]}


# ------------------------------------------------------------------ plain forms (fp32)

def _silu(v):
    return v * torch.sigmoid(v)


def _gates(s):
    """a, sqrt(1 - a^2), log a, R, G."""
    R, G = torch.sigmoid(s["r"].float()), torch.sigmoid(s["g"].float())
    # softplus in 64 bits: for very negative lam it is tiny and multiplies everything
    la = -C * torch.log1p(torch.exp(s["lam"].double())).float() * R
    return torch.exp(la), torch.sqrt(-torch.expm1(2 * la)), la, R, G


def _ends(s):
    """(row, position, sequence) of every non-empty sequence's first and last token."""
    if s["cu"] is not None:
        cu = s["cu"].long()
        seq = torch.nonzero(cu[1:] > cu[:-1])[:, 0]
        row = torch.zeros_like(seq)
        return (row, cu[:-1][seq], seq), (row, cu[1:][seq] - 1, seq)
    b, L = s["x"].shape[:2]
    seq = torch.arange(b, device=s["x"].device)
    return (seq, torch.zeros_like(seq), seq), (seq, torch.full_like(seq, L - 1), seq)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 (h_{-1} = 0), by doubling spans."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _forward(s, h0):
    a, m, _, _, G = _gates(s)
    b = m * G * s["x"].float()
    shape = b.shape
    if s["cu"] is not None:
        a, b = a[None], b[None]
    first, last = _ends(s)
    batch = s["case"]["batch"]
    start = torch.zeros(batch, shape[-1], device=b.device) if h0 is None else h0
    # a sequence's first token takes nothing from the token before it
    b[first[0], first[1]] += a[first[0], first[1]] * start[first[2]]
    a = a.clone()
    a[first[0], first[1]] = 0
    h = _scan(a, b)
    h_prev = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    h_prev[first[0], first[1]] = start[first[2]]
    h_end = start.clone()  # a sequence without tokens keeps its state
    h_end[last[2]] = h[last[0], last[1]]
    y = h.reshape(shape)
    y = (y if s["z"] is None else y * _silu(s["z"].float())).to(s["x"].dtype)
    return y, h_end, h, h_prev, first, last


def _power(byte):
    """2^(byte - 127), exactly."""
    bits = torch.where(byte == 0, 0x00400000, byte.to(torch.int32) << 23)
    return bits.to(torch.int32).view(torch.float32)


def _quantise(v, blk, codes):
    """Codes and biased exponents: the least power of two that keeps a block within the codes."""
    b, n = v.shape
    pad = -n % blk
    t = torch.nn.functional.pad(v, (0, pad)).reshape(b, -1, blk)
    amax = t.abs().amax(-1)
    frac, ex = torch.frexp(amax)  # amax = frac 2^ex, frac in [1/2, 1)
    if codes == torch.int8:
        e = ex - 7 + (frac > 127 / 128).int()
    else:
        e = ex - 9 + (frac > 448 / 512).int()
    byte = torch.where(amax > 0, (e + 127).clamp(min=0), 0)
    byte = torch.where(torch.isfinite(amax), byte, 255)
    q = t / _power(byte)[..., None]
    q = q.reshape(b, n + pad)[:, :n].contiguous()
    q = torch.where(torch.isfinite(q), q, 0)
    return (q.round().to(torch.int8) if codes == torch.int8 else q.to(codes)), byte.to(torch.uint8)


def _take(s, at, used):
    """Slots `at` of the cache into the rows `used` of the working states."""
    n, blk = s["case"]["row"], s["case"]["block"]
    codes = s["codes"].view(torch.uint8)[at].view(s["codes"].dtype).float()
    byte = s["scales"][at]
    scale = torch.where(byte == 255, math.nan, _power(byte)).repeat_interleave(blk, 1)[:, :n]
    s["out"][used] = (codes * scale).to(s["out"].dtype)


# ------------------------------------------------------------------ work and 64-bit values

def work(case):
    t = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("write", "read"):
        n = case["batch"] * case["row"]
        coded = n * (1 + 1 / case["block"])
        # writing: the state in, codes out; reading: codes in, the state out
        one = n * t + coded
        return {"bytes": one * (2 if case["kind"] == "write" else 1), "flops": 3.0 * n}
    D, b = case["width"], case["batch"]
    tokens = b if case["kind"] == "step" else case["seqlen"] * (1 if case["packed"] else b)
    n, z = tokens * D, int(case["gated"])
    state = b * D * 4 * (2 if case["kind"] == "step" or case["states_in"] else 1)
    forward = n * t * (4 + z) + state
    if case["kind"] != "train":
        return {"bytes": forward, "flops": 25.0 * n}
    # the backward call comes after the loss has given dy: it reads the inputs again
    return {"bytes": forward + n * t * (7 + 2 * z) + state, "flops": 75.0 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] in ("write", "read"):
        return _exact_cache(s, case)
    f = {k: s[k].double() for k in ("x", "r", "g", "z", "lam") if s[k] is not None}
    train = case["kind"] == "train"
    D = case["width"]
    if case["kind"] == "step":
        f = {k: (v if k == "lam" else v[:, None]) for k, v in f.items()}
        lens = [1] * case["batch"]
    elif case["packed"]:
        cu = s["cu"].tolist()
        lens = [q - p for p, q in zip(cu, cu[1:])]
    else:
        lens = [case["seqlen"]] * case["batch"]
    if train:
        for v in f.values():
            v.requires_grad_(True)
    a = torch.exp(-C * torch.nn.functional.softplus(f["lam"], threshold=100) * torch.sigmoid(f["r"]))
    b = torch.sqrt((1 - a) * (1 + a)) * torch.sigmoid(f["g"]) * f["x"]
    given = s.get("h0") if train else (s["h"] if case.get("states_in", True) else None)
    h0 = torch.zeros(case["batch"], D, device=b.device, dtype=torch.float64)
    h0 = h0 if given is None else given.double()
    if train:
        h0.requires_grad_(True)
    if case.get("packed"):  # sequence after sequence
        hs, ends, p = [], [], 0
        at, bt = a.unbind(0), b.unbind(0)
        for i, n in enumerate(lens):
            h = h0[i]
            for t in range(p, p + n):
                h = at[t] * h + bt[t]
                hs.append(h)
            ends.append(h)
            p += n
        h, h_end = torch.stack(hs), torch.stack(ends)
    else:
        hs, h = [], h0
        for at, bt in zip(a.unbind(1), b.unbind(1)):
            h = at * h + bt
            hs.append(h)
        h_end, h = h, torch.stack(hs, 1)
    y = h if s["z"] is None else h * torch.nn.functional.silu(f["z"])
    if not train:
        return {"y": y.reshape(s["x"].shape), "h": h_end}
    total = (y * s["dy"].double()).sum()
    if s["dh"] is not None:
        total = total + (h_end * s["dh"].double()).sum()
    total.backward()
    out = {"y": y.detach(), **{"d_" + k: v.grad for k, v in f.items()}}
    if s["h0"] is not None:
        out["d_h_state"] = h0.grad
    return out


def _exact_cache(s, case):
    """The values that the codes stand for, from the definition: every step below is exact in 64 bits."""
    n, blk, used = case["row"], case["block"], s["slots"] >= 0
    top, int8 = (127.0, True) if case["codes"] == "int8" else (448.0, False)
    out = torch.zeros(case["batch"], n, device="cuda", dtype=torch.float64)
    if case["kind"] == "read":
        unit = torch.exp2(s["scales"].double() - 127).repeat_interleave(blk, 1)[:, :n]
        return {"state": (s["codes"].double() * unit)[s["slots"].long()]}
    for i in torch.nonzero(used)[:, 0].tolist():
        v = torch.nn.functional.pad(s["state"][i].double(), (0, -n % blk)).reshape(-1, blk)
        amax = v.abs().amax(1, keepdim=True)
        e = torch.log2(amax.clamp(min=1e-30) / top).ceil()
        e = torch.where(amax <= top * torch.exp2(e - 1), e - 1, e)
        e = torch.where(amax > top * torch.exp2(e), e + 1, e).clamp(min=-127)
        q = v / torch.exp2(e)
        if not int8:  # e4m3: three bits after the leading one, none below 2^-9
            step = torch.exp2(torch.log2(q.abs().clamp(min=2.0 ** -6)).floor() - 3)
        else:
            step = torch.ones_like(q)
        out[i] = ((q / step).round() * step * torch.exp2(e)).reshape(-1)[:n]
    return {"state": out, "scales": None}
