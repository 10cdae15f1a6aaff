"""What is timed of the elementwise recurrences and of their training.

Five operators: the gated scan (``ssd_gated_scan``), its backward pass
(``ssd_gated_scan_backward``), its one-token step (``ssd_gated_step``), a
training pass of it whose saved inputs are held in 8 bits, and the backward
pass of the diagonal selective scan (``ssd_selective_scan_backward``).

``run`` computes them in elementary torch operations, or, where ``own`` is
true, by the library's calls; ``exact`` in 64 bits, token after token.
"""
import math

import torch

own = False

GATE_C = 8.0  # the gate's power: a = exp(-c softplus(lam) sigmoid(r))
BLOCK = 64    # tokens for each saved state and each 8-bit scale


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _gated(name, op, b, L, D, dtype="bf16", reset=False, h0=False):
    return {"name": name, "op": op, "batch": b, "seqlen": L, "channels": D, "dtype": dtype,
            "reset": reset, "h0": h0}


def _scan(name, b, L, D, N, G, dtype="bf16", softplus=True, zoh=True, clamp=False, h0=False):
    return {"name": name, "op": "scan_backward", "batch": b, "seqlen": L, "channels": D,
            "dstate": N, "ngroups": G, "dtype": dtype, "softplus": softplus, "zoh": zoh,
            "clamp": clamp, "h0": h0}


def listed():
    return [
        # prefill of a 2.7B-style layer's 5120 channels
        _gated("gated_b8_l2048_d5120", "gated", 8, 2048, 5120),
        # one long document carried on from a state: few lanes, a long axis
        _gated("gated_b1_l65536_d2048", "gated", 1, 65536, 2048, h0=True),
        # a small packed batch in fp32, odd channel count and length, resets
        _gated("gated_b3_l777_d1001_f32", "gated", 3, 777, 1001, "f32", reset=True),
        # the training batch's backward pass
        _gated("gated_bwd_b8_l2048_d5120", "gated_backward", 8, 2048, 5120),
        # a packed fp32 fine-tuning batch: ragged length, documents reset the state
        _gated("gated_bwd_b2_l5003_d1030_f32", "gated_backward", 2, 5003, 1030, "f32", reset=True,
               h0=True),
        # one user's next token: latency
        _gated("gated_step_b1_d2560", "gated_step", 1, 1, 2560),
        # a full decode batch of the serving configuration's 8192 channels
        _gated("gated_step_b256_d8192", "gated_step", 256, 1, 8192),
        # training with the saved inputs in 8 bits: forward and backward
        _gated("gated_ckpt8_b8_l2048_d5120", "gated_ckpt8", 8, 2048, 5120),
        # the same for one packed long row with an odd channel count
        _gated("gated_ckpt8_b1_l9001_d2049", "gated_ckpt8", 1, 9001, 2049, reset=True, h0=True),
        # training the 2.8B-style selective scan: softplus steps, zero-order hold
        _scan("scan_bwd_b8_l2048_d5120_n16", 8, 2048, 5120, 16, 1),
        # one long row, Euler weight: few channels, a long axis
        _scan("scan_bwd_b1_l16384_d2048_n16", 1, 16384, 2048, 16, 1, zoh=False, h0=True),
        # a small fp32 problem with two groups, clamped steps and a ragged end
        _scan("scan_bwd_b2_l333_d320_n8_f32", 2, 333, 320, 8, 2, "f32", clamp=True, h0=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated_backward", "gated_step", "gated_ckpt8", "scan_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    b = rng.choice([1, 1, 2, 3, 4, 8])
    h0 = rng.random() < 0.5
    if op == "scan_backward":
        N = rng.choice([4, 8, 16, 16])
        G = rng.choice([1, 1, 2])
        D = G * _log_int(rng, 24, 5120 // G)
        L = _log_int(rng, 20, 16384)
        while b * L * D * N > 500_000_000:
            L = max(1, L // 2)
        c = _scan("", b, L, D, N, G, dtype, rng.random() < 0.7, rng.random() < 0.5,
                  rng.random() < 0.3, h0)
    else:
        D = _log_int(rng, 200, 8192)
        if op == "gated_step":
            b, L = _log_int(rng, 1, 256), 1
        else:
            L = _log_int(rng, 16, 65536)
            while b * L * D > 80_000_000:
                L = max(1, L // 2)
        c = _gated("", op, b, L, D, dtype, op != "gated_step" and rng.random() < 0.5, h0)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _io(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    b, L, D, io = case["batch"], case["seqlen"], case["channels"], _io(case)

    def normal(*shape, std=1.0, dtype=io):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if case["op"] == "scan_backward":
        N, G = case["dstate"], case["ngroups"]
        s["x"], s["dy"] = normal(b, L, D), normal(b, L, D)
        # steps about log-uniform in [1e-3, 1e-1], as the layer's initialisation makes them
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
        if case["softplus"]:  # raw steps and the bias that softplus maps to them
            s["dt"], s["bias"] = normal(b, L, D, std=0.5), torch.log(torch.expm1(step))
        else:
            s["dt"], s["bias"] = (step * torch.exp(uniform(-0.7, 0.7, b, L, D))).to(io), None
        s["A"] = -torch.exp(uniform(0.0, math.log(16.0), D, N))
        s["B"], s["C"] = normal(b, L, G, N, std=N ** -0.5), normal(b, L, G, N, std=N ** -0.5)
        s["Dskip"] = 1.0 + normal(D, std=0.1, dtype=torch.float32)
        s["h0"] = normal(b, D, N, std=0.1, dtype=torch.float32) if case["h0"] else None
        s["dhf"] = normal(b, D, N, std=0.1, dtype=torch.float32) if case["h0"] else None
        s["limit"] = (2.0 ** -8, 3 * 2.0 ** -6) if case["clamp"] else None
        return s
    if case["op"] == "gated_step":
        s["h"] = normal(b, D, dtype=torch.float32)
        s["x"], s["r"], s["i"] = normal(b, D), normal(b, D), normal(b, D)
    else:
        s["x"], s["r"], s["i"] = normal(b, L, D), normal(b, L, D), normal(b, L, D)
        s["h0"] = normal(b, D, dtype=torch.float32) if case["h0"] else None
        s["reset"] = None
        if case["reset"]:  # documents of about 300 tokens, packed
            s["reset"] = (torch.rand((b, L), generator=g, device="cuda") < 1 / 300).to(torch.uint8)
    # lam so that exp(-c softplus(lam)) is uniform in [0.9, 0.999]
    keep = -torch.log(uniform(0.9, 0.999, D)) / GATE_C
    s["lam"] = torch.log(torch.expm1(keep))
    if case["op"] in ("gated_backward", "gated_ckpt8"):
        s["dy"] = normal(b, L, D)
        s["dhf"] = normal(b, D, dtype=torch.float32) if case["h0"] else None
    if case["op"] == "gated_backward":
        # the forward left the states that enter each block of 64 tokens
        h = _gated_forward(s)[0]
        first = s["h0"] if s["h0"] is not None else torch.zeros((b, D), device="cuda")
        s["states"] = torch.cat([first[:, None], h[:, BLOCK - 1:L - 1:BLOCK]], 1).contiguous()
    return s


# --------------------------------------------------------------------------
# the plain forms: elementary torch operations in 32 bits
# --------------------------------------------------------------------------

def _scan_time(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1 from h_{-1} = 0, by doubling; overwrites a and u."""
    k = 1
    while k < u.shape[1]:
        u[:, k:] += a[:, k:] * u[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return u


def _scan_back(a, u, last):
    """g_t = u_t + a_{t+1} g_{t+1} along axis 1, g_{L-1} = u_{L-1} + last."""
    u = u.flip(1)
    if last is not None:
        u[:, 0] += last
    step = torch.zeros_like(a)
    step[:, 1:] = a[:, 1:].flip(1)
    return _scan_time(step, u).flip(1)


def _gates(r, i, lam, reset):
    """sigmoid(r), sigmoid(i), s = log a, a and m = sqrt(1 - a^2); a reset token has a = 0, m = 1."""
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    s = -GATE_C * torch.log1p(torch.exp(lam)) * sr
    a, m = torch.exp(s), torch.sqrt(-torch.expm1(2 * s))
    if reset is not None:
        keep = (reset == 0).unsqueeze(-1)
        a, m = a * keep, torch.where(keep, m, torch.ones_like(m))
    return sr, si, s, a, m


def _gated_forward(s):
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    sr, si, _, a, m = _gates(r, i, s["lam"], s["reset"])
    u = m * si * x
    if s["h0"] is not None:
        u[:, 0] += a[:, 0] * s["h0"]
    h = _scan_time(a, u)
    return h, h[:, -1].clone()


def _gated_gradients(x, r, i, lam, reset, states, dy, dhf, io):
    b, L, D = x.shape
    sr, si, s, a, m = _gates(r, i, lam, reset)
    # the states before each token, block by block from the saved ones
    pad = -L % BLOCK
    blocks = [torch.nn.functional.pad(t, (0, 0, 0, pad)).reshape(-1, BLOCK, D)
              for t in (a, m * si * x)]
    entering = states.reshape(-1, D)
    blocks[1][:, 0] += blocks[0][:, 0] * entering
    h = _scan_time(blocks[0], blocks[1])
    before = torch.cat([entering[:, None], h[:, :-1]], 1).reshape(b, L + pad, D)[:, :L]
    G = _scan_back(a, dy.float(), dhf)
    ratio = torch.where(m > 0, a * a / m, torch.zeros_like(m))
    e = G * s * (a * before - ratio * si * x)  # a = 0 at a reset: no gradient for its gate
    sp = torch.log1p(torch.exp(lam))
    return {"dx": (G * m * si).to(io), "dr": (e * (1 - sr)).to(io),
            "di": (G * m * x * si * (1 - si)).to(io),
            "dlam": e.sum((0, 1)) * torch.sigmoid(lam) / sp, "dh0": a[:, 0] * G[:, 0]}


def _in_8_bits(v):
    """v (b, L, D) as int8 steps of 2^e for each channel and 64 tokens, e the least that holds
    the largest; given back as the values."""
    b, L, D = v.shape
    pad = -L % BLOCK
    w = torch.nn.functional.pad(v, (0, 0, 0, pad)).reshape(b, -1, BLOCK, D)
    f, k = torch.frexp(w.abs().amax(2, keepdim=True))
    e = torch.clamp(k - 7 + (f > 127 / 128), min=-126)
    q = torch.round(torch.ldexp(w, -e))
    return torch.ldexp(q, e).reshape(b, L + pad, D)[:, :L]


def _selective_gradients(s):
    case = s["case"]
    x, raw, dy = s["x"].float(), s["dt"].float(), s["dy"].float()
    A, G = s["A"], case["ngroups"]
    b, L, D = x.shape
    N = A.shape[1]
    pre = raw + s["bias"] if s["bias"] is not None else raw
    v = pre.clamp(min=0) + torch.log1p(torch.exp(-pre.abs())) if case["softplus"] else pre
    dt, through = v, torch.ones_like(v)
    if s["limit"] is not None:
        lo, hi = s["limit"]
        dt = v.clamp(lo, hi)
        # which side of a bound a step is on is found in 64 bits: its gradient is all or nothing
        v64 = raw.double() if s["bias"] is None else raw.double() + s["bias"].double()
        if case["softplus"]:
            v64 = v64.clamp(min=0) + torch.log1p(torch.exp(-v64.abs()))
        through = ((v64 >= lo) & (v64 <= hi)).float()
    if case["softplus"]:
        through = through * torch.sigmoid(pre)

    def channels(t):  # (b, L, G, N) -> each channel's row (b, L, D, N)
        return t.float().repeat_interleave(D // G, 2)

    z = dt.unsqueeze(-1) * A
    a = torch.exp(z)
    w = torch.expm1(z) / A if case["zoh"] else dt.unsqueeze(-1).expand_as(z)
    xB = x.unsqueeze(-1) * channels(s["B"])
    u = w * xB
    if s["h0"] is not None:
        u[:, 0] += a[:, 0] * s["h0"]
    h = _scan_time(a.clone(), u)
    dC = (dy.unsqueeze(-1) * h).reshape(b, L, G, D // G, N).sum(3)
    h = torch.cat([(s["h0"] if s["h0"] is not None else torch.zeros_like(h[:, 0]))[:, None],
                   h[:, :-1]], 1)
    R = _scan_back(a, dy.unsqueeze(-1) * channels(s["C"]), s["dhf"])
    dh0 = a[:, 0] * R[:, 0]
    ah = a * h
    del h
    # d(weight)/d(step) is a for the hold and 1 for Euler
    ddt = (R * (A * ah + (a * xB if case["zoh"] else xB))).sum(3)
    dA = (R * dt.unsqueeze(-1) * ah).sum((0, 1))
    del ah, a
    if case["zoh"]:
        # dw/dA = (dt e^z - w) / A = (z e^z - (e^z - 1)) / A^2: the difference in 64 bits
        z64 = z.double()
        slope = ((z64 * torch.exp(z64) - torch.expm1(z64)) / A.double() ** 2).float()
        del z64
        dA = dA + (R * slope * xB).sum((0, 1))
        del slope
    del xB, z
    Rw = R * w
    del w
    dx = (Rw * channels(s["B"])).sum(3) + s["Dskip"] * dy
    dB = (Rw * x.unsqueeze(-1)).reshape(b, L, G, D // G, N).sum(3)
    ddt = ddt * through
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (x * dy).sum((0, 1)),
            "ddt_bias": ddt.sum((0, 1)), "dh0": dh0}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _run_own(s):
    import selective_state_space_12_b200 as ssd

    case, op = s["case"], s["case"]["op"]
    if op == "gated":
        return ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], c=GATE_C, reset=s["reset"],
                                  h0=s["h0"])
    if op == "gated_step":
        y = ssd.ssd_gated_step(s["h"], s["x"], s["r"], s["i"], s["lam"], c=GATE_C)
        return y, s["h"]
    if op == "gated_backward":
        return ssd.ssd_gated_scan_backward(s["x"], s["r"], s["i"], s["lam"], s["states"], s["dy"],
                                           s["dhf"], c=GATE_C, reset=s["reset"])
    if op == "gated_ckpt8":
        b, L, D = s["x"].shape
        saved = ssd.GatedCheckpoint8(b, L, D, device=s["x"].device)
        y, hf = ssd.ssd_gated_scan(s["x"], s["r"], s["i"], s["lam"], c=GATE_C, reset=s["reset"],
                                   h0=s["h0"], checkpoint=saved)
        g = ssd.ssd_gated_scan_backward_ckpt8(saved, s["lam"], s["dy"], s["dhf"], c=GATE_C,
                                              reset=s["reset"])
        return {"y": y, "h_final": hf, **g}
    return ssd.ssd_selective_scan_backward(
        s["x"], s["dt"], s["A"], s["B"], s["C"], s["Dskip"], s["h0"], s["dy"], s["dhf"],
        dt_bias=s["bias"], dt_softplus=case["softplus"], dt_limit=s["limit"], zoh=case["zoh"])


def run(s):
    if own:
        return _run_own(s)
    op, io = s["case"]["op"], _io(s["case"])
    if op == "scan_backward":
        return _selective_gradients(s)
    if op == "gated_step":
        x = s["x"].float()
        _, si, _, a, m = _gates(s["r"].float(), s["i"].float(), s["lam"], None)
        s["h"].copy_(a * s["h"] + m * si * x)
        return s["h"].to(io), s["h"]
    if op == "gated":
        h, hf = _gated_forward(s)
        return h.to(io), hf
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    if op == "gated_backward":
        return _gated_gradients(x, r, i, s["lam"], s["reset"], s["states"], s["dy"], s["dhf"], io)
    h, hf = _gated_forward(s)
    first = s["h0"] if s["h0"] is not None else torch.zeros_like(hf)
    states = torch.cat([first[:, None], h[:, BLOCK - 1:x.shape[1] - 1:BLOCK]], 1)
    g = _gated_gradients(_in_8_bits(x), _in_8_bits(r), _in_8_bits(i), s["lam"], s["reset"], states,
                         s["dy"], s["dhf"], io)
    return {"y": h.to(io), "h_final": hf, **g}


# --------------------------------------------------------------------------
# the definition in 64 bits, token after token
# --------------------------------------------------------------------------

def _exact_gates(x, r, i, lam, reset):
    """(a, m, s, gate values) of every token in 64 bits."""
    x, r, i, lam = x.double(), r.double(), i.double(), lam.double()
    gr, gi = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    s = -GATE_C * torch.log(1 + torch.exp(lam)) * gr
    a = torch.exp(s)
    m = torch.sqrt(torch.clamp((1 - a) * (1 + a), min=0.0))
    if reset is not None:
        at = reset.bool()[..., None].expand_as(a)
        a, m = a.masked_fill(at, 0.0), m.masked_fill(at, 1.0)
    return x, gr, gi, s, a, m


def _exact_states(a, u, first):
    """(b, L + 1, D): the state before each token, and after the last."""
    b, L, D = u.shape
    out = torch.empty((b, L + 1, D), dtype=torch.float64, device=u.device)
    out[:, 0] = 0.0 if first is None else first.double()
    for t in range(L):
        torch.addcmul(u[:, t], a[:, t], out[:, t], out=out[:, t + 1])
    return out


def _exact_gated_gradients(x, r, i, lam, reset, states, dy, dhf):
    b, L, D = x.shape
    x, gr, gi, s, a, m = _exact_gates(x, r, i, lam, reset)
    u = m * gi * x
    before = torch.empty_like(u)
    for t in range(L):
        before[:, t] = states[:, t // BLOCK].double() if t % BLOCK == 0 else \
            torch.addcmul(u[:, t - 1], a[:, t - 1], before[:, t - 1])
    G = dy.double()
    carry = torch.zeros((b, D), dtype=torch.float64, device=x.device) if dhf is None \
        else dhf.double()
    for t in range(L - 1, -1, -1):
        G[:, t] += carry
        carry = a[:, t] * G[:, t]
    ds = G * (a * before - torch.where(m > 0, a * a / m, 0.0) * gi * x)
    if reset is not None:
        ds = ds.masked_fill(reset.bool()[..., None].expand_as(ds), 0.0)
    lam = lam.double()
    dlam = -(ds * gr).sum((0, 1)) * GATE_C / (1 + torch.exp(-lam))
    return {"dx": G * m * gi, "dr": ds * s * (1 - gr), "di": G * m * x * gi * (1 - gi),
            "dlam": dlam, "dh0": carry}


def _exact_8_bits(v):
    v = v.double()
    out = torch.empty_like(v)
    for t in range(0, v.shape[1], BLOCK):
        part = v[:, t:t + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        # the least power of two whose 127-fold reaches the largest value
        e = torch.floor(torch.log2(torch.clamp(top, min=2.0 ** -130) / 127))
        e = torch.where(127 * torch.exp2(e) < top, e + 1, e).clamp(min=-126)
        out[:, t:t + BLOCK] = torch.round(part / torch.exp2(e)) * torch.exp2(e)
    return out


def _exact_selective(s):
    case, A, Gn = s["case"], s["A"].double(), s["case"]["ngroups"]
    x, dy, raw = s["x"].double(), s["dy"].double(), s["dt"].double()
    b, L, D = x.shape
    N = A.shape[1]
    pre = raw if s["bias"] is None else raw + s["bias"].double()
    v = torch.logaddexp(pre, torch.zeros_like(pre)) if case["softplus"] else pre
    slope = 1 / (1 + torch.exp(-pre)) if case["softplus"] else torch.ones_like(pre)
    dt = v
    if s["limit"] is not None:
        lo, hi = s["limit"]
        dt = torch.minimum(torch.maximum(v, torch.full_like(v, lo)), torch.full_like(v, hi))
        slope = slope * (v >= lo) * (v <= hi)
    group = torch.arange(D, device=x.device) // (D // Gn)
    Bt, Ct = s["B"].double(), s["C"].double()
    H = torch.empty((L + 1, b, D, N), dtype=torch.float64, device=x.device)
    H[0] = 0.0 if s["h0"] is None else s["h0"].double()

    def token(t):
        z = dt[:, t, :, None] * A
        e = torch.exp(z)
        w = torch.expm1(z) / A if case["zoh"] else dt[:, t, :, None].expand_as(z)
        return z, e, w, Bt[:, t][:, group], x[:, t, :, None]

    for t in range(L):
        z, e, w, Br, xt = token(t)
        H[t + 1] = e * H[t] + w * xt * Br
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.empty_like(Bt), torch.empty_like(Ct)
    dA = torch.zeros_like(A)
    R = torch.zeros((b, D, N), dtype=torch.float64, device=x.device) if s["dhf"] is None \
        else s["dhf"].double()
    for t in range(L - 1, -1, -1):
        z, e, w, Br, xt = token(t)
        step = dt[:, t, :, None]
        R = R + dy[:, t, :, None] * Ct[:, t][:, group]
        dC[:, t] = (dy[:, t, :, None] * H[t + 1]).reshape(b, Gn, D // Gn, N).sum(2)
        dB[:, t] = (R * w * xt).reshape(b, Gn, D // Gn, N).sum(2)
        dx[:, t] = (R * w * Br).sum(2) + s["Dskip"].double() * dy[:, t]
        decay = e * H[t]
        if case["zoh"]:
            ddt[:, t] = (R * (A * decay + e * xt * Br)).sum(2)
            dA += (R * (step * decay + (step * e - w) / A * xt * Br)).sum(0)
        else:
            ddt[:, t] = (R * (A * decay + xt * Br)).sum(2)
            dA += (R * step * decay).sum(0)
        R = e * R
    ddt = ddt * slope
    return {"dx": dx, "ddt": ddt, "dA": dA, "dB": dB, "dC": dC, "dD": (x * dy).sum((0, 1)),
            "ddt_bias": ddt.sum((0, 1)), "dh0": R}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_backward":
        return _exact_selective(s)
    if op == "gated_step":
        x, gr, gi, _, a, m = _exact_gates(s["x"], s["r"], s["i"], s["lam"], None)
        h = a * s["h"].double() + m * gi * x
        return h, h
    if op == "gated_backward":
        return _exact_gated_gradients(s["x"], s["r"], s["i"], s["lam"], s["reset"], s["states"],
                                      s["dy"], s["dhf"])
    x, _, gi, _, a, m = _exact_gates(s["x"], s["r"], s["i"], s["lam"], s["reset"])
    h = _exact_states(a, m * gi * x, s["h0"])
    if op == "gated":
        return h[:, 1:], h[:, -1]
    g = _exact_gated_gradients(_exact_8_bits(s["x"]), _exact_8_bits(s["r"]), _exact_8_bits(s["i"]),
                               s["lam"], s["reset"], h[:, :-1:BLOCK], s["dy"], s["dhf"])
    return {"y": h[:, 1:], "h_final": h[:, -1], **g}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    b, L, D = case["batch"], case["seqlen"], case["channels"]
    io = 2 if case["dtype"] == "bf16" else 4
    n = b * L * D
    states = b * D * 4 * (2 if case["h0"] else 1)
    if case["op"] == "scan_backward":
        N, rows = case["dstate"], b * L * case["ngroups"] * case["dstate"]
        # x, dt, dy in, dx and ddt out (fp32); B, C in, dB and dC out; A, dA and the states; about
        # 16 operations for each state entry and token
        return {"bytes": n * (3 * io + 8) + rows * (2 * io + 8) + 8 * D * N + states * 2 * N
                + 16 * D, "flops": 16 * n * N}
    extra = b * L * (1 if case["reset"] else 0) + 4 * D
    if case["op"] == "gated":
        return {"bytes": n * 4 * io + states + extra, "flops": 12 * n}
    if case["op"] == "gated_step":
        return {"bytes": n * (4 * io + 8) + extra, "flops": 12 * n}
    blocks = b * -(-L // BLOCK) * D
    if case["op"] == "gated_backward":
        return {"bytes": n * 7 * io + 4 * blocks + states + extra + 4 * D, "flops": 30 * n}
    # forward: 3 in, 1 out and the checkpoint; backward: the checkpoint and dy in, 3 out
    return {"bytes": n * (8 * io + 6) + 2 * 7 * blocks + 2 * states + 2 * extra + 4 * D,
            "flops": 42 * n}
