"""The training-side operators of libgdn and the vector-state recurrence they
belong to, as cases that can be measured: the gated linear recurrence over
ragged sequences (serving and training), its backward pass with and without
8-bit checkpoints of its inputs, and the backward pass of the causal conv.

A case is a packed ragged batch: "lens" gives the sequence lengths, "channels"
the width, "act" and "state" the storage types.  Kinds:

  scan    forward only: h and the new state pages
  train   forward, then the backward pass from the activations themselves
  train8  forward that also keeps x, a and b in 8 bits, then the backward pass
          from those 8 bits
  conv    the backward pass of the width-4 causal conv + SiLU

With `own` false `run` computes in elementary torch operations; with `own`
true it makes the calls of the package.
"""
import math

import torch

own = False

#: Rows between two kept states: the backward pass recomputes h from the state before each such packed row.
BLOCK = 256
#: An 8-bit block: consecutive packed rows by consecutive channels that share one scale.
Q_ROWS, Q_CHANNELS = 16, 4

PROMPTS = "45,83,159,236,320,404,656,256"  # the short mixed prompts of this repository's benchmark
LONG = "8192,8192,8192,8192"
MAX_ELEMENTS = 32768 * 4096


def listed():
    return [
        # one decode step of a batch of 64 requests: one row each, where latency is what counts
        {"name": "scan decode 64x1", "kind": "scan", "lens": ",".join(["1"] * 64), "channels": 4096, "act": "bf16", "state": "f32"},
        # the prompts of a mixed prefill, packed
        {"name": "scan prompts", "kind": "scan", "lens": PROMPTS, "channels": 4096, "act": "bf16", "state": "f32"},
        # long prefill of four sequences
        {"name": "scan 4x8192", "kind": "scan", "lens": LONG, "channels": 4096, "act": "bf16", "state": "f32"},
        # one long document, few and odd channels, all fp32: little to do in parallel but the time axis
        {"name": "scan 1x30011 f32", "kind": "scan", "lens": "30011", "channels": 1001, "act": "f32", "state": "bf16"},
        # a small training step on short packed documents
        {"name": "train prompts", "kind": "train", "lens": PROMPTS, "channels": 4096, "act": "bf16", "state": "f32"},
        # a training step on long sequences
        {"name": "train 4x8192", "kind": "train", "lens": LONG, "channels": 4096, "act": "bf16", "state": "f32"},
        # ragged lengths, an odd width, fp32 throughout
        {"name": "train ragged f32", "kind": "train", "lens": "5000,1,0,3333,777,2,4099", "channels": 2050, "act": "f32", "state": "f32"},
        # the same steps with the activations held in 8 bits between the passes
        {"name": "train8 prompts", "kind": "train8", "lens": PROMPTS, "channels": 4096, "act": "bf16", "state": "f32"},
        {"name": "train8 4x8192", "kind": "train8", "lens": LONG, "channels": 4096, "act": "bf16", "state": "f32"},
        # the conv in front of the layer: 2 * 16 * 128 + 32 * 128 channels
        {"name": "conv prompts", "kind": "conv", "lens": PROMPTS, "channels": 8192, "act": "bf16", "state": "bf16"},
        {"name": "conv 4x8192", "kind": "conv", "lens": LONG, "channels": 8192, "act": "bf16", "state": "bf16"},
        # short and odd sequences, narrow, fp32
        {"name": "conv ragged f32", "kind": "conv", "lens": "1,700,2,3,0,1291,64,5", "channels": 672, "act": "f32", "state": "f32"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "train", "train8", "conv"])
    act = rng.choice(["bf16", "bf16", "f32"])
    state = act if kind == "conv" else rng.choice(["f32", "f32", "bf16"])
    channels = _log_uniform(rng, 32, 8192)
    if kind == "conv":
        channels = max(96, channels // 32 * 32)
    elif rng.random() < 0.5:
        channels = max(32, channels // 8 * 8)
    most = MAX_ELEMENTS // (2 if act == "f32" else 1) // channels
    rows = _log_uniform(rng, 16, min(40000, most))
    n = min(rows, _log_uniform(rng, 1, 64))
    if kind == "scan" and rng.random() < 0.3:  # a decode step: a few rows for each of many sequences
        lens = [rng.randint(1, 4) for _ in range(_log_uniform(rng, 1, 256))]
    else:
        cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    return {"kind": kind, "lens": ",".join(map(str, lens)), "channels": channels, "act": act, "state": state}


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens = [int(v) for v in case["lens"].split(",")]
    n, rows, C = len(lens), sum(lens), case["channels"]
    act, st = _DT[case["act"]], _DT[case["state"]]

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dt)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    cu = [sum(lens[:i]) for i in range(n + 1)]
    lens_t = torch.tensor(lens, device=dev)
    s = {"kind": case["kind"], "rows": rows, "channels": C, "lens": lens, "cu_host": cu, "act": case["act"],
         "state": case["state"], "max_len": max(lens),
         "cu": torch.tensor(cu, dtype=torch.int32, device=dev),
         # which sequence a packed row belongs to, and its place in it
         "seq": torch.repeat_interleave(torch.arange(n, device=dev), lens_t),
         "page": torch.randperm(n + 3, generator=gen, device=dev)[:n].to(torch.int32)}
    s["pos"] = torch.arange(rows, device=dev) - s["cu"].long()[s["seq"]]
    s["x"] = normal(rows, C, dt=act)
    if case["kind"] == "conv":
        s |= {"w": normal(C, 4, std=0.25, dt=act), "dy": normal(rows, C, dt=act),
              "window": normal(n + 3, 3, C, dt=act), "d_window": normal(n, 3, C)}
        return s
    # Decays from almost none to almost all: A in [1, 16], step sizes softplus(dt_bias) from 0.001 to 0.1
    step = torch.exp(uniform(C) * math.log(100.0) + math.log(1e-3))
    s |= {"a_log": torch.log(1.0 + 15.0 * uniform(C)), "dt_bias": torch.log(torch.expm1(step.double())).float(),
          "a": normal(rows, C, dt=act), "b": normal(rows, C, dt=act),
          "state_in": normal(n + 3, C, std=0.5, dt=st), "state_out": torch.zeros(n + 3, C, device=dev, dtype=st)}
    if case["kind"] != "scan":
        s |= {"dh": normal(rows, C, dt=act), "d_state": normal(n, C)}
    return s


# ------------------------------------------------------------ the plain forms


def _ahead(t, k, fill):
    """Row r of the result is row r - k of `t` (k > 0) or row r + |k|."""
    pad = torch.full((min(abs(k), t.shape[0]),) + t.shape[1:], fill, dtype=t.dtype, device=t.device)
    return torch.cat((pad, t[:-k]))[: t.shape[0]] if k > 0 else torch.cat((t[-k:], pad))[-t.shape[0]:]


def _recur(alpha, u, span, back=False):
    """y_t = alpha_t y_{t-1} + u_t over the rows (or from the last row to the first), where an alpha of 0 starts
    anew; no run is longer than `span`.  Each step doubles the reach."""
    reach = 1
    while reach < span:
        k = -reach if back else reach
        u = u + alpha * _ahead(u, k, 0.0)
        alpha = alpha * _ahead(alpha, k, 0.0)
        reach *= 2
    return u


def _gates(a, b, a_log, dt_bias):
    z = a + dt_bias
    sp = torch.clamp(z, min=0.0) + torch.log1p(torch.exp(-z.abs()))
    g = -torch.exp(a_log) * sp
    return z, g, torch.exp(g), 1.0 / (1.0 + torch.exp(-b))


def _stored(v):
    """The values that the 8-bit form of `v` stands for."""
    rows, C = v.shape
    pad_r, pad_c = -rows % Q_ROWS, -C % Q_CHANNELS
    w = torch.cat((v, v.new_zeros(pad_r, C))) if pad_r else v
    w = torch.cat((w, w.new_zeros(w.shape[0], pad_c)), 1) if pad_c else w
    w = w.view(w.shape[0] // Q_ROWS, Q_ROWS, w.shape[1] // Q_CHANNELS, Q_CHANNELS)
    top = w.abs().amax((1, 3), keepdim=True).double()
    live = top >= 2.0 ** -100
    up = torch.where(live, 127.0 / top, 0.0).float()
    scale = torch.where(live, top / 127.0, 0.0).float()
    q = torch.round(w.double() * up.double()).float()  # the product is exact in 64 bits: one rounding
    return (q * scale).view(rows + pad_r, C + pad_c)[:rows, :C].contiguous()


def _plain_scan(s):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    z, g, alpha, beta = _gates(a, b, s["a_log"], s["dt_bias"])
    first = (s["pos"] == 0)[:, None]
    h0 = s["state_in"].float()[s["page"].long()]
    u = beta * x
    u = torch.where(first, u + alpha * h0[s["seq"]], u)
    h = _recur(torch.where(first, 0.0, alpha), u, s["max_len"])
    last = s["cu"].long()[1:] - 1
    some = torch.tensor(s["lens"], device=x.device) > 0
    s["state_out"][s["page"].long()[some]] = h[last[some]].to(s["state_out"].dtype)
    return h


def _plain_scan_backward(s, h):
    x, a, b = s["x"].float(), s["a"].float(), s["b"].float()
    dh = s["dh"].float()
    seq, pos, page = s["seq"], s["pos"], s["page"].long()
    first = (pos == 0)[:, None]
    lens = torch.tensor(s["lens"], device=x.device)
    final = (pos == lens[seq] - 1)[:, None]
    h0 = s["state_in"].float()[page][seq]
    before = torch.where(first, h0, _ahead(h, 1, 0.0))
    if s["kind"] == "train8":
        x, a, b = _stored(x), _stored(a), _stored(b)
        z, g, alpha, beta = _gates(a, b, s["a_log"], s["dt_bias"])
        anew = first | (torch.arange(s["rows"], device=x.device) % BLOCK == 0)[:, None]
        u = beta * x
        h = _recur(torch.where(anew, 0.0, alpha), torch.where(anew, u + alpha * before, u), BLOCK)
        before = torch.where(anew, before, _ahead(h, 1, 0.0))
    else:
        z, g, alpha, beta = _gates(a, b, s["a_log"], s["dt_bias"])
    lam = _recur(torch.where(final, 0.0, _ahead(alpha, -1, 0.0)), torch.where(final, dh + s["d_state"][seq], dh), s["max_len"], back=True)
    dg = lam * alpha * before
    da = -torch.exp(s["a_log"]) * dg / (1.0 + torch.exp(-z))
    db = lam * x * beta * (1.0 - beta)
    starts = s["cu"].long()[:-1].clamp(max=max(s["rows"] - 1, 0))
    d_state0 = torch.where((lens > 0)[:, None], (alpha * lam)[starts], s["d_state"])
    act = s["dh"].dtype
    return {"dx": (beta * lam).to(act), "da": da.to(act), "db": db.to(act), "d_a_log": (dg.double() * g.double()).sum(0).float(),
            "d_dt_bias": da.double().sum(0).float(), "d_state0": d_state0}


def _plain_conv_backward(s):
    x, dy, w, seq, pos = s["x"].float(), s["dy"].float(), s["w"].float(), s["seq"], s["pos"]
    rows = torch.arange(s["rows"], device=x.device)
    window = s["window"].float()[s["page"].long()]
    taps = [torch.where((pos >= 3 - j)[:, None], x[(rows - 3 + j).clamp(min=0)], window[seq, (pos + j).clamp(max=2)]) for j in range(4)]
    z = taps[0] * w[:, 0] + taps[1] * w[:, 1] + taps[2] * w[:, 2] + taps[3] * w[:, 3]
    sig = 1.0 / (1.0 + torch.exp(-z))
    dz = dy * sig * (1.0 + z * (1.0 - sig))
    lens = torch.tensor(s["lens"], device=x.device)
    left = lens[seq] - 1 - pos
    dx = sum(torch.where((left >= 3 - j)[:, None], _ahead(dz, j - 3, 0.0) if j < 3 else dz, 0.0) * w[:, j] for j in range(4))
    dx = dx + torch.where((left < 3)[:, None], s["d_window"][seq, (2 - left).clamp(min=0)], 0.0)
    dw = torch.stack([(dz.double() * t.double()).sum(0) for t in taps], 1).float()
    # row i of the window before the sequence meets tap i - t of row t, and is still in the window after it where the sequence is short
    cu = s["cu"].long()

    def row(t):
        return torch.where((lens > t)[:, None], dz[(cu[:-1] + t).clamp(max=max(s["rows"] - 1, 0))], 0.0)

    d0 = [sum(w[:, i - t] * row(t) for t in range(i + 1)) for i in range(3)]
    keep = [torch.where((lens <= i)[:, None], s["d_window"].gather(1, (i - lens).clamp(min=0)[:, None, None].expand(-1, 1, w.shape[0]))[:, 0], 0.0) for i in range(3)]
    return {"dx": dx.to(s["x"].dtype), "d_conv_w": dw, "d_window0": torch.stack([p + q for p, q in zip(d0, keep)], 1)}


# ------------------------------------------------------- the package's calls


def _handles(s):
    """What a program keeps beside its tensors: dims, parameters, the batch, the pools and the workspaces."""
    import linear_attention_ssm_gdn_amd as g
    n = len(s["lens"])
    dev = s["x"].device
    batch = g.Batch(s["cu"], s["page"], None, s["max_len"], s["rows"])
    if s["kind"] == "conv":
        # any head split with this many channels: the conv knows no heads
        dims = g.Dims(1, 1, 32, s["channels"] - 64, act_dtype=s["act"], state_dtype="f32")
        return {"g": g, "batch": batch, "dims": dims, "ws": torch.empty(g.gdnt_conv_workspace_bytes(dims, n, s["rows"]), dtype=torch.uint8, device=dev),
                "pool": g.ConvPool(s["window"], None)}
    dims = g.ScanDims(s["channels"], act_dtype=s["act"], state_dtype=s["state"])
    own_ = {"g": g, "batch": batch, "dims": dims, "params": g.ScanParams(s["a_log"], s["dt_bias"]),
            "in": g.StatePool(s["state_in"]), "out": g.StatePool(s["state_out"]),
            "ws": torch.empty(g.gdnt_scan_workspace_bytes(dims, n, s["rows"]), dtype=torch.uint8, device=dev)}
    if s["kind"] != "scan":
        own_["saved"] = g.ScanSaved.alloc(dims, s["rows"], dev, ckpt=s["kind"] == "train8")
    return own_


def _own_run(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    o = s["handles"]
    g = o["g"]
    if s["kind"] == "conv":
        dx, dw, d0 = g.gdnt_conv_backward(o["dims"], s["w"], s["x"], s["dy"], o["batch"], o["pool"], d_window=s["d_window"], workspace=o["ws"])
        return {"dx": dx, "d_conv_w": dw, "d_window0": d0}
    saved = o.get("saved")
    h = g.gdnt_scan_forward(o["dims"], o["params"], s["x"], s["a"], s["b"], o["batch"], o["in"], o["out"], saved=saved, workspace=o["ws"])
    if s["kind"] == "scan":
        return {"h": h, "state": s["state_out"]}
    xab = {} if s["kind"] == "train8" else {"x": s["x"], "a": s["a"], "b": s["b"]}
    grads = g.gdnt_scan_backward(o["dims"], o["params"], o["batch"], o["in"], saved, s["dh"], d_state=s["d_state"], workspace=o["ws"], **xab)
    return {"h": h, "state": s["state_out"], **grads._asdict()}


def run(state):
    if own:
        return _own_run(state)
    if state["kind"] == "conv":
        return _plain_conv_backward(state)
    h = _plain_scan(state)
    out = {"h": h.to(state["x"].dtype), "state": state["state_out"]}
    if state["kind"] != "scan":
        out |= _plain_scan_backward(state, h)
    return out


def work(case):
    lens = [int(v) for v in case["lens"].split(",")]
    n, rows, C = len(lens), sum(lens), case["channels"]
    e = rows * C
    act, st = (2 if case["act"] == "bf16" else 4), (2 if case["state"] == "bf16" else 4)
    if case["kind"] == "conv":  # x, dy -> dx; the windows and their gradients
        return {"bytes": 3 * act * e + n * 3 * C * (act + 8) + C * 4 * (act + 4), "flops": 35 * e}
    if case["kind"] == "scan":  # x, a, b -> h; the states
        return {"bytes": 4 * act * e + n * C * 2 * st + 8 * C, "flops": 20 * e}
    # x, a, b, dh -> h, dx, da, db; the states and their gradients
    return {"bytes": 8 * act * e + n * C * (2 * st + 8) + 16 * C, "flops": 50 * e}


# ------------------------------------------- the definitions, row by row in 64 bits


def _order(lens):
    """The sequences from the longest to the shortest, and how many of them still have a row t, for each t."""
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    counts, k = [], len(order)
    for t in range(max(lens)):
        while k and lens[order[k - 1]] <= t:
            k -= 1
        counts.append(k)
    return order, counts


def _stored64(v):
    """The 8-bit values again, block by block of rows: integers by the stored scale (both scales are fp32 by definition)."""
    out = torch.empty_like(v)
    C = v.shape[1]
    wide = torch.cat((v, v.new_zeros(v.shape[0], -C % Q_CHANNELS)), 1)
    for r in range(0, v.shape[0], Q_ROWS):
        top = wide[r:r + Q_ROWS].abs().amax(0).view(-1, Q_CHANNELS).amax(1)
        live = top >= 2.0 ** -100
        up = torch.where(live, (127.0 / top).float().double(), 0.0).repeat_interleave(Q_CHANNELS)[:C]
        scale = torch.where(live, (top / 127.0).float().double(), 0.0).repeat_interleave(Q_CHANNELS)[:C]
        out[r:r + Q_ROWS] = (v[r:r + Q_ROWS] * up).round() * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    lens, cu, page = s["lens"], s["cu_host"], s["page"].long()
    order, counts = _order(lens)
    base = torch.tensor([cu[i] for i in order], device=page.device)
    perm = torch.tensor(order, device=page.device)
    if case["kind"] == "conv":
        w, x, dy = s["w"].to(D), s["x"].to(D), s["dy"].to(D)
        dx, dw = torch.zeros_like(x), torch.zeros(w.shape, dtype=D, device=w.device)
        d0 = torch.zeros(len(lens), 3, w.shape[0], dtype=D, device=w.device)
        for i, T in enumerate(lens):
            seq = torch.cat((s["window"][page[i]].to(D), x[cu[i]:cu[i] + T]))
            grad = torch.zeros_like(seq)
            z = sum(seq[j:j + T] * w[:, j] for j in range(4))
            sg = torch.sigmoid(z)
            dz = dy[cu[i]:cu[i] + T] * (sg + z * sg * torch.sigmoid(-z))
            for j in range(4):
                grad[j:j + T] += dz * w[:, j]
                dw[:, j] += (dz * seq[j:j + T]).sum(0)
            grad[T:] += s["d_window"][i].to(D)
            d0[i], dx[cu[i]:cu[i] + T] = grad[:3], grad[3:]
        return {"dx": dx, "d_conv_w": dw, "d_window0": d0}

    def gates(a, b):
        z = a + s["dt_bias"].to(D)
        g = -s["a_log"].to(D).exp() * torch.logaddexp(z, torch.zeros_like(z))
        return z, g, g.exp(), torch.sigmoid(b)

    x, a, b = s["x"].to(D), s["a"].to(D), s["b"].to(D)
    z, g, alpha, beta = gates(a, b)
    h, before = torch.zeros_like(x), torch.zeros_like(x)
    cur = s["state_in"].to(D)[page][perm]
    start = cur.clone()
    for t, k in enumerate(counts):
        at = base[:k] + t
        before[at] = cur[:k]
        cur[:k] = alpha[at] * cur[:k] + beta[at] * x[at]
        h[at] = cur[:k]
    state = s["state_out"].to(D)
    some = torch.tensor([i for i, T in enumerate(lens) if T > 0], device=page.device)
    ends = torch.empty_like(cur)
    ends[perm] = cur
    state[page[some]] = ends[some]
    out = {"h": h, "state": state}
    if case["kind"] == "scan":
        return out
    if case["kind"] == "train8":
        x, a, b = _stored64(x), _stored64(a), _stored64(b)
        z, g, alpha, beta = gates(a, b)
        cur = start
        for t, k in enumerate(counts):
            at = base[:k] + t
            kept = (at % BLOCK == 0)[:, None]  # the state before such a row was kept by the forward pass
            before[at] = torch.where(kept, before[at], cur[:k])
            cur[:k] = alpha[at] * before[at] + beta[at] * x[at]
    lam = torch.empty_like(x)
    dh = s["dh"].to(D)
    mu = s["d_state"].to(D)[perm]
    for t in range(len(counts) - 1, -1, -1):
        at = base[:counts[t]] + t
        now = dh[at] + mu[:counts[t]]
        lam[at] = now
        mu[:counts[t]] = alpha[at] * now
    dg = lam * alpha * before
    da = dg * -s["a_log"].to(D).exp() * torch.sigmoid(z)
    d0 = torch.empty_like(mu)
    d0[perm] = mu
    return out | {"dx": beta * lam, "da": da, "db": lam * x * beta * torch.sigmoid(-b), "d_a_log": (dg * g).sum(0),
                  "d_dt_bias": da.sum(0), "d_state0": d0}
