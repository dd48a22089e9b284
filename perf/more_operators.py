"""Linear attention with a decay for each head, what feeds it and what keeps
its state, as cases that can be measured.

A case is a packed ragged batch: "lens" gives the sequence lengths, "hk" and
"hv" the key and value heads, "dk" and "dv" their widths, "act" and "state" the
storage types.  Kinds:

  rotate        norms of queries and keys for each head and the rotation by position
  rotate_train  the same, then its backward pass
  attend        linear attention forward: o and the new state pages (prompts, or single tokens)
  attend_train  the same, then its backward pass
  cache         state pages written into 8-bit entries and read back into other pages

"decay" is "row" (a log decay for every row and value head, as a gate gives it)
or "head" (one number for each value head).

With `own` false `run` computes in elementary torch operations; with `own`
true it makes the calls of the package.
"""
import math

import torch

own = False

#: Rows that the plain form takes together between two states.
CHUNK = 64
#: Values of a state's row that share one scale in an 8-bit entry.
Q_COLS = 64
EPS = 1e-6

PROMPTS = "45,83,159,236,320,404,656,256"  # the short mixed prompts of this repository's benchmark
LONG = "8192,8192,8192,8192"
DECODE = ",".join(["1"] * 64)
LAYER = {"hk": 16, "hv": 32, "dk": 128, "dv": 128, "act": "bf16", "state": "f32"}  # the benchmark's layer
#: The most that a case costs: state entries times rows, and elements of q and k.
MOST, MOST_QK = 32768 * 32 * 128 * 128, 32768 * 32 * 128


def listed():
    return [
        # queries and keys of one decode step of 64 requests: latency counts
        {"name": "rotate decode 64x1", "kind": "rotate", "lens": DECODE, **LAYER, "rot": 128, "pairs": "halves", "norm": "rms"},
        # a training step's queries and keys
        {"name": "rotate train 4x8192", "kind": "rotate_train", "lens": LONG, **LAYER, "rot": 128, "pairs": "halves", "norm": "rms"},
        # ragged fp32, an odd width of which a part is rotated, neighbours as pairs, one key head for three of queries
        {"name": "rotate train ragged f32", "kind": "rotate_train", "lens": "700,1,0,1291,64,5", "hk": 3, "hv": 9, "dk": 80, "dv": 80, "act": "f32", "state": "f32", "rot": 48, "pairs": "neighbours", "norm": "l2"},
        # one decode step of a batch of 64 requests: 64 x 32 states read and written
        {"name": "attend decode 64x1", "kind": "attend", "lens": DECODE, **LAYER, "decay": "row"},
        # the prompts of a mixed prefill, packed
        {"name": "attend prompts", "kind": "attend", "lens": PROMPTS, **LAYER, "decay": "row"},
        # long prefill of four sequences
        {"name": "attend 4x8192", "kind": "attend", "lens": LONG, **LAYER, "decay": "row"},
        # one long document, four heads, all fp32, fixed decays: little to do in parallel but the time axis
        {"name": "attend 1x30011 f32", "kind": "attend", "lens": "30011", "hk": 4, "hv": 4, "dk": 64, "dv": 64, "act": "f32", "state": "f32", "decay": "head"},
        # a training step on short packed documents
        {"name": "train prompts", "kind": "attend_train", "lens": PROMPTS, **LAYER, "decay": "row"},
        # a training step on long sequences
        {"name": "train 4x8192", "kind": "attend_train", "lens": LONG, **LAYER, "decay": "row"},
        # ragged lengths and odd widths, fp32, two value heads to a key head, decays learned for each head
        {"name": "train ragged f32", "kind": "attend_train", "lens": "1500,1,0,777,2,63,64,65", "hk": 3, "hv": 6, "dk": 40, "dv": 72, "act": "f32", "state": "f32", "decay": "head"},
        # a few prefixes kept and restored
        {"name": "cache 3 pages", "kind": "cache", "lens": "1,1,1", **LAYER},
        # a whole batch's states swapped out and in
        {"name": "cache 96 pages", "kind": "cache", "lens": ",".join(["1"] * 96), **LAYER},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, rows, n):
    cuts = sorted(rng.randint(0, rows) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [rows])]


def draw(rng):
    kind = rng.choice(["rotate", "rotate_train", "attend", "attend", "attend_train", "attend_train", "cache"])
    act = rng.choice(["bf16", "bf16", "f32"])
    hk, group = _log_uniform(rng, 1, 16), rng.choice([1, 1, 2, 3, 4])
    case = {"kind": kind, "lens": "", "hk": hk, "hv": hk * group, "dk": 8 * rng.randint(2, 16), "dv": 8 * rng.randint(2, 16), "act": act, "state": rng.choice(["f32", "f32", "bf16"])}
    if rng.random() < 0.4:  # the common widths
        case |= {"dk": rng.choice([64, 128]), "dv": rng.choice([64, 128])}
    wide = 2 if act == "f32" else 1
    if kind.startswith("rotate"):
        most = MOST_QK // wide // (case["hk"] + case["hv"]) // case["dk"]
        case |= {"rot": 2 * rng.randint(0, case["dk"] // 2), "pairs": rng.choice(["halves", "neighbours"]), "norm": rng.choice(["rms", "l2"])}
    else:
        most = MOST // wide // case["hv"] // case["dk"] // case["dv"]
    if kind == "cache":
        lens = [1] * _log_uniform(rng, 1, min(96, 96 * 32 * 128 * 128 // (case["hv"] * case["dk"] * case["dv"])))
    elif kind == "attend" and rng.random() < 0.4:  # a decode step: a few rows for each of many sequences
        lens = [rng.randint(1, 4) for _ in range(_log_uniform(rng, 1, 128))]
    else:
        rows = _log_uniform(rng, 16, min(40000, most))
        lens = _split(rng, rows, min(rows, _log_uniform(rng, 1, 32)))
    if kind.startswith("attend"):
        case["decay"] = rng.choice(["row", "row", "head"])
    return case | {"lens": ",".join(map(str, lens))}


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    lens = [int(v) for v in case["lens"].split(",")]
    n, rows = len(lens), sum(lens)
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    act, st = _DT[case["act"]], _DT[case["state"]]

    def normal(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dt)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    s = dict(case) | {"n": n, "rows": rows}
    if case["kind"] == "cache":  # sequences at scattered pages, entries taken as they came free
        s |= {"page": torch.randperm(n + 3, generator=gen, device=dev)[:n].to(torch.int32), "entry": torch.randperm(n + 5, generator=gen, device=dev)[:n].to(torch.int32),
              "to": torch.randperm(n + 3, generator=gen, device=dev)[:n].to(torch.int32),
              "states": normal(n + 3, hv, dk, dv, dt=st) * torch.exp(normal(n + 3, hv, dk, 1)).to(st), "restored": torch.zeros(n + 3, hv, dk, dv, device=dev, dtype=st)}
        return s
    cu = [sum(lens[:i]) for i in range(n + 1)]
    lens_t = torch.tensor(lens, device=dev)
    s |= {"lens_host": lens, "cu_host": cu, "max_len": max(lens), "cu": torch.tensor(cu, dtype=torch.int32, device=dev),
          "page": torch.randperm(n + 3, generator=gen, device=dev)[:n].to(torch.int32)}
    if case["kind"].startswith("rotate"):  # hv heads of queries, hk of keys, all dk wide
        # decode steps stand far into their sequences, prompts begin at 0
        start = torch.randint(0, 100000, (n,), generator=gen, device=dev) if max(lens) <= 4 else torch.zeros(n, dtype=torch.long, device=dev)
        seq = torch.repeat_interleave(torch.arange(n, device=dev), lens_t)
        s |= {"q": normal(rows, hv * dk, dt=act), "k": normal(rows, hk * dk, dt=act), "wq": 1.0 + normal(dk, std=0.1), "wk": 1.0 + normal(dk, std=0.1),
              "pos": (start[seq] + torch.arange(rows, device=dev) - s["cu"].long()[seq]).to(torch.int32),
              "inv_freq": (10000.0 ** (-torch.arange(case["rot"] // 2, device=dev, dtype=torch.float64) * 2 / max(case["rot"], 1))).float()}
        if case["kind"] == "rotate_train":
            s |= {"d_yq": normal(rows, hv * dk, dt=act), "d_yk": normal(rows, hk * dk, dt=act)}
        return s
    if case["decay"] == "row":  # a gate in front: from almost no decay to almost all
        step = torch.exp(uniform(hv) * math.log(100.0) + math.log(1e-3))
        z = normal(rows, hv) + torch.log(torch.expm1(step.double())).float()
        s["g"] = -(1.0 + 15.0 * uniform(hv)) * torch.nn.functional.softplus(z)
    else:  # halving lengths, spread over the heads
        s["g"] = torch.log1p(-(2.0 ** -(2.0 + 7.0 * torch.arange(hv, device=dev) / hv)))
    s |= {"q": normal(rows, hk * dk, dt=act), "k": normal(rows, hk * dk, dt=act), "v": normal(rows, hv * dv, dt=act), "scale": dk ** -0.5,
          "state_in": normal(n + 3, hv, dk, dv, dt=st), "state_out": torch.zeros(n + 3, hv, dk, dv, device=dev, dtype=st)}
    if max(lens) <= 4:  # the sequences that have a row t, and that row
        live = [torch.tensor([i for i, v in enumerate(lens) if v > t], device=dev) for t in range(max(lens))]
        s["tokens"] = [(i, s["cu"].long()[i] + t) for t, i in enumerate(live)]
    if case["kind"] == "attend_train":
        s |= {"d_o": normal(rows, hv * dv, dt=act), "d_state": normal(n, hv, dk, dv)}
    return s


# ------------------------------------------------------------ the plain forms


def _angles(s):
    a = s["pos"].double()[:, None] * s["inv_freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotated(y, cos, sin, s):
    """The first `rot` values of each head, turned in pairs."""
    rot = s["rot"]
    if rot == 0:
        return y
    if s["pairs"] == "halves":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, y[..., rot:]), -1)
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), y[..., rot:]), -1)


def _root(x, s):
    square = x * x
    return torch.rsqrt((square.mean(-1, keepdim=True) if s["norm"] == "rms" else square.sum(-1, keepdim=True)) + EPS)


def _plain_rotate(s):
    cos, sin = _angles(s)
    out = {}
    for t in ("q", "k"):
        x = s[t].float().view(s["rows"], -1, s["dk"])
        out[t] = _rotated(x * _root(x, s) * s["w" + t], cos, sin, s).to(s[t].dtype).view(s[t].shape)
    if s["kind"] == "rotate":
        return out
    for t in ("q", "k"):
        x = s[t].float().view(s["rows"], -1, s["dk"])
        r = _root(x, s)
        dy = _rotated(s["d_y" + t].float().view(x.shape), cos, -sin, s)
        dn, unit = dy * s["w" + t], x * r
        mean = (dn * unit).sum(-1, keepdim=True) / (s["dk"] if s["norm"] == "rms" else 1)
        out["d_" + t] = (r * (dn - unit * mean)).to(s[t].dtype).view(s[t].shape)
        out["d_w" + t] = (dy.double() * unit.double()).sum((0, 1)).float()
    return out


def _chunk_rows(s):
    """The rows of every chunk, [chunks][CHUNK], with `rows` in the place of those behind a sequence's end; each chunk's
    sequence; each sequence's first and last chunk (any one for an empty sequence)."""
    dev = s["cu"].device
    per = [-(-v // CHUNK) for v in s["lens_host"]]
    first = [sum(per[:i]) for i in range(len(per))]
    seq = torch.repeat_interleave(torch.arange(s["n"], device=dev), torch.tensor(per, device=dev))
    nth = torch.arange(sum(per), device=dev) - torch.tensor(first, device=dev)[seq]
    at = s["cu"].long()[seq][:, None] + nth[:, None] * CHUNK + torch.arange(CHUNK, device=dev)
    at = torch.where(at < s["cu"].long()[seq + 1][:, None], at, s["rows"])
    ends = [(min(f, sum(per) - 1), max(f + p - 1, 0)) for f, p in zip(first, per)]
    return at, seq, torch.tensor([e[0] for e in ends], device=dev), torch.tensor([e[1] for e in ends], device=dev)


def _heads(t, at, heads, group=1):
    """[chunks][heads * group][CHUNK][width] of packed rows, zeros behind a sequence's end."""
    t = torch.cat((t.float(), t.new_zeros(1, t.shape[1], dtype=torch.float32)))[at]
    t = t.view(at.shape[0], CHUNK, heads, -1).transpose(1, 2)
    return t.repeat_interleave(group, 1) if group > 1 else t.contiguous()


def _packed(t, at, s, group=1):
    """Packed rows again, heads of a group summed."""
    if group > 1:
        t = t.view(t.shape[0], -1, group, *t.shape[2:]).sum(2)
    out = t.new_empty(s["rows"] + 1, t.shape[1] * t.shape[3])
    out[at.flatten()] = t.transpose(1, 2).reshape(at.numel(), -1)
    return out[:-1]


def _carried(local, total, seq, start, first, last, back=False):
    """The state in front of every chunk (`back`: behind it): what the chunks of its sequence on that side leave, each
    decayed by the chunks between, and the decayed `start`.  One product of matrices for a head."""
    U = total.cumsum(0)
    V = U - total  # up to the chunk, without it
    far = (V[None] - U[:, None]) if not back else (V[:, None] - U[None])  # between chunk c' (first axis) and chunk c
    i = torch.arange(total.shape[0], device=total.device)
    side = (i[:, None] < i[None]) if not back else (i[:, None] > i[None])
    between = torch.where((side & (seq[:, None] == seq[None]))[..., None], far, -math.inf).exp().float()  # [c'][c][head]
    got = between.permute(2, 1, 0) @ local.transpose(0, 1).flatten(2)
    edge = (V - V[first][seq]) if not back else (U[last][seq] - U)
    return got.transpose(0, 1).reshape(local.shape) + edge.exp().float()[..., None, None] * start[seq]


def _plain_tokens(s):
    """A few rows for each sequence: the recurrence as it stands, all sequences that still have a row together."""
    hk, hv = s["hk"], s["hv"]
    q, k, v = (s[t].float().view(s["rows"], h, -1).repeat_interleave(hv // h, 1) for t, h in (("q", hk), ("k", hk), ("v", hv)))
    decay = torch.exp(s["g"] if s["g"].dim() == 2 else s["g"].expand(s["rows"], hv))
    page = s["page"].long()
    S, o = s["state_in"].float()[page], torch.empty_like(v)
    for live, at in s["tokens"]:
        now = S[live] * decay[at][..., None, None] + k[at][..., :, None] * v[at][..., None, :]
        o[at] = s["scale"] * (q[at][..., None, :] @ now)[..., 0, :]
        s["state_out"][page[live]] = now.to(s["state_out"].dtype)
        S[live] = now
    return {"o": o.view(s["rows"], -1).to(s["q"].dtype), "state": s["state_out"]}


def _plain_attend(s):
    """A chunk's rows meet each other by products of matrices, and what went before as a state."""
    at, seq, first, last = _chunk_rows(s)
    hk, hv, scale = s["hk"], s["hv"], s["scale"]
    q, k, v = _heads(s["q"], at, hk, hv // hk), _heads(s["k"], at, hk, hv // hk), _heads(s["v"], at, hv)
    g = s["g"] if s["g"].dim() == 2 else s["g"].expand(s["rows"], hv)
    G = torch.cat((g.double(), g.new_zeros(1, hv)))[at].transpose(1, 2).cumsum(-1)
    past = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=at.device).tril()
    D = torch.where(past, torch.exp(G[..., :, None] - G[..., None, :]).float(), 0.0)
    into, rest, whole = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None], torch.exp(G[..., -1]).float()[..., None, None]
    page = s["page"].long()
    some = (s["cu"][1:] > s["cu"][:-1]).nonzero()[:, 0]
    local = (k * rest).transpose(-1, -2) @ v
    before = _carried(local, G[..., -1], seq, s["state_in"].float()[page], first, last)
    end = last[some]
    s["state_out"][page[some]] = (whole[end] * before[end] + local[end]).to(s["state_out"].dtype)
    P = D * (q @ k.transpose(-1, -2))
    o = scale * (into * (q @ before) + P @ v)
    out = {"o": _packed(o, at, s).to(s["q"].dtype), "state": s["state_out"]}
    if s["kind"] == "attend":
        return out
    do = _heads(s["d_o"], at, hv)
    local = scale * ((q * into).transpose(-1, -2) @ do)
    after = _carried(local, G[..., -1], seq, s["d_state"], first, last, back=True)
    begin = first[some]
    d_state0 = s["d_state"].clone()
    d_state0[some] = whole[begin] * after[begin] + local[begin]
    A = do @ v.transpose(-1, -2)
    M = scale * P * A  # how much row j gives to row i's part of the loss
    A = D * A
    dq_in, dk_out = scale * into * (do @ before.transpose(-1, -2)), rest * (v @ after.transpose(-1, -2))
    dq = dq_in + scale * (A @ k)
    dk = dk_out + scale * (A.transpose(-1, -2) @ q)
    dv = rest * (k @ after) + scale * (P.transpose(-1, -2) @ do)
    # the decay of row t lies between the rows before it, and the state, and the rows from it on, and the state behind
    through = (whole * before * after).sum((-1, -2))[..., None]
    r, c = (q * dq_in).sum(-1), (k * dk_out).sum(-1)
    across = (M.cumsum(-1) - M).flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)
    dg = through + r.flip(-1).cumsum(-1).flip(-1) + (c.cumsum(-1) - c) + across
    dg = _packed(dg[..., None], at, s)
    act = s["q"].dtype
    return out | {"dq": _packed(dq, at, s, hv // hk).to(act), "dk": _packed(dk, at, s, hv // hk).to(act), "dv": _packed(dv, at, s).to(act),
                  "dg": dg if s["g"].dim() == 2 else dg.double().sum(0).float(), "d_state0": d_state0}


def _plain_cache(s):
    v = s["states"].float()[s["page"].long()]
    n, pad = v.shape[0], -s["dv"] % Q_COLS
    w = torch.cat((v, v.new_zeros(*v.shape[:-1], pad)), -1).unflatten(-1, (-1, Q_COLS))
    top = w.abs().amax(-1, keepdim=True).double()
    live = top >= 2.0 ** -100
    up, scale = torch.where(live, 127.0 / top, 0.0).float(), torch.where(live, top / 127.0, 0.0).float()
    kept = torch.round(w.double() * up.double()).float() * scale  # the product is exact in 64 bits: one rounding
    s["restored"][s["to"].long()] = kept.flatten(-2)[..., :s["dv"]].to(s["restored"].dtype)
    return {"restored": s["restored"]}


# ------------------------------------------------------- the package's calls


def _handles(s):
    """What a program keeps beside its tensors: dims, the batch, the pools, the cache and the workspaces."""
    import linear_attention_ssm_gdn_amd as g
    if s["kind"].startswith("rotate"):
        dims = g.RotateDims(s["hv"], s["hk"], s["dk"], s["rot"], act_dtype=s["act"], norm=s["norm"], pairs=s["pairs"], eps=EPS)
        ws = g.gdnl_rotate_workspace_bytes(dims, s["rows"])
        return {"g": g, "dims": dims, "ws": torch.empty(ws, dtype=torch.uint8, device=s["q"].device)}
    dims = g.LinearDims(s["hk"], s["hv"], s["dk"], s["dv"], act_dtype=s.get("act", "bf16"), state_dtype=s["state"], scale=s.get("scale", 1.0))
    if s["kind"] == "cache":
        return {"g": g, "dims": dims, "from": g.StatePool(s["states"]), "to": g.StatePool(s["restored"]), "cache": g.StateCache.alloc(dims, s["n"] + 5, s["states"].device)}
    train = s["kind"] == "attend_train"
    return {"g": g, "dims": dims, "batch": g.Batch(s["cu"], s["page"], None, s["max_len"], s["rows"]), "in": g.StatePool(s["state_in"]), "out": g.StatePool(s["state_out"]),
            "ws": torch.empty(g.gdnl_attend_workspace_bytes(dims, s["n"], s["rows"], backward=train), dtype=torch.uint8, device=s["q"].device)}


def _own_run(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    g, dims = h["g"], h["dims"]
    if s["kind"] == "cache":
        g.gdnl_cache_store(dims, s["page"], s["entry"], h["from"], h["cache"])
        g.gdnl_cache_load(dims, s["entry"], s["to"], h["cache"], h["to"])
        return {"restored": s["restored"]}
    if s["kind"].startswith("rotate"):
        yq, yk = g.gdnl_rotate_forward(dims, s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"])
        out = {"q": yq, "k": yk}
        if s["kind"] == "rotate_train":
            d = g.gdnl_rotate_backward(dims, s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"], s["d_yq"], s["d_yk"], workspace=h["ws"])
            out |= {"d_q": d.dq, "d_k": d.dk, "d_wq": d.dwq, "d_wk": d.dwk}
        return out
    o = g.gdnl_attend_forward(dims, s["q"], s["k"], s["v"], s["g"], h["batch"], h["in"], h["out"], workspace=h["ws"])
    out = {"o": o, "state": s["state_out"]}
    if s["kind"] == "attend_train":
        d = g.gdnl_attend_backward(dims, s["q"], s["k"], s["v"], s["g"], h["batch"], h["in"], s["d_o"], d_state=s["d_state"], workspace=h["ws"])
        out |= d._asdict()
    return out


def run(state):
    if own:
        return _own_run(state)
    if state["kind"] == "cache":
        return _plain_cache(state)
    if state["kind"].startswith("rotate"):
        return _plain_rotate(state)
    return _plain_tokens(state) if state["kind"] == "attend" and state["max_len"] <= 4 else _plain_attend(state)


def work(case):
    lens = [int(v) for v in case["lens"].split(",")]
    n, rows = len(lens), sum(lens)
    hk, hv, dk, dv = (case[k] for k in ("hk", "hv", "dk", "dv"))
    act, st = (2 if case["act"] == "bf16" else 4), (2 if case["state"] == "bf16" else 4)
    if case["kind"] == "cache":  # pages read and written, entries written and read
        e = n * hv * dk
        return {"bytes": 2 * e * (dv * (st + 1) + 4 * -(-dv // Q_COLS)), "flops": 5 * e * dv}
    if case["kind"].startswith("rotate"):
        e, train = rows * (hv + hk) * dk, case["kind"] == "rotate_train"
        return {"bytes": (4 if train else 2) * act * e + (2 if train else 1) * (4 * rows + 8 * dk) + (act * e if train else 0), "flops": (30 if train else 9) * e}
    state, qkv, gates = n * hv * dk * dv, rows * (2 * hk * dk + hv * dv), 4 * hv * (rows if case["decay"] == "row" else 1)
    if case["kind"] == "attend":  # q, k, v -> o; the states.  A row's own share of the recurrence: decay, update, product with q
        return {"bytes": act * (qkv + rows * hv * dv) + gates + 2 * st * state, "flops": 4 * rows * hv * dk * dv}
    # q, k, v, do -> o, dq, dk, dv; the gates and states and their gradients
    return {"bytes": act * 2 * (qkv + rows * hv * dv) + 2 * gates + state * (2 * st + 8), "flops": 14 * rows * hv * dk * dv}


# ------------------------------------------- the definitions, row by row in 64 bits


def _exact_rotate(s):
    D = torch.float64
    rows, d, rot = s["rows"], s["dk"], s["rot"]
    first = torch.arange(rot // 2, device=s["pos"].device) * (2 if s["pairs"] == "neighbours" else 1)
    second = first + (1 if s["pairs"] == "neighbours" else rot // 2)
    turn = torch.polar(torch.ones((), dtype=D, device=first.device), s["pos"].to(D)[:, None] * s["inv_freq"].to(D))[:, None]

    def turned(y, t):
        y = y.clone()
        z = torch.complex(y[..., first], y[..., second]) * t
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    for t in ("q", "k"):
        x, w = s[t].to(D).view(rows, -1, d), s["w" + t].to(D)
        size = (x.square().sum(-1, keepdim=True) / (d if s["norm"] == "rms" else 1) + EPS).sqrt()
        out[t] = turned(x / size * w, turn).reshape(rows, -1)
        if s["kind"] == "rotate_train":
            dy = turned(s["d_y" + t].to(D).view(x.shape), turn.conj())
            along = (dy * w * x).sum(-1, keepdim=True) / (d if s["norm"] == "rms" else 1)
            out["d_" + t] = (dy * w / size - x * along / size ** 3).reshape(rows, -1)
            out["d_w" + t] = (dy * x / size).sum((0, 1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    D = torch.float64
    if case["kind"].startswith("rotate"):
        return _exact_rotate(s)
    if case["kind"] == "cache":
        out = s["restored"].to(D)
        for c in range(0, s["dv"], Q_COLS):
            v = s["states"][s["page"].long()][..., c:c + Q_COLS].to(D)
            top = v.abs().amax(-1, keepdim=True)
            live = top >= 2.0 ** -100  # both scales are fp32 by definition
            out[s["to"].long(), ..., c:c + Q_COLS] = (v * torch.where(live, (127.0 / top).float().to(D), 0.0)).round() * torch.where(live, (top / 127.0).float().to(D), 0.0)
        return {"restored": out}
    lens, cu, page = s["lens_host"], s["cu_host"], s["page"].long()
    hk, hv, dk, dv, rows, scale = s["hk"], s["hv"], s["dk"], s["dv"], s["rows"], s["scale"]
    train = case["kind"] == "attend_train"
    order = sorted(range(len(lens)), key=lambda i: -lens[i])
    live = [sum(v > t for v in lens) for t in range(max(lens))]  # sequences that still have a row t
    perm = torch.tensor(order, device=page.device)
    base = torch.tensor([cu[i] for i in order], device=page.device)

    def heads(name, h):
        t = s[name].to(D).view(rows, h, -1)
        return t.repeat_interleave(hv // h, 1)

    q, k, v = heads("q", hk), heads("k", hk), heads("v", hv)
    g = (s["g"] if s["g"].dim() == 2 else s["g"].expand(rows, hv)).to(D)
    decay = g.exp()[..., None, None]
    S = s["state_in"].to(D)[page][perm]
    o = torch.empty_like(v)
    if train:
        do, dq, dkk, dvv = heads("d_o", hv), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t, m in enumerate(live):
        at = base[:m] + t
        S[:m] = S[:m] * decay[at] + k[at][..., :, None] * v[at][..., None, :]
        o[at] = scale * (q[at][..., None, :] @ S[:m])[..., 0, :]
        if train:
            dq[at] = scale * (S[:m] @ do[at][..., :, None])[..., 0]
    state = s["state_out"].to(D)
    final = torch.empty_like(S)
    final[perm] = S
    some = torch.tensor([i for i, v_ in enumerate(lens) if v_ > 0], device=page.device)
    state[page[some]] = final[some]
    out = {"o": o.view(rows, -1), "state": state}
    if not train:
        return out
    E = s["d_state"].to(D)[perm]
    dG = (q * dq).sum(-1)
    for i, length in enumerate(lens):
        if length > 0:
            dG[cu[i + 1] - 1] += (final[i] * s["d_state"][i].to(D)).sum((-1, -2))
    for t in range(len(live) - 1, -1, -1):
        m = live[t]
        at = base[:m] + t
        E[:m] += scale * q[at][..., :, None] * do[at][..., None, :]
        dkk[at] = (E[:m] @ v[at][..., :, None])[..., 0]
        dvv[at] = (k[at][..., None, :] @ E[:m])[..., 0, :]
        E[:m] *= decay[at]
    dG -= (k * dkk).sum(-1)
    dg = torch.cat([dG[cu[i]:cu[i + 1]].flip(0).cumsum(0).flip(0) for i in range(len(lens))])
    d0 = torch.empty_like(E)
    d0[perm] = E
    group = lambda t: t.view(rows, hk, hv // hk, dk).sum(2).view(rows, -1)  # noqa: E731
    return out | {"dq": group(dq), "dk": group(dkk), "dv": dvv.view(rows, -1), "dg": dg if s["g"].dim() == 2 else dg.sum(0), "d_state0": d0}
