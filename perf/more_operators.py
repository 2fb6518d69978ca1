"""The operators between blocks, and the gated linear recurrence, measured: the residual stream's addition with its
dropout and root-mean-square norm (to the data type, or to 8 bits with scales; forward and backward), and the
recurrence over prompts, training batches and single tokens.

With ``own`` false, ``run`` computes them from their formulas in elementary torch operations; with ``own``
true it calls ``mamba_mimo_chunked_amd``. Sequences are handled as rows of one flat axis in both the plain
form and the reference in 64 bits: a dense batch is the packed batch of equal lengths.
"""

import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS, _RATE = 1e-5, 8.0
_TOP = {"e4m3": 448.0, "int8": 127.0}
_LEAST = 2.0 ** -100    # of the largest magnitude that a scale is made from


def listed():
    return [
        # token generation for one sequence: latency alone
        dict(name="recur_step_one", op="recur_step", seqs=1, width=1024, dtype="bf16", slots=1, gate=True, bias=True),
        # token generation for a batch whose states lie in a pool
        dict(name="recur_step_pool", op="recur_step", seqs=128, width=2048, dtype="fp16", slots=160, gate=True, bias=True),
        # one long prompt: little parallel work beside the long axis
        dict(name="recur_prompt", op="recur_fwd", seqs=1, tokens=8192, packed=False, width=2048, dtype="bf16", gate=True, bias=True),
        # prompts of unequal lengths, an odd width, full precision, the output gated elsewhere
        dict(name="recur_prompt_packed", op="recur_fwd", seqs=7, tokens=4100, packed=True, width=517, dtype="fp32", gate=False, bias=True),
        # a training batch
        dict(name="recur_train", op="recur_bwd", seqs=4, tokens=16384, packed=False, width=2048, dtype="bf16", gate=True, bias=True),
        # a small odd training batch of packed sequences
        dict(name="recur_train_odd", op="recur_bwd", seqs=3, tokens=903, packed=True, width=200, dtype="fp16", gate=True, bias=False),
        # token generation for one sequence, into an 8-bit product: latency alone
        dict(name="add_norm_token", op="add_norm_fwd", tokens=1, width=1024, dtype="bf16", wide=False, add=True, drop=0.0, to="e4m3", block=0),
        # a prompt into an 8-bit product with a scale for every 128 columns, the stream in full precision
        dict(name="add_norm_prompt", op="add_norm_fwd", tokens=8192, width=2048, dtype="bf16", wide=True, add=True, drop=0.0, to="e4m3", block=128),
        # the first block's norm, nothing added, into an integer product; a width that no access divides
        dict(name="add_norm_int8", op="add_norm_fwd", tokens=301, width=1003, dtype="fp16", wide=False, add=False, drop=0.0, to="int8", block=0),
        # training with dropout in front of the addition
        dict(name="add_norm_dropout", op="add_norm_fwd", tokens=8192, width=2048, dtype="bf16", wide=True, add=True, drop=0.1, to="", block=0),
        # its gradient, an odd number of rows
        dict(name="add_norm_train", op="add_norm_bwd", tokens=4100, width=4096, dtype="bf16", wide=False, add=True, drop=0.1),
        # a small odd training batch in full precision, without dropout
        dict(name="add_norm_train_odd", op="add_norm_bwd", tokens=1003, width=517, dtype="fp32", wide=False, add=True, drop=0.0),
    ]


def _between(rng, lo, hi):
    """Whole numbers from lo to hi, spread over their logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["recur_fwd", "recur_bwd", "recur_step", "add_norm_fwd", "add_norm_fwd", "add_norm_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op.startswith("add_norm"):
        c.update(tokens=_between(rng, 1, 8192), width=_between(rng, 16, 4096), wide=rng.random() < 0.4, add=rng.random() < 0.8,
                 drop=rng.choice([0.0, 0.0, 0.1, 0.25]))
        if op == "add_norm_fwd":
            c.update(to=rng.choice(["", "e4m3", "e4m3", "int8"]), block=rng.choice([0, 0, 32, 128]))
            c.update(block=c["block"] if c["to"] else 0)
        return c
    seqs = _between(rng, 1, 128 if op.endswith("step") else 16)
    c.update(seqs=seqs, gate=rng.random() < 0.7, bias=rng.random() < 0.7, width=_between(rng, 16, 2048))
    if op.endswith("step"):
        c.update(slots=seqs + rng.choice([0, 0, 3, 40]))
    else:
        each = _between(rng, 1, 16384 // seqs)
        c.update(packed=rng.random() < 0.5)
        c.update(tokens=seqs * each + (rng.randrange(seqs) if c["packed"] and each < 16384 // seqs else 0))
    return c


# ------------------------------------------------------------------------------------------------- inputs
def _cuts(case, gen):
    """Where the sequences begin and end, as numbers: equal lengths, or random ones (some may be empty)."""
    n, total = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [i * (total // n) for i in range(n + 1)]
    inner = torch.randint(0, total + 1, (n - 1,), generator=gen).sort().values.tolist()
    return [0] + inner + [total]


def _rows(case, cuts, device):
    """Where sequences lie on the flat axis, as a program that packs its batch has it in hand."""
    cu = torch.tensor(cuts, device=device)
    return {"cu": cu, "full": torch.nonzero(cu[1:] > cu[:-1])[:, 0], "longest": max(b - a for a, b in zip(cuts, cuts[1:]))}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    t, f32 = _TYPES[case["dtype"]], torch.float32
    op, D = case["op"], case["width"]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    s = {"case": dict(case)}
    if op.startswith("add_norm"):
        T, stream = case["tokens"], f32 if case["wide"] else t
        s["weight"] = 1 + 0.1 * normal(D, dtype=f32)
        s["seed"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=gen, device=dev) if case["drop"] else None
        if op == "add_norm_fwd":
            s["x"] = normal(T, D)
            # the stream has grown over the blocks before, in some channels more than in others
            s["residual"] = (3 * normal(T, D, dtype=f32) * (0.5 + torch.rand(D, generator=gen, device=dev))).to(stream) if case["add"] else None
        else:
            s["sum"] = (3 * normal(T, D, dtype=f32) * (0.5 + torch.rand(D, generator=gen, device=dev))).to(stream)
            s["dout"], s["dsum"] = normal(T, D), normal(T, D, dtype=stream)
        return s
    n = case["seqs"]
    if op.endswith("step"):
        lead = (n,)
        s["indices"] = torch.randperm(case["slots"], generator=gen, device=dev)[:n].to(torch.int32) if case["slots"] > 1 else None
    else:
        cuts = _cuts(case, host)
        s["rows"] = _rows(case, cuts, dev)
        s["cu_seqlens"] = s["rows"]["cu"].to(torch.int32) if case["packed"] else None
        lead = (cuts[-1],) if case["packed"] else (n, cuts[-1] // n)
    s["x"] = normal(*lead, D)                        # from the short convolution
    gates = normal(*lead, 2 * D)                     # one projection gives both gates
    s["r"], s["i"] = gates[..., :D], gates[..., D:]
    s["z"] = normal(*lead, 2 * D)[..., D:] if case["gate"] else None     # the other half of the input projection's rows
    # with an open gate a channel keeps 0.9 to 0.999 of its state
    keep = 0.9 + 0.099 * torch.rand(D, generator=gen, device=dev)
    s["decay"] = torch.log(torch.expm1(-torch.log(keep) / _RATE))
    s["r_bias"], s["i_bias"] = (normal(D, scale=0.3, dtype=f32), normal(D, scale=0.3, dtype=f32)) if case["bias"] else (None, None)
    if op == "recur_step":
        s["state"] = normal(case["slots"], D, dtype=f32)
    else:
        s["initial"] = normal(n, D, dtype=f32)
    if op == "recur_bwd":
        s["dout"] = normal(*lead, D)
        s["dstate"] = normal(n, D, dtype=f32)
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _flat(x):
    """A dense or packed batch as rows of one axis, in 32 bits."""
    return x.reshape(-1, x.shape[-1]).float()


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _silu_slope(x):
    g = _sigmoid(x)
    return g * (1 + x * (1 - g))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _recur(a, b, longest):
    """h with h_t = a_t h_{t-1} + b_t along the first axis, a zero where a sequence begins: the products and sums of
    1, 2, 4, ... tokens, each from two of the half length."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]]) if 2 * step < longest else a
        step *= 2
    return b


def _gates(s):
    """The inputs in 32 bits, the gates, the logarithm of what is kept, and what of the input enters."""
    x, r, i = (_flat(s[k]) for k in ("x", "r", "i"))
    r = _sigmoid(r if s["r_bias"] is None else r + s["r_bias"])
    i = _sigmoid(i if s["i_bias"] is None else i + s["i_bias"])
    kept = -_RATE * _softplus(s["decay"]) * r
    return x, r, i, kept, torch.sqrt(-torch.expm1(2 * kept))


def _recur_parts(s):
    rows = s["rows"]
    x, r, i, kept, enter = _gates(s)
    a = torch.exp(kept)
    full = rows["full"]
    begin, end = rows["cu"][full], rows["cu"][full + 1] - 1
    add = enter * i * x
    add[begin] = add[begin] + a[begin] * s["initial"][full]
    inner = a.clone()
    inner[begin] = 0
    return x, r, i, kept, enter, a, inner, _recur(inner, add, rows["longest"]), begin, end, full


def _recur_fwd(s):
    h, _, end, full = _recur_parts(s)[-4:]
    state = s["initial"].clone()
    state[full] = h[end]
    if s["z"] is not None:
        z = _flat(s["z"])
        h = h * z * _sigmoid(z)
    return {"out": h.to(s["x"].dtype).reshape(s["x"].shape), "state": state}


def _recur_bwd(s):
    t, shape = s["x"].dtype, s["x"].shape
    x, r, i, kept, enter, a, inner, h, begin, end, full = _recur_parts(s)
    dout = _flat(s["dout"])
    out = {}
    dh = dout
    if s["z"] is not None:
        z = _flat(s["z"])
        dh = dout * z * _sigmoid(z)
        out["dz"] = (dout * h * _silu_slope(z)).to(t).reshape(shape)
    add = dh.clone()
    add[end] = add[end] + s["dstate"][full]
    later = torch.cat([inner[1:], torch.zeros_like(inner[:1])])
    g = _recur(later.flip(0), add.flip(0), s["rows"]["longest"]).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[begin] = s["initial"][full]
    share = torch.where(enter > 0, kept / enter, 0)
    w = g * (kept * a * before - share * a * a * i * x)
    du = g * enter
    dr, di = (1 - r) * w, du * x * i * (1 - i)
    sp = _softplus(s["decay"])
    dinitial = s["dstate"].clone()
    dinitial[full] = a[begin] * g[begin]
    out.update(dx=(du * i).to(t).reshape(shape), dr=dr.to(t).reshape(shape), di=di.to(t).reshape(shape),
               ddecay=w.sum(0) * _sigmoid(s["decay"]) / sp, dinitial_state=dinitial)
    if s["r_bias"] is not None:
        out.update(dr_bias=dr.sum(0), di_bias=di.sum(0))
    return out


def _recur_step(s):
    x, r, i, kept, enter = _gates(s)
    state = s["state"]
    at = s["indices"].long() if s["indices"] is not None else torch.arange(x.shape[0], device=state.device)
    h = torch.exp(kept) * state[at] + enter * i * x
    state[at] = h
    if s["z"] is not None:
        z = s["z"].float()
        h = h * z * _sigmoid(z)
    return {"out": h.to(s["x"].dtype), "state": state}


def _kept(s, T, D, device):
    """Which elements dropout keeps, and their factor: Philox4x32 with ten rounds gives eight elements of a row their 16 bits."""
    cut = int(s["case"]["drop"] * 65536 + 0.5)
    low = 0xffffffff
    seed, offset = s["seed"][0], s["seed"][1]
    shape = (T, -(-D // 8))
    c0, c1, c2, c3 = (v.expand(shape) for v in (torch.arange(shape[1], device=device), torch.arange(T, device=device)[:, None],
                                                 offset & low, (offset >> 32) & low))
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([c & 0xffff if half == 0 else c >> 16 for c in (c0, c1, c2, c3) for half in (0, 1)], -1)
    return bits.reshape(T, -1)[:, :D] >= cut, 65536 / (65536 - cut)


def _add_norm_fwd(s):
    case, t, D = s["case"], s["x"].dtype, s["case"]["width"]
    v = s["x"].float()
    if case["drop"]:
        keep, factor = _kept(s, *v.shape, v.device)
        v = torch.where(keep, v * factor, 0)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    out = v / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS) * s["weight"]
    stream = torch.float32 if case["wide"] else t
    res = {"sum": v.to(stream)}
    if not case["to"]:
        return {**res, "out": out.to(t)}
    width = case["block"] or D
    blocks = -(-D // width)
    padded = torch.cat([out, out.new_zeros(out.shape[0], blocks * width - D)], 1).reshape(-1, blocks, width)
    scale = padded.abs().amax(-1).clamp(min=_LEAST) / _TOP[case["to"]]
    q = (padded / scale[..., None]).reshape(out.shape[0], -1)[:, :D]
    if case["to"] == "e4m3":
        return {**res, "out": q.to(torch.float8_e4m3fn), "scale": scale}
    q = q.round().reshape(out.shape[0], D)
    return {**res, "out": _values(q.to(torch.int8), scale, width), "scale": scale}


def _values(q, scale, width):
    """What whole numbers in 8 bits stand for."""
    return (q * scale.repeat_interleave(width, 1)[:, :q.shape[1]]).to(torch.bfloat16)


def _add_norm_bwd(s):
    case = s["case"]
    v, dout = s["sum"].float(), s["dout"].float()
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)
    hat, q = v * r, dout * s["weight"]
    dv = r * (q - hat * (q * hat).mean(-1, keepdim=True)) + s["dsum"].float()
    dx = dv
    if case["drop"]:
        keep, factor = _kept(s, *v.shape, v.device)
        dx = torch.where(keep, dv * factor, 0)
    out = {"dx": dx.to(s["dout"].dtype), "dweight": (dout * hat).sum(0)}
    if case["add"] and (case["drop"] or s["sum"].dtype != s["dout"].dtype):
        out["dresidual"] = dv.to(s["sum"].dtype)     # elsewhere it is dx
    return out


_PLAIN = {"recur_fwd": _recur_fwd, "recur_bwd": _recur_bwd, "recur_step": _recur_step, "add_norm_fwd": _add_norm_fwd, "add_norm_bwd": _add_norm_bwd}


# ------------------------------------------------------------------------------------------------- the framework's calls
def _own(s):
    import mamba_mimo_chunked_amd as m

    case = s["case"]
    if case["op"] == "recur_fwd":
        o = m.mamba_recur_fwd(s["x"], s["r"], s["i"], s["decay"], s["r_bias"], s["i_bias"], s["z"], s["initial"], s["cu_seqlens"],
                              rate=_RATE, return_state=True)
        return {"out": o.out, "state": o.state}
    if case["op"] == "recur_bwd":
        g = m.mamba_recur_bwd(s["dout"], s["x"], s["r"], s["i"], s["decay"], s["r_bias"], s["i_bias"], s["z"], s["initial"], s["dstate"],
                              s["cu_seqlens"], rate=_RATE)
        return {k: v for k, v in g._asdict().items() if v is not None}
    if case["op"] == "recur_step":
        return {"out": m.mamba_recur_step(s["x"], s["r"], s["i"], s["state"], s["decay"], s["r_bias"], s["i_bias"], s["z"], s["indices"],
                                          rate=_RATE), "state": s["state"]}
    if case["op"] == "add_norm_fwd":
        kinds = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
        o = m.mamba_add_norm_fwd(s["x"], s["weight"], s["residual"], eps=_EPS, dropout=case["drop"], seed=s["seed"],
                                 sum_dtype=torch.float32 if case["wide"] else None, out_dtype=kinds.get(case["to"]), block=case["block"] or None)
        res = {"sum": o.sum, "out": o.out}
        if case["to"]:
            res["scale"] = o.scale
        if case["to"] == "int8":
            res["out"] = _values(o.out, o.scale, case["block"] or case["width"])
        return res
    g = m.mamba_add_norm_bwd(s["dout"], s["sum"], s["weight"], s["dsum"], eps=_EPS, dropout=case["drop"], seed=s["seed"], residual=case["add"])
    out = {"dx": g.dx, "dweight": g.dweight}
    if g.dresidual is not None and g.dresidual is not g.dx:
        out["dresidual"] = g.dresidual
    return out


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------- in 64 bits
def _exact_recur(s):
    """The recurrence as it is defined, one token after another for all sequences, and its adjoint backwards."""
    case, F = s["case"], torch.nn.functional
    D = case["width"]
    speed = _RATE * F.softplus(s["decay"].double(), threshold=60)
    zero = torch.zeros(D, dtype=torch.float64, device=speed.device)
    rb, ib = (zero if s[k] is None else s[k].double() for k in ("r_bias", "i_bias"))
    x, pr, pi = (s[k].double().reshape(-1, D) for k in ("x", "r", "i"))
    z = None if s["z"] is None else s["z"].double().reshape(-1, D)

    def token(row, h):
        """(open gate, input gate, factor of the state, factor of the input, new state)"""
        r, i = torch.sigmoid(pr[row] + rb), torch.sigmoid(pi[row] + ib)
        a = torch.exp(-speed * r)
        enter = torch.sqrt((1 - a) * (1 + a))
        return r, i, a, enter, h * a + x[row] * i * enter

    if case["op"] == "recur_step":
        at = list(range(case["seqs"])) if s["indices"] is None else s["indices"].tolist()
        state = s["state"].double()
        h = token(slice(None), state[at])[-1]
        state[at] = h
        return {"out": h if z is None else h * F.silu(z), "state": state}
    cu = s["rows"]["cu"]
    lens = (cu[1:] - cu[:-1]).tolist()
    rank = sorted(range(case["seqs"]), key=lambda k: -lens[k])     # the longest first: those still running are a prefix
    order = torch.tensor(rank, device=cu.device)
    first = cu[order]
    past, now = torch.empty_like(x), torch.empty_like(x)
    h = s["initial"].double()[order]
    running = [sum(1 for k in rank if lens[k] > t) for t in range(lens[rank[0]])]
    for t, k in enumerate(running):
        row = first[:k] + t
        past[row] = h[:k]
        h[:k] = token(row, h[:k])[-1]
        now[row] = h[:k]
    if case["op"] == "recur_fwd":
        state = torch.empty_like(h)
        state[order] = h
        return {"out": (now if z is None else now * F.silu(z)).reshape(s["x"].shape), "state": state}
    dout = s["dout"].double().reshape(-1, D)
    dh, res = dout, {}
    if z is not None:
        sg = torch.sigmoid(z)
        dh, res["dz"] = dout * z * sg, (dout * now * (sg + z * sg * (1 - sg))).reshape(s["x"].shape)
    g, c = torch.empty_like(x), s["dstate"].double()[order]
    for t in range(len(running) - 1, -1, -1):
        k = running[t]
        row = first[:k] + t
        g[row] = dh[row] + c[:k]
        c[:k] = g[row] * torch.exp(-speed * torch.sigmoid(pr[row] + rb))
    dinitial = torch.empty_like(c)
    dinitial[order] = c
    r, i, a, enter, _ = token(slice(None), past)
    da = g * (past - x * i * a / enter)
    dspeed = -(da * a * r).sum(0)
    dr = -da * a * speed * r * (1 - r)
    di = g * x * enter * i * (1 - i)
    res.update(dx=(g * i * enter).reshape(s["x"].shape), dr=dr.reshape(s["x"].shape), di=di.reshape(s["x"].shape),
               ddecay=dspeed * _RATE * torch.sigmoid(s["decay"].double()), dinitial_state=dinitial)
    if s["r_bias"] is not None:
        res.update(dr_bias=dr.sum(0), di_bias=di.sum(0))
    return res


def _drawn_bits(s, T, D):
    """The 16 bits of every element, by numpy: one counter a row and eight columns."""
    seed, offset = (int(v) & (2 ** 64 - 1) for v in s["seed"].tolist())
    word, u = np.uint64(32), np.uint64
    low = u(0xffffffff)
    ctr = np.empty((4, T, -(-D // 8)), dtype=u)
    ctr[0], ctr[1], ctr[2], ctr[3] = np.arange(ctr.shape[2], dtype=u), np.arange(T, dtype=u)[:, None], u(offset) & low, u(offset) >> word
    for k in range(10):
        key = [u(((seed & 0xffffffff) + k * 0x9E3779B9) & 0xffffffff), u(((seed >> 32) + k * 0xBB67AE85) & 0xffffffff)]
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = np.stack([(b >> word) ^ ctr[1] ^ key[0], b & low, (a >> word) ^ ctr[3] ^ key[1], a & low])
    halves = np.ascontiguousarray(np.moveaxis(ctr, 0, -1), dtype="<u4").view("<u2")
    return halves.reshape(T, -1)[:, :D]


def _exact_add_norm(s):
    case = s["case"]
    f = 1.0
    source = s["x"] if case["op"] == "add_norm_fwd" else s["sum"]
    T, D = source.shape
    if case["drop"]:
        cut = int(case["drop"] * 65536 + 0.5)
        keep = torch.from_numpy((_drawn_bits(s, T, D).astype(np.int32) >= cut)).to(source.device)
        f = keep.double() / (1 - cut / 65536)
    w = s["weight"].double()
    if case["op"] == "add_norm_fwd":
        v = source.double() * f
        v = v if s["residual"] is None else v + s["residual"].double()
        out = w * v * torch.rsqrt(v.square().sum(-1, keepdim=True) / D + _EPS)
        if not case["to"]:
            return {"sum": v, "out": out}
        width = case["block"] or D
        scale = torch.stack([part.abs().amax(-1) for part in out.split(width, 1)], 1).clamp(min=_LEAST) / _TOP[case["to"]]
        wide = torch.cat([scale[:, k:k + 1].expand(T, part.shape[1]) for k, part in enumerate(out.split(width, 1))], 1)
        q = out / wide
        return {"sum": v, "out": q if case["to"] == "e4m3" else torch.round(q) * wide, "scale": scale}
    leaf = source.double().requires_grad_()
    wl = w.requires_grad_()
    with torch.enable_grad():
        out = wl * leaf * torch.rsqrt(leaf.square().sum(-1, keepdim=True) / D + _EPS)
        dv, dw = torch.autograd.grad(out, (leaf, wl), s["dout"].double())
    dv = dv + s["dsum"].double()
    res = {"dx": dv * f, "dweight": dw}
    if case["add"] and (case["drop"] or s["sum"].dtype != s["dout"].dtype):
        res["dresidual"] = dv
    return res


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_recur(s) if case["op"].startswith("recur") else _exact_add_norm(s)


# ------------------------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, D = case["op"], case["width"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op.startswith("add_norm"):
        T, stream = case["tokens"], 4 if case["wide"] else size
        if op == "add_norm_bwd":
            apart = case["add"] and (case["drop"] > 0 or stream != size)
            return {"bytes": T * D * (2 * size + (3 if apart else 2) * stream) + 8 * D, "flops": 16 * T * D}
        moved = case["add"] or case["drop"] > 0 or stream != size      # else the sum is the input
        blocks = (-(-D // case["block"]) if case["block"] else 1) if case["to"] else 0
        per = size + (stream if case["add"] else 0) + (stream if moved else 0) + (1 if case["to"] else size)
        return {"bytes": T * (D * per + 4 * blocks) + 4 * D, "flops": 8 * T * D}
    n = case["seqs"]
    T = n if op.endswith("step") else case["tokens"]
    state, weight = n * D * 4, (3 if case["bias"] else 1) * D * 4
    if op == "recur_bwd":
        return {"bytes": (9 if case["gate"] else 7) * T * D * size + 3 * state + 2 * weight, "flops": 70 * T * D}
    return {"bytes": (5 if case["gate"] else 4) * T * D * size + 2 * state + weight, "flops": 35 * T * D}
