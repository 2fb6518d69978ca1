"""The layer operators around the scan, measured: the short causal convolution, the selective scan and the
gated group norm, each forward and backward over prompts and packed batches, and as a step of one token.

With ``own`` false, ``run`` computes them from their formulas in elementary torch operations; with ``own``
true it calls ``mamba_mimo_chunked_amd``. Sequences are handled as rows of one flat axis in both the plain
form and the reference in 64 bits: a dense batch is the packed batch of equal lengths.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-5


def listed():
    return [
        # token generation for one sequence: latency alone
        dict(name="conv_step_one", op="conv_step", seqs=1, width=1024, taps=4, dtype="bf16", slots=1),
        # a long prompt; x is one half of the input projection's rows, and the state goes on to generation
        dict(name="conv_prompt", op="conv_fwd", seqs=1, tokens=8192, packed=False, width=2048, taps=4, dtype="bf16"),
        # a training batch with a length that no tile divides
        dict(name="conv_train", op="conv_bwd", seqs=4, tokens=16400, packed=False, width=2048, taps=4, dtype="bf16"),
        # ragged sequences in one packed batch, rows that are not aligned, full precision
        dict(name="conv_train_packed", op="conv_bwd", seqs=11, tokens=5003, packed=True, width=517, taps=3, dtype="fp32"),
        # token generation for one sequence: latency alone
        dict(name="scan_step_one", op="scan_step", seqs=1, width=1024, state=16, groups=1, dtype="bf16", slots=1),
        # token generation for a batch whose states lie in a pool
        dict(name="scan_step_pool", op="scan_step", seqs=128, width=2048, state=64, groups=4, dtype="bf16", slots=160),
        # one long prompt: little parallel work beside the long axis
        dict(name="scan_prompt", op="scan_fwd", seqs=1, tokens=8192, packed=False, width=1024, state=16, groups=1, dtype="bf16"),
        # prompts of unequal lengths, a wide state, several groups
        dict(name="scan_prompt_packed", op="scan_fwd", seqs=7, tokens=4100, packed=True, width=2048, state=64, groups=4, dtype="fp16"),
        # a training batch
        dict(name="scan_train", op="scan_bwd", seqs=4, tokens=16384, packed=False, width=1024, state=16, groups=1, dtype="bf16"),
        # a small odd training batch in full precision
        dict(name="scan_train_odd", op="scan_bwd", seqs=3, tokens=903, packed=True, width=200, state=24, groups=2, dtype="fp32"),
        # the norm behind a prompt's scan, gate before it, eight groups
        dict(name="norm_prompt", op="norm_fwd", tokens=8192, width=2048, groups=8, center=False, gate="before", bias=False, dtype="bf16"),
        # its gradient in training: one group, mean taken out, gate after it, an odd number of rows
        dict(name="norm_train", op="norm_bwd", tokens=4100, width=4096, groups=1, center=True, gate="after", bias=True, dtype="fp16"),
    ]


def _between(rng, lo, hi):
    """Whole numbers from lo to hi, spread over their logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_bwd", "scan_step", "norm_fwd", "norm_bwd"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op.startswith("norm"):
        c.update(tokens=_between(rng, 1, 8192), groups=rng.choice([1, 2, 4, 8]))
        c.update(width=c["groups"] * _between(rng, 16, 4096 // c["groups"]), center=rng.random() < 0.5,
                 gate=rng.choice(["before", "after", "none", "silu"]), bias=rng.random() < 0.5)
        return c
    seqs = _between(rng, 1, 128 if op.endswith("step") else 16)
    c.update(seqs=seqs)
    if op.endswith("step"):
        c.update(slots=seqs + rng.choice([0, 0, 3, 40]))
    else:
        each = _between(rng, 1, 16384 // seqs)
        c.update(packed=rng.random() < 0.5)
        c.update(tokens=seqs * each + (rng.randrange(seqs) if c["packed"] else 0))
    if op.startswith("conv"):
        c.update(width=_between(rng, 16, 2048), taps=rng.choice([2, 3, 4, 4, 4]))
    else:
        c.update(groups=rng.choice([1, 1, 2, 4]), state=rng.choice([1, 4, 8, 13, 16, 16, 16, 24, 32, 64]))
        most = 4096 * 16 // (max(16, c["state"]) * c["groups"]) if not op.endswith("step") else 2048 // c["groups"]
        c.update(width=c["groups"] * _between(rng, 8, min(most, 1024 // c["groups"])))
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
    """Index tensors over the flat axis that a program packing its batch has in hand."""
    cu = torch.tensor(cuts, device=device)
    lens = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=device), lens, output_size=cuts[-1])
    return {"cu": cu, "seq": seq, "full": torch.nonzero(lens > 0)[:, 0], "longest": max(b - a for a, b in zip(cuts, cuts[1:]))}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))
    t = _TYPES[case["dtype"]]
    op, D = case["op"], case["width"]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = {"case": dict(case)}
    f32 = torch.float32
    if op.startswith("norm"):
        T = case["tokens"]
        xz = normal(T, 2 * D)                       # the two halves come from one buffer, as projections give them
        s["x"] = xz[:, :D]
        s["z"] = xz[:, D:] if case["gate"] in ("before", "after") else None
        s["weight"] = 1 + 0.1 * normal(D, dtype=f32)
        s["bias"] = 0.1 * normal(D, dtype=f32) if case["bias"] else None
        s["dout"] = normal(T, D) if op == "norm_bwd" else None
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
    if op.startswith("conv"):
        W = case["taps"]
        s["x"] = normal(*lead, 2 * D)[..., :D]       # one half of the input projection's rows
        s["weight"] = uniform(D, W, lo=-1, hi=1) / math.sqrt(W)
        s["bias"] = uniform(D, lo=-1, hi=1) / math.sqrt(W)
        if op == "conv_step":
            s["state"] = normal(case["slots"], W - 1, D)
        else:
            s["initial"] = normal(n, W - 1, D)
        if op == "conv_bwd":
            s["dout"] = normal(*lead, D)
            s["dstate"] = normal(n, W - 1, D)
        return s
    N, G = case["state"], case["groups"]
    s["u"] = normal(*lead, D)
    s["dt"] = normal(*lead, D, scale=0.5)
    s["z"] = normal(*lead, 2 * D)[..., D:]
    s["b"] = normal(*lead, G, N)
    s["c"] = normal(*lead, G, N)
    # decays -1..-N, slightly off; step sizes from 0.001 to 0.1 through the softplus; a skip near one
    s["a"] = -(torch.arange(1, N + 1, device=dev, dtype=f32).expand(D, N) * uniform(D, N, lo=0.9, hi=1.1)).contiguous()
    dt0 = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(0.1)))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    s["d"] = 1 + 0.1 * normal(D, dtype=f32)
    if op == "scan_step":
        s["state"] = normal(case["slots"], D, N, scale=0.3, dtype=f32)
    else:
        s["initial"] = normal(n, D, N, scale=0.3, dtype=f32)
    if op == "scan_bwd":
        s["dout"] = normal(*lead, D)
        s["dstate"] = normal(n, D, N, scale=0.3, dtype=f32)
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _flat(x, keep):
    """A dense or packed batch as rows of one axis, in 32 bits; `keep` trailing axes stay."""
    return x.reshape(-1, *x.shape[x.dim() - keep:]).float()


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _silu_slope(x):
    g = _sigmoid(x)
    return g * (1 + x * (1 - g))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _extended(s, x, initial, W):
    """The rows of every sequence behind its W - 1 rows of state, and where the tokens and the state's rows are."""
    rows = s["rows"]
    back = torch.arange(W - 1, device=x.device)
    token = torch.arange(x.shape[0], device=x.device) + (rows["seq"] + 1) * (W - 1)
    first = rows["cu"][:-1, None] + (torch.arange(s["case"]["seqs"], device=x.device) * (W - 1))[:, None] + back
    last = first + (rows["cu"][1:] - rows["cu"][:-1])[:, None]
    e = x.new_empty(x.shape[0] + first.numel(), x.shape[1])
    e[first] = initial
    e[token] = x
    return e, token, first, last


def _conv_fwd(s):
    W, t = s["case"]["taps"], s["x"].dtype
    e, token, _, last = _extended(s, _flat(s["x"], 1), s["initial"].float(), W)
    window = e[token[:, None] + torch.arange(1 - W, 1, device=e.device)]
    pre = (window * s["weight"].t()).sum(1) + s["bias"]
    return {"out": (pre * _sigmoid(pre)).to(t).reshape(s["x"].shape), "state": e[last].to(t)}


def _conv_bwd(s):
    W, t = s["case"]["taps"], s["x"].dtype
    e, token, first, last = _extended(s, _flat(s["x"], 1), s["initial"].float(), W)
    taps = torch.arange(1 - W, 1, device=e.device)
    window = e[token[:, None] + taps]
    pre = (window * s["weight"].t()).sum(1) + s["bias"]
    dpre = _flat(s["dout"], 1) * _silu_slope(pre)
    late = e.new_zeros(e.shape[0] + W - 1, e.shape[1])
    late[token] = dpre
    reach = torch.arange(e.shape[0], device=e.device)[:, None] - taps
    de = (late[reach] * s["weight"].t()).sum(1)
    de = de.index_put((last,), s["dstate"].float(), accumulate=True)
    return {"dx": de[token].to(t).reshape(s["x"].shape), "dweight": (dpre[:, None] * window).sum(0).t().contiguous(),
            "dbias": dpre.sum(0), "dinitial_state": de[first].to(t)}


def _conv_step(s):
    t, state = s["x"].dtype, s["state"]
    at = s["indices"].long() if s["indices"] is not None else torch.arange(s["x"].shape[0], device=state.device)
    window = torch.cat([state[at].float(), s["x"].float()[:, None]], 1)
    pre = (window * s["weight"].t()).sum(1) + s["bias"]
    state[at] = window[:, 1:].to(t)
    return {"out": (pre * _sigmoid(pre)).to(t), "state": state}


def _recur(a, b, longest):
    """h with h_t = a_t h_{t-1} + b_t along the first axis, a zero where a sequence begins: the products and sums of
    1, 2, 4, ... tokens, each from two of the half length."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], torch.addcmul(b[step:], a[step:], b[:-step])])
        a = torch.cat([a[:step], a[step:] * a[:-step]]) if 2 * step < longest else a
        step *= 2
    return b


def _scan_parts(s):
    case, rows = s["case"], s["rows"]
    D, N, G = case["width"], case["state"], case["groups"]
    u, raw, z = (_flat(s[k], 1) for k in ("u", "dt", "z"))
    b, c = (_flat(s[k], 2).repeat_interleave(D // G, 1) for k in ("b", "c"))
    dt = _softplus(raw + s["dt_bias"])
    decay = torch.exp(dt[..., None] * s["a"])
    add = (dt * u)[..., None] * b
    full = rows["full"]
    begin, end = rows["cu"][full], rows["cu"][full + 1] - 1
    add[begin] = add[begin] + decay[begin] * s["initial"][full]
    inner = decay.clone()
    inner[begin] = 0
    h = _recur(inner, add, rows["longest"])
    return u, raw, z, b, c, dt, decay, inner, h, begin, end, full


def _scan_fwd(s):
    u, _, z, _, c, _, _, _, h, _, end, full = _scan_parts(s)
    y = (h * c).sum(-1) + s["d"] * u
    state = s["initial"].clone()
    state[full] = h[end]
    return {"out": (y * z * _sigmoid(z)).to(s["u"].dtype).reshape(s["u"].shape), "state": state}


def _scan_bwd(s):
    t, shape = s["u"].dtype, s["u"].shape
    T, G, N = s["rows"]["seq"].shape[0], s["case"]["groups"], s["case"]["state"]
    u, raw, z, b, c, dt, decay, inner, h, begin, end, full = _scan_parts(s)
    dout = _flat(s["dout"], 1)
    y = (h * c).sum(-1) + s["d"] * u
    dy = dout * z * _sigmoid(z)
    add = dy[..., None] * c
    add[end] = add[end] + s["dstate"][full]
    later = torch.cat([inner[1:], torch.zeros_like(inner[:1])])
    g = _recur(later.flip(0), add.flip(0), s["rows"]["longest"]).flip(0)
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[begin] = s["initial"][full]
    x = g * decay * before
    s_gb = (g * b).sum(-1)
    ddt = (u * s_gb + (x * s["a"]).sum(-1)) * _sigmoid(raw + s["dt_bias"])
    dinitial = s["dstate"].clone()
    dinitial[full] = decay[begin] * g[begin]
    by_group = (T, G, -1, N)
    return {"du": (dt * s_gb + s["d"] * dy).to(t).reshape(shape), "ddt": ddt.to(t).reshape(shape),
            "da": (x * dt[..., None]).sum(0), "db": (g * (dt * u)[..., None]).reshape(by_group).sum(2).to(t).reshape(s["b"].shape),
            "dc": (h * dy[..., None]).reshape(by_group).sum(2).to(t).reshape(s["c"].shape), "dd": (dy * u).sum(0),
            "dz": (dout * y * _silu_slope(z)).to(t).reshape(shape), "ddt_bias": ddt.sum(0), "dinitial_state": dinitial}


def _scan_step(s):
    D, G = s["case"]["width"], s["case"]["groups"]
    u, raw, z, state = s["u"].float(), s["dt"].float(), s["z"].float(), s["state"]
    b, c = (s[k].float().repeat_interleave(D // G, 1) for k in ("b", "c"))
    at = s["indices"].long() if s["indices"] is not None else torch.arange(u.shape[0], device=u.device)
    dt = _softplus(raw + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["a"]) * state[at] + (dt * u)[..., None] * b
    state[at] = h
    y = (h * c).sum(-1) + s["d"] * u
    return {"out": (y * z * _sigmoid(z)).to(s["u"].dtype), "state": state}


def _norm_parts(s):
    case = s["case"]
    x = s["x"].float()
    z = None if s["z"] is None else s["z"].float()
    v = x * z * _sigmoid(z) if case["gate"] == "before" else x
    v = v.reshape(case["tokens"], case["groups"], -1)
    if case["center"]:
        v = v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + _EPS)
    hat = v * r
    p = hat.reshape(x.shape) * s["weight"]
    return x, z, r, hat, p if s["bias"] is None else p + s["bias"]


def _norm_fwd(s):
    _, z, _, _, p = _norm_parts(s)
    gate = s["case"]["gate"]
    out = p * z * _sigmoid(z) if gate == "after" else p * _sigmoid(p) if gate == "silu" else p
    return {"out": out.to(s["x"].dtype)}


def _norm_bwd(s):
    case, t = s["case"], s["x"].dtype
    x, z, r, hat, p = _norm_parts(s)
    dout, gate = s["dout"].float(), case["gate"]
    dp = dout * z * _sigmoid(z) if gate == "after" else dout * _silu_slope(p) if gate == "silu" else dout
    dhat = (dp * s["weight"]).reshape(hat.shape)
    dv = dhat - hat * (dhat * hat).mean(-1, keepdim=True)
    if case["center"]:
        dv = dv - dhat.mean(-1, keepdim=True)
    dv = (r * dv).reshape(x.shape)
    out = {"dx": (dv * z * _sigmoid(z) if gate == "before" else dv).to(t), "dweight": (dp * hat.reshape(x.shape)).sum(0)}
    if s["bias"] is not None:
        out["dbias"] = dp.sum(0)
    if z is not None:
        out["dz"] = ((dv * x if gate == "before" else dout * p) * _silu_slope(z)).to(t)
    return out


_PLAIN = {"conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd, "conv_step": _conv_step, "scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd,
          "scan_step": _scan_step, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}


# ------------------------------------------------------------------------------------------------- the framework's calls
def _present(outputs):
    return {k: v for k, v in outputs._asdict().items() if v is not None}


def _norm_args(s):
    gate = s["case"]["gate"]
    return dict(bias=s["bias"], z=s["z"], groups=s["case"]["groups"], eps=_EPS, center=s["case"]["center"],
                gate="after" if gate == "after" else "before", activation="silu" if gate == "silu" else None)


def _own(s):
    import mamba_mimo_chunked_amd as m

    op = s["case"]["op"]
    if op == "conv_fwd":
        return _present(m.mamba_conv_fwd(s["x"], s["weight"], s["bias"], s["initial"], s["cu_seqlens"], activation="silu", return_state=True))
    if op == "conv_bwd":
        return _present(m.mamba_conv_bwd(s["dout"], s["x"], s["weight"], s["bias"], s["initial"], s["dstate"], s["cu_seqlens"], activation="silu"))
    if op == "conv_step":
        return {"out": m.mamba_conv_step(s["x"], s["state"], s["weight"], s["bias"], s["indices"], activation="silu"), "state": s["state"]}
    if op == "scan_fwd":
        return _present(m.mamba_scan_fwd(s["u"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"], s["initial"], s["cu_seqlens"],
                                         dt_softplus=True, return_state=True))
    if op == "scan_bwd":
        return _present(m.mamba_scan_bwd(s["dout"], s["u"], s["dt"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"], s["initial"], s["dstate"],
                                         s["cu_seqlens"], dt_softplus=True))
    if op == "scan_step":
        return {"out": m.mamba_scan_step(s["u"], s["dt"], s["state"], s["a"], s["b"], s["c"], s["d"], s["z"], s["dt_bias"], s["indices"],
                                         dt_softplus=True), "state": s["state"]}
    if op == "norm_fwd":
        return {"out": m.mamba_norm_fwd(s["x"], s["weight"], **_norm_args(s))}
    return _present(m.mamba_norm_bwd(s["dout"], s["x"], s["weight"], **_norm_args(s)))


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------- in 64 bits
def _exact_conv(s):
    """One token after another, the window carried along; gradients by the chain rule, tap by tap."""
    case, W = s["case"], s["case"]["taps"]
    w, bias = s["weight"].double(), s["bias"].double()
    if case["op"] == "conv_step":
        out, state = torch.empty(s["x"].shape, dtype=torch.float64, device=w.device), s["state"].double()
        for i in range(case["seqs"]):
            k = i if s["indices"] is None else int(s["indices"][i])
            rows = torch.vstack([state[k], s["x"][i].double()[None]])
            pre = (rows * w.t()).sum(0) + bias
            out[i], state[k] = torch.nn.functional.silu(pre), rows[1:]
        return {"out": out, "state": state}
    cu = s["rows"]["cu"].tolist()
    x, initial = s["x"].double().reshape(-1, case["width"]), s["initial"].double()
    out, state = torch.empty_like(x), torch.empty_like(initial)
    dx, dw, db, dinit = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(bias), torch.empty_like(initial)
    for i in range(case["seqs"]):
        lo, hi = cu[i], cu[i + 1]
        e = torch.vstack([initial[i], x[lo:hi]])
        pre = bias.expand(hi - lo, -1).clone()
        for k in range(W):
            pre += w[:, k] * e[k:k + hi - lo]
        out[lo:hi], state[i] = torch.nn.functional.silu(pre), e[hi - lo:]
        if case["op"] == "conv_bwd":
            g = torch.sigmoid(pre)
            dpre = s["dout"].reshape(x.shape)[lo:hi].double() * (g + pre * g * (1 - g))
            de = torch.zeros_like(e)
            de[hi - lo:] += s["dstate"][i].double()
            for k in range(W):
                de[k:k + hi - lo] += w[:, k] * dpre
                dw[:, k] += (dpre * e[k:k + hi - lo]).sum(0)
            db += dpre.sum(0)
            dinit[i], dx[lo:hi] = de[:W - 1], de[W - 1:]
    if case["op"] == "conv_fwd":
        return {"out": out.reshape(s["x"].shape), "state": state}
    return {"dx": dx.reshape(s["x"].shape), "dweight": dw, "dbias": db, "dinitial_state": dinit}


def _exact_scan(s):
    """The recurrence as it is defined, one token after another for all sequences, and its adjoint backwards."""
    case = s["case"]
    D, N, G = case["width"], case["state"], case["groups"]
    a, d, bias = s["a"].double(), s["d"].double(), s["dt_bias"].double()
    softplus, silu = torch.nn.functional.softplus, torch.nn.functional.silu

    def wide(v):
        return v.double().reshape(-1, G, 1, N).expand(-1, G, D // G, N).reshape(-1, D, N)

    if case["op"] == "scan_step":
        dt = softplus(s["dt"].double() + bias, threshold=60)
        at = torch.arange(case["seqs"], device=a.device) if s["indices"] is None else s["indices"].long()
        state = s["state"].double()
        h = state[at] * torch.exp(dt[:, :, None] * a) + wide(s["b"]) * (dt * s["u"].double())[:, :, None]
        state[at] = h
        y = (h * wide(s["c"])).sum(-1) + d * s["u"].double()
        return {"out": y * silu(s["z"].double()), "state": state}
    bwd = case["op"] == "scan_bwd"
    if case["tokens"] * D * N > 2 ** 30:
        return None
    cu = s["rows"]["cu"]
    lens = (cu[1:] - cu[:-1]).tolist()
    rank = sorted(range(case["seqs"]), key=lambda i: -lens[i])     # the longest first: those still running are a prefix
    order = torch.tensor(rank, device=a.device)
    u, raw, z = (s[k].double().reshape(-1, D) for k in ("u", "dt", "z"))
    b, c = s["b"].reshape(-1, G, N), s["c"].reshape(-1, G, N)
    dt = softplus(raw + bias, threshold=60)
    h, y = s["initial"].double()[order], torch.empty_like(u)
    past = torch.empty(u.shape[0], D, N, dtype=torch.float64, device=a.device) if bwd else None
    for t in range(lens[rank[0]]):
        k = sum(1 for i in rank if lens[i] > t)
        row = cu[order[:k]] + t
        if bwd:
            past[row] = h[:k]
        h[:k] = h[:k] * torch.exp(dt[row][:, :, None] * a) + wide(b[row]) * (dt[row] * u[row])[:, :, None]
        y[row] = (h[:k] * wide(c[row])).sum(-1) + d * u[row]
    if not bwd:
        state = torch.empty_like(h)
        state[order] = h
        return {"out": (y * silu(z)).reshape(s["u"].shape), "state": state}
    dout = s["dout"].double().reshape(-1, D)
    sg = torch.sigmoid(z)
    dy, dz = dout * z * sg, dout * y * (sg + z * sg * (1 - sg))
    du, ddt = torch.empty_like(u), torch.empty_like(u)
    db, dc = torch.empty(b.shape, dtype=torch.float64, device=a.device), torch.empty(c.shape, dtype=torch.float64, device=a.device)
    da, g = torch.zeros_like(a), s["dstate"].double()[order]
    for t in range(lens[rank[0]] - 1, -1, -1):
        k = sum(1 for i in rank if lens[i] > t)
        row = cu[order[:k]] + t
        bt, decay = wide(b[row]), torch.exp(dt[row][:, :, None] * a)
        now = past[row] * decay + bt * (dt[row] * u[row])[:, :, None]
        g[:k] += wide(c[row]) * dy[row][:, :, None]
        dc[row] = (now * dy[row][:, :, None]).reshape(k, G, D // G, N).sum(2)
        db[row] = (g[:k] * (dt[row] * u[row])[:, :, None]).reshape(k, G, D // G, N).sum(2)
        gb, x = (g[:k] * bt).sum(-1), g[:k] * decay * past[row]
        du[row] = gb * dt[row] + d * dy[row]
        ddt[row] = gb * u[row] + (x * a).sum(-1)
        da += (x * dt[row][:, :, None]).sum(0)
        g[:k] *= decay
    ddt = ddt * torch.sigmoid(raw + bias)
    dinitial = torch.empty_like(g)
    dinitial[order] = g
    shape = s["u"].shape
    return {"du": du.reshape(shape), "ddt": ddt.reshape(shape), "da": da, "db": db.reshape(s["b"].shape), "dc": dc.reshape(s["c"].shape),
            "dd": (dy * u).sum(0), "dz": dz.reshape(shape), "ddt_bias": ddt.sum(0), "dinitial_state": dinitial}


def _exact_norm(s):
    """The forward in 64 bits; the gradients are those that differentiation of it gives."""
    case = s["case"]
    gate = case["gate"]
    leaves = {k: s[k].double().requires_grad_() for k in ("x", "z", "weight", "bias") if s[k] is not None}
    with torch.enable_grad():
        v = leaves["x"] * torch.nn.functional.silu(leaves["z"]) if gate == "before" else leaves["x"]
        v = v.unflatten(-1, (case["groups"], -1))
        var = v.var(-1, keepdim=True, unbiased=False) if case["center"] else v.square().mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True) if case["center"] else v
        p = (v / torch.sqrt(var + _EPS)).flatten(-2) * leaves["weight"]
        p = p + leaves["bias"] if "bias" in leaves else p
        out = p * torch.nn.functional.silu(leaves["z"]) if gate == "after" else torch.nn.functional.silu(p) if gate == "silu" else p
        if case["op"] == "norm_fwd":
            return {"out": out.detach()}
        grads = torch.autograd.grad(out, list(leaves.values()), s["dout"].double())
    return {"d" + k: g for k, g in zip(leaves, grads)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return _exact_conv(s) if op.startswith("conv") else _exact_scan(s) if op.startswith("scan") else _exact_norm(s)


# ------------------------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op, D = case["op"], case["width"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op.startswith("norm"):
        T, z = case["tokens"], case["gate"] in ("before", "after")
        streams = (3 if z else 2) if op == "norm_fwd" else (5 if z else 3)
        return {"bytes": streams * T * D * size + 4 * D * (4 if op == "norm_bwd" else 2), "flops": (12 if op == "norm_fwd" else 30) * T * D}
    n = case["seqs"]
    T = n if op.endswith("step") else case["tokens"]
    if op.startswith("conv"):
        W = case["taps"]
        state, weight = n * (W - 1) * D * size, D * (W + 1) * 4
        if op == "conv_bwd":
            return {"bytes": 3 * T * D * size + 3 * state + 2 * weight, "flops": (6 * W + 8) * T * D}
        return {"bytes": 2 * T * D * size + 2 * state + weight, "flops": (2 * W + 5) * T * D}
    N, G = case["state"], case["groups"]
    state, weight = n * D * N * 4, D * (N + 2) * 4
    if op == "scan_bwd":
        return {"bytes": 7 * T * D * size + 4 * T * G * N * size + 3 * state + 2 * weight, "flops": 22 * T * D * N + 30 * T * D}
    return {"bytes": 4 * T * D * size + 2 * T * G * N * size + 2 * state + weight, "flops": 7 * T * D * N + 15 * T * D}
