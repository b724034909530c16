"""The operators of a decoder's pass over packed sequences, as they are timed: norms of
queries and keys with the position rotation, causal attention of grouped heads, and the log
probabilities of the given tokens, each with its gradient.

``run`` computes each in its plain form with elementary torch operations, or, with ``own``
set, through the calls of this library.  ``exact`` is the definition in float64.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # -- norms of queries and keys and their rotation; rows are tokens of a fused projection
        # one decoding step of a small batch: launch latency counts
        dict(name="rope_decode", op="rope", back=False, tokens=16, heads=32, kv_heads=8, dim=128,
             rot=128, pairs="halves", dtype="bf16"),
        # the prompts of a serving step
        dict(name="rope_prompt", op="rope", back=False, tokens=16384, heads=32, kv_heads=8,
             dim=128, rot=128, pairs="halves", dtype="bf16"),
        # gradient in fp32, half of each head rotated, neighbours paired, an odd token count
        dict(name="rope_back_f32", op="rope", back=True, tokens=1999, heads=16, kv_heads=4,
             dim=64, rot=32, pairs="neighbours", dtype="f32"),
        # gradient of a training batch
        dict(name="rope_back", op="rope", back=True, tokens=16384, heads=32, kv_heads=8, dim=128,
             rot=128, pairs="halves", dtype="bf16"),
        # -- attention over packed sequences of differing lengths (one empty, one of one token)
        # a handful of short prompts: latency
        dict(name="attn_short", op="attn", back=False, batch=6, tokens=300, heads=8, kv_heads=2,
             dim=64),
        # long prompts of a serving step
        dict(name="attn_prompt", op="attn", back=False, batch=4, tokens=16000, heads=32,
             kv_heads=8, dim=128),
        # gradient of a ragged batch, three heads to a key head, head dimension 64
        dict(name="attn_back_d64", op="attn", back=True, batch=12, tokens=4097, heads=12,
             kv_heads=4, dim=64),
        # gradient of a training batch
        dict(name="attn_back", op="attn", back=True, batch=5, tokens=8192, heads=32, kv_heads=8,
             dim=128),
        # -- log probabilities; rows are tokens, columns the vocabulary
        # the tokens that a decoding step drew, with five alternatives
        dict(name="logprob_decode", op="logprob", back=False, rows=4, cols=50304, k=5,
             dtype="bf16", temperature=1.0),
        # prompts scored, with twenty alternatives
        dict(name="logprob_score", op="logprob", back=False, rows=16384, cols=50304, k=20,
             dtype="bf16", temperature=1.0),
        # gradient over an odd vocabulary in fp32
        dict(name="logprob_back_f32", op="logprob", back=True, rows=255, cols=65537, k=0,
             dtype="f32", temperature=0.7),
        # gradient of a training batch
        dict(name="logprob_back", op="logprob", back=True, rows=8192, cols=50304, k=0,
             dtype="bf16", temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, back = rng.choice(["rope", "attn", "logprob"]), rng.random() < 0.5
    if op == "rope":
        dim = rng.choice([32, 64, 80, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 8])
        dtype = rng.choice(["f32", "bf16"])
        most = min(16384, 40 * 128 * 16384 * 2 // ((heads + kv) * dim * SIZE[dtype]))
        return dict(op=op, back=back, tokens=_log_int(rng, 1, most), heads=heads, kv_heads=kv,
                    dim=dim, rot=dim // rng.choice([1, 1, 2]),
                    pairs=rng.choice(["halves", "halves", "neighbours"]), dtype=dtype)
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        batch = _log_int(rng, 1, 64)
        return dict(op=op, back=back, batch=batch,
                    tokens=_log_int(rng, 16 + 4 * batch, 8192 if back else 16000),
                    heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=rng.choice([64, 128]))
    dtype = rng.choice(["f32", "bf16"])
    cols = _log_int(rng, 1000, 131072)
    rows = _log_int(rng, 1, min(16384, (400_000_000 if back else 800_000_000) * 2 // SIZE[dtype]
                                // cols))
    return dict(op=op, back=back, rows=rows, cols=cols, k=0 if back else rng.choice([0, 1, 5, 20]),
                dtype=dtype, temperature=rng.choice([1.0, 1.0, 0.7, 1.5]))


# ------------------------------------------------------------------- inputs ---

def _lengths(case):
    """Lengths of the packed sequences; the buffer's last rows belong to none."""
    n, room = case["batch"], case["tokens"]
    if n == 1:
        return [room]
    weight = [0.1 + ((b + 1) * 0.6180339887) % 1.0 for b in range(n)]
    if n >= 4:
        weight[1] = 0.0
    total = sum(weight)
    got = [int((room - n) * w / total) for w in weight]
    if n >= 4:
        got[2] = 1
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return {"rope": _prepare_rope, "attn": _prepare_attn,
            "logprob": _prepare_logprob}[case["op"]](case, g, dev)


def _prepare_rope(case, g, dev):
    T, H, KV, D, R = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rot"))
    dt = DT[case["dtype"]]
    # the fused projection's output: queries, keys and values of a token side by side
    qkv = torch.randn(T, H + 2 * KV, D, generator=g, device=dev)
    qkv = (qkv * (0.5 + 2.0 * torch.rand(1, H + 2 * KV, 1, generator=g, device=dev))).to(dt)
    reach = 32768
    angle = torch.arange(reach, dtype=torch.float64, device=dev)[:, None] * (
        500000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev) / R))
    # positions restart with each packed prompt, some of which continue a long context
    start = torch.randint(0, reach - T, (T // 700 + 1,), generator=g, device=dev)
    at = torch.arange(T, device=dev)
    st = dict(case=case, q=qkv[:, :H], k=qkv[:, H:H + KV],
              cos=angle.cos().float(), sin=angle.sin().float(),
              positions=(start[at // 700] + at % 700).int(),
              qw=(1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt),
              kw=(1.0 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt),
              a=torch.empty(T, H, D, dtype=dt, device=dev),
              b=torch.empty(T, KV, D, dtype=dt, device=dev))
    if case["back"]:
        st["dq"] = torch.randn(T, H, D, generator=g, device=dev).to(dt)
        st["dk"] = torch.randn(T, KV, D, generator=g, device=dev).to(dt)
        st["dqw"], st["dkw"] = torch.empty_like(st["qw"]), torch.empty_like(st["kw"])
    return st


def _prepare_attn(case, g, dev):
    T, H, KV, D = (case[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    bf = torch.bfloat16
    qkv = torch.randn(T, H + 2 * KV, D, generator=g, device=dev).to(bf)
    ends = [0]
    for n in _lengths(case):
        ends.append(ends[-1] + n)
    st = dict(case=case, q=qkv[:, :H], k=qkv[:, H:H + KV], v=qkv[:, H + KV:],
              cu=torch.tensor(ends, dtype=torch.int32, device=dev),
              o=torch.zeros(T, H, D, dtype=bf, device=dev), lse=torch.zeros(H, T, device=dev))
    if case["back"]:  # what the forward pass left, and the gradient of its output
        o, st["lse"] = _plain_attn(st)
        st["o"] = o
        st["do"] = torch.randn(T, H, D, generator=g, device=dev).to(bf)
        grads = torch.zeros(T, H + 2 * KV, D, dtype=bf, device=dev)
        st["dq"], st["dk"], st["dv"] = grads[:, :H], grads[:, H:H + KV], grads[:, H + KV:]
    return st


def _prepare_logprob(case, g, dev):
    R, V, T, k = (case[k] for k in ("rows", "cols", "temperature", "k"))
    logits = torch.empty(R, V, dtype=DT[case["dtype"]], device=dev)
    tokens = torch.empty(R, dtype=torch.int32, device=dev)
    stats = torch.empty(3, R, device=dev)
    step = max(1, 100_000_000 // V)
    for r in range(0, R, step):
        x = (3.0 * torch.randn(min(step, R - r), V, generator=g, device=dev)).to(logits.dtype)
        logits[r:r + step] = x
        x = x.float()
        e = torch.empty_like(x).exponential_(generator=g)
        tokens[r:r + step] = (x / T - e.log()).argmax(1)  # drawn from the row itself
        if case["back"]:  # what the forward pass saved
            m = x.amax(1, keepdim=True)
            z = (x - m) / T
            log_sum = torch.logsumexp(z, 1, keepdim=True)
            stats[0, r:r + step] = m[:, 0]
            stats[1, r:r + step] = log_sum[:, 0]
            stats[2, r:r + step] = (log_sum - (torch.exp(z - log_sum) * z).sum(1, True))[:, 0]
    tokens[torch.rand(R, generator=g, device=dev) < 0.05] = -100  # tokens that do not count
    st = dict(case=case, logits=logits, tokens=tokens)
    if case["back"]:
        stats[:, tokens == -100] = 0.0
        st |= dict(row_max=stats[0], log_sum=stats[1], entropy=stats[2],
                   g=torch.randn(R, generator=g, device=dev),
                   h=0.1 * torch.randn(R, generator=g, device=dev),
                   dlogits=torch.empty_like(logits))
        return st
    i32 = dict(dtype=torch.int32, device=dev)
    st |= dict(logprob=torch.empty(R, device=dev), entropy=torch.empty(R, device=dev),
               row_max=torch.empty(R, device=dev), log_sum=torch.empty(R, device=dev),
               rank=torch.empty(R, **i32))
    if k:
        st |= dict(top_index=torch.empty(R, k, **i32), top_logprob=torch.empty(R, k, device=dev))
    return st


# ---------------------------------------------------------------------- run ---

def run(state):
    what = state["case"]["op"] + ("_back" if state["case"]["back"] else "")
    if own:
        return {"rope": _own_rope, "rope_back": _own_rope_back, "attn": _own_attn,
                "attn_back": _own_attn_back, "logprob": _own_logprob,
                "logprob_back": _own_logprob_back}[what](state)
    return {"rope": _plain_rope, "rope_back": _plain_rope_back, "attn": _plain_attn,
            "attn_back": _plain_attn_back, "logprob": _plain_logprob,
            "logprob_back": _plain_logprob_back}[what](state)


def _own_rope(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"], s["positions"],
                           s["a"], s["b"], eps=EPS, interleaved=s["case"]["pairs"] != "halves")
    return s["a"], s["b"]


def _own_rope_back(s):
    import row_reduction_pass_gb300 as rr
    c = s["case"]
    if "workspace" not in s:  # kept by a training program from step to step
        n = rr.rr_qk_norm_rope_bwd_workspace_size(c["tokens"], c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    rr.rr_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["cos"], s["sin"],
                           s["positions"], s["a"], s["b"], s["dqw"], s["dkw"], eps=EPS,
                           interleaved=c["pairs"] != "halves", workspace=s["workspace"])
    return s["a"], s["b"], s["dqw"], s["dkw"]


def _own_attn(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_attention_packed_fwd(s["q"], s["k"], s["v"], s["cu"], s["o"], lse=s["lse"])
    return s["o"], s["lse"]


def _own_attn_back(s):
    import row_reduction_pass_gb300 as rr
    c = s["case"]
    if "workspace" not in s:  # kept by a training program from step to step
        n = rr.rr_attention_packed_bwd_workspace_size(c["tokens"], c["heads"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
    rr.rr_attention_packed_bwd(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["cu"],
                               s["dq"], s["dk"], s["dv"], workspace=s["workspace"])
    return s["dq"], s["dk"], s["dv"]


def _own_logprob(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_token_logprob_fwd(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"],
                            row_max=s["row_max"], log_sum=s["log_sum"], rank=s["rank"],
                            top_index=s.get("top_index"), top_logprob=s.get("top_logprob"),
                            temperature=s["case"]["temperature"])
    got = [s[k] for k in ("logprob", "entropy", "row_max", "log_sum", "rank")]
    return got + [s[k] for k in ("top_index", "top_logprob") if k in s]


def _own_logprob_back(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_token_logprob_bwd(s["logits"], s["tokens"], s["row_max"], s["log_sum"], s["g"],
                            s["dlogits"], entropy=s["entropy"], grad_entropy=s["h"],
                            temperature=s["case"]["temperature"])
    return s["dlogits"]


def _places(case):
    """(first, second) member of each rotated pair."""
    R = case["rot"]
    return (slice(0, R // 2), slice(R // 2, R)) if case["pairs"] == "halves" else (
        slice(0, R, 2), slice(1, R, 2))


def _turn(x, c, s, case):
    """Each pair (x_a, x_b) turned by its angle; what is behind the pairs stays."""
    a, b = _places(case)
    y = x.clone()
    y[..., a] = c * x[..., a] - s * x[..., b]
    y[..., b] = s * x[..., a] + c * x[..., b]
    return y


def _plain_rope(s):
    at = s["positions"].long()
    c, sn = s["cos"][at][:, None], s["sin"][at][:, None]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        return _turn(x, c, sn, s["case"]).to(w.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_rope_back(s):
    at = s["positions"].long()
    c, sn = s["cos"][at][:, None], s["sin"][at][:, None]

    def one(dy, x, w):
        x, g = x.float(), _turn(dy.float(), c, -sn, s["case"])
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        dw = (g * x).sum((0, 1))
        g = g * w.float()
        dx = r * (g - x * (g * x).mean(-1, keepdim=True))
        return dx.to(w.dtype), dw.to(w.dtype)

    dq, dqw = one(s["dq"], s["q"], s["qw"])
    dk, dkw = one(s["dk"], s["k"], s["kw"])
    return dq, dk, dqw, dkw


def _scores(s):
    """Probabilities [KV, G, T, T] of all rows at once, with each row's log of its sum; rows of
    other sequences and later ones are out of sight."""
    c = s["case"]
    T, H, KV, D = (c[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    q = s["q"].float().permute(1, 0, 2).reshape(KV, H // KV, T, D)
    k = s["k"].float().permute(1, 0, 2)[:, None]
    at = torch.arange(T, device=q.device)
    which = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    unseen = (which[:, None] != which[None, :]) | (at[:, None] < at[None, :])
    unseen |= (which == len(s["cu"]) - 1)[:, None]
    x = torch.matmul(q * (1.0 / math.sqrt(D)), k.transpose(-1, -2)).masked_fill_(unseen, -math.inf)
    m = x.amax(-1, keepdim=True)
    live = m > -math.inf
    x.sub_(torch.where(live, m, 0.0)).exp_()
    z = x.sum(-1, keepdim=True)
    x.div_(torch.where(live, z, 1.0))
    return x, torch.where(live, m + torch.log(z), 0.0).reshape(H, T)


def _plain_attn(s):
    c = s["case"]
    p, lse = _scores(s)
    v = s["v"].float().permute(1, 0, 2)[:, None]
    o = torch.matmul(p, v).reshape(c["heads"], c["tokens"], c["dim"]).permute(1, 0, 2)
    return o.to(torch.bfloat16).contiguous(), lse


def _plain_attn_back(s):
    c = s["case"]
    T, H, KV, D = (c[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    scale = 1.0 / math.sqrt(D)
    p = _scores(s)[0]
    do = s["do"].float().permute(1, 0, 2).reshape(KV, H // KV, T, D)
    q = s["q"].float().permute(1, 0, 2).reshape(KV, H // KV, T, D)
    k, v = s["k"].float().permute(1, 0, 2)[:, None], s["v"].float().permute(1, 0, 2)[:, None]
    dv = torch.matmul(p.transpose(-1, -2), do).sum(1).permute(1, 0, 2)
    dp = torch.matmul(do, v.transpose(-1, -2))
    p.mul_(dp.sub_((dp * p).sum(-1, keepdim=True)))
    dq = torch.matmul(p, k).mul_(scale).reshape(H, T, D).permute(1, 0, 2)
    dk = torch.matmul(p.transpose(-1, -2), q).sum(1).mul_(scale).permute(1, 0, 2)
    return tuple(x.to(torch.bfloat16).contiguous() for x in (dq, dk, dv))


def _plain_logprob(s):
    c = s["case"]
    V, k = c["cols"], c["k"]
    t, x = s["tokens"].long(), s["logits"].float()
    counts = t != -100
    t = torch.where(counts, t, 0)[:, None]
    at = torch.arange(V, device=x.device)
    xt = x.gather(1, t)
    rank = ((x > xt) | ((x == xt) & (at < t))).sum(1)
    m = x.amax(1, keepdim=True)
    top = None
    if k:  # a tie goes to the lowest column
        bits = (x + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * (1 << 32) + (V - 1 - at)
        top = torch.topk(order, k, dim=1).values
        top = V - 1 - (top & 0xffffffff)
        del bits, order
    z = (x - m) / c["temperature"]
    e = torch.exp(z)
    d = e.sum(1, keepdim=True)
    log_sum = torch.log(d)
    entropy = log_sum - e.mul_(z).sum(1, keepdim=True) / d
    got = [torch.where(counts, v[:, 0], 0.0)
           for v in (z.gather(1, t) - log_sum, entropy, m, log_sum)]
    got.append(torch.where(counts, rank, -1).int())
    if k:
        got.append(torch.where(counts[:, None], top, -1).int())
        got.append(torch.where(counts[:, None], z.gather(1, top) - log_sum, 0.0))
    return got


def _plain_logprob_back(s):
    T = s["case"]["temperature"]
    t = s["tokens"].long()
    counts = t != -100
    lp = (s["logits"].float() - s["row_max"][:, None]) / T - s["log_sum"][:, None]
    p = torch.exp(lp)
    d = p * (-s["g"][:, None] - s["h"][:, None] * (lp + s["entropy"][:, None]))
    d.scatter_add_(1, torch.where(counts, t, 0)[:, None], s["g"][:, None])
    return torch.where(counts[:, None], d / T, 0.0).to(s["logits"].dtype)


# --------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "rope":
        T, H, KV, D, R = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rot"))
        n = T * (H + KV) * D
        side = T * (4 + 4 * R) + 2 * D * SIZE[case["dtype"]]  # angles, positions, weights
        return {"bytes": n * SIZE[case["dtype"]] * (3 if case["back"] else 2) + side,
                "flops": n * (16 if case["back"] else 8)}
    if case["op"] == "attn":
        H, KV, D = (case[k] for k in ("heads", "kv_heads", "dim"))
        lens = _lengths(case)
        pairs, rows = sum(n * (n + 1) // 2 for n in lens), sum(lens)
        if case["back"]:  # q, o, do, dq; k, v, dk, dv; lse
            return {"bytes": rows * (2 * D * (4 * H + 4 * KV) + 4 * H),
                    "flops": 10 * D * H * pairs}
        return {"bytes": rows * (2 * D * (2 * H + 2 * KV) + 4 * H), "flops": 4 * D * H * pairs}
    n, E = case["rows"] * case["cols"], SIZE[case["dtype"]]
    if case["back"]:
        return {"bytes": 2 * n * E + 24 * case["rows"], "flops": 8 * n}
    return {"bytes": n * E + case["rows"] * (24 + 8 * case["k"]), "flops": 6 * n}


# -------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "logprob": _exact_logprob}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    D, R = c["dim"], c["rot"]
    dev = s["q"].device
    # the rotation as complex numbers, one for each pair
    at = s["positions"].long()
    unit = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None, :]
    pairs = torch.arange(R, device=dev)
    pairs = pairs.reshape(2, R // 2).T if c["pairs"] == "halves" else pairs.reshape(R // 2, 2)

    def rotate(u, z):
        y = u.clone()
        w = torch.view_as_complex(u[..., pairs].contiguous()) * z
        y[..., pairs] = torch.view_as_real(w)
        return y

    def forward(x, w):
        x = x.double()
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
        return rotate(x / norm * w.double(), unit)

    def backward(dy, x, w):
        x, w = x.double(), w.double()
        norm = torch.sqrt(x.square().sum(-1, keepdim=True) / D + EPS)
        du = rotate(dy.double(), unit.conj())
        dw = torch.einsum("thd,thd->d", du, x / norm)
        a = du * w
        # d(x / norm): the part along x is what the norm takes away
        dx = a / norm - x * (a * x).sum(-1, keepdim=True) / (D * norm ** 3)
        return dx, dw

    if not c["back"]:
        return forward(s["q"], s["qw"]), forward(s["k"], s["kw"])
    dq, dqw = backward(s["dq"], s["q"], s["qw"])
    dk, dkw = backward(s["dk"], s["k"], s["kw"])
    return dq, dk, dqw, dkw


def _exact_attn(s):
    c = s["case"]
    T, H, KV, D = (c[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    f64 = dict(dtype=torch.float64, device=s["q"].device)
    o, lse = torch.zeros(T, H, D, **f64), torch.zeros(H, T, **f64)
    dq, dk, dv = torch.zeros(T, H, D, **f64), torch.zeros(T, KV, D, **f64), torch.zeros(T, KV, D,
                                                                                         **f64)
    begin = 0
    for n in _lengths(c):
        rows = slice(begin, begin + n)
        begin += n
        if n == 0:
            continue
        hide = torch.ones(n, n, dtype=torch.bool, device=o.device).triu(1)
        for h in range(H):
            kv = h // (H // KV)
            q, k, v = s["q"][rows, h].double(), s["k"][rows, kv].double(), s["v"][rows, kv].double()
            x = (q @ k.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
            if not c["back"]:
                lse[h, rows] = torch.logsumexp(x, 1)
                o[rows, h] = torch.softmax(x, 1) @ v
                continue
            p = torch.softmax(x, 1)
            g = s["do"][rows, h].double()
            dv[rows, kv] += p.T @ g
            a = g @ v.T
            ds = p * (a - (p * a).sum(1, keepdim=True)) / math.sqrt(D)
            dq[rows, h] = ds @ k
            dk[rows, kv] += ds.T @ q
    return (dq, dk, dv) if c["back"] else (o, lse)


def _exact_logprob(s):
    c = s["case"]
    R, V, T, k = (c[k] for k in ("rows", "cols", "temperature", "k"))
    parts = []
    step = max(1, 40_000_000 // V)
    for r in range(0, R, step):
        x = s["logits"][r:r + step].double()
        t = s["tokens"][r:r + step].long()
        off = t < 0
        t = t.clamp_min(0)[:, None]
        lp = torch.log_softmax(x / T, 1)
        if c["back"]:
            # d lp_t = 1_t - p;  d H = -p (lp + H)
            hot = torch.zeros_like(lp).scatter_(1, t, 1.0)
            p = lp.exp()
            ent = -(p * lp).sum(1, keepdim=True)
            g, h = (s[n][r:r + step].double()[:, None] for n in ("g", "h"))
            d = (g * (hot - p) - h * p * (lp + ent)) / T
            parts.append([d.masked_fill_(off[:, None], 0.0)])
            continue
        m = x.amax(1)
        got = [lp.gather(1, t)[:, 0], -(lp.exp() * lp).sum(1), m,
               torch.log(torch.exp((x - m[:, None]) / T).sum(1))]
        got = [v.masked_fill_(off, 0.0) for v in got]
        got.append(None)
        if k:
            got.append(None)
            got.append(torch.topk(lp, k, dim=1).values.masked_fill_(off[:, None], 0.0))
        parts.append(got)
    whole = [None if p[0] is None else torch.cat(p) for p in zip(*parts)]
    return whole[0] if c["back"] else whole
