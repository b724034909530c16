"""The operators of a draft model's life, as they are timed: training it on a
teacher's top logits (distillation loss and its gradient in one pass), scoring
its tree of drafted tokens over a paged cache (attention), and accepting the
drafted tokens against the target's probabilities (verification).

``run`` computes each in its plain form with elementary torch operations, or,
with ``own`` set, through the calls of this library.  ``exact`` is the
definition in float64.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # -- distillation: rows are training tokens, columns the vocabulary
        # a probe batch of a small head: launch latency counts
        dict(name="distill_small_f32", op="distill", rows=64, cols=1000, k=8, dtype="f32",
             temperature=2.0, tail=False),
        # an odd vocabulary in fp32, the teacher's mass outside its list kept as one bucket
        dict(name="distill_odd_f32_tail", op="distill", rows=255, cols=65537, k=50, dtype="f32",
             temperature=1.0, tail=True),
        # a training micro-batch
        dict(name="distill_mid_bf16_tail", op="distill", rows=2048, cols=50304, k=100,
             dtype="bf16", temperature=1.5, tail=True),
        # a full training batch of tokens
        dict(name="distill_large_bf16", op="distill", rows=8192, cols=50304, k=64, dtype="bf16",
             temperature=2.0, tail=False),
        # -- attention over a paged cache
        # one user, one new token: the latency of plain decoding
        dict(name="tree_attn_token", op="attention", batch=1, nodes=1, heads=32, kv_heads=8,
             dim=128, ctx_min=4001, ctx_max=4001, page=16, branch=1),
        # a ragged serving batch, one new token each: the cache is read at memory speed
        dict(name="tree_attn_decode_batch", op="attention", batch=64, nodes=1, heads=32,
             kv_heads=8, dim=128, ctx_min=500, ctx_max=8000, page=64, branch=1),
        # small drafted trees over a ragged batch, head dimension 64
        dict(name="tree_attn_mid_d64", op="attention", batch=16, nodes=30, heads=16, kv_heads=4,
             dim=64, ctx_min=1000, ctx_max=4100, page=32, branch=2),
        # large trees over long contexts: the products dominate
        dict(name="tree_attn_large", op="attention", batch=8, nodes=62, heads=64, kv_heads=8,
             dim=128, ctx_min=12000, ctx_max=20000, page=128, branch=2),
        # -- verification
        # one user, a drafted chain: latency
        dict(name="verify_chain_one", op="verify", batch=1, nodes=5, cols=50304, dtype="bf16",
             branch=1, greedy=False),
        # drafted trees, three tries a node, fp32 logits of an odd vocabulary
        dict(name="verify_tree_f32", op="verify", batch=8, nodes=39, cols=65537, dtype="f32",
             branch=3, greedy=False),
        # a serving batch of chains, every second sequence greedy
        dict(name="verify_chain_mixed", op="verify", batch=48, nodes=7, cols=131072,
             dtype="bf16", branch=1, greedy=True),
        # the largest batch
        dict(name="verify_chain_batch", op="verify", batch=256, nodes=8, cols=50304,
             dtype="bf16", branch=1, greedy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["distill", "attention", "verify"])
    if op == "distill":
        dtype = rng.choice(["f32", "bf16"])
        cols = _log_int(rng, 1000, 131072)
        rows = _log_int(rng, 16, max(17, min(8192, 400_000_000 // (cols * SIZE[dtype] // 2))))
        return dict(op=op, rows=rows, cols=cols, k=_log_int(rng, 4, 128), dtype=dtype,
                    temperature=rng.choice([1.0, 1.5, 2.0, 4.0]), tail=rng.random() < 0.5)
    if op == "attention":
        batch = _log_int(rng, 1, 64)
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128])
        branch = rng.choice([1, 1, 2, 3])
        nodes = 1 if rng.random() < 0.4 else rng.randint(2, 64)
        ctx_max = _log_int(rng, 64, max(65, min(20000, 60_000_000 // (batch * kv * dim))))
        return dict(op=op, batch=batch, nodes=nodes, heads=kv * rng.choice([1, 3, 4, 8]),
                    kv_heads=kv, dim=dim, ctx_min=rng.randint(0, ctx_max), ctx_max=ctx_max,
                    page=rng.choice([16, 32, 48, 64, 128, 256]), branch=branch)
    dtype = rng.choice(["f32", "bf16"])
    branch = rng.choice([1, 1, 2, 3])
    cols = _log_int(rng, 1000, 131072)
    nodes = rng.randint(1, 8) if branch == 1 else rng.randint(4, 40)
    batch = _log_int(rng, 1, max(2, min(256, 200_000_000 // (cols * (2 * nodes + 1)))))
    return dict(op=op, batch=batch, nodes=nodes, cols=cols, dtype=dtype, branch=branch,
                greedy=rng.random() < 0.3)


# ------------------------------------------------------------------- inputs ---

def _parents(nodes, branch):
    """Parents of a tree whose nodes have `branch` children each, breadth first
    (branch 1: a chain); -1 is the root."""
    return [i // branch - 1 for i in range(nodes)]


def _lengths(case):
    """Context length of each sequence, spread evenly over the case's range."""
    lo, hi = case["ctx_min"], case["ctx_max"]
    return [lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) if case["batch"] > 1 else hi
            for b in range(case["batch"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if case["op"] == "distill":
        return _prepare_distill(case, g, dev)
    if case["op"] == "attention":
        return _prepare_attention(case, g, dev)
    return _prepare_verify(case, g, dev)


def _prepare_distill(case, g, dev):
    rows, cols, k, T = case["rows"], case["cols"], case["k"], case["temperature"]
    logits = (3.0 * torch.randn(rows, cols, generator=g, device=dev)).to(DT[case["dtype"]])
    index = torch.empty(rows, k, dtype=torch.int32, device=dev)
    value = torch.empty(rows, k, device=dev)
    for r in range(0, rows, 1024):  # the teacher's row is the student's with noise
        x = logits[r:r + 1024].float()
        x = x + torch.randn(x.shape, generator=g, device=dev)
        v, i = torch.topk(x, k, dim=1)
        if case["tail"]:  # log-probabilities at this temperature
            v = v / T - torch.logsumexp(x / T, dim=1, keepdim=True)
        index[r:r + 1024] = i
        value[r:r + 1024] = v
    # lists of differing lengths, and rows without a teacher
    keep = torch.randint(max(1, k // 2), k + 1, (rows, 1), generator=g, device=dev)
    keep[torch.rand(rows, 1, generator=g, device=dev) < 0.05] = 0
    index[torch.arange(k, device=dev)[None, :] >= keep] = -1
    weight = torch.rand(rows, generator=g, device=dev)
    return dict(case=case, logits=logits, index=index, value=value, weight=weight,
                loss=torch.empty(rows, device=dev), dlogits=torch.empty_like(logits))


def _prepare_attention(case, g, dev):
    B, n, H, KV, D, ps = (case[k] for k in ("batch", "nodes", "heads", "kv_heads", "dim", "page"))
    lens = _lengths(case)
    need = [(L + n + ps - 1) // ps for L in lens]
    width, pages = max(need), sum(need) + 3
    bf = torch.bfloat16
    q = torch.randn(B, n, H, D, generator=g, device=dev).to(bf)
    kc = torch.randn(pages, ps, KV, D, generator=g, device=dev).to(bf)
    vc = torch.randn(pages, ps, KV, D, generator=g, device=dev).to(bf)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    parents = None
    if case["branch"] > 1:
        parents = torch.tensor(_parents(n, case["branch"]), dtype=torch.int32,
                               device=dev).repeat(B, 1)
    st = dict(case=case, q=q, kc=kc, vc=vc, table=table, parents=parents,
              length=torch.tensor(lens, dtype=torch.int32, device=dev),
              o=torch.empty_like(q), lse=torch.empty(B, n, H, device=dev))
    if own:
        import row_reduction_pass_gb300 as rr
        st["workspace"] = torch.empty(rr.rr_attention_tree_workspace_size(B, n, H, KV, D),
                                      dtype=torch.uint8, device=dev)
    return st


def _prepare_verify(case, g, dev):
    B, n, V = case["batch"], case["nodes"], case["cols"]
    dt = DT[case["dtype"]]
    target = torch.empty(B, n + 1, V, dtype=dt, device=dev)
    draft = torch.empty(B, n, V, dtype=dt, device=dev)
    for i in range(n + 1):
        x = 3.0 * torch.randn(B, V, generator=g, device=dev)
        target[:, i] = x
        if i < n:
            draft[:, i] = x + 0.6 * torch.randn(B, V, generator=g, device=dev)
    temperature = 0.7 + 0.5 * torch.rand(B, generator=g, device=dev)
    if case["greedy"]:
        temperature[::2] = 0.0
    par = _parents(n, case["branch"])
    tokens = torch.empty(B, n, dtype=torch.int32, device=dev)
    T = temperature.clamp_min(0.05)[:, None]  # a greedy sequence drafts nearly greedily
    for i in range(n):
        e = torch.empty(B, V, device=dev).exponential_(generator=g)
        tokens[:, i] = (draft[:, par[i] + 1].float() / T - e.log()).argmax(1)
    # sequences that drafted fewer tokens
    short = torch.rand(B, generator=g, device=dev) < 0.1
    tokens[short, (n + 1) // 2:] = -1
    race = torch.empty(B, V, device=dev).exponential_(generator=g)
    parents = None
    if case["branch"] > 1:
        parents = torch.tensor(par, dtype=torch.int32, device=dev).repeat(B, 1)
    return dict(case=case, target=target, draft=draft, tokens=tokens, parents=parents,
                temperature=temperature, race=race,
                uniform=torch.rand(B, n, generator=g, device=dev),
                out_tokens=torch.empty(B, n + 1, dtype=torch.int32, device=dev),
                out_nodes=torch.empty(B, n + 1, dtype=torch.int32, device=dev),
                out_count=torch.empty(B, dtype=torch.int32, device=dev))


# ---------------------------------------------------------------------- run ---

def run(state):
    op = state["case"]["op"]
    if own:
        return {"distill": _own_distill, "attention": _own_attention,
                "verify": _own_verify}[op](state)
    return {"distill": _plain_distill, "attention": _plain_attention,
            "verify": _plain_verify}[op](state)


def _own_distill(s):
    import row_reduction_pass_gb300 as rr
    c = s["case"]
    rr.rr_distill_fwd_bwd(s["logits"], s["index"], s["value"], s["loss"], s["dlogits"],
                          grad=s["weight"], temperature=c["temperature"], tail=c["tail"])
    return s["loss"], s["dlogits"]


def _own_attention(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_attention_tree_fwd(s["q"], s["kc"], s["vc"], s["table"], s["length"], s["o"],
                             lse=s["lse"], parents=s["parents"], workspace=s["workspace"])
    return s["o"], s["lse"]


def _own_verify(s):
    import row_reduction_pass_gb300 as rr
    rr.rr_draft_verify(s["target"], s["draft"], s["tokens"], s["uniform"], s["race"],
                       s["out_tokens"], s["out_nodes"], s["out_count"], parents=s["parents"],
                       temperature=s["temperature"])
    return s["out_tokens"], s["out_nodes"], s["out_count"]


def _plain_distill(s):
    c = s["case"]
    T, tail, cols = c["temperature"], c["tail"], c["cols"]
    x, index, v, w = s["logits"].float() / T, s["index"].long(), s["value"], s["weight"]
    valid = (index >= 0) & (index < cols)
    some = valid.any(1)
    at = index.clamp(0, cols - 1)
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    Z = e.sum(1, keepdim=True)
    if tail:
        lt = v.masked_fill(~valid, -math.inf)
        t = torch.exp(lt)
        tt = (1.0 - t.sum(1, keepdim=True)).clamp_min(0.0)
    else:
        lt = (v / T).masked_fill(~valid, -math.inf)
        lt = lt - lt.amax(1, keepdim=True)
        lt = lt - torch.log(torch.exp(lt).sum(1, keepdim=True))
        lt = lt.masked_fill(~valid, -math.inf)
        t = torch.exp(lt)
        tt = torch.zeros_like(m)
    ls = x.gather(1, at) - m - torch.log(Z)
    term = torch.where(t > 0, t * (lt - ls), 0.0).sum(1, keepdim=True)
    d = e * ((t.sum(1, keepdim=True) + tt) / Z)
    if tail:
        free = torch.ones_like(x)
        free.scatter_reduce_(1, at, torch.where(valid, 0.0, 1.0), "amin")
        et = e * free
        Zt = et.sum(1, keepdim=True)
        term = term + torch.where(tt > 0, tt * (torch.log(tt) - torch.log(Zt / Z)), 0.0)
        d = d - et * (tt / Zt)
    d = d.scatter_add(1, at, -t)
    loss = torch.where(some, T * T * term[:, 0], 0.0)
    d = torch.where(some[:, None], d * (T * w[:, None]), 0.0)
    return loss, d.to(s["logits"].dtype)


def _seen(parents, n, batch, dev):
    """seen[b, i, j]: node i attends to node j (itself and its ancestors)."""
    if parents is None:
        return torch.ones(n, n, dtype=torch.bool, device=dev).tril().expand(batch, n, n)
    j = torch.arange(n, device=dev)
    a = (parents[:, :, None] == j) | (j[:, None] == j)
    steps = 1
    while steps < n:  # each product doubles the distance covered
        a = torch.matmul(a.float(), a.float()) > 0
        steps *= 2
    return a


def _plain_attention(s):
    c = s["case"]
    B, n, H, KV, D = (c[k] for k in ("batch", "nodes", "heads", "kv_heads", "dim"))
    G = H // KV
    table, length = s["table"].long(), s["length"].long()
    L = table.shape[1] * c["page"]
    dev = table.device
    k = s["kc"][table].reshape(B, L, KV, D).float().permute(0, 2, 3, 1)
    q = s["q"].float().reshape(B, n, KV, G, D).permute(0, 2, 1, 3, 4).reshape(B, KV, n * G, D)
    x = torch.matmul(q, k).reshape(B, KV, n, G, L) * (1.0 / math.sqrt(D))
    node = torch.arange(L, device=dev)[None, :] - length[:, None]
    tree = _seen(s["parents"], n, B, dev).gather(
        2, node.clamp(0, n - 1)[:, None, :].expand(B, n, L))
    seen = (node < 0)[:, None, :] | ((node >= 0) & (node < n))[:, None, :] & tree
    x = x.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(-1, keepdim=True)
    v = s["vc"][table].reshape(B, L, KV, D).float().permute(0, 2, 1, 3)
    o = torch.matmul((e / z).reshape(B, KV, n * G, L), v)
    o = o.reshape(B, KV, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H, D)
    lse = (m + torch.log(z))[..., 0].permute(0, 2, 1, 3).reshape(B, n, H)
    return o.to(s["q"].dtype), lse


def _plain_verify(s):
    c = s["case"]
    B, n, V = c["batch"], c["nodes"], c["cols"]
    tokens, u = s["tokens"].long(), s["uniform"]
    dev = u.device
    T = s["temperature"][:, None, None]
    greedy = T <= 0

    def probabilities(logits):
        x = logits.float()
        hot = torch.zeros_like(x).scatter_(2, x.argmax(2, keepdim=True), 1.0)
        x = x / torch.where(greedy, 1.0, T)
        e = torch.exp(x - x.amax(2, keepdim=True))
        return torch.where(greedy, hot, e / e.sum(2, keepdim=True))

    p, q = probabilities(s["target"]), probabilities(s["draft"])
    b = torch.arange(B, device=dev)
    cur = torch.full((B,), -1, dtype=torch.long, device=dev)
    ratio = torch.zeros(B, device=dev)  # the residual is max(p - ratio q, 0) / mass
    mass = torch.ones(B, device=dev)
    count = torch.zeros(B, dtype=torch.long, device=dev)
    out = torch.full((B, n + 2), -1, dtype=torch.long, device=dev)
    nodes = torch.full((B, n + 2), -1, dtype=torch.long, device=dev)
    for i in range(n):
        parent = s["parents"][:, i] if s["parents"] is not None else torch.full_like(cur, i - 1)
        x = tokens[:, i]
        tried = (parent == cur) & (x >= 0) & (x < V)
        pr, qr = p[b, cur + 1], q[b, (cur + 1).clamp_max(n - 1)]
        px, qx = pr[b, x.clamp(0, V - 1)], qr[b, x.clamp(0, V - 1)]
        yes = tried & (u[:, i] * mass * qx < px - ratio * qx)
        no = tried & ~yes
        slot = torch.where(yes, count, n + 1)
        out[b, slot], nodes[b, slot] = x, torch.full_like(x, i)
        count = count + yes
        ratio = torch.where(no, ratio + mass, torch.where(yes, 0.0, ratio))
        left = (pr - ratio[:, None] * qr).clamp_min(0.0).sum(1)
        mass = torch.where(no, left, torch.where(yes, 1.0, mass))
        cur = torch.where(yes, i, cur)
    pr, qr = p[b, cur + 1], q[b, (cur + 1).clamp_max(n - 1)]
    w = (pr - ratio[:, None] * qr).clamp_min(0.0)
    w = torch.where(mass[:, None] > 0, w, pr)
    score = torch.where(w > 0, w / s["race"], -1.0)
    best = torch.where(score.amax(1) >= 0, score.argmax(1), -1)
    step = torch.arange(n + 1, device=dev)[None, :]
    toks = torch.where(step < count[:, None], out[:, :n + 1],
                       torch.where(step == count[:, None], best[:, None], -1))
    nod = torch.where(step < count[:, None], nodes[:, :n + 1], -1)
    return toks.int(), nod.int(), count.int()


# --------------------------------------------------------------------- work ---

def work(case):
    if case["op"] == "distill":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + case["rows"] * (8 * case["k"] + 8),
                "flops": 6 * n}
    if case["op"] == "attention":
        B, n, H, KV, D = (case[k] for k in ("batch", "nodes", "heads", "kv_heads", "dim"))
        keys = sum(L + n for L in _lengths(case))
        return {"bytes": keys * KV * D * 4 + B * n * H * (4 * D + 4),
                "flops": 4 * n * H * D * keys}
    # the rows that a walk visits: one pair, and another for each accepted
    # token; drafts like these are accepted about seven times in ten a level
    B, n, V, E = case["batch"], case["nodes"], case["cols"], SIZE[case["dtype"]]
    depth, width = 0, 1
    left = n
    while left > 0:
        left -= min(left, case["branch"] * width)
        width *= case["branch"]
        depth += 1
    pairs = sum(0.7 ** d for d in range(depth + 1))
    return {"bytes": int(B * V * (2 * E * pairs + 4)), "flops": int(B * V * 10 * pairs)}


# -------------------------------------------------------------------- exact ---

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "distill":
        return _exact_distill(s)
    if case["op"] == "attention":
        return _exact_attention(s)
    return _exact_verify(s)


def _exact_distill(s):
    c = s["case"]
    T, V = c["temperature"], c["cols"]
    losses, grads = [], []
    step = max(1, 40_000_000 // V)
    for r in range(0, c["rows"], step):
        z = torch.log_softmax(s["logits"][r:r + step].double() / T, dim=1)
        prob = z.exp()
        idx = s["index"][r:r + step].long()
        val = s["value"][r:r + step].double()
        # the teacher as a dense row over the vocabulary, one spare column for absent entries
        R = z.shape[0]
        at = torch.where((idx >= 0) & (idx < V), idx, V)
        raw = torch.full((R, V + 1), -math.inf, dtype=torch.float64, device=z.device)
        raw.scatter_(1, at, val)
        raw = raw[:, :V]
        listed_ = torch.isfinite(raw)
        t = torch.where(listed_, (raw if c["tail"] else raw / T).exp(), 0.0)
        if not c["tail"]:
            t = t / t.sum(1, keepdim=True)
        kl = torch.xlogy(t, t).sum(1) - (t * torch.where(listed_, z, 0.0)).sum(1)
        grad = prob * t.sum(1, keepdim=True) - t
        if c["tail"]:
            rest = (1.0 - t.sum(1)).clamp_min(0.0)
            student = torch.where(listed_, 0.0, prob).sum(1)
            kl = kl + torch.xlogy(rest, rest) - torch.xlogy(rest, student)
            inside = torch.where(listed_, 0.0, prob) / student[:, None]
            grad = grad + rest[:, None] * (prob - inside)
        has = listed_.any(1)
        losses.append(torch.where(has, T * T * kl, 0.0))
        grad = grad * (T * s["weight"][r:r + step].double()[:, None])
        grads.append(torch.where(has[:, None], grad, 0.0))
    return torch.cat(losses), torch.cat(grads)


def _exact_attention(s):
    c = s["case"]
    B, n, H, KV, D, ps = (c[k] for k in ("batch", "nodes", "heads", "kv_heads", "dim", "page"))
    par = _parents(n, c["branch"])
    o = torch.empty(B, n, H, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(B, n, H, dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(_lengths(c)):
        pages = s["table"][b, :(L + n + ps - 1) // ps].long()
        hide = torch.ones(n, L + n, dtype=torch.bool)
        hide[:, :L] = False
        for i in range(n):
            a = i
            while a >= 0:
                hide[i, L + a] = False
                a = par[a]
        hide = hide.to(o.device)
        for h in range(KV):
            k = s["kc"][pages, :, h].reshape(-1, D)[:L + n].double()
            v = s["vc"][pages, :, h].reshape(-1, D)[:L + n].double()
            for head in range(h * (H // KV), (h + 1) * (H // KV)):
                x = s["q"][b, :, head].double() @ k.T / math.sqrt(D)
                x = x.masked_fill(hide, -math.inf)
                lse[b, :, head] = torch.logsumexp(x, 1)
                o[b, :, head] = torch.softmax(x, 1) @ v
    return o, lse


def _exact_verify(s):
    c = s["case"]
    n, V = c["nodes"], c["cols"]
    par = _parents(n, c["branch"])
    tokens, u = s["tokens"].tolist(), s["uniform"].double().tolist()
    temps = s["temperature"].double().tolist()
    toks = torch.full((c["batch"], n + 1), -1, dtype=torch.int32)
    nodes = toks.clone()
    count = torch.zeros(c["batch"], dtype=torch.int32)

    def dist(row, T):
        if T <= 0:
            hot = torch.zeros(V, dtype=torch.float64, device=row.device)
            hot[row.float().argmax()] = 1.0
            return hot
        return torch.softmax(row.double() / T, 0)

    for b in range(c["batch"]):
        cur, done = -1, 0
        while True:
            p = dist(s["target"][b, cur + 1], temps[b])
            kids = [i for i in range(cur + 1, n) if par[i] == cur and 0 <= tokens[b][i] < V]
            nxt = None
            rest = p
            if kids:
                q = dist(s["draft"][b, cur + 1], temps[b])
            for i in kids:
                x = tokens[b][i]
                if u[b][i] * float(q[x]) < float(rest[x]):
                    nxt = i
                    break
                # what is left of the target once the draft's mass is taken out
                left = (rest - q).clamp_min(0.0)
                if float(left.sum()) <= 0:
                    break
                rest = left / left.sum()
            if nxt is None:
                score = torch.where(rest > 0, rest / s["race"][b].double(), -1.0)
                toks[b, done] = int(score.argmax())
                count[b] = done
                break
            toks[b, done], nodes[b, done] = tokens[b][nxt], nxt
            done, cur = done + 1, nxt
    dev = s["race"].device
    return toks.to(dev), nodes.to(dev), count.to(dev)
