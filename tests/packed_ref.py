"""Plain float64 forms (torch on the CPU, straight from the definitions) of the operators of
a decoder's pass over packed sequences: norms of queries and keys with the position
rotation, causal attention of grouped heads, log probabilities of given tokens, and the
gradients.  They share no code with the GPU path.  Beside each result stands the sum of the
magnitudes that its rounding errors are relative to."""
from __future__ import annotations

import math

import torch

EPS = 2.0 ** -24  # half a step of float32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of a type


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def table(positions, rot, base=10000.0):
    """Cosines and sines (float32) of an angle for each position and pair."""
    a = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return a.cos().float(), a.sin().float()


def _angles(cos, sin, pos):
    """Of tokens beyond the table NaN, of padding (whose rows are zero) no turn."""
    at = pos.clamp(0, cos.shape[0] - 1)
    c, s = cos.double()[at], sin.double()[at]
    beyond, padding = (pos >= cos.shape[0])[:, None], (pos < 0)[:, None]
    c = torch.where(padding, 1.0, torch.where(beyond, math.nan, c))
    s = torch.where(padding, 0.0, torch.where(beyond, math.nan, s))
    return c[:, None, :], s[:, None, :]


def _kept(x, pos, eps):
    ms = (x * x).mean(-1, keepdim=True)
    return ms, (pos >= 0)[:, None, None] & torch.isfinite(ms) & (ms <= 3.4e38) & (ms + eps > 0)


def rope(x, w, cos, sin, pos, eps, interleaved):
    """y and its magnitudes for x [tokens, heads, dim]."""
    x, pos = x.double(), pos.long()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    ms, keep = _kept(x, pos, eps)
    u = x * w / torch.sqrt(ms + eps)
    a, b = pairs(2 * cos.shape[1], interleaved)
    c, s = _angles(cos, sin, pos)
    y, mag = u.clone(), u.abs()
    y[..., a], y[..., b] = c * u[..., a] - s * u[..., b], s * u[..., a] + c * u[..., b]
    mag[..., a] = (c * u[..., a]).abs() + (s * u[..., b]).abs()
    mag[..., b] = (s * u[..., a]).abs() + (c * u[..., b]).abs()
    zero = torch.zeros(())
    return torch.where(keep, y, zero.double()), torch.where(keep, mag, zero.double())


def rope_bwd(dy, x, w, cos, sin, pos, eps, interleaved):
    """(dx, magnitudes), (dw, magnitudes)."""
    x, dy, pos = x.double(), dy.double(), pos.long()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    ms, keep = _kept(x, pos, eps)
    r = 1.0 / torch.sqrt(ms + eps)
    a, b = pairs(2 * cos.shape[1], interleaved)
    c, s = _angles(cos, sin, pos)
    g, gm = dy.clone(), dy.abs()
    g[..., a], g[..., b] = c * dy[..., a] + s * dy[..., b], c * dy[..., b] - s * dy[..., a]
    gm[..., a] = (c * dy[..., a]).abs() + (s * dy[..., b]).abs()
    gm[..., b] = (c * dy[..., b]).abs() + (s * dy[..., a]).abs()
    xh = x * r
    dw = torch.where(keep, g * xh, 0.0).sum((0, 1))
    dwm = torch.where(keep, gm * xh.abs(), 0.0).sum((0, 1))
    h, hm = g * w, gm * w.abs()
    dx = r * (h - xh * (h * xh).mean(-1, keepdim=True))
    dxm = r * (hm + xh.abs() * (hm * xh.abs()).mean(-1, keepdim=True))
    return ((torch.where(keep, dx, 0.0), torch.where(keep, dxm, 0.0)), (dw, dwm))


def spans(cu, tokens):
    cu = [min(max(int(c), 0), tokens) for c in cu]
    return [(a, b) for a, b in zip(cu, cu[1:]) if b > a]


def attention(q, k, v, cu, scale):
    """o, lse, sum_j p |v|, and the largest error-carrying magnitude scale sum_d |q k| of
    each row (rows outside every sequence: NaN)."""
    T, H, D = q.shape
    G = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    o, lse = torch.full((T, H, D), math.nan).double(), torch.full((H, T), math.nan).double()
    om, sm = o.clone(), lse.clone()
    for a, b in spans(cu, T):
        hide = torch.ones(b - a, b - a, dtype=torch.bool).triu(1)
        for h in range(H):
            kk, vv = k[a:b, h // G], v[a:b, h // G]
            s = scale * (q[a:b, h] @ kk.T)
            s = s.masked_fill(hide, -math.inf)
            p = torch.softmax(s, 1)
            lse[h, a:b] = torch.logsumexp(s, 1)
            # 0 x NaN of an unseen row must not count
            for dst, val in ((o, vv), (om, vv.abs())):
                seen = torch.where(torch.isfinite(val), val, 0.0)
                dst[a:b, h] = p @ seen
                for j in torch.nonzero(~torch.isfinite(val).all(1)).flatten().tolist():
                    dst[a + j:b, h] = math.nan
            sm[h, a:b] = scale * (q[a:b, h].abs() @ kk.abs().T).masked_fill(hide, 0.0).amax(1)
    return o, lse, om, sm


def attention_bwd(do, q, k, v, o, cu, scale):
    """(dq, dk, dv) and their magnitudes, for o as it is given."""
    T, H, D = q.shape
    G = H // k.shape[1]
    do, q, k, v, o = (t.double() for t in (do, q, k, v, o))
    dq, dk, dv = (torch.zeros_like(t) for t in (q, k, v))
    mq, mk, mv = (torch.zeros_like(t) for t in (q, k, v))
    for a, b in spans(cu, T):
        hide = torch.ones(b - a, b - a, dtype=torch.bool).triu(1)
        for h in range(H):
            kv = h // G
            s = (scale * (q[a:b, h] @ k[a:b, kv].T)).masked_fill(hide, -math.inf)
            p = torch.softmax(s, 1)
            g = do[a:b, h]
            dp = g @ v[a:b, kv].T
            delta = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - delta) * scale
            dm = p * ((dp - delta).abs() + (g * o[a:b, h]).abs().sum(1, keepdim=True)) * scale
            dv[a:b, kv] += p.T @ g
            mv[a:b, kv] += p.T @ g.abs()
            dq[a:b, h] = ds @ k[a:b, kv]
            mq[a:b, h] = dm @ k[a:b, kv].abs()
            dk[a:b, kv] += ds.T @ q[a:b, h]
            mk[a:b, kv] += dm.T @ q[a:b, h].abs()
    return (dq, dk, dv), (mq, mk, mv)


def logprob(x, tokens, T, k, ignore=-100):
    """Dict of logprob, entropy, row_max, log_sum, rank, top_index, top_logprob, and the
    rows' magnitudes: `lp` of the logarithms, `ent` of the entropy."""
    R, V = x.shape
    x = x.double()
    out = {n: torch.zeros(R, dtype=torch.float64)
           for n in ("logprob", "entropy", "row_max", "log_sum", "lp", "ent")}
    out["rank"] = torch.full((R,), -1, dtype=torch.int64)
    out["top_index"] = torch.full((R, k), -1, dtype=torch.int64)
    out["top_logprob"] = torch.zeros(R, k, dtype=torch.float64)
    for r in range(R):
        t, row = int(tokens[r]), x[r]
        if t == ignore:
            continue
        good = 0 <= t < V
        if torch.isnan(row).any() or (row == math.inf).any():
            for n in ("logprob", "entropy", "row_max", "log_sum"):
                out[n][r] = math.nan
            out["top_logprob"][r] = math.nan
            continue
        m = row.max()
        out["row_max"][r] = m
        if good:
            at = torch.arange(V)
            out["rank"][r] = int(((row > row[t]) | ((row == row[t]) & (at < t))).sum())
        out["top_logprob"][r] = -math.inf
        if m == -math.inf:
            out["logprob"][r] = 0.0 if good else math.nan
            continue
        z = (row - m) / T
        e = torch.exp(z)
        ls = math.log(float(e.sum()))
        p = e / e.sum()
        zz = torch.where(p > 0, z, 0.0)
        out["log_sum"][r] = ls
        out["logprob"][r] = float(z[t]) - ls if good else math.nan
        out["entropy"][r] = ls - float((p * zz).sum())
        out["lp"][r] = 1.0 + ls + float((p * zz.abs()).sum()) + (abs(float(z[t])) if good and
                                                                 z[t] > -math.inf else 0.0)
        out["ent"][r] = 1.0 + ls + float((p * zz.abs() * (1.0 + zz.abs())).sum())
        order = torch.sort(-row, stable=True).indices[:k]
        order = order[row[order] > -math.inf]
        out["top_index"][r, :len(order)] = order
        out["top_logprob"][r, :len(order)] = z[order] - ls
    return out


def logprob_bwd(x, tokens, g, h, T, ignore=-100):
    """dlogits and its magnitudes."""
    R, V = x.shape
    x = x.double()
    g = torch.zeros(R) if g is None else g
    h = torch.zeros(R) if h is None else h
    d, mag = torch.zeros(R, V).double(), torch.zeros(R, V).double()
    for r in range(R):
        t, row = int(tokens[r]), x[r]
        if t == ignore or row.max() == -math.inf:
            continue
        lp = torch.log_softmax(row / T, 0)
        p = lp.exp()
        lz = torch.where(p > 0, lp, 0.0)
        ent = -(p * lz).sum()
        gr, hr = float(g[r]), float(h[r])
        d[r] = -gr * p - hr * p * (lz + ent)
        mag[r] = p * (abs(gr) + abs(hr) * (lz.abs() + ent)) * (1.0 + lz.abs())
        if 0 <= t < V:
            d[r, t] += gr
            mag[r, t] += abs(gr)
        d[r] /= T
        mag[r] /= T
    return d, mag
