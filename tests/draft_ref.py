"""Plain float64 forms (numpy, straight from the definitions) of the draft
model's operators: distillation from a teacher's top entries, attention of a
tree of new tokens over a paged cache, verification of drafted tokens.  They
share no code with the GPU path."""
from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24  # half a step of float32, relative


def f64(a):
    """float32 arrays, or bfloat16 bits in uint16, as float64."""
    a = np.asarray(a)
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return a.astype(np.float64)


def distill(x, index, value, grad=None, T=1.0, tail=False):
    """Loss and dlogits, and for each the sum of the magnitudes that its fp32
    rounding errors are relative to."""
    x, value = f64(x), f64(value)
    R, C = x.shape
    K = index.shape[1]
    g = np.ones(R) if grad is None else f64(grad)
    loss, dl = np.zeros(R), np.zeros((R, C))
    lmag, dmag = np.zeros(R), np.zeros((R, C))
    for r in range(R):
        ent = [(int(index[r, k]), value[r, k]) for k in range(K) if 0 <= index[r, k] < C]
        m = np.max(x[r])
        if not ent or m == -np.inf:
            continue
        v = np.array([e[1] for e in ent])
        cols = np.array([e[0] for e in ent])
        if tail:
            lt = v
        else:
            if v.max() == -np.inf:
                continue
            lt = v / T - v.max() / T
            lt = lt - np.log(np.exp(lt).sum())
        t = np.exp(lt)
        z = (x[r] - m) / T
        e = np.exp(z)
        Z = e.sum()
        s = e / Z
        unl = np.ones(C, bool)
        unl[cols] = False
        et = np.where(unl, e, 0.0)
        Zt = et.sum()
        tt = max(0.0, 1.0 - t.sum()) if tail and Zt > 0 else 0.0
        mass = t.sum() + tt if tail else 1.0
        on = t > 0
        ls = z[cols] - np.log(Z)
        loss[r] = T * T * np.sum(t[on] * (lt[on] - ls[on]))
        # t_k carries a relative error of about |ln t_k| steps, the student's
        # logarithm one of |x - m| / T steps
        zz = np.where(np.isfinite(z[cols]), np.abs(z[cols]), 0.0)
        step = np.abs(np.where(on, lt, 0.0)) + zz + np.log(Z) + 1
        lmag[r] = T * T * np.sum(t[on] * step[on] * (1 + np.abs(np.where(on, lt, 0))[on]))
        dl[r] = mass * s
        np.subtract.at(dl[r], cols, t)
        dmag[r] = mass * s * (1 + np.abs(np.where(np.isfinite(z), z, 0)))
        np.add.at(dmag[r], cols, t * (1 + np.abs(np.where(on, lt, 0.0))))
        if tail:
            st = Zt / Z
            dt = (K + 64) / 64  # the sum of t, in units of 64 steps
            if tt > 0:
                loss[r] += T * T * tt * (np.log(tt) - np.log(st))
                dl[r] -= tt * et / Zt
                dmag[r] += tt * et / Zt * (1 + np.abs(np.where(np.isfinite(z), z, 0)))
            if st > 0:
                lmag[r] += T * T * (dt + tt) * (abs(np.log(max(tt, 1e-7))) + abs(np.log(st)) + 2)
                dmag[r] += dt * (et / Zt)
        dl[r] *= g[r] * T
        dmag[r] *= abs(g[r]) * T
    return loss, dl, lmag, dmag


def ancestors(par, n):
    """seen[i, j] for one sequence; par None is a chain.  A row whose chain of
    parents does not end at -1 sees nothing."""
    seen = np.zeros((n, n), bool)
    here = np.ones(n, bool)
    for i in range(n):
        if par is None:
            seen[i, :i + 1] = True
            continue
        a = i
        while a >= 0:
            seen[i, a] = True
            up = int(par[a])
            if up < -1 or up >= a:
                here[i] = False
                break
            a = up
        if not here[i]:
            seen[i] = False
    return seen, here


def tree_attention(q, kc, vc, table, ctx, parents=None, scale=None):
    """o, lse and sum_j p_j |v_j| (bf16 bits in, float64 out)."""
    q = f64(q)
    B, n, H, D = q.shape
    pages, ps, KV, _ = kc.shape
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    o = np.zeros((B, n, H, D))
    mag = np.zeros((B, n, H, D))
    lse = np.full((B, n, H), -np.inf)
    for b in range(B):
        L = max(0, int(ctx[b]))
        seen, here = ancestors(None if parents is None else parents[b], n)
        pos = np.arange(min(L + n, table.shape[1] * ps))
        page = table[b][pos // ps] if len(pos) else np.zeros(0, int)
        ok = (page >= 0) & (page < pages)
        k = f64(kc[np.where(ok, page, 0), pos % ps]) if pages else np.zeros((len(pos), KV, D))
        v = f64(vc[np.where(ok, page, 0), pos % ps]) if pages else np.zeros((len(pos), KV, D))
        for i in range(n):
            if not here[i]:
                continue
            vis = ok & ((pos < L) | seen[i][np.clip(pos - L, 0, n - 1)])
            if not vis.any():
                continue
            for h in range(H):
                kv = h // (H // KV)
                s = scale * (k[vis, kv] @ q[b, i, h])
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                o[b, i, h] = p @ v[vis, kv]
                mag[b, i, h] = p @ np.abs(v[vis, kv])
                lse[b, i, h] = m + np.log(e.sum())
    return o, lse, mag


def softmax_row(x, T):
    if T <= 0:
        p = np.zeros(x.shape)
        if np.any(x > -np.inf):
            p[int(np.argmax(x))] = 1.0
        return p
    m = np.max(x)
    if m == -np.inf:
        return np.zeros(x.shape)
    e = np.exp((x - m) / T)
    return e / e.sum()


def verify(target, draft, tokens, uniform, race, parents=None, temperature=None):
    """out_tokens, out_nodes, out_count, and for each sequence how far its
    closest decision was from the other answer (relative)."""
    B, n1, V = target.shape
    n = n1 - 1
    toks = np.full((B, n1), -1, np.int32)
    nodes = np.full((B, n1), -1, np.int32)
    count = np.zeros(B, np.int32)
    margin = np.full(B, np.inf)
    for b in range(B):
        T = 1.0 if temperature is None else float(temperature[b])
        cur, done = -1, 0
        while True:
            p = softmax_row(f64(target[b, cur + 1]), T)
            if np.isnan(p).any() or not p.any():
                break
            rest, q, nxt = p, None, -1
            for i in range(cur + 1, n):
                x = int(tokens[b, i])
                up = i - 1 if parents is None else int(parents[b, i])
                if up != cur or not 0 <= x < V:
                    continue
                if q is None:
                    q = softmax_row(f64(draft[b, cur + 1]), T)
                lhs, rhs = float(uniform[b, i]) * q[x], rest[x]
                if T > 0 and max(lhs, rhs) > 0:
                    margin[b] = min(margin[b], abs(lhs - rhs) / max(p[x], q[x]))
                if lhs < rhs:
                    nxt = i
                    break
                left = np.maximum(rest - q, 0.0)
                if left.sum() <= 0:
                    break
                rest = left / left.sum()
            if nxt < 0:
                with np.errstate(divide="ignore", invalid="ignore"):
                    s = np.where(rest > 0, rest / f64(race[b]), -1.0)
                j = int(np.argmax(s))
                toks[b, done] = j
                if T > 0 and V > 1:
                    second = np.max(np.delete(s, j))
                    margin[b] = min(margin[b], (s[j] - second) / s[j] * min(1.0, rest[j] / p[j]))
                break
            toks[b, done], nodes[b, done] = tokens[b, nxt], nxt
            done, cur = done + 1, nxt
        count[b] = done
    return toks, nodes, count, margin
