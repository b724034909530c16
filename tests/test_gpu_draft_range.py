"""The draft model's operators at the ends of their ranges (distillation and
verification): lists that hold little of the mass, finite mask values, low
temperatures, NaN.  Both kernels of each operator."""
import numpy as np
import pytest
import torch

import draft_ref as ref
import row_reduction_pass_gb300 as rr

from test_gpu_draft import check_verify, run_verify, verify_inputs
from parity import check_guards, compare, empty_like_dev, host, store, to_dev

pytestmark = pytest.mark.gpu

LOWEST = {"f32": float(np.finfo(np.float32).min), "bf16": -3.3895313892515355e38}


def run_distill(x, index, value, g, dtype, T, tail, pads=(0, 0)):
    """pads that differ take the kernel of single-element accesses."""
    rows, k = index.shape
    dl, loss = empty_like_dev(x.shape, dtype, pads[1]), empty_like_dev((rows,), "f32")
    rr.rr_distill_fwd_bwd(to_dev(x, pads[0]), to_dev(index).view(rows, k),
                          to_dev(value).view(rows, k), loss, dl, grad=to_dev(g), temperature=T,
                          tail=tail)
    torch.cuda.synchronize()
    check_guards()
    assert rr.rr_read_device_error(0) == 0
    return host(loss), host(dl)


def small_list(rows, cols, k, T, dtype, seed):
    """A student's logits, and the top of a teacher's that are the student's with noise,
    as log-probabilities at temperature T."""
    rng = np.random.default_rng(seed)
    x = store(3.0 * rng.standard_normal((rows, cols)), dtype)
    t = ref.f64(x) + rng.standard_normal((rows, cols))
    index = np.argsort(-t, axis=1)[:, :k].astype(np.int32)
    z = t / T
    lse = np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) + z.max(1, keepdims=True)
    value = np.take_along_axis(z - lse, index.astype(np.int64), 1).astype(np.float32)
    return x, index, value, rng.uniform(0.5, 1.5, rows).astype(np.float32)


def tail_bounds(x, index, value, g, T, k):
    """What the fp32 arithmetic may be off by where list and student's list hold less
    than half of the mass, in units of EPS (half a step, relative):
      loss: a listed term t (lt - z + ln Z): lt, z = (x - m) / T (a difference, a product)
        and the difference one step of their size each, the product one, the sums of the
        list K / 32 + 6 (a lane's share one after the other, then five levels) of |lt - ref|
        and of st ln Z; t itself 5 (expf 2 ulp and its argument), which the loss feels as
        t (lt - ls - ln tt + ln st');
      the tail's term: the student's list, sl, 4 |z| + 8 for the exponentials (argument
        and ex2.approx, 2^-22, also where the parts are scaled to the row's maximum), 40
        for the sums of Z (at most 28 terms a thread in four chains, and the meetings), and
        two logarithms of 4 (1 ulp each of log1pf, and its argument);
      an unlisted gradient g T e / Z (st - tt Zl / Zt): st K / 32 + 14, sl as above.
    Each is allowed once, and half a step of the result's type."""
    X = ref.f64(x)
    cols = index.astype(np.int64)
    lt, z = value.astype(np.float64), X / T
    z = z - z.max(1, keepdims=True)
    lnZ = np.log(np.exp(z).sum(1, keepdims=True))
    zl = np.take_along_axis(z, cols, 1)
    t, s = np.exp(lt), np.exp(zl - lnZ)
    st, sl = t.sum(1, keepdims=True), s.sum(1, keepdims=True)
    assert st.max() < 0.5 and sl.max() < 0.5
    sums = k / 32 + 6
    felt = np.abs(lt - zl + lnZ) + np.abs(np.log1p(-st) - np.log1p(-sl))
    units = (t * (2 * np.abs(lt) + 3 * np.abs(zl) + sums * (np.abs(lt) + np.abs(zl) + lnZ)
                  + 5 * felt)).sum(1)
    units_sl = (s * (4 * np.abs(zl) + 48)).sum(1)
    units += units_sl + 4 * (np.abs(np.log1p(-st)) + np.abs(np.log1p(-sl)))[:, 0]
    per_unlisted = (sums + 8) * st[:, 0] + units_sl
    # tt = 1 - st and its product are rounded relative to themselves: 2 more of sl
    return T * T * units, (g * T * (per_unlisted + 2 * sl[:, 0]))[:, None] * np.exp(z - lnZ)


@pytest.mark.parametrize("pads", [(0, 0), (1, 0)])
@pytest.mark.parametrize("rows,cols,k,T,dtype", [
    (37, 131072, 4, 4.0, "f32"), (37, 131072, 4, 4.0, "bf16"), (60, 20000, 32, 4.0, "f32"),
    (60, 20011, 1, 4.0, "f32"), (90, 5003, 2, 8.0, "bf16"), (5, 300001, 4, 4.0, "f32")])
def test_distill_tail_of_a_list_with_little_mass(rows, cols, k, T, dtype, pads):
    x, index, value, g = small_list(rows, cols, k, T, dtype, cols + k)
    loss, dl = run_distill(x, index, value, g, dtype, T, True, pads)
    rl, rd, _, _ = ref.distill(x, index, value, g, T, True)
    lu, du = tail_bounds(x, index, value, g, T, k)
    compare("distill loss", loss, rl, ref.EPS, 0.0, scale=lu, scale_rtol=ref.EPS)
    if dtype == "f32":
        free = np.ones(x.shape, bool)
        np.put_along_axis(free, index.astype(np.int64), False, 1)
        # (a result's own exponential: 2 |z| + 6 steps of it, |z| at most 10 here)
        compare("unlisted dlogits", np.where(free, dl, 0.0), np.where(free, rd, 0.0),
                27 * ref.EPS, 0.0, scale=du, scale_rtol=ref.EPS)


def compare_distill(got, x, index, value, g, dtype, T, tail, atol=1e-30):
    rl, rd, lm, dm = ref.distill(x, index, value, g, T, tail)
    compare("distill loss", got[0], rl, 0.0, atol, scale=lm, scale_rtol=64 * ref.EPS)
    compare("distill dlogits", got[1], rd, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23, atol,
            scale=dm, scale_rtol=64 * ref.EPS)


@pytest.mark.parametrize("fill", ["lowest", -1e30, -1e10, -1e9])
@pytest.mark.parametrize("cols,dtype", [(97, "f32"), (1000, "bf16"), (4097, "bf16"), (50304, "bf16"),
                                        (50304, "f32"), (131075, "f32"), (300001, "f32")])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_columns_masked_by_a_finite_value(cols, tail, dtype, fill):
    """All but a run of columns and a few scattered ones hold a mask's value; some lists
    have a masked column (300001: the kernel of single-element accesses)."""
    rows, k, T = (24, 6, 0.3) if cols < 50000 else (6, 6, 0.3)
    rng = np.random.default_rng(cols)
    x = store(rng.standard_normal((rows, cols)) * 3.0, dtype)
    keep = np.zeros(cols, bool)
    keep[cols // 3:cols // 3 + cols // 20 + 8] = True
    keep[rng.choice(cols, 4, replace=False)] = True
    x[:, ~keep] = store(np.array([LOWEST[dtype] if fill == "lowest" else fill]), dtype)[0]
    index = np.stack([rng.choice(np.flatnonzero(keep), k, replace=False) for _ in range(rows)])
    z = rng.standard_normal((rows, k))
    value = z - np.log(np.exp(z).sum(1, keepdims=True)) - 0.4 if tail else z
    if fill != "lowest":
        index[::4, 2] = np.flatnonzero(~keep)[-1]
    index, value = index.astype(np.int32), value.astype(np.float32)
    g = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    got = run_distill(x, index, value, g, dtype, T, tail)
    compare_distill(got, x, index, value, g, dtype, T, tail)


@pytest.mark.parametrize("T", [1e-6, 1e-9, 1e-12, 2.0 ** -120])
@pytest.mark.parametrize("cols,dtype", [(97, "f32"), (4097, "bf16"), (50304, "f32"),
                                        (131075, "f32"), (300001, "f32")])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_low_temperatures(cols, tail, dtype, T):
    """The distributions are all on their largest logits; the loss, about T times a
    difference of logits, keeps its digits."""
    rows, k = 20 if cols < 50000 else 6, 5
    rng = np.random.default_rng(cols)
    x = store(rng.standard_normal((rows, cols)) * 6.0 + 7.0, dtype)
    index = np.stack([rng.choice(cols, k, replace=False) for _ in range(rows)]).astype(np.int32)
    index[::2, 0] = ref.f64(x)[::2].argmax(1)
    z = rng.standard_normal((rows, k))
    value = (z - np.log(np.exp(z).sum(1, keepdims=True)) - 0.4 if tail else z).astype(np.float32)
    g = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    got = run_distill(x, index, value, g, dtype, T, tail)
    # (T 1e-30: exponentials flushed to zero)
    compare_distill(got, x, index, value, g, dtype, T, tail, atol=T * 1e-30)


@pytest.mark.parametrize("T", [2.0 ** 30, 2.0 ** 60])
@pytest.mark.parametrize("cols", [97, 300001])
def test_distill_high_temperatures(cols, T):
    """Without a tail (T^2 times what the list's weights leave of 1 would be the loss)."""
    rows, k, rng = 5, 3, np.random.default_rng(cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    index = np.stack([rng.choice(cols, k, replace=False) for _ in range(rows)]).astype(np.int32)
    value, g = rng.standard_normal((rows, k)).astype(np.float32), np.ones(rows, np.float32)
    compare_distill(run_distill(x, index, value, g, "f32", T, False), x, index, value, g, "f32", T,
                    False)


@pytest.mark.parametrize("cols,dtype", [(2, "f32"), (97, "f32"), (4097, "bf16"), (50304, "bf16"),
                                        (131075, "f32"), (300001, "f32")])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_nan_and_inf_logits(cols, tail, dtype):
    """One NaN (or +inf) anywhere in a row, listed or not, makes the row's loss and
    dlogits NaN, and so does a row of NaN, or of NaN and -inf; the rows beside it are as
    they would be."""
    rng = np.random.default_rng(cols)
    rows, k, T = 16, 2, 2.0
    x = store(rng.standard_normal((rows, cols)) * 3.0, dtype)
    nan, inf, ninf = store(np.array([np.nan, np.inf, -np.inf]), dtype)
    index = np.stack([rng.choice(cols, k, replace=False) for _ in range(rows)]).astype(np.int32)
    z = rng.standard_normal((rows, k))
    value = (z - np.log(np.exp(z).sum(1, keepdims=True)) - 0.4 if tail else z).astype(np.float32)
    x[1] = nan
    x[2], x[2, cols // 2] = ninf, nan
    x[4, 0], x[5, cols - 1], x[6, cols // 2] = nan, nan, nan
    x[7, index[7, 1]] = nan
    x[8, cols // 3] = inf
    x[10, max(0, cols - 5):] = nan
    x[11], index[11] = nan, -1                   # no entry present: zeros
    x[13] = ninf                                 # fully masked: zeros
    g = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    loss, dl = run_distill(x, index, value, g, dtype, T, tail)
    bad = [1, 2, 4, 5, 6, 7, 8, 10]
    assert np.isnan(loss[bad]).all() and np.isnan(dl[bad]).all()
    assert loss[11] == 0 and (dl[11] == 0).all() and loss[13] == 0 and (dl[13] == 0).all()
    good = [r for r in range(rows) if r not in bad + [11]]
    compare_distill((loss[good], dl[good]), x[good], index[good], value[good], g[good], dtype, T,
                    tail)


@pytest.mark.parametrize("cols", [97, 50304, 300001])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("k", [1, 3, 200])
def test_distill_nan_values(cols, tail, k):
    """A NaN among the teacher's values, or all of them: no list without weight."""
    rng = np.random.default_rng(k)
    rows, k = 6, min(k, cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    index = np.stack([rng.choice(cols, k, replace=False) for _ in range(rows)]).astype(np.int32)
    value = (rng.standard_normal((rows, k)) - 9.0).astype(np.float32)
    value[1] = np.nan
    value[2, k // 2] = np.nan
    value[3], value[3, 0] = -np.inf, np.nan
    g = np.ones(rows, np.float32)
    loss, dl = run_distill(x, index, value, g, "f32", 1.0, tail)
    assert np.isnan(loss[1:4]).all() and np.isnan(dl[1:4]).all()
    good = [0, 4, 5]
    compare_distill((loss[good], dl[good]), x[good], index[good], value[good], g[good], "f32", 1.0,
                    tail)


# ------------------------------------------------------------- verification ---

def redraw(d, par, T, rng):
    """Tokens from the draft's distributions."""
    B, n, V = d.shape
    tok = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            up = i - 1 if par is None else par[b, i]
            tok[b, i] = rng.choice(V, p=ref.softmax_row(ref.f64(d[b, up + 1]), float(T[b])))
    return tok


@pytest.mark.parametrize("fill", ["lowest", -1e30, -1e10, -1e9])
@pytest.mark.parametrize("V,dtype", [(97, "f32"), (4097, "bf16"), (50304, "bf16"), (50304, "f32"),
                                     (300001, "f32")])
def test_verify_columns_masked_by_a_finite_value(V, dtype, fill):
    """All but a run of columns and a few scattered ones hold a mask's value, as a
    grammar's or a vocabulary's masks leave a row (300001: the one-block kernel)."""
    B, n = (16, 6) if V < 50000 else (4, 6)
    t, d, tok, u, e, par, T = verify_inputs(B, n, V, dtype, V, 2)
    T[::2] = 0.3
    rng = np.random.default_rng(V)
    keep = np.zeros(V, bool)
    keep[V // 3:V // 3 + V // 20 + 8] = True
    keep[rng.choice(V, 8)] = True
    bits = store(np.array([LOWEST[dtype] if fill == "lowest" else fill]), dtype)[0]
    t[:, :, ~keep], d[:, :, ~keep] = bits, bits
    tok = redraw(d, par, T, rng)
    want = check_verify(t, d, tok, u, e, par, T)
    assert (want[0][:, 0] >= 0).all() and want[2].max() > 0


@pytest.mark.parametrize("T", [1e-6, 1e-9, 1e-12, 2.0 ** -120])
@pytest.mark.parametrize("V,dtype", [(1003, "f32"), (50304, "bf16"), (300001, "f32")])
@pytest.mark.parametrize("branch", [0, 2])
def test_verify_low_temperatures(V, dtype, T, branch):
    B, n = (20, 6) if V < 50000 else (4, 6)
    t, d, tok, u, e, par, temps = verify_inputs(B, n, V, dtype, V + branch, branch, noise=0.1)
    temps[:] = T
    rng = np.random.default_rng(V)
    x = store(ref.f64(t) * 3 + 7, dtype), store(ref.f64(d) * 3 + 7, dtype)
    want = check_verify(*x, redraw(x[1], par, temps, rng), u, e, par, temps)
    assert (want[0][:, 0] >= 0).all() and want[2].max() > 0


@pytest.mark.parametrize("V", [200, 300001])
@pytest.mark.parametrize("branch", [0, 3])
def test_verify_undefined_draft_rows(V, branch):
    """A NaN or +inf in the draft's row: no child is accepted, and the token is that of a
    sequence in which nothing was drafted."""
    t, d, tok, u, e, par, T = verify_inputs(4, 5, V, "f32", V, branch)
    d[0, 0, 3], d[1, 0, V - 1], d[2, 0] = np.nan, np.inf, np.nan
    got = run_verify(t, d, tok, u, e, par, T)
    none = run_verify(t, d, np.full_like(tok, -1), u, e, par, T)
    for a, b in zip(got, none):
        assert (a[:3] == b[:3]).all()
    assert (got[0][:3, 0] >= 0).all()


# ---------------------------------------------------------------- attention ---

@pytest.mark.parametrize("batch", [2, 400])
def test_tree_attention_pages_but_no_table(batch):
    """A table of no width: nothing is seen, by either way of planning."""
    q = torch.randn(batch, 3, 4, 64, device="cuda").bfloat16()
    kc = torch.randn(5, 16, 2, 64, device="cuda").bfloat16()
    table = torch.empty(batch, 0, dtype=torch.int32, device="cuda")
    ctx = torch.full((batch,), 9, dtype=torch.int32, device="cuda")
    for par in (None, torch.full((batch, 3), -1, dtype=torch.int32, device="cuda")):
        o, l = torch.full_like(q, 7.0), torch.zeros(batch, 3, 4, device="cuda")
        rr.rr_attention_tree_fwd(q, kc, kc, table, ctx, o, lse=l, parents=par)
        torch.cuda.synchronize()
        assert rr.rr_read_device_error(0) == 0
        assert (o == 0).all() and torch.isneginf(l).all()
