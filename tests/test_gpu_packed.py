"""GPU parity of the packed-sequence operators (rr_qk_norm_rope, rr_attention_packed,
rr_token_logprob, forward and backward) with their float64 plain forms.

Tolerances, from the arithmetic (EPS = 2^-24, half a float32 step; HALF: half a step of the
storage type, relative):
  rotation: a value is two products of (x r w) with (c, s), r from a sum of dim squares over
    at most 32 lanes (dim / 32 + 5 additions) and rsqrt (4 EPS): 32 EPS of the magnitudes.
    Its gradient has a second such sum: 64 EPS.  The weights' gradients are sums over rows,
    at most a few hundred one after the other in a lane: 600 EPS of the sum of magnitudes.
  attention, float32 kernels: a score's error is dim EPS times scale sum |q k| (the plain form
    returns the largest of a row), a weight's relative error that plus 16 EPS, and a sum over
    n keys adds n EPS; on the tensor cores (bf16): products are exact, weights and ds are
    rounded (at most 2^-8 each), and so is the result (2^-8); delta carries the rounding of o
    (2^-8 of sum |dout o|).  2^-7 of the magnitudes is allowed beside the result's own
    rounding, as the float32 errors are far below.
  log probabilities: an exponential carries (|z| + 4) EPS, sums over a row some tens, the
    logarithm as much: 64 EPS of the magnitudes that the plain form returns.
Whole numbers are equal.
"""
import math

import pytest
import torch

import packed_ref as ref
import row_reduction_pass_gb300 as rr
from packed_ref import EPS, HALF

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(name, got, want, mag, rel, half=0.0, floor=1e-30):
    got, want = got.detach().double().cpu(), want.double()
    assert got.shape == want.shape
    both = torch.isnan(got) & torch.isnan(want) | (got == want)
    err = (got - want).abs()
    bound = floor + rel * mag + half * want.abs()
    bad = ~both & ~(err <= bound)
    if bad.any():
        i = int(torch.where(bad, torch.nan_to_num(err - bound, nan=math.inf), -1.0).argmax())
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} off; at {i}: got {got.flatten()[i]}, want "
            f"{want.flatten()[i]}, bound {torch.as_tensor(bound).expand_as(got).flatten()[i]}")


def rnd(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


class Buffer:
    """A device buffer of rows with room around and between them, filled with `fill`."""

    def __init__(self, rows, shape, dtype, gap=0, pad=0, fill=math.nan):
        width = math.prod(shape)
        self.raw = torch.full((64 + pad + rows * (width + gap) + 64,), fill, dtype=dtype,
                              device="cuda")
        flat = self.raw[64 + pad:64 + pad + rows * (width + gap)].view(rows, width + gap)
        self.view = flat[:, :width].view(rows, *shape)
        self.was = self.raw.clone()

    def untouched_around(self):
        """Nothing but the view was written."""
        now = self.raw.clone()
        keep = self.view.clone()
        self.view.copy_(torch.zeros_like(self.view))
        a = self.raw.clone()
        self.raw.copy_(self.was)
        self.view.copy_(torch.zeros_like(self.view))
        ok = torch.equal(a.view(torch.uint8), self.raw.clone().view(torch.uint8))
        self.raw.copy_(now)
        self.view.copy_(keep)
        return ok


def buf(t, gap=0, pad=0):
    b = Buffer(t.shape[0], t.shape[1:], t.dtype, gap, pad)
    b.view.copy_(t)
    b.was = b.raw.clone()
    return b


# ----------------------------------------------------------------- rotation ---

def check_rope(T, H, KV, D, R, dtype, interleaved=False, gap=0, pad=0, weights=True, seed=0,
               inplace=False, hard=False, eps=1e-6):
    dt = DT[dtype]
    q, k = rnd(seed, T, H, D, dtype=dt), rnd(seed + 1, T, KV, D, dtype=dt)
    gq, gk = rnd(seed + 2, T, H, D, dtype=dt), rnd(seed + 3, T, KV, D, dtype=dt)
    qw = (1 + 0.3 * rnd(seed + 4, D)).to(dt) if weights else None
    kw = (1 + 0.3 * rnd(seed + 5, D)).to(dt) if weights else None
    P = 500
    cos, sin = ref.table(P, R)
    pos = torch.randint(0, P, (T,), generator=torch.Generator().manual_seed(seed + 6))
    n_bad = 0
    if hard:
        q[0, 0, 1] = math.inf
        k[1, 0, 0] = math.nan
        q[2, 1] = 0.0
        q[3, 0] *= 1e-12 if dtype == "f32" else 1e-4
        pos[4], pos[5] = -1, -2 ** 31
        q[5] = math.nan
    cd, sd, pd = cos.cuda(), sin.cuda(), pos.int().cuda()
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    half, opt = HALF[dt], dict(eps=eps, interleaved=interleaved)
    bq, bk = buf(q, gap, pad), buf(k, gap, pad)
    oq = bq if inplace else Buffer(T, (H, D), dt, gap, pad)
    ok = bk if inplace else Buffer(T, (KV, D), dt, gap, pad)
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    rr.rr_qk_norm_rope_fwd(bq.view, bk.view, dev(qw), dev(kw), cd, sd, pd, oq.view, ok.view,
                           bad_position_count=count, **opt)
    for name, x, w, o in (("q", q, qw, oq), ("k", k, kw, ok)):
        want, mag = ref.rope(x, w, cos, sin, pos, eps, interleaved)
        close(name, o.view, want, mag, 32 * EPS, half)
        assert o.untouched_around()
    assert int(count) == n_bad
    # the gradient, from the inputs as they were
    bq, bk, dq, dk = (buf(t, gap, pad) for t in (q, k, gq, gk))
    oq = dq if inplace else Buffer(T, (H, D), dt, gap, pad)
    ok = dk if inplace else Buffer(T, (KV, D), dt, gap, pad)
    dqw, dkw = (torch.full((D,), math.nan, dtype=dt, device="cuda") for _ in range(2))
    rr.rr_qk_norm_rope_bwd(dq.view, dk.view, bq.view, bk.view, dev(qw), dev(kw), cd, sd, pd,
                           oq.view, ok.view, dqw, dkw, **opt)
    for name, dy, x, w, o, dw in (("q", gq, q, qw, oq, dqw), ("k", gk, k, kw, ok, dkw)):
        (want, mag), (wantw, magw) = ref.rope_bwd(dy, x, w, cos, sin, pos, eps, interleaved)
        close("d" + name, o.view, want, mag, 64 * EPS, half)
        close("dw" + name, dw, wantw, magw, 600 * EPS, half)
        assert o.untouched_around()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(2, 2), (6, 4), (16, 16), (32, 32), (64, 32), (80, 80), (96, 48),
                                 (128, 128), (130, 64), (256, 256), (256, 64)])
def test_rope(D, R, interleaved, dtype):
    check_rope(37, 6, 3, D, R, dtype, interleaved, seed=D + R)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,KV", [(1, 1, 1), (1, 32, 8), (3, 5, 1), (700, 3, 3), (2, 64, 8),
                                    (1300, 16, 4)])
def test_rope_shapes(T, H, KV, dtype):
    check_rope(T, H, KV, 128, 128, dtype, seed=T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gap,pad,inplace", [(64, 0, False), (64, 0, True), (3, 1, False),
                                             (3, 1, True), (8, 4, False)])
def test_rope_layouts(gap, pad, inplace, dtype):
    check_rope(21, 4, 2, 64, 64, dtype, gap=gap, pad=pad, inplace=inplace, seed=gap)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,eps", [(64, 1e-6), (64, 0.0), (10, 0.0)])
def test_rope_padding_and_nonfinite_heads(D, eps, dtype):
    check_rope(9, 3, 2, D, D, dtype, hard=True, eps=eps, weights=D == 64)


def test_rope_positions_beyond_the_table_and_without_positions():
    T, D = 7, 64
    cos, sin = ref.table(5, D)
    q = rnd(1, T, 2, D)
    out, count = torch.empty(T, 2, D, device="cuda"), torch.zeros(1, dtype=torch.int32,
                                                                  device="cuda")
    rr.rr_qk_norm_rope_fwd(q.cuda(), None, None, None, cos.cuda(), sin.cuda(), None, out, None,
                           bad_position_count=count)
    want, mag = ref.rope(q, None, cos, sin, torch.arange(T), 1e-6, False)
    close("q", out, want, mag, 32 * EPS, EPS)
    assert int(count) == 2 and bool(torch.isnan(out[5:]).all()) and not torch.isnan(out[:5]).any()
    dx = torch.empty_like(out)
    rr.rr_qk_norm_rope_bwd(torch.ones_like(out), None, q.cuda(), None, None, None, cos.cuda(),
                           sin.cuda(), None, dx, None)
    assert bool(torch.isnan(dx[5:]).all()) and not torch.isnan(dx[:5]).any()


# ---------------------------------------------------------------- attention ---

def check_attention(lens, H, KV, D, dtype, seed=0, first=0, tail=0, scale=None, gap=0, sigma=1.0,
                    poison=True, back=True):
    dt = DT[dtype]
    T = first + sum(lens) + tail
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    q, k, v, g = (rnd(seed + i, T, n, D).mul(sigma if i < 2 else 1.0).to(dt)
                  for i, n in enumerate((H, KV, KV, H)))
    out = torch.ones(T, dtype=torch.bool)
    for a, b in ref.spans(cu, T):
        out[a:b] = False
    if poison:  # rows of no sequence
        for t in (q, k, v, g):
            t[out] = math.nan
    bq, bk, bv = (buf(t, gap) for t in (q, k, v))
    bo = Buffer(T, (H, D), dt, gap, fill=7.0)
    lse = torch.full((H, T), 7.0, device="cuda")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    rr.rr_attention_packed_fwd(bq.view, bk.view, bv.view, cud, bo.view, lse=lse, scale=scale)
    want, wlse, mag, smag = ref.attention(q, k, v, cu, scale)
    inside = ~out
    fine = dtype == "f32" or D not in (64, 128)
    worst = float(torch.nan_to_num(smag).max())
    n = max(lens)
    rel = 4 * (D * worst + 16 + n) * EPS if fine else 2.0 ** -7
    close("o", bo.view[inside.cuda()], want[inside], mag[inside], rel, HALF[dt])
    close("lse", lse[:, inside.cuda()], wlse[:, inside], 1.0 + worst + wlse[:, inside].abs(),
          (D + 64) * EPS if fine else 1e-5)
    assert bool((bo.view[out.cuda()] == 7.0).all()) and bool((lse[:, out.cuda()] == 7.0).all())
    assert bo.untouched_around()
    if not back:
        return
    o = torch.nan_to_num(want).to(dt)
    bo.view.copy_(o)
    lse = torch.nan_to_num(wlse).float().cuda()
    bg = buf(g, gap)
    dq, dk, dv = (Buffer(T, (m, D), dt, gap, fill=7.0) for m in (H, KV, KV))
    rr.rr_attention_packed_bwd(bg.view, bq.view, bk.view, bv.view, bo.view, lse, cud, dq.view,
                               dk.view, dv.view, scale=scale)
    clean = [torch.where(out[:, None, None], torch.zeros((), dtype=dt), t) for t in (g, q, k, v)]
    (wq, wk, wv), (mq, mk, mv) = ref.attention_bwd(*clean, o, cu, scale)
    G = H // KV
    for name, b, w, m, terms in (("dq", dq, wq, mq, n), ("dk", dk, wk, mk, n * G),
                                 ("dv", dv, wv, mv, n * G)):
        # (S, dP and delta are sums of D terms each, rounded by EPS a term and exponential)
        rel = 8 * (D * (worst + 4) + 64 + terms) * EPS + HALF[dt] if fine else 2.0 ** -7
        close(name, b.view[inside.cuda()], w[inside], m[inside], rel, HALF[dt], floor=1e-6)
        assert bool((b.view[out.cuda()] == 7.0).all()), name
        assert b.untouched_around(), name


LENS = [[1], [2, 1], [0, 3, 0, 1], [64], [127, 128, 129], [255, 1, 257], [300, 0, 40, 513],
        [1, 1, 1, 1, 1, 31, 33]]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_attention_lengths(lens, D):
    check_attention(lens, 4, 2, D, "bf16", seed=sum(lens), first=3, tail=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,KV", [(1, 1), (2, 1), (3, 1), (6, 2), (8, 1), (5, 5), (16, 4)])
def test_attention_groups(H, KV, D):
    check_attention([200, 130, 1], H, KV, D, "bf16", seed=H, gap=D)


@pytest.mark.parametrize("dtype,D", [("f32", 4), ("f32", 64), ("f32", 128), ("f32", 256),
                                     ("bf16", 8), ("bf16", 80), ("bf16", 96), ("bf16", 256)])
@pytest.mark.parametrize("lens", [[1], [33, 0, 70], [130]])
def test_attention_other_dims(lens, dtype, D):
    check_attention(lens, 4, 2, D, dtype, seed=D, first=1, tail=2, gap=16)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_peaked_and_scaled(D):
    check_attention([400, 90], 2, 1, D, "bf16", sigma=3.0, back=False)
    check_attention([140], 2, 2, D, "bf16", scale=0.01)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_sequences(D):
    lens = [(7 * i) % 23 for i in range(700)]
    check_attention(lens, 2, 1, D, "bf16", seed=5)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_more_tiles_than_blocks(D):
    """Several tiles a block, of differing lengths: forward, dq and dk, dv."""
    check_attention([700, 333, 129, 257, 90, 1, 0, 128], 32, 32, D, "bf16", seed=7)
    check_attention([37 * i % 300 for i in range(140)], 4, 2, D, "bf16", seed=8)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_unseen_values_change_nothing(D):
    """NaN and infinities in the keys and values of later tokens, and of the sequences
    beside it, leave a token's output as it is."""
    T, H = 333, 2
    q, k, v = (rnd(i, T, H, D, dtype=torch.bfloat16).cuda() for i in range(3))
    cu = torch.tensor([0, 70, 333], dtype=torch.int32, device="cuda")
    outs = []
    for bad in (None, math.nan, math.inf, -math.inf):
        k2, v2 = k.clone(), v.clone()
        if bad is not None:
            k2[:70], v2[:70] = bad, bad
            k2[300:], v2[300:] = bad, bad
        o, lse = torch.empty_like(q), torch.empty(H, T, device="cuda")
        rr.rr_attention_packed_fwd(q, k2, v2, cu, o, lse=lse)
        outs.append((o[70:300].clone(), lse[:, 70:300].clone()))
    for o, lse in outs[1:]:
        assert torch.allclose(o.float(), outs[0][0].float(), atol=2e-2)
        assert torch.allclose(lse, outs[0][1], atol=1e-4)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_gradient_is_apart_from_other_sequences(D):
    T, H = 333, 2
    bf = torch.bfloat16
    q, k, v, g = (rnd(i, T, H, D, dtype=bf).cuda() for i in range(4))
    cu = torch.tensor([0, 70, 290, 333], dtype=torch.int32, device="cuda")
    got = []
    for bad in (None, math.nan, math.inf):
        t = [x.clone() for x in (q, k, v, g)]
        o, lse = torch.zeros_like(q), torch.zeros(H, T, device="cuda")
        rr.rr_attention_packed_fwd(*t[:3], cu, o, lse=lse)
        if bad is not None:
            for x in t + [o]:
                x[:70] = bad
                x[290:] = bad
            lse[:, :70] = bad
            lse[:, 290:] = bad
        d = [torch.empty_like(q) for _ in range(3)]
        rr.rr_attention_packed_bwd(t[3], *t[:3], o, lse, cu, *d)
        got.append([x[70:290].clone() for x in d])
    for d in got[1:]:
        for a, b in zip(d, got[0]):
            assert torch.equal(a, b)


def test_attention_bounds_outside_the_buffer():
    """Bounds beyond the tokens are taken as the nearest."""
    q = rnd(1, 50, 1, 64, dtype=torch.bfloat16).cuda()
    o, o2 = torch.empty_like(q), torch.empty_like(q)
    rr.rr_attention_packed_fwd(q, q, q, torch.tensor([-5, 20, 900], dtype=torch.int32,
                                                     device="cuda"), o)
    rr.rr_attention_packed_fwd(q, q, q, torch.tensor([0, 20, 50], dtype=torch.int32,
                                                     device="cuda"), o2)
    assert torch.equal(o, o2)


# -------------------------------------------------------- log probabilities ---

def logits(rows, cols, dtype, seed, hard=True):
    x = 3.0 * rnd(seed, rows, cols)
    if hard:
        g = torch.Generator().manual_seed(seed + 1)
        u = torch.rand(rows, cols, generator=g)
        x[u < 0.01] = -math.inf
        x[(u > 0.01) & (u < 0.012)] = 60.0
        for r in range(rows):
            if r % 11 == 5:
                x[r] = -math.inf
            elif r % 11 == 6:
                x[r, cols // 2] = math.nan
            elif r % 11 == 7:
                x[r, cols - 1] = math.inf
            elif r % 11 == 8:
                x[r] = 1.5                               # all alike
            elif r % 11 == 9:
                x[r, 3:] = -math.inf                     # three live columns
            elif r % 11 == 10:
                x[r] = torch.sort(x[r]).values
    return x.to(DT[dtype])


def check_logprob(rows, cols, dtype, k, T=1.0, seed=0, gap=0, pad=0, hard=True, inplace=False,
                  grads=(True, True)):
    x = logits(rows, cols, dtype, seed, hard)
    g = torch.Generator().manual_seed(seed + 2)
    tok = torch.randint(0, cols, (rows,), generator=g)
    n_bad = 0
    if hard and rows > 4:
        tok[1] = -100
        tok[3], tok[4] = cols, -7
        n_bad = 2
    want = ref.logprob(x, tok, T, k)
    bx = buf(x, gap, pad)
    f = {n: torch.full((rows,), math.nan, device="cuda")
         for n in ("logprob", "entropy", "row_max", "log_sum")}
    i32 = dict(dtype=torch.int32, device="cuda")
    rank, bad = torch.full((rows,), 77, **i32), torch.zeros(1, **i32)
    top = dict(top_index=torch.full((rows, k), 77, **i32),
               top_logprob=torch.full((rows, k), math.nan, device="cuda")) if k else {}
    td = tok.int().cuda()
    rr.rr_token_logprob_fwd(bx.view, td, rank=rank, bad_token_count=bad, temperature=T, **f, **top)
    assert torch.equal(rank.cpu().long(), want["rank"])
    assert int(bad) == n_bad
    for n in ("logprob", "log_sum"):
        close(n, f[n], want[n], want["lp"], 64 * EPS, EPS)
    close("entropy", f["entropy"], want["entropy"], want["ent"], 64 * EPS, EPS)
    close("row_max", f["row_max"], want["row_max"], 0.0, 0.0)
    if k:
        assert torch.equal(top["top_index"].cpu().long(), want["top_index"])
        close("top", top["top_logprob"], want["top_logprob"],
              want["lp"][:, None] + torch.nan_to_num(want["top_logprob"].abs(), posinf=0.0),
              64 * EPS, EPS)
    gl, gh = (rnd(seed + 3 + i, rows) if on else None for i, on in enumerate(grads))
    out = bx if inplace else Buffer(rows, (cols,), DT[dtype], gap, pad)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    rr.rr_token_logprob_bwd(bx.view, td, f["row_max"], f["log_sum"], dev(gl), out.view,
                            entropy=f["entropy"] if gh is not None else None,
                            grad_entropy=dev(gh), temperature=T)
    d, mag = ref.logprob_bwd(x, tok, gl, gh, T)
    # (rows with a NaN or an infinity: all NaN here, as the softmax is)
    close("dlogits", out.view, d, mag, 64 * EPS, HALF[DT[dtype]])
    assert out.untouched_around()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [1, 2, 7, 31, 97, 1000, 4097, 16385, 50304, 131075])
def test_logprob(cols, dtype):
    check_logprob(max(12, min(40, (1 << 19) // cols)), cols, dtype, min(20, 2 * cols),
                  T=0.8 if cols == 1000 else 1.0, seed=cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k", [0, 1, 2, 33, 128])
@pytest.mark.parametrize("cols", [100, 5003])
def test_logprob_lists(cols, k, dtype):
    check_logprob(23, cols, dtype, k, seed=k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gap,pad,inplace,grads", [
    (0, 1, False, (True, True)), (3, 0, True, (True, False)), (8, 0, False, (False, True)),
    (5, 3, True, (True, True))])
def test_logprob_layouts(gap, pad, inplace, grads, dtype):
    check_logprob(14, 1234, dtype, 5, gap=gap, pad=pad, inplace=inplace, grads=grads, seed=gap)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2.0 ** -120, 0.01, 3.0, 2.0 ** 120])
def test_logprob_temperatures(T, dtype):
    x = logits(12, 999, dtype, 3, hard=False)
    x[2, :40] = 3e38
    x[3, 5] = -3.3e38
    tok = x.float().argmax(1)
    lp, ent = (torch.empty(12, device="cuda") for _ in range(2))
    rr.rr_token_logprob_fwd(x.cuda(), tok.int().cuda(), lp, entropy=ent, temperature=T)
    want = ref.logprob(x, tok, T, 0)
    close("logprob", lp, want["logprob"], 1 + want["log_sum"], 64 * EPS, EPS)
    assert bool(torch.isfinite(ent).all())
    close("entropy", ent, want["entropy"], 1 + want["ent"], 256 * EPS, EPS)


@pytest.mark.parametrize("rows,cols,dtype,k,gap,pad", [
    (12, 33000, "bf16", 128, 0, 0), (200, 33001, "bf16", 20, 3, 1), (14, 40001, "f32", 5, 3, 1),
    (9, 270001, "f32", 33, 5, 3), (12, 270000, "bf16", 100, 0, 1), (13, 262144, "bf16", 0, 8, 0)])
def test_logprob_rows_over_several_blocks(rows, cols, dtype, k, gap, pad):
    check_logprob(rows, cols, dtype, k, T=0.9, seed=rows, gap=gap, pad=pad)


def test_logprob_more_rows_than_blocks():
    check_logprob(3001, 40, "bf16", 3, seed=9, hard=False)
    check_logprob(2501, 640, "f32", 2, seed=9, hard=False)


# ----------------------------------------------------------- used together ---

def pass_over(qkv, w, cos, sin, pos, cu, head, tok, H, KV):
    """One decoder attention block over packed sequences and the tokens' log probabilities."""
    T, D = qkv.shape[0], qkv.shape[2]
    dev = qkv.device
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    qr, kr = (torch.empty(T, n, D, dtype=qkv.dtype, device=dev) for n in (H, KV))
    rr.rr_qk_norm_rope_fwd(q, k, w[0], w[1], cos, sin, pos, qr, kr)
    o, lse = torch.zeros_like(qr), torch.zeros(H, T, device=dev)
    rr.rr_attention_packed_fwd(qr, kr, v, cu, o, lse=lse)
    x = (o.reshape(T, H * D).float() @ head).contiguous()
    s = {n: torch.empty(T, device=dev) for n in ("logprob", "entropy", "row_max", "log_sum")}
    rr.rr_token_logprob_fwd(x, tok, **s)
    return qr, kr, o, lse, x, s


def pass_back(qkv, w, cos, sin, pos, cu, head, tok, H, KV, saved, g, h):
    qr, kr, o, lse, x, s = saved
    T, D = qkv.shape[0], qkv.shape[2]
    dx = torch.empty_like(x)
    rr.rr_token_logprob_bwd(x, tok, s["row_max"], s["log_sum"], g, dx, entropy=s["entropy"],
                            grad_entropy=h)
    do = (dx @ head.T).reshape(T, H, D).to(qkv.dtype)
    d = torch.zeros_like(qkv)
    dqr, dkr = torch.zeros_like(qr), torch.zeros_like(kr)
    rr.rr_attention_packed_bwd(do, qr, kr, qkv[:, H + KV:], o, lse, cu, dqr, dkr, d[:, H + KV:])
    dw = [torch.empty_like(t) for t in w]
    rr.rr_qk_norm_rope_bwd(dqr, dkr, qkv[:, :H], qkv[:, H:H + KV], w[0], w[1], cos, sin, pos,
                           d[:, :H], d[:, H:H + KV], dw[0], dw[1])
    return d, dw


def make_pass(dtype, D, seed=0, H=4, KV=2, V=53):
    T = 90
    qkv = rnd(seed, T, H + 2 * KV, D, dtype=dtype).cuda()
    w = [(1 + 0.2 * rnd(seed + 1 + i, D)).to(dtype).cuda() for i in range(2)]
    cos, sin = (t.cuda() for t in ref.table(64, D))
    cu = torch.tensor([0, 40, 40, 41, 88], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(40), torch.arange(1), torch.arange(47), torch.tensor([-1, -1])])
    head = 0.2 * rnd(seed + 3, H * D, V).cuda()
    tok = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed)).int()
    tok[::9] = -100
    tok[88:] = -100
    return [qkv, w, cos, sin, pos.int().cuda(), cu, head, tok.cuda(), H, KV]


def autograd_pass(a, g, h):
    qkv, w, cos, sin, pos, cu, head, tok, H, KV = (
        t.double().cpu() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for t in a)
    w = [t.double().cpu() for t in w]
    leaves = [qkv.requires_grad_()] + [t.requires_grad_() for t in w]
    pos, cu, tok = pos.cpu(), cu.cpu().tolist(), tok.cpu().long()
    q, _ = ref.rope(qkv[:, :H], w[0], cos.float(), sin.float(), pos, 1e-6, False)
    k, _ = ref.rope(qkv[:, H:H + KV], w[1], cos.float(), sin.float(), pos, 1e-6, False)
    T, D = qkv.shape[0], qkv.shape[2]
    rows = []
    for s, e in ref.spans(cu, T):
        for hh in range(H):
            x = q[s:e, hh] @ k[s:e, hh * KV // H].T / math.sqrt(D)
            x = x.masked_fill(torch.ones(e - s, e - s).triu(1) > 0, -math.inf)
            rows.append((s, e, hh, torch.softmax(x, 1) @ qkv[s:e, H + KV + hh * KV // H]))
    o = torch.zeros(T, H, D, dtype=torch.float64)
    for s, e, hh, val in rows:
        o = o.index_put((torch.arange(s, e), torch.tensor(hh)), val)
    lp = torch.log_softmax(o.reshape(T, H * D) @ head, 1)
    live = tok >= 0
    ent = -(lp.exp() * lp).sum(1)
    got = lp[torch.arange(T), tok.clamp_min(0)]
    ((g * got + h * ent) * live).sum().backward()
    return got.detach() * live, [t.grad for t in leaves]


@pytest.mark.parametrize("dtype,D,tol", [(torch.float32, 32, 2e-5), (torch.bfloat16, 64, 4e-2)])
def test_the_operators_together(dtype, D, tol):
    """Rotation, attention and log probabilities of a packed batch, there and back, against
    autograd in float64 (relative 2-norm: float32 through six kernels; bf16: every tensor
    between them is rounded, 2^-9 each, some ten roundings deep)."""
    a = make_pass(dtype, D)
    T = a[0].shape[0]
    g, h = rnd(5, T), 0.3 * rnd(6, T)
    saved = pass_over(*a)
    d, dw = pass_back(*a, saved, g.cuda(), h.cuda())
    lp, grads = autograd_pass(a, g.double(), h.double())
    off = lambda x, y: float((x.double().cpu() - y).norm() / y.norm())  # noqa: E731
    assert off(saved[5]["logprob"], lp) < tol
    for x, y in zip([d] + dw, grads):
        assert off(x, y) < tol


def test_the_operators_in_a_graph_and_on_another_stream():
    a = make_pass(torch.bfloat16, 128, seed=3)
    T = a[0].shape[0]
    g, h = rnd(5, T).cuda(), rnd(6, T).cuda()
    want = pass_back(*a, pass_over(*a), g, h)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pass_back(*a, pass_over(*a), g, h)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and all(map(torch.equal, got[1], want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pass_back(*a, pass_over(*a), g, h)
    a[0].copy_(rnd(77, *a[0].shape, dtype=torch.bfloat16))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    new = pass_back(*a, pass_over(*a), g, h)
    assert torch.equal(got[0], new[0]) and all(map(torch.equal, got[1], new[1]))
    assert not torch.equal(new[0], want[0])
    assert rr.rr_read_device_error(0) == 0


def test_binding_refusals():
    q, o = (torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    f = rr.rr_attention_packed_fwd
    f(q, k, k, cu, o)
    for bad in (dict(q=q.float()), dict(k=k.cpu()), dict(o=o[:2]), dict(cu_seqlens=cu.long()),
                dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(v=k[..., :32])):
        with pytest.raises((ValueError, TypeError)):
            f(**(dict(q=q, k=k, v=k, cu_seqlens=cu, o=o) | bad))
    x, t, lp = torch.zeros(2, 9, device="cuda"), cu, torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        rr.rr_token_logprob_fwd(x, t, lp, top_index=torch.zeros(2, 3, dtype=torch.int32,
                                                                device="cuda"))
    with pytest.raises(rr.RRError):
        rr.rr_token_logprob_fwd(x, t, lp, temperature=0.0)


@pytest.mark.parametrize("index", [2 ** 31, -2 ** 31 - 1, 2 ** 32 - 100])
def test_binding_refuses_an_ignore_index_beyond_32_bits(index):
    x, t = torch.zeros(2, 9, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    f = [torch.zeros(2, device="cuda") for _ in range(3)]
    with pytest.raises(ValueError):
        rr.rr_token_logprob_fwd(x, t, f[0], ignore_index=index)
    with pytest.raises(ValueError):
        rr.rr_token_logprob_bwd(x, t, *f, x, ignore_index=index)
