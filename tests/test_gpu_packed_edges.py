"""The packed-sequence operators at the edges of what they accept: values that are not finite
where a token does not see them, long sequences, extreme magnitudes."""
import math

import pytest
import torch

import packed_ref as ref
import row_reduction_pass_gb300 as rr
from packed_ref import EPS, HALF

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def attend(q, k, v, cu, **kw):
    o, lse = torch.full_like(q, 7.0), torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    rr.rr_attention_packed_fwd(q, k, v, cu, o, lse=lse, **kw)
    return o, lse


# ---------------------------------------------------------------- attention ---

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_of_no_sequence_leave_the_same_bits(bad, D):
    """Whatever stands between, behind and in the sequences beside it: a sequence's rows come out
    the same to the bit, with lengths that end a tile early, at its end and a row after."""
    lens, H, KV = [70, 128, 129, 1, 255, 300], 4, 2
    T = 5 + sum(lens) + 40
    q, k, v = (rnd(i, T, n, D, dtype=BF).cuda() for i, n in enumerate((H, KV, KV)))
    ends = [5]
    for n in lens:
        ends.append(ends[-1] + n)
    want, wlse = attend(q, k, v, i32(ends))
    for b, n in enumerate(lens):
        mine = slice(ends[b], ends[b + 1])
        t = [x.clone() for x in (q, k, v)]
        for x in t:
            x[:mine.start] = bad
            x[mine.stop:] = bad
        o, lse = attend(*t, i32(ends))
        assert torch.equal(o[mine], want[mine]) and torch.equal(lse[:, mine], wlse[:, mine])
    assert rr.rr_read_device_error(0) == 0


def near(got, want, q, k, v, cu):
    """Two results with their own roundings, of the weights and of themselves (2^-8 each): 2^-6 of
    sum p |v|, which an attention over |v| gives to a few of these roundings."""
    mag = attend(q, k, v.abs(), cu)[0].float()
    return bool(((got.float() - want.float()).abs() <= 2.0 ** -6 * 1.05 * mag).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("first", [0, 130])
@pytest.mark.parametrize("at", [[0], [127], [128], [5, 6, 127, 200], [31, 32, 63, 64, 299], [40, 41]])
def test_single_values_reach_the_rows_and_columns_that_see_them(at, first, D):
    """A NaN or an infinity in one element of v: of the rows from its own on that column is NaN or
    infinite, and everything else is as with a zero in its place: to the bit, but in the rows of
    its tile before it."""
    T, H, KV = first + 301, 4, 2
    q, k, v = (rnd(i + 9, T, n, D, dtype=BF).cuda() for i, n in enumerate((H, KV, KV)))
    cu, bad = i32([0, first, T]), (math.inf, math.nan, -math.inf, math.inf)
    zeroed, add = v.clone(), torch.zeros(T, KV, D, device="cuda")
    same = torch.ones(T, dtype=torch.bool, device="cuda")
    for i, j in enumerate(at):
        same[first + j // 128 * 128:first + j] = False
        for kv in range(KV):
            c = 3 if at == [40, 41] else (17 * i + 5 * kv) % D  # (one column: inf, then -inf)
            f = (math.inf, -math.inf)[i] if at == [40, 41] else bad[(i + kv) % 4]
            v[first + j, kv, c], zeroed[first + j, kv, c] = f, 0.0
            add[first + j:, kv, c] += f
    base, wlse = attend(q, k, zeroed, cu)
    want = (base.float() + add.repeat_interleave(H // KV, 1)).to(BF)
    o, lse = attend(q, k, v, cu)
    assert torch.equal(lse, wlse) and not bool(torch.isfinite(want).all())
    assert torch.equal(torch.isnan(o), torch.isnan(want))
    assert torch.equal(torch.isinf(o), torch.isinf(want))
    assert torch.equal(torch.nan_to_num(o[same], nan=3.0), torch.nan_to_num(want[same], nan=3.0))
    fine = torch.isfinite(want)
    assert near(torch.where(fine, o, base), base, q, k, zeroed, cu)
    assert torch.equal(o[torch.isinf(want)], want[torch.isinf(want)])
    assert rr.rr_read_device_error(0) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_a_long_sequence_with_values_that_are_not_finite_beside_it(D):
    """Sequences of 100 001 tokens and fewer: NaN behind the last, at the long one's end, early and
    late in it change neither the others nor the rows before, and no wait runs out."""
    lens, H = [90, 100001, 513], 2
    T = sum(lens) + 100
    q, k, v = (rnd(i, T, n, D, dtype=BF).cuda() for i, n in enumerate((H, 1, 1)))
    ends = [0, 90, 90 + 100001, sum(lens)]
    cu = i32(ends)
    want, wlse = attend(q, k, v, cu)
    for row in (ends[2] - 1, ends[1] + 50, ends[1] + 60000):
        bad = v.clone()
        bad[row] = math.nan
        bad[ends[3]:] = math.nan
        o, lse = attend(q, k, bad, cu)
        assert rr.rr_read_device_error(0) == 0
        kept = torch.ones(T, dtype=torch.bool, device="cuda")
        kept[row:ends[2]] = False
        assert torch.equal(lse, wlse) and bool(torch.isnan(o[~kept]).all())
        o[~kept] = want[~kept]
        assert near(o, want, q, k, v, cu)
        kept[ends[1] + (row - ends[1]) // 128 * 128:row] = False  # (that tile's rows before it)
        assert torch.equal(o[kept], want[kept])
    bad = torch.full_like(v, math.nan)
    o, _ = attend(q, k, bad, cu)
    assert rr.rr_read_device_error(0) == 0 and bool(torch.isnan(o[:ends[3]]).all())


@pytest.mark.parametrize("D", [64, 128])
def test_more_tiles_a_block_than_have_a_bit_of_their_own(D):
    """Sequences of one tile, some thousands for each block, every seventh with a NaN in it."""
    n, H = 128, 4 * 160
    T = 1100 * n
    q, k, v = (rnd(i, T, 1, D, dtype=BF).cuda() for i in range(3))
    q = q.expand(T, H, D).contiguous()
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    want = torch.empty_like(q)
    rr.rr_attention_packed_fwd(q, k, v, cu, want)
    bad = v.clone()
    bad[100::7 * n] = math.nan
    o = torch.empty_like(q)
    rr.rr_attention_packed_fwd(q, k, bad, cu, o)
    same = torch.ones(T, dtype=torch.bool, device="cuda")
    for b in range(0, 1100, 7):
        same[b * n:(b + 1) * n] = False
        assert bool(torch.isnan(o[b * n + 100:(b + 1) * n]).all())
        assert float((o[b * n:b * n + 100] - want[b * n:b * n + 100]).float().abs().max()) < 0.05
    assert torch.equal(o[same], want[same]) and rr.rr_read_device_error(0) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_great_values(D):
    """200 values of 2^120, whose sum still is a float32, under scores that rise by 7 powers of
    two from the first tile to the second: the result is 2^120 (within its rounding and the
    weights', 2^-8 each)."""
    T = 200
    q = torch.zeros(T, 1, D, dtype=BF, device="cuda")
    q[..., 0] = 1.0
    k = torch.zeros_like(q)
    k[128:, 0, 0] = 7.0 * math.log(2.0)
    v = torch.full_like(q, 2.0 ** 120)
    o, _ = attend(q, k, v, i32([0, T]), scale=1.0)
    assert float(((o.double() / 2.0 ** 120) - 1.0).abs().max()) <= 2.0 ** -7


@pytest.mark.parametrize("D", [64, 128])
def test_rows_before_a_nan_against_the_plain_form(D):
    """Weights and the result are rounded to bf16 (2^-8 each): 2^-7 of sum p |v|."""
    T, H, KV = 333, 4, 2
    q, k, v = (rnd(i, T, n, D, dtype=BF) for i, n in enumerate((H, KV, KV)))
    cu = [0, 70, 333]
    want, wlse, mag, _ = ref.attention(q, k, v, cu, 1.0 / math.sqrt(D))
    v[300] = math.nan
    v[310:, :, 7] = math.inf
    o, lse = attend(q.cuda(), k.cuda(), v.cuda(), i32(cu))
    off = (o.double().cpu() - want).abs() - 2.0 ** -7 * mag
    assert float(off[:300].max()) <= 0.0
    assert float((lse.double().cpu() - wlse).abs().max()) <= 1e-5 * (1.0 + float(wlse.abs().max()))

def gradients_with_exact_delta(q, k, v, g, o, G, scale):
    """dq and dk of one sequence in float64, the bounds of their errors when delta is the weights'
    sum, and the gradients that delta = dout . o with the rounded o would give.  Relative error
    of a weight: a score of D products, lse, an exponential.  ds: that, dout . v and delta's sum of
    such products, and its own rounding to bf16 (2^-8, as the result's).  Beside a row whose
    one great weight all but cancels in dout . v - delta, o's rounding stands far above these."""
    D, n = q.shape[2], q.shape[0]
    q, k, v, g, o = (t.double() for t in (q, k, v, g, o))
    zero = [torch.zeros_like(q), torch.zeros_like(k)]
    out = [[t.clone() for t in zero] for _ in range(3)]
    hide = torch.ones(n, n, dtype=torch.bool).triu(1)
    for h in range(q.shape[1]):
        kv = h // G
        s = scale * (q[:, h] @ k[:, kv].T)
        lse = torch.logsumexp(s.masked_fill(hide, -math.inf), 1, keepdim=True)
        p = torch.exp(s - lse).masked_fill(hide, 0.0)
        dp, gm = g[:, h] @ v[:, kv].T, g[:, h].abs() @ v[:, kv].abs().T
        delta = (p * dp).sum(1, keepdim=True)
        rel = EPS * (D * scale * (q[:, h].abs() @ k[:, kv].abs().T) + lse.abs() + 16)
        ds = p * (dp - delta)
        e_delta = (p * (D * EPS * gm + dp.abs() * (rel + n * EPS))).sum(1, keepdim=True)
        e_ds = p * (D * EPS * gm + e_delta + (dp - delta).abs() * rel) + (2.0 ** -8 + n * EPS) * ds.abs()
        rounded = p * (dp - (g[:, h] * o[:, h]).sum(1, keepdim=True))
        for to, x, kk, qq in ((out[0], ds, k, q), (out[1], e_ds, k.abs(), q.abs()),
                              (out[2], rounded, k, q)):
            to[0][:, h] = scale * (x @ kk[:, kv])
            to[1][:, kv] += scale * (x.T @ qq[:, h])
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[37], [128], [3, 100, 0, 127]])
def test_gradients_of_first_rows_take_delta_from_the_weights(lens, D):
    H, KV, T = 4, 2, sum(lens)
    scale = 1.0 / math.sqrt(D)
    q, k, v, g = (rnd(i + 20, T, n, D).mul(3.0 if i < 2 else 1.0).to(BF)
                  for i, n in enumerate((H, KV, KV, H)))
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    want, wlse, _, _ = ref.attention(q, k, v, ends, scale)
    o = want.to(BF)
    dq, dk, dv = (torch.empty(T, n, D, dtype=BF, device="cuda") for n in (H, KV, KV))
    rr.rr_attention_packed_bwd(g.cuda(), q.cuda(), k.cuda(), v.cuda(), o.cuda(),
                               wlse.float().cuda(), i32(ends), dq, dk, dv)
    seen = [False, False]
    for a, b in ref.spans(ends, T):
        exact, bound, rounded = gradients_with_exact_delta(q[a:b], k[a:b], v[a:b], g[a:b], o[a:b],
                                                           H // KV, scale)
        for i, got in enumerate((dq, dk)):
            most = bound[i] + 2.0 ** -8 * exact[i].abs() + 1e-30
            assert float(((got[a:b].double().cpu() - exact[i]).abs() / most).max()) <= 1.0
            seen[i] |= bool(((rounded[i] - exact[i]).abs() > 2.0 * most).any())
    assert seen == [True, True]  # o's rounding would show in either


# -------------------------------------------------------- log probabilities ---

@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("T", [2.0 ** -120, 2.0 ** -60, 0.01, 2.0 ** 60, 2.0 ** 120])
def test_logprob_gradient_at_extreme_temperatures(T, dtype):
    """Gradients of log probability and entropy, masked columns (-infinity, the type's lowest, a
    finite -1e9) among them.  At a low temperature a column below the maximum has probability 0
    and gets 0; a row of two equal maxima has 1/2 for both.  The plain form in float64, within
    64 EPS of its magnitudes and the result's rounding, as at other temperatures.  A result below
    2^-126 may be 0, and so may a probability, whose factor is at most h 126 ln 2 < 2^9, over T."""
    rows, cols = 12, 999
    x = 3.0 * rnd(3, rows, cols).to(dtype)
    x[1, :40], x[2, :40], x[3, :40] = -math.inf, torch.finfo(dtype).min, -1e9
    x[4, 7] = x[4, 700] = 50.0
    x[5] = 1.5
    tok = x.float().argmax(1)
    tok[6:9] = torch.tensor([3, 400, -100])
    g, h = 0.5 + rnd(4, rows).abs(), rnd(5, rows)
    f = {n: torch.empty(rows, device="cuda") for n in ("logprob", "entropy", "row_max", "log_sum")}
    xd, td = x.cuda(), tok.int().cuda()
    rr.rr_token_logprob_fwd(xd, td, temperature=T, **f)
    for gl, gh in ((g, h), (None, h), (g, None)):
        d = torch.empty_like(xd)
        rr.rr_token_logprob_bwd(xd, td, f["row_max"], f["log_sum"],
                                None if gl is None else gl.cuda(), d,
                                entropy=None if gh is None else f["entropy"],
                                grad_entropy=None if gh is None else gh.cuda(), temperature=T)
        want, mag = ref.logprob_bwd(x, tok, gl, gh, T)
        # (a token's own term cancels with its probability: both carry the logarithms' error)
        close = (d.double().cpu() - want).abs() <= (64 * EPS * mag + HALF[dtype] * want.abs()
                                                    + 2.0 ** -126 + 2.0 ** -117 / T)
        assert bool(close.all()), (int((~close).sum()), d.cpu()[~close][:4], want[~close][:4])


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("pad", [0, 1])
def test_logprob_gradient_of_tokens_out_of_range_adds_nothing_anywhere(pad, dtype):
    """Tokens just below 0 and from the row's end on, with ragged rows and an output that starts at
    another alignment: only the probabilities' part."""
    rows, cols = 8, 133
    x = rnd(6, rows, cols).to(dtype)
    tok = torch.tensor([-1, -2, -3, -2 ** 31, cols, cols + 1, 2 ** 31 - 1, 132])
    g, h = rnd(7, rows), rnd(8, rows)
    f = {n: torch.empty(rows, device="cuda") for n in ("logprob", "entropy", "row_max", "log_sum")}
    xd, td = x.cuda(), tok.int().cuda()
    rr.rr_token_logprob_fwd(xd, td, **f)
    d = torch.empty(pad + rows * cols, dtype=dtype, device="cuda")[pad:].view(rows, cols)
    rr.rr_token_logprob_bwd(xd, td, f["row_max"], f["log_sum"], g.cuda(), d, entropy=f["entropy"],
                            grad_entropy=h.cuda())
    want, mag = ref.logprob_bwd(x, tok, g, h, 1.0)
    assert bool(((d.double().cpu() - want).abs() <= 64 * EPS * mag + HALF[dtype] * want.abs()
                 + 1e-30).all())


# --------------------------------------------------- batches padded with empty ones ---

def padded(lens, place, empty):
    """`empty` sequences of no tokens among `lens`: before, between or behind them."""
    if place == "behind":
        return lens + [0] * empty
    if place == "before":
        return [0] * empty + lens
    each = empty // len(lens)
    return sum(([n] + [0] * each for n in lens), [])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("place", ["behind", "before", "between"])
@pytest.mark.parametrize("live,empty", [(1, 128), (7, 3000), (128, 1280), (129, 1290), (200, 20000),
                                        (3, 30000)])
def test_empty_sequences_change_nothing(live, empty, place, D):
    """Any number of empty sequences anywhere: the same bits."""
    lens = [1 + (37 * i + 11 * live) % 290 for i in range(live)]
    T, H, KV = sum(lens), 4, 2
    q, k, v, g = (rnd(i, T, n, D, dtype=BF).cuda() for i, n in enumerate((H, KV, KV, H)))
    got = []
    for pad in (lens, padded(lens, place, empty)):
        cu = torch.zeros(len(pad) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(pad).cumsum(0)
        o, lse = attend(q, k, v, cu.cuda())
        d = [torch.full_like(x, 7.0) for x in (q, k, v)]
        rr.rr_attention_packed_bwd(g, q, k, v, o, lse, cu.cuda(), *d)
        got.append([o, lse] + d)
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert rr.rr_read_device_error(0) == 0


def test_nothing_but_empty_sequences():
    q = torch.zeros(5, 2, 64, dtype=BF, device="cuda")
    for batch in (1, 128, 129, 400, 20000):
        o, lse = attend(q, q, q, torch.full((batch + 1,), 3, dtype=torch.int32, device="cuda"))
        d = [torch.full_like(q, 7.0) for _ in range(3)]
        rr.rr_attention_packed_bwd(q, q, q, q, o, lse,
                                   torch.full((batch + 1,), 5, dtype=torch.int32, device="cuda"), *d)
        assert bool((o == 7.0).all()) and bool((lse == 7.0).all())
        assert all(bool((x == 7.0).all()) for x in d)
    assert rr.rr_read_device_error(0) == 0


@pytest.mark.parametrize("batch", [100, 300])
def test_decreasing_bounds_end_and_stay_inside(batch):
    """Results are not specified, but the calls end, and nothing around the tensors is written."""
    g = torch.Generator().manual_seed(batch)
    T, H = 500, 2
    cu = torch.randint(-20, 600, (batch + 1,), generator=g).int().cuda()
    raw = [torch.full((T + 200, H, 64), 7.0, dtype=BF, device="cuda") for _ in range(5)]
    q, o, dq, dk, dv = (t[100:100 + T] for t in raw)
    q.copy_(rnd(1, T, H, 64, dtype=BF))
    lse = torch.zeros(H, T, device="cuda")
    rr.rr_attention_packed_fwd(q, q, q, cu, o, lse=lse)
    rr.rr_attention_packed_bwd(q, q, q, q, o, lse, cu, dq, dk, dv)
    torch.cuda.synchronize()
    for t in raw:
        assert bool((t[:100] == 7.0).all()) and bool((t[100 + T:] == 7.0).all())
    assert rr.rr_read_device_error(0) == 0
