"""GPU parity of the draft model's operators (rr_distill_fwd_bwd,
rr_attention_tree_fwd, rr_draft_verify) with their float64 plain forms.

Tolerances, from the arithmetic (EPS = 2^-24, half a float32 step):
  distillation: an exponential 2^((x - m) c) carries (|x - m| / T + 2) steps (the
    argument's rounding, and ex2.approx's 2^-22), a sum over a row some tens of
    steps, a teacher weight |ln t| steps.  The plain form returns the sum of the
    magnitudes these are relative to; 64 EPS times it is allowed, plus half a step of
    the storage type (bf16 2^-8 |dlogits|, fp32 2^-23), plus 1e-30 for results
    flushed below the smallest normal float32.
  attention: products of bf16 are exact in fp32; weights p_j are rounded to bf16
    (2^-9) before P V and o to bf16 (2^-9 |o|): |o_gpu - o| <= 2^-8 sum p |v|, twice
    that is allowed; lse 1e-5 + 1e-5 relative.
  verification: whole numbers, equal.  A sequence one of whose decisions lies within
    1e-5 (relative) of the other answer is left out, since fp32 probabilities (sums
    over the row: some tens of EPS, 4e-6) may fall on either side.
"""
import numpy as np
import pytest
import torch

import draft_ref as ref
import row_reduction_pass_gb300 as rr

from parity import check_guards, compare, empty_like_dev, host, store, to_dev, zeros_i32

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- distillation ---

def distill_inputs(rows, cols, k, dtype, seed, tail, T, hard=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * 3.0
    if hard:
        x[rng.random((rows, cols)) < 0.01] = 1e4
        x[rng.random((rows, cols)) < 0.01] = -1e4
        x[rng.random((rows, cols)) < 0.01] = -np.inf
        x[5::17] = -np.inf                                   # fully masked rows
    xs = store(x, dtype)
    index = np.full((rows, k), -1, np.int32)
    value = np.zeros((rows, k), np.float32)
    for r in range(rows):
        kk = min(k, cols)
        index[r, :kk] = rng.choice(cols, kk, replace=False)
        z = rng.standard_normal(k) * 2.0
        value[r] = z - np.log(np.exp(z).sum()) + np.log(rng.uniform(0.3, 0.999)) if tail else z
        if hard and k > 0:
            n = rng.integers(0, k + 1)
            index[r, n:] = -1                                # a shorter list
            if k > 2 and r % 3 == 0:
                index[r, 1] = index[r, 0]                    # listed twice
            if r % 5 == 1:
                index[r, rng.integers(0, k)] = cols + 7      # out of range
            if r % 7 == 2:
                value[r, rng.integers(0, k)] = -np.inf
    return xs, index, value, rng.uniform(0.0, 2.0, rows).astype(np.float32)


def check_distill(rows, cols, k, dtype, tail, T, seed, pads=(0, 0), inplace=False, grad=True,
                  hard=True, loss_only=False):
    x, index, value, g = distill_inputs(rows, cols, k, dtype, seed, tail, T, hard)
    xd = to_dev(x, pads[0])
    dl = None if loss_only else xd if inplace else empty_like_dev(x.shape, dtype, pads[1])
    loss, bad = empty_like_dev((rows,), "f32"), zeros_i32(1)
    rr.rr_distill_fwd_bwd(xd, to_dev(index).view(rows, k), to_dev(value).view(rows, k), loss, dl,
                          grad=to_dev(g) if grad else None, temperature=T, tail=tail,
                          bad_index_count=bad)
    torch.cuda.synchronize()
    check_guards()
    rl, rd, lm, dm = ref.distill(x, index, value, g if grad else None, T, tail)
    compare("distill loss", host(loss), rl, 0.0, 1e-30, scale=lm, scale_rtol=64 * ref.EPS)
    if dl is not None:
        compare("distill dlogits", host(dl), rd, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23,
                1e-30, scale=dm, scale_rtol=64 * ref.EPS)
    assert int(bad.item()) == int((index >= cols).sum())


COLS = [1, 2, 31, 97, 1000, 4097, 16385, 50304, 65537, 131075]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("cols", COLS)
def test_distill(cols, tail, dtype):
    rows = int(max(3, min(300, (1 << 21) // cols)))
    check_distill(rows, cols, min(24, 2 * cols), dtype, tail, 2.0, 10 + cols)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("k", [0, 1, 2, 33, 300, 1024])
def test_distill_list_lengths(k, tail, dtype):
    check_distill(40, 5003, k, dtype, tail, 1.0, 100 + k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5, 1000, 4097, 50304])
@pytest.mark.parametrize("layout", ["inplace", "misaligned", "inplace_misaligned", "mixed",
                                    "loss_only"])
def test_distill_layouts(cols, layout, dtype):
    pads = {"misaligned": (1, 1), "inplace_misaligned": (1, 1), "mixed": (1, 0)}.get(layout, (0, 0))
    check_distill(37, cols, 8, dtype, cols == 1000, 1.5, 7 + cols, pads,
                  inplace=layout.startswith("inplace"), loss_only=layout == "loss_only",
                  grad=layout != "mixed")


def test_distill_every_column_listed_and_more_rows_than_blocks():
    check_distill(5000, 16, 16, "f32", True, 1.0, 4, hard=False)
    check_distill(5000, 16, 16, "f32", False, 3.0, 5, hard=False)


def test_distill_student_sure_of_the_list():
    """The unlisted columns hold 1e-9 of the student's mass: the tail's gradient
    keeps its digits (it is not the difference of two sums)."""
    rows, cols = 16, 3000
    rng = np.random.default_rng(1)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x[:, 17] = 30.0
    index, value = np.full((rows, 1), 17, np.int32), np.full((rows, 1), np.log(0.9), np.float32)
    xd, loss, dl = to_dev(x), empty_like_dev((rows,), "f32"), empty_like_dev(x.shape, "f32")
    rr.rr_distill_fwd_bwd(xd, to_dev(index).view(rows, 1), to_dev(value).view(rows, 1), loss, dl,
                          tail=True)
    rl, rd, lm, dm = ref.distill(x, index, value, tail=True)
    compare("loss", host(loss), rl, 0.0, 0.0, scale=lm, scale_rtol=64 * ref.EPS)
    compare("dlogits", host(dl), rd, 2.0 ** -23, 1e-30, scale=dm, scale_rtol=64 * ref.EPS)


@pytest.mark.parametrize("dtype,cols", [("bf16", 9733), ("bf16", 59183), ("f32", 19467),
                                        ("f32", 40971), ("bf16", 118347)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_rows_whose_last_chunk_moves(cols, tail, dtype):
    """Rows that end in one chunk or the next, by where they begin, so that its thread
    changes from row to row: right at every run, and the same bits."""
    rows = 700 if cols < 50000 else 200
    x, index, value, g = distill_inputs(rows, cols, 9, dtype, cols, tail, 2.0, hard=False)
    xd, idx, val, gd = to_dev(x), to_dev(index).view(rows, 9), to_dev(value).view(rows, 9), to_dev(g)
    outs = []
    for _ in range(8):
        loss, dl = empty_like_dev((rows,), "f32"), empty_like_dev(x.shape, dtype)
        rr.rr_distill_fwd_bwd(xd, idx, val, loss, dl, grad=gd, temperature=2.0, tail=tail)
        outs.append((loss, dl))
    torch.cuda.synchronize()
    check_guards()
    for loss, dl in outs[1:]:
        assert torch.equal(loss, outs[0][0]) and torch.equal(dl, outs[0][1])
    rl, rd, lm, dm = ref.distill(x, index, value, g, 2.0, tail)
    compare("distill loss", host(outs[0][0]), rl, 0.0, 1e-30, scale=lm, scale_rtol=64 * ref.EPS)
    compare("distill dlogits", host(outs[0][1]), rd, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23,
            1e-30, scale=dm, scale_rtol=64 * ref.EPS)


@pytest.mark.parametrize("dtype,cols,k", [("f32", 50304, 1024), ("bf16", 50304, 1024),
                                          ("f32", 207000, 300), ("f32", 262147, 1024),
                                          ("bf16", 420001, 7)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_long_rows_and_lists(cols, k, tail, dtype):
    """Long lists beside long rows; the longest rows a cluster holds, and longer ones."""
    check_distill(5, cols, k, dtype, tail, 2.0, k + cols)


# ---------------------------------------------------------------- attention ---

def tree_inputs(B, n, H, KV, D, lens, ps, seed, tree, spare=2):
    rng = np.random.default_rng(seed)
    need = [(max(L, 0) + n + ps - 1) // ps for L in lens]
    pages, width = sum(need) + spare, max(need + [1])
    q = store(rng.standard_normal((B, n, H, D)), "bf16")
    kc = store(rng.standard_normal((pages, ps, KV, D)), "bf16")
    vc = store(rng.standard_normal((pages, ps, KV, D)), "bf16")
    order = rng.permutation(pages)
    table = np.full((B, width), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    par = None
    if tree:
        par = np.array([[rng.integers(-1, i) if i else -1 for i in range(n)] for _ in range(B)],
                       np.int32)
    return q, kc, vc, table, np.array(lens, np.int32), par


def run_tree(q, kc, vc, table, ctx, par, lse=True):
    B, n, H, D = q.shape
    o = empty_like_dev((B, n, H, D), "bf16")
    l = empty_like_dev((B, n, H), "f32") if lse else None
    rr.rr_attention_tree_fwd(to_dev(q), to_dev(kc), to_dev(vc), to_dev(table).view(table.shape),
                             to_dev(ctx), o, lse=l,
                             parents=None if par is None else to_dev(par).view(par.shape))
    torch.cuda.synchronize()
    check_guards()
    assert rr.rr_read_device_error(0) == 0
    return o, l


def check_tree(q, kc, vc, table, ctx, par, scale=None):
    o, l = run_tree(q, kc, vc, table, ctx, par)
    ro, rl, mag = ref.tree_attention(q, kc, vc, table, ctx, par)
    compare("tree attention lse", host(l), rl, 1e-5, 1e-5)
    compare("tree attention o", host(o), ro, 0.0, 1e-6, scale=mag, scale_rtol=2.0 ** -7)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [1, 5, 16, 48, 64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_tree_attention_pages(D, ps, tree):
    check_tree(*tree_inputs(3, 7, 4, 2, D, [0, 130, 517], ps, ps + D, tree))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,H,KV", [(1, 1, 1), (1, 8, 1), (1, 32, 8), (5, 7, 1), (17, 6, 2),
                                    (33, 16, 4), (64, 8, 1), (130, 3, 1), (256, 2, 1)])
@pytest.mark.parametrize("tree", [False, True])
def test_tree_attention_heads(D, n, H, KV, tree):
    check_tree(*tree_inputs(2, n, H, KV, D, [63, 300], 16, n + H + D, tree))


@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention_lengths(D):
    """Contexts around every tile border, in one ragged batch."""
    lens = [0, 1, 15, 16, 17, 62, 63, 64, 65, 126, 127, 128, 129, 191, 255, 256, 257, 600]
    check_tree(*tree_inputs(len(lens), 3, 4, 2, D, lens, 16, D, True))
    check_tree(*tree_inputs(len(lens), 1, 4, 4, D, lens, 32, D + 1, False))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch,ctx", [(1, 6000), (3, 9001), (17, 900), (70, 200), (320, 60),
                                       (321, 60), (700, 33)])
def test_tree_attention_split_sequences(D, batch, ctx):
    """Long contexts shared between many blocks, and more sequences than blocks."""
    lens = [max(0, ctx - 13 * b) for b in range(batch)]
    check_tree(*tree_inputs(batch, 2, 2, 1, D, lens, 64, ctx + D, True))


@pytest.mark.parametrize("D,ps", [(128, 64), (64, 128)])
def test_tree_attention_many_sequences_a_block(D, ps):
    """Enough cache that memory is the bound, and sequences short enough that a
    block works through several of them, each with the rest of a page behind its end:
    six runs give the same bits and the float64 attention."""
    B, H, KV = 64, 32, 8
    g = torch.Generator("cuda").manual_seed(4)
    lens = [500 + int(3500 * ((b * 0.618034) % 1.0)) for b in range(B)]
    need = [(L + 1 + ps - 1) // ps for L in lens]
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(need), generator=g, device="cuda").int()
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, kc, vc = rnd(B, 1, H, D), rnd(at, ps, KV, D), rnd(at, ps, KV, D)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    runs = []
    for _ in range(6):
        o, l = torch.full_like(q, 7.0), torch.empty(B, 1, H, device="cuda")
        rr.rr_attention_tree_fwd(q, kc, vc, table, ctx, o, lse=l)
        runs.append((o, l))
    torch.cuda.synchronize()
    assert rr.rr_read_device_error(0) == 0
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])
    for b in range(B):
        pages = table[b, :need[b]].long()
        k = kc[pages].reshape(-1, KV, D)[:lens[b] + 1].double().repeat_interleave(H // KV, 1)
        v = vc[pages].reshape(-1, KV, D)[:lens[b] + 1].double().repeat_interleave(H // KV, 1)
        s = torch.einsum("hd,lhd->hl", q[b, 0].double(), k) / D ** 0.5
        p = torch.softmax(s, 1)
        compare("lse", host(runs[0][1][b, 0]), torch.logsumexp(s, 1).cpu().numpy(), 1e-5, 1e-5)
        compare("o", host(runs[0][0][b, 0]), torch.einsum("hl,lhd->hd", p, v).cpu().numpy(), 0.0,
                1e-6, scale=torch.einsum("hl,lhd->hd", p, v.abs()).cpu().numpy(),
                scale_rtol=2.0 ** -7)


def test_tree_attention_long_chain():
    """A prompt chunk: 600 new tokens, several tiles of query rows."""
    check_tree(*tree_inputs(2, 600, 2, 1, 64, [0, 77], 16, 3, False))


@pytest.mark.parametrize("ps", [5, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention_absent_nodes_and_bad_pages(ps, D):
    q, kc, vc, table, ctx, par = tree_inputs(4, 6, 4, 2, D, [0, 40, 100, -5], ps, 31 + ps, True)
    par[0, 2] = -2          # absent, and with it every node below
    par[0, 4] = 2
    par[1] = -2             # a sequence without nodes
    par[2, 3] = 3           # its own parent
    table[1, 1] = -1        # pages that do not exist
    table[2, 2] = kc.shape[0]
    table[2, 0] = 2 ** 31 - 1
    check_tree(q, kc, vc, table, ctx, par)
    o, l = run_tree(q, kc, vc, table, ctx, par)
    assert (host(o)[1] == 0).all() and np.isneginf(host(l)[1]).all()


@pytest.mark.parametrize("ps", [5, 16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_tree_attention_unseen_values_do_not_matter(ps, D, bad):
    """NaN and infinities in the rest of the last page, in unused pages, at
    absent nodes and at nodes that other nodes do not see."""
    lens = [0, 30, 125]
    q, kc, vc, table, ctx, par = tree_inputs(3, 9, 4, 2, D, lens, ps, 77 + ps, True)
    par[:, 1:3] = -1
    par[:, 3:] = np.array([1, 1, 2, 2, 5, 0])
    par[2, 8] = -3
    bits = store(np.array([bad]), "bf16")[0]
    used = np.zeros(kc.shape[:2], bool)
    for b, L in enumerate(lens):
        for p in range(L + 9):
            used[table[b, p // ps], p % ps] = True
    kc2, vc2 = kc.copy(), vc.copy()
    kc2[~used] = bits
    vc2[~used] = bits
    p8 = 125 + 8                                    # the absent node of sequence 2
    kc2[table[2, p8 // ps], p8 % ps] = bits
    vc2[table[2, p8 // ps], p8 % ps] = bits
    check_tree(q, kc, vc, table, ctx, par)
    a, b = run_tree(q, kc, vc, table, ctx, par), run_tree(q, kc2, vc2, table, ctx, par)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # node 2 of sequence 1 is seen by nodes 2, 5, 6 and 7 only
    p2 = 30 + 2
    vc2[table[1, p2 // ps], p2 % ps, :, 3] = bits
    c = run_tree(q, kc2, vc2, table, ctx, par)
    assert torch.equal(a[1], c[1])
    hit = np.zeros(a[0].shape, bool)
    hit[1, [2, 5, 6, 7], :, 3] = True
    ca, cc = host(a[0]), host(c[0])
    assert (ca[~hit] == cc[~hit]).all()
    assert (~np.isfinite(cc[hit])).all()


def test_tree_attention_no_table_and_no_pages():
    q = torch.randn(2, 3, 4, 64, device="cuda").bfloat16()
    kc = torch.empty(0, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    for table in (torch.empty(2, 0, dtype=torch.int32, device="cuda"),
                  torch.zeros(2, 4, dtype=torch.int32, device="cuda")):
        o, l = torch.full_like(q, 7.0), torch.zeros(2, 3, 4, device="cuda")
        ctx = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
        rr.rr_attention_tree_fwd(q, kc, kc, table, ctx, o, lse=l)
        torch.cuda.synchronize()
        assert (o == 0).all() and torch.isneginf(l).all()


@pytest.mark.parametrize("ps", [5, 16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_tree_attention_positions_beyond_the_table(ps, D, tree):
    """Contexts and nodes that the table does not cover, up to the largest length."""
    q, kc, vc, table, _, par = tree_inputs(4, 5, 4, 2, D, [300, 300, 300, 300], ps, ps + D, tree)
    table = np.ascontiguousarray(table[:, :128 // ps])
    edge = table.shape[1] * ps
    check_tree(q, kc, vc, table, np.array([edge - 3, edge, edge + 40, 2 ** 31 - 1], np.int32), par)


def test_tree_attention_sequences_share_pages():
    """One table row for all (a common prefix): page indexes that stand many times."""
    q, kc, vc, table, ctx, par = tree_inputs(3, 4, 8, 2, 128, [200, 200, 200], 16, 5, True)
    table[:] = table[0]
    table[:, 2] = table[:, 1]
    check_tree(q, kc, vc, table, ctx, par)


def test_tree_attention_odd_values_at_nodes_of_many_pieces():
    """Infinities in V at nodes that all of a sequence's rows see, of several row tiles
    and heads, in a batch where pipelines go on to other sequences: those rows and
    columns become infinite, all others stay as they are."""
    B, n, H, KV, D, ps = 40, 33, 32, 4, 64, 16
    lens = [100 + 37 * b for b in range(B)]
    q, kc, vc, table, ctx, par = tree_inputs(B, n, H, KV, D, lens, ps, 8, True)
    par[:, 1:] = np.maximum(par[:, 1:], 0)          # all below node 0
    a = run_tree(q, kc, vc, table, ctx, par)
    hit = np.zeros(a[0].shape, bool)
    inf = store(np.array([np.inf]), "bf16")[0]
    for b in range(0, B, 3):
        h, c = b % KV, 7 * b % D
        vc[table[b, lens[b] // ps], lens[b] % ps, h, c] = inf
        hit[b, :, h * (H // KV):(h + 1) * (H // KV), c] = True
    for _ in range(3):
        o, l = run_tree(q, kc, vc, table, ctx, par)
        assert torch.equal(l, a[1])
        assert (host(o)[~hit] == host(a[0])[~hit]).all()
        assert np.isposinf(host(o)[hit]).all()


def test_tree_attention_last_page_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements (4.3 GB): the pages at its end."""
    D, KV, ps = 128, 8, 64
    pages = (1 << 31) // (D * KV * ps) + 5
    kc = torch.zeros(pages, ps, KV, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v, table, ctx, par = tree_inputs(2, 3, 16, KV, D, [70, 100], ps, 9, True, spare=0)
    n = k.shape[0]
    dev = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    kc[pages - n:] = dev(k)
    vc[pages - n:] = dev(v)
    o, l = torch.empty(2, 3, 16, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        2, 3, 16, device="cuda")
    high = np.where(table >= 0, table + (pages - n), table).astype(np.int32)
    rr.rr_attention_tree_fwd(dev(q), kc, vc, torch.from_numpy(high).cuda(),
                             torch.from_numpy(ctx).cuda(), o, lse=l,
                             parents=torch.from_numpy(par).cuda())
    ro, rl, mag = ref.tree_attention(q, k, v, table, ctx, par)
    compare("o", host(o), ro, 0.0, 1e-6, scale=mag, scale_rtol=2.0 ** -7)
    compare("lse", host(l), rl, 1e-5, 1e-5)


# ------------------------------------------------------------- verification ---

def verify_inputs(B, n, V, dtype, seed, branch=0, noise=0.6, greedy=False):
    rng = np.random.default_rng(seed)
    t = rng.standard_normal((B, n + 1, V)) * 2.0
    d = t[:, :n] + noise * rng.standard_normal((B, n, V))
    t, d = store(t, dtype), store(d, dtype)
    T = rng.uniform(0.6, 1.5, B).astype(np.float32)
    if greedy:
        T[::2] = 0.0
    par = None
    if branch:
        par = np.array([[max(-1, i // branch - 1) for i in range(n)] for _ in range(B)], np.int32)
    tok = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            up = i - 1 if par is None else par[b, i]
            q = ref.softmax_row(ref.f64(d[b, up + 1]), float(T[b]) or 0.05)
            tok[b, i] = rng.choice(V, p=q)
    u = rng.random((B, n)).astype(np.float32)
    e = rng.exponential(size=(B, V)).astype(np.float32)
    return t, d, tok, u, e, par, T


def run_verify(t, d, tok, u, e, par, T, pad=0):
    B, n1, V = t.shape
    out = [empty_like_dev((B, n1), "i32", fill=99), empty_like_dev((B, n1), "i32", fill=99),
           empty_like_dev((B,), "i32", fill=99)]
    up = lambda a: None if a is None else to_dev(a).view(a.shape)  # noqa: E731
    rr.rr_draft_verify(to_dev(t, pad), to_dev(d, pad) if n1 > 1 else to_dev(t, pad)[:, :0].contiguous(),
                       up(tok), up(u), up(e), *out, parents=up(par), temperature=up(T))
    torch.cuda.synchronize()
    check_guards()
    assert rr.rr_read_device_error(0) == 0
    return [x.cpu().numpy() for x in out]


def check_verify(*a, pad=0, least=0.9):
    got = run_verify(*a, pad=pad)
    want = ref.verify(*a[:5], parents=a[5], temperature=a[6])
    clear = want[3] > 1e-5
    assert clear.mean() >= least
    for g, w in zip(got, want):
        assert (g[clear] == w[clear]).all()
    return want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50304])
@pytest.mark.parametrize("branch", [0, 2, 3])
def test_verify(V, branch, dtype):
    B, n = (40, 7) if V <= 1000 else (6, 6)
    w = check_verify(*verify_inputs(B, n, V, dtype, V + branch, branch), pad=V % 2)
    if V >= 1000:
        assert w[2].max() > 0 and w[2].min() < n


@pytest.mark.parametrize("V", [1, 31, 5003])
@pytest.mark.parametrize("branch", [0, 3])
def test_verify_greedy_and_sampled_sequences(V, branch):
    check_verify(*verify_inputs(30, 6, V, "bf16", V, branch, noise=0.2, greedy=True))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [3, 40, 1003, 50304, 300001])
def test_verify_greedy_trees_of_siblings(V, dtype):
    """All four ways: the target's largest logit is the first child's token, a later
    child's or none's, and the draft's largest is the target's or another."""
    B, n = 24 if V <= 1003 else 6, 7
    rng = np.random.default_rng(V)
    t, d, tok, u, e, par, _ = verify_inputs(B, n, V, dtype, V, 3)
    for b in range(B):
        for r in range(n + 1):
            best = int(ref.f64(t[b, r]).argmax())
            kids = [i for i in range(n) if par[b, i] == r - 1]
            if not kids:
                continue
            tok[b, kids] = rng.choice([x for x in range(min(V, 50)) if x != best], len(kids))
            way = rng.integers(0, 4)
            if way < 3:
                tok[b, kids[min(way, len(kids) - 1)]] = best
            if rng.random() < 0.5:
                d[b, r, best] = store(np.array([99.0]), dtype)[0]
    check_verify(t, d, tok, u, e, par, np.zeros(B, np.float32), least=1.0)


@pytest.mark.parametrize("n", [1, 2, 40])
def test_verify_poor_and_perfect_drafts(n):
    """Drafts unlike the target (every child is rejected, the residual is
    reduced many times), and equal to it (every token is accepted)."""
    a = verify_inputs(20, n, 333, "f32", n, 0 if n == 1 else n, noise=4.0)
    check_verify(*a)
    t, d, tok, u, e, par, T = verify_inputs(20, n, 333, "f32", n, 0, noise=0.0)
    out, nodes, count = run_verify(t, d, tok, u, e, par, T)
    assert (count == n).all() and (out[:, :n] == tok).all()
    assert (nodes[:, :n] == np.arange(n)).all()


def test_verify_no_nodes_draws_from_the_target():
    t, d, tok, u, e, par, T = verify_inputs(50, 0, 1000, "f32", 8)
    check_verify(t, d, tok, u, e, None, T)


def test_verify_large_batch():
    check_verify(*verify_inputs(700, 3, 64, "bf16", 2, 2))


@pytest.mark.parametrize("V,dtype", [(300001, "f32"), (524287, "bf16")])
@pytest.mark.parametrize("branch", [0, 2])
def test_verify_rows_longer_than_a_cluster_holds(V, dtype, branch):
    check_verify(*verify_inputs(3, 4, V, dtype, 77 + branch, branch, greedy=True), least=0.6)


def test_verify_more_nodes_than_shared_memory_holds():
    B, n, V = 2, 20000, 5
    rng = np.random.default_rng(3)
    t = rng.standard_normal((B, n + 1, V)).astype(np.float32)
    d = t[:, :n] + np.float32(0.05) * rng.standard_normal((B, n, V)).astype(np.float32)
    tok = rng.integers(0, V, (B, n)).astype(np.int32)
    par = np.array([[max(-1, i // 8 - 1) for i in range(n)] for _ in range(B)], np.int32)
    check_verify(t, d, tok, rng.random((B, n)).astype(np.float32),
                 rng.exponential(size=(B, V)).astype(np.float32), par, None)


def test_verify_absent_nodes_masked_and_undefined_rows():
    t, d, tok, u, e, par, T = verify_inputs(12, 6, 200, "f32", 21, 2)
    tok[0] = -1                               # nothing drafted
    tok[1, 0], tok[2, 1] = 200, 2 ** 31 - 1   # outside the vocabulary
    par[3, 3] = 5                             # a link that leads nowhere
    par[4, 2:] = -9
    t[5, 0, 10:] = -np.inf                    # most of the target masked
    t[6, 0] = -np.inf                         # all of it
    d[7, 0] = -np.inf                         # a draft row without a distribution
    t[8, 0, 3] = np.nan
    t[9, 0, 3] = np.inf
    T[10], t[10, 0] = 0.0, -np.inf
    u[11] = 0.0
    keep = [i for i in range(12) if i not in (7, 8, 9)]
    got = run_verify(t, d, tok, u, e, par, T)
    want = ref.verify(t, d, tok, u, e, parents=par, temperature=T)
    for g, w in zip(got, want):
        assert (g[keep] == w[keep]).all()
    for b in (6, 8, 9, 10):
        assert got[2][b] == 0 and (got[0][b] == -1).all()
    assert got[0][7, 0] == tok[7, 0]          # q = 0 there: the first child is accepted


def test_verify_first_token_has_the_targets_distribution():
    rng = np.random.default_rng(6)
    B, V = 60000, 7
    t1, d1 = rng.standard_normal((3, V)) * 1.5, rng.standard_normal((2, V)) * 1.5
    q = ref.softmax_row(d1[0], 1.0)
    t = np.broadcast_to(t1, (B, 3, V)).astype(np.float32).copy()
    d = np.broadcast_to(d1, (B, 2, V)).astype(np.float32).copy()
    tok = rng.choice(V, size=(B, 2), p=q).astype(np.int32)
    par = np.full((B, 2), -1, np.int32)
    out, _, _ = run_verify(t, d, tok, rng.random((B, 2)).astype(np.float32),
                           rng.exponential(size=(B, V)).astype(np.float32), par, None)
    p = ref.softmax_row(t1[0], 1.0)
    got = np.bincount(out[:, 0], minlength=V) / B
    assert np.all(np.abs(got - p) < 4.5 * np.sqrt(p * (1 - p) / B))


# ------------------------------------------------------------ as it is used ---

def test_draft_score_verify_and_distil_together():
    """One speculative step of a one-layer model: the tree's keys are in the
    cache, the tree is scored, greedily verified against step-by-step decoding
    in float64, and the draft is distilled on the target's top logits."""
    rng = np.random.default_rng(12)
    V, H, KV, D, ps, L, n, B = 211, 4, 2, 64, 16, 37, 7, 5
    emb = rng.standard_normal((V, H * D))
    wk, wv = (rng.standard_normal((H * D, KV * D)) / 16 for _ in range(2))
    head = rng.standard_normal((H * D, V)) / 4
    rnd = lambda a: ref.f64(store(np.asarray(a, np.float32), "bf16"))  # noqa: E731
    K = lambda tk: rnd(emb[tk] @ wk).reshape(-1, KV, D)  # noqa: E731
    W = lambda tk: rnd(emb[tk] @ wv).reshape(-1, KV, D)  # noqa: E731

    def next_logits(toks):  # the last token attends to all of toks
        q = rnd(emb[toks[-1]]).reshape(H, D)
        o = np.zeros((H, D))
        for h in range(H):
            s = K(toks)[:, h // 2] @ q[h] / np.sqrt(D)
            p = np.exp(s - s.max())
            o[h] = (p / p.sum()) @ W(toks)[:, h // 2]
        return o.reshape(-1) @ head

    q = np.zeros((B, n + 1, H, D))
    width = (L + n + ps) // ps + 1
    kc, vc = np.zeros((B * width, ps, KV, D)), np.zeros((B * width, ps, KV, D))
    table = rng.permutation(B * width).astype(np.int32).reshape(B, width)
    par = np.tile(np.array([-1, 0, 0, 1, 1, 2, 3, 5], np.int32), (B, 1))   # node 0: last token
    toks = np.zeros((B, n + 1), np.int32)
    want = []
    for b in range(B):
        prompt = list(rng.integers(0, V, L + 1))
        steps, seq = [], list(prompt)
        for _ in range(5):  # plain decoding, and how clear each choice is
            z = next_logits(np.array(seq))
            o = np.sort(z)
            steps.append((int(z.argmax()), o[-1] - o[-2]))
            seq.append(steps[-1][0])
        want.append(steps)
        toks[b] = rng.integers(0, V, n + 1)
        toks[b, 0] = prompt[-1]
        path = [1, 3, 6][:b]              # the drafted tokens that are right
        for depth, node in enumerate(path):
            toks[b, node] = steps[depth][0]
        allk = np.concatenate([K(np.array(prompt[:-1])), K(toks[b])])
        allv = np.concatenate([W(np.array(prompt[:-1])), W(toks[b])])
        for p in range(L + n + 1):
            kc[table[b, p // ps], p % ps], vc[table[b, p // ps], p % ps] = allk[p], allv[p]
        q[b] = emb[toks[b]].reshape(n + 1, H, D)
    a = (store(q, "bf16"), store(kc, "bf16"), store(vc, "bf16"), table,
         np.full(B, L, np.int32), par)
    o, _ = run_tree(*a)
    ro, _, mag = ref.tree_attention(*a)
    compare("o", host(o), ro, 0.0, 1e-6, scale=mag, scale_rtol=2.0 ** -7)
    target = (o.float().reshape(B, n + 1, H * D).double()
              @ torch.from_numpy(head).cuda()).float().contiguous()
    # the verified tree is that of nodes 1..n: node i there is node i + 1 here
    vpar = to_dev((par[:, 1:] - 1).astype(np.int32)).view(B, n)
    draft = (target[:, :n] + torch.randn(B, n, V, device="cuda",
                                         generator=torch.Generator("cuda").manual_seed(3)))
    dt = to_dev(np.ascontiguousarray(toks[:, 1:])).view(B, n)
    out = [torch.empty(B, n + 1, dtype=torch.int32, device="cuda"),
           torch.empty(B, n + 1, dtype=torch.int32, device="cuda"),
           torch.empty(B, dtype=torch.int32, device="cuda")]
    rr.rr_draft_verify(target, draft, dt, torch.zeros(B, n, device="cuda"),
                       torch.ones(B, V, device="cuda"), *out, parents=vpar,
                       temperature=torch.zeros(B, device="cuda"))
    tokens, count = out[0].cpu().numpy(), out[2].cpu().numpy()
    # how far the logits are from those of the float64 attention
    off = np.abs(host(target) - ro.reshape(B, n + 1, H * D) @ head).max(axis=(1, 2))
    called = 0
    for b in range(B):
        for depth in range(min(b, 3) + 1):
            tok, gap = want[b][depth]
            if gap < 2 * off[b]:
                break  # too close to call with o in bf16
            assert tokens[b, depth] == tok
            called += 1
        assert 0 <= count[b] <= n
    assert called >= 5
    rows = target[:, :n].reshape(B * n, V)
    value, index = torch.topk(rows, 8, dim=1)
    loss = torch.empty(B * n, device="cuda")
    dl = torch.empty(B * n, V, device="cuda")
    rr.rr_distill_fwd_bwd(draft.reshape(B * n, V), index.int(), value.contiguous(), loss, dl,
                          temperature=2.0)
    rl, rd, lm, dm = ref.distill(draft.reshape(B * n, V).cpu().numpy(), index.cpu().numpy(),
                                 value.cpu().numpy(), T=2.0)
    compare("loss", host(loss), rl, 0.0, 1e-30, scale=lm, scale_rtol=64 * ref.EPS)
    compare("dlogits", host(dl), rd, 2.0 ** -23, 1e-30, scale=dm, scale_rtol=64 * ref.EPS)


def test_calls_on_two_streams_at_once():
    """Each of the three on two streams that are not the current one, with workspaces of
    their own (the binding's too): bit for bit what calls one after the other give."""
    B, n, H, KV, D, ps, V, k = 9, 12, 16, 2, 128, 16, 30011, 20
    sides = []
    for seed in (1, 2):
        q, kc, vc, table, ctx, par = tree_inputs(B, n, H, KV, D, [700 * b % 4001 for b in range(B)],
                                                 ps, seed, True)
        dev = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
        a = [dev(q), dev(kc), dev(vc)] + [torch.from_numpy(x).cuda() for x in (table, ctx, par)]
        g = torch.Generator("cuda").manual_seed(seed)
        t = torch.randn(B, n + 1, V, device="cuda", generator=g)
        d = t[:, :n] + 0.3 * torch.randn(B, n, V, device="cuda", generator=g)
        v = [t, d.contiguous(), d.argmax(2).int(), torch.rand(B, n, device="cuda", generator=g),
             torch.rand(B, V, device="cuda", generator=g) + 0.01]
        idx = torch.randint(0, V, (B * n, k), dtype=torch.int32, device="cuda", generator=g)
        val = torch.randn(B * n, k, device="cuda", generator=g)
        sides.append((a, v, idx, val, torch.cuda.Stream()))

    def outs():
        i32 = dict(dtype=torch.int32, device="cuda")
        return [torch.zeros(B, n, H, D, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(B, n, H, device="cuda"), torch.zeros(B, n + 1, **i32),
                torch.zeros(B, n + 1, **i32), torch.zeros(B, **i32),
                torch.zeros(B * n, device="cuda"), torch.zeros(B * n, V, device="cuda")]

    def run(side, o, stream):
        a, v, idx, val, _ = side
        rr.rr_attention_tree_fwd(*a[:5], o[0], lse=o[1], parents=a[5], stream=stream)
        rr.rr_draft_verify(*v, *o[2:5], parents=a[5], stream=stream)
        rr.rr_distill_fwd_bwd(v[1].view(B * n, V), idx, val, o[5], o[6], stream=stream)

    want = [outs(), outs()]
    for side, o in zip(sides, want):
        run(side, o, None)
        torch.cuda.synchronize()
    got = [[outs() for _ in range(8)] for _ in sides]
    torch.cuda.synchronize()
    for i in range(8):
        for side, o in zip(sides, got):
            run(side, o[i], side[4])
    torch.cuda.synchronize()
    assert rr.rr_read_device_error(0) == 0
    for w, o in zip(want, got):
        for x in o:
            assert all(torch.equal(p, r) for p, r in zip(w, x))


def test_captured_calls_replay_on_new_inputs():
    """The three calls captured in one graph, replayed on other inputs (twice):
    bit for bit what direct calls give."""
    B, n, H, KV, D, ps, V, k = 3, 5, 8, 2, 64, 16, 5001, 9
    q, kc, vc, table, ctx, par = tree_inputs(B, n, H, KV, D, [20, 900, 333], ps, 1, True)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    q, kc, vc = dev(q), dev(kc), dev(vc)
    table, ctx, par = (torch.from_numpy(a).cuda() for a in (table, ctx, par))
    t, d, tok, u, e, _, T = (torch.from_numpy(a).cuda() if a is not None else None
                             for a in verify_inputs(B, n, V, "f32", 2, 2))
    idx = torch.randint(0, V, (B * n, k), dtype=torch.int32, device="cuda")
    val = torch.randn(B * n, k, device="cuda")
    ws = torch.empty(rr.rr_attention_tree_workspace_size(B, n, H, KV, D), dtype=torch.uint8,
                     device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(q), torch.empty(B, n, H, device="cuda"), torch.empty(B, n + 1, **i32),
            torch.empty(B, n + 1, **i32), torch.empty(B, **i32), torch.empty(B * n, device="cuda"),
            torch.empty(B * n, V, device="cuda")]

    def step():
        rr.rr_attention_tree_fwd(q, kc, vc, table, ctx, outs[0], lse=outs[1], parents=par,
                                 workspace=ws)
        rr.rr_draft_verify(t, d, tok, u, e, outs[2], outs[3], outs[4], parents=par, temperature=T)
        rr.rr_distill_fwd_bwd(d.view(B * n, V), idx, val, outs[5], outs[6], tail=False)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (5, 6):
        torch.manual_seed(seed)
        q.copy_(torch.randn_like(q.float()))
        t.copy_(torch.randn_like(t))
        d.copy_(t[:, :n] + 0.5 * torch.randn_like(d))
        val.copy_(torch.randn_like(val))
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in outs]
        for x in outs:
            x.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
