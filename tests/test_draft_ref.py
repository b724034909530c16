"""CPU checks of the draft model's operators: the float64 plain forms against
differences, closed forms and each other, and the refusals of the C entry
points (fake pointers, never dereferenced)."""
import ctypes

import numpy as np
import pytest

import draft_ref as ref
import row_reduction_pass_gb300 as rr_pkg

S0 = ctypes.c_void_p(0)
CF = ctypes.c_float


def P(i):
    return ctypes.c_void_p(0x100000000 * (i + 1))   # disjoint fake device buffers


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return rr_pkg.load_library()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_distill_gradient_is_the_difference_of_the_loss(tail, T):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 9))
    index = np.array([[2, 5, -1], [0, 8, 3], [1, 1, 4], [7, 100, -2]], np.int32)
    value = np.log(rng.uniform(0.05, 0.3, (4, 3)))
    g = rng.uniform(0.5, 2.0, 4)
    loss, dl, _, _ = ref.distill(x, index, value, g, T, tail)
    h = 1e-6
    for r in range(4):
        for j in range(9):
            a, b = x.copy(), x.copy()
            a[r, j] += h
            b[r, j] -= h
            la = ref.distill(a, index, value, g, T, tail)[0][r]
            lb = ref.distill(b, index, value, g, T, tail)[0][r]
            assert abs(g[r] * (la - lb) / (2 * h) - T * 0 - dl[r, j]) < 1e-6


def test_distill_closed_forms():
    # one entry, no tail: the cross-entropy of that column
    x = np.array([[0.0, 1.0, 2.0]])
    loss, dl, _, _ = ref.distill(x, np.array([[2]], np.int32), np.array([[7.0]]))
    s = np.exp(x[0]) / np.exp(x[0]).sum()
    assert np.isclose(loss[0], -np.log(s[2])) and np.allclose(dl[0], s - [0, 0, 1])
    # the student's own distribution, listed in full: loss 0, gradient 0
    loss, dl, _, _ = ref.distill(x, np.array([[0, 1, 2]], np.int32), x)
    assert abs(loss[0]) < 1e-14 and np.abs(dl).max() < 1e-15
    # its top entry as a log-probability, the rest in the tail: the same
    loss, dl, _, _ = ref.distill(x, np.array([[2]], np.int32), np.log(s[[2]])[None], tail=True)
    assert abs(loss[0]) < 1e-14 and np.abs(dl).max() < 1e-15


def test_verify_first_token_has_the_targets_distribution():
    """Whatever the draft, the first token out is distributed as the target
    (3 standard deviations per token, and one shared draw of inputs)."""
    rng = np.random.default_rng(5)
    V, N = 6, 20000
    t, d = rng.standard_normal((4, V)) * 1.5, rng.standard_normal((3, V)) * 1.5
    p, q = ref.softmax_row(t[0], 1.0), ref.softmax_row(d[0], 1.0)
    par = np.array([[-1, -1, 0]], np.int32)
    counts = np.zeros(V)
    for _ in range(N):
        tok = np.array([[rng.choice(V, p=q), rng.choice(V, p=q), 0]], np.int32)
        out, _, _, _ = ref.verify(t[None], d[None], tok, rng.random((1, 3)),
                                  rng.exponential(size=(1, V)), parents=par)
        counts[out[0, 0]] += 1
    sd = np.sqrt(p * (1 - p) / N)
    assert np.all(np.abs(counts / N - p) < 4 * sd)


def test_distill_argument_errors(lib):
    def f(rows=4, cols=8, k=2, T=1.0, dtype=0, **o):
        a = dict(x=P(0), i=P(1), v=P(2), g=P(3), l=P(4), y=P(5), bad=P(6))
        a.update(o)
        return lib.rr_distill_fwd_bwd(a["x"], a["i"], a["v"], a["g"], a["l"], a["y"], rows, cols,
                                      k, CF(T), 0, a["bad"], dtype, S0)
    assert f(dtype=3) == 2
    assert f(rows=-1) == 1 and f(cols=0) == 1 and f(k=-1) == 1 and f(k=1025) == 1
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-45):
        assert f(T=T) == 1
    assert f(cols=1 << 31) == 1
    assert f(rows=0) == 0
    assert f(x=None) == 1 and f(l=None) == 1 and f(i=None) == 1
    assert f(x=ctypes.c_void_p(0x100000002)) == 1           # fp32 alignment
    assert f(l=ctypes.c_void_p(0x500000002)) == 1
    assert f(y=ctypes.c_void_p(0x100000010)) == 3           # partly over logits
    assert f(l=P(0)) == 3 and f(l=P(1)) == 3 and f(l=P(3)) == 3 and f(y=P(2)) == 3
    assert f(bad=P(4)) == 3 and f(bad=P(5)) == 3 and f(bad=P(1)) == 3


def test_draft_verify_argument_errors(lib):
    def f(batch=2, nodes=3, cols=8, dtype=0, **o):
        a = {n: P(i) for i, n in enumerate("t d k p u r T ot on oc".split())}
        a.update(o)
        return lib.rr_draft_verify(a["t"], a["d"], a["k"], a["p"], a["u"], a["r"], a["T"],
                                   a["ot"], a["on"], a["oc"], batch, nodes, cols, dtype, S0)
    assert f(dtype=2) == 2
    assert f(batch=-1) == 1 and f(nodes=-1) == 1 and f(nodes=65536) == 1 and f(cols=0) == 1
    assert f(cols=1 << 31) == 1 and f(batch=1 << 40) == 1
    assert f(batch=0) == 0
    for n in ("t", "d", "k", "u", "r", "ot", "on", "oc"):
        assert f(**{n: None}) == 1, n
    assert f(u=ctypes.c_void_p(0x500000001)) == 1
    for n in ("t", "d", "k", "p", "u", "r", "T"):
        i = "t d k p u r T ot on oc".split().index(n)
        assert f(ot=P(i)) == 3 and f(on=P(i)) == 3 and f(oc=P(i)) == 3, n
    assert f(ot=P(8)) == 3 and f(oc=P(7)) == 3 and f(oc=P(8)) == 3


def test_attention_tree_argument_errors(lib):
    def f(b=2, n=3, h=8, kv=2, d=64, pages=10, ps=16, w=4, sc=0.125, dtype=1, ws=P(8),
          wsb=1 << 40, **o):
        a = {n_: P(i) for i, n_ in enumerate("q k v t c p o l".split())}
        a.update(o)
        return lib.rr_attention_tree_fwd(a["q"], a["k"], a["v"], a["t"], a["c"], a["p"], a["o"],
                                         a["l"], ws, wsb, b, n, h, kv, d, pages, ps, w, CF(sc),
                                         dtype, S0)
    assert f(dtype=0) == 2
    assert f(d=96) == 1 and f(h=7) == 1 and f(h=0) == 1 and f(kv=0) == 1
    assert f(b=-1) == 1 and f(n=-1) == 1 and f(ps=0) == 1 and f(w=-1) == 1 and f(pages=-1) == 1
    assert f(n=257) == 1                                     # a tree of more than 256 nodes
    assert f(b=1 << 20, n=1 << 20, p=None) == 1
    assert f(b=65537) == 1                                   # more sequences than are looked through
    assert f(b=1, n=1 << 16, h=16385, kv=1, p=None) == 1     # 2^30 rows
    assert f(b=65536, w=1 << 20) == 1                        # key tiles
    assert f(ps=16, w=(1 << 26) + 1) == 1                    # positions
    for sc in (0.0, -1.0, float("nan"), float("inf")):
        assert f(sc=sc) == 1
    assert f(b=0) == 0 and f(n=0) == 0
    for n_ in ("q", "k", "v", "t", "c", "o"):
        assert f(**{n_: None}) == 1, n_
    assert f(q=ctypes.c_void_p(0x100000008)) == 1
    assert f(t=ctypes.c_void_p(0x400000002)) == 1
    assert f(o=P(0)) == 3 and f(o=P(1)) == 3 and f(l=P(2)) == 3 and f(l=P(6)) == 3


def test_bindings_refuse_what_the_kernels_cannot_take():
    import torch
    x = torch.zeros(2, 8)
    i = torch.zeros(2, 2, dtype=torch.int32)
    v, l = torch.zeros(2, 2), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        rr_pkg.rr_distill_fwd_bwd(x, i, v, l)
    with pytest.raises(TypeError, match="top_index"):
        rr_pkg.rr_distill_fwd_bwd(x, i.long(), v, l)
    with pytest.raises(ValueError, match="loss must have shape"):
        rr_pkg.rr_distill_fwd_bwd(x, i, v, torch.zeros(3))
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="v_cache"):
        rr_pkg.rr_attention_tree_fwd(q, kc, kc[:2], i[:1], i[0, :1], q)
    with pytest.raises(ValueError, match="contiguous"):
        rr_pkg.rr_attention_tree_fwd(q.expand(1, 2, 4, 64).transpose(1, 2), kc, kc, i[:1],
                                     i[0, :1], torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16))
    t = torch.zeros(1, 3, 8)
    with pytest.raises(ValueError, match="draft_logits"):
        rr_pkg.rr_draft_verify(t, t, i[:1], v[:1], t[:, 0], i[:1], i[:1], i[0, :1])
