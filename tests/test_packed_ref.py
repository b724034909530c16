"""CPU checks of the packed-sequence operators: the plain float64 forms against autograd and
worked cases, and the library's refusals (fake pointers, never dereferenced)."""
import ctypes
import math

import pytest
import torch

import packed_ref as ref
import row_reduction_pass_gb300 as rr_pkg


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


# -------------------------------------------------------------- plain forms ---

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [2, 4, 6])
def test_rope_gradient_is_autograds(rot, interleaved):
    T, H, D = 5, 3, 6
    x, w, dy = rnd(T, H, D), 1 + 0.3 * rnd(D, seed=1), rnd(T, H, D, seed=2)
    cos, sin = ref.table(20, rot)
    pos = torch.tensor([0, 7, 19, 3, 3])
    x.requires_grad_()
    w.requires_grad_()
    y, _ = ref.rope(x, w, cos, sin, pos, 1e-3, interleaved)
    y.backward(dy)
    (dx, _), (dw, _) = ref.rope_bwd(dy, x.detach(), w.detach(), cos, sin, pos, 1e-3, interleaved)
    assert torch.allclose(dx, x.grad, atol=1e-12) and torch.allclose(dw, w.grad, atol=1e-12)


def test_rope_worked_case():
    """Two elements (3, 4), no eps: the norm is sqrt(12.5); a quarter turn takes (a, b) to
    (-b, a)."""
    cos, sin = torch.zeros(1, 1), torch.ones(1, 1)
    y, _ = ref.rope(torch.tensor([[[3.0, 4.0]]]), torch.tensor([1.0, 2.0]), cos, sin,
                    torch.tensor([0]), 0.0, False)
    r = 1 / math.sqrt(12.5)
    assert torch.allclose(y, torch.tensor([[[-8.0 * r, 3.0 * r]]]).double())


def test_rope_scores_depend_on_the_distance_only():
    cos, sin = ref.table(50, 8)
    q, k = rnd(1, 1, 8), rnd(1, 1, 8, seed=1)
    at = lambda x, p: ref.rope(x, None, cos, sin, torch.tensor([p]), 0.0, False)[0]  # noqa: E731
    a = (at(q, 13) * at(k, 5)).sum()
    b = (at(q, 41) * at(k, 33)).sum()
    assert abs(float(a - b)) < 1e-5  # (float32 tables)


def test_attention_gradient_is_autograds():
    T, H, KV, D = 9, 4, 2, 3
    q, k, v, do = rnd(T, H, D), rnd(T, KV, D, seed=1), rnd(T, KV, D, seed=2), rnd(T, H, D, seed=3)
    cu = [0, 4, 4, 5, 9]
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o = torch.zeros(T, H, D, dtype=torch.float64)
    for a, b in zip(cu, cu[1:]):
        for h in range(H):
            s = 0.7 * leaves[0][a:b, h] @ leaves[1][a:b, h // 2].T
            s = s.masked_fill(torch.ones(b - a, b - a).triu(1) > 0, -math.inf)
            o[a:b, h] = torch.softmax(s, 1) @ leaves[2][a:b, h // 2]
    o.backward(do)
    assert torch.allclose(ref.attention(q, k, v, cu, 0.7)[0], o.detach(), atol=1e-12)
    got, _ = ref.attention_bwd(do, q, k, v, o.detach(), cu, 0.7)
    for g, leaf in zip(got, leaves):
        assert torch.allclose(g, leaf.grad, atol=1e-12)


def test_logprob_gradient_is_autograds_and_differences():
    x, tok = rnd(3, 7), torch.tensor([2, 0, 6])
    g, h = rnd(3, seed=1), rnd(3, seed=2)
    leaf = x.clone().requires_grad_()

    def total(z):
        lp = torch.log_softmax(z / 0.8, 1)
        ent = -(lp.exp() * lp).sum(1)
        return (g * lp[torch.arange(3), tok] + h * ent).sum()

    total(leaf).backward()
    d, _ = ref.logprob_bwd(x, tok, g, h, 0.8)
    assert torch.allclose(d, leaf.grad, atol=1e-12)
    for r, j in ((0, 2), (1, 5)):
        e = torch.zeros_like(x)
        e[r, j] = 1e-5
        num = (total(x + e) - total(x - e)) / 2e-5
        assert abs(float(num - d[r, j])) < 1e-8


def test_logprob_worked_case():
    """Logits ln 1, ln 2, ln 1: probabilities 1/4, 1/2, 1/4; entropy 1.5 ln 2."""
    x = torch.tensor([[0.0, math.log(2.0), 0.0]])
    got = ref.logprob(x, torch.tensor([2]), 1.0, 3)
    assert abs(float(got["logprob"][0]) + 2 * math.log(2.0)) < 1e-7
    assert abs(float(got["entropy"][0]) - 1.5 * math.log(2.0)) < 1e-7
    assert got["rank"].tolist() == [2] and got["top_index"].tolist() == [[1, 0, 2]]


# ----------------------------------------------------------------- refusals ---

@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return rr_pkg.load_library()


def ptr(i):
    return ctypes.c_void_p((i + 1) << 36)  # far apart


F = ctypes.c_float
S0 = ctypes.c_void_p(0)


def rope_fwd(lib, **kw):
    a = dict(q=ptr(0), k=ptr(1), qw=ptr(2), kw=ptr(3), cos=ptr(4), sin=ptr(5), pos=ptr(6),
             qo=ptr(7), ko=ptr(8), T=0, H=4, KV=2, D=64, R=64, P=10, sq=256, sk=128, so=256, sp=128,
             eps=1e-6, inter=0, bad=None, dt=1) | kw
    v = list(a.values())
    v[19] = F(v[19])
    return lib.rr_qk_norm_rope_fwd(*v, S0)


def rope_bwd(lib, **kw):
    a = dict(gq=ptr(0), gk=ptr(1), q=ptr(2), k=ptr(3), qw=ptr(4), kw=ptr(5), cos=ptr(6),
             sin=ptr(7), pos=ptr(8), dq=ptr(9), dk=ptr(10), dqw=None, dkw=None, ws=None, n=0, T=0,
             H=4, KV=2, D=64, R=64, P=10, s0=256, s1=128, s2=256, s3=128, s4=256, s5=128, eps=1e-6,
             inter=0, bad=None, dt=1) | kw
    v = list(a.values())
    v[27] = F(v[27])
    return lib.rr_qk_norm_rope_bwd(*v, S0)


@pytest.mark.parametrize("call", [rope_fwd, rope_bwd])
@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(dt=5), 2), (dict(T=-1), 1), (dict(H=0), 1), (dict(KV=-1), 1), (dict(H=65536), 1),
    (dict(D=63), 1), (dict(D=258), 1), (dict(R=0), 1), (dict(R=66), 1), (dict(R=3), 1),
    (dict(P=-1), 1), (dict(P=2 ** 31), 1), (dict(eps=-1.0), 1), (dict(eps=math.inf), 1),
    (dict(eps=math.nan), 1), (dict(T=3, q=None), 1), (dict(T=3, k=None), 1),
    (dict(T=3, cos=None), 1), (dict(T=3, pos=ctypes.c_void_p(0x1002)), 1),
    (dict(T=3, qw=ctypes.c_void_p(0x1001)), 1), (dict(T=2 ** 31), 1)])
def test_rope_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_rope_strides_and_aliases(lib):
    assert rope_fwd(lib, sq=255) == 1 and rope_fwd(lib, sp=127) == 1
    assert rope_bwd(lib, s4=255) == 1 and rope_bwd(lib, s5=2 ** 28 + 1) == 1
    # side by side in one buffer: apart; a token on: not
    base = 1 << 36
    at = lambda e: ctypes.c_void_p(base + 2 * e)  # noqa: E731
    side = dict(T=5, q=at(0), k=at(256), sq=512, sk=512, so=512, sp=512, pos=ctypes.c_void_p(6))
    assert rope_fwd(lib, **side, qo=at(0), ko=at(256)) == 1            # (positions misaligned)
    side["pos"] = None
    assert rope_fwd(lib, **side, qo=at(8), ko=ptr(9)) == 3             # partly over q
    assert rope_fwd(lib, **side, qo=at(256), ko=ptr(9)) == 3           # over k
    assert rope_fwd(lib, **(side | dict(so=256)), qo=at(0), ko=ptr(9)) == 3  # another stride
    assert rope_fwd(lib, **side, qo=ptr(8), ko=ptr(8)) == 3
    assert rope_fwd(lib, **side, qo=at(0), ko=at(256), bad=at(0)) == 3
    assert rope_bwd(lib, T=3, dqw=ptr(20)) == 1                        # one weight gradient only
    assert rope_bwd(lib, T=3, dk=ptr(9)) == 3                          # dk over dq
    assert rope_bwd(lib, T=3, dk=ptr(2)) == 3                          # dk over q


def attn_fwd(lib, **kw):
    a = dict(q=ptr(0), k=ptr(1), v=ptr(2), cu=ptr(3), o=ptr(4), lse=ptr(5), T=0, B=2, H=4, KV=2,
             D=64, sq=256, sk=128, sv=128, so=256, scale=0.1, dt=1) | kw
    v = list(a.values())
    v[15] = F(v[15])
    return lib.rr_attention_packed_fwd(*v, S0)


def attn_bwd(lib, **kw):
    a = dict(do=ptr(0), q=ptr(1), k=ptr(2), v=ptr(3), o=ptr(4), lse=ptr(5), cu=ptr(6), dq=ptr(7),
             dk=ptr(8), dv=ptr(9), ws=ptr(10), n=1 << 30, T=0, B=2, H=4, KV=2, D=64, sdo=256,
             sq=256, sk=128, sv=128, so=256, sdq=256, sdk=128, sdv=128, scale=0.1, dt=1) | kw
    v = list(a.values())
    v[25] = F(v[25])
    return lib.rr_attention_packed_bwd(*v, S0)


@pytest.mark.parametrize("call", [attn_fwd, attn_bwd])
@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(T=5, B=0), 0), (dict(dt=3), 2), (dict(T=-1), 1), (dict(B=-1), 1),
    (dict(B=2 ** 20 + 1), 1), (dict(H=0), 1), (dict(KV=0), 1), (dict(H=5), 1), (dict(D=60), 1),
    (dict(D=264, sq=2048, sk=2048, so=2048), 1), (dict(D=0), 1), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(sq=255), 1), (dict(sk=129), 1),
    (dict(sv=120), 1), (dict(so=2 ** 28 + 8), 1), (dict(T=2 ** 31), 1),
    (dict(q=ctypes.c_void_p(8)), 1), (dict(lse=ctypes.c_void_p(6)), 1), (dict(T=4, q=None), 1),
    (dict(T=4, cu=None), 1), (dict(T=4, o=None), 1), (dict(T=4, cu=ctypes.c_void_p(6)), 1)])
def test_attention_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_attention_aliases_and_workspace(lib):
    assert attn_fwd(lib, T=4, o=ptr(0)) == 3 and attn_fwd(lib, T=4, lse=ptr(1)) == 3
    assert attn_fwd(lib, T=4, o=ptr(3)) == 3
    assert attn_bwd(lib, T=4, dq=ptr(0)) == 3 and attn_bwd(lib, T=4, dv=ptr(8)) == 3
    assert attn_bwd(lib, T=4, ws=ptr(5)) == 3 and attn_bwd(lib, T=4, dk=ptr(4)) == 3
    assert attn_bwd(lib, T=4, n=63) == 4 and attn_bwd(lib, T=4, ws=None) == 4
    assert attn_bwd(lib, T=4, dq=None) == 1 and attn_bwd(lib, T=4, lse=None) == 1
    assert lib.rr_attention_packed_bwd_workspace_size(0, 4) == 0
    assert lib.rr_attention_packed_bwd_workspace_size(5, 0) == 0


def lp_fwd(lib, **kw):
    a = dict(x=ptr(0), t=ptr(1), lp=ptr(2), en=ptr(3), rm=ptr(4), ls=ptr(5), rk=ptr(6), ti=ptr(7),
             tl=ptr(8), R=0, V=100, s=100, k=5, T=1.0, ig=-100, bad=None, dt=0) | kw
    v = list(a.values())
    v[13] = F(v[13])
    return lib.rr_token_logprob_fwd(*v, S0)


def lp_bwd(lib, **kw):
    a = dict(x=ptr(0), t=ptr(1), rm=ptr(2), ls=ptr(3), en=ptr(4), g=ptr(5), h=ptr(6), y=ptr(7),
             R=0, V=100, s=100, sy=100, T=1.0, ig=-100, dt=0) | kw
    v = list(a.values())
    v[12] = F(v[12])
    return lib.rr_token_logprob_bwd(*v, S0)


@pytest.mark.parametrize("call", [lp_fwd, lp_bwd])
@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(dt=2), 2), (dict(R=-1), 1), (dict(V=0), 1), (dict(s=99), 1),
    (dict(V=2 ** 31, s=2 ** 31), 1), (dict(T=0.0), 1), (dict(T=1e-40), 1), (dict(T=3e38), 1),
    (dict(T=math.nan), 1), (dict(R=2, x=None), 1), (dict(R=2, t=None), 1),
    (dict(R=2, x=ctypes.c_void_p(2)), 1), (dict(R=2, t=ctypes.c_void_p(6)), 1),
    (dict(R=2 ** 59), 1)])
def test_logprob_refusals(lib, call, kw, status):
    assert call(lib, **kw) == status


def test_logprob_lists_and_aliases(lib):
    assert lp_fwd(lib, k=129) == 1 and lp_fwd(lib, k=-1) == 1
    assert lp_fwd(lib, R=2, ti=None) == 1 and lp_fwd(lib, R=2, lp=None) == 1
    assert lp_fwd(lib, R=2, lp=ptr(0)) == 3 and lp_fwd(lib, R=2, en=ptr(2)) == 3
    assert lp_fwd(lib, R=2, tl=ptr(1)) == 3
    assert lp_bwd(lib, R=2, en=None) == 1                       # an entropy gradient without it
    assert lp_bwd(lib, R=2, sy=99) == 1 and lp_bwd(lib, R=2, y=None) == 1
    assert lp_bwd(lib, R=2, y=ctypes.c_void_p((1 << 36) + 4)) == 3
    assert lp_bwd(lib, R=2, y=ptr(0), sy=104) == 3              # in place with another stride
    assert lp_bwd(lib, R=2, y=ptr(5)) == 3
