"""The sizes up to which the packed-sequence operators say that they work: at the limit a call gets
as far as its (missing) tensors, above it the size is named."""
import ctypes

import pytest

import row_reduction_pass_gb300 as rr_pkg
from test_packed_ref import attn_bwd, attn_fwd, lp_bwd, ptr, rope_bwd, rope_fwd


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return rr_pkg.load_library()


def detail(lib, call, **kw):
    assert call(lib, **kw) == 1
    return lib.rr_last_error_detail().decode()


@pytest.mark.parametrize("call", [attn_fwd, attn_bwd])
def test_attention_limits(lib, call):
    wide = dict(H=1024, KV=1024, sq=65536, sk=65536, sv=65536, so=65536, q=None)
    for name in ("sdo", "sdq", "sdk", "sdv") if call is attn_bwd else ():
        wide[name] = 65536
    for sizes in (dict(T=2 ** 22, B=1), dict(H=1, KV=1, T=2 ** 31 - 1 - 4096, B=1)):
        assert "null pointer" in detail(lib, call, **(wide | sizes))
    for sizes in (dict(T=2 ** 22 + 1, B=1), dict(H=1, KV=1, T=2 ** 31 - 4096, B=1),
                  dict(H=65535, KV=65535, T=1, B=2 ** 15 + 1)):
        assert "too many" in detail(lib, call, **(wide | sizes))


@pytest.mark.parametrize("call", [rope_fwd, rope_bwd])
def test_rotation_limits(lib, call):
    assert "null pointer" in detail(lib, call, T=2 ** 31 - 1, q=None)
    assert "too many tokens" in detail(lib, call, T=2 ** 31, q=None)


def test_logprob_gradient_limits(lib):
    sizes = dict(V=4097, s=4097, sy=4097)  # fp32: two pieces of 16384 bytes a row
    assert "too many rows" in detail(lib, lp_bwd, R=2 ** 30, y=ptr(1 << 12), **{
        n: ptr((i + 1) << 5) for i, n in enumerate(("x", "t", "rm", "ls", "en", "g", "h"))}, **sizes)
