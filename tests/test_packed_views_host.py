"""Strides of the packed calls' and the rotation's tensors (no GPU): which are refused."""
import pytest

from test_packed_host import ALL, FAKE, heads, lib, packed, passed, rotary  # noqa: F401


@pytest.mark.parametrize("backward", (False, True))
def test_one_token_in_a_long_buffer_of_each_head(lib, backward):  # noqa: F811
    """The stride between tokens is not looked at where there is one, nor made up to be too large: a
    token of [heads][tokens][d] with 2^27 tokens a head, 128 heads."""
    q = heads(n=128, head=1 << 33, token=64)
    k = heads(n=2, head=1 << 33, token=64)
    assert passed(packed(lib, backward, q=q, o=q, g=q, dq=q, k=k, v=k, dk=k, dv=k, tq=1, tk=1, B=1))


@pytest.mark.parametrize("which", ALL, ids=str)
def test_one_token_of_a_long_buffer_turns(lib, which):  # noqa: F811
    q, k = heads(n=16, head=1 << 33, token=64), heads(n=2, head=1 << 33, token=64)
    assert passed(rotary(lib, q=q, qo=q, k=k, ko=k, N=1, **which))
