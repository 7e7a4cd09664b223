"""Strides of the packed calls' and the rotation's tensors (no GPU): which are refused."""
import pytest

from test_packed_host import ALL, FAKE, SHAPE, heads, lib, packed, passed, rotary  # noqa: F401


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


@pytest.mark.parametrize("which", ALL, ids=str)
def test_sequences_of_a_batch_that_overlap_are_refused(lib, which):  # noqa: F811
    same = dict(B=3, k=heads(n=2, batch=5120), ko=heads(n=2, batch=5120))
    fine = [heads(batch=2560),                       # one behind the other: 10 tokens of 4 heads of 64
            heads(batch=256, token=768),             # token by token
            heads(batch=64, head=192, token=768),    # head by head
            heads(batch=640, token=64, head=1920)]   # [heads][B][N][d]
    for q in fine:
        assert passed(rotary(lib, q=q, qo=q, **same, **which))
    for q in (heads(batch=64), heads(batch=256), heads(batch=2552), heads(batch=2304, token=256), heads(batch=128, token=768),
              heads(batch=1272, token=64, head=640)):
        assert rotary(lib, q=heads(batch=2560), qo=q, **same, **which) == SHAPE


def test_strides_whose_products_leave_64_bits(lib):  # noqa: F811
    """2^31 - 1 tokens 2^34 elements apart do not lie within a head of 64."""
    big = heads(n=2, token=1 << 34, head=64)
    n = (1 << 31) - 1
    assert passed(packed(lib, q=big, o=big, k=big, v=big, tq=n, tk=n, B=1))
    over = heads(n=2, token=1 << 34, head=1 << 34)
    assert packed(lib, q=over, o=over, k=over, v=over, tq=n, tk=n, B=1) == SHAPE
