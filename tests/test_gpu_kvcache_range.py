"""Tree decode where a row's weights, values or queries span many binades: one key with
much of the weight before a long flat tail, value rows of zeros among large ones, an
infinity in a query; drafts whose own rows were never written; and batches of many more
sequences than there are CTAs.

The bounds are those that the call promises, not the kernel's own: a probability to 2^-8
of its value, so that their part of o is off by at most 2^-8 sum p|v|, whatever the number
of keys (the 2^-29 of the row's largest that it may be off by besides is 2^-13 over 65536
keys, within what the kernel's 2^-9 leaves of the 2^-8); o rounded to bf16, off by 2^-8 of
its value; scores off by ds, as the tests of the other cases derive it.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
FMTS = ("e4m3", "bf16")


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_16_gb300 as m
    from exact_io_aware_16_gb300 import build

    build.build()
    m.library()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def values(t, s):
    x = t.double()
    return x if s is None else x * torch.exp2(s.double() - 127)[..., None]


def check(fa, cache, q, lens, o, lse, scale, pairs, mask=None):
    """The rows of `pairs` (sequence, key head) against 64 bits; masks causal unless given."""
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)
    B, Hkv, cap, d = cache.shape
    Hq, T = q.shape[1:3]
    G = Hq // Hkv
    j = torch.arange(T, device="cuda")
    for b, h in pairs:
        n = min(lens[b] + T, cap)
        k = values(cache.k[b, h, :n], None if cache.k_scale is None else cache.k_scale[b, h, :n])
        v = values(cache.v[b, h, :n], None if cache.v_scale is None else cache.v_scale[b, h, :n])
        sees = torch.ones(T, n, dtype=torch.bool, device="cuda")
        drafts = j[None] <= j[:, None] if mask is None else mask[b][:, None] >> j[None] & 1 != 0
        sees[:, lens[b]:] = drafts[:, : n - lens[b]]
        for r in range(h * G, h * G + G):
            x = q[b, r].double()
            s = torch.where(sees, x @ k.T * scale, -math.inf)
            want_lse = torch.logsumexp(s, -1)
            p = torch.where(sees, torch.exp(s - want_lse[:, None]), 0.0)
            want, a = p @ v, p @ v.abs()
            ds = 2.0 ** -23 * (d + 8) * scale * (x.abs() @ k.abs().T).amax(-1)
            if cache.format == "e4m3":
                ds = ds + 2.0 ** -12.8 * x.abs().amax(-1) * scale * k.abs().sum(-1).max()
            tol = a * (2.0 ** -8 + 2 * ds[:, None] + 2.0 ** -18) + 2.0 ** -8 * want.abs()
            err = (o[b, r].double() - want).abs()
            assert torch.isfinite(o[b, r]).all() and torch.isfinite(lse[b, r]).all(), (b, r)
            assert (err <= tol).all(), ("o", b, r, (err / tol.clamp(min=1e-300)).max().item())
            off = (lse[b, r].double() - want_lse).abs()
            assert (off <= ds + 2.0 ** -20 * (1 + want_lse.abs())).all(), ("lse", b, r, off.max().item())


# (B, Hq, Hkv, T): 16, 32 and 64 rows a CTA, with as many pairs or row tiles as CTAs, so
# that one CTA walks over whole pairs; and one pair that is spread over all CTAs
SHAPES = [(1, 304, 304, 1), (1, 304, 304, 24), (1, 152, 1, 64), (1, 2, 1, 3)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("weight,spread", ((0.5, 0.0), (0.75, 0.3), (0.9, 1.0)))
def test_one_heavy_key_before_a_long_tail(fa, fmt, d, shape, weight, spread):
    """The tail's keys have 2^-16 of the first key's weight each and, together, 10 to 50 %
    of the row's; the values have a mean, so that a lost weight shows."""
    B, Hq, Hkv, T = shape
    n = 65536 if Hkv == 1 else 8192
    g = gen(d + T)
    gap = math.log(weight / (1 - weight)) + math.log(n) + spread ** 2 / 2  # nats above the tail
    cache = fa.KvCache(B, Hkv, n + T, d, fmt)
    k = randn(g, B, Hkv, n, d) * (spread / math.sqrt(d))  # scores of the tail: spread nats
    k[..., 0] = 0
    k[:, :, 0] = 0
    k[:, :, 0, 0] = gap / 4
    v = randn(g, B, Hkv, n, d) + 0.5
    v[..., 1] = 1.0  # a channel that is the sum of the weights
    fa.fa_cache_write(cache, k.bfloat16(), v.bfloat16())
    q = randn(g, B, Hq, T, d)
    q[..., 0] = 4.0
    q = q.bfloat16()
    lens = [n - T]  # the last T of the tail are drafts
    o, lse = fa.fa_decode_tree(cache, q, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=1.0)
    check(fa, cache, q, lens, o, lse, 1.0, [(0, h) for h in range(0, Hkv, 101)])


# (over a bf16 cache, sums of 5e37 over many keys pass fp32)
@pytest.mark.parametrize("fmt,size", [(f, x) for f in FMTS for x in (1.0, 1e13, 1e25, 1e-30)] + [("e4m3", 5e37)])
@pytest.mark.parametrize("shape", ((1, 2, 1, 3), (1, 320, 320, 2), (2, 24, 1, 2), (1, 8, 1, 8)), ids=str)
@pytest.mark.parametrize("where", ("first", "last", "all", "every second"))
def test_value_rows_of_zeros_count_in_the_sum(fa, fmt, shape, size, where):
    """A row of zeros has the least scale exponent; its weight counts all the same, beside
    values of any size, in the same share and through the merge."""
    B, Hq, Hkv, T = shape
    d, n = 64, 40000 if Hkv == 1 else 700
    g = gen(int(math.log10(size)) + 40)
    cache = fa.KvCache(B, Hkv, n + T, d, fmt)
    k = randn(g, B, Hkv, n + T, d) * 0.5
    v = (randn(g, B, Hkv, n + T, d) + 0.5) * size
    if where == "first":
        v[:, :, : n // 2] = 0
    elif where == "last":
        v[:, :, n // 2:] = 0
    elif where == "all":
        v[:] = 0
    else:
        v[:, :, ::2] = 0
    fa.fa_cache_write(cache, k.bfloat16(), v.bfloat16())
    q = randn(g, B, Hq, T, d).bfloat16()
    lens = [n, n - 5][:B]
    o, lse = fa.fa_decode_tree(cache, q, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check(fa, cache, q, lens, o, lse, 1 / math.sqrt(d), [(b, h) for b in range(B) for h in range(0, Hkv, 97)])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("Hq", (1, 20, 48))
@pytest.mark.parametrize("sign", (1.0, -1.0))
def test_an_infinity_in_a_query_makes_its_row_nan(fa, fmt, d, Hq, sign):
    """Also where every score that the row sees is -inf, which no other row is."""
    cache = fa.KvCache(1, 1, 16, d, fmt)
    k = torch.ones(1, 1, 3, d, dtype=torch.bfloat16, device="cuda")
    fa.fa_cache_write(cache, k, k)
    q = torch.ones(1, Hq, 1, d, dtype=torch.bfloat16, device="cuda")
    q[0, Hq // 2, 0, 5] = sign * math.inf
    lens = torch.tensor([2], dtype=torch.int32, device="cuda")
    o, lse = fa.fa_decode_tree(cache, q, lens=lens)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)
    bad = torch.zeros(Hq, dtype=torch.bool)
    bad[Hq // 2] = True
    assert torch.equal(torch.isnan(lse[0, :, 0]).cpu(), bad)
    assert torch.equal(torch.isnan(o[0, :, 0]).cpu(), bad[:, None].expand(Hq, d))
    # a row that sees nothing has no scores: o = 0 and lse = -inf
    mask = torch.zeros(1, dtype=torch.int64, device="cuda")
    o, lse = fa.fa_decode_tree(cache, q, mask, lens=torch.zeros_like(lens))
    assert not o.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,Hq,Hkv,T,cap", ((5000, 1, 1, 1, 700), (700, 12, 3, 5, 300), (600, 8, 1, 20, 520), (9000, 1, 1, 1, 100)))
def test_batches_of_many_short_sequences(fa, fmt, B, Hq, Hkv, T, cap):
    """Many more pairs than CTAs: each share ends inside some pair, whose parts are merged."""
    d = 64
    g = gen(B)
    cache = fa.KvCache(B, Hkv, cap, d, fmt)
    x = randn(g, B, Hkv, cap, d)
    fa.fa_cache_write(cache, x.bfloat16(), (x.flip(-1) + 0.25).bfloat16())
    lens = torch.randint(0, cap - T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    q = randn(g, B, Hq, T, d).bfloat16()
    o, lse = fa.fa_decode_tree(cache, q, lens=lens)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)
    G = Hq // Hkv
    j = torch.arange(T, device="cuda")
    pos = torch.arange(cap, device="cuda")
    for b0 in range(0, B, 250):
        b = slice(b0, min(b0 + 250, B))
        k = values(cache.k[b], None if cache.k_scale is None else cache.k_scale[b])
        v = values(cache.v[b], None if cache.v_scale is None else cache.v_scale[b])
        qq = q[b].double().reshape(-1, Hkv, G * T, d)
        s = qq @ k.transpose(-1, -2) / math.sqrt(d)
        last = (lens[b, None] + j[None]).repeat(1, G)[:, None, :, None]  # causal drafts
        s = torch.where(pos <= last, s, -math.inf)
        want_lse = torch.logsumexp(s, -1)
        p = torch.softmax(s, -1)
        want, a = p @ v, p @ v.abs()
        ds = 2.0 ** -23 * (d + 8) * (qq.abs() @ k.abs().transpose(-1, -2)).amax(-1) / math.sqrt(d)
        if fmt == "e4m3":
            ds = ds + 2.0 ** -12.8 * qq.abs().amax(-1) * k.abs().sum(-1).amax(-1)[..., None] / math.sqrt(d)
        tol = a * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -18) + 2.0 ** -8 * want.abs()
        assert ((o[b].double().reshape(want.shape) - want).abs() <= tol).all(), b0
        off = (lse[b].double().reshape(want_lse.shape) - want_lse).abs()
        assert (off <= ds + 2.0 ** -20 * (1 + want_lse.abs())).all(), b0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("Hq,T", ((1, 5), (3, 8), (4, 16)))
def test_padded_drafts_that_see_their_own_unwritten_rows(fa, fmt, d, Hq, T):
    """A padded batch over memory that was never written: drafts behind a sequence's own
    see themselves, whose rows and scales hold anything.  The others' results are right."""
    lens, real = [130, 7], T - 2
    cap = 200
    g = gen(T)
    cache = fa.KvCache(2, 1, cap, d, fmt)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(255)  # NaN codes, bf16 NaN, scales of no value
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k, v = (randn(g, 2, 1, cap, d).bfloat16() for _ in range(2))
    fa.fa_cache_write(cache, k, v, lens=torch.zeros_like(n), counts=n + real)
    q = randn(g, 2, Hq, T, d).bfloat16()
    mask = torch.tensor([(2 << t) - 1 if t < real else 1 << t for t in range(T)], device="cuda").repeat(2, 1)
    o, lse = fa.fa_decode_tree(cache, q, mask, lens=n)
    rows = slice(0, real)
    check(fa, cache, q[:, :, rows], lens, o[:, :, rows], lse[:, :, rows], 1 / math.sqrt(d),
          [(0, 0), (1, 0)], mask[:, rows])
