"""The key/value cache operators on the GPU against their fp64 definitions:
writing (bit for bit), reading back, committing a path, tree decode, and the
serving loop that uses them together."""
import math

import numpy as np
import pytest
import torch

import kvcache_ref as ref

pytestmark = pytest.mark.gpu
FMTS = ("e4m3", "bf16")


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_16_gb300 as m
    from exact_io_aware_16_gb300 import build

    build.build()
    m.library()
    return m


def rnd(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def state(cache):
    """Everything the cache holds, as bytes."""
    return [t.view(torch.uint8).cpu().clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)
            if t is not None]


def poison(cache):
    """Fill the cache with NaN codes / NaN and scale bytes 255."""
    if cache.format == "e4m3":
        for t in (cache.k, cache.v):
            t.view(torch.uint8).fill_(0x7F)
        cache.k_scale.fill_(255)
        cache.v_scale.fill_(255)
    else:
        cache.k.fill_(math.nan)
        cache.v.fill_(math.nan)


def ok(fa):
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("B,H,N,cap,lens,counts", [
    (1, 1, 1, 16, [0], None),
    (3, 2, 5, 48, [0, 7, 43], [5, 0, 4]),
    (2, 3, 33, 64, [40, 3], None),          # the first sequence runs past the cache
    (2, 1, 9, 32, [-4, 30], [9, 7]),        # positions before and behind the cache
    (1, 5, 129, 144, [15], [128]),
])
def test_write_and_read(fa, fmt, d, B, H, N, cap, lens, counts):
    k, v = rnd(1, B, H, N, d), rnd(2, B, H, N, d, scale=7.0)
    k[0, 0, 0, : d // 2] *= 1000.0
    cache = fa.KvCache(B, H, cap, d, fmt)
    poison(cache)
    before = [x.numpy().copy() for x in state(cache)]
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), lens=i32(lens),
                      counts=None if counts is None else i32(counts))
    ok(fa)
    want = before
    if fmt == "bf16":
        want = [x.view(np.uint16).reshape(B, H, cap, d) for x in want]
    for b in range(B):
        for i in range(N if counts is None else counts[b]):
            p = lens[b] + i
            if not 0 <= p < cap:
                continue
            for j, x in enumerate((k, v)):
                if fmt == "e4m3":
                    c, s = ref.quantise(ref.to64(x[b, :, i]))
                    want[j][b, :, p] = c
                    want[2 + j][b, :, p] = s
                else:
                    want[j][b, :, p] = x[b, :, i].view(torch.int16).numpy().view(np.uint16)
    got = [x.numpy() for x in state(cache)]
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.reshape(-1), w.view(np.uint8).reshape(-1))
    # the rows written come back, zeros elsewhere
    first = [max(x, 0) for x in lens]
    many = [max(0, min(lens[b] + (N if counts is None else counts[b]), cap) - first[b]) for b in range(B)]
    rk, rv = fa.fa_cache_read(cache, N + 3, first=i32(first), counts=i32(many))
    ok(fa)
    kk, vv = ref.cache_values(cache)
    for r, x in ((rk, kk), (rv, vv)):
        w = np.zeros((B, H, N + 3, d))
        for b in range(B):
            w[b, :, : many[b]] = x[b, :, first[b]: first[b] + many[b]]
        np.testing.assert_array_equal(ref.to64(r), w)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
def test_rows_aligned_to_sixteen_bytes(fa, fmt, d):
    """Tensors whose addresses allow 16-byte accesses but none of 32 bytes."""
    B, H, N, cap = 2, 3, 37, 64
    shape = (B, H, N, d)

    def odd(x):
        t = torch.full((x.numel() + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        t[8:-8] = x.cuda().reshape(-1)
        v = t[8:-8].view(x.shape)
        assert v.data_ptr() % 32 == 16
        return t, v

    k, v = rnd(3, *shape), rnd(4, *shape)
    caches = [fa.KvCache(B, H, cap, d, fmt) for _ in range(2)]
    fa.fa_cache_write(caches[0], k.cuda(), v.cuda())
    fa.fa_cache_write(caches[1], odd(k)[1], odd(v)[1])
    for x, y in zip(state(caches[0]), state(caches[1])):
        assert torch.equal(x, y)
    n = i32([N, 11])
    want = fa.fa_cache_read(caches[0], N, counts=n)
    (tk, ok_), (tv, ov) = odd(torch.zeros(shape)), odd(torch.zeros(shape))
    fa.fa_cache_read(caches[0], N, counts=n, k=ok_, v=ov)
    fa.fa_cache_read(caches[1], N, counts=n, k=ok_)  # one of each
    ok(fa)
    assert torch.equal(ok_, want[0]) and torch.equal(ov, want[1])
    for t in (tk, tv):
        assert (t[:8] == 7).all() and (t[-8:] == 7).all()


def special_rows():
    """Rows at the borders of the quantiser, d = 64."""
    rows = []
    for m in (448.0, 452.0, 449.9, 1.75, 1.7578125, 2.0 ** -126, 2.0 ** -133, 3.38e38, 2.9775e38, 1e-30):
        r = torch.linspace(-1, 1, 64) * m
        r[0] = m
        rows.append(r)
    rows.append(torch.zeros(64))
    r = torch.linspace(-3, 3, 64)
    r[5], r[9], r[11] = math.nan, math.inf, -math.inf
    rows.append(r)
    rows.append(torch.full((64,), math.inf))
    rows.append(torch.full((64,), math.nan))
    for k in range(40):  # every midpoint between neighbouring codes of a few binades
        r = torch.full((64,), 448.0)
        r[1:] = torch.arange(63) * 2.0 ** -10 * (k + 1)
        rows.append(r)
    return torch.stack(rows).to(torch.bfloat16)


def test_write_borders(fa):
    rows = special_rows()
    n = rows.shape[0]
    k = rows.reshape(1, 1, n, 64).cuda()
    cache = fa.KvCache(1, 1, (n + 15) // 16 * 16, 64)
    fa.fa_cache_write(cache, k, -k)
    ok(fa)
    for t, s, x in ((cache.k, cache.k_scale, rows), (cache.v, cache.v_scale, -rows)):
        c, e = ref.quantise(ref.to64(x))
        c[(c & 127) == 127] = 127
        np.testing.assert_array_equal(s[0, 0, :n].cpu().numpy(), e)
        np.testing.assert_array_equal(ref.codes_np(t[0, 0, :n]), c)
    rk, _ = fa.fa_cache_read(cache, n, counts=i32([n]))
    ok(fa)
    np.testing.assert_array_equal(ref.to64(rk)[0, 0], ref.cache_values(cache)[0][0, 0, :n])


def test_quantisation_error_is_half_a_step(fa):
    """A value comes back within half an e4m3 step: 2^-4 of itself, or 2^-10 of
    the scale where the code is subnormal."""
    x = rnd(3, 2, 3, 200, 128, scale=3.0)
    cache = fa.KvCache(2, 3, 208, 128)
    fa.fa_cache_write(cache, x.cuda(), x.cuda())
    y, _ = fa.fa_cache_read(cache, 200, counts=i32([200, 200]))
    ok(fa)
    s = 2.0 ** (cache.k_scale[:, :, :200].cpu().numpy().astype(float) - 127)[..., None]
    err = np.abs(ref.to64(y) - ref.to64(x))
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(ref.to64(x)), 2.0 ** -10 * s))


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("B,H,T,cap,lens,n,path", [
    (1, 1, 1, 16, [3], [1], [[0]]),
    (2, 3, 4, 32, [0, 27], [2, 4], [[0, 3, 9, 9], [3, 2, 1, 0]]),
    (3, 9, 8, 48, [5, 40, 45], [8, 0, 7], [[0, 2, 2, 7, 4, 1, 1, 6]] * 3),   # 45 + drafts run out of the cache
    (4, 2, 3, 16, [-1, 17, 16, 2], [2, 2, 2, 9], [[1, 2, 0], [1, 2, 0], [1, 2, 0], [2, -1, 99]]),
    (2, 1, 64, 160, [1, 90], [64, 33], [list(range(63, -1, -1)), list(range(31, 64)) + [0] * 31]),
])
def test_commit(fa, fmt, d, B, H, T, cap, lens, n, path):
    cache = fa.KvCache(B, H, cap, d, fmt)
    x = rnd(4, B, H, cap, d)
    fa.fa_cache_write(cache, x.cuda(), (-3 * x).cuda(), lens=i32([0] * B))
    want = [t.clone() for t in state(cache)]
    olds = [t.clone() for t in want]
    new = list(lens)
    for b in range(B):
        if not 0 <= lens[b] <= cap:
            continue
        m = min(max(n[b], 0), T)
        new[b] = min(lens[b] + m, cap)
        for i in range(m):
            p = path[b][i]
            if 0 <= p < T and lens[b] + p < cap and lens[b] + i < cap:
                for w, o in zip(want, olds):
                    w[b, :, lens[b] + i] = o[b, :, lens[b] + p]
    got = fa.fa_cache_commit(cache, i32(path), i32(n), lens=i32(lens), new_lens=i32([7] * B))
    ok(fa)
    assert got.tolist() == new
    for g, w in zip(state(cache), want):
        assert torch.equal(g, w)


def test_commit_in_place_advances_the_lengths(fa):
    cache = fa.KvCache(3, 2, 32, 64)
    cache.lens.copy_(i32([1, 5, 31]))
    out = fa.fa_cache_commit(cache, torch.zeros((3, 4), dtype=torch.int32, device="cuda"), i32([2, 0, 4]))
    ok(fa)
    assert out.data_ptr() == cache.lens.data_ptr()
    assert cache.lens.tolist() == [3, 5, 32]


# ---------------------------------------------------------------- tree
def make_cache(fa, fmt, B, H, cap, d, lens, T, seed, junk=True):
    """A cache whose positions below min(lens + T, cap) hold rows, with a few
    large key channels; the others hold NaN codes."""
    cache = fa.KvCache(B, H, cap, d, fmt)
    if junk:
        poison(cache)
    n = [min(max(x, 0) + T, cap) for x in lens]
    k = rnd(seed, B, H, max(n), d)
    k[..., 3] *= 6
    v = rnd(seed + 1, B, H, max(n), d) * torch.logspace(-1, 1, max(n)).to(torch.bfloat16)[:, None]
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), lens=i32([0] * B), counts=i32(n))
    return cache


def random_masks(B, T, seed, empty=False):
    g = np.random.RandomState(seed)
    m = [[int(g.randint(0, 1 << 32)) << 32 | int(g.randint(0, 1 << 32)) | 1 << t for t in range(T)] for _ in range(B)]
    m = [[x & ((1 << T) - 1) for x in r] for r in m]
    if empty:
        for r in m:
            r[T // 2] = 0
    return m


def mask_tensor(m):
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in m], dtype=torch.int64, device="cuda")


def check_tree(got_o, got_lse, want):
    o, lse, o_tol, lse_tol = want
    go, gl = ref.to64(got_o), ref.to64(got_lse)
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(go[empty] == 0)
    assert np.all(np.isfinite(go)) and np.all(np.isfinite(gl[~empty]))
    assert np.all(np.abs(gl[~empty] - lse[~empty]) <= lse_tol[~empty]), \
        (np.abs(gl[~empty] - lse[~empty]) / lse_tol[~empty]).max()
    over = np.abs(go - o) - o_tol
    assert np.all(over <= 0), (over.max(), np.unravel_index(over.argmax(), over.shape))


CASES = [  # B, Hq, Hkv, T, cap, lens
    (1, 1, 1, 1, 16, [0]),
    (1, 1, 1, 1, 16, [15]),
    (1, 1, 1, 1, 16, [16]),                  # the cache is full: the draft has no place
    (2, 4, 1, 1, 144, [127, 128]),
    (3, 4, 2, 3, 288, [62, 125, 254]),       # drafts that cross a tile's end
    (2, 8, 8, 5, 301, [0, 299]),             # drafts past the cache's end; an odd capacity
    (1, 33, 1, 1, 80, [64]),                 # 33 rows a key head
    (1, 8, 1, 8, 80, [63]),                  # 64 rows
    (1, 13, 1, 5, 208, [193]),               # 65 rows
    (1, 8, 1, 16, 208, [129]),               # 128 rows
    (2, 3, 1, 43, 208, [10, 128]),           # 129 rows
    (1, 10, 2, 64, 400, [333]),              # 320 rows a key head
    (4, 6, 3, 2, 1040, [1000, 1, 513, 0]),
    (5, 2, 2, 7, 4000, [3993, -5, 5000, 700, 64]),   # lengths outside the cache
    (1, 8, 2, 4, 9600, [9590]),              # split over many CTAs
    (40, 2, 1, 2, 272, [(37 * i) % 271 for i in range(40)]),  # more sequences than a warp's lanes
    (1, 700, 1, 64, 64, [20]),               # more row tiles than CTA slots
    (4, 80, 40, 5, 1200, [1190, 700, 900, 3]),   # several tiles and pairs a CTA, 10 rows
    (3, 192, 32, 4, 2400, [2390, 1800, 2000]),   # 24 rows
    (3, 32, 32, 48, 2400, [2300, 1800, 2011]),   # 48 rows
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}q{c[1]}k{c[2]}t{c[3]}c{c[4]}")
def test_tree_matches_the_definition(fa, fmt, d, case):
    B, Hq, Hkv, T, cap, lens = case
    cache = make_cache(fa, fmt, B, Hkv, cap, d, lens, T, seed=cap + T)
    q = rnd(9, B, Hq, T, d)
    mask = random_masks(B, T, cap, empty=True)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.fa_decode_tree(cache, q.cuda(), mask_tensor(mask), lens=i32(lens))
    ok(fa)
    heads = range(Hq)
    if Hq * T > 300:  # the definition is slow: a sample of the heads
        heads = range(0, Hq, 97 if Hq > 192 else 13)
    k, v = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    for h in heads:
        kv = slice(h // (Hq // Hkv), h // (Hq // Hkv) + 1)
        want = ref.tree(ref.to64(q[:, h:h + 1]), k[:, kv], v[:, kv], lens, mask, scale, fmt,
                        None if vs is None else vs[:, kv], qmax=float(q.abs().max()))
        check_tree(o[:, h:h + 1], lse[:, h:h + 1], want)


@pytest.mark.parametrize("fmt", FMTS)
def test_tree_default_mask_is_causal_and_a_shared_mask_is_shared(fa, fmt):
    B, Hq, Hkv, T, d, cap, lens = 3, 4, 2, 6, 64, 160, [100, 0, 151]
    cache = make_cache(fa, fmt, B, Hkv, cap, d, lens, T, seed=5)
    q = rnd(6, B, Hq, T, d)
    k, v = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    cache.lens.copy_(i32(lens))
    o, lse = fa.fa_decode_tree(cache, q.cuda(), scale=0.3)
    ok(fa)
    chain = [[(2 << t) - 1 for t in range(T)]] * B
    check_tree(o, lse, ref.tree(ref.to64(q), k, v, lens, chain, 0.3, fmt, vs))
    parents = [-1, 0, 0, 1, 2, -1]
    m = fa.tree_mask(parents)
    o, lse = fa.fa_decode_tree(cache, q.cuda(), m.cuda(), scale=0.3)
    ok(fa)
    check_tree(o, lse, ref.tree(ref.to64(q), k, v, lens, [m.tolist()] * B, 0.3, fmt, vs))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("T,Hq", ((5, 2), (33, 4)))
def test_tree_nan_reaches_only_the_rows_that_see_it(fa, fmt, d, T, Hq):
    """NaN in the K and V rows of a draft that some rows do not see, and of one
    that no row sees; infinities too in a bf16 cache."""
    cap, lens = 416, [250, 3]
    cache = make_cache(fa, fmt, 2, 1, cap, d, lens, T, seed=8)
    mask = [[(1 << t) | 1 for t in range(T)] for _ in range(2)]
    mask[0][3] = mask[1][3] = 0b101  # draft 3 is dead, draft 2 is seen by rows 2 and 3
    want = None
    q = rnd(10, 2, Hq, T, d)
    k, v = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    want = ref.tree(ref.to64(q), k, v, lens, mask, 0.125, fmt, vs)
    for b in range(2):
        for t, what in ((cache.k, "k"), (cache.v, "v")):
            row = t[b, 0]
            if fmt == "e4m3":
                row = row.view(torch.uint8)
                row[lens[b] + 3] = 0x7F
                if what == "v":
                    row[lens[b] + 2, 5] = 0xFF
            else:
                row[lens[b] + 3] = math.inf if b else math.nan
                if what == "v":
                    row[lens[b] + 2, 5] = math.nan if b else -math.inf
    o, lse = fa.fa_decode_tree(cache, q.cuda(), mask_tensor(mask), lens=i32(lens), scale=0.125)
    ok(fa)
    got = ref.to64(o).copy()
    for b in range(2):
        bad = got[b, :, 2:4, 5]
        assert np.all(np.isneginf(bad)) if fmt == "bf16" and b == 0 else np.all(np.isnan(bad))
        got[b, :, 2:4, 5] = want[0][b, :, 2:4, 5]
    check_tree(torch.from_numpy(got), lse, want)
    # a NaN key: NaN in the rows that see it, nowhere else
    if fmt == "e4m3":
        cache.k.view(torch.uint8)[1, 0, lens[1] + 4, 7] = 0x7F
    else:
        cache.k[1, 0, lens[1] + 4, 7] = math.nan
    o, lse = fa.fa_decode_tree(cache, q.cuda(), mask_tensor(mask), lens=i32(lens), scale=0.125)
    ok(fa)
    sees = np.array([mask[1][t] >> 4 & 1 for t in range(T)], dtype=bool)
    assert np.all(np.isnan(ref.to64(o)[1][:, sees])) and np.all(np.isnan(ref.to64(lse)[1][:, sees]))
    rest = ref.to64(o)[1][:, ~sees]
    rest[:, 2:4, 5] = 0
    assert np.all(np.isfinite(rest))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d", (64, 128))
def test_tree_nan_query_and_queries_of_many_sizes(fa, fmt, d):
    """A query row with a NaN or an infinity is NaN and leaves the others alone; rows
    whose sizes differ by 2^20 each keep their result."""
    B, Hq, Hkv, T, cap, lens = 1, 6, 2, 4, 300, [290]
    cache = make_cache(fa, fmt, B, Hkv, cap, d, lens, T, seed=70)
    q = rnd(71, B, Hq, T, d) * (2.0 ** torch.linspace(1, -19, Hq * T)).reshape(Hq, T, 1).to(torch.bfloat16)
    k, v = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    chain = [[(2 << t) - 1 for t in range(T)]]
    want = ref.tree(ref.to64(q), k, v, lens, chain, 0.2, fmt, vs)
    q[0, 1, 2, 7], q[0, 4, 0, 3] = math.nan, math.inf
    o, lse = fa.fa_decode_tree(cache, q.cuda(), lens=i32(lens), scale=0.2)
    ok(fa)
    for h, t in ((1, 2), (4, 0)):
        assert torch.isnan(o[0, h, t]).all() and torch.isnan(lse[0, h, t])
        o[0, h, t], lse[0, h, t] = torch.from_numpy(want[0][0, h, t]).cuda(), float(want[1][0, h, t])
    check_tree(o, lse, want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,T", ((2, 6), (4, 12), (6, 40)))
def test_tree_padded_rows_leave_the_others_alone(fa, fmt, Hq, T):
    """Drafts behind a sequence's own hold anything, in q too: the rows of the others
    are within their own bounds, over several tiles of keys."""
    B, Hkv, d, cap, lens = 2, 2, 128, 600, [560, 140]
    cache = make_cache(fa, fmt, B, Hkv, cap, d, lens, T, seed=75)
    q = rnd(76, B, Hq, T, d)
    q[0, :, T - 2] = 1e30
    q[0, :, T - 1] = -3e38
    k, v = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    mask = [[(2 << t) - 1 for t in range(T - 2)] + [0, 0]] * B
    o, lse = fa.fa_decode_tree(cache, q.cuda(), mask_tensor(mask), lens=i32(lens))
    ok(fa)
    t = T - 2
    want = ref.tree(ref.to64(q[:, :, :t]), k, v, lens, [m[:t] for m in mask], 1 / math.sqrt(d), fmt, vs, qmax=math.inf)
    check_tree(o[:, :, :t], lse[:, :, :t], want)


@pytest.mark.parametrize("fmt", FMTS)
def test_tree_large_scores_and_scales(fa, fmt):
    """Rows whose scores spread over hundreds, keys and values over many binades."""
    B, Hq, Hkv, T, d, cap, lens = 1, 4, 1, 3, 128, 704, [690]
    cache = fa.KvCache(B, Hkv, cap, d, fmt)
    n = lens[0] + T
    k = rnd(11, B, Hkv, n, d) * torch.logspace(-3, 1.3, n)[:, None].to(torch.bfloat16)
    v = rnd(12, B, Hkv, n, d) * torch.logspace(2, -2, n)[:, None].to(torch.bfloat16)
    v[:, :, 5] = 0
    fa.fa_cache_write(cache, k.cuda(), v.cuda())
    q = rnd(13, B, Hq, T, d, scale=3.0)
    mask = [[7, 0, 5]]
    o, lse = fa.fa_decode_tree(cache, q.cuda(), mask_tensor(mask), lens=i32(lens))
    ok(fa)
    kk, vv = ref.cache_values(cache)
    vs = None if fmt == "bf16" else cache.v_scale.cpu().numpy()
    check_tree(o, lse, ref.tree(ref.to64(q), kk, vv, lens, mask, 1 / math.sqrt(d), fmt, vs))


@pytest.mark.parametrize("fmt", FMTS)
def test_tree_offsets_beyond_32_bits(fa, fmt):
    """The last head of a cache of more than 2^32 bytes and 2^31 elements."""
    cap, d = (1 << 24) + 16, 128
    cache = fa.KvCache(1, 2, cap, d, fmt)
    n = 300
    k, v = rnd(14, 1, 2, n, d), rnd(15, 1, 2, n, d)
    fa.fa_cache_write(cache, k.cuda(), v.cuda())
    q = rnd(16, 1, 2, 2, d)
    o, lse = fa.fa_decode_tree(cache, q.cuda(), lens=i32([n - 2]))
    ok(fa)
    kk, vv = (x[:, :, :n] for x in ref.cache_values(fa.KvCache.from_tensors(
        cache.k[:, :, :n].contiguous(), cache.v[:, :, :n].contiguous(),
        *(None if s is None else s[:, :, :n].contiguous() for s in (cache.k_scale, cache.v_scale)))))
    vs = None if fmt == "bf16" else cache.v_scale[:, :, :n].cpu().numpy()
    check_tree(o, lse, ref.tree(ref.to64(q), kk, vv, [n - 2], [[1, 3]], 1 / math.sqrt(d), fmt, vs))


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fmt", FMTS)
def test_serving_loop(fa, fmt):
    """Prompt, then rounds of drafts, tree attention and a committed path; every
    round's outputs are those of the definition on the history of the tokens."""
    B, Hq, Hkv, d, cap, T = 3, 8, 2, 64, 512, 7
    cache = fa.KvCache(B, Hkv, cap, d, fmt)
    prompt = [200, 1, 65]
    k, v = rnd(20, B, Hkv, 200, d), rnd(21, B, Hkv, 200, d)
    fa.fa_cache_write(cache, k.cuda(), v.cuda(), counts=i32(prompt))
    cache.lens.copy_(i32(prompt))
    hist = [[(k[b, :, i], v[b, :, i]) for i in range(prompt[b])] for b in range(B)]
    parents = [-1, 0, 0, 1, 2, 3, 3]
    m = fa.tree_mask(parents)
    paths = [[0, 1, 3, 6], [0, 2, 4], [0]]
    for step in range(4):
        dk, dv, q = (rnd(30 + 3 * step + i, B, h, T, d) for i, h in ((0, Hkv), (1, Hkv), (2, Hq)))
        fa.fa_cache_write(cache, dk.cuda(), dv.cuda())
        o, lse = fa.fa_decode_tree(cache, q.cuda(), m.cuda())
        lens = [len(h) for h in hist]
        assert cache.lens.tolist() == lens
        # the definition, on a cache rebuilt from the tokens
        full = fa.KvCache(B, Hkv, cap, d, fmt)
        hk = torch.zeros(B, Hkv, cap, d, dtype=torch.bfloat16)
        hv = hk.clone()
        for b in range(B):
            for i, (x, y) in enumerate(hist[b] + [(dk[b, :, t], dv[b, :, t]) for t in range(T)]):
                hk[b, :, i], hv[b, :, i] = x, y
        fa.fa_cache_write(full, hk.cuda(), hv.cuda())
        kk, vv = ref.cache_values(full)
        vs = None if fmt == "bf16" else full.v_scale.cpu().numpy()
        check_tree(o, lse, ref.tree(ref.to64(q), kk, vv, lens, [m.tolist()] * B, 0.125, fmt, vs))
        path = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            p = paths[(b + step) % 3]
            path[b, : len(p)] = torch.tensor(p)
            hist[b] += [(dk[b, :, t], dv[b, :, t]) for t in p]
        fa.fa_cache_commit(cache, path.cuda(), i32([len(paths[(b + step) % 3]) for b in range(B)]))
    rk, rv = fa.fa_cache_read(cache, cap)
    ok(fa)
    for b in range(B):
        n = len(hist[b])
        for r, j in ((rk, 0), (rv, 1)):
            x = ref.to64(torch.stack([h[j] for h in hist[b]], 1))
            want = x if fmt == "bf16" else ref.dequantise(*ref.quantise(x))
            np.testing.assert_array_equal(ref.to64(r)[b, :, :n], want)
            assert not r[b, :, n:].any()


@pytest.mark.parametrize("fmt", FMTS)
def test_captured_step_replays_with_new_lengths(fa, fmt):
    """One decode step (write, attend, commit) captured in a graph and replayed:
    the lengths live on the device, so each replay continues the last."""
    B, Hq, Hkv, d, cap = 2, 4, 2, 128, 400
    cache, eager = fa.KvCache(B, Hkv, cap, d, fmt), fa.KvCache(B, Hkv, cap, d, fmt)
    k, v, q = (torch.zeros(B, h, 1, d, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    path = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    one = i32([1] * B)
    ws = torch.empty(max(256, fa.fa_decode_tree_workspace_size(cache, Hq, 1)), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")

    def step(c, o, lse, w):
        fa.fa_cache_write(c, k, v)
        fa.fa_decode_tree(c, q, o=o, lse=lse, workspace=w)
        fa.fa_cache_commit(c, path, one)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cache, o, lse, ws)  # warm-up
    torch.cuda.current_stream().wait_stream(s)
    cache.lens.copy_(i32([300, 0]))
    eager.lens.copy_(i32([300, 0]))
    for c in (cache, eager):
        hk = rnd(40, B, Hkv, 300, d).cuda()
        fa.fa_cache_write(c, hk, hk, lens=i32([0, 0]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(cache, o, lse, ws)
    for i in range(5):
        for j, t in enumerate((k, v, q)):
            t.copy_(rnd(50 + 3 * i + j, *t.shape))
        g.replay()
        oe, le = torch.empty_like(o), torch.empty_like(lse)
        step(eager, oe, le, None)
        ok(fa)
        assert torch.equal(o, oe) and torch.equal(lse, le)
        assert cache.lens.tolist() == eager.lens.tolist() == [301 + i, 1 + i]


def test_tree_on_two_streams_and_repeated(fa):
    """Calls that overlap on two streams, each with its own workspace, and
    repeated calls give the same bits."""
    B, Hq, Hkv, T, d, cap = 2, 8, 2, 8, 128, 4096
    lens = [4000, 1234]
    cache = make_cache(fa, "e4m3", B, Hkv, cap, d, lens, T, seed=60)
    q = rnd(61, B, Hq, T, d).cuda()
    n = i32(lens)
    want = fa.fa_decode_tree(cache, q, lens=n)
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        with torch.cuda.stream(ss[i % 2]):
            got.append(fa.fa_decode_tree(cache, q, lens=n))
    ok(fa)
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("Hkv", (1, 8))
@pytest.mark.parametrize("T", (1, 5, 24))
def test_tree_one_workspace_for_many_calls(fa, Hkv, T):
    """One workspace, its contents arbitrary at first, serves calls of changing lengths
    one after the other: each gives the bits of a call with a workspace of its own."""
    B, d, cap = 3, 128, 6000
    cache = make_cache(fa, "e4m3", B, Hkv, cap, d, [cap] * B, T, seed=80, junk=False)
    q = rnd(81, B, 4 * Hkv, T, d).cuda()
    ws = torch.full((fa.fa_decode_tree_workspace_size(cache, 4 * Hkv, T),), 0xA5, dtype=torch.uint8, device="cuda")
    g = np.random.RandomState(82)
    got, want = [], []
    for i in range(40):
        n = i32([int(x) for x in g.randint(0, cap - T, B)])
        got.append(fa.fa_decode_tree(cache, q, lens=n, workspace=ws))
        want.append(fa.fa_decode_tree(cache, q, lens=n))
    ok(fa)
    for (o, lse), (o2, lse2) in zip(got, want):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_graphs_share_a_workspace(fa):
    """Two captured calls of different shapes on one workspace, replayed in turn."""
    d, cap, T = 128, 5000, 12
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    calls = []
    for fmt, B, Hkv, seed in (("e4m3", 1, 1, 100), ("bf16", 2, 4, 101)):
        cache = make_cache(fa, fmt, B, Hkv, cap, d, [cap] * B, T, seed=seed, junk=False)
        q, n = rnd(seed + 10, B, 2 * Hkv, T, d).cuda(), i32([4900] * B)
        assert fa.fa_decode_tree_workspace_size(cache, 2 * Hkv, T) <= ws.numel()
        fa.fa_decode_tree(cache, q, lens=n, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fa.fa_decode_tree(cache, q, lens=n, workspace=ws)
        calls.append((cache, q, n, g, out))
    for i in range(6):
        for cache, q, n, g, (o, lse) in calls:
            n.fill_(4900 - 700 * i)
            g.replay()
            oe, le = fa.fa_decode_tree(cache, q, lens=n)
            ok(fa)
            assert torch.equal(o, oe) and torch.equal(lse, le)


def test_tree_on_a_raw_stream_allocates_there(fa):
    """A call given a stream by its handle: its own tensors belong to that stream."""
    cache = make_cache(fa, "bf16", 1, 2, 2000, 64, [1900], 4, seed=90)
    q, n = rnd(91, 1, 4, 4, 64).cuda(), i32([1900])
    want = fa.fa_decode_tree(cache, q, lens=n)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        o, lse = fa.fa_decode_tree(cache, q, lens=n, stream=stream)
        k, v = fa.fa_cache_read(cache, 10, counts=n, stream=stream)
        ok(fa)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert torch.equal(k, cache.k[:, :, :10]) and torch.equal(v, cache.v[:, :, :10])
