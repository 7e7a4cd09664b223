"""Attention over packed sequences on the GPU against its fp64 definition: lengths
from zero on, grouped heads, chunks over earlier keys, strides, rows that see nothing,
what lies outside the sequences, and its use in graphs and on streams."""
import math

import pytest
import torch

import packed_ref as ref

pytestmark = pytest.mark.gpu


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


def ok(fa):
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)


def check(name, got, want, tol):
    got, fine = got.cpu().double(), ~torch.isnan(want)
    assert torch.equal(torch.isneginf(got) & fine, torch.isneginf(want)), name
    fine &= ~torch.isneginf(want)
    assert not torch.isnan(got[fine]).any(), name
    over = ((got - want).abs() - tol)[fine]
    assert over.numel() == 0 or over.max() <= 1e-30, f"{name}: {over.max()} beyond its bound"
    norm = want[fine].norm()
    if norm > 0 and fine.sum() > 1000:
        print(name, float((got - want)[fine].norm() / norm))


def run_both(fa, lens_q, lens_k, Hq, Hkv, d, causal, seed=1, scale=None):
    cu_q = ref.starts(lens_q)
    cu_k = cu_q if lens_k is None else ref.starts(lens_k)
    q, k, v = rnd(seed, cu_q[-1], Hq, d), rnd(seed + 1, cu_k[-1], Hkv, d), rnd(seed + 2, cu_k[-1], Hkv, d)
    dO = rnd(seed + 3, cu_q[-1], Hq, d)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    want = ref.attention(q, k, v, cu_q, cu_k, scale, causal, dO, tol=True)
    g = [t.cuda() for t in (q, k, v, dO)]
    cq, ck = i32(cu_q), None if lens_k is None else i32(cu_k)
    o, lse = fa.fa_forward_packed(g[0], g[1], g[2], cq, ck, causal=causal, scale=scale)
    dq, dk, dv = fa.fa_backward_packed(g[0], g[1], g[2], o, g[3], lse, cq, ck, causal=causal, scale=scale)
    ok(fa)
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got, want[name], want["tol"][name])


LENGTHS = [
    [1], [2], [17], [127], [128], [129], [300], [0, 5], [1, 0, 0, 3], [64, 1, 32, 0, 33, 2],
    [255, 256, 257], [513, 1, 260, 0], [1] * 40,
]


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_lengths(fa, lens, d, causal):
    run_both(fa, lens, None, 4, 2, d, causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (7, 1), (8, 1), (14, 2), (16, 1), (17, 1), (20, 1), (24, 1),
                                    (32, 1), (12, 4)])
@pytest.mark.parametrize("d", (64, 128))
def test_groups_of_heads(fa, Hq, Hkv, d):
    run_both(fa, [70, 131, 0, 9], None, Hq, Hkv, d, True, seed=5)
    run_both(fa, [33, 150], None, Hq, Hkv, d, False, seed=6)


CHUNKS = [
    ([1], [1000]), ([5, 40, 130], [105, 40, 830]), ([16, 300], [129, 301]), ([1, 0, 2], [64, 50, 65]),
    # fewer keys than queries: the first queries see nothing; no keys at all
    ([130, 70], [20, 0]), ([5], [0]), ([300, 3], [299, 128]),
]


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 64), (8, 2, 128), (7, 1, 128)])
@pytest.mark.parametrize("lens_q,lens_k", CHUNKS, ids=str)
def test_chunks_over_other_keys(fa, lens_q, lens_k, Hq, Hkv, d, causal):
    run_both(fa, lens_q, lens_k, Hq, Hkv, d, causal, seed=9)


@pytest.mark.parametrize("d", (64, 128))
def test_long_sequences(fa, d):
    run_both(fa, [1500, 2, 900], None, 4, 1, d, True, seed=11)
    run_both(fa, [257], [3001], 4, 2, d, True, seed=12)


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 1), (7, 1)])
@pytest.mark.parametrize("lens_q,lens_k,causal", [
    ([2100, 1030], None, True), ([1537], None, True), ([1300, 1200], None, False), ([1100], [3000], True), ([1300, 0, 1900], [1290, 5, 1900], True)],
    ids=str)
def test_sequences_long_enough_for_two_blocks_to_share_their_tiles(fa, lens_q, lens_k, causal, Hq, Hkv):
    run_both(fa, lens_q, lens_k, Hq, Hkv, 128, causal, seed=30)


@pytest.mark.parametrize("d", (64, 128))
def test_thousands_of_short_sequences(fa, d):
    run_both(fa, [b * b % 7 for b in range(2500)], None, 2, 1, d, True, seed=31)
    run_both(fa, [b % 3 for b in range(1100)], [b % 5 for b in range(1100)], 2, 2, d, False, seed=32)


@pytest.mark.parametrize("scale", (1e-3, 1.0, 4.0))
def test_scales(fa, scale):
    run_both(fa, [200, 31], None, 4, 2, 64, True, seed=13, scale=scale)


@pytest.mark.parametrize("rise", (0.5, -0.5))
def test_scores_that_rise_and_fall_along_the_keys(fa, rise):
    """The running maximum moves in every tile, or never after the first."""
    n, d = 700, 64
    q, k, v, dO = (rnd(20 + i, n, 2, d) for i in range(4))
    q[..., 0] = 8.0
    k[..., 0] = (torch.arange(n)[:, None] * rise / 8).to(torch.bfloat16)
    cu = [0, n]
    want = ref.attention(q, k, v, cu, cu, 0.125, True, dO, tol=True)
    g = [t.cuda() for t in (q, k, v, dO)]
    o, lse = fa.fa_forward_packed(*g[:3], i32(cu), causal=True)
    grads = fa.fa_backward_packed(*g[:3], o, g[3], lse, i32(cu), causal=True)
    ok(fa)
    for name, got in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)):
        check(name, got, want[name], want["tol"][name])


@pytest.mark.parametrize("layout", ("fused", "heads_first", "gaps"))
@pytest.mark.parametrize("d", (64, 128))
def test_strides(fa, layout, d):
    """Parts of one tensor, [heads][tokens][d], rows with gaps: inputs and outputs."""
    cu, Hq, Hkv = [0, 130, 131, 290], 6, 2
    n, scale = cu[-1], 0.1

    def room(heads, name=[0]):
        if layout == "heads_first":
            return torch.full((heads, n, d), 9.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
        big = torch.full((n + 2, heads + 3, d + 24), 9.0, dtype=torch.bfloat16, device="cuda")
        return big[1:-1, 2:-1, 8: 8 + d]

    q, k, v, dO = rnd(1, n, Hq, d), rnd(2, n, Hkv, d), rnd(3, n, Hkv, d), rnd(4, n, Hq, d)
    want = ref.attention(q, k, v, cu, cu, scale, True, dO, tol=True)
    if layout == "fused":
        x = torch.cat([q, k, v], 1).cuda()
        y = torch.full_like(x, 9.0)
        gq, gk, gv = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
        dq, dk, dv = y[:, :Hq], y[:, Hq: Hq + Hkv], y[:, Hq + Hkv:]
        o, g = torch.empty(n, Hq, d, dtype=torch.bfloat16, device="cuda"), dO.cuda()
    else:
        gq, gk, gv, o, g = room(Hq), room(Hkv), room(Hkv), room(Hq), room(Hq)
        dq, dk, dv = room(Hq), room(Hkv), room(Hkv)
        for a, b in ((gq, q), (gk, k), (gv, v), (g, dO)):
            a.copy_(b)
    _, lse = fa.fa_forward_packed(gq, gk, gv, i32(cu), causal=True, scale=scale, o=o)
    fa.fa_backward_packed(gq, gk, gv, o, g, lse, i32(cu), causal=True, scale=scale, dq=dq, dk=dk, dv=dv)
    ok(fa)
    for name, got in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, got, want[name], want["tol"][name])
    if layout == "gaps":
        for t in (o, dq, dk, dv):
            base = t._base
            inside = torch.zeros(base.shape, dtype=torch.bool)
            inside[1:-1, 2:-1, 8: 8 + d] = True
            assert (base.cpu()[~inside] == 9.0).all()


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("causal", (True, False))
def test_what_lies_outside_a_sequence_does_not_reach_it(fa, d, causal):
    """Sequences of NaN and infinities, and tokens of no sequence, between others; what
    lies in no sequence stays as it was."""
    lens, Hq, Hkv = [37, 5, 130, 128, 64, 3], 4, 2
    cu = ref.starts(lens, 7)
    n = cu[-1] + 9
    q, k, v, dO = rnd(1, n, Hq, d), rnd(2, n, Hkv, d), rnd(3, n, Hkv, d), rnd(4, n, Hq, d)
    bad = [slice(0, 7), slice(cu[1], cu[2]), slice(cu[3], cu[4]), slice(cu[-1], n)]
    for t, x in ((q, math.nan), (k, math.inf), (v, math.nan), (dO, -math.inf)):
        for s in bad:
            t[s] = x
    want = ref.attention(*(torch.nan_to_num(t) for t in (q, k, v)), cu, cu, 0.1, causal, torch.nan_to_num(dO), tol=True)
    g = [t.cuda() for t in (q, k, v, dO)]
    o, dq = (torch.full((n, Hq, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dk, dv = (torch.full((n, Hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.full((Hq, n), 9.0, device="cuda")
    fa.fa_forward_packed(*g[:3], i32(cu), causal=causal, scale=0.1, o=o, lse=lse)
    fa.fa_backward_packed(*g[:3], o, g[3], lse, i32(cu), causal=causal, scale=0.1, dq=dq, dk=dk, dv=dv)
    ok(fa)
    for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        w = want[name].clone()
        for s in bad:
            w[s] = math.nan
        check(name, got, w, want["tol"][name])
        assert (got[:7] == 9.0).all() and (got[cu[-1]:] == 9.0).all(), name
    w = want["lse"].clone()
    for s in bad:
        w[:, s] = math.nan
    check("lse", lse, w, want["tol"]["lse"])
    assert (lse[:, :7] == 9.0).all() and (lse[:, cu[-1]:] == 9.0).all()


def test_empty_tensors(fa):
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    kv = rnd(1, 30, 2, 64).cuda()
    cu0, cu = i32([0, 0, 0]), i32([0, 30, 30])
    o, lse = fa.fa_forward_packed(e, kv, kv, cu0, cu)
    dq, dk, dv = fa.fa_backward_packed(e, kv, kv, o, e, lse, cu0, cu)
    ok(fa)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0) and dq.shape == (0, 4, 64)
    assert (dk == 0).all() and (dv == 0).all()
    q, none = rnd(2, 30, 4, 64).cuda(), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.fa_forward_packed(q, none, none, cu, cu0)
    dq, dk, dv = fa.fa_backward_packed(q, none, none, o, q, lse, cu, cu0)
    ok(fa)
    assert (o == 0).all() and torch.isneginf(lse).all() and (dq == 0).all() and dk.shape == (0, 2, 64)


@pytest.mark.parametrize("cu", [[0, 50, 20, 60], [-5, 30, 1000, 60], [60, 0, 60, 60], [2**31 - 1, -2**31, 5, 2**31 - 1],
                                [0, 60, 0, 60]])
def test_starts_that_make_no_sense_stay_inside_the_tensors(fa, cu):
    n, d = 60, 64
    guard = torch.full((3 * n, 4, d), 9.0, dtype=torch.bfloat16, device="cuda")
    o, q = guard[n: 2 * n], rnd(1, n, 4, d).cuda()
    lse_all = torch.full((3, 4, n), 9.0, device="cuda")
    grads = [g.clone() for g in (guard, guard, guard)]
    fa.fa_forward_packed(q, q, q, i32(cu), causal=True, o=o, lse=lse_all[1])
    fa.fa_backward_packed(q, q, q, o, q, lse_all[1], i32(cu), causal=True, dq=grads[0][n: 2 * n], dk=grads[1][n: 2 * n],
                          dv=grads[2][n: 2 * n])
    ok(fa)
    for t in (guard, *grads):
        assert (t[:n] == 9.0).all() and (t[2 * n:] == 9.0).all()
    assert (lse_all[0] == 9.0).all() and (lse_all[2] == 9.0).all()


def test_the_same_call_twice_gives_the_same_bits(fa):
    lens = [1000, 3, 700, 256, 1]
    cu = ref.starts(lens)
    q, k, v, dO = (rnd(i, cu[-1], h, 128).cuda() for i, h in enumerate((8, 2, 2, 8)))
    runs = []
    for _ in range(3):
        o, lse = fa.fa_forward_packed(q, k, v, i32(cu), causal=True)
        runs.append((o, lse, *fa.fa_backward_packed(q, k, v, o, dO, lse, i32(cu), causal=True)))
    ok(fa)
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_the_dense_call_gives_the_same(fa):
    """Equal lengths and heads: fa_forward and fa_backward on [B][H][N][d], within the
    rounding of bf16 results computed twice."""
    B, H, N, d = 2, 3, 260, 64
    q, k, v, dO = (rnd(i, B, H, N, d).cuda() for i in range(4))
    o0, lse0 = fa.fa_forward(q, k, v, causal=True)
    g0 = fa.fa_backward(q, k, v, o0, dO, lse0, causal=True)
    pack = lambda t: t.transpose(1, 2).reshape(B * N, H, d)  # noqa: E731
    cu = i32([0, N, 2 * N])
    o, lse = fa.fa_forward_packed(pack(q), pack(k), pack(v), cu, causal=True)
    g = fa.fa_backward_packed(pack(q), pack(k), pack(v), o, pack(dO), lse, cu, causal=True)
    ok(fa)
    torch.testing.assert_close(lse.view(H, B, N).transpose(0, 1), lse0, atol=2e-5, rtol=0)
    for a, b in zip((o, *g), (o0, *g0)):
        a, b = a.float(), pack(b).float()
        assert (a - b).norm() <= 5e-3 * b.norm()


def test_captured_calls_replay_with_new_lengths_and_share_a_workspace(fa):
    n, Hq, Hkv, d, B = 400, 4, 2, 128, 5
    q, k, v, dO = (rnd(i, n, h, d).cuda() for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    need = fa.fa_backward_packed_workspace_size(B, n, n, Hq, Hkv, d)
    assert need >= fa.fa_forward_packed_workspace_size(B, n, n, Hq, Hkv, d) > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    lens = [[100, 0, 200, 1, 99], [1, 1, 1, 396, 1], [400, 0, 0, 0, 0]]
    cu = i32(ref.starts(lens[0]))

    def step():
        o, lse = fa.fa_forward_packed(q, k, v, cu, causal=True, workspace=ws)
        return (o, lse, *fa.fa_backward_packed(q, k, v, o, dO, lse, cu, causal=True, workspace=ws))

    step()  # an eager run before, as a warm-up
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for ln in lens:
        cu.copy_(i32(ref.starts(ln)))
        for g, out in graphs:
            for t in out:
                t.fill_(7.0)
            g.replay()
        ok(fa)
        want = ref.attention(q.cpu(), k.cpu(), v.cpu(), ref.starts(ln), ref.starts(ln), d ** -0.5, True, dO.cpu(), tol=True)
        for _, out in graphs:
            for name, got in zip(("o", "lse", "dq", "dk", "dv"), out):
                check(name, got, want[name], want["tol"][name])


def test_another_stream_and_raw_handles(fa):
    cu = i32([0, 90, 91, 300])
    q, k, v = (rnd(i, 300, 2, 64).cuda() for i in range(3))
    o0, lse0 = fa.fa_forward_packed(q, k, v, cu, causal=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        o, lse = fa.fa_forward_packed(q, k, v, cu, causal=True, stream=stream)
        g = fa.fa_backward_packed(q, k, v, o, q, lse, cu, causal=True, stream=stream)
        s.synchronize()
        assert torch.equal(o, o0) and torch.equal(lse, lse0)
    with torch.cuda.stream(s):
        g2 = fa.fa_backward_packed(q, k, v, o, q, lse, cu, causal=True)
    ok(fa)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


def test_two_calls_at_once_have_workspaces_of_their_own(fa):
    cu = [i32([0, 1500, 2000]), i32([0, 3, 700, 2000])]
    q, k, v = (rnd(i, 2000, 4, 128).cuda() for i in range(3))
    alone = [fa.fa_forward_packed(q, k, v, c, causal=True) for c in cu]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [[fa.fa_forward_packed(q, k, v, c, causal=True, stream=s) for c, s in zip(cu, streams)] for _ in range(5)]
    ok(fa)
    for pair in both:
        for a, b in zip(pair, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", (64, 128))
def test_a_short_sequence_ends_an_allocation(fa, d):
    """The last token ends a block of memory of its own: nothing behind it is read (what lies there
    need not be mapped)."""
    n, lens = 12 * 2 ** 20 // (2 * d * 2), [200, 70, 3, 1]
    cu = ref.starts(lens)
    near = [rnd(60 + i, cu[-1], 2, d).cuda() for i in range(4)]
    o1, lse1 = fa.fa_forward_packed(*near[:3], i32(cu), causal=True)
    want = fa.fa_backward_packed(*near[:3], o1, near[3], lse1, i32(cu), causal=True)
    whole = [torch.zeros(n, 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for t, s in zip(whole, near):
        t[-cu[-1]:] = s
    at = i32(ref.starts(lens, n - cu[-1]))
    o, lse = fa.fa_forward_packed(*whole[:3], at, causal=True)
    got = fa.fa_backward_packed(*whole[:3], o, whole[3], lse, at, causal=True)
    ok(fa)
    assert torch.equal(o[-cu[-1]:], o1) and torch.equal(lse[:, -cu[-1]:], lse1)
    assert all(torch.equal(a[-cu[-1]:], b) for a, b in zip(got, want))


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("d", (64, 128))
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(fa, d, causal):
    """By the definition, exp(-inf - -inf); a row that sees no key stays 0, and no other changes."""
    lens_q, lens_k, Hq, Hkv = [150, 9], [140, 30], 4, 2
    cu_q, cu_k = ref.starts(lens_q), ref.starts(lens_k)
    q, k, v = rnd(70, cu_q[-1], Hq, d), rnd(71, cu_k[-1], Hkv, d), rnd(72, cu_k[-1], Hkv, d)
    k[:, :, 0] = -k[:, :, 0].abs() - 0.5
    args = [t.cuda() for t in (q, k, v)]
    o0, lse0 = fa.fa_forward_packed(*args, i32(cu_q), i32(cu_k), causal=causal)
    rows, head = [100, 152], 1
    args[0][rows, head] = 0.0
    args[0][rows, head, 0] = math.inf
    o, lse = fa.fa_forward_packed(*args, i32(cu_q), i32(cu_k), causal=causal)
    ok(fa)
    for i in rows:
        assert torch.isnan(o[i, head]).all() and torch.isneginf(lse[head, i])
    o[rows, head], lse[head, rows] = o0[rows, head], lse0[head, rows]
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    if causal:  # queries 0 to 9 of the first sequence see no key
        assert (o[:10] == 0).all() and torch.isneginf(lse[:, :10]).all()


def test_heads_in_chunks(fa):
    """Many items: the heads are taken some at a time (of 32 here six, five times, and two), which
    changes the order of the work and no bit of its results."""
    lens = [241 + b % 31 for b in range(80)]
    cu = ref.starts(lens)
    q, k, v, dO = (rnd(40 + i, cu[-1], 32, 128).cuda() for i in range(4))
    o, lse = fa.fa_forward_packed(q, k, v, i32(cu), causal=True)
    grads = fa.fa_backward_packed(q, k, v, o, dO, lse, i32(cu), causal=True)
    for h in range(0, 32, 8):
        p = slice(h, h + 8)
        o8, lse8 = fa.fa_forward_packed(q[:, p], k[:, p], v[:, p], i32(cu), causal=True)
        g8 = fa.fa_backward_packed(q[:, p], k[:, p], v[:, p], o8, dO[:, p], lse8, i32(cu), causal=True)
        ok(fa)
        assert torch.equal(o[:, p], o8) and torch.equal(lse[p], lse8)
        assert all(torch.equal(a[:, p], b) for a, b in zip(grads, g8))


@pytest.mark.slow
def test_tokens_beyond_4_GiB(fa):
    """The last of 17 million tokens, 4.4 GB into each tensor; about 36 GB of device memory."""
    n, lens, d = 17_000_000, [200, 100], 128
    assert (n - 300) * d * 2 > 2 ** 32
    near = [rnd(50 + i, 300, 1, d).cuda() for i in range(4)]
    cu = ref.starts(lens)
    o1, lse1 = fa.fa_forward_packed(*near[:3], i32(cu), causal=True)
    want = fa.fa_backward_packed(*near[:3], o1, near[3], lse1, i32(cu), causal=True)
    far = [torch.empty(n, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for t, s in zip(far, near):
        t[-300:] = s
    at = i32(ref.starts(lens, n - 300))
    o, lse = fa.fa_forward_packed(*far[:3], at, causal=True)
    got = fa.fa_backward_packed(*far[:3], o, far[3], lse, at, causal=True)
    ok(fa)
    assert torch.equal(o[-300:], o1) and torch.equal(lse[:, -300:], lse1)
    assert all(torch.equal(a[-300:], b) for a, b in zip(got, want))
