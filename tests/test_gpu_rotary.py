"""The rotation of queries and keys, and the norm before it, on the GPU against their
fp64 definitions: pairs, parts of a head, positions near and far, strides, in place,
the gradients, and a training and a serving step of which they are a part."""
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


def spots(seed, *shape, far=5000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, shape, generator=g, dtype=torch.int32)


def ok(fa):
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)


def check(name, got, want, tol):
    over = (got.cpu().double() - want).abs() - tol
    assert not torch.isnan(over).any() and over.max() <= 1e-30, f"{name}: {float(over.max())} beyond its bound"


# cos and sin are off by at most 2^-22 (the phase cut to 24 bits of a half turn: pi 2^-25;
# sincospif: 2 ulp, 2^-23; the product with the amplitude 2^-24), the products and their sum
# by 3 2^-24 of |x| + |y|, bf16 by 2^-8 of the result
def turn_tol(x, want, rot, interleaved, amplitude=1.0):
    return abs(amplitude) * 2.0 ** -21 * ref.pair_size(x, rot, interleaved) + 1.01 * ref.BF * want.abs()


SHAPES = [
    # d, rot, interleaved, q shape, heads of k
    (128, 128, False, (1, 32, 128), 8), (128, 128, True, (37, 5, 128), 1), (64, 64, False, (200, 12, 64), 12),
    (64, 48, False, (33, 3, 64), 2), (128, 16, True, (5, 9, 128), 3), (128, 80, False, (1000, 4, 128), 4),
    (64, 32, True, (3, 7, 11, 64), 2), (128, 112, False, (2, 32, 1, 128), 8), (64, 16, False, (2, 1, 300, 64), 1),
]


@pytest.mark.parametrize("d,rot,inter,shape,hk", SHAPES, ids=str)
def test_rotation_and_its_gradient(fa, d, rot, inter, shape, hk):
    r = fa.Rotary(d, rot=rot, interleaved=inter, amplitude=1.25)
    ks = (shape[0], hk, d) if len(shape) == 3 else (shape[0], hk, shape[2], d)
    q, k = rnd(1, *shape), rnd(2, *ks, scale=4.0)
    pos = spots(3, shape[0]) if len(shape) == 3 else spots(3, shape[0], shape[2])
    turns = r.turns.cpu()
    for back, call in ((False, fa.fa_rotary), (True, fa.fa_rotary_backward)):
        got = call(r, q.cuda(), k.cuda(), pos.cuda())
        alone = call(r, q.cuda(), positions=pos.cuda())
        ok(fa)
        assert alone[1] is None and torch.equal(alone[0], got[0])
        for name, x, y in (("q", q, got[0]), ("k", k, got[1])):
            want = ref.rotate(x.double(), turns, pos, inter, 1.25, back)
            check(name, y, want, turn_tol(x.double(), want, rot, inter, 1.25))
            assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("inter", (False, True))
def test_positions_of_any_size(fa, inter):
    """As exact at the ends of int32 as at one."""
    pos = torch.tensor([0, 1, -1, 7, 2**20, 2**24 + 1, 10**9 + 7, 2**31 - 1, -2**31], dtype=torch.int32)
    q = rnd(1, len(pos), 3, 128)
    r = fa.Rotary(128, interleaved=inter)
    got, _ = fa.fa_rotary(r, q.cuda(), positions=pos.cuda())
    ok(fa)
    want = ref.rotate(q.double(), r.turns.cpu(), pos, inter)
    check("q", got, want, turn_tol(q.double(), want, 128, inter))
    assert torch.equal(got[0].cpu(), q[0])  # position 0 turns nothing


def test_no_positions_are_the_places_of_the_tokens(fa):
    r = fa.Rotary(64)
    x = rnd(1, 2, 3, 50, 64).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    a, _ = fa.fa_rotary(r, x)
    b, _ = fa.fa_rotary(r, x, positions=pos.expand(2, 50).contiguous())
    y = x[0].transpose(0, 1)
    c, _ = fa.fa_rotary(r, y)
    ok(fa)
    assert torch.equal(a, b) and torch.equal(c, a[0].transpose(0, 1))


def norm_case(fa, d, rot, inter, shape, hk, wdtype):
    r = fa.Rotary(d, rot=rot, interleaved=inter, amplitude=0.9)
    ks = (shape[0], hk, d) if len(shape) == 3 else (shape[0], hk, shape[2], d)
    q, k = rnd(1, *shape), rnd(2, *ks, scale=30.0)
    dq, dk = rnd(3, *shape), rnd(4, *ks)
    wq, wk = (1 + 0.3 * rnd(5, d).float()).to(wdtype), (rnd(6, d).float()).to(wdtype)
    pos = spots(3, shape[0]) if len(shape) == 3 else spots(3, shape[0], shape[2])
    return r, q, k, dq, dk, wq, wk, pos





@pytest.mark.parametrize("wdtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("d,rot,inter,shape,hk", SHAPES, ids=str)
def test_norm_and_rotation_and_their_gradients(fa, d, rot, inter, shape, hk, wdtype):
    """Bounds: 1 / sqrt and the sum under it are off by 2^-19 in all (128 additions of
    2^-24 and two functions), as is the mean of the backward pass; then as above."""
    eps = 1e-5
    r, q, k, dq, dk, wq, wk, pos = norm_case(fa, d, rot, inter, shape, hk, wdtype)
    turns = r.turns.cpu()
    g = [t.cuda() for t in (q, k, dq, dk, pos, wq, wk)]
    y = fa.fa_norm_rotary(r, g[0], g[1], g[4], g[5], g[6], eps=eps)
    b = fa.fa_norm_rotary_backward(r, g[2], g[3], g[0], g[1], g[4], g[5], g[6], eps=eps)
    one = fa.fa_norm_rotary_backward(r, g[2], None, g[0], None, g[4], g[5], eps=eps)
    ok(fa)
    assert one[1] is None and one[3] is None and torch.equal(one[0], b[0])
    for name, x, w, dy, y1, dx, dw in (("q", q, wq, dq, y[0], b[0], b[2]), ("k", k, wk, dk, y[1], b[1], b[3])):
        x, w, dy = x.double(), w.double(), dy.double()
        n = ref.norm(x, w, eps)
        want = ref.rotate(n, turns, pos, inter, 0.9)
        small = 2.0 ** -19 * ref.pair_size(n, rot, inter)
        check(name, y1, want, small + turn_tol(n, want, rot, inter, 0.9))
        back = ref.rotate(dy, turns, pos, inter, 0.9, back=True)
        gx, gw = ref.norm_backward(back, x, w, eps)
        e = 2.0 ** -21 * ref.pair_size(dy, rot, inter) + 2.0 ** -24 * back.abs()  # of the gradient turned back
        inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        xh = (x * inv).abs()
        u, eu = (w * back).abs(), (w.abs() * e)
        big = inv * (eu + xh * (eu * xh).mean(-1, keepdim=True) + 2.0 ** -18 * (u + xh * (u * xh).mean(-1, keepdim=True)))
        check("d" + name, dx, gx, big + 1.01 * ref.BF * gx.abs())
        rows = x.numel() // d
        tol = ((e + (2.0 ** -19 + rows * 2.0 ** -24) * back.abs()) * xh).flatten(0, -2).sum(0)
        check("w" + name, dw, gw, tol)


def test_gradients_are_the_differences(fa):
    """The norm's and rotation's gradients against central differences of the fp64
    definition: truncation of order h^2, far below the bf16 rounding of the results."""
    d, rot, eps, h = 64, 48, 1e-3, 1e-4
    r = fa.Rotary(d, rot=rot)
    x, dy, w, pos = rnd(1, 4, 2, d), rnd(2, 4, 2, d), (1 + 0.3 * rnd(3, d).float()), spots(4, 4)
    dx, _, dw, _ = fa.fa_norm_rotary_backward(r, dy.cuda(), None, x.cuda(), None, pos.cuda(), w.cuda(), eps=eps)
    ok(fa)
    turns = r.turns.cpu()
    f = lambda x, w: (ref.rotate(ref.norm(x, w, eps), turns, pos, False) * dy.double()).sum()  # noqa: E731
    x, w = x.double(), w.double()
    for t, e in ((0, 0), (1, 20), (2, 47), (3, 63)):
        a = torch.zeros_like(x)
        a[t, 1, e] = h
        diff = (f(x + a, w) - f(x - a, w)) / (2 * h)
        assert abs(dx[t, 1, e].cpu().double() - diff) <= 2.0 ** -8 * abs(diff) + 2e-5
        b = torch.zeros_like(w)
        b[e] = h
        diff = (f(x, w + b) - f(x, w - b)) / (2 * h)
        assert abs(dw[e].cpu().double() - diff) <= 1e-5 * (1 + abs(diff))


@pytest.mark.parametrize("d", (64, 128))
def test_strides_and_in_place(fa, d):
    n, Hq, Hkv = 77, 6, 2
    r = fa.Rotary(d, rot=d // 2)
    pos = spots(1, n).cuda()
    x = rnd(2, n, Hq + 2 * Hkv, d).cuda()
    w = (1 + 0.1 * rnd(3, d).float()).cuda()
    q, k = x[:, :Hq], x[:, Hq: Hq + Hkv]
    want = fa.fa_norm_rotary(r, q.contiguous(), k.contiguous(), pos, w, w)
    plain = fa.fa_rotary(r, q.contiguous(), k.contiguous(), pos)
    big = torch.full((n, Hq + 3, d + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    q_out, k_out = big[:, 1: 1 + Hq, 8:], torch.empty(Hkv, n, d, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    fa.fa_norm_rotary(r, q, k, pos, w, w, q_out=q_out, k_out=k_out)
    ok(fa)
    assert torch.equal(q_out, want[0]) and torch.equal(k_out, want[1])
    assert (big[:, 0] == 9.0).all() and (big[:, 1 + Hq:] == 9.0).all() and (big[:, :, :8] == 9.0).all()
    # [B, heads, N, d] as the rest of the library takes it, by a view of the same tensor
    q4, k4 = q.transpose(0, 1)[None], k.transpose(0, 1)[None]
    a = fa.fa_norm_rotary(r, q4, k4, pos[None], w, w)
    # in place, both calls
    y = x.clone()
    fa.fa_rotary(r, y[:, :Hq], y[:, Hq: Hq + Hkv], pos, q_out=y[:, :Hq], k_out=y[:, Hq: Hq + Hkv])
    z = x.clone()
    fa.fa_norm_rotary(r, z[:, :Hq], z[:, Hq: Hq + Hkv], pos, w, w, q_out=z[:, :Hq], k_out=z[:, Hq: Hq + Hkv])
    ok(fa)
    assert torch.equal(a[0][0].transpose(0, 1), want[0]) and torch.equal(a[1][0].transpose(0, 1), want[1])
    assert torch.equal(y[:, :Hq], plain[0]) and torch.equal(y[:, Hq: Hq + Hkv], plain[1])
    assert torch.equal(z[:, :Hq], want[0]) and torch.equal(z[:, Hq: Hq + Hkv], want[1])
    for t in (y, z):
        assert torch.equal(t[:, Hq + Hkv:], x[:, Hq + Hkv:])
    dq, dk = rnd(5, n, Hq, d).cuda(), rnd(6, n, Hkv, d).cuda()
    g = fa.fa_norm_rotary_backward(r, dq, dk, q, k, pos, w, w)
    g2 = fa.fa_norm_rotary_backward(r, dq, dk, q, k, pos, w, w, dq_in=dq, dk_in=dk)
    ok(fa)
    assert all(torch.equal(u, v) for u, v in zip(g, g2))


def test_rows_keep_to_themselves(fa):
    """NaN and infinity in one row stay there; a row of zeros has a finite norm."""
    r = fa.Rotary(128)
    x, w = rnd(1, 40, 8, 128).cuda(), torch.ones(128, device="cuda")
    want, _ = fa.fa_norm_rotary(r, x, None, None, w)
    y = x.clone()
    y[3, 2, 5], y[7, 0, 0], y[9, 1] = math.nan, math.inf, 0.0
    got, _ = fa.fa_norm_rotary(r, y, None, None, w)
    ok(fa)
    keep = torch.ones(40, 8, dtype=torch.bool, device="cuda")
    keep[3, 2] = keep[7, 0] = keep[9, 1] = False
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[3, 2]).all() and (got[9, 1] == 0).all()


def test_many_tokens_of_few_heads(fa):
    """Weight gradients over many rows, and rows that do not fill a warp."""
    n, d = 30000, 64
    r = fa.Rotary(d)
    x, dy, w = rnd(1, n, 1, d), rnd(2, n, 1, d), 1 + 0.2 * rnd(3, d).float()
    runs = [fa.fa_norm_rotary_backward(r, dy.cuda(), dy.cuda(), x.cuda(), x.cuda(), None, w.cuda(), w.cuda()) for _ in range(2)]
    ok(fa)
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    back = ref.rotate(dy.double(), r.turns.cpu(), torch.arange(n, dtype=torch.int32), False, back=True)
    gx, gw = ref.norm_backward(back, x.double(), w.double(), 1e-6)
    for dw in runs[0][2:]:
        assert (dw.cpu().double() - gw).norm() <= 1e-5 * gw.norm()
    assert (runs[0][0].cpu().double() - gx).norm() <= 4e-3 * gx.norm()


def test_captured_and_on_another_stream(fa):
    r = fa.Rotary(128, rot=64, interleaved=True)
    q, k, w = rnd(1, 9, 8, 128).cuda(), rnd(2, 9, 2, 128).cuda(), torch.ones(128, device="cuda")
    pos, ws = spots(3, 9).cuda(), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        y = fa.fa_norm_rotary(r, q, k, pos, w, w)
        return (*y, *fa.fa_norm_rotary_backward(r, *y, q, k, pos, w, w, workspace=ws), *fa.fa_rotary(r, q, k, pos))

    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    ok(fa)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    pos.add_(100)
    graph.replay()
    again = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = fa.fa_norm_rotary(r, q, k, pos, w, w, stream=s)
    z = fa.fa_rotary(r, q, k, pos, stream=s.cuda_stream)
    ok(fa)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert torch.equal(y[0], again[0]) and torch.equal(y[1], again[1])
    assert torch.equal(z[0], again[6]) and torch.equal(z[1], again[7])


def test_training_step(fa):
    """Projection's output -> norm and rotation -> packed attention -> backward, against
    autograd on the fp64 definition (2 % of each gradient's norm: four bf16 roundings
    a value on the way there and back)."""
    lens, Hq, Hkv, d, eps = [50, 1, 130, 0, 77], 4, 2, 64, 1e-6
    cu = ref.starts(lens)
    n = cu[-1]
    r = fa.Rotary(d, rot=32)
    x, dO = rnd(1, n, Hq + 2 * Hkv, d).cuda(), rnd(2, n, Hq, d).cuda()
    wq, wk = ((1 + 0.2 * rnd(s, d).float()).cuda() for s in (3, 4))
    pos = torch.cat([torch.arange(m) for m in lens]).to(torch.int32)
    cuda_cu, p = torch.tensor(cu, dtype=torch.int32, device="cuda"), pos.cuda()
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv:]
    qr, kr = fa.fa_norm_rotary(r, q, k, p, wq, wk)
    o, lse = fa.fa_forward_packed(qr, kr, v, cuda_cu, causal=True)
    dx = torch.empty_like(x)
    dq, dk, _ = fa.fa_backward_packed(qr, kr, v, o, dO, lse, cuda_cu, causal=True, dv=dx[:, Hq + Hkv:])
    _, _, dwq, dwk = fa.fa_norm_rotary_backward(r, dq, dk, q, k, p, wq, wk, dq_in=dx[:, :Hq], dk_in=dx[:, Hq: Hq + Hkv])
    ok(fa)
    X = x.cpu().double().requires_grad_()
    W = [w.cpu().double().requires_grad_() for w in (wq, wk)]
    turns = r.turns.cpu()

    def turned(t, w):
        y = ref.norm(t, w, eps)
        a = 2 * math.pi * ref.fractions(turns, pos)[:, None]
        u, z = y[..., :16], y[..., 16:32]
        return torch.cat([u * a.cos() - z * a.sin(), z * a.cos() + u * a.sin(), y[..., 32:]], -1)

    Q, K, V = turned(X[:, :Hq], W[0]), turned(X[:, Hq: Hq + Hkv], W[1]), X[:, Hq + Hkv:]
    O = []
    for a, b in zip(cu, cu[1:]):
        for h in range(Hq):
            s = (Q[a:b, h] @ K[a:b, h // 2].T) * d ** -0.5
            s = s.masked_fill(~ref.seen(b - a, b - a, True), -math.inf)
            O.append((torch.softmax(s, -1) @ V[a:b, h // 2] * dO[a:b, h].cpu().double()).sum())
    torch.stack(O).sum().backward()
    for got, want in ((dx, X.grad), (dwq, W[0].grad), (dwk, W[1].grad)):
        assert (got.cpu().double() - want).norm() <= 0.02 * want.norm()


def test_serving_step(fa):
    """A prompt by the packed attention, then single tokens: norm and rotation, cache,
    decode; each token gets what one packed call over all of it gives."""
    Hq, Hkv, d, prompt, more = 8, 2, 128, 150, 3
    n = prompt + more
    r = fa.Rotary(d)
    w = torch.ones(d, device="cuda")
    q, k, v = rnd(1, n, Hq, d).cuda(), rnd(2, n, Hkv, d).cuda(), rnd(3, n, Hkv, d).cuda()
    qr, kr = fa.fa_norm_rotary(r, q, k, None, w, w)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want, want_lse = fa.fa_forward_packed(qr, kr, v, cu, causal=True)
    cache = fa.KvCache(1, Hkv, 256, d, "bf16")
    heads = lambda t: t.transpose(0, 1)[None].contiguous()  # noqa: E731
    fa.fa_cache_write(cache, heads(kr[:prompt]), heads(v[:prompt]))
    cache.lens.fill_(prompt)
    for t in range(prompt, n):
        at = torch.full((1, 1), t, dtype=torch.int32, device="cuda")
        q1, k1 = fa.fa_norm_rotary(r, q[t][None, :, None], k[t][None, :, None], at, w, w)
        assert torch.equal(q1[0, :, 0], qr[t]) and torch.equal(k1[0, :, 0], kr[t])
        fa.fa_cache_write(cache, k1, v[t][None, :, None].contiguous())
        o, lse = fa.fa_decode_tree(cache, q1)
        cache.lens.add_(1)
        ok(fa)
        torch.testing.assert_close(lse[0, :, 0], want_lse[:, t], atol=2e-5, rtol=0)
        assert (o[0, :, 0].float() - want[t].float()).norm() <= 8e-3 * want[t].float().norm()
    # the same tokens as a chunk over the keys before them
    cq, ck = torch.tensor([0, more], dtype=torch.int32, device="cuda"), cu
    o, _ = fa.fa_forward_packed(qr[prompt:], kr, v, cq, ck, causal=True)
    ok(fa)
    assert (o.float() - want[prompt:].float()).norm() <= 5e-3 * want[prompt:].float().norm()


@pytest.mark.slow
def test_tokens_beyond_4_GiB(fa):
    """The last of 17 million tokens, 4.4 GB into each tensor."""
    n, d = 17_000_000, 128
    r = fa.Rotary(d)
    g = torch.Generator().manual_seed(3)
    x, y = (torch.randn(50, 1, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, dq = (torch.zeros(n, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[-50:], dq[-50:] = x, y
    last = pos[-50:].contiguous()
    assert torch.equal(fa.fa_rotary(r, q, None, pos)[0][-50:], fa.fa_rotary(r, x, None, last)[0])
    assert torch.equal(fa.fa_norm_rotary(r, q, None, pos, w)[0][-50:], fa.fa_norm_rotary(r, x, None, last, w)[0])
    far, _, dw, _ = fa.fa_norm_rotary_backward(r, dq, None, q, None, pos, w)
    near, _, dw1, _ = fa.fa_norm_rotary_backward(r, y, None, x, None, last, w)
    assert torch.equal(far[-50:], near)
    # the same 50 addends in another order: 2^-23 of their sizes' sum each time
    assert ((dw - dw1).abs() <= 100 * 2.0 ** -23 * 50 * 6 * 6).all()
    assert (torch.cuda.synchronize(), fa.fa_get_device_error())[1] == (0, 0)


@pytest.mark.parametrize("eps", (1e-6, 0.0, 1e-30))
@pytest.mark.parametrize("d", (64, 128))
def test_norm_of_the_largest_and_smallest_rows(fa, d, eps):
    """Rows whose squares leave fp32, or (where eps does not hide them) vanish in it, beside
    ordinary ones; their gradients."""
    r = fa.Rotary(d)
    g = torch.Generator().manual_seed(8)
    n = 9
    sizes = torch.tensor([1.0, 2.0 ** 126, 2.0 ** 70, 2.0 ** 61, 1.0, 2.0 ** -40, 2.0 ** -70, 2.0 ** -120, 2.0 ** 10])
    x = (torch.randn(n, 3, d, generator=g).clamp(-1.9, 1.9) * sizes[:, None, None]).to(torch.bfloat16)
    dy = torch.randn(n, 3, d, generator=g).to(torch.bfloat16)
    w = torch.linspace(0.5, 1.5, d)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")  # (no turn: the norm alone)
    y, _ = fa.fa_norm_rotary(r, x.cuda(), None, pos, w.cuda(), eps=eps)
    # the gradient of rows below 2^-20 or so leaves bf16 for the smallest eps: those of the others
    keep = sizes >= 2.0 ** -40
    dx, _, dw, _ = fa.fa_norm_rotary_backward(r, dy.cuda(), None, x.cuda(), None, pos, w.cuda(), eps=eps)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)
    xd, gd, wd = x.double(), dy.double(), w.double()
    s = (xd.square().mean(-1, keepdim=True) + float(torch.tensor(eps))) ** -0.5
    want = wd * xd * s
    # one rounding to bf16, and 2^-18 for the fp32 steps before it
    assert ((y.cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs() + 2.0 ** -133).all()
    h = xd * s
    inner = (wd * gd * h).mean(-1, keepdim=True)
    wdx = s * (wd * gd - h * inner)
    room = (2.0 ** -8) * wdx.abs() + 2.0 ** -16 * s * ((wd * gd).abs() + (h * inner).abs()) + 2.0 ** -133
    assert ((dx.cpu().double() - wdx).abs() <= room)[keep].all()
    wdw = (gd * h).sum((0, 1))
    assert ((dw.cpu().double() - wdw).abs() <= 2.0 ** -16 * (gd * h).abs().sum((0, 1))).all()
