"""How exact the gradients of packed attention are where bf16 tells most: scores so sharp that few
keys share a row, and keys that all lie far to one side, whose common part drops out of dq.

A value rounded to bf16 is off by 2^-8 of its leading bit at most, evenly spread: with leading digits
spread over their logarithm, 2^-8 / sqrt(3) * sqrt((1 / ln 2) * integral_1^2 x^-3 dx) = 0.425 * 2^-8
of the value in the root mean square.  dS is rounded once, then dq and dk once, all independently of
each other, so that the squares add up: for dq sum_j (0.425 * 2^-8 scale dS_ij K_jc)^2 + (0.425 * 2^-8
dq_ic)^2.  All other steps are in fp32, a hundred times finer.  An error of D, which dS has in common
along a row, would come on top of that: of a D from the bf16 o alone 0.34 to 0.7 times as much.
"""
import math

import pytest
import torch

import packed_ref as ref

pytestmark = pytest.mark.gpu

RMS = 0.425 * 2.0 ** -8


@pytest.fixture(scope="module")
def fa():
    import exact_io_aware_16_gb300 as m
    from exact_io_aware_16_gb300 import build

    build.build()
    m.library()
    return m


def inputs(kind, n, Hq, Hkv, d):
    g = torch.Generator().manual_seed(17)
    q, k, v, dO = (torch.randn(n, h, d, generator=g) for h in (Hq, Hkv, Hkv, Hq))
    if kind == "sharp":
        q, k = 2 * q, 2 * k
    elif kind == "offset":
        k = k + 20
    elif kind == "channels":
        k[..., :4] += 20
    return [t.to(torch.bfloat16) for t in (q, k, v, dO)]


CASES = [
    # scores, lengths, query and key heads, d, causal: one head a tile, two, three and four, short and long
    ("sharp", [2048], 2, 2, 128, True), ("sharp", [1500, 548], 4, 2, 128, True), ("sharp", [1100], 3, 1, 128, False),
    ("sharp", [3000, 70], 2, 2, 64, True), ("sharp", [900, 200], 4, 1, 64, False),
    ("offset", [512], 2, 2, 64, True), ("offset", [700, 65], 4, 2, 128, True), ("offset", [300, 129, 500], 3, 1, 128, True),
    ("channels", [700], 4, 1, 64, True), ("channels", [1300], 2, 1, 128, False), ("channels", [80, 100, 120] * 4, 2, 2, 128, True),
    ("plain", [1000, 20], 4, 2, 128, True), ("plain", [400], 2, 1, 64, False),
]


@pytest.mark.parametrize("kind,lens,Hq,Hkv,d,causal", CASES, ids=str)
def test_gradients_are_as_exact_as_their_roundings(fa, kind, lens, Hq, Hkv, d, causal):
    cu, scale, G = ref.starts(lens), d ** -0.5, Hq // Hkv
    q, k, v, dO = inputs(kind, cu[-1], Hq, Hkv, d)
    g = [t.cuda() for t in (q, k, v, dO)]
    starts = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, lse = fa.fa_forward_packed(*g[:3], starts, causal=causal)
    dq, dk, dv = fa.fa_backward_packed(*g[:3], o, g[3], lse, starts, causal=causal)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == (0, 0)
    want = ref.attention(q, k, v, cu, cu, scale, causal, dO)
    var = {"dq": (RMS * want["dq"]) ** 2, "dk": (RMS * want["dk"]) ** 2}
    for a, b in zip(cu, cu[1:]):
        mask = ref.seen(b - a, b - a, causal)
        for h in range(Hq):
            Q, K, V, X = (t[a:b, i].double() for t, i in ((q, h), (k, h // G), (v, h // G), (dO, h)))
            P = torch.softmax((Q @ K.T * scale).masked_fill(~mask, -math.inf), -1)
            dP = X @ V.T
            dS2 = (RMS * scale * P * (dP - (P * dP).sum(-1, keepdim=True))) ** 2
            var["dq"][a:b, h] += dS2 @ K ** 2
            var["dk"][a:b, h // G] += dS2.T @ Q ** 2
    for name, got in (("dq", dq), ("dk", dk)):
        err = (got.cpu().double() - want[name]).norm()
        room = var[name].sum().sqrt()
        print(name, kind, "error %.2f of its roundings', %.4f of its norm" % (err / room, err / want[name].norm()))
        # 1.2: the spread of a sum over some thousand rows of few keys, and the fp32 steps
        assert err <= 1.2 * room, name


@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 2), (3, 1), (7, 1)])
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("causal", (True, False))
def test_a_sequence_has_the_same_bits_whatever_else_is_in_the_batch(fa, d, Hq, Hkv, causal):
    """Alone, among shorter sequences and beside a long one: the same results, to the bit."""
    lens = [130, 64, 21]
    alone = {}
    for others in ([], [9] * 40, [2300], [700] * 3):
        cu = ref.starts(lens + others)
        q, k, v, dO = inputs("sharp", cu[-1], Hq, Hkv, d)
        n = sum(lens)
        if not alone:
            first = [t.clone() for t in (q, k, v, dO)]
        for t, x in zip((q, k, v, dO), first):
            t[:n] = x
        g = [t.cuda() for t in (q, k, v, dO)]
        starts = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = fa.fa_forward_packed(*g[:3], starts, causal=causal)
        dq, dk, dv = fa.fa_backward_packed(*g[:3], o, g[3], lse, starts, causal=causal)
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == (0, 0)
        got = dict(o=o[:n], lse=lse[:, :n], dq=dq[:n], dk=dk[:n], dv=dv[:n])
        alone = alone or got
        for name in got:
            assert torch.equal(got[name], alone[name]), (name, len(others))
