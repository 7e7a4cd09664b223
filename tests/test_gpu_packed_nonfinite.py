"""NaN and infinities in packed attention and its gradients: rows whose scores are all -inf, and what a
row that is not finite may and may not reach."""
import math

import pytest
import torch

import packed_ref as ref
from test_gpu_packed import fa, i32, ok, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


def both(fa, t, cu_q, cu_k, causal):  # noqa: F811
    o, lse = fa.fa_forward_packed(*t[:3], i32(cu_q), i32(cu_k), causal=causal)
    grads = fa.fa_backward_packed(*t[:3], o, t[3], lse, i32(cu_q), i32(cu_k), causal=causal)
    ok(fa)
    return dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads)))


@pytest.mark.parametrize("causal", (True, False))
@pytest.mark.parametrize("lens_q,lens_k", [([150, 9], [140, 30]), ([40, 3], [33, 50]), ([20, 300], [600, 300])], ids=str)
@pytest.mark.parametrize("d", (64, 128))
def test_gradients_of_a_row_whose_scores_are_all_minus_infinity(fa, d, lens_q, lens_k, causal):  # noqa: F811
    """P = exp(-inf + inf) is NaN for the keys that the row sees, whatever the lengths: so is its dq, and the dk
    and dv of those keys.  The other queries' results, the other key head and the other sequence do not change."""
    Hq, Hkv, head = 4, 2, 1
    cu_q, cu_k = ref.starts(lens_q), ref.starts(lens_k)
    q, k, v, dO = rnd(70, cu_q[-1], Hq, d), rnd(71, cu_k[-1], Hkv, d), rnd(72, cu_k[-1], Hkv, d), rnd(73, cu_q[-1], Hq, d)
    k[:, :, 0] = -k[:, :, 0].abs() - 0.5
    t = [x.cuda() for x in (q, k, v, dO)]
    want = both(fa, t, cu_q, cu_k, causal)
    row = lens_q[0] - 2  # sees all keys of the first sequence, or all but one
    t[0][row, head] = 0.0
    t[0][row, head, 0] = math.inf
    got = both(fa, t, cu_q, cu_k, causal)
    seen = lens_k[0] - 1 if causal else lens_k[0]
    assert torch.isneginf(got["lse"][head, row])
    assert torch.isnan(got["o"][row, head]).all() and torch.isnan(got["dq"][row, head]).all()
    for x in ("dk", "dv"):
        assert torch.isnan(got[x][:seen, 0]).all(), x
        assert torch.equal(got[x][:, 1], want[x][:, 1]) and torch.equal(got[x][lens_k[0]:], want[x][lens_k[0]:]), x
    for x in ("o", "dq"):
        got[x][row, head] = want[x][row, head]
        assert torch.equal(got[x], want[x]), x
    if causal and lens_k[0] < lens_q[0]:  # the first queries see nothing
        none = lens_q[0] - lens_k[0]
        assert (got["dq"][:none] == 0).all() and torch.isneginf(got["lse"][:, :none]).all()


@pytest.mark.parametrize("lens_q,lens_k", [([150], [140]), ([90, 200], [30, 170])], ids=str)
@pytest.mark.parametrize("d", (64, 128))
def test_a_query_that_sees_no_key_has_no_gradient_whatever_it_holds(fa, d, lens_q, lens_k):  # noqa: F811
    cu_q, cu_k = ref.starts(lens_q), ref.starts(lens_k)
    q, k, v, dO = (rnd(80 + i, n, h, d).cuda() for i, (n, h) in
                   enumerate(((cu_q[-1], 4), (cu_k[-1], 2), (cu_k[-1], 2), (cu_q[-1], 4))))
    want = both(fa, (q, k, v, dO), cu_q, cu_k, True)
    q[cu_q[-2] + 2], dO[cu_q[-2] + 3], dO[cu_q[-2] + 4] = math.nan, math.inf, math.nan
    got = both(fa, (q, k, v, dO), cu_q, cu_k, True)
    for x in ("o", "lse", "dq"):
        assert torch.equal(got[x], want[x]), x


@pytest.mark.parametrize("bad", (math.nan, math.inf))
@pytest.mark.parametrize("which", ("q", "k", "v", "dO"))
@pytest.mark.parametrize("d", (64, 128))
def test_how_far_a_row_that_is_not_finite_reaches(fa, d, which, bad):  # noqa: F811
    """Other sequences and other key heads' groups never change; of its own, only what the row can reach."""
    lens, at = [70, 300, 45], 170  # a token of the second sequence
    cu = ref.starts(lens)
    t = dict(q=rnd(90, cu[-1], 4, d), k=rnd(91, cu[-1], 2, d), v=rnd(92, cu[-1], 2, d), dO=rnd(93, cu[-1], 4, d))
    t = {x: y.cuda() for x, y in t.items()}
    want = both(fa, list(t.values()), cu, cu, True)
    t[which][cu[1] + at, 0] = bad
    got = both(fa, list(t.values()), cu, cu, True)
    own = slice(cu[1], cu[2])
    keep = {x: torch.ones(y.shape[:2] if x != "lse" else y.T.shape, dtype=torch.bool, device="cuda") for x, y in got.items()}
    heads = dict(o=slice(0, 2), lse=slice(0, 2), dq=slice(0, 2), dk=slice(0, 1), dv=slice(0, 1))
    if which in ("q", "dO"):  # a row of query head 0: of o, lse and dq its own alone
        for x in ("o", "lse", "dq") if which == "q" else ("dq",):
            keep[x][cu[1] + at, 0] = False
        keep["dk"][own, 0] = keep["dv"][own, 0] = False
    elif which == "k":  # o and lse of the queries that see it
        for x in ("o", "lse"):
            keep[x][cu[1] + at: cu[2], heads[x]] = False
        for x in ("dq", "dk", "dv"):
            keep[x][own, heads[x]] = False
    else:  # neither lse nor dv depends on the values
        for x in ("o", "dq", "dk"):
            keep[x][own, heads[x]] = False
    for x in got:
        a, b = (y.T if x == "lse" else y for y in (got[x], want[x]))
        assert torch.equal(a[keep[x]], b[keep[x]]), x
    # and the row's own result says so
    mine = dict(q="dq", k="dk", v="dk", dO="dq")[which]
    assert not torch.isfinite(got[mine][cu[1] + at, 0]).all()
