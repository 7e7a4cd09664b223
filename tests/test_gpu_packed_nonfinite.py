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
