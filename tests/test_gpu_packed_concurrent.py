"""Backward passes of packed attention on several streams at once, each with a workspace of its own."""
import pytest
import torch

import packed_ref as ref
from test_gpu_packed import fa, i32, ok, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("own", (False, True))
def test_backward_passes_at_once(fa, d, own):  # noqa: F811
    """Long samples, short ones and a batch of single tokens on three streams, five times over: the same bits as one
    after the other. Workspaces by the binding, or the caller's own, kept from call to call."""
    lens = [[1500, 500], [40] * 50, [1] * 2000, [1024, 3, 700, 273]]
    Hq, Hkv = 4, 2
    q, k, v, dO = (rnd(100 + i, 2000, h, d).cuda() for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    cu = [i32(ref.starts(x)) for x in lens]
    first = [fa.fa_forward_packed(q, k, v, c, causal=True) for c in cu]
    alone = [fa.fa_backward_packed(q, k, v, o, dO, lse, c, causal=True) for c, (o, lse) in zip(cu, first)]
    streams = [torch.cuda.Stream() for _ in lens]
    room = [None] * len(lens)
    if own:
        room = [torch.empty(fa.fa_backward_packed_workspace_size(len(x), 2000, 2000, Hq, Hkv, d), dtype=torch.uint8,
                            device="cuda") for x in lens]
    torch.cuda.synchronize()
    runs = []
    for _ in range(5):
        for c, (o, lse), s, w in zip(cu, first, streams, room):
            runs.append(fa.fa_backward_packed(q, k, v, o, dO, lse, c, causal=True, workspace=w, stream=s))
    ok(fa)
    for i, got in enumerate(runs):
        assert all(torch.equal(a, b) for a, b in zip(got, alone[i % len(lens)])), i


@pytest.mark.parametrize("d", (64, 128))
def test_whole_steps_at_once(fa, d):  # noqa: F811
    """Forward and backward pass of each batch on a stream of its own."""
    lens = [[900, 100], [250] * 4, [20] * 50]
    q, k, v, dO = (rnd(110 + i, 1000, h, d).cuda() for i, h in enumerate((8, 2, 2, 8)))
    cu = [i32(ref.starts(x)) for x in lens]

    def step(c, stream=None):
        o, lse = fa.fa_forward_packed(q, k, v, c, causal=False, stream=stream)
        return (o, lse, *fa.fa_backward_packed(q, k, v, o, dO, lse, c, causal=False, stream=stream))

    alone = [step(c) for c in cu]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cu]
    runs = [[step(c, s) for c, s in zip(cu, streams)] for _ in range(5)]
    ok(fa)
    for r in runs:
        for got, want in zip(r, alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
