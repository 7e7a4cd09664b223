"""The operators on packed sequences and the rotation on the host (no GPU): argument checks of
the C ABI and of the Python binding, workspace sizes, and the tables of rotations."""
import ctypes
import math

import pytest
import torch

import exact_io_aware_16_gb300 as fa
from exact_io_aware_16_gb300 import _binding as bd
from exact_io_aware_16_gb300 import build as fabuild
from test_binding_checks import StubLib

FAKE = 0x10000  # aligned, never dereferenced: validation returns first
NULL, SHAPE, HEADDIM, ALIGN, ARCH, WORKSPACE, CUDA = -1, -2, -3, -4, -5, -6, -7


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.library()


def heads(p=FAKE, batch=0, token=None, head=None, n=4, d=64):
    head = d if head is None else head
    return bd._pack_heads(p or 0, batch, head * n if token is None else token, head, n)


def passed(status):
    """Past all checks but that of the GPU, of which this machine has none."""
    return status in (ARCH, CUDA)


# ---------------------------------------------------------------- packed attention
def packed(lib, backward=False, q=None, k=None, v=None, o=None, g=None, dq=None, dk=None, dv=None, lse=FAKE, cu_q=FAKE,
           cu_k=None, B=2, tq=100, tk=100, d=64, scale=0.1, ws=FAKE, wb=1 << 40):
    q, k, v, o = (heads() if q is None else q, heads(n=2) if k is None else k, heads(n=2) if v is None else v,
                  heads() if o is None else o)
    if not backward:
        return lib.fa_forward_packed(q, k, v, o, lse, cu_q, cu_k, B, tq, tk, d, scale, 1, ws, wb, None)
    g, dq, dk, dv = (heads() if g is None else g, heads() if dq is None else dq, heads(n=2) if dk is None else dk,
                     heads(n=2) if dv is None else dv)
    return lib.fa_backward_packed(q, k, v, o, g, lse, dq, dk, dv, cu_q, cu_k, B, tq, tk, d, scale, 1, ws, wb, None)


@pytest.mark.parametrize("backward", (False, True))
def test_packed_calls_that_are_right_reach_the_gpu_check(lib, backward):
    for kw in (dict(), dict(cu_k=FAKE, tk=300), dict(tq=0, tk=0, lse=None), dict(cu_k=FAKE, tk=0), dict(B=(1 << 20) - 1),
               dict(q=heads(token=2048, head=64 * 7)),          # rows with gaps
               dict(q=heads(token=64, head=6400)),              # [heads][tokens][d]
               dict(tq=1, tk=1, q=heads(token=3, head=64)),     # a stride that no element depends on
               dict(cu_k=FAKE, tk=0, k=heads(p=None, n=2), v=heads(p=None, n=2))):
        assert passed(packed(lib, backward, **kw)), kw


REFUSED = [
    (dict(lse=None), NULL), (dict(cu_q=None), NULL), (dict(q=heads(p=None)), NULL),
    (dict(B=0), SHAPE), (dict(B=1 << 20), SHAPE), (dict(tq=-1), SHAPE), (dict(tk=-1, cu_k=FAKE), SHAPE),
    (dict(tk=99), SHAPE),                                                       # cu_k is needed
    (dict(d=96), HEADDIM), (dict(d=0), HEADDIM),
    (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE),
    (dict(k=heads(n=3)), SHAPE), (dict(k=heads(n=0)), SHAPE), (dict(q=heads(n=0)), SHAPE),
    (dict(v=heads(n=4)), SHAPE), (dict(o=heads(n=2)), SHAPE),
    (dict(tq=2**31 - 1, tk=2**31 - 1, q=heads(n=64), o=heads(n=64)), SHAPE),    # 2^31 items
    (dict(q=heads(p=FAKE + 8)), ALIGN), (dict(k=heads(n=2, token=132)), ALIGN), (dict(v=heads(n=2, head=68)), ALIGN),
    (dict(o=heads(p=FAKE + 2)), ALIGN), (dict(lse=FAKE + 2), ALIGN), (dict(cu_q=FAKE + 1), ALIGN),
    (dict(cu_k=FAKE + 2), ALIGN),
    (dict(q=heads(token=0)), SHAPE), (dict(q=heads(head=0)), SHAPE), (dict(q=heads(token=-256)), SHAPE),
    (dict(q=heads(token=128, head=64)), SHAPE),                                 # rows that overlap
    (dict(q=heads(token=1 << 40)), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 16), WORKSPACE), (dict(wb=1000), WORKSPACE),
]


@pytest.mark.parametrize("backward", (False, True))
@pytest.mark.parametrize("kw,status", REFUSED, ids=[str(i) for i in range(len(REFUSED))])
def test_packed_refusals(lib, kw, status, backward):
    assert packed(lib, backward, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(g=heads(n=2)), SHAPE), (dict(dq=heads(p=None)), NULL), (dict(dk=heads(n=4)), SHAPE),
    (dict(dv=heads(n=2, p=FAKE + 4)), ALIGN), (dict(dk=heads(n=2, token=64, head=64)), SHAPE)])
def test_backward_refusals(lib, kw, status):
    assert packed(lib, True, **kw) == status


def test_workspace_sizes(lib):
    fwd, bwd = lib.fa_forward_packed_workspace_size, lib.fa_backward_packed_workspace_size
    for bad in ((0, 1, 1, 1, 1, 64), (1, -1, 1, 1, 1, 64), (1, 1, 1, 3, 2, 64), (1, 1, 1, 1, 1, 80), (1, 1, 1, 0, 1, 64)):
        assert fwd(*bad) == bwd(*bad) == 0
    for args in ((1, 17, 17, 32, 8, 128), (64, 16384, 16384, 12, 12, 64), (5, 0, 0, 4, 2, 64), (1000, 5, 700000, 7, 1, 128)):
        B, tq, tk, Hq, _, d = args
        assert 0 < fwd(*args) < 1024 * B + 8 * tq + 4096
        assert 4 * Hq * tq < bwd(*args) < 4 * Hq * tq + 1400 * B + 16 * tq + tk + 8192
        assert fwd(*args) % 256 == bwd(*args) % 256 == 0
        # exactly what is asked for is enough, a byte less is not
        q, k = heads(n=Hq, d=d), heads(n=args[4], d=d)
        for size, back in ((fwd(*args), False), (bwd(*args), True)):
            kw = dict(q=q, k=k, v=k, o=q, g=q, dq=q, dk=k, dv=k, B=B, tq=tq, tk=tk, d=d, cu_k=FAKE)
            assert passed(packed(lib, back, wb=size, **kw))
            assert packed(lib, back, wb=size - 1, **kw) == WORKSPACE


# ---------------------------------------------------------------- rotation
def rotation(turns=FAKE, rot=32, inter=0, amplitude=1.0):
    return ctypes.byref(bd._RotationStruct(turns, rot, inter, amplitude))


def rotary(lib, r=None, q=None, k=None, qo=None, ko=None, pos=FAKE, B=1, N=10, d=64, norm=False, back=False, wq=FAKE, wk=FAKE,
           fmt=0, eps=1e-6, dwq=FAKE, dwk=FAKE, ws=FAKE, wb=1 << 20, alone=False):
    r = rotation() if r is None else r
    q, qo = heads() if q is None else q, heads() if qo is None else qo
    k, ko = (None, None) if alone else (heads(n=2) if k is None else k, heads(n=2) if ko is None else ko)
    if norm and back:
        return lib.fa_norm_rotary_backward(r, q, k, q, k, qo, ko, dwq, dwk, pos, wq, wk, fmt, eps, B, N, d, ws, wb, None)
    if norm:
        return lib.fa_norm_rotary(r, q, k, qo, ko, pos, wq, wk, fmt, eps, B, N, d, None)
    return (lib.fa_rotary_backward if back else lib.fa_rotary)(r, q, k, qo, ko, pos, B, N, d, None)


ALL = [dict(norm=n, back=b) for n in (False, True) for b in (False, True)]


@pytest.mark.parametrize("which", ALL, ids=str)
def test_rotations_that_are_right_reach_the_gpu_check(lib, which):
    for kw in (dict(), dict(pos=None), dict(alone=True, wk=None, dwk=None), dict(r=rotation(rot=64, inter=1, amplitude=0.0)),
               dict(B=3, q=heads(batch=2560), qo=heads(batch=2560), k=heads(n=2, batch=2560), ko=heads(n=2, batch=2560)),
               dict(fmt=1), dict(eps=0.0)):
        assert passed(rotary(lib, **which, **kw)), kw


@pytest.mark.parametrize("which", ALL, ids=str)
@pytest.mark.parametrize("kw,status", [
    (dict(r=rotation(turns=None)), NULL), (dict(q=heads(p=None)), NULL), (dict(ko=heads(n=2, p=None)), NULL),
    (dict(r=rotation(rot=0)), SHAPE), (dict(r=rotation(rot=24)), SHAPE), (dict(r=rotation(rot=80)), SHAPE),
    (dict(r=rotation(rot=-16)), SHAPE), (dict(r=rotation(amplitude=math.inf)), SHAPE), (dict(d=32), HEADDIM),
    (dict(B=0), SHAPE), (dict(N=0), SHAPE), (dict(N=2**31 - 1, B=2), SHAPE), (dict(N=2**30), SHAPE),
    (dict(qo=heads(n=2)), SHAPE), (dict(q=heads(p=FAKE + 8)), ALIGN), (dict(qo=heads(token=260)), ALIGN),
    (dict(q=heads(token=64, head=64)), SHAPE), (dict(pos=FAKE + 1), ALIGN), (dict(r=rotation(turns=FAKE + 4)), ALIGN),
])
def test_rotation_refusals(lib, which, kw, status):
    assert rotary(lib, **which, **kw) == status


@pytest.mark.parametrize("back", (False, True))
@pytest.mark.parametrize("kw,status", [
    (dict(wq=None), NULL), (dict(wk=None), NULL), (dict(fmt=2), SHAPE), (dict(eps=-1e-9), SHAPE), (dict(eps=math.nan), SHAPE),
    (dict(wq=FAKE + 8), ALIGN), (dict(wk=FAKE + 4), ALIGN)])
def test_norm_refusals(lib, back, kw, status):
    assert rotary(lib, norm=True, back=back, **kw) == status


def test_norm_backward_refusals(lib):
    for kw, status in ((dict(dwq=None), NULL), (dict(dwk=None), NULL), (dict(dwq=FAKE + 4), ALIGN), (dict(ws=None), WORKSPACE),
                       (dict(wb=(1 << 20) - 1), WORKSPACE), (dict(ws=FAKE + 128), WORKSPACE)):
        assert rotary(lib, norm=True, back=True, **kw) == status, kw


def table(lib, rot, base, scaling=0, factor=1.0, original=0.0, low=1.0, high=32.0):
    t = (ctypes.c_ulonglong * (rot // 2))()
    assert lib.fa_rotary_table(t, rot, base, scaling, factor, original, low, high) == 0
    return [x / 2.0 ** 64 * 2 * math.pi for x in t]


@pytest.mark.parametrize("rot", (16, 48, 64, 128))
def test_tables_of_every_scaling(lib, rot):
    """Against the formulas in 64 bits: 2^-50 for the functions' roundings, 2^-64 of a turn."""
    base, s, L, low, high = 10000.0, 8.0, 4096.0, 1.0, 32.0
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]

    def near(got, want):
        assert all(abs(a - b) <= 2.0 ** -49 * b + 2.0 ** -61 for a, b in zip(got, want))

    near(table(lib, rot, base), f)
    near(table(lib, rot, base, 1, s), [x / s for x in f])
    b = table(lib, rot, base, 2, s)
    near(b, [x * s ** (-2 * i / (rot - 2)) for i, x in enumerate(f)])
    assert abs(b[0] - 1) < 1e-14 and abs(b[-1] * s / f[-1] - 1) < 1e-13
    g = [min(max((L * x / (2 * math.pi) - low) / (high - low), 0), 1) for x in f]
    near(table(lib, rot, base, 3, s, L, low, high), [a * x + (1 - a) * x / s for a, x in zip(g, f)])
    at = lambda t: rot * math.log(L / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    i0, i1 = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    g = [min(max(1 - (i - i0) / max(i1 - i0, 1e-3), 0), 1) for i in range(rot // 2)]
    near(table(lib, rot, base, 4, s, L, low, high), [a * x + (1 - a) * x / s for a, x in zip(g, f)])


def test_tables_refused(lib):
    t = (ctypes.c_ulonglong * 64)()
    ok = dict(rot=32, base=1e4, scaling=4, factor=2.0, original=4096.0, low=1.0, high=32.0)
    call = lambda **kw: lib.fa_rotary_table(t, *{**ok, **kw}.values())  # noqa: E731
    assert call() == 0
    assert lib.fa_rotary_table(None, *ok.values()) == NULL
    for kw in (dict(rot=8), dict(rot=40), dict(rot=144), dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(scaling=5),
               dict(scaling=-1), dict(factor=0.5), dict(factor=math.inf), dict(original=0.0), dict(low=0.0), dict(high=1.0),
               dict(high=math.inf)):
        assert call(**kw) == SHAPE, kw


# ---------------------------------------------------------------- the binding
@pytest.fixture
def stub(monkeypatch):
    class Lib(StubLib):
        def __getattr__(self, name):
            fn = super().__getattr__(name)
            out = (lambda *a: (fn(*a), 4096)[1]) if name.endswith("workspace_size") else fn
            out.__name__ = name
            return out

    lib = Lib()
    monkeypatch.setattr(bd, "library", lambda: lib)
    monkeypatch.setattr(bd, "_on_device", lambda t: True)
    return lib


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


TABLE = torch.zeros(32, dtype=torch.int64)


def arguments():
    """One accepted call of each function: (function, positional tensors by name, keywords)."""
    r = fa.Rotary.from_table(64, TABLE)
    q, k, v, o, g, cu = bf(30, 4, 64), bf(30, 2, 64), bf(30, 2, 64), bf(30, 4, 64), bf(30, 4, 64), i32(0, 10, 30)
    lse, pos, w = torch.zeros(4, 30), torch.arange(30, dtype=torch.int32), torch.ones(64)
    return {
        "fa_forward_packed": (dict(q=q, k=k, v=v, cu_q=cu, cu_k=cu), dict(o=o, lse=lse)),
        "fa_backward_packed": (dict(q=q, k=k, v=v, o=o, dO=g, lse=lse, cu_q=cu, cu_k=cu), dict(dq=q, dk=k, dv=v)),
        "fa_rotary": (dict(rotary=r, q=q, k=k, positions=pos), dict(q_out=q, k_out=k)),
        "fa_rotary_backward": (dict(rotary=r, dq=q, dk=k, positions=pos), dict(dq_in=q, dk_in=k)),
        "fa_norm_rotary": (dict(rotary=r, q=q, k=k, positions=pos, q_weight=w, k_weight=w), dict(q_out=q, k_out=k)),
        "fa_norm_rotary_backward": (dict(rotary=r, dq=q, dk=k, q=q, k=k, positions=pos, q_weight=w, k_weight=w),
                                    dict(dq_in=q, dk_in=k, dq_weight=w, dk_weight=w)),
    }


NAMES = ["fa_forward_packed", "fa_backward_packed", "fa_rotary", "fa_rotary_backward", "fa_norm_rotary", "fa_norm_rotary_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_every_wrapper_reaches_its_library_function(stub, name):
    args, outs = arguments()[name]
    getattr(fa, name)(**args, stream=0)
    assert stub.calls[-1] == name
    getattr(fa, name)(**args, **outs, stream=0)
    assert stub.calls[-1] == name


@pytest.mark.parametrize("name", NAMES)
def test_bad_tensors_are_refused_before_the_library(stub, name):
    args, outs = arguments()[name]
    every = {**args, **outs}
    for which, t in every.items():
        if not isinstance(t, torch.Tensor):
            continue
        bad = [t.to(torch.float64), t[:-1].clone() if t.dim() == 1 else t[..., :-1].clone()]
        if t.dim() == 3:
            bad += [t.transpose(-1, -2).contiguous().transpose(-1, -2)]  # rows that are not contiguous
        for b in bad:
            with pytest.raises((TypeError, ValueError)):
                getattr(fa, name)(**{**every, which: b}, stream=0)
    assert [c for c in stub.calls if not c.endswith("workspace_size")] == []


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_gpu_are_refused(stub, monkeypatch, name):
    args, outs = arguments()[name]
    every = {**args, **outs}
    for which, t in every.items():
        if not isinstance(t, torch.Tensor):
            continue
        other = t.clone()
        # -1 (a CPU tensor's index) for the rest: accepted calls switch no device
        monkeypatch.setattr(bd, "_device_index", lambda x: 1 if x is other else -1)
        with pytest.raises(ValueError, match="device"):
            getattr(fa, name)(**{**every, which: other}, stream=0)
    assert [c for c in stub.calls if not c.endswith("workspace_size")] == []


def test_shapes_of_the_binding(stub):
    r = fa.Rotary.from_table(64, TABLE)
    q, k, cu = bf(30, 4, 64), bf(30, 2, 64), i32(0, 30)
    with pytest.raises(ValueError, match="cu_k is needed"):
        fa.fa_forward_packed(q, bf(31, 2, 64), bf(31, 2, 64), cu)
    with pytest.raises(ValueError):
        fa.fa_forward_packed(bf(1, 30, 4, 64), k, k, cu)
    with pytest.raises(ValueError):
        fa.fa_forward_packed(q, k, k, i32(0))
    with pytest.raises(TypeError):
        fa.fa_forward_packed(q, k, k, cu.long())
    with pytest.raises(TypeError):
        fa.fa_forward_packed(q, k, k, cu, workspace=torch.zeros(9999))
    with pytest.raises(ValueError):
        fa.fa_rotary(r, bf(30, 4, 128))
    with pytest.raises(ValueError):
        fa.fa_rotary(r, q, k[None])
    with pytest.raises(TypeError):
        fa.fa_rotary(r, q, positions=torch.arange(30))
    with pytest.raises(ValueError, match="k_weight"):
        fa.fa_norm_rotary(r, q, k, None, torch.ones(64))
    with pytest.raises(TypeError):  # both weights of one type
        fa.fa_norm_rotary(r, q, k, None, torch.ones(64), torch.ones(64).bfloat16())
    with pytest.raises(TypeError):
        fa.fa_norm_rotary(r, q, k, None, torch.ones(64, dtype=torch.float16))
    with pytest.raises(ValueError, match="dk"):
        fa.fa_norm_rotary_backward(r, q, None, q, k, None, torch.ones(64), torch.ones(64))
    assert [c for c in stub.calls if not c.endswith("workspace_size")] == []
    # four axes, positions of each sequence
    fa.fa_rotary(r, bf(2, 4, 15, 64), bf(2, 2, 15, 64), torch.zeros(2, 15, dtype=torch.int32), stream=0)
    fa.fa_rotary(r, bf(2, 4, 15, 64), stream=0)
    assert stub.calls[-2:] == ["fa_rotary"] * 2
    out = fa.fa_rotary(r, q, None, None, stream=0)
    assert out[0].shape == q.shape and out[1] is None


def test_rotary_objects(lib):
    r = fa.Rotary(128, rot=64, base=500.0, interleaved=True, scaling="linear", factor=4.0, amplitude=1.5, device="cpu")
    assert (r.d, r.rot, r.interleaved, r.amplitude) == (128, 64, True, 1.5) and r.turns.shape == (32,)
    want = [500.0 ** (-2 * i / 64) / 4 / (2 * math.pi) for i in range(32)]
    assert all(abs(int(t) / 2.0 ** 64 - w) <= 2.0 ** -49 * w for t, w in zip(r.turns, want))
    for kw in (dict(rot=24), dict(rot=144), dict(rot=0), dict(scaling="other")):
        with pytest.raises(ValueError):
            fa.Rotary(128, device="cpu", **kw)
    for kw in (dict(scaling="turns", factor=2.0), dict(base=0.5), dict(scaling="linear", factor=0.0)):
        with pytest.raises(fa.FaError):
            fa.Rotary(128, device="cpu", **kw)
