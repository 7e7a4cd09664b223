"""The key/value cache operators on the host (no GPU): argument checks of the C
ABI and of the Python binding, the tree masks, and the fp64 definition's own
quantiser against a search over all codes."""
import ctypes

import numpy as np
import pytest
import torch

import exact_io_aware_16_gb300 as fa
import kvcache_ref as ref
from exact_io_aware_16_gb300 import _binding as bd
from exact_io_aware_16_gb300 import build as fabuild

FAKE = 0x10000  # aligned, never dereferenced: validation returns first


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.library()


def cache(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, B=2, Hkv=3, cap=64, d=64, fmt=1):
    return ctypes.byref(bd._CacheStruct(k, v, ks, vs, B, Hkv, cap, d, fmt))


BAD_CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(B=0), -2), (dict(Hkv=-1), -2), (dict(cap=0), -2), (dict(d=96), -3), (dict(d=0), -3),
    (dict(cap=(1 << 31) - 1), -2),            # positions and a tile fit an int32
    (dict(fmt=2), -2), (dict(fmt=-1), -2),
    (dict(B=1 << 16, Hkv=1 << 15), -2),       # B*Hkv = 2^31
    (dict(B=1 << 20, Hkv=64, cap=2048), -2),  # 2^31 tiles of 64 tokens
    (dict(k=FAKE + 8), -4), (dict(v=FAKE + 2), -4), (dict(ks=FAKE + 1), -4), (dict(vs=FAKE + 8), -4),
]


def write(lib, c, k=FAKE, v=FAKE, lens=FAKE, counts=None, N=4):
    return lib.fa_cache_write(c, k, v, lens, counts, N, None)


def read(lib, c, k=FAKE, v=FAKE, first=None, counts=FAKE, N=4):
    return lib.fa_cache_read(c, k, v, first, counts, N, None)


def commit(lib, c, lens=FAKE, path=FAKE, n=FAKE, new=FAKE, T=4):
    return lib.fa_cache_commit(c, lens, path, n, new, T, None)


def tree(lib, c, q=FAKE, lens=FAKE, mask=None, stride=0, o=FAKE, lse=FAKE, Hq=6, T=4, scale=0.125,
         ws=FAKE * 16, wb=1 << 40):
    return lib.fa_decode_tree(c, q, lens, mask, stride, o, lse, Hq, T, scale, ws, wb, None)


@pytest.mark.parametrize("kw,status", BAD_CACHES, ids=[str(c[0]) for c in BAD_CACHES])
def test_bad_caches_are_refused_by_every_call(lib, kw, status):
    # an unaligned argument of its own would only be looked at later
    assert write(lib, cache(**kw)) == status
    assert read(lib, cache(**kw)) == status
    assert commit(lib, cache(**kw)) == status
    assert tree(lib, cache(**kw)) == status
    if status != -4:
        assert lib.fa_decode_tree_workspace_size(cache(**kw), 6, 4) == 0


def test_null_cache(lib):
    assert write(lib, None) == read(lib, None) == commit(lib, None) == tree(lib, None) == -1
    assert lib.fa_decode_tree_workspace_size(None, 6, 4) == 0


def test_a_bf16_cache_needs_no_scales_and_any_capacity_will_do(lib):
    assert write(lib, cache(cap=73), k=FAKE + 8) == -4
    c = cache(ks=None, vs=None, cap=71, fmt=0)
    assert write(lib, c, k=FAKE + 8) == -4  # past the shape checks
    assert tree(lib, c, q=FAKE + 8) == -4
    assert lib.fa_decode_tree_workspace_size(c, 6, 4) > 0


def test_write_read_commit_refusals(lib):
    c = cache()
    for kw, st in ((dict(k=None), -1), (dict(v=None), -1), (dict(lens=None), -1), (dict(N=0), -2), (dict(N=-1), -2),
                   (dict(N=1 << 28), -2), (dict(k=FAKE + 8), -4), (dict(v=FAKE + 4), -4), (dict(lens=FAKE + 2), -4),
                   (dict(counts=FAKE + 1), -4)):
        assert write(lib, c, **kw) == st, kw
    for kw, st in ((dict(k=None), -1), (dict(v=None), -1), (dict(counts=None), -1), (dict(N=0), -2), (dict(N=1 << 28), -2),
                   (dict(k=FAKE + 8), -4), (dict(first=FAKE + 2), -4), (dict(counts=FAKE + 1), -4)):
        assert read(lib, c, **kw) == st, kw
    for kw, st in ((dict(lens=None), -1), (dict(path=None), -1), (dict(n=None), -1), (dict(new=None), -1),
                   (dict(T=0), -2), (dict(T=65), -2), (dict(lens=FAKE + 2), -4), (dict(path=FAKE + 1), -4),
                   (dict(n=FAKE + 2), -4), (dict(new=FAKE + 2), -4)):
        assert commit(lib, c, **kw) == st, kw


def test_tree_refusals(lib):
    c = cache()
    need = lib.fa_decode_tree_workspace_size(c, 6, 4)
    assert need > 0 and need % 256 == 0
    for kw, st in ((dict(q=None), -1), (dict(lens=None), -1), (dict(o=None), -1), (dict(lse=None), -1),
                   (dict(T=0), -2), (dict(T=65), -2), (dict(Hq=0), -2), (dict(Hq=7), -2), (dict(Hq=-3), -2),
                   (dict(Hq=3 << 28), -2), (dict(mask=FAKE, stride=5), -2), (dict(mask=FAKE, stride=-4), -2),
                   (dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2),
                   (dict(ws=None), -6), (dict(wb=need - 1), -6), (dict(ws=FAKE * 16 + 16), -6),
                   (dict(q=FAKE + 8), -4), (dict(o=FAKE + 2), -4), (dict(lse=FAKE + 2), -4), (dict(lens=FAKE + 2), -4),
                   (dict(mask=FAKE + 4, stride=4), -4)):
        assert tree(lib, c, **kw) == st, kw
    for Hq, T in ((0, 4), (7, 4), (6, 0), (6, 65), (3 << 28, 64)):
        assert lib.fa_decode_tree_workspace_size(c, Hq, T) == 0


@pytest.mark.parametrize("B,Hkv,cap,st", [
    (65537, 1, 16, -2),          # more sequences than a CTA walks over
    (65536, 1, 16, -6),
    (65536, 1 << 12, 16, -2),    # 2^28 pairs of 5 units
    (2, 1, 2147483392, -6),      # the largest capacity
    (65, 1, 2147483392, -2),     # more than 2^30 units
])
def test_tree_size_limits(lib, B, Hkv, cap, st):
    """-6: the shape passes, and the workspace of no bytes is refused."""
    c = cache(B=B, Hkv=Hkv, cap=cap)
    assert tree(lib, c, Hq=Hkv, T=1, wb=0) == st
    assert (lib.fa_decode_tree_workspace_size(c, Hkv, 1) > 0) == (st == -6)


# ---------------------------------------------------------------- binding
class StubLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if not name.startswith("fa_"):
            raise AttributeError(name)

        def fn(*args):
            self.calls.append(name)
            return 512 if name.endswith("workspace_size") else 0

        fn.__name__ = name
        return fn


@pytest.fixture
def stub(monkeypatch):
    s = StubLib()
    monkeypatch.setattr(bd, "library", lambda: s)
    monkeypatch.setattr(bd, "_on_device", lambda t: True)
    return s


def held(fmt="e4m3", B=2, H=3, cap=32, d=64):
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.bfloat16
    k, v = torch.zeros(B, H, cap, d, dtype=dt), torch.zeros(B, H, cap, d, dtype=dt)
    s = [torch.zeros(B, H, cap, dtype=torch.uint8) for _ in range(2)] if fmt == "e4m3" else [None, None]
    return k, v, *s


def test_cache_objects(stub):
    k, v, ks, vs = held()
    c = fa.KvCache.from_tensors(k, v, ks, vs)
    assert c.format == "e4m3" and c.shape == (2, 3, 32, 64) and c.lens.tolist() == [0, 0]
    assert c.k is k and c.v_scale is vs
    with pytest.raises(AttributeError):
        c.k = v
    assert fa.KvCache(2, 3, 32, 64, "bf16", device="cpu").format == "bf16"
    for bad in ((k, v, ks, None), (k, v, None, vs), (k, v[:1], ks, vs), (k, v.bfloat16(), ks, vs),
                (k.float(), v.float(), None, None), (k.bfloat16(), v.bfloat16(), ks, vs), (k[0], v[0], ks, vs),
                (k, v, ks[:1], vs), (k, v, ks.int(), vs), (k.transpose(0, 1), v.transpose(0, 1), ks, vs)):
        with pytest.raises((TypeError, ValueError)):
            fa.KvCache.from_tensors(*bad)
    with pytest.raises(TypeError):
        fa.KvCache.from_tensors(k, v, ks, vs, lens=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        fa.KvCache(2, 3, 32, 64, "fp8", device="cpu")


def calls(c, i=torch.int32):
    """Per call: its good arguments, by name."""
    B, H, cap, d = c.shape
    bf = torch.bfloat16
    return {
        "fa_cache_write": dict(k=torch.zeros(B, H, 5, d, dtype=bf), v=torch.zeros(B, H, 5, d, dtype=bf),
                               lens=torch.zeros(B, dtype=i), counts=torch.zeros(B, dtype=i)),
        "fa_cache_read": dict(N=5, k=torch.zeros(B, H, 5, d, dtype=bf), v=torch.zeros(B, H, 5, d, dtype=bf),
                              first=torch.zeros(B, dtype=i), counts=torch.zeros(B, dtype=i)),
        "fa_cache_commit": dict(path=torch.zeros(B, 4, dtype=i), n_accept=torch.zeros(B, dtype=i),
                                lens=torch.zeros(B, dtype=i), new_lens=torch.zeros(B, dtype=i)),
        "fa_decode_tree": dict(q=torch.zeros(B, 2 * H, 4, d, dtype=bf), mask=torch.zeros(B, 4, dtype=torch.int64),
                               lens=torch.zeros(B, dtype=i), o=torch.zeros(B, 2 * H, 4, d, dtype=bf),
                               lse=torch.zeros(B, 2 * H, 4), workspace=torch.zeros(512, dtype=torch.uint8)),
    }


@pytest.mark.parametrize("fmt", ("e4m3", "bf16"))
def test_binding_refuses_what_does_not_fit(stub, monkeypatch, fmt):
    c = fa.KvCache.from_tensors(*held(fmt))
    for name, kw in calls(c).items():
        getattr(fa, name)(c, **kw, stream=0)
        assert stub.calls[-1] == name
        n = len(stub.calls)
        for arg, t in kw.items():
            if not isinstance(t, torch.Tensor):
                continue
            bad = [t.double(), t[:1].contiguous() if arg != "workspace" else t.float()]
            if t.dim() > 1:
                bad.append(torch.zeros(t.shape[::-1], dtype=t.dtype).permute(*range(t.dim() - 1, -1, -1)))
            for x in bad:
                with pytest.raises((TypeError, ValueError)):
                    getattr(fa, name)(c, **{**kw, arg: x}, stream=0)
            # on another GPU than the cache
            with monkeypatch.context() as m:
                m.setattr(bd, "_device_index", lambda x, t=t: 1 if x is t else -1)
                with pytest.raises(ValueError, match="device"):
                    getattr(fa, name)(c, **kw, stream=0)
        assert [x for x in stub.calls[n:] if not x.endswith("workspace_size")] == []
    # the defaults
    fa.fa_cache_write(c, kw_k := torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16), kw_k, stream=0)
    fa.fa_cache_read(c, 3, stream=0)
    fa.fa_decode_tree(c, torch.zeros(2, 3, 1, 64, dtype=torch.bfloat16), stream=0)
    assert fa.fa_cache_commit(c, torch.zeros(2, 4, dtype=torch.int32), c.lens, stream=0) is c.lens


def test_calls_run_with_the_caches_device_current(stub, monkeypatch):
    current, seen = {"dev": 0}, []

    class SwitchTo:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.prev, current["dev"] = current["dev"], self.dev

        def __exit__(self, *exc):
            current["dev"] = self.prev

    monkeypatch.setattr(bd.torch.cuda, "current_device", lambda: current["dev"])
    monkeypatch.setattr(bd.torch.cuda, "device", SwitchTo)
    monkeypatch.setattr(bd, "_device_index", lambda t: 1)
    real = StubLib.__getattr__
    monkeypatch.setattr(StubLib, "__getattr__", lambda self, n: (
        lambda *a: (seen.append((n, current["dev"])), real(self, n)(*a))[1]))
    c = fa.KvCache.from_tensors(*held())
    for name, kw in calls(c).items():
        getattr(fa, name)(c, **kw, stream=0)
        assert seen[-1] == (name, 1)
    assert current["dev"] == 0


# ---------------------------------------------------------------- masks, definition
def test_tree_mask():
    assert fa.tree_mask([-1]).tolist() == [1]
    assert fa.tree_mask([-1, 0, 0, 1, -1]).tolist() == [1, 3, 5, 11, 16]
    m = fa.tree_mask([-1] + list(range(63)))
    assert m.dtype == torch.int64 and [x & (2**64 - 1) for x in m.tolist()] == [(2 << t) - 1 for t in range(64)]
    for bad in ([], [0], [-1, 1], [-1, -2], list(range(-1, 64))):
        with pytest.raises(ValueError):
            fa.tree_mask(bad)


def test_the_definitions_quantiser_takes_the_nearest_code():
    g = np.random.RandomState(0)
    x = g.standard_normal((200, 64)) * 10.0 ** g.uniform(-6, 6, (200, 1))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    c, s = ref.quantise(x)
    e = s.astype(int) - 127
    amax = np.abs(x).max(-1)
    assert np.all(amax <= 448 * 2.0 ** e) and np.all(amax > 448 * 2.0 ** (e - 1))
    y = x / 2.0 ** e[:, None].astype(float)
    best = np.nanmin(np.abs(y[..., None] - ref.CODES), -1)
    np.testing.assert_array_equal(np.abs(y - ref.CODES[c]), best)
    # torch's own conversion rounds ties to the even code as well
    t = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.CODES[t], ref.CODES[c])
