"""What the operators of the key/value cache are measured on: writing a cache
(quantised to e4m3 or kept in bf16), reading it back, attention of a tree of
drafted tokens over it, and committing the accepted path.

`run` computes them in plain torch operations, or, where `own` is true, with
the library's kernels.  `prepare` makes the inputs of a case from a seed.
"""
import math

import torch

own = False

F8_MAX = 448.0      # largest e4m3 value
E_MIN, E_MAX = -100, 119  # scale exponents of a cache row
BIAS = 127          # stored scale byte = exponent + 127


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of eight sequences enters the cache (every decode step)
        dict(name="write_token", op="write", fmt="e4m3", B=8, Hkv=8, N=1, d=128, cap=2048, lo=100, hi=2000, ragged=False),
        # a ragged batch of drafted tokens, odd count, small heads
        dict(name="write_drafts", op="write", fmt="e4m3", B=32, Hkv=4, N=17, d=64, cap=1008, lo=0, hi=990, ragged=True),
        # a prompt of the benchmark's length enters the cache
        dict(name="write_prompt", op="write", fmt="e4m3", B=4, Hkv=8, N=8192, d=128, cap=8448, lo=0, hi=200, ragged=False),
        # a short window of a few sequences comes back in bf16
        dict(name="read_window", op="read", fmt="e4m3", B=2, Hkv=8, N=333, d=64, cap=2048, lo=300, hi=333, ragged=True),
        # whole prompts come back for the prefill kernel of a follow-up turn
        dict(name="read_prompt", op="read", fmt="e4m3", B=4, Hkv=8, N=8192, d=128, cap=8448, lo=7000, hi=8192, ragged=True),
        # one token of one sequence, grouped heads: latency
        dict(name="tree_token", op="tree", fmt="e4m3", B=1, Hq=32, Hkv=8, T=1, d=128, cap=1040, lo=1000, hi=1000),
        # a ragged batch, eight drafted tokens each
        dict(name="tree_batch", op="tree", fmt="e4m3", B=32, Hq=32, Hkv=8, T=8, d=128, cap=4112, lo=500, hi=4096),
        # a few long contexts
        dict(name="tree_long", op="tree", fmt="e4m3", B=4, Hq=32, Hkv=8, T=16, d=128, cap=65552, lo=32768, hi=65536),
        # wide trees on a bf16 cache: 256 query rows for each key head
        dict(name="tree_wide", op="tree", fmt="bf16", B=8, Hq=32, Hkv=8, T=64, d=128, cap=8256, lo=4000, hi=8192),
        # as many key heads as query heads, 64-wide, odd counts
        dict(name="tree_mha", op="tree", fmt="bf16", B=16, Hq=16, Hkv=16, T=5, d=64, cap=2053, lo=1, hi=2048),
        # the accepted path of a few sequences
        dict(name="commit_few", op="commit", fmt="e4m3", B=4, Hkv=8, T=16, n=5, d=128, cap=4096, lo=0, hi=4000),
        # the accepted paths of a large batch of wide trees
        dict(name="commit_batch", op="commit", fmt="bf16", B=64, Hkv=8, T=64, n=16, d=128, cap=2048, lo=10, hi=1900),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of these ranges, no costlier than the largest listed one."""
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["write", "read", "tree", "tree", "tree", "commit"])
        c = dict(op=op, fmt=rng.choice(["e4m3", "e4m3", "bf16"]), d=rng.choice([64, 128]))
        c["B"] = _log(rng, 1, 64)
        c["Hkv"] = rng.choice([1, 2, 4, 5, 8, 16, 32])
        if op in ("write", "read"):
            c["N"] = _log(rng, 1, 8192)
            c["ragged"] = rng.random() < 0.5
            if op == "write":
                c["lo"], c["hi"] = 0, _log(rng, 1, 2000)
                need = c["hi"] + c["N"]
            else:
                c["lo"], c["hi"] = rng.randint(0, c["N"]), c["N"]
                need = c["N"] + 64
        elif op == "tree":
            c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8])
            c["T"] = _log(rng, 1, 64)
            c["hi"] = _log(rng, 16, 65536)
            c["lo"] = rng.randint(0, c["hi"])
            need = c["hi"] + c["T"]
        else:
            c["T"] = _log(rng, 1, 64)
            c["n"] = rng.randint(1, (c["T"] + 1) // 2)
            c["lo"], c["hi"] = 0, _log(rng, 16, 4000)
            need = c["hi"] + c["T"]
        # an e4m3 cache holds a multiple of 16 tokens; a bf16 one any number
        c["cap"] = (need + 15) // 16 * 16 if c["fmt"] == "e4m3" else need
        held = c["B"] * c["Hkv"] * c["cap"] * c["d"]
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and held <= 1.2 * 4 * 8 * 65552 * 128:
            return c


def _spread(c, count, lo, hi):
    """`count` whole numbers over [lo, hi], both ends among them: the lengths
    of a ragged batch.  They follow from the case; a seed orders them."""
    if count == 1:
        return [hi]
    return [lo + round((hi - lo) * ((i * 0.6180339887) % 1.0)) if 0 < i < count - 1 else (lo if i == 0 else hi)
            for i in range(count)]


def _counts(c):
    """New rows of each sequence of a write, or rows read of each sequence."""
    if c["op"] == "write":
        return _spread(c, c["B"], (c["N"] + 1) // 2, c["N"]) if c["ragged"] else [c["N"]] * c["B"]
    return _spread(c, c["B"], c["lo"], c["hi"]) if c["ragged"] else [c["hi"]] * c["B"]


def work(c):
    """Bytes and operations of one pass that no implementation can avoid."""
    row = c["d"] + 1 if c["fmt"] == "e4m3" else 2 * c["d"]  # one row of one cache
    if c["op"] == "write":
        return {"bytes": 2 * c["Hkv"] * sum(_counts(c)) * (2 * c["d"] + row), "flops": 0}
    if c["op"] == "read":  # rows past a sequence's count are written as zeros
        return {"bytes": 2 * c["Hkv"] * (sum(_counts(c)) * row + c["B"] * c["N"] * 2 * c["d"]), "flops": 0}
    if c["op"] == "tree":
        keys = sum(n + c["T"] for n in _spread(c, c["B"], c["lo"], c["hi"]))
        rows = c["B"] * c["Hq"] * c["T"]
        return {"bytes": 2 * c["Hkv"] * keys * row + rows * (4 * c["d"] + 4),
                "flops": 4 * c["Hq"] * c["T"] * keys * c["d"]}
    n = sum(_spread(c, c["B"], 1, c["n"]))
    return {"bytes": 4 * c["Hkv"] * n * row + 8 * c["B"], "flops": 0}


# ---------------------------------------------------------------- inputs
def _pow2(e):
    """2^e in fp32 for whole numbers e of -126 .. 127, from the bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """(e4m3 codes, scale bytes) of rows x [..., d]: 2^e is the least power of
    two with max|x| 2^-e <= 448, codes are x 2^-e rounded to nearest even."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # max|x| = m 2^e, 1/2 <= m < 1
    e = torch.where(m > F8_MAX / 512, e - 8, e - 9)
    e = torch.where(m == 0, E_MIN, e).clamp(E_MIN, E_MAX)
    codes = (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + BIAS).to(torch.uint8)


def _dequantise(codes, scale):
    return codes.float() * _pow2(scale.int() - BIAS)[..., None]


def _bf16(g, *shape, outliers=False):
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:  # keys: a few channels carry much larger values
        x *= 1.0 + 5.0 * (torch.rand(shape[-1], generator=g, device="cuda") > 0.95)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    B, H, cap, d = c["B"], c["Hkv"], c["cap"], c["d"]

    def ints(values):
        return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=cpu)].cuda()

    s = dict(case=c)
    if c["op"] == "write":  # a fresh cache, and new keys and values
        s["new_k"], s["new_v"] = _bf16(g, B, H, c["N"], d, outliers=True), _bf16(g, B, H, c["N"], d)
        s["lens"] = ints(_spread(c, B, c["lo"], c["hi"]))
        s["counts"] = ints(_counts(c)) if c["ragged"] else None
        k = torch.zeros(B, H, cap, d, dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
    else:  # a cache that holds tokens
        k, v = _bf16(g, B, H, cap, d, outliers=True), _bf16(g, B, H, cap, d)
    if c["fmt"] == "e4m3":
        (s["k"], s["k_scale"]), (s["v"], s["v_scale"]) = _quantise(k), _quantise(v)
    else:
        s["k"], s["v"], s["k_scale"], s["v_scale"] = k, v, None, None
    if c["op"] == "read":
        s["counts"] = ints(_counts(c))
        s["first"] = torch.randint(0, cap - c["N"] + 1, (B,), generator=cpu, dtype=torch.int32).cuda()
    if c["op"] in ("tree", "commit"):
        s["lens"] = ints(_spread(c, B, c["lo"], c["hi"]))
    if c["op"] == "tree":
        T = c["T"]
        s["q"] = _bf16(g, B, c["Hq"], T, d)
        # a random tree: token i's parent is one of those before it
        masks = torch.zeros(B, T, dtype=torch.int64)
        for i in range(T):
            up = torch.randint(0, i, (B,), generator=cpu) if i else None
            bit = -(1 << 63) if i == 63 else 1 << i
            masks[:, i] = (masks[torch.arange(B), up] if i else 0) | bit
        s["mask"] = masks.cuda()
        s["scale"] = 1.0 / math.sqrt(d)
    if c["op"] == "commit":
        # the root (draft 0), then drafts that lie behind the committed rows:
        # a pass can be run again on what it left
        n, T = c["n"], c["T"]
        path = torch.zeros(B, T, dtype=torch.int32)
        for b in range(B):
            later = n + torch.randperm(T - n, generator=cpu)[: n - 1].sort().values
            path[b, 1 : 1 + len(later)] = later.int()
        s["path"] = path.cuda()
        s["n_accept"] = ints(_spread(c, B, 1, n))
    return s


# ---------------------------------------------------------------- plain forms
def _rows(cache, at):
    """Rows `at` [B, n] of a cache tensor [B, H, cap, ...], as [B, n, H, ...]."""
    b = torch.arange(cache.shape[0], device=cache.device)[:, None]
    return cache.transpose(1, 2)[b, at]


def _store(cache, at, rows, keep):
    """Rows [B, n, H, ...] where `keep` [B, n] holds; the others stay."""
    b = torch.arange(cache.shape[0], device=cache.device)[:, None]
    keep = keep.reshape(keep.shape + (1,) * (rows.dim() - 2))
    view = cache.transpose(1, 2)
    view[b, at] = torch.where(keep, rows, view[b, at])


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _plain_write(s):
    c = s["case"]
    i = torch.arange(c["N"], device="cuda")[None]
    at = s["lens"][:, None].long() + i
    keep = i < (s["counts"][:, None] if s["counts"] is not None else c["N"])
    keep = keep.expand(c["B"], c["N"])
    for x, cache, scale in ((s["new_k"], s["k"], s["k_scale"]), (s["new_v"], s["v"], s["v_scale"])):
        x = x.transpose(1, 2)
        if scale is not None:
            x, e = _quantise(x)
            _store(scale, at, e, keep)
        _store(_bytes(cache), at, _bytes(x), keep)
    return _cache(s)


def _plain_read(s):
    c = s["case"]
    i = torch.arange(c["N"], device="cuda")[None]
    at = s["first"][:, None].long() + i
    keep = (i < s["counts"][:, None])[:, :, None, None]
    out = []
    for cache, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        x = _rows(_bytes(cache), at)
        x = x.float() if scale is None else _dequantise(x.view(torch.float8_e4m3fn), _rows(scale, at))
        out.append(torch.where(keep, x, 0.0).transpose(1, 2).to(torch.bfloat16).contiguous())
    return out


def _visible(s):
    """[B, T, cap]: which cache position each drafted token sees."""
    c = s["case"]
    j = torch.arange(c["cap"], device="cuda")[None, None] - s["lens"][:, None, None].long()
    drafted = (s["mask"][:, :, None] >> j.clamp(0, 63)) & 1
    return (j < 0) | ((j < c["T"]) & (drafted != 0))


def _plain_tree(s):
    c = s["case"]
    B, H, T, d, G = c["B"], c["Hkv"], c["T"], c["d"], c["Hq"] // c["Hkv"]
    k, v = s["k"], s["v"]
    k = k.float() if s["k_scale"] is None else _dequantise(k, s["k_scale"])
    v = v.float() if s["v_scale"] is None else _dequantise(v, s["v_scale"])
    q = s["q"].float().reshape(B, H, G * T, d)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(B, H, G, T, c["cap"])
    x.masked_fill_(~_visible(s)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.clamp(min=-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * T, c["cap"]), v).view(B, H, G, T, d)
    o = torch.where(l > 0, o / l, 0.0).reshape(B, c["Hq"], T, d).to(torch.bfloat16)
    return {"o": o, "lse": (m + l.log()).reshape(B, c["Hq"], T)}


def _plain_commit(s):
    c = s["case"]
    i = torch.arange(c["T"], device="cuda")[None]
    lens = s["lens"][:, None].long()
    keep = i < s["n_accept"][:, None]
    for t in (s["k"], s["v"], s["k_scale"], s["v_scale"]):
        if t is not None:
            t = _bytes(t)
            _store(t, lens + i, _rows(t, lens + s["path"].long()), keep)
    return dict(_cache(s), lens=s["lens"] + s["n_accept"])


def _cache(s):
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale") if s[n] is not None}


# ---------------------------------------------------------------- the library
def _handle(s):
    """The cache object that a serving program keeps beside its tensors."""
    if "handle" not in s:
        import exact_io_aware_16_gb300 as fa

        s["fa"] = fa
        s["handle"] = fa.KvCache.from_tensors(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["fa"], s["handle"]


def _own_run(s):
    fa, cache = _handle(s)
    op = s["case"]["op"]
    if op == "write":
        fa.fa_cache_write(cache, s["new_k"], s["new_v"], lens=s["lens"], counts=s["counts"])
        return _cache(s)
    if op == "read":
        return list(fa.fa_cache_read(cache, s["case"]["N"], first=s["first"], counts=s["counts"]))
    if op == "tree":
        o, lse = fa.fa_decode_tree(cache, s["q"], s["mask"], lens=s["lens"], scale=s["scale"])
        return {"o": o, "lse": lse}
    lens = fa.fa_cache_commit(cache, s["path"], s["n_accept"], lens=s["lens"], new_lens=torch.empty_like(s["lens"]))
    return dict(_cache(s), lens=lens)


def run(state):
    if own:
        return _own_run(state)
    return {"write": _plain_write, "read": _plain_read, "tree": _plain_tree, "commit": _plain_commit}[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _value64(s, name):
    """A cache tensor's values in 64 bits, from the bits of its codes."""
    t = s[name]
    if s[name + "_scale"] is None:
        return t.double()
    b = t.view(torch.uint8).long()
    ex, ma = (b >> 3) & 15, b & 7
    x = torch.where(ex > 0, (8 + ma).double() * _pow2_64(ex - 10), ma.double() * 2.0**-9)
    x = torch.where(b > 127, -x, x)
    return x * _pow2_64(s[name + "_scale"].long() - BIAS)[..., None]


def _codes64(x):
    """(values of the codes, exponents) of rows x in 64 bits, from the
    definition: e by logarithm, corrected at the borders, and codes by rounding
    to the step of each value's binade."""
    a = x.abs().amax(-1)
    e = torch.ceil(torch.log2(a.clamp(min=2.0**-140) / F8_MAX))
    e = torch.where(a > F8_MAX * _pow2_64(e), e + 1, e)
    e = torch.where(a <= F8_MAX * _pow2_64(e - 1), e - 1, e).clamp(E_MIN, E_MAX)
    y = x / _pow2_64(e)[..., None]
    _, binade = torch.frexp(y.abs().clamp(min=2.0**-6))
    step = _pow2_64(binade - 4)
    return torch.round(y / step) * step, e


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, H, G = c["B"], c["Hkv"], c.get("Hq", 0) // c["Hkv"]
    if c["op"] == "write":
        out = {}
        for n in ("k", "v"):
            new = s["new_" + n].double()
            held, scale = s[n].double(), s[n + "_scale"]
            codes, e = _codes64(new) if scale is not None else (new, None)
            for b in range(B):
                at, m = int(s["lens"][b]), int(s["counts"][b]) if s["counts"] is not None else c["N"]
                held[b, :, at : at + m] = codes[b, :, :m]
                if scale is not None:
                    scale[b, :, at : at + m] = (e[b, :, :m] + BIAS).to(torch.uint8)
            out[n] = held
            if scale is not None:
                out[n + "_scale"] = scale
        return out
    if c["op"] == "read":
        out = []
        for n in ("k", "v"):
            held = _value64(s, n)
            x = torch.zeros(B, H, c["N"], c["d"], dtype=torch.float64, device="cuda")
            for b in range(B):
                at, m = int(s["first"][b]), int(s["counts"][b])
                x[b, :, :m] = held[b, :, at : at + m]
            out.append(x)
        return out
    if c["op"] == "tree":
        T, d = c["T"], c["d"]
        o = torch.zeros(B, c["Hq"], T, d, dtype=torch.float64, device="cuda")
        lse = torch.full((B, c["Hq"], T), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(s["lens"][b])
            one = {x: (s[x][b : b + 1, :, : n + T] if s[x] is not None else None) for x in ("k", "v", "k_scale", "v_scale")}
            k, v = _value64(one, "k")[0], _value64(one, "v")[0]
            seen = torch.ones(T, n + T, dtype=torch.bool)
            for t in range(T):
                bits = int(s["mask"][b, t]) & (2**64 - 1)
                seen[t, n:] = torch.tensor([bits >> j & 1 for j in range(T)], dtype=torch.bool)
            seen = seen.cuda()
            for h in range(H):
                q = s["q"][b, h * G : (h + 1) * G].double()
                x = (q @ k[h].T) * s["scale"]
                x = torch.where(seen[None], x, -math.inf)
                lse[b, h * G : (h + 1) * G] = torch.logsumexp(x, -1)
                o[b, h * G : (h + 1) * G] = torch.softmax(x, -1) @ v[h]
        return {"o": o, "lse": lse}
    out = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        if s[n] is not None:
            t = s[n].clone() if n.endswith("scale") else s[n].double()
            for b in range(B):
                at, m = int(s["lens"][b]), int(s["n_accept"][b])
                t[b, :, at : at + m] = t[b, :, at + s["path"][b, :m].long()].clone()
            out[n] = t
    out["lens"] = s["lens"] + s["n_accept"]
    return out
