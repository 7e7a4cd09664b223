"""What the operators of packed sequences are measured on: attention of sequences
of different lengths that lie one behind the other, with grouped heads, alone
(a prompt, a chunk of one) and with its backward pass; the rotation of queries
and keys by their positions; and that rotation with a norm of each head before it,
forward and backward.

`run` computes them in plain torch operations, or, where `own` is true, with
the library's kernels.  `prepare` makes the inputs of a case from a seed.
"""
import math

import torch

own = False

EPS = 1e-6  # of the norms


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short line enters an empty conversation: latency
        dict(name="prompt_line", op="prompt", seqs=1, lo=17, hi=17, past=0, Hq=32, Hkv=8, d=128, causal=True, fused=True),
        # the prompts of many requests at once, one token to two thousand each
        dict(name="prompt_ragged", op="prompt", seqs=24, lo=1, hi=2048, past=0, Hq=32, Hkv=8, d=128, causal=True, fused=True),
        # two long documents
        dict(name="prompt_long", op="prompt", seqs=2, lo=8192, hi=8192, past=0, Hq=32, Hkv=8, d=128, causal=True, fused=True),
        # follow-up turns: some hundred new tokens each, over what was said before
        dict(name="prompt_chunk", op="prompt", seqs=16, lo=40, hi=500, past=8000, Hq=28, Hkv=4, d=128, causal=True, fused=False),
        # a training step of many short samples, small heads
        dict(name="train_short", op="train", seqs=64, lo=1, hi=512, past=0, Hq=12, Hkv=12, d=64, causal=True, fused=True),
        # a training step of a few long samples
        dict(name="train_long", op="train", seqs=4, lo=1000, hi=8192, past=0, Hq=32, Hkv=8, d=128, causal=True, fused=True),
        # an encoder's step: all tokens of a sample see each other, empty samples among them
        dict(name="train_encoder", op="train", seqs=31, lo=0, hi=1500, past=0, Hq=16, Hkv=2, d=64, causal=False, fused=False),
        # the next token of eight sequences, far into their contexts: latency
        dict(name="rotary_token", op="rotary", seqs=8, tokens=1, far=100000, Hq=32, Hkv=8, d=128, rot=128, pairs="half", scaling="none", back=False, fused=False),
        # a training step's tokens, half of each head turned, stretched for a longer context
        dict(name="rotary_train", op="rotary", seqs=2, tokens=8192, far=0, Hq=32, Hkv=8, d=128, rot=64, pairs="interleaved", scaling="linear", back=True, fused=True),
        # the next token of sixty-four sequences
        dict(name="norm_token", op="norm", seqs=64, tokens=1, far=30000, Hq=32, Hkv=8, d=128, rot=128, pairs="half", scaling="none", back=False, fused=False),
        # an odd number of tokens, small heads, part of each turned
        dict(name="norm_odd", op="norm", seqs=7, tokens=143, far=5000, Hq=12, Hkv=12, d=64, rot=48, pairs="half", scaling="turns", back=True, fused=True),
        # a training step's tokens
        dict(name="norm_train", op="norm", seqs=2, tokens=8192, far=0, Hq=32, Hkv=8, d=128, rot=128, pairs="half", scaling="index", back=True, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of these ranges, no costlier than the largest listed one."""
    while True:
        op = rng.choice(["prompt", "prompt", "train", "train", "rotary", "norm", "norm"])
        c = dict(op=op, d=rng.choice([64, 128]), Hkv=rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), fused=rng.random() < 0.5)
        c["Hq"] = c["Hkv"] * rng.choice([1, 1, 2, 3, 4, 6, 7, 8])
        c["seqs"] = _log(rng, 1, 64)
        if op in ("prompt", "train"):
            # gradients of queries and keys are zero where a token sees itself alone
            c["hi"] = _log(rng, 1 if op == "prompt" else 8, 8192)
            c["lo"] = rng.choice([0, rng.randint(0, c["hi"]), c["hi"]])
            c["past"] = _log(rng, 1, 8192) if op == "prompt" and rng.random() < 0.4 else 0
            c["causal"] = rng.random() < 0.75
        else:
            c["tokens"] = _log(rng, 1, 8192)
            c["far"] = _log(rng, 1, 1000000)
            c["rot"] = c["d"] if rng.random() < 0.5 else 16 * rng.randint(1, c["d"] // 16)
            c["pairs"] = rng.choice(["half", "half", "interleaved"])
            c["scaling"] = rng.choice(["none", "none", "linear", "base", "turns", "index"])
            c["back"] = rng.random() < 0.5
        if c["Hq"] > 64 or (op in ("prompt", "train") and sum(_lengths(c)[0]) == 0):
            continue
        most = [max(work(x)[k] for x in listed() if x["op"] == op) for k in ("bytes", "flops")]
        w = work(c)
        # the plain form works on whole rectangles of queries and keys
        area = sum(n * m for n, m in zip(*_lengths(c))) * c["Hq"] if op in ("prompt", "train") else 0
        if w["bytes"] <= most[0] and w["flops"] <= most[1] and area <= 32 * 2 * 8192**2 // (1 if op == "prompt" else 2):
            return c


def _spread(count, lo, hi):
    """`count` whole numbers over [lo, hi], both ends among them: the lengths
    of a ragged batch.  They follow from the case; a seed orders them."""
    if count == 1:
        return [hi]
    return [lo + round((hi - lo) * ((i * 0.6180339887) % 1.0)) if 0 < i < count - 1 else (lo if i == 0 else hi)
            for i in range(count)]


def _lengths(c):
    """Queries and keys of each sequence: the keys are those of the tokens
    before, if any, and of the queries' own tokens."""
    new = _spread(c["seqs"], c["lo"], c["hi"])
    if not c["past"]:
        return new, new
    before = _spread(c["seqs"], c["past"] // 4, c["past"])
    return new, [n + b for n, b in zip(new, before[::-1])]


def work(c):
    """Bytes and operations of one pass that no implementation can avoid."""
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    if c["op"] in ("prompt", "train"):
        new, keys = _lengths(c)
        seen = sum(n * (m - n) + n * (n + 1) // 2 if c["causal"] else n * m for n, m in zip(new, keys))
        q, kv = 2 * sum(new) * Hq * d, 2 * sum(keys) * Hkv * d
        lse = 4 * sum(new) * Hq
        if c["op"] == "prompt":  # q, k, v -> o, lse
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * seen * Hq * d}
        # q, k, v, do -> o, lse, dq, dk, dv
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * seen * Hq * d}
    tokens = c["seqs"] * c["tokens"]
    elements = tokens * (Hq + Hkv) * d
    if c["op"] == "rotary":
        turned = tokens * (Hq + Hkv) * c["rot"]
        return {"bytes": (8 if c["back"] else 4) * elements + 4 * tokens, "flops": (6 if c["back"] else 3) * turned}
    # a step reads q, k and the gradients of the results, and writes q, k and their gradients
    return {"bytes": (8 if c["back"] else 4) * elements + 4 * tokens + (16 if c["back"] else 8) * d,
            "flops": (20 if c["back"] else 7) * elements}


# ---------------------------------------------------------------- inputs
def _bf16(g, *shape, outliers=False):
    x = torch.randn(shape, generator=g, device="cuda")
    if outliers:  # keys: a few channels carry much larger values
        x *= 1.0 + 5.0 * (torch.rand(shape[-1], generator=g, device="cuda") > 0.95)
    return x.to(torch.bfloat16)


def _qkv(g, c, tokens, keys):
    """Queries, keys and values by token and head: three tensors, or, as a
    projection of all three leaves them, parts of one."""
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["fused"] and tokens == keys:
        x = _bf16(g, tokens, Hq + 2 * Hkv, d)
        x[:, Hq : Hq + Hkv] = _bf16(g, tokens, Hkv, d, outliers=True)
        return x[:, :Hq], x[:, Hq : Hq + Hkv], x[:, Hq + Hkv :]
    return _bf16(g, tokens, Hq, d), _bf16(g, keys, Hkv, d, outliers=True), _bf16(g, keys, Hkv, d)


def _starts(lengths):
    """Where each of the sequences starts, and the end of the last."""
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] in ("prompt", "train"):
        order = torch.randperm(c["seqs"], generator=cpu).tolist()
        new, keys = ([x[i] for i in order] for x in _lengths(c))
        s["at_q"], s["at_k"] = _starts(new), _starts(keys)
        s["cu_q"] = torch.tensor(s["at_q"], dtype=torch.int32).cuda()
        s["cu_k"] = torch.tensor(s["at_k"], dtype=torch.int32).cuda() if c["past"] else s["cu_q"]
        s["q"], s["k"], s["v"] = _qkv(g, c, sum(new), sum(keys))
        if c["op"] == "train":
            s["do"] = _bf16(g, sum(new), c["Hq"], c["d"])
        s["scale"] = 1.0 / math.sqrt(c["d"])
        return s
    tokens, Hq, Hkv, d = c["seqs"] * c["tokens"], c["Hq"], c["Hkv"], c["d"]
    first = torch.randint(0, c["far"] + 1, (c["seqs"], 1), generator=cpu, dtype=torch.int32)
    at = (first + torch.arange(c["tokens"], dtype=torch.int32)).cuda()
    s["freqs"] = _frequencies(c)
    s["amplitude"] = _amplitude(c)
    if c["tokens"] == 1:  # a serving step: [sequences, heads, 1, d]
        s["q"], s["k"] = _bf16(g, c["seqs"], Hq, 1, d), _bf16(g, c["seqs"], Hkv, 1, d, outliers=True)
        s["positions"] = at
    else:
        s["q"], s["k"], _ = _qkv(g, c, tokens, tokens)
        s["positions"] = at.reshape(-1)
    if c["op"] == "norm":
        for n in ("q", "k"):
            s[n + "_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
    if c["back"]:
        s["dq"], s["dk"] = (_bf16(g, *s[n].shape) for n in ("q", "k"))
    return s


# The long context that a scaled table is made for: `factor` times the
# `original` one; of the frequencies that turn less than `low` times within the
# original context all are divided by factor, of those above `high` none.
SCALES = dict(none={}, linear=dict(factor=4.0), base=dict(factor=8.0),
              turns=dict(factor=8.0, original=8192.0, low=1.0, high=4.0),
              index=dict(factor=16.0, original=4096.0, low=1.0, high=32.0))
BASE = 10000.0


def _amplitude(c):
    return 0.1 * math.log(SCALES["index"]["factor"]) + 1.0 if c["scaling"] == "index" else 1.0


def _frequencies(c):
    """Radians a position of each pair, 64 bits."""
    rot, kind = c["rot"], c["scaling"]
    x = SCALES[kind]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2.0 * i / rot)
    if kind == "linear":
        f = f / x["factor"]
    elif kind == "base":
        f = (BASE * x["factor"] ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
    elif kind == "turns":
        keep = ((x["original"] * f / (2 * math.pi) - x["low"]) / (x["high"] - x["low"])).clamp(0, 1)
        f = f * (keep + (1 - keep) / x["factor"])
    elif kind == "index":
        ends = [rot * math.log(x["original"] / (t * 2 * math.pi)) / (2 * math.log(BASE)) for t in (x["high"], x["low"])]
        a, b = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
        keep = 1 - ((i - a) / max(b - a, 1e-3)).clamp(0, 1)
        f = f * (keep + (1 - keep) / x["factor"])
    return f


# ---------------------------------------------------------------- plain forms
def _sequences(s):
    """(queries, keys) of each sequence, as slices; none of those without queries."""
    for a, b, x, y in zip(s["at_q"], s["at_q"][1:], s["at_k"], s["at_k"][1:]):
        if b > a:
            yield slice(a, b), slice(x, y)


def _groups(c, n, m):
    """Key heads at a time: as many as keep the scores within 4 GB."""
    G = c["Hq"] // c["Hkv"]
    step = max(1, min(c["Hkv"], (1 << 30) // max(1, G * n * m)))
    return [(h, min(h + step, c["Hkv"])) for h in range(0, c["Hkv"], step)]


def _rows(x, part, heads, G):
    """[heads, G * tokens, d] in 32 bits of the given tokens and key heads of x."""
    x = x[part, heads[0] * G : heads[1] * G].float()
    n, H, d = x.shape
    return x.view(n, H // G, G, d).permute(1, 2, 0, 3).reshape(H // G, G * n, d)


def _back(x, G):
    """[heads, G * n, d] -> [n, heads * G, d] in bf16."""
    H, r, d = x.shape
    return x.view(H, G, r // G, d).permute(2, 0, 1, 3).reshape(r // G, H * G, d).to(torch.bfloat16)


def _scores(s, q, k, n, m, G):
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    if s["case"]["causal"]:
        i = torch.arange(n, device="cuda")[:, None] + (m - n)
        hidden = torch.arange(m, device="cuda")[None] > i
        x.view(-1, G, n, m).masked_fill_(hidden, -math.inf)
    return x


def _plain_attention(s):
    c = s["case"]
    G, train = c["Hq"] // c["Hkv"], c["op"] == "train"
    tq, tk, d = s["at_q"][-1], s["at_k"][-1], c["d"]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    out = dict(o=torch.zeros(tq, c["Hq"], d, **bf), lse=torch.full((c["Hq"], tq), -math.inf, device="cuda"))
    if train:
        out.update(dq=torch.zeros(tq, c["Hq"], d, **bf), dk=torch.zeros(tk, c["Hkv"], d, **bf), dv=torch.zeros(tk, c["Hkv"], d, **bf))
    for new, keys in _sequences(s):
        n, m = new.stop - new.start, keys.stop - keys.start
        for h in _groups(c, n, m):
            heads = slice(h[0] * G, h[1] * G)
            q, k, v = _rows(s["q"], new, h, G), _rows(s["k"], keys, h, 1), _rows(s["v"], keys, h, 1)
            p = _scores(s, q, k, n, m, G)
            top = p.amax(-1, keepdim=True)
            p = p.sub_(top).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l)
            o = torch.matmul(p, v)
            out["o"][new, heads] = _back(o, G)
            out["lse"][heads, new] = (top + l.log()).view(-1, n)
            if train:
                do = _rows(s["do"], new, h, G)
                out["dv"][keys, h[0] : h[1]] = _back(torch.matmul(p.transpose(-1, -2), do), 1)
                dp = torch.matmul(do, v.transpose(-1, -2))
                ds = dp.sub_((o * do).sum(-1, keepdim=True)).mul_(p)
                out["dq"][new, heads] = _back(torch.matmul(ds, k).mul_(s["scale"]), G)
                out["dk"][keys, h[0] : h[1]] = _back(torch.matmul(ds.transpose(-1, -2), q).mul_(s["scale"]), 1)
    return out


def _turns(s):
    """Cosines and sines of each token's angles [..., rot / 2], found in 64 bits
    (far positions turn many times) and kept in 32."""
    a = s["positions"].double()[..., None] * s["freqs"]
    cos, sin = a.cos().float() * s["amplitude"], a.sin().float() * s["amplitude"]
    return cos[:, None], sin[:, None]  # the same for all heads


def _rotate(c, x, cos, sin):
    """x in 32 bits, its first `rot` elements turned: the pairs are the two
    halves of them, or neighbours."""
    r = c["rot"]
    if c["pairs"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rotary(s):
    c = s["case"]
    cos, sin = _turns(s)
    out = {n: _rotate(c, s[n].float(), cos, sin).to(torch.bfloat16) for n in ("q", "k")}
    if c["back"]:
        out.update({n: _rotate(c, s[n].float(), cos, -sin).to(torch.bfloat16) for n in ("dq", "dk")})
    return out


def _plain_norm(s):
    c = s["case"]
    cos, sin = _turns(s)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
        x = x * r
        out[n] = _rotate(c, x * w, cos, sin).to(torch.bfloat16)
        if c["back"]:
            g = _rotate(c, s["d" + n].float(), cos, -sin)
            out["d" + n + "_weight"] = (g * x).sum(tuple(range(x.dim() - 1)))
            g = g * w
            out["d" + n] = (r * (g - x * (g * x).mean(-1, keepdim=True))).to(torch.bfloat16)
    return out


# ---------------------------------------------------------------- the library
def _handle(s):
    """The table of rotations that a program keeps beside its weights."""
    if "handle" not in s:
        import exact_io_aware_16_gb300 as fa

        c = s["case"]
        s["fa"] = fa
        if "rot" in c:
            scaling = None if c["scaling"] == "none" else c["scaling"]
            s["handle"] = fa.Rotary(c["d"], rot=c["rot"], base=BASE, interleaved=c["pairs"] == "interleaved",
                                    scaling=scaling, amplitude=s["amplitude"], **SCALES[c["scaling"]])
        else:
            s["handle"] = None
    return s["fa"], s["handle"]


def _own_run(s):
    fa, table = _handle(s)
    c = s["case"]
    if c["op"] in ("prompt", "train"):
        cu_k = s["cu_k"] if c["past"] else None
        o, lse = fa.fa_forward_packed(s["q"], s["k"], s["v"], s["cu_q"], cu_k, causal=c["causal"], scale=s["scale"])
        if c["op"] == "prompt":
            return dict(o=o, lse=lse)
        dq, dk, dv = fa.fa_backward_packed(s["q"], s["k"], s["v"], o, s["do"], lse, s["cu_q"], cu_k, causal=c["causal"], scale=s["scale"])
        return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    at = s["positions"]
    if c["op"] == "rotary":
        q, k = fa.fa_rotary(table, s["q"], s["k"], at)
        if not c["back"]:
            return dict(q=q, k=k)
        dq, dk = fa.fa_rotary_backward(table, s["dq"], s["dk"], at)
        return dict(q=q, k=k, dq=dq, dk=dk)
    wq, wk = s["q_weight"], s["k_weight"]
    q, k = fa.fa_norm_rotary(table, s["q"], s["k"], at, wq, wk, eps=EPS)
    if not c["back"]:
        return dict(q=q, k=k)
    dq, dk, dwq, dwk = fa.fa_norm_rotary_backward(table, s["dq"], s["dk"], s["q"], s["k"], at, wq, wk, eps=EPS)
    return dict(q=q, k=k, dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk)


def run(state):
    if own:
        return _own_run(state)
    return {"rotary": _plain_rotary, "norm": _plain_norm}.get(state["case"]["op"], _plain_attention)(state)


# ---------------------------------------------------------------- 64 bits
def _exact_attention(c, s):
    """Head by head, from the definition: softmax and its derivative."""
    G, train = c["Hq"] // c["Hkv"], c["op"] == "train"
    f64 = dict(dtype=torch.float64, device="cuda")
    shape_q, shape_k = s["q"].shape, s["k"].shape
    out = dict(o=torch.zeros(shape_q, **f64), lse=torch.full((c["Hq"], shape_q[0]), -math.inf, **f64))
    if train:
        out.update(dq=torch.zeros(shape_q, **f64), dk=torch.zeros(shape_k, **f64), dv=torch.zeros(shape_k, **f64))
    for b in range(c["seqs"]):
        q0, q1, k0, k1 = s["at_q"][b], s["at_q"][b + 1], s["at_k"][b], s["at_k"][b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0 or m == 0:
            continue
        seen = torch.ones(n, m, dtype=torch.bool, device="cuda")
        if c["causal"]:
            seen = seen.tril(m - n)
        for h in range(c["Hq"]):
            q, k, v = s["q"][q0:q1, h].double(), s["k"][k0:k1, h // G].double(), s["v"][k0:k1, h // G].double()
            x = torch.where(seen, (q @ k.T) * s["scale"], -math.inf)
            out["lse"][h, q0:q1] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            out["o"][q0:q1, h] = p @ v
            if train:
                do = s["do"][q0:q1, h].double()
                out["dv"][k0:k1, h // G] += p.T @ do
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True))
                out["dq"][q0:q1, h] = (ds @ k) * s["scale"]
                out["dk"][k0:k1, h // G] += (ds.T @ q) * s["scale"]
    return out


def _exact_frequency(c, i):
    """Radians a position of pair i, by the scaling's definition."""
    x, rot, f = SCALES[c["scaling"]], c["rot"], BASE ** (-2.0 * i / c["rot"])
    if c["scaling"] == "none":
        return f
    if c["scaling"] == "linear":
        return f / x["factor"]
    if c["scaling"] == "base":  # pair 0 as it is, the last pair factor times slower
        return f * x["factor"] ** (-2.0 * i / (rot - 2.0))
    if c["scaling"] == "turns":
        t = x["original"] * f / (2 * math.pi)
        share = min(max((t - x["low"]) / (x["high"] - x["low"]), 0.0), 1.0)
    else:
        # the pairs that turn `high` and `low` times within the original context
        def at(t):
            return rot / 2 * math.log(x["original"] / (2 * math.pi * t), BASE)

        a, b = max(math.floor(at(x["high"])), 0), min(math.ceil(at(x["low"])), rot - 1)
        share = 1.0 - min(max((i - a) / max(b - a, 1e-3), 0.0), 1.0)
    return share * f + (1.0 - share) * f / x["factor"]


def _exact_turn(c, s, x, sign):
    """x in 64 bits with each pair turned as one complex number."""
    r = c["rot"]
    f = torch.tensor([_exact_frequency(c, i) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    a = sign * s["positions"].double()[..., None] * f
    z = torch.polar(torch.full_like(a, _amplitude(c)), a)[:, None]
    if c["pairs"] == "half":
        y = torch.complex(x[..., : r // 2], x[..., r // 2 : r]) * z
        return torch.cat([y.real, y.imag, x[..., r:]], -1)
    y = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * z).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("prompt", "train"):
        return _exact_attention(c, s)
    out = {}
    for n in ("q", "k"):
        x = s[n].double()
        if c["op"] == "rotary":
            out[n] = _exact_turn(c, s, x, 1.0)
            if c["back"]:
                out["d" + n] = _exact_turn(c, s, s["d" + n].double(), -1.0)
            continue
        w = s[n + "_weight"].double()
        rms = torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        out[n] = _exact_turn(c, s, x / rms * w, 1.0)
        if c["back"]:
            g = _exact_turn(c, s, s["d" + n].double(), -1.0)
            out["d" + n + "_weight"] = (g * x / rms).flatten(0, -2).sum(0)
            g = g * w
            # y = x / rms: dx = g / rms - x (g . x) / (d rms^3)
            out["d" + n] = g / rms - x * (g * x).sum(-1, keepdim=True) / (c["d"] * rms**3)
    return out
