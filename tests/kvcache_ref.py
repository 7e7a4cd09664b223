"""Plain fp64 definitions of the key/value cache operators (numpy, test code).

A cache row of e4m3 codes c and scale byte s stands for c * 2^(s - 127); the
writer takes the least exponent with max|x| 2^-e <= 448 (finite elements,
-100 .. 119) and rounds x 2^-e to nearest even.
"""
import numpy as np
import torch

E_MIN, E_MAX = -100, 119


def code_values():
    """The 256 e4m3 values by code (0x7f and 0xff: NaN)."""
    v = np.empty(256)
    for c in range(256):
        ex, ma = c >> 3 & 15, c & 7
        x = (8 + ma) * 2.0 ** (ex - 10) if ex else ma * 2.0 ** -9
        v[c] = np.nan if c & 127 == 127 else (-x if c > 127 else x)
    return v


CODES = code_values()
POSITIVE = CODES[:127]  # ascending


def to64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def quantise(x):
    """(codes uint8, scale bytes uint8) of rows x [..., d] (fp64 of bf16)."""
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = fin.max(-1)
    e = np.full(amax.shape, E_MIN)
    pos = amax > 0
    ea = np.floor(np.log2(np.where(pos, amax, 1.0))).astype(int) - 10
    for _ in range(4):  # the least e with amax 2^-e <= 448
        ea = np.where(np.where(pos, amax, 0.0) > 448.0 * 2.0 ** ea, ea + 1, ea)
    e = np.clip(np.where(pos, ea, E_MIN), E_MIN, E_MAX)
    with np.errstate(invalid="ignore"):
        y = np.minimum(np.abs(x) * 2.0 ** -e[..., None].astype(float), 448.0)
    y0 = np.where(np.isfinite(x), y, 0.0)
    hi = np.clip(np.searchsorted(POSITIVE, y0, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = y0 - POSITIVE[lo], POSITIVE[hi] - y0
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))  # codes order by value: ties to the even code
    c = np.where(up, hi, lo)
    c = np.where(y0 == 0, 0, c) | (np.signbit(x) * 128)
    c = np.where(np.isfinite(x), c, 127).astype(np.uint8)
    return c, (e + 127).astype(np.uint8)


def dequantise(codes, scale):
    return CODES[codes] * 2.0 ** (scale.astype(float) - 127)[..., None]


def codes_np(t):
    """uint8 codes of a float8 tensor, NaN codes without their sign."""
    c = t.view(torch.uint8).cpu().numpy().copy()
    c[(c & 127) == 127] = 127
    return c


def cache_values(cache):
    """(k, v) of a KvCache in fp64."""
    if cache.format == "bf16":
        return to64(cache.k), to64(cache.v)
    return tuple(dequantise(t.view(torch.uint8).cpu().numpy(), s.cpu().numpy())
                 for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))


def tree(q, k, v, lens, mask, scale, fmt, v_scale=None, qmax=None):
    """(o, lse, o_tol, lse_tol) of fa_decode_tree in fp64.

    q [B,Hq,T,d], k, v [B,Hkv,cap,d] fp64; mask: python ints [B][T].

    The bounds follow from the arithmetic, for the keys a row sees:
     - scores: products are exact and added in fp32 (at most d + 8 roundings or
       truncations of 2^-23 of sum|q k|, scaled); an e4m3 cache splits q into
       two e4m3 pieces of a power-of-two scale.  An element is off by at most 2^-10
       in the units in which the largest |q| of the rows that share a tile (qmax; all
       of q unless given) is in (224, 448], 2^-17.8 of qmax; or, where the rows'
       exponents differ by more than 4, in those of its own row, so by no more than
       2^-12.8 of the row's largest.  ds is the sum of both; e^s is off by at most
       2 ds + 2^-20 (ex2 and the fp32 sums).
     - probabilities: rounded to bf16 (2^-8 of the value), or through fp16 (2^-11)
       to two e4m3 pieces (cut to four bits, the rest rounded to four: 2^-8), where
       the first is subnormal off by at most 2^-13, in units in which the largest
       p_j 2^e_j of the row is 7 .. 448: 2^-15.8 of that largest one, times the codes.
     - o: rounded to bf16 once (2^-8).
    """
    B, Hq, T, d = q.shape
    Hkv, cap = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qmax = np.abs(q).max() if qmax is None else qmax
    o = np.zeros((B, Hq, T, d))
    lse = np.full((B, Hq, T), -np.inf)
    o_tol = np.zeros_like(o)
    lse_tol = np.zeros_like(lse)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        for t in range(T):
            see = list(range(n)) + [n + j for j in range(T) if mask[b][t] >> j & 1 and n + j < cap]
            if not see:
                continue
            for h in range(Hq):
                kk, vv = k[b, h // G, see], v[b, h // G, see]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[b, h, t] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p /= l
                    o[b, h, t] = p @ vv
                    lse[b, h, t] = m + np.log(l)
                    ds = 2.0 ** -23 * (d + 8) * scale * (np.abs(kk) @ np.abs(q[b, h, t])).max()
                    a = p @ np.abs(vv)
                    floor = 0.0
                    if fmt == "e4m3":
                        off = min(2.0 ** -17.8 * qmax, 2.0 ** -12.8 * np.abs(q[b, h, t]).max())
                        ds += off * scale * np.abs(kk).sum(-1).max()
                        w = 2.0 ** (v_scale[b, h // G, see].astype(float) - 127)
                        floor = 2.0 ** -15.8 * (p * w).max() * (np.abs(vv) / w[:, None]).sum(0)
                    each = 2.0 ** -8 if fmt == "bf16" else 2.0 ** -8 + 2.0 ** -11
                    o_tol[b, h, t] = a * (each + 2 * ds + 2.0 ** -18) + floor \
                        + 2.0 ** -8 * 1.02 * np.abs(o[b, h, t])
                    lse_tol[b, h, t] = ds + 2.0 ** -20 * (1 + abs(lse[b, h, t]))
    return o, lse, o_tol, lse_tol
