"""Plain fp64 definitions of the operators on packed sequences and of the rotation,
with bounds on what bf16 and fp32 arithmetic may add (torch on the CPU, test code).

A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24; fp32
sums on the tensor core may cut instead of rounding: 2^-23 an addition.
"""
import math

import torch

BF = 2.0 ** -8
ACC = 2.0 ** -23


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def seen(n, m, causal):
    s = torch.ones(n, m, dtype=torch.bool)
    return s.tril(m - n) if causal else s


def attention(q, k, v, cu_q, cu_k, scale, causal, dO=None, tol=False):
    """fp64 {o, lse[, dq, dk, dv]} of q [tq, Hq, d], k, v [tk, Hkv, d]; NaN in tokens of
    no sequence.  With `tol` also the same under "tol": bounds for each element.

    With S = scale q k, the score is off by ds = (d + 8) 2^-23 scale |q| |k| and the
    statistics by as much, so that e^(s - m) and P are off by ep = 2 ds + 2^-18 of
    themselves (2^-18: ex2 and the sums of l).  o sums bf16 P: (2^-8 + ep) P |v|, and
    2^-23 an addition.  dP is off by (d + 8) 2^-23 |dO| |v|; D, from the bf16 o, by
    |dO| times o's bound.  dS = P (dP - D) is then off by P (ddP + dD) + (ep + 2^-8) |dS|,
    2^-8 for its rounding to bf16.
    """
    tq, Hq, d = q.shape
    tk, Hkv, _ = k.shape
    G = Hq // Hkv
    nan = dict(dtype=torch.float64)
    out = dict(o=torch.full((tq, Hq, d), math.nan, **nan), lse=torch.full((Hq, tq), math.nan, **nan))
    if dO is not None:
        out.update(dq=torch.full((tq, Hq, d), math.nan, **nan), dk=torch.full((tk, Hkv, d), math.nan, **nan),
                   dv=torch.full((tk, Hkv, d), math.nan, **nan))
    bound = {x: torch.zeros_like(y) for x, y in out.items()}
    for b in range(len(cu_q) - 1):
        i0, i1, j0, j1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = i1 - i0, j1 - j0
        if dO is not None:
            out["dk"][j0:j1] = 0
            out["dv"][j0:j1] = 0
        if n == 0:
            continue
        mask = seen(n, m, causal)
        some = mask.any(-1, keepdim=True)
        for h in range(Hq):
            qq, kk, vv = q[i0:i1, h].double(), k[j0:j1, h // G].double(), v[j0:j1, h // G].double()
            s = torch.where(mask, qq @ kk.T * scale, -math.inf)
            lse = torch.logsumexp(s, -1) if m else torch.full((n,), -math.inf, **nan)
            p = torch.where(some, torch.exp(s - torch.where(some[:, 0], lse, 0)[:, None]), 0.0)
            o = p @ vv
            out["o"][i0:i1, h], out["lse"][h, i0:i1] = o, lse
            ds = torch.where(mask, (d + 8) * ACC * scale * (qq.abs() @ kk.abs().T), 0.0)
            ds = ds.amax(-1, keepdim=True) if m else torch.zeros(n, 1, **nan)
            ep = 2 * ds + 2.0 ** -18
            eo = (BF + ep + (m + 8) * ACC) * (p @ vv.abs()) + 1.02 * BF * o.abs()
            bound["o"][i0:i1, h] = eo
            bound["lse"][h, i0:i1] = ds[:, 0] + 2.0 ** -20 * (1 + torch.where(some[:, 0], lse, 0).abs())
            if dO is None:
                continue
            g = dO[i0:i1, h].double()
            dp = g @ vv.T
            D = (g * o).sum(-1, keepdim=True)
            dS = p * (dp - D)
            out["dq"][i0:i1, h] = scale * dS @ kk
            out["dk"][j0:j1, h // G] += scale * dS.T @ qq
            out["dv"][j0:j1, h // G] += p.T @ g
            ddp = (d + 8) * ACC * (g.abs() @ vv.abs().T)
            dD = (g.abs() * (eo + d * ACC * o.abs())).sum(-1, keepdim=True)
            eS = p * (ddp + dD) + (ep + 1.02 * BF) * dS.abs()
            add = dS.abs() + eS
            bound["dq"][i0:i1, h] = scale * (eS + (m + 8) * ACC * add) @ kk.abs()
            bound["dk"][j0:j1, h // G] += scale * (eS + (n * G + 8) * ACC * add).T @ qq.abs()
            bound["dv"][j0:j1, h // G] += ((BF + ep + (n * G + 8) * ACC) * p).T @ g.abs()
    for x in ("dq", "dk", "dv"):
        if x in out:
            bound[x] += 1.02 * BF * out[x].abs()
    if tol:
        out["tol"] = bound
    return out


def fractions(turns, positions):
    """Angles in turns [..., rot / 2] (-1/2 .. 1/2), exact to 2^-53: whole numbers
    modulo 2^64."""
    flat = [[(int(p) * (int(t) % (1 << 64))) % (1 << 64) for t in turns.tolist()]
            for p in positions.reshape(-1).tolist()]
    x = [[(a - (1 << 64) if a >> 63 else a) / 2.0 ** 64 for a in r] for r in flat]
    return torch.tensor(x, dtype=torch.float64).view(*positions.shape, len(turns))


def rotate(x, turns, positions, interleaved, amplitude=1.0, back=False):
    """x fp64 [tokens, H, d] or [B, H, N, d] with positions [tokens] or [B, N]."""
    r = 2 * len(turns)
    a = 2 * math.pi * fractions(turns, positions) * (-1.0 if back else 1.0)
    c, s = amplitude * a.cos()[:, None], amplitude * a.sin()[:, None]
    y = x.clone()
    if interleaved:
        u, w = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = u * c - w * s, w * c + u * s
    else:
        u, w = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = u * c - w * s, w * c + u * s
    return y


def pair_size(x, rot, interleaved):
    """|x| + |y| of each element's pair, |x| where it does not turn."""
    z = x.abs().clone()
    if interleaved:
        both = z[..., 0:rot:2] + z[..., 1:rot:2]
        z[..., 0:rot:2] = both
        z[..., 1:rot:2] = both
    else:
        both = z[..., : rot // 2] + z[..., rot // 2: rot]
        z[..., : rot // 2] = both
        z[..., rot // 2: rot] = both
    return z


def norm(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def norm_backward(g, x, w, eps):
    """(dx, dw) of norm() for the gradient g of its result."""
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u = w * g
    dx = r * (u - x * r * (u * x * r).mean(-1, keepdim=True))
    return dx, (g * x * r).flatten(0, -2).sum(0)
