"""64-bit plain implementations of the multi-head cross attention and of the paged cache's
operators, with the error that the kernels' roundings may cause, element by element.

Where the kernels round: the weights P and the score gradients dS enter a product as bf16
(off by at most 2^-8 of the value: half a step, torch.finfo(bfloat16).eps / 2), and an output
is rounded to bf16 once (2^-8 of the value). Everything else is fp32. A score is a sum of d
products: off by at most (d + 2) 2^-24 times the sum of their magnitudes; exp2 and log2 add
2^-21. With `s` the largest such score error of a row, a weight is off by at most
2 s + 2^-20 of its value (numerator and denominator), and a sum over n terms in fp32 by
(n + 2) 2^-24 of the sum of magnitudes at the very most (n counted per 128-row tile plus the
tiles). Below 2^-126, the smallest normal fp32 (and bf16) number, a result may become 0: that
moves each weight, each dS and each product by up to TINY = 2^-126, so a gradient that sums
n of them by up to n TINY times the other factor (visible only where the scores differ by
more than 87 and whole gradients are that small).
"""
import math

import torch

HALF = 2.0 ** -8          # half a step of bf16
TINY = 2.0 ** -126        # the smallest normal number of fp32 and bf16


def _sum_err(n):
    return (128 + n / 128 + 2) * 2.0 ** -24


def cross(Q, qo, K, V, ko, mask=None, scale=None, dout=None, rest=False):
    """Q [n, H, d], K, V [m, Hkv, d]; offsets lists; returns dict of (value, bound) pairs:
    out, lse, wide (out + rest) and, with dout, dQ, dK, dV (rest: with the rest given). Rows outside the offsets hold 0 and bound inf."""
    H, d = Q.shape[1:]
    Hkv = K.shape[1]
    G = H // Hkv
    scale = d ** -0.5 if scale is None else scale
    dev = Q.device
    z64 = dict(dtype=torch.float64, device=dev)
    Qd, Kd, Vd = Q.double(), K.double(), V.double()
    out, oerr = torch.zeros(Q.shape, **z64), torch.full(Q.shape, math.inf, **z64)
    lse, lerr = torch.zeros(Q.shape[:2], **z64), torch.full(Q.shape[:2], math.inf, **z64)
    res = {"out": (out, oerr), "lse": (lse, lerr), "wide": (out, torch.full(Q.shape, math.inf, **z64))}
    if dout is not None:
        gd = dout.double()
        for n, x in (("dQ", Q), ("dK", K), ("dV", V)):
            res[n] = (torch.zeros(x.shape, **z64), torch.full(x.shape, math.inf, **z64))
    for u in range(len(qo) - 1):
        a, b = qo[u], qo[u + 1]
        rows = torch.arange(ko[u], ko[u + 1], device=dev)
        keep = rows if mask is None else rows[mask[rows].bool()]
        for n in ("dK", "dV"):
            if n in res:
                res[n][1][rows] = 0.0
        if dout is not None:
            res["dQ"][1][a:b] = 0.0
        oerr[a:b], lerr[a:b], res["wide"][1][a:b] = 0.0, 0.0, 0.0
        if len(keep) == 0:
            lse[a:b] = -math.inf
            continue
        if a == b:
            continue
        for h in range(H):
            q, k, v = Qd[a:b, h], Kd[keep, h // G], Vd[keep, h // G]
            z = q @ k.T * scale
            zerr = (q.abs() @ k.abs().T * scale * (d + 2) * 2.0 ** -24).amax(1, keepdim=True) + 2.0 ** -21
            l = torch.logsumexp(z, 1, keepdim=True)
            w = torch.exp(z - l)
            n = len(keep)
            rel = 2 * zerr + 2.0 ** -20 + _sum_err(n)     # of a weight, before its rounding
            A = w @ v.abs()
            o = w @ v
            out[a:b, h], lse[a:b, h] = o, l[:, 0]
            # the weight's rounding, the sums' and the output's
            e = (HALF + 2 * rel) * A
            oe = e + HALF * (o.abs() + e)
            oerr[a:b, h] = oe
            res["wide"][1][a:b, h] = e + HALF ** 2 * (o.abs() + e) + TINY
            lerr[a:b, h] = (zerr + rel)[:, 0] + l[:, 0].abs() * 2.0 ** -22
            if dout is None:
                continue
            g = gd[a:b, h]
            D = (g * o).sum(1, keepdim=True)
            # delta is formed from the rounded out, or from out + rest: rest is at most HALF of out, and
            # off by HALF of itself
            Derr = (g.abs() * (e + HALF ** 2 * (o.abs() + e) + TINY if rest else oe)).sum(1, keepdim=True) + \
                (g.abs() * o.abs()).sum(1, keepdim=True) * (d + 2) * 2.0 ** -24
            dp = g @ v.T
            dperr = (g.abs() @ v.abs().T) * (d + 2) * 2.0 ** -24
            ds = w * (dp - D) * scale
            prel = 2 * rel                                 # exp(z - lse): z and lse both off
            dserr = w * scale * (dperr + Derr) * (1 + prel) + prel * ds.abs()
            dserr = dserr + TINY * (1 + scale * ((dp - D).abs() + dperr + Derr))
            dserr = dserr + HALF * (ds.abs() + dserr)      # its rounding to bf16
            dq = ds @ k
            e = dserr @ k.abs() + _sum_err(n) * (ds.abs() @ k.abs())
            res["dQ"][0][a:b, h] = dq
            res["dQ"][1][a:b, h] = e + HALF * (dq.abs() + e) + TINY
            m = b - a
            res["dK"][0][keep, h // G] += ds.T @ q
            res["dK"][1][keep, h // G] += (dserr.T + 2 * _sum_err(m * G) * ds.abs().T) @ q.abs()
            res["dV"][0][keep, h // G] += w.T @ g
            res["dV"][1][keep, h // G] += ((HALF + prel.T + 2 * _sum_err(m * G)) * w.T + TINY) @ g.abs()
    for n in ("dK", "dV"):
        if n in res:
            v, e = res[n]
            res[n] = (v, e + HALF * (v.abs() + e) + TINY)
    return res


def check(got, ref, names):
    """Every element of got[name] within its bound; infinite values equal. Rows with bound inf
    (outside the offsets) are not compared."""
    for n in names:
        v, e = ref[n]
        x = got[n].double()
        cmp = torch.isfinite(e)
        fin = torch.isfinite(v) & cmp
        assert torch.equal(x[cmp & ~fin], v[cmp & ~fin]), n
        assert torch.isfinite(x[fin]).all(), f"{n}: not finite"
        bad = (x - v).abs() > e
        bad &= fin
        if bad.any():
            i = tuple(int(t[0]) for t in torch.nonzero(bad, as_tuple=True))
            raise AssertionError(f"{n}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                                 f"{float(x[i])} against {float(v[i])} +- {float(e[i])}")


def gather(cache, table, lens, page, window=0):
    """The rows of every request as ragged K, V [n, Hkv, d] in 64 bits, and their offsets."""
    ks, vs, off = [], [], [0]
    for r, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        p = torch.arange(first, n, device=cache["K"].device)
        pg, row = table[r].long()[p // page], p % page
        for x, sc, to in (("K", "k_scales", ks), ("V", "v_scales", vs)):
            if cache[sc] is None:
                t = cache[x][pg, :, row].double()
            else:
                t = cache[x].view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float().double()
                t = t * cache[sc][pg, :, row].double()[..., None]
            to.append(t)
        off.append(off[-1] + max(0, n - first))
    return torch.cat(ks), torch.cat(vs), off


def tables(cached, new, free, used, table, page, n_slots):
    """The block table, slots, offsets, lengths and taken pages after one sa_page_tables call
    (plain Python)."""
    table = [list(row) for row in table]
    slots, off, at = [], [0], used
    for r, (c, n) in enumerate(zip(cached, new)):
        for p in range(-(-c // page), -(-(c + n) // page)):
            table[r][p] = free[at]
            at += 1
        for pos in range(c, c + n):
            pg = table[r][pos // page]
            slots.append(pg * page + pos % page if pg >= 0 else -1)
        off.append(off[-1] + n)
    slots += [-1] * (n_slots - len(slots))
    return table, slots, off, [c + n for c, n in zip(cached, new)], at
