"""Users of at most 128 keys: the forward's weights enter the second product as two bf16, so out + rest and the
gradients' delta = dout . out carry 2^-16 of a weight in place of 2^-8. Bounds as in attn_reference.py
with that figure; and the whole gradients' errors beside those of fp32 products and one rounding, where dS's
rounding to bf16 alone gives sqrt(2)."""
import math

import pytest
import torch

import attn_reference as ref
from test_gpu_cross import _inputs, _offsets, _run

pytestmark = pytest.mark.gpu
HALF, TINY, P_HALF = ref.HALF, ref.TINY, 2.0 ** -16


def _bounds(Q, qo, K, V, ko, mask, dout):
    """(value, bound) of out, wide (out + rest) and dQ; rows of users without kept keys: 0."""
    H, d = Q.shape[1:]
    G, scale = H // K.shape[1], d ** -0.5
    res = {n: (torch.zeros(Q.shape, dtype=torch.float64, device="cuda"), torch.zeros(Q.shape, dtype=torch.float64, device="cuda"))
           for n in ("out", "wide", "dQ")}
    for u in range(len(qo) - 1):
        a, b = qo[u], qo[u + 1]
        keep = torch.arange(ko[u], ko[u + 1], device="cuda")
        keep = keep if mask is None else keep[mask[keep]]
        if len(keep) == 0 or a == b:
            continue
        for h in range(H):
            q, k, v, g = Q[a:b, h].double(), K[keep, h // G].double(), V[keep, h // G].double(), dout[a:b, h].double()
            z = q @ k.T * scale
            zerr = (q.abs() @ k.abs().T * scale * (d + 2) * 2.0 ** -24).amax(1, keepdim=True) + 2.0 ** -21
            w = torch.softmax(z, 1)
            rel = 2 * zerr + 2.0 ** -20 + (len(keep) + 2) * 2.0 ** -24
            o = w @ v
            e = (P_HALF + 2 * rel) * (w @ v.abs())
            we = e + HALF ** 2 * (o.abs() + e) + TINY
            derr = (g.abs() * we).sum(1, keepdim=True) + (g.abs() * o.abs()).sum(1, keepdim=True) * (d + 2) * 2.0 ** -24
            dp = g @ v.T
            ds = w * (dp - (g * o).sum(1, keepdim=True)) * scale
            dse = w * scale * ((g.abs() @ v.abs().T) * (d + 2) * 2.0 ** -24 + derr) * (1 + 2 * rel) + 2 * rel * ds.abs()
            dse = dse + TINY * (1 + scale * dp.abs().amax())
            dse = dse + HALF * (ds.abs() + dse)
            dq = ds @ k
            qe = dse @ k.abs() + (len(keep) + 2) * 2.0 ** -24 * (ds.abs() @ k.abs())
            for n, x, y in (("out", o, e + HALF * (o.abs() + e)), ("wide", o, we), ("dQ", dq, qe + HALF * (dq.abs() + qe) + TINY)):
                res[n][0][a:b, h], res[n][1][a:b, h] = x, y
    return res


@pytest.mark.parametrize("lq,lk", [([1], [1]), ([40, 3, 129], [2, 128, 127]), ([300, 1, 7, 256], [5, 64, 100, 33]),
                                   ([2] * 200, [1 + i % 128 for i in range(200)]), ([5, 0, 9], [0, 17, 65])])
@pytest.mark.parametrize("H,Hkv,d", [(4, 4, 64), (6, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("masked", [False, True])
def test_within_the_narrower_bounds(lq, lk, H, Hkv, d, masked):
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=40 + H)
    qo, ko = _offsets(lq), _offsets(lk)
    mask = None
    if masked:
        mask = torch.rand(ko[-1], generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < 0.6
    got = _run(Q, qo, K, V, ko, dout, mask)
    got["wide"] = got["out"].double() + got["rest"].double()
    ref.check(got, _bounds(Q, qo, K, V, ko, mask, dout), ("out", "wide", "dQ"))


@pytest.mark.parametrize("keys", [2, 3, 8, 40, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_gradients_are_off_by_two_roundings(keys, d):
    """A value rounded to bf16 is off by u / sqrt(3) in the mean square, u = 2^-9 to 2^-8 of it; two independent
    ones (dS, the gradient) by sqrt(2) times one. Another 3 percent for what the scores' and exponentials'
    fp32 errors add and for the spread of 4,000 rows' mean square; P's rounding in delta made it 1.5 and more."""
    lq, lk = [40] * 25, [keys] * 25
    Q, K, V, dout = _inputs(lq, lk, 4, 2, d, seed=keys)
    qo, ko = _offsets(lq), _offsets(lk)
    got, want = _run(Q, qo, K, V, ko, dout), ref.cross(Q, qo, K, V, ko, dout=dout)
    for n in ("dQ", "dK"):
        w = want[n][0]
        one = float((w.to(torch.bfloat16).double() - w).norm())
        assert float((got[n].double() - w).norm()) <= 1.03 * math.sqrt(2) * one, n
