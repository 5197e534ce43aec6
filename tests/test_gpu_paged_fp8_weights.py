"""FP8 paged attention where value rows' scales and softmax weights are far apart: a row of zeros (scale 1)
among small rows, rows with a large scale and next to no weight, scales that grow or fall along the positions.

The bound. A product t = w v_scale (w the softmax weight) enters the second product as fp16: off by 2^-11 of its value, or,
where it is small beside the largest product of its head, by 2^-25 of a unit of at most twice that
largest product: 2^-24 of it. Codes are exact. Scores: a sum of d products in fp32, (d + 2) 2^-24 of
their magnitudes, four more roundings for the scales, exp2 2^-21; queries lose at most 2^-33 of the
head's largest value. The output is rounded to bf16 once (2^-8). So an output element may be off by
  sum_j (2^-11 + rel) t_j |code_j| + 2^-24 max_j t_j sum_j |code_j|, and 2^-8 of the result."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn
HALF = 2.0 ** -8


def _reference(Q, Kc, ks, Vc, vs, lens, starts):
    """Q [R, H, d]; codes [n, Hkv, d] and scales [n, Hkv] of all requests' rows, in order."""
    R, H, d = Q.shape
    G = H // Kc.shape[1]
    scale = d ** -0.5
    o = torch.zeros(R, H, d, dtype=torch.float64, device=Q.device)
    err = torch.zeros_like(o)
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device=Q.device)
    lerr = torch.zeros_like(lse)
    for r, (n, s0) in enumerate(zip(lens, starts)):
        if n == 0:
            continue
        for h in range(H):
            q = Q[r, h].double()
            k, v = Kc[s0:s0 + n, h // G].float().double(), Vc[s0:s0 + n, h // G].float().double()
            kk, vv = ks[s0:s0 + n, h // G].double(), vs[s0:s0 + n, h // G].double()
            z = (k @ q) * kk * scale
            mag = (k.abs() @ q.abs()) * kk * scale
            zerr = float(((d + 6) * 2.0 ** -24 * mag + 2.0 ** -33 * q.abs().max() * k.abs().sum(1) * kk * scale).max()) + 2.0 ** -21
            l = torch.logsumexp(z, 0)
            rel = 2 * zerr + 2.0 ** -20 + (128 + n / 128 + 2) * 2.0 ** -24
            t = torch.exp(z - l) * vv
            e = ((2.0 ** -11 + 2 * rel) * t) @ v.abs() + 2.0 ** -24 * t.max() * v.abs().sum(0)
            o[r, h] = t @ v
            err[r, h] = e + HALF * (o[r, h].abs() + e) + 2.0 ** -126
            lse[r, h] = l
            lerr[r, h] = zerr + rel + l.abs() * 2.0 ** -22
    return o, err, lse, lerr


def _run(Q, K, V, lens, page=16):
    """Rows K, V [n, Hkv, d] appended to an FP8 cache and attended to; the codes and scales that it holds."""
    from prototype_sketch_attention_b200 import binding as b
    R = len(lens)
    n, Hkv, d = K.shape
    cnt = [-(-x // page) for x in lens]
    cache = b.paged_cache(sum(cnt) + 1, Hkv, page, d, fmt=b.SA_CODEC_FP8)
    cache["K"].view(torch.uint8).fill_(0x7F)  # NaN where nothing is written
    cache["V"].view(torch.uint8).fill_(0x7F)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.full((R, max(cnt)), -1, **i32)
    t = b.page_tables(torch.zeros(R, **i32), torch.tensor(lens, **i32), torch.randperm(sum(cnt), device="cuda").to(torch.int32),
                      table, page, n)
    b.paged_append(K, V, t["slots"], cache)
    pg, row = t["slots"] // page, t["slots"] % page
    held = [cache["K"].view(torch.uint8)[pg, :, row].view(F8), cache["k_scales"][pg, :, row],
            cache["V"].view(torch.uint8)[pg, :, row].view(F8), cache["v_scales"][pg, :, row]]
    got = b.paged_attention(Q, cache, table, t["seq_lens"])
    assert b.device_status(t["_ws"]) == 0 and b.device_status(got["_ws"]) == 0
    return got, held


def _check(Q, K, V, lens):
    got, held = _run(Q, K, V, lens)
    starts = [sum(lens[:r]) for r in range(len(lens))]
    o, err, lse, lerr = _reference(Q, *held, lens, starts)
    off = (got["out"].double() - o).abs() / err
    assert not (off > 1).any() and not off.isnan().any(), f"out {float(off.max())} times the bound"
    off = (got["lse"].double() - lse).abs() / lerr
    assert not (off > 1).any() and not off.isnan().any(), f"lse {float(off.max())} times the bound"


HEADS = [(8, 1, 128), (16, 1, 128), (8, 2, 64), (32, 2, 64), (3, 3, 128)]
LENS = [[4000], [1, 40, 333, 1500], [17] * 60]


def _rows(lens, H, Hkv, d, seed, amp):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(*s, generator=g, device="cuda")
    n = sum(lens)
    return r(len(lens), H, d).to(BF), r(n, Hkv, d).to(BF), (amp * r(n, Hkv, d)).to(BF)


@pytest.mark.parametrize("amp", [0.02, 1e-3, 1e-4, 1e-6, 1e-30, 1e4, 1e30])
@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=["one", "ragged", "many"])
def test_a_row_of_zeros_among_small_ones(lens, H, Hkv, d, amp):
    """The append gives a row of zeros the scale 1, whatever its neighbours hold."""
    Q, K, V = _rows(lens, H, Hkv, d, 11, amp)
    at = 0
    for n in lens:
        V[at + n // 3] = 0
        at += n
    _check(Q, K, V, lens)


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=["one", "ragged", "many"])
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_a_large_row_without_weight(lens, H, Hkv, d, place):
    """A value row 10^5 times the others, whose score lies 40 and more below the largest."""
    Q, K, V = _rows(lens, H, Hkv, d, 12, 1e-3)
    K = K.float() * 0.2
    Q = (Q.float().abs() + 0.5).to(BF)
    at = 0
    for n in lens:
        if n > 1:
            j = at + {"first": 0, "middle": n // 2, "last": n - 1}[place]
            K[j] = -8.0
            V[j] = V[j].float() * 1e5
        at += n
    _check(Q, K.to(BF), V, lens)


@pytest.mark.parametrize("H,Hkv,d", HEADS)
def test_heads_of_a_key_head_want_different_units(H, Hkv, d):
    """Every other query head takes the large rows, the heads between them do not."""
    lens = [900, 70]
    Q, K, V = _rows(lens, H, Hkv, d, 13, 1e-4)
    K = K.float() * 0.1
    K[5::37] += 1.0
    V = V.float()
    V[5::37] *= 1e5
    sign = torch.tensor([1.0 if h % 2 else -1.0 for h in range(H)], device="cuda")
    Q = (Q.float().abs() + 0.5) * sign[:, None]
    _check(Q.to(BF), K.to(BF), V.to(BF), lens)


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("scores,values", [(1, 1), (1, -1), (-1, 1), (-1, -1), (0, 1), (0, -1), (1, 0)])
def test_scores_and_scales_that_run(H, Hkv, d, scores, values):
    """Along 3,000 positions the scores rise or fall by some hundred, the values by twelve decades."""
    lens = [3000, 200]
    Q, K, V = _rows(lens, H, Hkv, d, 14, 1.0)
    Q = (Q.float().abs() + 0.5).to(BF)
    run = torch.cat([torch.linspace(-1, 1, n, device="cuda") for n in lens])[:, None, None]
    K = (0.05 * K.float() + scores * 6.0 * run).to(BF)
    V = (V.float() * 10.0 ** (6 * values * run)).to(BF)
    _check(Q, K, V, lens)


def test_only_rows_of_zeros():
    Q, K, V = _rows([300, 5], 16, 2, 128, 15, 0.0)
    got, _ = _run(Q, K, V, [300, 5])
    assert (got["out"] == 0).all() and got["lse"].isfinite().all()
