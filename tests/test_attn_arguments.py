"""The multi-head cross attention and the paged cache: refusals (C ABI and binding) before any
CUDA call, and the 64-bit reference against autograd and differences. CPU only."""
import ctypes
import math

import pytest
import torch

import attn_reference as ref


@pytest.fixture(scope="module")
def b():
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding
    return binding


def _cross(b, back=False, **kw):
    a = dict(Q=16, qs=256, qo=8, R=1, n_q=4, H=2, d=128, K=16, ks=128, V=16, vs=128, ko=8, n_kv=5, Hkv=1, mask=None,
             scale=0.1, out=16, rest=None, lse=16, dout=16, dQ=16, dK=16, dV=16, ws=256, nb=1 << 30)
    a.update(kw)
    head = [a[n] for n in ("Q", "qs", "qo", "R", "n_q", "H", "d", "K", "ks", "V", "vs", "ko", "n_kv", "Hkv", "mask",
                           "scale", "out", "rest", "lse")]
    if back:
        return b.sa_cross_attn_backward(*head, a["dout"], a["dQ"], a["dK"], a["dV"], a["ws"], a["nb"], None)
    return b.sa_cross_attn_forward(*head, a["ws"], a["nb"], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(d=96), 2), (dict(H=3, Hkv=2), 1), (dict(Hkv=0), 1), (dict(H=2048, Hkv=1), 1), (dict(R=-1), 1),
    (dict(n_q=-1), 1), (dict(n_kv=1 << 31), 1), (dict(scale=0.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(scale=-1.0), 1), (dict(Q=None), 1), (dict(K=None), 1), (dict(V=24), 1),
    (dict(qo=None), 1), (dict(ko=12), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(qs=255), 1),
    (dict(qs=128), 1), (dict(ks=132), 1), (dict(vs=64), 1), (dict(out=8), 1), (dict(rest=8), 1),
    (dict(n_q=(1 << 31) - 1, H=1024, qs=1024 * 128), 2),
])
def test_cross_attention_refuses(b, back, kw, code):
    assert _cross(b, back, **kw) == code


@pytest.mark.parametrize("kw", [dict(dout=None), dict(dQ=None), dict(dK=None), dict(dV=20)])
def test_cross_attention_backward_refuses(b, kw):
    assert _cross(b, True, **kw) == 1


def _tables(b, **kw):
    a = dict(c=4, n=4, R=2, page=16, free=4, n_free=8, used=8, table=4, mp=4, n_slots=9, slots=8, off=8, lens=4,
             out=8, ws=256, nb=256)
    a.update(kw)
    return b.sa_page_tables(*[a[n] for n in ("c", "n", "R", "page", "free", "n_free", "used", "table", "mp", "n_slots",
                                             "slots", "off", "lens", "out", "ws", "nb")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(page=12), 2), (dict(page=4), 2), (dict(page=512), 2), (dict(R=-1), 1), (dict(n_free=-1), 1),
    (dict(n_slots=1 << 31), 1), (dict(mp=-1), 1), (dict(c=None), 1), (dict(free=None), 1), (dict(table=None), 1),
    (dict(slots=None), 1), (dict(slots=12), 1), (dict(off=None), 1), (dict(out=None), 1), (dict(lens=2), 1),
    (dict(used=4), 1),
])
def test_page_tables_refuses(b, kw, code):
    assert _tables(b, **kw) == code


def _append(b, **kw):
    a = dict(K=16, ks=256, V=16, vs=256, slots=8, n=3, Hkv=2, d=128, fmt=1, kc=16, vc=16, sk=16, sv=16, pages=4, page=16)
    a.update(kw)
    return b.sa_paged_append(*[a[n] for n in ("K", "ks", "V", "vs", "slots", "n", "Hkv", "d", "fmt", "kc", "vc", "sk",
                                              "sv", "pages", "page")], None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=32), 2), (dict(page=3), 2), (dict(fmt=2), 1), (dict(n=-1), 1), (dict(pages=-1), 1), (dict(Hkv=0), 1),
    (dict(sk=None), 1), (dict(vc=None), 1), (dict(K=None), 1), (dict(slots=None), 1), (dict(ks=128), 1),
    (dict(vs=260), 1), (dict(kc=8), 1), (dict(pages=1 << 30), 2),
])
def test_paged_append_refuses(b, kw, code):
    assert _append(b, **kw) == code


def _attend(b, **kw):
    a = dict(Q=16, qs=512, R=2, H=4, d=128, kc=16, vc=16, sk=16, sv=16, fmt=1, pages=4, page=16, Hkv=2, table=4, mp=2,
             lens=4, window=0, scale=0.1, out=16, lse=16, ws=256, nb=1 << 30)
    a.update(kw)
    return b.sa_paged_attn(*[a[n] for n in ("Q", "qs", "R", "H", "d", "kc", "vc", "sk", "sv", "fmt", "pages", "page",
                                            "Hkv", "table", "mp", "lens", "window", "scale", "out", "lse", "ws", "nb")],
                           None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=32), 2), (dict(page=24), 2), (dict(fmt=5), 1), (dict(H=5), 1), (dict(H=130, Hkv=2, qs=130 * 128), 2),
    (dict(R=-1), 1), (dict(window=-1), 1), (dict(scale=0.0), 1), (dict(Q=None), 1), (dict(out=None), 1),
    (dict(lens=None), 1), (dict(table=None), 1), (dict(sv=None), 1), (dict(qs=511), 1), (dict(table=6), 1),
    (dict(mp=1 << 30), 2),
])
def test_paged_attention_refuses(b, kw, code):
    assert _attend(b, **kw) == code


def test_workspace_sizes_refuse(b):
    assert b.sa_cross_attn_workspace_size(1, 4, 4, 3, 2, 128, 0) == 0
    assert b.sa_cross_attn_workspace_size(1, 4, 4, 2, 2, 80, 1) == 0
    assert b.sa_paged_attn_workspace_size(-1, 4, 2, 128) == 0
    assert b.sa_paged_attn_workspace_size(1, 65, 1, 128) == 0


# ---------------------------------------------------------------- the binding's own checks
def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_binding_refuses_cross_inputs(b):
    Q, K, o = _bf(4, 4, 64), _bf(6, 2, 64), torch.tensor([0, 4])
    for args, kw, msg in [
        ((Q.float(), o, K, K, o), {}, "Q has dtype"), ((Q, o, K, _bf(6, 1, 64), o), {}, "V has shape"),
        ((Q, o, _bf(6, 3, 64), _bf(6, 3, 64), o), {}, "cannot share"), ((Q, o.int(), K, K, o), {}, "q_offsets has dtype"),
        ((Q, o, K, K, torch.tensor([0, 1, 2])), {}, "kv_offsets has shape"),
        ((Q, o, K, K, o), dict(key_mask=torch.ones(5, dtype=torch.bool)), "key_mask has shape"),
        ((Q, o, K, K, o), dict(key_mask=torch.ones(6)), "key_mask must be"), ((Q[0], o, K, K, o), {}, "Q must be"),
        ((Q, o, K, K, o), {}, "CUDA devices only"),
    ]:
        with pytest.raises(b.SketchAttentionError, match=msg):
            b.cross_attention(*args, **kw)
    with pytest.raises(b.SketchAttentionError, match="CUDA devices only"):
        b.cross_attention_backward(Q, o, K, K, o, {}, Q)


def test_binding_refuses_cache_inputs(b):
    cache = b.paged_cache(4, 2, 16, 64, device="cpu")
    f8 = b.paged_cache(4, 2, 16, 64, fmt=b.SA_CODEC_FP8, device="cpu")
    K, sl = _bf(3, 2, 64), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(b.SketchAttentionError, match="unknown format"):
        b.paged_cache(4, 2, 16, 64, fmt=3, device="cpu")
    for args, msg in [((K, K[:2], sl, cache), "V has shape"), ((K, K, sl.int(), cache), "slots has dtype"),
                      ((K, K, sl, {**f8, "k_scales": None}), "k_scales is required"),
                      ((K, K, sl, {**cache, "v_scales": f8["v_scales"]}), "belongs to an FP8"),
                      ((K, K, sl, {"K": K}), "cache must hold"), ((K, K, sl, f8), "CUDA devices only")]:
        with pytest.raises(b.SketchAttentionError, match=msg):
            b.paged_append(*args)
    Q, t, ln = _bf(2, 4, 64), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args, msg in [((_bf(2, 4, 128), cache, t, ln), "Q has shape"), ((Q, cache, t.long(), ln), "block_table has dtype"),
                      ((Q, cache, t[:1], ln), "block_table has shape"), ((_bf(2, 3, 64), cache, t, ln), "cannot share"),
                      ((Q, cache, t, ln.long()), "seq_lens has dtype"), ((Q, cache, t, ln), "CUDA devices only")]:
        with pytest.raises(b.SketchAttentionError, match=msg):
            b.paged_attention(*args)
    for args, msg in [((ln.long(), ln, ln, t, 16, 4), "cached_lens has dtype"), ((ln, ln, t, t, 16, 4), "free_pages must be"),
                      ((ln, ln, ln, ln, 16, 4), "block_table must be"), ((ln, ln, ln, t, 16, 4), "CUDA devices only")]:
        with pytest.raises(b.SketchAttentionError, match=msg):
            b.page_tables(*args)


# ---------------------------------------------------------------- the reference itself
def test_reference_gradients_against_autograd_and_differences():
    g = torch.Generator().manual_seed(3)
    qo, ko = [0, 3, 3, 5], [0, 4, 6, 13]
    Q, K, V = (torch.randn(n, h, 8, generator=g, dtype=torch.float64) for n, h in ((5, 4), (13, 2), (13, 2)))
    dout = torch.randn(5, 4, 8, generator=g, dtype=torch.float64)
    mask = torch.rand(13, generator=g) < 0.7
    r = ref.cross(Q, qo, K, V, ko, mask, dout=dout)

    def loss(Q, K, V):
        tot = 0.0
        for u in range(3):
            keep = torch.arange(ko[u], ko[u + 1])[mask[ko[u]:ko[u + 1]]]
            for h in range(4):
                z = Q[qo[u]:qo[u + 1], h] @ K[keep, h // 2].T / math.sqrt(8)
                tot = tot + ((torch.softmax(z, 1) @ V[keep, h // 2]) * dout[qo[u]:qo[u + 1], h]).sum()
        return tot

    xs = [x.clone().requires_grad_() for x in (Q, K, V)]
    for name, grad in zip(("dQ", "dK", "dV"), torch.autograd.grad(loss(*xs), xs)):
        assert torch.allclose(r[name][0], grad, rtol=1e-10, atol=1e-12), name
    for i, name in enumerate(("dQ", "dK", "dV")):
        x = [Q, K, V]
        dirn = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        hi, lo = list(x), list(x)
        hi[i], lo[i] = x[i] + 1e-5 * dirn, x[i] - 1e-5 * dirn
        diff = float(loss(*hi) - loss(*lo)) / 2e-5
        assert abs(diff - float((r[name][0] * dirn).sum())) < 1e-7 * (1 + abs(diff)), name


def test_reference_tables():
    t = [[7, -1, -1], [-1, -1, -1], [3, 4, -1]]
    table, slots, off, lens, used = ref.tables([3, 0, 16], [6, 0, 2], [9, 1, 5, 6], 1, t, 8, 10)
    assert table == [[7, 1, -1], [-1, -1, -1], [3, 4, 5]]
    assert slots == [59, 60, 61, 62, 63, 8, 40, 41, -1, -1]
    assert (off, lens, used) == ([0, 6, 6, 8], [9, 0, 18], 3)


def test_short_calls_leave_what_is_not_plain_to_python(b):
    """_calls returns None, and touches nothing, for whatever is not a plain call on CUDA tensors."""
    calls = b._calls
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i, o = torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    counts = {"cross_forward": 9, "cross_backward": 12, "page_tables": 8, "paged_append": 7, "paged_attention": 10}
    for name, n in counts.items():
        f = getattr(calls, name)
        for arg in (None, 3, "x", x, i, o, torch.nn.Parameter(x.float())):
            assert f(*[arg] * n) is None
        assert f() is None and f(*[x] * (n + 1)) is None
    assert calls.cross_forward(x, o, x, x, o, None, None, True, None) is None
    assert calls.paged_attention(x, x, x, None, None, i, i, 0, None, None) is None
