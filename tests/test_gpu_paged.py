"""GPU paged key-value cache: block tables and slot maps, the append, and the attention of one
new token per request, each against plain implementations (attn_reference.py), and a run of
them together with the cross attention over the same rows."""
import math
import random

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- block tables and slot maps
def _tables(cached, new, page, *, used=0, spare=3, pad=0, width=None, free_pages=None):
    """Runs sa_page_tables; returns its results as lists, the reference's, and the status."""
    from prototype_sketch_attention_b200 import binding as b
    r = random.Random(len(cached) + page)
    have = [-(-c // page) for c in cached]
    want = [-(-(c + n) // page) for c, n in zip(cached, new)]
    width = max(want + [1]) if width is None else width
    ids = list(range(sum(have) + sum(want) + used + spare))
    r.shuffle(ids)
    table = [[ids.pop() for _ in range(h)][:width] + [-1] * (width - h) for h in have]
    free = ids if free_pages is None else ids[:free_pages]
    n_slots = sum(new) + pad
    t = torch.tensor(table, dtype=torch.int32, device="cuda").reshape(len(cached), width)
    out = b.page_tables(_i32(cached), _i32(new), _i32(free), t, page, n_slots,
                        free_used=torch.tensor([used], dtype=torch.int64, device="cuda"))
    st = b.device_status(out["_ws"])
    got = (t.tolist(), out["slots"].tolist(), out["new_offsets"].tolist(), out["seq_lens"].tolist(),
           int(out["free_used"]))
    return got, table, free, n_slots, st


@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("cached,new", [
    ([0], [1]), ([0], [0]), ([5], [0]), ([7, 8, 9], [1, 1, 1]), ([0, 0, 0], [300, 0, 1]),
    ([1000, 3, 0, 255, 256], [17, 5000, 64, 1, 256]), ([3] * 700, [1] * 700),
    ([(i * 37) % 90 for i in range(1300)], [(i * 11) % 23 for i in range(1300)]),
])
def test_tables_match(page, cached, new):
    got, table, free, n_slots, st = _tables(cached, new, page, used=2, pad=5)
    assert st == 0
    want = ref.tables(cached, new, free, 2, table, page, n_slots)
    for x, y, name in zip(got, want, ("table", "slots", "new_offsets", "seq_lens", "free_used")):
        assert x == y, name


def test_tables_without_requests_and_without_free_used():
    from prototype_sketch_attention_b200 import binding as b
    t = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    out = b.page_tables(_i32([]), _i32([]), _i32([]), t, 16, 6)
    assert out["slots"].tolist() == [-1] * 6 and out["new_offsets"].tolist() == [0]
    assert int(out["free_used"]) == 0 and b.device_status(out["_ws"]) == 0


@pytest.mark.parametrize("why,code,kw", [
    ("free pages", 8, dict(cached=[8, 3], new=[40, 60], page=16, free_pages=4)),
    ("row too short", 8, dict(cached=[8, 3], new=[40, 60], page=16, width=3)),
    ("negative new", 6, dict(cached=[8, 3], new=[-1, 6], page=16)),
    ("negative cached", 6, dict(cached=[8, -3], new=[1, 6], page=16)),
    ("too many new", 6, dict(cached=[8, 3], new=[10, 6], page=16, pad=-1)),
    ("free list used up", 8, dict(cached=[8], new=[40], page=16, used=10 ** 6)),
])
def test_tables_refuse_on_the_device(why, code, kw):
    """All or nothing: nothing is taken and nothing written but the empty answer."""
    from prototype_sketch_attention_b200 import binding as b
    kw = dict(kw)
    cached, new, page = kw.pop("cached"), kw.pop("new"), kw.pop("page")
    have = [max(0, -(-c // page)) for c in cached]
    width = kw.get("width", 8)
    table = torch.arange(len(cached) * width, dtype=torch.int32, device="cuda").reshape(len(cached), width)
    before = table.clone()
    used = torch.tensor([kw.get("used", 0)], dtype=torch.int64, device="cuda")
    free = _i32(list(range(100, 100 + kw.get("free_pages", 50))))
    n_slots = max(0, sum(new)) + kw.get("pad", 0)
    out = b.page_tables(_i32(cached), _i32(new), free, table, page, n_slots, free_used=used)
    assert b.device_status(out["_ws"]) == code, (why, have)
    assert torch.equal(table, before) and torch.equal(out["free_used"], used)
    assert (out["slots"] == -1).all() and (out["new_offsets"] == 0).all() and out["seq_lens"].tolist() == cached


def test_tables_held_page_without_id_gives_no_slot():
    from prototype_sketch_attention_b200 import binding as b
    table = _i32([[-1, -1]])
    out = b.page_tables(_i32([5]), _i32([6]), _i32([9]), table, 8, 6)
    assert out["slots"].tolist() == [-1, -1, -1, 72, 73, 74] and table.tolist() == [[-1, 9]]


# ---------------------------------------------------------------- append
def _cache(pages, Hkv, page, d, fp8, fill=0.0):
    from prototype_sketch_attention_b200 import binding as b
    c = b.paged_cache(pages, Hkv, page, d, fmt=b.SA_CODEC_FP8 if fp8 else b.SA_CODEC_BF16)
    for n in ("K", "V"):
        c[n].copy_(torch.full(c[n].shape, fill, device="cuda").to(c[n].dtype))
    if fp8:
        c["k_scales"].fill_(3.0)
        c["v_scales"].fill_(3.0)
    return c


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,Hkv,page,d,fused", [(1, 1, 8, 64, False), (37, 3, 16, 128, True), (500, 2, 64, 64, True),
                                                (2001, 8, 256, 128, False), (0, 2, 16, 128, False)])
def test_append_is_exact(fp8, n, Hkv, page, d, fused):
    """bf16 rows bit for bit; FP8 codes and scales as the sketch cache codec's reference makes
    them; rows of other slots stay."""
    from oracle import codec
    from prototype_sketch_attention_b200 import binding as b
    g = torch.Generator(device="cuda").manual_seed(n)
    KV = torch.randn(n, 2, Hkv, d, generator=g, device="cuda") * 10 ** torch.empty(n, 2, Hkv, 1, device="cuda").uniform_(
        -6, 3, generator=g)
    KV = KV.to(BF)
    if n > 2:
        KV[1, :, 0] = 0.0
        KV[2, 1, 0] = -0.0
    K, V = (KV[:, 0], KV[:, 1]) if fused else (KV[:, 0].contiguous(), KV[:, 1].contiguous())
    pages = max(1, -(-n * 3 // (2 * page)))
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:n]
    if n > 5:
        slots[3], slots[4] = -1, pages * page  # padding, and a slot past the cache
    cache = _cache(pages, Hkv, page, d, fp8, fill=1.5)
    b.paged_append(K, V, slots, cache)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < pages * page)
    pg, row = slots[ok] // page, slots[ok] % page
    for x, name, sc in ((K, "K", "k_scales"), (V, "V", "v_scales")):
        if not fp8:
            want = torch.full((pages, Hkv, page, d), 1.5, device="cuda").to(BF)
            want[pg, :, row] = x[ok]
            assert torch.equal(cache[name].view(torch.int16), want.view(torch.int16)), name
            continue
        want = torch.full((pages, Hkv, page, d), 1.5, device="cuda").to(F8).view(torch.uint8)
        wsc = torch.full((pages, Hkv, page), 3.0, device="cuda")
        if n:
            codes, scales = codec.fp8_encode(x[ok].float().cpu().numpy())
            want[pg, :, row] = torch.from_numpy(codes).cuda()
            wsc[pg, :, row] = torch.from_numpy(scales).cuda()
        assert torch.equal(cache[name].view(torch.uint8), want), name
        assert torch.equal(cache[sc], wsc), sc


# ---------------------------------------------------------------- attention
def _filled(lens, H, Hkv, d, page, fp8, seed, poison=True):
    """A cache with shuffled pages; what no request may read holds NaN."""
    from prototype_sketch_attention_b200 import binding as b
    g = torch.Generator(device="cuda").manual_seed(seed)
    cnt = [-(-n // page) for n in lens]
    pages = sum(cnt) + 2
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    width = max(cnt + [1]) + 1
    table = torch.full((len(lens), width), -5, dtype=torch.int32)
    own = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for r, n in enumerate(lens):
        for p in range(cnt[r]):
            table[r, p] = ids[at]
            own[ids[at], :min(page, n - p * page)] = True
            at += 1
    own = own.cuda()
    cache = b.paged_cache(pages, Hkv, page, d, fmt=b.SA_CODEC_FP8 if fp8 else b.SA_CODEC_BF16)
    for name, sc in (("K", "k_scales"), ("V", "v_scales")):
        x = torch.randn(pages, Hkv, page, d, generator=g, device="cuda")
        gone = ~own[:, None, :].expand(pages, Hkv, page)
        if fp8:
            s = x.abs().amax(-1) / 448
            q = (x / s[..., None]).to(F8).view(torch.uint8)
            q[gone] = 0x7F  # NaN
            s[gone] = math.nan
            cache[name].view(torch.uint8).copy_(q)
            cache[sc].copy_(s)
        else:
            x[gone] = math.nan
            cache[name].copy_(x.to(BF))
    Q = torch.randn(len(lens), H, d, generator=g, device="cuda").to(BF)
    return Q, cache, table.cuda(), _i32(lens)


def _check(Q, cache, table, lens, page, window, got, scale=None):
    K, V, off = ref.gather(cache, table, lens.tolist(), page, window)
    R, H, d = Q.shape
    r = ref.cross(Q, list(range(R + 1)), K, V, off, scale=scale)
    ref.check(got, r, ("out", "lse"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d,page,window", [
    ([1], 1, 1, 64, 8, 0),
    ([0, 1, 7, 8, 9], 4, 4, 64, 8, 0),
    ([63, 64, 65, 0, 300], 8, 2, 128, 16, 0),
    ([1000, 129], 12, 4, 128, 64, 100),
    ([5000], 16, 1, 128, 16, 0),
    ([5000, 33], 17, 1, 64, 32, 4097),
    ([257, 4096, 31], 64, 1, 128, 256, 0),
    ([20000, 3], 6, 2, 64, 128, 1),
    ([40 * i for i in range(40)], 24, 8, 128, 16, 333),
    ([17] * 400, 3, 3, 64, 16, 0),
    ([60001], 8, 8, 64, 64, 0),
    ([100], 40, 2, 128, 8, 0),
])
def test_attention_against_reference(lens, H, Hkv, d, page, window, fp8):
    from prototype_sketch_attention_b200 import binding as b
    Q, cache, table, ln = _filled(lens, H, Hkv, d, page, fp8, seed=len(lens) + H)
    got = b.paged_attention(Q, cache, table, ln, window=window)
    torch.cuda.synchronize()
    assert b.device_status(got["_ws"]) == 0
    _check(Q, cache, table, ln, page, window, got)


def test_attention_strided_queries_scale_and_no_requests():
    from prototype_sketch_attention_b200 import binding as b
    Q, cache, table, ln = _filled([100, 50], 4, 2, 128, 16, False, seed=3)
    wide = torch.full((2, 9, 128), float("nan"), dtype=BF, device="cuda")
    wide[:, 2:6] = Q
    got = b.paged_attention(wide[:, 2:6], cache, table, ln, scale=0.2)
    _check(Q, cache, table, ln, 16, 0, got, scale=0.2)
    got = b.paged_attention(Q[:0], cache, table[:0].contiguous(), ln[:0].contiguous())
    assert got["out"].shape == (0, 4, 128) and b.device_status(got["_ws"]) == 0


def test_attention_sharp_scores():
    from prototype_sketch_attention_b200 import binding as b
    for fp8 in (False, True):
        Q, cache, table, ln = _filled([3000, 700], 8, 1, 128, 64, fp8, seed=9)
        Q *= 30.0
        got = b.paged_attention(Q, cache, table, ln)
        _check(Q, cache, table, ln, 64, 0, got)


@pytest.mark.parametrize("what,code", [("page past the cache", 8), ("negative page", 8), ("length past the table", 6),
                                       ("negative length", 6)])
def test_attention_latches_bad_pages_and_lengths(what, code):
    from prototype_sketch_attention_b200 import binding as b
    Q, cache, table, ln = _filled([100, 500], 4, 2, 64, 16, False, seed=4)
    good = (table.clone(), ln.clone())
    if what == "page past the cache":
        table[1, 17] = cache["K"].shape[0]
    elif what == "negative page":
        table[0, 0] = -1
    elif what == "length past the table":
        ln[1] = table.shape[1] * 16 + 1
    else:
        ln[0] = -7
    got = b.paged_attention(Q, cache, table, ln)
    assert b.device_status(got["_ws"]) == code
    got = b.paged_attention(Q, cache, *good, ws=got["_ws"])  # the same workspace, good inputs
    assert b.device_status(got["_ws"]) == 0
    _check(Q, cache, *good, 16, 0, got)
    # a bad id behind the length or before the window is not read as one
    table, ln = good
    table[0, 7:], table[1, 0] = 10 ** 6, -3
    got = b.paged_attention(Q, cache, table, ln, window=300)
    assert b.device_status(got["_ws"]) == 0


def test_attention_deterministic_on_streams_and_from_a_graph():
    from prototype_sketch_attention_b200 import binding as b
    lens = [9000, 17, 0, 2500]
    Q, cache, table, ln = _filled(lens, 16, 2, 128, 64, True, seed=12)
    base = b.paged_attention(Q, cache, table, ln)
    torch.cuda.synchronize()
    res = [b.paged_attention(Q, cache, table, ln, stream=s) for s in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    for r in res:
        assert torch.equal(r["out"], base["out"]) and torch.equal(r["lse"], base["lse"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = b.paged_attention(Q, cache, table, ln, ws=base["_ws"])
    ln.copy_(_i32([3, 0, 0, 1999]))
    Q.mul_(0.5)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert b.device_status(base["_ws"]) == 0
    _check(Q, cache, table, ln, 64, 0, r)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_then_decode_steps(fp8):
    """An encoder's states go into the cache (tables, append), then each step adds one row per
    request and its token attends over everything: equal to the cross attention over the same
    rows in one piece (bf16), and to the 64-bit reference over what the cache holds."""
    from prototype_sketch_attention_b200 import binding as b
    H, Hkv, d, page = 8, 2, 128, 16
    lens = [100, 1, 0, 333]
    R = len(lens)
    g = torch.Generator(device="cuda").manual_seed(77)
    cache = b.paged_cache(80, Hkv, page, d, fmt=b.SA_CODEC_FP8 if fp8 else b.SA_CODEC_BF16)
    free = torch.randperm(80, generator=g, device="cuda").to(torch.int32)
    table = torch.full((R, 30), -1, dtype=torch.int32, device="cuda")
    held = torch.zeros(R, dtype=torch.int32, device="cuda")
    used, rows = None, [[] for _ in range(R)]
    for step in range(18):
        new = lens if step == 0 else [1] * R
        n = sum(new)
        KV = torch.randn(n, 2, Hkv, d, generator=g, device="cuda").to(BF)
        t = b.page_tables(held, _i32(new), free, table, page, n + 3, free_used=used)
        pad = torch.zeros(3, 2, Hkv, d, dtype=BF, device="cuda")
        KVp = torch.cat([KV, pad])
        b.paged_append(KVp[:, 0], KVp[:, 1], t["slots"], cache)
        at = 0
        for r in range(R):
            rows[r].append(KV[at:at + new[r]])
            at += new[r]
        held, used = t["seq_lens"], t["free_used"]
        Q = torch.randn(R, H, d, generator=g, device="cuda").to(BF)
        got = b.paged_attention(Q, cache, table, held)
        assert b.device_status(t["_ws"]) == 0 and b.device_status(got["_ws"]) == 0
        _check(Q, cache, table, held, page, 0, got)
    if not fp8:
        flat = torch.cat([torch.cat(x) for x in rows])
        off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(held.long(), 0)])
        f = b.cross_attention(Q, torch.arange(R + 1, device="cuda"), flat[:, 0], flat[:, 1], off)
        K, V = flat[:, 0].contiguous(), flat[:, 1].contiguous()
        r = ref.cross(Q, list(range(R + 1)), K, V, off.tolist())
        ref.check(f, r, ("out", "lse"))
        ref.check(got, r, ("out", "lse"))


@pytest.mark.parametrize("H,Hkv,d", [(8, 2, 64), (16, 1, 128), (4, 4, 128)])
@pytest.mark.parametrize("amp", [1e-6, 1.0, 1e3])
def test_attention_fp8_scales_of_many_magnitudes(H, Hkv, d, amp):
    """Row scales over nine decades, K against the query's magnitude: a row's product is scaled in fp32."""
    from prototype_sketch_attention_b200 import binding as b
    lens = [1, 70, 1500, 4000]
    Q, cache, table, ln = _filled(lens, H, Hkv, d, 32, True, seed=600 + H)
    g = torch.Generator(device="cuda").manual_seed(601)
    p = cache["k_scales"].shape
    cache["k_scales"].mul_(10.0 ** (torch.rand(p, generator=g, device="cuda") * 3 - 3) / amp)
    cache["v_scales"].mul_(10.0 ** (torch.rand(p, generator=g, device="cuda") * 9 - 6))
    Q.mul_(amp)
    got = b.paged_attention(Q, cache, table, ln)
    torch.cuda.synchronize()
    assert b.device_status(got["_ws"]) == 0
    _check(Q, cache, table, ln, 32, 0, got)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,H,Hkv,d", [([5, 300, 9000], 4, 2, 64), ([20000], 32, 2, 128)])
def test_attention_nan_in_reach_stays_with_its_request_and_heads(lens, H, Hkv, d, fp8):
    from prototype_sketch_attention_b200 import binding as b
    Q, cache, table, ln = _filled(lens, H, Hkv, d, 16, fp8, seed=901)
    clean = b.paged_attention(Q, cache, table, ln)
    K = cache["K"].view(torch.uint8) if fp8 else cache["K"]
    for r, pos in [(x, p) for x in range(len(lens)) for p in (0, lens[x] // 2, lens[x] - 1)]:
        at = (int(table[r, pos // 16]), 1, pos % 16, 7)
        old = K[at].clone()
        K[at] = 0x7F if fp8 else math.nan
        got = b.paged_attention(Q, cache, table, ln)
        K[at] = old
        hit = torch.zeros(Q.shape[:2], dtype=torch.bool, device="cuda")
        hit[r, H // Hkv:] = True
        assert got["out"][hit].isnan().all() and got["lse"][hit].isnan().all()
        assert torch.equal(got["out"][~hit], clean["out"][~hit]) and torch.equal(got["lse"][~hit], clean["lse"][~hit])


@pytest.mark.parametrize("fp8", [False, True])
def test_short_calls_and_stepwise_calls_agree(fp8):
    """A call with a stream goes through Python's checks, one without through the extension's."""
    from prototype_sketch_attention_b200 import binding as b
    R, H, Hkv, d, page = 5, 4, 2, 128, 16
    cached, new = [3, 0, 40, 16, 7], [1, 30, 2, 16, 0]
    g = torch.Generator(device="cuda").manual_seed(950)
    K, V = (torch.randn(sum(new) + 2, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))  # and two of padding
    Q = torch.randn(R, H, d, generator=g, device="cuda").to(BF)
    free = _i32(range(20, 60))
    got = []
    for stream in (None, torch.cuda.current_stream()):
        table = _i32(range(R * 6)).view(R, 6) % 20
        cache = b.paged_cache(64, Hkv, page, d, fmt=b.SA_CODEC_FP8 if fp8 else b.SA_CODEC_BF16)
        for x in cache.values():
            if x is not None:
                x.view(torch.uint8).zero_()
        t = b.page_tables(_i32(cached), _i32(new), free, table, page, sum(new) + 2, stream=stream)
        b.paged_append(K, V, t["slots"], cache, stream=stream)
        a = b.paged_attention(Q, cache, table, t["seq_lens"], window=20, stream=stream)
        q, k = _i32([0, 1, 2, 3, 4, 5]).long(), _i32([0, 7, 7, 20, 30, 45]).long()
        f = b.cross_attention(Q, q, K[:45], V[:45], k, stream=stream)
        r = b.cross_attention_backward(Q, q, K[:45], V[:45], k, f, Q, stream=stream)
        torch.cuda.synchronize()
        assert all(b.device_status(x["_ws"]) == 0 for x in (t, a, f, r))
        got.append([table, *(t[n] for n in ("slots", "new_offsets", "seq_lens", "free_used")), a["out"], a["lse"],
                    f["out"], f["lse"], f["rest"], r["dQ"], r["dK"], r["dV"]])
        got[-1] += [x.view(torch.uint8) for x in cache.values() if x is not None]
    assert len(got[0]) == len(got[1])
    for x, y in zip(*got):
        assert x.shape == y.shape and x.dtype == y.dtype and torch.equal(x, y)
    assert isinstance(b._calls.paged_attention(Q, cache["K"], cache["V"], cache["k_scales"], cache["v_scales"], table,
                                               t["seq_lens"], 0, None, None), dict)
    assert b._calls.paged_append(K, V, t["slots"], cache["K"], cache["V"], cache["k_scales"],
                                 cache["v_scales"]) == 0
    with pytest.raises(b.SketchAttentionError):  # a status of the C ABI (an uneven workspace)
        b.paged_attention(Q, cache, table, t["seq_lens"], ws=torch.empty(300, dtype=torch.uint8, device="cuda")[1:])
