"""Cases of the multi-head cross attention and of its paged serving cache, measured.

Five operators, in the order in which a program uses them:

  train     multi-head cross attention from ragged queries to an encoder's states of other
            lengths (shared heads, key masks), forward and backward
  fwd       its forward alone
  tables    block tables and slot maps of a paged key-value cache, from request lengths
  append    new key and value rows into the cache's pages (bf16, or FP8 E4M3 with row scales)
  attend    attention of one new token per request over the paged cache

A case is a dict of plain values. `own` chooses between the plain form (elementary torch
operations in 32 bits) and the library's calls. Lengths come from the case's own "shape"
number, values from the seed.
"""
import math
import random

import torch

own = False

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one user's candidates over that user's sketch rows: the smallest call, latency counts
        dict(name="fwd_one_user", op="fwd", R=1, q_lo=40, q_hi=40, k_lo=1024, k_hi=1024, H=4, Hkv=4, d=64,
             masked=False, shape=1),
        # the training batch's 40 users x 300 candidates over the recent 10K history rows
        dict(name="fwd_recent_40x300", op="fwd", R=40, q_lo=300, q_hi=300, k_lo=10000, k_hi=10000, H=8, Hkv=2,
             d=128, masked=False, shape=2),
        # the same candidates over sketches of 1024 rows, every head with its own keys
        dict(name="train_sketch_40x300", op="train", R=40, q_lo=300, q_hi=300, k_lo=1024, k_hi=1024, H=8, Hkv=8,
             d=64, masked=False, shape=3),
        # ragged histories of up to 10K rows with padding inside them masked, heads shared by pairs
        dict(name="train_recent_masked", op="train", R=40, q_lo=100, q_hi=300, k_lo=1000, k_hi=10000, H=8, Hkv=4,
             d=128, masked=True, shape=4),
        # a small odd batch: a user without keys, one whose mask leaves nothing, three heads per key head
        dict(name="train_odd", op="train", R=7, q_lo=1, q_hi=131, k_lo=0, k_hi=777, H=6, Hkv=2, d=128, masked=True,
             shape=5),
        # a decode step of the serving batch: one token for each of 300 requests
        dict(name="tables_decode_300", op="tables", R=300, c_lo=1000, c_hi=100000, n_lo=1, n_hi=1, page=64, shape=6),
        # the serving batch's whole histories laid out in pages at once
        dict(name="tables_prefill_300", op="tables", R=300, c_lo=0, c_hi=0, n_lo=1000, n_hi=100000, page=16,
             shape=7),
        # that decode step's rows, in FP8
        dict(name="append_decode_fp8", op="append", n=300, Hkv=8, d=128, page=16, fp8=True, shape=8),
        # histories written in one call, in bf16, some slots of the padded batch unused
        dict(name="append_prefill_bf16", op="append", n=300001, Hkv=2, d=128, page=64, fp8=False, shape=9),
        # one request with a short history: latency counts
        dict(name="attend_one", op="attend", R=1, lo=1900, hi=1900, H=8, Hkv=8, d=64, page=16, fp8=False, window=0,
             shape=10),
        # the training batch's users reading their recent 10K rows, three heads per key head
        dict(name="attend_recent_40", op="attend", R=40, lo=10000, hi=100000, H=12, Hkv=4, d=128, page=16,
             fp8=False, window=10000, shape=11),
        # the serving batch over whole histories in FP8, one key head for eight
        dict(name="attend_serving_300", op="attend", R=300, lo=1000, hi=100000, H=8, Hkv=1, d=128, page=64, fp8=True,
             window=0, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "train", "train", "tables", "append", "attend", "attend"])
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        c = dict(op=op, shape=rng.randrange(1 << 30))
        if op in ("fwd", "train"):
            hkv = rng.choice([1, 2, 3, 4, 8])
            q, k = _log(rng, 1, 600), _log(rng, 1, 10000)
            c.update(R=_log(rng, 1, 40), q_lo=rng.choice([q, q // 3]), q_hi=q, k_lo=rng.choice([k, k // 8, 0]), k_hi=k,
                     H=hkv * rng.choice([1, 2, 3, 4, 8]), Hkv=hkv, d=rng.choice([64, 128]), masked=rng.random() < 0.4)
        elif op == "tables":
            n = _log(rng, 1, 100000)
            c.update(R=_log(rng, 1, 1000), c_lo=0, c_hi=rng.choice([0, _log(rng, 1, 100000)]),
                     n_lo=rng.choice([n, n // 100]), n_hi=n, page=rng.choice([8, 16, 32, 64, 128]))
        elif op == "append":
            c.update(n=_log(rng, 1, 300000), Hkv=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([64, 128]),
                     page=rng.choice([8, 16, 32, 64, 128]), fp8=rng.random() < 0.5)
        else:
            hkv, hi = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 100000)
            c.update(R=_log(rng, 1, 300), lo=rng.choice([hi, hi // 10, 0]), hi=hi, H=hkv * rng.choice([1, 2, 3, 4, 8, 16]),
                     Hkv=hkv, d=rng.choice([64, 128]), page=rng.choice([8, 16, 32, 64, 128]), fp8=rng.random() < 0.5,
                     window=rng.choice([0, 0, _log(rng, 1, 10000)]))
        if _cost(c) <= most and _padded(c) <= 4.2e9 and (op != "tables" or c["R"] * c["n_hi"] <= 3e7):
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _padded(c):
    """Values of the largest padded array that the plain form makes of a case."""
    if c["op"] in ("fwd", "train"):
        return c["R"] * c["H"] * c["q_hi"] * c["k_hi"]
    if c["op"] == "attend":
        return c["R"] * c["Hkv"] * c["d"] * (min(c["hi"], c["window"]) if c["window"] else c["hi"])
    return 0


def _lengths(c, salt, n, lo, hi):
    """n lengths in [lo, hi], spread over their logarithm; the first is hi, and lo = 0 gives some of 0."""
    r = random.Random(c["shape"] * 7919 + salt)
    a = [int(round(math.exp(r.uniform(math.log(max(lo, 1)), math.log(max(hi, 1)))))) if hi else 0 for _ in range(n)]
    if lo == 0 and hi:
        a = [0 if r.random() < 0.2 else x for x in a]
    return [hi] + a[1:]


def _cross_lengths(c):
    return _lengths(c, 1, c["R"], c["q_lo"], c["q_hi"]), _lengths(c, 2, c["R"], c["k_lo"], c["k_hi"])


def _span(c, n):
    return min(n, c["window"]) if c["window"] else n


def work(c):
    """Bytes with each input read and each output written once, and the products' operations."""
    if c["op"] in ("fwd", "train"):
        lq, lk = _cross_lengths(c)
        pairs = sum(a * b for a, b in zip(lq, lk)) * c["H"]
        q, k = sum(lq) * c["H"] * c["d"] * 2, sum(lk) * c["Hkv"] * c["d"] * 2
        small = sum(lq) * c["H"] * 4 + (sum(lk) if c["masked"] else 0) + 16 * (c["R"] + 1)
        if c["op"] == "fwd":  # Q, K, V; out, lse
            return {"bytes": 2 * q + 2 * k + small, "flops": 4 * c["d"] * pairs}
        return {"bytes": 4 * q + 4 * k + small, "flops": 14 * c["d"] * pairs}  # and dout; dQ, dK, dV
    if c["op"] == "tables":
        cached, new, p = *_table_lengths(c), c["page"]
        pages = sum(-(-(a + b) // p) - -(-a // p) for a, b in zip(cached, new))
        return {"bytes": 8 * sum(new) + 8 * pages + 24 * c["R"], "flops": 0}  # slots; free list, new entries; lengths
    if c["op"] == "append":
        row = c["Hkv"] * (c["d"] * (3 if c["fp8"] else 4) + (4 if c["fp8"] else 0))
        return {"bytes": c["n"] * (2 * row + 8), "flops": 0}
    ls = [_span(c, n) for n in _lengths(c, 3, c["R"], c["lo"], c["hi"])]
    row = c["Hkv"] * (c["d"] + 4 if c["fp8"] else 2 * c["d"])
    io = c["R"] * c["H"] * (4 * c["d"] + 4)
    return {"bytes": sum(ls) * 2 * row + sum(-(-n // c["page"]) for n in ls) * 4 + io,
            "flops": 4 * c["d"] * c["H"] * sum(ls)}


# ---------------------------------------------------------------- inputs
def _table_lengths(c):
    return _lengths(c, 4, c["R"], min(c["c_lo"], c["c_hi"]), c["c_hi"]), _lengths(c, 5, c["R"], c["n_lo"], c["n_hi"])


def _offsets(lengths):
    o = [0]
    for n in lengths:
        o.append(o[-1] + n)
    return torch.tensor(o, dtype=torch.int64).cuda()


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(BF16)


def _pages(g, lengths, page, spare=0):
    """Every request's pages, shuffled over the cache as a server's are: (table [R, width] int32, pages)."""
    counts = [-(-n // page) for n in lengths]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(max(counts), 1)
    cnt = torch.tensor(counts).cuda()
    start = torch.cumsum(cnt, 0) - cnt
    col = torch.arange(width, device="cuda")
    at = (start[:, None] + col).clamp(max=max(total - 1, 0))
    none = torch.zeros((), dtype=torch.int32, device="cuda")
    return torch.where(col < cnt[:, None], order[at] if total else none, none), max(total, 1)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(c=c)
    if c["op"] in ("fwd", "train"):
        lq, lk = _cross_lengths(c)
        s.update(Q=_randn(g, sum(lq), c["H"], c["d"]), K=_randn(g, sum(lk), c["Hkv"], c["d"]),
                 V=_randn(g, sum(lk), c["Hkv"], c["d"]), qo=_offsets(lq), ko=_offsets(lk), mask=None)
        if c["masked"]:
            s["mask"] = torch.rand(sum(lk), generator=g, device="cuda") < 0.9
            if c["R"] > 1:  # the last user's mask leaves nothing
                s["mask"][sum(lk[:-1]):] = False
        if c["op"] == "train":
            s["dout"] = _randn(g, sum(lq), c["H"], c["d"])
    elif c["op"] == "tables":
        cached, new = _table_lengths(c)
        p = c["page"]
        table, used = _pages(g, cached, p)
        need = sum(-(-(a + b) // p) - -(-a // p) for a, b in zip(cached, new))
        width = max(max(-(-(a + b) // p) for a, b in zip(cached, new)), table.shape[1])
        s["table"] = torch.full((c["R"], width), -1, dtype=torch.int32, device="cuda")
        s["table"][:, :table.shape[1]] = table
        skip = 1 + seed % 5  # pages of the free list that earlier steps took
        s.update(cached=torch.tensor(cached, dtype=torch.int32).cuda(), new=torch.tensor(new, dtype=torch.int32).cuda(),
                 free=(torch.randperm(need + skip + 9, generator=g, device="cuda") + used).to(torch.int32),
                 free_used=torch.tensor([skip], dtype=torch.int64).cuda(), n_slots=sum(new))
    elif c["op"] == "append":
        pages = -(-c["n"] * 5 // (4 * c["page"])) + 1
        slots = torch.randperm(pages * c["page"], generator=g, device="cuda")[:c["n"]]
        if c["n"] > 100:  # the padding of a batch of fixed size
            slots[-7:] = -1
        kind = F8 if c["fp8"] else BF16
        s["cache"] = _empty_cache(pages, c, kind)
        s.update(K=_randn(g, c["n"], c["Hkv"], c["d"]), V=_randn(g, c["n"], c["Hkv"], c["d"]), slots=slots)
    else:
        ls = _lengths(c, 3, c["R"], c["lo"], c["hi"])
        s["table"], pages = _pages(g, ls, c["page"], spare=3)
        s["cache"] = _empty_cache(pages, c, F8 if c["fp8"] else BF16)
        for name in ("K", "V"):
            if c["fp8"]:
                x = torch.randn(s["cache"][name].shape, generator=g, device="cuda")
                sc = x.abs().amax(-1) / 448
                s["cache"][name] = (x / sc[..., None]).to(F8)
                s["cache"][name.lower() + "_scales"] = sc
            else:
                s["cache"][name] = _randn(g, *s["cache"][name].shape)
        s.update(Q=_randn(g, c["R"], c["H"], c["d"]), lens=torch.tensor(ls, dtype=torch.int32).cuda())
    return s


def _empty_cache(pages, c, kind):
    shape = (pages, c["Hkv"], c["page"], c["d"])
    cache = {"K": torch.zeros(shape, device="cuda").to(kind), "V": torch.zeros(shape, device="cuda").to(kind),
             "k_scales": None, "v_scales": None}
    if kind == F8:
        cache["k_scales"] = torch.ones(shape[:3], device="cuda")
        cache["v_scales"] = torch.ones(shape[:3], device="cuda")
    return cache


# ---------------------------------------------------------------- one pass
def run(s):
    return _RUN[s["c"]["op"]](s)


def _run_fwd(s):
    if own:
        from prototype_sketch_attention_b200 import binding
        f = binding.cross_attention(s["Q"], s["qo"], s["K"], s["V"], s["ko"], key_mask=s["mask"])
        return f["out"], f["lse"]
    o, lse, *_ = _plain_forward(s)
    return o.to(BF16), lse


def _run_train(s):
    if own:
        from prototype_sketch_attention_b200 import binding
        f = binding.cross_attention(s["Q"], s["qo"], s["K"], s["V"], s["ko"], key_mask=s["mask"])
        b = binding.cross_attention_backward(s["Q"], s["qo"], s["K"], s["V"], s["ko"], f, s["dout"],
                                             key_mask=s["mask"])
        return f["out"], f["lse"], b["dQ"], b["dK"], b["dV"]
    return _plain_train(s)


def _run_tables(s):
    if own:
        from prototype_sketch_attention_b200 import binding
        t = binding.page_tables(s["cached"], s["new"], s["free"], s["table"], s["c"]["page"], s["n_slots"],
                                free_used=s["free_used"])
        return s["table"], t["slots"], t["new_offsets"], t["seq_lens"], t["free_used"]
    return _plain_tables(s)


def _run_append(s):
    if own:
        from prototype_sketch_attention_b200 import binding
        binding.paged_append(s["K"], s["V"], s["slots"], s["cache"])
    else:
        _plain_append(s)
    return s["cache"]


def _run_attend(s):
    if own:
        from prototype_sketch_attention_b200 import binding
        f = binding.paged_attention(s["Q"], s["cache"], s["table"], s["lens"], window=s["c"]["window"])
        return f["out"], f["lse"]
    return _plain_attend(s)


# ---------------------------------------------------------------- plain forms
def _where(offsets, n):
    """Every row's user and its place in the user's rows."""
    i = torch.arange(n, device=offsets.device)
    u = torch.searchsorted(offsets, i, right=True) - 1
    return u, i - offsets[u]


def _rows(offsets, width, n):
    """[R, width] row numbers of the users' rows, and which of them are rows of that user."""
    j = torch.arange(width, device=offsets.device)
    return (offsets[:-1, None] + j).clamp(max=max(n - 1, 0)), j < (offsets[1:] - offsets[:-1])[:, None]


def _padded_inputs(s):
    """Queries as [R, Hkv, G Lq, d], keys and values as [R, Hkv, Lk, d], in 32 bits, and which keys count."""
    c = s["c"]
    R, H, Hkv, d = c["R"], c["H"], c["Hkv"], c["d"]
    nq, nk = s["Q"].shape[0], s["K"].shape[0]
    qi, qok = _rows(s["qo"], c["q_hi"], nq)
    ki, kok = _rows(s["ko"], max(c["k_hi"], 1), nk)

    def heads(x):  # [n, H, d] -> [R, Hkv, G Lq, d]
        x = x.float()[qi] * qok[:, :, None, None]
        return x.view(R, -1, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4).reshape(R, Hkv, -1, d)

    def keys(x):
        if nk == 0:
            return torch.zeros(R, Hkv, ki.shape[1], d, device=x.device)
        return (x.float()[ki] * kok[:, :, None, None]).permute(0, 2, 1, 3)

    if s["mask"] is not None and nk:
        kok = kok & s["mask"][ki]
    return heads, heads(s["Q"]), keys(s["K"]), keys(s["V"]), kok[:, None, None, :]


def _ragged(x, offsets, n, H):
    """[R, Hkv, G L, ...] -> [n, H, ...]"""
    u, p = _where(offsets, n)
    R, Hkv = x.shape[:2]
    x = x.reshape(R, H, -1, *x.shape[3:])
    return x[u, :, p]


def _softmax(z, ok):
    """exp(z - max) of what counts, its sum and the log of the sum of exp; rows without anything give 0 and -inf."""
    z = z.masked_fill_(~ok, -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z.sub_(torch.where(m > -math.inf, m, 0.0)))
    l = e.sum(-1, keepdim=True)
    return e, l, (m + torch.log(l))[..., 0]


def _plain_forward(s):
    c = s["c"]
    heads, q, k, v, ok = _padded_inputs(s)
    e, l, lse = _softmax(q @ k.transpose(-1, -2) / math.sqrt(c["d"]), ok)
    o = (e @ v) / torch.where(l > 0, l, 1.0)
    n = s["Q"].shape[0]
    return _ragged(o, s["qo"], n, c["H"]), _ragged(lse, s["qo"], n, c["H"]), heads, q, k, v, e, l, o


def _plain_train(s):
    c = s["c"]
    out, lse, heads, q, k, v, e, l, o = _plain_forward(s)
    p = e.div_(torch.where(l > 0, l, 1.0))
    do = heads(s["dout"])
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).div_(math.sqrt(c["d"]))
    dq, dk = ds @ k, ds.transpose(-1, -2) @ q
    n, nk = s["Q"].shape[0], s["K"].shape[0]
    return (out.to(BF16), lse, _ragged(dq, s["qo"], n, c["H"]).to(BF16), _ragged(dk, s["ko"], nk, c["Hkv"]).to(BF16),
            _ragged(dv, s["ko"], nk, c["Hkv"]).to(BF16))


def _plain_tables(s):
    p = s["c"]["page"]
    cached, new = s["cached"].long(), s["new"].long()
    end = cached + new
    have, want = (cached + p - 1) // p, (end + p - 1) // p
    need = want - have
    first = s["free_used"] + torch.cumsum(need, 0) - need
    col = torch.arange(s["table"].shape[1], device=new.device)
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][at], s["table"]))
    off = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    u, i = _where(off, s["n_slots"])
    pos = cached[u] + i
    slots = s["table"][u, pos // p].long() * p + pos % p
    return s["table"], slots, off, end.to(torch.int32), s["free_used"] + need.sum()


def _plain_append(s):
    cache, page = s["cache"], s["c"]["page"]
    used = s["slots"] >= 0
    # unused slots write what the first row's slot gets: the same value twice
    src = torch.where(used, torch.arange(used.numel(), device=used.device), 0)
    at = s["slots"][src]
    pg, row = at // page, at % page
    for x, name in ((s["K"], "K"), (s["V"], "V")):
        x = x[src].float()
        if cache["k_scales"] is not None:
            m = x.abs().amax(-1)
            sc = torch.where(m > 0, m / 448, 1.0)
            cache[name.lower() + "_scales"][pg, :, row] = sc
            cache[name].view(torch.uint8)[pg, :, row] = (x / sc[..., None]).to(F8).view(torch.uint8)
        else:
            cache[name][pg, :, row] = x.to(BF16)


def _plain_attend(s):
    c, cache, lens = s["c"], s["cache"], s["lens"].long()
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    width = max(_span(c, c["hi"]), 1)
    j = first[:, None] + torch.arange(width, device=lens.device)
    ok = j < lens[:, None]
    j = j.clamp(max=s["table"].shape[1] * c["page"] - 1)
    pg, row = torch.gather(s["table"], 1, j // c["page"]).long(), j % c["page"]

    def rows(name):  # [R, Hkv, width, d]
        codes, sc = cache[name], cache[name.lower() + "_scales"]
        x = codes.view(torch.uint8)[pg, :, row].view(F8).float() if sc is not None else codes[pg, :, row].float()
        return (x.mul_(sc[pg, :, row][..., None]) if sc is not None else x).transpose(1, 2)

    R, H, Hkv, d = c["R"], c["H"], c["Hkv"], c["d"]
    z = s["Q"].float().view(R, Hkv, H // Hkv, d) @ rows("K").transpose(-1, -2) / math.sqrt(d)
    e, l, lse = _softmax(z, ok[:, None, None, :])
    o = (e @ rows("V")) / torch.where(l > 0, l, 1.0)
    return o.reshape(R, H, d).to(BF16), lse.reshape(R, H)


_RUN = {"fwd": _run_fwd, "train": _run_train, "tables": _run_tables, "append": _run_append, "attend": _run_attend}


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    """run()'s numbers from the definition in 64 bits, one user (and head) at a time."""
    if c["op"] == "tables":
        return None  # whole numbers
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s) if c["op"] == "attend" else _exact_cross(s)


def _exact_one(q, k, v, scale):
    """Softmax attention of q [m, d] over k, v [n, d]: output, log of the sum of exp, weights."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), q.new_full((q.shape[0],), -math.inf), q.new_zeros(q.shape[0], 0)
    z = (q @ k.T) * scale
    lse = torch.logsumexp(z, dim=1)
    w = torch.exp(z - lse[:, None])
    return w @ v, lse, w


def _exact_cross(s):
    c = s["c"]
    G, scale = c["H"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    Q, K, V = s["Q"].double(), s["K"].double(), s["V"].double()
    out, lse = torch.zeros_like(Q), torch.zeros(Q.shape[:2], dtype=torch.float64, device="cuda")
    dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    qo, ko = s["qo"].tolist(), s["ko"].tolist()
    for u in range(c["R"]):
        a, b = qo[u], qo[u + 1]
        keep = torch.arange(ko[u], ko[u + 1], device="cuda")
        if s["mask"] is not None:
            keep = keep[s["mask"][keep]]
        for h in range(c["H"]):
            q, k, v = Q[a:b, h], K[keep, h // G], V[keep, h // G]
            o, l, w = _exact_one(q, k, v, scale)
            out[a:b, h], lse[a:b, h] = o, l
            if c["op"] == "train":
                g = s["dout"][a:b, h].double()
                dz = w * (g @ v.T - (g * o).sum(1, keepdim=True)) * scale
                dQ[a:b, h] = dz @ k
                dK[keep, h // G] += dz.T @ q
                dV[keep, h // G] += w.T @ g
    return (out, lse) if c["op"] == "fwd" else (out, lse, dQ, dK, dV)


def _exact_append(s):
    page, cache = s["c"]["page"], s["cache"]
    n = int((s["slots"] >= 0).sum())
    pg, row = s["slots"][:n] // page, s["slots"][:n] % page
    if s["c"]["fp8"]:  # the codes themselves are whole steps of the type: only the scales are numbers
        got = {"K": None, "V": None}
        for name, x in (("k_scales", s["K"]), ("v_scales", s["V"])):
            got[name] = cache[name].double()
            got[name][pg, :, row] = x[:n].double().abs().amax(-1) / 448
        return got
    got = {"k_scales": None, "v_scales": None}
    for name in ("K", "V"):
        got[name] = cache[name].double()
        got[name][pg, :, row] = s[name][:n].double()
    return got


def _exact_attend(s):
    c, cache = s["c"], s["cache"]
    G, scale = c["H"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    out = torch.zeros(c["R"], c["H"], c["d"], dtype=torch.float64, device="cuda")
    lse = torch.zeros(c["R"], c["H"], dtype=torch.float64, device="cuda")
    for u, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n - _span(c, n), n, device="cuda")
        pg, row = s["table"][u].long()[j // c["page"]], j % c["page"]
        for h in range(c["Hkv"]):
            k, v = (cache[x][:, h].view(torch.uint8)[pg, row].view(F8).double() if c["fp8"] else
                    cache[x][:, h][pg, row].double() for x in ("K", "V"))
            if c["fp8"]:
                k, v = k * cache["k_scales"][pg, h, row][:, None], v * cache["v_scales"][pg, h, row][:, None]
            o, l, _ = _exact_one(s["Q"][u, h * G:(h + 1) * G].double(), k, v, scale)
            out[u, h * G:(h + 1) * G], lse[u, h * G:(h + 1) * G] = o, l
    return out, lse
