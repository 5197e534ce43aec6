"""Calls with a given stream: where their results and workspaces come from, and how long their
tensors stay allocated.

The caching allocator hands a freed block out again to its own stream at once, although work queued
there may still use it. A call whose kernels run on another stream may therefore not write into a
block of the current stream's pool. On the CPU the library and the streams are replaced by records; on the
GPU a block that queued work still needs is free while the call is made."""
import contextlib

import pytest
import torch

BF, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def _tensors(dev):
    """Inputs of every call: 2 users, 6 queries or tokens, 9 keys, heads 4 over 2 of 64; 8 pages of 16."""
    g = torch.Generator().manual_seed(1)

    def r(*s, dt=BF):
        return torch.randn(*s, generator=g).to(dt).to(dev)

    def i(x, dt=I64):
        return torch.tensor(x, dtype=dt, device=dev)
    d = 128
    x = dict(X=r(6, d), off=i([0, 2, 6]), P=r(16, d), W=r(d, d, dt=F32).mul(0.1).to(BF), S=r(2, 16, d, dt=F32),
             mass=torch.ones(2, 16, device=dev), dS=r(2, 16, d, dt=F32), cand=r(6, d), dcand=r(6, d, dt=F32),
             kb=i([0, 3]), ke=i([3, 6]), offh=torch.tensor([0, 2, 6]),
             Q=r(6, 4, 64), K=r(9, 2, 64), V=r(9, 2, 64), ko=i([0, 4, 9]), dO=r(6, 4, 64),
             cached=i([3, 0], I32), new=i([1, 2], I32), free=i(list(range(2, 8)), I32), table=i([[0, 1], [1, 0]], I32),
             slots=i([3, 16, 17]), lens=i([4, 3], I32), q1=r(2, 4, 64), lse=r(6, 4, dt=F32))
    x["cache"] = {"K": r(8, 2, 16, 64), "V": r(8, 2, 16, 64), "k_scales": None, "v_scales": None}
    return x


def _calls(b, x, stream):
    """(name, call, tensors the call is given)"""
    W = x["W"]
    sk = {"sketch": x["S"], "mass": x["mass"], "xsketch": x["S"]}
    cr = (x["Q"], x["off"], x["K"], x["V"], x["ko"])
    c = x["cache"]
    keys = (x["cand"], x["off"], x["X"], x["kb"], x["ke"], W, W, W)
    return [
        ("forward", lambda: b.forward(x["X"], x["off"], x["P"], W, W, stream=stream), [x["X"], x["off"], x["P"]]),
        ("backward", lambda: b.backward(x["X"], x["off"], x["P"], W, W, sk, x["dS"], stream=stream), [x["S"], x["dS"]]),
        ("combine", lambda: b.combine(x["S"], x["mass"], W, stream=stream), [x["S"], x["mass"], W]),
        ("stca_forward", lambda: b.stca_forward(x["cand"], x["off"], x["S"], W, W, W, stream=stream), [x["cand"]]),
        ("stca_backward", lambda: b.stca_backward(x["cand"], x["off"], x["S"], W, W, W, x["dcand"],
                                                  cand_offsets_host=x["offh"], stream=stream), [x["dcand"]]),
        ("recent_ranges", lambda: b.recent_ranges(x["off"], 2, stream=stream), [x["off"]]),
        ("stca_keys_forward", lambda: b.stca_keys_forward(*keys, stream=stream), [x["kb"], x["ke"]]),
        ("stca_keys_backward", lambda: b.stca_keys_backward(*keys, x["dcand"], stream=stream), [x["dcand"], W]),
        ("sketch_pack", lambda: b.sketch_pack(x["S"], stream=stream), [x["S"]]),
        ("sketch_unpack", lambda: b.sketch_unpack({"codes": x["K"].view(torch.int16).view(18, 64), "format": 0},
                                                  stream=stream), []),
        ("cross_attention", lambda: b.cross_attention(*cr, stream=stream), list(cr)),
        ("cross_attention_backward",
         lambda: b.cross_attention_backward(*cr, {"out": x["dO"], "lse": x["lse"]}, x["dO"], stream=stream),
         [*cr, x["dO"], x["lse"]]),
        ("page_tables", lambda: b.page_tables(x["cached"], x["new"], x["free"], x["table"], 16, 3, stream=stream),
         [x["cached"], x["new"], x["free"], x["table"]]),
        ("paged_append", lambda: b.paged_append(x["K"][:3], x["V"][:3], x["slots"], c, stream=stream),
         [x["slots"], c["K"], c["V"]]),
        ("paged_attention", lambda: b.paged_attention(x["q1"], c, x["table"], x["lens"], stream=stream),
         [x["q1"], x["table"], x["lens"], c["K"], c["V"]]),
    ]


NAMES = [n for n, *_ in _calls(None, _tensors("cpu"), None)]


def _flat(res):
    if isinstance(res, torch.Tensor):
        return [res]
    vals = res.values() if isinstance(res, dict) else res or ()
    return [t for t in vals if isinstance(t, torch.Tensor)]


class _Library:
    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith("workspace_size") else 0


class _FakeStream:
    device, cuda_stream = torch.device("cpu"), 0


@pytest.mark.parametrize("name", NAMES)
def test_allocations_come_from_the_given_stream(name, monkeypatch):
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding as b
    x, given, callers = _tensors("cpu"), _FakeStream(), object()
    current, made, recorded = [callers], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def empty(*a, real=torch.empty, **kw):
        made.append(current[-1])
        return real(*a, **kw)
    monkeypatch.setattr(b, "_lib", _Library())
    monkeypatch.setattr(b, "_check_cuda", lambda *a: None)
    monkeypatch.setattr(b, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    _, call, inputs = next(c for c in _calls(b, x, given) if c[0] == name)
    res = _flat(call())
    assert made or name == "paged_append"
    assert all(s is given for s in made)
    for t in inputs:  # a tensor dropped early stays allocated until the given stream has passed the call
        assert (t.data_ptr(), given) in recorded
    for t in res:     # and a result until the caller's stream has
        assert (t.data_ptr(), callers) in recorded


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding as b
    monkeypatch.setattr(b, "_check_cuda", lambda *a: None)

    class Other(_FakeStream):
        device = torch.device("cuda", 1)
    for _, call, _ in _calls(b, _tensors("cpu"), Other()):
        with pytest.raises(b.SketchAttentionError, match="stream"):
            call()


def _named(res):
    if isinstance(res, torch.Tensor):
        return {"": res}
    items = res.items() if isinstance(res, dict) else enumerate(res or ())
    return {n: t for n, t in items if isinstance(t, torch.Tensor) and n != "_ws"}


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_a_block_that_queued_work_still_needs_is_not_written(name):
    """Blocks of every result's size are freed on the current stream while copies out of them wait there;
    the call on another stream at once leaves them alone, and gives what it gives without a stream."""
    from prototype_sketch_attention_b200 import binding as b
    x, s = _tensors("cuda"), torch.cuda.Stream()
    plain, call = (next(c for c in _calls(b, x, to) if c[0] == name)[1] for to in (None, s))
    first = plain()
    want = {n: t.clone() for n, t in _named(first).items()}
    sizes = [t.nbytes for t in _flat(first)]
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    kept = [torch.empty_like(t) for t in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    while blocks:
        kept[len(blocks) - 1].copy_(blocks.pop())
    got = call()
    s.synchronize()
    got = {n: t.clone() for n, t in _named(got).items()}
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in kept)
    assert got.keys() == want.keys()
    for n, w in want.items():
        # the single-head gradients' fp32 reductions meet in L2, in no fixed order: off by 2^-24 of the terms'
        # magnitudes a term, which are at most some hundred times the largest result
        a, w = got[n].double(), w.double()
        assert (a - w).abs().max() <= 1e-4 * w.abs().max() if w.numel() else a.numel() == 0, n
