"""A bf16 cache that is a dictionary of K and V alone is the same cache with and without a given stream."""
import contextlib

import pytest
import torch

BF, I32 = torch.bfloat16, torch.int32


def _inputs(b, dev):
    g = torch.Generator().manual_seed(3)

    def r(*s):
        return torch.randn(*s, generator=g).to(BF).to(dev)
    cache = {"K": r(4, 2, 16, 64), "V": r(4, 2, 16, 64)}
    return (cache, r(2, 4, 64), r(3, 2, 64), r(3, 2, 64), torch.tensor([5, 6, 40], device=dev),
            torch.tensor([[0, 1], [2, 3]], dtype=I32, device=dev), torch.tensor([20, 9], dtype=I32, device=dev))


def test_without_scales_on_the_steps_of_python(monkeypatch):
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding as b

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(a) or (256 if name.endswith("workspace_size") else 0)
    seen = []
    monkeypatch.setattr(b, "_lib", Library())
    monkeypatch.setattr(b, "_check_cuda", lambda *a: None)
    monkeypatch.setattr(b, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(b, "_stream", lambda *a: 0)
    cache, Q, K, V, slots, table, lens = _inputs(b, "cpu")
    b.paged_append(K, V, slots, cache)
    b.paged_attention(Q, cache, table, lens)
    assert len(seen) == 3 and seen[0][11:13] == (None, None) and seen[2][7:9] == (None, None)


@pytest.mark.gpu
def test_without_scales_with_and_without_a_stream():
    from prototype_sketch_attention_b200 import binding as b
    got = []
    for stream in (None, torch.cuda.current_stream()):
        cache, Q, K, V, slots, table, lens = _inputs(b, "cuda")
        b.paged_append(K, V, slots, cache, stream=stream)
        got.append([b.paged_attention(Q, cache, table, lens, stream=stream)["out"], cache["K"], cache["V"]])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*got))
