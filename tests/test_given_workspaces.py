"""A workspace that the caller gives: of another device, or with fewer bytes than its shape says, it is
refused before its pointer reaches the library."""
import contextlib

import pytest
import torch

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


@pytest.fixture(scope="module")
def b():
    from prototype_sketch_attention_b200 import build
    build.build()
    from prototype_sketch_attention_b200 import binding
    return binding


def _calls(b, dev):
    def z(*s, dt=BF):
        return torch.zeros(*s, dtype=dt, device=dev)
    off = torch.tensor([0, 2, 6], device=dev)
    X, W, S, P, g = z(6, 128), z(128, 128), z(2, 16, 128, dt=F32), z(16, 128), z(6, 128, dt=F32)
    kb, ke = torch.tensor([0, 2], device=dev), torch.tensor([2, 6], device=dev)
    one = torch.ones(2, 16, device=dev)
    sk = {"sketch": S, "mass": one, "xsketch": S}
    cr = (z(6, 4, 64), off, z(6, 2, 64), z(6, 2, 64), off)
    f = {"out": z(6, 4, 64), "lse": z(6, 4, dt=F32)}
    cache = {"K": z(8, 2, 16, 64), "V": z(8, 2, 16, 64), "k_scales": None, "v_scales": None}
    ln, table = torch.tensor([4, 3], dtype=I32, device=dev), z(2, 2, dt=I32)
    return {
        "forward": lambda ws: b.forward(X, off, P, W, W, ws=ws),
        "backward": lambda ws: b.backward(X, off, P, W, W, sk, S, ws=ws),
        "stca_forward": lambda ws: b.stca_forward(X, off, S, W, W, W, ws=ws),
        "stca_backward": lambda ws: b.stca_backward(X, off, S, W, W, W, g, ws=ws),
        "stca_keys_forward": lambda ws: b.stca_keys_forward(X, off, X, kb, ke, W, W, W, ws=ws),
        "stca_keys_backward": lambda ws: b.stca_keys_backward(X, off, X, kb, ke, W, W, W, g, ws=ws),
        "cross_attention": lambda ws: b.cross_attention(*cr, ws=ws),
        "cross_attention_backward": lambda ws: b.cross_attention_backward(*cr, f, cr[0], ws=ws),
        "page_tables": lambda ws: b.page_tables(ln, ln, ln, table, 16, 7, ws=ws),
        "paged_attention": lambda ws: b.paged_attention(cr[0][:2], cache, table, ln, ws=ws),
    }


NAMES = list(_calls(None, "cpu"))


def _bad(dev):
    other = "meta" if dev == "cpu" else "cpu"
    return {"of another device": torch.empty(1 << 20, dtype=torch.uint8, device=other),
            "expanded": torch.empty(1, dtype=torch.uint8, device=dev).expand(1 << 20),
            "strided": torch.empty(1 << 20, dtype=torch.uint8, device=dev)[::2],
            "no tensor": 1 << 20}


class _Library:
    """Stands in for the library: sizes, and success of every call that should not have been made."""
    def __getattr__(self, name):
        if name == "sa_status_string":
            return lambda *a: b"refused"
        return lambda *a: 256 if name.endswith("workspace_size") else 0


@pytest.mark.parametrize("what", list(_bad("cpu")))
@pytest.mark.parametrize("name", NAMES)
def test_unusable_workspace_is_refused(b, name, what, monkeypatch):
    monkeypatch.setattr(b, "_lib", _Library())
    monkeypatch.setattr(b, "_check_cuda", lambda *a: None)
    monkeypatch.setattr(b, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(b, "_stream", lambda *a: 0)
    call = _calls(b, "cpu")[name]
    call(torch.empty(1 << 20, dtype=torch.uint8))  # a good one
    with pytest.raises(b.SketchAttentionError, match="ws must be") as e:
        call(_bad("cpu")[what])
    assert e.value.status == b.SA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_unusable_workspace_is_refused_on_the_gpu(b, name):
    """The short calls' extension, too, hands such a call back, and the reason is given in Python."""
    call = _calls(b, "cuda")[name]
    for what, ws in _bad("cuda").items():
        with pytest.raises(b.SketchAttentionError, match="ws must be"):
            call(ws)
