"""The extension of the short calls is an addition: without it every operator is there, through Python's own
steps, and one that was compiled against another torch or Python is neither used nor taken for current."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def build():
    from prototype_sketch_attention_b200 import build
    build.build()
    return build


@pytest.mark.parametrize("state", ["missing", "of another machine"])
def test_the_package_imports_without_it(build, state, tmp_path):
    path = tmp_path / "calls.so"
    if state != "missing":
        path.write_text("not an extension")
    code = f"""
import warnings
from prototype_sketch_attention_b200 import build
build.calls_path = lambda: {str(path)!r}
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from prototype_sketch_attention_b200 import binding as b
import torch
assert b._calls is None
assert torch.version.cuda is None or any("short calls" in str(w.message) for w in seen)
o = torch.tensor([0, 4])
q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
i = torch.zeros(4, dtype=torch.int32)
cache = b.paged_cache(4, 2, 16, 64, device="cpu")
for call in (lambda: b.cross_attention(q, o, k, k, o), lambda: b.cross_attention_backward(q, o, k, k, o, {{"out": q, "lse": q.float()[:, :, 0].contiguous()}}, q),
             lambda: b.page_tables(i, i, i, i.view(4, 1), 16, 4), lambda: b.paged_append(k, k, torch.zeros(4, dtype=torch.int64), cache),
             lambda: b.paged_attention(q, cache, i.view(4, 1), i)):
    try:
        call()
        raise SystemExit("accepted CPU tensors")
    except b.SketchAttentionError as e:
        assert "CUDA devices only" in str(e), e
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_its_name_says_what_it_was_compiled_against(build, monkeypatch):
    here = build.calls_path()
    assert os.path.exists(here) == (torch.version.cuda is not None)
    monkeypatch.setattr(torch, "__version__", "99.0.0")
    assert build.calls_path() != here and not os.path.exists(build.calls_path())


def test_another_torch_gets_its_own(build, monkeypatch):
    """The build is not content with a newer file that belongs to another torch; without CUDA in torch there
    is nothing to compile against, and the library alone is built."""
    ran = []

    class Done:
        returncode, stdout, stderr = 1, "", "stopped by the test"
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or Done())
    build._build_calls(False)  # current
    assert not ran
    monkeypatch.setattr(torch, "__version__", "99.0.0")
    if torch.version.cuda is not None:
        with pytest.raises(RuntimeError, match="stopped by the test"):
            build._build_calls(False)
        assert ran and any("99.0.0" in x for x in ran[0])
    ran.clear()
    monkeypatch.setattr(torch.version, "cuda", None)
    build._build_calls(True)
    assert not ran


@pytest.mark.gpu
def test_results_without_it_are_the_same(monkeypatch):
    from prototype_sketch_attention_b200 import binding as b
    assert b._calls is not None
    g = torch.Generator(device="cuda").manual_seed(1)

    def draw(*s):
        return torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    Q, K, V = draw(70, 4, 64), draw(300, 2, 64), draw(300, 2, 64)
    q, k = torch.tensor([0, 60, 70], device="cuda"), torch.tensor([0, 40, 300], device="cuda")

    def run():
        f = b.cross_attention(Q, q, K, V, k)
        r = b.cross_attention_backward(Q, q, K, V, k, f, Q)
        torch.cuda.synchronize()
        return [f["out"], f["lse"], f["rest"], r["dQ"], r["dK"], r["dV"]]
    want = run()
    monkeypatch.setattr(b, "_calls", None)
    assert all(torch.equal(x, y) for x, y in zip(run(), want))
