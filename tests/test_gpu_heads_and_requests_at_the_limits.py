"""Heads up to 1,024 (tiles of one token by 128 heads, several head groups to a key head, every head its own
keys), 64 heads to a cached key head, thousands of users and requests of few positions."""
import pytest
import torch

import attn_reference as ref
from test_gpu_cross import NAMES, _inputs, _offsets, _run
from test_gpu_paged import _check, _filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,d", [(128, 1, 64), (256, 1, 128), (1024, 1, 64), (96, 1, 128), (192, 2, 64), (1024, 1024, 64),
                                     (768, 256, 64)])
@pytest.mark.parametrize("masked", [False, True])
def test_cross_attention_of_many_heads(H, Hkv, d, masked):
    lq, lk = [3, 0, 5, 1], [140, 9, 0, 1]
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=H + d)
    qo, ko = _offsets(lq), _offsets(lk)
    mask = None
    if masked:
        mask = torch.rand(ko[-1], generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") < 0.5
    got = _run(Q, qo, K, V, ko, dout, mask)
    ref.check(got, ref.cross(Q, qo, K, V, ko, mask, dout=dout, rest=True), NAMES)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,Hkv,d", [(1024, 16, 64), (1024, 1024, 64), (192, 3, 128)])
def test_paged_attention_of_many_heads(H, Hkv, d, fp8):
    from prototype_sketch_attention_b200 import binding as b
    Q, cache, table, ln = _filled([70, 0, 1], H, Hkv, d, 16, fp8, seed=H)
    got = b.paged_attention(Q, cache, table, ln, window=50)
    assert b.device_status(got["_ws"]) == 0
    _check(Q, cache, table, ln, 16, 50, got)


@pytest.mark.parametrize("fp8", [False, True])
def test_paged_attention_of_many_requests(fp8):
    from prototype_sketch_attention_b200 import binding as b
    lens = [0 if i % 7 == 3 else (i * 29) % 41 for i in range(3001)]
    lens[1700] = 9000
    Q, cache, table, ln = _filled(lens, 1, 1, 64, 8, fp8, seed=5)
    got = b.paged_attention(Q, cache, table, ln)
    assert b.device_status(got["_ws"]) == 0
    _check(Q, cache, table, ln, 8, 0, got)


def test_cross_attention_of_many_users():
    lq = [(i * 5) % 3 for i in range(2500)]
    lk = [(i * 11) % 6 for i in range(2500)]
    Q, K, V, dout = _inputs(lq, lk, 1, 1, 64, seed=77)
    qo, ko = _offsets(lq), _offsets(lk)
    ref.check(_run(Q, qo, K, V, ko, dout), ref.cross(Q, qo, K, V, ko, dout=dout, rest=True), NAMES)
