"""The cross attention with many items a block (8 a multiprocessor and more, and just below that), one very
long user among short ones with them, against the 64-bit reference: several key tiles and head
groups, masks, the output's rest, users without queries or keys."""
import pytest
import torch

import attn_reference as ref
from test_gpu_cross import NAMES, _inputs, _offsets, _run

pytestmark = pytest.mark.gpu


def _items(lq, H, Hkv):
    G = H // Hkv
    pg = min(G & -G, 128)
    return sum(-(-n // (256 // pg)) for n in lq) * (H // pg)


def _lengths(n, q, k):
    lq = [1 + (17 * i) % q for i in range(n)]
    lk = [(131 * i) % k for i in range(n)]
    return lq, lk


CASES = [
    # users, most queries, most keys, H, Hkv, longest: with a user of that many keys among the others
    (170, 40, 700, 8, 8, 0),
    (130, 60, 300, 12, 4, 0),
    (160, 300, 400, 16, 4, 0),
    (320, 5, 513, 4, 4, 20000),
    (110, 40, 700, 8, 8, 0),  # below
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("users,q,k,H,Hkv,longest", CASES)
def test_against_reference(users, q, k, H, Hkv, longest, masked, d):
    lq, lk = _lengths(users, q, k)
    lq[3], lk[users // 2] = 0, longest or lk[users // 2]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (_items(lq, H, Hkv) >= 8 * sms) == (users != 110)
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=1000 + users)
    qo, ko = _offsets(lq), _offsets(lk)
    mask = None
    if masked:
        mask = torch.rand(ko[-1], generator=torch.Generator(device="cuda").manual_seed(9), device="cuda") < 0.7
        mask[ko[7]:ko[7] + 128] = False
    got = _run(Q, qo, K, V, ko, dout, mask)
    got["wide"] = got["out"].double() + got["rest"].double()
    ref.check(got, ref.cross(Q, qo, K, V, ko, mask, dout=dout, rest=True), (*NAMES, "wide"))
