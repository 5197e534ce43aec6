"""GPU multi-head cross attention, forward and gradients, against the 64-bit reference at
element-wise bounds (attn_reference.py): lengths from zero and one to several tiles, shared
heads, masks that leave rows empty, NaN where nothing may be read, strided rows, rows behind
the last user, streams and graphs."""
import math

import pytest
import torch

import attn_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _offsets(lens):
    o = [0]
    for n in lens:
        o.append(o[-1] + n)
    return o


def _inputs(lq, lk, H, Hkv, d, seed, fused=False, amp=1.0, behind=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    nq, nk = sum(lq) + behind, sum(lk) + behind
    Q = (amp * torch.randn(nq, H, d, generator=g, device="cuda")).to(BF)
    KV = torch.randn(nk, 2, Hkv, d, generator=g, device="cuda").to(BF)
    K, V = (KV[:, 0], KV[:, 1]) if fused else (KV[:, 0].contiguous(), KV[:, 1].contiguous())
    dout = torch.randn(nq, H, d, generator=g, device="cuda").to(BF)
    return Q, K, V, dout


def _dev(o):
    return torch.tensor(o, dtype=torch.int64, device="cuda")


def _run(Q, qo, K, V, ko, dout, mask=None, scale=None):
    from prototype_sketch_attention_b200 import binding as b
    f = b.cross_attention(Q, _dev(qo), K, V, _dev(ko), key_mask=mask, scale=scale)
    g = b.cross_attention_backward(Q, _dev(qo), K, V, _dev(ko), f, dout, key_mask=mask, scale=scale)
    torch.cuda.synchronize()
    assert b.device_status(f["_ws"]) == 0 and b.device_status(g["_ws"]) == 0
    return {**f, **g}


NAMES = ("out", "lse", "dQ", "dK", "dV")

CASES = [
    # lq, lk, H, Hkv, d
    ([1], [1], 1, 1, 64),
    ([1], [1], 3, 1, 128),
    ([0, 5, 130, 1], [7, 0, 3, 129], 4, 2, 128),
    ([128], [128], 2, 2, 64),
    ([129, 1, 64], [257, 128, 65], 6, 2, 128),
    ([300, 17], [1000, 260], 8, 8, 64),
    ([33, 5], [500, 1200], 16, 1, 128),
    ([2, 3, 1, 4], [1500, 7, 64, 900], 12, 4, 64),
    ([257], [383], 5, 5, 128),
    ([1, 1, 1], [4000, 1, 2047], 32, 2, 128),
    ([700], [130], 24, 8, 64),
]


@pytest.mark.parametrize("lq,lk,H,Hkv,d", CASES)
@pytest.mark.parametrize("masked", [False, True])
def test_against_reference(lq, lk, H, Hkv, d, masked):
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=sum(lq) + 7 * H)
    qo, ko = _offsets(lq), _offsets(lk)
    mask = None
    if masked:
        g = torch.Generator(device="cuda").manual_seed(5)
        mask = torch.rand(ko[-1], generator=g, device="cuda") < 0.6
        mask[ko[-2]:ko[-2] + 130] = False  # a whole first tile of the last user (or all of it)
    got = _run(Q, qo, K, V, ko, dout, mask)
    ref.check(got, ref.cross(Q, qo, K, V, ko, mask, dout=dout), NAMES)


@pytest.mark.parametrize("lq,lk,H,Hkv,d,fused", [([5, 40], [1, 3], 4, 4, 64, True), ([70, 200], [200, 70], 4, 2, 128, True),
                                                 ([3, 9], [300, 5], 8, 1, 128, False)])
def test_strided_rows(lq, lk, H, Hkv, d, fused):
    """Keys and values as halves of one projection, queries inside wider rows."""
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=11, fused=fused)
    wide = torch.full((Q.shape[0], H + 3, d), float("nan"), dtype=BF, device="cuda")
    wide[:, 1:H + 1] = Q
    qo, ko = _offsets(lq), _offsets(lk)
    got = _run(wide[:, 1:H + 1], qo, K, V, ko, dout)
    ref.check(got, ref.cross(Q, qo, K, V, ko, dout=dout), NAMES)


@pytest.mark.parametrize("d", [64, 128])
def test_dropped_rows_are_never_used(d):
    """NaN and infinities in dropped key rows, in other users' rows and behind the last one do
    not reach any output; gradients of dropped rows are 0; rows behind stay as they were."""
    from prototype_sketch_attention_b200 import binding as b
    lq, lk, H, Hkv = [3, 70, 2], [150, 40, 9], 4, 2
    qo, ko = _offsets(lq), _offsets(lk)
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=21, behind=5)
    mask = torch.ones(ko[-1] + 5, dtype=torch.bool, device="cuda")
    drop = torch.tensor([0, 1, 77, 128, 149, 151], device="cuda")
    mask[drop] = False
    mask[ko[2]:ko[3]] = False  # the last user keeps nothing
    clean = ref.cross(Q, qo, K, V, ko, mask, dout=dout)
    bad = torch.tensor([math.nan, math.inf, -math.inf, 3.3895e38, -3.3895e38], device="cuda").to(BF)
    for x, rows in ((K, [*drop.tolist(), *range(ko[2], ko[3] + 5)]), (V, [*drop.tolist(), *range(ko[2], ko[3] + 5)]),
                    (Q, range(qo[-1], qo[-1] + 5)), (dout, range(qo[-1], qo[-1] + 5))):
        for i, r in enumerate(rows):
            x[r] = bad[i % 5]
    out = {"out": torch.full_like(dout, 7.0), "lse": torch.full(dout.shape[:2], 7.0, device="cuda")}
    f = b.cross_attention(Q, _dev(qo), K, V, _dev(ko), key_mask=mask, out=out)
    grads = {"dQ": torch.full_like(Q, 7.0), "dK": torch.full_like(K, 7.0), "dV": torch.full_like(V, 7.0)}
    g = b.cross_attention_backward(Q, _dev(qo), K, V, _dev(ko), f, dout, key_mask=mask, out=grads)
    got = {**f, **g}
    ref.check(got, clean, NAMES)
    for n, x in got.items():
        if n != "_ws":
            end = qo[-1] if n in ("out", "lse", "dQ") else ko[-1]
            assert (x[end:] == 7.0).all(), n
    assert (got["dK"][drop] == 0).all() and (got["dV"][drop] == 0).all()
    assert (got["lse"][qo[2]:qo[3]] == -math.inf).all() and (got["out"][qo[2]:qo[3]] == 0).all()


@pytest.mark.parametrize("amp", [12.0, 60.0])
def test_sharp_rows(amp):
    """Scores far apart, growing along the keys so that the running maximum is raised often."""
    lq, lk = [40, 3], [900, 300]
    Q, K, V, dout = _inputs(lq, lk, 4, 2, 128, seed=31, amp=amp)
    K *= torch.linspace(0.05, 1.0, sum(lk), device="cuda")[:, None, None].to(BF)
    got = _run(Q, _offsets(lq), K, V, _offsets(lk), dout)
    ref.check(got, ref.cross(Q, _offsets(lq), K, V, _offsets(lk), dout=dout), NAMES)


def test_scale_argument_and_keys_of_the_lowest_value():
    lq, lk = [9, 20], [200, 31]
    Q, K, V, dout = _inputs(lq, lk, 2, 2, 64, seed=41)
    qo, ko = _offsets(lq), _offsets(lk)
    got = _run(Q, qo, K, V, ko, dout, scale=0.5)
    ref.check(got, ref.cross(Q, qo, K, V, ko, scale=0.5, dout=dout), NAMES)


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit forward against the kernels' gradients."""
    lq, lk = [20, 3], [150, 40]
    Q, K, V, dout = _inputs(lq, lk, 4, 2, 64, seed=51)
    qo, ko = _offsets(lq), _offsets(lk)
    got = _run(Q, qo, K, V, ko, dout)
    r = ref.cross(Q, qo, K, V, ko, dout=dout)
    g = torch.Generator(device="cuda").manual_seed(52)
    base = [x.double() for x in (Q, K, V)]
    for i, name in enumerate(("dQ", "dK", "dV")):
        u = torch.randn(base[i].shape, generator=g, dtype=torch.float64, device="cuda")
        val = []
        for e in (1e-4, -1e-4):
            x = [*base]
            x[i] = x[i] + e * u
            val.append(float((ref.cross(*[x[0], qo, x[1], x[2], ko])["out"][0] * dout.double()).sum()))
        diff = (val[0] - val[1]) / 2e-4
        slack = float((r[name][1] * u.abs()).sum()) + 1e-5 * abs(diff)  # bounds, and the difference's own 1e-8 term
        assert abs(diff - float((got[name].double() * u).sum())) <= slack, name


def test_long_keys_few_queries_and_many_users():
    for lq, lk, H, Hkv, d in (([1], [30000], 8, 2, 128), ([1] * 500, [3] * 500, 2, 1, 64),
                              ([2] * 1500, [(7 * i) % 5 for i in range(1500)], 1, 1, 64)):
        Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=61)
        qo, ko = _offsets(lq), _offsets(lk)
        ref.check(_run(Q, qo, K, V, ko, dout), ref.cross(Q, qo, K, V, ko, dout=dout), NAMES)


def test_no_rows_at_all():
    for lq, lk in (([0], [0]), ([4, 2], [0, 0]), ([0, 0], [3, 140]), ([], [])):
        Q, K, V, dout = _inputs(lq, lk, 4, 2, 64, seed=71)
        got = _run(Q, _offsets(lq), K, V, _offsets(lk), dout)
        ref.check(got, ref.cross(Q, _offsets(lq), K, V, _offsets(lk), dout=dout), NAMES)


def test_bad_offsets_are_latched():
    from prototype_sketch_attention_b200 import binding as b
    Q, K, V, dout = _inputs([6], [9], 2, 1, 64, seed=81)
    good_q, good_k = _dev([0, 2, 6]), _dev([0, 4, 9])
    for qo, ko in (([0, 7, 6], [0, 4, 9]), ([1, 2, 6], [0, 4, 9]), ([0, 2, 6], [0, 10, 9]), ([0, 2, 7], [0, 4, 9]),
                   ([0, 2, 6], [0, 4, 10]), ([0, -1, 6], [0, 4, 9])):
        f = b.cross_attention(Q, _dev(qo), K, V, _dev(ko))
        assert b.device_status(f["_ws"]) == b.SA_ERR_BAD_OFFSETS, (qo, ko)
        g = b.cross_attention_backward(Q, _dev(qo), K, V, _dev(ko), f, dout)
        assert b.device_status(g["_ws"]) == b.SA_ERR_BAD_OFFSETS
    f = b.cross_attention(Q, good_q, K, V, good_k, ws=f["_ws"])  # the word is cleared by the next call
    assert b.device_status(f["_ws"]) == 0


def test_small_workspace_is_refused():
    from prototype_sketch_attention_b200 import binding as b
    Q, K, V, dout = _inputs([6], [9], 2, 1, 64, seed=82)
    ws = torch.empty(128, dtype=torch.uint8, device="cuda")
    with pytest.raises(b.SketchAttentionError) as e:
        b.cross_attention(Q, _dev([0, 6]), K, V, _dev([0, 9]), ws=ws)
    assert e.value.status == b.SA_ERR_WORKSPACE


def test_deterministic_and_on_two_streams():
    from prototype_sketch_attention_b200 import binding as b
    Q, K, V, dout = _inputs([300, 41], [1300, 2000], 8, 2, 128, seed=91)
    qo, ko = _offsets([300, 41]), _offsets([1300, 2000])
    base = _run(Q, qo, K, V, ko, dout)
    streams, res = [torch.cuda.Stream() for _ in range(2)], []
    qd, kd = _dev(qo), _dev(ko)
    torch.cuda.synchronize()
    for s in streams:  # two calls at once, a workspace each
        f = b.cross_attention(Q, qd, K, V, kd, stream=s)
        res.append({**f, **b.cross_attention_backward(Q, qd, K, V, kd, f, dout, stream=s), "fws": f["_ws"]})
    torch.cuda.synchronize()
    for r in res:
        for n in NAMES:
            assert torch.equal(r[n], base[n]), n


def test_replays_from_a_graph():
    from prototype_sketch_attention_b200 import binding as b
    lq, lk = [40, 0, 129], [700, 30, 1]
    Q, K, V, dout = _inputs(lq, lk, 6, 2, 64, seed=95)
    qd, kd = _dev(_offsets(lq)), _dev(_offsets(lk))
    wf = b.cross_attention(Q, qd, K, V, kd)
    wb = b.cross_attention_backward(Q, qd, K, V, kd, wf, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = b.cross_attention(Q, qd, K, V, kd, ws=wf["_ws"])
        r = b.cross_attention_backward(Q, qd, K, V, kd, f, dout, ws=wb["_ws"])
    Q2, K2, V2, d2 = _inputs([129, 3, 37], [31, 600, 100], 6, 2, 64, seed=96)
    for x, y in ((Q, Q2), (K, K2), (V, V2), (dout, d2)):
        x.copy_(y)
    qd.copy_(_dev(_offsets([129, 3, 37])))  # other lengths in the same buffers
    kd.copy_(_dev(_offsets([31, 600, 100])))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    want = _run(Q2, _offsets([129, 3, 37]), K2, V2, _offsets([31, 600, 100]), d2)
    for n in NAMES:
        assert torch.equal({**f, **r}[n], want[n]), n


@pytest.mark.parametrize("lq,lk,H,Hkv,d", [([40], [300], 4, 2, 64), ([0, 70, 9], [12, 500, 900], 8, 2, 128),
                                           ([3, 200], [2000, 1], 16, 1, 128)])
@pytest.mark.parametrize("masked", [False, True])
def test_rest_of_the_output(lq, lk, H, Hkv, d, masked):
    """out + rest has the digits that rounding took, and the gradients formed with it are held to the
    narrower bound; without it out is the same and the gradients keep theirs."""
    from prototype_sketch_attention_b200 import binding as b
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=301)
    qo, ko = _offsets(lq), _offsets(lk)
    mask = torch.rand(ko[-1], generator=torch.Generator(device="cuda").manual_seed(6), device="cuda") < 0.5 if masked else None
    qd, kd = _dev(qo), _dev(ko)
    got = _run(Q, qo, K, V, ko, dout, mask)
    got["wide"] = got["out"].double() + got["rest"].double()
    assert (got["rest"].double().abs() <= ref.HALF * got["out"].double().abs() + ref.TINY).all()
    ref.check(got, ref.cross(Q, qo, K, V, ko, mask, dout=dout, rest=True), (*NAMES, "wide"))
    f = b.cross_attention(Q, qd, K, V, kd, key_mask=mask, want_rest=False)
    assert f.get("rest") is None and torch.equal(f["out"], got["out"]) and torch.equal(f["lse"], got["lse"])
    g = b.cross_attention_backward(Q, qd, K, V, kd, f, dout, key_mask=mask)
    torch.cuda.synchronize()
    ref.check({**f, **g}, ref.cross(Q, qo, K, V, ko, mask, dout=dout), NAMES)


REPEATED = [
    # lq, lk, H, Hkv, d: persistent blocks take many items each, of every kind, in changing order
    ([700, 1, 0, 130, 400] * 6, [900, 64, 500, 0, 1] * 6, 8, 2, 64),
    ([700, 1, 0, 130, 400] * 6, [900, 64, 500, 0, 1] * 6, 8, 2, 128),
    ([100, 0, 60] * 30, [100, 0, 128, 0, 129, 1] * 15, 12, 12, 64),
    ([100, 0, 60] * 30, [100, 0, 128, 0, 129, 1] * 15, 12, 12, 128),
    ([1024] * 12, [1024] * 12, 8, 8, 64),
    ([300] * 8, [4000] * 8, 8, 8, 128),
]


@pytest.mark.parametrize("lq,lk,H,Hkv,d", REPEATED)
def test_repeated_calls_agree_bit_for_bit(lq, lk, H, Hkv, d):
    """Calls back to back, two inputs in turn, with no wait between them: every result is the first one's."""
    from prototype_sketch_attention_b200 import binding as b
    qo, ko = _dev(_offsets(lq)), _dev(_offsets(lk))
    sets = [_inputs(lq, lk, H, Hkv, d, seed=400 + i) for i in range(2)]
    mask = torch.rand(sum(lk), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda") < 0.9
    runs, first = [], {}
    for n in range(24):
        Q, K, V, dout = sets[n & 1]
        m = mask if n & 2 else None
        f = b.cross_attention(Q, qo, K, V, ko, key_mask=m)
        g = b.cross_attention_backward(Q, qo, K, V, ko, f, dout, key_mask=m)
        base = first.setdefault(n & 3, {**f, **g})
        runs.append((n, torch.stack([(x[name] != base[name]).sum() for x in ({**f, **g},) for name in (*NAMES, "rest")]),
                     f["_ws"], g["_ws"]))
    torch.cuda.synchronize()
    for n, off, fw, gw in runs:
        assert not off.any(), (n, off.tolist())
        assert b.device_status(fw) == 0 and b.device_status(gw) == 0


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (4, 1, 128)])
def test_items_without_steps_between_others(H, Hkv, d):
    """Users with one key tile, no keys or no queries between longer ones."""
    lq = [1, 0, 3, 300, 2, 0, 140, 1, 1] * 20
    lk = [1, 5, 0, 128, 0, 0, 127, 129, 700, 2, 0] * 18
    lq, lk = lq[:180], lk[:180]
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=500)
    qo, ko = _offsets(lq), _offsets(lk)
    ref.check(_run(Q, qo, K, V, ko, dout), ref.cross(Q, qo, K, V, ko, dout=dout, rest=True), NAMES)


def test_history_to_sketch_to_heads_and_back():
    """A training step's chain: histories to sketches, keys and values of heads from the sketch rows,
    cross attention, its gradients, and back into the histories' gradients, against 64-bit autograd
    of the whole. Tolerance on the relative L2 error: 1e-2 of the sketch's backward (its own tests'),
    and one half step of bf16, 2^-8, for each of what is rounded between: the sketch, K or V, the
    weights, dS, dK or dV, out."""
    from prototype_sketch_attention_b200 import binding as b
    g = torch.Generator(device="cuda").manual_seed(700)
    n, lq, k, d, H, Hkv, dh = [700, 64, 1500], [40, 3, 129], 128, 128, 4, 2, 64
    off, qo, ko = _offsets(n), _offsets(lq), _offsets([k] * 3)

    def draw(*shape, amp=1.0):
        return (amp * torch.randn(*shape, generator=g, device="cuda")).to(BF)
    X, P = draw(sum(n), d), draw(k, d)
    Wk, Wv, Ak, Av = (draw(d, m, amp=d ** -0.5) for m in (d, d, Hkv * dh, Hkv * dh))
    Q, dout = draw(sum(lq), H, dh), draw(sum(lq), H, dh)

    fw = b.forward(X, _dev(off), P, Wk, Wv)
    rows = fw["sketch"].reshape(-1, d).to(BF)
    K, V = (rows @ Ak).view(-1, Hkv, dh), (rows @ Av).view(-1, Hkv, dh)
    f = b.cross_attention(Q, _dev(qo), K, V, _dev(ko))
    c = b.cross_attention_backward(Q, _dev(qo), K, V, _dev(ko), f, dout)
    ds = c["dK"].view(-1, Hkv * dh).float() @ Ak.float().T + c["dV"].view(-1, Hkv * dh).float() @ Av.float().T
    gr = b.backward(X, _dev(off), P, Wk, Wv, fw, ds.view(3, k, d).contiguous())
    torch.cuda.synchronize()

    leaves = [x.double().requires_grad_() for x in (X, P, Wk, Wv, Q)]
    Xd, Pd, Wkd, Wvd, Qd = leaves
    total = 0
    for u in range(3):
        x = Xd[off[u]:off[u + 1]]
        a = torch.softmax((x @ Wkd) @ Pd.T * d ** -0.5, 1)
        s = a.T @ (x @ Wvd) / a.sum(0)[:, None]
        kk, vv = ((s @ A.double()).view(k, Hkv, dh).repeat_interleave(H // Hkv, 1) for A in (Ak, Av))
        z = torch.einsum("thd,khd->htk", Qd[qo[u]:qo[u + 1]], kk) * dh ** -0.5
        o = torch.einsum("htk,khd->thd", torch.softmax(z, 2), vv)
        total = total + (o * dout[qo[u]:qo[u + 1]].double()).sum()
    want = torch.autograd.grad(total, leaves)
    for name, w, x in zip(("dX", "dP", "dWk", "dWv", "dQ"), want, (gr["dX"], gr["dP"], gr["dWk"], gr["dWv"], c["dQ"])):
        err = float((x.double() - w).norm() / w.norm())
        assert err <= 1e-2 + 6 * ref.HALF, (name, err)


@pytest.mark.parametrize("lq,lk,d", [([3, 200, 7], [40, 700, 20000], 64), ([300, 1], [513, 9000], 128)])
def test_nan_in_a_kept_row_stays_with_its_user_and_heads(lq, lk, d):
    """A NaN that is attended to is in out and lse of every head that shares its key head, and nowhere else."""
    from prototype_sketch_attention_b200 import binding as b
    H, Hkv = 6, 2
    Q, K, V, dout = _inputs(lq, lk, H, Hkv, d, seed=801)
    qo, ko = _offsets(lq), _offsets(lk)
    clean = b.cross_attention(Q, _dev(qo), K, V, _dev(ko))
    for u, row in [(x, r) for x in range(len(lq)) for r in (0, lk[x] // 2, lk[x] - 1)]:
        bad = K.clone()
        bad[ko[u] + row, 1, 5] = math.nan
        f = b.cross_attention(Q, _dev(qo), bad, V, _dev(ko))
        hit = torch.zeros(Q.shape[:2], dtype=torch.bool, device="cuda")
        hit[qo[u]:qo[u + 1], 3:] = True
        assert f["out"][hit].isnan().all() and f["lse"][hit].isnan().all()
        assert torch.equal(f["out"][~hit], clean["out"][~hit]) and torch.equal(f["lse"][~hit], clean["lse"][~hit])
    assert b.device_status(f["_ws"]) == 0


def test_short_calls_follow_the_current_stream_and_take_parameters():
    """The extension's calls run on the stream that is current; nn.Parameter inputs give the same results."""
    from prototype_sketch_attention_b200 import binding as b
    Q, K, V, dout = _inputs([70, 3], [300, 40], 4, 2, 64, seed=990)
    qo, ko = _dev(_offsets([70, 3])), _dev(_offsets([300, 40]))
    base = _run(Q, [0, 70, 73], K, V, [0, 300, 340], dout)
    s, gate = torch.cuda.Stream(), torch.cuda.Event()
    late = torch.empty_like(K)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):  # K is written on this stream first: another one would read it too early
        torch.cuda._sleep(20_000_000)
        late.copy_(K)
        f = b.cross_attention(Q, qo, late, V, ko)
        g = b.cross_attention_backward(Q, qo, late, V, ko, f, dout)
        gate.record()
    gate.synchronize()
    assert all(torch.equal({**f, **g}[n], base[n]) for n in NAMES)
    P = [torch.nn.Parameter(x) for x in (Q, K, V)]
    f = b.cross_attention(P[0], qo, P[1], P[2], ko)
    g = b.cross_attention_backward(P[0], qo, P[1], P[2], ko, f, dout)
    torch.cuda.synchronize()
    assert all(torch.equal({**f, **g}[n], base[n]) and not {**f, **g}[n].requires_grad for n in NAMES)
