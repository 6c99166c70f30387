"""q/k normalisation with rotation (gdn_qk_norm_rope_fwd, gdn_qk_norm_rope_bwd) against the fp64
form of oracle/qk_rope.py, element by element.  Tolerances are the oracle's fp32 error bounds plus,
for a bf16 result, half a step of its own rounding (2^-8 of the value)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_99_b200 as gdn
from oracle import qk_rope as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TINY = 2.0 ** -126


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, err, name):
    half = torch.finfo(got.dtype).eps / 2
    got = np64(got)
    assert got.shape == want.shape
    tol = err + half * (np.abs(want) + err) + TINY
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, first at %s: %r for %r +- %r" % (
        name, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), got[bad][0], want[bad][0],
        np.broadcast_to(tol, want.shape)[bad][0])


def draw(B, T, Hq, Hk, d, rot, dtype="bf16", weights=True, far=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    v = dict(q=r(B, T, Hq, d), k=r(B, T, Hk, d) * torch.exp(r(B, T, Hk, 1)), dqo=r(B, T, Hq, d),
             dko=r(B, T, Hk, d))
    v = {n: t.to(DT[dtype]) for n, t in v.items()}
    v["inv_freq"] = torch.pow(1e4, -torch.arange(0, rot, 2).double() / max(rot, 1)).float()
    v["positions"] = (torch.randint(-far, far, (B, T), generator=gen).to(torch.int32) if far else None)
    v["q_weight"] = 1 + 0.3 * r(d) if weights else None
    v["k_weight"] = r(d) if weights else None
    return v


def run_and_check(v, norm="rms", eps=None, interleaved=False, on=lambda t: t.cuda()):
    B, T, Hq, d = v["q"].shape
    rot = 2 * v["inv_freq"].numel()
    dev = {n: None if t is None else t.cuda() for n, t in v.items()}
    for n in ("q", "k", "dqo", "dko"):
        dev[n] = on(v[n])
    kw = dict(inv_freq=dev["inv_freq"] if rot else None, positions=dev["positions"], norm=norm,
              q_weight=dev["q_weight"], k_weight=dev["k_weight"], eps=eps, interleaved=interleaved)
    out = gdn.gdn_qk_norm_rope_fwd(dev["q"], dev["k"], **kw)
    grads = gdn.gdn_qk_norm_rope_bwd(dev["q"], dev["k"], dev["dqo"], dev["dko"], **kw)
    pos = (np.arange(T, dtype=np.float64)[None].repeat(B, 0) if v["positions"] is None else
           np64(v["positions"]))
    e = float(np.float32({"rms": 1e-6, "l2": 0.0, None: 0.0}[norm] if eps is None else eps))
    for i, (x, dy, w) in enumerate((("q", "dqo", "q_weight"), ("k", "dko", "k_weight"))):
        wt = np.ones(d) if v[w] is None else np64(v[w])
        args = (pos, np64(v["inv_freq"]), norm, wt, e, interleaved)
        close(out[i], *ref.fwd(np64(v[x]), *args), x + "o")
        (dx, dw), (edx, edw) = ref.bwd(np64(v[x]), np64(v[dy]), *args)
        close(grads[i], dx, edx, "d" + x)
        if v[w] is None:
            assert grads[2 + i] is None
        else:
            close(grads[2 + i], dw, edw, "d" + w)
    return out + grads


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (256, 256), (2, 2), (10, 6), (80, 80),
                                   (96, 48), (192, 20), (66, 34), (16, 0), (250, 250), (80, 40), (12, 8),
                                   (100, 36), (256, 2), (256, 40)])
def test_row_sizes(d, rot, interleaved, norm, dtype):
    v = draw(2, 5, 3, 2, d, rot, dtype, weights=norm != "l2", seed=d + rot)
    run_and_check(v, norm, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (1, 1, 16, 16), (7, 1, 16, 4), (3, 33, 5, 1),
                                       (2, 150, 4, 6), (1, 2100, 2, 1), (1, 3, 70, 33)])
def test_token_and_head_counts(B, T, Hq, Hk, dtype):
    run_and_check(draw(B, T, Hq, Hk, 128, 128, dtype, seed=T + Hq))
    run_and_check(draw(B, T, Hq, Hk, 64, 32, dtype, seed=T + Hq, far=5000), "l2", interleaved=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hk,d,rot,interleaved", [(8, 2, 64, 64, False), (3, 1, 64, 32, True), (5, 3, 32, 8, True),
                                                     (1, 1, 16, 0, False), (2, 1, 128, 48, False), (1, 1, 24, 24, True),
                                                     (2, 1, 256, 256, False), (1, 7, 8, 8, True)])
def test_few_heads_of_many_tokens(Hq, Hk, d, rot, interleaved, dtype):
    """A warp takes several tokens at once, fewer at the end; in column slices of one projection too."""
    v = draw(3, 2501, Hq, Hk, d, rot, dtype, seed=d + rot, far=100000)
    want = run_and_check(v, interleaved=interleaved)
    v["positions"] = None
    run_and_check(v, "l2", interleaved=interleaved)
    v["positions"] = draw(3, 2501, Hq, Hk, d, rot, dtype, seed=d + rot, far=100000)["positions"]

    def sliced(t):
        wide = torch.full(t.shape[:2] + (t.shape[2] + 2, d), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :, 1:-1] = t.cuda()
        return wide[:, :, 1:-1]
    for one, two in zip(want, run_and_check(v, interleaved=interleaved, on=sliced)):
        assert torch.equal(one, two)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_far_and_negative_positions(dtype):
    v = draw(2, 40, 2, 2, 128, 128, dtype, far=1 << 20)
    v["positions"][0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1 << 24])
    for interleaved in (False, True):
        run_and_check(v, interleaved=interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 32), (64, 24), (10, 6), (128, 0), (80, 72)])
def test_non_finite_values_that_are_not_turned_stay_where_they_are(d, rot, interleaved, dtype):
    """Without a norm a value behind the rotated ones touches no other, and no gradient but its weight's."""
    v = draw(2, 6, 3, 2, d, rot, dtype, seed=d + rot)
    dev = {n: None if t is None else t.cuda() for n, t in v.items()}
    kw = dict(inv_freq=dev["inv_freq"] if rot else None, norm=None, q_weight=dev["q_weight"],
              k_weight=dev["k_weight"], interleaved=interleaved)
    fwd = lambda: gdn.gdn_qk_norm_rope_fwd(dev["q"], dev["k"], **kw)
    bwd = lambda: gdn.gdn_qk_norm_rope_bwd(dev["q"], dev["k"], dev["dqo"], dev["dko"], **kw)
    q, k = fwd()
    grads = bwd()
    hit = torch.zeros(v["q"].shape, dtype=torch.bool, device="cuda")
    for i, bad in enumerate((float("inf"), -float("inf"), float("nan"))):
        for at in range(rot + i, d, 3):
            dev["q"][i % 2, i, (at + i) % 3, at] = bad
            hit[i % 2, i, (at + i) % 3, at] = True
    q2, k2 = fwd()
    assert torch.equal(q2[~hit], q[~hit]) and not torch.isfinite(q2[hit]).any() and torch.equal(k2, k)
    dq, dk, dqw, dkw = bwd()
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1]) and torch.equal(dkw, grads[3])
    assert torch.equal(dqw[:rot], grads[2][:rot])


def test_one_weight_only_and_given_eps():
    v = draw(2, 9, 3, 2, 64, 64, "fp32")
    v["q_weight"] = None
    run_and_check(v, "rms", eps=0.25)
    run_and_check(v, "l2", eps=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zero_rows_and_rows_of_far_magnitudes(dtype):
    v = draw(1, 12, 2, 2, 64, 64, dtype, weights=False)
    v["q"][0, 3, 1] = 0
    v["k"][0, 5] = 0
    v["q"][0, 6] *= 1e15
    v["k"][0, 7] *= 1e-15
    for norm in ("l2", "rms"):
        qo, ko, dq, dk = run_and_check(v, norm)[:4]
        assert (qo[0, 3, 1] == 0).all() and (ko[0, 5] == 0).all()
        if norm == "l2":
            assert (dq[0, 3, 1] == 0).all() and (dk[0, 5] == 0).all()


def test_non_finite_values_stay_in_their_row():
    v = draw(1, 9, 2, 2, 64, 64)
    want = run_and_check(v)
    v["q"][0, 2, 1, 7] = float("nan")
    v["k"][0, 4, 0, 3] = float("inf")
    v["dqo"][0, 5, 0, 9] = float("nan")
    d = {n: None if t is None else t.cuda() for n, t in v.items()}
    kw = {n: d[n] for n in ("inv_freq", "q_weight", "k_weight")}
    got = gdn.gdn_qk_norm_rope_fwd(d["q"], d["k"], **kw)
    got += gdn.gdn_qk_norm_rope_bwd(d["q"], d["k"], d["dqo"], d["dko"], **kw)[:2]
    rows = [(0, 2, 1)], [(0, 4, 0)], [(0, 2, 1), (0, 5, 0)], [(0, 4, 0)]
    for a, b, bad in zip(got, want, rows):
        same = (a == b).all(-1).cpu()
        for i in bad:
            assert not same[i]
            same[i] = True
        assert same.all()


@pytest.mark.parametrize("d,pad", [(128, 8), (64, 24), (66, 16), (66, 17)])
def test_column_slices_of_one_projection(d, pad):
    """Rows inside wider ones, with values beside them that must not be read, and outputs into
    slices whose neighbours must not be written."""
    def inside(t):
        B, T, H, _ = t.shape
        wide = torch.full((B, T, H * d + pad), float("nan"), dtype=t.dtype, device="cuda")
        part = wide[..., 8:8 + H * d].unflatten(-1, (H, d))
        part.copy_(t)
        return part

    v = draw(2, 21, 3, 2, d, d)
    want = run_and_check(v)
    got = run_and_check(v, on=inside)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dev = {n: None if t is None else t.cuda() for n, t in v.items()}
    kw = {n: dev[n] for n in ("inv_freq", "q_weight", "k_weight")}
    wide = [torch.full((2, 21, H * d + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            for H in (3, 2, 3, 2)]
    parts = [w[..., 8:8 + H * d].unflatten(-1, (H, d)) for w, H in zip(wide, (3, 2, 3, 2))]
    gdn.gdn_qk_norm_rope_fwd(dev["q"], dev["k"], qo=parts[0], ko=parts[1], **kw)
    gdn.gdn_qk_norm_rope_bwd(dev["q"], dev["k"], dev["dqo"], dev["dko"],
                             grads=(parts[2], parts[3], None, None), **kw)
    for w, p, t in zip(wide, parts, want):
        assert torch.equal(p, t)
        n = p.shape[2] * d
        assert (w[..., :8] == 7).all() and (w[..., 8 + n:] == 7).all()


def test_one_token_slices_of_a_batch_of_rows():
    v = draw(5, 3, 2, 1, 64, 64)
    q, k, f = v["q"].cuda(), v["k"].cuda(), v["inv_freq"].cuda()
    pos = torch.tensor([[7], [0], [1 << 20], [3], [9]], dtype=torch.int32, device="cuda")
    for t in range(3):
        got = gdn.gdn_qk_norm_rope_fwd(q[:, t:t + 1], k[:, t:t + 1], f, pos)
        want = gdn.gdn_qk_norm_rope_fwd(q[:, t:t + 1].contiguous(), k[:, t:t + 1].contiguous(), f, pos)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradients_against_differences():
    v = draw(1, 3, 2, 1, 6, 4, "fp32", far=50)
    got = run_and_check(v)
    pos, f = np64(v["positions"]), np64(v["inv_freq"])
    for i, (x, dy, w) in enumerate((("q", "dqo", "q_weight"), ("k", "dko", "k_weight"))):
        base = [np64(v[x]), np64(v[w])]
        eps = float(np.float32(1e-6))
        loss = lambda a, b: (np64(v[dy]) * ref.fwd(a, pos, f, "rms", b, eps, False)[0]).sum()
        for j, grad in enumerate((got[2 + i], got[4 + i])):
            for at in np.ndindex(base[j].shape):
                hi, lo = base[j].copy(), base[j].copy()
                hi[at] += 1e-5
                lo[at] -= 1e-5
                diff = (loss(*[hi if k == j else b for k, b in enumerate(base)]) -
                        loss(*[lo if k == j else b for k, b in enumerate(base)])) / 2e-5
                assert abs(np64(grad)[at] - diff) <= 1e-5 * (1 + abs(diff))


def test_l2_equals_the_layers_own_normalisation():
    """Without rotation and with norm "l2" the rows are those that gdn_fwd's qk_l2norm option forms
    (fp32 inputs: the same layer output to rounding)."""
    v = draw(1, 70, 2, 2, 64, 0, "fp32", weights=False)
    q, k = v["q"].cuda(), v["k"].cuda()
    x = torch.randn(1, 70, 2, 64, device="cuda")
    g, beta = -torch.rand(1, 70, 2, device="cuda"), torch.rand(1, 70, 2, device="cuda")
    o1, h1 = gdn.gdn_fwd(q, k, x, g, beta, qk_l2norm=True)
    qn, kn = gdn.gdn_qk_norm_rope_fwd(q, k, norm="l2")
    o2, h2 = gdn.gdn_fwd(qn, kn, x, g, beta)
    for a, b in ((o1, o2), (h1, h2)):
        assert (a - b).abs().max() <= 1e-5 * a.abs().max()


def test_same_results_every_time_on_another_stream_and_replayed():
    v = draw(2, 300, 4, 2, 128, 128, far=9999)
    want = run_and_check(v)
    d = {n: t.cuda() for n, t in v.items()}
    kw = {n: d[n] for n in ("inv_freq", "positions", "q_weight", "k_weight")}
    call = lambda **more: (gdn.gdn_qk_norm_rope_fwd(d["q"], d["k"], **kw, **more) +
                           gdn.gdn_qk_norm_rope_bwd(d["q"], d["k"], d["dqo"], d["dko"], **kw, **more))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = call(stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn on values that change
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out))
    v2 = draw(2, 300, 4, 2, 128, 128, far=9999, seed=8)
    want2 = run_and_check(v2)
    for values, expected in ((v2, want2), (v, want)):
        for n in d:
            d[n].copy_(values[n])
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, expected):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 values of q: the last tokens of a long row of many heads."""
    T, H, d = 65536 + 3, 256, 128
    q = torch.zeros(1, T, H, d, dtype=torch.bfloat16, device="cuda")
    q[0, -1] = 1
    q[0, 7, 3] = 2
    k = q[:, :, :1].contiguous()
    qo, ko = gdn.gdn_qk_norm_rope_fwd(q, k, norm="l2")
    one = torch.full((d,), d ** -0.5, dtype=torch.bfloat16, device="cuda")
    assert (qo[0, -1] == one).all() and (qo[0, 7, 3] == one).all() and (qo[0, -2] == 0).all()
    assert (ko[0, -1] == one).all()
    del qo
    dq, dk, _, _ = gdn.gdn_qk_norm_rope_bwd(q, k, q, k, norm="l2")
    # the gradient along the row itself is 0 up to the rounding of <u, x r> (x's own scale: 1)
    assert dq.abs().max() <= 2.0 ** -18 and dk.abs().max() <= 2.0 ** -18


def test_empty_rows():
    q = torch.zeros(1, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    qo, ko = gdn.gdn_qk_norm_rope_fwd(q, q, q_weight=w)
    dq, dk, dqw, dkw = gdn.gdn_qk_norm_rope_bwd(q, q, q, q, q_weight=w)
    assert qo.shape == dq.shape == q.shape and (dqw == 0).all() and dkw is None


def test_planted_launch_failure_is_reported():
    v = draw(1, 3, 2, 2, 64, 64)
    q, k = v["q"].cuda(), v["k"].cuda()
    gdn.set_test_hook(gdn.GDN_TEST_FAIL_LAUNCH)
    try:
        for call in (lambda: gdn.gdn_qk_norm_rope_fwd(q, k),
                     lambda: gdn.gdn_qk_norm_rope_bwd(q, k, q, k)):
            with pytest.raises(gdn.GdnError) as e:
                call()
            assert e.value.code == 5
    finally:
        gdn.set_test_hook(0)
    run_and_check(v)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_rows_whose_sum_of_squares_passes_fp32(norm, dtype):
    """Rows of 1e18 are right (64 squares sum to 6e37); rows of 1e20, whose sum is infinite, have r = 0:
    zeros, and zero gradients, and their neighbours are as ever."""
    v = draw(1, 12, 2, 2, 64, 64, dtype, weights=norm == "rms")
    v["q"][0, 6] *= 1e18 / 4
    want = run_and_check(v, norm)
    far = {n: None if t is None else t.clone() for n, t in v.items()}
    far["q"][0, 3, 1] = 1e20
    far["k"][0, 5, 0] = -1e20
    dev = {n: None if t is None else t.cuda() for n, t in far.items()}
    kw = dict(norm=norm, **{n: dev[n] for n in ("inv_freq", "q_weight", "k_weight")})
    got = gdn.gdn_qk_norm_rope_fwd(dev["q"], dev["k"], **kw)
    got += gdn.gdn_qk_norm_rope_bwd(dev["q"], dev["k"], dev["dqo"], dev["dko"], **kw)[:2]
    for a, b, row in zip(got, want, ((0, 3, 1), (0, 5, 0)) * 2):
        assert (a[row] == 0).all()
        a[row] = b[row]
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,T", [(3, 3200), (1, 9601)])
@pytest.mark.parametrize("Hq,Hk,d,rot,dtype,interleaved,grouped", [
    (4, 4, 64, 64, "bf16", False, "both"), (2, 1, 128, 128, "bf16", False, "both"),
    (1, 1, 64, 64, "bf16", True, "both"), (3, 2, 32, 32, "bf16", False, "both"),
    (2, 2, 64, 64, "fp32", False, "both"), (1, 2, 64, 64, "fp32", True, "both"),
    (4, 2, 64, 32, "bf16", False, "both"), (2, 1, 64, 24, "fp32", True, "both"),
    (1, 1, 24, 24, "bf16", False, "both"), (8, 2, 64, 64, "bf16", False, "bwd"),
    (8, 1, 64, 32, "fp32", True, "bwd"), (16, 16, 128, 128, "bf16", False, "none")])
def test_several_tokens_per_warp_are_taken_and_right(Hq, Hk, d, rot, dtype, interleaved, grouped, B, T):
    """The kernels that take several tokens of few heads per warp: with tokens for every warp's lanes (9600, by
    which rows need no mask where heads and tokens fill the lanes) and with fewer in the last warp (9601)."""
    v = draw(B, T, Hq, Hk, d, rot, dtype, seed=d + rot + Hq)
    with gdn.LaunchTrace(16) as trace:
        run_and_check(v, interleaved=interleaved)
    torch.cuda.synchronize()
    names = {"qk_norm_rope" + ("_group" if grouped == "both" else ""),
             "qk_norm_rope_bwd" + ("" if grouped == "none" else "_group"), "qk_norm_rope_dw"}
    assert set(trace.per_kernel()) == names


WEIGHTS = [(4, 4, 64, 64, "bf16", 9600), (4, 4, 64, 64, "bf16", 9601), (2, 1, 128, 128, "bf16", 9600),
           (8, 2, 64, 64, "bf16", 9603), (8, 1, 64, 32, "fp32", 9601), (1, 1, 64, 64, "bf16", 9599),
           (16, 16, 128, 128, "bf16", 3001), (3, 5, 256, 256, "fp32", 1200), (3, 3, 66, 34, "bf16", 2001),
           (2, 2, 250, 250, "fp32", 700), (40, 3, 80, 0, "bf16", 5)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,rot,dtype,T", WEIGHTS)
def test_weight_gradients_have_every_row_once(Hq, Hk, d, rot, dtype, T, interleaved):
    """Without a norm and turned by no angle dw = sum of dy x: with whole numbers from 1 to 3 of either sign it is
    exact in fp32 (below 9 x 9603 x 16 < 2^24 in any order), and every row left out or taken twice shows."""
    gen = torch.Generator().manual_seed(T + d)

    def whole(H):
        n = torch.randint(1, 4, (1, T, H, d), generator=gen)
        return torch.where(torch.rand(n.shape, generator=gen) < 0.5, n, -n)

    q, k, dq, dk = whole(Hq), whole(Hk), whole(Hq), whole(Hk)
    on = lambda t: t.to(DT[dtype]).cuda()
    w = torch.ones(d, device="cuda")
    f = torch.zeros(rot // 2, device="cuda") if rot else None
    got = gdn.gdn_qk_norm_rope_bwd(on(q), on(k), on(dq), on(dk), f, norm=None, q_weight=w, k_weight=w,
                                   interleaved=interleaved)
    assert torch.equal(got[0], on(dq)) and torch.equal(got[1], on(dk))
    for dw, x, dy in ((got[2], q, dq), (got[3], k, dk)):
        assert torch.equal(dw.cpu().long(), (x * dy).sum((0, 1, 2)))


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("H,d,rot,dtype,side,T", [(4, 64, 64, "bf16", 8, 9600), (4, 64, 64, "fp32", 4, 9601),
                                                  (16, 128, 128, "bf16", 4, 3001), (2, 250, 100, "fp32", 1, 700)])
def test_weight_gradients_of_normalised_rows(H, d, rot, dtype, side, T, norm):
    """dw = sum of u x r within the rounding of the sums that are made: a lane adds its rows (the 148 blocks of
    each tensor have 8 warps, each of which takes the H heads of ceil(T / 1184) tokens at most, `side` of them in
    lanes beside each other), then come 5 joins of lanes, 8 of warps, 5 of blocks and 32 of their sums."""
    v = draw(1, T, H, H, d, rot, dtype, seed=T)
    dev = {n: None if t is None else t.cuda() for n, t in v.items()}
    kw = dict(norm=norm, **{n: dev[n] for n in ("inv_freq", "q_weight", "k_weight")})
    got = gdn.gdn_qk_norm_rope_bwd(dev["q"], dev["k"], dev["dqo"], dev["dko"], **kw)
    depth = -(-T // 1184) * -(-H // side) + 5 + 8 + 5 + 32
    angle = np.arange(T, dtype=np.float64)[None, :, None, None] * np64(v["inv_freq"])
    eps = float(np.float32(1e-6)) if norm == "rms" else 0.0
    for x, dy, dw in ((v["q"], v["dqo"], got[2]), (v["k"], v["dko"], got[3])):
        x, c = np64(x), 1 / d if norm == "rms" else 1.0
        xn = x / np.sqrt(c * (x * x).sum(-1, keepdims=True) + eps)
        u, m = ref.turn(np64(dy), angle, False, back=True)
        err = (np.abs(xn) * ref.U * (ref.TRIG + 2) * m + ref.U * (ref.NORM + 2 + depth) * np.abs(u * xn)).sum((0, 1, 2))
        want = (u * xn).sum((0, 1, 2))
        assert err.max() < np.abs(u * xn).mean()  # one row of all that is left out or taken twice shows
        close(dw, want, err, "dw")
