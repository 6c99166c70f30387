"""Gated linear recurrence (gdn_linrec_fwd, gdn_linrec_bwd, gdn_linrec_decode) against the fp64
token-by-token form of oracle/linrec.py, element by element.  Tolerances are the oracle's fp32 error
bounds plus, for a bf16 result, half a step of its own rounding (2^-8 of the value)."""
import numpy as np
import pytest
import torch

import gated_delta_rule_99_b200 as gdn
from oracle import linrec as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")]
TINY = 2.0 ** -126  # results below the smallest normal fp32 may be flushed


def draw(B, T, D, dtype="bf16", gate="bf16", N=None, seed=0, decay=0.1, state=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    N = B if N is None else N
    x = r(B, T, D).to(DT[dtype])
    g = (-torch.nn.functional.softplus(r(B, T, D)) * decay).to(DT[gate])
    h0 = r(N, D) if state else None
    return dict(x=x, g=g, h0=h0, do=r(B, T, D).to(DT[dtype]), dhT=r(N, D) if state else None)


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, err, name):
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 2.0 ** -24
    got = np64(got).reshape(want.shape)
    tol = err + half * (np.abs(want) + err) + TINY
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d off, first at %s: %r for %r +- %r" % (
        name, bad.sum(), bad.size, tuple(np.argwhere(bad)[0]), got[bad][0], want[bad][0],
        np.broadcast_to(tol, want.shape)[bad][0])


def run_and_check(v, lengths=None, complement=False, bwd=True, on=lambda t: t.cuda(), **kw):
    """fwd (with and without saved states), bwd (the same) and every output against the oracle."""
    B, T, D = v["x"].shape
    cu = None if lengths is None else np.concatenate([[0], np.cumsum(lengths)]).tolist()
    cu_t = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    N = B if cu is None else len(lengths)
    segs = ref.segments(B, T, cu)
    flat = lambda t: np64(t).reshape(B * T, D)
    h0 = np.zeros((N, D)) if v["h0"] is None else np64(v["h0"])
    dhT = np.zeros((N, D)) if v["dhT"] is None else np64(v["dhT"])
    o, hT, _, eo, ehT, _ = ref.fwd(flat(v["x"]), flat(v["g"]), h0, segs, complement)
    d = {k: None if t is None else (on(t) if k in ("x", "g", "do") else t.cuda()) for k, t in v.items()}
    args = dict(cu_seqlens=None if cu is None else cu_t.cuda(), cu_seqlens_host=cu_t, h0=d["h0"],
                complement=complement, **kw)
    go, ghT = gdn.gdn_linrec_fwd(d["x"], d["g"], **args)
    go2, ghT2, states = gdn.gdn_linrec_fwd(d["x"], d["g"], save_states=True, **args)
    close(go, o, eo, "o")
    close(ghT, hT, ehT, "hT")
    assert torch.equal(go, go2) and torch.equal(ghT, ghT2)
    if not bwd:
        return go, ghT
    want, err = ref.bwd(flat(v["x"]), flat(v["g"]), h0, flat(v["do"]), dhT, segs, complement)
    one = gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], dhT=d["dhT"], states=states, **args)
    two = gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], dhT=d["dhT"], **args)
    for name, a, b, w, e in zip(("dx", "dg", "dh0"), one, two, want, err):
        close(a, w, e, name)
        assert torch.equal(a, b), name
    return (go, ghT) + one


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 3, 5), (1, 15, 64), (1, 16, 66), (3, 17, 31),
                                   (1, 127, 64), (2, 128, 72), (2, 129, 130), (1, 1030, 65),
                                   (1, 2500, 128), (5, 40, 256), (70, 2, 33), (300, 1, 8)])
def test_sizes(B, T, D, complement, types):
    run_and_check(draw(B, T, D, *types, seed=B + T + D), complement=complement)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("lengths", [[1], [0, 5, 0, 0, 3, 0], [128, 128], [127, 1, 1, 127, 256, 0],
                                     [1] * 200, [300, 1, 0, 700, 16, 15, 17], [0, 0, 2049]])
def test_packed_documents(lengths, types):
    v = draw(1, sum(lengths), 72, *types, N=len(lengths), seed=len(lengths))
    run_and_check(v, lengths=lengths, complement=len(lengths) % 2 == 1)


def test_many_documents_of_odd_lengths():
    lengths = [int(n) for n in np.random.default_rng(3).integers(0, 60, size=150)]
    run_and_check(draw(1, sum(lengths), 40, N=150, seed=3), lengths=lengths)


def test_thousands_of_documents_of_no_one_or_a_few_tokens():
    """Longer searches for a token's document, in both directions, and long runs of empty ones."""
    rng = np.random.default_rng(8)
    lengths = [int(n) for n in rng.choice([0, 0, 0, 0, 1, 2, 40], size=4000)]
    lengths[100:1500] = [0] * 1400
    run_and_check(draw(1, sum(lengths), 8, N=4000, seed=8), lengths=lengths)


@pytest.mark.parametrize("B,T,D", [(700, 3, 2048), (9001, 1, 770), (1301, 63, 190)])
def test_many_short_rows(B, T, D):
    """More rows than fill a tile go through one stream, and the last stream has fewer."""
    run_and_check(draw(B, T, D, seed=B))


def test_rows_of_no_token():
    x = torch.zeros(3, 0, 40, device="cuda")
    h0, dhT = torch.randn(3, 40, device="cuda"), torch.randn(3, 40, device="cuda")
    assert torch.equal(gdn.gdn_linrec_fwd(x, x, h0=h0)[1], h0)
    assert torch.equal(gdn.gdn_linrec_bwd(x, x, x, dhT=dhT)[2], dhT)
    assert (gdn.gdn_linrec_fwd(x, x)[1] == 0).all()


def test_one_token_slices_of_a_batch_of_rows():
    """x[:, t:t + 1] of (B, T, D): tokens a whole row apart."""
    v = draw(5, 7, 64, seed=14)
    x, g = v["x"].cuda(), v["g"].cuda()
    a, b = v["h0"].cuda(), v["h0"].cuda()
    for t in range(7):
        o = gdn.gdn_linrec_decode(x[:, t:t + 1], g[:, t:t + 1], a)
        want = gdn.gdn_linrec_decode(x[:, t:t + 1].contiguous(), g[:, t:t + 1].contiguous(), b)
        assert torch.equal(o, want) and torch.equal(a, b)
    for got, want in zip(gdn.gdn_linrec_fwd(x[:, 3:4], g[:, 3:4]),
                         gdn.gdn_linrec_fwd(x[:, 3:4].contiguous(), g[:, 3:4].contiguous())):
        assert torch.equal(got, want)


def test_long_memory_keeps_its_precision():
    """Factors around 0.999: an exponential that is low by a fraction of an ulp on average would show
    in a state that sums up thousands of tokens.  Bound: rounding of every step, one ulp each, in
    the same direction for no more than the memory's length: 2^-23 / (1 - 0.999) = 1.2e-4 of the
    sum of magnitudes is certain; unbiased roundings add up like their square root, 4e-6, and ten
    times less than the former is asked for."""
    T = 20000
    gen = torch.Generator().manual_seed(2)
    g = -torch.rand(1, T, 64, generator=gen) * 0.002
    x = torch.ones(1, T, 64)
    o, hT = gdn.gdn_linrec_fwd(x.cuda(), g.cuda())
    want = np.zeros(64)
    for a in np.exp(np64(g)[0]):
        want = a * want + 1
    assert (np.abs(np64(hT)[0] - want) <= 1.2e-5 * want).all()


def test_two_host_threads():
    from concurrent.futures import ThreadPoolExecutor
    v = [draw(2, 300, 72, seed=s) for s in (40, 41)]
    want = [run_and_check(a) for a in v]
    dev = [{k: t.cuda() for k, t in a.items()} for a in v]
    torch.cuda.synchronize()

    def work(i):
        d = dev[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                out = gdn.gdn_linrec_fwd(d["x"], d["g"], h0=d["h0"])
                out += gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], h0=d["h0"], dhT=d["dhT"])
            torch.cuda.current_stream().synchronize()
        return out

    with ThreadPoolExecutor(2) as pool:
        for got, expected in zip(pool.map(work, (0, 1)), want):
            for a, b in zip(got, expected):
                assert torch.equal(a, b)


def test_no_initial_and_final_states():
    v = draw(2, 200, 48, state=False)
    args = {k: t.cuda() for k, t in v.items() if t is not None}
    o, hT = gdn.gdn_linrec_fwd(args["x"], args["g"], output_final_state=False)
    assert hT is None
    dx, dg, dh0 = gdn.gdn_linrec_bwd(args["x"], args["g"], args["do"], want_dh0=False)
    assert dh0 is None
    run_and_check(v)
    for got, want in zip((o, dx, dg), run_and_check(v)[0:1] + run_and_check(v)[2:4]):
        assert torch.equal(got, want)


@pytest.mark.parametrize("D,types", [(64, TYPES[0]), (65, TYPES[0]), (66, TYPES[1]), (65, TYPES[2])])
def test_column_slices_of_a_wider_tensor(D, types):
    """x, g and do inside rows of another width, with values beside them that must not be read, and
    outputs into slices whose neighbours must not be written."""
    def inside(t):
        wide = torch.full(t.shape[:2] + (D + 24,), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., 8:8 + D] = t.cuda()
        return wide[..., 8:8 + D]

    v = draw(2, 150, D, *types, seed=D)
    want = run_and_check(v)
    got = run_and_check(v, on=inside)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    d = {k: t.cuda() for k, t in v.items()}
    wide = [torch.full((2, 150, D + 24), 7.0, dtype=dt, device="cuda")
            for dt in (d["x"].dtype, d["x"].dtype, d["g"].dtype)]
    o, dx, dg = (w[..., 8:8 + D] for w in wide)
    gdn.gdn_linrec_fwd(d["x"], d["g"], h0=d["h0"], o=o)
    gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], h0=d["h0"], dhT=d["dhT"],
                       grads=(dx, dg, torch.empty_like(d["h0"])))
    for w, t in zip(wide, (want[0], want[2], want[3])):
        assert torch.equal(w[..., 8:8 + D], t)
        assert (w[..., :8] == 7).all() and (w[..., 8 + D:] == 7).all()


@pytest.mark.parametrize("types", TYPES)
def test_resets_strong_decays_and_growth(types):
    """-inf gates (resets), gates far below the fp32 range of exp, and growing states."""
    v = draw(1, 300, 40, *types, seed=9)
    v["g"][0, 7::50] = -float("inf")
    v["g"][0, 13::50] = -200.0
    v["g"][0, 100:110] = 0.25
    v["g"][0, 33] = 0.0
    for complement in (False, True):
        run_and_check(v, complement=complement)


def test_non_finite_values_stay_in_their_channel_and_document():
    lengths = [40, 100, 30]
    v = draw(1, 170, 40, N=3, seed=5)
    want = run_and_check(v, lengths=lengths)
    v["x"][0, 60, 3] = float("nan")
    v["x"][0, 20, 5] = float("inf")
    v["do"][0, 90, 7] = float("nan")
    d = {k: t.cuda() for k, t in v.items()}
    cu = torch.tensor([0, 40, 140, 170], dtype=torch.int32)
    kw = dict(cu_seqlens=cu.cuda(), cu_seqlens_host=cu, h0=d["h0"])
    o, hT = gdn.gdn_linrec_fwd(d["x"], d["g"], **kw)
    dx, dg, dh0 = gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], dhT=d["dhT"], **kw)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(lengths))
    touched = {3: 1, 5: 0, 7: 1}
    for got, ref_ in zip((o, dx, dg), (want[0], want[2], want[3])):
        same = (got == ref_)[0].cpu()
        for c in range(40):
            bad = seq == touched[c] if c in touched else torch.zeros(170, dtype=torch.bool)
            assert same[~bad, c].all(), c
    assert o[0, 60:140, 3].isnan().all() and o[0, 20:40, 5].isinf().all()
    assert dx[0, 40:91, 7].isnan().all()
    for got, ref_ in zip((hT, dh0), (want[1], want[4])):
        same = (got == ref_).cpu()
        for c in range(40):
            for n in range(3):
                assert same[n, c] or touched.get(c) == n


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 1, 31), (2, 4, 130), (64, 1, 256), (1, 2, 515)])
def test_decode(B, T, D, types):
    for complement in (False, True):
        v = draw(B, T, D, *types, seed=T + D)
        o, hT, _, eo, ehT, _ = ref.fwd(np64(v["x"]).reshape(-1, D), np64(v["g"]).reshape(-1, D),
                                       np64(v["h0"]), ref.segments(B, T), complement)
        state = v["h0"].cuda()
        go = gdn.gdn_linrec_decode(v["x"].cuda(), v["g"].cuda(), state, complement=complement)
        close(go, o, eo, "o")
        close(state, hT, ehT, "state")


def test_prefill_then_decode_carries_the_state():
    v = draw(2, 303, 96, "fp32", "fp32", seed=12)
    d = {k: t.cuda() for k, t in v.items()}
    o, hT, _, eo, ehT, _ = ref.fwd(np64(v["x"]).reshape(-1, 96), np64(v["g"]).reshape(-1, 96),
                                   np64(v["h0"]), ref.segments(2, 303))
    o0, h = gdn.gdn_linrec_fwd(d["x"][:, :300].contiguous(), d["g"][:, :300].contiguous(), h0=d["h0"])
    parts = [o0] + [gdn.gdn_linrec_decode(d["x"][:, t:t + 1].contiguous(),
                                          d["g"][:, t:t + 1].contiguous(), h) for t in range(300, 303)]
    close(torch.cat(parts, 1), o.reshape(2, 303, 96), eo.reshape(2, 303, 96), "o")
    close(h, hT, ehT, "state")


def test_gradients_against_differences():
    """Central differences of sum(do * o) + sum(dhT * hT) in fp64 through the oracle's forward agree
    with the kernel's gradients (fp32, so to its error bound and the difference's own h^2)."""
    lengths = [9, 0, 4]
    v = draw(1, 13, 3, "fp32", "fp32", N=3, seed=21, decay=0.7)
    x, g, h0, do, dhT = (np64(v[k]).reshape(-1, 3) for k in ("x", "g", "h0", "do", "dhT"))
    segs = ref.segments(1, 13, [0, 9, 9, 13])
    for complement in (False, True):
        def loss(x, g, h0):
            o, hT = ref.fwd(x, g, h0, segs, complement)[:2]
            return (do * o).sum() + (dhT * hT).sum()

        got = run_and_check(v, lengths=lengths, complement=complement)[2:]
        for i, grad in enumerate(got):
            args = [x, g, h0]
            for at in np.ndindex(args[i].shape):
                hi, lo = args[i].copy(), args[i].copy()
                hi[at] += 1e-5
                lo[at] -= 1e-5
                diff = (loss(*[hi if j == i else a for j, a in enumerate(args)]) -
                        loss(*[lo if j == i else a for j, a in enumerate(args)])) / 2e-5
                assert abs(np64(grad).reshape(args[i].shape)[at] - diff) <= 1e-5 * (1 + abs(diff))


def test_same_results_every_time_and_on_another_stream():
    v = draw(3, 700, 136, seed=30)
    first = run_and_check(v)
    d = {k: t.cuda() for k, t in v.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o, hT, states = gdn.gdn_linrec_fwd(d["x"], d["g"], h0=d["h0"], save_states=True, stream=s)
        grads = gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], h0=d["h0"], dhT=d["dhT"], states=states,
                                   stream=s)
        s.synchronize()
        for a, b in zip((o, hT) + grads, first):
            assert torch.equal(a, b)


def test_captured_calls_replay_on_new_values():
    """A captured forward and backward without host synchronisation, replayed on other inputs and
    other document borders (the mirror is only looked at when the call is made)."""
    lengths = [[100, 50, 150], [10, 0, 290]]
    v = [draw(1, 300, 64, N=3, seed=s) for s in (1, 2)]
    want = [run_and_check(a, lengths=b) for a, b in zip(v, lengths)]
    cu = [torch.tensor([0] + np.cumsum(b).tolist(), dtype=torch.int32) for b in lengths]
    buf = {k: t.cuda() for k, t in v[0].items()}
    cu_dev = cu[0].cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kw = dict(cu_seqlens=cu_dev, cu_seqlens_host=cu[0], h0=buf["h0"])
        out = gdn.gdn_linrec_fwd(buf["x"], buf["g"], **kw)
        out += gdn.gdn_linrec_bwd(buf["x"], buf["g"], buf["do"], dhT=buf["dhT"], **kw)
    for i in (0, 1, 0):
        for k in buf:
            buf[k].copy_(v[i][k])
        cu_dev.copy_(cu[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)


def test_capture_without_the_host_mirror_is_refused():
    v = draw(1, 30, 8, N=2)
    x, g = v["x"].cuda(), v["g"].cuda()
    cu = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda")
    o, hT = gdn.gdn_linrec_fwd(x, g, cu_seqlens=cu)  # without a capture: copied to the host
    desc = gdn.GdnLinrecDesc(1, 30, 8, 2, 0, 0, 0, 0, 0, gdn.GDN_BF16, gdn.GDN_BF16, 0, 0)
    import ctypes
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc = gdn.lib().gdn_linrec_fwd(ctypes.byref(desc), x.data_ptr(), g.data_ptr(), cu.data_ptr(),
                                      None, None, o.data_ptr(), None, None,
                                      torch.cuda.current_stream().cuda_stream)
        o.zero_()
    assert rc == 1


def test_state_offsets_past_32_bits():
    """More than 2^31 elements of x: the last tokens of a wide, long row."""
    D, T = 1 << 16, 32784 + 50
    x = torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda")
    x[0, -1] = 1
    x[0, 5] = 2
    o, hT = gdn.gdn_linrec_fwd(x, g)
    assert (o[0, -1] == 3).all() and (o[0, -2] == 2).all() and (o[0, :5] == 0).all()
    assert (o[0, 5:-1:97] == 2).all() and (hT == 3).all()
    del o
    do = torch.zeros_like(x)
    do[0, -1] = 1
    dx, dg, dh0 = gdn.gdn_linrec_bwd(x, g, do)
    assert (dx[0, ::97] == 1).all() and (dg[0, 6:-1:97] == 2).all() and (dh0 == 1).all()
    assert (dg[0, :6] == 0).all() and (dg[0, -1] == 2).all()


def test_planted_launch_failure_is_reported():
    v = draw(1, 30, 8)
    x, g, st = v["x"].cuda(), v["g"].cuda(), v["h0"].cuda()
    gdn.set_test_hook(gdn.GDN_TEST_FAIL_LAUNCH)
    try:
        for call in (lambda: gdn.gdn_linrec_fwd(x, g), lambda: gdn.gdn_linrec_bwd(x, g, x),
                     lambda: gdn.gdn_linrec_decode(x, g, st)):
            with pytest.raises(gdn.GdnError) as e:
                call()
            assert e.value.code == 5
    finally:
        gdn.set_test_hook(0)
    run_and_check(v)


def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    """The first CTA waits for 16 bytes more than its cluster sends: it gives up after the limit,
    then so do the others, and the kernel ends."""
    v = draw(1, 2000, 64, seed=4)
    d = {k: t.cuda() for k, t in v.items()}
    gdn.set_wait_limit(1 << 12)
    gdn.set_test_hook(gdn.GDN_TEST_STALL_COPY)
    try:
        _, _, states = gdn.gdn_linrec_fwd(d["x"], d["g"], save_states=True)
        assert gdn.linrec_status() == 6 and gdn.linrec_status() == 0
        gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], states=states)
        assert gdn.linrec_status() == 6
    finally:
        gdn.set_test_hook(0)
        gdn.set_wait_limit(0)
    run_and_check(v)
    assert gdn.linrec_status() == 0


def test_launch_trace_names_the_kernels():
    v = draw(1, 300, 64)
    d = {k: t.cuda() for k, t in v.items()}
    with gdn.LaunchTrace(16) as trace:
        gdn.gdn_linrec_fwd(d["x"], d["g"])
        gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"])
        gdn.gdn_linrec_decode(d["x"], d["g"], d["h0"])
    torch.cuda.synchronize()
    assert {k: n for k, (n, _) in trace.per_kernel().items()} == {
        "linrec_fwd": 2, "linrec_bwd": 1, "linrec_decode": 1}


def test_empty_rows_pass_the_states_through():
    x = torch.zeros(1, 0, 40, dtype=torch.bfloat16, device="cuda")
    h0, dhT = torch.randn(3, 40, device="cuda"), torch.randn(3, 40, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32)
    o, hT = gdn.gdn_linrec_fwd(x, x, cu_seqlens=cu.cuda(), cu_seqlens_host=cu, h0=h0)
    assert o.shape == x.shape and torch.equal(hT, h0)
    dh0 = gdn.gdn_linrec_bwd(x, x, x, cu_seqlens=cu.cuda(), cu_seqlens_host=cu, dhT=dhT)[2]
    assert torch.equal(dh0, dhT)


def test_a_device_tensor_as_the_mirror_of_the_offsets_is_refused():
    v = draw(1, 30, 8, N=2)
    d = {k: t.cuda() for k, t in v.items()}
    cu = torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 30, 1, 64, device="cuda")
    s = torch.zeros(1, 30, 1, device="cuda")
    for call in (lambda **k: gdn.gdn_linrec_fwd(d["x"], d["g"], **k),
                 lambda **k: gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], **k),
                 lambda **k: gdn.gdn_fwd(q, q, q, s, s, **k),
                 lambda **k: gdn.gdn_bwd(q, q, q, s, s, q, **k)):
        for kw in (dict(cu_seqlens=cu), dict()):
            with pytest.raises(ValueError, match="CPU tensor"):
                call(cu_seqlens_host=cu, **kw)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("B,T,D", [(1, 200, 64), (1, 1100, 8), (1, 9000, 64), (3, 5000, 130), (2, 40000, 66)])
def test_clusters_that_give_up_end_with_every_map_accounted_for(B, T, D, types):
    """Waits that run out in the first step (planted), or wherever a limit of few polls makes them: clusters
    of one step and of many, in both directions.  The calls end, and the ones after them are right."""
    v = draw(B, T, D, *types, seed=T)
    d = {k: t.cuda() for k, t in v.items()}
    run = lambda: gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], states=gdn.gdn_linrec_fwd(
        d["x"], d["g"], h0=d["h0"], save_states=True)[2], h0=d["h0"], dhT=d["dhT"])
    want = run()
    gdn.linrec_status()
    try:
        gdn.set_wait_limit(256)
        gdn.set_test_hook(gdn.GDN_TEST_STALL_COPY)
        run()
        assert gdn.linrec_status() == 6
        gdn.set_test_hook(0)
        for polls in (1, 2, 5, 20):
            gdn.set_wait_limit(polls)
            for _ in range(5):
                run()
            assert gdn.linrec_status() in (0, 6)
    finally:
        gdn.set_test_hook(0)
        gdn.set_wait_limit(0)
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    assert gdn.linrec_status() == 0


def test_a_timeout_is_told_of_its_own_stream_and_to_every_thread():
    from concurrent.futures import ThreadPoolExecutor
    v = draw(1, 2000, 64, seed=4)
    x, g = v["x"].cuda(), v["g"].cuda()
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    torch.cuda.synchronize()

    def stalled(call):
        gdn.set_wait_limit(256)
        gdn.set_test_hook(gdn.GDN_TEST_STALL_COPY)
        try:
            call()
        finally:
            gdn.set_test_hook(0)
            gdn.set_wait_limit(0)

    with ThreadPoolExecutor(1) as other:
        there = lambda *args: other.submit(gdn.linrec_status, *args).result()
        for s in (a, b, c):
            assert gdn.linrec_status(s) == 0 and there(s) == 0
        stalled(lambda: gdn.gdn_linrec_fwd(x, g, stream=a))
        gdn.gdn_linrec_fwd(x, g, stream=b)
        assert gdn.linrec_status(b) == 0
        assert gdn.linrec_status(a) == 6 and gdn.linrec_status(a) == 0
        assert there(b) == 0 and there(a) == 6 and there(a) == 0
        # captured calls: told of whichever stream is asked for, once to each thread
        graph = torch.cuda.CUDAGraph()

        def capture():
            with torch.cuda.graph(graph):
                gdn.gdn_linrec_fwd(x, g)

        stalled(capture)
        with torch.cuda.stream(c):
            graph.replay()
        assert gdn.linrec_status(c) == 6 and gdn.linrec_status(c) == 0 and gdn.linrec_status(b) == 0
        assert there(c) == 6 and there(c) == 0


def test_the_status_of_a_stream_that_is_captured_is_refused():
    x = torch.zeros(1, 300, 64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = gdn.gdn_linrec_fwd(x, x)
        assert gdn.linrec_status() == 1
    graph.replay()
    assert gdn.linrec_status() == 0 and (o == 0).all()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("complement", [False, True])
@pytest.mark.parametrize("lengths", [None, [700, 0, 4100, 1, 4199]])
def test_gates_that_are_nan_stay_in_their_channel(types, complement, lengths):
    """NaN of both signs in g, in tiles of several CTAs of a cluster: the channel beside it (in the same lane)
    and the other documents keep their bits."""
    T, D = 9000, 66
    N = 1 if lengths is None else len(lengths)
    v = draw(1, T, D, *types, N=N, seed=3)
    d = {k: t.cuda() for k, t in v.items()}
    cu = None if lengths is None else torch.tensor([0] + np.cumsum(lengths).tolist(), dtype=torch.int32)
    kw = dict(cu_seqlens=None if cu is None else cu.cuda(), cu_seqlens_host=cu, h0=d["h0"], complement=complement)

    def run():
        o, hT, states = gdn.gdn_linrec_fwd(d["x"], d["g"], save_states=True, **kw)
        return (o, hT) + gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], dhT=d["dhT"], states=states, **kw)

    want = run()
    nan = torch.tensor([float("nan")])
    at = {0: 5, 3: 1000, 33: 4500, 64: 8500, 65: 8500}
    for i, (c, t) in enumerate(at.items()):
        d["g"][0, t, c] = torch.copysign(nan, torch.tensor(1.0 - 2 * (i % 2))).to(d["g"].dtype).item()
    assert d["g"].isnan().sum() == len(at)
    o, hT, dx, dg, dh0 = run()
    segs = ref.segments(1, T, None if cu is None else cu.tolist())
    for c in range(D):
        t = at.get(c)
        n, (t0, t1) = (-1, (0, 0)) if t is None else next((n, s) for n, s in enumerate(segs) if s[0] <= t < s[1])
        here = torch.zeros(T, dtype=torch.bool, device="cuda")
        here[t0:t1] = True  # the document of the NaN, and in it the tokens from it on, or up to it
        late, early = here.clone(), here.clone()
        if t is not None:
            late[:t] = False
            early[t + complement:] = False  # dx of the token itself has the factor 1 - exp(NaN)
        for got, ref_, bad in ((o, want[0], late), (dx, want[2], early), (dg, want[3], here)):
            assert got[0, bad, c].isnan().all() and torch.equal(got[0, ~bad, c], ref_[0, ~bad, c])
        for got, ref_ in ((hT, want[1]), (dh0, want[4])):
            for m in range(N):
                assert got[m, c].isnan() if m == n else got[m, c] == ref_[m, c]


@pytest.mark.parametrize("types,complement", [(TYPES[0], True), (TYPES[1], False), (TYPES[1], True), (TYPES[2], False),
                                              (TYPES[2], True)])
@pytest.mark.parametrize("B,T,D", [(700, 3, 1160), (9001, 1, 260), (601, 63, 66), (1201, 16, 130)])
def test_many_short_rows_of_every_type(B, T, D, types, complement):
    """Streams of more rows than fill a tile, in every type and with both write strengths."""
    run_and_check(draw(B, T, D, *types, seed=B + 1), complement=complement)


def test_a_backward_behind_a_forward_that_gave_up_runs_on_and_is_reported():
    """Without saved states the backward recomputes them first: if that stalls, the call is undefined in its
    values, writes nothing beside its outputs, and is reported once."""
    v = draw(2, 3000, 72, seed=6)
    want = run_and_check(v)[2:]
    d = {k: t.cuda() for k, t in v.items()}
    wide = [torch.full((2, 3000, 80), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dx, dg = (w[..., :72] for w in wide)
    dh0 = torch.empty_like(d["h0"])
    call = lambda: gdn.gdn_linrec_bwd(d["x"], d["g"], d["do"], h0=d["h0"], dhT=d["dhT"], grads=(dx, dg, dh0))
    gdn.set_wait_limit(256)
    gdn.set_test_hook(gdn.GDN_TEST_STALL_COPY)
    try:
        call()
    finally:
        gdn.set_test_hook(0)
        gdn.set_wait_limit(0)
    assert gdn.linrec_status() == 6 and gdn.linrec_status() == 0
    assert all((w[..., 72:] == 7).all() for w in wide)
    for a, b in zip(call(), want):
        assert torch.equal(a, b)
    assert gdn.linrec_status() == 0


def test_a_captured_timeout_is_told_once_whatever_streams_are_asked_for():
    v = draw(1, 2000, 64, seed=4)
    x, g = v["x"].cuda(), v["g"].cuda()
    gdn.set_wait_limit(256)
    gdn.set_test_hook(gdn.GDN_TEST_STALL_COPY)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gdn.gdn_linrec_fwd(x, g)
    finally:
        gdn.set_test_hook(0)
        gdn.set_wait_limit(0)
    streams = [torch.cuda.Stream() for _ in range(24)]
    for s in streams[:3]:
        gdn.linrec_status(s)
    graph.replay()
    torch.cuda.synchronize()
    assert [gdn.linrec_status(s) for s in streams] == [6] + [0] * 23
    graph.replay()
    torch.cuda.synchronize()
    assert [gdn.linrec_status(s) for s in streams[::-1]] == [6] + [0] * 23
