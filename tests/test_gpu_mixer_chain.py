"""The operators run together as a token-mixing layer uses them: the values are mixed along the tokens
by the gated linear recurrence, q and k are normalised and rotated, and the delta rule reads all
three; forward and backward over packed documents, and a prefill followed by one-token steps that
carry the recurrence's state, the delta rule's state and the position.  Against the fp64 forms of
oracle/, with the layer's own tolerances (largest error over largest value): 1e-4 for fp32 inputs, 2e-2
for bf16 ones."""
import numpy as np
import pytest
import torch

import gated_delta_rule_99_b200 as gdn
import oracle
from oracle import linrec as ref_linrec
from oracle import qk_rope as ref_qk

from _util import maxnorm_err

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"fp32": 1e-4, "bf16": 2e-2}
H, K = 2, 64


def inputs(T, dtype, N, seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    D = H * K
    return dict(
        # one projection holds q, k, the values and their gates side by side
        proj=torch.cat([r(1, T, 2 * D), r(1, T, D), -torch.nn.functional.softplus(r(1, T, D))],
                       -1).to(DT[dtype]),
        g=-torch.nn.functional.softplus(r(1, T, H)) * 0.1, beta=torch.sigmoid(r(1, T, H)),
        s0=r(N, D) * 0.1, h0=r(N, H, K, K) * 0.1, wq=1 + 0.1 * r(K), wk=(1 + 0.1 * r(K)) / 8,
        inv_freq=torch.pow(1e4, -torch.arange(0, K, 2).double() / K).float(),
        do=r(1, T, H, K).to(DT[dtype]), dhT=r(N, H, K, K) * 0.1, dsT=r(N, D) * 0.1)


def parts(proj):
    D = H * K
    q, k, v, a = proj.split(D, -1)
    T = proj.shape[1]
    return q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v, a, T


def positions(cu):
    return torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])])[None].to(torch.int32)


def forward(d, cu_dev, cu_host, pos):
    q, k, v, a, T = parts(d["proj"])
    u, sT, states = gdn.gdn_linrec_fwd(v, a, cu_seqlens=cu_dev, cu_seqlens_host=cu_host, h0=d["s0"],
                                       complement=True, save_states=True)
    qr, kr = gdn.gdn_qk_norm_rope_fwd(q, k, d["inv_freq"], pos, q_weight=d["wq"], k_weight=d["wk"])
    o, hT = gdn.gdn_fwd(qr, kr, u.view(1, T, H, K), d["g"], d["beta"], cu_seqlens=cu_dev,
                        cu_seqlens_host=cu_host, h0=d["h0"])
    return (u, sT, states, qr, kr, o, hT)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_forward_and_backward_over_packed_documents(dtype):
    cu = [0, 70, 70, 71, 200, 330]
    x = inputs(330, dtype, 5, 3)
    d = {n: t.cuda() for n, t in x.items()}
    cu_host = torch.tensor(cu, dtype=torch.int32)
    cu_dev, pos = cu_host.cuda(), positions(cu)
    q, k, v, a, T = parts(d["proj"])
    u, sT, states, qr, kr, o, hT = forward(d, cu_dev, cu_host, pos.cuda())
    dqr, dkr, du, dg, dbeta, dh0 = gdn.gdn_bwd(qr, kr, u.view(1, T, H, K), d["g"], d["beta"], d["do"],
                                               cu_seqlens=cu_dev, cu_seqlens_host=cu_host, h0=d["h0"],
                                               dhT=d["dhT"])
    # the gradients go into the slices of one projection's gradient
    dproj = torch.full_like(d["proj"], float("nan"))
    dq, dk, dv, da, _ = parts(dproj)
    ds0 = torch.empty_like(d["s0"])
    gdn.gdn_linrec_bwd(v, a, du.view(1, T, H * K), cu_seqlens=cu_dev, cu_seqlens_host=cu_host,
                       h0=d["s0"], dhT=d["dsT"], complement=True, states=states, grads=(dv, da, ds0))
    dwq, dwk = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    gdn.gdn_qk_norm_rope_bwd(q, k, dqr, dkr, d["inv_freq"], pos.cuda(), q_weight=d["wq"],
                             k_weight=d["wk"], grads=(dq, dk, dwq, dwk))
    assert gdn.linrec_status() == 0

    # the same in 64 bits, from the same inputs
    n64 = lambda t: t.double().numpy()
    cq, ck, cv, ca, _ = parts(x["proj"])
    segs = ref_linrec.segments(1, T, cu)
    ru, rsT = ref_linrec.fwd(n64(cv)[0], n64(ca)[0], n64(x["s0"]), segs, True)[:2]
    qk = (n64(pos), n64(x["inv_freq"]), "rms")
    rq = ref_qk.fwd(n64(cq), *qk, n64(x["wq"]), 1e-6, False)[0]
    rk = ref_qk.fwd(n64(ck), *qk, n64(x["wk"]), 1e-6, False)[0]
    rv = ru.reshape(1, T, H, K)
    args = (rq, rk, rv, n64(x["g"]), n64(x["beta"]))
    ro, rhT = oracle.gdn_fwd(*args, cu_seqlens=cu_host, h0=n64(x["h0"]))
    rdq, rdk, rdv, rdg, rdbeta, rdh0 = oracle.gdn_bwd(*args, n64(x["do"]), cu_seqlens=cu_host,
                                                      h0=n64(x["h0"]), dhT=n64(x["dhT"]))
    (rdx, rda, rds0), _ = ref_linrec.bwd(n64(cv)[0], n64(ca)[0], n64(x["s0"]),
                                         rdv.reshape(T, H * K), n64(x["dsT"]), segs, True)
    (rdq, rdwq), _ = ref_qk.bwd(n64(cq), rdq, *qk, n64(x["wq"]), 1e-6, False)
    (rdk, rdwk), _ = ref_qk.bwd(n64(ck), rdk, *qk, n64(x["wk"]), 1e-6, False)
    errs = {name: maxnorm_err(got, want.reshape(got.shape)) for name, got, want in (
        ("u", u, ru), ("sT", sT, rsT), ("o", o, ro), ("hT", hT, rhT), ("dg", dg, rdg),
        ("dbeta", dbeta, rdbeta), ("dh0", dh0, rdh0), ("dv", dv, rdx), ("da", da, rda),
        ("ds0", ds0, rds0), ("dq", dq, rdq), ("dk", dk, rdk), ("dwq", dwq, rdwq), ("dwk", dwk, rdwk))}
    print(" ".join("%s=%.1e" % e for e in errs.items()))
    assert all(e <= TOL[dtype] for e in errs.values()), errs


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prefill_then_one_token_steps(dtype):
    """150 tokens at once and 4 one by one give what 154 at once give (a bf16 value passes the same
    roundings in both; sums associate differently, so single values may round to the neighbour)."""
    x = inputs(154, dtype, 1, 5)
    d = {n: t.cuda() for n, t in x.items()}
    pos = torch.arange(154, dtype=torch.int32, device="cuda")[None]
    whole = forward(d, None, None, pos)
    cut = lambda t, a, b: t[:, a:b].clone()  # its own, aligned memory
    head = dict(d, proj=cut(d["proj"], 0, 150), g=cut(d["g"], 0, 150), beta=cut(d["beta"], 0, 150))
    u, state, _, _, _, o, h = forward(head, None, None, pos[:, :150])
    outs = [o]
    for t in range(150, 154):
        q, k, v, a, _ = parts(cut(d["proj"], t, t + 1))
        u = gdn.gdn_linrec_decode(v, a, state, complement=True)
        qr, kr = gdn.gdn_qk_norm_rope_fwd(q, k, d["inv_freq"], pos[:, t:t + 1],
                                          q_weight=d["wq"], k_weight=d["wk"])
        outs.append(gdn.gdn_decode(qr, kr, u.view(1, 1, H, K), cut(d["g"], t, t + 1),
                                   cut(d["beta"], t, t + 1), h))
    tol = {"fp32": 1e-5, "bf16": 2e-2}[dtype]
    assert maxnorm_err(state, whole[1]) <= 1e-5
    assert maxnorm_err(torch.cat(outs, 1), whole[5]) <= tol
    assert maxnorm_err(h, whole[6]) <= tol


def test_two_streams_at_once():
    """The same calls on two streams at the same time, with nothing shared but the inputs."""
    x = inputs(2000, "bf16", 1, 7)
    d = {n: t.cuda() for n, t in x.items()}
    pos = torch.arange(2000, dtype=torch.int32, device="cuda")[None]
    want = forward(d, None, None, pos)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(forward(d, None, None, pos))
    torch.cuda.synchronize()
    for g in got:
        for i in (0, 1, 3, 4, 5, 6):
            assert torch.equal(g[i], want[i])
    assert gdn.linrec_status() == 0


def test_first_calls_inside_a_capture():
    """A fresh process whose first calls of the operators are captured into a graph."""
    import subprocess
    import sys
    code = """
import torch, gated_delta_rule_99_b200 as gdn
x = torch.randn(1, 700, 96, device="cuda").bfloat16(); g = -torch.rand_like(x)
q = torch.randn(1, 700, 2, 64, device="cuda"); w = torch.ones(64, device="cuda"); f = torch.rand(32, device="cuda")
st = torch.zeros(1, 96, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def run():
    o, hT, states = gdn.gdn_linrec_fwd(x, g, save_states=True)
    a = gdn.gdn_linrec_bwd(x, g, x, states=states)
    b = gdn.gdn_qk_norm_rope_bwd(q, q, q, q, f, q_weight=w, k_weight=w)
    return (o, hT) + a + gdn.gdn_qk_norm_rope_fwd(q, q, f, q_weight=w) + b
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__import__("os").path.dirname(__import__("os").path.dirname(
                           __import__("os").path.abspath(__file__))))
    assert "captured" in r.stdout, r.stderr[-2000:]
