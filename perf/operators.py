"""Measured cases of the gated linear recurrence and of the q/k normalisation with rotation.

Gated linear recurrence (per sequence and channel, state in fp32):

    h_t = a_t h_{t-1} + w_t x_t,   a_t = exp(g_t),   w_t = 1, or 1 - a_t ("complement"),   o_t = h_t

with packed documents, initial and final states, its gradients, and the one-token form that updates a
state in place.  q/k normalisation with rotation (per token and head, rows of d values):

    y = R(p) (weight * x / sqrt(c |x|^2 + eps)),   c = 1 ("l2") or 1/d ("rms")

where R(p) turns the pairs of the first `rot` values by the angles p * inv_freq[i], with its gradients.

`own = False` computes them with elementary torch operations in 32 bits (angles and weight gradients in
64); `own = True` calls the library.  `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases
def _linrec(name, mode, B, T, D, dtype="bf16", gate="bf16", complement=False, docs=0, least=0,
            fused=False, gate_scale=0.1):
    """docs: documents of a packed row, each of `least` tokens or more (0: dense rows).  fused: x and g are column slices
    of one projection, as a layer that computes both with one matrix product has them."""
    return dict(name=name, op="linrec", mode=mode, B=B, T=T, D=D, dtype=dtype, gate=gate,
                complement=complement, docs=docs, least=least, fused=fused, gate_scale=gate_scale)


def _qk(name, mode, B, T, Hq, Hk, d, rot, dtype="bf16", norm="rms", interleaved=False, docs=0,
        least=0, far=0, fused=False):
    """far: positions are drawn from [0, far) instead of counting from each row's or document's start."""
    return dict(name=name, op="qk", mode=mode, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot, dtype=dtype,
                norm=norm, interleaved=interleaved, docs=docs, least=least, far=far, fused=fused)


def listed():
    return [
        # one token for one sequence of 16 heads x 128 channels: interactive serving, latency counts
        _linrec("linrec_decode_1x2048", "decode", 1, 1, 2048, gate="fp32"),
        # one token for each of a full batch of sequences
        _linrec("linrec_decode_256x2048", "decode", 256, 1, 2048),
        # prefill of a packed row of documents, fp32 gates as the delta rule has them
        _linrec("linrec_prefill_packed_16384x2048", "fwd", 1, 16384, 2048, gate="fp32", docs=9, least=64),
        # a training step of four rows, input and gate from one projection, write strength 1 - a
        _linrec("linrec_train_4x4096x2048", "train", 4, 4096, 2048, complement=True, fused=True),
        # a training step of one long row: few channels, all parallelism along the tokens
        _linrec("linrec_train_1x262144x1024", "train", 1, 262144, 1024, gate_scale=0.02),
        # an fp32 training step of odd sizes
        _linrec("linrec_train_fp32_3x1237x515", "train", 3, 1237, 515, dtype="fp32", gate="fp32"),
        # one token of one sequence, 16 + 16 heads, far into its context
        _qk("qk_decode_1_h16_d128", "fwd", 1, 1, 16, 16, 128, 128, far=1 << 20),
        # one token for each of a full batch, query heads over fewer key heads, slices of one projection
        _qk("qk_decode_256_h16_4_d128", "fwd", 256, 1, 16, 4, 128, 128, far=131072, fused=True),
        # a packed row with the layer's weightless x / |x|, positions from each document's start
        _qk("qk_packed_16384_h16_d128_l2", "fwd", 1, 16384, 16, 16, 128, 128, norm="l2", docs=9, least=64),
        # a training step of four rows with learned weights
        _qk("qk_train_4x4096_h16_d128", "train", 4, 4096, 16, 16, 128, 128),
        # an fp32 training step of odd sizes, adjacent pairs, part of each row rotated
        _qk("qk_train_fp32_3x777_h6_2_d64", "train", 3, 777, 6, 2, 64, 48, dtype="fp32", interleaved=True),
        # one long row, head dim 256 with half of each row rotated
        _qk("qk_fwd_1x131072_h8_d256", "fwd", 1, 131072, 8, 8, 256, 128),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.55:
        mode = rng.choice(["decode", "fwd", "train", "train"])
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        gate = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
        D = _spread(rng, 24, 4096)
        if rng.random() < 0.6:
            D = -(-D // 8) * 8
        if mode == "decode":
            B, T, docs, least = _spread(rng, 1, 512), rng.choice([1, 1, 1, 2, 4]), 0, 0
        else:
            T = _spread(rng, 1, 32768)
            most = max(1, min(64, (1 << 25) // (T * D)))
            B, docs, least = _spread(rng, 1, most), 0, 0
            if rng.random() < 0.4:  # packed: where `least` is 0, a few empty documents among them
                B, docs = 1, _spread(rng, 1, max(1, T // 8))
                least = min(T // docs, rng.choice([0, 1, 16]))
        fused = D % 8 == 0 and gate == dtype and rng.random() < 0.5
        return _linrec("", mode, B, T, D, dtype, gate, rng.random() < 0.5, docs, least, fused,
                       rng.choice([0.02, 0.1]))
    mode, dtype = rng.choice(["fwd", "fwd", "train"]), rng.choice(["bf16", "bf16", "fp32"])
    d = rng.choice([32, 64, 80, 96, 128, 192, 256])
    rot = rng.choice([d, d, d // 2, d // 4 * 2])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4])
    T = _spread(rng, 1, 16384)
    B = _spread(rng, 1, max(1, min(256, (1 << 25) // (T * d * (Hq + Hk)))))
    docs = least = far = 0
    if rng.random() < 0.3:
        B, docs, least = 1, _spread(rng, 1, max(1, T // 8)), 1
    elif rng.random() < 0.5:
        far = _spread(rng, 1024, 1 << 20)
    return _qk("", mode, B, T, Hq, Hk, d, rot, dtype, rng.choice(["rms", "rms", "l2"]),
               rng.random() < 0.4, docs, least, far, rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _offsets(case, seed):
    """Documents' first tokens and the row's end: `docs` lengths of `least` or more, cut at random places."""
    gen = torch.Generator().manual_seed(seed + 1000)
    n, least = case["docs"], case["least"]
    cuts = torch.randint(0, case["T"] - n * least + 1, (n - 1,), generator=gen).sort()[0]
    cuts = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([case["T"] - n * least])])
    return (cuts + least * torch.arange(n + 1)).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    B, T, dt = case["B"], case["T"], DTYPES[case["dtype"]]
    s = dict(case)
    cu = None
    if case["docs"]:  # packed documents: offsets on the device, and the host's copy of them
        cu = _offsets(case, seed)
    s["cu_host"], s["cu"] = cu, None if cu is None else cu.to(dev)
    if case["op"] == "linrec":
        D, gdt = case["D"], DTYPES[case["gate"]]
        N = B if cu is None else cu.numel() - 1
        x = randn(B, T, D).to(dt)
        g = (-torch.nn.functional.softplus(randn(B, T, D)) * case["gate_scale"]).to(gdt)
        if case["fused"]:
            x, g = torch.cat([x, g], -1).split(D, -1)
        s.update(x=x, g=g, h0=randn(N, D) * 0.5)
        if case["mode"] == "train":
            s.update(do=randn(B, T, D).to(dt), dhT=randn(N, D) * 0.1)
        return s
    Hq, Hk, d, rot = case["Hq"], case["Hk"], case["d"], case["rot"]
    qk = (randn(B, T, Hq + Hk, d) * torch.exp(0.5 * randn(B, T, Hq + Hk, 1))).to(dt)
    q, k = qk.split([Hq, Hk], 2)
    s.update(q=q if case["fused"] else q.contiguous(), k=k if case["fused"] else k.contiguous())
    # rotation frequencies 10000^(-2i / rot), as a model keeps them
    s["inv_freq"] = torch.pow(1e4, -torch.arange(0, rot, 2, dtype=torch.float64) / rot).float().to(dev)
    if case["far"]:
        pos = torch.randint(0, case["far"], (B, T), generator=gen, device=dev)
    elif cu is not None:
        at = torch.arange(T, device=dev)
        pos = (at - s["cu"][:-1].long()[torch.searchsorted(s["cu"][1:].long(), at, right=True)])[None]
    else:
        pos = None
    s["positions"] = None if pos is None else pos.to(torch.int32)
    s["wq"] = s["wk"] = None
    if case["norm"] == "rms":
        s["wq"], s["wk"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
    if case["mode"] == "train":
        s.update(dqo=randn(B, T, Hq, d).to(dt), dko=randn(B, T, Hk, d).to(dt))
    return s


# ---------------------------------------------------------------- plain forms
def _firsts(s, device):
    """First tokens of the sequences that have any, and the indices of those sequences."""
    if s["cu"] is None:
        n = torch.arange(s["B"], device=device)
        return n * s["T"], n, (n + 1) * s["T"] - 1
    lens = s["cu"][1:] - s["cu"][:-1]
    n = torch.nonzero(lens > 0)[:, 0]
    return s["cu"][:-1].long()[n], n, s["cu"][1:].long()[n] - 1


def _scan(a, b, longest):
    """b_t <- a_t b_{t-1} + b_t along the tokens, in place, by doubling distances; a is overwritten."""
    step = 1
    while step < longest:
        b[step:] += a[step:] * b[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _linrec_parts(s):
    D = s["D"]
    x, g = s["x"].reshape(-1, D).float(), s["g"].reshape(-1, D).float()
    a = torch.exp(g)
    w = -torch.expm1(g) if s["complement"] else torch.ones_like(g)
    return x, a, w


def _linrec_forward(s, x, a, w):
    first, n, last = _firsts(s, x.device)
    A, h = a.clone(), w * x
    h[first] += a[first] * s["h0"][n]
    A[first] = 0
    _scan(A, h, s["T"])
    hT = s["h0"].clone()
    hT[n] = h[last]
    return h, hT


def _linrec_backward(s, x, a, w, h):
    first, n, last = _firsts(s, x.device)
    e = s["do"].reshape(-1, s["D"]).float().clone()
    e[last] += s["dhT"][n]
    A = torch.zeros_like(a)
    A[:-1] = a[1:]
    A[last] = 0
    e = _scan(A.flip(0), e.flip(0), s["T"]).flip(0)
    before = torch.zeros_like(h)
    before[1:] = h[:-1]
    before[first] = s["h0"][n]
    if s["complement"]:
        before = before - x
    dh0 = s["dhT"].clone()
    dh0[n] = (a * e)[first]
    return w * e, a * e * before, dh0


def _linrec_plain(s):
    shape, xt, gt = s["x"].shape, s["x"].dtype, s["g"].dtype
    if s["mode"] == "decode":
        x, a, w = (v.view(shape) for v in _linrec_parts(s))
        out = []
        for t in range(s["T"]):
            s["h0"].copy_(a[:, t] * s["h0"] + w[:, t] * x[:, t])
            out.append(s["h0"].to(xt))
        return torch.stack(out, 1), s["h0"]
    x, a, w = _linrec_parts(s)
    h, hT = _linrec_forward(s, x, a, w)
    out = (h.to(xt).view(shape), hT)
    if s["mode"] == "train":
        dx, dg, dh0 = _linrec_backward(s, x, a, w, h)
        out += (dx.to(xt).view(shape), dg.to(gt).view(shape), dh0)
    return out


def _angles(s):
    """cos and sin of position x frequency, [B, T, 1, rot/2], the angle in 64 bits."""
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(s["T"], device=s["q"].device).expand(s["B"], -1)
    angle = pos.double()[..., None, None] * s["inv_freq"].double()
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, interleaved):
    """The pairs of x's first 2 * cos.shape[-1] values turned by the angles; the others as they are."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, v = a * cos - b * sin, a * sin + b * cos
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _norm_consts(s):
    return (1.0 / s["d"], 1e-6) if s["norm"] == "rms" else (1.0, 0.0)


def _unit(s, x):
    """x in 32 bits and 1 / its norm (0 for a zero row without eps)."""
    c, eps = _norm_consts(s)
    x = x.float()
    m = c * (x * x).sum(-1, keepdim=True) + eps
    return x, torch.where(m > 0, m.rsqrt(), torch.zeros_like(m))


def _qk_one(s, x, w, dy, cos, sin):
    dt = x.dtype
    x, r = _unit(s, x)
    w = torch.ones(s["d"], device=x.device) if w is None else w
    if dy is None:
        return (_turn(x * r * w, cos, sin, s["interleaved"]).to(dt),)
    y = _turn(x * r * w, cos, sin, s["interleaved"])
    u = _turn(dy.float(), cos, -sin, s["interleaved"])
    xn = x * r
    c, _ = _norm_consts(s)
    dx = r * (u * w - xn * (c * (u * w * xn).sum(-1, keepdim=True)))
    dw = (u * xn).double().sum((0, 1, 2)).float()
    return y.to(dt), dx.to(dt), dw


def _qk_plain(s):
    cos, sin = _angles(s)
    q = _qk_one(s, s["q"], s["wq"], s.get("dqo"), cos, sin)
    k = _qk_one(s, s["k"], s["wk"], s.get("dko"), cos, sin)
    if s["norm"] == "l2":  # no weights, no gradients of them
        q, k = q[:2], k[:2]
    return q, k


# ---------------------------------------------------------------- one pass
def _linrec_own(s):
    import gated_delta_rule_99_b200 as gdn
    kw = dict(complement=s["complement"])
    if s["mode"] == "decode":
        return gdn.gdn_linrec_decode(s["x"], s["g"], s["h0"], **kw), s["h0"]
    kw.update(cu_seqlens=s["cu"], cu_seqlens_host=s["cu_host"], h0=s["h0"])
    if s["mode"] == "fwd":
        return gdn.gdn_linrec_fwd(s["x"], s["g"], **kw)
    o, hT, states = gdn.gdn_linrec_fwd(s["x"], s["g"], save_states=True, **kw)
    return (o, hT) + tuple(gdn.gdn_linrec_bwd(s["x"], s["g"], s["do"], dhT=s["dhT"], states=states, **kw))


def _qk_own(s):
    import gated_delta_rule_99_b200 as gdn
    kw = dict(inv_freq=s["inv_freq"], positions=s["positions"], norm=s["norm"], q_weight=s["wq"],
              k_weight=s["wk"], interleaved=s["interleaved"])
    qo, ko = gdn.gdn_qk_norm_rope_fwd(s["q"], s["k"], **kw)
    if s["mode"] == "fwd":
        return (qo,), (ko,)
    dq, dk, dwq, dwk = gdn.gdn_qk_norm_rope_bwd(s["q"], s["k"], s["dqo"], s["dko"], **kw)
    return ((qo, dq), (ko, dk)) if s["norm"] == "l2" else ((qo, dq, dwq), (ko, dk, dwk))


def run(state):
    if own:
        return _linrec_own(state) if state["op"] == "linrec" else _qk_own(state)
    return _linrec_plain(state) if state["op"] == "linrec" else _qk_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"bf16": 2, "fp32": 4}
    es, train = size[case["dtype"]], case["mode"] == "train"
    if case["op"] == "linrec":
        n = case["B"] * case["T"] * case["D"]
        gs = size[case["gate"]]
        seqs = case["docs"] or case["B"]
        per, flops, states = 2 * es + gs, 4 + case["complement"], 2
        if train:  # x, g and do in, dx and dg out besides
            per, flops, states = per + 3 * es + 2 * gs, flops + 8, 5
        return {"bytes": n * per + 4 * states * seqs * case["D"], "flops": n * flops}
    n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["d"]
    return {"bytes": n * es * (5 if train else 2) + case["B"] * case["T"] * 4, "flops": n * (22 if train else 8)}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_linrec(s):
    """Token after token, from the definition."""
    D = s["D"]
    x, g = s["x"].double().reshape(-1, D), s["g"].double().reshape(-1, D)
    a = g.exp()
    put = (-torch.expm1(g)) * x if s["complement"] else x
    if s["cu"] is None:
        steps, runs = s["T"], [(0, s["T"])]
        x, a, put, g = (v.view(s["B"], s["T"], D).transpose(0, 1) for v in (x, a, put, g))
        of = [slice(None)]
    else:
        c = s["cu_host"].tolist()
        steps, runs = s["T"], list(zip(c, c[1:]))
        x, a, put, g = (v[:, None] for v in (x, a, put, g))
        of = [slice(i, i + 1) for i in range(len(runs))]
    h, before = torch.empty_like(x), torch.empty_like(x)
    hT = s["h0"].double().clone()
    for (t0, t1), i in zip(runs, of):
        cur = hT[i]
        for t in range(t0, t1):
            cur = torch.addcmul(put[t], a[t], cur, out=h[t])
        if t1 > t0:
            before[t0], before[t0 + 1:t1] = hT[i], h[t0:t1 - 1]
            hT[i] = cur
    rows = lambda v: v.transpose(0, 1).reshape(s["x"].shape)  # noqa: E731
    if s["mode"] == "decode":
        return rows(h), hT
    if s["mode"] == "fwd":
        return rows(h), hT
    do = s["do"].double().reshape(s["B"], steps, D).transpose(0, 1)
    e, dh0 = do.clone(), s["dhT"].double().clone()
    for (t0, t1), i in zip(runs, of):
        if t1 > t0:
            e[t1 - 1] += dh0[i]
            for t in range(t1 - 2, t0 - 1, -1):
                e[t].addcmul_(a[t + 1], e[t + 1])
            dh0[i] = a[t0] * e[t0]
    if s["complement"]:
        dx, dg = -torch.expm1(g) * e, e * a * (before - x)
    else:
        dx, dg = e, e * a * before
    return rows(h), hT, rows(dx), rows(dg), dh0


def _exact_rows(s, x, w):
    """The rows as complex numbers, one for each pair, turned by unit complex numbers."""
    c, eps = (1.0 / s["d"], 1e-6) if s["norm"] == "rms" else (1.0, 0.0)
    y = x / torch.sqrt(c * x.square().sum(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w
    rot = s["rot"]
    pairs = (y[..., :rot].unflatten(-1, (rot // 2, 2)) if s["interleaved"] else
             y[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2))
    pos = torch.arange(s["T"], device=x.device)[None] if s["positions"] is None else s["positions"]
    angle = pos.double()[:, :, None, None] * s["inv_freq"].double()
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle))
    z = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linrec":
        return _exact_linrec(s)
    out = []
    for x, w, dy in ((s["q"], s["wq"], s.get("dqo")), (s["k"], s["wk"], s.get("dko"))):
        if dy is None:
            out.append((_exact_rows(s, x.double(), None if w is None else w.double()),))
            continue
        x = x.double().requires_grad_()
        w = None if w is None else w.double().requires_grad_()
        y = _exact_rows(s, x, w)
        grads = torch.autograd.grad(y, [x] if w is None else [x, w], dy.double())
        out.append((y.detach(),) + grads)
    return tuple(out)
