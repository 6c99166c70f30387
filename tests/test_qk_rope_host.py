"""Host side of the q/k normalisation with rotation: its fp64 form pinned by invariants and
differences, and every refusal, which come before anything touches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_99_b200 as gdn
from oracle import qk_rope as ref

FAKE = 0x7F0000000000  # a 256-byte aligned address that is never dereferenced


def case(norm="rms", seed=0):
    rng = np.random.default_rng(seed)
    x, dy = rng.standard_normal((2, 3, 2, 8)), rng.standard_normal((2, 3, 2, 8))
    return x, dy, rng.integers(-99, 99, (2, 3)), rng.random(3), norm, 1 + rng.random(8), 0.01


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_invariants(interleaved):
    x, dy, pos, f, norm, w, eps = case()
    y, _ = ref.fwd(x, pos, f, None, np.ones(8), 0.0, interleaved)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))            # a rotation keeps lengths
    assert np.array_equal(y[..., 6:], x[..., 6:])                   # values from rot on stay
    at0, _ = ref.fwd(x, 0 * pos, f, None, np.ones(8), 0.0, interleaved)
    assert np.allclose(at0, x)
    # <R(p) a, R(p + s) b> depends on s alone
    a, b = x, dy
    dots = [(ref.fwd(a, pos + o, f, None, np.ones(8), 0.0, interleaved)[0] *
             ref.fwd(b, pos + o + 5, f, None, np.ones(8), 0.0, interleaved)[0]).sum(-1) for o in (0, 17)]
    assert np.allclose(dots[0], dots[1])
    # the pair (1, 0) of frequency 1 at position p becomes (cos p, sin p)
    e = np.zeros((1, 1, 1, 8))
    e[..., 0] = 1
    t, _ = ref.fwd(e, np.array([[2]]), np.ones(4), None, np.ones(8), 0.0, interleaved)
    assert np.allclose(t[0, 0, 0, [0, 1 if interleaved else 4]], [np.cos(2), np.sin(2)])
    n, _ = ref.fwd(x, pos, f, "l2", np.ones(8), 0.0, interleaved)
    assert np.allclose((n * n).sum(-1), 1)
    n, _ = ref.fwd(3 * x, pos, f, "rms", np.ones(8), 0.0, interleaved)
    assert np.allclose((n * n).mean(-1), 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
def test_oracle_gradients_against_differences(norm, interleaved):
    x, dy, pos, f, _, w, eps = case()
    grads, _ = ref.bwd(x, dy, pos, f, norm, w, eps, interleaved)
    loss = lambda a, b: (dy * ref.fwd(a, pos, f, norm, b, eps, interleaved)[0]).sum()
    base = [x, w]
    for i, grad in enumerate(grads):
        for at in np.ndindex(base[i].shape):
            hi, lo = base[i].copy(), base[i].copy()
            hi[at] += 1e-6
            lo[at] -= 1e-6
            d = (loss(*[hi if j == i else b for j, b in enumerate(base)]) -
                 loss(*[lo if j == i else b for j, b in enumerate(base)])) / 2e-6
            assert abs(grad[at] - d) < 1e-7 * (1 + abs(d))


def desc(**kw):
    f = dict(B=2, T=100, Hq=4, Hk=2, d=64, rot=64, q_stride=0, k_stride=0, qo_stride=0, ko_stride=0,
             dq_stride=0, dk_stride=0, dtype=0, norm=2, flags=0, eps=1e-6)
    f.update(kw)
    return gdn.GdnQkDesc(*f.values())


def fwd(d, **kw):
    p = dict(q=FAKE, k=FAKE, pos=None, inv_freq=FAKE, qw=None, kw=None, qo=FAKE, ko=FAKE)
    p.update(kw)
    return gdn.lib().gdn_qk_norm_rope_fwd(ctypes.byref(d), *p.values(), None)


def bwd(d, ws=FAKE, ws_bytes=1 << 40, **kw):
    p = dict(q=FAKE, k=FAKE, pos=None, inv_freq=FAKE, qw=None, kw=None, dqo=FAKE, dko=FAKE, dq=FAKE,
             dk=FAKE, dqw=FAKE, dkw=None)
    p.update(kw)
    return gdn.lib().gdn_qk_norm_rope_bwd(ctypes.byref(d), *p.values(), ws, ws_bytes, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(Hk=0), 1), (dict(Hq=65536), 1),
    (dict(Hk=1 << 40), 1), (dict(d=0, rot=0), 2), (dict(d=63, rot=0), 2), (dict(d=258), 2),
    (dict(rot=66), 1), (dict(rot=-2), 1), (dict(rot=3), 1), (dict(B=1 << 40, T=1 << 40), 1),
    (dict(dtype=2), 2), (dict(norm=3), 2), (dict(norm=-1), 2), (dict(flags=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(q_stride=255), 1),
    (dict(k_stride=127), 1), (dict(qo_stride=-256), 1), (dict(ko_stride=1), 1),
    (dict(dq_stride=1 << 31), 1), (dict(dk_stride=100), 1)])
def test_bad_descriptors(bad, code):
    d = desc(**bad)
    assert gdn.lib().gdn_qk_norm_rope_bwd_workspace_size(ctypes.byref(d)) == 0
    assert fwd(d) == code and bwd(d) == code


def test_null_and_misaligned_pointers():
    d = desc()
    for call, names in ((fwd, ("q", "k", "qo", "ko")), (bwd, ("q", "k", "dqo", "dko", "dq", "dk"))):
        for name in names:
            assert call(d, **{name: None}) == 1
            assert call(d, **{name: FAKE + 8}) == 3
        for name in ("pos", "inv_freq", "qw", "kw"):
            assert call(d, **{name: FAKE + 2}) == 3
        assert call(d, inv_freq=None) == 1
    assert bwd(d, dqw=FAKE + 2) == 3 and bwd(d, dkw=FAKE + 2) == 3


def test_workspace_of_the_backward():
    d = desc()
    need = gdn.lib().gdn_qk_norm_rope_bwd_workspace_size(ctypes.byref(d))
    assert need > 0
    assert bwd(d, ws=None) == 4
    assert bwd(d, ws=FAKE + 16) == 3
    assert bwd(d, ws_bytes=need - 1) == 4


def test_binding_refuses_before_any_call():
    q = torch.zeros(1, 8, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_qk_norm_rope_fwd(q, q)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_qk_norm_rope_bwd(q, q, q, q)


def test_head_strides():
    from gated_delta_rule_99_b200._binding import _row_stride
    stride = lambda t: _row_stride(t, "q", torch.float32, tuple(t.shape))
    wide = torch.zeros(2, 5, 40)
    assert stride(wide[..., 8:24].unflatten(-1, (2, 8))) == 40
    for bad in (wide.unflatten(-1, (5, 8))[:, :, ::2], wide.unflatten(-1, (5, 8))[..., :4],
                torch.zeros(2, 3, 5, 8).transpose(1, 2)):
        with pytest.raises(ValueError):
            stride(bad)


def test_refusals_do_not_depend_on_earlier_calls():
    """Descriptors are kept by what they are made of; a call that is refused the first time is refused after
    a like one that was not."""
    from gated_delta_rule_99_b200._binding import _qk_plan
    q, f = torch.zeros(1, 3, 2, 64), torch.zeros(32)
    plan = lambda f: _qk_plan(q, q, f, "rms", None, False, -1, (None, None), (None, None))
    for _ in range(2):
        assert plan(f)[0].rot == 64 and plan(None)[0].rot == 0 and plan(f[:0])[0].rot == 0
        with pytest.raises(ValueError, match="inv_freq must have one dimension"):
            plan(f.view(2, 16))
