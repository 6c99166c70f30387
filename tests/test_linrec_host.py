"""Host side of the gated linear recurrence: its fp64 form pinned by closed forms and differences,
and every refusal of the C ABI and the binding, which come before anything touches a GPU."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_99_b200 as gdn
from oracle import linrec as ref

FAKE = 0x7F0000000000  # a 256-byte aligned address that is never dereferenced


def test_oracle_equals_the_weighted_sum_of_all_earlier_tokens():
    rng = np.random.default_rng(0)
    T, D = 11, 3
    x, g, h0 = rng.standard_normal((T, D)), -rng.random((T, D)), rng.standard_normal((2, D))
    for complement in (False, True):
        w = 1 - np.exp(g) if complement else np.ones((T, D))
        o, hT, before, *_ = ref.fwd(x, g, h0, [(0, 7), (7, 11)], complement)
        for n, (t0, t1) in enumerate([(0, 7), (7, 11)]):
            for t in range(t0, t1):
                want = h0[n] * np.exp(g[t0:t + 1].sum(0))
                for j in range(t0, t + 1):
                    want = want + np.exp(g[j + 1:t + 1].sum(0)) * w[j] * x[j]
                assert np.allclose(o[t], want, rtol=1e-13, atol=1e-13)
                assert np.allclose(before[t], h0[n] if t == t0 else o[t - 1], rtol=0, atol=0)
            assert np.array_equal(hT[n], o[t1 - 1])


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(1)
    T, D = 9, 2
    segs = [(0, 4), (4, 4), (4, 9)]
    x, g, do = (rng.standard_normal((T, D)) for _ in range(3))
    h0, dhT = rng.standard_normal((3, D)), rng.standard_normal((3, D))
    for complement in (False, True):
        def loss(x, g, h0):
            o, hT = ref.fwd(x, g, h0, segs, complement)[:2]
            return (do * o).sum() + (dhT * hT).sum()

        grads, _ = ref.bwd(x, g, h0, do, dhT, segs, complement)
        for i, grad in enumerate(grads):
            base = [x, g, h0]
            for at in np.ndindex(base[i].shape):
                hi, lo = base[i].copy(), base[i].copy()
                hi[at] += 1e-6
                lo[at] -= 1e-6
                d = (loss(*[hi if j == i else b for j, b in enumerate(base)]) -
                     loss(*[lo if j == i else b for j, b in enumerate(base)])) / 2e-6
                assert abs(grad[at] - d) < 1e-7 * (1 + abs(d))


def desc(**kw):
    f = dict(B=2, T=100, D=40, n_seqs=0, x_stride=0, g_stride=0, o_stride=0, dx_stride=0,
             dg_stride=0, dtype=0, g_dtype=0, flags=0, reserved=0)
    f.update(kw)
    return gdn.GdnLinrecDesc(*f.values())


def fwd(d, cu=None, cu_host=None, **kw):
    p = dict(x=FAKE, g=FAKE, h0=None, o=FAKE, hT=None, states=None)
    p.update(kw)
    return gdn.lib().gdn_linrec_fwd(ctypes.byref(d), p["x"], p["g"], cu, cu_host, p["h0"], p["o"],
                                    p["hT"], p["states"], None)


def bwd(d, cu=None, cu_host=None, ws=FAKE, ws_bytes=1 << 40, **kw):
    p = dict(x=FAKE, g=FAKE, h0=None, do=FAKE, dhT=None, dx=FAKE, dg=FAKE, dh0=None, states=None)
    p.update(kw)
    return gdn.lib().gdn_linrec_bwd(ctypes.byref(d), p["x"], p["g"], cu, cu_host, p["h0"], p["do"],
                                    p["dhT"], p["dx"], p["dg"], p["dh0"], p["states"], ws, ws_bytes,
                                    None)


def decode(d, **kw):
    p = dict(x=FAKE, g=FAKE, state=FAKE, o=FAKE)
    p.update(kw)
    return gdn.lib().gdn_linrec_decode(ctypes.byref(d), *p.values(), None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(D=(1 << 20) + 1), 1), (dict(n_seqs=-1), 1),
    (dict(n_seqs=2), 1), (dict(B=1 << 20, T=1 << 11), 1), (dict(B=1 << 40, T=1 << 40), 1),
    (dict(dtype=2), 2), (dict(g_dtype=2), 2), (dict(dtype=1, g_dtype=0), 2), (dict(flags=2), 1),
    (dict(reserved=1), 1), (dict(x_stride=39), 1), (dict(g_stride=-40), 1), (dict(o_stride=1), 1),
    (dict(dx_stride=39), 1), (dict(dg_stride=1 << 31), 1)])
def test_bad_descriptors(bad, code):
    d = desc(**bad)
    assert gdn.lib().gdn_linrec_states_size(ctypes.byref(d)) == 0
    assert fwd(d) == code and bwd(d) == code and decode(d) == code
    assert gdn.lib().gdn_linrec_states_size(None) == 0


def test_null_and_misaligned_pointers():
    d = desc()
    for name in ("x", "g", "o"):
        assert fwd(d, **{name: None}) == 1
        assert fwd(d, **{name: FAKE + 8}) == 3
    for name in ("h0", "hT", "states"):
        assert fwd(d, **{name: FAKE + 4}) == 3
    for name in ("x", "g", "do", "dx", "dg"):
        assert bwd(d, **{name: None}) == 1
        assert bwd(d, **{name: FAKE + 2}) == 3
    for name in ("h0", "dhT", "dh0", "states"):
        assert bwd(d, **{name: FAKE + 4}) == 3
    for name in ("x", "g", "state", "o"):
        assert decode(d, **{name: None}) == 1
        assert decode(d, **{name: FAKE + 8}) == 3


def test_states_in_place_are_refused():
    assert fwd(desc(), h0=FAKE, hT=FAKE) == 1
    assert bwd(desc(), dhT=FAKE, dh0=FAKE) == 1


def test_workspace_of_the_backward():
    d = desc(T=200)
    need = gdn.lib().gdn_linrec_states_size(ctypes.byref(d))
    assert need >= 2 * 2 * 40 * 4
    assert bwd(d, ws=None) == 4
    assert bwd(d, ws=FAKE + 16) == 3
    assert bwd(d, ws_bytes=need - 1) == 4


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 100], [0, 50, 99], [0, 50, 101]])
def test_bad_document_offsets(cu):
    d = desc(B=1, n_seqs=len(cu) - 1)
    host = ctypes.cast((ctypes.c_int32 * len(cu))(*cu), ctypes.c_void_p)
    assert fwd(d, cu=FAKE, cu_host=host) == 1 and bwd(d, cu=FAKE, cu_host=host) == 1


def test_document_offsets_need_the_device_copy_and_a_packed_descriptor():
    host = ctypes.cast((ctypes.c_int32 * 3)(0, 40, 100), ctypes.c_void_p)
    packed = desc(B=1, n_seqs=2)
    assert fwd(packed, cu=None, cu_host=host) == 1 and bwd(packed, cu=None, cu_host=host) == 1
    assert fwd(packed, cu=FAKE + 2, cu_host=host) == 3
    assert fwd(desc(B=1), cu=FAKE, cu_host=host) == 1
    assert decode(desc(B=1, n_seqs=1)) == 1 and decode(desc(T=0)) == 1


def test_states_size_counts_every_tile():
    size = lambda **kw: gdn.lib().gdn_linrec_states_size(ctypes.byref(desc(**kw)))
    assert size(B=1, T=0) == 256
    for B, T, D in ((1, 4096, 2048), (3, 1237, 515), (1, 1 << 20, 1024), (1024, 8, 64)):
        tiles = -(-T // 64) * B if T > 64 else 0  # a shorter row starts within its tile
        assert size(B=B, T=T, D=D) >= 4 * D * tiles


def test_binding_refuses_before_any_call():
    x = torch.zeros(1, 8, 16)
    for call in (lambda: gdn.gdn_linrec_fwd(x, x), lambda: gdn.gdn_linrec_bwd(x, x, x),
                 lambda: gdn.gdn_linrec_decode(x, x, torch.zeros(1, 16))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_token_strides():
    from gated_delta_rule_99_b200._binding import _row_stride

    def stride(t, shape=None):
        return _row_stride(t, "x", torch.float32, tuple(shape or t.shape))

    wide = torch.zeros(2, 5, 24)
    assert stride(wide) == 0 and stride(wide[..., 8:16]) == 24
    assert stride(wide[:, :1, :8]) == 120 and stride(wide[:1, :, :8]) == 24
    assert stride(wide[:1, :1, :8]) in (0, 8)
    for bad in (wide.transpose(1, 2), wide[..., ::2], wide[:, :4], wide[:1, :1].expand(2, 5, 24),
                wide[:, :1].expand(2, 5, 24), wide[..., :1].expand(2, 5, 24)):
        with pytest.raises(ValueError):
            stride(bad)
    with pytest.raises(ValueError):
        stride(wide, (2, 5, 25))
    with pytest.raises(ValueError):
        _row_stride(wide, "x", torch.bfloat16, (2, 5, 24))


def test_the_mirror_of_the_offsets_must_be_on_the_host():
    from gated_delta_rule_99_b200._binding import _offsets, _seqlens

    cu = torch.tensor([0, 3, 8], dtype=torch.int32)
    elsewhere = torch.empty(3, dtype=torch.int32, device="meta")  # no host address either
    for call in (lambda: _offsets(cu, elsewhere, -1), lambda: _offsets(None, elsewhere, 0),
                 lambda: _offsets(cu.long(), elsewhere, 0), lambda: _seqlens(cu, elsewhere, "cpu"),
                 lambda: _seqlens(None, elsewhere.long(), "cpu")):
        with pytest.raises(ValueError, match="cu_seqlens_host must be a CPU tensor"):
            call()
    assert _offsets(cu, cu.clone(), -1)[3] == 2


def test_the_status_is_read_on_the_device_of_the_calls(monkeypatch):
    """The calls run on their tensors' device, whatever the current one is; so does the read of
    their status.  Two devices, with a timeout on the second one."""
    from gated_delta_rule_99_b200 import _binding

    class Stream:
        def __init__(self, index, handle):
            self.device, self.cuda_stream = torch.device("cuda", index), handle

    class Device:
        current = 0

        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, Device.current = Device.current, self.index

        def __exit__(self, *exc):
            Device.current = self.before

    class Lib:
        calls = []

        def gdn_linrec_status(self, stream):
            self.calls.append((Device.current, stream.value))
            return 6 if Device.current == 1 else 0

    def current_stream(device=None):
        index = Device.current if device is None else device if isinstance(device, int) else device.index
        return Stream(index, 100 + index)

    monkeypatch.setattr(_binding, "lib", Lib)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "device", Device)
    assert gdn.linrec_status() == 0
    assert gdn.linrec_status(Stream(1, 7)) == 6 and gdn.linrec_status(stream=Stream(0, 9)) == 0
    assert gdn.linrec_status(device=1) == 6 and gdn.linrec_status(device=torch.device("cuda", 1)) == 6
    assert Lib.calls == [(0, 100), (1, 7), (0, 9), (1, 101), (1, 101)] and Device.current == 0


def test_offsets_too_many_for_the_host_are_an_error_code():
    """Without the mirror the offsets are copied to the host: where their memory cannot be had, the call
    returns an error, and the process goes on.  In a process of its own, whose address space is limited."""
    import os
    import subprocess
    import sys
    code = """
import ctypes, resource
import gated_delta_rule_99_b200 as gdn
L, fake, n = gdn.lib(), 0x7F0000000000, 1 << 29
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (1 << 30), used + (1 << 30)))
d = gdn.make_desc(1, 100, 1, 64, 64, n_seqs=n)
print(L.gdn_fwd(ctypes.byref(d), fake, fake, fake, fake, fake, fake, None, None, fake, None, fake, 1 << 60, None))
d = gdn.GdnLinrecDesc(1, 100, 64, (1 << 31) - 1, 0, 0, 0, 0, 0, 0, 0, 0, 0)
print(L.gdn_linrec_fwd(ctypes.byref(d), fake, fake, fake, None, None, fake, None, None, None))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.split() == ["5", "5"], r.stdout + r.stderr[-2000:]


def test_device_offsets_must_be_as_many_as_the_mirrors():
    from gated_delta_rule_99_b200._binding import _seqlens

    class OnDevice(torch.Tensor):
        is_cuda = True

    cu = torch.tensor([0, 3, 8, 9], dtype=torch.int32)
    with pytest.raises(ValueError, match="3 values, its host mirror 4"):
        _seqlens(cu[:3].as_subclass(OnDevice), cu, "cpu")
    assert _seqlens(cu.as_subclass(OnDevice), cu[:3], "cpu")[1].numel() == 3
