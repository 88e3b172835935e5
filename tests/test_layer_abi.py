"""Refusals of the operators around the attention, on the host: status codes
before any device call, and the binding's own checks."""
import ctypes

import numpy as np
import pytest
import torch

from recurrent_states_b200 import build as B
from recurrent_states_b200 import taylor_attn as TA


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


P = 1 << 20  # an aligned, never-dereferenced address
INV, UNS, MIS, OK = TA.TAYLOR_ERR_INVALID_ARG, TA.TAYLOR_ERR_UNSUPPORTED, TA.TAYLOR_ERR_MISALIGNED, TA.TAYLOR_OK


def _three(*v):
    return (ctypes.c_int64 * 3)(*v)


def _qk(backward=False, **over):
    """Status of one call with everything in order but what `over` says."""
    N, H, d = 5, 2, 16
    a = dict(q=P, k=P, dqo=P, dko=P, qw=None, kw=None, pos=None, pos0=0, rot=16, inter=0, yq=P, yk=P, dqw=None,
             dkw=None, B=1, N=N, Hq=H, Hk=H, d=d, qs=_three(N * H * d, H * d, d), ks=_three(N * H * d, H * d, d),
             dqs=_three(N * H * d, H * d, d), dks=_three(N * H * d, H * d, d), eps=0.0,
             freqs=np.ones(32))
    a.update(over)
    f = a["freqs"]
    f = None if f is None else f.ctypes.data
    grads = [a["dqo"], a["dko"]] if backward else []
    weights = [a["dqw"], a["dkw"]] if backward else []
    ys = [a["dqs"], a["dks"]] if backward else []
    fn = TA.lib().taylor_attn_qk_norm_rope_backward if backward else TA.lib().taylor_attn_qk_norm_rope
    return fn(a["q"], a["k"], *grads, a["qw"], a["kw"], a["pos"], a["pos0"], f, a["rot"], a["inter"], a["yq"],
              a["yk"], *weights, a["B"], a["N"], a["Hq"], a["Hk"], a["d"], a["qs"], a["ks"], *ys, a["eps"], None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(d=0), UNS), (dict(d=65), UNS), (dict(rot=17), UNS), (dict(rot=18), UNS), (dict(rot=15), UNS),
    (dict(rot=-2), INV), (dict(B=-1), INV), (dict(N=-1), INV), (dict(Hk=-1), INV), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(freqs=None), INV),
    (dict(freqs=np.full(32, np.inf)), INV), (dict(q=None), INV), (dict(yk=None), INV), (dict(qs=None), INV),
    (dict(q=P + 1), MIS), (dict(yq=P + 1), MIS), (dict(qw=P + 2), MIS), (dict(pos=P + 4), MIS),
    (dict(qs=_three(160, -32, 16)), INV), (dict(B=1 << 20, N=1 << 11), UNS),
    (dict(B=1 << 15, N=1 << 15, Hq=1 << 2), UNS),
    (dict(B=0, q=None), OK), (dict(N=0, yk=None), OK), (dict(Hq=0, Hk=0, q=None, k=None), OK),
])
def test_qk_norm_rope_refuses(backward, over, status):
    assert _qk(backward, **over) == status


def test_qk_norm_rope_backward_refuses_more():
    assert _qk(True, dqo=None) == INV and _qk(True, dks=None) == INV and _qk(True, dko=P + 1) == MIS
    assert _qk(True, dqw=P) == INV                       # a weight's gradient without the weight
    assert _qk(True, dqs=_three(160, 16, 16)) == INV     # tokens on top of heads
    assert _qk(True, dks=_three(0, 0, 0)) == INV


def test_binding_refuses_cpu_tensors():
    q = torch.zeros(1, 2, 3, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        TA.taylor_attn_qk_norm_rope(q, q, TA.rope_freqs(16))


def test_rope_freqs():
    np.testing.assert_allclose(TA.rope_freqs(4, 100.0), [1.0, 0.1])
    assert len(TA.rope_freqs(0)) == 0


def _two(*v):
    return (ctypes.c_int64 * 2)(*v)


def _scan(backward=False, **over):
    B, N, D = 2, 5, 8
    a = dict(gate=P, x=P, h=P, dh=P, h0=None, lengths=None, dl=None, y=P, dgate=P, dx=P, end=None, B=B, N=N, D=D,
             gs=_two(N * D, D), xs=_two(N * D, D), dgs=_two(N * D, D), dxs=_two(N * D, D))
    a.update(over)
    L = TA.lib()
    if backward:
        return L.taylor_attn_gated_scan_backward(a["gate"], a["x"], a["h"], a["dh"], a["h0"], a["lengths"], a["dl"],
                                                 a["dgate"], a["dx"], a["end"], a["B"], a["N"], a["D"], a["gs"],
                                                 a["xs"], a["dgs"], a["dxs"], 1, None)
    return L.taylor_attn_gated_scan(a["gate"], a["x"], a["h0"], a["lengths"], a["y"], a["end"], a["B"], a["N"],
                                    a["D"], a["gs"], a["xs"], 1, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INV), (dict(N=-1), INV), (dict(D=-1), INV), (dict(gate=None), INV), (dict(x=None), INV),
    (dict(gs=None), INV), (dict(xs=_two(40, -8)), INV), (dict(gate=P + 1), MIS), (dict(h0=P + 2), MIS),
    (dict(lengths=P + 1), MIS), (dict(end=P + 2), MIS), (dict(B=1 << 16, N=1 << 15), UNS),
    (dict(B=1 << 16, D=1 << 15), UNS), (dict(B=0, gate=None), OK), (dict(D=0, x=None), OK),
    (dict(N=0, gate=None, x=None), OK),
])
def test_gated_scan_refuses(backward, over, status):
    assert _scan(backward, **over) == status


def test_gated_scan_refuses_more():
    assert _scan(y=None) == INV
    for name in ("h", "dh", "dgate", "dx", "dgs", "dxs"):
        assert _scan(True, **{name: None}) == INV, name
    assert _scan(True, dgs=_two(0, 8)) == INV and _scan(True, dxs=_two(40, 4)) == INV
    assert _scan(True, dx=P + 1) == MIS and _scan(True, dl=P + 1) == MIS


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INV), (dict(D=-1), INV), (dict(gs=-1), INV), (dict(gate=None), INV), (dict(out=None), INV),
    (dict(state=None), INV), (dict(gate=P + 1), MIS), (dict(state=P + 2), MIS), (dict(B=0, gate=None), OK),
    (dict(D=0, out=None), OK),
])
def test_gated_step_refuses(over, status):
    a = dict(gate=P, x=P, state=P, out=P, B=2, D=8, gs=8, xs=8)
    a.update(over)
    assert TA.lib().taylor_attn_gated_step(a["gate"], a["x"], a["state"], a["state"], a["out"], a["B"], a["D"],
                                           a["gs"], a["xs"], 1, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INV), (dict(H=-1), INV), (dict(cap=-1), INV), (dict(cap=0), INV), (dict(tau=float("inf")), INV),
    (dict(n=0), UNS), (dict(n=6), UNS), (dict(d=65), UNS), (dict(d=0), UNS), (dict(dv=62), UNS), (dict(dv=260), UNS),
    (dict(B=1 << 12, H=1 << 12), UNS), (dict(cap=(1 << 30) + 1), UNS), (dict(q=None), INV), (dict(state=None), INV), (dict(kc=None), INV),
    (dict(lengths=None), INV), (dict(out=None), INV), (dict(vc=P + 8), MIS), (dict(state=P + 4), MIS),
    (dict(lengths=P + 2), MIS), (dict(B=0, q=None), OK), (dict(H=0, out=None), OK),
])
def test_shared_prefix_decode_refuses(over, status):
    a = dict(q=P, k=P, v=P, state=P, kc=P, vc=P, lengths=P, out=P, B=2, H=2, cap=4, d=16, dv=64, n=3, tau=2.0)
    a.update(over)
    assert TA.lib().taylor_attn_shared_prefix_decode(
        a["q"], a["k"], a["v"], a["state"], a["kc"], a["vc"], a["lengths"], a["out"], a["B"], a["H"], a["cap"],
        a["d"], a["dv"], a["n"], a["tau"], None) == status
