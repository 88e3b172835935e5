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
