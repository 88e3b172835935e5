"""Norms of queries and keys with the position rotation, forward and gradient,
against the float64 oracle on the same inputs.

Tolerances.  u = 2^-24 is fp32's half step, t that of the output's type
(torch.finfo(t).eps / 2).  Forward: an entry is x_i inv w_i cos -+ x_m inv w_m
sin.  inv carries the sum of at most 64 squares (per lane at most 8, then 5
levels of a tree, each u) and the reciprocal root (2 steps); the fraction of a
turn is rounded once to fp32 (u of at most pi/2 after the doubling) and sine
and cosine are within 2 steps; weights, products and the sum add 4 roundings:
under 32 u (|u_i| + |u_m|) <= 64 u max|u|, plus one rounding to the type.
Gradient: g = du w has the same 32 u relative to the row's largest |g|, the
projection a sum over 64 products: under 128 u max|g| sqrt(d) inv in all.
Weight gradients are sums of at most M = tokens x heads terms: (M + 64) u sum
of |terms|."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from recurrent_states_b200 import taylor_attn as TA
from tests.gpu_common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FORWARD = {"bf16": TA.taylor_attn_qk_norm_rope, "f32": TA.taylor_attn_qk_norm_rope_f32}
BACKWARD = {"bf16": TA.taylor_attn_qk_norm_rope_backward, "f32": TA.taylor_attn_qk_norm_rope_backward_f32}


def _half(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def _inputs(dtype, B, N, Hq, Hk, d, seed, packed=False, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    if packed:
        rows = (scale * torch.randn(B, N, (Hq + Hk) * d + 3 * d, generator=g)).to(t).to(DEV)
        q = rows[..., :Hq * d].unflatten(-1, (Hq, d))
        k = rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    else:
        q = (scale * torch.randn(B, N, Hq, d, generator=g)).to(t).to(DEV)
        k = (scale * torch.randn(B, N, Hk, d, generator=g)).to(t).to(DEV)
    dqo = torch.randn(B, Hq, N, d, generator=g).to(t).to(DEV)
    dko = torch.randn(B, Hk, N, d, generator=g).to(t).to(DEV)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(DEV) for _ in range(2)]
    pos = torch.randint(-5, 100_000, (B, N), generator=g).to(DEV)
    return q, k, dqo, dko, w, pos


def _check_forward(got, x, freqs, pos, w, inter, eps, dtype):
    want = L.norm_rope(f64(x), freqs, pos, None if w is None else f64(w), inter, eps)
    big = np.abs(want).max(-1, keepdims=True) * np.sqrt(2)
    err = np.abs(f64(got) - want)
    limit = _half(dtype) * np.abs(want) * (1 + 1e-3) + 64 * U * big if dtype == "bf16" else 64 * U * big
    assert (err <= limit).all(), float((err / np.where(limit > 0, limit, 1)).max())


def _check_backward(dx, dw, x, dy, freqs, pos, w, inter, eps, dtype):
    wd = None if w is None else f64(w)
    want, wantw = L.norm_rope_grad(f64(x), f64(dy), freqs, pos, wd, inter, eps)
    xd, d = f64(x), x.shape[-1]
    inv = L._inv(xd, eps)
    R = L.rotation(pos, freqs, d, inter)
    du = np.einsum("bnij,bhni->bnhj", R, f64(dy))
    g = du if wd is None else du * wd
    big = np.abs(g).max(-1, keepdims=True) * np.sqrt(2 * d) * inv
    limit = 128 * U * big + (_half(dtype) * np.abs(want) * (1 + 1e-3) if dtype == "bf16" else 0)
    err = np.abs(f64(dx) - want)
    assert (err <= limit).all(), float((err / np.where(limit > 0, limit, 1)).max())
    if w is None:
        assert dw is None
    else:
        terms = np.abs(du * xd * inv).sum((0, 1, 2))
        M = x.shape[0] * x.shape[1] * x.shape[2]
        assert (np.abs(f64(dw) - wantw) <= (M + 64) * U * terms).all()


CASES = [
    # B, N, Hq, Hk, d, rot, interleaved, weights, packed, eps
    (1, 1, 1, 1, 16, 16, False, False, False, 0.0),
    (64, 1, 16, 16, 16, 16, False, False, True, 0.0),     # one decode step
    (2, 100, 8, 8, 16, 16, False, True, True, 0.0),
    (1, 333, 4, 4, 64, 64, False, True, False, 1e-6),
    (2, 37, 3, 1, 64, 64, True, True, True, 0.0),
    (1, 129, 5, 2, 32, 16, False, False, True, 0.0),      # half of each row rotated
    (3, 77, 6, 2, 20, 12, True, True, False, 0.0),
    (2, 50, 2, 2, 24, 24, False, True, True, 1e-5),
    (1, 65, 3, 3, 7, 6, False, True, True, 0.0),          # odd d: element by element
    (2, 31, 2, 2, 63, 62, True, True, False, 0.0),
    (1, 40, 2, 2, 64, 0, False, True, False, 0.0),        # no rotation
    (1, 33, 1, 1, 1, 0, False, True, False, 0.1),
    (2, 20, 2, 2, 2, 2, False, False, True, 0.0),
    (2, 45, 3, 3, 34, 34, False, True, True, 0.0),        # pairs a multiple of one entry apart
    (1, 60, 2, 4, 40, 36, True, False, True, 0.0),
    (1, 700, 31, 1, 48, 32, False, True, False, 0.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,inter,weights,packed,eps", CASES)
def test_forward_and_gradient_match_the_oracle(dtype, B, N, Hq, Hk, d, rot, inter, weights, packed, eps):
    q, k, dqo, dko, (qw, kw), pos = _inputs(dtype, B, N, Hq, Hk, d, seed=N + d, packed=packed)
    qw, kw = (qw, kw) if weights else (None, None)
    freqs = TA.rope_freqs(rot)
    more = dict(positions=pos, q_weight=qw, k_weight=kw, interleaved=inter, eps=eps)
    qo, ko = FORWARD[dtype](q, k, freqs, **more)
    p = pos.cpu().numpy()
    eps32 = float(np.float32(eps))
    _check_forward(qo, q, freqs, p, qw, inter, eps32, dtype)
    _check_forward(ko, k, freqs, p, kw, inter, eps32, dtype)
    dq, dk, dqw, dkw = BACKWARD[dtype](q, k, dqo, dko, freqs, **more)
    _check_backward(dq, dqw, q, dqo, freqs, p, qw, inter, eps32, dtype)
    _check_backward(dk, dkw, k, dko, freqs, p, kw, inter, eps32, dtype)


def test_positions_default_to_the_token_plus_an_offset():
    q, k, *_ = _inputs("f32", 2, 19, 2, 2, 16, seed=1)
    freqs = TA.rope_freqs(16)
    p = (torch.arange(19) + 1000)[None].expand(2, 19).contiguous().to(DEV)
    a = TA.taylor_attn_qk_norm_rope_f32(q, k, freqs, positions=p)
    b = TA.taylor_attn_qk_norm_rope_f32(q, k, freqs, pos0=1000)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [16, 9])
def test_far_positions_keep_their_angles(d):
    """2^31 + 7 turns of the fastest pair: fp32 angles would be off by hundreds of radians."""
    q, k, *_ = _inputs("f32", 1, 3, 1, 1, d, seed=2)
    pos = torch.tensor([[0, 2 ** 31 + 7, 2 ** 40 + 3]], device=DEV)
    freqs = TA.rope_freqs(d // 2 * 2)
    qo, _ = TA.taylor_attn_qk_norm_rope_f32(q, k, freqs, positions=pos)
    # an angle of 2^40 radians carries 2^40 2^-53 of rounding in the oracle and 2 pi 2^-53 of its turns in the kernel
    want = L.norm_rope(f64(q), freqs, pos.cpu().numpy())
    assert np.abs(f64(qo) - want).max() <= 64 * U * np.sqrt(2) + 4 * 2.0 ** -13


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 13])
def test_rows_of_zeros_and_of_extreme_size(dtype, d):
    q, k, dqo, dko, (qw, kw), pos = _inputs(dtype, 1, 8, 2, 2, d, seed=5)
    q, k = q.clone(), k.clone()
    q[0, 1, 0] = 0
    scales = [1e-30, 1e30, 1e-22, 1e19, 3e37, 1.0]
    for i, s in enumerate(scales):
        k[0, i, 1] = (k[0, i, 1].float() * s).clamp(-3e38, 3e38).to(k.dtype)
    freqs = TA.rope_freqs(d // 2 * 2)
    qo, ko = FORWARD[dtype](q, k, freqs, positions=pos)
    assert (qo[0, 0, 1] == 0).all()
    p = pos.cpu().numpy()
    _check_forward(qo, q, freqs, p, None, False, 0.0, dtype)
    _check_forward(ko, k, freqs, p, None, False, 0.0, dtype)
    dq, dk, _, _ = BACKWARD[dtype](q, k, dqo, dko, freqs, positions=pos)
    assert (dq[0, 1, 0] == 0).all()
    assert torch.isfinite(dk).all() and torch.isfinite(ko).all()
    _check_backward(dk[:, 5:], None, k[:, 5:], dko[:, :, 5:], freqs, p[:, 5:], None, False, 0.0, dtype)


# The size of a row, and eps beside it: eps that outweighs the row, that is of its order, and that is nothing beside it;
# squares that leave fp32's range in either direction, and an eps that does so too.  Gradients stay inside the types'
# range: dy / |x| at most 1e31.  Beside eps 1e38 a row of 1e-20 has outputs of 1e-39, below the types' normal numbers,
# where a half step is h = 2^-150 in fp32 and 2^-134 in bf16 whatever the value: the row scaled by sqrt(eps) is rounded
# to its type and enters as two entries times cosine, sine and weight (sqrt(2) max|w| h), the output is rounded (h).
EXTREME = [(0.0, [1e-30, 1e-22, 1e-16, 1e19, 1e30, 1.0]),
           (1e-6, [1e-22, 1e-23, 1e-24, 1e-30, 1e-36, 1e-4, 1e20]),
           (1e-5, [1e-25, 1e-33, 1e-18, 1e-2]),
           (1.0, [1e-20, 1e-21, 1e-36, 1e18, 1e30]),
           (1e-31, [1e-24, 1e-17, 1e-15, 1e-12, 1e-36]),
           (1e-38, [1e-19, 1e-20, 1e-30, 1e-36, 1.0]),
           (1e38, [1e-20, 1.0, 1e18, 1e19, 1e24])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,inter", [(16, False), (64, True), (20, False), (13, False), (41, True)])
@pytest.mark.parametrize("eps,scales", EXTREME)
def test_rows_of_extreme_size_with_and_without_eps(dtype, d, inter, eps, scales):
    """Outputs and every row's gradient, weights' gradients among them, for rows in pieces and element by element."""
    N = len(scales) + 2
    q, k, dqo, dko, (qw, kw), pos = _inputs(dtype, 2, N, 2, 3, d, seed=d)
    for x in (q, k):
        for i, s in enumerate(scales):
            x[0, i, 1] = (x[0, i, 1].double() * s).to(x.dtype)
            x[1, i + 1] = (x[1, i + 1].double() * s).to(x.dtype)
        x[1, 0, 0] = 0
    freqs, p, eps32 = TA.rope_freqs(d // 2 * 2), pos.cpu().numpy(), float(np.float32(eps))
    more = dict(positions=pos, q_weight=qw, k_weight=kw, interleaved=inter, eps=eps)
    qo, ko = FORWARD[dtype](q, k, freqs, **more)
    h = 2.0 ** -134 if dtype == "bf16" else 2.0 ** -150
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want = L.norm_rope(f64(x), freqs, p, f64(w), inter, eps32)
        limit = 64 * U * 2 ** 0.5 * np.abs(want).max(-1, keepdims=True) + (1 + 2 ** 0.5 * float(w.abs().max())) * h
        if dtype == "bf16":
            limit = limit + _half(dtype) * np.abs(want) * (1 + 1e-3)
        assert (np.abs(f64(got) - want) <= limit).all(), float((np.abs(f64(got) - want) / limit).max())
    dq, dk, dqw, dkw = BACKWARD[dtype](q, k, dqo, dko, freqs, **more)
    _check_backward(dq, dqw, q, dqo, freqs, p, qw, inter, eps32, dtype)
    _check_backward(dk, dkw, k, dko, freqs, p, kw, inter, eps32, dtype)
    plain = dict(positions=pos, interleaved=inter, eps=eps)
    dq, dk, _, _ = BACKWARD[dtype](q, k, dqo, dko, freqs, **plain)
    _check_backward(dq, None, q, dqo, freqs, p, None, inter, eps32, dtype)
    _check_backward(dk, None, k, dko, freqs, p, None, inter, eps32, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,inter", [(16, 16, False), (16, 16, True), (64, 64, False), (24, 14, True), (34, 34, False)])
def test_tokens_that_do_not_exist_leave_the_weight_gradients_alone(dtype, d, rot, inter):
    """A few tokens fill a part of a CTA; the rest of its angles' places hold what the call before left there: NaN, from
    frequencies whose angles overflow."""
    q, k, dqo, dko, (qw, kw), pos = _inputs(dtype, 1, 3, 1, 2, d, seed=d)
    many = _inputs(dtype, 4, 4096, 1, 2, d, seed=1)
    freqs, p = TA.rope_freqs(rot), pos.cpu().numpy()
    for _ in range(3):
        bad = BACKWARD[dtype](*many[:4], np.full(rot // 2, 1e308), pos0=1 << 40, q_weight=qw, k_weight=kw, interleaved=inter)
        assert torch.isnan(bad[0]).any()
        dq, dk, dqw, dkw = BACKWARD[dtype](q, k, dqo, dko, freqs, positions=pos, q_weight=qw, k_weight=kw, interleaved=inter)
        _check_backward(dq, dqw, q, dqo, freqs, p, qw, inter, 0.0, dtype)
        _check_backward(dk, dkw, k, dko, freqs, p, kw, inter, 0.0, dtype)


def test_gradients_into_slices_of_a_packed_gradient():
    B, N, H, d = 2, 21, 4, 16
    q, k, dqo, dko, (qw, kw), pos = _inputs("bf16", B, N, H, H, d, seed=8)
    freqs = TA.rope_freqs(d)
    want = TA.taylor_attn_qk_norm_rope_backward(q, k, dqo, dko, freqs, positions=pos, q_weight=qw, k_weight=kw)
    rows = torch.full((B, N, 3 * H * d), 7.0, dtype=torch.bfloat16, device=DEV)
    dq, dk = (rows[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(2))
    got = TA.taylor_attn_qk_norm_rope_backward(q, k, dqo, dko, freqs, positions=pos, q_weight=qw, k_weight=kw, dq=dq,
                                               dk=dk)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert (rows[..., 2 * H * d:] == 7).all()


def test_odd_offsets_and_head_major_inputs():
    """Rows that start at an odd element, and inputs that are head-major already."""
    g = torch.Generator().manual_seed(3)
    flat = torch.randn(1 + 2 * 9 * 3 * 16, generator=g).bfloat16().to(DEV)
    q = flat[1:].view(2, 9, 3, 16)
    freqs = TA.rope_freqs(16)
    want = TA.taylor_attn_qk_norm_rope(q.clone(), q.clone(), freqs)
    got = TA.taylor_attn_qk_norm_rope(q, q, freqs)
    for x, y in zip(want, got):
        torch.testing.assert_close(x, y, rtol=2.0 ** -7, atol=0)
    major = q.transpose(1, 2).contiguous().transpose(1, 2)
    got = TA.taylor_attn_qk_norm_rope(major, major, freqs)
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_empty_calls():
    e = torch.empty((2, 0, 3, 16), dtype=torch.bfloat16, device=DEV)
    qo, ko = TA.taylor_attn_qk_norm_rope(e, e, TA.rope_freqs(16))
    assert qo.shape == (2, 3, 0, 16)
    w = torch.ones(16, device=DEV)
    _, _, dw, _ = TA.taylor_attn_qk_norm_rope_backward(e, e, qo, ko, TA.rope_freqs(16), q_weight=w)
    assert (dw == 0).all()
    k0 = torch.empty((2, 5, 0, 16), dtype=torch.bfloat16, device=DEV)
    q = torch.randn(2, 5, 3, 16, device=DEV).bfloat16()
    qo, ko = TA.taylor_attn_qk_norm_rope(q, k0, TA.rope_freqs(16))
    want, _ = TA.taylor_attn_qk_norm_rope(q, q, TA.rope_freqs(16))
    assert torch.equal(qo, want) and ko.numel() == 0
    for d in (16, 7):   # keys alone, in pieces and element by element
        k, none = torch.randn(2, 5, 3, d, device=DEV).bfloat16(), torch.empty((2, 5, 0, d), dtype=torch.bfloat16, device=DEV)
        both = TA.taylor_attn_qk_norm_rope(k, k, TA.rope_freqs(d // 2 * 2))
        qo, ko = TA.taylor_attn_qk_norm_rope(none, k, TA.rope_freqs(d // 2 * 2))
        assert qo.numel() == 0 and torch.equal(ko, both[1])
        w = torch.ones(d, device=DEV)
        more = dict(q_weight=w, k_weight=w)
        _, dk, dqw, dkw = TA.taylor_attn_qk_norm_rope_backward(none, k, qo, ko, TA.rope_freqs(d // 2 * 2), **more)
        _, dk2, _, dkw2 = TA.taylor_attn_qk_norm_rope_backward(k, k, ko, ko, TA.rope_freqs(d // 2 * 2), **more)
        assert torch.equal(dk, dk2) and (dqw == 0).all()
        torch.testing.assert_close(dkw, dkw2, rtol=1e-5, atol=1e-5)


def test_streams_graphs_and_repeats():
    """Two captured graphs whose workspaces come from one pool, replayed in turn
    and on other inputs, and a call on another stream: the same bits."""
    freqs = TA.rope_freqs(64)
    sets = [_inputs("bf16", 2, 200, 4, 4, 64, seed=s) for s in (1, 2)]
    call = lambda s: TA.taylor_attn_qk_norm_rope_backward(  # noqa: E731
        s[0], s[1], s[2], s[3], freqs, positions=s[5], q_weight=s[4][0], k_weight=s[4][1])
    want = [[t.clone() for t in call(s)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = TA.taylor_attn_qk_norm_rope_backward(*sets[0][:4], freqs, positions=sets[0][5], q_weight=sets[0][4][0],
                                               k_weight=sets[0][4][1], stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[0], got))
    graphs, outs = [], []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(s))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, y) for x, y in zip(w, o))
    sets[0][0].copy_(sets[1][0])
    graphs[0].replay()
    fresh = call(sets[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(fresh, outs[0]))
