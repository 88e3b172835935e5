"""Gated linear recurrence: scan, gradient and step against the float64 oracle.

Tolerances, by running error analysis with u = 2^-24.  e = exp(-gate) is formed
as 2^t: t carries 1 rounding, so e is off by |t| ln 2 u + 2 steps of the
exponential, under 16 u for |gate| <= 10; a = 1 / (1 + e) and 1 - a = e a add 4
more.  Every term of h_t is a product of a's and one b, each factor within 20 u
and each multiplication and addition (of the chunk's sums and of the state
carried in) within u, two of each a step: with the majorant
M_t = a_t M_{t-1} + |b_t| the error obeys E_t = a_t E_{t-1} + 24 u M_t.  The
gradient's G the same, backwards; dgate and dx multiply it by factors within
48 u.  Outputs add half a step of their type.  The gradient takes h as the
forward call stored it."""
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
SCAN = {"bf16": TA.taylor_attn_gated_scan, "f32": TA.taylor_attn_gated_scan_f32}
BACK = {"bf16": TA.taylor_attn_gated_scan_backward, "f32": TA.taylor_attn_gated_scan_backward_f32}
STEP = {"bf16": TA.taylor_attn_gated_step, "f32": TA.taylor_attn_gated_step_f32}


def _half(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def _inputs(dtype, B, N, D, seed, packed=False):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    bias = 1 + 4 * torch.rand(D, generator=g)
    gate, x = (torch.randn(B, N, D, generator=g) + bias).clamp(-9, 9), torch.randn(B, N, D, generator=g)
    if packed:
        rows = torch.cat([x, gate, x[..., :3]], -1).to(t).to(DEV)
        x, gate = rows[..., :D], rows[..., D:2 * D]
    else:
        gate, x = gate.to(t).to(DEV), x.to(t).to(DEV)
    h0 = torch.randn(B, D, generator=g).to(DEV)
    dh = torch.randn(B, N, D, generator=g).to(t).to(DEV)
    dl = torch.randn(B, D, generator=g).to(DEV)
    return gate, x, h0, dh, dl


def _bounds(gate, x, coupled, h0, lengths):
    """Majorants and errors of h [B, N, D] and of the last state."""
    gate, x = f64(gate), np.abs(f64(x))
    B, N, D = gate.shape
    M, E = np.zeros((B, N, D)), np.zeros((B, N, D))
    last = np.zeros((B, D))
    for b in range(B):
        m, e = (np.zeros(D) if h0 is None else np.abs(f64(h0[b]))), np.zeros(D)
        for t in range(N if lengths is None else lengths[b]):
            a = L.sigmoid(gate[b, t])
            m = a * m + (L.sigmoid(-gate[b, t]) * x[b, t] if coupled else x[b, t])
            e = a * e + 24 * U * m
            M[b, t], E[b, t] = m, e
        last[b] = e
    return E, last


def _check(got, want, err, half):
    got, want = f64(got), np.asarray(want)
    off = np.abs(got - want)
    limit = err + half * (np.abs(want) + err)
    assert (off <= limit).all(), float((off / np.where(limit > 0, limit, 1e-300)).max())


def _check_all(dtype, gate, x, h0, dh, dl, coupled, lengths, h, last, dgate, dx, dh0):
    ref_h, ref_last = L.gated_scan(f64(gate), f64(x), coupled, None if h0 is None else f64(h0), lengths)
    E, El = _bounds(gate, x, coupled, h0, lengths)
    half = _half(dtype) if dtype == "bf16" else 0.0
    _check(h, ref_h, E, half)
    _check(last, ref_last, El, 0.0)
    if dgate is None:
        return
    g, xs, hs = f64(gate), f64(x), f64(h)
    want = L.gated_scan_grad(g, xs, f64(dh), coupled, None if h0 is None else f64(h0), lengths,
                             None if dl is None else f64(dl), h=hs)
    B, N, D = g.shape
    Eg, Ex, E0 = np.zeros((B, N, D)), np.zeros((B, N, D)), np.zeros((B, D))
    for b in range(B):
        m, e = (np.zeros(D) if dl is None else np.abs(f64(dl[b]))), np.zeros(D)   # of the carry a G
        for t in reversed(range(N if lengths is None else lengths[b])):
            a, keep = L.sigmoid(g[b, t]), L.sigmoid(-g[b, t])
            m, e = m + np.abs(f64(dh[b, t])), e
            before = np.abs(hs[b, t - 1]) if t else (np.zeros(D) if h0 is None else np.abs(f64(h0[b])))
            by = (before + np.abs(xs[b, t]) if coupled else before) * a * keep
            Eg[b, t] = by * (e + 48 * U * m)
            Ex[b, t] = (keep if coupled else 1.0) * (e + 48 * U * m)
            m = a * m
            e = a * e + 24 * U * m
        E0[b] = e
    _check(dgate, want[0], Eg, half)
    _check(dx, want[1], Ex, half)
    if dh0 is not None:
        _check(dh0, want[2], E0, 0.0)


CASES = [
    # B, N, D, coupled, h0, lengths, packed
    (1, 1, 1, True, False, None, False),
    (2, 1, 64, True, True, None, False),
    (1, 2, 33, False, True, None, True),
    (2, 31, 32, True, False, None, False),
    (2, 127, 40, True, True, [127, 1], True),
    (1, 128, 36, False, True, None, False),
    (3, 129, 30, True, True, [0, 129, 64], True),      # pairs of channels
    (2, 255, 96, True, False, None, False),
    (2, 256, 7, False, True, [255, 256], True),        # odd width: one channel at a time
    (1, 257, 64, True, True, None, True),
    (1, 513, 65, True, True, None, False),
    (2, 1000, 100, True, True, [999, 513], False),
    (1, 2049, 34, False, True, None, True),
    (1, 4100, 72, True, True, None, False),            # several chunks a CTA
    (5, 300, 333, True, False, [300, 0, 299, 7, 128], False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,D,coupled,carried,lengths,packed", CASES)
def test_scan_and_gradient_match_the_oracle(dtype, B, N, D, coupled, carried, lengths, packed):
    gate, x, h0, dh, dl = _inputs(dtype, B, N, D, seed=N + D, packed=packed)
    h0 = h0 if carried else None
    dl = dl if carried else None
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    h, last = SCAN[dtype](gate, x, coupled=coupled, h0=h0, lengths=lens, h_last=True)
    dgate, dx, dh0 = BACK[dtype](gate, x, h, dh, coupled=coupled, h0=h0, lengths=lens, dh_last=dl, dh0=True)
    _check_all(dtype, gate, x, h0, dh, dl, coupled, lengths, h, last, dgate, dx, dh0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tiles_fill_the_gpu_more_than_once(dtype):
    """More channel tiles than CTAs fit at once, and sequences that end inside a chunk."""
    B, N, D = 24, 70, 1200
    gate, x, h0, dh, dl = _inputs(dtype, B, N, D, seed=1)
    lengths = [(7 * i) % (N + 1) for i in range(B)]
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    h, last = SCAN[dtype](gate, x, h0=h0, lengths=lens, h_last=True)
    dgate, dx, dh0 = BACK[dtype](gate, x, h, dh, h0=h0, lengths=lens, dh_last=dl, dh0=True)
    _check_all(dtype, gate, x, h0, dh, dl, True, lengths, h, last, dgate, dx, dh0)


# Channel tiles enough for CTAs of four warps, few enough that several of them share a sequence, and several rounds of
# each cluster: the shapes of a training step.  Clusters of 4, of 6 (a last round of which some chunks are empty, ragged
# lengths) and of 6 at an odd width.
TRAINING = [
    # B, N, D, coupled, lengths
    (4, 1500, 1024, True, None),
    (3, 1300, 1000, False, [1300, 771, 1]),
    (3, 1100, 999, True, [640, 1100, 1099]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,N,D,coupled,lengths", TRAINING)
def test_training_shapes_match_the_oracle(dtype, B, N, D, coupled, lengths):
    """Forward, gradient, and both again with the states written over the ones read."""
    gate, x, h0, dh, dl = _inputs(dtype, B, N, D, seed=D)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    more = dict(coupled=coupled, lengths=lens)
    TA.taylor_attn_device_errors(clear=True)
    h, last = SCAN[dtype](gate, x, h0=h0, h_last=True, **more)
    dgate, dx, dh0 = BACK[dtype](gate, x, h, dh, h0=h0, dh_last=dl, dh0=True, **more)
    _check_all(dtype, gate, x, h0, dh, dl, coupled, lengths, h, last, dgate, dx, dh0)
    state, carry = h0.clone(), dl.clone()
    h2, _ = SCAN[dtype](gate, x, h0=state, h_last=state, **more)
    dgate2, dx2, _ = BACK[dtype](gate, x, h, dh, h0=h0, dh_last=carry, dh0=carry, **more)
    assert torch.equal(h, h2) and torch.equal(state, last)
    assert torch.equal(dgate, dgate2) and torch.equal(dx, dx2) and torch.equal(carry, dh0)
    assert TA.taylor_attn_device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 33])
def test_padding_is_never_read(dtype, D):
    """NaN in every padded row of every input changes nothing; lengths past N count as N, negative ones as 0."""
    B, N = 4, 150
    gate, x, h0, dh, dl = _inputs(dtype, B, N, D, seed=4)
    lens = torch.tensor([0, 150, 77, 1], dtype=torch.int32, device=DEV)
    h, last = SCAN[dtype](gate, x, h0=h0, lengths=lens, h_last=True)
    grads = BACK[dtype](gate, x, h, dh, h0=h0, lengths=lens, dh_last=dl, dh0=True)
    pad = (torch.arange(N, device=DEV)[None] >= lens[:, None])[..., None]
    bad = [t.masked_fill(pad, float("nan")) for t in (gate, x, dh)]
    wild = torch.tensor([-3, 1000, 77, 1], dtype=torch.int32, device=DEV)
    h2, last2 = SCAN[dtype](bad[0], bad[1], h0=h0, lengths=wild, h_last=True)
    hn = h2.masked_fill(pad, float("nan"))
    grads2 = BACK[dtype](bad[0], bad[1], hn, bad[2], h0=h0, lengths=wild, dh_last=dl, dh0=True)
    assert torch.equal(h, h2) and torch.equal(last, last2)
    assert all(torch.equal(p, q) for p, q in zip(grads, grads2))
    assert (h[pad.expand_as(h)] == 0).all() and torch.equal(last[0], h0[0]) and torch.equal(grads[2][0], dl[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_gates_reset_and_hold(dtype):
    """-inf starts over from x, +inf holds the state; their gradients are zero, and NaN stays in its channel."""
    gate, x, h0, dh, dl = _inputs(dtype, 1, 300, 64, seed=6)
    gate[0, 100], gate[0, 200] = float("-inf"), float("inf")
    h, last = SCAN[dtype](gate, x, h0=h0, h_last=True)
    fresh, fresh_last = SCAN[dtype](gate[:, 100:], x[:, 100:], h_last=True)
    assert torch.equal(h[:, 100], x[:, 100])
    # token 200 may open another run of tokens than 199 closes: the state that enters it is then (prod a) c + b of
    # the run before, 199's own value the same sum walked token by token; both are within E of the exact state (the
    # module's analysis, which counts the sums' and the state's roundings), so they are within 2 E of one another,
    # and a rounding to the type each
    finite = gate.clone()
    finite[0, 100], finite[0, 200] = -9, 9
    E, _ = _bounds(finite, x, True, h0, None)
    apart = np.abs(f64(h[:, 200]) - f64(h[:, 199]))
    assert (apart <= 2 * E[:, 199] + 2 * (_half(dtype) if dtype == "bf16" else 0) * np.abs(f64(h[:, 199]))).all()
    torch.testing.assert_close(h[:, 100:], fresh, rtol=2 * _half(dtype) + 1e-4 * (dtype == "f32"), atol=1e-5)
    dgate, dx, _ = BACK[dtype](gate, x, h, dh, h0=h0, dh_last=dl)
    assert torch.isfinite(dgate).all() and torch.isfinite(dx).all()
    assert (dgate[0, 100].abs() < 1e-30).all() and (dgate[0, 200] == 0).all() and (dx[0, 200] == 0).all()
    gate[0, 50, 3] = float("nan")
    h, _ = SCAN[dtype](gate, x, h0=h0)
    clean = torch.ones(64, dtype=torch.bool, device=DEV)
    clean[3] = False
    assert torch.isnan(h[0, 50:, 3]).all() and torch.isfinite(h[0, :, clean]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [48, 37])
def test_parts_and_steps_make_the_whole(dtype, D):
    """A scan continued from its state, in place, and single steps follow the scan of the whole."""
    B, N = 3, 300
    gate, x, h0, *_ = _inputs(dtype, B, N, D, seed=9)
    E, El = _bounds(gate, x, True, h0, None)
    ref, ref_last = L.gated_scan(f64(gate), f64(x), True, f64(h0))
    half = _half(dtype) if dtype == "bf16" else 0.0
    state, parts = h0.clone(), []
    for lo, hi in ((0, 1), (1, 140), (140, 140), (140, 290)):
        h, state = SCAN[dtype](gate[:, lo:hi], x[:, lo:hi], h0=state, h_last=state)
        parts.append(h)
    for t in range(290, N):
        parts.append(STEP[dtype](gate[:, t], x[:, t], state)[:, None])
    _check(torch.cat(parts, 1), ref, E, half)
    _check(state, ref_last, El, 0.0)
    new = torch.empty_like(state)
    keep = state.clone()
    out = STEP[dtype](gate[:, 0], x[:, 0], state, state_out=new)
    assert torch.equal(state, keep) and torch.equal(new.to(out.dtype), out)


@pytest.mark.parametrize("N,D", [(5000, 40), (700, 33)])
def test_states_may_be_written_over_the_ones_read(N, D):
    """h_last over h0 and dh0 over dh_last, with several CTAs to a sequence."""
    gate, x, h0, dh, dl = _inputs("bf16", 2, N, D, seed=5)
    h, last = TA.taylor_attn_gated_scan(gate, x, h0=h0, h_last=True)
    dgate, dx, dh0 = TA.taylor_attn_gated_scan_backward(gate, x, h, dh, h0=h0, dh_last=dl, dh0=True)
    state, carry = h0.clone(), dl.clone()
    h2, _ = TA.taylor_attn_gated_scan(gate, x, h0=state, h_last=state)
    dgate2, dx2, _ = TA.taylor_attn_gated_scan_backward(gate, x, h, dh, h0=h0, dh_last=carry, dh0=carry)
    assert torch.equal(h, h2) and torch.equal(state, last)
    assert torch.equal(dgate, dgate2) and torch.equal(dx, dx2) and torch.equal(carry, dh0)


@pytest.mark.parametrize("coupled", [True, False])
def test_the_gradient_is_that_of_exact_states_within_their_rounding(coupled):
    """bf16: dgate against the gradient that has the states in 64 bits.  The stored h_{t-1} is off by E (the module's
    analysis) and half a step, and enters dgate times |G| a (1 - a); the kernel adds its own bound and a rounding."""
    B, N, D = 2, 400, 72
    gate, x, h0, dh, dl = _inputs("bf16", B, N, D, seed=21)
    h, _ = TA.taylor_attn_gated_scan(gate, x, coupled=coupled, h0=h0)
    dgate, dx, dh0 = TA.taylor_attn_gated_scan_backward(gate, x, h, dh, coupled=coupled, h0=h0, dh_last=dl, dh0=True)
    g, xs, half = f64(gate), f64(x), _half("bf16")
    want = L.gated_scan_grad(g, xs, f64(dh), coupled, f64(h0), None, f64(dl))
    a, keep = L.sigmoid(g), L.sigmoid(-g)
    states, _ = L.gated_scan(g, xs, coupled, f64(h0))
    E, _ = _bounds(gate, x, coupled, h0, None)
    before = np.concatenate([f64(h0)[:, None], states[:, :-1]], 1)
    rounding = np.concatenate([np.zeros((B, 1, D)), E[:, :-1] + half * (np.abs(states[:, :-1]) + E[:, :-1])], 1)
    m, e, limit = np.abs(f64(dl)), np.zeros((B, D)), np.zeros((B, N, D))
    for t in reversed(range(N)):
        m = m + np.abs(f64(dh[:, t]))
        size = np.abs(before[:, t]) + rounding[:, t] + (np.abs(xs[:, t]) if coupled else 0.0)
        limit[:, t] = a[:, t] * keep[:, t] * (m * rounding[:, t] + size * (e + 48 * U * m))
        m, e = a[:, t] * m, a[:, t] * e + 24 * U * a[:, t] * m
    _check(dgate, want[0], limit, half)


def test_uncoupled_step():
    gate, x, h0, *_ = _inputs("f32", 4, 1, 20, seed=2)
    h, last = SCAN["f32"](gate, x, coupled=False, h0=h0, h_last=True)
    state = h0.clone()
    out = STEP["f32"](gate[:, 0], x[:, 0], state, coupled=False)
    torch.testing.assert_close(out, h[:, 0], rtol=2 ** -22, atol=1e-7)
    torch.testing.assert_close(state, last, rtol=2 ** -22, atol=1e-7)


def test_empty_calls():
    e = torch.empty(2, 0, 8, dtype=torch.bfloat16, device=DEV)
    h0 = torch.randn(2, 8, device=DEV)
    h, last = TA.taylor_attn_gated_scan(e, e, h0=h0, h_last=True)
    assert h.shape == (2, 0, 8) and torch.equal(last, h0)
    _, last = TA.taylor_attn_gated_scan(e, e, h_last=True)
    assert (last == 0).all()
    _, _, dh0 = TA.taylor_attn_gated_scan_backward(e, e, h, e, dh_last=h0, dh0=True)
    assert torch.equal(dh0, h0)
    n = torch.empty(0, 5, 8, dtype=torch.bfloat16, device=DEV)
    assert TA.taylor_attn_gated_scan(n, n)[0].numel() == 0


def test_gradients_into_slices_of_a_packed_gradient():
    gate, x, h0, dh, dl = _inputs("bf16", 2, 90, 32, seed=3, packed=True)
    h, _ = TA.taylor_attn_gated_scan(gate, x, h0=h0)
    want = TA.taylor_attn_gated_scan_backward(gate, x, h, dh, h0=h0, dh_last=dl)
    rows = torch.full((2, 90, 100), 5.0, dtype=torch.bfloat16, device=DEV)
    got = TA.taylor_attn_gated_scan_backward(gate, x, h, dh, h0=h0, dh_last=dl, dgate=rows[..., 4:36],
                                             dx=rows[..., 40:72])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    rest = torch.cat([rows[..., :4], rows[..., 36:40], rows[..., 72:]], -1)
    assert (rest == 5).all()


def test_repeats_streams_and_graphs_give_the_same_bits():
    gate, x, h0, dh, dl = _inputs("bf16", 2, 3000, 64, seed=12)

    def both(stream=None):
        h, last = TA.taylor_attn_gated_scan(gate, x, h0=h0, h_last=True, stream=stream)
        return (h, last) + TA.taylor_attn_gated_scan_backward(gate, x, h, dh, h0=h0, dh_last=dl, dh0=True,
                                                              stream=stream)

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, out))
    gate.copy_(gate.flip(1))
    graph.replay()
    again = both()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(again, out))
