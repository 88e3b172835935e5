"""The operators around the attention in one run, as a decoder uses them: a
recurrent layer feeds projections, queries and keys are normalised and rotated,
the attention takes the whole prompt once, and a batch of sequences continues
from it token by token; and the gradients of the recurrent layer and the norms
chained through the projection."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from oracle import taylor_oracle as T
from recurrent_states_b200 import taylor_attn as TA
from tests.gpu_common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TAU = 2.0


def _weights(D, H, d, dv, seed):
    g = torch.Generator().manual_seed(seed)
    w_in = torch.randn(D, 2 * D, generator=g) / D ** 0.5                     # gate | x
    w_qkv = torch.randn(D, H * (2 * d + dv), generator=g) / D ** 0.5         # q | k | v
    return w_in.to(DEV), w_qkv.to(DEV)


def _split(rows, H, d, dv):
    q = rows[..., :H * d].unflatten(-1, (H, d))
    k = rows[..., H * d:2 * H * d].unflatten(-1, (H, d))
    return q, k, rows[..., 2 * H * d:].unflatten(-1, (H, dv))


@pytest.mark.parametrize("d,n", [(16, 3), (16, 4), (64, 3)])
def test_a_batch_continues_a_shared_prompt(d, n):
    """fp32 throughout.  The oracle runs every sequence whole, prompt and
    continuation, from the same projections' outputs of the kernels' own states
    (the recurrent layer is compared on its own), so what is compared is norms,
    rotation and attention: tolerance 1e-5 of the row's largest output, that of
    the fp32 attention path."""
    D, H, dv, P, B, steps = 48, 2, 16, 70, 3, 5
    w_in, w_qkv = _weights(D, H, d, dv, seed=d + n)
    g = torch.Generator().manual_seed(1)
    prompt, later = torch.randn(1, P, D, generator=g).to(DEV), torch.randn(B, steps, D, generator=g).to(DEV)
    freqs = TA.rope_freqs(d)

    # the prompt, once
    rows = prompt @ w_in
    h, state = TA.taylor_attn_gated_scan_f32(rows[..., :D], rows[..., D:], h_last=True)
    q, k, v = _split(h @ w_qkv, H, d, dv)
    qn, kn = TA.taylor_attn_qk_norm_rope_f32(q, k, freqs)
    out, prefix = TA.taylor_attn_prefill_f32(qn, kn, v.transpose(1, 2).contiguous(), n, TAU, state_out=True)
    ref_h, ref_last = L.gated_scan(f64(rows[..., :D]), f64(rows[..., D:]))
    np.testing.assert_allclose(f64(h), ref_h, rtol=1e-5, atol=1e-6)

    # the batch, from the prompt's two states
    state = state.expand(B, D).contiguous()
    cap = steps
    k_cache, v_cache = torch.zeros(B, H, cap, d, device=DEV), torch.zeros(B, H, cap, dv, device=DEV)
    lengths = torch.zeros(B, dtype=torch.int32, device=DEV)
    got, keys, queries, values, gates, xs = [], [], [], [], [], []
    for s in range(steps):
        rows_s = later[:, s] @ w_in
        gates.append(rows_s[:, :D])
        xs.append(rows_s[:, D:])
        hs = TA.taylor_attn_gated_step_f32(rows_s[:, :D], rows_s[:, D:], state)
        q1, k1, v1 = _split((hs @ w_qkv)[:, None], H, d, dv)
        pos = torch.full((B, 1), P + s, dtype=torch.int64, device=DEV)
        qo, ko = TA.taylor_attn_qk_norm_rope_f32(q1, k1, freqs, positions=pos)
        queries.append(q1)
        keys.append(k1)
        values.append(v1)
        got.append(TA.taylor_attn_shared_prefix_decode_f32(qo[:, :, 0], ko[:, :, 0], v1[:, 0].contiguous(), prefix,
                                                           k_cache, v_cache, lengths, n, TAU))
        lengths += 1
    got = torch.stack(got, 2)

    whole, last = L.gated_scan(np.concatenate([np.repeat(f64(rows[..., :D]), B, 0), f64(torch.stack(gates, 1))], 1),
                               np.concatenate([np.repeat(f64(rows[..., D:]), B, 0), f64(torch.stack(xs, 1))], 1))
    np.testing.assert_allclose(f64(state), last, rtol=1e-5, atol=1e-6)
    pos = np.arange(P + steps)[None].repeat(B, 0)
    joined = lambda one, rest: np.concatenate([np.repeat(f64(one), B, 0), f64(torch.cat(rest, 1))], 1)  # noqa: E731
    Q, K = (L.norm_rope(joined(a, b), freqs, pos) for a, b in ((q, queries), (k, keys)))
    V = joined(v, values).transpose(0, 2, 1, 3)
    want = T.attention_direct(Q, K, V, n, TAU)
    for have, ref in ((f64(out), want[:1, :, :P]), (f64(got), want[:, :, P:])):
        scale = np.abs(ref).max(-1, keepdims=True)
        assert (np.abs(have - ref) <= 1e-5 * scale).all(), float((np.abs(have - ref) / scale).max())


def test_gradients_chain_through_the_layer():
    """d loss of the packed input projection through recurrence, projection, norms and rotation, against float64
    differences of the oracle: fp32 kernels, so 1e-4 of the largest gradient (differences of step 1e-5 in float64
    are good to 1e-9; the chain multiplies fp32 roundings by sums of some hundred terms)."""
    B, N, D, H, d = 2, 9, 12, 2, 6
    w_in, w_qkv = _weights(D, H, d, 4, seed=3)
    g = torch.Generator().manual_seed(2)
    rows = torch.randn(B, N, 2 * D, generator=g).to(DEV)
    dqo, dko = torch.randn(B, H, N, d, generator=g).to(DEV), torch.randn(B, H, N, d, generator=g).to(DEV)
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(DEV)
    freqs = TA.rope_freqs(4)

    h, _ = TA.taylor_attn_gated_scan_f32(rows[..., :D], rows[..., D:])
    proj = h @ w_qkv
    q, k, _ = _split(proj, H, d, 4)
    dproj = torch.zeros_like(proj)
    dq, dk, _ = _split(dproj, H, d, 4)
    TA.taylor_attn_qk_norm_rope_backward_f32(q, k, dqo, dko, freqs, q_weight=w, k_weight=w, dq=dq, dk=dk)
    drows = torch.empty_like(rows)
    TA.taylor_attn_gated_scan_backward_f32(rows[..., :D], rows[..., D:], h, dproj @ w_qkv.T, dgate=drows[..., :D],
                                           dx=drows[..., D:])

    def loss(r):
        h64, _ = L.gated_scan(r[..., :D], r[..., D:])
        p = h64 @ f64(w_qkv)
        pos = np.arange(N)[None].repeat(B, 0)
        y = [L.norm_rope(p[..., i * H * d:(i + 1) * H * d].reshape(B, N, H, d), freqs, pos, f64(w)) for i in range(2)]
        return (y[0] * f64(dqo)).sum() + (y[1] * f64(dko)).sum()

    r = f64(rows)
    want = np.zeros_like(r)
    for i in np.ndindex(r.shape):
        e = np.zeros_like(r)
        e[i] = 1e-5
        want[i] = (loss(r + e) - loss(r - e)) / 2e-5
    assert np.abs(f64(drows) - want).max() <= 1e-4 * np.abs(want).max()


@pytest.mark.parametrize("capture", [False, True])
def test_two_streams_at_once(capture):
    """Calls of every operator on two streams at the same time (and two captured graphs replayed together) give what
    they give alone."""
    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
        q, k, w = r(4, 300, 4, 64), r(4, 300, 4, 64), torch.rand(64, generator=g).to(DEV) + 0.5
        gate, x = r(2, 2500, 64), r(2, 2500, 64)
        unit = lambda z: torch.nn.functional.normalize(z.float(), dim=-1).bfloat16()  # noqa: E731
        kp = unit(r(1, 4, 200, 64))
        state = TA.taylor_attn_prefill(kp, kp, r(1, 4, 200, 64), 3, TAU, state_out=True)[1]
        lens = torch.randint(0, 90, (5,), generator=g, dtype=torch.int32).to(DEV)
        return q, k, w, gate, x, unit(r(5, 4, 64)), r(5, 4, 64), state, unit(r(5, 4, 90, 64)), r(5, 4, 90, 64), lens

    def calls(a):
        q, k, w, gate, x, q1, v1, state, kc, vc, lens = a
        freqs = TA.rope_freqs(64)
        qo, ko = TA.taylor_attn_qk_norm_rope(q, k, freqs, q_weight=w, k_weight=w)
        dq, dk, dqw, dkw = TA.taylor_attn_qk_norm_rope_backward(q, k, qo, ko, freqs, q_weight=w, k_weight=w)
        h, last = TA.taylor_attn_gated_scan(gate, x, h_last=True)
        dgate, dx, _ = TA.taylor_attn_gated_scan_backward(gate, x, h, h)
        o = TA.taylor_attn_shared_prefix_decode(q1, q1, v1, state, kc, vc, lens, 3, TAU)
        return qo, ko, dq, dk, dqw, dkw, h, last, dgate, dx, o

    sets = [inputs(s) for s in (1, 2)]
    want = [[t.clone() for t in calls(a)] for a in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    if capture:
        for a in sets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = calls(a)
            graphs.append((g, out))
    for _ in range(3):
        got = []
        for i, a in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                if capture:
                    graphs[i][0].replay()
                    got.append(graphs[i][1])
                else:
                    got.append(calls(a))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(w, o))


FIRST = {
    "norms": "TA.taylor_attn_qk_norm_rope_backward(q, q, o, o, TA.rope_freqs(64), q_weight=w)",
    "scan": "TA.taylor_attn_gated_scan(g, g)",
    "prefix": "TA.taylor_attn_shared_prefix_decode(r(2, 4, 64), r(2, 4, 64), r(2, 4, 64), state, kc, kc, lens, 3, 2.0)",
}


@pytest.mark.parametrize("name", FIRST)
def test_a_process_may_make_its_first_call_inside_a_capture(name):
    """The workspace pool and the error word are set up by the first call that needs them."""
    code = f"""
import torch
from recurrent_states_b200 import taylor_attn as TA
r = lambda *s: torch.randn(*s, device="cuda").bfloat16()
q, o, g, w = r(2, 40, 4, 64), r(2, 4, 40, 64), r(2, 900, 64), torch.ones(64, device="cuda")
state = torch.ones(4, TA.taylor_attn_state_stride(64, 64, 3), device="cuda")
kc, lens = r(2, 4, 9, 64), torch.tensor([3, 8], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = {FIRST[name]}
graph.replay()
torch.cuda.synchronize()
out = out if isinstance(out, tuple) else (out,)
assert all(torch.isfinite(t).all() for t in out if t is not None)
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-1500:]


def test_sizes_past_32_bits_are_refused():
    """Sizes that a C int does not hold (expanded tensors) are refused before anything is allocated or launched; they
    were taken modulo 2^32, which left all but a few rows of the outputs as they were allocated."""
    many, one = (1 << 32) + 1, torch.ones(1, device=DEV)
    none = TA.rope_freqs(0)
    rows, flat, cache = one.expand(1, many, 1), one.expand(many, 1), one.expand(1, 1, many, 1)
    calls = [lambda: TA.taylor_attn_qk_norm_rope_f32(rows[..., None], rows[..., None], none),
             lambda: TA.taylor_attn_qk_norm_rope_backward_f32(rows[..., None], rows[..., None], cache, cache, none),
             lambda: TA.taylor_attn_gated_scan_f32(rows, rows),
             lambda: TA.taylor_attn_gated_scan_backward_f32(rows, rows, rows, rows),
             lambda: TA.taylor_attn_gated_step_f32(flat, flat, flat),
             lambda: TA.taylor_attn_shared_prefix_decode_f32(one.view(1, 1, 1), one.view(1, 1, 1), one.expand(1, 1, 4), one,
                                                             cache, cache, one, 2, TAU)]
    for call in calls:
        with pytest.raises(TA.TaylorAttnError) as refused:
            call()
        assert refused.value.status == TA.TAYLOR_ERR_UNSUPPORTED
