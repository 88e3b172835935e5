"""Decoding a batch that shares a prefix, against the float64 oracle.

Tolerance.  y is a sum of products: over F features phi_f(q) S_f, over L + 1
own tokens K(tau q.k_j) v_j.  phi is a product of at most 4 entries and a
weight (6 roundings), both of its product's factors are held as two tf32 parts
(within 2^-21 = 8 u each, by truncation, and lo lo left out, 4 u), K a
polynomial of degree 4 in a dot product of at most 64 terms; sums run over at most F + L + 1 terms in strips and trees of which no
chain is longer than (F + L) / 8 + 64.  With A the sum of the terms' absolute
values (for K the polynomial of |q|.|k|) and u = 2^-24 the numerator and the
denominator are within (96 + (F + L) / 8) u A of theirs, and the quotient adds
one rounding and the denominator's relative error."""
import math

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from oracle import taylor_oracle as T
from recurrent_states_b200 import taylor_attn as TA
from tests.gpu_common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DECODE = {"bf16": TA.taylor_attn_shared_prefix_decode, "f32": TA.taylor_attn_shared_prefix_decode_f32}
TAU = 2.0


def _unit(g, *shape):
    x = torch.randn(*shape, generator=g, dtype=torch.float64)
    return x / x.norm(dim=-1, keepdim=True)


def _inputs(dtype, B, H, d, dv, n, cap, lengths, seed, P=40):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    kp, vp = _unit(g, H, P, d).numpy(), torch.randn(H, P, dv, generator=g, dtype=torch.float64).numpy()
    logical = T.state_of(kp[None], vp[None], n)[0]
    state = TA.state_flat(torch.from_numpy(logical), d, dv, n).to(DEV)
    q, k = _unit(g, B, H, d).to(t).to(DEV), _unit(g, B, H, d).to(t).to(DEV)
    v = torch.randn(B, H, dv, generator=g).to(t).to(DEV)
    kc, vc = _unit(g, B, H, cap, d).to(t).to(DEV), torch.randn(B, H, cap, dv, generator=g).to(t).to(DEV)
    return q, k, v, state, kc, vc, torch.tensor(lengths, dtype=torch.int32, device=DEV)


def _check(out, q, k, v, state, kc, vc, lengths, n):
    """kc, vc as they were before the call."""
    d, dv = q.shape[-1], v.shape[-1]
    S = f64(TA.state_logical(state.cpu(), d, dv, n))
    want = L.shared_prefix_decode(f64(q), f64(k), f64(v), S, f64(kc), f64(vc), lengths.tolist(), n, TAU)
    size = L.shared_prefix_decode(np.abs(f64(q)), np.abs(f64(k)), np.abs(f64(v)), np.abs(S), np.abs(f64(kc)),
                                  np.abs(f64(vc)), lengths.tolist(), n, TAU)  # majorant quotient: A / A_z
    phi = T.feature_map(f64(q), n) * T.query_coeffs(d, n, TAU)
    den = np.einsum("bhf,hf->bh", phi, S[..., -1])
    aden = np.einsum("bhf,hf->bh", T.feature_map(np.abs(f64(q)), n) * T.query_coeffs(d, n, TAU), np.abs(S[..., -1]))
    for b, m in enumerate(lengths.tolist()):
        keys = np.concatenate([f64(kc)[b, :, :m], f64(k)[b, :, None]], 1)
        den[b] += T.taylor_kernel(TAU * np.einsum("hld,hd->hl", keys, f64(q)[b]), n).sum(-1)
        aden[b] += T.taylor_kernel(TAU * np.einsum("hld,hd->hl", np.abs(keys), np.abs(f64(q)[b])), n).sum(-1)
    F = S.shape[1]
    c = (96 + (F + int(lengths.max())) / 8) * U
    ratio = (aden / np.abs(den))[..., None]
    limit = c * ratio * (size + np.abs(want)) + U * np.abs(want)
    err = np.abs(f64(out) - want)
    assert (err <= limit).all(), float((err / limit).max())


CASES = [
    # B, H, d, dv, n, cap, lengths
    (1, 1, 16, 64, 3, 1, [0]),                       # the first token past the prefix
    (3, 2, 16, 64, 3, 70, [0, 69, 33]),
    (5, 3, 16, 64, 5, 40, [1, 39, 17, 0, 8]),
    (2, 2, 16, 64, 4, 300, [299, 257]),
    (4, 2, 64, 64, 3, 130, [128, 129, 127, 0]),
    (2, 1, 64, 128, 3, 20, [19, 4]),
    (3, 1, 32, 64, 4, 33, [32, 31, 16]),
    (2, 2, 64, 256, 2, 50, [49, 3]),
    (3, 2, 7, 12, 3, 90, [89, 0, 64]),               # odd key rows
    (2, 3, 24, 20, 3, 60, [59, 2]),
    (2, 1, 1, 4, 1, 9, [8, 0]),
    (1, 2, 3, 36, 5, 17, [11]),
    (2, 2, 20, 100, 2, 64, [63, 32]),
    (37, 2, 16, 64, 3, 12, list(range(12)) * 3 + [11]),
    (70, 1, 64, 64, 3, 5, [i % 5 for i in range(70)]),   # more sequences than a tile of queries
    (130, 3, 16, 16, 2, 3, [i % 3 for i in range(130)]),
    (1, 2, 16, 64, 3, 5000, [4999]),                 # a long suffix of few heads
    (40, 8, 16, 64, 3, 700, [(i * 17) % 700 for i in range(40)]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,dv,n,cap,lengths", CASES)
def test_decode_matches_the_oracle_and_appends(dtype, B, H, d, dv, n, cap, lengths):
    q, k, v, state, kc, vc, lens = _inputs(dtype, B, H, d, dv, n, cap, lengths, seed=d + cap)
    before = kc.clone(), vc.clone()
    out = DECODE[dtype](q, k, v, state, kc, vc, lens, n, TAU)
    _check(out, q, k, v, state, *before, lens, n)
    rows = torch.arange(B, device=DEV)
    before[0][rows, :, lens.long()] = k
    before[1][rows, :, lens.long()] = v
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


# Enough heads of short caches for CTAs of four warps, at every way of reading keys (rows of 64, 32 and 16 entries, and
# any other) and every count of a lane's columns; and shares of more than 256 features, whose descriptors are formed
# several times, with the last group of features not a whole one (F 4,845, 2,145 and 6,545).
MANY = [(19, 16, d, dv, 3, 40, [(i * 7) % 40 for i in range(19)]) for d in (64, 32, 16, 20) for dv in (20, 64, 100, 128, 256)]
LARGE_SHARES = [
    (17, 8, 16, 64, 5, 30, [(i * 11) % 30 for i in range(17)]),
    (3, 32, 64, 64, 3, 6, [5, 0, 3]),
    (70, 16, 64, 64, 3, 3, [i % 3 for i in range(70)]),
    (4, 16, 32, 36, 4, 5, [4, 0, 1, 2]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,dv,n,cap,lengths", MANY + LARGE_SHARES)
def test_many_heads_and_large_shares(dtype, B, H, d, dv, n, cap, lengths):
    q, k, v, state, kc, vc, lens = _inputs(dtype, B, H, d, dv, n, cap, lengths, seed=d + dv)
    before = kc.clone(), vc.clone()
    out = DECODE[dtype](q, k, v, state, kc, vc, lens, n, TAU)
    _check(out, q, k, v, state, *before, lens, n)
    rows = torch.arange(B, device=DEV)
    before[0][rows, :, lens.long()] = k
    before[1][rows, :, lens.long()] = v
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(16, 64), (9, 20)])
def test_rows_behind_a_sequence_are_never_read(dtype, d, dv):
    q, k, v, state, kc, vc, lens = _inputs(dtype, 3, 2, d, dv, 3, 50, [0, 20, 49], seed=1)
    want = DECODE[dtype](q, k, v, state, kc, vc, lens, 3, TAU)
    behind = (torch.arange(50, device=DEV)[None] >= lens[:, None])[:, None, :, None]
    kn, vn = kc.masked_fill(behind, float("nan")), vc.masked_fill(behind, float("nan"))
    got = DECODE[dtype](q, k, v, state, kn, vn, lens, 3, TAU)
    assert torch.equal(want, got)
    past = (torch.arange(50, device=DEV)[None] > lens[:, None])[:, None, :, None]
    assert torch.isnan(kn[past.expand_as(kn)]).all() and torch.isnan(vn[past.expand_as(vn)]).all()


def test_lengths_out_of_range_are_reported():
    q, k, v, state, kc, vc, lens = _inputs("bf16", 4, 2, 16, 64, 3, 10, [3, 10, -1, 9], seed=2)
    before = kc.clone(), vc.clone()
    TA.taylor_attn_device_errors(clear=True)
    out = TA.taylor_attn_shared_prefix_decode(q, k, v, state, kc, vc, lens, 3, TAU)
    assert TA.taylor_attn_device_errors(clear=True) == 32
    assert torch.isnan(out[1:3]).all() and torch.isfinite(out[[0, 3]]).all()
    assert torch.equal(kc[1:3], before[0][1:3]) and torch.equal(vc[1:3], before[1][1:3])
    good = torch.tensor([3, 0, 0, 9], dtype=torch.int32, device=DEV)
    kc.copy_(before[0]), vc.copy_(before[1])
    again = TA.taylor_attn_shared_prefix_decode(q, k, v, state, kc, vc, good, 3, TAU)
    assert torch.equal(out[[0, 3]], again[[0, 3]]) and TA.taylor_attn_device_errors() == 0


@pytest.mark.parametrize("d,n,dv", [(16, 3, 64), (64, 3, 64), (16, 5, 64)])
def test_it_is_a_decode_from_copies_of_the_prefix(d, n, dv):
    """Steps of the batch against taylor_attn_decode_f32 on a copy of the state for each sequence."""
    B, H, cap = 3, 2, 8
    q, k, v, state, kc, vc, lens = _inputs("f32", B, H, d, dv, n, cap, [0, 0, 0], seed=3)
    states = state[None].repeat(B, 1, 1)
    g = torch.Generator().manual_seed(4)
    for step in range(cap):
        q, k = _unit(g, B, H, d).float().to(DEV), _unit(g, B, H, d).float().to(DEV)
        v = torch.randn(B, H, dv, generator=g).to(DEV)
        want = TA.taylor_attn_decode_f32(q, k, v, states, n, TAU)
        got = TA.taylor_attn_shared_prefix_decode_f32(q, k, v, state, kc, vc, lens, n, TAU)
        torch.testing.assert_close(got, want, rtol=1e-5, atol=1e-5)
        lens += 1
    with pytest.raises(TA.TaylorAttnError):
        TA.taylor_attn_shared_prefix_decode_f32(q, k, v, state, kc[:, :, :0], vc[:, :, :0], lens, n, TAU)


def test_graphs_streams_and_repeats_give_the_same_bits():
    """Two captured calls with workspaces of their own, replayed in turn, and one on another stream."""
    sets = [_inputs("bf16", 40, 4, 64, 64, 3, 400, [(i * s) % 400 for i in range(40)], seed=s) for s in (7, 11)]
    call = lambda s: TA.taylor_attn_shared_prefix_decode(*s, 3, TAU)  # noqa: E731
    want = [call(s).clone() for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = TA.taylor_attn_shared_prefix_decode(*sets[0], 3, TAU, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
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
    assert all(torch.equal(w, o) for w, o in zip(want, outs))
    sets[0][0].copy_(sets[1][0])
    graphs[0].replay()
    fresh = call(sets[0])
    torch.cuda.synchronize()
    assert torch.equal(fresh, outs[0])


def test_empty_batch():
    e = torch.empty(0, 2, 16, dtype=torch.bfloat16, device=DEV)
    v = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    state = torch.zeros(2, TA.taylor_attn_state_stride(16, 64, 3), device=DEV)
    out = TA.taylor_attn_shared_prefix_decode(e, e, v, state, e[:, :, None], v[:, :, None],
                                              torch.empty(0, dtype=torch.int32, device=DEV), 3, TAU)
    assert out.shape == (0, 2, 64)
