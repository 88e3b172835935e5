"""The operators of a decoder around Taylor attention, as they are timed and compared.

Three operators, each in the forms that training and serving use:

qk      norms of queries and keys for each head with the position rotation in
        the same pass, from the projection's token-major layout to the
        head-major one that the attention calls take; and its gradient
prefix  one new token per sequence for a batch whose sequences share a long
        prefix: the prefix's Taylor state is read once for the whole batch,
        each sequence's own tokens come from its key and value cache
gate    the gated linear recurrence h_t = a_t h_{t-1} + b_t per channel: the
        scan over a sequence, its gradient, and the step for single tokens

With ``own`` false, ``run`` computes them from elementary torch operations in
32 bits (angles in 64) and rounds once at the end; with ``own`` true it calls
the library.
"""
import itertools
import math

import numpy as np
import torch

own = False

TAU = 2.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def _qk(name, B, N, Hq, Hk, d, rot, dtype, weights, grad, interleaved, packed, given):
    return dict(name=name, op="qk", B=B, N=N, Hq=Hq, Hk=Hk, d=d, rot=rot, dtype=dtype, weights=weights, grad=grad,
                interleaved=interleaved, packed=packed, given=given)


def _prefix(name, B, H, d, dv, n, most, dtype):
    return dict(name=name, op="prefix", B=B, H=H, d=d, dv=dv, n=n, most=most, dtype=dtype)


def _gate(name, form, B, N, D, dtype, coupled, carried, ragged):
    return dict(name=name, op="gate", form=form, B=B, N=N, D=D, dtype=dtype, coupled=coupled, carried=carried,
                ragged=ragged)


def listed():
    return [
        # one decode step's q and k of 64 sequences, each at its own position: latency
        _qk("qk_step", 64, 1, 16, 16, 16, 16, "bf16", False, False, False, True, True),
        # the main prefill's q and k, sliced out of a packed projection
        _qk("qk_prefill", 1, 4096, 8, 8, 16, 16, "bf16", False, False, False, True, False),
        # a training step at the large head's width, with learned weights: forward and gradient
        _qk("qk_train", 4, 8192, 16, 16, 64, 64, "bf16", True, True, False, True, False),
        # odd sizes: fewer key heads, a partial rotation of neighbouring pairs, fp32
        _qk("qk_train_odd", 3, 777, 6, 2, 20, 12, "f32", True, True, True, False, True),
        # a few sequences just after the shared prefix: latency
        _prefix("prefix_few", 4, 8, 16, 64, 3, 32, "bf16"),
        # the decode workload's heads, each sequence up to 512 tokens past the prefix
        _prefix("prefix_decode", 64, 16, 16, 64, 3, 512, "bf16"),
        # the large head: 2,145 features, up to 1,024 tokens past the prefix
        _prefix("prefix_large_head", 64, 16, 64, 64, 3, 1024, "bf16"),
        # the highest order over an odd batch in fp32: the shared state is the larger part
        _prefix("prefix_order5", 17, 8, 16, 64, 5, 300, "f32"),
        # one decode step of a recurrent layer
        _gate("gate_step", "step", 64, 1, 1024, "bf16", True, True, False),
        # a prompt continued from a carried state, one sequence: few channels, split over the length
        _gate("gate_prefill", "scan", 1, 4096, 512, "bf16", True, True, False),
        # a training step over long sequences: forward and gradient
        _gate("gate_train", "train", 4, 8192, 1024, "bf16", True, False, False),
        # odd sizes: ragged lengths in a padded batch, an odd width, inputs not scaled by 1 - a, fp32
        _gate("gate_train_odd", "train", 3, 1999, 333, "f32", False, True, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk", "prefix", "gate", "gate"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "qk":
        d = rng.choice([rng.randint(2, 64), 16, 32, 64])
        rot = rng.choice([d // 2 * 2, d // 2 * 2, d // 4 * 2])
        B, Hq = _log(rng, 1, 64), _log(rng, 1, 32)
        Hk = rng.choice([Hq, max(1, Hq // 4)])
        most = max(1, 32_000_000 // (B * (Hq + Hk) * d))
        N = min(_log(rng, 1, 16384), most)
        case = _qk(None, B, N, Hq, Hk, d, rot, dtype, rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3,
                   rng.random() < 0.6, rng.random() < 0.5)
    elif op == "prefix":
        d, n = rng.choice([(16, 3), (16, 3), (16, 4), (16, 5), (64, 3), (32, 3), (rng.randint(3, 24), 2), (24, 3)])
        B, H = _log(rng, 1, 96), _log(rng, 1, 16)
        dv = rng.choice([64, 64, 128, 4 * rng.randint(1, 20)])
        most = min(_log(rng, 1, 2048), max(1, 60_000_000 // (B * H * (d + dv))))
        case = _prefix(None, B, H, d, dv, n, most, dtype)
    else:
        form = rng.choice(["step", "scan", "train", "train"])
        B, D = _log(rng, 1, 32), _log(rng, 32, 4096)
        N = 1 if form == "step" else min(_log(rng, 1, 65536), max(1, 16_000_000 // (B * D)))
        case = _gate(None, form, B, N, D, dtype, rng.random() < 0.6, form == "step" or rng.random() < 0.5,
                     form != "step" and rng.random() < 0.4)
    del case["name"]
    return case


def _lengths(B, most):
    """Lengths from zero to `most`, spread over the batch by its index alone."""
    if B == 1:
        return [most]
    return [most * ((i * 37) % B) // (B - 1) if B % 37 else most * i // (B - 1) for i in range(B)]


# ------------------------------------------------------------------ the inputs

def _features(d, n):
    """Per degree: the packed monomials' indices and weights sqrt(m!/alpha!)."""
    found = []
    for m in range(n):
        tuples = list(itertools.combinations_with_replacement(range(d), m))
        weights = [math.sqrt(math.factorial(m) / math.prod(math.factorial(t.count(i)) for i in set(t)))
                   for t in tuples]
        found.append((tuples, weights))
    return found


def _phi(x, table):
    """phi of x [..., d], degree-major, in x's type."""
    parts = []
    for tuples, weights in table:
        w = torch.tensor(weights, dtype=x.dtype, device=x.device)
        if not tuples[0]:
            parts.append(w.expand(x.shape[:-1] + (1,)))
            continue
        index = torch.tensor(tuples, device=x.device)
        parts.append(x[..., index].prod(-1) * w)
    return torch.cat(parts, -1)


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _stride(F, dv):
    return (F * (dv + 1) + 31) // 32 * 32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    t = DTYPES[case["dtype"]]
    B, s = case["B"], {"case": case}
    if case["op"] == "qk":
        N, Hq, Hk, d = case["N"], case["Hq"], case["Hk"], case["d"]
        if case["packed"]:  # q | k | v rows of one projection, v as wide as q
            rows = normal(B, N, (2 * Hq + Hk) * d).to(t)
            s["q"] = rows[..., :Hq * d].unflatten(-1, (Hq, d))
            s["k"] = rows[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
        else:
            s["q"], s["k"] = normal(B, N, Hq, d).to(t), normal(B, N, Hk, d).to(t)
        s["freqs"] = 10000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"]) if case["rot"] else np.zeros(0)
        s["positions"] = None
        if case["given"]:
            s["positions"] = (torch.randint(0, 65536 - N + 1, (B, 1), generator=g, device="cuda")
                              + torch.arange(N, device="cuda"))
        s["qw"] = s["kw"] = None
        if case["weights"]:
            s["qw"], s["kw"] = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
        if case["grad"]:
            s["dqo"], s["dko"] = normal(B, Hq, N, d).to(t), normal(B, Hk, N, d).to(t)
    elif case["op"] == "prefix":
        H, d, dv, n, most = case["H"], case["d"], case["dv"], case["n"], case["most"]
        s["table"] = _features(d, n)
        # the state of 512 tokens per head, each counted eight times over
        k, v = _unit(normal(H, 512, d)), normal(H, 512, dv)
        phi = _phi(k, s["table"])
        F = phi.shape[-1]
        logical = 8 * (phi.transpose(1, 2) @ torch.cat([v, torch.ones_like(v[..., :1])], -1))
        flat = torch.zeros(H, _stride(F, dv), device="cuda")
        flat[:, :F * dv] = logical[..., :dv].reshape(H, F * dv)
        flat[:, F * dv:F * (dv + 1)] = logical[..., dv]
        s["state"] = flat
        s["lengths"] = torch.tensor(_lengths(B, most), dtype=torch.int32, device="cuda")
        s["q"], s["k"], s["v"] = _unit(normal(B, H, d)).to(t), _unit(normal(B, H, d)).to(t), normal(B, H, dv).to(t)
        s["k_cache"], s["v_cache"] = _unit(normal(B, H, most + 1, d)).to(t), normal(B, H, most + 1, dv).to(t)
    else:
        N, D = case["N"], case["D"]
        # memories of a few to a few hundred tokens, by channel
        bias = 1 + 5 * torch.rand(D, generator=g, device="cuda")
        rows = (B, D) if case["form"] == "step" else (B, N, D)
        s["gate"], s["x"] = (normal(*rows) + bias).to(t), normal(*rows).to(t)
        s["h0"] = normal(B, D) if case["carried"] else None
        s["lengths"] = (torch.tensor([max(1, v) for v in _lengths(B, N)], dtype=torch.int32, device="cuda")
                        if case["ragged"] else None)
        if case["form"] == "train":
            s["dh"], s["dh_last"] = normal(B, N, D).to(t), normal(B, D)
    return s


# ------------------------------------------------------------------ the plain forms

def _turn(x, s, sign):
    """x [B, N, H, d] in 32 bits with its first `rot` entries rotated by the tokens' angles."""
    case, rot = s["case"], s["case"]["rot"]
    if not rot:
        return x
    pos = s["positions"] if s["positions"] is not None else torch.arange(x.shape[1], device=x.device)[None]
    angle = pos.double()[..., None] * torch.from_numpy(s["freqs"]).to(x.device)
    cos, sin = angle.cos().float()[:, :, None], sign * angle.sin().float()[:, :, None]
    if case["interleaved"]:
        one, two = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([one * cos - two * sin, two * cos + one * sin], -1).flatten(-2)
    else:
        one, two = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([one * cos - two * sin, two * cos + one * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _norm_rope(x, w, s):
    x = x.float()
    u = x * (x * x).sum(-1, keepdim=True).rsqrt()
    if w is not None:
        u = u * w
    return _turn(u, s, 1.0).transpose(1, 2)


def _norm_rope_grad(x, w, dy, s):
    x = x.float()
    inv = (x * x).sum(-1, keepdim=True).rsqrt()
    unit = x * inv
    du = _turn(dy.float().transpose(1, 2), s, -1.0)
    dw = (du * unit).sum((0, 1, 2)) if w is not None else None
    dunit = du if w is None else du * w
    return inv * (dunit - unit * (unit * dunit).sum(-1, keepdim=True)), dw


def _run_qk(s):
    case, t = s["case"], DTYPES[s["case"]["dtype"]]
    if own:
        from recurrent_states_b200 import taylor_attn as TA

        more = dict(positions=s["positions"], q_weight=s["qw"], k_weight=s["kw"], interleaved=case["interleaved"])
        f32 = case["dtype"] == "f32"
        forward = TA.taylor_attn_qk_norm_rope_f32 if f32 else TA.taylor_attn_qk_norm_rope
        q_out, k_out = forward(s["q"], s["k"], s["freqs"], **more)
        out = {"q_out": q_out, "k_out": k_out}
        if case["grad"]:
            backward = TA.taylor_attn_qk_norm_rope_backward_f32 if f32 else TA.taylor_attn_qk_norm_rope_backward
            dq, dk, dqw, dkw = backward(s["q"], s["k"], s["dqo"], s["dko"], s["freqs"], **more)
            out |= {"dq": dq, "dk": dk}
            if case["weights"]:
                out |= {"dqw": dqw, "dkw": dkw}
        return out
    out = {"q_out": _norm_rope(s["q"], s["qw"], s).to(t).contiguous(),
           "k_out": _norm_rope(s["k"], s["kw"], s).to(t).contiguous()}
    if case["grad"]:
        dq, dqw = _norm_rope_grad(s["q"], s["qw"], s["dqo"], s)
        dk, dkw = _norm_rope_grad(s["k"], s["kw"], s["dko"], s)
        out |= {"dq": dq.to(t), "dk": dk.to(t)}
        if case["weights"]:
            out |= {"dqw": dqw, "dkw": dkw}
    return out


def _series(x, n):
    return sum(x ** m / math.factorial(m) for m in range(n))


def _run_prefix(s):
    case = s["case"]
    B, H, d, dv, n = (case[c] for c in ("B", "H", "d", "dv", "n"))
    if own:
        from recurrent_states_b200 import taylor_attn as TA

        f32 = case["dtype"] == "f32"
        decode = TA.taylor_attn_shared_prefix_decode_f32 if f32 else TA.taylor_attn_shared_prefix_decode
        out = decode(s["q"], s["k"], s["v"], s["state"], s["k_cache"], s["v_cache"], s["lengths"], n, TAU)
        return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    at = s["lengths"].long()
    row = torch.arange(B, device=at.device)
    s["k_cache"][row, :, at] = s["k"]
    s["v_cache"][row, :, at] = s["v"]
    q = s["q"].float()
    coeff = torch.cat([torch.full((len(t),), TAU ** m / math.factorial(m), device=q.device)
                       for m, (t, _) in enumerate(s["table"])])
    phi = (_phi(q, s["table"]) * coeff).transpose(0, 1)
    F = phi.shape[-1]
    num = phi @ s["state"][:, :F * dv].unflatten(1, (F, dv))
    den = phi @ s["state"][:, F * dv:F * (dv + 1), None]
    score = (s["k_cache"].float() @ q[..., None])[..., 0] * TAU
    seen = torch.arange(score.shape[-1], device=at.device) <= at[:, None, None]
    weight = torch.where(seen, _series(score, n), 0.0)
    num = num.transpose(0, 1) + (weight[:, :, None] @ s["v_cache"].float())[:, :, 0]
    den = den.transpose(0, 1) + weight.sum(-1, keepdim=True)
    return {"out": num / den, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from zero, by doubling: after a round every row holds the sum over
    twice as many tokens. A scan with products has no elementary operation, so these are the rounds."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return b


def _run_gate(s):
    case, t = s["case"], DTYPES[s["case"]["dtype"]]
    coupled, form = case["coupled"], case["form"]
    if own:
        from recurrent_states_b200 import taylor_attn as TA

        f32 = case["dtype"] == "f32"
        if form == "step":
            step = TA.taylor_attn_gated_step_f32 if f32 else TA.taylor_attn_gated_step
            state = torch.empty_like(s["h0"])
            out = step(s["gate"], s["x"], s["h0"], coupled=coupled, state_out=state)
            return {"out": out, "state": state}
        forward = TA.taylor_attn_gated_scan_f32 if f32 else TA.taylor_attn_gated_scan
        h, h_last = forward(s["gate"], s["x"], coupled=coupled, h0=s["h0"], lengths=s["lengths"], h_last=True)
        out = {"h": h, "h_last": h_last}
        if form == "train":
            backward = TA.taylor_attn_gated_scan_backward_f32 if f32 else TA.taylor_attn_gated_scan_backward
            dgate, dx, dh0 = backward(s["gate"], s["x"], h, s["dh"], coupled=coupled, h0=s["h0"],
                                      lengths=s["lengths"], dh_last=s["dh_last"], dh0=case["carried"])
            out |= {"dgate": dgate, "dx": dx}
            if case["carried"]:
                out["dh0"] = dh0
        return out
    gate, x = s["gate"].float(), s["x"].float()
    a, keep = torch.sigmoid(gate), torch.sigmoid(-gate)
    b = keep * x if coupled else x
    if form == "step":
        state = a * s["h0"] + b
        return {"out": state.to(t), "state": state}
    live = None
    if s["lengths"] is not None:  # a padded row keeps the state
        live = (torch.arange(a.shape[1], device=a.device) < s["lengths"][:, None])[..., None]
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros_like(a[:, 0])
    h = _scan(a, torch.cat([b[:, :1] + a[:, :1] * h0[:, None], b[:, 1:]], 1))
    out = {"h": (h if live is None else torch.where(live, h, 0.0)).to(t), "h_last": h[:, -1]}
    if form == "train":
        dh = s["dh"].float() if live is None else torch.where(live, s["dh"].float(), 0.0)
        after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_last"][:, None]], 1)
        grad = _scan(after.flip(1), dh.flip(1)).flip(1)
        before = torch.cat([h0[:, None], h[:, :-1]], 1)
        dgate = grad * (before - x if coupled else before) * a * keep
        dx = grad * keep if coupled else grad
        if live is not None:
            dgate, dx = torch.where(live, dgate, 0.0), torch.where(live, dx, 0.0)
        out |= {"dgate": dgate.to(t), "dx": dx.to(t)}
        if case["carried"]:
            out["dh0"] = a[:, 0] * grad[:, 0]
    return out


def run(state):
    return {"qk": _run_qk, "prefix": _run_prefix, "gate": _run_gate}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    z, B = SIZE[case["dtype"]], case["B"]
    if case["op"] == "qk":
        values = B * case["N"] * (case["Hq"] + case["Hk"]) * case["d"]
        tables = (8 * B * case["N"] if case["given"] else 0) + (8 * case["d"] if case["weights"] else 0)
        nbytes, flops = 2 * values * z + tables, 7 * values
        if case["grad"]:  # the gradient reads the outputs' gradients too; q and k are read once for both
            nbytes, flops = nbytes + 2 * values * z + (8 * case["d"] if case["weights"] else 0), flops + 16 * values
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "prefix":
        H, d, dv, n = case["H"], case["d"], case["dv"], case["n"]
        F = math.comb(d + n - 1, n - 1)
        tokens = H * (sum(_lengths(B, case["most"])) + B)
        nbytes = 4 * H * F * (dv + 1) + tokens * (d + dv) * z + B * H * ((2 * d + dv) * z + 4 * dv) + 4 * B
        return {"bytes": nbytes, "flops": 2 * B * H * F * (dv + 1) + tokens * (2 * (d + dv + 1) + 2 * n)}
    values = B * case["N"] * case["D"]
    if case["ragged"]:
        values = sum(max(1, v) for v in _lengths(B, case["N"])) * case["D"]
    out = B * case["N"] * case["D"]  # a padded row is written too
    nbytes, flops = (2 * values + out) * z + 4 * B * case["D"] * (2 if case["carried"] else 1), 12 * values
    if case["form"] == "train":
        nbytes += (values + 2 * out) * z + 4 * B * case["D"] * (2 if case["carried"] else 1)
        flops += 16 * values
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ in 64 bits, from the definitions

def _exact_qk(case, s):
    d, rot = case["d"], case["rot"]

    def pairs(x):  # [..., rot] -> complex [..., rot / 2]
        return (torch.view_as_complex(x.unflatten(-1, (rot // 2, 2)).contiguous()) if case["interleaved"]
                else torch.complex(x[..., :rot // 2], x[..., rot // 2:]))

    def flat(z):
        return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)

    pos = s["positions"] if s["positions"] is not None else torch.arange(case["N"], device="cuda")[None]
    theta = pos.double()[:, None, :, None] * torch.tensor(s["freqs"], device="cuda")
    spin = torch.polar(torch.ones_like(theta), theta)

    def turn(x, by):
        return torch.cat([flat(pairs(x[..., :rot]) * by), x[..., rot:]], -1) if rot else x

    out, grads, weights = {}, {}, {}
    for c in "qk":
        x = s[c].double().permute(0, 2, 1, 3)
        w = s[c + "w"].double() if case["weights"] else torch.ones(d, dtype=torch.float64, device="cuda")
        length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        out[c + "_out"] = turn(x / length * w, spin)
        if case["grad"]:
            du = turn(s[f"d{c}o"].double(), spin.conj())
            weights[f"d{c}w"] = torch.einsum("bhnd,bhnd->d", du, x / length)
            along = torch.einsum("bhnd,bhnd->bhn", du * w, x)[..., None] / length ** 2
            grads["d" + c] = ((du * w - along * x) / length).permute(0, 2, 1, 3)
    return out | grads | (weights if case["weights"] else {})


def _exact_prefix(case, s):
    B, H, d, dv, n = (case[c] for c in ("B", "H", "d", "dv", "n"))
    q = s["q"].double().cpu().numpy()
    F = math.comb(d + n - 1, n - 1)
    flat = s["state"].double().cpu().numpy()
    table = np.concatenate([flat[:, :F * dv].reshape(H, F, dv), flat[:, F * dv:F * (dv + 1), None]], -1)
    phi, f = np.empty((H, B, F)), 0
    for m in range(n):
        for t in itertools.combinations_with_replacement(range(d), m):
            # tau^m / m! sqrt(m!/alpha!) on the query's side
            value = TAU ** m / math.sqrt(math.factorial(m) * math.prod(math.factorial(t.count(i)) for i in set(t)))
            for i in t:
                value = value * q[:, :, i].T
            phi[:, :, f] = value
            f += 1
    y = phi @ table
    at, out = s["lengths"].tolist(), np.empty((B, H, dv))
    for b in range(B):
        keys = torch.cat([s["k_cache"][b, :, :at[b]], s["k"][b, :, None]], 1).double().cpu().numpy()
        values = torch.cat([s["v_cache"][b, :, :at[b]], s["v"][b, :, None]], 1).double().cpu().numpy()
        x = TAU * np.einsum("hld,hd->hl", keys, q[b])
        w = np.ones_like(x)
        for m in range(n - 1, 0, -1):
            w = 1 + w * x / m
        out[b] = (y[:, b, :dv] + np.einsum("hl,hlc->hc", w, values)) / (y[:, b, dv] + w.sum(1))[:, None]
    return {"out": torch.from_numpy(out), "k_cache": None, "v_cache": None}


def _exact_gate(case, s):
    step = case["form"] == "step"
    gate, x = s["gate"].double(), s["x"].double()
    gate, x = (gate[:, None], x[:, None]) if step else (gate, x)
    B, N, D = gate.shape
    a = 1 / (1 + torch.exp(-gate))
    scale = 1 / (1 + torch.exp(gate)) if case["coupled"] else torch.ones_like(gate)
    state = s["h0"].double() if case["carried"] else torch.zeros(B, D, dtype=torch.float64, device="cuda")
    start, live = state, None
    if s["lengths"] is not None:
        live = torch.arange(N, device="cuda")[:, None] < s["lengths"][None, :]
    h = torch.zeros_like(gate)
    for i in range(N):
        new = a[:, i] * state + scale[:, i] * x[:, i]
        state = new if live is None else torch.where(live[i][:, None], new, state)
        h[:, i] = state if live is None else state * live[i][:, None]
    if step:
        return {"out": state, "state": state}
    out = {"h": h, "h_last": state}
    if case["form"] == "train":
        dgate, dx, carry = torch.zeros_like(gate), torch.zeros_like(gate), s["dh_last"].double()
        for i in range(N - 1, -1, -1):
            g = carry + s["dh"][:, i].double()
            before = h[:, i - 1] if i else start
            da = g * (before - x[:, i] if case["coupled"] else before)
            row, on = da * a[:, i] * (1 / (1 + torch.exp(gate[:, i]))), 1.0
            if live is not None:
                on = live[i][:, None].double()
            dgate[:, i], dx[:, i] = on * row, on * (g * scale[:, i])
            back = g * a[:, i]
            carry = back if live is None else torch.where(live[i][:, None], back, carry)
        out |= {"dgate": dgate, "dx": dx}
        if case["carried"]:
            out["dh0"] = carry
    return out


def exact(case, seed):
    if case["op"] == "gate" and case["N"] > 20_000:
        return None  # one row after another: over half a minute
    return {"qk": _exact_qk, "prefix": _exact_prefix, "gate": _exact_gate}[case["op"]](case, prepare(case, seed))
