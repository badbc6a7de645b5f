"""What is measured of the operators of a recurrent language model's layer.

Three operators that a training or serving step runs around the diagonal scan:

  gates   the gated linear recurrence: decays and inputs made from gates in
          the same pass as the scan,
              rg = sigmoid(r), ig = sigmoid(i), log a = -c softplus(lam) rg,
              h_t = a_t h_{t-1} + sqrt(1 - a_t^2) ig_t x_t      (c = 8)
          (a_t = 0 where segment_pos is 0), its backward pass, and its form
          for single tokens on a pool of states;
  conv    the short causal convolution of each channel in front of it,
              y_t = bias + sum_k w[K-1-k] x_{t-k}
          within a segment, its backward pass, and its single-token form;
  embed   the embedding lookup with scaling, scale * weight[ids] (a row of
          zeros for a negative id), and its gradient, a sum over the tokens.

``run`` computes them in plain torch operations, or (``own``) by the calls of
this package.  A plain scan in time takes log2(T) vectorised doubling steps:
the one loop of the plain form.
"""
import math

import numpy as np
import torch

own = False

C = 8.0  # the decay's exponent scale
K = 4    # taps of the causal convolution
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode step of 32 running requests: one token each, states in a pool
        {"name": "gates step 32", "kind": "gates_step", "B": 32, "D": 2560, "dtype": "bf16"},
        # the prefill of a prompt that continues an earlier one (carried state), an odd length
        {"name": "gates prefill odd", "kind": "gates_fwd", "B": 1, "T": 1999, "D": 2560, "dtype": "bf16", "carry": True},
        # a training step's forward and backward on the package's gated workload; r and i are halves of one projection
        {"name": "gates train bf16", "kind": "gates_train", "B": 8, "T": 2048, "D": 2560, "dtype": "bf16", "fused": True},
        # long packed documents in fp32: the package's long-sequence workload with restarts
        {"name": "gates train long", "kind": "gates_train", "B": 1, "T": 65536, "D": 2560, "dtype": "f32", "packed": 1500},
        # few channels and a very long sequence (bytes or audio frames)
        {"name": "gates fwd few lanes", "kind": "gates_fwd", "B": 1, "T": 1 << 20, "D": 64, "dtype": "bf16"},
        # odd sizes throughout: rows that no 16-byte copy can start on
        {"name": "gates train ragged", "kind": "gates_train", "B": 3, "T": 777, "D": 1001, "dtype": "bf16", "packed": 100},
        # the convolution of the same training step, on packed documents
        {"name": "conv train bf16", "kind": "conv_train", "B": 8, "T": 2048, "D": 2560, "dtype": "bf16", "packed": 400},
        # the convolution of a decode step
        {"name": "conv step 32", "kind": "conv_step", "B": 32, "D": 2560, "dtype": "bf16"},
        # the tokens of a training step, table in fp32 and activations in bf16
        {"name": "embed lookup", "kind": "embed_fwd", "N": 16384, "V": 32768, "D": 2560, "weight": "f32", "dtype": "bf16"},
        # their gradient: token frequencies fall as in text, so that a few rows collect many tokens
        {"name": "embed grad", "kind": "embed_bwd", "N": 16384, "V": 32768, "D": 2560, "weight": "f32", "dtype": "bf16"},
        # a small odd table in one type, padded batch
        {"name": "embed grad odd", "kind": "embed_bwd", "N": 3001, "V": 5003, "D": 777, "weight": "bf16", "dtype": "bf16", "pad": True},
        # the lookup of a decode step
        {"name": "embed lookup 32", "kind": "embed_fwd", "N": 32, "V": 32768, "D": 2560, "weight": "bf16", "dtype": "bf16"},
    ]


def _size(rng, lo, hi, unit=1):
    """A power of two times `unit` (half of the time) or an odd multiple of `unit`, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    if rng.random() < 0.5:
        return max(lo, min(hi, 2 ** int(round(math.log2(v)))))
    return max(unit, min(hi, (int(v / unit) // 2 * 2 + 1) * unit))


def draw(rng):
    kind = rng.choice(["gates_step", "gates_fwd", "gates_train", "gates_train", "conv_train", "conv_step", "embed_fwd", "embed_bwd"])
    case = {"kind": kind, "D": _size(rng, 64, 4096, rng.choice([1, 8, 8, 8]))}
    if kind.startswith("embed"):
        case["N"] = _size(rng, 1, min(65536, (1 << 26) // case["D"]))
        case["V"] = _size(rng, 256, min(131072, (1 << 27) // case["D"]))
        case["weight"], case["dtype"] = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
        case["pad"] = rng.random() < 0.3
        return case
    case["dtype"] = rng.choice(["bf16", "f32"])
    if kind.endswith("step"):
        case["B"] = _size(rng, 1, 512)
        return case
    case["B"] = _size(rng, 1, 32)
    case["T"] = _size(rng, 1, max(2, min(131072, (1 << 25) // (case["B"] * case["D"]))))
    if rng.random() < 0.5:
        case["packed"] = _size(rng, 16, 2048)
    if kind != "conv_train":
        case["carry"] = rng.random() < 0.5
        case["fused"] = rng.random() < 0.5
    return case


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _positions(gen, B, T, mean):
    """int32 [B, T] positions within documents of about `mean` tokens, packed one after another."""
    start = torch.rand((B, T), generator=gen, device="cuda") < 1.0 / mean
    start[:, 0] = True
    t = torch.arange(T, device="cuda").expand(B, T)
    return (t - torch.cummax(torch.where(start, t, 0), dim=1).values).to(torch.int32)


def _frequencies(V):
    p = 1.0 / (np.arange(V) + 2.7)  # token frequencies by rank
    return p / p.sum()


def _tokens(gen, case):
    p = torch.from_numpy(np.cumsum(_frequencies(case["V"]))).to("cuda", torch.float32)
    rank = torch.searchsorted(p, torch.rand(case["N"], generator=gen, device="cuda")).clamp_(max=case["V"] - 1)
    names = torch.randperm(case["V"], generator=gen, device="cuda")  # an id says nothing of its frequency
    ids = names[rank]
    if case.get("pad"):
        ids = torch.where(torch.rand(case["N"], generator=gen, device="cuda") < 0.2, -1, ids)
    return ids


def prepare(case, seed):
    gen, kind, D = _generator(seed), case["kind"], case["D"]
    dt = DTYPES[case["dtype"]]
    s = {"kind": kind}
    if kind.startswith("embed"):
        s["ids"] = _tokens(gen, case)
        s["V"], s["scale"], s["dtype"], s["weight_dtype"] = case["V"], math.sqrt(D), dt, DTYPES[case["weight"]]
        if kind == "embed_fwd":
            s["weight"] = _normal(gen, (case["V"], D), torch.float32).mul_(D ** -0.5).to(s["weight_dtype"])
        else:
            s["grad_out"] = _normal(gen, (case["N"], D), dt)
        return s
    B = case["B"]
    if kind.startswith("gates"):
        u = torch.empty(D, device="cuda").uniform_(0.9, 0.999, generator=gen)
        s["lam"] = torch.log(torch.expm1(-torch.log(u) / C))  # a = u where the recurrence gate is open
    else:
        s["w"] = _normal(gen, (D, K), torch.float32).mul_(K ** -0.5)
        s["bias"] = _normal(gen, (D,), torch.float32).mul_(0.1)
    if kind.endswith("step"):
        s["slots"] = torch.randperm(2 * B, generator=gen, device="cuda")[:B].to(torch.int32)
        s["x"] = _normal(gen, (B, D), dt)
        if kind == "gates_step":
            s["r"], s["i"] = _normal(gen, (B, D), dt), _normal(gen, (B, D), dt)
            s["state"] = _normal(gen, (2 * B, D), torch.float32)
        else:
            s["state"] = _normal(gen, (2 * B, K - 1, D), dt)
        return s
    T = case["T"]
    s["x"] = _normal(gen, (B, T, D), dt)
    s["segment_pos"] = _positions(gen, B, T, case["packed"]) if case.get("packed") else None
    s["grad_out"] = _normal(gen, (B, T, D), dt) if kind.endswith("train") else None
    if kind.startswith("gates"):
        if case.get("fused"):
            both = _normal(gen, (B, T, 2 * D), dt)
            s["r"], s["i"] = both[..., :D], both[..., D:]
        else:
            s["r"], s["i"] = _normal(gen, (B, T, D), dt), _normal(gen, (B, T, D), dt)
        s["h0"] = _normal(gen, (B, D), torch.float32) if case.get("carry") else None
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1, by doubling: after a step of distance n each pair holds the map of 2n tokens."""
    a, h, n = a.clone(), b.clone(), 1
    while n < h.shape[1]:
        h[:, n:] += a[:, n:] * h[:, :-n].clone()
        a[:, n:] *= a[:, :-n].clone()
        n *= 2
    return h


def _gates(s):
    r, i = torch.sigmoid(s["r"].float()), torch.sigmoid(s["i"].float())
    la = (-C * torch.log1p(torch.exp(s["lam"]))) * r
    a, m = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    return r, i, la, a, m


def _plain_gates(s):
    r, i, la, a, m = _gates(s)
    dt, x, h0 = s["x"].dtype, s["x"].float(), s["h0"]
    if s["segment_pos"] is not None:
        first = (s["segment_pos"] == 0)[..., None]
        a, m = torch.where(first, 0.0, a), torch.where(first, 1.0, m)
    b = m * i * x
    if h0 is not None:
        b[:, 0] += a[:, 0] * h0
    h = _scan(a, b)
    if s["grad_out"] is None:
        return h.to(dt), h[:, -1].clone()
    # g_t = grad_out_t + a_{t+1} g_{t+1}
    up = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _scan(up.flip(1), s["grad_out"].float().flip(1)).flip(1)
    before = torch.cat([h[:, :1] * 0 if h0 is None else h0[:, None], h[:, :-1]], 1)
    gla = g * (before * a - i * x * a * a / m)  # the gradient of log a; none where a is 0
    gr = gla * la * (1 - r)
    gi = g * m * x * i * (1 - i)
    glam = (gla * r).sum((0, 1)) * (-C) * torch.sigmoid(s["lam"])
    grads = [gr.to(dt), gi.to(dt), (g * m * i).to(dt), glam]
    return [h.to(dt), h[:, -1].clone(), *grads] + ([] if h0 is None else [a[:, 0] * g[:, 0]])


def _plain_gates_step(s):
    r, i, la, a, m = _gates(s)
    h = a * s["state"][s["slots"].long()] + m * i * s["x"].float()
    s["state"][s["slots"].long()] = h
    return h.to(s["x"].dtype), s["state"]


def _shifted(x, k, seg):
    """x_{t-k}, or 0 before the segment's first token."""
    y = torch.cat([torch.zeros_like(x[:, :k]), x[:, : max(0, x.shape[1] - k)]], 1)
    return y if seg is None or k == 0 else torch.where((seg >= k)[..., None], y, 0.0)


def _advanced(g, k, seg):
    """g_{t+k} where token t is in the segment of token t+k, or 0."""
    g = g if seg is None or k == 0 else torch.where((seg >= k)[..., None], g, 0.0)
    return torch.cat([g[:, k:], torch.zeros_like(g[:, :k])], 1)


def _plain_conv(s):
    x, g, w, seg = s["x"].float(), s["grad_out"].float(), s["w"], s["segment_pos"]
    y = s["bias"] + sum(w[:, K - 1 - k] * _shifted(x, k, seg) for k in range(K))
    gx = sum(w[:, K - 1 - k] * _advanced(g, k, seg) for k in range(K))
    gw = torch.stack([(g * _shifted(x, K - 1 - k, seg)).sum((0, 1)) for k in range(K)], 1)
    return y.to(s["x"].dtype), gx.to(s["x"].dtype), gw, g.sum((0, 1))


def _plain_conv_step(s):
    at = s["slots"].long()
    window = torch.cat([s["state"][at], s["x"][:, None]], 1)
    s["state"][at] = window[:, 1:]
    return (s["bias"] + (window.float() * s["w"].t()).sum(1)).to(s["x"].dtype), s["state"]


def _plain_embed(s):
    rows = s["weight"][s["ids"].clamp(min=0)].float() * s["scale"]
    return torch.where((s["ids"] >= 0)[:, None], rows, 0.0).to(s["dtype"])


def _plain_embed_grad(s):
    rows = torch.where((s["ids"] >= 0)[:, None], s["grad_out"].float(), 0.0)
    total = torch.zeros((s["V"], rows.shape[1]), device=rows.device)
    total.index_add_(0, s["ids"].clamp(min=0), rows)
    return (total * s["scale"]).to(s["weight_dtype"])


PLAIN = {"gates_step": _plain_gates_step, "gates_fwd": _plain_gates, "gates_train": _plain_gates, "conv_train": _plain_conv,
         "conv_step": _plain_conv_step, "embed_fwd": _plain_embed, "embed_bwd": _plain_embed_grad}


# --------------------------------------------------------------------------
# the package's operators
# --------------------------------------------------------------------------
def _own(s):
    from linear_recurrence_scan_lrscan_gb300 import lrscan as L
    kind = s["kind"]
    if kind == "gates_step":
        return L.lrscan_step_gates(s["r"], s["i"], s["x"], s["lam"], s["state"], slots=s["slots"]), s["state"]
    if kind == "conv_step":
        return L.lrscan_step_conv(s["x"], s["w"], s["state"], bias=s["bias"], slots=s["slots"]), s["state"]
    if kind == "gates_fwd":
        return L.lrscan_fwd_gates(s["r"], s["i"], s["x"], s["lam"], h0=s["h0"], segment_pos=s["segment_pos"])[:2]
    if kind == "gates_train":
        out, last, saved = L.lrscan_fwd_gates(s["r"], s["i"], s["x"], s["lam"], h0=s["h0"], segment_pos=s["segment_pos"],
                                              want_saved=True)
        grads = L.lrscan_bwd_gates(s["r"], s["i"], s["x"], s["lam"], saved, s["grad_out"], segment_pos=s["segment_pos"],
                                   want_grad_h0=s["h0"] is not None)
        return [out, last, *grads[:4]] + ([] if s["h0"] is None else [grads[4]])
    if kind == "conv_train":
        out, _ = L.lrscan_fwd_conv(s["x"], s["w"], s["bias"], segment_pos=s["segment_pos"])
        return out, *L.lrscan_bwd_conv(s["x"], s["w"], s["grad_out"], segment_pos=s["segment_pos"])[:3]
    if kind == "embed_fwd":
        return L.lrscan_fwd_embed(s["ids"], s["weight"], scale=s["scale"], dtype=s["dtype"])
    return L.lrscan_bwd_embed(s["ids"], s["grad_out"], s["V"], scale=s["scale"], dtype=s["weight_dtype"])


def run(state):
    return _own(state) if own else PLAIN[state["kind"]](state)


# --------------------------------------------------------------------------
# the definition in 64 bits, and what a pass cannot do without
# --------------------------------------------------------------------------
def _walk(a, b, h):
    """h_t = a_t h_{t-1} + b_t token by token, in blocks of about sqrt(T) tokens that walk side by side."""
    B, T, D = a.shape
    n = max(1, int(math.isqrt(T)))
    m = -(-T // n)
    a = torch.cat([a, torch.ones((B, m * n - T, D), device=a.device, dtype=a.dtype)], 1).view(B, m, n, D)
    b = torch.cat([b, torch.zeros((B, m * n - T, D), device=b.device, dtype=b.dtype)], 1).view(B, m, n, D)
    out, prod, p, q = torch.empty_like(b), torch.empty_like(a), torch.ones_like(a[:, :, 0]), torch.zeros_like(a[:, :, 0])
    for t in range(n):
        q = a[:, :, t] * q + b[:, :, t]
        p = p * a[:, :, t]
        out[:, :, t], prod[:, :, t] = q, p
    for j in range(m):
        out[:, j] += prod[:, j] * h[:, None]
        h = out[:, j, -1].clone()
    return out.view(B, m * n, D)[:, :T]


def _exact_gates(s):
    f = torch.float64
    x, lam = s["x"].to(f), s["lam"].to(f)
    rg, ig = 1 / (1 + torch.exp(-s["r"].to(f))), 1 / (1 + torch.exp(-s["i"].to(f)))
    sp = torch.nn.functional.softplus(lam, threshold=1000.0)
    la = -C * sp * rg
    a = torch.exp(la)
    m2 = -torch.expm1(2 * la)
    if s["kind"] == "gates_step":
        at = s["slots"].long()
        state = s["state"].to(f)
        state[at] = a * state[at] + m2.sqrt() * ig * x
        return state[at], state
    B, T, D = x.shape
    seg = torch.ones((B, T), device=x.device) if s["segment_pos"] is None else s["segment_pos"]
    keep = (seg != 0).to(f)[..., None]
    m = torch.where(keep > 0, m2, torch.ones_like(m2)).sqrt()
    h0 = torch.zeros((B, D), device=x.device, dtype=f) if s["h0"] is None else s["h0"].to(f)
    h = _walk(a * keep, m * ig * x, h0)
    if s["grad_out"] is None:
        return h, h[:, -1]
    # c_t = a_t g_t is what token t hands to token t-1: c_t = a_t grad_out_t + a_t c_{t+1}
    ak = (a * keep).flip(1)
    go = s["grad_out"].to(f)
    c = _walk(ak, ak * go.flip(1), torch.zeros_like(h0)).flip(1)
    g = go + torch.cat([c[:, 1:], torch.zeros_like(c[:, :1])], 1)
    del ak, go
    prev = torch.cat([h0[:, None], h[:, :-1]], 1)
    # d/d(log a) of a h_{t-1} + sqrt(1 - a^2) i x
    q = g * keep * a * (prev - a / m * ig * x)
    grads = [q * -C * sp * rg * (1 - rg), g * m * x * ig * (1 - ig), g * m * ig, (q * -C * rg).sum((0, 1)) / (1 + torch.exp(-lam))]
    return [h, h[:, -1], *grads] + ([] if s["h0"] is None else [c[:, 0]])


def _exact_conv(s):
    f = torch.float64
    x, w, bias = s["x"].to(f), s["w"].to(f), s["bias"].to(f)
    if s["kind"] == "conv_step":
        at, state = s["slots"].long(), s["state"].to(f)
        y = bias + w[:, K - 1] * x
        for k in range(1, K):
            y = y + w[:, K - 1 - k] * state[at, K - 1 - k]
        state[at] = torch.cat([state[at, 1:], x[:, None]], 1)
        return y, state
    g = s["grad_out"].to(f)
    T = x.shape[1]
    seg = torch.full(x.shape[:2], T + K, device=x.device) if s["segment_pos"] is None else s["segment_pos"]
    y, gx, gw = bias.expand_as(x).clone(), torch.zeros_like(x), torch.zeros_like(w)
    for k in range(min(K, T)):
        inside = (seg[:, k:] >= k).to(f)[..., None]
        y[:, k:] += w[:, K - 1 - k] * x[:, : T - k] * inside
        gx[:, : T - k] += w[:, K - 1 - k] * g[:, k:] * inside
        gw[:, K - 1 - k] = (g[:, k:] * x[:, : T - k] * inside).sum((0, 1))
    return y, gx, gw, g.sum((0, 1))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("gates"):
        return _exact_gates(s)
    if case["kind"].startswith("conv"):
        return _exact_conv(s)
    ids, f = s["ids"], torch.float64
    seen = ids >= 0
    if case["kind"] == "embed_fwd":
        out = torch.zeros((ids.numel(), case["D"]), device=ids.device, dtype=f)
        out[seen] = s["weight"].to(f)[ids[seen]] * s["scale"]
        return out
    return torch.zeros((s["V"], case["D"]), device=ids.device, dtype=f).index_add_(0, ids[seen], s["grad_out"].to(f)[seen]) * s["scale"]


def work(case):
    kind, D = case["kind"], case["D"]
    e = 4 if case["dtype"] == "f32" else 2
    if kind.startswith("embed"):
        N, V = case["N"], case["V"]
        we = 4 if case["weight"] == "f32" else 2
        tokens = N * (0.8 if case.get("pad") else 1.0)
        if kind == "embed_bwd":  # the tokens' gradients in, the table's gradient out
            return {"bytes": N * 8 + tokens * D * e + V * D * we, "flops": tokens * D + V * D}
        rows = float(np.sum(1 - (1 - _frequencies(V)) ** tokens))  # distinct ids expected
        return {"bytes": N * 8 + rows * D * we + N * D * e, "flops": N * D}
    if kind == "gates_step":  # r, i, x in, out out; the state in and out
        return {"bytes": case["B"] * D * (4 * e + 8) + 4 * D, "flops": 30 * case["B"] * D}
    if kind == "conv_step":  # x in, out out; the window in and out
        return {"bytes": case["B"] * D * e * (2 + 2 * (K - 1)) + D * 4 * (K + 1), "flops": 2 * K * case["B"] * D}
    n = case["B"] * case["T"] * D
    planes = {"gates_fwd": 4, "gates_train": 8, "conv_train": 4}[kind]
    flops = {"gates_fwd": 30, "gates_train": 90, "conv_train": 6 * K}[kind]
    return {"bytes": n * planes * e + (4 * case["B"] * case["T"] if case.get("packed") else 0), "flops": n * flops}
