"""The operators around the scan in CUDA graphs and back to back: every kernel may
begin while the one before it ends, so a chain of calls on changing buffers has to
give what the same calls give one at a time."""
import pytest
import torch

from linear_recurrence_scan_lrscan_gb300 import lrscan as L

pytestmark = pytest.mark.gpu


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    B, T, D, V = 3, 210, 192, 500
    return {"ids": torch.randint(-1, V, (B, T), generator=g).cuda(), "table": n(V, D), "w": n(D, 4) / 2, "bias": n(D),
            "r": n(B, T, D), "i": n(B, T, D), "lam": torch.linspace(-8.0, -4.0, D).cuda(), "go": n(B, T, D),
            "windows": n(5, 3, D), "states": n(5, D), "slots": torch.tensor([4, 0, 2], dtype=torch.int32).cuda()}


def chain(s, out):
    """Each call reads what the one before it wrote."""
    L.lrscan_fwd_embed(s["ids"], s["table"], scale=0.5, out=out["x"])
    L.lrscan_fwd_conv(out["x"], s["w"], s["bias"], out=out["u"])
    L.lrscan_fwd_gates(s["r"], s["i"], out["u"], s["lam"], out=out["h"], last=out["last"], saved=out["saved"])
    L.lrscan_bwd_gates(s["r"], s["i"], out["u"], s["lam"], out["saved"], s["go"], grad_r=out["gr"], grad_i=out["gi"],
                       grad_x=out["gu"], grad_lam=out["glam"], want_grad_h0=False)
    L.lrscan_bwd_conv(out["x"], s["w"], out["gu"], grad_x=out["gx"], grad_w=out["gw"], grad_bias=out["gb"])
    L.lrscan_bwd_embed(s["ids"], out["gx"], s["table"].shape[0], scale=0.5, grad_weight=out["gtable"])
    L.lrscan_step_conv(out["gx"][:, -1], s["w"], out["windows"], bias=s["bias"], slots=s["slots"], out=out["u1"])
    L.lrscan_step_gates(s["r"][:, -1], s["i"][:, -1], out["u1"], s["lam"], out["states"], slots=s["slots"], out=out["h1"])


def outputs(s):
    B, T, D = s["r"].shape
    e = lambda *shape: torch.full(shape, float("nan"), device="cuda")  # noqa: E731
    out = {k: e(B, T, D) for k in ("x", "u", "h", "gr", "gi", "gu", "gx")}
    out.update(last=e(B, D), saved=e(B, (T + 15) // 16, D), glam=e(D), gw=e(D, 4), gb=e(D), gtable=e(*s["table"].shape),
               u1=e(B, D), h1=e(B, D), windows=s["windows"].clone(), states=s["states"].clone())
    return out


def apart(s):
    """The same calls, each finished before the next."""
    out = outputs(s)
    names = [n for n in dir(L) if n.startswith("lrscan_") and n.split("_")[1] in ("fwd", "bwd", "step")]
    kept = {n: getattr(L, n) for n in names}
    try:
        for n, f in kept.items():
            setattr(L, n, lambda *a, f=f, **k: (f(*a, **k), torch.cuda.synchronize())[0])
        chain(s, out)
    finally:
        for n, f in kept.items():
            setattr(L, n, f)
    return out


def same(got, want):
    for k in want:
        assert torch.isfinite(want[k]).all() and torch.equal(got[k], want[k]), k


def test_calls_back_to_back():
    sets = [inputs(k) for k in range(3)]
    want = [apart(s) for s in sets]
    outs = [[outputs(s) for s in sets] for _ in range(4)]
    torch.cuda.synchronize()
    for turn in outs:
        for s, out in zip(sets, turn):
            chain(s, out)
    assert L.lrscan_sync_check() == 0
    for turn in outs:
        for out, w in zip(turn, want):
            same(out, w)


def test_chain_in_a_graph():
    s = inputs(7)
    want = apart(s)
    st = torch.cuda.Stream()
    out = outputs(s)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        chain(s, out)  # scratch is made before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        chain(s, out)
    for _ in range(3):
        for k, v in outputs(s).items():
            out[k].copy_(v)
        graph.replay()
    torch.cuda.synchronize()
    same(out, want)
    assert L.lrscan_sync_check() == 0
