"""GPU tests of the causal convolution against its definition in 64 bits: taps 2
to 8, both types, sizes around a walk's edges, restarts, carried tokens, both
gradients of them, strided rows, single tokens and refusals.

Bounds (u = 2^-24): an output is a sum of K + 1 products taken in fused
multiply-adds, so it is within (K + 1) u of the sum of its terms' magnitudes;
grad_w and grad_bias are sums of B T products, 32 in a walk, 8 walks, the CTAs'
sums every 32nd in a warp and 32 warps (64 slices where there are many), so
within (32 + 8 + rows / 32 + 32 + 66) u of theirs."""
import pytest
import torch

from gates_reference import U
from linear_recurrence_scan_lrscan_gb300 import lrscan as L

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.lib()
    yield
    assert L.lrscan_sync_check() == 0


def close(got, ref, bound, dtype, what):
    got, half = got.detach().double().cpu(), 2.0 ** -8 if dtype == torch.bfloat16 else U
    allowed = bound + half * (ref.abs() + bound) + 1e-37
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: not finite in other places"
    off = ((got - ref).abs() - allowed)[fine]
    assert off.numel() == 0 or off.max() <= 0, f"{what}: {int((off > 0).sum())} over the bound, by {off.max():.3g}"


def valid(seg, k, T):
    """[B, T] whether tap k of token t counts."""
    ok = torch.ones(seg.shape, dtype=torch.bool)
    for j in range(k):  # no restart at t - j
        s = torch.ones_like(ok)
        s[:, j:] = seg[:, : T - j] != 0 if j else seg != 0
        ok &= s
    return ok


def reference(x, w, bias, x0, seg, go=None, gl=None):
    """{name: (value, bound)}"""
    B, T, D = x.shape
    K = w.shape[1]
    f = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    x, w, bias, x0, go, gl = f(x), f(w), f(bias), f(x0), f(go), f(gl)
    seg = torch.ones((B, T), dtype=torch.int32) if seg is None else seg.cpu()
    ext = torch.cat([torch.zeros((B, K - 1, D), dtype=torch.float64) if x0 is None else x0, x], 1)
    y, my = torch.zeros_like(x), torch.zeros_like(x)
    gext, mext = torch.zeros_like(ext), torch.zeros_like(ext)
    gw, mw = torch.zeros_like(w), torch.zeros_like(w)
    for k in range(K):
        ok = valid(seg, k, T)[..., None]
        past = torch.where(ok, ext[:, K - 1 - k : K - 1 - k + T], 0.0)
        y += w[:, K - 1 - k] * past
        my += (w[:, K - 1 - k] * past).abs()
        if go is not None:
            g = torch.where(ok, go, 0.0)
            gext[:, K - 1 - k : K - 1 - k + T] += w[:, K - 1 - k] * g
            mext[:, K - 1 - k : K - 1 - k + T] += (w[:, K - 1 - k] * g).abs()
            gw[:, K - 1 - k] = (g * past).sum((0, 1))
            mw[:, K - 1 - k] = (g * past).abs().sum((0, 1))
    if bias is not None:
        y, my = y + bias, my + bias.abs()
    out = {"out": (y, (K + 1) * U * my), "last": (ext[:, T:], torch.zeros_like(ext[:, T:]))}
    if go is not None:
        if gl is not None:
            gext[:, T:] += gl
            mext[:, T:] += gl.abs()
        rows = B * ((T + 255) // 256)
        n = (32 + 8 + rows / 32 + 32 + 66) * U
        out |= {"grad_x": (gext[:, K - 1:], (K + 1) * U * mext[:, K - 1:]), "grad_x0": (gext[:, : K - 1], (K + 1) * U * mext[:, : K - 1]),
                "grad_w": (gw, n * mw), "grad_bias": (go.sum((0, 1)), n * go.abs().sum((0, 1)))}
    return out


def draw(B, T, D, K, dt, seed, *, carry, packed, wide=False):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dtype = DT[dt]
    x, go = n(B, T, 2 * D).to(dtype).cuda(), n(B, T, 2 * D).to(dtype).cuda()
    cut = (lambda t: t[..., D:]) if wide else (lambda t: t[..., D:].contiguous())
    seg = (torch.rand((B, T), generator=g) >= 1.0 / packed).to(torch.int32).cuda() if packed else None
    return {"x": cut(x), "go": cut(go), "w": n(D, K).cuda(), "bias": n(D).cuda(), "seg": seg, "dtype": dtype,
            "x0": n(B, K - 1, D).to(dtype).cuda() if carry else None,
            "gl": n(B, K - 1, D).to(dtype).cuda() if carry else None}


def check(s):
    out, last = L.lrscan_fwd_conv(s["x"], s["w"], s["bias"], x0=s["x0"], segment_pos=s["seg"], want_last=True)
    gx, gw, gb, g0 = L.lrscan_bwd_conv(s["x"], s["w"], s["go"], x0=s["x0"], segment_pos=s["seg"], grad_last=s["gl"],
                                       want_grad_x0=True)
    want = reference(s["x"], s["w"], s["bias"], s["x0"], s["seg"], s["go"], s["gl"])
    got = {"out": out, "last": last, "grad_x": gx, "grad_x0": g0, "grad_w": gw, "grad_bias": gb}
    for name, (ref, bound) in want.items():
        close(got[name], ref, bound, torch.float32 if name in ("grad_w", "grad_bias") else s["dtype"], name)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4, 5, 6, 7, 8])
def test_conv_every_tap_count(K, dt):
    check(draw(2, 67, 40, K, dt, K, carry=True, packed=9))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 1, 64), (2, 2, 129), (1, 32, 128), (2, 33, 132), (1, 256, 260), (2, 257, 127), (1, 1000, 33)])
def test_conv_sizes(shape, dt):
    check(draw(*shape, 4, dt, 20, carry=False, packed=0))
    check(draw(*shape, 4, dt, 21, carry=True, packed=5, wide=True))


def test_conv_many_rows_of_partial_sums():
    # 1300 CTAs in time: the reduction takes slices
    check(draw(26, 256 * 50 - 3, 8, 4, "f32", 22, carry=False, packed=100))


def test_conv_restart_stops_infinities_and_nan():
    s = draw(1, 80, 64, 4, "f32", 23, carry=True, packed=0)
    s["seg"] = torch.ones((1, 80), dtype=torch.int32, device="cuda")
    s["seg"][:, [0, 33, 50]] = 0
    s["x0"][:] = float("nan")
    s["x"][:, 32] = float("inf")
    s["x"][:, 49] = float("nan")
    out, _ = L.lrscan_fwd_conv(s["x"], s["w"], s["bias"], x0=s["x0"], segment_pos=s["seg"])
    bad = torch.zeros(80, dtype=torch.bool)
    bad[[32, 49]] = True
    assert torch.equal((~torch.isfinite(out)).all(2)[0].cpu(), bad) and torch.isfinite(out[:, ~bad.cuda()]).all()
    s["go"][:, 50] = float("inf")
    gx, _, _, g0 = L.lrscan_bwd_conv(s["x"], s["w"], s["go"], x0=s["x0"], segment_pos=s["seg"], want_grad_x0=True)
    assert torch.isfinite(gx[:, :50]).all() and torch.isfinite(gx[:, 51:]).all() and not g0.any()


def test_conv_two_calls_continue():
    s = draw(2, 100, 64, 4, "bf16", 24, carry=True, packed=30)
    # a restart less than three tokens back is not in the carried tokens: the second call begins at least 3 after one
    seg = s["seg"].clone()
    seg[:, 34:37] = 1
    o0, m0 = L.lrscan_fwd_conv(s["x"], s["w"], s["bias"], x0=s["x0"], segment_pos=seg, want_last=True)
    o1, mid = L.lrscan_fwd_conv(s["x"][:, :37], s["w"], s["bias"], x0=s["x0"], segment_pos=seg[:, :37].contiguous(),
                                want_last=True)
    o2, m2 = L.lrscan_fwd_conv(s["x"][:, 37:], s["w"], s["bias"], x0=mid, segment_pos=seg[:, 37:].contiguous(),
                               want_last=True)
    assert torch.equal(torch.cat([o1, o2], 1), o0) and torch.equal(m0, m2)


def test_conv_empty():
    x = torch.empty((2, 0, 16), device="cuda")
    w, x0 = torch.randn((16, 4), device="cuda"), torch.randn((2, 3, 16), device="cuda")
    _, last = L.lrscan_fwd_conv(x, w, x0=x0, want_last=True)
    assert torch.equal(last, x0)
    _, gw, gb, g0 = L.lrscan_bwd_conv(x, w, x, grad_last=x0, want_grad_x0=True)
    assert not gw.any() and not gb.any() and torch.equal(g0, x0)


def test_conv_autograd_differences_and_repeat():
    s = draw(2, 45, 36, 4, "f32", 25, carry=True, packed=11)
    leaves = [s[k].clone().requires_grad_() for k in ("x", "w", "bias", "x0")]
    out, last = L.causal_conv(*leaves, segment_pos=s["seg"])
    ((out * s["go"]).sum() + (last * s["gl"]).sum()).backward()
    want = reference(s["x"], s["w"], s["bias"], s["x0"], s["seg"], s["go"], s["gl"])
    go, gl = s["go"].double().cpu(), s["gl"].double().cpu()
    gen = torch.Generator().manual_seed(26)
    for k, name in enumerate(("grad_x", "grad_w", "grad_bias", "grad_x0")):
        v = torch.randn(leaves[k].shape, generator=gen, dtype=torch.float64)
        loss = []
        for eps in (0.5, -0.5):  # linear in each argument: no truncation
            moved = [t.detach().double().cpu() for t in leaves]
            moved[k] = moved[k] + eps * v
            r = reference(*moved, s["seg"])
            loss.append(float((r["out"][0] * go).sum() + (r["last"][0] * gl).sum()))
        ref, bound = want[name]
        allowed = float(((bound + U * ref.abs()) * v.abs()).sum()) + 1e-12 * float((ref * v).abs().sum() + 1)
        got = float((leaves[k].grad.double().cpu() * v).sum())
        assert abs(got - (loss[0] - loss[1])) <= allowed, name
    again = L.lrscan_bwd_conv(s["x"], s["w"], s["go"], x0=s["x0"], segment_pos=s["seg"], grad_last=s["gl"])
    assert torch.equal(again[1], leaves[1].grad) and torch.equal(again[0], leaves[0].grad)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,K", [(1, 1, 2), (5, 300, 4), (33, 64, 8)])
def test_conv_step(B, D, K, dt):
    s = draw(B, 1, D, K, dt, 27, carry=True, packed=0)
    pool = torch.randn((2 * B + 1, K - 1, D), device="cuda").to(s["dtype"])
    slots = torch.randperm(2 * B + 1)[:B].to(torch.int32).cuda()
    slots[B // 2] = -1
    before, live = pool.clone(), slots >= 0
    at = slots[live].long()
    out = L.lrscan_step_conv(s["x"][:, 0], s["w"], pool, bias=s["bias"], slots=slots)
    ref = reference(s["x"][live], s["w"], s["bias"], before[at], None)
    close(out[live], ref["out"][0][:, 0], ref["out"][1][:, 0], s["dtype"], "out")
    want = before.clone()
    want[at] = torch.cat([before[at][:, 1:], s["x"][live]], 1)
    assert torch.equal(pool, want) and not out[~live].any()


def test_conv_step_reports_a_slot_out_of_range():
    x, pool = torch.randn((2, 64), device="cuda"), torch.zeros((3, 3, 64), device="cuda")
    L.lrscan_step_conv(x, torch.randn((64, 4), device="cuda"), pool,
                       slots=torch.tensor([3, -7], dtype=torch.int32, device="cuda"))
    assert L.lrscan_sync_check() == L.LRSCAN_EINVAL
    assert not pool.any()


def test_conv_refusals():
    s = draw(2, 10, 16, 4, "f32", 28, carry=True, packed=3)
    x, w = s["x"], s["w"]
    bad = [
        (ValueError, lambda: L.lrscan_fwd_conv(x, w.t())),
        (ValueError, lambda: L.lrscan_fwd_conv(x, w[:15])),
        (ValueError, lambda: L.lrscan_fwd_conv(x, w.double())),
        (ValueError, lambda: L.lrscan_fwd_conv(x.cpu(), w)),
        (ValueError, lambda: L.lrscan_fwd_conv(x, w, x0=s["x0"][:, :2])),
        (ValueError, lambda: L.lrscan_fwd_conv(x, w, s["bias"][:3])),
        (ValueError, lambda: L.lrscan_fwd_conv(x, w, segment_pos=s["seg"].long())),
        (L.LrscanError, lambda: L.lrscan_fwd_conv(x, w[:, :1].contiguous())),
        (L.LrscanError, lambda: L.lrscan_fwd_conv(x, torch.zeros((16, 9), device="cuda"))),
        (ValueError, lambda: L.lrscan_bwd_conv(x, w, s["go"][:, :3])),
        (ValueError, lambda: L.lrscan_step_conv(x[:, 0], w, s["x0"][:, :2])),
        (L.LrscanError, lambda: L.lrscan_step_conv(x[:, 0], w, s["x0"][:1].contiguous())),
        (L.LrscanError, lambda: L.lrscan_bwd_conv(x, w, s["go"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
    ]
    for what, call in bad:
        with pytest.raises(what):
            call()
    assert L.lrscan_sync_check() == 0
