"""GPU tests of the gated recurrence against its definition in 64 bits: both
directions, both storage types, sizes around a tile's edges, carried state and
segment restarts, strided and unaligned rows, extreme gates, long sequences on
the tree of maps, single tokens, and the calls it refuses."""
import numpy as np
import pytest
import torch

import gates_reference as R
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


def draw(B, T, D, dt, seed, *, lam_lo=0.9, lam_hi=0.999, carry=False, packed=0, wide=False):
    """Inputs on the GPU; wide: r and i are slices of one projection."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dtype = DT[dt]
    u = torch.empty(D).uniform_(lam_lo, lam_hi, generator=g)
    lam = torch.log(torch.expm1(-torch.log(u) / 8))
    both = n(B, T, 2 * D).to(dtype).cuda()
    r, i = (both[..., :D], both[..., D:]) if wide else (both[..., :D].contiguous(), both[..., D:].contiguous())
    seg = None
    if packed:
        start = torch.rand((B, T), generator=g) < 1.0 / packed
        t = torch.arange(T).expand(B, T)
        seg = (t - torch.cummax(torch.where(start, t, -5), dim=1).values).to(torch.int32).cuda()
    return {"r": r, "i": i, "x": n(B, T, D).to(dtype).cuda(), "lam": lam.cuda(),
            "h0": n(B, D).cuda() if carry else None, "seg": seg, "go": n(B, T, D).to(dtype).cuda(),
            "gl": n(B, D).cuda() if carry else None, "dtype": dtype}


def run_fwd(s, **kw):
    return L.lrscan_fwd_gates(s["r"], s["i"], s["x"], s["lam"], h0=s["h0"], segment_pos=s["seg"], want_saved=True, **kw)


def run_bwd(s, saved, **kw):
    return L.lrscan_bwd_gates(s["r"], s["i"], s["x"], s["lam"], saved, s["go"], segment_pos=s["seg"],
                              grad_last=s["gl"], **kw)


def check(s):
    out, last, saved = run_fwd(s)
    ref, rlast, e, elast = R.forward(s["r"], s["i"], s["x"], s["lam"], 8.0, s["h0"], s["seg"])
    R.assert_within(out, ref, e, s["dtype"], "out")
    R.assert_within(last, rlast, elast, torch.float32, "last")
    B, T, D = ref.shape
    h0 = torch.zeros((B, D), dtype=torch.float64) if s["h0"] is None else s["h0"].double().cpu()
    before = torch.cat([h0[:, None], ref], 1)[:, :T:16]
    ebefore = torch.cat([torch.zeros_like(h0)[:, None], e], 1)[:, :T:16]
    R.assert_within(saved, before, ebefore, torch.float32, "saved")
    grads = dict(zip(("grad_r", "grad_i", "grad_x", "grad_lam", "grad_h0"), run_bwd(s, saved)))
    want = R.backward(s["r"], s["i"], s["x"], s["lam"], s["go"], 8.0, s["h0"], s["seg"], s["gl"])
    for name, (w, b) in want.items():
        R.assert_within(grads[name], w, b, s["dtype"] if name in ("grad_r", "grad_i", "grad_x") else torch.float32, name)
    assert L.lrscan_sync_check() == 0


SHAPES = [(1, 1, 64), (2, 1, 1), (1, 63, 64), (3, 64, 128), (2, 65, 40), (1, 129, 1001), (2, 200, 72), (2, 700, 190)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gates_plain(shape, dt):
    check(draw(*shape, dt, 1))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_gates_with_state_restarts_and_slices(shape, dt):
    check(draw(*shape, dt, 2, carry=True, packed=23, wide=True))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 33])
def test_gates_on_every_level_of_the_tree(dt, D):
    # 64-token tiles: over 16 * 16 of them, so tile, group and state words are all read
    check(draw(1, 64 * 300 + 17, D, dt, 3, carry=True))


def test_gates_tree_with_restarts():
    check(draw(1, 64 * 270, 64, "f32", 4, carry=True, packed=3000))


@pytest.mark.parametrize("D", [64, 65])
def test_gates_fast_decays(D):
    # rates far over 1/4: the exponential instead of its series
    check(draw(2, 150, D, "f32", 5, lam_lo=1e-6, lam_hi=0.9))


def test_gates_repeat_bit_for_bit():
    s = draw(2, 64 * 40 + 3, 320, "bf16", 6, carry=True, packed=500)
    one = [*run_fwd(s), *run_bwd(s, run_fwd(s)[2])]
    for _ in range(3):
        two = [*run_fwd(s), *run_bwd(s, run_fwd(s)[2])]
        assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("D", [64, 65])
def test_gates_extreme_gates(D):
    s = draw(1, 90, D, "f32", 7, carry=True)
    s["r"][:, 10:20] = -float("inf")   # the state stays as it is
    s["r"][:, 30:35] = 200.0
    s["i"][:, 40:45] = -float("inf")
    s["i"][:, 50:55] = float("inf")
    s["r"][:, 60:62] = -100.0          # decays that differ from one by less than a rounding
    check(s)
    out, _, saved = run_fwd(s)
    assert torch.equal(out[:, 10:16], out[:, 9:10].expand(-1, 6, -1))  # tokens of one thread
    assert all(torch.isfinite(g).all() for g in run_bwd(s, saved))


@pytest.mark.parametrize("D", [64, 65])
def test_gates_restart_stops_infinities_and_nan(D):
    s = draw(1, 200, D, "f32", 8, carry=True)
    s["seg"] = torch.ones((1, 200), dtype=torch.int32, device="cuda")
    s["seg"][:, [0, 50, 130]] = 0
    s["h0"][:] = float("nan")          # token 0 starts a segment: the carried state is not used
    s["x"][:, 40] = float("inf")
    s["x"][:, 100] = float("nan")
    out, last, saved = run_fwd(s)
    assert torch.isfinite(out[:, :40]).all() and torch.isinf(out[:, 40:50]).all()
    assert torch.isfinite(out[:, 50:100]).all() and torch.isnan(out[:, 100:130]).all()
    assert torch.isfinite(out[:, 130:]).all() and torch.isfinite(last).all()
    gr, gi, gx, _, gh0 = run_bwd(s, saved)
    assert torch.isfinite(gx).all()    # the adjoint holds no value of x
    assert torch.isfinite(gr[:, :40]).all() and torch.isfinite(gr[:, 50:100]).all() and torch.isfinite(gr[:, 130:]).all()
    assert not gh0.any()


def test_gates_nan_passes_without_a_restart():
    s = draw(1, 300, 64, "f32", 9)
    s["r"][0, 100, 5] = float("nan")
    out, last, _ = run_fwd(s)
    assert torch.isnan(out[0, 100:, 5]).all() and torch.isnan(last[0, 5])
    assert torch.isfinite(out[0, :, :5]).all() and torch.isfinite(out[0, :100, 5]).all()


def test_gates_split_in_two_calls_continues():
    s = draw(2, 300, 64, "f32", 10, carry=True)
    out, last, _ = run_fwd(s)
    cut = 111
    head = {**s, **{k: s[k][:, :cut] for k in ("r", "i", "x")}}
    o1, l1, _ = run_fwd(head)
    tail = {**s, **{k: s[k][:, cut:] for k in ("r", "i", "x")}, "h0": l1}
    o2, l2, _ = run_fwd(tail)
    ref, rlast, e, elast = R.forward(s["r"], s["i"], s["x"], s["lam"], 8.0, s["h0"])
    R.assert_within(torch.cat([o1, o2], 1), ref, e, torch.float32, "out in two calls")
    R.assert_within(l2, rlast, elast, torch.float32, "last of two calls")


def test_gates_empty():
    x = torch.empty((2, 0, 16), device="cuda")
    h0 = torch.randn((2, 16), device="cuda")
    lam = torch.zeros(16, device="cuda")
    out, last, saved = L.lrscan_fwd_gates(x, x, x, lam, h0=h0, want_saved=True)
    assert torch.equal(last, h0) and saved.shape == (2, 0, 16)
    g = L.lrscan_bwd_gates(x, x, x, lam, saved, x, grad_last=h0)
    assert not g[3].any() and torch.equal(g[4], h0)
    x = torch.empty((0, 5, 16), device="cuda")
    out, last, saved = L.lrscan_fwd_gates(x, x, x, lam, want_saved=True)
    assert not L.lrscan_bwd_gates(x, x, x, lam, saved, x)[3].any()


def test_gates_strided_gradients_and_layouts():
    """Gradients written into one projection's gradient; time-major tensors; an offset base."""
    B, T, D = 2, 130, 64
    s = draw(B, T, D, "bf16", 11, wide=True)
    ref = run_bwd(s, run_fwd(s)[2])
    both = torch.zeros((B, T, 2 * D), device="cuda", dtype=torch.bfloat16)
    run_bwd(s, run_fwd(s)[2], grad_r=both[..., :D], grad_i=both[..., D:])
    assert torch.equal(both[..., :D], ref[0]) and torch.equal(both[..., D:], ref[1])
    tm = {**s, **{k: s[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("r", "i", "x", "go")}}
    check(tm)  # plain loads instead of bulk copies: the same within the bounds, not bit for bit
    time_major = torch.empty((T, B, D), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    assert torch.equal(run_fwd(tm, out=time_major)[0], run_fwd(tm)[0])
    buf = torch.empty(B * T * D + 3, device="cuda", dtype=torch.bfloat16)
    shifted = buf[3:].view(B, T, D).copy_(s["x"])
    check({**s, "x": shifted})
    # one gate for all requests: a broadcast input
    rb = s["r"][:1].expand(B, T, D)
    check({**s, "r": rb})


def test_gates_autograd_and_differences():
    """Autograd against central differences of the 64-bit definition along random directions."""
    s = draw(2, 90, 40, "f32", 12, carry=True, packed=31)
    leaves = [s[k].clone().requires_grad_() for k in ("r", "i", "x", "lam", "h0")]
    out, last = L.gate_scan(*leaves[:4], h0=leaves[4], segment_pos=s["seg"])
    ((out * s["go"]).sum() + (last * s["gl"]).sum()).backward()
    want = R.backward(s["r"], s["i"], s["x"], s["lam"], s["go"], 8.0, s["h0"], s["seg"], s["gl"])
    go, gl = s["go"].double().cpu(), s["gl"].double().cpu()
    gen = torch.Generator().manual_seed(13)
    for k, leaf in enumerate(leaves):
        v = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)
        loss = []
        for eps in (1e-5, -1e-5):
            moved = [t.detach().double().cpu() for t in leaves]
            moved[k] = moved[k] + eps * v
            o, l, _, _ = R.forward(*moved[:4], 8.0, moved[4], s["seg"])
            loss.append(float((o * go).sum() + (l * gl).sum()))
        slope = (loss[0] - loss[1]) / 2e-5
        name = ("grad_r", "grad_i", "grad_x", "grad_lam", "grad_h0")[k]
        # the bound of the gradient along v; 1e-7 of the terms for the differences themselves
        allowed = float((want[name][1] * v.abs()).sum()) + 1e-7 * float((want[name][0] * v).abs().sum()) + R.U * float(
            (want[name][0] * v).abs().sum())
        got = float((leaf.grad.double().cpu() * v).sum())
        assert abs(got - slope) <= allowed, (name, got, slope, allowed)


def test_gates_on_another_stream_and_in_a_graph():
    s = draw(2, 64 * 20, 128, "bf16", 14)
    ref = run_fwd(s)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        run_bwd(s, run_fwd(s)[2])
        out, last, saved = run_fwd(s)
        grads = run_bwd(s, saved)
    st.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(last, ref[1])
    outs = [torch.zeros_like(t) for t in (out, last, saved)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        run_fwd(s, out=outs[0], last=outs[1], saved=outs[2])
    for _ in range(2):
        outs[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], out) and torch.equal(outs[1], last)
    ws = torch.empty(L.lrscan_gates_workspace_bytes(2, 64 * 20, 128, "bf16", "bwd"), dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(grads, run_bwd(s, saved, workspace=ws)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (5, 300), (33, 64)])
def test_gates_step(B, D, dt):
    s = draw(B, 1, D, dt, 15)
    S = 2 * B + 1
    pool = torch.randn((S, D), device="cuda")
    slots = torch.randperm(S)[:B].to(torch.int32).cuda()
    slots[B // 2] = -1
    before = pool.clone()
    live = slots >= 0
    at = slots[live].long()
    out = L.lrscan_step_gates(s["r"][:, 0], s["i"][:, 0], s["x"][:, 0], s["lam"], pool, slots=slots)
    ref, rlast, e, elast = R.forward(s["r"][live], s["i"][live], s["x"][live], s["lam"], 8.0, before[at])
    R.assert_within(out[live], ref[:, 0], e[:, 0], s["dtype"], "out")
    R.assert_within(pool[at], rlast, elast, torch.float32, "state")
    assert not out[~live].any()
    rest = torch.ones(S, dtype=torch.bool)
    rest[at.cpu()] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])


def test_gates_step_matches_the_sequence():
    s = draw(3, 20, 72, "bf16", 16, carry=True)
    out, last, _ = run_fwd(s)
    state = s["h0"].clone()
    ref, _, e, _ = R.forward(s["r"], s["i"], s["x"], s["lam"], 8.0, s["h0"])
    for t in range(20):
        y = L.lrscan_step_gates(s["r"][:, t], s["i"][:, t], s["x"][:, t], s["lam"], state)
        R.assert_within(y, ref[:, t], e[:, t], torch.bfloat16, f"token {t}")


def test_gates_step_reports_a_slot_out_of_range():
    x = torch.randn((3, 64), device="cuda")
    pool = torch.randn((4, 64), device="cuda")
    before = pool.clone()
    slots = torch.tensor([1, 4, 0], dtype=torch.int32, device="cuda")
    out = L.lrscan_step_gates(x, x, x, torch.zeros(64, device="cuda"), pool, slots=slots)
    assert L.lrscan_sync_check() == L.LRSCAN_EINVAL
    assert L.lrscan_sync_check() == 0
    assert not out[1].any() and torch.equal(pool[2:], before[2:]) and not torch.equal(pool[0], before[0])


def test_gates_refusals():
    s = draw(2, 10, 16, "f32", 17)
    r, i, x, lam = s["r"], s["i"], s["x"], s["lam"]
    _, _, saved = run_fwd(s)
    bad = [
        (TypeError, lambda: L.lrscan_fwd_gates(r, i, np.zeros((2, 10, 16)), lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r, i, x[0], lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r.cpu(), i, x, lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r.bfloat16(), i, x, lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r.half(), i.half(), x.half(), lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r[:, :5], i, x, lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r.transpose(1, 2).contiguous().transpose(1, 2), i, x, lam)),
        (ValueError, lambda: L.lrscan_fwd_gates(r, i, x, lam.double())),
        (ValueError, lambda: L.lrscan_fwd_gates(r, i, x, lam, h0=torch.zeros((2, 15), device="cuda"))),
        (ValueError, lambda: L.lrscan_fwd_gates(r, i, x, lam, segment_pos=torch.zeros((2, 10), device="cuda"))),
        (L.LrscanError, lambda: L.lrscan_fwd_gates(r, i, x, lam, c=0.0)),
        (L.LrscanError, lambda: L.lrscan_fwd_gates(r, i, x, lam, c=float("nan"))),
        (L.LrscanError, lambda: L.lrscan_fwd_gates(r, i, x, lam, out=x[:1].expand(2, 10, 16))),
        (ValueError, lambda: L.lrscan_bwd_gates(r, i, x, lam, saved[:, :0], s["go"])),
        (ValueError, lambda: L.lrscan_step_gates(x[:, 0], x[:, 0], x[:, 0], lam, saved)),
        (L.LrscanError, lambda: L.lrscan_step_gates(x[:, 0], x[:, 0], x[:, 0], lam, torch.zeros((1, 16), device="cuda"))),
        (L.LrscanError, lambda: L.lrscan_fwd_gates(*(torch.zeros((1, 200, 64), device="cuda"),) * 3,
                                                   torch.zeros(64, device="cuda"),
                                                   workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
    ]
    for what, call in bad:
        with pytest.raises(what):
            call()
    assert L.lrscan_sync_check() == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_rows_that_share_memory(dt):
    # one row for all batch rows, one token for all tokens: strides of zero
    s = draw(3, 150, 64, dt, 21, carry=True)
    s["r"] = s["r"][:1].expand(3, -1, -1)
    s["x"] = s["x"][:, :1].expand(-1, 150, -1)
    s["go"] = s["go"][:1, :1].expand(3, 150, -1)
    check(s)


def test_gates_gradient_of_broadcast_inputs():
    # the gradient of what was broadcast is the sum over where it went
    s = draw(3, 90, 64, "f32", 22)
    r, x, i = (s[k].clone().requires_grad_() for k in ("r", "x", "i"))
    one_r, one_x = s["r"][:1].clone().requires_grad_(), s["x"][:, :1].clone().requires_grad_()
    L.gate_scan(one_r.expand(3, -1, -1), i, one_x.expand(-1, 90, -1), s["lam"])[0].sum().backward()
    with torch.no_grad():
        r.copy_(s["r"][:1].expand(3, -1, -1))
        x.copy_(s["x"][:, :1].expand(-1, 90, -1))
    L.gate_scan(r, s["i"], x, s["lam"])[0].sum().backward()
    # the same gradients, summed over 3 rows or 90 tokens in fp32 either way
    for got, parts, dim, n in ((one_r.grad, r.grad, 0, 3), (one_x.grad, x.grad, 1, 90)):
        bound = n * 2.0 ** -23 * parts.abs().sum(dim, keepdim=True)
        assert ((got - parts.sum(dim, keepdim=True)).abs() <= bound + 1e-30).all()


@pytest.mark.parametrize("packed", [0, 20])
@pytest.mark.parametrize("D", [64, 33])
def test_gates_many_lane_tiles(D, packed):
    # a lane tile for every fourth SM and more: bf16 forward takes fewer, wider teams
    check(draw(40, 150, D, "bf16", 23, carry=True, packed=packed))


@pytest.mark.parametrize("D", [64, 65])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gates_restart_stops_a_nan_gate(dt, D):
    s = draw(1, 200, D, dt, 24)
    s["seg"] = torch.ones((1, 200), dtype=torch.int32, device="cuda")
    s["seg"][:, [0, 50, 130]] = 0
    s["r"][:, 100] = float("nan")
    s["r"][:, 130] = float("nan")      # a segment's first token: its decay is not used
    out, last, saved = run_fwd(s)
    assert torch.isfinite(out[:, :100]).all() and torch.isnan(out[:, 100:130]).all()
    assert torch.isfinite(out[:, 130:]).all() and torch.isfinite(last).all()
    for grad in run_bwd(s, saved)[:3]:
        # back from token 100 to its segment's start, and in grad_r on to its end
        assert torch.isfinite(grad[:, :50]).all() and torch.isfinite(grad[:, 130:]).all()
