"""GPU tests of the token embedding and its gradient: types of table, tokens and
ids, widths that take wide and narrow accesses, frequent and rare ids, tables of
one to several digits of the sort, tokens that are none, ids out of range, and
refusals.

Bounds (u = 2^-24): the lookup is one fp32 product and one rounding to the
result's type; a row of the gradient is a sum of its c tokens in some fixed
order times the scale, so within (c + 1) u of the sum of their magnitudes."""
import pytest
import torch

from gates_reference import U
from linear_recurrence_scan_lrscan_gb300 import lrscan as L

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PAIRS = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L.lib()
    yield
    assert L.lrscan_sync_check() == 0


def tokens(N, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((N,), V - 1)
    elif kind == "few":  # a handful of frequent ids among rare ones
        ids = torch.where(torch.rand(N, generator=g) < 0.7, torch.randint(0, min(V, 3), (N,), generator=g),
                          torch.randint(0, V, (N,), generator=g))
    else:
        ids = torch.randint(0, V, (N,), generator=g)
    if kind == "padded":
        ids[torch.rand(N, generator=g) < 0.4] = -1
    return ids.cuda()


def check_grad(ids, go, V, scale, wdt, base=None):
    got = L.lrscan_bwd_embed(ids, go, V, scale=scale, dtype=DT[wdt], grad_weight=None if base is None else base.clone(),
                             accumulate=base is not None)
    flat, rows = ids.reshape(-1).cpu(), go.reshape(-1, go.shape[-1]).double().cpu()
    live = flat >= 0
    zero = lambda: torch.zeros((V, rows.shape[1]), dtype=torch.float64)  # noqa: E731
    ref = zero().index_add_(0, flat[live], rows[live]) * scale
    mag = zero().index_add_(0, flat[live], rows[live].abs()) * abs(scale)
    count = torch.zeros(V, dtype=torch.float64).index_add_(0, flat[live], torch.ones(int(live.sum()), dtype=torch.float64))
    bound = (count[:, None] + 1) * U * mag
    if base is not None:
        ref = ref + base.double().cpu()
        bound = bound + U * ref.abs()
    half = 2.0 ** -8 if wdt == "bf16" else U
    off = (got.double().cpu() - ref).abs() - bound - half * (ref.abs() + bound) - 1e-37
    assert off.max() <= 0, f"{int((off > 0).sum())} values over the bound, by {off.max():.3g}"
    untouched = (count == 0).cuda()
    assert torch.equal(got[untouched], torch.zeros_like(got[untouched]) if base is None else base[untouched])
    return got


@pytest.mark.parametrize("wdt,odt", PAIRS)
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (5, 7, 8), (1000, 33, 264), (333, 1000, 77), (3, 5, 4104)])
def test_embed_lookup(N, V, D, wdt, odt):
    weight = torch.randn((V, D), device="cuda").to(DT[wdt])
    ids = tokens(N, V, "padded", N)
    scale = 1.7
    out = L.lrscan_fwd_embed(ids, weight, scale=scale, dtype=DT[odt])
    want = (weight.float()[ids.clamp(min=0)] * torch.tensor(scale, dtype=torch.float32)).to(DT[odt])
    want[ids < 0] = 0
    assert torch.equal(out, want)
    assert torch.equal(L.lrscan_fwd_embed(ids.to(torch.int32), weight, scale=scale, dtype=DT[odt]), want)


@pytest.mark.parametrize("gdt,wdt", PAIRS)
@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (40, 7, 8), (1000, 33, 264), (333, 5000, 77), (31, 5, 4104)])
def test_embed_grad(N, V, D, gdt, wdt):
    go = torch.randn((N, D), device="cuda").to(DT[gdt])
    for kind in ("uniform", "padded"):
        ids = tokens(N, V, kind, N)
        got = check_grad(ids, go, V, 0.7, wdt)
        assert torch.equal(got, L.lrscan_bwd_embed(ids.to(torch.int32), go, V, scale=0.7, dtype=DT[wdt]))


@pytest.mark.parametrize("N,V,D", [(20000, 300, 40), (20000, 70000, 8), (9000, 600000, 8), (5000, 2 ** 20 + 1, 3)])
@pytest.mark.parametrize("kind", ["uniform", "few", "one"])
def test_embed_grad_frequent_ids_and_wide_tables(N, V, D, kind):
    # tables of one, two and three digits; ids that take hundreds of stretches
    ids = tokens(N, V, kind, V)
    go = torch.randn((N, D), device="cuda")
    first = check_grad(ids, go, V, 1.0, "f32")
    for _ in range(2):
        assert torch.equal(first, L.lrscan_bwd_embed(ids, go, V))


def test_embed_grad_edges_of_stretches():
    # runs of every length from 1 to 70, so that runs begin and end at each place of a stretch
    ids = torch.repeat_interleave(torch.arange(70), torch.arange(1, 71)).cuda()
    ids = ids[torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(1)).cuda()]
    check_grad(ids, torch.randn((ids.numel(), 16), device="cuda"), 80, 1.0, "f32")


def test_embed_grad_accumulates():
    ids, go = tokens(500, 90, "padded", 2), torch.randn((500, 48), device="cuda")
    for dt in ("f32", "bf16"):
        check_grad(ids, go, 90, 0.5, dt, base=torch.randn((90, 48), device="cuda").to(DT[dt]))


def test_embed_all_tokens_none_and_no_tokens():
    go = torch.randn((6, 16), device="cuda")
    none = torch.full((6,), -1, device="cuda")
    assert not L.lrscan_bwd_embed(none, go, 9).any()
    assert not L.lrscan_fwd_embed(none, torch.randn((9, 16), device="cuda")).any()
    empty = torch.empty(0, dtype=torch.int64, device="cuda")
    assert not L.lrscan_bwd_embed(empty, go[:0], 9).any()
    base = torch.randn((9, 16), device="cuda")
    assert torch.equal(L.lrscan_bwd_embed(empty, go[:0], 9, grad_weight=base.clone(), accumulate=True), base)
    assert L.lrscan_fwd_embed(empty, base).shape == (0, 16)


def test_embed_reports_ids_out_of_range():
    w, go = torch.randn((9, 16), device="cuda"), torch.randn((4, 16), device="cuda")
    ids = torch.tensor([3, 9, 2 ** 40, 8], device="cuda")
    out = L.lrscan_fwd_embed(ids, w)
    assert L.lrscan_sync_check() == L.LRSCAN_EINVAL and L.lrscan_sync_check() == 0
    assert torch.equal(out[[0, 3]], w[[3, 8]]) and not out[1:3].any()
    g = L.lrscan_bwd_embed(ids, go, 9)
    assert L.lrscan_sync_check() == L.LRSCAN_EINVAL
    assert torch.equal(g[3], go[0]) and torch.equal(g[8], go[3]) and not g[:3].any()


def test_embed_autograd_and_differences():
    ids = tokens(60, 20, "padded", 3).view(4, 15)
    w = torch.randn((20, 24), device="cuda").requires_grad_()
    go = torch.randn((4, 15, 24), device="cuda")
    out = L.embed(ids, w, scale=3.0)
    assert out.shape == (4, 15, 24)
    (out * go).sum().backward()
    check_grad(ids, go, 20, 3.0, "f32")
    v = torch.randn(w.shape, dtype=torch.float64)
    rows = torch.where((ids >= 0)[..., None].cpu(), v[ids.clamp(min=0).cpu()], 0.0)
    slope = 3.0 * float((rows * go.double().cpu()).sum())  # linear in the table
    mag = 3.0 * float((rows * go.double().cpu()).abs().sum())
    assert abs(float((w.grad.double().cpu() * v).sum()) - slope) <= (60 + 2) * U * mag


def test_embed_unaligned_and_workspace():
    buf = torch.randn(9 * 16 + 1, device="cuda")
    w = buf[1:].view(9, 16)
    ids = tokens(50, 9, "uniform", 4)
    assert torch.equal(L.lrscan_fwd_embed(ids, w), w[ids])
    go = torch.randn(50 * 16 + 1, device="cuda")[1:].view(50, 16)
    ws = torch.empty(L.lrscan_embed_workspace_bytes(50, 9, 16), dtype=torch.uint8, device="cuda")
    assert torch.equal(L.lrscan_bwd_embed(ids, go, 9, workspace=ws), L.lrscan_bwd_embed(ids, go.clone(), 9))


def test_embed_refusals():
    w, ids, go = torch.randn((9, 16), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.randn((4, 16), device="cuda")
    bad = [
        (ValueError, lambda: L.lrscan_fwd_embed(ids.float(), w)),
        (ValueError, lambda: L.lrscan_fwd_embed(ids.cpu(), w)),
        (ValueError, lambda: L.lrscan_fwd_embed(ids, w.t())),
        (ValueError, lambda: L.lrscan_fwd_embed(ids, w.half())),
        (ValueError, lambda: L.lrscan_fwd_embed(ids, w, dtype=torch.float16)),
        (ValueError, lambda: L.lrscan_fwd_embed(ids, w[0])),
        (ValueError, lambda: L.lrscan_fwd_embed(ids[::2], w)),
        (L.LrscanError, lambda: L.lrscan_fwd_embed(ids, w[:0])),
        (ValueError, lambda: L.lrscan_bwd_embed(ids, go[:3], 9)),
        (ValueError, lambda: L.lrscan_bwd_embed(ids, go, 9, accumulate=True)),
        (ValueError, lambda: L.lrscan_bwd_embed(ids, go, 9, grad_weight=torch.zeros((8, 16), device="cuda"))),
        (L.LrscanError, lambda: L.lrscan_bwd_embed(ids, go, 9, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))),
    ]
    for what, call in bad:
        with pytest.raises(what):
            call()
    assert L.lrscan_sync_check() == 0
