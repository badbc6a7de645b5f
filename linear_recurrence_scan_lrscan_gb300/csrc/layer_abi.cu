// Host side of the operators around the scan declared in include/lrscan.h:
// argument checks, plans, workspace layout and launches of the gated
// recurrence.
#include <cmath>
#include <cstdarg>

#include "gates_args.h"
#include "launch.h"
#include "lrscan.h"

namespace lrscan {
namespace {

size_t pad256(size_t x) { return (x + 255) / 256 * 256; }
int elem(int dtype) { return dtype == LRSCAN_F32 ? 4 : 2; }

// Rows of a [B, T, D] argument: the pointer's alignment, and strides that do
// not matter (one row, one token) as those of a contiguous tensor.
int rows_of(const char *name, const lrscan_rows *in, int64_t B, int64_t T, int64_t D, int dtype, bool output,
            RowsArg *out) {
    if (!in || !in->ptr) return report_errorf(LRSCAN_EINVAL, "NULL %s", name);
    if (reinterpret_cast<uintptr_t>(in->ptr) % elem(dtype))
        return report_errorf(LRSCAN_EINVAL, "%s is not aligned to its elements", name);
    int64_t st = in->stride_t, sb = in->stride_b, far = 0, rows = 0;
    if (st < 0 || sb < 0) return report_errorf(LRSCAN_EINVAL, "%s has a negative stride", name);
    if (T == 1) st = D;
    if (B == 1 && __builtin_mul_overflow(T, st, &sb)) return report_errorf(LRSCAN_EINVAL, "%s: strides overflow", name);
    if (__builtin_mul_overflow(T - 1, st, &far) || __builtin_mul_overflow(B - 1, sb, &rows) ||
        __builtin_add_overflow(far, rows, &far) || far > (INT64_MAX / 8) - D)
        return report_errorf(LRSCAN_EINVAL, "%s: strides overflow", name);
    // tokens of an output must not share memory: either dimension may be the outer one
    if (output && !(st >= D && (B == 1 || sb >= (T - 1) * st + D)) && !(sb >= D && st >= (B - 1) * sb + D))
        return report_errorf(LRSCAN_EINVAL, "%s: rows overlap (strides %lld, %lld)", name, static_cast<long long>(sb),
                             static_cast<long long>(st));
    out->p = in->ptr;
    out->sb = sb;
    out->st = st;
    return LRSCAN_OK;
}

// Whether a row tensor can be read by bulk tensor copies.
bool bulk_rows(const RowsArg &r, int64_t B, int64_t T, int64_t D, int dtype) {
    const int64_t e = elem(dtype);
    return reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && r.st * e % 16 == 0 && r.sb * e % 16 == 0 && r.st >= D &&
           r.sb >= T * r.st && r.sb * e < (1ll << 40);
}
// Whether pairs of lanes can be stored to it at once.
bool pair_rows(const RowsArg &r, int dtype) {
    return reinterpret_cast<uintptr_t>(r.p) % (2 * elem(dtype)) == 0 && r.st % 2 == 0 && r.sb % 2 == 0;
}

int check_f32(const char *name, const void *p, bool required) {
    if (!p) return required ? report_errorf(LRSCAN_EINVAL, "NULL %s", name) : LRSCAN_OK;
    if (reinterpret_cast<uintptr_t>(p) % 4) return report_errorf(LRSCAN_EINVAL, "%s is not 4-byte aligned", name);
    return LRSCAN_OK;
}

int launch_failed(const char *what) {
    return report_errorf(LRSCAN_ECUDA, "launch of %s: %s", what, cudaGetErrorString(cudaGetLastError()));
}

// ----------------------------------------------------------------------------
// Gated recurrence
// ----------------------------------------------------------------------------
struct GatesScratch {
    int64_t nl, nc, n1, n2;
    size_t head, a1, a2, a3, part;  // bytes
    size_t sync() const { return head + a1 + a2 + a3; }
    size_t total() const { return sync() + part; }
};
// Ticket and published maps (only where tiles follow one another in time),
// then the backward's partial sums of the lam gradient.
GatesScratch gates_scratch(int64_t B, int64_t T, int64_t D, int dtype, int dir) {
    GatesScratch s{};
    const int64_t rows = gates_tile_rows(dtype, dir);
    s.nl = B * ((D + kGatesLanes - 1) / kGatesLanes);
    s.nc = (T + rows - 1) / rows;
    s.n1 = (s.nc + kGatesRadix - 1) / kGatesRadix;
    s.n2 = (s.n1 + kGatesRadix - 1) / kGatesRadix;
    if (s.nc > 1) {
        const size_t tile = static_cast<size_t>(s.nl) * kGatesLanes * 8;
        s.head = 256;
        s.a1 = pad256(tile * s.nc);
        s.a2 = pad256(tile * s.n1);
        s.a3 = pad256(tile * s.n2);
    }
    if (dir == 1) s.part = pad256(static_cast<size_t>(B * s.nc + gates_finish_splits(B * s.nc)) * D * 4);
    return s;
}

int gates_common(GatesLaunch *L, const lrscan_rows *r, const lrscan_rows *i, const lrscan_rows *x, const float *lam,
                 float c, const lrscan_state *state, int64_t B, int64_t T, int64_t D, int dtype) {
    int rc;
    if ((rc = rows_of("r", r, B, T, D, dtype, false, &L->a.r))) return rc;
    if ((rc = rows_of("i", i, B, T, D, dtype, false, &L->a.i))) return rc;
    if ((rc = rows_of("x", x, B, T, D, dtype, false, &L->a.x))) return rc;
    if ((rc = check_f32("lam", lam, true))) return rc;
    if (!(c > 0.0f) || std::isinf(c)) return report_errorf(LRSCAN_EINVAL, "c = %g is not a positive number", c);
    if (state) {
        const void *ps[4] = {state->h0, state->segment_pos, state->grad_last, state->grad_h0};
        for (const void *p : ps)
            if ((rc = check_f32("a state pointer", p, false))) return rc;
        L->a.seg = state->segment_pos;
    }
    L->a.lam = lam;
    L->a.c = c;
    L->a.B = B;
    L->a.T = T;
    L->a.D = D;
    L->a.ndt = static_cast<int>((D + kGatesLanes - 1) / kGatesLanes);
    L->bulk = D % 2 == 0 && bulk_rows(L->a.r, B, T, D, dtype) && bulk_rows(L->a.i, B, T, D, dtype) &&
              bulk_rows(L->a.x, B, T, D, dtype);
    return LRSCAN_OK;
}

// Everything after the checks: device, workspace, tensor maps, launch.
int gates_run(GatesLaunch *L, int dtype, int dir, float *grad_lam, void *stream, const lrscan_opts *opts) {
    const int64_t B = L->a.B, T = L->a.T, D = L->a.D;
    const GatesScratch sc = gates_scratch(B, T, D, dtype, dir);
    if (sc.nl > 0x7fffffffLL || sc.nl * sc.nc > 0x7fffffffLL)
        return report_errorf(LRSCAN_EINVAL, "too many tiles: B %lld, T %lld, D %lld", static_cast<long long>(B),
                             static_cast<long long>(T), static_cast<long long>(D));
    CallCtx ctx;
    int rc = call_device(&ctx);
    if (rc) return rc;
    const cudaStream_t st = call_stream(stream);
    void *ws = nullptr;
    if (sc.total() > 0 && (rc = call_workspace(ctx, st, sc.total(), opts, &ws))) return rc;
    char *base = static_cast<char *>(ws);
    GatesArgs &a = L->a;
    a.nl = static_cast<int>(sc.nl);
    a.nc = static_cast<int>(sc.nc);
    if (sc.nc > 1) {
        a.ticket = reinterpret_cast<unsigned int *>(base);
        a.agg1 = reinterpret_cast<uint64_t *>(base + sc.head);
        a.agg2 = reinterpret_cast<uint64_t *>(base + sc.head + sc.a1);
        a.agg3 = reinterpret_cast<uint64_t *>(base + sc.head + sc.a1 + sc.a2);
    }
    if (dir == 1) a.part = reinterpret_cast<float *>(base + sc.sync());
    a.status = ctx.status;
    a.timeout_ns = ctx.timeout_ns;
    L->stream = st;
    if (L->bulk) {
        const RowsArg *in[4] = {&a.r, &a.i, &a.x, &a.go};
        for (int k = 0; k < (dir ? 4 : 3); ++k)
            if ((rc = encode_rows_map(&L->maps[k], in[k]->p, in[k]->sb, in[k]->st, dtype, B, T, D, kGatesLanes,
                                      gates_tile_rows(dtype, dir))))
                return rc;
    }
    if (sc.nc > 1 && cudaMemsetAsync(ws, 0xff, sc.sync(), st) != cudaSuccess) {
        cudaGetLastError();
        return report_errorf(LRSCAN_ECUDA, "clearing the workspace failed");
    }
    if (gates_launch(*L, dtype, dir, ctx.sm_count)) return launch_failed("the gated recurrence");
    if (dir == 1 && gates_finish_launch(a.part, B * sc.nc, D, a.lam, grad_lam, st))
        return launch_failed("the reduction of grad_lam");
    return LRSCAN_OK;
}

}  // namespace
}  // namespace lrscan

using namespace lrscan;

extern "C" {

size_t lrscan_gates_workspace_bytes(int64_t B, int64_t T, int64_t D, int dtype, int dir) {
    if (call_shape(B, T, D, dtype) || B == 0 || T == 0 || D == 0 || dir < 0 || dir > 1) return 0;
    return gates_scratch(B, T, D, dtype, dir).total();
}

int lrscan_fwd_gates(const lrscan_rows *r, const lrscan_rows *i, const lrscan_rows *x, const float *lam, float c,
                     const lrscan_rows *out, float *last, float *saved, const lrscan_state *state, int64_t B,
                     int64_t T, int64_t D, int dtype, void *stream, const lrscan_opts *opts) {
    begin_call();
    int rc = call_shape(B, T, D, dtype);
    if (rc) return rc;
    if (B == 0 || D == 0) return LRSCAN_OK;
    if ((rc = check_f32("last", last, false)) || (rc = check_f32("saved", saved, false))) return rc;
    if (T == 0) return call_copy_or_zero(last, state ? state->h0 : nullptr, B, D, call_stream(stream));
    GatesLaunch L{};
    if ((rc = gates_common(&L, r, i, x, lam, c, state, B, T, D, dtype))) return rc;
    if ((rc = rows_of("out", out, B, T, D, dtype, true, &L.a.o0))) return rc;
    L.a.h0 = state ? state->h0 : nullptr;
    L.a.edge = last;
    L.a.saved = saved;
    L.bulk = L.bulk && pair_rows(L.a.o0, dtype);
    return gates_run(&L, dtype, 0, nullptr, stream, opts);
}

int lrscan_bwd_gates(const lrscan_rows *r, const lrscan_rows *i, const lrscan_rows *x, const float *lam, float c,
                     const float *saved, const lrscan_rows *grad_out, const lrscan_rows *grad_r,
                     const lrscan_rows *grad_i, const lrscan_rows *grad_x, float *grad_lam, const lrscan_state *state,
                     int64_t B, int64_t T, int64_t D, int dtype, void *stream, const lrscan_opts *opts) {
    begin_call();
    int rc = call_shape(B, T, D, dtype);
    if (rc) return rc;
    if (D == 0) return LRSCAN_OK;
    if ((rc = check_f32("grad_lam", grad_lam, true))) return rc;
    const cudaStream_t st = call_stream(stream);
    if (B == 0 || T == 0) {
        if ((rc = call_copy_or_zero(grad_lam, nullptr, 1, D, st))) return rc;
        return call_copy_or_zero(state ? state->grad_h0 : nullptr, state ? state->grad_last : nullptr, B, D, st);
    }
    GatesLaunch L{};
    if ((rc = gates_common(&L, r, i, x, lam, c, state, B, T, D, dtype))) return rc;
    if ((rc = check_f32("saved", saved, true))) return rc;
    if ((rc = rows_of("grad_out", grad_out, B, T, D, dtype, false, &L.a.go))) return rc;
    if ((rc = rows_of("grad_r", grad_r, B, T, D, dtype, true, &L.a.o0))) return rc;
    if ((rc = rows_of("grad_i", grad_i, B, T, D, dtype, true, &L.a.o1))) return rc;
    if ((rc = rows_of("grad_x", grad_x, B, T, D, dtype, true, &L.a.o2))) return rc;
    L.a.grad_last = state ? state->grad_last : nullptr;
    L.a.edge = state ? state->grad_h0 : nullptr;
    L.a.saved = const_cast<float *>(saved);
    L.bulk = L.bulk && bulk_rows(L.a.go, B, T, D, dtype) && pair_rows(L.a.o0, dtype) && pair_rows(L.a.o1, dtype) &&
             pair_rows(L.a.o2, dtype);
    return gates_run(&L, dtype, 1, grad_lam, stream, opts);
}

int lrscan_step_gates(const lrscan_rows *r, const lrscan_rows *i, const lrscan_rows *x, const float *lam, float c,
                      float *state, const int32_t *slots, const lrscan_rows *out, int64_t B, int64_t S, int64_t D,
                      int dtype, void *stream) {
    begin_call();
    int rc = call_shape(B, 1, D, dtype);
    if (rc || (rc = call_shape(S, 1, D, LRSCAN_F32))) return rc;
    if (B == 0 || D == 0) return LRSCAN_OK;
    RowsArg in[3], o;
    if ((rc = rows_of("r", r, B, 1, D, dtype, false, &in[0]))) return rc;
    if ((rc = rows_of("i", i, B, 1, D, dtype, false, &in[1]))) return rc;
    if ((rc = rows_of("x", x, B, 1, D, dtype, false, &in[2]))) return rc;
    if ((rc = rows_of("out", out, B, 1, D, dtype, true, &o))) return rc;
    if ((rc = check_f32("lam", lam, true)) || (rc = check_f32("state", state, true)) ||
        (rc = check_f32("slots", slots, false)))
        return rc;
    if (!(c > 0.0f) || std::isinf(c)) return report_errorf(LRSCAN_EINVAL, "c = %g is not a positive number", c);
    if (!slots && S < B)
        return report_errorf(LRSCAN_EINVAL, "a state of %lld rows for %lld requests without slots",
                             static_cast<long long>(S), static_cast<long long>(B));
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    GatesStep g{};
    g.r = in[0].p; g.i = in[1].p; g.x = in[2].p;
    g.sr = in[0].sb; g.si = in[1].sb; g.sx = in[2].sb; g.so = o.sb;
    g.out = o.p;
    g.lam = lam; g.c = c;
    g.state = state; g.slots = slots;
    g.S = S; g.B = B; g.D = D;
    g.status = ctx.status;
    g.stream = call_stream(stream);
    return gates_step_launch(g, dtype) ? launch_failed("the single-token gated recurrence") : LRSCAN_OK;
}

}  // extern "C"
