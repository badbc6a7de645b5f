// Host side of the operators around the scan declared in include/lrscan.h:
// argument checks, workspace layout and launches of the gated recurrence, the
// causal convolution and the token embedding.
#include <cmath>
#include <cstdarg>

#include "conv_args.h"
#include "embed_args.h"
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
    size_t head, a1, a2, a3, rate, part;  // bytes
    size_t sync() const { return head + a1 + a2 + a3; }
    size_t total() const { return sync() + rate + part; }
};
// Ticket, published maps and rates (only where tiles follow one another in
// time), then the backward's partial sums of the lam gradient.
GatesScratch gates_scratch(int64_t B, int64_t T, int64_t D, int dir) {
    GatesScratch s{};
    const int64_t rows = kGatesTileRows;
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
        s.rate = pad256(static_cast<size_t>(D) * 4);
    }
    if (dir == 1) s.part = pad256(static_cast<size_t>(B * s.nc + gates_finish_slices(B * s.nc)) * D * 4);
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
    const GatesScratch sc = gates_scratch(B, T, D, dir);
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
        a.rate = reinterpret_cast<float *>(base + sc.sync());
    }
    if (dir == 1) a.part = reinterpret_cast<float *>(base + sc.sync() + sc.rate);
    a.status = ctx.status;
    a.timeout_ns = ctx.timeout_ns;
    L->stream = st;
    if (L->bulk) {
        const RowsArg *in[4] = {&a.r, &a.i, &a.x, &a.go};
        for (int k = 0; k < (dir ? 4 : 3); ++k)
            if ((rc = encode_rows_map(&L->maps[k], in[k]->p, in[k]->sb, in[k]->st, dtype, B, T, D, kGatesLanes,
                                      kGatesTileRows)))
                return rc;
    }
    if (sc.nc > 1 && gates_begin_launch(ws, sc.sync(), a.lam, a.c, D, const_cast<float *>(a.rate), ctx.sm_count, st))
        return launch_failed("the gated recurrence's first kernel");
    if (gates_launch(*L, dtype, dir, ctx.sm_count)) return launch_failed("the gated recurrence");
    if (dir == 1 && gates_finish_launch(a.part, B * sc.nc, D, a.lam, grad_lam, st))
        return launch_failed("the reduction of grad_lam");
    return LRSCAN_OK;
}

// ----------------------------------------------------------------------------
// Causal convolution
// ----------------------------------------------------------------------------
constexpr int64_t kConvTokens = static_cast<int64_t>(kConvSteps) * kConvSplit;  // a CTA's

int64_t conv_chunks(int64_t T) { return (T + kConvTokens - 1) / kConvTokens; }

int conv_common(ConvArgs *a, const lrscan_rows *x, const float *w, int K, const void *x0, const int32_t *segment_pos,
                int64_t B, int64_t T, int64_t D, int dtype) {
    int rc;
    if ((rc = rows_of("x", x, B, T, D, dtype, false, &a->x)) || (rc = check_f32("w", w, true)) ||
        (rc = check_f32("segment_pos", segment_pos, false)))
        return rc;
    if (conv_chunks(T) * ((D + 31) / 32) > 0x7fffffffLL)
        return report_errorf(LRSCAN_EINVAL, "T and D are too large together");
    a->w = w;
    a->x0 = x0;
    a->seg = segment_pos;
    a->B = B;
    a->T = T;
    a->D = D;
    a->chunks = static_cast<unsigned>(conv_chunks(T));
    return LRSCAN_OK;
}
int check_taps(int K) {
    if (K < kConvMinTaps || K > kConvMaxTaps)
        return report_errorf(LRSCAN_EINVAL, "%d taps: %d to %d are supported", K, kConvMinTaps, kConvMaxTaps);
    return LRSCAN_OK;
}
int check_elem(const char *name, const void *p, int dtype) {
    if (p && reinterpret_cast<uintptr_t>(p) % elem(dtype))
        return report_errorf(LRSCAN_EINVAL, "%s is not aligned to its elements", name);
    return LRSCAN_OK;
}
// Whether four lanes of a row can be accessed at once (rows of a tensor; a dense tensor).
bool quads(const RowsArg &r, int dtype) {
    return reinterpret_cast<uintptr_t>(r.p) % (4 * elem(dtype)) == 0 && r.st % 4 == 0 && r.sb % 4 == 0;
}
bool quads(const void *p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (4 * elem(dtype)) == 0; }

int copy_rows(void *dst, const void *src, size_t bytes, cudaStream_t st) {
    if (!dst || bytes == 0) return LRSCAN_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(dst, 0, bytes, st);
    if (e == cudaSuccess) return LRSCAN_OK;
    cudaGetLastError();
    return report_errorf(LRSCAN_ECUDA, "state copy: %s", cudaGetErrorString(e));
}

// ----------------------------------------------------------------------------
// Token embedding
// ----------------------------------------------------------------------------
struct EmbedScratch {
    size_t list, runs, part;
    int bits, passes, per;
    size_t total() const { return 4 * list + runs + part; }
};
EmbedScratch embed_scratch(int64_t N, int64_t V, int64_t D, int sm_count) {
    EmbedScratch s{};
    int bits = 5;  // of the largest key, V itself (a token that is none)
    while (bits < 32 && (V >> bits) != 0) ++bits;
    s.passes = (bits + kSortBits - 1) / kSortBits;
    s.bits = (bits + s.passes - 1) / s.passes;
    if (s.bits < 5) s.bits = 5;
    // stretches short enough for two CTAs an SM, and long enough that few sums are left in between
    s.per = 32;
    while (s.per > 4 && N / s.per < 2LL * sm_count) s.per /= 2;
    s.list = pad256(static_cast<size_t>(N) * 4);
    s.runs = 256 + pad256(static_cast<size_t>(N / kLongRun + 1) * 4);
    s.part = pad256(static_cast<size_t>((N + s.per - 1) / s.per) * 2 * D * 4);
    return s;
}

int embed_common(EmbedArgs *a, const void *ids, int id_bytes, const void *in, int idtype, void *out, int odtype,
                 float scale, int64_t N, int64_t V, int64_t D) {
    if (id_bytes != 4 && id_bytes != 8) return report_errorf(LRSCAN_EINVAL, "ids of %d bytes", id_bytes);
    if (N > 0 && (!ids || !in)) return report_errorf(LRSCAN_EINVAL, "NULL ids or input");
    if (!out) return report_errorf(LRSCAN_EINVAL, "NULL output");
    if (reinterpret_cast<uintptr_t>(ids) % id_bytes || reinterpret_cast<uintptr_t>(in) % elem(idtype) ||
        reinterpret_cast<uintptr_t>(out) % elem(odtype))
        return report_errorf(LRSCAN_EINVAL, "a pointer is not aligned to its elements");
    a->ids = ids;
    a->wide = id_bytes == 8;
    a->in = in;
    a->out = out;
    a->scale = scale;
    a->N = N;
    a->V = V;
    a->D = D;
    a->vec = D % 8 == 0 && reinterpret_cast<uintptr_t>(in) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    return LRSCAN_OK;
}
int embed_shape(int64_t N, int64_t V, int64_t D, int wdtype, int odtype) {
    int rc;
    if ((rc = call_shape(N, 1, D, odtype)) || (rc = call_shape(V, 1, D, wdtype))) return rc;
    if (N > 0x7fffffffLL || V > 0x7ffffffeLL) return report_errorf(LRSCAN_EINVAL, "N or V above 2^31 - 2");
    return LRSCAN_OK;
}

}  // namespace
}  // namespace lrscan

using namespace lrscan;

extern "C" {

size_t lrscan_gates_workspace_bytes(int64_t B, int64_t T, int64_t D, int dtype, int dir) {
    if (call_shape(B, T, D, dtype) || B == 0 || T == 0 || D == 0 || dir < 0 || dir > 1) return 0;
    return gates_scratch(B, T, D, dir).total();
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

size_t lrscan_conv_workspace_bytes(int64_t B, int64_t T, int64_t D, int K) {
    if (call_shape(B, T, D, LRSCAN_F32) || B == 0 || T == 0 || D == 0 || check_taps(K)) return 0;
    const int64_t rows = B * conv_chunks(T);
    return pad256(static_cast<size_t>(rows + conv_finish_slices(rows)) * (K + 1) * D * 4);
}

int lrscan_fwd_conv(const lrscan_rows *x, const float *w, const float *bias, int K, const void *x0,
                    const int32_t *segment_pos, const lrscan_rows *out, void *last, int64_t B, int64_t T, int64_t D,
                    int dtype, void *stream) {
    begin_call();
    int rc = call_shape(B, T, D, dtype);
    if (rc || (rc = check_taps(K)) || (rc = check_elem("x0", x0, dtype)) || (rc = check_elem("last", last, dtype)))
        return rc;
    if (B == 0 || D == 0) return LRSCAN_OK;
    const cudaStream_t st = call_stream(stream);
    if (T == 0) return copy_rows(last, x0, static_cast<size_t>(B) * (K - 1) * D * elem(dtype), st);
    ConvArgs a{};
    if ((rc = conv_common(&a, x, w, K, x0, segment_pos, B, T, D, dtype)) ||
        (rc = rows_of("out", out, B, T, D, dtype, true, &a.o)) || (rc = check_f32("bias", bias, false)))
        return rc;
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    a.bias = bias;
    a.last = last;
    a.vec = D % 4 == 0 && quads(a.x, dtype) && quads(a.o, dtype) && quads(x0, dtype) && quads(last, dtype);
    a.stream = st;
    return conv_fwd_launch(a, K, dtype) ? launch_failed("the causal convolution") : LRSCAN_OK;
}

int lrscan_bwd_conv(const lrscan_rows *x, const float *w, int K, const void *x0, const int32_t *segment_pos,
                    const lrscan_rows *grad_out, const void *grad_last, const lrscan_rows *grad_x, float *grad_w,
                    float *grad_bias, void *grad_x0, int64_t B, int64_t T, int64_t D, int dtype, void *stream,
                    const lrscan_opts *opts) {
    begin_call();
    int rc = call_shape(B, T, D, dtype);
    if (rc || (rc = check_taps(K)) || (rc = check_elem("x0", x0, dtype)) ||
        (rc = check_elem("grad_last", grad_last, dtype)) || (rc = check_elem("grad_x0", grad_x0, dtype)))
        return rc;
    if (D == 0) return LRSCAN_OK;
    if ((rc = check_f32("grad_w", grad_w, true)) || (rc = check_f32("grad_bias", grad_bias, false))) return rc;
    const cudaStream_t st = call_stream(stream);
    if (B == 0 || T == 0) {
        if ((rc = copy_rows(grad_w, nullptr, static_cast<size_t>(D) * K * 4, st)) ||
            (rc = copy_rows(grad_bias, nullptr, static_cast<size_t>(D) * 4, st)))
            return rc;
        return copy_rows(grad_x0, grad_last, static_cast<size_t>(B) * (K - 1) * D * elem(dtype), st);
    }
    ConvArgs a{};
    if ((rc = conv_common(&a, x, w, K, x0, segment_pos, B, T, D, dtype)) ||
        (rc = rows_of("grad_out", grad_out, B, T, D, dtype, false, &a.go)) ||
        (rc = rows_of("grad_x", grad_x, B, T, D, dtype, true, &a.o)))
        return rc;
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    void *ws = nullptr;
    if ((rc = call_workspace(ctx, st, lrscan_conv_workspace_bytes(B, T, D, K), opts, &ws))) return rc;
    a.part = static_cast<float *>(ws);
    a.grad_last = grad_last;
    a.grad_x0 = grad_x0;
    a.vec = D % 4 == 0 && quads(a.x, dtype) && quads(a.o, dtype) && quads(a.go, dtype) && quads(x0, dtype) &&
            quads(grad_last, dtype) && quads(grad_x0, dtype);
    a.stream = st;
    if (conv_bwd_launch(a, K, dtype)) return launch_failed("the causal convolution's backward");
    return conv_finish_launch(a.part, B * a.chunks, D, K, grad_w, grad_bias, st)
               ? launch_failed("the reduction of grad_w")
               : LRSCAN_OK;
}

int lrscan_step_conv(const lrscan_rows *x, const float *w, const float *bias, int K, void *state, const int32_t *slots,
                     const lrscan_rows *out, int64_t B, int64_t S, int64_t D, int dtype, void *stream) {
    begin_call();
    int rc = call_shape(B, 1, D, dtype);
    if (rc || (rc = call_shape(S, kConvMaxTaps, D, dtype)) || (rc = check_taps(K))) return rc;
    if (B == 0 || D == 0) return LRSCAN_OK;
    RowsArg in, o;
    if ((rc = rows_of("x", x, B, 1, D, dtype, false, &in)) || (rc = rows_of("out", out, B, 1, D, dtype, true, &o)) ||
        (rc = check_f32("w", w, true)) || (rc = check_f32("bias", bias, false)) ||
        (rc = check_f32("slots", slots, false)) || (rc = check_elem("state", state, dtype)))
        return rc;
    if (!state) return report_errorf(LRSCAN_EINVAL, "NULL state");
    if (!slots && S < B)
        return report_errorf(LRSCAN_EINVAL, "a state of %lld rows for %lld requests without slots",
                             static_cast<long long>(S), static_cast<long long>(B));
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    const ConvStep g{in.p, in.sb, o.sb, o.p, w, bias, state, slots, S, B, D, ctx.status, call_stream(stream)};
    return conv_step_launch(g, K, dtype) ? launch_failed("the single-token convolution") : LRSCAN_OK;
}

int lrscan_fwd_embed(const void *ids, int id_bytes, const void *weight, int wdtype, float scale, void *out, int odtype,
                     int64_t N, int64_t V, int64_t D, void *stream) {
    begin_call();
    int rc = embed_shape(N, V, D, wdtype, odtype);
    if (rc) return rc;
    if (N == 0 || D == 0) return LRSCAN_OK;
    if (V == 0) return report_errorf(LRSCAN_EINVAL, "an empty table");
    EmbedArgs a{};
    if ((rc = embed_common(&a, ids, id_bytes, weight, wdtype, out, odtype, scale, N, V, D))) return rc;
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    a.status = ctx.status;
    a.sm_count = ctx.sm_count;
    a.stream = call_stream(stream);
    return embed_fwd_launch(a, wdtype, odtype) ? launch_failed("the embedding lookup") : LRSCAN_OK;
}

size_t lrscan_embed_workspace_bytes(int64_t N, int64_t V, int64_t D) {
    if (embed_shape(N, V, D, LRSCAN_F32, LRSCAN_F32) || N == 0 || V == 0 || D == 0) return 0;
    CallCtx ctx;
    return embed_scratch(N, V, D, call_device(&ctx) ? 152 : ctx.sm_count).total();
}

int lrscan_bwd_embed(const void *ids, int id_bytes, const void *grad_out, int gdtype, float scale, void *grad_weight,
                     int wdtype, int accumulate, int64_t N, int64_t V, int64_t D, void *stream,
                     const lrscan_opts *opts) {
    begin_call();
    int rc = embed_shape(N, V, D, wdtype, gdtype);
    if (rc) return rc;
    if (V == 0 || D == 0) return LRSCAN_OK;
    EmbedArgs a{};
    if ((rc = embed_common(&a, ids, id_bytes, grad_out, gdtype, grad_weight, wdtype, scale, N, V, D))) return rc;
    const cudaStream_t st = call_stream(stream);
    if (N == 0)
        return accumulate ? LRSCAN_OK : copy_rows(grad_weight, nullptr, static_cast<size_t>(V) * D * elem(wdtype), st);
    CallCtx ctx;
    if ((rc = call_device(&ctx))) return rc;
    const EmbedScratch sc = embed_scratch(N, V, D, ctx.sm_count);
    void *ws = nullptr;
    if ((rc = call_workspace(ctx, st, sc.total(), opts, &ws))) return rc;
    char *base = static_cast<char *>(ws);
    for (int k = 0; k < 2; ++k) {
        a.keys[k] = reinterpret_cast<uint32_t *>(base + k * sc.list);
        a.vals[k] = reinterpret_cast<uint32_t *>(base + (2 + k) * sc.list);
    }
    a.runs = reinterpret_cast<int *>(base + 4 * sc.list);
    a.run_at = reinterpret_cast<uint32_t *>(base + 4 * sc.list + 256);
    a.part = reinterpret_cast<float *>(base + 4 * sc.list + sc.runs);
    a.bits = sc.bits;
    a.passes = sc.passes;
    a.per = sc.per;
    a.add = accumulate != 0;
    a.status = ctx.status;
    a.sm_count = ctx.sm_count;
    a.stream = st;
    return embed_bwd_launch(a, gdtype, wdtype) ? launch_failed("the embedding's backward") : LRSCAN_OK;
}

}  // extern "C"
