// C ABI of the layer operators (channel scan, gated feed-forward, linear cross entropy):
// host-side argument validation and dispatch. Every check happens before anything is enqueued;
// see include/gdr.h for the contract.
#include "../../include/gdr.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_host.hpp"
#include "gdr_kernels.hpp"
#include "layer_kernels.hpp"

using gdr::aligned;
using gdr::elem_size;
using gdr::fail;
using gdr::g_last_error;
using gdr::overlap;
using gdr::prod;
using gdr::Range;
using gdr::rng;

namespace {

// One buffer of a call: its bytes, and whether it may be NULL.
struct Buf {
    Range r;
    bool optional;
    Buf(const char *name, const void *p, int64_t bytes, bool opt = false) : r(rng(name, p, bytes)), optional(opt) {}
};

// Presence and alignment of every buffer, and no output overlapping an input or another output.
template <size_t NI, size_t NO>
gdr_status_t check_buffers(const Buf (&ins)[NI], const Buf (&outs)[NO]) {
    auto one = [](const Buf &b) -> gdr_status_t {
        if (b.r.lo == 0 && !b.optional && b.r.hi > 0) return fail(GDR_ERR_NULL, "%s is NULL", b.r.name);
        if (b.r.lo % 16) return fail(GDR_ERR_ALIGN, "%s is not 16-byte aligned", b.r.name);
        return GDR_OK;
    };
    for (const Buf &b : ins) {
        const gdr_status_t s = one(b);
        if (s != GDR_OK) return s;
    }
    for (const Buf &b : outs) {
        const gdr_status_t s = one(b);
        if (s != GDR_OK) return s;
    }
    for (const Buf &o : outs) {
        for (const Buf &i : ins)
            if (overlap(o.r, i.r)) return fail(GDR_ERR_ALIAS, "%s overlaps %s", o.r.name, i.r.name);
        for (const Buf &o2 : outs)
            if (&o2 != &o && overlap(o.r, o2.r)) return fail(GDR_ERR_ALIAS, "%s overlaps %s", o.r.name, o2.r.name);
    }
    return GDR_OK;
}

gdr_status_t check_dtype(int32_t dtype) {
    if (dtype != GDR_F32 && dtype != GDR_BF16)
        return fail(GDR_ERR_DTYPE, "dtype %d is not GDR_F32 or GDR_BF16", dtype);
    return GDR_OK;
}

gdr_status_t launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(GDR_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return GDR_OK;
}

// rows are walked with 32-bit offsets within a tile or a block of tokens
constexpr int64_t kMaxWidth = INT64_C(1) << 20;

// ------------------------------------------------------------------ channel scan

struct ScanSizes {
    int64_t nseq, slots, n, ns;  // sequences, blocks, elements, state elements
};

gdr_status_t scan_sizes(const gdr_scan_dims_t *dims, bool packed, ScanSizes *z) {
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    const gdr_scan_dims_t &d = *dims;
    const gdr_status_t s = check_dtype(d.dtype);
    if (s != GDR_OK) return s;
    if (d.flags & ~GDR_REVERSE) return fail(GDR_ERR_FLAGS, "flags 0x%x: the channel scan takes GDR_REVERSE only", d.flags);
    if (d.B < 0 || d.T < 0 || d.D < 1)
        return fail(GDR_ERR_DIMS, "B (%lld) and T (%lld) must be >= 0 and D (%lld) >= 1", (long long)d.B, (long long)d.T, (long long)d.D);
    if (d.T > INT32_MAX) return fail(GDR_ERR_DIMS, "T must be below 2^31");
    z->nseq = d.B;
    if (packed) {
        if (d.B != 1) return fail(GDR_ERR_DIMS, "cu_seqlens needs B == 1 (got %lld)", (long long)d.B);
        if (d.num_seqs < 1) return fail(GDR_ERR_DIMS, "num_seqs (%lld) must be >= 1 with cu_seqlens", (long long)d.num_seqs);
        z->nseq = d.num_seqs;
    }
    const int64_t CB = gdr::kScanBlock;
    z->slots = packed ? d.T / CB + d.num_seqs + 1 : prod({d.B, (d.T + CB - 1) / CB});
    z->n = prod({d.B, d.T, d.D});
    z->ns = prod({z->nseq, d.D});
    if (z->n < 0 || z->ns < 0 || z->slots < 0 || z->n > (INT64_C(1) << 58) || z->ns > (INT64_C(1) << 58) ||
        prod({z->slots, d.D}) < 0 || prod({z->slots, d.D}) > (INT64_C(1) << 58))
        return fail(GDR_ERR_DIMS, "sizes overflow");
    if (d.D > kMaxWidth) return fail(GDR_ERR_DIMS, "D (%lld) must be at most 2^20", (long long)d.D);
    // the launches hold a block per (sequence or block of tokens, 16 channels) at most
    if (prod({z->nseq + z->slots, (d.D + 15) / 16}) > INT32_MAX)
        return fail(GDR_ERR_DIMS, "too many sequences or channels");
    return GDR_OK;
}

void scan_args(gdr::ScanArgs *a, const gdr_scan_dims_t &d, const ScanSizes &z, const void *x, const void *ra, const void *rb,
               const float *A_log, const float *dt_bias, const int32_t *cu) {
    *a = gdr::ScanArgs{};
    a->x = x; a->a = ra; a->b = rb;
    a->A_log = A_log; a->dt_bias = dt_bias;
    a->cu_seqlens = cu;
    a->B = d.B; a->T = d.T; a->D = d.D;
    a->nseq = z.nseq; a->slots = z.slots;
    a->flags = d.flags;
}

gdr_status_t check_workspace(const void *ws, int64_t have, int64_t need) {
    if (need > 0 && !ws) return fail(GDR_ERR_NULL, "workspace is NULL");
    if (have < need)
        return fail(GDR_ERR_DIMS, "workspace_bytes %lld is below the %lld bytes this call needs", (long long)have, (long long)need);
    return GDR_OK;
}

// ------------------------------------------------------------------ feed-forward and cross entropy

gdr_status_t ffn_sizes(const gdr_ffn_dims_t *dims) {
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    const gdr_ffn_dims_t &d = *dims;
    const gdr_status_t s = check_dtype(d.dtype);
    if (s != GDR_OK) return s;
    const int32_t act = d.act & ~GDR_FFN_KEEP_F32;
    if (act != GDR_ACT_SILU && act != GDR_ACT_GELU_TANH)
        return fail(GDR_ERR_FLAGS, "act %d is not GDR_ACT_SILU or GDR_ACT_GELU_TANH", d.act);
    if (d.M < 0 || d.D < 1 || d.F < 1 || d.D > kMaxWidth || d.F > kMaxWidth || d.M > INT32_MAX)
        return fail(GDR_ERR_DIMS, "M (%lld) must be in [0, 2^31), D (%lld) and F (%lld) in [1, 2^20]", (long long)d.M, (long long)d.D, (long long)d.F);
    // at most one workgroup per 64 x 64 tile of any of the products
    if (((d.M + 63) / 64) * ((d.F + 63) / 64 + (d.D + 63) / 64) > INT32_MAX / 4 || prod({d.M, d.F + 8}) / 256 > INT32_MAX / 4)
        return fail(GDR_ERR_DIMS, "M (%lld) is too large for these widths", (long long)d.M);
    return GDR_OK;
}

// the type gate and up are kept in: dtype, or fp32
bool ffn_wide(const gdr_ffn_dims_t &d) { return (d.act & GDR_FFN_KEEP_F32) != 0; }
int64_t ffn_kept_bytes(const gdr_ffn_dims_t &d) { return d.M * d.F * (ffn_wide(d) ? 4 : elem_size(d.dtype)); }

gdr_status_t ce_sizes(const gdr_ce_dims_t *dims) {
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    const gdr_ce_dims_t &d = *dims;
    const gdr_status_t s = check_dtype(d.dtype);
    if (s != GDR_OK) return s;
    if (d.flags) return fail(GDR_ERR_FLAGS, "flags 0x%x has unknown bits", d.flags);
    if (d.N < 0 || d.D < 1 || d.V < 1 || d.D > kMaxWidth || d.N > INT32_MAX || d.V > INT32_MAX)
        return fail(GDR_ERR_DIMS, "N (%lld) must be in [0, 2^31), V (%lld) in [1, 2^31), D (%lld) in [1, 2^20]", (long long)d.N, (long long)d.V, (long long)d.D);
    if (prod({(d.N + 63) / 64, (d.V + 63) / 64}) > INT32_MAX / 4)
        return fail(GDR_ERR_DIMS, "N (%lld) is too large for this vocabulary", (long long)d.N);
    return GDR_OK;
}

}  // namespace

extern "C" {

int64_t gdr_channel_scan_states_elems(const gdr_scan_dims_t *dims, int32_t packed) {
    ScanSizes z;
    if (scan_sizes(dims, packed != 0, &z) != GDR_OK) return -1;
    return z.slots * dims->D;
}

int64_t gdr_channel_scan_fwd_workspace_bytes(const gdr_scan_dims_t *dims, int32_t packed) {
    ScanSizes z;
    if (scan_sizes(dims, packed != 0, &z) != GDR_OK) return -1;
    return gdr::scan_fwd_ws_bytes(dims->T, dims->D, z.nseq, packed != 0, dims->dtype);
}

int64_t gdr_channel_scan_bwd_workspace_bytes(const gdr_scan_dims_t *dims, int32_t packed) {
    ScanSizes z;
    if (scan_sizes(dims, packed != 0, &z) != GDR_OK) return -1;
    return gdr::scan_bwd_ws_bytes(dims->T, dims->D, z.nseq, packed != 0, dims->dtype);
}

gdr_status_t gdr_channel_scan_fwd(const void *x, const void *a, const void *b, const float *A_log, const float *dt_bias,
                                  const float *h0, const int32_t *cu_seqlens, void *out, float *hT, float *states,
                                  void *workspace, int64_t workspace_bytes, const gdr_scan_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    ScanSizes z;
    gdr_status_t s = scan_sizes(dims, cu_seqlens != nullptr, &z);
    if (s != GDR_OK) return s;
    const gdr_scan_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = gdr::scan_fwd_ws_bytes(d.T, d.D, z.nseq, cu_seqlens != nullptr, d.dtype);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    if (cu_seqlens && !aligned(cu_seqlens, 4)) return fail(GDR_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
    // hT may be exactly h0: a state is read before it is written, by one thread
    const bool in_place = hT && hT == h0;
    const Buf ins[] = {Buf("x", x, z.n * es), Buf("a", a, z.n * es), Buf("b", b, z.n * es), Buf("A_log", A_log, d.D * 4),
                       Buf("dt_bias", dt_bias, d.D * 4), Buf("h0", in_place ? nullptr : h0, z.ns * 4, true)};
    const Buf outs[] = {Buf("out", out, z.n * es), Buf("hT", hT, z.ns * 4, true),
                        Buf("states", states, z.slots * d.D * 4, true), Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    const Range rcu = rng("cu_seqlens", cu_seqlens, cu_seqlens ? (z.nseq + 1) * 4 : 0);
    for (const Buf &o : outs)
        if (overlap(o.r, rcu)) return fail(GDR_ERR_ALIAS, "%s overlaps cu_seqlens", o.r.name);
    gdr::ScanArgs g;
    scan_args(&g, d, z, x, a, b, A_log, dt_bias, cu_seqlens);
    g.h0 = h0; g.out = out; g.hT = hT; g.states = states;
    g.ws = static_cast<float *>(workspace);
    return launched(gdr::launch_scan_fwd(g, d.dtype, reinterpret_cast<hipStream_t>(stream)), "channel scan");
}

gdr_status_t gdr_channel_scan_bwd(const void *x, const void *a, const void *b, const float *A_log, const float *dt_bias,
                                  const float *states, const int32_t *cu_seqlens, const void *dout, const float *dhT,
                                  void *dx, void *da, void *db, float *dA_log, float *ddt_bias, float *dh0,
                                  void *workspace, int64_t workspace_bytes, const gdr_scan_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    ScanSizes z;
    gdr_status_t s = scan_sizes(dims, cu_seqlens != nullptr, &z);
    if (s != GDR_OK) return s;
    const gdr_scan_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = gdr::scan_bwd_ws_bytes(d.T, d.D, z.nseq, cu_seqlens != nullptr, d.dtype);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    if (cu_seqlens && !aligned(cu_seqlens, 4)) return fail(GDR_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
    const Buf ins[] = {Buf("x", x, z.n * es), Buf("a", a, z.n * es), Buf("b", b, z.n * es), Buf("A_log", A_log, d.D * 4),
                       Buf("dt_bias", dt_bias, d.D * 4), Buf("states", states, z.n ? z.slots * d.D * 4 : 0),
                       Buf("dout", dout, z.n * es), Buf("dhT", dhT, z.ns * 4, true)};
    const Buf outs[] = {Buf("dx", dx, z.n * es), Buf("da", da, z.n * es), Buf("db", db, z.n * es),
                        Buf("dA_log", dA_log, d.D * 4), Buf("ddt_bias", ddt_bias, d.D * 4), Buf("dh0", dh0, z.ns * 4, true),
                        Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    const Range rcu = rng("cu_seqlens", cu_seqlens, cu_seqlens ? (z.nseq + 1) * 4 : 0);
    for (const Buf &o : outs)
        if (overlap(o.r, rcu)) return fail(GDR_ERR_ALIAS, "%s overlaps cu_seqlens", o.r.name);
    gdr::ScanArgs g;
    scan_args(&g, d, z, x, a, b, A_log, dt_bias, cu_seqlens);
    g.states = const_cast<float *>(states);
    g.dout = dout; g.dhT = dhT;
    g.dx = dx; g.da = da; g.db = db; g.dA_log = dA_log; g.ddt_bias = ddt_bias; g.dh0 = dh0;
    g.ws = static_cast<float *>(workspace);
    return launched(gdr::launch_scan_bwd(g, d.dtype, reinterpret_cast<hipStream_t>(stream)), "channel scan backward");
}

gdr_status_t gdr_channel_scan_step(const void *x, const void *a, const void *b, const float *A_log, const float *dt_bias,
                                   const float *state_in, float *state_out, void *out, const gdr_scan_dims_t *dims,
                                   void *stream) {
    g_last_error[0] = '\0';
    ScanSizes z;
    gdr_status_t s = scan_sizes(dims, false, &z);
    if (s != GDR_OK) return s;
    const gdr_scan_dims_t &d = *dims;
    if (d.T != 1) return fail(GDR_ERR_DIMS, "T must be 1 for a step (got %lld)", (long long)d.T);
    if (d.flags) return fail(GDR_ERR_FLAGS, "flags 0x%x: a step takes none", d.flags);
    const int64_t es = elem_size(d.dtype);
    const bool in_place = state_out && state_out == state_in;
    if (z.ns > 0 && !state_in) return fail(GDR_ERR_NULL, "state_in is NULL");
    const Buf ins[] = {Buf("x", x, z.n * es), Buf("a", a, z.n * es), Buf("b", b, z.n * es), Buf("A_log", A_log, d.D * 4),
                       Buf("dt_bias", dt_bias, d.D * 4), Buf("state_in", in_place ? nullptr : state_in, z.ns * 4, true)};
    const Buf outs[] = {Buf("out", out, z.n * es), Buf("state_out", state_out, z.ns * 4)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::ScanArgs g;
    scan_args(&g, d, z, x, a, b, A_log, dt_bias, nullptr);
    g.h0 = state_in; g.hT = state_out; g.out = out;
    return launched(gdr::launch_scan_step(g, d.dtype, reinterpret_cast<hipStream_t>(stream)), "channel scan step");
}

gdr_status_t gdr_gated_ffn_fwd(const void *x, const void *w_gate, const void *w_up, void *h, void *gate, void *up,
                               const gdr_ffn_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = ffn_sizes(dims);
    if (s != GDR_OK) return s;
    const gdr_ffn_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), nx = d.M * d.D * es, nw = d.F * d.D * es, nh = d.M * d.F * es;
    if (nh > 0 && (gate == nullptr) != (up == nullptr)) return fail(GDR_ERR_NULL, "gate and up are kept together or not at all");
    const Buf ins[] = {Buf("x", x, nx), Buf("w_gate", w_gate, nw), Buf("w_up", w_up, nw)};
    const int64_t nk = ffn_kept_bytes(d);
    const Buf outs[] = {Buf("h", h, nh), Buf("gate", gate, nk, true), Buf("up", up, nk, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::FfnArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up;
    a.h = h; a.gate = gate; a.up = up;
    a.M = d.M; a.D = d.D; a.F = d.F; a.act = d.act & ~GDR_FFN_KEEP_F32; a.wide = ffn_wide(d);
    return launched(gdr::launch_ffn_fwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "gated feed-forward");
}

int64_t gdr_gated_ffn_bwd_workspace_bytes(const gdr_ffn_dims_t *dims) {
    if (ffn_sizes(dims) != GDR_OK) return -1;
    return gdr::ffn_bwd_ws_bytes(dims->M, dims->D, dims->F, dims->dtype);
}

gdr_status_t gdr_gated_ffn_bwd(const void *x, const void *w_gate, const void *w_up, const void *gate, const void *up,
                               const void *dh, void *dx, void *dw_gate, void *dw_up, void *workspace,
                               int64_t workspace_bytes, const gdr_ffn_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = ffn_sizes(dims);
    if (s != GDR_OK) return s;
    const gdr_ffn_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), nx = d.M * d.D * es, nw = d.F * d.D * es, nh = d.M * d.F * es;
    const int64_t need = gdr::ffn_bwd_ws_bytes(d.M, d.D, d.F, d.dtype), nk = ffn_kept_bytes(d);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    const Buf ins[] = {Buf("x", x, nx), Buf("w_gate", w_gate, nw), Buf("w_up", w_up, nw),
                       Buf("gate", gate, nk), Buf("up", up, nk), Buf("dh", dh, nh)};
    const Buf outs[] = {Buf("dx", dx, nx), Buf("dw_gate", dw_gate, nw), Buf("dw_up", dw_up, nw),
                        Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::FfnArgs a{};
    a.x = x; a.wg = w_gate; a.wu = w_up;
    a.gate = const_cast<void *>(gate); a.up = const_cast<void *>(up);
    a.dh = dh; a.dx = dx; a.dwg = dw_gate; a.dwu = dw_up; a.ws = workspace;
    a.M = d.M; a.D = d.D; a.F = d.F; a.act = d.act & ~GDR_FFN_KEEP_F32; a.wide = ffn_wide(d);
    return launched(gdr::launch_ffn_bwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "gated feed-forward backward");
}

int64_t gdr_linear_ce_fwd_workspace_bytes(const gdr_ce_dims_t *dims) {
    if (ce_sizes(dims) != GDR_OK) return -1;
    return gdr::ce_fwd_ws_bytes(dims->N, dims->D, dims->V, dims->dtype);
}

int64_t gdr_linear_ce_bwd_workspace_bytes(const gdr_ce_dims_t *dims) {
    if (ce_sizes(dims) != GDR_OK) return -1;
    return gdr::ce_bwd_ws_bytes(dims->N, dims->D, dims->V, dims->dtype);
}

gdr_status_t gdr_linear_ce_fwd(const void *x, const void *w, const int64_t *targets, float *loss, float *lse,
                               void *workspace, int64_t workspace_bytes, const gdr_ce_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = ce_sizes(dims);
    if (s != GDR_OK) return s;
    const gdr_ce_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = gdr::ce_fwd_ws_bytes(d.N, d.D, d.V, d.dtype);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    const Buf ins[] = {Buf("x", x, d.N * d.D * es), Buf("w", w, d.V * d.D * es), Buf("targets", targets, d.N * 8)};
    const Buf outs[] = {Buf("loss", loss, d.N * 4), Buf("lse", lse, d.N * 4), Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::CeArgs a{};
    a.x = x; a.w = w; a.t = targets;
    a.loss = loss; a.lse = lse; a.ws = workspace;
    a.N = d.N; a.D = d.D; a.V = d.V;
    return launched(gdr::launch_ce_fwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "linear cross entropy");
}

gdr_status_t gdr_linear_ce_bwd(const void *x, const void *w, const int64_t *targets, const float *lse, const float *dloss,
                               void *dx, void *dw, void *workspace, int64_t workspace_bytes, const gdr_ce_dims_t *dims,
                               void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = ce_sizes(dims);
    if (s != GDR_OK) return s;
    const gdr_ce_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = gdr::ce_bwd_ws_bytes(d.N, d.D, d.V, d.dtype);
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    const Buf ins[] = {Buf("x", x, d.N * d.D * es), Buf("w", w, d.V * d.D * es), Buf("targets", targets, d.N * 8),
                       Buf("lse", lse, d.N * 4), Buf("dloss", dloss, d.N * 4)};
    const Buf outs[] = {Buf("dx", dx, d.N * d.D * es), Buf("dw", dw, d.V * d.D * es), Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::CeArgs a{};
    a.x = x; a.w = w; a.t = targets;
    a.lse_in = lse; a.dloss = dloss;
    a.dx = dx; a.dw = dw; a.ws = workspace;
    a.N = d.N; a.D = d.D; a.V = d.V;
    return launched(gdr::launch_ce_bwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "linear cross entropy backward");
}

}  // extern "C"
