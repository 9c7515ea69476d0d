// C ABI of the layer operators (channel scan, gated feed-forward, linear cross entropy, linear attention, norms of queries and keys):
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

// ------------------------------------------------------------------ linear attention

struct AttnSizes {
    int64_t nseq, nq, nv, na, ns;  // sequences; elements of q, of v, of log_alpha and of the states
};

gdr_status_t attn_heads(int64_t Hk, int64_t Hv, int64_t dk, int64_t dv, int32_t dtype, uint32_t flags) {
    const gdr_status_t s = check_dtype(dtype);
    if (s != GDR_OK) return s;
    if (flags & ~GDR_HEAD_DECAY) return fail(GDR_ERR_FLAGS, "flags 0x%x: linear attention takes GDR_HEAD_DECAY only", flags);
    if (Hk < 1 || Hv < 1 || Hv % Hk)
        return fail(GDR_ERR_DIMS, "Hv (%lld) must be a positive multiple of Hk (%lld)", (long long)Hv, (long long)Hk);
    if (dk != 64 && dk != 128) return fail(GDR_ERR_UNSUPPORTED, "dk must be 64 or 128 (got %lld)", (long long)dk);
    if (dv < 32 || dv > 256 || dv % 32)
        return fail(GDR_ERR_UNSUPPORTED, "dv must be a multiple of 32, at most 256 (got %lld)", (long long)dv);
    return GDR_OK;
}

gdr_status_t attn_sizes(const gdr_chunk_dims_t *dims, bool packed, AttnSizes *z) {
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    const gdr_chunk_dims_t &d = *dims;
    const gdr_status_t s = attn_heads(d.Hk, d.Hv, d.dk, d.dv, d.dtype, d.flags);
    if (s != GDR_OK) return s;
    // (tokens are counted in 32 bits, a chunk past a sequence's end too)
    if (d.B < 0 || d.T < 0 || d.T > INT32_MAX - 4096)
        return fail(GDR_ERR_DIMS, "B (%lld) must be >= 0 and T (%lld) in [0, 2^31 - 4096)", (long long)d.B, (long long)d.T);
    z->nseq = d.B;
    if (packed) {
        if (d.B != 1) return fail(GDR_ERR_DIMS, "cu_seqlens needs B == 1 (got %lld)", (long long)d.B);
        if (d.num_seqs < 1) return fail(GDR_ERR_DIMS, "num_seqs (%lld) must be >= 1 with cu_seqlens", (long long)d.num_seqs);
        z->nseq = d.num_seqs;
    }
    z->nq = prod({d.B, d.Hk, d.T, d.dk});
    z->nv = prod({d.B, d.Hv, d.T, d.dv});
    z->na = d.flags & GDR_HEAD_DECAY ? d.Hv : prod({d.B, d.Hv, d.T});
    z->ns = prod({z->nseq, d.Hv, d.dk, d.dv});
    // the gradients of shared heads and the segments' states take some times as much
    const int64_t most = INT64_C(1) << 52;
    if (z->nq < 0 || z->nv < 0 || z->na < 0 || z->ns < 0 || z->nq > most || z->nv > most || z->ns > most ||
        prod({d.B, d.Hv, d.T, d.dk}) < 0 || prod({d.B, d.Hv, d.T, d.dk}) > most)
        return fail(GDR_ERR_DIMS, "sizes overflow");
    if (!gdr::attn_numbered(z->nseq, d.B, d.T, d.Hv)) return fail(GDR_ERR_DIMS, "too many sequences or heads");
    return GDR_OK;
}

gdr::AttnSpace attn_space_of(const gdr_chunk_dims_t &d, const AttnSizes &z, bool packed, bool backward) {
    const int64_t units = backward ? d.Hv : d.Hv * gdr::attn_slices(d.dv);
    return gdr::attn_space(gdr::attn_plan(d.T, z.nseq, units, packed, backward), d.B, d.T, d.Hk, d.Hv, z.nseq, d.dk, d.dv, backward);
}

void attn_call(gdr::AttnCall *c, const gdr_chunk_dims_t &d, const AttnSizes &z, const void *q, const void *k, const void *v,
               const float *log_alpha, const float *h0, const int32_t *cu, void *workspace) {
    *c = gdr::AttnCall{};
    c->q = q; c->k = k; c->v = v;
    c->la = log_alpha; c->h0 = h0;
    c->cu = cu;
    c->ws = static_cast<char *>(workspace);
    c->B = d.B; c->T = d.T; c->Hk = d.Hk; c->Hv = d.Hv; c->nseq = z.nseq;
    c->dk_size = d.dk; c->dv_size = d.dv;
    c->la_token = !(d.flags & GDR_HEAD_DECAY);
}

// ------------------------------------------------------------------ norms of queries and keys

gdr_status_t qk_sizes(const gdr_qk_dims_t *dims, bool backward) {
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    const gdr_qk_dims_t &d = *dims;
    const gdr_status_t s = check_dtype(d.dtype);
    if (s != GDR_OK) return s;
    if (d.flags & ~GDR_ROPE_NEIGHBOURS) return fail(GDR_ERR_FLAGS, "flags 0x%x: only GDR_ROPE_NEIGHBOURS is known here", d.flags);
    if (d.d < 8 || d.d > 256 || d.d % 8) return fail(GDR_ERR_UNSUPPORTED, "d must be a multiple of 8, at most 256 (got %lld)", (long long)d.d);
    if (d.rot < 0 || d.rot > d.d || d.rot % 8)
        return fail(GDR_ERR_UNSUPPORTED, "rot must be a multiple of 8 in [0, d] (got %lld)", (long long)d.rot);
    const int64_t rows = prod({d.B, d.T});
    if (d.B < 0 || d.T < 0 || rows < 0 || rows > INT32_MAX)
        return fail(GDR_ERR_DIMS, "B (%lld) and T (%lld) must be >= 0, their product below 2^31", (long long)d.B, (long long)d.T);
    if (d.Hq < 1 || d.Hk < 1 || d.Hq > (1 << 16) || d.Hk > (1 << 16))
        return fail(GDR_ERR_DIMS, "Hq (%lld) and Hk (%lld) must be in [1, 2^16]", (long long)d.Hq, (long long)d.Hk);
    const struct {
        const char *name;
        int64_t stride, least;
        bool read;
    } rows_of[] = {{"q_stride", d.q_stride, d.Hq * d.d, true}, {"k_stride", d.k_stride, d.Hk * d.d, true},
                   {"dq_stride", d.dq_stride, d.Hq * d.d, backward}, {"dk_stride", d.dk_stride, d.Hk * d.d, backward}};
    for (const auto &r : rows_of)
        if (r.read && (r.stride < r.least || r.stride % 4 || r.stride > (INT64_C(1) << 30)))
            return fail(GDR_ERR_DIMS, "%s (%lld) must be a multiple of 4, at least the heads' %lld and at most 2^30", r.name, (long long)r.stride, (long long)r.least);
    if (!(d.eps >= 0.f) || d.eps > 3e38f) return fail(GDR_ERR_DIMS, "eps must be finite and >= 0");
    // a launch holds a workgroup per four tokens and step of heads at most (some hundred past its last where the grid has rows)
    if (prod({rows / 4 + 1, d.Hq + d.Hk}) > INT32_MAX - 4096) return fail(GDR_ERR_DIMS, "too many tokens or heads");
    return GDR_OK;
}

// bytes that H heads in rows `stride` elements apart span
int64_t qk_span(const gdr_qk_dims_t &d, int64_t H, int64_t stride) {
    const int64_t rows = d.B * d.T;
    return rows ? ((rows - 1) * stride + H * d.d) * elem_size(d.dtype) : 0;
}

void qk_args(gdr::QkArgs *a, const gdr_qk_dims_t &d, const void *q, const void *k, const float *w_q, const float *w_k, const float *inv_freq,
             const int64_t *positions) {
    *a = gdr::QkArgs{};
    a->q = q; a->k = k;
    a->w_q = w_q; a->w_k = w_k;
    a->inv_freq = inv_freq;
    a->positions = positions;
    a->rows = d.B * d.T;
    a->T = d.T > 0 ? d.T : 1;
    a->q_stride = d.q_stride; a->k_stride = d.k_stride; a->dq_stride = d.dq_stride; a->dk_stride = d.dk_stride;
    a->Hq = (int)d.Hq; a->Hk = (int)d.Hk; a->d = (int)d.d; a->rot = (int)d.rot;
    a->eps = d.eps;
    a->next = (d.flags & GDR_ROPE_NEIGHBOURS) != 0;
}

}  // namespace

extern "C" {

gdr_status_t gdr_qk_norm_rope_fwd(const void *q, const void *k, const float *w_q, const float *w_k, const float *inv_freq,
                                  const int64_t *positions, void *out_q, void *out_k, const gdr_qk_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = qk_sizes(dims, false);
    if (s != GDR_OK) return s;
    const gdr_qk_dims_t &d = *dims;
    const int64_t rows = d.B * d.T, es = elem_size(d.dtype);
    const Buf ins[] = {Buf("q", q, qk_span(d, d.Hq, d.q_stride)), Buf("k", k, qk_span(d, d.Hk, d.k_stride)), Buf("w_q", w_q, d.d * 4, true),
                       Buf("w_k", w_k, d.d * 4, true), Buf("inv_freq", inv_freq, d.rot * 2), Buf("positions", positions, rows * 8, true)};
    const Buf outs[] = {Buf("out_q", out_q, rows * d.Hq * d.d * es), Buf("out_k", out_k, rows * d.Hk * d.d * es)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::QkArgs a;
    qk_args(&a, d, q, k, w_q, w_k, inv_freq, positions);
    a.oq = out_q; a.ok = out_k;
    return launched(gdr::launch_qk_fwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "norms of queries and keys");
}

int64_t gdr_qk_norm_rope_bwd_workspace_bytes(const gdr_qk_dims_t *dims) {
    if (qk_sizes(dims, true) != GDR_OK) return -1;
    return gdr::qk_bwd_ws_bytes(dims->B * dims->T, dims->d);
}

gdr_status_t gdr_qk_norm_rope_bwd(const void *q, const void *k, const float *w_q, const float *w_k, const float *inv_freq,
                                  const int64_t *positions, const void *dout_q, const void *dout_k, void *dq, void *dk, float *dw_q,
                                  float *dw_k, void *workspace, int64_t workspace_bytes, const gdr_qk_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    gdr_status_t s = qk_sizes(dims, true);
    if (s != GDR_OK) return s;
    const gdr_qk_dims_t &d = *dims;
    const int64_t rows = d.B * d.T, es = elem_size(d.dtype), need = dw_q || dw_k ? gdr::qk_bwd_ws_bytes(rows, d.d) : 0;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    const Buf ins[] = {Buf("q", q, qk_span(d, d.Hq, d.q_stride)), Buf("k", k, qk_span(d, d.Hk, d.k_stride)), Buf("w_q", w_q, d.d * 4, true),
                       Buf("w_k", w_k, d.d * 4, true), Buf("inv_freq", inv_freq, d.rot * 2), Buf("positions", positions, rows * 8, true),
                       Buf("dout_q", dout_q, rows * d.Hq * d.d * es), Buf("dout_k", dout_k, rows * d.Hk * d.d * es)};
    // dq and dk may be parts of the same rows
    const int64_t sq = qk_span(d, d.Hq, d.dq_stride), sk = qk_span(d, d.Hk, d.dk_stride);
    if (overlap(rng("dq", dq, sq), rng("dk", dk, sk))) {
        const int64_t row = d.dq_stride * es;
        const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(dk) - reinterpret_cast<uintptr_t>(dq));
        const int64_t at = (apart % row + row) % row;
        if (d.dq_stride != d.dk_stride || at < d.Hq * d.d * es || at + d.Hk * d.d * es > row)
            return fail(GDR_ERR_ALIAS, "dq overlaps dk");
    }
    const Buf outs_q[] = {Buf("dq", dq, sq), Buf("dw_q", dw_q, d.d * 4, true), Buf("dw_k", dw_k, d.d * 4, true), Buf("workspace", workspace, need, true)};
    const Buf outs_k[] = {Buf("dk", dk, sk), outs_q[1], outs_q[2], outs_q[3]};
    s = check_buffers(ins, outs_q);
    if (s != GDR_OK) return s;
    s = check_buffers(ins, outs_k);
    if (s != GDR_OK) return s;
    gdr::QkArgs a;
    qk_args(&a, d, q, k, w_q, w_k, inv_freq, positions);
    a.doq = dout_q; a.dok = dout_k;
    a.dq = dq; a.dk = dk; a.dw_q = dw_q; a.dw_k = dw_k;
    a.part = need ? static_cast<double *>(workspace) : nullptr;
    return launched(gdr::launch_qk_bwd(a, d.dtype, reinterpret_cast<hipStream_t>(stream)), "norms of queries and keys backward");
}

int64_t gdr_linear_attn_fwd_workspace_bytes(const gdr_chunk_dims_t *dims, int32_t packed) {
    AttnSizes z;
    if (attn_sizes(dims, packed != 0, &z) != GDR_OK) return -1;
    return attn_space_of(*dims, z, packed != 0, false).total;
}

int64_t gdr_linear_attn_bwd_workspace_bytes(const gdr_chunk_dims_t *dims, int32_t packed) {
    AttnSizes z;
    if (attn_sizes(dims, packed != 0, &z) != GDR_OK) return -1;
    return attn_space_of(*dims, z, packed != 0, true).total;
}

gdr_status_t gdr_linear_attn_fwd(const void *q, const void *k, const void *v, const float *log_alpha, const float *h0,
                                 const int32_t *cu_seqlens, void *out, float *hT, void *workspace, int64_t workspace_bytes,
                                 const gdr_chunk_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    AttnSizes z;
    const bool packed = cu_seqlens != nullptr;
    gdr_status_t s = attn_sizes(dims, packed, &z);
    if (s != GDR_OK) return s;
    const gdr_chunk_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = attn_space_of(d, z, packed, false).total;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    if (!aligned(cu_seqlens, 4)) return fail(GDR_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
    // hT may be exactly h0: a workgroup reads its part of a state before it writes it
    const bool in_place = hT && hT == h0;
    const Buf ins[] = {Buf("q", q, z.nq * es), Buf("k", k, z.nq * es), Buf("v", v, z.nv * es), Buf("log_alpha", log_alpha, z.na * 4),
                       Buf("h0", in_place ? nullptr : h0, z.ns * 4, true)};
    const Buf outs[] = {Buf("out", out, z.nv * es), Buf("hT", hT, z.ns * 4, true), Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    const Range rcu = rng("cu_seqlens", cu_seqlens, packed ? (z.nseq + 1) * 4 : 0);
    for (const Buf &o : outs)
        if (overlap(o.r, rcu)) return fail(GDR_ERR_ALIAS, "%s overlaps cu_seqlens", o.r.name);
    gdr::AttnCall c;
    attn_call(&c, d, z, q, k, v, log_alpha, h0, cu_seqlens, workspace);
    c.out = out; c.hT = hT;
    return launched(gdr::launch_attn_fwd(c, d.dtype, reinterpret_cast<hipStream_t>(stream)), "linear attention");
}

gdr_status_t gdr_linear_attn_bwd(const void *q, const void *k, const void *v, const float *log_alpha, const float *h0,
                                 const int32_t *cu_seqlens, const void *dout, const float *dhT, void *dq, void *dk, void *dv,
                                 float *dlog_alpha, float *dh0, void *workspace, int64_t workspace_bytes,
                                 const gdr_chunk_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    AttnSizes z;
    const bool packed = cu_seqlens != nullptr;
    gdr_status_t s = attn_sizes(dims, packed, &z);
    if (s != GDR_OK) return s;
    const gdr_chunk_dims_t &d = *dims;
    const int64_t es = elem_size(d.dtype), need = attn_space_of(d, z, packed, true).total;
    s = check_workspace(workspace, workspace_bytes, need);
    if (s != GDR_OK) return s;
    if (!aligned(cu_seqlens, 4)) return fail(GDR_ERR_ALIGN, "cu_seqlens is not 4-byte aligned");
    const Buf ins[] = {Buf("q", q, z.nq * es), Buf("k", k, z.nq * es), Buf("v", v, z.nv * es), Buf("log_alpha", log_alpha, z.na * 4),
                       Buf("h0", h0, z.ns * 4, true), Buf("dout", dout, z.nv * es), Buf("dhT", dhT, z.ns * 4, true)};
    const Buf outs[] = {Buf("dq", dq, z.nq * es), Buf("dk", dk, z.nq * es), Buf("dv", dv, z.nv * es), Buf("dlog_alpha", dlog_alpha, z.na * 4),
                        Buf("dh0", dh0, z.ns * 4, true), Buf("workspace", workspace, need, true)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    const Range rcu = rng("cu_seqlens", cu_seqlens, packed ? (z.nseq + 1) * 4 : 0);
    for (const Buf &o : outs)
        if (overlap(o.r, rcu)) return fail(GDR_ERR_ALIAS, "%s overlaps cu_seqlens", o.r.name);
    gdr::AttnCall c;
    attn_call(&c, d, z, q, k, v, log_alpha, h0, cu_seqlens, workspace);
    c.dout = dout; c.dhT = dhT;
    c.dq = dq; c.dk = dk; c.dv = dv; c.dla = dlog_alpha; c.dh0 = dh0;
    return launched(gdr::launch_attn_bwd(c, d.dtype, reinterpret_cast<hipStream_t>(stream)), "linear attention backward");
}

gdr_status_t gdr_linear_attn_step(const void *q, const void *k, const void *v, const float *log_alpha, const float *state_in,
                                  float *state_out, void *out, const gdr_decode_dims_t *dims, void *stream) {
    g_last_error[0] = '\0';
    if (!dims) return fail(GDR_ERR_NULL, "dims is NULL");
    // one token a sequence
    const gdr_chunk_dims_t d{dims->N, 1, dims->Hk, dims->Hv, dims->dk, dims->dv, 0, dims->dtype, dims->flags};
    if (dims->N < 0) return fail(GDR_ERR_DIMS, "N (%lld) must be >= 0", (long long)dims->N);
    AttnSizes z;
    gdr_status_t s = attn_sizes(&d, false, &z);
    if (s != GDR_OK) return s;
    const int64_t es = elem_size(d.dtype);
    const bool in_place = state_out && state_out == state_in;
    if (z.ns > 0 && !state_in) return fail(GDR_ERR_NULL, "state_in is NULL");
    const Buf ins[] = {Buf("q", q, z.nq * es), Buf("k", k, z.nq * es), Buf("v", v, z.nv * es), Buf("log_alpha", log_alpha, z.na * 4),
                       Buf("state_in", in_place ? nullptr : state_in, z.ns * 4, true)};
    const Buf outs[] = {Buf("state_out", state_out, z.ns * 4), Buf("out", out, z.nv * es)};
    s = check_buffers(ins, outs);
    if (s != GDR_OK) return s;
    gdr::AttnCall c;
    attn_call(&c, d, z, q, k, v, log_alpha, state_in, nullptr, nullptr);
    c.out = out; c.hT = state_out;
    return launched(gdr::launch_attn_step(c, d.dtype, reinterpret_cast<hipStream_t>(stream)), "linear attention step");
}

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
