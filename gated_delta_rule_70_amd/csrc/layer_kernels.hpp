// Host-side launch interface of the layer operators (channel scan, gated feed-forward, linear
// cross entropy, linear attention, norms of queries and keys) between the C ABI (layer_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_plan.hpp"

namespace gdr {

// A launch takes fewer than 2^32 threads along x: more workgroups go along y as well. A kernel numbers
// them with block_id(), and those past its last one have nothing to do.
inline dim3 grid_of(int64_t blocks, int threads) {
    const int64_t most = INT64_C(0xffffffff) / threads, rows = (blocks + most - 1) / most;
    return rows < 2 ? dim3((unsigned)blocks) : dim3((unsigned)((blocks + rows - 1) / rows), (unsigned)rows);
}
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

struct ScanArgs {
    const void *x, *a, *b;          // [B][T][D]
    const float *A_log, *dt_bias;   // [D]
    const float *h0;                // [nseq][D] or null
    const int32_t *cu_seqlens;
    void *out;                      // [B][T][D]
    float *hT;                      // [nseq][D] or null
    float *states;                  // [slots][D] or null (forward writes, backward reads)
    // backward
    const void *dout;
    const float *dhT;
    void *dx, *da, *db;
    float *dA_log, *ddt_bias, *dh0;
    float *ws;
    int64_t B, T, D, nseq, slots;
    uint32_t flags;
};

struct FfnArgs {
    const void *x, *wg, *wu;        // [M][D], [F][D], [F][D]
    void *h, *gate, *up;            // [M][F]; gate, up null unless kept, in fp32 with `wide`
    // backward (gate and up as the forward kept them)
    const void *dh;
    void *dx, *dwg, *dwu;
    void *ws;
    int64_t M, D, F;
    int act;
    bool wide;
};

struct CeArgs {
    const void *x, *w;              // [N][D], [V][D]
    const int64_t *t;               // [N]
    float *loss, *lse;              // [N]
    const float *lse_in, *dloss;
    void *dx, *dw;
    void *ws;
    int64_t N, D, V;
};

// One sweep of linear attention, out = A(x, y, z) in linear_attn.hip's terms: x, y [B][H][T][da], z and out [B][H][T][db]
// with the key heads (xk, yk, zk, ok) or the value heads; a state is [da][db].
struct AttnRole {
    const void *x, *y, *z;
    void *out;           // of value heads, in the tensors' type, or fp32 where the value heads of a key head are summed
    const void *other;   // like out: each row's product with out's goes to dot, [B][Hv][T], if that is wanted
    float *dot;
    const float *s_in;   // entering states by slot (in_slots) or sequence, or null for zeros
    const float *s_cuts; // with cuts: entering states of the segments of cut sequences, by slot and turned (s_in is for the others)
    float *s_out;        // states that sequences end with; without outputs, the segments' own, by slot
    float *decay;        // without outputs: the segments' decays [slots][Hv]
    int32_t da, db;
    bool xk, yk, zk, ok, reverse, in_turned, out_turned, in_slots;  // *_turned: the state is stored as [db][da]
    bool cuts;           // forwards: only segments that another one follows have a state of their own
    bool shares;         // mixed form: out is fp32
};

struct AttnArgs {
    AttnRole roles[3];
    const float *la;     // [B][Hv][T] (la_token) or [Hv]
    const int32_t *cu;
    int64_t B, T, Hk, Hv, nseq;
    int64_t seg, per_seq, slots, slices;  // seg 0: slots are sequences
    int64_t cuts;                         // where a sequence may be cut: slots without the sequences
    bool la_token;
    uint32_t group;                       // value heads of a key head
    Divisor by_inner, by_roles, by_slices, by_Hk, by_per, by_cuts, by_seg;
};

// A call of linear attention: forward, backward or step (x, y, z of the roles unused).
struct AttnCall {
    const void *q, *k, *v;
    const float *la, *h0;
    const int32_t *cu;
    void *out;
    float *hT;
    // backward
    const void *dout;
    const float *dhT;
    void *dq, *dk, *dv;
    float *dla, *dh0;
    char *ws;
    int64_t B, T, Hk, Hv, nseq, dk_size, dv_size;
    bool la_token;
};

struct QkArgs {
    const void *q, *k;               // rows of a token, q_stride and k_stride elements apart: [rows][H][d]
    const float *w_q, *w_k;          // [d] or null
    const float *inv_freq;           // [rot / 2]
    const int64_t *positions;        // [rows] or null: the token's place in its batch row
    void *oq, *ok;                   // [B][H][T][d]
    // backward
    const void *doq, *dok;           // like oq, ok
    void *dq, *dk;                   // rows as q and k, dq_stride and dk_stride elements apart
    float *dw_q, *dw_k;              // [d] or null
    double *part;                    // one row of [2][d] a workgroup, or null: no weights' gradients
    int64_t rows, T, q_stride, k_stride, dq_stride, dk_stride;
    int Hq, Hk, d, rot;
    float eps, inv_d;
    bool next;                       // neighbours are paired, not halves
    // the launch
    int64_t tiles;
    int q_steps, all_steps, steps, chunks;
    Divisor by_chunks, by_T;
};

hipError_t launch_scan_fwd(const ScanArgs &a, int dtype, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs &a, int dtype, hipStream_t s);
// out = one token of nseq sequences: h0 is the state read, hT the state written
hipError_t launch_scan_step(const ScanArgs &a, int dtype, hipStream_t s);
int64_t scan_fwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype);
int64_t scan_bwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype);

hipError_t launch_attn_fwd(const AttnCall &c, int dtype, hipStream_t s);
hipError_t launch_attn_bwd(const AttnCall &c, int dtype, hipStream_t s);
// one token of nseq sequences: h0 is the state read, hT the state written
hipError_t launch_attn_step(const AttnCall &c, int dtype, hipStream_t s);

hipError_t launch_qk_fwd(const QkArgs &a, int dtype, hipStream_t s);
hipError_t launch_qk_bwd(const QkArgs &a, int dtype, hipStream_t s);

hipError_t launch_ffn_fwd(const FfnArgs &a, int dtype, hipStream_t s);
hipError_t launch_ffn_bwd(const FfnArgs &a, int dtype, hipStream_t s);
int64_t ffn_bwd_ws_bytes(int64_t M, int64_t D, int64_t F, int dtype);

hipError_t launch_ce_fwd(const CeArgs &a, int dtype, hipStream_t s);
hipError_t launch_ce_bwd(const CeArgs &a, int dtype, hipStream_t s);
int64_t ce_fwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype);
int64_t ce_bwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype);

}  // namespace gdr
