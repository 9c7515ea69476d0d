// Host-side launch interface of the layer operators (channel scan, gated feed-forward, linear
// cross entropy) between the C ABI (layer_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// Tokens per block of the channel scan: the forward keeps the state that enters each block of a
// sequence when the backward will run. Packed sequences: the blocks of sequence s start at slot
// cu[s] / kScanBlock + s, so that no two sequences share one.
constexpr int kScanBlock = 256;

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
    void *h, *gate, *up;            // [M][F]; gate, up null unless kept
    // backward (gate and up as the forward kept them)
    const void *dh;
    void *dx, *dwg, *dwu;
    void *ws;
    int64_t M, D, F;
    int act;
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

hipError_t launch_scan_fwd(const ScanArgs &a, int dtype, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs &a, int dtype, hipStream_t s);
// out = one token of nseq sequences: h0 is the state read, hT the state written
hipError_t launch_scan_step(const ScanArgs &a, int dtype, hipStream_t s);
int64_t scan_fwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype);
int64_t scan_bwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype);

hipError_t launch_ffn_fwd(const FfnArgs &a, int dtype, hipStream_t s);
hipError_t launch_ffn_bwd(const FfnArgs &a, int dtype, hipStream_t s);
int64_t ffn_bwd_ws_bytes(int64_t M, int64_t D, int64_t F, int dtype);

hipError_t launch_ce_fwd(const CeArgs &a, int dtype, hipStream_t s);
hipError_t launch_ce_bwd(const CeArgs &a, int dtype, hipStream_t s);
int64_t ce_fwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype);
int64_t ce_bwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype);

}  // namespace gdr
