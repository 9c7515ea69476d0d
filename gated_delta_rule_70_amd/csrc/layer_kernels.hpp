// Host-side launch interface of the layer operators (channel scan, gated feed-forward, linear
// cross entropy) between the C ABI (layer_api.cpp) and the kernels.
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
