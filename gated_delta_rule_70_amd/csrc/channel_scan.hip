// Channel scan on gfx950: the gated linear recurrence of one number per channel,
//
//   u = a_t + dt_bias,  la = -e^{A_log} softplus(u),  alpha = e^{la},  beta = sigmoid(b_t)
//   h_t = alpha h_{t-1} + beta x_t,  out_t = h_t
//
// and its adjoint, given dout and the final state's gradient:
//
//   g_t = dout_t + alpha_{t+1} g_{t+1}            (g past the last token: the final state's gradient)
//   dx = beta g,  db = beta (1 - beta) x g,  dla = alpha h_{t-1} g,  da = -e^{A_log} sigmoid(u) dla
//   dA_log = sum dla la,  ddt_bias = sum da,  dh0 = alpha_1 g_1
//
// One thread per (sequence, channel) walks the tokens; neighbouring threads hold neighbouring
// channels.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_kernels.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

// The gates of one element. softplus(u) = max(u, 0) + log1p(z), z = e^{-|u|}; below 2^-5 the
// logarithm is taken by its series (next term z^5/5 < 2^-27 z), where log(1 + z) would lose z's
// low bits: the decay's logarithm enters the gradient of A_log by itself.
struct Gates {
    float alpha, beta, la, rs;  // rs = e^{A_log} sigmoid(u)
};
__device__ __forceinline__ Gates gates_of(float a, float b, float bias, float rate) {
    const float u = a + bias;
    const float z = __expf(-fabsf(u));
    const float series = z * (1.f - z * (0.5f - z * (0.33333333f - z * 0.25f)));
    const float l1p = z < 0.03125f ? series : __logf(1.f + z);
    const float inv = __builtin_amdgcn_rcpf(1.f + z);
    Gates g;
    // finite, so that la times a vanished alpha is 0
    g.la = fmaxf(-rate * (fmaxf(u, 0.f) + l1p), -1e30f);
    g.alpha = __expf(g.la);
    g.beta = __builtin_amdgcn_rcpf(1.f + __expf(-b));
    g.rs = rate * (u >= 0.f ? inv : z * inv);
    return g;
}

struct Span {
    int64_t row0, len, slot0;
    int step;  // +1, or -1 for a reversed scan (row0 is then the last row)
};
__device__ __forceinline__ Span span_of(const ScanArgs &a, int64_t s) {
    Span p;
    if (a.cu_seqlens) {
        const int64_t c0 = a.cu_seqlens[s];
        p.row0 = c0;
        p.len = a.cu_seqlens[s + 1] - c0;
        p.slot0 = c0 / kScanBlock + s;
    } else {
        p.row0 = s * a.T;
        p.len = a.T;
        p.slot0 = s * ((a.T + kScanBlock - 1) / kScanBlock);
    }
    p.step = 1;
    if (a.flags & kFlagReverse) {
        p.row0 += p.len - 1;
        p.step = -1;
    }
    return p;
}

template <typename E>
__global__ __launch_bounds__(64) void scan_fwd_kernel(ScanArgs a, int64_t ntile) {
    const int64_t s = blockIdx.x / ntile, d = (blockIdx.x % ntile) * 64 + threadIdx.x;
    if (d >= a.D) return;
    const Span p = span_of(a, s);
    const E *x = (const E *)a.x, *ra = (const E *)a.a, *rb = (const E *)a.b;
    E *out = (E *)a.out;
    const float rate = expf(a.A_log[d]), bias = a.dt_bias[d];
    float h = a.h0 ? a.h0[s * a.D + d] : 0.f;
    for (int64_t t = 0; t < p.len; ++t) {
        if (a.states && t % kScanBlock == 0) a.states[(p.slot0 + t / kScanBlock) * a.D + d] = h;
        const int64_t i = (p.row0 + p.step * t) * a.D + d;
        const Gates g = gates_of((float)ra[i], (float)rb[i], bias, rate);
        h = g.alpha * h + g.beta * (float)x[i];
        out[i] = (E)h;
    }
    if (a.hT) a.hT[s * a.D + d] = h;
}

template <typename E>
__global__ __launch_bounds__(64) void scan_bwd_kernel(ScanArgs a, int64_t ntile) {
    __shared__ float hbuf[kScanBlock][64];
    const int64_t s = blockIdx.x / ntile, d = (blockIdx.x % ntile) * 64 + threadIdx.x;
    if (d >= a.D) return;
    const Span p = span_of(a, s);
    const E *x = (const E *)a.x, *ra = (const E *)a.a, *rb = (const E *)a.b, *dout = (const E *)a.dout;
    E *dx = (E *)a.dx, *da = (E *)a.da, *db = (E *)a.db;
    const float rate = expf(a.A_log[d]), bias = a.dt_bias[d];
    float g = a.dhT ? a.dhT[s * a.D + d] : 0.f, sA = 0.f, sb = 0.f;
    const int64_t nb = (p.len + kScanBlock - 1) / kScanBlock;
    for (int64_t k = nb - 1; k >= 0; --k) {
        const int n = (int)(p.len - k * kScanBlock < kScanBlock ? p.len - k * kScanBlock : kScanBlock);
        float h = a.states[(p.slot0 + k) * a.D + d];
        for (int t = 0; t < n; ++t) {
            const int64_t i = (p.row0 + p.step * (k * kScanBlock + t)) * a.D + d;
            const Gates q = gates_of((float)ra[i], (float)rb[i], bias, rate);
            hbuf[t][threadIdx.x] = h;
            h = q.alpha * h + q.beta * (float)x[i];
        }
        for (int t = n - 1; t >= 0; --t) {
            const int64_t i = (p.row0 + p.step * (k * kScanBlock + t)) * a.D + d;
            const Gates q = gates_of((float)ra[i], (float)rb[i], bias, rate);
            g += (float)dout[i];
            const float dla = q.alpha * hbuf[t][threadIdx.x] * g, dai = -q.rs * dla;
            dx[i] = (E)(q.beta * g);
            db[i] = (E)(q.beta * (1.f - q.beta) * (float)x[i] * g);
            da[i] = (E)dai;
            sA += dla * q.la;
            sb += dai;
            g *= q.alpha;
        }
    }
    if (a.dh0) a.dh0[s * a.D + d] = g;
    a.ws[(2 * s) * a.D + d] = sA;
    a.ws[(2 * s + 1) * a.D + d] = sb;
}

// dA_log and ddt_bias: the partial sums [n][2][D] added in order
__global__ __launch_bounds__(64) void scan_param_kernel(const float *ws, int64_t n, int64_t D, float *dA, float *db) {
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (d >= D) return;
    float sA = 0.f, sb = 0.f;
    for (int64_t i = 0; i < n; ++i) {
        sA += ws[2 * i * D + d];
        sb += ws[(2 * i + 1) * D + d];
    }
    dA[d] = sA;
    db[d] = sb;
}

template <typename E>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.nseq * a.D) return;
    const int64_t d = i % a.D;
    const Gates g = gates_of((float)((const E *)a.a)[i], (float)((const E *)a.b)[i], a.dt_bias[d], expf(a.A_log[d]));
    const float h = g.alpha * a.h0[i] + g.beta * (float)((const E *)a.x)[i];
    a.hT[i] = h;
    ((E *)a.out)[i] = (E)h;
}

}  // namespace

int64_t scan_fwd_ws_bytes(int64_t, int64_t, int64_t) { return 0; }
int64_t scan_bwd_ws_bytes(int64_t D, int64_t nseq, int64_t) { return nseq * D * 8; }

hipError_t launch_scan_fwd(const ScanArgs &a, int dtype, hipStream_t s) {
    const int64_t ntile = (a.D + 63) / 64;
    if (a.nseq == 0) return hipSuccess;
    const dim3 grid((unsigned)(ntile * a.nseq)), block(64);
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((scan_fwd_kernel<__bf16>), grid, block, 0, s, a, ntile);
    else hipLaunchKernelGGL((scan_fwd_kernel<float>), grid, block, 0, s, a, ntile);
    return hipGetLastError();
}

hipError_t launch_scan_bwd(const ScanArgs &a, int dtype, hipStream_t s) {
    const int64_t ntile = (a.D + 63) / 64;
    if (a.nseq > 0) {
        const dim3 grid((unsigned)(ntile * a.nseq)), block(64);
        if (dtype == kDtypeBf16) hipLaunchKernelGGL((scan_bwd_kernel<__bf16>), grid, block, 0, s, a, ntile);
        else hipLaunchKernelGGL((scan_bwd_kernel<float>), grid, block, 0, s, a, ntile);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(scan_param_kernel, dim3((unsigned)ntile), dim3(64), 0, s, a.ws, a.nseq, a.D, a.dA_log, a.ddt_bias);
    return hipGetLastError();
}

hipError_t launch_scan_step(const ScanArgs &a, int dtype, hipStream_t s) {
    const int64_t n = a.nseq * a.D;
    if (n == 0) return hipSuccess;
    const dim3 grid((unsigned)((n + 255) / 256)), block(256);
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((scan_step_kernel<__bf16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((scan_step_kernel<float>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace gdr
