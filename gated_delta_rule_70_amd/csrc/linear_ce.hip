// Softmax cross entropy of a linear layer over a large vocabulary on gfx950, in pieces of the
// vocabulary, the logits never kept.
//
//   l = x W^T,  lse_n = log sum_v e^{l_nv},  loss_n = lse_n - l_{n, t_n}
//   dl_nv = (e^{l_nv - lse_n} - [v = t_n]) dloss_n,  dx = dl W,  dW = dl^T x
//
// A token whose target is outside 0 .. V-1 bears no loss and no gradient.
//
// Forward: each wave reduces its tile of logits to one (max, sum of e^{l - max}) per token, in 32
// bits, and the lane that holds the target's logit writes it out; a second kernel joins the
// partial sums of a token. Backward: for each piece of the vocabulary the logits are formed again
// and turned into dl (in the inputs' type, as the operand of two products), then
// dW's rows of the piece are complete and dx is summed over the pieces in 32 bits.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gdr_kernels.hpp"
#include "layer_gemm.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

// vocabulary columns per partial sum
template <typename E>
int64_t strip_of(int64_t D) {
    return whole_pieces<E>(D) ? kTileCols : kAnyCols;
}

struct StatEpi {
    const int64_t *t;
    float2 *part;  // [strips][M]
    float *tgt;    // [M]
    int64_t M, V;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0) const {
        constexpr int SJ = NI < kTileCols / 16 ? NI : kTileCols / 16;  // tiles per strip
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c;
            const int64_t tm = m < M ? t[m] : -1;
#pragma unroll
            for (int s = 0; s < NI / SJ; ++s) {
                const int64_t ns = n0 + 16 * SJ * s;
                if (ns >= V) continue;
                const int left = V - ns < 16 * SJ ? (int)(V - ns) : 16 * SJ;        // columns in range
                const int want = tm >= ns && tm < ns + left ? (int)(tm - ns) : -1;  // the target's column
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int n = 16 * j + 4 * g + r;
                        if (n < left) top = fmaxf(top, acc[0][i][SJ * s + j][r]);
                        if (n == want) tgt[m] = acc[0][i][SJ * s + j][r];
                    }
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * j + 4 * g + r < left) sum += __expf(acc[0][i][SJ * s + j][r] - ref);
                sum += __shfl_xor(sum, 16, 64);
                sum += __shfl_xor(sum, 32, 64);
                if (g == 0 && m < M) part[(ns / (16 * SJ)) * M + m] = make_float2(top, sum);
            }
        }
    }
};

// dl of one piece: rows of ld elements, the piece's columns past the vocabulary's end zero
template <typename E>
struct GradEpi {
    const int64_t *t;
    const float *lse, *dloss;
    E *dl;
    int64_t M, V, v0, width, ld;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0) const {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c;
            if (m >= M) continue;
            const int64_t tm = t[m];
            const bool on = tm >= 0 && tm < V;
            const float ls = lse[m], sc = on ? dloss[m] : 0.f;
            // the target's column and the piece's end, from this wave's first column
            const int want = tm - v0 >= n0 && tm - v0 < n0 + 16 * NI ? (int)(tm - v0 - n0) : -1;
            const int left = !on ? 0 : width - n0 < 16 * NI ? (int)(width - n0) : 16 * NI;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int k = 16 * j + 4 * g;
                const int64_t n = n0 + k;
                if (n >= ld) continue;
                floatx4 v;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = __expf(acc[0][i][j][r] - ls) - (k + r == want ? 1.f : 0.f);
                    v[r] = k + r < left ? p * sc : 0.f;
                }
                store4(dl + m * ld + n, v, ld - n, true);
            }
        }
    }
};

// one thread per token joins its partial sums in order
__global__ __launch_bounds__(64) void ce_join_kernel(const float2 *part, const float *tgt, const int64_t *t, float *loss,
                                                     float *lse, int64_t N, int64_t V, int64_t strips) {
    const int64_t n = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (n >= N) return;
    float top = -INFINITY, sum = 0.f;
    for (int64_t s = 0; s < strips; ++s) {
        const float2 p = part[s * N + n];
        const float m = fmaxf(top, p.x), ref = m == -INFINITY ? 0.f : m;
        sum = sum * expf(top - ref) + p.y * expf(p.x - ref);
        top = m;
    }
    const float l = top + logf(sum);
    lse[n] = l;
    loss[n] = t[n] >= 0 && t[n] < V ? l - tgt[n] : 0.f;
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }
template <typename E>
int64_t strips_of(int64_t D, int64_t V) {
    return (V + strip_of<E>(D) - 1) / strip_of<E>(D);
}

// Vocabulary columns per piece of the backward: dl of a piece takes at most about 512 MB.
int64_t piece_of(int64_t N, int64_t V) {
    int64_t p = (INT64_C(1) << 28) / (N > 0 ? N : 1) / 256 * 256;
    if (p < 2048) p = 2048;
    const int64_t all = (V + 7) / 8 * 8;
    return p < all ? p : all;
}

template <typename E>
hipError_t fwd_t(const CeArgs &a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    const int64_t strips = strips_of<E>(a.D, a.V);
    float *tgt = (float *)a.ws;
    float2 *part = (float2 *)((char *)a.ws + up256(a.N * 4));
    const GemmOp g{{a.x, nullptr}, {a.w, nullptr}, a.D, a.D, a.N, a.V, a.D, 1};
    const hipError_t e = launch_gemm<E, true, true, 1>(g, StatEpi{a.t, part, tgt, a.N, a.V}, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ce_join_kernel, dim3((unsigned)((a.N + 63) / 64)), dim3(64), 0, s, part, tgt, a.t, a.loss, a.lse,
                       a.N, a.V, strips);
    return hipGetLastError();
}

template <typename E>
hipError_t bwd_t(const CeArgs &a, hipStream_t s) {
    const int64_t piece = piece_of(a.N, a.V);
    E *dl = (E *)a.ws;
    float *acc = (float *)((char *)a.ws + up256(a.N * piece * (int64_t)sizeof(E)));
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t width = a.V - v0 < piece ? a.V - v0 : piece;
        const E *w = (const E *)a.w + v0 * a.D;
        const GemmOp gl{{a.x, nullptr}, {w, nullptr}, a.D, a.D, a.N, width, a.D, 1};
        hipError_t e = launch_gemm<E, true, true, 1>(
            gl, GradEpi<E>{a.t, a.lse_in, a.dloss, dl, a.N, a.V, v0, width, piece}, s);
        if (e != hipSuccess) return e;
        const GemmOp gw{{dl, nullptr}, {a.x, nullptr}, piece, a.D, width, a.D, a.N, 1};
        e = launch_gemm<E, false, false, 1>(gw, StoreEpi<E>{(E *)a.dw + v0 * a.D, nullptr, nullptr, width, a.D, a.D}, s);
        if (e != hipSuccess) return e;
        const bool last = v0 + piece >= a.V;
        const GemmOp gx{{dl, nullptr}, {w, nullptr}, piece, a.D, a.N, a.D, width, 1};
        e = launch_gemm<E, true, false, 1>(
            gx, StoreEpi<E>{last ? (E *)a.dx : nullptr, v0 ? acc : nullptr, acc, a.N, a.D, a.D}, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t ce_fwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype) {
    const int64_t strips = dtype == kDtypeBf16 ? strips_of<__bf16>(D, V) : strips_of<float>(D, V);
    return up256(N * 4) + strips * N * 8;
}
int64_t ce_bwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype) {
    const int64_t piece = piece_of(N, V);
    return up256(N * piece * (dtype == kDtypeBf16 ? 2 : 4)) + (piece < V ? N * D * 4 : 0);
}

hipError_t launch_ce_fwd(const CeArgs &a, int dtype, hipStream_t s) {
    return dtype == kDtypeBf16 ? fwd_t<__bf16>(a, s) : fwd_t<float>(a, s);
}
hipError_t launch_ce_bwd(const CeArgs &a, int dtype, hipStream_t s) {
    return dtype == kDtypeBf16 ? bwd_t<__bf16>(a, s) : bwd_t<float>(a, s);
}

}  // namespace gdr
