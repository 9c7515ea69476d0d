// The gated feed-forward block on gfx950: both projections, the activation and the product in
// one kernel, and the gradients.
//
//   G = x Wg^T,  U = x Wu^T,  h = act(G) * U
//   dU = dh * act(G),  dG = dh * U * act'(G)
//   dx = dG Wg + dU Wu,  dWg = dG^T x,  dWu = dU^T x
//
// Products are summed in 32 bits. With bf16 inputs dG and dU enter the backward's products in bf16: one rounding of a
// matrix operand, of the size of the inputs' own (products of two bf16 halves a value would double the
// backward's matrix instructions). G and U are kept for the backward in 32 bits, or in bf16 where the caller would rather
// have the memory: gradients (relative Frobenius, against 64 bits) 2.3e-3 off and a training pass of 16384 tokens, 2048 x
// 8192, in 3.36 ms, or 3.1e-3 and 3.12 ms; the results' own rounding alone is 1.7e-3.
//
// Matrix instructions bound the large sizes: 16384 tokens, 2048 x 8192, bf16: forward 932 us (1180 TFLOP/s), 1048 with G
// and U kept in bf16 and 1190 in fp32 (their 537 MB and 1074 MB of stores come in bursts at each tile's end), dx
// 839 us (1311 TFLOP/s), both weights' gradients 818 us (1344). The weights' read
// bounds few tokens: one token 14.8 us (67 MB, 4.5 TB/s), 256 tokens 24.8 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_kernels.hpp"
#include "layer_gemm.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

constexpr float kGeluC = 0.7978845608028654f, kGeluA = 0.044715f;  // sqrt(2 / pi)

__device__ __forceinline__ float sigmoid_f(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// silu(x) = x sigmoid(x); gelu(x) = x sigmoid(2 c (x + a x^3)), the tanh form written as a sigmoid
__device__ __forceinline__ float act_f(float x, int act) {
    const float s = act == 0 ? x : 2.f * kGeluC * (x + kGeluA * x * x * x);
    return x * sigmoid_f(s);
}
// the value and the derivative
__device__ __forceinline__ void act_grad_f(float x, int act, float &val, float &der) {
    const float s = act == 0 ? x : 2.f * kGeluC * (x + kGeluA * x * x * x);
    // q (1 - q) vanishes long before |x| is 1e3; x^2 stays finite for it
    const float y = __builtin_amdgcn_fmed3f(x, -1e3f, 1e3f), ds = act == 0 ? 1.f : 2.f * kGeluC * (1.f + 3.f * kGeluA * y * y);
    const float q = sigmoid_f(s);
    val = x * q;
    der = q + x * q * (1.f - q) * ds;
}

// S: the type gate and up are kept in
template <typename E, typename S>
struct GluEpi {
    E *h;
    S *gate, *up;
    int64_t M, F;
    int act;
    static constexpr bool whole = true;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[2][MI][NI], int64_t m0, int64_t n0, int, char *st) const {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            floatx4 v[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[j][r] = act_f(acc[0][i][j][r], act) * acc[1][i][j][r];
            store_rows<E, MI, NI>(st, v, h, F, m0 + 16 * i, n0, M, F);
            if (gate) {
                store_rows<S, MI, NI>(st, acc[0][i], gate, F, m0 + 16 * i, n0, M, F);
                store_rows<S, MI, NI>(st, acc[1][i], up, F, m0 + 16 * i, n0, M, F);
            }
        }
    }
};

// dG and dU, rows of ld elements, columns F .. ld-1 zero; 16 bytes of dh a thread. Bound by memory: three
// reads and two writes, for 16384 x 8192 bf16 1.34 GB in 256 us (5.2 TB/s; 388 us with 2 bytes a thread), with gate and
// up in fp32 1.88 GB in 367 us (5.1 TB/s).
// Apart from the products: each value of dG and dU is an operand of two of them.
template <typename E, typename S, typename G>
__global__ __launch_bounds__(256) void glu_grad_kernel(const S *gate, const S *up, const E *dh, G *dg, G *du, int64_t M,
                                                       int64_t F, int64_t ld, int act) {
    constexpr int V = 16 / sizeof(E);
    typedef E Piece __attribute__((ext_vector_type(V)));
    typedef S Kept __attribute__((ext_vector_type(V), aligned(16)));
    typedef G Grad __attribute__((ext_vector_type(V), aligned(16)));
    const int64_t i = block_id() * 256 + threadIdx.x, pieces = ld / V;
    if (i >= M * pieces) return;
    const int64_t m = i / pieces, n = (i - m * pieces) * V, k = m * F + n;
    Kept g, u;
    Piece d;
    // Whole pieces inside the row; ld may hold one more than F (fp32, F % 8 == 4), which is all zeros.
    if (F % V == 0 && n < F) {
        g = *reinterpret_cast<const Kept *>(gate + k);
        u = *reinterpret_cast<const Kept *>(up + k);
        d = *reinterpret_cast<const Piece *>(dh + k);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool in = n + j < F;
            g[j] = in ? gate[k + j] : (S)0.f;
            u[j] = in ? up[k + j] : (S)0.f;
            d[j] = in ? dh[k + j] : (E)0.f;
        }
    }
    Grad pg, pu;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float val, der;
        act_grad_f((float)g[j], act, val, der);
        const float dj = (float)d[j];
        pg[j] = (G)(dj * (float)u[j] * der);
        pu[j] = (G)(dj * val);
    }
    *reinterpret_cast<Grad *>(dg + i * V) = pg;
    *reinterpret_cast<Grad *>(du + i * V) = pu;
}

template <typename E, typename S>
hipError_t fwd_t(const FfnArgs &a, hipStream_t s) {
    GemmOp g = ffn_fwd_product(a.M, a.D, a.F);
    g.A[0] = a.x;
    g.B[0] = a.wg, g.B[1] = a.wu;
    return launch_gemm<E, true, true, 2>(g, GluEpi<E, S>{(E *)a.h, (S *)a.gate, (S *)a.up, a.M, a.F, a.act}, s);
}

// the products of the backward: dx, and both weights' gradients side by side
GemmOp dx_op(const FfnArgs &a, const void *dg, const void *du) {
    GemmOp g = ffn_dx_product(a.M, a.D, a.F);
    g.A[0] = dg, g.A[1] = du;
    g.B[0] = a.wg, g.B[1] = a.wu;
    return g;
}
GemmOp dw_op(const FfnArgs &a, const void *dg, const void *du) {
    GemmOp g = ffn_dw_product(a.M, a.D, a.F);
    g.A[0] = dg, g.A[1] = du;
    g.B[0] = g.B[1] = a.x;
    return g;
}
// workspace: dG and dU, then the partial products of one product at a time
template <typename E>
int64_t bwd_bytes(const FfnArgs &a) {
    const int64_t x = store_ws_bytes<E>(dx_op(a, nullptr, nullptr)), w = store_ws_bytes<E>(dw_op(a, nullptr, nullptr));
    const int64_t es = whole_pieces(a.D, sizeof(E)) ? sizeof(E) : 4;
    return 2 * a.M * grad_ld(a.F) * es + (x > w ? x : w);
}

// G: the type of dG and dU. Where rows of D elements are not whole 16-byte pieces both products run on fp32 matrix
// instructions, and dG and dU are left in 32 bits.
template <typename E, typename S, typename G>
hipError_t bwd_t(const FfnArgs &a, hipStream_t s) {
    const int64_t ld = grad_ld(a.F);
    G *dg = (G *)a.ws, *du = dg + a.M * ld;
    const StoreEpi<E> to_x{{(E *)a.dx, nullptr}, nullptr, nullptr, nullptr, nullptr, a.M, a.D, a.D},
        to_w{{(E *)a.dwg, (E *)a.dwu}, nullptr, nullptr, nullptr, nullptr, a.F, a.D, a.D};
    void *part = du + a.M * ld;
    if (a.M > 0) {
        const int64_t blocks = (a.M * ld / (16 / (int64_t)sizeof(E)) + 255) / 256;
        hipLaunchKernelGGL((glu_grad_kernel<E, S, G>), grid_of(blocks, 256), dim3(256), 0, s, (const S *)a.gate,
                           (const S *)a.up, (const E *)a.dh, dg, du, a.M, a.F, ld, a.act);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if constexpr (sizeof(G) > sizeof(E)) e = launch_gemm_any_op<G, E, true, false, 1>(dx_op(a, dg, du), to_x, s);
        else e = launch_gemm_store<E, true, false>(dx_op(a, dg, du), to_x, part, s);
        if (e != hipSuccess) return e;
    }
    if constexpr (sizeof(G) > sizeof(E)) return launch_gemm_any_op<G, E, false, false, 1>(dw_op(a, dg, du), to_w, s);
    else return launch_gemm_store<E, false, false>(dw_op(a, dg, du), to_w, part, s);
}
template <typename S>
hipError_t bwd_bf16(const FfnArgs &a, hipStream_t s) {
    return whole_pieces(a.D, 2) ? bwd_t<__bf16, S, __bf16>(a, s) : bwd_t<__bf16, S, float>(a, s);
}

}  // namespace

int64_t ffn_bwd_ws_bytes(int64_t M, int64_t D, int64_t F, int dtype) {
    FfnArgs a{};
    a.M = M;
    a.D = D;
    a.F = F;
    return dtype == kDtypeBf16 ? bwd_bytes<__bf16>(a) : bwd_bytes<float>(a);
}

hipError_t launch_ffn_fwd(const FfnArgs &a, int dtype, hipStream_t s) {
    if (dtype != kDtypeBf16) return fwd_t<float, float>(a, s);
    return a.wide ? fwd_t<__bf16, float>(a, s) : fwd_t<__bf16, __bf16>(a, s);
}
hipError_t launch_ffn_bwd(const FfnArgs &a, int dtype, hipStream_t s) {
    if (dtype != kDtypeBf16) return bwd_t<float, float, float>(a, s);
    return a.wide ? bwd_bf16<float>(a, s) : bwd_bf16<__bf16>(a, s);
}

}  // namespace gdr
