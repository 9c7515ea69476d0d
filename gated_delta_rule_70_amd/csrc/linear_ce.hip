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
// and turned into dl (in the inputs' type, as the operand of two products, its common factor apart), then
// dW's rows of the piece are complete and dx is summed over the pieces in 32 bits.
//
// Matrix instructions bound it where there are many tokens: 16384 tokens, 2048 x 65536, bf16: forward
// 3.46 ms (1270 TFLOP/s), backward 4 x (1.07 ms for dl, of which 0.1 its 537 MB of stores; 0.89 for dx;
// 0.82 for dW: 1026, 1241 and 1340 TFLOP/s). Keeping the logits instead of forming them again would take 2.1 GB
// in bf16 and round them. With few tokens the read of W does: 16 tokens 74 us (268 MB, 3.6 TB/s with the
// join's 7 us).
#include <hip/hip_runtime.h>
#include <math.h>
#include <initializer_list>
#include <type_traits>
#include <stdint.h>

#include "gdr_kernels.hpp"
#include "layer_gemm.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

// The difference is taken before the change of base: at a logit equal to its reference the
// exponential is 1 exactly.
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// The forward's epilogue: per token and strip of kTileCols columns (max, sum of e^{l - max}).
struct StatEpi {
    const int64_t *t;
    float2 *part;  // [strips][M]
    float *tgt;    // [M]
    int64_t M, V;
    static constexpr bool whole = false;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0, int, char *st) const {
        constexpr int SJ = NI < kTileCols / 16 ? NI : kTileCols / 16, S = NI / SJ;  // tiles per strip, strips
        const int lane = epilogue_lane(), g = lane >> 4, c = lane & 15;
        const int left = V - n0 < 16 * NI ? (int)(V - n0) : 16 * NI;  // columns in range
        int want[MI];                                                 // the target's column among the wave's
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c, n = (m < M ? t[m] : -1) - n0;
            want[i] = n >= 0 && n < left ? (int)n : -1;
        }
        // The sums of every row first, without a branch (the accumulators stay where they are), then
        // what a lane has to write.
        float2 sums[MI][S];
        float found[MI];
        const int last = left - 4 * g;  // in-range columns of this lane: 16 j + r below it
        auto reduce = [&](auto ragged) GDR_INLINE {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            found[i] = 0.f;
            const int at = want[i] - 4 * g;  // the target's 16 j + r, if this lane holds it
#pragma unroll
            for (int s = 0; s < S; ++s) {
                floatx4 v[SJ];
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int n = 16 * (SJ * s + j) + r;
                        const float l = acc[0][i][SJ * s + j][r];
                        found[i] = n == at ? l : found[i];
                        v[j][r] = !ragged.value || n < last ? l : -INFINITY;
                        top = fmaxf(top, v[j][r]);
                    }
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
                for (int j = 0; j < SJ; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum += exp_f(v[j][r] - ref);
                sum += __shfl_xor(sum, 16, 64);
                sum += __shfl_xor(sum, 32, 64);
                sums[i][s] = make_float2(top, sum);
                __builtin_amdgcn_sched_barrier(0);  // one strip's values in registers at a time
            }
        }
        };
        if (left == 16 * NI) reduce(std::false_type{});
        else reduce(std::true_type{});
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c;
            // lane (g, c) holds columns 16 j + 4 g ..: the target's is among them where want / 4 % 4 == g
            if (want[i] >= 0 && ((want[i] >> 2) & 3) == g) tgt[m] = found[i];
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (g == s % 4 && m < M && 16 * SJ * s < left) part[(n0 / (16 * SJ) + s) * M + m] = sums[i][s];
        }
    }
};

// dl of one piece: rows of ld elements, the piece's columns past the vocabulary's end zero
template <typename E>
struct GradEpi {
    const int64_t *t;
    const float *lse, *dloss;
    const float *inv;  // 1 / the factor taken out of dl
    E *dl;
    int64_t M, V, v0, width, ld;
    static constexpr bool whole = true;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0, int, char *st) const {
        const int lane = epilogue_lane(), g = lane >> 4, c = lane & 15;
        float ls[MI], sc[MI];
        const float inv_scale = *inv;
        int want[MI], left[MI];  // the target's column and the piece's end, from this wave's first column
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c;
            const int64_t tm = m < M ? t[m] : -1, tv = tm - v0 - n0;
            const bool on = tm >= 0 && tm < V;
            ls[i] = on ? lse[m] : 0.f;
            sc[i] = on ? dloss[m] * inv_scale : 0.f;
            want[i] = tv >= 0 && tv < 16 * NI ? (int)tv : -1;
            left[i] = !on ? 0 : width - n0 < 16 * NI ? (int)(width - n0) : 16 * NI;
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            floatx4 v[NI];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[j][r] = exp_f(acc[0][i][j][r] - ls[i]) * sc[i];
            if (__any(want[i] >= 0)) {
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * j + 4 * g + r == want[i])
                            v[j][r] = (exp_f(acc[0][i][j][r] - ls[i]) - 1.f) * sc[i];
            }
            if (__any(left[i] < 16 * NI)) {
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (16 * j + 4 * g + r >= left[i]) v[j][r] = 0.f;
            }
            store_rows<E, MI, NI>(st, v, dl, ld, m0 + 16 * i, n0, M, ld);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};

// What the backward's products need of the tokens, in one launch.
// Workgroup 0: the largest |dloss| of a token that bears a loss, and its inverse (1 and 1 where there is none). It is
// taken out of dl before dl is rounded to the inputs' type and multiplied back into dx and dW, in 32 bits: with a
// mean over tokens every dloss is the same number, whose rounding would be a common error of all of dl (2.9e-3 of dW
// in bf16 against 64 bits; without it the large entries, p - 1 at the targets, are near -1 and lose little).
// The others: a copy of x for dW = dl^T x, with zeros in the rows of the tokens without a loss. Their dl is 0, but
// 0 times what a padded row may hold, NaN or infinity, would be in all of dW. 29 us for 16384 x 2048 bf16 (134 MB,
// 4.7 TB/s), next to 11 ms; 5.4 us for 1021 x 1024.
template <typename E>
__global__ __launch_bounds__(1024) void ce_tokens_kernel(const float *dloss, const int64_t *t, const E *x, int64_t N, int64_t D,
                                                         int64_t V, float *scale, E *kept) {
    __shared__ float held[16];
    const int64_t id = block_id();
    if (id > 0) {
        constexpr int W = 16 / sizeof(E);
        typedef E Piece __attribute__((ext_vector_type(W)));
        const int64_t first = ((id - 1) * 4096 + threadIdx.x) * W;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t i = first + k * 1024 * W;
            if (D % W == 0) {
                if (i >= N * D) return;
                const int64_t v = t[i / D];
                Piece p = *reinterpret_cast<const Piece *>(x + i);
                if (v < 0 || v >= V) p = Piece{};
                *reinterpret_cast<Piece *>(kept + i) = p;
            } else {
                for (int64_t j = i; j < i + W && j < N * D; ++j) {
                    const int64_t v = t[j / D];
                    kept[j] = v < 0 || v >= V ? (E)0.f : x[j];
                }
            }
        }
        return;
    }
    float top = 0.f;
#pragma unroll 4
    for (int64_t n = threadIdx.x; n < N; n += 1024)
        if (t[n] >= 0 && t[n] < V) top = fmaxf(top, fabsf(dloss[n]));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if ((threadIdx.x & 63) == 0) held[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, held[i]);
    // a factor whose inverse is a normal number
    const bool fit = top > 1e-37f && top < 1e37f;
    scale[0] = fit ? top : 1.f;
    scale[1] = fit ? 1.f / top : 1.f;
}

// Joins the partial sums of 16 tokens: 64 threads a token each take every 64th strip in order, then
// the 64 are joined in pairs. 30 us for 16384 tokens x 1024 strips (134 MB, 4.5 TB/s), 7 us for 16 tokens.
__global__ __launch_bounds__(1024) void ce_join_kernel(const float2 *part, const float *tgt, const int64_t *t, float *loss,
                                                       float *lse, int64_t N, int64_t V, int64_t strips) {
    __shared__ float2 held[64][16];
    const int c = threadIdx.x & 15, slot = threadIdx.x >> 4;
    const int64_t n = block_id() * 16 + c;
    auto join = [](float2 p, float2 q) {
        const float m = fmaxf(p.x, q.x), ref = m == -INFINITY ? 0.f : m;
        return make_float2(m, p.y * expf(p.x - ref) + q.y * expf(q.x - ref));
    };
    float2 mine = make_float2(-INFINITY, 0.f);
    if (n < N) {
#pragma unroll 4
        for (int64_t s = slot; s < strips; s += 64) mine = join(mine, part[s * N + n]);
    }
    held[slot][c] = mine;
    for (int k = 32; k > 0; k >>= 1) {
        __syncthreads();
        if (slot < k) held[slot][c] = mine = join(mine, held[slot + k][c]);
    }
    if (slot == 0 && n < N) {
        const float l = mine.x + logf(mine.y);
        lse[n] = l;
        loss[n] = t[n] >= 0 && t[n] < V ? l - tgt[n] : 0.f;
    }
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }
// partial sums of a token
template <typename E>
int64_t strips_of(int64_t N, int64_t D, int64_t V) {
    const int64_t cols = wave_cols(N, V, D, sizeof(E));
    return (V + cols - 1) / cols;
}

template <typename E>
hipError_t fwd_t(const CeArgs &a, hipStream_t s) {
    if (a.N == 0) return hipSuccess;
    const int64_t strips = strips_of<E>(a.N, a.D, a.V);
    float *tgt = (float *)a.ws;
    float2 *part = (float2 *)((char *)a.ws + up256(a.N * 4));
    GemmOp g = ce_logits_product(a.N, a.D, a.V);
    g.A[0] = a.x;
    g.B[0] = a.w;
    const hipError_t e = launch_gemm<E, true, true, 1>(g, StatEpi{a.t, part, tgt, a.N, a.V}, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ce_join_kernel, grid_of((a.N + 15) / 16, 1024), dim3(1024), 0, s, part, tgt, a.t, a.loss, a.lse,
                       a.N, a.V, strips);
    return hipGetLastError();
}

// the products of one piece of the backward (`width` columns from w)
template <typename E>
GemmOp dw_op(const CeArgs &a, const E *dl, const E *x, int64_t piece, int64_t width) {
    GemmOp g = ce_dw_product(a.N, a.D, piece, width);
    g.A[0] = dl;
    g.B[0] = x;
    return g;
}
template <typename E>
GemmOp dx_op(const CeArgs &a, const E *dl, const E *w, int64_t piece, int64_t width) {
    GemmOp g = ce_dx_product(a.N, a.D, piece, width);
    g.A[0] = dl;
    g.B[0] = w;
    return g;
}
// workspace: the two factors, x without the rows of tokens without a loss, dl of a piece, dx in 32 bits where
// there are several, the partial products of one product at a time
struct BwdLayout {
    int64_t x, dl, acc, part, total;
};
template <typename E>
BwdLayout bwd_layout(const CeArgs &a) {
    const int64_t piece = ce_piece(a.N, a.V), tail = a.V % piece ? a.V % piece : piece;
    const E *none = nullptr;
    int64_t part = 0;
    for (int64_t width : {piece < a.V ? piece : a.V, tail}) {
        const int64_t w = store_ws_bytes<E>(dw_op(a, none, none, piece, width)), x = store_ws_bytes<E>(dx_op(a, none, none, piece, width));
        part = part > w ? part : w;
        part = part > x ? part : x;
    }
    BwdLayout l;
    l.x = 256;
    l.dl = l.x + up256(a.N * a.D * (int64_t)sizeof(E));
    l.acc = l.dl + up256(a.N * piece * (int64_t)sizeof(E));
    l.part = l.acc + (piece < a.V ? up256(a.N * a.D * 4) : 0);
    l.total = l.part + part;
    return l;
}

template <typename E>
hipError_t bwd_t(const CeArgs &a, hipStream_t s) {
    const int64_t piece = ce_piece(a.N, a.V);
    const BwdLayout l = bwd_layout<E>(a);
    float *scale = (float *)a.ws;
    E *x = (E *)((char *)a.ws + l.x), *dl = (E *)((char *)a.ws + l.dl);
    float *acc = (float *)((char *)a.ws + l.acc);
    void *part = (char *)a.ws + l.part;
    const int64_t copied = 4096 * (16 / (int64_t)sizeof(E));  // elements of x a workgroup
    hipLaunchKernelGGL((ce_tokens_kernel<E>), grid_of(1 + (a.N * a.D + copied - 1) / copied, 1024), dim3(1024), 0, s, a.dloss, a.t,
                       (const E *)a.x, a.N, a.D, a.V, scale, x);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
        const int64_t width = a.V - v0 < piece ? a.V - v0 : piece;
        const E *w = (const E *)a.w + v0 * a.D;
        GemmOp gl = ce_logits_product(a.N, a.D, width);
        gl.A[0] = a.x;
        gl.B[0] = w;
        e = launch_gemm<E, true, true, 1>(
            gl, GradEpi<E>{a.t, a.lse_in, a.dloss, scale + 1, dl, a.N, a.V, v0, width, piece}, s);
        if (e != hipSuccess) return e;
        e = launch_gemm_store<E, false, false>(
            dw_op(a, dl, x, piece, width),
            StoreEpi<E>{{(E *)a.dw + v0 * a.D, nullptr}, nullptr, nullptr, nullptr, scale, width, a.D, a.D}, part, s);
        if (e != hipSuccess) return e;
        const bool last = v0 + piece >= a.V;
        e = launch_gemm_store<E, true, false>(
            dx_op(a, dl, w, piece, width),
            StoreEpi<E>{{last ? (E *)a.dx : nullptr, nullptr}, v0 ? acc : nullptr, acc, nullptr, scale, a.N, a.D, a.D}, part, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t ce_fwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype) {
    const int64_t strips = dtype == kDtypeBf16 ? strips_of<__bf16>(N, D, V) : strips_of<float>(N, D, V);
    return up256(N * 4) + strips * N * 8;
}
int64_t ce_bwd_ws_bytes(int64_t N, int64_t D, int64_t V, int dtype) {
    CeArgs a{};
    a.N = N;
    a.D = D;
    a.V = V;
    return dtype == kDtypeBf16 ? bwd_layout<__bf16>(a).total : bwd_layout<float>(a).total;
}

hipError_t launch_ce_fwd(const CeArgs &a, int dtype, hipStream_t s) {
    return dtype == kDtypeBf16 ? fwd_t<__bf16>(a, s) : fwd_t<float>(a, s);
}
hipError_t launch_ce_bwd(const CeArgs &a, int dtype, hipStream_t s) {
    return dtype == kDtypeBf16 ? bwd_t<__bf16>(a, s) : bwd_t<float>(a, s);
}

}  // namespace gdr
