// Matrix products of the layer operators (gated feed-forward, linear cross entropy) on gfx950.
//
//   C[m][n] = sum over pairs p, sum over k of A_p(m, k) B_p(n, k)
//
// Every kernel hands its result to an epilogue as 16x16 accumulator tiles of one wave, held
// transposed (B's rows are the matrix instruction's rows): lane l = 16 g + c holds, of tile
// (i, j), row m = m0 + 16 i + c and columns n = n0 + 16 j + 4 g + r, r = 0..3, so that a lane's
// four values are neighbours in a row of C. With NB = 2 one A meets two B matrices of the same
// shape and the epilogue gets both products' tiles at the same (m, n).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_mfma.hpp"

namespace gdr {

// Operand strides in elements; one of the two of each operand is 1.
struct AnyGemmArgs {
    const void *A[2], *B[2];
    int64_t am, ak, bn, bk;
    int64_t M, N, K;
    int pairs;  // products summed over; with NB = 2 the two B matrices of one A, and pairs is 1
};

// Any sizes, strides and alignments: 64 x 64 tiles staged in LDS as fp32, fp32 matrix
// instructions, every load checked. Four waves of 32 x 32. The sum over k is taken in blocks of
// kSumK terms that are added up afterwards: one running fp32 sum over the 60,000 tokens of a weight
// gradient was 2.1e-5 off (relative Frobenius), in blocks the error stops growing with the length.
constexpr int kAnyK = 16, kAnyLd = kAnyK + 1, kSumK = 512;
template <typename E, int NB, class Epi>
__global__ __launch_bounds__(256) void gemm_any_kernel(AnyGemmArgs a, Epi epi) {
    __shared__ float As[64 * kAnyLd], Bs[NB][64 * kAnyLd];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
    const int64_t nm = (a.M + 63) / 64;
    const int64_t m0 = (blockIdx.x % nm) * 64, n0 = (blockIdx.x / nm) * 64;
    const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
    floatx4 acc[NB][2][2], total[NB][2][2];
    auto each = [&](auto f) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) f(acc[b][i][j], total[b][i][j]);
    };
    each([](floatx4 &p, floatx4 &t) { p = t = zero4(); });

    auto stage = [&](float *dst, const E *src, int64_t r0, int64_t rows, int64_t k0, int64_t sr, int64_t sk) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = sk == 1 ? tid / 16 + 16 * j : tid % 64, k = sk == 1 ? tid % 16 : tid / 64 + 4 * j;
            float v = 0.f;
            if (r0 + row < rows && k0 + k < a.K) v = (float)src[(r0 + row) * sr + (k0 + k) * sk];
            dst[row * kAnyLd + k] = v;
        }
    };
    for (int p = 0; p < a.pairs; ++p)
        for (int64_t k0 = 0; k0 < a.K; k0 += kAnyK) {
            stage(As, (const E *)a.A[p], m0, a.M, k0, a.am, a.ak);
#pragma unroll
            for (int b = 0; b < NB; ++b) stage(Bs[b], (const E *)a.B[NB == 2 ? b : p], n0, a.N, k0, a.bn, a.bk);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kAnyK; k += 4)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[b][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(Bs[b][(wn + 16 * j + c) * kAnyLd + k + g],
                                                                               As[(wm + 16 * i + c) * kAnyLd + k + g],
                                                                               acc[b][i][j], 0, 0, 0);
            __syncthreads();
            if ((k0 + kAnyK) % kSumK == 0) each([](floatx4 &q, floatx4 &t) { t += q; q = zero4(); });
        }
    each([](floatx4 &q, floatx4 &t) { q += t; });
    epi(acc, m0 + wm, n0 + wn);
}

template <typename E, int NB, class Epi>
hipError_t launch_gemm_any(const AnyGemmArgs &a, const Epi &epi, hipStream_t s) {
    const int64_t blocks = ((a.M + 63) / 64) * ((a.N + 63) / 64);
    if (blocks == 0) return hipSuccess;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_any_kernel<E, NB, Epi>), dim3((unsigned)blocks), dim3(256), 0, s, a, epi);
    return hipGetLastError();
}

// ---------------------------------------------------------------- stores

// four neighbours of a row, the first `n` of them inside the matrix; `wide` when rows keep the
// alignment of four elements
template <typename E>
__device__ __forceinline__ void store4(E *p, floatx4 v, int64_t n, bool wide) {
    if (wide && n >= 4) {
        *reinterpret_cast<typename Vec4<E>::type *>(p) = cvt4<E>(v);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < n) p[r] = (E)v[r];
    }
}

// C = (acc_in +) the product, rounded to E in `out`, or kept in 32 bits in `acc_out`.
template <typename E>
struct StoreEpi {
    E *out;
    const float *acc_in;
    float *acc_out;
    int64_t M, N, ld;
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0) const {
        const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
        const bool wide = (ld & 3) == 0;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int64_t m = m0 + 16 * i + c;
            if (m >= M) continue;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int64_t n = n0 + 16 * j + 4 * g;
                if (n >= N) continue;
                floatx4 v = acc[0][i][j];
                if (acc_in) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < N) v[r] += acc_in[m * ld + n + r];
                }
                if (out) store4(out + m * ld + n, v, N - n, wide);
                else store4(acc_out + m * ld + n, v, N - n, wide);
            }
        }
    }
};

}  // namespace gdr
