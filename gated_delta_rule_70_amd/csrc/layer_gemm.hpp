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

// ---------------------------------------------------------------- tiled product

// The tiled product for operands whose rows are multiples of 16 bytes (every pointer of the C ABI
// is 16-byte aligned, so whole 16-byte pieces are inside or outside a matrix).
//
// A workgroup of WM x WN waves computes BM x (BN / NB) columns of C; a block of 128 bytes of k (64 bf16
// or 32 fp32) of both operands is copied straight from global memory into one half of LDS while
// the other half is multiplied, one barrier a block. An operand
// comes in either order:
//   KC (k contiguous, rows of ld elements): LDS holds rows of 128 bytes, eight 16-byte pieces, piece p
//      of row r at p ^ (r & 7), so that the 16 rows a fragment read touches spread over the banks;
//   otherwise (row index contiguous, k strided): LDS holds one row per k. bf16 fragments come
//      from the transpose read (each 16-lane group takes a 4 x 16 block), fp32 ones from four
//      scalar reads; pieces are XORed by bits of k that differ between the rows one read touches.
// Both orders give a lane the same k values of a fragment (8g .. 8g+7 of a 32-deep bf16 step, 4g ..
// 4g+3 of a 16-deep fp32 one), so any two can be paired.
//
// Reads past a matrix: the buffer descriptor ends with the 16-byte piece of the matrix's last
// element (rows are whole pieces, so that piece is the matrix's own), and pieces that begin past
// the row's end in k are sent past the descriptor; both arrive in LDS as zeros. A k-contiguous
// operand whose K is not whole pieces holds zeros up to the piece's end. In the k-strided order
// columns past the row's end are the next row's values: they reach only columns of C that are
// not stored.
//
// Work is laid out so that the 32 or so tiles an XCD runs at a time are neighbours (its L2 holds
// their operand rows): workgroup i runs on XCD i % 8 and takes tiles from the i % 8 th contiguous
// eighth, in columns of eight tiles of m.
struct TileGemmArgs {
    const void *A[2], *B[2];
    int64_t lda, ldb;
    int64_t M, N, K;
    int pairs;
    int nm, nn;  // tiles
};

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from the buffer into LDS at m0 + 16 lane. Written in assembly because the
// compiler would wait for every copy before its next LDS read; each wave waits for its own copies
// before the barrier that hands the block over.
__device__ __forceinline__ void copy_b128(unsigned lds, u32x4 rsrc, int voff) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(voff), "s"(rsrc), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ u32x4 buffer_at(const char *p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    // bytes clamped to 0 .. 2^31 - 1, in 32-bit halves (there is no scalar 64-bit less-than)
    const int hi = (int)(bytes >> 32);
    const unsigned lo = (unsigned)bytes;
    const unsigned n = hi < 0 ? 0u : hi > 0 || lo > 0x7fffffffu ? 0x7fffffffu : lo;
    u32x4 r;
    r.x = __builtin_amdgcn_readfirstlane((unsigned)a);
    r.y = __builtin_amdgcn_readfirstlane((unsigned)(a >> 32) & 0xffffu);
    r.z = __builtin_amdgcn_readfirstlane(n);
    r.w = 0x00020000;  // raw, untyped
    // A vector instruction's write of a scalar register (readfirstlane) needs five wait states before
    // a buffer access reads it; the compiler does not count them for an access inside assembly.
    asm volatile("s_nop 4" : "+s"(r));
    return r;
}

__device__ __forceinline__ bf16x4 read_tr(const char *p) {
    return __builtin_bit_cast(
        bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) shortx4 *)(p)));
}

// One operand's tile of R rows (the m or n index) by 128 bytes of k.
template <typename E, bool KC, int R, int NW>
struct Operand {
    static constexpr int es = sizeof(E), KB = 128 / es, L = R / 8 / NW;  // copies per wave
    static constexpr int PPR = R * es / 16;                              // pieces per k row (k strided)
    static_assert(L >= 1 && L * 8 * NW == R, "tile shape");
    const char *base;
    int64_t limit, step;  // bytes from base to the matrix's end, and per block of k
    int voff[L], kpiece;  // kpiece: the byte of k this lane's pieces start at (KC)
    int64_t kbytes;

    static __device__ __forceinline__ int swz(int k) {
        if constexpr (es == 2) return PPR >= 16 ? 2 * (k & 3) + 8 * ((k >> 3) & 1) : 2 * (k & 3);
        else return 4 * ((k >> 2) & 3);
    }
    __device__ __forceinline__ void init(const void *p, int64_t ld, int64_t r0, int64_t rows, int64_t K, int wave, int lane) {
        kbytes = K * es;
        if constexpr (KC) {
            const int64_t n = rows - r0 < R ? rows - r0 : R;
            base = (const char *)p + r0 * ld * es;
            limit = ((n - 1) * ld * es + kbytes + 15) / 16 * 16;
            step = 128;
            kpiece = ((lane & 7) ^ ((lane >> 3) & 7)) * 16;
#pragma unroll
            for (int i = 0; i < L; ++i) voff[i] = (8 * (wave * L + i) + (lane >> 3)) * (int)(ld * es) + kpiece;
        } else {
            base = (const char *)p + r0 * es;
            limit = (((K - 1) * ld + rows - r0) * es + 15) / 16 * 16;
            step = KB * ld * es;
            kpiece = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int at = 64 * (wave * L + i) + lane, k = at / PPR, slot = at % PPR;
                voff[i] = k * (int)(ld * es) + (slot ^ swz(k)) * 16;
            }
        }
    }
    // Block kb of the operand, this wave's copy i into LDS at `lds` (byte address). A block past the
    // last reads nothing: in the k-strided order its descriptor holds no bytes (kb KB >= K rows of
    // ld >= rows - r0 elements lie behind it), in the k-contiguous one each piece begins past the
    // row's end.
    u32x4 rsrc;
    bool in;
    __device__ __forceinline__ void begin(const char *b, int kb) {
        rsrc = buffer_at(b + kb * step, limit - kb * step);
        in = !KC || (int64_t)kb * 128 + kpiece < kbytes;
    }
    __device__ __forceinline__ void copy(int i, unsigned lds, int wave) const {
        copy_b128(lds + (wave * L + i) * 1024, rsrc, in ? voff[i] : 0x7fffffff);
    }
};

// Fragments of one operand for the wave's rows r0 .. r0 + 16 I - 1 (r0 a multiple of 16).
template <typename E, bool KC, int R, int I>
struct Fragments;
template <bool KC, int R, int I>
struct Fragments<__bf16, KC, R, I> {
    typedef bf16x8 type;
    int off[KC ? 1 : I];
    __device__ __forceinline__ void init(int r0, int lane) {
        const int g = lane >> 4, c = lane & 15;
        if constexpr (KC) {
            off[0] = (r0 + c) * 128 + ((g ^ (c & 7)) << 4);
        } else {
            const int k = 8 * g + (c >> 2);
#pragma unroll
            for (int i = 0; i < I; ++i)
                off[i] = k * R * 2 + (((r0 / 8 + 2 * i + ((c & 3) >> 1)) ^ Operand<__bf16, false, R, 1>::swz(k)) << 4) + 8 * (c & 1);
        }
    }
    __device__ __forceinline__ type read(const char *buf, int i, int ks) const {
        if constexpr (KC) {
            return *reinterpret_cast<const bf16x8 *>(buf + (off[0] ^ (ks << 6)) + 2048 * i);
        } else {
            const char *p = buf + off[i] + ks * 32 * R * 2;
            return __builtin_shufflevector(read_tr(p), read_tr(p + 4 * R * 2), 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};
template <bool KC, int R, int I>
struct Fragments<float, KC, R, I> {
    typedef floatx4 type;
    int off[KC ? 1 : I];
    __device__ __forceinline__ void init(int r0, int lane) {
        const int g = lane >> 4, c = lane & 15;
        if constexpr (KC) {
            off[0] = (r0 + c) * 128 + ((g ^ (c & 7)) << 4);
        } else {
#pragma unroll
            for (int i = 0; i < I; ++i)
                off[i] = 4 * g * R * 4 + (((r0 + 16 * i + c) / 4 ^ Operand<float, false, R, 1>::swz(4 * g)) << 4) + 4 * (c & 3);
        }
    }
    __device__ __forceinline__ type read(const char *buf, int i, int ks) const {
        if constexpr (KC) {
            return *reinterpret_cast<const floatx4 *>(buf + (off[0] ^ (ks << 6)) + 2048 * i);
        } else {
            const char *p = buf + off[i] + ks * 16 * R * 4;
            floatx4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float *>(p + j * R * 4);
            return v;
        }
    }
};
__device__ __forceinline__ floatx4 mma_step(floatx4 acc, bf16x8 a, bf16x8 b) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mma_step(floatx4 acc, floatx4 a, floatx4 b) { return mma16(acc, a, b); }

// The same with the accumulator held to AGPRs: left to itself the compiler moved a quarter of the
// large tile's 256 accumulators between register files in every block (588 instructions a block
// next to 128 matrix ones; 330 this way).
__device__ __forceinline__ void mma_step_agpr(floatx4 &acc, bf16x8 a, bf16x8 b) {
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}

template <typename E, bool AKC, bool BKC, int NB, int BM, int BN, int WM, int WN, class Epi>
__global__ __launch_bounds__(64 * WM * WN, (BM / WM) * (BN / WN) > 128 * 64 ? 1 : 2) void gemm_tile_kernel(TileGemmArgs a, Epi epi) {
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / NB / WN, MI = TM / 16, NI = TN / 16, KB = 128 / (int)sizeof(E);
    static_assert(NB == 1 || BKC, "two B matrices come k contiguous");
    __shared__ __align__(1024) char lds[2][(BM + BN) * 128];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    int64_t m0, n0;
    {
        const int total = a.nm * a.nn, id = blockIdx.x, x = id & 7, q = total >> 3, r = total & 7;
        const int t = x * q + (x < r ? x : r) + (id >> 3);
        const int span = 8 * a.nn, group = t / span, in = t % span;
        const int high = a.nm - group * 8 < 8 ? a.nm - group * 8 : 8;
        m0 = (int64_t)(group * 8 + in % high) * BM;
        n0 = (int64_t)(in / high) * (BN / NB);
    }
    Operand<E, AKC, BM, NW> A;
    A.init(a.A[0], a.lda, m0, a.M, a.K, wave, lane);
    // with two B matrices the first half of the waves copies one, the second half the other
    Operand<E, BKC, BN / NB, NW / NB> B;
    const int bhalf = NB == 2 ? wave / (NW / 2) : 0, bwave = NB == 2 ? wave % (NW / 2) : wave;
    B.init(a.B[bhalf], a.ldb, n0, a.N, a.K, bwave, lane);
    // the second pair of a sum of two products (never with two B matrices)
    const bool two = NB == 1 && a.pairs == 2;
    const char *abase2 = two ? A.base + ((const char *)a.A[1] - (const char *)a.A[0]) : A.base;
    const char *bbase2 = two ? B.base + ((const char *)a.B[1] - (const char *)a.B[0]) : B.base;

    Fragments<E, AKC, BM, MI> fa;
    Fragments<E, BKC, BN / NB, NI> fb;
    fa.init(wm * TM, lane);
    fb.init(wn * TN, lane);

    const int nkb = (int)((a.K + KB - 1) / KB), total_kb = two ? 2 * nkb : nkb;
    const unsigned lds0 = __builtin_amdgcn_readfirstlane(
        (unsigned)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)&lds[0][0]));
    constexpr int LA = Operand<E, AKC, BM, NW>::L, LB = Operand<E, BKC, BN / NB, NW / NB>::L;
    auto begin_copy = [&](int kb) {
        const bool second = two && kb >= nkb;
        const int k = second ? kb - nkb : kb;
        A.begin(second ? abase2 : A.base, k);
        B.begin(second ? bbase2 : B.base, k);
    };
    // this wave's copies i0 .. i1 - 1 of the LA + LB of block kb
    auto copy = [&](int kb, int i0, int i1) {
        const unsigned at = lds0 + (kb & 1) * (BM + BN) * 128;
#pragma unroll
        for (int i = 0; i < LA + LB; ++i)
            if (i >= i0 && i < i1) {
                if (i < LA) A.copy(i, at, wave);
                else B.copy(i - LA, at + BM * 128 + bhalf * (BN / NB) * 128, bwave);
            }
    };

    // 256 accumulators a lane are the AGPRs
    constexpr bool in_agprs = NB * MI * NI > 32;
    floatx4 acc[NB][MI][NI];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[b][i][j] = zero4();
    // fp32 sums are taken in blocks, as in gemm_any_kernel
    constexpr bool blocked = sizeof(E) == 4;
    floatx4 total[blocked ? NB : 1][blocked ? MI : 1][blocked ? NI : 1];
    if constexpr (blocked)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) total[b][i][j] = zero4();

    // fragments of the two halves of a block
    typename Fragments<E, AKC, BM, MI>::type va[2][MI], vb[2][NB * NI];
    // reads i0 .. i1 - 1 of the NB NI + MI of half ks of block kb
    auto read = [&](int kb, int ks, int i0, int i1) {
        const char *buf = lds[kb & 1];
#pragma unroll
        for (int i = 0; i < NB * NI + MI; ++i)
            if (i >= i0 && i < i1) {
                if (i < NB * NI) vb[ks][i] = fb.read(buf + BM * 128 + (i / NI) * (BN / NB) * 128, i % NI, ks);
                else va[ks][i - NB * NI] = fa.read(buf, i - NB * NI, ks);
            }
    };
    // Multiplies half ks row by row of the wave's tiles; `side(i)` is issued before row i, in the
    // shadow of the matrix instructions of the row before.
    auto multiply = [&](int ks, auto side) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            side(i);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    if constexpr (in_agprs) mma_step_agpr(acc[b][i][j], vb[ks][b * NI + j], va[ks][i]);
                    else acc[b][i][j] = mma_step(acc[b][i][j], vb[ks][b * NI + j], va[ks][i]);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // this wave's copies have landed and its reads of the block in use are done, then everyone's
    auto hand_over = [] {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // The first half of a block is multiplied while its second half is read from LDS; then the halves
    // of LDS change hands, and the second half is multiplied while the next block's first is read
    // and the block after it is copied in.
    constexpr int NR = NB * NI + MI, NC = LA + LB;
    begin_copy(0);
    copy(0, 0, NC);
    hand_over();
    begin_copy(1);
    copy(1, 0, NC);
    read(0, 0, 0, NR);
    for (int kb = 0; kb < total_kb; ++kb) {
        multiply(0, [&](int i) { read(kb, 1, i * NR / MI, (i + 1) * NR / MI); });
        hand_over();
        begin_copy(kb + 2);
        multiply(1, [&](int i) {
            read(kb + 1, 0, i * NR / MI, (i + 1) * NR / MI);
            copy(kb + 2, i * NC / MI, (i + 1) * NC / MI);
        });
        if constexpr (blocked)
            if ((kb + 1) % (kSumK / KB) == 0) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j) {
                            total[b][i][j] += acc[b][i][j];
                            acc[b][i][j] = zero4();
                        }
            }
    }
    // the copies past the end land before the wave ends
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (blocked)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[b][i][j] += total[b][i][j];
    // matrix results are read by other instructions from here on: 18 wait states
    if constexpr (in_agprs) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) asm volatile("" : "+a"(acc[b][i][j]));
        asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    }
    epi(acc, m0 + wm * TM, n0 + wn * TN);
}

template <typename E, bool AKC, bool BKC, int NB, int BM, int BN, int WM, int WN, class Epi>
hipError_t launch_gemm_tile(TileGemmArgs a, const Epi &epi, hipStream_t s) {
    const int64_t nm = (a.M + BM - 1) / BM, nn = (a.N + BN / NB - 1) / (BN / NB);
    if (nm * nn == 0) return hipSuccess;
    if (nm * nn > INT32_MAX / 16 || a.pairs < 1 || a.pairs > 3 - NB) return hipErrorInvalidValue;
    a.nm = (int)nm;
    a.nn = (int)nn;
    hipLaunchKernelGGL((gemm_tile_kernel<E, AKC, BKC, NB, BM, BN, WM, WN, Epi>), dim3((unsigned)(nm * nn)),
                       dim3(64 * WM * WN), 0, s, a, epi);
    return hipGetLastError();
}

// columns of C per wave are a multiple of this in the tiled and in the any-size kernel
constexpr int kTileCols = 64, kAnyCols = 32;

// C = sum of A_p B_p^T in the order given by AKC and BKC (true: k contiguous, the leading dimension
// between rows; false: rows contiguous, the leading dimension between k).
struct GemmOp {
    const void *A[2], *B[2];
    int64_t lda, ldb, M, N, K;
    int pairs;
};
// whether rows of ld elements are whole 16-byte pieces
template <typename E>
bool whole_pieces(int64_t ld) {
    return ld * (int64_t)sizeof(E) % 16 == 0;
}
template <typename E, bool AKC, bool BKC, int NB, class Epi>
hipError_t launch_gemm(const GemmOp &o, const Epi &epi, hipStream_t s) {
    if (whole_pieces<E>(o.lda) && whole_pieces<E>(o.ldb)) {
        TileGemmArgs t{{o.A[0], o.A[1] ? o.A[1] : o.A[0]}, {o.B[0], o.B[1] ? o.B[1] : o.B[0]}, o.lda, o.ldb, o.M, o.N, o.K, o.pairs, 0, 0};
        const int64_t big = ((o.M + 255) / 256) * ((o.N * NB + 255) / 256);
        if constexpr (sizeof(E) == 2)
            if (big >= 192) return launch_gemm_tile<E, AKC, BKC, NB, 256, 256, 2, 2>(t, epi, s);
        return launch_gemm_tile<E, AKC, BKC, NB, 128, 128, 2, 2>(t, epi, s);
    }
    AnyGemmArgs g{{o.A[0], o.A[1]}, {o.B[0], o.B[1]}, AKC ? o.lda : 1, AKC ? 1 : o.lda, BKC ? o.ldb : 1, BKC ? 1 : o.ldb,
                  o.M, o.N, o.K, o.pairs};
    return launch_gemm_any<E, NB>(g, epi, s);
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
