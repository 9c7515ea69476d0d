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
#include "layer_kernels.hpp"

// a lambda of a kernel, whose captures have to stay in registers
#define GDR_INLINE __attribute__((always_inline))

namespace gdr {

// Operand strides in elements; one of the two of each operand is 1.
struct AnyGemmArgs {
    const void *A[2], *B[2];
    int64_t am, ak, bn, bk;
    int64_t M, N, K;
    int pairs;  // products summed over; with NB = 2 the two B matrices of one A, and pairs is 1
    int batch;  // passed to the epilogue
};

// Any sizes, strides and alignments: 64 x 64 tiles staged in LDS as fp32, fp32 matrix
// instructions, every load checked. Four waves of 32 x 32. The sum over k is taken in blocks of
// kSumK terms that are added up afterwards: one running fp32 sum over the 60,000 tokens of a weight
// gradient was 2.1e-5 off (relative Frobenius), in blocks the error stops growing with the length. Its
// loads and LDS accesses are of single elements, which bounds it: 1021 x 2 x 2731 x 1023 takes 257 us in fp32 and 250 in bf16 (44 and 46 TFLOP/s), against 125 and 43 us
// in gemm_tile_kernel for a width of 1024; with an operand whose k is strided 17 TFLOP/s.
constexpr int kAnyK = 16, kAnyLd = kAnyK + 1, kSumK = 512;
// EA and EB: the operands' types.
template <typename EA, typename EB, int NB, class Epi>
__global__ __launch_bounds__(256) void gemm_any_kernel(AnyGemmArgs a, Epi epi) {
    __shared__ float As[64 * kAnyLd], Bs[NB][64 * kAnyLd];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
    const int64_t nm = (a.M + 63) / 64, id = block_id(), m0 = (id % nm) * 64, n0 = (id / nm) * 64;
    if (n0 >= a.N) return;
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

    auto stage = [&](float *dst, const auto *src, int64_t r0, int64_t rows, int64_t k0, int64_t sr, int64_t sk) {
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
            stage(As, (const EA *)a.A[p], m0, a.M, k0, a.am, a.ak);
#pragma unroll
            for (int b = 0; b < NB; ++b) stage(Bs[b], (const EB *)a.B[NB == 2 ? b : p], n0, a.N, k0, a.bn, a.bk);
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
    epi(acc, m0 + wm, n0 + wn, a.batch, nullptr);
}

template <typename EA, typename EB, int NB, class Epi>
hipError_t launch_gemm_any(const AnyGemmArgs &a, const Epi &epi, hipStream_t s) {
    const int64_t blocks = ((a.M + 63) / 64) * ((a.N + 63) / 64);
    if (blocks == 0) return hipSuccess;
    if (blocks > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_any_kernel<EA, EB, NB, Epi>), grid_of(blocks, 256), dim3(256), 0, s, a, epi);
    return hipGetLastError();
}

// ---------------------------------------------------------------- tiled product

// The tiled product for operands whose rows are multiples of 16 bytes (every pointer of the C ABI
// is 16-byte aligned, so whole 16-byte pieces are inside or outside a matrix).
//
// A workgroup of WM x WN waves computes BM x (BN / NB) columns of C; blocks of 128 bytes of k (64 bf16 or
// 32 fp32) of both operands are copied straight from global memory into a ring of S slots of LDS, one
// barrier a block. An operand
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
// The launch holds as many workgroups as the chip runs at a time; each takes tile after tile, and the
// blocks of its tiles are one stream: the next tile's first blocks are copied in while this one's
// last are multiplied and its results are stored. Work is laid out so that the 32 or so tiles an XCD
// runs at a time are neighbours (its L2 holds their operand rows): workgroup i runs on XCD i % 8 and
// takes tiles from the i % 8 th contiguous eighth, in columns of eight tiles of m.
//
// Bound by the matrix instructions and their feeding: 1.2 to 1.34 PFLOP/s on the large bf16 products
// (16384 x 16384 x 2048 and the like; the instruction alone, operands in registers, sustains 2.05; the
// large tile holds one wave a SIMD, so what a wave waits for at a hand-over is not hidden), 92 TFLOP/s
// on 1021 x 2731 x 1024 fp32, whose tiles do not fill the last round.
struct TileGemmArgs {
    const void *A[2], *B[2];
    int64_t lda, ldb;
    int64_t M, N, K;
    int pairs;   // products summed over
    int batch;   // products side by side (A[0] B[0], A[1] B[1])
    int slices;  // slices of k, of `kper` blocks each (the last may have fewer): partial products
    int kper;
    int nm, nn;  // tiles
};
// LDS of one wave for 16 rows of results on their way to memory (RowStore)
constexpr int stage_bytes(int MI) { return 16 * ((MI == 8 ? 256 : MI == 4 ? 128 : 64) + 16); }

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

// a value that is the same in every lane, in scalar registers
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)x), hi = __builtin_amdgcn_readfirstlane((unsigned)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// One operand's tile of R rows (the m or n index) by 128 bytes of k.
template <typename E, bool KC, int R, int NW>
struct Operand {
    static constexpr int es = sizeof(E), KB = 128 / es, L = R / 8 / NW;  // copies per wave
    static constexpr int PPR = R * es / 16;                              // pieces per k row (k strided)
    static_assert(L >= 1 && L * 8 * NW == R, "tile shape");
    const char *cur;     // where the next block of k begins
    int64_t left, step;  // bytes from there to the matrix's end (none left: nothing is read), and per block
    int kleft;           // bytes of k left in a row (KC)
    int voff[L], kpiece; // kpiece: the byte of k this lane's pieces start at (KC)

    static __device__ __forceinline__ int swz(int k) {
        if constexpr (es == 2) return PPR >= 16 ? 2 * (k & 3) + 8 * ((k >> 3) & 1) : 2 * (k & 3);
        else return 4 * ((k >> 2) & 3);
    }
    __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
        if constexpr (KC) {
            step = 128;
            kpiece = ((lane & 7) ^ ((lane >> 3) & 7)) * 16;
#pragma unroll
            for (int i = 0; i < L; ++i) voff[i] = (8 * (wave * L + i) + (lane >> 3)) * (int)(ld * es) + kpiece;
        } else {
            step = uniform(KB * ld * es);
            kpiece = 0;
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int at = 64 * (wave * L + i) + lane, k = at / PPR, slot = at % PPR;
                voff[i] = k * (int)(ld * es) + (slot ^ swz(k)) * 16;
            }
        }
    }
    // rows r0 .. of the matrix at p (of `rows` rows), from its block `at` on
    __device__ __forceinline__ void place(const void *p, int64_t ld, int64_t r0, int64_t rows, int64_t K, int at) {
        if constexpr (KC) {
            const int64_t n = rows - r0 < R ? rows - r0 : R;
            cur = (const char *)uniform((int64_t)p + r0 * ld * es + at * step);
            left = uniform(((((n - 1) * ld + K) * es + 15) & ~15) - at * step);
            kleft = (int)(K * es) - at * 128;
        } else {
            cur = (const char *)uniform((int64_t)p + r0 * es + at * step);
            left = uniform(((((K - 1) * ld + rows - r0) * es + 15) & ~15) - at * step);
        }
    }
    // the next block of the operand, then this wave's copy i of it into LDS at `lds` (byte address)
    u32x4 rsrc;
    bool in;
    __device__ __forceinline__ void begin() {
        rsrc = buffer_at(cur, left);
        cur += step;
        left -= step;
        if constexpr (KC) {
            in = kpiece < kleft;
            kleft -= 128;
        }
    }
    __device__ __forceinline__ void copy(int i, unsigned lds, int wave) const {
        copy_b128(lds + (wave * L + i) * 1024, rsrc, !KC || in ? voff[i] : 0x7fffffff);
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

template <typename E, bool AKC, bool BKC, int NB, int BM, int BN, int WM, int WN, int S, class Epi>
__global__ __launch_bounds__(64 * WM * WN, (BM / WM) * (BN / WN) > 128 * 64 ? 1 : WM * WN / 2) void gemm_tile_kernel(TileGemmArgs, Epi) {
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / NB / WN, MI = TM / 16, NI = TN / 16, KB = 128 / (int)sizeof(E);
    static_assert(NB == 1 || BKC, "two B matrices come k contiguous");
    __shared__ __align__(1024) char lds[S][(BM + BN) * 128];
    __shared__ __align__(16) char stage[NW][stage_bytes(MI)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // The arguments are read where they are used, once a tile: held through the loop they do not fit
    // the scalar registers (45 to 70 of them were spilled to vector registers and back in every block; what is
    // spilled now, 70 where the large tile reduces logits, 44 where it forms dl and 12 elsewhere, is nearly all
    // outside the loop over k).
    typedef __attribute__((address_space(4))) const char arg_char;
    auto arg_at = [](int at) GDR_INLINE {
        arg_char *p = (arg_char *)__builtin_amdgcn_kernarg_segment_ptr() + at;
        asm volatile("" : "+s"(p));
        return p;
    };
    typedef __attribute__((address_space(4))) const TileGemmArgs arg_gemm;

    // this workgroup's tiles: tile, tile + stride, ... below tile_end
    int tile, tile_end, stride;
    {
        arg_gemm &a = *(arg_gemm *)arg_at(0);
        const int all = a.nm * a.nn * a.batch * a.slices, id = blockIdx.x, x = id & 7, q = all >> 3, r = all & 7;
        const int first = x * q + (x < r ? x : r);
        tile = first + (id >> 3);
        tile_end = first + q + (x < r ? 1 : 0);
        stride = ((int)gridDim.x - x + 7) >> 3;
    }
    // tz: batch x slices + slice
    auto locate = [&](int t, int &tm, int &tn, int &tz) GDR_INLINE {
        arg_gemm &a = *(arg_gemm *)arg_at(0);
        const int per = a.nm * a.nn;
        tz = t / per;
        t -= tz * per;
        const int span = 8 * a.nn, group = t / span, in = t % span;
        const int high = a.nm - group * 8 < 8 ? a.nm - group * 8 : 8;
        tm = group * 8 + in % high;
        tn = in / high;
    };
    Operand<E, AKC, BM, NW> A;
    // with two B matrices the first half of the waves copies one, the second half the other
    Operand<E, BKC, BN / NB, NW / NB> B;
    const int bhalf = NB == 2 ? wave / (NW / 2) : 0, bwave = NB == 2 ? wave % (NW / 2) : wave;
    Fragments<E, AKC, BM, MI> fa;
    Fragments<E, BKC, BN / NB, NI> fb;
    fa.init(wm * TM, lane);
    fb.init(wn * TN, lane);
    bool two;  // a sum of two products (never with two B matrices)
    int nkb;   // blocks of one product
    int slices, kper;
    {
        arg_gemm &a = *(arg_gemm *)arg_at(0);
        A.init(a.lda, wave, lane);
        B.init(a.ldb, bwave, lane);
        two = NB == 1 && a.pairs == 2;
        nkb = (int)((a.K + KB - 1) / KB);
        slices = a.slices;
        kper = a.kper;
    }
    // blocks of one product in slice z % slices
    auto blocks_of = [&](int z) GDR_INLINE {
        const int at = slices == 1 ? 0 : z % slices * kper;
        return nkb - at < kper ? nkb - at : kper;
    };
    const unsigned lds0 = __builtin_amdgcn_readfirstlane(
        (unsigned)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)&lds[0][0]));
    constexpr int LA = Operand<E, AKC, BM, NW>::L, LB = Operand<E, BKC, BN / NB, NW / NB>::L;
    // The stream of copies: blocks of product copy_pair of tile copy_tile, copy_left of them. Past the
    // last tile the operands have no bytes: the copies read nothing.
    int copy_tile = tile, copy_pair = 0, copy_left = 0;
    auto place = [&]() GDR_INLINE {
        const bool some = copy_tile < tile_end;
        int tm, tn, tz;
        locate(some ? copy_tile : tile, tm, tn, tz);
        arg_gemm &a = *(arg_gemm *)arg_at(0);
        const int tb = slices == 1 ? tz | copy_pair : tz / slices, at = slices == 1 ? 0 : tz % slices * kper;
        copy_left = blocks_of(tz);
        A.place(tb ? a.A[1] : a.A[0], a.lda, (int64_t)tm * BM, a.M, a.K, at);
        B.place(bhalf | tb ? a.B[1] : a.B[0], a.ldb, (int64_t)tn * (BN / NB), a.N, a.K, at);
        A.left = some ? A.left : 0;
        B.left = some ? B.left : 0;
    };
    auto begin_copy = [&]() GDR_INLINE {
        A.begin();
        B.begin();
        if (--copy_left == 0) {
            copy_pair = two ? copy_pair ^ 1 : 0;
            if (!copy_pair) copy_tile += stride;
            place();
        }
    };
    // this wave's copies i0 .. i1 - 1 of the LA + LB of the block begun, into slot h of the ring
    auto copy = [&](int h, int i0, int i1) GDR_INLINE {
        const unsigned at = lds0 + h * (BM + BN) * 128;
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
    // fp32 sums are taken in blocks, as in gemm_any_kernel
    constexpr bool blocked = sizeof(E) == 4;
    floatx4 total[blocked ? NB : 1][blocked ? MI : 1][blocked ? NI : 1];
    auto each = [&](auto f) GDR_INLINE {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) f(acc[b][i][j], total[blocked ? b : 0][blocked ? i : 0][blocked ? j : 0]);
    };

    // What is on one side of this stays there: a wait between two of them separates the accumulators' writers from
    // their readers, which nothing else holds to their places around an instruction in assembly.
    auto held = [&]() GDR_INLINE { each([](floatx4 &p, floatx4 &) GDR_INLINE { asm volatile("" : "+a"(p)); }); };

    // fragments of the two halves of a block
    typename Fragments<E, AKC, BM, MI>::type va[2][MI], vb[2][NB * NI];
    // reads i0 .. i1 - 1 of the NB NI + MI of half ks of the block in slot h
    auto read = [&](int h, int ks, int i0, int i1) GDR_INLINE {
        const char *buf = lds[h];
#pragma unroll
        for (int i = 0; i < NB * NI + MI; ++i)
            if (i >= i0 && i < i1) {
                if (i < NB * NI) vb[ks][i] = fb.read(buf + BM * 128 + (i / NI) * (BN / NB) * 128, i % NI, ks);
                else va[ks][i - NB * NI] = fa.read(buf, i - NB * NI, ks);
            }
    };
    // Multiplies half ks row by row of the wave's tiles; `side(i)` is issued before row i, in the
    // shadow of the matrix instructions of the row before.
    auto multiply = [&](int ks, auto side) GDR_INLINE {
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
    // The first half of a block is multiplied while its second half is read from LDS; then its slot changes
    // hands, and the second half is multiplied while the next block's first is read and the block S
    // later is copied into the slot. At the hand-over this wave's reads of the block are done and its
    // copies of the next block have landed (those of the S - 2 blocks after it may be in flight, and
    // whatever an epilogue issued since only makes the wait longer), then everyone's.
    constexpr int NR = NB * NI + MI, NC = LA + LB;
    auto hand_over = [&]() GDR_INLINE {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"((S - 2) * NC) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    int h = 0;  // the slot in use
    place();
#pragma unroll
    for (int i = 0; i < S; ++i) {
        begin_copy();
        copy(i, 0, NC);
    }
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"((S - 1) * NC) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(0, 0, 0, NR);
    for (; tile < tile_end; tile += stride) {
        each([](floatx4 &p, floatx4 &t) GDR_INLINE {
            p = zero4();
            if constexpr (blocked) t = zero4();
        });
        if constexpr (in_agprs) {  // written before the matrix instructions in assembly read them
            held();
            asm volatile("s_nop 7");
            held();
        }
        int tm, tn, tz;
        locate(tile, tm, tn, tz);
        const int total_kb = two ? 2 * nkb : blocks_of(tz);
        for (int kb = 0; kb < total_kb; ++kb) {
            multiply(0, [&](int i) GDR_INLINE { read(h, 1, i * NR / MI, (i + 1) * NR / MI); });
            hand_over();
            begin_copy();
            const int next = h + 1 == S ? 0 : h + 1;
            multiply(1, [&](int i) GDR_INLINE {
                read(next, 0, i * NR / MI, (i + 1) * NR / MI);
                copy(h, i * NC / MI, (i + 1) * NC / MI);
            });
            h = next;
            if constexpr (blocked)
                if ((kb + 1) % (kSumK / KB) == 0) each([](floatx4 &p, floatx4 &t) GDR_INLINE {
                    t += p;
                    p = zero4();
                });
        }
        if constexpr (blocked) each([](floatx4 &p, floatx4 &t) GDR_INLINE { p += t; });
        // matrix results are read by other instructions from here on: 18 wait states
        if constexpr (in_agprs) {
            held();
            asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
            held();
        }
        Epi epi;
        {
            static_assert(sizeof(Epi) % 8 == 0 && alignof(Epi) == 8 && sizeof(TileGemmArgs) % 8 == 0, "argument layout");
            __attribute__((address_space(4))) const uint64_t *p =
                (__attribute__((address_space(4))) const uint64_t *)arg_at(sizeof(TileGemmArgs));
            uint64_t words[sizeof(Epi) / 8];
#pragma unroll
            for (int i = 0; i < (int)(sizeof(Epi) / 8); ++i) words[i] = p[i];
            __builtin_memcpy(&epi, words, sizeof(Epi));
        }
        epi(acc, (int64_t)tm * BM + wm * TM, (int64_t)tn * (BN / NB) + wn * TN, tz, stage[wave]);
    }
    // the copies past the end land before the wave ends
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
}

template <typename E, bool AKC, bool BKC, int NB, int BM, int BN, int WM, int WN, int S, class Epi>
hipError_t launch_gemm_tile(TileGemmArgs a, const Epi &epi, hipStream_t s) {
    const int64_t nm = (a.M + BM - 1) / BM, nn = (a.N + BN / NB - 1) / (BN / NB);
    if (nm * nn == 0) return hipSuccess;
    const int64_t all = nm * nn * a.batch * a.slices, nkb = (a.K * (int64_t)sizeof(E) + 127) / 128;
    if (all > INT32_MAX / 2 || a.K < 1 || a.pairs * a.batch * NB > 2 || a.pairs * a.batch < 1 || nkb > INT32_MAX / 4 ||
        a.slices < 1 || (a.pairs > 1 && a.slices > 1))
        return hipErrorInvalidValue;
    // slices of whole blocks, none of them empty
    a.kper = (int)((nkb + a.slices - 1) / a.slices);
    if ((int64_t)a.kper * (a.slices - 1) >= nkb) return hipErrorInvalidValue;
    constexpr int64_t resident = kComputeUnits * (163840 / (S * (BM + BN) * 128 + WM * WN * stage_bytes(BM / WM / 16)));
    a.nm = (int)nm;
    a.nn = (int)nn;
    hipLaunchKernelGGL((gemm_tile_kernel<E, AKC, BKC, NB, BM, BN, WM, WN, S, Epi>), dim3((unsigned)(all < resident ? all : resident)),
                       dim3(64 * WM * WN), 0, s, a, epi);
    return hipGetLastError();
}

// ---------------------------------------------------------------- few rows

// The product for a few rows of A (a decode batch), 16 MT of them a workgroup: B's rows, the weights, are read once, straight into
// matrix operands, and that read is all it costs. A workgroup of eight waves owns 16 NT rows of each B: NT
// tiles of 16, and KS = 8 / NT waves share a tile's k in turns of 128 bytes, so that a wave's loads
// cover whole lines and enough of them are in flight (four turns a wave: 64 KB a workgroup, two workgroups a
// compute unit). The waves' sums are added in order through LDS and the first wave runs the epilogue. A's
// rows come from L2 (rows past M repeat the last one; their columns are not stored). Both operands k
// contiguous, rows whole 16-byte pieces. Bound by that read: feed-forward forward of one token, 2048 x 8192
// (67 MB of weights), 14.8 us (4.5 TB/s), 23.3 us with the tiled kernel; 16 tokens in 65,536 columns
// of 2048 (268 MB) 68 us (3.9 TB/s).
template <typename E, int NB, int MT, int NT, class Epi>
__global__ __launch_bounds__(512, MT == 1 ? 4 : 2) void gemm_rows_kernel(TileGemmArgs a, Epi epi) {
    constexpr int KS = 8 / NT, es = sizeof(E), step = 64 / es, G = 4 / MT;  // step: k of one matrix step; G: turns in flight
    typedef typename Fragments<E, true, 16, 1>::type Piece;
    __shared__ floatx4 held[KS][NT][NB][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
    const int nt = wave % NT, ks = wave / NT;
    const int64_t n0 = block_id() * (16 * NT), n = n0 + 16 * nt + c;
    if (n0 >= a.N) return;
    const int kl = g * (16 / es);  // this lane's first k of a step
    const E *w[NB], *x[MT];
#pragma unroll
    for (int b = 0; b < NB; ++b) w[b] = (const E *)a.B[b] + (n < a.N ? n : a.N - 1) * a.ldb + kl;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = (int64_t)blockIdx.z * (16 * MT) + 16 * i + c;
        x[i] = (const E *)a.A[0] + (m < a.M ? m : a.M - 1) * a.lda + kl;
    }
    floatx4 acc[NB][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[b][i] = zero4();
    const Piece none = {};
    const int64_t turns = (a.K + 2 * step - 1) / (2 * step);
    for (int64_t t0 = ks; t0 < turns; t0 += G * KS) {
        Piece pw[G][2][NB], px[G][2][MT];
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (t0 + q * KS) * 2 * step + h * step;
                const bool in = k + kl < a.K;
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    pw[q][h][b] = in ? __builtin_nontemporal_load(reinterpret_cast<const Piece *>(w[b] + k)) : none;
#pragma unroll
                for (int i = 0; i < MT; ++i) px[q][h][i] = in ? *reinterpret_cast<const Piece *>(x[i] + k) : none;
            }
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[b][i] = mma_step(acc[b][i], pw[q][h][b], px[q][h][i]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MT; ++i) held[ks][nt][b][i][lane] = acc[b][i];
    __syncthreads();
    if (wave) return;
    floatx4 sum[NB][MT][NT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                sum[b][i][j] = held[0][j][b][i][lane];
#pragma unroll
                for (int k = 1; k < KS; ++k) sum[b][i][j] += held[k][j][b][i][lane];
            }
    epi(sum, (int64_t)blockIdx.z * (16 * MT), n0, 0, nullptr);
}

template <typename E, int NB, int MT, int NT, class Epi>
hipError_t launch_gemm_rows(const TileGemmArgs &a, const Epi &epi, hipStream_t s) {
    const int64_t blocks = (a.N + 16 * NT - 1) / (16 * NT);
    dim3 grid = grid_of(blocks, 512);
    grid.z = (unsigned)((a.M + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((gemm_rows_kernel<E, NB, MT, NT, Epi>), grid, dim3(512), 0, s, a, epi);
    return hipGetLastError();
}

// The product on gemm_any_kernel, the products side by side one after the other.
template <typename EA, typename EB, bool AKC, bool BKC, int NB, class Epi>
hipError_t launch_gemm_any_op(const GemmOp &o, const Epi &epi, hipStream_t s) {
    for (int b = 0; b < o.batch; ++b) {
        const AnyGemmArgs g{{o.A[b], o.A[1]}, {o.B[b], o.B[1]}, AKC ? o.lda : 1, AKC ? 1 : o.lda, BKC ? o.ldb : 1,
                            BKC ? 1 : o.ldb, o.M, o.N, o.K, o.pairs, b};
        const hipError_t e = launch_gemm_any<EA, EB, NB>(g, epi, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The product in the order given by AKC and BKC (true: k contiguous, the leading dimension between rows; false:
// rows contiguous, the leading dimension between k), on the kernel that path_of names.
template <typename E, bool AKC, bool BKC, int NB, class Epi>
hipError_t launch_gemm(const GemmOp &o, const Epi &epi, hipStream_t s) {
    const Path how = path_of(o, sizeof(E), NB, AKC && BKC, Epi::whole);
    if (how.kind != Path::kAny) {
        const TileGemmArgs t{{o.A[0], o.A[1]}, {o.B[0], o.B[1]}, o.lda, o.ldb, o.M, o.N, o.K, o.pairs, o.batch, o.slices, 0, 0, 0};
        if constexpr (AKC && BKC)
            if (how.kind == Path::kRows) {
                if constexpr (NB == 1)
                    if (how.nt == 4)
                        return how.mt == 1   ? launch_gemm_rows<E, NB, 1, 4>(t, epi, s)
                               : how.mt == 2 ? launch_gemm_rows<E, NB, 2, 4>(t, epi, s)
                                             : launch_gemm_rows<E, NB, 4, 4>(t, epi, s);
                return how.mt == 1   ? launch_gemm_rows<E, NB, 1, 1>(t, epi, s)
                       : how.mt == 2 ? launch_gemm_rows<E, NB, 2, 1>(t, epi, s)
                                     : launch_gemm_rows<E, NB, 4, 1>(t, epi, s);
            }
        if constexpr (sizeof(E) == 2)
            if (how.tile == 256) return launch_gemm_tile<E, AKC, BKC, NB, 256, 256, 2, 2, 2>(t, epi, s);
        if (how.tile == 128) return launch_gemm_tile<E, AKC, BKC, NB, 128, 128, 4, 2, 2>(t, epi, s);
        return launch_gemm_tile<E, AKC, BKC, NB, 64, 128, 2, 2, 3>(t, epi, s);
    }
    return launch_gemm_any_op<E, E, AKC, BKC, NB>(o, epi, s);
}

// ---------------------------------------------------------------- stores

// The lane, computed anew: what an epilogue derives from it is not kept in registers through the
// next tile's products.
__device__ __forceinline__ int epilogue_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

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

// Sixteen rows of a wave's results (v[j]: lane (g, c) holds row c, columns 16 j + 4 g ..) to rows m0 ..
// of C (of M rows), columns n0 .. (below N). Where whole 16-byte pieces of every row are in range the
// rows go through the wave's stage in LDS (pitch 16 bytes over the row, which spreads the 16 rows
// over the banks) and leave as 16 bytes a lane, whole rows side by side: 5.1 TB/s into HBM on 512 MB,
// against 4.3 TB/s for the accumulator layout's own 32-byte runs. `st` null: no stage.
template <typename E, int MI, int NI>
__device__ __forceinline__ void store_rows(char *st, const floatx4 (&v)[NI], E *C, int64_t ld, int64_t m0, int64_t n0,
                                           int64_t M, int64_t N) {
    constexpr int es = sizeof(E), most = (stage_bytes(MI) / 16 - 16) / (16 * es), NJ = NI < most ? NI : most;
    constexpr int pieces = NJ * es, pitch = 16 * pieces + 16, rows = pieces < 4 ? 16 : 64 / pieces;  // rows per store
    static_assert(NI % NJ == 0 && 64 % pieces == 0, "stage shape");
    const int lane = epilogue_lane(), g = lane >> 4, c = lane & 15;
    // (a single tile of bf16 is not worth a stage)
    if (pieces >= 4 && st && n0 + 16 * NI <= N && ld * es % 16 == 0) {
#pragma unroll
        for (int j0 = 0; j0 < NI; j0 += NJ) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                *reinterpret_cast<typename Vec4<E>::type *>(st + c * pitch + (16 * j + 4 * g) * es) = cvt4<E>(v[j0 + j]);
            wave_lds_sync();
            uint4 piece[16 / rows];
#pragma unroll
            for (int q = 0; q < 16 / rows; ++q)
                piece[q] = *reinterpret_cast<const uint4 *>(st + (q * rows + lane / pieces) * pitch + (lane % pieces) * 16);
            wave_lds_sync();
#pragma unroll
            for (int q = 0; q < 16 / rows; ++q) {
                const int64_t m = m0 + q * rows + lane / pieces;
                if (m < M)
                    *reinterpret_cast<uint4 *>(C + m * ld + n0 + 16 * j0 + (lane % pieces) * (16 / es)) = piece[q];
            }
        }
        return;
    }
    const int64_t m = m0 + c;
    if (m >= M) return;
    const bool wide = (ld & 3) == 0;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int64_t n = n0 + 16 * j + 4 * g;
        if (n < N) store4(C + m * ld + n, v[j], N - n, wide);
    }
}

// C = (acc_in +) the product, times *scale (where given) and rounded to E in out[batch], or kept in 32 bits
// in `acc_out`; a slice of k goes to `part` [batch x slices][M][ld] as it is.
template <typename E>
struct StoreEpi {
    E *out[2];
    const float *acc_in;
    float *acc_out;
    float *part;
    const float *scale;
    int64_t M, N, ld;
    static constexpr bool whole = true;  // the epilogue stores the whole tile
    template <int MI, int NI>
    __device__ __forceinline__ void operator()(const floatx4 (&acc)[1][MI][NI], int64_t m0, int64_t n0, int z, char *st) const {
        const int lane = epilogue_lane(), g = lane >> 4, c = lane & 15;
        E *C = part ? nullptr : z ? out[1] : out[0];
        float *C32 = part ? part + z * M * ld : acc_out;
        const float by = C && scale ? *scale : 1.f;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            floatx4 v[NI];
            const int64_t m = m0 + 16 * i + c;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                v[j] = acc[0][i][j];
                const int64_t n = n0 + 16 * j + 4 * g;
                if (acc_in && m < M && n < N) {
                    const float *p = acc_in + m * ld + n;
                    if ((ld & 3) == 0) v[j] += *reinterpret_cast<const floatx4 *>(p);
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (n + r < N) v[j][r] += p[r];
                }
                v[j] *= by;
            }
            if (C) store_rows<E, MI, NI>(st, v, C, ld, m0 + 16 * i, n0, M, N);
            else store_rows<float, MI, NI>(st, v, C32, ld, m0 + 16 * i, n0, M, N);
        }
    }
};

// C[b] = (acc_in +) the sum of its `parts` partial products, in order; four neighbours a thread. n: elements
// of one product, a multiple of 4. Bound by memory: 6.8 us for 1021 x 1024 in eight slices (36 MB, 5.2 TB/s).
template <typename E>
__global__ __launch_bounds__(256) void gemm_sum_kernel(const float *part, int parts, int64_t n, E *out0, E *out1,
                                                       const float *acc_in, float *acc_out, const float *scale) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int b = blockIdx.y;
    floatx4 v = acc_in ? *reinterpret_cast<const floatx4 *>(acc_in + i) : zero4();
    for (int p = 0; p < parts; ++p) v += *reinterpret_cast<const floatx4 *>(part + ((int64_t)b * parts + p) * n + i);
    E *out = b ? out1 : out0;
    if (out) *reinterpret_cast<typename Vec4<E>::type *>(out + i) = cvt4<E>(scale ? v * *scale : v);
    else *reinterpret_cast<floatx4 *>(acc_out + i) = v;
}

// bytes of partial products launch_gemm_store needs
template <typename E>
int64_t store_ws_bytes(const GemmOp &o) {
    const int64_t s = store_choice(o, sizeof(E)).slices;
    return s > 1 ? s * o.pairs * o.batch * o.M * o.N * 4 : 0;
}
// The plain product (epi.part is set here), cut where store_choice says so.
template <typename E, bool AKC, bool BKC>
hipError_t launch_gemm_store(const GemmOp &o, StoreEpi<E> epi, void *ws, hipStream_t s) {
    epi.part = nullptr;
    const Choice how = store_choice(o, sizeof(E));
    GemmOp run = o;
    run.tile = how.tile;
    if (how.slices == 1) return launch_gemm<E, AKC, BKC, 1>(run, epi, s);
    if (epi.ld != o.N) return hipErrorInvalidValue;
    run.pairs = 1;
    run.batch = o.pairs * o.batch;
    run.slices = how.slices;
    StoreEpi<E> to_part = epi;
    to_part.part = (float *)ws;
    to_part.acc_in = nullptr;
    const hipError_t e = launch_gemm<E, AKC, BKC, 1>(run, to_part, s);
    if (e != hipSuccess) return e;
    const int64_t n = o.M * o.N;
    hipLaunchKernelGGL((gemm_sum_kernel<E>), dim3((unsigned)((n / 4 + 255) / 256), (unsigned)o.batch), dim3(256), 0, s, (const float *)ws,
                       how.slices * o.pairs, n, epi.out[0], epi.out[1], epi.acc_in, epi.acc_out, epi.scale);
    return hipGetLastError();
}

}  // namespace gdr
