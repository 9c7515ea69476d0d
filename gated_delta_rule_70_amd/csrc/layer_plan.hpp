// How the layer operators (channel scan, gated feed-forward, linear cross entropy) lay a call out: what runs as
// one launch or two, in which tiles, slices and pieces. Host arithmetic on sizes alone.
#pragma once

#include <stdint.h>

namespace gdr {

constexpr int kComputeUnits = 256;

// ---------------------------------------------------------------- channel scan

// Tokens per block of the channel scan: the forward keeps the state that enters each block of a
// sequence when the backward will run. Packed sequences: the blocks of sequence s start at slot
// cu[s] / kScanBlock + s, so that no two sequences share one.
constexpr int kScanBlock = 256;

// How a launch walks the sequences: whole, or in chunks of `chunk` tokens. Packed chunks of sequence
// s begin at slot cu[s] / chunk + s.
struct ScanPlan {
    int64_t chunk;   // 0: not split
    int64_t units;   // sequences, or chunk slots
    int64_t ntile;   // channel tiles
    int64_t per_seq; // chunks of a sequence (not packed)
};

// Channels a thread: 64-byte runs of a row for 16 lanes, as two bf16 a lane or one fp32 (two fp32, a third of
// whose backward's registers spilled: 0.214 ms against 0.142 ms on packed fp32 sequences of 520 channels);
// one bf16 where rows are not whole pairs.
inline int scan_vec(int64_t D, int es) { return es == 2 && D % 2 == 0 ? 2 : 1; }

// Split where whole sequences would leave compute units idle: fewer than 224 workgroups (of 256), or,
// packed, fewer than 1024 (their lengths differ and are not known here). Chunks are whole blocks, of a
// size that gives about 768 workgroups: three a compute unit, which evens out the ends.
inline ScanPlan scan_plan(int64_t T, int64_t D, int64_t nseq, bool packed, int vec) {
    ScanPlan p;
    const int64_t cols = 16 * vec;
    p.ntile = (D + cols - 1) / cols;
    p.chunk = 0;
    p.units = nseq;
    p.per_seq = 1;
    const int64_t rows = packed ? T : nseq * T, blocks = (rows + kScanBlock - 1) / kScanBlock;
    if (nseq == 0 || T <= kScanBlock || nseq * p.ntile >= (packed ? 1024 : 224)) return p;
    const int64_t per = (blocks * p.ntile + 767) / 768;
    p.chunk = per * kScanBlock;
    p.per_seq = (T + p.chunk - 1) / p.chunk;
    p.units = packed ? T / p.chunk + nseq + 1 : nseq * p.per_seq;
    return p;
}

// ---------------------------------------------------------------- products

// C = sum of A_p B_p^T, M x N over K, A's and B's rows lda and ldb elements apart (their k index where k is the
// strided one).
struct GemmOp {
    const void *A[2], *B[2];
    int64_t lda, ldb, M, N, K;
    int pairs = 1, batch = 1;  // at most one of them 2: A[0] B[0] + A[1] B[1], or the two side by side
    int slices = 1;            // of k: the epilogue gets partial products (batch x slices + slice)
    int tile = 0;              // the tile to use; 0: chosen here
};

// The operators' products, without the operands.
inline int64_t grad_ld(int64_t F) { return (F + 7) / 8 * 8; }  // rows of dG and dU
inline GemmOp ffn_fwd_product(int64_t M, int64_t D, int64_t F) { return GemmOp{{}, {}, D, D, M, F, D}; }
inline GemmOp ffn_dx_product(int64_t M, int64_t D, int64_t F) { return GemmOp{{}, {}, grad_ld(F), D, M, D, F, 2, 1}; }
inline GemmOp ffn_dw_product(int64_t M, int64_t D, int64_t F) { return GemmOp{{}, {}, grad_ld(F), D, F, D, M, 1, 2}; }
inline GemmOp ce_logits_product(int64_t N, int64_t D, int64_t width) { return GemmOp{{}, {}, D, D, N, width, D}; }
inline GemmOp ce_dx_product(int64_t N, int64_t D, int64_t piece, int64_t width) { return GemmOp{{}, {}, piece, D, N, D, width}; }
inline GemmOp ce_dw_product(int64_t N, int64_t D, int64_t piece, int64_t width) { return GemmOp{{}, {}, piece, D, width, D, N}; }

// Vocabulary columns per piece of the backward: dl of a piece takes at most about 512 MB, and its rows at most
// 2^20 elements, as the other operands' (the products' offsets within a tile are 32 bits).
inline int64_t ce_piece(int64_t N, int64_t V) {
    int64_t p = (INT64_C(1) << 28) / (N > 0 ? N : 1) / 256 * 256;
    if (p < 2048) p = 2048;
    if (p > INT64_C(1) << 20) p = INT64_C(1) << 20;
    const int64_t all = (V + 7) / 8 * 8;
    return p < all ? p : all;
}

// columns of a wave's partial sum in the tiled and in the any-size kernel
constexpr int kTileCols = 64, kAnyCols = 32;
// whether rows of ld elements of es bytes are whole 16-byte pieces
inline bool whole_pieces(int64_t ld, int es) { return ld * es % 16 == 0; }
// blocks of 128 bytes of k
inline int64_t k_blocks(int64_t K, int es) { return (K * es + 127) / 128; }

// How a product is run. Tiles of 256 x 256 (bf16, one workgroup a compute unit), 128 x 128 or 64 x 128 (two); a
// plain product's k may be cut into slices that are summed afterwards. The choice is the least of
//   rounds (blocks a slice * block + fixed) + what summing the slices costs,
// rounds = tiles * slices / resident workgroups, rounded up, with the times measured on this chip: a block of
// 128 bytes of k with every compute unit busy 1.6, 1.1 and 0.8 us (fp32: 4.6 and 2.0 us, of which the matrix
// instructions 3.6 and 1.8), a tile's start and end 24 (16 where the epilogue does not store the whole tile), 3.5
// and 3 us, a slice's 4 bytes at 3 TB/s and a launch. The 128 x 128 tile has eight waves, so that one of a
// SIMD's four multiplies while another stores: at 16 blocks of k (1021 x 32003 x 1024) its stored products take 91 us,
// 105 with four waves and 103 in 256 x 256 tiles, at 32 and more the large tile wins. What the model is for: 129 tiles of 256 x 256 are one round that leaves half the chip idle, 516 of 128 x
// 128 are two of which one is empty (cross entropy dx of 10904 x 744 in 22,528 columns: 722 us so).
struct Choice {
    int tile, slices;
};
inline Choice choose(int64_t M, int64_t N, int64_t nkb, int products, bool bf16, bool cut, bool whole) {
    struct {
        int tile, rows, cols, resident;
        double block, fixed;
    } const kinds[] = {{256, 256, 256, kComputeUnits, 1.6, whole ? 24. : 16.},
                 {128, 128, 128, 2 * kComputeUnits, bf16 ? 1.1 : 4.6, 3.5},
                 {64, 64, 128, 2 * kComputeUnits, bf16 ? 0.8 : 2.0, 3.}};
    Choice best{64, 1};
    double least = -1.;
    for (const auto &k : kinds) {
        if (k.tile == 256 && !bf16) continue;
        const int64_t tiles = ((M + k.rows - 1) / k.rows) * ((N + k.cols - 1) / k.cols) * products;
        for (int64_t want = 1; want <= (cut ? 32 : 1); ++want) {
            if (want > 1 && nkb < 4 * want) break;
            const int64_t kper = (nkb + want - 1) / want, s = (nkb + kper - 1) / kper;  // no slice empty
            const int64_t rounds = (tiles * s + k.resident - 1) / k.resident;
            const double sum = s > 1 ? 5. + (double)(s * products * M * N) * 4e-6 / 3. : 0.;
            const double time = rounds * (kper * k.block + k.fixed) + sum;
            if (least < 0. || time < least) {
                least = time;
                best = Choice{k.tile, (int)s};
            }
        }
    }
    return best;
}

// Whether the product (both operands k contiguous, `cols` rows of all B matrices) goes by rows: up to 64 rows
// the weights' read is all there is; up to 256 it still wins where 64 x 128 tiles would leave half of the
// compute units idle (85 rows, 1600 x 2 x 1181 fp32: 64 us in 38 tiles).
inline bool by_rows(int64_t M, int64_t cols) {
    return M > 0 && (M <= 64 || (M <= 256 && ((M + 63) / 64) * ((cols + 127) / 128) < 128));
}
// Columns of C of a workgroup that goes by rows, over 16: with one B four tiles of 16 where there are plenty
// (16 rows x 2048 x 65536: 74 us with four, 79 us with two, which leave more partial sums to join), else one.
inline int rows_tiles(int64_t N, int NB) { return NB == 1 && N >= 64 * 512 ? 4 : 1; }

// The kernel a product runs on. `both`: both operands k contiguous; `whole`: the epilogue stores whole tiles.
struct Path {
    enum { kAny, kRows, kTile } kind;
    int tile;    // kTile: 256, 128 or 64
    int mt, nt;  // kRows: tiles of 16 rows and of 16 columns a workgroup
};
inline Path path_of(const GemmOp &o, int es, int NB, bool both, bool whole) {
    if (!whole_pieces(o.lda, es) || !whole_pieces(o.ldb, es) || o.K < 1) return Path{Path::kAny, 0, 0, 0};
    if (both && by_rows(o.M, o.N * NB)) return Path{Path::kRows, 0, o.M <= 16 ? 1 : o.M <= 32 ? 2 : 4, rows_tiles(o.N, NB)};
    if (o.tile) return Path{Path::kTile, o.tile, 0, 0};
    return Path{Path::kTile, choose(o.M, o.N * NB, o.pairs * k_blocks(o.K, es), o.batch * o.slices, es == 2, false, whole).tile, 0, 0};
}
// The tile and the slices of k of a plain product (rows of N elements); a sum of two products is cut at the
// seam first. The same for the workspace's size and for the launch.
inline Choice store_choice(const GemmOp &o, int es) {
    if (!whole_pieces(o.lda, es) || !whole_pieces(o.ldb, es) || o.M < 1 || o.K < 1) return Choice{0, 1};
    const Choice whole = choose(o.M, o.N, o.pairs * k_blocks(o.K, es), o.batch, es == 2, false, true);
    if (o.N % 4) return whole;
    const Choice cut = choose(o.M, o.N, k_blocks(o.K, es), o.pairs * o.batch, es == 2, true, true);
    return cut.slices > 1 ? cut : whole;
}
// Columns of C of one wave's partial sum when x W^T (rows of ld elements) is reduced as it is formed.
inline int64_t wave_cols(int64_t M, int64_t N, int64_t ld, int es) {
    if (!whole_pieces(ld, es)) return kAnyCols;
    return by_rows(M, N) ? 16 * rows_tiles(N, 1) : kTileCols;
}

}  // namespace gdr
