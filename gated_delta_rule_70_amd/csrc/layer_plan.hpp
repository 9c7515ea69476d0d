// How the layer operators (channel scan, linear attention, gated feed-forward, linear cross entropy) lay a call out: what runs as
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

// ---------------------------------------------------------------- linear attention

constexpr int kAttnChunk = 64;  // tokens of a bf16 chunk; fp32 chunks are half of it

// How a call walks the sequences: whole (seg 0), or in segments that are walked side by side once a pass has left each
// one's own state. Packed segments of sequence s begin at slot cu[s] / seg + s; where one is followed by another, a sequence has a
// cut, and the forward forms states of the segments before those alone.
struct AttnPlan {
    int64_t seg, per_seq, slots;
};
// `units`: workgroups of a whole sequence (heads and column slices). Split, into about 512 of whole chunks, where whole sequences
// leave too many compute units idle to be worth less than the states' sweep and the second read: fewer than 192 of them, 96 in
// the backward, which has each twice. Sequences of 4096 tokens of 16 heads of 128, bf16, split and whole: forward 8 of them (128)
// 239 and 289 us, 12 (192) 404 and 385, 18 570 and 499, 23 894 and 531; backward 4 (64) 382 and 479, 6 (96) 640 and 577, 10 990
// and 670; of 1024 tokens forward 8 89 and 86, backward 4 149 and 132; forward fp32 4 316 and 497, 8 527 and 504. Values of 256
// channels, whose gradients of q and k have one workgroup a compute unit: 6 1051 and 1168, 8 1345 and 1187. 512 workgroups: 4
// sequences forward in segments of 512 tokens take 125 us, of 256 154, of 1024 146 (backward 351, 425 and 366); 2048 tokens of 16
// heads would take 42 in 128 or 256, 51 in the 64 that this gives. Up to 256 tokens one workgroup's few chunks take less than the
// two launches that a split adds, or as long: 192 tokens of 16 heads 20 us whole and 23 split, 256 24 and 23, 320 28 and 24,
// backward 49 and 44. The backward's segments end at 4096 tokens, since sums over them cancel. Packed, fewer than 1024 workgroups
// are split, since their lengths differ and are not known here.
//
// Packed sequences of 1024 workgroups and more: the forward cuts only those that are longer than their heads' share of the card,
// for two launches that find nothing to do otherwise. 16 heads of 128: a document of 100,000 tokens among 63 of 500 takes 913 us
// so, 9289 whole; 3000 among 63 of 40 86 us and 298; 64 of 100 tokens 83 and 68, 64 of 512 202 and 203. Not below 2048 tokens,
// nor where sequences are shorter than a chunk in the mean, since the workspace has a state for each of them. The backward's
// states are of all segments.
inline AttnPlan attn_plan(int64_t T, int64_t nseq, int64_t units, bool packed, bool backward) {
    AttnPlan p{0, 1, nseq};
    const int64_t rows = packed ? T : nseq * T;
    if (nseq == 0 || T <= 256) return p;
    int64_t seg = (rows * units + 511) / 512;
    seg = (seg + kAttnChunk - 1) / kAttnChunk * kAttnChunk;
    if (packed ? nseq * units >= 1024 && (backward || T <= 2048 || T < kAttnChunk * nseq) : nseq * units >= (backward ? 96 : 192)) seg = T;
    if (backward && seg > 4096) seg = 4096;
    if (seg >= T) return p;
    p.seg = seg;
    p.per_seq = (T + seg - 1) / seg;
    p.slots = packed ? T / seg + nseq : nseq * p.per_seq;
    return p;
}

// Division by a number that the host knows, of numerators below 2^31.
struct Divisor {
    uint32_t d = 1, m = 0, s = 0;
    constexpr Divisor() = default;
    explicit Divisor(int64_t by) : d((uint32_t)by) {
        while ((uint64_t(1) << s) < d) ++s;
        m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
    }
    constexpr uint32_t operator()(uint32_t n) const { return (uint32_t)(((uint64_t)n * m >> 32) + n) >> s; }
};

// Columns of a workgroup of 4 waves: a wave takes 16 or 32 (every column slice forms the scores again). 16 also where the slices
// may be narrower and no more than 256 workgroups come of 32, so that the chip holds two of the others side by side: 77 tokens of
// 16 heads of 128 take 15.2 us so, 19.6 with 32 (fp32 17.9 and 25.9), 256 tokens 24.4 and 31.6 (fp32 37.1 and 56.6). With up to
// 512 workgroups 8192 tokens take 98 us so, 84 with 32.
inline int attn_tiles(int64_t db, int64_t workgroups = INT64_MAX) { return db <= 64 || workgroups <= kComputeUnits ? 1 : 2; }
inline int64_t attn_slices(int64_t db, int tiles) { return (db + 64 * tiles - 1) / (64 * tiles); }
inline int64_t attn_slices(int64_t db) { return attn_slices(db, attn_tiles(db)); }

// Whether the backward's gradients of q, k and v are one launch: where the same kernel takes keys' and values' sizes. A backward
// of 77 tokens of 16 heads of 128 takes 28 us so, 43 in two launches (256 tokens: 42 and 65; four value heads to a key head: 38
// and 52), 16 x 512 tokens 160 and 165, 64 x 512 561 and 585, 4 x 4096 353 and 372, 32 heads of 32,768 tokens 1293 and 1329; fp32
// 34 and 51, 66 and 101, 312 and 325, 1149 and 1205, 765 and 791, 2906 and 2969.
inline bool attn_together(int64_t dk, int64_t dv) { return dv <= 128 && (dv <= 64) == (dk <= 64); }

// Elements that a chunk's n rows of `width` span from column `first` on: what a workgroup may touch from there. None where there
// is no row (a negative number would be a bound without an end).
constexpr int attn_extent(int n, int width, int first) { return n > 0 ? n * width - first : 0; }

// Whether every launch's workgroups can be numbered in 31 bits. Per sequence and value head they are 32 at most: the blocks of a
// 128 x 256 state where segments are joined; a step has 8, a sweep two roles of four column slices for twice the sequences (the last
// segment of each is a part of one). Per token and value head they are an eighth at most: the sums of two value heads' gradients of 128
// channels; a sweep has 8 in 4096 tokens, and with shorter segments some thousand in all. Sweeps round up to eight key heads.
inline bool attn_numbered(int64_t nseq, int64_t B, int64_t T, int64_t Hv) {
    if (nseq > INT32_MAX || B > INT32_MAX || T > INT32_MAX || Hv > INT32_MAX) return false;
    const __int128 units = (__int128)nseq + (__int128)B * (T / 256 + 1) + 8;
    return units * Hv * 32 <= INT32_MAX;
}

// The workspace's parts, in bytes from its beginning.
struct AttnSpace {
    int64_t states, decays;                            // forward; the backward's first pair
    int64_t back, back_decays, ends, last, dq_dot, dk_dot, part, dq, dk;
    int64_t total;
};
inline int64_t attn_whole(int64_t bytes) { return (bytes + 255) / 256 * 256; }
inline AttnSpace attn_space(const AttnPlan &p, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t nseq, int64_t dk, int64_t dv, bool backward) {
    AttnSpace s{};
    int64_t at = 0;
    auto take = [&](int64_t bytes) { const int64_t here = at; at += attn_whole(bytes); return here; };
    const int64_t state = Hv * dk * dv * 4, split = p.seg ? p.slots : 0;
    s.states = take(split * state);
    s.decays = take(split * Hv * 4);
    if (backward) {
        s.back = take(split * state);
        s.back_decays = take(split * Hv * 4);
        s.ends = take(split * Hv * (dk * dv / 1024) * 8);
        s.last = take(nseq * state);
        s.dq_dot = take(B * Hv * T * 4);
        s.dk_dot = take(B * Hv * T * 4);
        s.part = take(p.slots * Hv * 8);
        const int64_t shared = Hk < Hv ? B * Hv * T * dk * 4 : 0;
        s.dq = take(shared);
        s.dk = take(shared);
    }
    s.total = at;
    return s;
}

// ---------------------------------------------------------------- norms of queries and keys

// Tokens of a workgroup, which takes `rows_a_step` rows (a head of a token) at a time: more where four tokens' heads are few steps
// and there are tokens enough.
inline int qk_tokens(int64_t rows, int64_t heads, int rows_a_step) { return heads * 4 < 6 * rows_a_step && rows >= 16384 ? 16 : 4; }
// Steps of a workgroup: all of its tokens' heads, so that their angles are formed once, unless there are too few tokens to
// fill the card so.
inline int64_t qk_steps(int64_t tiles, int64_t all) {
    const int64_t per = (tiles * all + 2047) / 2048;
    return per < 1 ? 1 : per < all ? per : all;
}
// Workgroups of the backward, each of which leaves one row of the weights' gradients: four a compute unit.
inline int64_t qk_groups(int64_t items) { return items < 4 * kComputeUnits ? items : 4 * kComputeUnits; }
inline int64_t qk_bwd_ws_bytes(int64_t rows, int64_t d) { return rows > 0 ? 4 * kComputeUnits * 2 * d * 8 : 0; }

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
