// Linear attention with a decay for each head (gfx950): the chunk form over whole sequences, its gradients, and the
// step of one token.
//
//   H_t = alpha_t H_{t-1} + k_t v_t^T,   o_t = H_t^T q_t
//
// One operator, walked over a sequence in chunks of C tokens with c the sum of log alpha within the chunk:
//
//   A(x, y, z)_i = e^{c_i} H^T x_i + sum_{j <= i} e^{c_i - c_j} (x_i . y_j) z_j,   H <- e^{c_C} H + sum_j y_j (e^{c_C - c_j} z_j)^T
//
// is the forward with (x, y, z) = (q, k, v). Its gradients are the same operator: dq = A(dout, v, k) with the state H^T, and
// run from each sequence's last token with the adjoint state G_t = q_t dout_t^T + alpha_{t+1} G_{t+1}: dv = A(k, q, dout) with
// G, dk = A(v, dout, q) with G^T. Backwards a token's decay applies on the way to the one before it, so that the sums c go up
// to the token before, and nothing else changes. log alpha_t scales all that goes on from t:
//   dlog_alpha_t = sum_{s >= t} (q_s . dq_s - k_s . dk_s) + <the adjoint that enters from behind, H there>,
// with the sum taken to the end of t's segment.
//
// Rounding. q, k, v and dout are matrix operands as they are. What is formed from them and is an operand in turn (the state, the
// scores, the decayed rows) enters as a sum of three bf16 numbers, which is off by 2^-25 of it at most: results whose terms
// cancel are those of fp32 products. Two (2^-17) in the forward and dv took 434 us for 131,072 tokens of 8 heads where three take
// 474, and 490 for 498 in training 4 x 4096 tokens of 16 heads.
//
// What bounds it. A chunk of 64 tokens of a 128 x 128 head is 48 KB in, 16 KB out and 6.3 MFLOP, 15 as executed (in parts). Two
// workgroups of four waves share a compute unit; eight chunks of a forward sweep of 4 x 4096 tokens of 16 heads take the 512 of
// them 170,000 cycles (88 to 101 us), of which the matrix cores are busy 35% and LDS 45%, and the waves wait 34% for memory, LDS
// and barriers and 34% to issue. Without any of the products the same copies and barriers take 52 us (5.8 TB/s). So the long
// sweeps are bound by the order copies, scores, products, state in two waves a SIMD. Eight waves a workgroup (one on a compute
// unit) were slower by a tenth or more, two such workgroups too (registers: 128 a thread spill). The gradients' sweep of 128
// columns takes all 256 registers of its two waves a SIMD and spills 3 to 7 of them (16 to 32 bytes a lane; the next chunk's rows
// and the rows of the products are held over the chunk). That of values of more than 128 channels (x and y are values there)
// leaves one workgroup a compute unit, 106 of its accumulators in AGPRs: the backward of 4 x 4096 tokens of 16 heads takes 668 us
// for values of 160 channels, which are multiplied as 256, 778
// for 256, 383 for 128 (forward 204, 244 and 153).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gdr_kernels.hpp"
#include "gdr_mfma.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

constexpr double kLog2e = 1.4426950408889634074;
constexpr float kLeast = -104.f;  // e^-104 is 0 in fp32: a log decay below it (-infinity too) is this one

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

template <typename E>
constexpr bool is_bf16() { return std::is_same<E, __bf16>::value; }
// tokens of a chunk: fp32 chunks take the same memory
template <typename E>
constexpr int chunk_of() { return is_bf16<E>() ? kAttnChunk : kAttnChunk / 2; }

// ---------------------------------------------------------------- operands

// x as an operand. bf16 tensors: the sum of its bf16 part, the bf16 part of what is left, and that of what is left then.
template <typename E, int N>
struct Parts {
    Frag<E> part[N];
};
template <int N>
__device__ __forceinline__ void split4(floatx4 x, bf16x4 (&part)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        part[i] = cvt4<__bf16>(x);
        if (i + 1 < N) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] -= (float)part[i][e];
        }
    }
}
template <typename E>
constexpr int parts_of(int n) { return is_bf16<E>() ? n : 1; }
template <typename E, int N>
__device__ __forceinline__ Parts<E, N> parts(floatx4 top, floatx4 bottom) {
    Parts<E, N> t;
    if constexpr (is_bf16<E>()) {
        bf16x4 lo[N], hi[N];
        split4(top, lo);
        split4(bottom, hi);
#pragma unroll
        for (int i = 0; i < N; ++i) t.part[i] = Frag<E>{lo[i], hi[i]};
    } else {
        static_assert(N == 1, "fp32 operands are whole");
        t.part[0] = Frag<E>{top, bottom};
    }
    return t;
}

typedef __attribute__((address_space(3))) shortx4 lds_shortx4;
__device__ __forceinline__ bf16x4 tr16(const __bf16 *p) {
    return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4 *)(p)));
}
// An operand whose k index runs down the columns of a row-major matrix: lane (g, c) gets X[k0 + 4g + s] and X[k0 + 16 + 4g + s],
// s = 0..3, at column col0 + step (c / 4) + c % 4. bf16 through the transpose read: in each 16-lane group, lane i receives
// element i % 4 of the 8-byte pieces addressed by lanes 4v + i / 4.
template <typename E>
__device__ __forceinline__ Frag<E> down(const E *X, int ld, int col0, int step, int k0) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    Frag<E> f;
    if constexpr (is_bf16<E>()) {
        const E *p = X + (k0 + 4 * g + (c >> 2)) * ld + col0 + step * (c & 3);
        f.lo = tr16(p);
        f.hi = tr16(p + 16 * ld);
    } else {
        const E *p = X + (k0 + 4 * g) * ld + col0 + step * (c >> 2) + (c & 3);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            f.lo[s] = p[s * ld];
            f.hi[s] = p[(16 + s) * ld];
        }
    }
    return f;
}

typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
typedef unsigned uintx2 __attribute__((ext_vector_type(2)));

// A chunk's rows in memory: what is read past its bytes is zero, what is written there is dropped. p and bytes are the same in
// every lane.
typedef __amdgpu_buffer_rsrc_t Rows;
__device__ __forceinline__ Rows rows_at(const void *p, int bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)u), hi = (unsigned)__builtin_amdgcn_readfirstlane((int)(unsigned)(u >> 32));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(hi << 32 | lo), 0, __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
constexpr int kNowhere = 0x40000000;  // an offset past every chunk
// Results are stored past the caches' keeping, which leaves them to k and v, read again by the next launch: 4 x 4096 tokens of 16
// heads train in 471 us so, 474 without; 131,072 tokens forward take 458 us either way.
constexpr int kPast = 2;
// N elements of a row from a byte offset on
template <typename E, int N>
struct Piece {
    typename Vec4<E>::type v[N / 4];
};
template <typename E, int N>
__device__ __forceinline__ Piece<E, N> read_piece(Rows r, int off) {
    Piece<E, N> p;
    if constexpr (sizeof(p) == 8) {
        p = __builtin_bit_cast(Piece<E, N>, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    } else {
        struct U {
            uintx4 u[sizeof(p) / 16];
        } u;
#pragma unroll
        for (int i = 0; i < (int)sizeof(p) / 16; ++i) u.u[i] = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0);
        p = __builtin_bit_cast(Piece<E, N>, u);
    }
    return p;
}
template <typename E, int N>
__device__ __forceinline__ void write_piece(const Piece<E, N> &p, Rows r, int off) {
    if constexpr (sizeof(p) == 8) {
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2, p), r, off, 0, kPast);
    } else {
        struct U {
            uintx4 u[sizeof(p) / 16];
        };
        const U u = __builtin_bit_cast(U, p);
#pragma unroll
        for (int i = 0; i < (int)sizeof(p) / 16; ++i) __builtin_amdgcn_raw_buffer_store_b128(u.u[i], r, off + 16 * i, 0, kPast);
    }
}

// whether a 16-byte piece holds infinity or NaN (every exponent bit set)
template <typename E>
__device__ __forceinline__ unsigned odd_bits(uintx4 u) {
    unsigned r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r |= is_bf16<E>() ? ((u[i] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u : ((u[i] & 0x7fffffffu) + 0x00800000u) & 0x80000000u;
    return r;
}
__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) < __builtin_inff(); }

// ---------------------------------------------------------------- where a workgroup works

struct Span {
    int seq, row, t0;   // sequence, its batch row and first token there
    int lo, hi, len;    // the segment's tokens, of the sequence's len
    int slot;
    bool some;          // the slot is one of the sequence's
    __device__ __forceinline__ bool first() const { return lo == 0; }
    __device__ __forceinline__ bool last() const { return hi >= len; }
};
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// The last of n sequences whose key is not past `at` (the first one if all are), by all lanes of a wave at once.
template <typename Key>
__device__ __forceinline__ unsigned last_up_to(unsigned at, unsigned n, Key key) {
    const unsigned lane = threadIdx.x & 63;
    unsigned lo = 0;
    while (n > 1) {
        const unsigned step = (n + 63) / 64, on = lane * step;
        const unsigned m = (unsigned)__popcll(__ballot(on < n && key(lo + on) <= at)), skip = m > 1 ? (m - 1) * step : 0;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    return (unsigned)uniform((int)lo);
}

// Slots are segments of a.seg tokens; without a split (a.seg 0) slots are sequences. Packed: the segments of sequence s begin at
// slot cu[s] / seg + s. Cuts are where a segment ends and its sequence goes on: those of sequence s begin at cut cu[s] / seg (s
// (per_seq - 1) if not packed), so that cut i of sequence s lies behind slot i + s. With `cut`, the segment before a cut is asked
// for. Boundaries are held inside the row whatever cu_seqlens has.
__device__ __forceinline__ Span span_of(const AttnArgs &a, unsigned slot, bool cut = false) {
    Span p;
    const unsigned seg = (unsigned)a.seg;
    const int T = (int)a.T;
    int from = 0, end = T;
    unsigned piece = 0;
    p.slot = (int)slot;
    if (!a.cu) {
        const Divisor &by = cut ? a.by_cuts : a.by_per;  // (one segment a sequence without a split)
        const unsigned s = by(slot);
        p.seq = p.row = (int)s;
        piece = slot - s * by.d;
    } else {
        unsigned s = slot;
        if (seg) {
            // whose first slot or cut is not past this one
            s = last_up_to(slot, (unsigned)a.nseq, [&](unsigned i) { return a.by_seg((unsigned)a.cu[i]) + (cut ? 0 : i); });
            piece = slot - (a.by_seg((unsigned)uniform(a.cu[s])) + (cut ? 0 : s));
        }
        p.seq = (int)s;
        p.row = 0;
        from = uniform(a.cu[s]);
        from = from < 0 ? 0 : from > T ? T : from;
        end = uniform(a.cu[s + 1]);
        end = end < from ? from : end > T ? T : end;
    }
    if (cut) p.slot += p.seq;
    p.t0 = from;
    p.len = end - from;
    const int64_t lo = (int64_t)piece * seg;
    p.some = cut ? lo + seg < p.len : piece == 0 || lo < p.len;
    p.lo = p.some ? (int)lo : 0;
    p.hi = seg && (int64_t)p.lo + seg < p.len ? p.lo + (int)seg : p.len;
    return p;
}

// ---------------------------------------------------------------- the sweep

// tables of a chunk, by position in walking order (a token each): the log2 decay c, e^c and e^{total - c}
template <int C>
struct Gates {
    double c[C];
    double sum;  // log2 of total
    float total;
    float pad;
    float in[C], on[C];
};

template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double v) {  // v of the lane that the control names, 0 where there is none
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, kCtrl, kRows, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), kCtrl, kRows, 0xf, false);
    return __builtin_bit_cast(double, (uint64_t)(unsigned)hi << 32 | (unsigned)lo);
}
__device__ __forceinline__ double from_lane(double v, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)u, lane), hi = (unsigned)__builtin_amdgcn_readlane((int)(unsigned)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// the sums over the lanes up to each one: within rows of 16, then the rows before
__device__ __forceinline__ double lane_sums(double v) {
    v += moved<0x111, 0xf>(v);  // from 1, 2, 4 and 8 lanes before
    v += moved<0x112, 0xf>(v);
    v += moved<0x114, 0xf>(v);
    v += moved<0x118, 0xf>(v);
    v += moved<0x142, 0xa>(v);  // a row's last lane to the next row, for rows 1 and 3
    v += moved<0x143, 0xc>(v);  // lane 31's to rows 2 and 3
    return v;
}
// by one wave, lane = position; la: the token's log decay
template <int C>
__device__ __forceinline__ void make_gates(Gates<C> *t, float la, int n, bool reverse) {
    const int lane = threadIdx.x & 63;
    const double own = lane < n ? (double)(la < kLeast ? kLeast : la) * kLog2e : 0.;
    const double v = lane_sums(own), total = from_lane(v, C - 1);
    const double c = reverse ? moved<0x138, 0xf>(v) : v;  // (backwards up to the token before, whatever this one's decay is)
    if (lane < C) {
        t->c[lane] = c;
        t->in[lane] = ex2((float)c);
        t->on[lane] = ex2((float)(total - c));
    }
    if (lane == 0) {
        t->sum = total;
        t->total = ex2((float)total);
    }
}

// What a sweep leaves: the segments' states; the results; or the results and their rows' products with another tensor's rows, the
// results in fp32 where they are shares of a key head's (of some roles, in the mixed form).
enum Form { kStates, kResults, kProducts, kShares, kMixed };

template <typename E, int DA, int NT, int NW, Form F>
struct Shape {
    static constexpr bool OUT = F != kStates, kDots = F == kProducts || F == kShares || F == kMixed;
    static constexpr int C = chunk_of<E>();
    static constexpr int NB = 16 * NT * NW;                     // columns of a workgroup
    static constexpr int kPad = 16 / sizeof(E);
    static constexpr int LA = DA + kPad, LB = NB + kPad, LP = C + 4;
    static constexpr int kPlanes = parts_of<E>(3);              // parts of the state and the scores as operands
    struct Lds {
        E y[C * LA];
        E z[C * LB];
        E x[OUT ? C * LA : 8];
        E p[OUT ? kPlanes * C * LP : 8];
        Gates<C> gates[2];
        unsigned odd[NW];
        // each wave's part of a row's product lies in the padding of x's and y's rows
        __device__ __forceinline__ float *dot(int w, int i) { return reinterpret_cast<float *>((w < 4 ? x : y) + i * LA + DA) + w % 4; }
    };
};

// One workgroup walks one segment of one value head for NB columns of z. The states form leaves the segment's own state (from
// zero) and total decay; the others begin from the entering state and write A(x, y, z).
//
// A wave holds 16 NT columns of the state in registers, [DA][16 NT] in the accumulators' layout, which as it stands is the
// operand of H^T x: the state never leaves the registers. Scores are shared out over the waves by tiles and go through LDS.
// The next chunk's rows are loaded into registers while this one is multiplied. Rows and columns past the tensors' are zeros.
template <typename E, int DA, int NT, int NW, Form F>
__global__ __launch_bounds__(NW * 64, DA > 128 ? 1 : NW / 2) void sweep_kernel(AttnArgs a, int first_role, unsigned nouter) {
    typedef Shape<E, DA, NT, NW, F> S;
    constexpr bool OUT = S::OUT, kDots = S::kDots;
    constexpr int C = S::C, LA = S::LA, LB = S::LB, LP = S::LP, kThreads = NW * 64;
    constexpr int TI = C / 16, TA = DA / 16, KS = C / 32;       // token tiles, state tiles, 32-deep steps over the tokens
    constexpr int kElems = 16 / sizeof(E), es = (int)sizeof(E);  // of a 16-byte piece
    constexpr int PA = DA / kElems, PB = S::NB / kElems;        // pieces of a row
    constexpr int RA = kThreads / PA, RB = kThreads / PB;       // rows that the threads' pieces cover
    constexpr int NA = C / RA, NZ = C / RB;
    constexpr int N = S::kPlanes;
    static_assert(kThreads % PA == 0 && kThreads % PB == 0 && C % RA == 0 && C % RB == 0, "pieces are shared out evenly");
    __shared__ __align__(16) typename S::Lds m;

    // what reads the same rows goes to one XCD (workgroups go round them in turn): roles, column slices, heads of a key head
    const unsigned Hk = (unsigned)a.Hk, Hv = (unsigned)a.Hv, id = (unsigned)block_id(), at = id / 8, round = a.by_inner(at), outer = round * 8 + id % 8;
    if (outer >= nouter) return;
    const unsigned in = at - round * a.by_inner.d, unit = a.by_roles(in), member = a.by_slices(unit), slot = a.by_Hk(outer);
    const AttnRole &r = a.roles[first_role + (in - unit * a.by_roles.d)];
    const unsigned slice = unit - member * a.by_slices.d, kh = outer - slot * Hk, head = kh * a.group + member;
    const Span sp = span_of(a, slot, !OUT && r.cuts);
    if (!sp.some) return;

    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int wave = uniform(tid >> 6);
    const int da = r.da, db = r.db, col0 = (int)slice * S::NB, left = db - col0;  // left: columns from this workgroup's first on
    const int wcol = 16 * NT * wave;
    const bool active = wcol < left;                            // (db is a multiple of a wave's columns)
    const bool reverse = r.reverse, dots = kDots;
    auto slab = [&](const void *p, bool key, int d) {
        const int64_t h = key ? kh : head, H = key ? Hk : Hv;
        return reinterpret_cast<const char *>(p) + ((sp.row * H + h) * a.T + sp.t0 + sp.lo) * d * es;
    };
    const char *gx = OUT ? slab(r.x, r.xk, da) : nullptr, *gy = slab(r.y, r.yk, da), *gz = slab(r.z, r.zk, db) + col0 * es;
    const char *go = dots ? slab(r.other, r.ok, db) + col0 * es : nullptr;
    const int64_t scalars = (sp.row * (int64_t)Hv + head) * a.T + sp.t0 + sp.lo;
    typedef typename std::conditional<F == kShares, float, E>::type R;  // of the results, unless shares of the mixed form
    const int osize = F == kMixed && r.shares ? 4 : (int)sizeof(R);
    char *out = OUT ? reinterpret_cast<char *>(r.out) + (scalars * db + col0) * osize : nullptr;
    const int len = sp.hi - sp.lo, nch = (len + C - 1) / C;

    // chunk k in walking order: its first token (in the segment) and how many it has; the token at a position p of a chunk of n
    // is turn p + from
    auto first_token = [&](int k) { return (reverse ? nch - 1 - k : k) * C; };
    auto count = [&](int k) { return k >= nch ? 0 : len - first_token(k) < C ? len - first_token(k) : C; };
    const int turn = reverse ? -1 : 1;
    auto from = [&](int n) { return reverse ? n - 1 : 0; };

    // this thread's pieces: of every RA-th row of x and y and every RB-th of z
    const int row_a = tid / PA, col_a = tid % PA * kElems, row_b = tid / PB, col_b = tid % PB * kElems;
    const int off_a = col_a < da ? (turn * row_a * da + col_a) * es : kNowhere, off_b = col_b < left ? (turn * row_b * db + col_b) * es : kNowhere;
    uintx4 rx[NA], ry[NA], rz[NZ];
    auto load = [&](int k) {
        const int64_t t = first_token(k);
        const int n = count(k);
        const Rows py = rows_at(gy + t * (da * es), attn_extent(n, da, 0) * es), pz = rows_at(gz + t * (db * es), attn_extent(n, db, col0) * es);
        const Rows px = OUT ? rows_at(gx + t * (da * es), attn_extent(n, da, 0) * es) : py;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int off = off_a + (from(n) + turn * i * RA) * da * es;
            if (OUT) rx[i] = __builtin_amdgcn_raw_buffer_load_b128(px, off, 0, 0);
            ry[i] = __builtin_amdgcn_raw_buffer_load_b128(py, off, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) rz[i] = __builtin_amdgcn_raw_buffer_load_b128(pz, off_b + (from(n) + turn * i * RB) * db * es, 0, 0);
    };
    float la = 0.f;
    auto load_decay = [&](int k) {
        if (wave == 0 && k < nch) {
            const int n = count(k);
            la = 0.f;
            if (lane < n) la = a.la_token ? a.la[scalars + first_token(k) + from(n) + turn * lane] : a.la[head];
        }
    };
    if (nch > 0) {
        load_decay(0);
        load(0);
    }

    // column of this lane in tile nt of its wave's columns: the tiles alternate by fours, so that a lane's results of all of
    // them are neighbours
    constexpr int kStep = 4 * NT;
    const int lcol = wcol + kStep * (c >> 2) + (c & 3);

    // the state, and its element at (16 t + 4 g, this lane's column) of the stored [da][db] or [db][da]
    floatx4 h[TA][NT];
#pragma unroll
    for (int t = 0; t < TA; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n) h[t][n] = zero4();
    // (of a sequence that is cut the first one too: its last one may write over the state that the sequence begins with)
    const bool of_cut = OUT && r.cuts && !(sp.first() && sp.last());
    const float *s_in = of_cut ? r.s_cuts : r.s_in;
    if (OUT && s_in && active) {
        const float *p = s_in + ((int64_t)(of_cut || r.in_slots ? sp.slot : sp.seq) * Hv + head) * da * db;
        if (of_cut || r.in_turned) {
#pragma unroll
            for (int t = 0; t < TA; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int row = 16 * t < da ? 16 * t + 4 * g : 0;  // (rows past da are zeroed below)
                    h[t][n] = *reinterpret_cast<const floatx4 *>(p + (unsigned)((col0 + lcol + 4 * n) * da + row));
                }
        } else {
#pragma unroll
            for (int t = 0; t < TA; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 16 * t < da ? 16 * t + 4 * g + e : 0;
                        h[t][n][e] = p[(unsigned)(row * db + col0 + lcol + 4 * n)];
                    }
        }
#pragma unroll
        for (int t = 0; t < TA; ++t)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (16 * t >= da) h[t][n] = zero4();
    }

    if (OUT) {  // the score tiles above the diagonal that a 32-deep step covers stay zero
        static_assert(C * LP % kElems == 0, "planes are whole pieces");
        for (int i = tid; i < N * C * LP / kElems; i += kThreads) *reinterpret_cast<uintx4 *>(&m.p[i * kElems]) = uintx4{0, 0, 0, 0};
    }
    const bool ends = OUT && r.s_out && (reverse ? sp.first() : sp.last());  // the sequence ends here, and its state is wanted
    double decay = 0.;  // the segment's total, of the states form
    if (nch > 0) {
        if (wave == 0) make_gates<C>(&m.gates[0], la, count(0), reverse);
        load_decay(1);
    }
    auto put_dots = [&](int k) {
        const int n = count(k);
        if (kDots && r.dot && tid < n) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) s += *m.dot(w, tid);
            r.dot[scalars + first_token(k) + from(n) + turn * tid] = s;
        }
    };
    auto store_rows = [&]() {
        unsigned odd = 0;
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int off = (row_a + i * RA) * LA + col_a;
            if (OUT) *reinterpret_cast<uintx4 *>(&m.x[off]) = rx[i];
            *reinterpret_cast<uintx4 *>(&m.y[off]) = ry[i];
        }
#pragma unroll
        for (int i = 0; i < NZ; ++i) {
            *reinterpret_cast<uintx4 *>(&m.z[(row_b + i * RB) * LB + col_b]) = rz[i];
            if (OUT) odd |= odd_bits<E>(rz[i]);
        }
        if (OUT) {
            const bool any = __ballot(odd != 0) != 0;
            if (lane == 0) m.odd[wave] = any;
        }
    };
    if (nch > 0) store_rows();

    // Memory operations end in order, stores too: the next chunk's loads are asked for before this one's results are stored, in
    // the same round of the loop, so that the wait for them leaves the stores in flight.
    for (int k = 0; k < nch; ++k) {
        const Gates<C> &gt = m.gates[k & 1];
        const int64_t t0 = first_token(k);
        const int n = count(k);
        __syncthreads();
        if (wave == 0 && k + 1 < nch) {
            make_gates<C>(&m.gates[(k + 1) & 1], la, count(k + 1), reverse);
            load_decay(k + 2);
        }
        int off[TI];
#pragma unroll
        for (int ti = 0; ti < TI; ++ti) off[ti] = active ? (from(n) + turn * (16 * ti + c)) * db + wcol + kStep * g : kNowhere / 4;
        Piece<E, 4 * NT> w[kDots ? TI : 1];
        if (dots) {  // the rows that the results are multiplied with
            const Rows po = rows_at(go + t0 * (db * es), attn_extent(n, db, col0) * es);
#pragma unroll
            for (int ti = 0; ti < TI; ++ti) w[ti] = read_piece<E, 4 * NT>(po, off[ti] * es);
        }
        load(k + 1);
        const float total = gt.total;
        Frag<E> z[KS][NT];
        auto load_z = [&]() {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) z[ks][nt] = down<E>(m.z, LB, wcol + 4 * nt, kStep, 32 * ks);
        };

        if constexpr (OUT) {
            // scores of tile (ti, tj), transposed: lane (g, c) holds those of token 16 ti + c with 16 tj + 4g + e
            constexpr int kTiles = TI * (TI + 1) / 2, kPer = (kTiles + NW - 1) / NW;  // of a wave: every NW-th
            int ti_[kPer], tj_[kPer];
            floatx4 s[kPer];
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int t = wave + q * NW < kTiles ? wave + q * NW : kTiles - 1;
                ti_[q] = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
                tj_[q] = t - ti_[q] * (ti_[q] + 1) / 2;
                s[q] = zero4();
            }
#pragma unroll
            for (int ks = 0; ks < DA / 32; ++ks)
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    s[q] = mma32(s[q], frag_rows<E>(m.y, LA, 16 * tj_[q], 32 * ks), frag_rows<E>(m.x, LA, 16 * ti_[q], 32 * ks));
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int i = 16 * ti_[q] + c, j = 16 * tj_[q] + 4 * g;
                const double ci = gt.c[i];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float v = s[q][e] * ex2((float)(ci - gt.c[j + e]));
                    asm("" : "+v"(v));  // a select, not a branch round the exponential
                    s[q][e] = j + e <= i ? v : 0.f;
                }
            }
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                E *p = m.p + (16 * ti_[q] + c) * LP + 16 * tj_[q] + 4 * g;
                if constexpr (is_bf16<E>()) {
                    bf16x4 part[N];
                    split4(s[q], part);
                    if (wave + q * NW < kTiles) {
#pragma unroll
                        for (int w = 0; w < N; ++w) *reinterpret_cast<bf16x4 *>(p + w * C * LP) = part[w];
                    }
                } else {
                    if (wave + q * NW < kTiles) *reinterpret_cast<floatx4 *>(p) = s[q];
                }
            }
            // e^c H^T x. Products go before the other workgroup's copies and scores: training 471 us so, 479
            // without, 131,072 tokens forward 458 and 471.
            __builtin_amdgcn_s_setprio(1);
            floatx4 o[TI][NT];
#pragma unroll
            for (int ti = 0; ti < TI; ++ti)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) o[ti][nt] = zero4();
#pragma unroll
            for (int ks = 0; ks < DA / 32; ++ks) {
                Parts<E, N> hs[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) hs[nt] = parts<E, N>(h[2 * ks][nt], h[2 * ks + 1][nt]);
#pragma unroll
                for (int ti = 0; ti < TI; ++ti) {
                    const Frag<E> x = frag_rows<E>(m.x, LA, 16 * ti, 32 * ks);
#pragma unroll
                    for (int q = N - 1; q >= 0; --q)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) o[ti][nt] = mma32(o[ti][nt], hs[nt].part[q], x);
                }
            }
#pragma unroll
            for (int ti = 0; ti < TI; ++ti) {
                const float e = gt.in[16 * ti + c];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) o[ti][nt] *= e;
            }
            __syncthreads();
            load_z();
            unsigned bad = 0;
#pragma unroll
            for (int q = 0; q < NW; ++q) bad |= m.odd[q];
            bad = uniform(bad);
            if (__builtin_expect(bad != 0, 0)) {
                // Infinities and NaN in z must not meet the zero scores of tokens before theirs: they are taken out of the
                // product and added pair by pair.
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (!finite((float)z[ks][nt].lo[e])) z[ks][nt].lo[e] = (E)0.f;
                            if (!finite((float)z[ks][nt].hi[e])) z[ks][nt].hi[e] = (E)0.f;
                        }
#pragma unroll
                for (int ti = 0; ti < TI; ++ti) {
#pragma unroll 1
                    for (int j = 0; j <= 16 * ti + c; ++j) {
                        float p = 0.f;
#pragma unroll
                        for (int q = N - 1; q >= 0; --q) p += (float)m.p[(q * C + 16 * ti + c) * LP + j];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float zj = (float)m.z[j * LB + wcol + kStep * g + 4 * nt + e];
                                if (!finite(zj)) o[ti][nt][e] += p * zj;
                            }
                    }
                }
            }
#pragma unroll
            for (int ti = 0; ti < TI; ++ti)
#pragma unroll
                for (int ks = 0; ks <= ti / 2; ++ks)
#pragma unroll
                    for (int q = N - 1; q >= 0; --q) {
                        const Frag<E> p = frag_rows<E>(m.p + q * C * LP, LP, 16 * ti, 32 * ks);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) o[ti][nt] = mma32(o[ti][nt], z[ks][nt], p);
                    }
            if (__builtin_expect(bad != 0, 0)) load_z();
            __builtin_amdgcn_s_setprio(0);
            const Rows to = rows_at(out + t0 * (db * osize), attn_extent(n, db, col0) * osize);
            auto put_rows = [&](auto like) {
                typedef decltype(like) P;
#pragma unroll
                for (int ti = 0; ti < TI; ++ti) {
                    Piece<P, 4 * NT> p;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) p.v[nt] = cvt4<P>(o[ti][nt]);
                    write_piece(p, to, off[ti] * (int)sizeof(P));
                }
            };
            if (F == kMixed && r.shares) put_rows(float{});
            else put_rows(R{});
            if (dots) {
#pragma unroll
                for (int ti = 0; ti < TI; ++ti) {
                    float dot = 0.f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) dot += (float)w[ti].v[nt][e] * o[ti][nt][e];
                    dot += __shfl_xor(dot, 16, 64);
                    dot += __shfl_xor(dot, 32, 64);
                    if (g == 0) *m.dot(wave, 16 * ti + c) = dot;
                }
            }
        } else {
            load_z();
        }
        // the state, unless nothing reads it any more
        if (!OUT || k + 1 < nch || ends) {
#pragma unroll
            for (int t = 0; t < TA; ++t)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) h[t][nt] *= total;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const floatx4 lo = *reinterpret_cast<const floatx4 *>(&gt.on[32 * ks + 4 * g]);
                const floatx4 hi = *reinterpret_cast<const floatx4 *>(&gt.on[32 * ks + 16 + 4 * g]);
                Parts<E, N> zs[NT];  // z decayed to the chunk's end
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    floatx4 zl, zh;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        zl[e] = (float)z[ks][nt].lo[e] * lo[e];
                        zh[e] = (float)z[ks][nt].hi[e] * hi[e];
                    }
                    zs[nt] = parts<E, N>(zl, zh);
                }
#pragma unroll
                for (int t = 0; t < TA; ++t) {
                    const Frag<E> y = down<E>(m.y, LA, 16 * t, 4, 32 * ks);
#pragma unroll
                    for (int q = N - 1; q >= 0; --q)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) h[t][nt] = mma32(h[t][nt], y, zs[nt].part[q]);
                }
            }
        }
        if (!OUT) decay += gt.sum;
        __syncthreads();
        if (dots) put_dots(k);
        store_rows();
    }
    if (active && (OUT ? ends : r.s_out != nullptr)) {
        float *p = r.s_out + ((int64_t)(OUT ? sp.seq : sp.slot) * Hv + head) * da * db;
#pragma unroll
        for (int t = 0; t < TA; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int row = 16 * t + 4 * g, col = col0 + lcol + 4 * nt;
                if (16 * t < da) {
                    if (r.out_turned) {
                        *reinterpret_cast<floatx4 *>(p + (unsigned)(col * da + row)) = h[t][nt];
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[(unsigned)((row + e) * db + col)] = h[t][nt][e];
                    }
                }
            }
    }
    if (!OUT && r.decay && slice == 0 && tid == 0) r.decay[(int64_t)sp.slot * Hv + head] = ex2((float)decay);
}

// ---------------------------------------------------------------- states between segments

// The sum over a workgroup of 256 threads, for every thread.
__device__ __forceinline__ double sum_all(double v, double *held) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) held[threadIdx.x >> 6] = v;
    __syncthreads();
    return held[0] + held[1] + held[2] + held[3];
}

// Four elements of one head's state a thread: each segment's own state is replaced by the one that enters it. States are
// [rows][cols] here, init and last the same or, turned, [cols][rows]. With `ends` (backwards, behind the forward's states), each
// workgroup leaves its part of <the adjoint that enters segment i from behind, the state there>, which enters segment i + 1. With
// `cuts`, packed sequences of one segment are left out (a sequence's first cut names the workgroup).
struct Join {
    float *states;
    const float *decays, *init;
    float *last;
    const float *other, *other_last;
    double *ends;  // [slots][Hv][blocks of a state]
    int rows, cols;
    bool turned, reverse, cuts;
};
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, Join j) {
    __shared__ double held[4];
    const int64_t elems = (int64_t)j.rows * j.cols;
    const unsigned blocks = (unsigned)(elems / 1024), id = (unsigned)block_id(), unit = id / blocks, block = id % blocks;
    const unsigned which = unit / (unsigned)a.Hv, head = unit % (unsigned)a.Hv;
    if (which >= (j.cuts && a.cu ? a.cuts : a.nseq)) return;
    const int64_t e = block * 1024 + threadIdx.x * 4;
    unsigned seq = which;
    int first = (int)(which * a.per_seq), n = (int)a.per_seq;
    if (j.cuts && a.cu) {
        const Span sp = span_of(a, which, true);
        if (!sp.some || !sp.first()) return;
        seq = (unsigned)sp.seq;
        first = sp.slot;
        n = (sp.len - 1) / (int)a.seg + 1;
        if ((int64_t)first + n > a.slots) return;  // boundaries that are none
    } else if (a.cu) {
        const int from = a.cu[seq], len = a.cu[seq + 1] - from;
        first = (int)(a.by_seg((unsigned)from) + seq);
        n = len > a.seg ? (int)((len + a.seg - 1) / a.seg) : 1;
        if (first < 0 || (int64_t)first + n > a.slots) return;  // boundaries that are none
    }
    const int row = (int)(e / j.cols), col = (int)(e % j.cols);
    const int64_t at = ((int64_t)seq * a.Hv + head) * elems;
    auto outside = [&](int i) { return at + (j.turned ? (int64_t)(col + i) * j.rows + row : e + i); };
    floatx4 h = zero4();
    if (j.init) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = j.init[outside(i)];
    }
    constexpr int kAhead = 4;
    for (int i = 0; i < n; i += kAhead) {
        floatx4 s[kAhead], x[kAhead];
        float d[kAhead];
        auto slot = [&](int p) { return (int64_t)(j.reverse ? first + n - 1 - p : first + p); };
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            s[p] = x[p] = zero4();
            d[p] = 0.f;
            if (i + p + 1 < n || (i + p < n && j.last)) {
                s[p] = *reinterpret_cast<const floatx4 *>(j.states + (slot(i + p) * a.Hv + head) * elems + e);
                d[p] = j.decays[slot(i + p) * a.Hv + head];
            }
            if (j.ends && i + p < n) {
                if (i + p > 0) x[p] = *reinterpret_cast<const floatx4 *>(j.other + ((slot(i + p) + 1) * a.Hv + head) * elems + e);
                else if (j.other_last) x[p] = *reinterpret_cast<const floatx4 *>(j.other_last + at + e);
            }
        }
#pragma unroll
        for (int p = 0; p < kAhead; ++p)
            if (i + p < n) {
                if (j.ends) {
                    double v = 0.;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v += (double)h[q] * x[p][q];
                    v = sum_all(v, held);
                    if (threadIdx.x == 0) j.ends[(slot(i + p) * a.Hv + head) * blocks + block] = v;
                }
                *reinterpret_cast<floatx4 *>(j.states + (slot(i + p) * a.Hv + head) * elems + e) = h;
                h = d[p] * h + s[p];
            }
    }
    if (j.last) {
#pragma unroll
        for (int i = 0; i < 4; ++i) j.last[outside(i)] = h[i];
    }
}

// ---------------------------------------------------------------- the decays' gradient

struct DecayGrad {
    const double *ends;          // what enters each segment from behind, in parts (with a split)
    const float *last, *dhT;     // the same without: the final states and their gradients, by sequence (dhT null: zero)
    const float *dq_dot, *dk_dot;
    float *dla;                  // [B][Hv][T]
    double *part;                // [slots][Hv]: the slot's sum, where a head has one decay
    int elems;
    // for tokens that are not finite: the inputs, and the states that enter the segments (with a split by slot) from both sides
    const void *q, *k, *v, *dout;
    const float *before, *behind;
    int dk, dv;
    bool split;
};

template <typename E>
__device__ __forceinline__ bool finite_row(const E *p, int n) {
    bool all = true;
    for (int i = 0; i < n; ++i) all = all && finite((float)p[i]);
    return all;
}

// The gradient at the segment's first token whose key or value is not finite: alpha_t <G_t, H_{t-1}>, where neither G nor H holds
// that token's key and value, from the recurrences themselves. Returns the token, or -1 where there is none, or where a query or
// an output's gradient from it on is not finite either, which every token up to it holds.
template <typename E>
__device__ __forceinline__ int first_bad(const AttnArgs &a, const DecayGrad &d, const Span &sp, unsigned head, double *held, double &grad) {
    __shared__ int bounds[2];
    const int tid = threadIdx.x;
    const unsigned kh = head / a.group;
    const int64_t keys = (sp.row * a.Hk + kh) * a.T + sp.t0, values = (sp.row * a.Hv + head) * a.T + sp.t0;
    const E *q = reinterpret_cast<const E *>(d.q) + keys * d.dk, *k = reinterpret_cast<const E *>(d.k) + keys * d.dk;
    const E *v = reinterpret_cast<const E *>(d.v) + values * d.dv, *dout = reinterpret_cast<const E *>(d.dout) + values * d.dv;
    if (tid == 0) {
        bounds[0] = sp.hi;
        bounds[1] = -1;
    }
    __syncthreads();
    int first = sp.hi, last = -1;
    for (int t = sp.lo + tid; t < sp.hi; t += 256) {
        const int64_t tk = (int64_t)t * d.dk, tv = (int64_t)t * d.dv;
        if (first == sp.hi && !(finite_row(k + tk, d.dk) && finite_row(v + tv, d.dv))) first = t;
        if (!(finite_row(q + tk, d.dk) && finite_row(dout + tv, d.dv))) last = t;
    }
    if (first < sp.hi) atomicMin(&bounds[0], first);
    if (last >= 0) atomicMax(&bounds[1], last);
    __syncthreads();
    const int bad = bounds[0];
    if (bad == sp.hi || bounds[1] >= bad) return -1;
    auto alpha = [&](int t) {
        const float la = a.la_token ? a.la[values + t] : a.la[head];
        return ex2((float)((double)(la < kLeast ? kLeast : la) * kLog2e));
    };
    const int64_t from = (int64_t)(d.split ? sp.slot : sp.seq) * a.Hv + head;
    double sum = 0.;
    for (int e = tid; e < d.elems; e += 256) {
        const int r = e / d.dv, c = e % d.dv;
        float h = d.before ? d.before[from * d.elems + e] : 0.f, g = d.behind ? d.behind[from * d.elems + e] : 0.f;
        for (int t = sp.lo; t < bad; ++t) h = alpha(t) * h + (float)k[(int64_t)t * d.dk + r] * (float)v[(int64_t)t * d.dv + c];
        for (int t = sp.hi - 1; t > bad; --t) g = alpha(t) * (g + (float)q[(int64_t)t * d.dk + r] * (float)dout[(int64_t)t * d.dv + c]);
        g += (float)q[(int64_t)bad * d.dk + r] * (float)dout[(int64_t)bad * d.dv + c];
        sum += (double)g * h;
    }
    grad = alpha(bad) * sum_all(sum, held);
    return bad;
}

// A workgroup takes a segment of a head. The sums run over up to thousands of tokens and cancel: they are held in 64 bits. A
// decay of nothing left has no gradient, whatever the sums leave of theirs. The sums hold each later token's q . dq and k . dk,
// where a bad key or value would reach all earlier tokens, which do not depend on it: such a segment's are taken again up to there.
template <typename E>
__global__ __launch_bounds__(256) void decay_grad_kernel(AttnArgs a, DecayGrad d) {
    __shared__ double held[4], waves[4];
    const unsigned id = (unsigned)block_id(), slot = id / (unsigned)a.Hv, head = id % (unsigned)a.Hv;
    if (slot >= a.slots) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Span sp = span_of(a, slot);
    double sum = 0.;
    if (sp.some) {
        double carry = 0.;
        if (d.ends) {
            const int blocks = d.elems / 1024;
            for (int i = 0; i < blocks; ++i) carry += d.ends[((int64_t)slot * a.Hv + head) * blocks + i];
        } else if (d.dhT) {
            const int64_t at = ((int64_t)sp.seq * a.Hv + head) * d.elems;
            for (int e = tid * 4; e < d.elems; e += 1024) {
                const floatx4 x = *reinterpret_cast<const floatx4 *>(d.last + at + e), y = *reinterpret_cast<const floatx4 *>(d.dhT + at + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) carry += (double)x[i] * y[i];
            }
            carry = sum_all(carry, held);
        }
        const int64_t base = ((int64_t)sp.row * a.Hv + head) * a.T + sp.t0;
        // the tokens before `end`, behind which the sum is `carry`; whether all sums were finite
        auto walk = [&](int end, double carry) {
            bool fine = true;
            for (; end > sp.lo; end -= 256) {
                const int t = end - 1 - tid;  // thread 0 has the last token
                const float la = t < sp.lo ? 0.f : a.la_token ? a.la[base + t] : a.la[head];
                double v = lane_sums(t >= sp.lo ? (double)d.dq_dot[base + t] - (double)d.dk_dot[base + t] : 0.);
                __syncthreads();
                if (lane == 63) waves[wave] = v;
                __syncthreads();
                v += carry;
                for (int w = 0; w < wave; ++w) v += waves[w];
                carry += waves[0] + waves[1] + waves[2] + waves[3];
                if (t >= sp.lo) {
                    fine = fine && finite((float)v);
                    if (la <= kLeast) v *= 0.;
                    if (a.la_token) d.dla[base + t] = (float)v;
                    else sum += v;
                }
            }
            return fine;
        };
        if (__builtin_expect(__syncthreads_or(!walk(sp.hi, carry)), 0)) {
            double grad;
            const int bad = first_bad<E>(a, d, sp, head, held, grad);
            if (bad >= 0) {
                if (a.la_token) {
                    if (tid == 0) d.dla[base + bad] = (float)grad;
                } else {
                    sum = tid ? 0. : bad + 1 < sp.hi ? __builtin_nan("") : grad;  // (tokens behind it hold it)
                }
                walk(bad, grad);
            }
        }
    }
    if (!a.la_token) {
        sum = sum_all(sum, held);
        if (tid == 0) d.part[(int64_t)slot * a.Hv + head] = sum;
    }
}

// The gradient of a head's one decay: its segments' sums in order.
__global__ __launch_bounds__(256) void head_decay_kernel(const double *part, float *dla, int64_t slots, int64_t Hv) {
    __shared__ double held[4];
    const int64_t head = block_id();
    if (head >= Hv) return;
    double s = 0.;
    for (int64_t i = threadIdx.x; i < slots; i += 256) s += part[i * Hv + head];
    s = sum_all(s, held);
    if (threadIdx.x == 0) dla[head] = (float)s;
}

// The gradients of shared key heads: the sum over their value heads, [B][Hv][T][d] to [B][Hk][T][d] (`slab` elements of a head's T
// rows), four elements a thread. Rows outside the packed sequences are left as they are.
template <typename E>
__global__ __launch_bounds__(256) void shared_kernel(const float *pq, const float *pk, E *dq, E *dk, int64_t slab, int64_t group, int64_t n, int d,
                                                     const int32_t *cu, int64_t nseq) {
    const int64_t i = (block_id() * 256 + threadIdx.x) * 4;
    if (i >= 2 * n) return;
    const float *p = i < n ? pq : pk;
    E *out = i < n ? dq : dk;
    const int64_t e = i < n ? i : i - n, head = e / slab, in = e - head * slab, at = head * group * slab + in;
    if (cu && (in < (int64_t)cu[0] * d || in >= (int64_t)cu[nseq] * d)) return;
    floatx4 s = *reinterpret_cast<const floatx4 *>(p + at);
    for (int64_t j = 1; j < group; ++j) s += *reinterpret_cast<const floatx4 *>(p + at + j * slab);
    *reinterpret_cast<typename Vec4<E>::type *>(out + e) = cvt4<E>(s);
}

// ---------------------------------------------------------------- one token

// A workgroup takes 32 columns of one head's state: a thread 4 adjacent columns of every 32nd row. The state is read and written
// once, past the caches' keeping; the sum over the rows goes over lanes and then LDS.
template <typename E, int DK>
__global__ __launch_bounds__(256) void step_kernel(AttnCall a) {
    constexpr int RPT = DK / 32;
    __shared__ floatx4 held[4][8];
    const int64_t slices = a.dv_size / 32, id = block_id(), unit = id / slices;
    if (unit >= a.nseq * a.Hv) return;
    const int64_t col0 = id % slices * 32, head = unit % a.Hv, n = unit / a.Hv;
    const int tid = threadIdx.x, cg = tid & 7, rg = tid >> 3;
    const float *in = a.h0 + unit * DK * a.dv_size + col0 + 4 * cg;
    float *to = a.hT + unit * DK * a.dv_size + col0 + 4 * cg;
    floatx4 h[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) h[i] = __builtin_nontemporal_load(reinterpret_cast<const floatx4 *>(in + (rg + 32 * i) * a.dv_size));
    const int64_t kh = n * a.Hk + head / (a.Hv / a.Hk);
    const E *q = reinterpret_cast<const E *>(a.q) + kh * DK, *k = reinterpret_cast<const E *>(a.k) + kh * DK;
    const typename Vec4<E>::type v4 = *reinterpret_cast<const typename Vec4<E>::type *>(reinterpret_cast<const E *>(a.v) + unit * a.dv_size + col0 + 4 * cg);
    floatx4 v, o = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)v4[e];
    const float alpha = expf(a.la[a.la_token ? unit : head]);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = rg + 32 * i;
        const float kr = (float)k[row], qr = (float)q[row];
        h[i] = alpha * h[i] + kr * v;
        o += qr * h[i];
        __builtin_nontemporal_store(h[i], reinterpret_cast<floatx4 *>(to + row * a.dv_size));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int off = 8; off < 64; off <<= 1) o[e] += __shfl_xor(o[e], off, 64);
    if ((tid & 63) < 8) held[tid >> 6][cg] = o;
    __syncthreads();
    if (tid < 8) {
        o = held[0][cg] + held[1][cg] + held[2][cg] + held[3][cg];
        *reinterpret_cast<typename Vec4<E>::type *>(reinterpret_cast<E *>(a.out) + unit * a.dv_size + col0 + 4 * cg) = cvt4<E>(o);
    }
}

// ---------------------------------------------------------------- launches

template <typename E, int DA, int NT, Form F>
hipError_t sweep_t(AttnArgs a, int first, int n, hipStream_t s) {
    constexpr int NW = 4;
    const int64_t outer = (F == kStates && a.roles[first].cuts ? a.cuts : a.slots) * a.Hk, inner = n * a.slices * a.group;
    if (outer == 0) return hipSuccess;
    a.by_inner = Divisor(inner);
    a.by_roles = Divisor(n);
    a.by_slices = Divisor(a.slices);
    hipLaunchKernelGGL((sweep_kernel<E, DA, NT, NW, F>), grid_of((outer + 7) / 8 * 8 * inner, NW * 64), dim3(NW * 64), 0, s, a, first,
                       (unsigned)outer);
    return hipGetLastError();
}
// n roles of one size, from the first one on
template <typename E, Form F>
hipError_t sweep(AttnArgs a, int first, int n, hipStream_t s) {
    const AttnRole &r = a.roles[first];
    // (the results' products with q and k are formed by the one workgroup that has all columns)
    const bool narrow = F == kStates || F == kResults;
    const int nt = narrow ? attn_tiles(r.db, (r.cuts && F == kStates ? a.cuts : a.slots) * a.Hv * n * attn_slices(r.db)) : attn_tiles(r.db);
    a.slices = attn_slices(r.db, nt);
    if (r.da <= 64) return nt == 1 ? sweep_t<E, 64, 1, F>(a, first, n, s) : sweep_t<E, 64, 2, F>(a, first, n, s);
    if (r.da <= 128) return nt == 1 ? sweep_t<E, 128, 1, F>(a, first, n, s) : sweep_t<E, 128, 2, F>(a, first, n, s);
    // values, which have more channels, are x and y where the results go on to the decays' gradient
    if constexpr (F == kProducts || F == kShares) return nt == 1 ? sweep_t<E, 256, 1, F>(a, first, n, s) : sweep_t<E, 256, 2, F>(a, first, n, s);
    return hipErrorInvalidValue;
}

hipError_t join(const AttnArgs &a, const Join &j, hipStream_t s) {
    hipLaunchKernelGGL(join_kernel, grid_of((j.cuts && a.cu ? a.cuts : a.nseq) * a.Hv * (j.rows * j.cols / 1024), 256), dim3(256), 0, s, a, j);
    return hipGetLastError();
}

AttnArgs args_of(const AttnCall &c, const AttnPlan &p) {
    AttnArgs a{};
    a.la = c.la;
    a.cu = c.cu;
    a.B = c.B; a.T = c.T; a.Hk = c.Hk; a.Hv = c.Hv; a.nseq = c.nseq;
    a.seg = p.seg; a.per_seq = p.per_seq; a.slots = p.slots; a.cuts = p.slots - c.nseq;
    a.la_token = c.la_token;
    a.group = (uint32_t)(c.Hv / c.Hk);
    a.by_Hk = Divisor(c.Hk);
    a.by_per = Divisor(p.per_seq);
    a.by_cuts = Divisor(p.per_seq > 1 ? p.per_seq - 1 : 1);
    a.by_seg = Divisor(p.seg ? p.seg : 1);
    return a;
}

template <typename E>
hipError_t fwd(const AttnCall &c, hipStream_t s) {
    const int dk = (int)c.dk_size, dv = (int)c.dv_size;
    const AttnPlan p = attn_plan(c.T, c.nseq, c.Hv * attn_slices(dv), c.cu != nullptr, false);
    const AttnSpace w = attn_space(p, c.B, c.T, c.Hk, c.Hv, c.nseq, dk, dv, false);
    AttnArgs a = args_of(c, p);
    AttnRole &r = a.roles[0];
    r.x = c.q; r.y = c.k; r.z = c.v;
    r.xk = r.yk = true;
    r.da = dk; r.db = dv;
    if (p.seg) {
        float *states = reinterpret_cast<float *>(c.ws + w.states), *decays = reinterpret_cast<float *>(c.ws + w.decays);
        r.s_out = states;
        r.decay = decays;
        r.out_turned = true;  // a lane of the sweep then reads 16 bytes at a time
        r.cuts = true;
        hipError_t e = sweep<E, kStates>(a, 0, 1, s);
        if (e != hipSuccess) return e;
        e = join(a, Join{states, decays, c.h0, nullptr, nullptr, nullptr, nullptr, dv, dk, true, false, true}, s);
        if (e != hipSuccess) return e;
        r.s_cuts = states;
        r.out_turned = false;
    }
    r.s_in = c.h0;
    r.out = c.out;
    r.s_out = c.hT;
    return sweep<E, kResults>(a, 0, 1, s);
}

template <typename E>
hipError_t bwd(const AttnCall &c, hipStream_t s) {
    const int dk = (int)c.dk_size, dv = (int)c.dv_size;
    const int64_t group = c.Hv / c.Hk;
    const AttnPlan p = attn_plan(c.T, c.nseq, c.Hv, c.cu != nullptr, true);
    const AttnSpace w = attn_space(p, c.B, c.T, c.Hk, c.Hv, c.nseq, dk, dv, true);
    auto at = [&](int64_t off) { return reinterpret_cast<float *>(c.ws + off); };
    float *states = at(w.states), *decays = at(w.decays), *back = at(w.back), *back_decays = at(w.back_decays), *last = at(w.last);
    double *ends = reinterpret_cast<double *>(c.ws + w.ends);
    AttnArgs a = args_of(c, p);
    hipError_t e;
    if (p.seg) {
        AttnRole &f = a.roles[0], &b = a.roles[1];
        f.y = c.k; f.z = c.v; f.yk = true;
        f.da = dk; f.db = dv;
        f.s_out = states;
        f.decay = decays;
        b = f;
        b.y = c.q; b.z = c.dout;
        b.s_out = back;
        b.decay = back_decays;
        b.reverse = true;
        e = sweep<E, kStates>(a, 0, 2, s);
        if (e != hipSuccess) return e;
        e = join(a, Join{states, decays, c.h0, c.dhT ? last : nullptr, nullptr, nullptr, nullptr, dk, dv, false, false, false}, s);
        if (e != hipSuccess) return e;
        e = join(a, Join{back, back_decays, c.dhT, c.dh0, states, c.dhT ? last : nullptr, ends, dk, dv, false, true, false}, s);
        if (e != hipSuccess) return e;
    }
    AttnRole &q = a.roles[0], &k = a.roles[1], &v = a.roles[2];
    q = AttnRole{};
    q.x = c.dout; q.y = c.v; q.z = c.k; q.zk = true;
    q.da = dv; q.db = dk;
    q.out = group > 1 ? c.ws + w.dq : c.dq;
    q.other = c.q; q.ok = true;
    q.dot = at(w.dq_dot);
    q.in_turned = q.out_turned = true;
    q.in_slots = p.seg != 0;
    q.s_in = p.seg ? states : c.h0;
    q.s_out = !p.seg && c.dhT ? last : nullptr;
    k = q;
    k.x = c.v; k.y = c.dout; k.z = c.q;
    k.out = group > 1 ? c.ws + w.dk : c.dk;
    k.other = c.k;
    k.dot = at(w.dk_dot);
    k.reverse = true;
    k.s_in = p.seg ? back : c.dhT;
    k.s_out = nullptr;
    v = AttnRole{};
    v.x = c.k; v.y = c.q; v.z = c.dout; v.xk = v.yk = true;
    v.da = dk; v.db = dv;
    v.out = c.dv;
    v.reverse = true;
    v.in_slots = k.in_slots;
    v.s_in = k.s_in;
    v.s_out = p.seg ? nullptr : c.dh0;
    if (attn_together(dk, dv)) {
        v.other = c.dout;  // read and multiplied with as the other roles' are; the products go nowhere
        q.shares = k.shares = group > 1;
        if constexpr (is_bf16<E>()) {
            a.slices = 1;
            if (dk == 64) e = group > 1 ? sweep_t<E, 64, 1, kMixed>(a, 0, 3, s) : sweep_t<E, 64, 1, kProducts>(a, 0, 3, s);
            else e = group > 1 ? sweep_t<E, 128, 2, kMixed>(a, 0, 3, s) : sweep_t<E, 128, 2, kProducts>(a, 0, 3, s);
        } else {
            e = sweep<E, kProducts>(a, 0, 3, s);
        }
        if (e != hipSuccess) return e;
    } else {
        if constexpr (is_bf16<E>()) e = group > 1 ? sweep<E, kShares>(a, 0, 2, s) : sweep<E, kProducts>(a, 0, 2, s);
        else e = sweep<E, kProducts>(a, 0, 2, s);
        if (e != hipSuccess) return e;
        e = sweep<E, kResults>(a, 2, 1, s);
        if (e != hipSuccess) return e;
    }
    const DecayGrad d{p.seg ? ends : nullptr, last, c.dhT, at(w.dq_dot), at(w.dk_dot), c.dla, reinterpret_cast<double *>(c.ws + w.part), dk * dv,
                      c.q, c.k, c.v, c.dout, p.seg ? states : c.h0, p.seg ? back : c.dhT, dk, dv, p.seg != 0};
    if (p.slots) {
        hipLaunchKernelGGL((decay_grad_kernel<E>), grid_of(p.slots * c.Hv, 256), dim3(256), 0, s, a, d);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (!c.la_token) {
        hipLaunchKernelGGL(head_decay_kernel, grid_of(c.Hv, 256), dim3(256), 0, s, d.part, c.dla, p.slots, c.Hv);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t n = c.B * c.Hk * c.T * dk;
    if (group > 1 && n) {
        hipLaunchKernelGGL((shared_kernel<E>), grid_of((2 * n / 4 + 255) / 256, 256), dim3(256), 0, s, at(w.dq), at(w.dk), reinterpret_cast<E *>(c.dq),
                           reinterpret_cast<E *>(c.dk), c.T * dk, group, n, dk, c.cu, c.nseq);
        e = hipGetLastError();
    }
    return e;
}

template <typename E>
hipError_t step(const AttnCall &c, hipStream_t s) {
    const dim3 grid = grid_of(c.nseq * c.Hv * (c.dv_size / 32), 256);
    if (c.dk_size == 64) hipLaunchKernelGGL((step_kernel<E, 64>), grid, dim3(256), 0, s, c);
    else hipLaunchKernelGGL((step_kernel<E, 128>), grid, dim3(256), 0, s, c);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_fwd(const AttnCall &c, int dtype, hipStream_t s) { return dtype == kDtypeBf16 ? fwd<__bf16>(c, s) : fwd<float>(c, s); }
hipError_t launch_attn_bwd(const AttnCall &c, int dtype, hipStream_t s) { return dtype == kDtypeBf16 ? bwd<__bf16>(c, s) : bwd<float>(c, s); }
hipError_t launch_attn_step(const AttnCall &c, int dtype, hipStream_t s) {
    if (c.nseq == 0) return hipSuccess;
    return dtype == kDtypeBf16 ? step<__bf16>(c, s) : step<float>(c, s);
}

}  // namespace gdr
