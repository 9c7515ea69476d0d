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
// A step is the affine map h -> alpha h + beta x, and maps compose: (P, H) over several steps, P the
// product of their alphas and H the end state from zero. A workgroup owns 16 V neighbouring channels
// of a sequence and walks it in blocks of 256 tokens: 32 time slots of 8
// tokens side by side, 16 lanes of V channels each. A thread composes its 8 steps in registers, the
// slots' maps are joined (shuffles within a wave, LDS between the eight waves, one barrier a
// block), and the thread runs its steps again from the state that enters them: 8 more
// multiply-adds, no second read. The next block's inputs are on their way meanwhile. The adjoint of
// a block runs backwards with the same maps' products: (P, C) with C the gradient that leaves the
// steps at their front; both directions' maps of a block are joined behind one barrier, the forward
// one starting at the block's kept state.
//
// Memory is what bounds it: a read of x, a, b (and dout) and a write of the results, each once. Where
// there are too few (sequence, channel tile) pairs for the 256 compute units the time axis is split
// too: a first launch composes each chunk's map, and each workgroup of the second composes the
// chunks before its own (behind it, in the backward) before it starts, at the cost of reading the
// inputs of the maps twice.
//
// Measured (bf16): 4 x 4096 tokens x 2048 channels forward 71 us (268 MB, 3.8 TB/s), backward 133 us
// (470 MB, 3.5 TB/s); the device's own large copy moves 4.9 TB/s. Per element the gates are 5
// transcendental and about 25 other instructions, which at eight waves a compute unit nearly take the
// time that the bytes take and do not all hide behind them. The backward holds 245 registers (fp32: 160), so that
// a compute unit has one workgroup of it. Split, 131,072 tokens x 1024 channels:
// 217 us for the maps (805 MB, 3.7 TB/s) and 265 us for the scan (1074 MB, 4.0 TB/s). The chunks'
// order is fixed, so the results do not depend on which workgroup comes first.
//
// A sequence takes whole blocks, so short ones leave slots idle: 2^14 tokens x 2048 channels as sequences of 4096, 256,
// 64, 16 and 1 tokens take 60, 53, 184, 680 and 10310 us forward and 133, 151, 506, 1920 and 29,280 us backward. (One
// token at a time without a gradient is scan_step_kernel's.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gdr_kernels.hpp"
#include "layer_kernels.hpp"

namespace gdr {

namespace {

// The gates of one element, in base 2: softplus(u) log2 e = max(u, 0) log2 e + log2(1 + z), z =
// e^{-|u|}. 1 + z is rounded; d is what it lost, and d / (1 + z) (its quotient to a tenth: d is below
// 2^-24) puts it back, so that small softplus keep their bits: the decay's logarithm enters the
// gradient of A_log by itself.
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
__device__ __forceinline__ float sigmoid_of(float b) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * b));
}
// log2 of alpha; z and 1 + z for the sigmoid of u
__device__ __forceinline__ float log2_alpha(float u, float rate, float &z, float &w) {
    z = __builtin_amdgcn_exp2f(-kLog2e * fabsf(u));
    w = 1.f + z;
    const float d = z - (w - 1.f);
    const float l = fmaf(d, fmaf(-0.5f * kLog2e, z, kLog2e), __builtin_amdgcn_logf(w));
    return -rate * fmaf(__builtin_amdgcn_fmed3f(u, 0.f, INFINITY), kLog2e, l);
}
__device__ __forceinline__ float alpha_of(float u, float rate) {
    float z, w;
    return __builtin_amdgcn_exp2f(log2_alpha(u, rate, z, w));
}
// The backward needs 1 - beta too, and to its own bits: by subtraction it is 1e-3 off at b = 10 and 0 from 17
// on. One number holds both: the smaller of the two, with the sign bit set where that is 1 - beta.
struct Gates {
    float alpha, sig, la, rs;  // la = log2 alpha, rs = e^{A_log} sigmoid(u)
    __device__ __forceinline__ bool open() const { return __float_as_int(sig) < 0; }
    __device__ __forceinline__ float beta() const { return open() ? 1.f + sig : sig; }
    __device__ __forceinline__ float shut() const { return open() ? -sig : 1.f - sig; }  // 1 - beta
    // computed anew from here on: what was derived is not kept through a phase of the block
    __device__ __forceinline__ void forget() { asm("" : "+v"(sig)); }
};
__device__ __forceinline__ Gates gates_of(float a, float b, float bias, float rate) {
    const float u = a + bias;
    float z, w;
    Gates g;
    // not -infinity, so that la times a vanished alpha is 0; a comparison, which lets NaN through
    const float la = log2_alpha(u, rate, z, w);
    g.la = la < -1e30f ? -1e30f : la;
    g.alpha = __builtin_amdgcn_exp2f(g.la);
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(b)), s = e * __builtin_amdgcn_rcpf(1.f + e);
    g.sig = b > 0.f ? -s : s;
    g.rs = rate * (u >= 0.f ? 1.f : z) * __builtin_amdgcn_rcpf(w);
    return g;
}

constexpr int kThreads = 512, kWaves = kThreads / 64, kSlots = 4 * kWaves, kLen = kScanBlock / kSlots;
static_assert(kLen * kSlots == kScanBlock, "block shape");

// One unit: tokens [t0, t1) of a sequence in scan order.
struct Unit {
    int64_t s, row0, len, slot0;  // sequence, its first row, its tokens, its first block slot
    int64_t c, base, t0, t1;      // the chunk and the unit index of the sequence's first chunk
    bool last;                    // the sequence ends with this unit
};
__device__ __forceinline__ Unit unit_of(const ScanArgs &a, const ScanPlan &p, int64_t u) {
    Unit n;
    n.s = u;
    n.c = 0;
    n.base = u;
    if (p.chunk) {
        if (a.cu_seqlens) {  // the last sequence whose first chunk is at or before u
            int64_t lo = 0, hi = a.nseq - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) / 2;
                if (a.cu_seqlens[mid] / p.chunk + mid <= u) lo = mid;
                else hi = mid - 1;
            }
            n.s = lo;
            n.base = a.cu_seqlens[lo] / p.chunk + lo;
        } else {
            n.s = u / p.per_seq;
            n.base = n.s * p.per_seq;
        }
        n.c = u - n.base;
    }
    if (a.cu_seqlens) {
        n.row0 = a.cu_seqlens[n.s];
        n.len = a.cu_seqlens[n.s + 1] - n.row0;
        n.slot0 = n.row0 / kScanBlock + n.s;
    } else {
        n.row0 = n.s * a.T;
        n.len = a.T;
        n.slot0 = n.s * ((a.T + kScanBlock - 1) / kScanBlock);
    }
    n.t0 = p.chunk ? n.c * p.chunk : 0;
    n.t1 = p.chunk && n.t0 + p.chunk < n.len ? n.t0 + p.chunk : n.len;
    n.last = n.t1 == n.len && (n.t0 < n.len || n.c == 0);
    return n;
}

// What a thread is: V channels from d0, slot `slot` of the block.
template <typename E, int V>
struct Lane {
    typedef E Raw __attribute__((ext_vector_type(V)));
    int wave, sub, col, slot;
    int64_t d0;
    bool on;                 // its channels exist
    unsigned off[kLen];      // bytes from a block's first row (in memory) to its tokens' channels (to the
                             // tile's first where the thread's own do not exist)
    unsigned safe;           // ... to an address that any block with a token has

    __device__ __forceinline__ void init(const ScanArgs &a, int64_t tile) {
        const int lane = threadIdx.x & 63;
        wave = threadIdx.x >> 6;
        sub = lane >> 4;
        col = lane & 15;
        slot = 4 * wave + sub;
        d0 = (tile * 16 + col) * V;
        on = d0 < a.D;
        const bool rev = a.flags & kFlagReverse;
        const unsigned pitch = (unsigned)(a.D * sizeof(E));
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            const int t = slot * kLen + j;
            off[j] = (rev ? kScanBlock - 1 - t : t) * pitch + (unsigned)((on ? d0 : tile * 16 * V) * sizeof(E));
        }
        safe = rev ? (kScanBlock - 1) * pitch : 0;
    }
    // whether token j of the thread's slot is among the first n of the block
    __device__ __forceinline__ bool has(int j, int n) const { return on && slot * kLen + j < n; }
    // offsets of the loads of a block of n tokens; tokens it does not have read a safe address
    __device__ __forceinline__ void places(unsigned (&o)[kLen], int n) const {
#pragma unroll
        for (int j = 0; j < kLen; ++j) o[j] = off[j];
        if (n < kScanBlock) {
#pragma unroll
            for (int j = 0; j < kLen; ++j) o[j] = has(j, n) ? off[j] : safe;
        }
    }
    __device__ __forceinline__ void load(Raw (&r)[kLen], const E *p, const unsigned (&o)[kLen]) const {
#pragma unroll
        for (int j = 0; j < kLen; ++j) r[j] = *reinterpret_cast<const Raw *>(reinterpret_cast<const char *>(p) + o[j]);
    }
    __device__ __forceinline__ void store(E *p, int j, const float (&v)[V]) const {
        Raw r;
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = (E)v[i];
        *reinterpret_cast<Raw *>(reinterpret_cast<char *>(p) + off[j]) = r;
    }
};

// The first row, in memory, of the block that begins at token t of unit n's sequence.
__device__ __forceinline__ int64_t block_row(const ScanArgs &a, const Unit &n, int64_t t) {
    return a.flags & kFlagReverse ? n.row0 + n.len - t - kScanBlock : n.row0 + t;
}

// Joins the slots' maps (P, H) in time order. `in` becomes the state entering the thread's slot
// when `carry` enters the block, `carry` the state that leaves the block, `whole` (the product of
// all alphas so far) is multiplied on. BACK joins from the last slot to the first.
template <int V>
struct WaveMap {
    float P[V], H[V];
};
template <int V, bool BACK>
__device__ __forceinline__ void join_in_wave(int sub, const float (&P)[V], const float (&H)[V], WaveMap<V> &all, WaveMap<V> &before) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = P[i], h = H[i];
#pragma unroll
        for (int d = 1; d < 4; d *= 2) {
            const float q = BACK ? __shfl_down(p, 16 * d, 64) : __shfl_up(p, 16 * d, 64);
            const float g = BACK ? __shfl_down(h, 16 * d, 64) : __shfl_up(h, 16 * d, 64);
            if (BACK ? sub + d < 4 : sub >= d) {
                h = fmaf(p, g, h);
                p *= q;
            }
        }
        all.P[i] = p;
        all.H[i] = h;
        const float q = BACK ? __shfl_down(p, 16, 64) : __shfl_up(p, 16, 64);
        const float g = BACK ? __shfl_down(h, 16, 64) : __shfl_up(h, 16, 64);
        const bool first = BACK ? sub == 3 : sub == 0;
        before.P[i] = first ? 1.f : q;
        before.H[i] = first ? 0.f : g;
    }
}
template <int V, bool BACK>
__device__ __forceinline__ void join_waves(const WaveMap<V> (*rec)[16], int wave, int col, const WaveMap<V> &before,
                                           float (&carry)[V], float (&whole)[V], float (&in)[V]) {
    float mine[V];
#pragma unroll
    for (int k = 0; k < kWaves; ++k) {
        const int w = BACK ? kWaves - 1 - k : k;
        const WaveMap<V> m = rec[w][col];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (w == wave) mine[i] = carry[i];
            carry[i] = fmaf(m.P[i], carry[i], m.H[i]);
            whole[i] *= m.P[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) in[i] = fmaf(before.P[i], mine[i], before.H[i]);
}

// The state entering chunk n.c of a sequence (BACK: the gradient entering it from behind): the maps of
// the chunks before it (behind it), composed by the 32 slots side by side and then joined.
template <int V, bool BACK>
__device__ __forceinline__ void fold_chunks(const ScanArgs &a, const Unit &n, const ScanPlan &p, const float2 *agg, int slot, int sub,
                                            int wave, int col, int64_t d0, bool on, WaveMap<V> (*rec)[16], float (&carry)[V]) {
    const int64_t chunks = (n.len + p.chunk - 1) / p.chunk;
    const int64_t first = BACK ? n.c + 1 : 0, count = BACK ? chunks - first : n.c;
    float P[V], H[V], in[V], whole[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        P[i] = whole[i] = 1.f;
        H[i] = 0.f;
    }
    const int64_t lo = first + count * slot / kSlots, hi = first + count * (slot + 1) / kSlots;
    if (on)
        for (int64_t k = lo; k < hi; ++k) {
            const int64_t c = BACK ? lo + hi - 1 - k : k;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float2 m = agg[(n.base + c) * a.D + d0 + i];
                if (!BACK && c == 0) m.x = 0.f;  // holds the initial state, see scan_fwd_kernel
                H[i] = fmaf(m.x, H[i], m.y);
                P[i] *= m.x;
            }
        }
    WaveMap<V> all, before;
    join_in_wave<V, BACK>(sub, P, H, all, before);
    if (sub == (BACK ? 0 : 3)) rec[wave][col] = all;
    __syncthreads();
    join_waves<V, BACK>(rec, wave, col, before, carry, whole, in);
}

enum ScanMode { kWhole, kCompose, kApply };

// workgroup -> (unit, channel tile), the tiles of a unit side by side on one XCD: their rows share
// 128-byte lines
__device__ __forceinline__ int64_t xcd_order(int64_t id, int64_t all) {
    const int64_t x = id & 7, q = all >> 3, r = all & 7;
    return x * q + (x < r ? x : r) + (id >> 3);
}

template <typename E, int V, int MODE>
__global__ __launch_bounds__(kThreads, 2) void scan_fwd_kernel(ScanArgs a, ScanPlan p, float2 *agg) {
    __shared__ WaveMap<V> rec[2][kWaves][16];
    const int64_t all = p.units * p.ntile, id = block_id();
    if (id >= all) return;
    const int64_t w = xcd_order(id, all), u = w / p.ntile;
    const Unit n = unit_of(a, p, u);
    if (p.chunk && n.t0 >= n.len && n.c > 0) return;  // a slot without a chunk
    Lane<E, V> ln;
    ln.init(a, w % p.ntile);
    typedef typename Lane<E, V>::Raw Raw;

    float rate[V], bias[V], carry[V], whole[V], initial[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t d = ln.on ? ln.d0 + i : 0;
        rate[i] = expf(a.A_log[d]);
        bias[i] = a.dt_bias[d];
        // Split: the first launch takes the initial state into the first chunk's map and keeps a copy of
        // it where that map's product would stand; the second does not read h0, which its last chunk
        // may overwrite (hT in place).
        if (MODE == kApply) carry[i] = n.c == 0 && ln.on ? agg[u * a.D + d].x : 0.f;
        else carry[i] = n.c == 0 && a.h0 && ln.on ? a.h0[n.s * a.D + d] : 0.f;
        whole[i] = 1.f;
        initial[i] = carry[i];
    }
    if (MODE == kApply) {
        fold_chunks<V, false>(a, n, p, agg, ln.slot, ln.sub, ln.wave, ln.col, ln.d0, ln.on, rec[1], carry);
    }

    Raw rx[kLen], ra[kLen], rb[kLen];
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
        const int64_t row = block_row(a, n, t) * a.D;
        const int left = n.t1 - t < kScanBlock ? (int)(n.t1 - t) : kScanBlock;
        unsigned o[kLen];
        ln.places(o, left);
        ln.load(rx, (const E *)a.x + row, o);
        ln.load(ra, (const E *)a.a + row, o);
        ln.load(rb, (const E *)a.b + row, o);
    };
    if (n.t0 < n.t1) fetch(n.t0);
    int buf = 0;
    for (int64_t t = n.t0; t < n.t1; t += kScanBlock, buf ^= 1) {
        const int left = n.t1 - t < kScanBlock ? (int)(n.t1 - t) : kScanBlock;
        Raw x[kLen], ga[kLen], gb[kLen];
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            x[j] = rx[j];
            ga[j] = ra[j];
            gb[j] = rb[j];
        }
        if (t + kScanBlock < n.t1) fetch(t + kScanBlock);
        if (MODE != kCompose && a.states && ln.slot == 0 && ln.on) {
#pragma unroll
            for (int i = 0; i < V; ++i) a.states[(n.slot0 + t / kScanBlock) * a.D + ln.d0 + i] = carry[i];
        }
        float al[kLen][V], v[kLen][V], P[V], H[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            P[i] = 1.f;
            H[i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                al[j][i] = alpha_of((float)ga[j][i] + bias[i], rate[i]);
                v[j][i] = sigmoid_of((float)gb[j][i]) * (float)x[j][i];
            }
        if (left < kScanBlock) {  // past the end: the identity
#pragma unroll
            for (int j = 0; j < kLen; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    al[j][i] = ln.has(j, left) ? al[j][i] : 1.f;
                    v[j][i] = ln.has(j, left) ? v[j][i] : 0.f;
                }
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                H[i] = fmaf(al[j][i], H[i], v[j][i]);
                P[i] *= al[j][i];
            }
        WaveMap<V> all, before;
        join_in_wave<V, false>(ln.sub, P, H, all, before);
        if (ln.sub == 3) rec[buf][ln.wave][ln.col] = all;
        __syncthreads();
        float h[V];
        join_waves<V, false>(rec[buf], ln.wave, ln.col, before, carry, whole, h);
        if (MODE == kCompose) continue;
        E *out = (E *)a.out + block_row(a, n, t) * a.D;
        float hs[kLen][V];
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) hs[j][i] = h[i] = fmaf(al[j][i], h[i], v[j][i]);
        if (left == kScanBlock) {
            if (ln.on)
#pragma unroll
                for (int j = 0; j < kLen; ++j) ln.store(out, j, hs[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kLen; ++j)
                if (ln.has(j, left)) ln.store(out, j, hs[j]);
        }
    }
    if (ln.slot == 0 && ln.on) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (MODE == kCompose) agg[u * a.D + ln.d0 + i] = make_float2(n.c == 0 ? initial[i] : whole[i], carry[i]);
            else if (a.hT && n.last) a.hT[n.s * a.D + ln.d0 + i] = carry[i];
        }
    }
}

// MODE kCompose: the maps (P, C) of the chunks' adjoints, which need a and dout alone.
template <typename E, int V, int MODE>
__global__ __launch_bounds__(kThreads, 2) void scan_bwd_kernel(ScanArgs a, ScanPlan p, float2 *agg, float *sums) {
    __shared__ WaveMap<V> rec[2][kWaves][16], rec_back[2][kWaves][16];
    __shared__ float part[2][V][kSlots][16];
    const int64_t all = p.units * p.ntile, id = block_id();
    if (id >= all) return;
    const int64_t w = xcd_order(id, all), u = w / p.ntile;
    const Unit n = unit_of(a, p, u);
    Lane<E, V> ln;
    ln.init(a, w % p.ntile);
    const bool none = p.chunk && n.t0 >= n.len && n.c > 0;  // a slot without a chunk
    if (none) {
        if (MODE != kCompose && ln.slot == 0 && ln.on)
#pragma unroll
            for (int i = 0; i < V; ++i) sums[2 * u * a.D + ln.d0 + i] = sums[(2 * u + 1) * a.D + ln.d0 + i] = 0.f;
        return;
    }
    typedef typename Lane<E, V>::Raw Raw;

    float rate[V], bias[V], carry[V], whole[V], sA[V], sb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t d = ln.on ? ln.d0 + i : 0;
        rate[i] = expf(a.A_log[d]);
        bias[i] = a.dt_bias[d];
        carry[i] = MODE != kCompose && a.dhT && ln.on ? a.dhT[n.s * a.D + d] : 0.f;
        whole[i] = 1.f;
        sA[i] = sb[i] = 0.f;
    }
    if (MODE == kApply) {
        fold_chunks<V, true>(a, n, p, agg, ln.slot, ln.sub, ln.wave, ln.col, ln.d0, ln.on, rec_back[1], carry);
        __syncthreads();
    }

    Raw rx[kLen], ra[kLen], rb[kLen], rg[kLen];
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
        const int64_t row = block_row(a, n, t) * a.D;
        const int left = n.t1 - t < kScanBlock ? (int)(n.t1 - t) : kScanBlock;
        unsigned o[kLen];
        ln.places(o, left);
        ln.load(ra, (const E *)a.a + row, o);
        ln.load(rg, (const E *)a.dout + row, o);
        if (MODE != kCompose) {
            ln.load(rx, (const E *)a.x + row, o);
            ln.load(rb, (const E *)a.b + row, o);
        }
    };
    const int64_t blocks = (n.t1 - n.t0 + kScanBlock - 1) / kScanBlock;
    if (blocks > 0) fetch(n.t0 + (blocks - 1) * kScanBlock);
    int buf = 0;
    for (int64_t k = blocks - 1; k >= 0; --k, buf ^= 1) {
        const int64_t t = n.t0 + k * kScanBlock;
        const int left = n.t1 - t < kScanBlock ? (int)(n.t1 - t) : kScanBlock;
        Raw x[kLen], ga[kLen], gb[kLen], go[kLen];
#pragma unroll
        for (int j = 0; j < kLen; ++j) {
            x[j] = rx[j];
            ga[j] = ra[j];
            gb[j] = rb[j];
            go[j] = rg[j];
        }
        float start[V];
        if (MODE != kCompose) {
#pragma unroll
            for (int i = 0; i < V; ++i) start[i] = a.states[(n.slot0 + t / kScanBlock) * a.D + (ln.on ? ln.d0 + i : 0)];
        }
        if (k > 0) fetch(t - kScanBlock);
        Gates q[kLen][V];
        float P[V], H[V], C[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            P[i] = 1.f;
            H[i] = C[i] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (MODE == kCompose) q[j][i].alpha = alpha_of((float)ga[j][i] + bias[i], rate[i]);
                else q[j][i] = gates_of((float)ga[j][i], (float)gb[j][i], bias[i], rate[i]);
            }
        // Past the end: the identity, with no gradient of its own. x and beta are what the safe address
        // holds, maybe another channel's NaN: they reach states past the end only.
        if (left < kScanBlock) {
#pragma unroll
            for (int j = 0; j < kLen; ++j) {
                const bool in = ln.has(j, left);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    q[j][i].alpha = in ? q[j][i].alpha : 1.f;
                    go[j][i] = in ? go[j][i] : (E)0.f;
                    if (MODE != kCompose) {
                        q[j][i].la = in ? q[j][i].la : 0.f;
                        q[j][i].rs = in ? q[j][i].rs : 0.f;
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (MODE != kCompose) H[i] = fmaf(q[j][i].alpha, H[i], q[j][i].beta() * (float)x[j][i]);
                P[i] *= q[j][i].alpha;
            }
#pragma unroll
        for (int j = kLen - 1; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < V; ++i) C[i] = q[j][i].alpha * ((float)go[j][i] + C[i]);
        WaveMap<V> all, before, all_back, before_back;
        join_in_wave<V, true>(ln.sub, P, C, all_back, before_back);
        if (ln.sub == 0) rec_back[buf][ln.wave][ln.col] = all_back;
        if (MODE != kCompose) {
            join_in_wave<V, false>(ln.sub, P, H, all, before);
            if (ln.sub == 3) rec[buf][ln.wave][ln.col] = all;
        }
        __syncthreads();
        float c[V];
        join_waves<V, true>(rec_back[buf], ln.wave, ln.col, before_back, carry, whole, c);
        if (MODE == kCompose) continue;
        float h[V], prev[kLen][V], unused[V];
#pragma unroll
        for (int i = 0; i < V; ++i) unused[i] = 1.f;
        join_waves<V, false>(rec[buf], ln.wave, ln.col, before, start, unused, h);
#pragma unroll
        for (int j = 0; j < kLen; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                prev[j][i] = h[i];
                q[j][i].forget();
                h[i] = fmaf(q[j][i].alpha, h[i], q[j][i].beta() * (float)x[j][i]);
            }
        if (left < kScanBlock) {  // the states past the end, out of the sums
#pragma unroll
            for (int j = 0; j < kLen; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) prev[j][i] = ln.has(j, left) ? prev[j][i] : 0.f;
        }
        const int64_t row = block_row(a, n, t) * a.D;
        E *dx = (E *)a.dx + row, *da = (E *)a.da + row, *db = (E *)a.db + row;
#pragma unroll
        for (int j = kLen - 1; j >= 0; --j) {
            float vx[V], va[V], vb[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                Gates &g = q[j][i];
                g.forget();
                const float up = (float)go[j][i] + c[i];
                const float dla = g.alpha * prev[j][i] * up;
                vx[i] = g.beta() * up;
                va[i] = -g.rs * dla;
                vb[i] = vx[i] * g.shut() * (float)x[j][i];
                sA[i] = fmaf(dla, g.la, sA[i]);
                sb[i] += va[i];
                c[i] = g.alpha * up;
            }
            if (left == kScanBlock ? ln.on : ln.has(j, left)) {
                ln.store(dx, j, vx);
                ln.store(da, j, va);
                ln.store(db, j, vb);
            }
        }
    }
    if (MODE == kCompose) {
        if (ln.slot == 0 && ln.on)
#pragma unroll
            for (int i = 0; i < V; ++i) agg[u * a.D + ln.d0 + i] = make_float2(whole[i], carry[i]);
        return;
    }
    // the parameters' sums of this unit: the slots' in order
#pragma unroll
    for (int i = 0; i < V; ++i) {
        part[0][i][ln.slot][ln.col] = sA[i];
        part[1][i][ln.slot][ln.col] = sb[i];
    }
    __syncthreads();
    if (ln.slot < 2 && ln.on) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) s += part[ln.slot][i][k][ln.col];
            sums[(2 * u + ln.slot) * a.D + ln.d0 + i] = ln.slot == 0 ? s * kLn2 : s;  // la was in base 2
        }
    }
    if (ln.slot == 0 && ln.on && a.dh0 && n.c == 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) a.dh0[n.s * a.D + ln.d0 + i] = carry[i];
    }
}

// dA_log and ddt_bias: the units' sums [units][2][D], 16 slices of the units side by side and then
// in order. 4.6 us for 2048 channels, most of it the launch.
__global__ __launch_bounds__(1024) void scan_param_kernel(const float *sums, int64_t units, int64_t D, float *dA, float *db) {
    __shared__ float held[2][16][64];
    const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t d = (int64_t)blockIdx.x * 64 + lane;
    float sA = 0.f, sb = 0.f;
    if (d < D)
        for (int64_t i = units * slice / 16; i < units * (slice + 1) / 16; ++i) {
            sA += sums[2 * i * D + d];
            sb += sums[(2 * i + 1) * D + d];
        }
    held[0][slice][lane] = sA;
    held[1][slice][lane] = sb;
    __syncthreads();
    if (slice < 2 && d < D) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += held[slice][k][lane];
        (slice ? db : dA)[d] = s;
    }
}

// One token: a channel of a sequence a thread. Latency is all of it: 5.3 us as a launch for 256 x 4096
// bf16 (16.8 MB, which the large copy's rate would move in 3.4).
template <typename E>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanArgs a) {
    const int64_t i = block_id() * 256 + threadIdx.x;
    if (i >= a.nseq * a.D) return;
    const int64_t d = i % a.D;
    const float alpha = alpha_of((float)((const E *)a.a)[i] + a.dt_bias[d], expf(a.A_log[d]));
    const float h = fmaf(alpha, a.h0[i], sigmoid_of((float)((const E *)a.b)[i]) * (float)((const E *)a.x)[i]);
    a.hT[i] = h;
    ((E *)a.out)[i] = (E)h;
}

int vec_of(int64_t D, int dtype) { return scan_vec(D, dtype == kDtypeBf16 ? 2 : 4); }
ScanPlan plan_of(const ScanArgs &a, int vec) { return scan_plan(a.T, a.D, a.nseq, a.cu_seqlens != nullptr, vec); }

template <typename E, int V>
hipError_t fwd_t(const ScanArgs &a, hipStream_t s) {
    const ScanPlan p = plan_of(a, V);
    const dim3 grid = grid_of(p.units * p.ntile, kThreads), block(kThreads);
    float2 *agg = (float2 *)a.ws;
    if (!p.chunk) {
        hipLaunchKernelGGL((scan_fwd_kernel<E, V, kWhole>), grid, block, 0, s, a, p, agg);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((scan_fwd_kernel<E, V, kCompose>), grid, block, 0, s, a, p, agg);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_fwd_kernel<E, V, kApply>), grid, block, 0, s, a, p, agg);
    return hipGetLastError();
}

template <typename E, int V>
hipError_t bwd_t(const ScanArgs &a, hipStream_t s) {
    const ScanPlan p = plan_of(a, V);
    const dim3 grid = grid_of(p.units * p.ntile, kThreads), block(kThreads);
    float *sums = a.ws;
    float2 *agg = (float2 *)(a.ws + 2 * p.units * a.D);
    if (a.nseq > 0) {
        if (p.chunk) {
            hipLaunchKernelGGL((scan_bwd_kernel<E, V, kCompose>), grid, block, 0, s, a, p, agg, sums);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((scan_bwd_kernel<E, V, kApply>), grid, block, 0, s, a, p, agg, sums);
        } else {
            hipLaunchKernelGGL((scan_bwd_kernel<E, V, kWhole>), grid, block, 0, s, a, p, agg, sums);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(scan_param_kernel, dim3((unsigned)((a.D + 63) / 64)), dim3(1024), 0, s, sums, a.nseq ? p.units : 0, a.D,
                       a.dA_log, a.ddt_bias);
    return hipGetLastError();
}

}  // namespace

int64_t scan_fwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype) {
    const ScanPlan p = scan_plan(T, D, nseq, packed, vec_of(D, dtype));
    return p.chunk ? p.units * D * 8 : 0;
}
int64_t scan_bwd_ws_bytes(int64_t T, int64_t D, int64_t nseq, bool packed, int dtype) {
    const ScanPlan p = scan_plan(T, D, nseq, packed, vec_of(D, dtype));
    return p.units * D * (p.chunk ? 16 : 8);
}

hipError_t launch_scan_fwd(const ScanArgs &a, int dtype, hipStream_t s) {
    if (a.nseq == 0) return hipSuccess;
    if (dtype == kDtypeBf16) return vec_of(a.D, dtype) == 2 ? fwd_t<__bf16, 2>(a, s) : fwd_t<__bf16, 1>(a, s);
    return fwd_t<float, 1>(a, s);
}

hipError_t launch_scan_bwd(const ScanArgs &a, int dtype, hipStream_t s) {
    if (dtype == kDtypeBf16) return vec_of(a.D, dtype) == 2 ? bwd_t<__bf16, 2>(a, s) : bwd_t<__bf16, 1>(a, s);
    return bwd_t<float, 1>(a, s);
}

hipError_t launch_scan_step(const ScanArgs &a, int dtype, hipStream_t s) {
    const int64_t n = a.nseq * a.D;
    if (n == 0) return hipSuccess;
    const dim3 grid = grid_of((n + 255) / 256, 256), block(256);
    if (dtype == kDtypeBf16) hipLaunchKernelGGL((scan_step_kernel<__bf16>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((scan_step_kernel<float>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace gdr
