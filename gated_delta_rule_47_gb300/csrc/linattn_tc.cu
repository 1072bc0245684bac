// linattn_tc.cu -- linear attention with a decay for each head over whole
// prompts on the tensor cores (bf16, tcgen05), in chunks of 128 tokens.  The
// formulas are linattn.cu's.
//
// prompt_kernel is the forward, in one launch or, where few long sequences are
// cut into pieces, behind the one that plans them.  A CTA owns 64 value columns of
// one head (columns are independent) and walks a sequence's chunks with the
// fp32 state in registers, so q, k, v and o cross the memory once (a head's two
// CTAs run side by side and share q and k in L2).  A chunk is four products:
// T = Q K^T; P V with P = T under the decay mask, in tensor memory; Q S; and
// the chunk's own share of the state K^T diag(w) V, which does not depend on
// the state, so the walk itself costs one multiply-add an element.
// The weighted values w v go in as two or three bf16 terms (x = hi + mid + lo
// to 2^-24): with one, the state would carry 2^-9 of rounding in every term,
// against inputs that are exact; sums and state stay in fp32.  P and S enter
// their products rounded to bf16: each adds about as much as the output's own
// rounding does.
//
// state_kernel is the walk alone, for the backward, which wants the state that
// enters each chunk and (backwards) the gradient of the one that leaves it.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <type_traits>

#include "gdn_internal.h"
#include "linattn.cuh"
#include "tc_util.cuh"

namespace gdn {

using namespace tc;

namespace la {
namespace {

constexpr int kC = 128;

__device__ unsigned int g_la_error = 0;  // set when a bounded wait gives up
constexpr unsigned long long kDrainNs = 200000000ull;

// Waits for the phase of the given parity, until the CTA's deadline at most.
// Small on purpose: the roles' loops share the instruction cache.  The deadline
// is a reference so that one in shared memory is read when it is looked at.
__device__ __forceinline__ bool la_wait(uint64_t *bar, uint32_t parity, const uint64_t &deadline) {
#pragma unroll 1
    while (!mbar_try_wait_sleep(bar, parity, 20000u))
        if (global_timer_ns() > deadline) {
            *reinterpret_cast<volatile unsigned *>(&g_la_error) = 1u;
            return false;
        }
    return true;
}

// When a CTA that walks n chunks gives up: the wait limit, and 50 us a chunk
// for the work itself.
__device__ __forceinline__ uint64_t deadline_after(unsigned long long limit, int n) {
    return global_timer_ns() + limit + 50000ull * n;
}

// A wait's outcome made uniform across the warp, so that the warp's
// .sync.aligned TMEM accesses that follow are reached by all of its lanes.
__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }
// A barrier (1) of THREADS of the CTA's threads, and whether all of them say so.
template <int THREADS>
__device__ __forceinline__ bool all_of(bool ok) {
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all)
                 : "r"(ok ? 1u : 0u), "n"(THREADS)
                 : "memory");
    return all != 0;
}
__device__ __forceinline__ uint32_t lane_base(int warp) { return (uint32_t)(32 * (warp & 3)) << 16; }

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A weight as bf16 terms, each twice in a word: w = h + m + l to 2^-24.
struct Weight {
    uint32_t h, m, l;
};
__device__ __forceinline__ Weight split_weight(float w) {
    Weight r;
    r.h = pack_bf16(w, w);
    w -= __uint_as_float(r.h & 0xffff0000u);
    r.m = pack_bf16(w, w);
    w -= __uint_as_float(r.m & 0xffff0000u);
    r.l = pack_bf16(w, w);
    return r;
}

// Two values times a weight as a sum of bf16 terms, in packed bf16 arithmetic.
// hi is the rounded product with the weight's first term and r what that
// rounding left, exactly (a product of two 8-bit mantissas has 16 bits).
// Two terms: lo = v m + r, 2^-17 of the product off.  Three: the product with
// the second term is split in the same way, the two parts of that size are
// added with the sum's own rounding error kept (exact in any order of size),
// and what is left goes into lo: 2^-24 or so off.
__device__ __forceinline__ void weigh2(uint32_t v, const Weight &w, uint32_t &hi, uint32_t &lo) {
    hi = mul2(v, w.h);
    lo = fma2(v, w.m, fma2(v, w.h, hi ^ 0x80008000u));
}
__device__ __forceinline__ void weigh3(uint32_t v, const Weight &w, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = mul2(v, w.h);
    const uint32_t r = fma2(v, w.h, hi ^ 0x80008000u);
    const uint32_t m = mul2(v, w.m), mr = fma2(v, w.m, m ^ 0x80008000u);
    mid = add2(r, m);
    const uint32_t b = sub2(mid, r);
    const uint32_t e = add2(sub2(r, sub2(mid, b)), sub2(m, b));
    lo = fma2(v, w.l, add2(mr, e));
}

// A forward whose long sequences are cut into pieces of whole chunks: a piece
// but the last of its sequence has its own share of the state made first (a
// row of the tables here, one item a head and 64 columns), and a piece starts
// from the shares before it.
struct Plan {
    int *head;        // {next item, rows of shares, pieces, chunks of a piece at most}; null: no plan
    int4 *shares;     // [rows] {sequence, first token, tokens, piece of its sequence}
    int4 *pieces;     // {sequence, first token, tokens, 32 first row of its sequence's shares + 2 piece + last}
    unsigned *flags;  // [rows][items of a row] made
    float *decay;     // [rows][items of a row] e^(sum of the piece's log-decays)
    float *share;     // [rows][items of a row][DK][64]
    int rows;         // places
};

// A backward whose walks are cut into pieces of `len` chunks (0: they are not):
// the shares of the pieces first, in a launch of their own.
struct Cut {
    View pieces;   // chunks of len * kC tokens
    int len;
    float *share;  // [piece][direction][H][DV / 64][DK][64]
    float *decay;  // [piece][direction][H]
};

// What the tensor-core kernels take besides their maps.
struct TcArgs {
    LinAttnArgs a;
    View v;
    Plan plan;
    Cut cut;
    uint16_t *S[3], *R[3];  // [chunk][H][DK][DV], in three bf16 terms: the states that enter the chunks, and the
                            // gradients of those that leave them
    float *gates;         // [chunk][H][4][128] decays for the gradients, see state_kernel
    float *dqh, *dkh;     // [B,H,T,DK] fp32, where value heads share dq and dk
    float *dgt;           // dg by token, with its strides
    Strides sdg;
    unsigned long long timeout_ns;
    int wide;             // o's rows are 32-byte aligned
};

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// smem_desc in two halves: what varies is the low one, an address (and the
// leading stride) in 16-byte units, to which a product's steps add constants.
// The warps that issue products run converged, so that all of this stays in
// uniform registers; a step is then two instructions.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) { return (saddr >> 4) | (lbo_bytes >> 4) << 16; }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32 | lo;
}

// A chunk's log-decays, lane's tokens 4 lane ..: summed up to each from the
// chunk's start, and after it to the end, each way by itself: weights near the
// end are made from few terms, not from the difference of two large sums.
struct Sums {
    float cum[4], to_end[4], all;
};
__device__ __forceinline__ Sums scan_sums(const float (&g)[4]) {
    const int lane = threadIdx.x & 31;
    Sums r;
    r.cum[0] = g[0], r.cum[1] = g[0] + g[1], r.cum[2] = r.cum[1] + g[2], r.cum[3] = r.cum[2] + g[3];
    r.to_end[3] = 0.f, r.to_end[2] = g[3], r.to_end[1] = g[3] + g[2], r.to_end[0] = r.to_end[1] + g[1];
    float up = r.cum[3], down = r.cum[3];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float x = __shfl_up_sync(~0u, up, m), y = __shfl_down_sync(~0u, down, m);
        if (lane >= m) up += x;
        if (lane + m < 32) down += y;
    }
    r.all = __shfl_sync(~0u, up, 31);
    up = __shfl_up_sync(~0u, up, 1);
    down = __shfl_down_sync(~0u, down, 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (lane > 0) r.cum[j] += up;
        if (lane < 31) r.to_end[j] += down;
    }
    return r;
}

// 32 bytes to a 32-byte aligned address: whole sectors.
__device__ __forceinline__ void st_global_32(void *p, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Four lanes (rows) of four words of 32 bytes each exchange them: before, z[e] is
// word e of the lane's row; after, z[e] is word lane % 4 of the e-th row.  A store
// is then of 8 whole lines and not of a piece of 32.
__device__ __forceinline__ void exchange(uint32_t (&z)[4][8]) {
#pragma unroll
    for (int m = 2; m; m >>= 1) {
        const bool up = threadIdx.x & m;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (!(e & m))
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t got = __shfl_xor_sync(~0u, up ? z[e][j] : z[e | m][j], m);
                    if (up) z[e][j] = got;
                    else z[e | m][j] = got;
                }
    }
}

// D[tmem] (+)= A * B[smem]^T with A in shared memory, or (ts) in tensor memory:
// rows are lanes, two bf16 of a row a column.  ADD is a constant: as a run-time
// operand it costs more instructions than all the rest of a product.
template <int ADD>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "n"(ADD)
        : "memory");
}
template <int ADD>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "n"(ADD)
        : "memory");
}

// KS steps of 16; a(ks) and b(ks) are the operands' low descriptor words.
// mma_more adds to what is there.
template <int KS, class A, class B>
__device__ __forceinline__ void mma_steps(uint32_t d, uint32_t idesc, const A &a, const B &b) {
    mma_ss<0>(d, desc_of(a(0)), desc_of(b(0)), idesc);
#pragma unroll
    for (int ks = 1; ks < KS; ++ks) mma_ss<1>(d, desc_of(a(ks)), desc_of(b(ks)), idesc);
}
template <int KS, class A, class B>
__device__ __forceinline__ void mma_more(uint32_t d, uint32_t idesc, const A &a, const B &b) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) mma_ss<1>(d, desc_of(a(ks)), desc_of(b(ks)), idesc);
}

// The backward's tensors; boxes of 64 columns, the states' of DK rows.
struct GradMaps {
    CUtensorMap q, k, v, o, s[3], r[3], dq, dk, dv;
};

// ================================================================ state kernel
// Warps: 0 TMA, 1 products, 2 decays, 4..7 state, 8..15 weighting.
constexpr int kStateThreads = 512;
constexpr int kStages = 2, kWRing = 4;

template <int DK>
struct StateSmem {
    static constexpr uint32_t KB = DK * 256, VB = 16384;  // a chunk's K (or Q) and 64 columns of V (or dO)
    static constexpr uint32_t STAGE = KB + VB;
    // with DK = 64 the product's rows 64..127 read the bytes after K, in the
    // stage's own V tile: rows that nobody looks at
    static constexpr uint32_t X = kStages * STAGE;        // [half][3][64 tokens][128 B] weighted values
    static constexpr uint32_t OUT = X + 2 * 3 * 8192;     // [3][DK][128 B] the state's terms on their way out
    static constexpr uint32_t W = OUT + 3 * DK * 128;       // [ring][3][128] weights, then [ring] chunk decays
    static constexpr uint32_t BAR = W + kWRing * 1536 + 64;
    enum { FULL = 0, EMPTY = 2, XREADY = 4, XEMPTY = 6, UFULL = 8, UEMPTY = 10, WFULL = 12, WEMPTY = 16, DRAIN = 20, NUM = 21 };
    static constexpr uint32_t TSLOT = BAR + 8 * NUM;
    static constexpr uint32_t BYTES = TSLOT + 16;
};
static_assert(StateSmem<128>::BYTES <= 232448, "state kernel fits the shared memory of one CTA");

// Grid (2 DV / 64, H, n_seq or pieces): the states that enter a sequence's chunks, and
// (the second half of x) backwards over them the gradients of the states that
// leave them, with Q and dO in the places of K and V.  They go out as three
// bf16 terms, which the gradients' products take as operands: dg is fp32, and
// with two terms of S (2^-17) it was 4e-6 off where a state comes in.
// Bound by what it writes, 48 KB a CTA and chunk, and by the waves of CTAs: 125
// us at B4 H16 T4096 (670 MB, 256 CTAs on 152 SMs), 1.7 us a chunk alone.  Two
// smaller CTAs an SM wait for each other's stores and were no faster.
// SHARE: a piece's share of the state after it (before it, backwards) and
// nothing else; the walk of a piece then starts from the shares on its way.
template <int DK, int DV, bool SHARE>
__global__ void __launch_bounds__(kStateThreads, 1)
    state_kernel(const __grid_constant__ GradMaps m, TcArgs p) {
    using L = StateSmem<DK>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::TSLOT);
    uint32_t *wring = reinterpret_cast<uint32_t *>(sm + L::W);
    float *dring = reinterpret_cast<float *>(wring + kWRing * 384);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool rev = blockIdx.x >= DV / 64;
    const int slice = blockIdx.x % (DV / 64), h = blockIdx.y;
    int seq = blockIdx.z, first = 0, pieces = 1, piece = 0;  // its sequence's pieces, and which it is
    if (p.cut.len) {
        const int z = blockIdx.z, over = z - p.cut.pieces.n_chunks;
        seq = over >= 0 ? over : p.a.cu ? p.cut.pieces.chunks[z].w : z / p.cut.pieces.per_row;
        if (seq < 0) return;  // tokens of no sequence
        const int2 all = seq_at(p.cut.pieces, seq);
        if (over >= 0 && all.y) return;  // those of sequences without tokens
        first = all.x, pieces = max(all.y, 1), piece = over >= 0 ? 0 : z - first;
        if (piece >= pieces) return;
        if (SHARE && (over >= 0 || piece == (rev ? 0 : pieces - 1))) return;
    }
    const Span sp = span_of(p.a, seq);
    const int2 sq = seq_at(p.v, seq);
    const int c0 = piece * p.cut.len, n = p.cut.len ? min(p.cut.len, sq.y - c0) : sq.y, row0 = p.a.cu ? 0 : seq;
    const uint64_t end = deadline_after(p.timeout_ns, n);
    auto number = [&](int i) { return c0 + (rev ? n - 1 - i : i); };
    auto chunk = [&](int i) { return Chunk{row0, sp.start + number(i) * kC, min(kC, sp.len - number(i) * kC), seq}; };
    auto share_of = [&](int i) { return ((size_t)(first + i) * 2 + rev) * p.a.H + h; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[L::FULL + s], 1);
            mbar_init(&bars[L::EMPTY + s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars[L::XREADY + x], 256);
            mbar_init(&bars[L::XEMPTY + x], 1);
            mbar_init(&bars[L::UFULL + x], 1);
            mbar_init(&bars[L::UEMPTY + x], 128);
        }
        for (int w = 0; w < kWRing; ++w) {
            mbar_init(&bars[L::WFULL + w], 32);
            mbar_init(&bars[L::WEMPTY + w], 256 + 128);
        }
        mbar_init(&bars[L::DRAIN], 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, 128);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tslot;
    const uint32_t sbase = smem_u32(sm);

    if (warp == 0) {
        if (lane == 0) {
            const int hk = h / (p.a.H / p.a.Hk);
            const CUtensorMap *m1 = rev ? &m.q : &m.k, *m2 = rev ? &m.o : &m.v;
            int i = 0;
#pragma unroll 1
            for (; i < n; ++i) {
                const int s = i % kStages;
                if (i >= kStages && !la_wait(&bars[L::EMPTY + s], ((i / kStages) - 1) & 1, end)) break;
                const Chunk c = chunk(i);
                uint8_t *st = sm + s * L::STAGE;
                mbar_arrive_expect_tx(&bars[L::FULL + s], L::STAGE);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x) tma_load_4d(st + x * 16384, m1, &bars[L::FULL + s], 64 * x, c.t0, hk, c.row);
                tma_load_4d(st + L::KB, m2, &bars[L::FULL + s], 64 * slice, c.t0, h, c.row);
            }
            // no copy is in flight when the CTA ends
#pragma unroll 1
            for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
                mbar_wait(&bars[L::FULL + j % kStages], (j / kStages) & 1, kDrainNs);
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16(128, 64, true, true);
        const bool leader = elect_one();
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
            const int s = i % kStages, acc = i & 1;
            ok = la_wait(&bars[L::FULL + s], (i / kStages) & 1, end);
            if (i >= 2) ok = ok && la_wait(&bars[L::UEMPTY + acc], ((i >> 1) - 1) & 1, end);
            tc_fence_after_sync();
            const uint32_t d = tmem + 64u * acc;
            // sums in the tensor core are cut off, not rounded, and what is added
            // to little loses little: the half of smaller weights first, and in
            // it the smallest terms
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                const int half = rev ? 1 - j : j;
                ok = ok && la_wait(&bars[L::XREADY + half], i & 1, end);
                if (!ok) break;
                const uint32_t k = desc_lo(sbase + s * L::STAGE, 16384) + half * 512, x = desc_lo(sbase + L::X + half * 3 * 8192, 8192);
                if (leader) {
                    if (j == 0) mma_ss<0>(d, desc_of(k), desc_of(x + 1024), id);
                    else mma_ss<1>(d, desc_of(k), desc_of(x + 1024), id);
#pragma unroll
                    for (int e = 1; e < 12; ++e)
                        mma_ss<1>(d, desc_of(k + (e & 3) * 128), desc_of(x + (2 - (e >> 2)) * 512 + (e & 3) * 128), id);
                    if (j == 1) mma_commit(&bars[L::UFULL + acc]);
                    mma_commit(&bars[L::XEMPTY + half]);
                    if (j == 1) mma_commit(&bars[L::EMPTY + s]);
                }
            }
        }
        // every MMA issued here is complete before TMEM is released
        if (leader) mma_commit(&bars[L::DRAIN]);
        mbar_wait(&bars[L::DRAIN], 0, kDrainNs);
    } else if (warp == 2) {
        // the weights: e^{G - c_t}, or backwards scale e^{c_t}; the next chunk's
        // gates are on their way meanwhile
        const bool per_head = p.a.flags & GDN_G_PER_HEAD;
        float next[4], whole = 0.f;
        auto fetch = [&](int i) {
            if (i >= n) return;
            load_gates<kC>(gate_ptr(p.a, chunk(i), h), p.a.sg.t, chunk(i).len, per_head, next);
        };
        fetch(0);
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int w = i % kWRing;
            const Gates<kC> g = scan_gates<kC>(next);
            fetch(i + 1);
            if (i >= kWRing && !la_wait(&bars[L::WEMPTY + w], ((i / kWRing) - 1) & 1, end)) break;
            Weight wt[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wt[j] = split_weight(rev ? p.a.scale * expf(g.cum[j].hi) : expf(g.to_end(j)));
            if (!SHARE && blockIdx.x == 0) {
                // the gradient kernel's decays: c_t as a pair, G - c_t, and
                // e^{c_r - c_t} with r the last token of t's block of 32
                const float rh = __shfl_sync(~0u, g.cum[3].hi, lane | 7), rl = __shfl_sync(~0u, g.cum[3].lo, lane | 7);
                float4 *out = reinterpret_cast<float4 *>(p.gates + ((size_t)(sq.x + number(i)) * p.a.H + h) * 512) + lane;
                float cf[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) cf[j] = expf(((rh - g.cum[j].hi) + (rl - g.cum[j].lo)));
                out[0] = make_float4(g.cum[0].hi, g.cum[1].hi, g.cum[2].hi, g.cum[3].hi);
                out[32] = make_float4(g.cum[0].lo, g.cum[1].lo, g.cum[2].lo, g.cum[3].lo);
                out[64] = make_float4(g.to_end(0), g.to_end(1), g.to_end(2), g.to_end(3));
                out[96] = make_float4(cf[0], cf[1], cf[2], cf[3]);
            }
            uint4 *ws = reinterpret_cast<uint4 *>(wring + w * 384);
            ws[lane] = make_uint4(wt[0].h, wt[1].h, wt[2].h, wt[3].h);
            ws[lane + 32] = make_uint4(wt[0].m, wt[1].m, wt[2].m, wt[3].m);
            ws[lane + 64] = make_uint4(wt[0].l, wt[1].l, wt[2].l, wt[3].l);
            if (lane == 0) dring[w] = expf(g.all.hi);
            whole += g.all.hi;
            if (SHARE && slice == 0 && i == n - 1 && lane == 0) p.cut.decay[share_of(piece)] = expf(whole);
            mbar_arrive(&bars[L::WFULL + w]);
        }
    } else if (warp >= 8) {
        // the weighted values, in two halves of 64 tokens: row r, 16 columns
        const int ct = threadIdx.x - 256, r = ct >> 2, c0 = (ct & 3) * 16;
        const uint32_t off[2] = {sw128_offset(r, c0), sw128_offset(r, c0 + 8)};
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int s = i % kStages, w = i % kWRing, len = chunk(i).len;
            ok = la_wait(&bars[L::FULL + s], (i / kStages) & 1, end) && la_wait(&bars[L::WFULL + w], (i / kWRing) & 1, end);
            if (!ok) break;
            uint8_t *st = sm + s * L::STAGE;
            if (len < kC) {
                // rows past the chunk's tokens are another sequence's: zeros, so
                // that nothing of theirs (an infinity, say) meets a zero weight
#pragma unroll 1
                for (int e = ct; e < (kC - len) * (DK / 8); e += 256) {
                    const int row = len + e / (DK / 8), col = (e % (DK / 8)) * 8;
                    *reinterpret_cast<uint4 *>(st + (col >> 6) * 16384 + sw128_offset(row, col & 63)) = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                const int half = rev ? 1 - j : j, t = half * 64 + r;
                const uint32_t *wr = wring + w * 384 + t;
                const Weight wt = {wr[0], wr[128], wr[256]};
                uint4 v[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    v[u] = *reinterpret_cast<const uint4 *>(st + L::KB + half * 8192 + off[u]);
                    if (t >= len) v[u] = make_uint4(0, 0, 0, 0);
                }
                if (i >= 1 && !la_wait(&bars[L::XEMPTY + half], (i - 1) & 1, end)) {
                    ok = false;
                    break;
                }
                uint8_t *xb = sm + L::X + half * 3 * 8192;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint4 x, y, z;
                    weigh3(v[u].x, wt, x.x, y.x, z.x), weigh3(v[u].y, wt, x.y, y.y, z.y);
                    weigh3(v[u].z, wt, x.z, y.z, z.z), weigh3(v[u].w, wt, x.w, y.w, z.w);
                    *reinterpret_cast<uint4 *>(xb + off[u]) = x;
                    *reinterpret_cast<uint4 *>(xb + 8192 + off[u]) = y;
                    *reinterpret_cast<uint4 *>(xb + 16384 + off[u]) = z;
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars[L::XREADY + half]);
            }
            if (!ok) break;
            mbar_arrive(&bars[L::WEMPTY + w]);
        }
    } else if (warp >= 4) {
        // the state: one row of 64 columns a thread
        const int row = 32 * (warp & 3) + lane;
        const bool mine = row < DK;
        float S[64];
        const int start = rev ? pieces - 1 : 0;  // the piece where the sequence's walk starts
        const float *from = piece != start ? nullptr : rev ? p.a.dsf : p.a.s0;
        const size_t page = (((size_t)seq * p.a.H + h) * DK + row) * DV + 64 * slice;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine && from) x = *reinterpret_cast<const float4 *>(from + page + e);
            S[e] = x.x, S[e + 1] = x.y, S[e + 2] = x.z, S[e + 3] = x.w;
        }
        if (!SHARE && mine)
#pragma unroll 1
            for (int j = start; j != piece; j += rev ? -1 : 1) {  // the shares on the way, the first with s0 in it
                const float d = j == start ? 0.f : p.cut.decay[share_of(j)];
                const float4 *x4 = reinterpret_cast<const float4 *>(p.cut.share + ((share_of(j) * (DV / 64) + slice) * DK + row) * 64);
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    const float4 x = x4[e / 4];
                    S[e] = fmaf(d, S[e], x.x), S[e + 1] = fmaf(d, S[e + 1], x.y);
                    S[e + 2] = fmaf(d, S[e + 2], x.z), S[e + 3] = fmaf(d, S[e + 3], x.w);
                }
            }
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int acc = i & 1, w = i % kWRing;
            if constexpr (!SHARE) {
            // the terms leave through a tile each, whole lines at a time: by the
            // threads' own stores, 32 bytes of 32 lines an instruction, the walks
            // took 167 us (B4 H16 T4096)
            if (i >= 1 && threadIdx.x == 128) tma_store_wait_read<0>();
            // a warp whose wait gave up comes to this barrier all the same, and none
            // of the four goes on
            ok = all_of<128>(ok);
            if (!ok) break;
            if (mine)
#pragma unroll
                for (int e = 0; e < 64; e += 8) {
                    uint32_t a[4], b[4], c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x = S[e + 2 * j], y = S[e + 2 * j + 1];
                        a[j] = pack_bf16(x, y);
                        x -= __uint_as_float(a[j] << 16), y -= __uint_as_float(a[j] & 0xffff0000u);
                        b[j] = pack_bf16(x, y);
                        x -= __uint_as_float(b[j] << 16), y -= __uint_as_float(b[j] & 0xffff0000u);
                        c[j] = pack_bf16(x, y);
                    }
                    uint8_t *to = sm + L::OUT + sw128_offset(row, e);
                    *reinterpret_cast<uint4 *>(to) = make_uint4(a[0], a[1], a[2], a[3]);
                    *reinterpret_cast<uint4 *>(to + DK * 128) = make_uint4(b[0], b[1], b[2], b[3]);
                    *reinterpret_cast<uint4 *>(to + 2 * DK * 128) = make_uint4(c[0], c[1], c[2], c[3]);
                }
            fence_proxy_async_smem();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (threadIdx.x == 128) {
                const int item = (sq.x + number(i)) * p.a.H + h;
#pragma unroll
                for (int e = 0; e < 3; ++e) tma_store_3d(rev ? &m.r[e] : &m.s[e], sm + L::OUT + e * DK * 128, 64 * slice, 0, item);
                tma_store_commit();
            }
            }
            ok = warp_ok(la_wait(&bars[L::WFULL + w], (i / kWRing) & 1, end) && la_wait(&bars[L::UFULL + acc], (i >> 1) & 1, end));
            if (!ok) {
                if (SHARE) break;
                continue;
            }
            const float d = dring[w];
            tc_fence_after_sync();
#pragma unroll
            for (int e = 0; e < 64; e += 16) {
                uint32_t u[16];
                tmem_ld16(tmem + lane_base(warp) + 64u * acc + e, u);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) S[e + j] = fmaf(d, S[e + j], __uint_as_float(u[j]));
            }
            tc_fence_before_sync();
            mbar_arrive(&bars[L::UEMPTY + acc]);
            mbar_arrive(&bars[L::WEMPTY + w]);
        }
        if (!SHARE && threadIdx.x == 128) tma_store_wait_all<0>();
        float *to = SHARE                               ? p.cut.share + ((share_of(piece) * (DV / 64) + slice) * DK + row) * 64
                    : piece != (rev ? 0 : pieces - 1)   ? nullptr
                    : rev                               ? (p.a.ds0 ? p.a.ds0 + page : nullptr)
                                                        : nullptr;
        if (to && mine && ok)
#pragma unroll
            for (int e = 0; e < 64; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 128);
    }
}

// ================================================================ prompt kernel
// Warps: 0 TMA, 1 and 2 products, 3 decays, 4..7 state, 8..11 P, 12..15
// weighting, 16..19 outputs.  One warp of each on each of the SM's four
// schedulers, so every instruction is fetched for one warp alone, and
// straight-line code is bound by its fetching (a third of an instruction a
// cycle here): the roles' bodies are short loops.
constexpr int kFwdThreads = 640;
constexpr int kQKStages = 2, kVStages = 3, kXMax = 3, kGRing = 4;

template <int DK>
struct FwdSmem {
    static constexpr uint32_t TB = DK * 256;                 // a chunk's Q or K
    static constexpr uint32_t QK = 0;                        // [stage] K | Q
    static constexpr uint32_t V = kQKStages * 2 * TB;        // [stage] 64 columns of V
    static constexpr uint32_t X = V + kVStages * 16384;      // [slot][term][32 tokens][128 B] weighted values
    static constexpr uint32_t S = X + 6 * 4096;              // [DK][128 B] the state as an operand
    static constexpr uint32_t W = S + DK * 128;              // [ring][3][128] weights
    static constexpr uint32_t G = W + kGRing * 1536;         // [ring] log2 decays | block factors, 128 each
    static constexpr uint32_t D = G + kGRing * 1024;         // [ring] chunk decays
    static constexpr uint32_t ITEM = D + 16;                 // the item, and the next one
    static constexpr uint32_t BAR = D + 112;
    enum { KFULL = 0, KEMPTY = 2, QFULL = 4, QEMPTY = 6, VFULL = 8, VREADY = 11, VEMPTY = 14, XREADY = 17,
           XEMPTY = XREADY + kXMax, UFULL = XEMPTY + kXMax,
           UEMPTY, SREADY, SEMPTY, TFULL, PREADY = TFULL + 2, OFULL = PREADY + 2, OEMPTY, GFULL, GEMPTY = GFULL + kGRing,
           DRAIN = GEMPTY + kGRing, NUM = DRAIN + 2 };
    static constexpr uint32_t TSLOT = BAR + 8 * NUM;
    static constexpr uint32_t BYTES = TSLOT + 16;
};
static_assert(FwdSmem<128>::BYTES <= 232448, "prompt kernel fits the shared memory of one CTA");
// TMEM columns: Q K^T twice (P, two bf16 a column, takes its first half), Q S
// twice, P V, the chunk's share of the state
constexpr uint32_t TM_T = 0, TM_OS = 256, TM_OP = 384, TM_U = 448;

// ---- the plan: how a call's sequences are cut.  Costs are in chunks that a
// CTA walks (2 us); one of a share alone is kShareCost of it (0.9 us), an item's
// start and end kItemCost, a share that a piece adds up kJoinCost, making the
// plan kPlanCost.
constexpr int kSms = 152, kShareItems = 4 * kSms, kMostPieces = 16;
constexpr float kCutShare = 0.6f;  // a share's chunk in the backward's walks
constexpr float kShareCost = 0.45f, kItemCost = 2.5f, kJoinCost = 0.4f, kPlanCost = 1.5f;
// With the longest sequence in p pieces of up to len chunks: chunks and shared
// chunks of the call (over heads and columns), its items and shares.  What runs
// at once takes as long as the longest walk, what does not is spread over the
// SMs to half a walk or so.
__host__ __device__ inline float plan_cost(long long chunks, long long shared, int len, long long items, long long shares, int p) {
    const float chain = p > 1 ? (1.f + kShareCost) * len + 2 * kItemCost + kJoinCost * p + kPlanCost : len + kItemCost;
    const float work = chunks + kShareCost * shared + kItemCost * items + kJoinCost * 0.5f * p * shares;
    const float even = work / kSms + 0.5f * len;
    return items > kSms && even > chain ? even : chain;
}
__host__ __device__ inline int pieces_of(int n, int len) { return n > len ? (n + len - 1) / len : 1; }

// One CTA.  Cuts packed sequences by the lengths that are there, which the host
// does not know (known: rows, in pieces of that many chunks).
// Items are taken in order: shares, then pieces, long ones first.
constexpr int kPlanThreads = 256;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(LinAttnArgs a, Plan pl, int slots, int known) {
    __shared__ float costs[kMostPieces + 1];  // by pieces of the longest
    __shared__ unsigned long long all;
    __shared__ int longest, some, len, rows, place[4];
    if (threadIdx.x == 0) all = 0, longest = some = rows = 0;
    if (threadIdx.x < 4) place[threadIdx.x] = 0;
    __syncthreads();
    if (known) {
        if (threadIdx.x == 0) len = known;
    } else {
#pragma unroll 1
        for (int s = threadIdx.x; s < a.n_seq; s += kPlanThreads) {
            const int n = (span_of(a, s).len + kC - 1) / kC;
            if (!n) continue;
            atomicAdd(&all, (unsigned long long)n);
            atomicMax(&longest, n);
            atomicAdd(&some, 1);
        }
        __syncthreads();
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (int p = 2 + (threadIdx.x >> 5); p <= kMostPieces && longest; p += kPlanThreads / 32) {
            const int most = (longest + p - 1) / p;
            unsigned r = 0, c = 0;  // rows and chunks of shares
#pragma unroll 1
            for (int s = lane; s < a.n_seq; s += 32) {
                const int n = (span_of(a, s).len + kC - 1) / kC, k = pieces_of(n, most);
                if (k > 1) r += k - 1, c += (k - 1) * ((n + k - 1) / k);
            }
            r = __reduce_add_sync(~0u, r), c = __reduce_add_sync(~0u, c);
            if (lane == 0)
                costs[p] = r > pl.rows ? 1e30f
                                       : plan_cost((long long)all * slots, (long long)c * slots, most,
                                                   (some + 2ll * r) * slots, (long long)r * slots, p);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            len = max(longest, 1);
            float best = plan_cost((long long)all * slots, 0, longest, (long long)some * slots, 0, 1);
#pragma unroll 1
            for (int p = 2; p <= kMostPieces && longest; ++p)
                if (costs[p] < best) best = costs[p], len = (longest + p - 1) / p;
        }
    }
    __syncthreads();
    auto size = [&](int n, int &q) {  // pieces of a sequence of n chunks, and their chunks
        int k = pieces_of(n, len);
        q = (n + k - 1) / k;
        return max((n + q - 1) / max(q, 1), 1);
    };
    auto bucket = [&](int chunks) { return 2 * chunks > len ? 0 : 4 * chunks > len ? 1 : 8 * chunks > len ? 2 : 3; };
#pragma unroll 1
    for (int s = threadIdx.x; s < a.n_seq; s += kPlanThreads) {
        int q;
        const int n = (span_of(a, s).len + kC - 1) / kC, k = size(n, q);
        if (k > 1) atomicAdd(&place[bucket(q)], k - 1);
        atomicAdd(&place[bucket(n - (k - 1) * q)], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        for (int &x : place) {
            const int y = x;
            x = at, at += y;
        }
        pl.head[0] = 0, pl.head[2] = at, pl.head[3] = len;
    }
    __syncthreads();
#pragma unroll 1
    for (int s = threadIdx.x; s < a.n_seq; s += kPlanThreads) {
        const Span sp = span_of(a, s);
        int q;
        const int n = (sp.len + kC - 1) / kC, k = size(n, q);
        const int row = k > 1 ? atomicAdd(&rows, k - 1) : 0;
        int at = k > 1 ? atomicAdd(&place[bucket(q)], k - 1) : 0;
#pragma unroll 1
        for (int j = 0; j < k - 1; ++j) {
            const int t0 = sp.start + j * q * kC;
            pl.shares[row + j] = make_int4(s, t0, q * kC, j);
            pl.pieces[at + j] = make_int4(s, t0, q * kC, 32 * row + 2 * j);
        }
        const int done = (k - 1) * q;
        at = atomicAdd(&place[bucket(n - done)], 1);
        pl.pieces[at] = make_int4(s, sp.start + done * kC, sp.len - done * kC, 32 * row + 2 * (k - 1) + 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) pl.head[1] = rows;
#pragma unroll 1
    for (int e = threadIdx.x; e < rows * slots; e += kPlanThreads) pl.flags[e] = 0u;
}

// An item: some chunks of one sequence for 64 value columns of one head.
enum { kNone = 0, kShare = 1, kPiece = 2, kFill = 3 };
struct Item {
    int seq, t0, tokens, kind;
    int slot, row, piece;  // head and columns; the sequence's first row of shares; 2 piece + last
    int base, full;        // the CTA's chunks before it, and those of pieces
    uint64_t end;          // when its waits give up
};
static_assert(sizeof(Item) == 48, "two items take 96 bytes");

// Waits for a share that another CTA makes.
__device__ __forceinline__ bool share_wait(const unsigned *flag, const uint64_t &deadline) {
    for (;;) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
        if (v) return true;
        if (global_timer_ns() > deadline) {
            *reinterpret_cast<volatile unsigned *>(&g_la_error) = 1u;
            return false;
        }
        __nanosleep(200);
    }
}

// Bound by a chunk's chain of products, decays and shared-memory traffic: about
// 4,000 cycles.  Measured, bf16, D 128: 4 x 4096 of 16 heads 68 us (40 at the
// memory's rate); cut, 1 x 32768 of 16 heads 257 us (uncut 532), of 2 heads 89.
// Grid (DV / 64, H, n_seq, and one more for the tokens of no sequence): a CTA
// walks the chunks of one sequence for 64 value columns of one head.  TERMS of
// a weighted value: three where the final state, an fp32 output, is asked for;
// for bf16 outputs alone two (2^-16) are far below their rounding.  With a
// plan, as many CTAs as there are SMs that take the plan's items in order, so
// that the shares a piece waits for have all been started.  Rings and phases go
// on from item to item.
template <int DK, int DV, bool PLANNED, int TERMS>
__global__ void __launch_bounds__(kFwdThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                  const __grid_constant__ CUtensorMap mV, TcArgs p) {
    using L = FwdSmem<DK>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::TSLOT);
    float *gring = reinterpret_cast<float *>(sm + L::G), *dring = reinterpret_cast<float *>(sm + L::D);
    uint32_t *wring = reinterpret_cast<uint32_t *>(sm + L::W);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Item *item = reinterpret_cast<Item *>(sm + L::ITEM);
    const int slots = p.a.H * (DV / 64);
    auto take = [&](Item *to, int base, int full) {  // thread 0's
        const int t = atomicAdd(p.plan.head, 1), rows = p.plan.head[1], u = t / slots - rows;
        Item x = {0, 0, 0, kNone, t % slots, 0, 1, base, full, 0};
        if (u < 0) {
            const int4 e = p.plan.shares[t / slots];
            x.seq = e.x, x.t0 = e.y, x.tokens = e.z, x.kind = kShare, x.row = t / slots, x.piece = 2 * e.w;
        } else if (u < p.plan.head[2]) {
            const int4 e = p.plan.pieces[u];
            x.seq = e.x, x.t0 = e.y, x.tokens = e.z, x.kind = kPiece, x.row = e.w >> 5, x.piece = e.w & 31;
        } else if (u == p.plan.head[2] && p.a.cu) {
            x.kind = kFill;
        }
        x.end = deadline_after(p.timeout_ns, x.tokens / kC + 1 + p.plan.head[3]);  // a share's time included
        *to = x;
    };
    if (threadIdx.x == 0) {
        if (PLANNED) {
            take(item, 0, 0);
        } else {
            const int seq = blockIdx.z;
            const Span sp = seq < p.a.n_seq ? span_of(p.a, seq) : Span{0, 0};
            *item = {seq, sp.start, sp.len, seq < p.a.n_seq ? kPiece : kFill, (int)(blockIdx.y * gridDim.x + blockIdx.x), 0, 1, 0, 0,
                     deadline_after(p.timeout_ns, sp.len / kC + 1)};
        }
    }
    constexpr int kXRing = TERMS == 3 ? 2 : 3;  // slots of X: 24 KB in all

    if (threadIdx.x == 0) {
        for (int s = 0; s < kQKStages; ++s) {
            mbar_init(&bars[L::KFULL + s], 1);
            mbar_init(&bars[L::KEMPTY + s], 2);
            mbar_init(&bars[L::QFULL + s], 1);
            mbar_init(&bars[L::QEMPTY + s], 1);
            mbar_init(&bars[L::DRAIN + s], 1);
            mbar_init(&bars[L::TFULL + s], 1);
            mbar_init(&bars[L::PREADY + s], 128);
        }
        for (int s = 0; s < kXMax; ++s) {
            mbar_init(&bars[L::XREADY + s], 128);
            mbar_init(&bars[L::XEMPTY + s], 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(&bars[L::VFULL + s], 1);
            mbar_init(&bars[L::VREADY + s], 128);
            mbar_init(&bars[L::VEMPTY + s], 129);
        }
        for (int s = 0; s < kGRing; ++s) {
            mbar_init(&bars[L::GFULL + s], 32);
            mbar_init(&bars[L::GEMPTY + s], 512);
        }
        mbar_init(&bars[L::UFULL], 1);
        mbar_init(&bars[L::UEMPTY], 128);
        mbar_init(&bars[L::SREADY], 128);
        mbar_init(&bars[L::SEMPTY], 1);
        mbar_init(&bars[L::OFULL], 1);
        mbar_init(&bars[L::OEMPTY], 128);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's
    const uint32_t sbase = smem_u32(sm);

#pragma unroll 1
    for (;;) {
        const Item &it = *item;
        // the same in all lanes, which the compiler is to see (uniform registers)
        auto same = [](int x) { return __shfl_sync(~0u, x, 0); };
        const int kind = same(it.kind);
        if (kind == kNone) break;
        const bool share = PLANNED && kind == kShare;
        const int slice = it.slot % (DV / 64), h = it.slot / (DV / 64), seq = it.seq, row = p.a.cu ? 0 : seq;
        const int tokens = same(it.tokens), t0 = same(it.t0), n = (tokens + kC - 1) / kC;
        const int base = PLANNED ? same(it.base) : 0, full = PLANNED ? same(it.full) : 0;
        auto chunk = [&](int i) { return Chunk{row, t0 + i * kC, min(kC, tokens - i * kC), seq}; };
        const uint64_t &end = it.end;
        bool ok = true;
        if (kind == kFill) {  // packed: zeros for the tokens of no sequence
            const int T = p.a.T, head = min(max(p.a.cu[0], 0), T), tail = min(max(p.a.cu[p.a.n_seq], 0), T);
#pragma unroll 1
            for (long long e = threadIdx.x; e < ((long long)head + T - tail) * 8; e += kFwdThreads) {
                const long long i = e >> 3, t = i < head ? i : tail + i - head;
                *reinterpret_cast<uint4 *>(at(static_cast<__nv_bfloat16 *>(p.a.o), p.a.so, 0, h, (int)t) + 64 * slice + (e & 7) * 8) =
                    make_uint4(0, 0, 0, 0);
            }
            if (PLANNED && threadIdx.x == 0) take(item + 1, base, full);
        } else if (warp == 0) {
            if (lane == 0) {
                const int hk = h / (p.a.H / p.a.Hk);
                int ik = 0, iq = 0, iv = 0;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const Chunk c = chunk(i);
                    const int gi = base + i, fi = full + i, s = gi % kQKStages, v = gi % kVStages, f = fi % kQKStages;
                    uint8_t *st = sm + L::QK + s * 2 * L::TB, *sq = sm + L::QK + f * 2 * L::TB + L::TB;
                    if (gi >= kVStages && !(ok = la_wait(&bars[L::VEMPTY + v], (gi / kVStages - 1) & 1, end))) break;
                    mbar_arrive_expect_tx(&bars[L::VFULL + v], 16384);
                    tma_load_4d(sm + L::V + v * 16384, &mV, &bars[L::VFULL + v], 64 * slice, c.t0, h, c.row);
                    ++iv;
                    if (gi >= kQKStages && !(ok = la_wait(&bars[L::KEMPTY + s], (gi / kQKStages - 1) & 1, end))) break;
                    mbar_arrive_expect_tx(&bars[L::KFULL + s], L::TB);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x) tma_load_4d(st + x * 16384, &mK, &bars[L::KFULL + s], 64 * x, c.t0, hk, c.row);
                    ++ik;
                    if (share) continue;
                    if (fi >= kQKStages && !(ok = la_wait(&bars[L::QEMPTY + f], (fi / kQKStages - 1) & 1, end))) break;
                    mbar_arrive_expect_tx(&bars[L::QFULL + f], L::TB);
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x)
                        tma_load_4d(sq + x * 16384, &mQ, &bars[L::QFULL + f], 64 * x, c.t0, hk, c.row);
                    ++iq;
                }
                if (PLANNED) take(item + 1, base + n, share ? full : full + n);
                // no copy is in flight when the item ends
                auto drain = [&](int bar, int stages, int first, int count) {
#pragma unroll 1
                    for (int j = count > stages ? first + count - stages : first; j < first + count; ++j)
                        mbar_wait(&bars[bar + j % stages], (j / stages) & 1, kDrainNs);
                };
                drain(L::KFULL, kQKStages, base, ik);
                drain(L::QFULL, kQKStages, full, iq);
                drain(L::VFULL, kVStages, base, iv);
            }
        } else if (warp == 1) {
            // the products of the outputs: Q K^T a chunk ahead, Q S and P V.  All
            // lanes wait, one issues.
            constexpr uint32_t idT = idesc_bf16(128, 128, false, false), idO = idesc_bf16(128, 64, false, true);
            const bool leader = elect_one();
            if (share) {  // K and V pass by
#pragma unroll 1
                for (int gi = base; gi < base + n && ok; ++gi) {
                    const int s = gi % kQKStages, v = gi % kVStages;
                    ok = la_wait(&bars[L::KFULL + s], (gi / kQKStages) & 1, end) && la_wait(&bars[L::VFULL + v], (gi / kVStages) & 1, end);
                    if (leader && ok) {
                        mbar_arrive(&bars[L::KEMPTY + s]);
                        mbar_arrive(&bars[L::VEMPTY + v]);
                    }
                }
            }
#pragma unroll 1
            for (int i = share ? n : -1; i < n; ++i) {
                if (i + 1 < n) {
                    // T's place is free: P V of two chunks before, the last to read
                    // it, was issued before (products run in the order of their issue)
                    const int gj = base + i + 1, fj = full + i + 1, st = gj % kQKStages, sq = fj % kQKStages;
                    if (!(ok = la_wait(&bars[L::KFULL + st], (gj / kQKStages) & 1, end))) break;
                    if (!(ok = la_wait(&bars[L::QFULL + sq], (fj / kQKStages) & 1, end))) break;
                    const uint32_t k = desc_lo(sbase + L::QK + st * 2 * L::TB, 16);
                    const uint32_t q = desc_lo(sbase + L::QK + sq * 2 * L::TB + L::TB, 16), d = TM_T + 128u * (fj & 1);
                    if (leader) {
                        mma_steps<DK / 16>(d, idT, [&](int ks) { return q + (ks >> 2) * 1024 + (ks & 3) * 2; },
                                           [&](int ks) { return k + (ks >> 2) * 1024 + (ks & 3) * 2; });
                        mma_commit(&bars[L::TFULL + (fj & 1)]);
                        mma_commit(&bars[L::KEMPTY + st]);
                    }
                }
                if (i < 0) continue;
                const int gi = base + i, fi = full + i;
                if (!(ok = la_wait(&bars[L::SREADY], fi & 1, end))) break;
                if (leader) {  // into the place that P V of one chunk before has waited for
                    const uint32_t q = desc_lo(sbase + L::QK + (fi % kQKStages) * 2 * L::TB + L::TB, 16), x = desc_lo(sbase + L::S, 8192);
                    mma_steps<DK / 16>(TM_OS + 64u * (fi & 1), idO, [&](int ks) { return q + (ks >> 2) * 1024 + (ks & 3) * 2; },
                                       [&](int ks) { return x + ks * 128; });
                    mma_commit(&bars[L::SEMPTY]);
                    mma_commit(&bars[L::QEMPTY + fi % kQKStages]);
                }
                if (!(ok = la_wait(&bars[L::PREADY + (fi & 1)], (fi / 2) & 1, end))) break;
                if (!(ok = la_wait(&bars[L::VREADY + gi % kVStages], (gi / kVStages) & 1, end))) break;
                if (fi >= 1 && !(ok = la_wait(&bars[L::OEMPTY], (fi - 1) & 1, end))) break;
                tc_fence_after_sync();
                const uint32_t v = desc_lo(sbase + L::V + (gi % kVStages) * 16384, 8192), t = TM_T + 128u * (fi & 1);
                if (leader) {
                    mma_ts<0>(TM_OP, t, desc_of(v), idO);
#pragma unroll
                    for (int ks = 1; ks < kC / 16; ++ks) mma_ts<1>(TM_OP, t + 8 * ks, desc_of(v + ks * 128), idO);
                    mma_commit(&bars[L::OFULL]);
                    mma_commit(&bars[L::VEMPTY + gi % kVStages]);
                }
            }
        } else if (warp == 2) {
            // the chunk's share of the state, as far as the weighted values are there
            constexpr uint32_t idU = idesc_bf16(128, 64, true, true);
            const bool leader = elect_one();
            int xs = 4 * base % kXRing;  // slot of X, and its phase
            uint32_t xp = (4 * base / kXRing) & 1;
#pragma unroll 1
            for (int gi = base; gi < base + n; ++gi) {
                const int st = gi % kQKStages;
                uint32_t k = desc_lo(sbase + L::QK + st * 2 * L::TB, 16384);
                ok = la_wait(&bars[L::KFULL + st], (gi / kQKStages) & 1, end);
                if (gi >= 1) ok = ok && la_wait(&bars[L::UEMPTY], (gi - 1) & 1, end);
                tc_fence_after_sync();
#pragma unroll 1
                for (int qd = 0; qd < 4; ++qd, k += 256) {
                    ok = ok && la_wait(&bars[L::XREADY + xs], xp, end);
                    if (!ok) break;
                    const uint32_t x = desc_lo(sbase + L::X + xs * TERMS * 4096, 8192);
                    if (leader) {
                        if (qd == 0) mma_ss<0>(TM_U, desc_of(k), desc_of(x), idU);
                        else mma_ss<1>(TM_U, desc_of(k), desc_of(x), idU);
                        mma_ss<1>(TM_U, desc_of(k + 128), desc_of(x + 128), idU);
                        mma_ss<1>(TM_U, desc_of(k), desc_of(x + 256), idU);
                        mma_ss<1>(TM_U, desc_of(k + 128), desc_of(x + 384), idU);
                        if constexpr (TERMS == 3) {
                            mma_ss<1>(TM_U, desc_of(k), desc_of(x + 512), idU);
                            mma_ss<1>(TM_U, desc_of(k + 128), desc_of(x + 640), idU);
                        }
                        if (qd == 3) mma_commit(&bars[L::UFULL]);
                        mma_commit(&bars[L::XEMPTY + xs]);
                        if (qd == 3) mma_commit(&bars[L::KEMPTY + st]);
                    }
                    if (++xs == kXRing) xs = 0, xp ^= 1;
                }
                if (!ok) break;
            }
        } else if (warp == 3) {
            // a chunk's decays: e^{G - c_t}, log2(e) c_t, e^{c_r - c_t} with r the last
            // token of t's block of 32, and e^G; the next chunk's gates are on their
            // way meanwhile
            const bool per_head = p.a.flags & GDN_G_PER_HEAD;
            float next[4], whole = 0.f;
            auto fetch = [&](int i) {
                if (i >= n) return;
                load_gates<kC>(gate_ptr(p.a, chunk(i), h), p.a.sg.t, chunk(i).len, per_head, next);
            };
            fetch(0);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int gi = base + i, w = gi % kGRing;
                const Sums g = scan_sums(next);
                fetch(i + 1);
                if (gi >= kGRing && !(ok = la_wait(&bars[L::GEMPTY + w], (gi / kGRing - 1) & 1, end))) break;
                Weight wt[4];
                float c2[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    wt[j] = split_weight(exp2_fast(g.to_end[j] * kLog2e));
                    c2[j] = g.cum[j] * kLog2e;
                }
                uint4 *ws = reinterpret_cast<uint4 *>(wring + w * 384);
                ws[lane] = make_uint4(wt[0].h, wt[1].h, wt[2].h, wt[3].h);
                ws[lane + 32] = make_uint4(wt[0].m, wt[1].m, wt[2].m, wt[3].m);
                ws[lane + 64] = make_uint4(wt[0].l, wt[1].l, wt[2].l, wt[3].l);
                float4 *slot = reinterpret_cast<float4 *>(gring + w * 256);
                slot[lane] = make_float4(c2[0], c2[1], c2[2], c2[3]);
                const float r = __shfl_sync(~0u, c2[3], lane | 7);
                slot[lane + 32] = make_float4(exp2_fast(r - c2[0]), exp2_fast(r - c2[1]), exp2_fast(r - c2[2]), exp2_fast(r - c2[3]));
                if (lane == 0) dring[w] = expf(g.all);
                whole += g.all;
                if (share && i == n - 1 && lane == 0) p.plan.decay[(size_t)it.row * slots + it.slot] = expf(whole);
                mbar_arrive(&bars[L::GFULL + w]);
            }
        } else if (warp < 8) {
            // the state: a row of 64 columns a thread, in registers
            const int row = 32 * (warp & 3) + lane;
            const bool mine = row < DK;
            float S[64];
            const size_t page = (((size_t)seq * p.a.H + h) * DK + row) * DV + 64 * slice;
            const int piece = PLANNED ? it.piece >> 1 : 0;
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine && p.a.s0 && piece == 0) x = *reinterpret_cast<const float4 *>(p.a.s0 + page + e);
                S[e] = x.x, S[e + 1] = x.y, S[e + 2] = x.z, S[e + 3] = x.w;
            }
            if (PLANNED && !share)
#pragma unroll 1
                for (int j = 0; j < piece; ++j) {  // the shares before the piece, the first with s0 in it
                    const size_t at = (size_t)(it.row + j) * slots + it.slot;
                    ok = warp_ok(ok && share_wait(p.plan.flags + at, end));
                    if (!ok) break;
                    const float d = j ? __ldcg(p.plan.decay + at) : 0.f;
                    const float4 *from = reinterpret_cast<const float4 *>(p.plan.share + (at * DK + (mine ? row : 0)) * 64);
#pragma unroll
                    for (int e = 0; e < 64; e += 4) {
                        const float4 x = __ldcg(from + e / 4);
                        S[e] = fmaf(d, S[e], x.x), S[e + 1] = fmaf(d, S[e + 1], x.y);
                        S[e + 2] = fmaf(d, S[e + 2], x.z), S[e + 3] = fmaf(d, S[e + 3], x.w);
                    }
                }
            auto step = [&](int gi) {  // S = e^G S + the chunk's share
                const int w = gi % kGRing;
                ok = warp_ok(ok && la_wait(&bars[L::GFULL + w], (gi / kGRing) & 1, end) && la_wait(&bars[L::UFULL], gi & 1, end));
                if (!ok) return;
                const float d = dring[w];
                tc_fence_after_sync();
#pragma unroll
                for (int e = 0; e < 64; e += 16) {
                    uint32_t u[16];
                    tmem_ld16(tmem + lane_base(warp) + TM_U + e, u);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[e + j] = fmaf(d, S[e + j], __uint_as_float(u[j]));
                }
                tc_fence_before_sync();
                mbar_arrive(&bars[L::UEMPTY]);
                mbar_arrive(&bars[L::GEMPTY + w]);
            };
            if (share) {
#pragma unroll 1
                for (int gi = base; gi < base + n && ok; ++gi) step(gi);
            } else {
#pragma unroll 1
                for (int gi = base; gi < base + n && ok; ++gi) {
                    ok = la_wait(&bars[L::SEMPTY], (gi + full - base + 1) & 1, end);  // the first passes
                    if (mine)
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
                            *reinterpret_cast<uint4 *>(sm + L::S + sw128_offset(row, e)) =
                                make_uint4(pack_bf16(S[e], S[e + 1]), pack_bf16(S[e + 2], S[e + 3]), pack_bf16(S[e + 4], S[e + 5]),
                                           pack_bf16(S[e + 6], S[e + 7]));
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[L::SREADY]);
                    step(gi);
                }
            }
            if (share) {
                const size_t at = (size_t)it.row * slots + it.slot;
                if (mine && ok)
#pragma unroll
                    for (int e = 0; e < 64; e += 4)
                        *reinterpret_cast<float4 *>(p.plan.share + (at * DK + row) * 64 + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (ok && threadIdx.x == 128) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.plan.flags + at), "r"(1u) : "memory");
            } else if (p.a.sf && (it.piece & 1) && mine && ok) {
#pragma unroll
                for (int e = 0; e < 64; e += 4)
                    *reinterpret_cast<float4 *>(p.a.sf + page + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
            }
        } else if (share && (warp < 12 || warp >= 16)) {  // the decays pass by
#pragma unroll 1
            for (int gi = base; gi < base + n && ok; ++gi) {
                ok = la_wait(&bars[L::GFULL + gi % kGRing], (gi / kGRing) & 1, end);
                if (ok) mbar_arrive(&bars[L::GEMPTY + gi % kGRing]);
            }
        } else if (warp < 12) {
            // P in blocks of 16 columns, thread's row t.  On the warp's diagonal (32
            // columns) the decay is e^{c_t - c_s}; before it e^{c_t - c_r} e^{c_r - c_s}
            // with r the last token of s's block of 32, whose factors are both at most
            // 1 for decays, so that a row costs one exponential a block.
            const int t = 32 * (warp & 3) + lane, diag = 32 * (warp & 3);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int gi = base + i, fi = full + i, w = gi % kGRing;
                ok = warp_ok(la_wait(&bars[L::GFULL + w], (gi / kGRing) & 1, end) && la_wait(&bars[L::TFULL + (fi & 1)], (fi / 2) & 1, end));
                if (!ok) break;
                tc_fence_after_sync();
                const float *c2 = gring + w * 256, *cf = c2 + 128;
                const float ct = c2[t];
                const uint32_t tt = tmem + lane_base(warp) + TM_T + 128u * (fi & 1);
                uint32_t u[16], y[8];
#pragma unroll 1
                for (int s = 0; s < diag; s += 16) {
                    tmem_ld16(tt + s, u);
                    const float rf = exp2_fast(ct - c2[s | 31]);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(cf + s + j);
                        y[j / 2] = pack_bf16(__uint_as_float(u[j]) * (rf * f.x), __uint_as_float(u[j + 1]) * (rf * f.y));
                        y[j / 2 + 1] = pack_bf16(__uint_as_float(u[j + 2]) * (rf * f.z), __uint_as_float(u[j + 3]) * (rf * f.w));
                    }
                    tmem_st8(tt + s / 2, y);
                }
#pragma unroll 1
                for (int s = diag; s < diag + 32; s += 16) {
                    tmem_ld16(tt + s, u);
                    tmem_wait_ld();
                    const int last = t - s;  // the row's last column of the block
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 cs = *reinterpret_cast<const float4 *>(c2 + s + j);
                        const float x0 = j + 0 <= last ? __uint_as_float(u[j]) * exp2_fast(ct - cs.x) : 0.f;
                        const float x1 = j + 1 <= last ? __uint_as_float(u[j + 1]) * exp2_fast(ct - cs.y) : 0.f;
                        const float x2 = j + 2 <= last ? __uint_as_float(u[j + 2]) * exp2_fast(ct - cs.z) : 0.f;
                        const float x3 = j + 3 <= last ? __uint_as_float(u[j + 3]) * exp2_fast(ct - cs.w) : 0.f;
                        y[j / 2] = pack_bf16(x0, x1);
                        y[j / 2 + 1] = pack_bf16(x2, x3);
                    }
                    tmem_st8(tt + s / 2, y);
                }
                // P's columns past the diagonal take the place of T's that have been read
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = 0u;
#pragma unroll 1
                for (int s = diag + 32; s < kC; s += 16) tmem_st8(tt + s / 2, y);
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(&bars[L::PREADY + (fi & 1)]);
                mbar_arrive(&bars[L::GEMPTY + w]);
            }
        } else if (warp < 16) {
            // the weighted values, in quarters of 32 tokens: row r of each, 16 columns
            const int ct = threadIdx.x - 384, r = ct >> 2, c0 = (ct & 3) * 16;
            const uint32_t off[2] = {sw128_offset(r, c0), sw128_offset(r, c0 + 8)};
            int xs = 4 * base % kXRing;  // slot of X, and the phase of its last release
            uint32_t xp = (4 * base / kXRing + 1) & 1;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                const int gi = base + i, v = gi % kVStages, w = gi % kGRing, len = chunk(i).len;
                ok = la_wait(&bars[L::VFULL + v], (gi / kVStages) & 1, end) && la_wait(&bars[L::GFULL + w], (gi / kGRing) & 1, end);
                uint8_t *vt = sm + L::V + v * 16384;
                if (len < kC) {
                    // rows past the chunk's tokens are another sequence's: zeros, so
                    // that nothing of theirs (an infinity, say) meets a zero weight
                    ok = ok && la_wait(&bars[L::KFULL + gi % kQKStages], (gi / kQKStages) & 1, end);
                    uint8_t *k = sm + L::QK + (gi % kQKStages) * 2 * L::TB;
                    if (ok) {
#pragma unroll 1
                        for (int row = r; row < kC; row += 32)
                            if (row >= len) {
                                *reinterpret_cast<uint4 *>(vt + (row - r) * 128 + off[0]) = make_uint4(0, 0, 0, 0);
                                *reinterpret_cast<uint4 *>(vt + (row - r) * 128 + off[1]) = make_uint4(0, 0, 0, 0);
                            }
#pragma unroll 1
                        for (int e = ct; e < (kC - len) * (DK / 8); e += 128) {
                            const int row = len + e / (DK / 8), col = (e % (DK / 8)) * 8;
                            *reinterpret_cast<uint4 *>(k + (col >> 6) * 16384 + sw128_offset(row, col & 63)) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                }
                if (ok) mbar_arrive(&bars[L::VREADY + v]);
                const uint32_t *wr = wring + w * 384 + r;
#pragma unroll 1
                for (int qd = 0; qd < 4; ++qd, wr += 32, vt += 4096) {
                    const uint4 x[2] = {*reinterpret_cast<const uint4 *>(vt + off[0]), *reinterpret_cast<const uint4 *>(vt + off[1])};
                    const Weight wt = {wr[0], wr[128], wr[256]};
                    ok = ok && la_wait(&bars[L::XEMPTY + xs], xp, end);
                    if (!ok) break;
                    uint8_t *xb = sm + L::X + xs * TERMS * 4096;
                    if constexpr (TERMS == 3) {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint4 a, b, d;
                            weigh3(x[u].x, wt, a.x, b.x, d.x), weigh3(x[u].y, wt, a.y, b.y, d.y);
                            weigh3(x[u].z, wt, a.z, b.z, d.z), weigh3(x[u].w, wt, a.w, b.w, d.w);
                            *reinterpret_cast<uint4 *>(xb + off[u]) = a;
                            *reinterpret_cast<uint4 *>(xb + 4096 + off[u]) = b;
                            *reinterpret_cast<uint4 *>(xb + 8192 + off[u]) = d;
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint4 a, b;
                            weigh2(x[u].x, wt, a.x, b.x), weigh2(x[u].y, wt, a.y, b.y);
                            weigh2(x[u].z, wt, a.z, b.z), weigh2(x[u].w, wt, a.w, b.w);
                            *reinterpret_cast<uint4 *>(xb + off[u]) = a;
                            *reinterpret_cast<uint4 *>(xb + 4096 + off[u]) = b;
                        }
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[L::XREADY + xs]);
                    if (++xs == kXRing) xs = 0, xp ^= 1;
                }
                if (!ok) break;
                mbar_arrive(&bars[L::VEMPTY + v]);
                mbar_arrive(&bars[L::GEMPTY + w]);
            }
        } else {
            // the rows of O: scale (e^c (Q S) + P V)
            const int t = 32 * (warp & 3) + lane;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int gi = base + i, fi = full + i, w = gi % kGRing;
                ok = warp_ok(la_wait(&bars[L::OFULL], fi & 1, end));
                if (!ok) break;
                tc_fence_after_sync();
                const Chunk c = chunk(i);
                const float f = exp2_fast(gring[w * 256 + t]) * p.a.scale;
                const uint32_t ts = tmem + lane_base(warp) + TM_OS + 64u * (fi & 1), tp = tmem + lane_base(warp) + TM_OP;
                uint32_t z[4][8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x[16], y[16];
                    tmem_ld16(ts + 16 * e, x);
                    tmem_ld16(tp + 16 * e, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        z[e][j] = pack_bf16(fmaf(f, __uint_as_float(x[2 * j]), p.a.scale * __uint_as_float(y[2 * j])),
                                            fmaf(f, __uint_as_float(x[2 * j + 1]), p.a.scale * __uint_as_float(y[2 * j + 1])));
                }
                tc_fence_before_sync();
                mbar_arrive(&bars[L::OEMPTY]);
                mbar_arrive(&bars[L::GEMPTY + w]);
                exchange(z);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int u = (t & ~3) + e;
                    if (u >= c.len) break;
                    __nv_bfloat16 *out = at(static_cast<__nv_bfloat16 *>(p.a.o), p.a.so, c.row, h, c.t0 + u) + 64 * slice + 16 * (lane & 3);
                    if (p.wide) {
                        st_global_32(out, z[e]);
                    } else {
                        reinterpret_cast<uint4 *>(out)[0] = make_uint4(z[e][0], z[e][1], z[e][2], z[e][3]);
                        reinterpret_cast<uint4 *>(out)[1] = make_uint4(z[e][4], z[e][5], z[e][6], z[e][7]);
                    }
                }
            }
        }
        if (!PLANNED) break;
        __syncwarp();
        tc_fence_before_sync();
        const bool bad = __syncthreads_or(!ok);
        if (threadIdx.x == 0) *item = item[1];
        if (bad) break;
        __syncthreads();
        tc_fence_after_sync();
    }
    if (warp == 1 || warp == 2) {  // every MMA issued here is complete before TMEM is released
        if (elect_one()) mma_commit(&bars[L::DRAIN + warp - 1]);
        mbar_wait(&bars[L::DRAIN + warp - 1], 0, kDrainNs);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ================================================================ grad kernel
// Warps: 0..15 arithmetic (rows by lane quarter, columns in four parts), 16
// loads and products.
constexpr int kGradWork = 512, kGradThreads = kGradWork + 32;

struct GradSmem {
    static constexpr uint32_t Q = 0, K = 32768, V = 65536, O = 98304;  // V: later P
    // S hi, then R lo, then dv; S lo, then R's last term, then N, then dq; S's last term, then R hi, then dk
    static constexpr uint32_t X = 131072, Y = 163840, Z = 196608;
    static constexpr uint32_t G = 229376;                              // the chunk's decays, as state_kernel wrote them
    static constexpr uint32_t RED = G + 2048;
    static constexpr uint32_t BAR = RED + 64;  // 16 floats
    enum { QK = 0, OV, SS, RR, GT, LOADS = 5, CT = 5, CN, CQ, CK, DONE, TAIL, XREAD, READY, XFREE, ROWS, STORED, DRAIN, NUM };
    static constexpr uint32_t TSLOT = BAR + 8 * NUM;
    static constexpr uint32_t BYTES = TSLOT + 16;
};
static_assert(GradSmem::BYTES <= 232448, "grad kernel fits the shared memory of one CTA");
// TMEM columns: Q K^T, then P | N by blocks, then K R; dO V^T, then P^T dO; dQ; dK
constexpr uint32_t TM_A = 0, TM_B = 128, TM_Q = 256, TM_K = 384;

// Sums of x[j] over the warp's lanes (rows): lane's is column lane / 2.
__device__ __forceinline__ float column_sums(float (&x)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 8; m; m >>= 1) {
        const bool up = lane & (2 * m);
#pragma unroll
        for (int j = 0; j < m; ++j) {
            const float keep = up ? x[j + m] : x[j], give = up ? x[j] : x[j + m];
            x[j] = keep + __shfl_xor_sync(~0u, give, 2 * m);
        }
    }
    return x[0] + __shfl_xor_sync(~0u, x[0], 1);
}

// The chunks' gradients (the formulas are linattn.cu's): one CTA an SM takes
// (chunk, head) items in turn, the next item's tiles coming in as this one's
// places get free.
// Products: T = Q K^T and dO V^T; dO S^T and V R^T with S and R in terms; then,
// with P and N = dO V^T under the decay mask rounded to bf16, N K, N^T Q, P^T dO
// and K R.  What dg is made of never passes through a rounded operand: the
// pairs' terms A come from the fp32 products, the terms through S and R from
// the split ones.  Bound by the bytes and the chain of products and arithmetic
// behind them: 320 KB in, 96 KB out a chunk; at B4 H16 T4096, D 128, 171 us,
// 852 MB at 5.0 TB/s (74% of a plain copy's rate).
// dv's part through R takes R's first term alone (2^-9, as dv's own rounding); so
// do P and N, which costs dq and dk 2^-9 of each value head's part: where heads of
// one key cancel to 2^-4, up to 6e-2 of what is left of a chunk of more than 64
// tokens.
// P and N of a chunk of up to 64 tokens go into their products in two bf16 terms,
// in the tiles' other half: few pairs do not average the rounding out, and heads
// that share keys may cancel (1 token: dq 6e-2 off with one term).  The chunk
// alone decides, so that a sequence's precision does not depend on the call that it
// is in.  Both ways of the pairs' loop are compiled apart: as conditions in one
// loop they cost the long chunks 186 us in place of 171 (registers).
template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1) grad_kernel_tc(const __grid_constant__ GradMaps m, TcArgs p) {
    using L = GradSmem;
    using T = __nv_bfloat16;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::TSLOT);
    const float *hi = reinterpret_cast<const float *>(sm + L::G), *lo = hi + 128, *te = lo + 128, *cf = te + 128;
    float *red = reinterpret_cast<float *>(sm + L::RED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int items = p.v.n_chunks * p.a.H;
    const bool shared = p.a.H != p.a.Hk;
    const uint64_t end = deadline_after(p.timeout_ns, items / (int)gridDim.x + 1);
    if (threadIdx.x == 0) {
        for (int b = 0; b < L::NUM; ++b)
            mbar_init(&bars[b], b == L::XREAD || b == L::READY || b == L::TAIL || b == L::ROWS ? kGradWork : b == L::XFREE ? 32 : 1);
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's
    const uint32_t sbase = smem_u32(sm);

    if (warp == 16) {
        const bool leader = elect_one();
        int loads[L::LOADS] = {0, 0, 0, 0, 0};  // arrivals ordered on each of the loads' barriers
        auto order = [&](int bar, uint32_t bytes) {
            ++loads[bar];
            if (leader) mbar_arrive_expect_tx(&bars[bar], bytes);
        };
        auto tile = [&](const CUtensorMap *map, uint32_t to, int bar, int d, int head, const Chunk &c) {
            if (leader)
#pragma unroll
                for (int x = 0; x < d / 64; ++x) tma_load_4d(sm + to + x * 16384, map, &bars[bar], 64 * x, c.t0, head, c.row);
        };
        auto state = [&](const CUtensorMap *map, uint32_t to, int bar, int item) {
            if (leader)
#pragma unroll
                for (int x = 0; x < DV / 64; ++x) tma_load_3d(sm + to + x * (DK * 128), map, &bars[bar], 64 * x, 0, item);
        };
        // operands' low descriptor words: K-major tiles step by 32 bytes in a
        // block of 64 columns, MN-major ones by 16 rows
        auto km = [&](uint32_t at_, int rows) { return [=](int ks) { return desc_lo(sbase + at_, 16) + (ks >> 2) * (rows * 8) + (ks & 3) * 2; }; };
        auto mn = [&](uint32_t at_, uint32_t stride) { return [=](int ks) { return desc_lo(sbase + at_, stride) + ks * 128; }; };
        bool ok = true;
        uint32_t ph = 0, tails = 0;
        bool first = true;
#pragma unroll 1
        for (int it = blockIdx.x; it < items; it += gridDim.x) {
            const int ci = it / p.a.H, h = it - ci * p.a.H, hk = h / (p.a.H / p.a.Hk);
            const Chunk c = chunk_at<kC>(p.v, p.a.T, ci);
            if (c.len <= 0 || c.seq < 0) continue;
            // the item before this one: its products are done, and the tiles and
            // decays with them; its gradients' rows leave through X, Y and Z
            order(L::QK, 2 * DK * 256);
            tile(&m.q, L::Q, L::QK, DK, hk, c);
            tile(&m.k, L::K, L::QK, DK, hk, c);
            order(L::OV, 2 * DV * 256);
            tile(&m.o, L::O, L::OV, DV, h, c);
            tile(&m.v, L::V, L::OV, DV, h, c);
            order(L::GT, 2048);
            if (leader) bulk_load_global(sm + L::G, p.gates + (size_t)it * 512, 2048, &bars[L::GT]);
            if (!first) ok = la_wait(&bars[L::ROWS], ph ^ 1, end);
            if (!ok) break;
            tc_fence_after_sync();
            ok = la_wait(&bars[L::QK], ph, end);
            if (ok && c.len < kC) ok = la_wait(&bars[L::TAIL], tails++ & 1, end);
            if (!ok) break;
            if (leader) {
                mma_steps<DK / 16>(TM_A, idesc_bf16(128, 128, false, false), km(L::Q, 128), km(L::K, 128));
                mma_commit(&bars[L::CT]);
            }
            ok = la_wait(&bars[L::OV], ph, end);
            if (!ok) break;
            if (leader) {
                mma_steps<DV / 16>(TM_B, idesc_bf16(128, 128, false, false), km(L::O, 128), km(L::V, 128));
                mma_commit(&bars[L::CN]);
            }
            if (!first) ok = la_wait(&bars[L::STORED], ph ^ 1, end);
            if (!ok) break;
            first = false;
            order(L::SS, 3 * DK * DV * 2);
            state(&m.s[2], L::Z, L::SS, it);
            state(&m.s[1], L::Y, L::SS, it);
            state(&m.s[0], L::X, L::SS, it);
            constexpr uint32_t idk = idesc_bf16(128, DK, false, false);
            ok = la_wait(&bars[L::SS], ph, end);
            if (!ok) break;
            if (leader) {
                mma_steps<DV / 16>(TM_Q, idk, km(L::O, 128), km(L::Z, DK));  // the smaller terms first, as in state_kernel
                mma_more<DV / 16>(TM_Q, idk, km(L::O, 128), km(L::Y, DK));
                mma_more<DV / 16>(TM_Q, idk, km(L::O, 128), km(L::X, DK));
                mma_commit(&bars[L::CQ]);
            }
            // R's terms in S's places, which have been multiplied and read
            ok = la_wait(&bars[L::CQ], ph, end) && la_wait(&bars[L::XREAD], ph, end);
            if (!ok) break;
            order(L::RR, 3 * DK * DV * 2);
            state(&m.r[2], L::Y, L::RR, it);
            state(&m.r[1], L::X, L::RR, it);
            state(&m.r[0], L::Z, L::RR, it);
            ok = la_wait(&bars[L::RR], ph, end);
            if (!ok) break;
            if (leader) {
                mma_steps<DV / 16>(TM_K, idk, km(L::V, 128), km(L::Y, DK));
                mma_more<DV / 16>(TM_K, idk, km(L::V, 128), km(L::X, DK));
                mma_more<DV / 16>(TM_K, idk, km(L::V, 128), km(L::Z, DK));
                mma_commit(&bars[L::CK]);
            }
            ok = la_wait(&bars[L::READY], ph, end);
            if (!ok) break;
            tc_fence_after_sync();
            if (leader) {
                mma_more<kC / 16>(TM_Q, idesc_bf16(128, DK, false, true), km(L::Y, 128), mn(L::K, 16384));
                mma_more<kC / 16>(TM_K, idesc_bf16(128, DK, true, true), mn(L::Y, 16384), mn(L::Q, 16384));
                mma_steps<kC / 16>(TM_B, idesc_bf16(128, DV, true, true), mn(L::V, 16384), mn(L::O, 16384));
                mma_steps<DK / 16>(TM_A, idesc_bf16(128, DV, false, true), km(L::K, 128), mn(L::Z, DK * 128));
                mma_commit(&bars[L::DONE]);
            }
            ok = la_wait(&bars[L::DONE], ph, end);
            if (!ok) break;
            ph ^= 1;
        }
        if (!warp_ok(ok)) {  // no copy and no product is in flight when the CTA ends
            if (leader) mma_commit(&bars[L::DRAIN]);
            mbar_wait(&bars[L::DRAIN], 0, kDrainNs);
#pragma unroll
            for (int b = 0; b < L::LOADS; ++b)
                if (loads[b]) mbar_wait(&bars[b], (loads[b] - 1) & 1, kDrainNs);
        }
    } else {
        const int t = 32 * (warp & 3) + lane, four = warp >> 2, tid = threadIdx.x;
        const uint32_t lanes = tmem + lane_base(warp);
        bool ok = true;
        uint32_t ph = 0;
        // these warps' barrier.  A warp whose wait gave up comes to it all the
        // same, and none of them goes on.
        auto meet = [&] { ok = all_of<kGradWork>(ok); };
        auto wait = [&](int bar) { ok = warp_ok(ok && la_wait(&bars[bar], ph, end)); };
        // Scales the thread's part of its row of dQ or dK and gives its product
        // with the row of Q or K.
        auto scale_rows = [&](uint32_t col, float f, uint32_t tile_at) {
            float x = 0.f;
#pragma unroll 1
            for (int e = 0; e < DK / 4; e += 16) {
                const int d0 = four * (DK / 4) + e;
                uint32_t u[16];
                tmem_ld16(lanes + col + d0, u);
                float q[16];
#pragma unroll
                for (int j = 0; j < 16; j += 8) {
                    float y[8];
                    unpack8(*reinterpret_cast<const uint4 *>(sm + tile_at + ((d0 + j) >> 6) * 16384 + sw128_offset(t, (d0 + j) & 63)), y);
#pragma unroll
                    for (int k = 0; k < 8; ++k) q[j + k] = y[k];
                }
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float y = f * __uint_as_float(u[j]);
                    x = fmaf(q[j], y, x);
                    u[j] = __float_as_uint(y);
                }
                tmem_st16(lanes + col + d0, u);
            }
            return x;
        };
#pragma unroll 1
        for (int it = blockIdx.x; it < items; it += gridDim.x) {
            const int ci = it / p.a.H, h = it - ci * p.a.H, hk = h / (p.a.H / p.a.Hk);
            const Chunk c = chunk_at<kC>(p.v, p.a.T, ci);
            if (c.len <= 0) continue;
            T *dq = at(static_cast<T *>(p.a.dq), p.a.sq, c.row, hk, c.t0), *dk = at(static_cast<T *>(p.a.dk), p.a.sk, c.row, hk, c.t0);
            T *dv = at(static_cast<T *>(p.a.dv), p.a.sv, c.row, h, c.t0);
            float *dg = at(p.dgt, p.sdg, c.row, h, c.t0);
            const size_t wide_row = (((size_t)c.row * p.a.H + h) * p.a.T + c.t0) * DK;
            if (c.seq < 0) {  // tokens of no sequence
                auto zeros = [&](T *x, long long step, int d) {
#pragma unroll 1
                    for (int e = tid; e < c.len * (d / 8); e += kGradWork)
                        *reinterpret_cast<uint4 *>(x + (e / (d / 8)) * step + (e % (d / 8)) * 8) = make_uint4(0, 0, 0, 0);
                };
                if (shared) {
#pragma unroll 1
                    for (int e = tid; e < c.len * DK; e += kGradWork) p.dqh[wide_row + e] = p.dkh[wide_row + e] = 0.f;
                } else {
                    zeros(dq, p.a.sq.t, DK);
                    zeros(dk, p.a.sk.t, DK);
                }
                zeros(dv, p.a.sv.t, DV);
                for (int e = tid; e < c.len; e += kGradWork) dg[e * p.sdg.t] = 0.f;
                continue;
            }
            if (c.len < kC) {
                // another sequence's rows: zeros, so that nothing of theirs (an
                // infinity, say) reaches this one, and zeros come out of them
                wait(L::QK);
                wait(L::OV);
#pragma unroll 1
                for (int e = tid; e < (kC - c.len) * 16; e += kGradWork) {
                    const int row = c.len + (e >> 4), col = (e & 15) * 8;
                    const uint32_t o = (col >> 6) * 16384 + sw128_offset(row, col & 63);
                    if (col < DK) *reinterpret_cast<uint4 *>(sm + L::Q + o) = make_uint4(0, 0, 0, 0);
                    if (col < DK) *reinterpret_cast<uint4 *>(sm + L::K + o) = make_uint4(0, 0, 0, 0);
                    if (col < DV) *reinterpret_cast<uint4 *>(sm + L::O + o) = make_uint4(0, 0, 0, 0);
                    if (col < DV) *reinterpret_cast<uint4 *>(sm + L::V + o) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                if (ok) mbar_arrive(&bars[L::TAIL]);
            }
            const bool half = c.len <= 64;
            float rowa = 0.f, cola[2] = {0.f, 0.f}, dot = 0.f, xt = 0.f, yt = 0.f;
            wait(L::GT);
            wait(L::CT);
            wait(L::CN);
            tc_fence_after_sync();
            // P, N and A of the thread's row, a block of 16 columns at a time (every
            // fourth is this warp's).  The decays as in
            // prompt_kernel, with c_t - c_s from the pairs.
            const float ht = hi[t], lt = lo[t];
            auto pairs = [&](auto two) __attribute__((always_inline)) {
                constexpr bool TWO = decltype(two)::value;
#pragma unroll 1
                for (int k = 0; k < (TWO ? 1 : 2) && ok; ++k) {
                    const int sb = 16 * (4 * k + four), diag = 32 * (warp & 3);
                    uint32_t u[16];
                    if (sb >= diag + 32) {  // past the diagonal for every row of the warp
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = 0u;
                        tmem_st16(lanes + TM_A + sb, u);
                        if constexpr (TWO) tmem_st16(lanes + TM_A + 64 + sb, u);
                        continue;
                    }
                    uint32_t w[16];
                    float a[16];
                    tmem_ld16(lanes + TM_A + sb, u);
                    tmem_ld16(lanes + TM_B + sb, w);
                    const int r = sb | 31;
                    const float rf = p.a.scale * expf(((ht - hi[r]) + (lt - lo[r])));
                    tmem_wait_ld();
                    if (sb < diag) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 f4 = *reinterpret_cast<const float4 *>(cf + sb + j);
                            const float f[4] = {rf * f4.x, rf * f4.y, rf * f4.z, rf * f4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float qk = __uint_as_float(u[j + e]), nn = __uint_as_float(w[j + e]) * f[e];
                                a[j + e] = qk * nn;
                                u[j + e] = __float_as_uint(qk * f[e]);
                                w[j + e] = __float_as_uint(nn);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int s = sb + j;
                            const float f = s <= t ? p.a.scale * expf(((ht - hi[s]) + (lt - lo[s]))) : 0.f;
                            const float qk = __uint_as_float(u[j]), nn = __uint_as_float(w[j]) * f;
                            a[j] = s < t ? qk * nn : 0.f;
                            u[j] = __float_as_uint(qk * f);
                            w[j] = __float_as_uint(nn);
                        }
                    }
                    uint32_t pn[16];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        pn[j] = pack_bf16(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
                        pn[j + 8] = pack_bf16(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
                        rowa += a[2 * j] + a[2 * j + 1];
                    }
                    tmem_st16(lanes + TM_A + sb, pn);  // until their tiles' places are free
                    if constexpr (TWO) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            pn[j] = pack_bf16(__uint_as_float(u[2 * j]) - __uint_as_float(pn[j] << 16),
                                              __uint_as_float(u[2 * j + 1]) - __uint_as_float(pn[j] & 0xffff0000u));
                            pn[j + 8] = pack_bf16(__uint_as_float(w[2 * j]) - __uint_as_float(pn[j + 8] << 16),
                                                  __uint_as_float(w[2 * j + 1]) - __uint_as_float(pn[j + 8] & 0xffff0000u));
                        }
                        tmem_st16(lanes + TM_A + 64 + sb, pn);
                    }
                    const float sum = column_sums(a);
#pragma unroll
                    for (int j = 0; j < 2; ++j) cola[j] = j == k ? sum : cola[j];
                }
            };
            if (half) pairs(std::true_type{});
            else pairs(std::false_type{});
            // the thread's part of S for <R, S>, until R is there
            constexpr int NV = DK * DV / 8 / kGradWork;  // 16-byte words of a term a thread
            auto words = [&](int e, float (&x)[8], uint32_t t0, uint32_t t1, uint32_t t2) {  // t0's are the largest
                const uint32_t o = (tid + kGradWork * e) * 16;
                float y[8], z[8];
                unpack8(*reinterpret_cast<const uint4 *>(sm + t0 + o), x);
                unpack8(*reinterpret_cast<const uint4 *>(sm + t1 + o), y);
                unpack8(*reinterpret_cast<const uint4 *>(sm + t2 + o), z);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] += y[j] + z[j];
            };
            wait(L::SS);
            float sw[NV][8];
#pragma unroll
            for (int e = 0; e < NV; ++e) words(e, sw[e], L::X, L::Y, L::Z);
            if (ok) mbar_arrive(&bars[L::XREAD]);
            // dQ's part through S: scaled by its row, and x_t = q_t . it
            const float fe = expf(te[t]), whole = expf(hi[c.len - 1]);
            wait(L::CQ);
            tc_fence_after_sync();
            if (ok) xt = scale_rows(TM_Q, p.a.scale * expf(ht), L::Q);
            wait(L::RR);
#pragma unroll
            for (int e = 0; e < NV; ++e) {
                float r[8];
                words(e, r, L::Z, L::X, L::Y);
#pragma unroll
                for (int j = 0; j < 8; ++j) dot = fmaf(sw[e][j], r[j], dot);
            }
            wait(L::CK);
            tc_fence_after_sync();
            if (ok) yt = scale_rows(TM_K, fe, L::K);
            meet();
            if (ok) {
                // R's last term and V have been multiplied, and read by all: N and P
                // take their places
                tmem_wait_st();
                if (half) {
                    // rows 64.. repeat the rows 64 before them, for the second terms
                    auto repeat = [&](uint32_t tile_at, int d) {
                        for (int e = four * (d / 4); e < (four + 1) * (d / 4); e += 8) {
                            uint8_t *x = sm + tile_at + (e >> 6) * 16384 + sw128_offset(t, e & 63);
                            *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(x - 8192);
                        }
                    };
                    if (warp & 2) {
                        repeat(L::Q, DK);
                        repeat(L::K, DK);
                        repeat(L::O, DV);
                    } else {
                        const uint32_t at_[2] = {sw128_offset(t, 16 * four), sw128_offset(t, 16 * four + 8)};
#pragma unroll 1
                        for (int k = 0; k < 2; ++k) {  // first and second terms: P | N of 16 columns
                            uint32_t pn[16];
                            tmem_ld16(lanes + TM_A + 64 * k + 16 * four, pn);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint4 zero = make_uint4(0, 0, 0, 0);
                                const uint4 pp = make_uint4(pn[4 * x], pn[4 * x + 1], pn[4 * x + 2], pn[4 * x + 3]);
                                const uint4 nn = make_uint4(pn[4 * x + 8], pn[4 * x + 9], pn[4 * x + 10], pn[4 * x + 11]);
                                uint8_t *v = sm + L::V + at_[x], *y = sm + L::Y + at_[x];
                                *reinterpret_cast<uint4 *>(v + 8192 * k) = pp;
                                *reinterpret_cast<uint4 *>(v + 16384 + 8192 * k) = zero;
                                *reinterpret_cast<uint4 *>(y + 8192 * k) = nn;
                                *reinterpret_cast<uint4 *>(y + 16384 + 8192 * k) = zero;
                                if (k) *reinterpret_cast<uint4 *>(y + 16384) = nn;
                            }
                        }
                    }
                } else
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int sb = 16 * (4 * k + four);
                    uint32_t pn[16];
                    tmem_ld16(lanes + TM_A + sb, pn);
                    tmem_wait_ld();
                    const uint32_t o = (sb >> 6) * 16384, o0 = o + sw128_offset(t, sb & 63), o1 = o + sw128_offset(t, (sb & 63) + 8);
                    *reinterpret_cast<uint4 *>(sm + L::V + o0) = make_uint4(pn[0], pn[1], pn[2], pn[3]);
                    *reinterpret_cast<uint4 *>(sm + L::V + o1) = make_uint4(pn[4], pn[5], pn[6], pn[7]);
                    *reinterpret_cast<uint4 *>(sm + L::Y + o0) = make_uint4(pn[8], pn[9], pn[10], pn[11]);
                    *reinterpret_cast<uint4 *>(sm + L::Y + o1) = make_uint4(pn[12], pn[13], pn[14], pn[15]);
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                mbar_arrive(&bars[L::READY]);
            }
            // dg meanwhile, through R lo's place: partial sums by token, A's rows, x
            // and y (4 parts of the columns), A's columns (4 quarters of the rows)
            float *part = reinterpret_cast<float *>(sm + L::X);
            meet();
            part[four * 128 + t] = rowa;
            part[512 + four * 128 + t] = xt;
            part[1024 + four * 128 + t] = yt;
            if (!(lane & 1))
#pragma unroll
                for (int k = 0; k < 2; ++k) part[1536 + (warp & 3) * 128 + 16 * (4 * k + four) + lane / 2] = cola[k];
#pragma unroll
            for (int i = 16; i; i >>= 1) dot += __shfl_xor_sync(~0u, dot, i);
            if (lane == 0) red[warp] = dot;
            meet();
            if (warp == 0 && ok) {
                // dg_u = sum_{t >= u} (x_t + A's row t - A's column t) + sum_{t < u} y_t + e^G <R, S>
                float x[4], y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float *q = part + 4 * lane + j;
                    auto four_of = [&](int i) { return (q[i] + q[i + 128]) + (q[i + 256] + q[i + 384]); };
                    x[j] = four_of(512) + (four_of(0) - four_of(1536));
                    y[j] = four_of(1024);
                }
                float d = 0.f;
#pragma unroll
                for (int w = 0; w < kGradWork / 32; ++w) d += red[w];
                d *= whole;
                mbar_arrive(&bars[L::XFREE]);
                x[2] += x[3], x[1] += x[2], x[0] += x[1];
                float from = x[0], before = (y[0] + y[1]) + (y[2] + y[3]);
#pragma unroll
                for (int i = 1; i < 32; i <<= 1) {
                    const float a = __shfl_down_sync(~0u, from, i), b = __shfl_up_sync(~0u, before, i);
                    if (lane + i < 32) from += a;
                    if (lane >= i) before += b;
                }
                const float after = __shfl_down_sync(~0u, from, 1), prior = __shfl_up_sync(~0u, before, 1);
                float low = lane > 0 ? prior : 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int u = 4 * lane + j;
                    if (u < c.len) dg[u * p.sdg.t] = (x[j] + (lane < 31 ? after : 0.f)) + (low + d);
                    low += y[j];
                }
            }
            wait(L::DONE);
            tc_fence_after_sync();
            // the rows of the gradients: bf16 through the tiles Y, Z and X, so that
            // the stores are whole rows; fp32 (shared heads) straight
            auto rows = [&](uint32_t col, uint32_t tile_at, int d, float *wide, bool both) {
                if (wide && d == 128) {
                    uint32_t z[4][8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) tmem_ld8(lanes + col + four * 32 + 8 * e, z[e]);
                    tmem_wait_ld();
                    exchange(z);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = (t & ~3) + e;
                        if (u < c.len) st_global_32(wide + (size_t)u * d + four * 32 + 8 * (lane & 3), z[e]);
                    }
                    return;
                }
#pragma unroll 1
                for (int e = 0; e < d / 4; e += 16) {
                    const int d0 = four * (d / 4) + e;
                    uint32_t u[16], w[16];
                    tmem_ld16(lanes + col + d0, u);
                    if (both) tmem_ld16(lanes + TM_B + d0, w);
                    tmem_wait_ld();
                    if (both)
#pragma unroll
                        for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(fmaf(fe, __uint_as_float(u[j]), __uint_as_float(w[j])));
                    if (wide) {
                        if (t < c.len)
#pragma unroll
                            for (int j = 0; j < 16; j += 8) {
                                const uint32_t y[8] = {u[j], u[j + 1], u[j + 2], u[j + 3], u[j + 4], u[j + 5], u[j + 6], u[j + 7]};
                                st_global_32(wide + (size_t)t * d + d0 + j, y);
                            }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = pack_bf16(__uint_as_float(u[j + 2 * k]), __uint_as_float(u[j + 2 * k + 1]));
                            *reinterpret_cast<uint4 *>(sm + tile_at + ((d0 + j) >> 6) * 16384 + sw128_offset(t, (d0 + j) & 63)) =
                                make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
            };
            wait(L::XFREE);
            if (ok) {
#pragma unroll 1
                for (int k = 0; k < 2; ++k)
                    rows(k ? TM_K : TM_Q, k ? L::Z : L::Y, DK, shared ? (k ? p.dkh : p.dqh) + wide_row : nullptr, false);
                rows(TM_A, L::X, DV, nullptr, true);
            }
            fence_proxy_async_smem();
            tc_fence_before_sync();
            if (ok) mbar_arrive(&bars[L::ROWS]);
            meet();
            if (!ok) break;
            if (c.len == kC) {
                if (tid == 0) {
#pragma unroll
                    for (int x = 0; x < DK / 64; ++x) {
                        if (shared) break;
                        tma_store_4d(&m.dq, sm + L::Y + x * 16384, 64 * x, c.t0, hk, c.row);
                        tma_store_4d(&m.dk, sm + L::Z + x * 16384, 64 * x, c.t0, hk, c.row);
                    }
#pragma unroll
                    for (int x = 0; x < DV / 64; ++x) tma_store_4d(&m.dv, sm + L::X + x * 16384, 64 * x, c.t0, h, c.row);
                    tma_store_commit();
                    tma_store_wait_read<0>();
                    mbar_arrive(&bars[L::STORED]);
                }
            } else {
                auto store = [&](T *x, long long step, int d, uint32_t tile_at) {
#pragma unroll 1
                    for (int e = tid; e < c.len * (d / 8); e += kGradWork) {
                        const int row = e / (d / 8), col = (e % (d / 8)) * 8;
                        *reinterpret_cast<uint4 *>(x + row * step + col) =
                            *reinterpret_cast<const uint4 *>(sm + tile_at + (col >> 6) * 16384 + sw128_offset(row, col & 63));
                    }
                };
                if (!shared) {
                    store(dq, p.a.sq.t, DK, L::Y);
                    store(dk, p.a.sk.t, DK, L::Z);
                }
                store(dv, p.a.sv.t, DV, L::X);
                meet();
                if (tid == 0) mbar_arrive(&bars[L::STORED]);
            }
            ph ^= 1;
        }
        if (tid == 0) tma_store_wait_all<0>();
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ==================================================================== host side
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}

// 4-D map over a strided [B][heads][T][D] bf16 tensor with a box of 64 columns
// and `rows` tokens of one head.
bool strided_map(CUtensorMap *m, const void *base, const Strides &s, int B, int heads, int T, int D, int rows) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)B};
    // a dimension of one element has no stride that matters, but the map wants one
    const cuuint64_t strides[3] = {(cuuint64_t)(T > 1 ? 2 * s.t : 2 * D), (cuuint64_t)(heads > 1 ? 2 * s.h : 2 * D),
                                   (cuuint64_t)(B > 1 ? 2 * s.b : 2 * D)};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Strides that a map can hold (0: an expanded tensor).
bool mappable(const Strides &s, int B, int heads, int T) {
    auto ok = [](int n, long long x) { return n <= 1 || (x > 0 && x < (1LL << 38)); };
    return ok(B, s.b) && ok(heads, s.h) && ok(T, s.t);
}

// Over the chunk states [n][DK][DV].
bool state_map(CUtensorMap *m, const void *base, long long n, int DK, int DV) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)DV, (cuuint64_t)DK, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)DV * 2, (cuuint64_t)DV * DK * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)DK, 1}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up(size_t x) { return (x + 1023) / 1024 * 1024; }

int launched() {
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

// Raises a kernel's shared-memory limit, once for each device.
template <auto F>
bool smem_limit(uint32_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(F, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Chunks of a piece where cutting may pay (0: it does not): of the rows, whose
// length is known, or, packed, if one sequence had all of the tokens.  What it
// must save is more there, as lengths that need no cut lose by the plan and the
// costs are up to a fifth off for ragged ones (32760 tokens of 32 heads, states
// out: one sequence 517 -> 472 us, but eight equal ones 283 -> 318 and eight of
// 21001 tokens and fewer 357 -> 413; of 16 heads: one 560 -> 290, so those are cut
// and these are not).
int plan_len(const LinAttnArgs &a) {
    const int slots = a.H * (a.Dv / 64), seqs = a.cu ? 1 : a.B;
    const int n = (int)(((long long)a.T + kC - 1) / kC);
    const long long chunks = (long long)seqs * n * slots;
    float best = (a.cu ? 0.6f : 0.8f) * plan_cost(chunks, 0, n, (long long)seqs * slots, 0, 1);
    int found = 0;
    for (int p = 2; p <= kMostPieces; ++p) {
        const int len = (n + p - 1) / p;
        const long long rows = (long long)seqs * (pieces_of(n, len) - 1);
        if (rows * slots > kShareItems) break;
        const float cost = plan_cost(chunks, rows * len * slots, len, (seqs + 2 * rows) * slots, rows * slots, p);
        if (cost < best) best = cost, found = len;
    }
    return found;
}

Plan plan_at(const LinAttnArgs &a, void *ws, size_t *bytes) {
    Plan l{};
    *bytes = 0;
    if (!plan_len(a)) return l;
    const size_t slots = (size_t)a.H * (a.Dv / 64);
    l.rows = (int)(kShareItems / slots);
    const uintptr_t p0 = up(reinterpret_cast<uintptr_t>(ws));
    uintptr_t p = p0;
    auto room = [&](size_t n) {
        const uintptr_t at = p;
        p += up(n);
        return at;
    };
    l.head = reinterpret_cast<int *>(room(16));
    l.shares = reinterpret_cast<int4 *>(room(16 * (size_t)l.rows));
    l.pieces = reinterpret_cast<int4 *>(room(16 * ((size_t)a.n_seq + l.rows)));
    l.flags = reinterpret_cast<unsigned *>(room(4 * l.rows * slots));
    l.decay = reinterpret_cast<float *>(room(4 * l.rows * slots));
    l.share = reinterpret_cast<float *>(room(256 * l.rows * slots * a.Dk));
    *bytes = p - p0 + 1024;
    return l;
}

template <int DK, int DV, int TERMS>
int launch_prompt(const CUtensorMap &mQ, const CUtensorMap &mK, const CUtensorMap &mV, const TcArgs &p, cudaStream_t stream) {
    const LinAttnArgs &a = p.a;
    constexpr uint32_t bytes = FwdSmem<DK>::BYTES;
    if (!p.plan.head) {
        if (!smem_limit<prompt_kernel<DK, DV, false, TERMS>>(bytes)) return GDN_ERR_CUDA;
        const dim3 grid(DV / 64, a.H, a.n_seq + (a.cu ? 1 : 0));
        prompt_kernel<DK, DV, false, TERMS><<<grid, kFwdThreads, bytes, stream>>>(mQ, mK, mV, p);
        return launched();
    }
    if (!smem_limit<prompt_kernel<DK, DV, true, TERMS>>(bytes)) return GDN_ERR_CUDA;
    plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, p.plan, a.H * (DV / 64), a.cu ? 0 : plan_len(a));
    const int st = launched();
    if (st != GDN_OK) return st;
    prompt_kernel<DK, DV, true, TERMS><<<device_sm_count(), kFwdThreads, bytes, stream>>>(mQ, mK, mV, p);
    return launched();
}

template <int DK, int DV>
int run_fwd(const TcArgs &p, cudaStream_t stream) {
    const LinAttnArgs &a = p.a;
    if (!mappable(a.sq, a.B, a.Hk, a.T) || !mappable(a.sk, a.B, a.Hk, a.T) || !mappable(a.sv, a.B, a.H, a.T))
        return GDN_ERR_UNSUPPORTED;
    CUtensorMap mQ, mK, mV;
    if (!strided_map(&mQ, a.q, a.sq, a.B, a.Hk, a.T, DK, kC) || !strided_map(&mK, a.k, a.sk, a.B, a.Hk, a.T, DK, kC) ||
        !strided_map(&mV, a.v, a.sv, a.B, a.H, a.T, DV, kC))
        return GDN_ERR_CUDA;
    TcArgs w = p;
    w.wide = ((reinterpret_cast<uintptr_t>(a.o) | 2 * a.so.b | 2 * a.so.h | 2 * a.so.t) & 31) == 0;
    return a.sf ? launch_prompt<DK, DV, 3>(mQ, mK, mV, w, stream) : launch_prompt<DK, DV, 2>(mQ, mK, mV, w, stream);
}

// Chunks of a piece of the backward's walks (0: they are not cut), as plan_len:
// two launches of the walks' CTAs, of which the shares write no states.  Where
// the CTAs fill the SMs a chunk takes 1.4 of its time alone (the bytes bound it).
// D 128: 1 x 32768 tokens of 4 heads 115 us, uncut 404; 1 x 4096 of one head 29
// and 55; but of 16 heads 490 and 451, which are left uncut.
int cut_len(const LinAttnArgs &a) {
    const int slots = 2 * a.H * (a.Dv / 64), seqs = a.cu ? 1 : a.B;
    const int n = (int)(((long long)a.T + kC - 1) / kC);
    auto pass = [](long long items, int len) {
        return items <= kSms ? (float)len : fmaxf((float)len, 1.4f * items * len / kSms + 0.5f * len);
    };
    float best = (a.cu ? 0.6f : 0.8f) * pass((long long)seqs * slots, n);
    int found = 0;
    for (int p = 2; p <= kMostPieces; ++p) {
        const int len = (n + p - 1) / p, k = pieces_of(n, len);
        if (((long long)chunk_bound(a, len * kC)) * slots > 2 * kShareItems) break;
        const float cost = kCutShare * pass((long long)seqs * slots * (k - 1), len) + pass((long long)seqs * slots * k, len) +
                           2 * kItemCost + kJoinCost * k;
        if (cost < best) best = cost, found = len;
    }
    return found;
}

struct BwdWs {
    char *S[6];  // the terms of S, then R's
    float *gates, *dqh, *dkh, *dgt, *share, *decay;
    void *tables;  // the pieces'
    int len;
    size_t bytes;
};

BwdWs bwd_ws(const LinAttnArgs &a, void *ws) {
    const size_t states = up(2 * (size_t)chunk_bound(a, kC) * a.H * a.Dk * a.Dv);
    const size_t heads = a.H != a.Hk ? up(4 * (size_t)a.B * a.H * a.T * a.Dk) : 0;
    // 1024-byte alignment for the kernels' wide stores, whatever the caller's
    char *p = reinterpret_cast<char *>(up(reinterpret_cast<uintptr_t>(ws) + table_bytes(a, kC)));
    BwdWs w{};
    for (char *&s : w.S) s = p, p += states;
    w.gates = reinterpret_cast<float *>(p), p += up(2048 * (size_t)chunk_bound(a, kC) * a.H);
    w.dqh = reinterpret_cast<float *>(p), p += heads;
    w.dkh = reinterpret_cast<float *>(p), p += heads;
    w.dgt = reinterpret_cast<float *>(p), p += (a.flags & GDN_G_PER_HEAD) ? up(4 * (size_t)a.B * a.H * a.T) : 0;
    if ((w.len = cut_len(a))) {
        const size_t pieces = chunk_bound(a, w.len * kC);
        w.tables = p, p += up(table_bytes(a, w.len * kC));
        w.share = reinterpret_cast<float *>(p), p += up(8 * pieces * a.H * a.Dk * a.Dv);
        w.decay = reinterpret_cast<float *>(p), p += up(8 * pieces * a.H);
    }
    w.bytes = p - static_cast<char *>(ws) + 1024;
    return w;
}

template <int DK, int DV>
int run_bwd(const TcArgs &p, cudaStream_t stream) {
    const LinAttnArgs &a = p.a;
    if (!mappable(a.sq, a.B, a.Hk, a.T) || !mappable(a.sk, a.B, a.Hk, a.T) || !mappable(a.sv, a.B, a.H, a.T) ||
        !mappable(a.sdo, a.B, a.H, a.T))
        return GDN_ERR_UNSUPPORTED;
    GradMaps m;
    for (int i = 0; i < 3; ++i)
        if (!state_map(&m.s[i], p.S[i], (long long)p.v.n_chunks * a.H, DK, DV) ||
            !state_map(&m.r[i], p.R[i], (long long)p.v.n_chunks * a.H, DK, DV))
            return GDN_ERR_CUDA;
    if (!strided_map(&m.q, a.q, a.sq, a.B, a.Hk, a.T, DK, kC) || !strided_map(&m.k, a.k, a.sk, a.B, a.Hk, a.T, DK, kC) ||
        !strided_map(&m.v, a.v, a.sv, a.B, a.H, a.T, DV, kC) || !strided_map(&m.o, a.dout, a.sdo, a.B, a.H, a.T, DV, kC) ||
        !strided_map(&m.dq, a.dq, a.sq, a.B, a.Hk, a.T, DK, kC) || !strided_map(&m.dk, a.dk, a.sk, a.B, a.Hk, a.T, DK, kC) ||
        !strided_map(&m.dv, a.dv, a.sv, a.B, a.H, a.T, DV, kC))
        return GDN_ERR_CUDA;
    constexpr uint32_t bytes = StateSmem<DK>::BYTES;
    if (!smem_limit<state_kernel<DK, DV, false>>(bytes) || !smem_limit<state_kernel<DK, DV, true>>(bytes) ||
        !smem_limit<grad_kernel_tc<DK, DV>>(GradSmem::BYTES))
        return GDN_ERR_CUDA;
    int st = GDN_OK;
    dim3 grid(2 * DV / 64, a.H, a.n_seq);
    if (p.cut.len) {
        grid.z = p.cut.pieces.n_chunks + (a.cu ? a.n_seq : 0);
        state_kernel<DK, DV, true><<<grid, kStateThreads, bytes, stream>>>(m, p);
        if ((st = launched()) != GDN_OK) return st;
    }
    state_kernel<DK, DV, false><<<grid, kStateThreads, bytes, stream>>>(m, p);
    if ((st = launched()) != GDN_OK) return st;
    const long long items = (long long)p.v.n_chunks * a.H;
    const int sms = device_sm_count();
    const unsigned ctas = (unsigned)(items < sms ? items : sms);
    grad_kernel_tc<DK, DV><<<ctas, kGradThreads, GradSmem::BYTES, stream>>>(m, p);
    return launched();
}

}  // namespace
}  // namespace la

using namespace la;

bool linattn_tc_supported(const LinAttnArgs &a) {
    return a.dtype == GDN_BF16 && !(a.flags & GDN_PATH_SIMT) && sm100_family();
}

size_t linattn_tc_fwd_workspace(const LinAttnArgs &a) {
    size_t bytes;
    plan_at(a, nullptr, &bytes);
    return bytes;
}

int launch_linattn_tc_fwd(const LinAttnArgs &a, cudaStream_t stream) {
    TcArgs p{};
    p.a = a;
    p.timeout_ns = wait_limit_ns();
    size_t bytes;
    p.plan = plan_at(a, a.ws, &bytes);
    if (a.Dk == 128) return a.Dv == 128 ? run_fwd<128, 128>(p, stream) : run_fwd<128, 64>(p, stream);
    return a.Dv == 128 ? run_fwd<64, 128>(p, stream) : run_fwd<64, 64>(p, stream);
}

size_t linattn_tc_bwd_workspace(const LinAttnArgs &a) { return bwd_ws(a, nullptr).bytes; }

int launch_linattn_tc_bwd(const LinAttnArgs &a, cudaStream_t stream) {
    TcArgs p{};
    p.a = a;
    p.timeout_ns = wait_limit_ns();
    const BwdWs w = bwd_ws(a, a.ws);
    int st = make_view(a, kC, a.ws, &p.v, stream);
    if (st != GDN_OK) return st;
    for (int i = 0; i < 3; ++i) {
        p.S[i] = reinterpret_cast<uint16_t *>(w.S[i]);
        p.R[i] = reinterpret_cast<uint16_t *>(w.S[3 + i]);
    }
    if (w.len) {
        st = make_view(a, w.len * kC, w.tables, &p.cut.pieces, stream);
        if (st != GDN_OK) return st;
        p.cut.len = w.len, p.cut.share = w.share, p.cut.decay = w.decay;
    }
    p.gates = w.gates, p.dqh = w.dqh, p.dkh = w.dkh;
    const bool per_head = a.flags & GDN_G_PER_HEAD;
    p.dgt = per_head ? w.dgt : a.dg;
    p.sdg = per_head ? Strides{(long long)a.H * a.T, a.T, 1} : a.sg;
    if (a.Dk == 128) st = a.Dv == 128 ? run_bwd<128, 128>(p, stream) : run_bwd<128, 64>(p, stream);
    else st = a.Dv == 128 ? run_bwd<64, 128>(p, stream) : run_bwd<64, 64>(p, stream);
    if (st == GDN_OK && a.H != a.Hk) st = launch_group_sum(a, w.dqh, w.dkh, stream);
    if (st == GDN_OK && per_head) st = launch_head_sum(w.dgt, a.dg, a.B, a.H, a.T, stream);
    return st;
}

int linattn_tc_read_clear_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_la_error, sizeof(v)) != cudaSuccess) return GDN_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_la_error, &zero, sizeof(zero)) != cudaSuccess) return GDN_ERR_CUDA;
    return v ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
