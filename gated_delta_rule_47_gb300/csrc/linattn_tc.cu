// linattn_tc.cu -- linear attention with a decay for each head over whole
// prompts on the tensor cores (bf16, tcgen05), in chunks of 128 tokens.  The
// formulas are linattn.cu's.  Two launches:
//
// state_kernel walks a sequence's chunks with the state in registers and
// writes the state that enters each chunk as a bf16 operand.  A CTA owns 64
// value columns of one head (columns are independent, and only the value
// tile is weighted, so nothing is computed twice).  The chunk's own share
// K^T diag(w) V is one product that does not depend on the state, so the walk
// itself costs one multiply-add an element and chunk.  The weighted values
// w v go in as three bf16 terms (x = hi + mid + lo to 2^-24): with one, the
// state would carry 2^-9 of rounding in every term, against inputs that are
// exact; sums and state stay in fp32.
//
// out_kernel takes every chunk by itself: O = e^c (Q S) + (Q K^T o D) V with
// the decay mask D applied in fp32 between the two products.  P and S enter
// the products rounded to bf16: each adds about as much as the output's own
// rounding does.
//
// Both are bound by the bytes of q, k, v, o and the states (k and v are read
// twice, a state is 32 KB a chunk and head written and read).
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

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

// Waits for the phase of the given parity for at most limit ns; gives up at
// once when another wait has.
__device__ __forceinline__ bool la_wait(uint64_t *bar, uint32_t parity, unsigned code, unsigned long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
        if (*reinterpret_cast<volatile unsigned *>(&g_la_error) != 0u) return false;
        if (global_timer_ns() - t0 > limit) {
            atomicOr(&g_la_error, code);
            return false;
        }
    }
}

// A wait's outcome made uniform across the warp, so that the warp's
// .sync.aligned TMEM accesses that follow are reached by all of its lanes.
__device__ __forceinline__ bool warp_ok(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }
__device__ __forceinline__ uint32_t lane_base(int warp) { return (uint32_t)(32 * (warp & 3)) << 16; }

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
// x[0..7] -> bf16(x), leaving x - bf16(x)
__device__ __forceinline__ uint4 take8(float (&x)[8]) {
    const uint4 p = pack8(x);
    float h[8];
    unpack8(p, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] -= h[e];
    return p;
}

// What the tensor-core kernels take besides their maps.
struct TcArgs {
    LinAttnArgs a;
    View v;
    uint16_t *Shi, *Slo;  // [chunk][H][DK][DV] bf16: the states that enter the chunks (lo: the backward's)
    uint16_t *Rhi, *Rlo;  // gradients of the states that leave them
    float *dot;           // [chunk][H][DV / 64][4] shares of <R, S>
    unsigned long long timeout_ns;
};

// ================================================================ state kernel
constexpr int kStages = 3;
constexpr int kStateThreads = 480;  // warp 0 TMA, 1 MMA, 2..9 weighting, 10..13 state, 14 gates
constexpr int kConv = 256, kSt = 128;
constexpr int kWRing = 4;

template <int DK>
struct StateSmem {
    static constexpr uint32_t KB = DK * 256, VB = 16384;  // a chunk's K (or Q) and 64 columns of V (or dO)
    static constexpr uint32_t STAGE = KB + VB;
    // with DK = 64 the product's rows 64..127 read the bytes after K, in the
    // stage's own V tile: rows that nobody looks at
    static constexpr uint32_t X = kStages * STAGE;        // [half][3][64 tokens][128 B] weighted values
    static constexpr uint32_t W = X + 2 * 3 * 8192;       // [ring][128] weights, then [ring] chunk decays
    static constexpr uint32_t BAR = W + kWRing * 512 + 64;
    enum { FULL = 0, EMPTY = 3, XREADY = 6, XEMPTY = 8, UFULL = 10, UEMPTY = 12, WFULL = 14, WEMPTY = 18, DRAIN = 22, NUM = 23 };
    static constexpr uint32_t TSLOT = BAR + 8 * NUM;
    static constexpr uint32_t BYTES = TSLOT + 16 + 1024;
};
static_assert(StateSmem<128>::BYTES <= 232448, "state kernel fits the shared memory of one CTA");

// Grid (DV / 64, H, n_seq).  REV: the gradient's walk, backwards over the
// chunks, with Q and dO in the places of K and V.  LO: also the states' lower
// bf16 halves (the backward's products take both).
template <int DK, int DV, bool REV, bool LO>
__global__ void __launch_bounds__(kStateThreads, 1)
    state_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV, TcArgs p) {
    using L = StateSmem<DK>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::TSLOT);
    float *wring = reinterpret_cast<float *>(sm + L::W), *dring = wring + kWRing * 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slice = blockIdx.x, h = blockIdx.y, seq = blockIdx.z;
    const int2 sq = seq_at(p.v, seq);
    const int n = sq.y;
    const unsigned long long lim = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars[L::FULL + s], 1);
            mbar_init(&bars[L::EMPTY + s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars[L::XREADY + x], kConv);
            mbar_init(&bars[L::XEMPTY + x], 1);
            mbar_init(&bars[L::UFULL + x], 1);
            mbar_init(&bars[L::UEMPTY + x], kSt);
        }
        for (int w = 0; w < kWRing; ++w) {
            mbar_init(&bars[L::WFULL + w], 32);
            mbar_init(&bars[L::WEMPTY + w], kConv + kSt);
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
    auto chunk_of = [&](int i) { return sq.x + (REV ? n - 1 - i : i); };

    if (warp == 0) {
        if (lane == 0) {
            const int hk = h / (p.a.H / p.a.Hk);
            int i = 0;
            for (; i < n; ++i) {
                const int s = i % kStages;
                if (i >= kStages && !la_wait(&bars[L::EMPTY + s], ((i / kStages) - 1) & 1, 1u, lim)) break;
                const Chunk c = chunk_at<kC>(p.v, p.a.T, chunk_of(i));
                uint8_t *st = sm + s * L::STAGE;
                mbar_arrive_expect_tx(&bars[L::FULL + s], L::STAGE);
#pragma unroll
                for (int x = 0; x < DK / 64; ++x)
                    tma_load_4d(st + x * 16384, &mK, &bars[L::FULL + s], 64 * x, c.t0, hk, c.row);
                tma_load_4d(st + L::KB, &mV, &bars[L::FULL + s], 64 * slice, c.t0, h, c.row);
            }
            // no copy is in flight when the CTA ends
            for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
                mbar_wait(&bars[L::FULL + j % kStages], (j / kStages) & 1, kDrainNs);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, 64, true, true);
            bool ok = true;
            for (int i = 0; i < n && ok; ++i) {
                const int s = i % kStages, acc = i & 1;
                ok = la_wait(&bars[L::FULL + s], (i / kStages) & 1, 2u, lim);
                if (ok && i >= 2) ok = la_wait(&bars[L::UEMPTY + acc], ((i >> 1) - 1) & 1, 2u, lim);
                for (int half = 0; half < 2 && ok; ++half) {
                    ok = la_wait(&bars[L::XREADY + half], i & 1, 2u, lim);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t ka = sbase + s * L::STAGE, xb = sbase + L::X + half * 3 * 8192;
#pragma unroll
                    for (int t = 0; t < 3; ++t)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_bf16_ss(tmem + 64u * acc, smem_desc(ka + (half * 4 + ks) * 2048, 16384, 1024),
                                        smem_desc(xb + t * 8192 + ks * 2048, 8192, 1024), id,
                                        (half | t | ks) ? 1u : 0u);
                    mma_commit(&bars[L::XEMPTY + half]);
                }
                if (ok) {
                    mma_commit(&bars[L::EMPTY + s]);
                    mma_commit(&bars[L::UFULL + acc]);
                }
            }
            // every MMA issued here is complete before TMEM is released
            mma_commit(&bars[L::DRAIN]);
            mbar_wait(&bars[L::DRAIN], 0, kDrainNs);
        }
    } else if (warp < 10) {
        // the weighted values, in two halves of 64 tokens: row r, 16 columns
        const int ct = threadIdx.x - 64, r = ct >> 2, c0 = (ct & 3) * 16;
        for (int i = 0; i < n; ++i) {
            const int s = i % kStages, w = i % kWRing;
            bool ok = la_wait(&bars[L::FULL + s], (i / kStages) & 1, 4u, lim);
            ok = ok && la_wait(&bars[L::WFULL + w], (i / kWRing) & 1, 4u, lim);
            if (!warp_ok(ok)) break;
            uint8_t *st = sm + s * L::STAGE;
            const Chunk c = chunk_at<kC>(p.v, p.a.T, chunk_of(i));
            if (c.len < kC) {
                // rows past the chunk's tokens are another sequence's: zeros, so
                // that nothing of theirs (an infinity, say) meets a zero weight
                for (int e = ct; e < (kC - c.len) * (DK / 8); e += kConv) {
                    const int row = c.len + e / (DK / 8), col = (e % (DK / 8)) * 8;
                    *reinterpret_cast<uint4 *>(st + (col >> 6) * 16384 + sw128_offset(row, col & 63)) = make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t = half * 64 + r;
                const float wt = wring[w * 128 + t];
                float x[2][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    unpack8(*reinterpret_cast<const uint4 *>(st + L::KB + sw128_offset(t, c0 + 8 * u)), x[u]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[u][e] = t < c.len ? x[u][e] * wt : 0.f;
                }
                if (i >= 1 && !la_wait(&bars[L::XEMPTY + half], (i - 1) & 1, 4u, lim)) ok = false;
                if (!warp_ok(ok)) break;
                uint8_t *xb = sm + L::X + half * 3 * 8192;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t off = sw128_offset(r, c0 + 8 * u);
                    *reinterpret_cast<uint4 *>(xb + off) = take8(x[u]);
                    *reinterpret_cast<uint4 *>(xb + 8192 + off) = take8(x[u]);
                    *reinterpret_cast<uint4 *>(xb + 16384 + off) = pack8(x[u]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&bars[L::XREADY + half]);
            }
            if (!warp_ok(ok)) break;
            mbar_arrive(&bars[L::WEMPTY + w]);
        }
    } else if (warp < 14) {
        // the state: one row of 64 columns a thread
        const int row = 32 * (warp & 3) + lane;
        const bool mine = row < DK;
        float S[64];
        const float *from = REV ? p.a.dsf : p.a.s0;
        const size_t page = (((size_t)seq * p.a.H + h) * DK + row) * DV + 64 * slice;
#pragma unroll
        for (int e = 0; e < 64; e += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine && from) x = *reinterpret_cast<const float4 *>(from + page + e);
            S[e] = x.x, S[e + 1] = x.y, S[e + 2] = x.z, S[e + 3] = x.w;
        }
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const int acc = i & 1, w = i % kWRing;
            const size_t ci = (size_t)chunk_of(i) * p.a.H + h;
            const size_t at = (ci * DK + row) * DV + 64 * slice;
            uint16_t *hi = (REV ? p.Rhi : p.Shi) + at, *lo = (REV ? p.Rlo : p.Slo) + at;
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = S[e + j];
                if (REV && mine) {
                    float a[8], b[8];
                    unpack8(*reinterpret_cast<const uint4 *>(p.Shi + at + e), a);
                    unpack8(*reinterpret_cast<const uint4 *>(p.Slo + at + e), b);
#pragma unroll
                    for (int j = 0; j < 8; ++j) dot = fmaf(x[j], a[j] + b[j], dot);
                }
                const uint4 top = take8(x);
                if (mine) {
                    *reinterpret_cast<uint4 *>(hi + e) = top;
                    if (LO) *reinterpret_cast<uint4 *>(lo + e) = pack8(x);
                }
            }
            if (REV) {
#pragma unroll
                for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(~0u, dot, m);
                if (lane == 0) p.dot[(ci * (DV / 64) + slice) * 4 + (warp & 3)] = dot;
            }
            ok = la_wait(&bars[L::WFULL + w], (i / kWRing) & 1, 8u, lim);
            const float d = ok ? dring[w] : 0.f;
            ok = ok && la_wait(&bars[L::UFULL + acc], (i >> 1) & 1, 8u, lim);
            if (!warp_ok(ok)) break;
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
        float *to = REV ? p.a.ds0 : p.a.sf;
        if (to && mine && warp_ok(ok))
#pragma unroll
            for (int e = 0; e < 64; e += 4)
                *reinterpret_cast<float4 *>(to + page + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    } else {
        // the weights: e^{G - c_t}, or (REV) scale e^{c_t}
        for (int i = 0; i < n; ++i) {
            const int w = i % kWRing;
            if (i >= kWRing && !la_wait(&bars[L::WEMPTY + w], ((i / kWRing) - 1) & 1, 16u, lim)) break;
            const Chunk c = chunk_at<kC>(p.v, p.a.T, chunk_of(i));
            const Gates<kC> g = warp_gates<kC>(gate_ptr(p.a, c, h), p.a.sg.t, c.len, p.a.flags & GDN_G_PER_HEAD);
            float4 x;
            if (REV) x = make_float4(expf((float)g.cum[0]), expf((float)g.cum[1]), expf((float)g.cum[2]), expf((float)g.cum[3]));
            else x = make_float4(expf((float)(g.all - g.cum[0])), expf((float)(g.all - g.cum[1])),
                                 expf((float)(g.all - g.cum[2])), expf((float)(g.all - g.cum[3])));
            if (REV) x.x *= p.a.scale, x.y *= p.a.scale, x.z *= p.a.scale, x.w *= p.a.scale;
            reinterpret_cast<float4 *>(wring + w * 128)[lane] = x;
            if (lane == 0) dring[w] = expf((float)g.all);
            mbar_arrive(&bars[L::WFULL + w]);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 128);
    }
}

// ================================================================== out kernel
constexpr int kOutThreads = 256;

template <int DK, int DV>
struct OutSmem {
    static constexpr uint32_t Q = 0;              // later the rows of O
    static constexpr uint32_t K = 32768;          // later P
    static constexpr uint32_t S = 65536;          // later V
    static constexpr uint32_t G = 98304;          // [2][128] decays
    static constexpr uint32_t BAR = G + 1536;
    enum { QK = 0, ST, VL, DQK, DQS, DPV, DRAIN, NUM };
    static constexpr uint32_t TSLOT = BAR + 8 * NUM;
    static constexpr uint32_t BYTES = TSLOT + 16 + 1024;
};
static_assert(2 * (OutSmem<128, 128>::BYTES + 1024) <= 233472, "two CTAs of the out kernel share an SM");

// A chunk's outputs.  Grid (chunks, H), two CTAs an SM: one's loads and
// stores run under the other's products.
template <int DK, int DV>
__global__ void __launch_bounds__(kOutThreads, 2)
    out_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
               const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mS, TcArgs p) {
    using L = OutSmem<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::TSLOT);
    float *hi = reinterpret_cast<float *>(sm + L::G), *lo = hi + 128, *te = lo + 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ci = blockIdx.x, h = blockIdx.y;
    const Chunk c = chunk_at<kC>(p.v, p.a.T, ci);
    __nv_bfloat16 *out = at(static_cast<__nv_bfloat16 *>(p.a.o), p.a.so, c.row, h, c.t0);
    if (c.len <= 0) return;
    if (c.seq < 0) {  // tokens of no sequence
        for (int e = threadIdx.x; e < c.len * (DV / 8); e += kOutThreads)
            *reinterpret_cast<uint4 *>(out + (e / (DV / 8)) * p.a.so.t + (e % (DV / 8)) * 8) = make_uint4(0, 0, 0, 0);
        return;
    }
    // a first chunk without an initial state has nothing to read
    const bool with_state = p.a.s0 != nullptr || seq_at(p.v, c.seq).x != ci;
    const unsigned long long lim = p.timeout_ns;
    if (threadIdx.x == 0) {
        for (int b = 0; b < L::NUM; ++b) mbar_init(&bars[b], 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, 256);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tslot;
    const uint32_t sbase = smem_u32(sm);
    const int hk = h / (p.a.H / p.a.Hk);
    bool ok = true, v_armed = false;
    auto load_v = [&] {
        v_armed = true;
        mbar_arrive_expect_tx(&bars[L::VL], DV * 256);
#pragma unroll
        for (int x = 0; x < DV / 64; ++x) tma_load_4d(sm + L::S + x * 16384, &mV, &bars[L::VL], 64 * x, c.t0, h, c.row);
    };
    if (warp == 0 && lane == 0) {
        mbar_arrive_expect_tx(&bars[L::QK], 2 * DK * 256);
#pragma unroll
        for (int x = 0; x < DK / 64; ++x) {
            tma_load_4d(sm + L::Q + x * 16384, &mQ, &bars[L::QK], 64 * x, c.t0, hk, c.row);
            tma_load_4d(sm + L::K + x * 16384, &mK, &bars[L::QK], 64 * x, c.t0, hk, c.row);
        }
        if (with_state) {
            mbar_arrive_expect_tx(&bars[L::ST], DK * DV * 2);
#pragma unroll
            for (int x = 0; x < DV / 64; ++x)
                tma_load_3d(sm + L::S + x * (DK * 128), &mS, &bars[L::ST], 64 * x, 0, ci * p.a.H + h);
        } else {
            load_v();
        }
        ok = la_wait(&bars[L::QK], 0, 32u, lim);
        if (ok) {
            const uint32_t id = idesc_bf16(128, 128, false, false);
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks)
                mma_bf16_ss(tmem, smem_desc(sbase + L::Q + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024),
                            smem_desc(sbase + L::K + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024), id, ks > 0);
            mma_commit(&bars[L::DQK]);
        }
        if (with_state) {
            ok = la_wait(&bars[L::ST], 0, 32u, lim) && ok;
            if (ok) {
                const uint32_t id = idesc_bf16(128, DV, false, true);
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks)
                    mma_bf16_ss(tmem + 128, smem_desc(sbase + L::Q + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024),
                                smem_desc(sbase + L::S + ks * 2048, DK * 128, 1024), id, ks > 0);
                mma_commit(&bars[L::DQS]);
                ok = la_wait(&bars[L::DQS], 0, 32u, lim);  // S's place is V's now
                if (ok) load_v();
            }
        }
    } else if (warp == 2) {
        gates<kC>(gate_ptr(p.a, c, h), p.a.sg.t, c.len, p.a.flags & GDN_G_PER_HEAD, hi, lo, te);
    }
    __syncwarp();
    __syncthreads();  // the decays are there
    // P: thread's row t, columns s of its half
    const int t = 32 * (warp & 3) + lane, s0 = 64 * (warp >> 2);
    if (!warp_ok(la_wait(&bars[L::DQK], 0, 64u, lim))) ok = false;
    if (warp_ok(ok)) {
        tc_fence_after_sync();
        const float ht = hi[t], lt = lo[t];
#pragma unroll
        for (int e = 0; e < 64; e += 16) {
            uint32_t u[16];
            float x[16];
            if (32 * (warp & 3) + 31 >= s0 + e) {  // some row of the warp reaches these columns
                tmem_ld16(tmem + lane_base(warp) + s0 + e, u);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int s = s0 + e + j;
                    x[j] = s <= t ? __uint_as_float(u[j]) * __expf((ht - hi[s]) + (lt - lo[s])) : 0.f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 16; j += 8)
                *reinterpret_cast<uint4 *>(sm + L::K + (s0 >> 6) * 16384 + sw128_offset(t, e + j)) =
                    make_uint4(pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3]), pack_bf16(x[j + 4], x[j + 5]),
                               pack_bf16(x[j + 6], x[j + 7]));
        }
    }
    ok = warp_ok(la_wait(&bars[L::VL], 0, 64u, lim)) && ok;
    if (c.len < kC && ok) {  // another sequence's rows: zeros, as in state_kernel
        for (int e = threadIdx.x; e < (kC - c.len) * (DV / 8); e += kOutThreads) {
            const int row = c.len + e / (DV / 8), col = (e % (DV / 8)) * 8;
            *reinterpret_cast<uint4 *>(sm + L::S + (col >> 6) * 16384 + sw128_offset(row, col & 63)) = make_uint4(0, 0, 0, 0);
        }
    }
    fence_proxy_async_smem();
    tc_fence_before_sync();
    ok = __syncthreads_and(ok);
    if (ok) {
        if (warp == 0 && lane == 0) {
            tc_fence_after_sync();
            const uint32_t id = idesc_bf16(128, DV, false, true);
#pragma unroll
            for (int ks = 0; ks < kC / 16; ++ks)
                mma_bf16_ss(tmem, smem_desc(sbase + L::K + (ks >> 2) * 16384 + (ks & 3) * 32, 16, 1024),
                            smem_desc(sbase + L::S + ks * 2048, 16384, 1024), id, ks > 0);
            mma_commit(&bars[L::DPV]);
        }
        __syncwarp();
        ok = warp_ok(la_wait(&bars[L::DPV], 0, 128u, lim));
    }
    if (ok) {
        // the rows of O: scale (e^c (Q S) + P V), through Q's place, so that
        // the stores are whole rows
        tc_fence_after_sync();
        const float f = __expf(hi[t]) * p.a.scale;
        constexpr int W = DV / 2;  // columns of a thread
        const int w0 = W * (warp >> 2);
#pragma unroll
        for (int e = 0; e < W; e += 16) {
            uint32_t u[16], y[16];
            tmem_ld16(tmem + lane_base(warp) + w0 + e, u);
            if (with_state) tmem_ld16(tmem + 128 + lane_base(warp) + w0 + e, y);
            tmem_wait_ld();
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                x[j] = p.a.scale * __uint_as_float(u[j]);
                if (with_state) x[j] = fmaf(f, __uint_as_float(y[j]), x[j]);
            }
#pragma unroll
            for (int j = 0; j < 16; j += 8) {
                const int ch = (w0 + e + j) >> 3;
                *reinterpret_cast<uint4 *>(sm + L::Q + t * (DV * 2) + ((ch ^ (t & 7)) << 4)) =
                    make_uint4(pack_bf16(x[j], x[j + 1]), pack_bf16(x[j + 2], x[j + 3]), pack_bf16(x[j + 4], x[j + 5]),
                               pack_bf16(x[j + 6], x[j + 7]));
            }
        }
    }
    tc_fence_before_sync();
    ok = __syncthreads_and(ok);
    if (ok)
        for (int e = threadIdx.x; e < c.len * (DV / 8); e += kOutThreads) {
            const int row = e / (DV / 8), ch = e % (DV / 8);
            *reinterpret_cast<uint4 *>(out + row * p.a.so.t + ch * 8) =
                *reinterpret_cast<const uint4 *>(sm + L::Q + row * (DV * 2) + ((ch ^ (row & 7)) << 4));
        }
    if (!ok) {  // a wait gave up: no copy and no product is in flight when the CTA ends
        if (threadIdx.x == 0) {
            mma_commit(&bars[L::DRAIN]);
            mbar_wait(&bars[L::DRAIN], 0, kDrainNs);
            mbar_wait(&bars[L::QK], 0, kDrainNs);
            if (with_state) mbar_wait(&bars[L::ST], 0, kDrainNs);
            if (v_armed) mbar_wait(&bars[L::VL], 0, kDrainNs);
        }
        __syncwarp();
        tc_fence_before_sync();
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 256);
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
size_t state_bytes(const LinAttnArgs &a) { return up(2 * (size_t)chunk_bound(a, kC) * a.H * a.Dk * a.Dv); }

int launched() {
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

template <class F>
bool smem_limit(F f, uint32_t bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <int DK, int DV, bool REV, bool LO>
int run_state(const CUtensorMap &mK, const CUtensorMap &mV, const TcArgs &p, cudaStream_t stream) {
    auto kern = state_kernel<DK, DV, REV, LO>;
    if (!smem_limit(kern, StateSmem<DK>::BYTES)) return GDN_ERR_CUDA;
    kern<<<dim3(DV / 64, p.a.H, p.a.n_seq), kStateThreads, StateSmem<DK>::BYTES, stream>>>(mK, mV, p);
    return launched();
}

template <int DK, int DV>
int run_fwd(const TcArgs &p, cudaStream_t stream) {
    const LinAttnArgs &a = p.a;
    if (!mappable(a.sq, a.B, a.Hk, a.T) || !mappable(a.sk, a.B, a.Hk, a.T) || !mappable(a.sv, a.B, a.H, a.T))
        return GDN_ERR_UNSUPPORTED;
    CUtensorMap mQ, mK, mV, mS;
    if (!strided_map(&mQ, a.q, a.sq, a.B, a.Hk, a.T, DK, kC) || !strided_map(&mK, a.k, a.sk, a.B, a.Hk, a.T, DK, kC) ||
        !strided_map(&mV, a.v, a.sv, a.B, a.H, a.T, DV, kC) ||
        !state_map(&mS, p.Shi, (long long)p.v.n_chunks * a.H, DK, DV))
        return GDN_ERR_CUDA;
    // one chunk a sequence, no state in or out: the outputs are all
    if (a.cu || a.T > kC || a.s0 || a.sf) {
        const int st = run_state<DK, DV, false, false>(mK, mV, p, stream);
        if (st != GDN_OK) return st;
    }
    using L = OutSmem<DK, DV>;
    auto kern = out_kernel<DK, DV>;
    if (!smem_limit(kern, L::BYTES)) return GDN_ERR_CUDA;
    kern<<<dim3(p.v.n_chunks, a.H), kOutThreads, L::BYTES, stream>>>(mQ, mK, mV, mS, p);
    return launched();
}

}  // namespace
}  // namespace la

using namespace la;

bool linattn_tc_supported(const LinAttnArgs &a) {
    return a.dtype == GDN_BF16 && !(a.flags & GDN_PATH_SIMT) && sm100_family();
}

size_t linattn_tc_fwd_workspace(const LinAttnArgs &a) { return up(table_bytes(a, kC)) + state_bytes(a) + 1024; }

int launch_linattn_tc_fwd(const LinAttnArgs &a, cudaStream_t stream) {
    TcArgs p{};
    p.a = a;
    p.timeout_ns = wait_limit_ns();
    const int st = make_view(a, kC, a.ws, &p.v, stream);
    if (st != GDN_OK) return st;
    p.Shi = reinterpret_cast<uint16_t *>(static_cast<char *>(a.ws) + up(table_bytes(a, kC)));
    if (a.Dk == 128) return a.Dv == 128 ? run_fwd<128, 128>(p, stream) : run_fwd<128, 64>(p, stream);
    return a.Dv == 128 ? run_fwd<64, 128>(p, stream) : run_fwd<64, 64>(p, stream);
}

size_t linattn_tc_bwd_workspace(const LinAttnArgs &a) { return linattn_bwd_workspace(a); }
int launch_linattn_tc_bwd(const LinAttnArgs &a, cudaStream_t stream) { return launch_linattn_bwd(a, stream); }

int linattn_tc_read_clear_error() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_la_error, sizeof(v)) != cudaSuccess) return GDN_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_la_error, &zero, sizeof(zero)) != cudaSuccess) return GDN_ERR_CUDA;
    return v ? GDN_ERR_TIMEOUT : GDN_OK;
}

}  // namespace gdn
