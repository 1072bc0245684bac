// ssm_scan_bwd.cu -- backward of the selective state space scan (ssm.cuh).  With
// dy' = dy silu(z) and g_t the gradient of h_t:
//
//   g_t = C_t dy'_t + exp(D_{t+1} A) g_{t+1},     p_t = g_t exp(D_t A) h_{t-1}
//   dA = sum_t D_t p_t,  dx_t = D_t sum_n g_t B_t + skip dy'_t,
//   dD_t = x_t sum_n g_t B_t + sum_n A p_t,       ddt_t = dD_t sigmoid(dt_t + bias)
//   dB_t = sum_c g_t D_t x_t,  dC_t = sum_c dy'_t h_t,  dz_t = dy_t (C_t.h_t + skip x_t) silu'(z_t)
//
// Three launches.  share_kernel walks every chunk forwards from 0 and writes the
// state before every 4 tokens, what the chunk leaves, and what gradient it
// passes to the chunk before it (through the running product of its decays, so
// that one exponential serves both).  grad_kernel walks the chunks backwards: four
// tokens' states are made anew from the one before them and stay in registers.
// sum_kernel adds up, in order, what groups of channels give to dB and dC and what
// chunks give to dA, dskip and dbias.  Three exponentials a (token, channel,
// state); states every 4 tokens take Di N bytes a token, written and read once behind
// the arithmetic.  Every 8 took half of that and 7% longer: 64 registers more, of
// which some went through memory, and twice the code to fetch.
// Measured, bf16, 4 x 4096 x 2048 x 16 with a gate: 879 us, of them share_kernel
// 235 and grad_kernel about 630.  Instructions bound it, not bytes (0.47 GB and 1.07
// of states, 230 us): 21 for a warp's 32 tokens x channels x states in grad_kernel,
// at 43% of the issue slots of 8 warps an SM, which is what shared memory leaves room
// for.  (12 warps, with 168 registers and one block of 4 tokens at a time, spilled and
// waited for its loads: 1,104 us.)
//
// A thread holds 4 channels x 4 states, as pairs of channels: what belongs to a
// channel is loaded as a pair, and B and C lie in shared memory twice over.  The
// sums over a channel's lanes and, for dB and dC, over the channels' go through
// shared memory, two or four tokens at a time (matrix instructions with ones, in two
// parts a value, took 64 instructions a token and warp for the former).  The other
// way round (all states of a channel in a thread, as forwards) would need 32 values
// of a token summed over 32 lanes.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "ssm.cuh"

namespace gdn {
namespace {

using namespace ssm;
using mx::Run;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kBlock = 8;  // tokens that are fetched and converted at once
constexpr int kHalf = 4;   // tokens between two states in memory

template <typename T, int N>
struct Shape {
    static constexpr int L = N / 4;       // lanes of a channel's states
    static constexpr int G = 32 / L;      // lanes of the channels
    static constexpr int CH = 4 * G;      // channels a warp
    static constexpr int V = kWide<T>;
    // a token's channels in shared memory: lanes of 32 bytes, of two tokens in a quarter warp, meet in no bank
    static constexpr int ROW = CH + (V == 8 ? 4 : 0);
    static constexpr int RV = CH / V;     // vectors of a token's channels
    static constexpr int NV = kBlock * RV, VPL = (NV + 31) / 32;  // of a block; of a lane
    static constexpr int BV = N / V;      // vectors of a token's B
    // dB's and dC's halves trade places in rows that would meet in a bank
    static __device__ __forceinline__ int swap(int g) { return N == 16 ? (g & 1) * 16 : N == 8 ? (g >> 1 & 1) * 8 : 0; }
    // tokens that are summed at once over the states' lanes, and over the channels' (dB and dC): of fp32 rows fewer, so
    // that two CTAs fit on an SM (2 x 4096 x 2048 x 16 647 -> 518 us, 1999 x 512 59 -> 62)
    static constexpr int TOK = sizeof(T) == 2 ? 2 : 1;
    static constexpr int SLOTS = sizeof(T) == 2 && N == 16 ? 4 : 2;
    static constexpr int NB = kBlock * BV, BPL = (2 * NB + 31) / 32;
};

// How a row is cut, and where a call's intermediates are.
struct Plan {
    int len, chunks;     // tokens of a chunk, a multiple of kBlock
    int groups, halves;  // CTAs over the channels; half blocks of tokens a row
    float *left, *back;  // [row][chunk][Di][N]: the state that a chunk leaves, the gradient that it passes on
    float *steps;        // [row][chunk][Di]: the sum of its steps
    float *state;        // [row][half block][warp's channels][4][32] float4: the state before it, from 0 at the chunk's start
    float *upto;         // [row][half block][warp's channels]: the steps from the chunk's start to it
    float *dA, *dD, *db; // [row][chunk][Di][N], [row][chunk][Di] twice
    float *dBC;          // [group][row][T][2 N]
};

template <typename T, int N>
struct Mem {
    using S = Shape<T, N>;
    uint4 raw[2][4][S::NV];  // x, dt, dy, z as loaded, twice: one on its way
    uint4 bc[2][2 * S::NB];
    float step[kBlock][S::ROW], x[kBlock][S::ROW], dy[kBlock][S::ROW];  // then D's and x's gradients, and y
    float b[kBlock][2 * N], c[kBlock][2 * N];                        // every value twice
    int seq[kBlock];                                                // the sequences that start or end in the block
};
template <typename T, int N>
struct GradMem : Mem<T, N> {
    using S = Shape<T, N>;
    float4 saved[5][32];                      // a half block's state and steps, as the lanes take them
    float4 start[4][32];                      // the state that enters the chunk
    float part[2][kBlock][2 * N];             // a block's dB and dC of this warp
    float over_states[S::TOK][3][S::L][S::CH + 8];  // some tokens' D's and x's gradients and y, of each lane of a channel
    float over_channels[S::SLOTS][S::G][2 * N];  // some tokens' dB and dC, of each lane of the channels; swizzled
    float4 acc[2][S::VPL * S::V / 4][32];     // dskip and dbias of each lane's vectors
};

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_done(bool all) {
    if (all) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else asm volatile("cp.async.wait_group 1;" ::: "memory");
}
__device__ __forceinline__ void copies_out() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// A warp's place: channels c0 .., and the thread's four.
struct Place {
    int row, chunk, group, t0, t1, c0, c, q, g;
};
template <typename T, int N>
__device__ __forceinline__ Place place_of(const SsmArgs &a, const Plan &p) {
    using S = Shape<T, N>;
    Place w;
    const int lane = threadIdx.x & 31, item = blockIdx.x / p.groups;
    w.group = blockIdx.x % p.groups;
    w.row = item / p.chunks, w.chunk = item - w.row * p.chunks;
    w.t0 = w.chunk * p.len, w.t1 = min(w.t0 + p.len, a.T);
    w.c0 = (w.group * kWarps + (threadIdx.x >> 5)) * S::CH;
    w.q = lane % S::L, w.g = lane / S::L;
    w.c = w.c0 + 4 * w.g;
    return w;
}

// Starts the copies of the block of tokens at t.
template <typename T, int N>
__device__ __forceinline__ void fetch(const SsmArgs &a, const Place &w, Mem<T, N> &m, int buf, int t) {
    using S = Shape<T, N>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < S::VPL; ++i) {
        const int j = i * 32 + lane, tok = t + j / S::RV, c = w.c0 + j % S::RV * S::V;
        if (j < S::NV && tok < w.t1 && c < a.Di) {
            copy16(&m.raw[buf][0][j], static_cast<const T *>(a.x) + w.row * a.sx.b + tok * a.sx.t + c);
            copy16(&m.raw[buf][1][j], static_cast<const T *>(a.dt) + w.row * a.sdt.b + tok * a.sdt.t + c);
            copy16(&m.raw[buf][2][j], static_cast<const T *>(a.dy) + w.row * a.sy.b + tok * a.sy.t + c);
            if (a.z) copy16(&m.raw[buf][3][j], static_cast<const T *>(a.z) + w.row * a.sz.b + tok * a.sz.t + c);
        }
    }
#pragma unroll
    for (int i = 0; i < S::BPL; ++i) {
        const int j = i * 32 + lane, k = j % S::NB, tok = t + k / S::BV, n = k % S::BV * S::V;
        if (j < 2 * S::NB && tok < w.t1)
            copy16(&m.bc[buf][j], j < S::NB ? static_cast<const T *>(a.Bt) + w.row * a.sB.b + tok * a.sB.t + n
                                            : static_cast<const T *>(a.Ct) + w.row * a.sC.b + tok * a.sC.t + n);
    }
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const uint4 &p, float (&x)[V]) {
    Vec<T, V>::unpack(p, x);
}
template <int V>
__device__ __forceinline__ void put(float *to, const float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}
template <int V>
__device__ __forceinline__ void get(const float *from, float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        const float4 y = *reinterpret_cast<const float4 *>(from + e);
        x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
    }
}
template <int V>
__device__ __forceinline__ void vector_of(const float *p, int c, float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p) y = __ldg(reinterpret_cast<const float4 *>(p + c + e));
        x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
    }
}

// Steps, x and dy' of a block, and its B and C, in fp32; zeros for tokens of no
// sequence (bits of `dead`), which then change nothing.
template <typename T, int N>
__device__ __forceinline__ void convert(const SsmArgs &a, const Place &w, Mem<T, N> &m, int buf, int t, unsigned dead) {
    using S = Shape<T, N>;
    const int lane = threadIdx.x & 31;
    const bool soft = a.flags & GDN_DT_SOFTPLUS;
#pragma unroll
    for (int i = 0; i < S::VPL; ++i) {
        const int j = i * 32 + lane, tok = j / S::RV, c = j % S::RV * S::V;
        if (j >= S::NV) break;
        float x[S::V], d[S::V], g[S::V];
        if (t + tok < w.t1 && w.c0 + c < a.Di && !(dead >> tok & 1)) {
            float bias[S::V];
            vector_of<S::V>(a.bias, w.c0 + c, bias);
            unpack<T, S::V>(m.raw[buf][0][j], x);
            unpack<T, S::V>(m.raw[buf][1][j], d);
            unpack<T, S::V>(m.raw[buf][2][j], g);
#pragma unroll
            for (int e = 0; e < S::V; e += 2) {
                const F2 v = mx::add2(pair(d[e], d[e + 1]), pair(bias[e], bias[e + 1]));
                split(soft ? mx::softplus2(v) : v, d[e], d[e + 1]);
            }
            if (a.z) {
                float z[S::V];
                unpack<T, S::V>(m.raw[buf][3][j], z);
#pragma unroll
                for (int e = 0; e < S::V; e += 2) split(mul2(pair(g[e], g[e + 1]), mx::silu2(pair(z[e], z[e + 1]))), g[e], g[e + 1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < S::V; ++e) x[e] = d[e] = g[e] = 0.f;
        }
        put<S::V>(&m.x[tok][c], x);
        put<S::V>(&m.step[tok][c], d);
        put<S::V>(&m.dy[tok][c], g);
    }
    // two values a lane, so that the doubled ones of a quarter warp lie side by side
    constexpr int PAIRS = kBlock * N / 2;
    using Two = typename Vec<T, 2>::Raw;
#pragma unroll
    for (int i = 0; i < 2 * PAIRS; i += 32) {
        const int j = i + lane, k = j % PAIRS, tok = k / (N / 2), n = k % (N / 2) * 2;
        float x[2];
        Vec<T, 2>::unpack(reinterpret_cast<const Two *>(m.bc[buf])[j], x);
        if (t + tok >= w.t1 || (dead >> tok & 1)) x[0] = x[1] = 0.f;
        float *to = j < PAIRS ? &m.b[tok][2 * n] : &m.c[tok][2 * n];
        *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[0], x[1], x[1]);
    }
}

// Which tokens of a block start a sequence, end one, or are in none (or past the
// chunk); r: the run of its first token.
struct Marks {
    unsigned starts, ends, dead;
};
__device__ __forceinline__ Marks marks_of(const SsmArgs &a, const Place &w, int t, Run &r, int *seq) {
    if (t < r.start || t >= r.end) r = mx::run_at(a.cu, a.n_seq, a.T, w.row, t);
    const int n = min(kBlock, w.t1 - t), lane = threadIdx.x & 31;
    const unsigned past = 0xffu << n & 0xffu;
    if (r.end >= t + n) {
        if (lane < kBlock) seq[lane] = r.s;
        if (r.s < 0) return {0, 0, 0xffu};
        return {r.start == t ? 1u : 0u, r.end == t + n ? 1u << (n - 1) : 0u, past};
    }
    Run mine{-1, 0, 0};
    if (lane < n) mine = mx::run_at(a.cu, a.n_seq, a.T, w.row, t + lane);
    if (lane < kBlock) seq[lane] = mine.s;
    return {__ballot_sync(~0u, mine.s >= 0 && mine.start == t + lane), __ballot_sync(~0u, mine.s >= 0 && mine.end == t + lane + 1),
            __ballot_sync(~0u, mine.s < 0) & 0xffu};
}

// A thread's 4 channels x 4 states: [pair of channels][state].
using Quad = F2[2][4];

// .. of a [Di,N] page, 0 where there is none.
template <int N>
__device__ __forceinline__ void load16(const SsmArgs &a, const Place &w, const float *page, Quad &h) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (page && w.c < a.Di) {
            x = *reinterpret_cast<const float4 *>(page + (size_t)(w.c + 2 * p) * N + 4 * w.q);
            y = *reinterpret_cast<const float4 *>(page + (size_t)(w.c + 2 * p + 1) * N + 4 * w.q);
        }
        h[p][0] = pair(x.x, y.x), h[p][1] = pair(x.y, y.y), h[p][2] = pair(x.z, y.z), h[p][3] = pair(x.w, y.w);
    }
}
template <int N>
__device__ __forceinline__ void store16(const SsmArgs &a, const Place &w, float *page, const Quad &h) {
    if (w.c >= a.Di) return;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        float4 x, y;
        split(h[p][0], x.x, y.x), split(h[p][1], x.y, y.y), split(h[p][2], x.z, y.z), split(h[p][3], x.w, y.w);
        *reinterpret_cast<float4 *>(page + (size_t)(w.c + 2 * p) * N + 4 * w.q) = x;
        *reinterpret_cast<float4 *>(page + (size_t)(w.c + 2 * p + 1) * N + 4 * w.q) = y;
    }
}
// Vector e of the quad, as it lies in a block's saved state.
__device__ __forceinline__ ulonglong2 quad_vector(const Quad &h, int e) { return make_ulonglong2(h[e >> 1][2 * (e & 1)], h[e >> 1][2 * (e & 1) + 1]); }
__device__ __forceinline__ void set_vector(Quad &h, int e, const ulonglong2 &v) { h[e >> 1][2 * (e & 1)] = v.x, h[e >> 1][2 * (e & 1) + 1] = v.y; }

// Four channels' values of a token, as pairs; four states', each twice.
__device__ __forceinline__ void channels(const float *p, F2 (&x)[2]) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    x[0] = v.x, x[1] = v.y;
}
__device__ __forceinline__ void states(const float *p, F2 (&x)[4]) {
    const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(p), v = *reinterpret_cast<const ulonglong2 *>(p + 4);
    x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
}
// h <- exp(D A) h + D x B of one token, from `from`.
__device__ __forceinline__ void advance(const Quad &from, Quad &h, const Quad &A, const F2 (&d)[2], const F2 (&u)[2], const F2 (&b)[4]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int n = 0; n < 4; ++n) h[p][n] = fma2(exp2_2(mul2(d[p], A[p][n])), from[p][n], mul2(u[p], b[n]));
}

template <int N>
__device__ __forceinline__ void load_decays(const SsmArgs &a, const Place &w, Quad &d) {
    load16<N>(a, w, a.A, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i >> 2][i & 3] = mul2(d[i >> 2][i & 3], both(mx::kLog2e));
}
__device__ __forceinline__ void zero16(Quad &h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i >> 2][i & 3] = 0;
}
// Where a half block's saved state and steps are, of this warp's channels.
template <typename T, int N>
__device__ __forceinline__ size_t saved_at(const SsmArgs &a, const Plan &p, const Place &w, int t) {
    return ((size_t)w.row * p.halves + t / kHalf) * (p.groups * kWarps) + w.c0 / Shape<T, N>::CH;
}
__device__ __forceinline__ size_t chunk_at(const SsmArgs &a, const Plan &p, int row, int chunk) {
    return ((size_t)row * p.chunks + chunk) * a.Di;
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4) share_kernel(SsmArgs a, Plan p) {
    using S = Shape<T, N>;
    extern __shared__ __align__(16) char smem[];
    Mem<T, N> &m = reinterpret_cast<Mem<T, N> *>(smem)[threadIdx.x >> 5];
    mx::let_follow();
    const Place w = place_of<T, N>(a, p);
    if (w.c0 >= a.Di) return;  // warps do not wait for one another here
    fetch<T, N>(a, w, m, 0, w.t0);
    copies_out();
    const int lane = threadIdx.x & 31;
    Quad h, A, prod, back;
    F2 total[2] = {0, 0};
    load_decays<N>(a, w, A);
    zero16(h);
    zero16(back);
#pragma unroll
    for (int i = 0; i < 8; ++i) prod[i >> 2][i & 3] = both(1.f);
    const size_t page = (size_t)a.Di * N;
    Run r = mx::run_at(a.cu, a.n_seq, a.T, w.row, w.t0);
    // up to where the chunk passes a gradient to the one before
    const int until = r.s >= 0 && r.start < w.t0 ? min(r.end, w.t1) : w.t0;
    const int last_of = r.end, seq = r.s;
    int buf = 0;
    for (int t = w.t0; t < w.t1; t += kBlock, buf ^= 1) {
        const bool more = t + kBlock < w.t1;
        if (more) fetch<T, N>(a, w, m, buf ^ 1, t + kBlock), copies_out();
        const Marks k = marks_of(a, w, t, r, m.seq);
        auto save = [&](int u) {
            const size_t at = saved_at<T, N>(a, p, w, t + u);
            ulonglong2 *to = reinterpret_cast<ulonglong2 *>(p.state) + at * 128 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) to[e * 32] = quad_vector(h, e);
            if (w.q == 0) *reinterpret_cast<ulonglong2 *>(p.upto + at * S::CH + 4 * w.g) = make_ulonglong2(total[0], total[1]);
        };
        copies_done(!more);
        __syncwarp();
        convert<T, N>(a, w, m, buf, t, k.dead);
        __syncwarp();
        auto token = [&](int u, bool pass) {
            F2 d[2], x[2], b[4];
            channels(&m.step[u][4 * w.g], d);
            channels(&m.x[u][4 * w.g], x);
            states(&m.b[u][8 * w.q], b);
            const F2 in[2] = {mul2(d[0], x[0]), mul2(d[1], x[1])};
            total[0] = mx::add2(total[0], d[0]), total[1] = mx::add2(total[1], d[1]);
            if (!pass) {
                advance(h, h, A, d, in, b);
                return;
            }
            F2 g[2], c[4];
            channels(&m.dy[u][4 * w.g], g);
            states(&m.c[u][8 * w.q], c);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const F2 dec = exp2_2(mul2(d[i], A[i][n]));
                    h[i][n] = fma2(dec, h[i][n], mul2(in[i], b[n]));
                    prod[i][n] = mul2(prod[i][n], dec);
                    back[i][n] = fma2(prod[i][n], mul2(g[i], c[n]), back[i][n]);
                }
        };
        if (k.starts == 0 && (t + kBlock <= until || t >= until)) {
            const bool pass = t < until;
#pragma unroll 1
            for (int v = 0; v < kBlock; v += kHalf) {
                save(v);
                if (pass) {
#pragma unroll 4
                    for (int u = v; u < v + kHalf; ++u) token(u, true);
                } else {
#pragma unroll 4
                    for (int u = v; u < v + kHalf; ++u) token(u, false);
                }
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < kBlock; ++u) {
                if (u % kHalf == 0) save(u);
                if (k.starts >> u & 1) load16<N>(a, w, a.s0 ? a.s0 + m.seq[u] * page : nullptr, h);
                if (t + u < until) token(u, true);
                else token(u, false);
            }
        }
        __syncwarp();
    }
    if (a.dsf && until > w.t0 && last_of <= w.t1) {  // the sequence ends here: its final state's share
        Quad s;
        load16<N>(a, w, a.dsf + seq * page, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) back[i >> 2][i & 3] = fma2(prod[i >> 2][i & 3], s[i >> 2][i & 3], back[i >> 2][i & 3]);
    }
    const size_t at = chunk_at(a, p, w.row, w.chunk);
    store16<N>(a, w, p.left + at * N, h);
    store16<N>(a, w, p.back + at * N, back);
    if (w.q == 0 && w.c < a.Di) *reinterpret_cast<ulonglong2 *>(p.steps + at + w.c) = make_ulonglong2(total[0], total[1]);
}

template <typename T, int N, bool GATE>
__global__ void __launch_bounds__(kThreads, 2) grad_kernel(SsmArgs a, Plan p) {
    using S = Shape<T, N>;
    extern __shared__ __align__(16) char smem[];
    GradMem<T, N> *all = reinterpret_cast<GradMem<T, N> *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    GradMem<T, N> &m = all[warp];
    const Place w = place_of<T, N>(a, p);
    const size_t page = (size_t)a.Di * N;
    const bool soft = a.flags & GDN_DT_SOFTPLUS;
    // the copies of a half block's saved state: a lane's are its own
    auto fetch_saved = [&](int t) {
        if (w.c0 < a.Di) {
            const size_t at = saved_at<T, N>(a, p, w, t);
            const float4 *from = reinterpret_cast<const float4 *>(p.state) + at * 128 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) copy16(&m.saved[e][lane], from + e * 32);
            copy16(&m.saved[4][lane], p.upto + at * S::CH + 4 * w.g);
        }
    };
    const int last = w.t0 + (w.t1 - 1 - w.t0) / kBlock * kBlock;
    mx::let_follow();
    fetch<T, N>(a, w, m, 0, last);
    mx::follow_on();
    fetch_saved(last + kHalf);
    copies_out();
    Quad A, g, dA;
    load_decays<N>(a, w, A);
    zero16(g);
    zero16(dA);
#pragma unroll
    for (int i = 0; i < S::VPL * S::V / 4; ++i) m.acc[0][i][lane] = m.acc[1][i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    // sequences without tokens pass their gradient on
    if (a.cu && a.ds0) {
        for (int s0 = w.chunk * 32; s0 < a.n_seq; s0 += p.chunks * 32) {
            const int s = s0 + lane;
            unsigned e = __ballot_sync(~0u, s < a.n_seq && mx::no_tokens(a.cu, a.T, min(s, a.n_seq - 1)));
            for (; e; e &= e - 1) {
                const size_t at = (size_t)(s0 + __ffs(e) - 1) * page;
                Quad h;
                load16<N>(a, w, a.dsf ? a.dsf + at : nullptr, h);
                store16<N>(a, w, a.ds0 + at, h);
            }
        }
    }
    // x <- what chunk j gives + its decay x, for n chunks from j on in steps of `step`;
    // four chunks' loads at a time
    auto join = [&](const float *from, int j, int step, int n, Quad &x) {
        for (int i0 = 0; i0 < n; i0 += 4) {
            Quad v[4];
            F2 d[4][2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k < n) {
                    const size_t at = chunk_at(a, p, w.row, j + (i0 + k) * step);
                    load16<N>(a, w, from + at * N, v[k]);
                    d[k][0] = d[k][1] = 0;
                    if (w.c < a.Di) channels(p.steps + at + w.c, d[k]);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k < n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            x[i][q] = i0 + k == 0 ? v[k][i][q] : fma2(exp2_2(mul2(d[k][i], A[i][q])), x[i][q], v[k][i][q]);
        }
    };
    Run r = mx::run_at(a.cu, a.n_seq, a.T, w.row, w.t0);
    const int entered = r.s >= 0 && r.start < w.t0 ? r.end : w.t0;  // the entering state matters up to here
    {
        Quad h;
        zero16(h);
        if (entered > w.t0) {
            const int first = min(r.start / p.len, w.chunk - 1);
            join(p.left, first, 1, w.chunk - first, h);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<ulonglong2 *>(&m.start[e][lane]) = quad_vector(h, e);
        r = mx::run_at(a.cu, a.n_seq, a.T, w.row, w.t1 - 1);
        if (r.s >= 0 && r.end > w.t1) {
            const int end = max((r.end - 1) / p.len, w.chunk + 1);
            join(p.back, end, -1, end - w.chunk, g);
        }
    }
    int buf = 0;
    for (int t = last; t >= w.t0; t -= kBlock, buf ^= 1) {
        copies_done(true);
        const Marks k = marks_of(a, w, t, r, m.seq);
        __syncwarp();
        if (t > w.t0) fetch<T, N>(a, w, m, buf ^ 1, t - kBlock);
        convert<T, N>(a, w, m, buf, t, k.dead);
        __syncwarp();
#pragma unroll 1
        for (int half = kBlock - kHalf; half >= 0; half -= kHalf) {
            if (half == 0) copies_done(true);
            Quad h0;  // before the half block
            {
                const bool there = w.c < a.Di;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    set_vector(h0, e, there ? *reinterpret_cast<const ulonglong2 *>(&m.saved[e][lane]) : make_ulonglong2(0, 0));
                if (there && t + half < entered) {
                    F2 d[2];
                    Quad s;
                    channels(reinterpret_cast<const float *>(&m.saved[4][lane]), d);
#pragma unroll
                    for (int e = 0; e < 4; ++e) set_vector(s, e, *reinterpret_cast<const ulonglong2 *>(&m.start[e][lane]));
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int n = 0; n < 4; ++n) h0[i][n] = fma2(exp2_2(mul2(d[i], A[i][n])), s[i][n], h0[i][n]);
                }
            }
            if (t + half > w.t0) fetch_saved(t + half - kHalf);
            copies_out();
            // the half block, with or without sequences that start or end in it or tokens of none
            auto block = [&](auto marked) {
                constexpr bool MARKED = decltype(marked)::value;  // few blocks: their states go through local memory
                constexpr int UNROLL = MARKED ? 1 : kHalf;
                Quad hs[kHalf + 1];  // before the half block, and after each of its tokens
#pragma unroll
                for (int i = 0; i < 8; ++i) hs[0][i >> 2][i & 3] = h0[i >> 2][i & 3];
#pragma unroll UNROLL
                for (int u = 0; u < kHalf; ++u) {
                    const int v = half + u;
                    if (MARKED && (k.dead >> v & 1)) {  // no state of a sequence before it passes here: it may be infinite
                        zero16(hs[u + 1]);
                        continue;
                    }
                    F2 d[2], x[2], b[4];
                    channels(&m.step[v][4 * w.g], d);
                    channels(&m.x[v][4 * w.g], x);
                    states(&m.b[v][8 * w.q], b);
                    const F2 in[2] = {mul2(d[0], x[0]), mul2(d[1], x[1])};
                    if (MARKED && (k.starts >> v & 1)) {
                        Quad first;
                        load16<N>(a, w, a.s0 ? a.s0 + m.seq[v] * page : nullptr, first);
                        advance(first, hs[u + 1], A, d, in, b);
                    } else {
                        advance(hs[u], hs[u + 1], A, d, in, b);
                    }
                }
#pragma unroll UNROLL
                for (int u = kHalf - 1; u >= 0; --u) {
                    const int v = half + u;
                    if (MARKED && (k.ends >> v & 1)) load16<N>(a, w, a.dsf ? a.dsf + m.seq[v] * page : nullptr, g);
                    F2 d[2], x[2], dy[2], b[4], c[4], dx[2], ds[2], y[2];
                    channels(&m.step[v][4 * w.g], d);
                    channels(&m.x[v][4 * w.g], x);
                    channels(&m.dy[v][4 * w.g], dy);
                    states(&m.b[v][8 * w.q], b);
                    states(&m.c[v][8 * w.q], c);
                    F2 dB[4], dC[4];
                    auto token = [&](const Quad &before) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const F2 in = mul2(d[i], x[i]);
                            F2 gb, ap, cy;
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                g[i][n] = fma2(c[n], dy[i], g[i][n]);
                                dC[n] = i ? fma2(hs[u + 1][i][n], dy[i], dC[n]) : mul2(hs[u + 1][i][n], dy[i]);
                                dB[n] = i ? fma2(g[i][n], in, dB[n]) : mul2(g[i][n], in);
                                if (GATE) cy = n ? fma2(hs[u + 1][i][n], c[n], cy) : mul2(hs[u + 1][i][n], c[n]);
                                gb = n ? fma2(g[i][n], b[n], gb) : mul2(g[i][n], b[n]);
                                g[i][n] = mul2(exp2_2(mul2(d[i], A[i][n])), g[i][n]);
                                const F2 passed = mul2(g[i][n], before[i][n]);
                                dA[i][n] = fma2(passed, d[i], dA[i][n]);
                                ap = n ? fma2(passed, A[i][n], ap) : mul2(passed, A[i][n]);
                            }
                            dx[i] = mul2(d[i], gb);
                            ds[i] = fma2(x[i], gb, mul2(ap, both(mx::kLn2)));
                            y[i] = cy;
                        }
                    };
                    if (MARKED && (k.dead >> v & 1)) {
                        zero16(g);
#pragma unroll
                        for (int n = 0; n < 4; ++n) dB[n] = dC[n] = 0;
                        dx[0] = dx[1] = ds[0] = ds[1] = y[0] = y[1] = 0;
                    } else if (MARKED && (k.starts >> v & 1)) {  // what came before is the sequence's initial state
                        Quad first;
                        load16<N>(a, w, a.s0 ? a.s0 + m.seq[v] * page : nullptr, first);
                        token(first);
                        if (a.ds0) store16<N>(a, w, a.ds0 + m.seq[v] * page, g);
                        zero16(g);
                    } else {
                        token(hs[u]);
                    }
                    auto put = [&](int what, const F2 (&v)[2]) {
                        *reinterpret_cast<ulonglong2 *>(&m.over_states[u % S::TOK][what][w.q][4 * w.g]) = make_ulonglong2(v[0], v[1]);
                    };
                    put(0, ds);
                    put(1, dx);
                    if (GATE) put(2, y);
                    float *row = m.over_channels[u % S::SLOTS][w.g];
                    *reinterpret_cast<float4 *>(row + (4 * w.q ^ S::swap(w.g))) = make_float4(sum(dB[0]), sum(dB[1]), sum(dB[2]), sum(dB[3]));
                    *reinterpret_cast<float4 *>(row + (N + 4 * w.q ^ S::swap(w.g))) = make_float4(sum(dC[0]), sum(dC[1]), sum(dC[2]), sum(dC[3]));
                    if (u % S::TOK != 0) continue;
                    __syncwarp();
                    // over step, x and dy of the tokens, which all lanes have read
                    constexpr int each = S::TOK * S::CH / 4, items = (GATE ? 3 : 2) * each;
#pragma unroll
                    for (int i0 = 0; i0 < items; i0 += 32) {
                        const int i = i0 + lane;
                        if (i >= items) break;
                        const int what = i / each, tok = i % each / (S::CH / 4), c4 = i % (S::CH / 4) * 4;
                        F2 p0 = 0, p1 = 0;
#pragma unroll
                        for (int q = 0; q < S::L; ++q) {
                            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&m.over_states[tok][what][q][c4]);
                            p0 = mx::add2(p0, v.x), p1 = mx::add2(p1, v.y);
                        }
                        *reinterpret_cast<ulonglong2 *>(&m.step[0][0] + (what * kBlock + v + tok) * S::ROW + c4) = make_ulonglong2(p0, p1);
                    }
                    if (u % S::SLOTS == 0)
#pragma unroll
                        for (int i = lane; i < S::SLOTS * N / 2; i += 32) {
                            const int tok = i / (N / 2), n = i % (N / 2) * 4;
                            F2 p0 = 0, p1 = 0;
#pragma unroll
                            for (int q = 0; q < S::G; ++q) {
                                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(&m.over_channels[tok][q][n ^ S::swap(q)]);
                                p0 = mx::add2(p0, v.x), p1 = mx::add2(p1, v.y);
                            }
                            *reinterpret_cast<ulonglong2 *>(&m.part[buf][v + tok][n]) = make_ulonglong2(p0, p1);
                        }
                    __syncwarp();
                }
            };
            if (k.starts | k.ends | k.dead) block(std::true_type{});
            else block(std::false_type{});
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < S::VPL; ++i) {
            const int j = i * 32 + lane, tok = j / S::RV, cv = j % S::RV * S::V, c = w.c0 + cv;
            if (j >= S::NV || t + tok >= w.t1 || c >= a.Di) continue;
            const size_t at = ((size_t)w.row * a.T + t + tok) * a.Di + c;
            float dx[S::V], dv[S::V], dz[S::V];
            if (k.dead >> tok & 1) {
#pragma unroll
                for (int e = 0; e < S::V; ++e) dx[e] = dv[e] = dz[e] = 0.f;
            } else {
                float x[S::V], dt[S::V], dy[S::V], bias[S::V], skip[S::V];
                get<S::V>(&m.x[tok][cv], dx);
                get<S::V>(&m.step[tok][cv], dv);
                unpack<T, S::V>(m.raw[buf][0][j], x);
                unpack<T, S::V>(m.raw[buf][1][j], dt);
                unpack<T, S::V>(m.raw[buf][2][j], dy);
                vector_of<S::V>(a.bias, c, bias);
                vector_of<S::V>(a.D, c, skip);
                float z[S::V];
                if (GATE) {
                    unpack<T, S::V>(m.raw[buf][3][j], z);
                    get<S::V>(&m.dy[tok][cv], dz);
                }
#pragma unroll
                for (int e = 0; e < S::V; e += 4) {
                    ulonglong2 &p = reinterpret_cast<ulonglong2 &>(m.acc[0][(i * S::V + e) / 4][lane]);
                    ulonglong2 &q = reinterpret_cast<ulonglong2 &>(m.acc[1][(i * S::V + e) / 4][lane]);
#pragma unroll
                    for (int f = e; f < e + 4; f += 2) {  // two at once
                        const F2 x2 = pair(x[f], x[f + 1]), skip2 = pair(skip[f], skip[f + 1]);
                        F2 dy2 = pair(dy[f], dy[f + 1]), dv2 = pair(dv[f], dv[f + 1]);
                        if (GATE) {
                            const F2 z2 = pair(z[f], z[f + 1]), s = mx::sigmoid2(z2);
                            const F2 out = mul2(dy2, fma2(skip2, x2, pair(dz[f], dz[f + 1])));
                            split(mul2(out, mx::silu_slope2(z2, s)), dz[f], dz[f + 1]);
                            dy2 = mul2(dy2, mul2(z2, s));
                        }
                        split(fma2(skip2, dy2, pair(dx[f], dx[f + 1])), dx[f], dx[f + 1]);
                        if (soft) dv2 = mul2(dv2, mx::sigmoid2(mx::add2(pair(dt[f], dt[f + 1]), pair(bias[f], bias[f + 1]))));
                        split(dv2, dv[f], dv[f + 1]);
                        F2 &pf = f == e ? p.x : p.y, &qf = f == e ? q.x : q.y;
                        pf = fma2(dy2, x2, pf), qf = mx::add2(qf, dv2);
                    }
                }
            }
            using Raw = typename Vec<T, S::V>::Raw;
            __stcs(reinterpret_cast<Raw *>(static_cast<T *>(a.dx) + at), Vec<T, S::V>::pack(dx));
            __stcs(reinterpret_cast<Raw *>(static_cast<T *>(a.ddt) + at), Vec<T, S::V>::pack(dv));
            if (GATE) __stcs(reinterpret_cast<Raw *>(static_cast<T *>(a.dz) + at), Vec<T, S::V>::pack(dz));
        }
        // dB and dC of the CTA's channels: the warps take turns at adding the four
        // shares, and the two buffers need one barrier a block
        __syncthreads();
        if (warp == (t / kBlock) % kWarps)
            for (int i = lane; i < kBlock * 2 * N; i += 32) {
                const int tok = i / (2 * N), n = i % (2 * N);
                float x = 0.f;
#pragma unroll
                for (int k2 = 0; k2 < kWarps; ++k2) x += all[k2].part[buf][tok][n];
                if (t + tok < w.t1) p.dBC[(((size_t)w.group * a.B + w.row) * a.T + t + tok) * 2 * N + n] = x;
            }
    }
    const size_t at = chunk_at(a, p, w.row, w.chunk);
    store16<N>(a, w, p.dA + at * N, dA);
    __syncwarp();
    for (int i = lane; i < S::CH; i += 32) {
        if (w.c0 + i >= a.Di) break;
        float x = 0.f, y = 0.f;
        for (int j = i / S::V; j < S::NV; j += S::RV) {
            const int v = j / 32 * S::V + i % S::V;
            x += reinterpret_cast<const float *>(&m.acc[0][v / 4][j % 32])[v % 4];
            y += reinterpret_cast<const float *>(&m.acc[1][v / 4][j % 32])[v % 4];
        }
        p.dD[at + w.c0 + i] = x;
        p.db[at + w.c0 + i] = y;
    }
}

// dB and dC from the groups' shares, a thread four of a token's values; then dA,
// dskip and dbias from the chunks'.
template <typename T, int N>
__global__ void __launch_bounds__(256) sum_kernel(SsmArgs a, Plan p, int tokens_ctas) {
    mx::follow_on();
    if (blockIdx.x < tokens_ctas) {
        const long long n = (long long)a.B * a.T * (N / 2), i = (long long)blockIdx.x * 256 + threadIdx.x;
        if (i >= n) return;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < p.groups; ++k) {
            const float4 v = __ldcs(reinterpret_cast<const float4 *>(p.dBC) + k * n + i);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const long long tok = i / (N / 2);
        const int at = (int)(i - tok * (N / 2)) * 4;
        const float out[4] = {s.x, s.y, s.z, s.w};
        T *to = static_cast<T *>(at < N ? a.dB : a.dC) + tok * N + at % N;
        *reinterpret_cast<typename Vec<T, 4>::Raw *>(to) = Vec<T, 4>::pack(out);
        return;
    }
    const long long i = (long long)(blockIdx.x - tokens_ctas) * 256 + threadIdx.x, each = (long long)a.Di * N;
    const int items = a.B * p.chunks;
    const float *from;
    float *to;
    long long step;
    if (i < each) from = p.dA + i, to = a.dA + i, step = each;
    else if (i < each + a.Di) from = p.dD + (i - each), to = a.dD ? a.dD + (i - each) : nullptr, step = a.Di;
    else if (i < each + 2 * a.Di) from = p.db + (i - each - a.Di), to = a.dbias ? a.dbias + (i - each - a.Di) : nullptr, step = a.Di;
    else return;
    if (!to) return;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < items; ++k) s += from[k * step];
    *to = s;
}

// CTAs of grad_kernel on an SM, by its shared memory (228 KB, 1 KB of it for each).
template <typename T, int N>
constexpr int kPerSm = 2 * (sizeof(GradMem<T, N>) * kWarps + 1024) <= 228 * 1024 ? 2 : 1;
int per_sm(int N, int dtype) {
    using B16 = __nv_bfloat16;
    if (dtype == GDN_BF16) return N == 8 ? kPerSm<B16, 8> : N == 16 ? kPerSm<B16, 16> : kPerSm<B16, 32>;
    return N == 8 ? kPerSm<float, 8> : N == 16 ? kPerSm<float, 16> : kPerSm<float, 32>;
}
int channels(int N) { return kWarps * 4 * (32 / (N / 4)); }

// The chunks' length: what a wave of grad_kernel's CTAs takes is about its tokens
// and half a token's time for each chunk of the row, which it joins at its start.
// Candidates are what fills up to four waves, and lengths a quarter apart.
Plan plan(int B, int T, int Di, int N, int dtype, float *ws, size_t *bytes) {
    Plan p{};
    p.groups = (Di + channels(N) - 1) / channels(N);
    const long long whole = (long long)B * p.groups, resident = 152LL * per_sm(N, dtype);
    double best = 0.;
    auto consider = [&](long long tokens) {
        const long long len = std::min((std::max(tokens, 1LL) + kBlock - 1) / kBlock * kBlock, ((long long)T + kBlock - 1) / kBlock * kBlock);
        const long long chunks = (T + len - 1) / len, waves = (whole * chunks + resident - 1) / resident;
        const double cost = (double)waves * ((double)len + 0.5 * (double)chunks);
        if (p.len == 0 || cost < best) best = cost, p.len = (int)len, p.chunks = (int)chunks;
    };
    for (int w = 1; w <= 4; ++w) {
        const long long chunks = std::max(1LL, w * resident / whole);
        consider((T + chunks - 1) / chunks);
    }
    for (long long len = kBlock; len < T; len += std::max((long long)kBlock, len / 4)) consider(len);
    p.halves = (T + kBlock - 1) / kBlock * (kBlock / kHalf);
    size_t at = 0;
    auto take = [&](float **x, size_t n) { *x = ws ? ws + at : nullptr, at += (n + 3) / 4 * 4; };
    // a half block's places are of whole warps
    const size_t per_chunk = (size_t)B * p.chunks * Di, per_half = (size_t)B * p.halves * p.groups * channels(N);
    take(&p.left, per_chunk * N);
    take(&p.back, per_chunk * N);
    take(&p.steps, per_chunk);
    take(&p.state, per_half * N);
    take(&p.upto, per_half);
    take(&p.dA, per_chunk * N);
    take(&p.dD, per_chunk);
    take(&p.db, per_chunk);
    take(&p.dBC, (size_t)p.groups * B * T * 2 * N);
    *bytes = at * sizeof(float);
    return p;
}

// Shared memory above 48 KB is asked for once on each device.
template <auto F>
bool room(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return false;
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(F, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

template <typename T, int N>
int bwd(const SsmArgs &a, cudaStream_t stream) {
    size_t bytes;
    const Plan p = plan(a.B, a.T, a.Di, N, a.dtype, static_cast<float *>(a.ws), &bytes);
    constexpr int one = sizeof(Mem<T, N>) * kWarps, two = sizeof(GradMem<T, N>) * kWarps;
    if (!room<share_kernel<T, N>>(one) || !room<grad_kernel<T, N, false>>(two) || !room<grad_kernel<T, N, true>>(two)) return GDN_ERR_CUDA;
    const unsigned ctas = (unsigned)((long long)p.groups * a.B * p.chunks);
    share_kernel<T, N><<<ctas, kThreads, one, stream>>>(a, p);
    int st = mx::launched();
    if (st != GDN_OK) return st;
    mx::follow(a.z ? grad_kernel<T, N, true> : grad_kernel<T, N, false>, ctas, kThreads, two, stream, a, p);
    st = mx::launched();
    if (st != GDN_OK) return st;
    const long long tokens = ((long long)a.B * a.T * (N / 2) + 255) / 256, rest = ((long long)a.Di * (N + 2) + 255) / 256;
    mx::follow(sum_kernel<T, N>, (unsigned)(tokens + rest), 256, 0, stream, a, p, (int)tokens);
    return mx::launched();
}

}  // namespace

size_t ssm_bwd_workspace(int B, int T, int Di, int N, int dtype) {
    size_t bytes;
    plan(B, T, Di, N, dtype, nullptr, &bytes);
    return bytes;
}

int launch_ssm_bwd(const SsmArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.N == 8 ? bwd<B16, 8>(a, stream) : a.N == 16 ? bwd<B16, 16>(a, stream) : bwd<B16, 32>(a, stream);
    return a.N == 8 ? bwd<float, 8>(a, stream) : a.N == 16 ? bwd<float, 16>(a, stream) : bwd<float, 32>(a, stream);
}

}  // namespace gdn
