// ssm_scan.cu -- the selective state space scan over prompts (ssm.cuh), and its
// single token.
//
// A thread holds all N states of its channels, a warp a block of
// consecutive channels; B and C of a token are the same for all of them and come
// from shared memory, where the warp has put a tile of tokens in fp32.  Warps do
// not wait for one another.  Exponentials bound it from below, one instruction of
// 32 a clock and SM; as it stands the issue does: 6.4 instructions a token, channel
// and state for a warp's 32 (4.2 in share_kernel), of them one exponential and 2
// packed multiply-adds, at 59% of the issue slots of 12 warps an SM, which is what
// the registers allow.  (Channels' states over four lanes, 20 warps an SM: 686 us
// for 498, by the shared memory through which their steps and sums go.)  Few rows
// and channels are cut into chunks of tokens: share_kernel walks each chunk but the
// last from 0, then every chunk starts from what the chunks before it leave, so
// that each exponential is taken twice.
// Measured, bf16, 16 states, gate: 32 x 1024 x 2048 whole 387 us, 1 x 32760 x 2048
// cut into 57 chunks 498 (exponentials alone 110 and 220), 4 x 4096 x 2048 262,
// 1 x 130 x 2048 12 (9 one after another).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ssm.cuh"

namespace gdn {
namespace {

using namespace ssm;
using mx::Run;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens of B and C in shared memory
constexpr int kGroup = 4;  // tokens of x, dt and z on their way
constexpr int kStates = 32, kCtas = 3;
constexpr long long kResident = 152 * kCtas * kWarps;  // warps

// How a row is cut.
struct Plan {
    int len, chunks;  // tokens of a chunk, a multiple of kTile; chunks of a row
    int blocks;       // of channels
    float *state;     // [row][chunk][block][V][32] float4: the state that the chunk leaves from 0
    float *steps;     // [row][chunk][block][CH][32]: the sum of its steps
    bool joined;      // join_kernel has put in `state` what each chunk leaves with all before it
};

constexpr int channels_of(int N) { return N >= kStates ? 1 : kStates / N; }  // a thread, where there are many

template <int N, int CH>
struct Shape {
    static constexpr int P = N / 2;                            // pairs of states a channel
    static constexpr int V = CH * N / 4;                       // vectors of 4 states a thread
    static constexpr int BLOCK = 32 * CH;                      // channels a warp
};

// A warp's tile of B (and C): [token][N] fp32, C behind B.
template <typename T, int N, bool WITH_C>
struct Tile {
    static constexpr int V = kWide<T>;               // elements a vector
    static constexpr int PER = N / V;                // vectors a token
    static constexpr int ALL = kTile * PER, K = (ALL + 31) / 32;  // vectors of a tile, of a lane
    using Raw = typename Vec<T, V>::Raw;
    Raw b[K], c[K];
    __device__ __forceinline__ void fetch(const SsmArgs &a, const T *B, const T *C, int t, int t1) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int j = i * 32 + lane, tok = t + j / PER;
            if (j < ALL && tok < t1) {
                b[i] = __ldg(reinterpret_cast<const Raw *>(B + tok * a.sB.t) + j % PER);
                if (WITH_C) c[i] = __ldg(reinterpret_cast<const Raw *>(C + tok * a.sC.t) + j % PER);
            }
        }
    }
    __device__ __forceinline__ void put(float *s) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int j = i * 32 + lane;
            if (j >= ALL) break;
            float x[V];
#pragma unroll
            for (int m = 0; m <= (WITH_C ? 1 : 0); ++m) {
                Vec<T, V>::unpack(m ? c[i] : b[i], x);
                float *to = s + (j / PER) * (WITH_C ? 2 * N : N) + m * N + (j % PER) * V;
#pragma unroll
                for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
        }
    }
};

// The steps D of a token's channels from dt as loaded, two at once where there are.
template <int CH>
__device__ __forceinline__ void steps_of(const float (&dt)[CH], const float (&bias)[CH], bool soft, float (&step)[CH]) {
    if constexpr (CH == 1) {
        const float v = dt[0] + bias[0];
        step[0] = soft ? mx::softplus(v) : v;
    } else {
#pragma unroll
        for (int e = 0; e < CH; e += 2) {
            const F2 v = mx::add2(pair(dt[e], dt[e + 1]), pair(bias[e], bias[e + 1]));
            split(soft ? mx::softplus2(v) : v, step[e], step[e + 1]);
        }
    }
}
template <int CH>
__device__ __forceinline__ void gate(const float (&z)[CH], float (&g)[CH]) {
#pragma unroll
    for (int e = 0; e < CH; ++e) g[e] = mx::silu(z[e]);
}

// h <- exp(D A) h + D x B of a token; `bc` points at its B (and C behind), the
// answer is C . h where OUT.
template <int N, int CH, bool OUT>
__device__ __forceinline__ void advance(F2 (&h)[CH][N / 2], const F2 (&A)[CH][N / 2], const float (&step)[CH], const float (&x)[CH],
                                        const float *bc, float (&y)[CH]) {
    F2 d[CH], u[CH], acc[2][CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) d[e] = both(step[e]), u[e] = both(step[e] * x[e]), acc[0][e] = acc[1][e] = 0;
#pragma unroll
    for (int n = 0; n < N / 2; n += 2) {
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(bc + 2 * n);
        ulonglong2 c;
        if (OUT) c = *reinterpret_cast<const ulonglong2 *>(bc + N + 2 * n);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < CH; ++e) {
                F2 &s = h[e][n + m];
                s = fma2(exp2_2(mul2(d[e], A[e][n + m])), s, mul2(u[e], m ? b.y : b.x));
                if (OUT) acc[m][e] = fma2(m ? c.y : c.x, s, acc[m][e]);
            }
    }
    if (OUT)
#pragma unroll
        for (int e = 0; e < CH; ++e) y[e] = sum(mx::add2(acc[0][e], acc[1][e]));
}

// A thread's states [Di,N] from or to memory, 0 where there are none.
template <int N, int CH>
__device__ __forceinline__ void load_states(const float *from, int c, F2 (&h)[CH][N / 2]) {
#pragma unroll
    for (int e = 0; e < CH; ++e)
#pragma unroll
        for (int n = 0; n < N / 2; n += 2) {
            ulonglong2 v = make_ulonglong2(0, 0);
            if (from) v = __ldg(reinterpret_cast<const ulonglong2 *>(from + (size_t)(c + e) * N + 2 * n));
            h[e][n] = v.x, h[e][n + 1] = v.y;
        }
}
template <int N, int CH>
__device__ __forceinline__ void store_states(float *to, int c, const F2 (&h)[CH][N / 2]) {
#pragma unroll
    for (int e = 0; e < CH; ++e)
#pragma unroll
        for (int n = 0; n < N / 2; n += 2)
            *reinterpret_cast<ulonglong2 *>(to + (size_t)(c + e) * N + 2 * n) = make_ulonglong2(h[e][n], h[e][n + 1]);
}

template <int N, int CH>
__device__ __forceinline__ void load_decays(const float *A, int c, bool there, F2 (&d)[CH][N / 2]) {
    load_states<N, CH>(there ? A : nullptr, c, d);
#pragma unroll
    for (int e = 0; e < CH; ++e)
#pragma unroll
        for (int n = 0; n < N / 2; ++n) d[e][n] = mul2(d[e][n], both(mx::kLog2e));
}

// A warp's place.
struct Place {
    int block, chunk, row, c, t0, t1;
    bool there;  // the thread's channels exist
};
template <int N, int CH>
__device__ __forceinline__ bool place_of(const SsmArgs &a, const Plan &p, int chunks, Place *w) {
    const long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const long long item = i / p.blocks;
    w->block = (int)(i - item * p.blocks);
    w->row = (int)(item / chunks), w->chunk = (int)(item - (long long)w->row * chunks);
    if (w->row >= a.B) return false;
    w->c = w->block * Shape<N, CH>::BLOCK + (threadIdx.x & 31) * CH;
    w->there = w->c < a.Di;
    w->t0 = w->chunk * p.len, w->t1 = min(w->t0 + p.len, a.T);
    return true;
}
__device__ __forceinline__ size_t share_at(const Plan &p, int row, int chunk, int block) {
    return ((size_t)row * p.chunks + chunk) * p.blocks + block;
}

// What a chunk leaves: from 0, or from the state of a sequence that starts in it
// and goes on behind it.
template <typename T, int N, int CH>
__global__ void __launch_bounds__(kThreads, kCtas) share_kernel(SsmArgs a, Plan p) {
    constexpr int P = Shape<N, CH>::P;
    using Raw = typename Vec<T, CH>::Raw;
    __shared__ __align__(16) float tiles[kWarps][kTile * N];
    mx::let_follow();
    Place w;
    if (!place_of<N, CH>(a, p, p.chunks - 1, &w)) return;
    const Run r = mx::run_at(a.cu, a.n_seq, a.T, w.row, w.t1 - 1);
    if (r.s < 0 || r.end <= w.t1) return;  // no sequence goes on behind the chunk
    const int ts = max(w.t0, r.start);
    const bool soft = a.flags & GDN_DT_SOFTPLUS;
    float *tile = tiles[threadIdx.x >> 5];
    const int c = w.there ? w.c : 0;
    F2 h[CH][P], A[CH][P];
    float bias[CH], total[CH];
    load_decays<N, CH>(a.A, c, w.there, A);
    load_states<N, CH>(ts == r.start && a.s0 && w.there ? a.s0 + (size_t)r.s * a.Di * N : nullptr, c, h);
#pragma unroll
    for (int e = 0; e < CH; ++e) bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f, total[e] = 0.f;
    const T *x = static_cast<const T *>(a.x) + w.row * a.sx.b + c, *dt = static_cast<const T *>(a.dt) + w.row * a.sdt.b + c;
    const T *B = static_cast<const T *>(a.Bt) + w.row * a.sB.b;
    Raw nx[kGroup], nt[kGroup];
    auto fetch = [&](int t) {
        const T *px = x + t * a.sx.t, *pt = dt + t * a.sdt.t;
        const bool whole = t + kGroup <= w.t1;
#pragma unroll
        for (int u = 0; u < kGroup; ++u, px += a.sx.t, pt += a.sdt.t)
            if (whole || t + u < w.t1) nx[u] = __ldg(reinterpret_cast<const Raw *>(px)), nt[u] = __ldg(reinterpret_cast<const Raw *>(pt));
    };
    auto step_of = [&](const Raw &vt, float (&step)[CH]) {
        float dv[CH];
        Vec<T, CH>::unpack(vt, dv);
        steps_of<CH>(dv, bias, soft, step);
    };
    auto token = [&](const Raw &vx, const float (&step)[CH], const float *b) {
        float xv[CH], none[CH];
        Vec<T, CH>::unpack(vx, xv);
#pragma unroll
        for (int e = 0; e < CH; ++e) total[e] += step[e];
        advance<N, CH, false>(h, A, step, xv, b, none);
    };
    Tile<T, N, false> next;
    next.fetch(a, B, nullptr, ts, w.t1);
    fetch(ts);
    for (int t = ts; t < w.t1; t += kTile) {
        __syncwarp();
        next.put(tile);
        next.fetch(a, B, nullptr, t + kTile, w.t1);
        __syncwarp();
#pragma unroll 1
        for (int g = 0; g < kTile && t + g < w.t1; g += kGroup) {
            Raw cx[kGroup], ct[kGroup];
#pragma unroll
            for (int u = 0; u < kGroup; ++u) cx[u] = nx[u], ct[u] = nt[u];
            fetch(t + g + kGroup);
            const float *b = tile + g * N;
            if (t + g + kGroup <= w.t1) {
                float step[kGroup][CH];  // their chains side by side
#pragma unroll
                for (int u = 0; u < kGroup; ++u) step_of(ct[u], step[u]);
#pragma unroll
                for (int u = 0; u < kGroup; ++u) token(cx[u], step[u], b + u * N);
            } else {  // the chunk's last tokens
#pragma unroll 1
                for (int i = t + g; i < w.t1; ++i, b += N) {
                    float step[CH];
                    step_of(ct[0], step);
                    token(cx[0], step, b);
#pragma unroll
                    for (int u = 0; u + 1 < kGroup; ++u) cx[u] = cx[u + 1], ct[u] = ct[u + 1];
                }
            }
        }
    }
    const size_t at = share_at(p, w.row, w.chunk, w.block);
    const int lane = threadIdx.x & 31;
    float4 *to = reinterpret_cast<float4 *>(p.state) + at * Shape<N, CH>::V * 32 + lane;
    const F2 *hs = &h[0][0];
#pragma unroll
    for (int i = 0; i < Shape<N, CH>::V; ++i) *reinterpret_cast<ulonglong2 *>(to + i * 32) = make_ulonglong2(hs[2 * i], hs[2 * i + 1]);
#pragma unroll
    for (int e = 0; e < CH; ++e) p.steps[(at * CH + e) * 32 + lane] = total[e];
}

// What the chunks of a row leave, each with those before it of its sequence, in
// place: a thread 4 of a block's states, the next chunks' loads on their way.  A
// warp that joins all chunks before its own takes the latency of each.
template <int N, int CH>
__global__ void __launch_bounds__(32 * Shape<N, CH>::V) join_kernel(SsmArgs a, Plan p) {
    constexpr int P = Shape<N, CH>::P, V = Shape<N, CH>::V, AHEAD = 8;
    const int row = blockIdx.x / p.blocks, block = blockIdx.x - row * p.blocks;
    const int lane = threadIdx.x & 31, i = threadIdx.x >> 5, e = 2 * i / P, n = 2 * i % P * 2;  // vector i of the lane's
    const int c = block * Shape<N, CH>::BLOCK + lane * CH + e;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < a.Di) A = __ldg(reinterpret_cast<const float4 *>(a.A + (size_t)c * N + n));
    const F2 A0 = mul2(pair(A.x, A.y), both(mx::kLog2e)), A1 = mul2(pair(A.z, A.w), both(mx::kLog2e));
    mx::let_follow();
    mx::follow_on();
    ulonglong2 *state = reinterpret_cast<ulonglong2 *>(p.state) + i * 32 + lane;
    const float *steps = p.steps + e * 32 + lane;
    F2 h0 = 0, h1 = 0;
    int starts = 0;  // where the run at the end of chunk j + lane starts, for each 32 chunks
    for (int j0 = 0; j0 + 1 < p.chunks; j0 += AHEAD) {
        if (j0 % 32 == 0) starts = mx::run_at(a.cu, a.n_seq, a.T, row, (int)min((long long)(j0 + lane + 1) * p.len, (long long)a.T) - 1).start;
        ulonglong2 v[AHEAD];
        float d[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (j0 + k + 1 < p.chunks) {
                const size_t at = share_at(p, row, j0 + k, block);
                v[k] = state[at * V * 32], d[k] = steps[at * CH * 32];
            }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int j = j0 + k;
            if (j + 1 >= p.chunks) break;
            if (__shfl_sync(~0u, starts, j % 32) >= j * p.len) h0 = v[k].x, h1 = v[k].y;
            else h0 = fma2(exp2_2(mul2(both(d[k]), A0)), h0, v[k].x), h1 = fma2(exp2_2(mul2(both(d[k]), A1)), h1, v[k].y);
            state[share_at(p, row, j, block) * V * 32] = make_ulonglong2(h0, h1);
        }
    }
}

template <typename T, int N, int CH, bool GATE>
__global__ void __launch_bounds__(kThreads, kCtas) scan_kernel(SsmArgs a, Plan p) {
    constexpr int P = Shape<N, CH>::P, V = Shape<N, CH>::V;
    using Raw = typename Vec<T, CH>::Raw;
    __shared__ __align__(16) float tiles[kWarps][kTile * 2 * N];
    Place w;
    if (!place_of<N, CH>(a, p, p.chunks, &w)) return;
    const bool soft = a.flags & GDN_DT_SOFTPLUS;
    const int lane = threadIdx.x & 31;
    float *tile = tiles[threadIdx.x >> 5];
    const int c = w.there ? w.c : 0;
    const size_t page = (size_t)a.Di * N;
    const T *x = static_cast<const T *>(a.x) + w.row * a.sx.b + c, *dt = static_cast<const T *>(a.dt) + w.row * a.sdt.b + c;
    const T *z = GATE ? static_cast<const T *>(a.z) + w.row * a.sz.b + c : nullptr;
    const T *B = static_cast<const T *>(a.Bt) + w.row * a.sB.b, *C = static_cast<const T *>(a.Ct) + w.row * a.sC.b;
    T *y = static_cast<T *>(a.y) + w.row * a.sy.b + c;
    Raw nx[kGroup], nt[kGroup], nz[kGroup];
    auto fetch = [&](int t) {
        const T *px = x + t * a.sx.t, *pt = dt + t * a.sdt.t, *pz = z + t * a.sz.t;
        const bool whole = t + kGroup <= w.t1;
#pragma unroll
        for (int u = 0; u < kGroup; ++u, px += a.sx.t, pt += a.sdt.t, pz += a.sz.t)
            if (whole || t + u < w.t1) {
                nx[u] = __ldg(reinterpret_cast<const Raw *>(px)), nt[u] = __ldg(reinterpret_cast<const Raw *>(pt));
                if (GATE) nz[u] = __ldg(reinterpret_cast<const Raw *>(pz));
            }
    };
    Tile<T, N, true> next;
    next.fetch(a, B, C, w.t0, w.t1);
    fetch(w.t0);
    F2 h[CH][P], A[CH][P];
    float bias[CH], skip[CH];
    load_decays<N, CH>(a.A, c, w.there, A);
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        bias[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
        skip[e] = a.D ? __ldg(a.D + c + e) : 0.f;
    }
    mx::follow_on();
    // sequences without tokens pass their state on
    if (a.cu && a.sf) {
        for (int s0 = w.chunk * 32; s0 < a.n_seq; s0 += p.chunks * 32) {
            const int s = s0 + lane;
            unsigned m = __ballot_sync(~0u, s < a.n_seq && mx::no_tokens(a.cu, a.T, min(s, a.n_seq - 1)));
            for (; m; m &= m - 1) {
                const size_t q = (size_t)(s0 + __ffs(m) - 1) * page;
                load_states<N, CH>(a.s0 && w.there ? a.s0 + q : nullptr, c, h);
                if (w.there) store_states<N, CH>(a.sf + q, c, h);
            }
        }
    }
    Run r = mx::run_at(a.cu, a.n_seq, a.T, w.row, w.t0);
    auto enter = [&](bool fresh) { load_states<N, CH>(fresh && r.s >= 0 && a.s0 && w.there ? a.s0 + r.s * page : nullptr, c, h); };
    enter(r.start == w.t0);
    if (r.s >= 0 && r.start < w.t0) {  // what the chunks before this one leave
        if (p.joined) {
            const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(p.state) + share_at(p, w.row, w.chunk - 1, w.block) * V * 32 + lane;
            F2 *hs = &h[0][0];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const ulonglong2 v = from[i * 32];
                hs[2 * i] = v.x, hs[2 * i + 1] = v.y;
            }
        } else {
            const int first = min(r.start / p.len, w.chunk - 1);
            for (int j = first; j < w.chunk; ++j) {
                const size_t at = share_at(p, w.row, j, w.block);
                const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(p.state) + at * V * 32 + lane;
                F2 d[CH];
#pragma unroll
                for (int e = 0; e < CH; ++e) d[e] = both(p.steps[(at * CH + e) * 32 + lane]);
                F2 *hs = &h[0][0];
                const F2 *As = &A[0][0];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const ulonglong2 v = from[i * 32];
                    hs[2 * i] = j == first ? v.x : fma2(exp2_2(mul2(d[2 * i / P], As[2 * i])), hs[2 * i], v.x);
                    hs[2 * i + 1] = j == first ? v.y : fma2(exp2_2(mul2(d[(2 * i + 1) / P], As[2 * i + 1])), hs[2 * i + 1], v.y);
                }
            }
        }
    }
    auto factors_of = [&](const Raw &vt, const Raw &vz, float (&step)[CH], float (&g)[CH]) {
        float dv[CH];
        Vec<T, CH>::unpack(vt, dv);
        steps_of<CH>(dv, bias, soft, step);
        if (GATE) {
            float zv[CH];
            Vec<T, CH>::unpack(vz, zv);
            gate<CH>(zv, g);
        }
    };
    auto token = [&](const Raw &vx, const float (&step)[CH], const float (&g)[CH], const float *bc, T *to) {
        float xv[CH], out[CH];
        Vec<T, CH>::unpack(vx, xv);
        advance<N, CH, true>(h, A, step, xv, bc, out);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            out[e] = fmaf(skip[e], xv[e], out[e]);
            if (GATE) out[e] *= g[e];
        }
        if (w.there) __stcs(reinterpret_cast<Raw *>(to), r.s < 0 ? Raw{} : Vec<T, CH>::pack(out));
    };
    for (int t = w.t0; t < w.t1; t += kTile) {
        __syncwarp();
        next.put(tile);
        next.fetch(a, B, C, t + kTile, w.t1);
        __syncwarp();
#pragma unroll 1
        for (int g = 0; g < kTile && t + g < w.t1; g += kGroup) {
            Raw cx[kGroup], ct[kGroup], cz[kGroup];
#pragma unroll
            for (int u = 0; u < kGroup; ++u) cx[u] = nx[u], ct[u] = nt[u], cz[u] = nz[u];
            fetch(t + g + kGroup);
            const float *bc = tile + g * 2 * N;
            T *to = y + (t + g) * a.sy.t;
            if (t + g + kGroup <= w.t1 && t + g + kGroup <= r.end && t + g < r.end) {
                float step[kGroup][CH], g[kGroup][CH];  // their chains side by side
#pragma unroll
                for (int u = 0; u < kGroup; ++u) factors_of(ct[u], cz[u], step[u], g[u]);
#pragma unroll
                for (int u = 0; u < kGroup; ++u, to += a.sy.t) token(cx[u], step[u], g[u], bc + u * 2 * N, to);
            } else {
#pragma unroll 1
                for (int i = t + g; i < w.t1 && i < t + g + kGroup; ++i, bc += 2 * N, to += a.sy.t) {
                    if (i == r.end) {
                        if (a.sf && r.s >= 0 && w.there) store_states<N, CH>(a.sf + r.s * page, c, h);
                        r = mx::run_at(a.cu, a.n_seq, a.T, w.row, i);
                        enter(true);
                    }
                    float step[CH], g[CH];
                    factors_of(ct[0], cz[0], step, g);
                    token(cx[0], step, g, bc, to);
#pragma unroll
                    for (int u = 0; u + 1 < kGroup; ++u) cx[u] = cx[u + 1], ct[u] = ct[u + 1], cz[u] = cz[u + 1];
                }
            }
        }
    }
    if (a.sf && r.s >= 0 && w.there && r.end == w.t1) store_states<N, CH>(a.sf + r.s * page, c, h);
}

// Few warps are cut into more: as many as are resident at once.  A row that fills
// half of them by itself stays whole, as every exponential of a cut row is taken
// twice.  A chunk has sqrt(T) tokens or more: joining a chunk takes a launch about
// as long as walking one more token (40 channels of 18531 tokens: 442 us in 1158
// chunks, 98 in 129).
constexpr int kJoin = 16;  // from so many chunks of a row on they are joined by a launch of its own
template <int N, int CH>
Plan plan(int B, int T, int Di) {
    Plan p{};
    p.blocks = (Di + Shape<N, CH>::BLOCK - 1) / Shape<N, CH>::BLOCK;
    const long long whole = (long long)B * p.blocks;
    const long long chunks = whole * 2 >= kResident ? 1 : kResident / whole;
    const long long len = std::max((T + chunks - 1) / chunks, (long long)std::sqrt((double)T));
    p.len = (int)((len + kTile - 1) / kTile * kTile);
    p.chunks = (T + p.len - 1) / p.len;
    return p;
}
// A call that does not fill the SMs takes as long as a warp's tokens, which half as
// many channels a warp shorten: up to seven eighths of the warps that fit, if so
// many more fit at once.  Full, it is slower by what B and C from shared memory
// cost.  Measured, bf16, 2048 channels of 16 states, one channel a thread against
// two: 130 tokens 9.0 and 13.6 us, 500 17.0 and 20.3, 2048 45.7 and 52.6, 4096 (full)
// 82.9 and 79.9; 32 rows of 1024 (2048 warps where 1824 fit) 455 and 385.
template <int N>
bool thin(int B, int T, int Di) {
    constexpr int CH = channels_of(N), HALF = CH > 1 ? CH / 2 : 1;
    const Plan p = plan<N, CH>(B, T, Di), q = plan<N, HALF>(B, T, Di);
    return CH > 1 && (long long)B * p.chunks * p.blocks * 8 <= 7 * kResident && (long long)B * q.chunks * q.blocks <= kResident;
}
template <int N, int CH>
size_t shares(int B, int T, int Di) {
    const Plan p = plan<N, CH>(B, T, Di);
    return p.chunks == 1 ? 0 : (size_t)B * p.chunks * p.blocks * 32 * CH * (N + 1) * sizeof(float);
}
template <int N>
size_t workspace(int B, int T, int Di) {
    constexpr int CH = channels_of(N), HALF = CH > 1 ? CH / 2 : 1;
    return thin<N>(B, T, Di) ? shares<N, HALF>(B, T, Di) : shares<N, CH>(B, T, Di);
}

template <typename T, int N, int CH>
int fwd_with(const SsmArgs &a, cudaStream_t stream) {
    Plan p = plan<N, CH>(a.B, a.T, a.Di);
    const size_t n = (size_t)a.B * p.chunks * p.blocks;
    p.state = static_cast<float *>(a.ws);
    p.steps = p.state + n * 128 * Shape<N, CH>::V;
    auto ctas = [&](int chunks) { return (unsigned)(((long long)a.B * chunks * p.blocks + kWarps - 1) / kWarps); };
    if (p.chunks > 1) {
        share_kernel<T, N, CH><<<ctas(p.chunks - 1), kThreads, 0, stream>>>(a, p);
        int st = mx::launched();
        if (st != GDN_OK) return st;
        p.joined = p.chunks >= kJoin;
        if (p.joined) {
            mx::follow(join_kernel<N, CH>, (unsigned)((long long)a.B * p.blocks), 32 * Shape<N, CH>::V, 0, stream, a, p);
            st = mx::launched();
            if (st != GDN_OK) return st;
        }
    }
    const auto kernel = a.z ? scan_kernel<T, N, CH, true> : scan_kernel<T, N, CH, false>;
    if (p.chunks > 1) mx::follow(kernel, ctas(p.chunks), kThreads, 0, stream, a, p);
    else kernel<<<ctas(p.chunks), kThreads, 0, stream>>>(a, p);
    return mx::launched();
}
template <typename T, int N>
int fwd(const SsmArgs &a, cudaStream_t stream) {
    constexpr int CH = channels_of(N), HALF = CH > 1 ? CH / 2 : 1;
    return thin<N>(a.B, a.T, a.Di) ? fwd_with<T, N, HALF>(a, stream) : fwd_with<T, N, CH>(a, stream);
}

// One token a row: eight states a thread, the N/8 threads of a channel together,
// R rows a thread, whose A is read once.  The bytes of the states bound it, read
// and written once; with four states a thread what belongs to the channel (its
// step, its gate) was worked out four times over and took as long.  Measured: 256 rows of 2048 bf16
// channels of 16 states 16.4 us (70 MB at 4.3 TB/s).
constexpr int kStepThreads = 128;
template <typename T, int N, int R>
__global__ void __launch_bounds__(kStepThreads) step_kernel(SsmStepArgs a) {
    constexpr int L = N / 8;  // lanes of a channel, which take its float4 q and q + L
    const int i = blockIdx.x * kStepThreads + threadIdx.x, c = i / L, q = i % L, groups = (a.B + R - 1) / R;
    const int b0 = blockIdx.y;  // rows b0, b0 + groups, ..
    if (c >= a.Di) return;  // a channel's lanes are there or not together
    using One = typename Vec<T, 1>::Raw;
    using Four = typename Vec<T, 4>::Raw;
    auto load = [](const void *p, long long i, auto *to) {
        using Raw = std::remove_pointer_t<decltype(to)>;
        *to = __ldg(reinterpret_cast<const Raw *>(static_cast<const T *>(p) + i));
    };
    auto one = [](const One &p) {
        float v[1];
        Vec<T, 1>::unpack(p, v);
        return v[0];
    };
    auto two = [](const float4 &v, F2 (&x)[2]) { x[0] = pair(v.x, v.y), x[1] = pair(v.z, v.w); };
    int slot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = b0 + r * groups;
        slot[r] = b >= a.B ? -1 : a.slots ? __ldg(a.slots + b) : b;
        if (slot[r] >= a.n_slots) slot[r] = -1;
    }
    // all of the rows' loads before any of their arithmetic
    float4 state[R][2];
    One x[R], dt[R], z[R];
    Four B[R][2], C[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (slot[r] >= 0) {
            const int b = b0 + r * groups;
            const float4 *page = reinterpret_cast<const float4 *>(a.state + ((size_t)slot[r] * a.Di + c) * N);
            state[r][0] = __ldcs(page + q), state[r][1] = __ldcs(page + q + L);
            load(a.x, b * a.sx + c, &x[r]);
            load(a.dt, b * a.sdt + c, &dt[r]);
            if (a.z) load(a.z, b * a.sz + c, &z[r]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                load(a.Bt, b * a.sB + 4 * (q + k * L), &B[r][k]);
                load(a.Ct, b * a.sC + 4 * (q + k * L), &C[r][k]);
            }
        }
    F2 A[2][2];
    two(__ldg(reinterpret_cast<const float4 *>(a.A + (size_t)c * N) + q), A[0]);
    two(__ldg(reinterpret_cast<const float4 *>(a.A + (size_t)c * N) + q + L), A[1]);
    const float bias = a.bias ? __ldg(a.bias + c) : 0.f, skip = a.D ? __ldg(a.D + c) : 0.f;
    const unsigned mask = L == 1 ? 1u << (threadIdx.x & 31) : (L == 2 ? 0x3u : 0xfu) << ((threadIdx.x & 31) / L * L);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int b = b0 + r * groups;
        if (b >= a.B) break;
        float out[1] = {0.f};
        if (slot[r] >= 0) {
            const float xv = one(x[r]), v = one(dt[r]) + bias;
            const float step = (a.flags & GDN_DT_SOFTPLUS) ? mx::softplus(v) : v;
            const F2 u = both(step * xv), d = both(step * mx::kLog2e);
            F2 o = 0;
            float4 *page = reinterpret_cast<float4 *>(a.state_out + ((size_t)slot[r] * a.Di + c) * N);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                F2 h[2], bs[2], cs[2];
                mx::unpack2<T, 4>(B[r][k], bs);
                mx::unpack2<T, 4>(C[r][k], cs);
                two(state[r][k], h);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    h[m] = fma2(exp2_2(mul2(d, A[k][m])), h[m], mul2(u, bs[m]));
                    o = fma2(cs[m], h[m], o);
                }
                float4 n;
                split(h[0], n.x, n.y), split(h[1], n.z, n.w);
                __stcs(page + q + k * L, n);
            }
            out[0] = sum(o);
#pragma unroll
            for (int m = 1; m < L; m <<= 1) out[0] += __shfl_xor_sync(mask, out[0], m);
            out[0] = fmaf(skip, xv, out[0]);
            if (a.z) out[0] *= mx::silu(one(z[r]));
        }
        if (q == 0) *reinterpret_cast<One *>(static_cast<T *>(a.y) + (size_t)b * a.Di + c) = Vec<T, 1>::pack(out);
    }
}

template <typename T, int N>
int step(const SsmStepArgs &a, cudaStream_t stream) {
    const size_t size = sizeof(T);
    for (int b0 = 0; b0 < a.B; b0 += 65535) {  // grid.y's limit
        SsmStepArgs p = a;
        p.B = std::min(a.B - b0, 65535);
        auto at = [&](const void *x, long long row) { return x ? static_cast<const char *>(x) + (size_t)b0 * row * size : nullptr; };
        p.x = at(a.x, a.sx), p.dt = at(a.dt, a.sdt), p.Bt = at(a.Bt, a.sB), p.Ct = at(a.Ct, a.sC), p.z = at(a.z, a.sz);
        p.y = const_cast<char *>(at(a.y, a.Di));
        if (a.slots) {
            p.slots = a.slots + b0;
        } else {
            p.state = a.state + (size_t)b0 * a.Di * N, p.state_out = a.state_out + (size_t)b0 * a.Di * N;
            p.n_slots = a.n_slots - b0;
        }
        const unsigned ctas = (unsigned)(((long long)a.Di * (N / 8) + kStepThreads - 1) / kStepThreads);
        // two rows a thread where that leaves each SM eight CTAs; four were slower (256 rows of 2048 channels: 22 us against 16)
        if ((long long)ctas * p.B >= 2LL * 8 * device_sm_count()) step_kernel<T, N, 2><<<dim3(ctas, (p.B + 1) / 2), kStepThreads, 0, stream>>>(p);
        else step_kernel<T, N, 1><<<dim3(ctas, p.B), kStepThreads, 0, stream>>>(p);
        const int st = mx::launched();
        if (st != GDN_OK) return st;
    }
    return GDN_OK;
}

}  // namespace

size_t ssm_fwd_workspace(int B, int T, int Di, int N, int) {
    return N == 8 ? workspace<8>(B, T, Di) : N == 16 ? workspace<16>(B, T, Di) : workspace<32>(B, T, Di);
}

int launch_ssm_fwd(const SsmArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.N == 8 ? fwd<B16, 8>(a, stream) : a.N == 16 ? fwd<B16, 16>(a, stream) : fwd<B16, 32>(a, stream);
    return a.N == 8 ? fwd<float, 8>(a, stream) : a.N == 16 ? fwd<float, 16>(a, stream) : fwd<float, 32>(a, stream);
}

int launch_ssm_step(const SsmStepArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.N == 8 ? step<B16, 8>(a, stream) : a.N == 16 ? step<B16, 16>(a, stream) : step<B16, 32>(a, stream);
    return a.N == 8 ? step<float, 8>(a, stream) : a.N == 16 ? step<float, 16>(a, stream) : step<float, 32>(a, stream);
}

}  // namespace gdn
