// ssm_scan.cu -- the selective state space scan over prompts (ssm.cuh), and its
// single token.
//
// A thread holds all N states of its channels (32 states), a warp a block of
// consecutive channels; B and C of a token are the same for all of them and come
// from shared memory, where the warp has put a tile of tokens in fp32.  Warps do
// not wait for one another.  Exponentials bound it: one instruction of 32 a clock
// and SM.  Few rows and channels are cut into chunks of tokens: share_kernel
// walks each chunk but the last from 0, then every chunk starts from what the
// chunks before it leave, so that each exponential is taken twice.
#include <algorithm>

#include "ssm.cuh"

namespace gdn {
namespace {

using namespace ssm;
using mx::Run;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens of B and C in shared memory
constexpr int kGroup = 4;  // tokens of x, dt and z on their way

// How a row is cut.
struct Plan {
    int len, chunks;  // tokens of a chunk, a multiple of kTile; chunks of a row
    int blocks;       // of channels
    float *state;     // [row][chunk][block][8][32] float4: the state that the chunk leaves from 0
    float *steps;     // [row][chunk][block][CH][32]: the sum of its steps
};

template <int N>
struct Shape {
    static constexpr int CH = 32 / N;           // channels a thread
    static constexpr int P = N / 2;             // pairs of states a channel
    static constexpr int BLOCK = 32 * CH;       // channels a warp
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

// The steps D of a token's channels from dt as loaded.
template <int CH>
__device__ __forceinline__ void steps_of(const float (&dt)[CH], const float (&bias)[CH], bool soft, float (&step)[CH]) {
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float v = dt[e] + bias[e];
        step[e] = soft ? mx::softplus(v) : v;
    }
}

// h <- exp(D A) h + D x B of a token; `bc` points at its B (and C behind), the
// answer is C . h where OUT.
template <int N, int CH, bool OUT>
__device__ __forceinline__ void advance(F2 (&h)[CH][N / 2], const F2 (&A)[CH][N / 2], const float (&step)[CH], const float (&x)[CH],
                                        const float *bc, float (&y)[CH]) {
    F2 d[CH], u[CH], acc[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) d[e] = both(step[e]), u[e] = both(step[e] * x[e]), acc[e] = 0;
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
                if (OUT) acc[e] = fma2(m ? c.y : c.x, s, acc[e]);
            }
    }
    if (OUT)
#pragma unroll
        for (int e = 0; e < CH; ++e) y[e] = sum(acc[e]);
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
template <int N>
__device__ __forceinline__ bool place_of(const SsmArgs &a, const Plan &p, int chunks, Place *w) {
    const int groups = (p.blocks + kWarps - 1) / kWarps;
    const int g = blockIdx.x % groups, item = blockIdx.x / groups;
    w->block = g * kWarps + (threadIdx.x >> 5);
    w->row = item / chunks, w->chunk = item - w->row * chunks;
    if (w->block >= p.blocks) return false;
    w->c = w->block * Shape<N>::BLOCK + (threadIdx.x & 31) * Shape<N>::CH;
    w->there = w->c < a.Di;
    w->t0 = w->chunk * p.len, w->t1 = min(w->t0 + p.len, a.T);
    return true;
}
__device__ __forceinline__ size_t share_at(const Plan &p, int row, int chunk, int block) {
    return ((size_t)row * p.chunks + chunk) * p.blocks + block;
}

// What a chunk leaves: from 0, or from the state of a sequence that starts in it
// and goes on behind it.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 4) share_kernel(SsmArgs a, Plan p) {
    constexpr int CH = Shape<N>::CH, P = Shape<N>::P;
    using Raw = typename Vec<T, CH>::Raw;
    __shared__ __align__(16) float tiles[kWarps][kTile * N];
    Place w;
    if (!place_of<N>(a, p, p.chunks - 1, &w)) return;
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
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (t + u < w.t1) {
                nx[u] = __ldg(reinterpret_cast<const Raw *>(x + (t + u) * a.sx.t));
                nt[u] = __ldg(reinterpret_cast<const Raw *>(dt + (t + u) * a.sdt.t));
            }
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
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                if (t + g + u >= w.t1) break;
                float xv[CH], dv[CH], step[CH], none[CH];
                Vec<T, CH>::unpack(cx[u], xv);
                Vec<T, CH>::unpack(ct[u], dv);
                steps_of<CH>(dv, bias, soft, step);
#pragma unroll
                for (int e = 0; e < CH; ++e) total[e] += step[e];
                advance<N, CH, false>(h, A, step, xv, tile + (g + u) * N, none);
            }
        }
    }
    const size_t at = share_at(p, w.row, w.chunk, w.block);
    const int lane = threadIdx.x & 31;
    float4 *to = reinterpret_cast<float4 *>(p.state) + at * 8 * 32 + lane;
    const F2 *hs = &h[0][0];
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<ulonglong2 *>(to + i * 32) = make_ulonglong2(hs[2 * i], hs[2 * i + 1]);
#pragma unroll
    for (int e = 0; e < CH; ++e) p.steps[(at * CH + e) * 32 + lane] = total[e];
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 3) scan_kernel(SsmArgs a, Plan p) {
    constexpr int CH = Shape<N>::CH, P = Shape<N>::P;
    using Raw = typename Vec<T, CH>::Raw;
    __shared__ __align__(16) float tiles[kWarps][kTile * 2 * N];
    Place w;
    if (!place_of<N>(a, p, p.chunks, &w)) return;
    const bool soft = a.flags & GDN_DT_SOFTPLUS;
    const int lane = threadIdx.x & 31;
    float *tile = tiles[threadIdx.x >> 5];
    const int c = w.there ? w.c : 0;
    const size_t page = (size_t)a.Di * N;
    const T *x = static_cast<const T *>(a.x) + w.row * a.sx.b + c, *dt = static_cast<const T *>(a.dt) + w.row * a.sdt.b + c;
    const T *z = a.z ? static_cast<const T *>(a.z) + w.row * a.sz.b + c : nullptr;
    const T *B = static_cast<const T *>(a.Bt) + w.row * a.sB.b, *C = static_cast<const T *>(a.Ct) + w.row * a.sC.b;
    T *y = static_cast<T *>(a.y) + w.row * a.sy.b + c;
    Raw nx[kGroup], nt[kGroup], nz[kGroup];
    auto fetch = [&](int t) {
#pragma unroll
        for (int u = 0; u < kGroup; ++u)
            if (t + u < w.t1) {
                nx[u] = __ldg(reinterpret_cast<const Raw *>(x + (t + u) * a.sx.t));
                nt[u] = __ldg(reinterpret_cast<const Raw *>(dt + (t + u) * a.sdt.t));
                if (z) nz[u] = __ldg(reinterpret_cast<const Raw *>(z + (t + u) * a.sz.t));
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
        const int first = min(r.start / p.len, w.chunk - 1);
        for (int j = first; j < w.chunk; ++j) {
            const size_t at = share_at(p, w.row, j, w.block);
            const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(p.state) + at * 8 * 32 + lane;
            F2 d[CH];
#pragma unroll
            for (int e = 0; e < CH; ++e) d[e] = both(p.steps[(at * CH + e) * 32 + lane]);
            F2 *hs = &h[0][0];
            const F2 *As = &A[0][0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const ulonglong2 v = from[i * 32];
                hs[2 * i] = j == first ? v.x : fma2(exp2_2(mul2(d[2 * i / P], As[2 * i])), hs[2 * i], v.x);
                hs[2 * i + 1] = j == first ? v.y : fma2(exp2_2(mul2(d[(2 * i + 1) / P], As[2 * i + 1])), hs[2 * i + 1], v.y);
            }
        }
    }
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
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                const int i = t + g + u;
                if (i >= w.t1) break;
                if (i == r.end) {
                    if (a.sf && r.s >= 0 && w.there) store_states<N, CH>(a.sf + r.s * page, c, h);
                    r = mx::run_at(a.cu, a.n_seq, a.T, w.row, i);
                    enter(true);
                }
                float xv[CH], dv[CH], step[CH], out[CH];
                Vec<T, CH>::unpack(cx[u], xv);
                Vec<T, CH>::unpack(ct[u], dv);
                steps_of<CH>(dv, bias, soft, step);
                advance<N, CH, true>(h, A, step, xv, tile + (g + u) * 2 * N, out);
#pragma unroll
                for (int e = 0; e < CH; ++e) out[e] = fmaf(skip[e], xv[e], out[e]);
                if (z) {
                    float zv[CH];
                    Vec<T, CH>::unpack(cz[u], zv);
#pragma unroll
                    for (int e = 0; e < CH; ++e) out[e] *= mx::silu(zv[e]);
                }
                if (r.s < 0)
#pragma unroll
                    for (int e = 0; e < CH; ++e) out[e] = 0.f;
                if (w.there) __stcs(reinterpret_cast<Raw *>(y + i * a.sy.t), Vec<T, CH>::pack(out));
            }
        }
    }
    if (a.sf && r.s >= 0 && w.there && r.end == w.t1) store_states<N, CH>(a.sf + r.s * page, c, h);
}

// Few warps are cut into more: as many as are resident at once.  A row that fills
// half of them by itself stays whole, as every exponential of a cut row is taken
// twice.
constexpr int kResident = 152 * 3 * kWarps;
template <int N>
Plan plan(int B, int T, int Di) {
    Plan p{};
    p.blocks = (Di + Shape<N>::BLOCK - 1) / Shape<N>::BLOCK;
    const long long whole = (long long)B * p.blocks;
    long long chunks = whole * 2 >= kResident ? 1 : kResident / whole;
    long long len = ((T + chunks - 1) / chunks + kTile - 1) / kTile * kTile;
    p.len = (int)len;
    p.chunks = (int)((T + len - 1) / len);
    return p;
}
Plan plan_of(int B, int T, int Di, int N) { return N == 8 ? plan<8>(B, T, Di) : N == 16 ? plan<16>(B, T, Di) : plan<32>(B, T, Di); }

template <typename T, int N>
int fwd(const SsmArgs &a, cudaStream_t stream) {
    Plan p = plan<N>(a.B, a.T, a.Di);
    const size_t shares = (size_t)a.B * p.chunks * p.blocks;
    p.state = static_cast<float *>(a.ws);
    p.steps = p.state + shares * 1024;
    const long long groups = (p.blocks + kWarps - 1) / kWarps;
    if (p.chunks > 1) {
        share_kernel<T, N><<<(unsigned)(groups * a.B * (p.chunks - 1)), kThreads, 0, stream>>>(a, p);
        const int st = mx::launched();
        if (st != GDN_OK) return st;
    }
    scan_kernel<T, N><<<(unsigned)(groups * a.B * p.chunks), kThreads, 0, stream>>>(a, p);
    return mx::launched();
}

// One token a row: four states a thread, the N/4 threads of a channel together.
// The bytes of the states bound it, read and written once.
constexpr int kStepThreads = 256;
template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads) step_kernel(SsmStepArgs a) {
    constexpr int L = N / 4;  // lanes of a channel
    const int i = blockIdx.x * kStepThreads + threadIdx.x, c = i / L, q = i % L, b = blockIdx.y;
    const bool there = c < a.Di;
    const int slot = a.slots ? a.slots[b] : b;
    T *y = static_cast<T *>(a.y) + (size_t)b * a.Di + c;
    if (slot < 0 || slot >= a.n_slots) {  // an idle row
        float none[1] = {0.f};
        if (there && q == 0) *reinterpret_cast<typename Vec<T, 1>::Raw *>(y) = Vec<T, 1>::pack(none);
        return;
    }
    if (!there) return;
    auto at = [](const void *p, long long i) {
        float v[1];
        Vec<T, 1>::unpack(__ldg(reinterpret_cast<const typename Vec<T, 1>::Raw *>(static_cast<const T *>(p) + i)), v);
        return v[0];
    };
    const size_t place = ((size_t)slot * a.Di + c) * N + 4 * q;
    const float4 h = __ldcs(reinterpret_cast<const float4 *>(a.state + place));
    const float4 A = __ldg(reinterpret_cast<const float4 *>(a.A + (size_t)c * N) + q);
    float B[4], C[4];
    Vec<T, 4>::unpack(__ldg(reinterpret_cast<const typename Vec<T, 4>::Raw *>(static_cast<const T *>(a.Bt) + b * a.sB) + q), B);
    Vec<T, 4>::unpack(__ldg(reinterpret_cast<const typename Vec<T, 4>::Raw *>(static_cast<const T *>(a.Ct) + b * a.sC) + q), C);
    const float x = at(a.x, b * a.sx + c), v = at(a.dt, b * a.sdt + c) + (a.bias ? __ldg(a.bias + c) : 0.f);
    const float step = (a.flags & GDN_DT_SOFTPLUS) ? mx::softplus(v) : v, u = step * x, d = step * mx::kLog2e;
    float4 n;
    n.x = fmaf(mx::exp2_fast(d * A.x), h.x, u * B[0]), n.y = fmaf(mx::exp2_fast(d * A.y), h.y, u * B[1]);
    n.z = fmaf(mx::exp2_fast(d * A.z), h.z, u * B[2]), n.w = fmaf(mx::exp2_fast(d * A.w), h.w, u * B[3]);
    __stcs(reinterpret_cast<float4 *>(a.state_out + place), n);
    float o = fmaf(C[0], n.x, fmaf(C[1], n.y, fmaf(C[2], n.z, C[3] * n.w)));
    // a channel's lanes are there or not together
    const unsigned mask = (L == 8 ? 0xffu : L == 4 ? 0xfu : 0x3u) << ((threadIdx.x & 31) / L * L);
#pragma unroll
    for (int m = 1; m < L; m <<= 1) o += __shfl_xor_sync(mask, o, m);
    if (q == 0) {
        if (a.D) o = fmaf(__ldg(a.D + c), x, o);
        if (a.z) o *= mx::silu(at(a.z, b * a.sz + c));
        float out[1] = {o};
        *reinterpret_cast<typename Vec<T, 1>::Raw *>(y) = Vec<T, 1>::pack(out);
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
        const long long lanes = (long long)a.Di * (N / 4);
        step_kernel<T, N><<<dim3((unsigned)((lanes + kStepThreads - 1) / kStepThreads), p.B), kStepThreads, 0, stream>>>(p);
        const int st = mx::launched();
        if (st != GDN_OK) return st;
    }
    return GDN_OK;
}

}  // namespace

size_t ssm_fwd_workspace(int B, int T, int Di, int N, int) {
    const Plan p = plan_of(B, T, Di, N);
    if (p.chunks == 1) return 0;
    return (size_t)B * p.chunks * p.blocks * (1024 + 32 * (32 / N)) * sizeof(float);
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
