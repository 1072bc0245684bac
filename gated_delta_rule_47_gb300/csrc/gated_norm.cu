// gated_norm.cu -- the norm of a mixer's output by head, with its gate, in front of
// the output projection; and its backward.
//
//   y = w n(x) act(g),  n(u) = u / sqrt(mean u^2 + eps) over a head's D columns,
//   or with GDN_GATE_FIRST  y = w n(x act(g));   act: SiLU or the sigmoid
//
// backward, r = 1 / sqrt(..), u = x or x act(g), t = w dy act(g) or w dy:
//   du = r (t - n mean(n t)),   dw = sum dy n act(g) or dy n
//   dg = dy w n act'(g) or du x act'(g),   dx = du or du act(g)
//
// One pass: NT threads hold a row's head in registers between its sums and its
// outputs; the bytes bound it.  A group of threads keeps to one head and walks the
// tokens, the next row's loads on their way, so that the weights stay in
// registers, and the head's share of dw does too.
#include "mixer.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Where a group of NT threads works: head h of tokens first, first + step, ..
struct Walk {
    int h, first, step, tid;
};
template <int NT>
__device__ __forceinline__ Walk walk_of(const GatedNormArgs &a, int strips) {
    const long long slot = (long long)blockIdx.x * (kThreads / NT) + threadIdx.x / NT;
    const int strip = (int)(slot / a.H);
    return {(int)(slot - (long long)strip * a.H), strip < strips ? strip : 0x7fffffff, strips, (int)threadIdx.x % NT};
}
template <typename T>
__device__ __forceinline__ T *row_at(T *p, const HeadStrides &s, int b, int t, int h) {
    return p + b * s.b + t * s.t + h * s.h;
}

// Sums over the NT threads of a group; where it spans warps, `s` alternates.
template <int NT, int K>
__device__ __forceinline__ void group_sum(float (&x)[K], float (*s)[kThreads / 32]) {
#pragma unroll
    for (int m = (NT < 32 ? NT : 32) / 2; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(~0u, x[k], m);
    if constexpr (NT > 32) {
        const int warp = threadIdx.x >> 5, first = threadIdx.x / NT * (NT / 32);
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) s[k][warp] = x[k];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / NT), "n"(NT) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = 0.f;
#pragma unroll
            for (int i = 0; i < NT / 32; ++i) x[k] += s[k][first + i];
        }
    }
}

using mx::F2;

// The gate's activation and its slope, of pairs: act = s m and slope = s ((1 - s) m
// + k) with s the sigmoid; SiLU has m = gate and k = 1, the sigmoid m = 1 and k = 0.
struct Act {
    F2 k, rest;
    __device__ __forceinline__ explicit Act(bool sigmoid) : k(mx::both(sigmoid ? 0.f : 1.f)), rest(mx::both(sigmoid ? 1.f : 0.f)) {}
    __device__ __forceinline__ F2 factor(F2 gate) const { return mx::fma2(gate, k, rest); }
    __device__ __forceinline__ F2 slope(F2 s, F2 m) const {
        return mx::mul2(s, mx::fma2(mx::fma2(s, mx::both(-1.f), mx::both(1.f)), m, k));
    }
};

// V vectors a thread: vector j of thread t is number j NT + t; what a row lacks is 0
// and stays so.  Measured, bf16: 4 x 4096 tokens of 16 heads of 128 36 us (201 MB at
// 5.6 TB/s), calls back to back in a graph.
template <typename T, int NT, int V, bool FIRST>
__global__ void __launch_bounds__(kThreads) gated_kernel(GatedNormArgs a, int strips) {
    constexpr int N = kWide<T>, P = N / 2;
    using Raw = typename Vec<T, N>::Raw;
    __shared__ float red[2][1][kThreads / 32];
    const Walk k = walk_of<NT>(a, strips);
    const int nv = a.D / N, tokens = a.B * a.T;
    const Act act(a.flags & GDN_GATE_SIGMOID);
    F2 w[V][P];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + k.tid;
        mx::weights2<N>(a.w + ((a.flags & GDN_W_SHARED) ? 0 : k.h * a.D) + i * N, a.w && i < nv, w[j]);
    }
    Raw nx[V], ng[V];
    auto fetch = [&](int token) {
        const int b = token / a.T, t = token - b * a.T;
        const Raw *x = reinterpret_cast<const Raw *>(row_at(static_cast<const T *>(a.x), a.sx, b, t, k.h));
        const Raw *g = reinterpret_cast<const Raw *>(row_at(static_cast<const T *>(a.gate), a.sg, b, t, k.h));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + k.tid;
            nx[j] = ng[j] = Raw{};
            if (token < tokens && i < nv) nx[j] = __ldcs(x + i), ng[j] = __ldcs(g + i);
        }
    };
    // every group of a CTA takes as many turns, so that warps stay whole
    const int turns = (tokens - 1) / strips + 1;
    int token = k.first < tokens ? k.first : tokens, buf = 0;
    fetch(token);
    for (int turn = 0; turn < turns; ++turn, buf ^= 1) {
        F2 x[V][P], g[V][P], s2 = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mx::unpack2<T, N>(nx[j], x[j]);
            mx::unpack2<T, N>(ng[j], g[j]);
        }
        const int now = token;
        token = token < tokens - k.step ? token + k.step : tokens;
        fetch(token);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) {
                g[j][e] = mx::mul2(mx::sigmoid2(g[j][e]), act.factor(g[j][e]));
                if (FIRST) x[j][e] = mx::mul2(x[j][e], g[j][e]);
                s2 = mx::fma2(x[j][e], x[j][e], s2);
            }
        float ss[1] = {mx::sum(s2)};
        group_sum<NT, 1>(ss, red[buf]);
        const F2 r = mx::both(rsqrtf(ss[0] / a.D + a.eps));
        if (now >= tokens) continue;
        Raw *y = reinterpret_cast<Raw *>(static_cast<T *>(a.y) + ((size_t)now * a.H + k.h) * a.D);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                x[j][e] = mx::mul2(x[j][e], mx::mul2(r, w[j][e]));
                if (!FIRST) x[j][e] = mx::mul2(x[j][e], g[j][e]);
            }
            if (j * NT + k.tid < nv) __stcs(y + j * NT + k.tid, mx::pack2<T, N>(x[j]));
        }
    }
}

// part: with a weight for each head [strips][H][D]; with one for all, a CTA's
// groups are added up: [gridDim.x][D].  Measured, bf16: 4 x 4096 tokens of 16 heads of 128 68
// us (335 MB at 4.9 TB/s) and 6 for the sum; with single instead of paired
// arithmetic 77.  Another row on its way made no difference.
template <typename T, int NT, int V, bool FIRST>
__global__ void __launch_bounds__(kThreads, V == 1 ? 2 : 1) gated_bwd_kernel(GatedNormArgs a, int strips, float *part) {
    mx::let_follow();
    constexpr int N = kWide<T>, P = N / 2, GROUPS = kThreads / NT;
    using Raw = typename Vec<T, N>::Raw;
    __shared__ float red[2][2][kThreads / 32];
    extern __shared__ __align__(16) float share[];  // [GROUPS][D], where the weight is shared
    const Walk k = walk_of<NT>(a, strips);
    const int nv = a.D / N, tokens = a.B * a.T;
    const bool shared = a.flags & GDN_W_SHARED;
    const Act act(a.flags & GDN_GATE_SIGMOID);
    F2 w[V][P], dw[V][P];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + k.tid;
        mx::weights2<N>(a.w + (shared ? 0 : k.h * a.D) + i * N, a.w && i < nv, w[j]);
#pragma unroll
        for (int e = 0; e < P; ++e) dw[j][e] = 0;
    }
    Raw nx[V], ng[V], nd[V];
    auto fetch = [&](int token) {
        const int b = token / a.T, t = token - b * a.T;
        const Raw *x = reinterpret_cast<const Raw *>(row_at(static_cast<const T *>(a.x), a.sx, b, t, k.h));
        const Raw *g = reinterpret_cast<const Raw *>(row_at(static_cast<const T *>(a.gate), a.sg, b, t, k.h));
        const Raw *d = reinterpret_cast<const Raw *>(row_at(static_cast<const T *>(a.dy), a.sdy, b, t, k.h));
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + k.tid;
            nx[j] = ng[j] = nd[j] = Raw{};
            if (token < tokens && i < nv) nx[j] = __ldcs(x + i), ng[j] = __ldcs(g + i), nd[j] = __ldcs(d + i);
        }
    };
    const int turns = (tokens - 1) / strips + 1;
    int token = k.first < tokens ? k.first : tokens, buf = 0;
    fetch(token);
    for (int turn = 0; turn < turns; ++turn, buf ^= 1) {
        F2 x[V][P], m[V][P], s[V][P], d[V][P], s2 = 0, p2 = 0;  // m: the activation's factor
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mx::unpack2<T, N>(nx[j], x[j]);
            mx::unpack2<T, N>(ng[j], s[j]);
            mx::unpack2<T, N>(nd[j], d[j]);
        }
        const int now = token;
        token = token < tokens - k.step ? token + k.step : tokens;
        fetch(token);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < P; ++e) {
                m[j][e] = act.factor(s[j][e]);
                s[j][e] = mx::sigmoid2(s[j][e]);
                const F2 f = mx::mul2(s[j][e], m[j][e]);
                const F2 u = FIRST ? mx::mul2(x[j][e], f) : x[j][e], t = FIRST ? d[j][e] : mx::mul2(d[j][e], f);
                s2 = mx::fma2(u, u, s2);
                p2 = mx::fma2(u, mx::mul2(t, w[j][e]), p2);
            }
        float sums[2] = {mx::sum(s2), mx::sum(p2)};
        group_sum<NT, 2>(sums, red[buf]);
        const float r1 = rsqrtf(sums[0] / a.D + a.eps);
        const F2 r = mx::both(r1), mean = mx::both(-r1 * r1 * (sums[1] / a.D));
        if (now >= tokens) continue;
        const int b = now / a.T, t0 = now - b * a.T;
        Raw *dx = reinterpret_cast<Raw *>(row_at(static_cast<T *>(a.dx), a.sdx, b, t0, k.h));
        Raw *dg = reinterpret_cast<Raw *>(static_cast<T *>(a.dgate) + ((size_t)now * a.H + k.h) * a.D);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            F2 ox[P], og[P];
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const F2 f = mx::mul2(s[j][e], m[j][e]), slope = act.slope(s[j][e], m[j][e]);
                const F2 u = FIRST ? mx::mul2(x[j][e], f) : x[j][e], t = FIRST ? d[j][e] : mx::mul2(d[j][e], f);
                const F2 du = mx::mul2(r, mx::fma2(u, mean, mx::mul2(t, w[j][e]))), n = mx::mul2(u, r);
                ox[e] = FIRST ? mx::mul2(du, f) : du;
                og[e] = mx::mul2(slope, FIRST ? mx::mul2(du, x[j][e]) : mx::mul2(n, mx::mul2(d[j][e], w[j][e])));
                dw[j][e] = mx::fma2(t, n, dw[j][e]);
            }
            if (j * NT + k.tid < nv) {
                __stcs(dx + j * NT + k.tid, mx::pack2<T, N>(ox));
                __stcs(dg + j * NT + k.tid, mx::pack2<T, N>(og));
            }
        }
    }
    const bool mine = k.first < strips;  // groups past the last strip have nothing
    float *to = shared ? share + (threadIdx.x / NT) * a.D : part + ((size_t)(mine ? k.first : 0) * a.H + k.h) * a.D;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + k.tid;
        if (i < nv && (mine || shared))
#pragma unroll
            for (int e = 0; e < P; e += 2) *reinterpret_cast<ulonglong2 *>(to + i * N + 2 * e) = make_ulonglong2(dw[j][e], dw[j][e + 1]);
    }
    if (!shared) return;
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kThreads) {
        float x = share[i];
#pragma unroll 4
        for (int q = 1; q < GROUPS; ++q) x += share[q * a.D + i];
        part[(size_t)blockIdx.x * a.D + i] = x;
    }
}

__global__ void __launch_bounds__(1024) gated_sum_kernel(const float *part, float *out, int n, long long C) {
    const long long c = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
    mx::follow_on();
    const float x = mx::column_sum<32>(part, n, C, c);
    if (threadIdx.x < 32 && c < C) out[c] = x;
}

// Threads of a group and vectors a thread, by a head's vectors; and how the tokens
// of a head are shared out.
int group_threads(int nv) {
    int nt = 8;
    while (nt < 256 && nt < nv) nt *= 2;
    return nv <= 8 ? 8 : nt;
}
struct Cut {
    int strips, ctas;
};
constexpr int kMostCtas = 152 * 3;  // of a backward, whose workspace holds their sums
Cut cut_tokens(int B, int T, int H, int groups, int most) {
    const long long tokens = (long long)B * T;
    long long strips = (long long)most * groups / H;
    if (strips < 1) strips = 1;
    if (strips > tokens) strips = tokens;
    return {(int)strips, (int)((strips * H + groups - 1) / groups)};
}

template <typename T, int NT, int V, bool FIRST>
int fwd(const GatedNormArgs &a, cudaStream_t stream) {
    const Cut c = cut_tokens(a.B, a.T, a.H, kThreads / NT, mx::resident_ctas<gated_kernel<T, NT, V, FIRST>, kThreads>());
    gated_kernel<T, NT, V, FIRST><<<c.ctas, kThreads, 0, stream>>>(a, c.strips);
    return mx::launched();
}
template <typename T, int NT, int V, bool FIRST>
int bwd(const GatedNormArgs &a, cudaStream_t stream) {
    constexpr int GROUPS = kThreads / NT;
    const int fit = mx::resident_ctas<gated_bwd_kernel<T, NT, V, FIRST>, kThreads>();
    const Cut c = cut_tokens(a.B, a.T, a.H, GROUPS, fit < kMostCtas ? fit : kMostCtas);
    const bool shared = a.flags & GDN_W_SHARED;
    float *part = static_cast<float *>(a.ws);
    const size_t room = shared ? sizeof(float) * GROUPS * a.D : 0;  // at most 32 KB: a group's threads grow with D
    gated_bwd_kernel<T, NT, V, FIRST><<<c.ctas, kThreads, room, stream>>>(a, c.strips, part);
    const int st = mx::launched();
    if (st != GDN_OK) return st;
    const long long C = shared ? a.D : (long long)a.H * a.D;  // up to 2^31 - 1
    mx::follow(gated_sum_kernel, (unsigned)((C + 31) / 32), 1024, 0, stream, part, a.dw, shared ? c.ctas : c.strips, C);
    return mx::launched();
}

// A row of up to NT vectors has one a thread, up to 1024 (bf16) or 2048 (fp32) four or eight.
template <typename T, bool BACK>
int launch(const GatedNormArgs &a, cudaStream_t stream) {
    const int nv = a.D / kWide<T>;
#define GO(NT, V)                                                                                        \
    return a.flags & GDN_GATE_FIRST ? (BACK ? bwd<T, NT, V, true>(a, stream) : fwd<T, NT, V, true>(a, stream)) \
                                    : (BACK ? bwd<T, NT, V, false>(a, stream) : fwd<T, NT, V, false>(a, stream))
    switch (group_threads(nv)) {
        case 8: GO(8, 1);
        case 16: GO(16, 1);
        case 32: GO(32, 1);
        case 64: GO(64, 1);
        case 128: GO(128, 1);
        default:
            if (nv <= 256) GO(256, 1);
            if (nv <= 512) GO(256, 2);
            if (nv <= 1024) GO(256, 4);
            GO(256, sizeof(T) == 2 ? 4 : 8);
    }
#undef GO
}

}  // namespace

int launch_gated_norm(const GatedNormArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16, false>(a, stream) : launch<float, false>(a, stream);
}
size_t gated_norm_bwd_workspace(int B, int T, int H, int D, unsigned flags) {
    // the types' groups differ: the larger of both
    size_t most = 0;
    for (int n = 4; n <= 8; n += 4) {
        const Cut c = cut_tokens(B, T, H, kThreads / group_threads(D / n), kMostCtas);
        const size_t rows = (flags & GDN_W_SHARED) ? (size_t)c.ctas : (size_t)c.strips * H;
        most = rows > most ? rows : most;
    }
    return sizeof(float) * most * D;
}
int launch_gated_norm_bwd(const GatedNormArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16, true>(a, stream) : launch<float, true>(a, stream);
}

}  // namespace gdn
