// causal_conv.cu -- the short causal convolution in front of a mixer: each
// channel of a token sees its own last W inputs, with a bias and SiLU.
//
//   z_t = b + sum_j w[j] x_{t-W+1+j};   y = silu(z) or z
//
// Inputs before a sequence's start are its window's W-1 rows, or 0; the window
// it leaves is the last W-1 inputs, counted over window and tokens.  Backward:
//   dz = dy silu'(z),  dx_t = sum_j w[j] dz_{t+W-1-j},
//   dw[j] = sum_t dz_t x_{t-W+1+j},  db = sum_t dz_t
//
// The bytes bound it: 2 rows a token forwards, 3 backwards.  A thread walks a
// strip of tokens of its channels with the last inputs (and the unfinished
// gradients) in registers, so that a row is read once but for the W-1 rows
// around a strip's ends; strips are as long as one wave of threads allows.
#include "mixer.cuh"

namespace gdn {
namespace {

using mx::F2;
using mx::Run;
using mx::pack2;
using mx::unpack2;

// Weights [C,W] of channels c .. c+N-1.
template <int N, int W>
__device__ __forceinline__ void load_taps(const float *w, int c, float (&t)[W][N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if constexpr (W == 4) {
            const float4 y = __ldg(reinterpret_cast<const float4 *>(w) + c + e);
            t[0][e] = y.x, t[1][e] = y.y, t[2][e] = y.z, t[3][e] = y.w;
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) t[j][e] = __ldg(w + (size_t)(c + e) * W + j);
        }
    }
}

template <typename T, int N>
__device__ __forceinline__ void load(const T *p, float (&x)[N]) {
    Vec<T, N>::unpack(*reinterpret_cast<const typename Vec<T, N>::Raw *>(p), x);
}
template <typename T, int N>
__device__ __forceinline__ void store(T *p, const float (&x)[N]) {
    *reinterpret_cast<typename Vec<T, N>::Raw *>(p) = Vec<T, N>::pack(x);
}
template <int N>
__device__ __forceinline__ void zero(float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
}

// One thread's place: vector `v` of the channels, tokens t0 .. t1-1 of a row.
struct Strip {
    int c, row, t0, t1, index, strips;
};
template <int N>
__device__ __forceinline__ bool strip_of(const ConvArgs &a, int len, int per_row, Strip *s) {
    const int nv = a.C / N;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int strip = (int)(i / nv);
    s->strips = per_row * a.B;
    if (strip >= s->strips) return false;
    s->c = (int)(i - (long long)strip * nv) * N;
    s->index = strip;
    s->row = strip / per_row;
    s->t0 = (strip - s->row * per_row) * len;
    s->t1 = min(s->t0 + len, a.T);
    return true;
}

// The inputs before token t of run r, x[t-1] first.
template <typename T, int N, int W>
__device__ __forceinline__ void load_past(const ConvArgs &a, const T *x, const Run &r, int t, int c, float (&past)[W - 1][N]) {
#pragma unroll
    for (int k = 1; k < W; ++k) {
        zero<N>(past[k - 1]);
        if (r.s < 0) continue;
        if (t - k >= r.start) load<T, N>(x + (t - k) * a.sx.t, past[k - 1]);
        else if (a.win) load<T, N>(static_cast<const T *>(a.win) + ((size_t)r.s * (W - 1) + (W - 1 + t - r.start - k)) * a.C + c, past[k - 1]);
    }
}

// The windows of sequences without tokens are passed on, sequence s by strip s, s + strips, ..
template <typename T, int N>
__device__ __forceinline__ void pass_windows(const ConvArgs &a, const Strip &s, int rows, const void *from, void *to) {
    if (!a.cu || !to) return;
    for (int q = s.index; q < a.n_seq; q += s.strips) {
        if (!mx::no_tokens(a.cu, a.T, q)) continue;
        for (int r = 0; r < rows; ++r) {
            const size_t at = ((size_t)q * rows + r) * a.C + s.c;
            float x[N];
            zero<N>(x);
            if (from) load<T, N>(static_cast<const T *>(from) + at, x);
            store<T, N>(static_cast<T *>(to) + at, x);
        }
    }
}

constexpr int kThreads = 128;

template <int N>
__device__ __forceinline__ void pairs(const float (&v)[N], F2 (&x)[N / 2]) {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) x[e] = mx::pair(v[2 * e], v[2 * e + 1]);
}

// N channels a thread: 16 bytes.  Tokens go in groups of U; a group inside one run
// has no conditions.  Measured, bf16, W 4, SiLU: 32760 x
// 8192 packed, windows in and out, 178 us (1.07 GB at 6.0 TB/s), 4 x 4096 x 6144 74
// (5.4); with four tokens on their way, 32 KB an SM, 183.
template <typename T, int N, int W>
__global__ void __launch_bounds__(kThreads, 3) conv_kernel(ConvArgs a, int len, int per_row) {
    using Raw = typename Vec<T, N>::Raw;
    constexpr int U = sizeof(T) == 2 ? 8 : 4, P = N / 2;
    Strip s;
    if (!strip_of<N>(a, len, per_row, &s)) return;
    const bool act = a.flags & GDN_SILU;
    F2 w[W][P], bias[P], past[W - 1][P];
    {
        float t[W][N], b[N];
        load_taps<N, W>(a.w, s.c, t);
#pragma unroll
        for (int j = 0; j < W; ++j) pairs<N>(t[j], w[j]);
#pragma unroll
        for (int e = 0; e < N; ++e) b[e] = a.bias ? __ldg(a.bias + s.c + e) : 0.f;
        pairs<N>(b, bias);
    }
    const T *x = static_cast<const T *>(a.x) + s.row * a.sx.b + s.c;
    T *y = static_cast<T *>(a.y) + s.row * a.sy.b + s.c;
    Raw next[U];
    auto fetch = [&](int t) {
        const T *p = x + t * a.sx.t;
        if (t + U <= s.t1) {
#pragma unroll
            for (int u = 0; u < U; ++u, p += a.sx.t) next[u] = __ldg(reinterpret_cast<const Raw *>(p));
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u, p += a.sx.t)
                if (t + u < s.t1) next[u] = __ldg(reinterpret_cast<const Raw *>(p));
        }
    };
    fetch(s.t0);
    pass_windows<T, N>(a, s, W - 1, a.win, a.win_out);
    Run r = mx::run_at(a.cu, a.n_seq, a.T, s.row, s.t0);
    auto enter = [&](int t) {
        float p[W - 1][N];
        load_past<T, N, W>(a, x, r, t, s.c, p);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) pairs<N>(p[k], past[k]);
    };
    enter(s.t0);
    auto token = [&](const Raw &in, T *to) {
        F2 v[P], z[P];
        unpack2<T, N>(in, v);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            z[e] = mx::fma2(w[W - 1][e], v[e], bias[e]);
#pragma unroll
            for (int k = 1; k < W; ++k) z[e] = mx::fma2(w[W - 1 - k][e], past[k - 1][e], z[e]);
            if (act) z[e] = mx::mul2(z[e], mx::sigmoid2(z[e]));
#pragma unroll
            for (int k = W - 1; k > 1; --k) past[k - 1][e] = past[k - 2][e];
            past[0][e] = v[e];
        }
        __stcs(reinterpret_cast<Raw *>(to), r.s < 0 ? Raw{} : pack2<T, N>(z));
    };
    for (int t = s.t0; t < s.t1; t += U) {
        Raw now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        fetch(t + U);
        T *to = y + t * a.sy.t;
        if (t + U <= s.t1 && t + U < r.end) {
#pragma unroll
            for (int u = 0; u < U; ++u, to += a.sy.t) token(now[u], to);
            continue;
        }
#pragma unroll
        for (int u = 0; u < U; ++u, to += a.sy.t) {
            if (t + u >= s.t1) break;
            if (t + u == r.end) {
                r = mx::run_at(a.cu, a.n_seq, a.T, s.row, t + u);
                enter(t + u);
            }
            token(now[u], to);
            if (a.win_out && r.s >= 0 && t + u + 1 == r.end)
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    *reinterpret_cast<Raw *>(static_cast<T *>(a.win_out) + ((size_t)r.s * (W - 1) + (W - 2 - k)) * a.C + s.c) =
                        pack2<T, N>(past[k]);
        }
    }
}

// Backward, N channels a thread: 4, as twice as many would leave too few threads
// resident beside the taps, their gradients, the inputs and the unfinished dx.
// A strip goes on for the W-1 tokens behind it, whose dz its last dx need; dw and
// db count its own.  part: [strips][W+1][C].  Tokens go in groups as forwards: the
// conditions of a strip's and a run's ends took three times the arithmetic's
// instructions.  Measured, bf16, W 4, SiLU: 4 x 4096 x 6144 121 us (604 MB at 5.0
// TB/s; 278 with the conditions at every token, 129 with four tokens on their way).
template <typename T, int N, int W>
__global__ void __launch_bounds__(kThreads, 3) conv_bwd_kernel(ConvArgs a, int len, int per_row, float *part) {
    mx::let_follow();
    using Raw = typename Vec<T, N>::Raw;
    constexpr int U = sizeof(T) == 2 ? 8 : 2, P = N / 2;
    Strip s;
    if (!strip_of<N>(a, len, per_row, &s)) return;
    const bool act = a.flags & GDN_SILU;
    F2 w[W][P], bias[P], past[W - 1][P], dw[W][P], db[P];
    F2 open[W - 1][P];  // dx so far of tokens t-1, t-2, ..
    {
        float t[W][N], b[N];
        load_taps<N, W>(a.w, s.c, t);
#pragma unroll
        for (int j = 0; j < W; ++j) pairs<N>(t[j], w[j]);
#pragma unroll
        for (int e = 0; e < N; ++e) b[e] = a.bias ? __ldg(a.bias + s.c + e) : 0.f;
        pairs<N>(b, bias);
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
        db[e] = 0;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0;
    }
    const T *x = static_cast<const T *>(a.x) + s.row * a.sx.b + s.c;
    const T *dy = static_cast<const T *>(a.dy) + s.row * a.sy.b + s.c;
    T *dx = static_cast<T *>(a.dx) + (size_t)s.row * a.T * a.C + s.c;
    const int stop = min(s.t1 + W - 1, a.T);
    Raw nx[U], nd[U];
    auto fetch = [&](int t) {
        const T *p = x + t * a.sx.t, *d = dy + t * a.sy.t;
        if (t + U <= stop) {
#pragma unroll
            for (int u = 0; u < U; ++u, p += a.sx.t, d += a.sy.t) {
                nx[u] = __ldg(reinterpret_cast<const Raw *>(p));
                nd[u] = __ldg(reinterpret_cast<const Raw *>(d));
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u, p += a.sx.t, d += a.sy.t)
                if (t + u < stop) {
                    nx[u] = __ldg(reinterpret_cast<const Raw *>(p));
                    nd[u] = __ldg(reinterpret_cast<const Raw *>(d));
                }
        }
    };
    fetch(s.t0);
    pass_windows<T, N>(a, s, W - 1, a.dwin_out, a.dwin);
    Run r = mx::run_at(a.cu, a.n_seq, a.T, s.row, s.t0);
    auto enter = [&](int t) {
        float p[W - 1][N];
        load_past<T, N, W>(a, x, r, t, s.c, p);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            pairs<N>(p[k], past[k]);
#pragma unroll
            for (int e = 0; e < P; ++e) open[k][e] = 0;
        }
    };
    enter(s.t0);
    // dx of token t of run r, or of its window's row
    auto put = [&](int t, const F2 (&g)[P]) {
        if (t >= r.start) {
            if (t >= s.t0 && t < s.t1) __stcs(reinterpret_cast<Raw *>(dx + (size_t)t * a.C), pack2<T, N>(g));
        } else if (a.dwin && r.start >= s.t0 && r.start < s.t1) {
            *reinterpret_cast<Raw *>(static_cast<T *>(a.dwin) + ((size_t)r.s * (W - 1) + (W - 1 + t - r.start)) * a.C + s.c) = pack2<T, N>(g);
        }
    };
    // what the run's last W-1 inputs get, where it ends before token t
    auto close = [&](int t) {
        if (r.s < 0) return;
#pragma unroll
        for (int k = 1; k < W; ++k) {
            if (a.dwin_out) {
                F2 g[P];
                unpack2<T, N>(*reinterpret_cast<const Raw *>(static_cast<const T *>(a.dwin_out) +
                                                             ((size_t)r.s * (W - 1) + (W - 1 - k)) * a.C + s.c), g);
#pragma unroll
                for (int e = 0; e < P; ++e) open[k - 1][e] = mx::add2(open[k - 1][e], g[e]);
            }
            put(t - k, open[k - 1]);
        }
    };
    // one token: `last` is what dx of the token W-1 before has got in all; `own`: dw and db count it
    auto token = [&](const Raw &in, const Raw &grad, bool own, F2 (&last)[P]) {
        F2 v[P], g[P];
        unpack2<T, N>(in, v);
        unpack2<T, N>(grad, g);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            if (act) {
                F2 z = mx::fma2(w[W - 1][e], v[e], bias[e]);
#pragma unroll
                for (int k = 1; k < W; ++k) z = mx::fma2(w[W - 1 - k][e], past[k - 1][e], z);
                g[e] = mx::mul2(g[e], mx::silu_slope2(z, mx::sigmoid2(z)));
            }
            if (own) {
                db[e] = mx::add2(db[e], g[e]);
                dw[W - 1][e] = mx::fma2(g[e], v[e], dw[W - 1][e]);
#pragma unroll
                for (int k = 1; k < W; ++k) dw[W - 1 - k][e] = mx::fma2(g[e], past[k - 1][e], dw[W - 1 - k][e]);
            }
            last[e] = mx::fma2(w[0][e], g[e], open[W - 2][e]);
#pragma unroll
            for (int k = W - 1; k > 1; --k) open[k - 1][e] = mx::fma2(w[W - k][e], g[e], open[k - 2][e]);
            open[0][e] = mx::mul2(w[W - 1][e], g[e]);
#pragma unroll
            for (int k = W - 1; k > 1; --k) past[k - 1][e] = past[k - 2][e];
            past[0][e] = v[e];
        }
    };
    bool done = false;
    for (int t = s.t0; t < stop && !done; t += U) {
        Raw cx[U], cd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) cx[u] = nx[u], cd[u] = nd[u];
        fetch(t + U);
        if (r.s >= 0 && t - (W - 1) >= max(r.start, s.t0) && t + U <= min(r.end, s.t1) && t < r.end) {
            T *to = dx + (size_t)(t - (W - 1)) * a.C;
#pragma unroll
            for (int u = 0; u < U; ++u, to += a.C) {
                F2 last[P];
                token(cx[u], cd[u], true, last);
                __stcs(reinterpret_cast<Raw *>(to), pack2<T, N>(last));
            }
            continue;
        }
#pragma unroll 1
        for (int i = t; i < t + U; ++i) {
            if (i >= stop) break;
            const Raw vx = cx[0], vd = cd[0];
#pragma unroll
            for (int u = 0; u + 1 < U; ++u) cx[u] = cx[u + 1], cd[u] = cd[u + 1];
            if (i == r.end) {
                close(i);
                if (i >= s.t1) {
                    done = true;
                    break;
                }
                r = mx::run_at(a.cu, a.n_seq, a.T, s.row, i);
                enter(i);
            }
            if (r.s < 0) {
                if (i < s.t1) __stcs(reinterpret_cast<Raw *>(dx + (size_t)i * a.C), Raw{});
                continue;
            }
            F2 last[P];
            token(vx, vd, i < s.t1, last);
            put(i - (W - 1), last);
        }
    }
    if (!done && stop == a.T) close(a.T);
    float *to = part + (size_t)s.index * (W + 1) * a.C + s.c;
#pragma unroll
    for (int j = 0; j < W; ++j) *reinterpret_cast<typename Vec<float, N>::Raw *>(to + (size_t)j * a.C) = pack2<float, N>(dw[j]);
    *reinterpret_cast<typename Vec<float, N>::Raw *>(to + (size_t)W * a.C) = pack2<float, N>(db);
}

// dw [C,W] and db [C] from the strips' shares [n][W+1][C].
template <int STRANDS>
__global__ void __launch_bounds__(32 * STRANDS) conv_sum_kernel(const float *part, float *dw, float *db, int n, int C, int W) {
    const long long all = (long long)(W + 1) * C, i = (long long)blockIdx.x * 32 + (threadIdx.x & 31);
    mx::follow_on();
    const float x = mx::column_sum<STRANDS>(part, n, all, i);
    if (threadIdx.x >= 32 || i >= all) return;
    const int j = (int)(i / C), c = (int)(i - (long long)j * C);
    if (j < W) dw[(size_t)c * W + j] = x;
    else if (db) db[c] = x;
}

// One token a row: the window's rows are read, shifted and written.  R rows a
// thread, whose taps are read once: with one, the taps were half of what the call
// read.  Measured: 256 rows of 8192 bf16 channels 10.2 us (33 MB), 14.3 with one.
template <typename T, int N, int W, int R>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStepArgs a) {
    using Raw = typename Vec<T, N>::Raw;
    constexpr int P = N / 2;
    const int nv = a.C / N, groups = (a.B + R - 1) / R;
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b0 = (int)(i / nv);  // rows b0, b0 + groups, ..
    if (b0 >= groups) return;
    const int c = (int)(i - (long long)b0 * nv) * N;
    Raw x[R], past[R][W - 1];
    int slot[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int b = b0 + q * groups;
        slot[q] = b >= a.B ? -1 : a.slots ? __ldg(a.slots + b) : b;
        if (slot[q] >= a.n_slots) slot[q] = -1;
    }
#pragma unroll
    for (int q = 0; q < R; ++q)
        if (slot[q] >= 0) {
            const T *page = static_cast<const T *>(a.win) + (size_t)slot[q] * (W - 1) * a.C + c;
            x[q] = __ldg(reinterpret_cast<const Raw *>(static_cast<const T *>(a.x) + (b0 + q * groups) * a.sx + c));
#pragma unroll
            for (int k = 0; k < W - 1; ++k) past[q][k] = __ldcs(reinterpret_cast<const Raw *>(page + (size_t)k * a.C));
        }
    float taps[W][N], bs[N];
    F2 w[W][P], bias[P];
    load_taps<N, W>(a.w, c, taps);
#pragma unroll
    for (int j = 0; j < W; ++j) pairs<N>(taps[j], w[j]);
#pragma unroll
    for (int e = 0; e < N; ++e) bs[e] = a.bias ? __ldg(a.bias + c + e) : 0.f;
    pairs<N>(bs, bias);
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int b = b0 + q * groups;
        if (b >= a.B) break;
        Raw out{};
        if (slot[q] >= 0) {
            F2 v[P], z[P];
            unpack2<T, N>(x[q], v);
#pragma unroll
            for (int e = 0; e < P; ++e) z[e] = mx::fma2(w[W - 1][e], v[e], bias[e]);
#pragma unroll
            for (int k = W - 2; k >= 0; --k) {
                unpack2<T, N>(past[q][k], v);
#pragma unroll
                for (int e = 0; e < P; ++e) z[e] = mx::fma2(w[k][e], v[e], z[e]);
            }
            if (a.flags & GDN_SILU)
#pragma unroll
                for (int e = 0; e < P; ++e) z[e] = mx::mul2(z[e], mx::sigmoid2(z[e]));
            out = pack2<T, N>(z);
            T *page = static_cast<T *>(a.win_out) + (size_t)slot[q] * (W - 1) * a.C + c;
#pragma unroll
            for (int k = 1; k < W - 1; ++k) __stcs(reinterpret_cast<Raw *>(page + (size_t)(k - 1) * a.C), past[q][k]);
            __stcs(reinterpret_cast<Raw *>(page + (size_t)(W - 2) * a.C), x[q]);
        }
        __stcs(reinterpret_cast<Raw *>(static_cast<T *>(a.y) + (size_t)b * a.C + c), out);  // 0 for an idle row
    }
}

// Strips of a row: as many as fill `threads`, of at least 8 tokens.
struct Cut {
    int len, per_row;
};
Cut cut_rows(int B, int T, int nv, long long threads, int most) {
    long long strips = threads / nv;
    if (strips > most) strips = most;
    long long per_row = strips / B;
    if (per_row < 1) per_row = 1;
    long long len = (T + per_row - 1) / per_row;
    if (len < 8) len = 8;
    return {(int)len, (int)((T + len - 1) / len)};
}

template <typename T, int N, int W>
int fwd(const ConvArgs &a, cudaStream_t stream) {
    const int nv = a.C / N;
    const Cut c = cut_rows(a.B, a.T, nv, (long long)mx::resident_ctas<conv_kernel<T, N, W>, kThreads>() * kThreads, 1 << 20);
    const long long threads = (long long)nv * c.per_row * a.B;
    conv_kernel<T, N, W><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a, c.len, c.per_row);
    return mx::launched();
}

// The shares of dw that a backward makes: at most this many strips, or a strip a row.
constexpr int kMostStrips = 2048;
constexpr long long kBwdThreads = 152 * 3 * kThreads;  // resident at once
Cut bwd_cut(int B, int T, int C) { return cut_rows(B, T, C / 4, kBwdThreads, kMostStrips); }

template <typename T, int W>
int bwd(const ConvArgs &a, cudaStream_t stream) {
    constexpr int N = 4;
    const Cut c = bwd_cut(a.B, a.T, a.C);
    const long long threads = (long long)(a.C / N) * c.per_row * a.B;
    float *part = static_cast<float *>(a.ws);
    conv_bwd_kernel<T, N, W><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a, c.len, c.per_row, part);
    const int st = mx::launched();
    if (st != GDN_OK) return st;
    const unsigned ctas = (unsigned)(((long long)(W + 1) * a.C + 31) / 32);
    const int n = c.per_row * a.B;
    if (n <= 256) mx::follow(conv_sum_kernel<8>, ctas, 256, 0, stream, part, a.dw, a.db, n, a.C, W);
    else mx::follow(conv_sum_kernel<32>, ctas, 1024, 0, stream, part, a.dw, a.db, n, a.C, W);
    return mx::launched();
}

template <typename T, int N, int W>
int step(const ConvStepArgs &a, cudaStream_t stream) {
    const long long vectors = (long long)(a.C / N) * a.B;
    // four rows a thread where that leaves each SM two CTAs
    if (vectors >= 4LL * 2 * kThreads * device_sm_count()) {
        const long long threads = (long long)(a.C / N) * ((a.B + 3) / 4);
        conv_step_kernel<T, N, W, 4><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    } else {
        conv_step_kernel<T, N, W, 1><<<(unsigned)((vectors + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
    }
    return mx::launched();
}

}  // namespace

int launch_conv_fwd(const ConvArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.W == 2 ? fwd<B16, 8, 2>(a, stream) : a.W == 3 ? fwd<B16, 8, 3>(a, stream) : fwd<B16, 8, 4>(a, stream);
    return a.W == 2 ? fwd<float, 4, 2>(a, stream) : a.W == 3 ? fwd<float, 4, 3>(a, stream) : fwd<float, 4, 4>(a, stream);
}

size_t conv_bwd_workspace(int B, int T, int C, int W) {
    const Cut c = bwd_cut(B, T, C);
    return sizeof(float) * (size_t)c.per_row * B * (W + 1) * C;
}

int launch_conv_bwd(const ConvArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.W == 2 ? bwd<B16, 2>(a, stream) : a.W == 3 ? bwd<B16, 3>(a, stream) : bwd<B16, 4>(a, stream);
    return a.W == 2 ? bwd<float, 2>(a, stream) : a.W == 3 ? bwd<float, 3>(a, stream) : bwd<float, 4>(a, stream);
}

int launch_conv_step(const ConvStepArgs &a, cudaStream_t stream) {
    using B16 = __nv_bfloat16;
    if (a.dtype == GDN_BF16) return a.W == 2 ? step<B16, 8, 2>(a, stream) : a.W == 3 ? step<B16, 8, 3>(a, stream) : step<B16, 8, 4>(a, stream);
    return a.W == 2 ? step<float, 4, 2>(a, stream) : a.W == 3 ? step<float, 4, 3>(a, stream) : step<float, 4, 4>(a, stream);
}

}  // namespace gdn
