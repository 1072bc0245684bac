// block_norm.cu -- the norm after a block, its scale, the residual's sum and the
// norm before the next block; and their backward.
//
//   h = res + s n(x) w1,   y = n(h) w2,   n(u) = u / sqrt(mean u^2 + eps) over C columns
//
// s: a factor for each column, of every row or of each of `groups` runs of rows.
// backward, at the h that the forward stored, with r1, r2 the norms' factors:
//   dres = dh + r2 (w2 dy - h r2^2 mean(h w2 dy))
//   dx = r1 (m dres - x r1^2 mean(x m dres)),  m = s w1
//   dw2 = sum dy h r2,  dw1 = sum s dres x r1,  ds = w1 sum over the group dres x r1
//
// One pass: NT threads hold a row in registers over both norms; the bytes bound it
// (4 rows forwards, 6 backwards).  The next row's loads are on their way
// meanwhile, the weights stay in registers.  Sums are in fp32; h enters its norm
// before it is rounded for the store.  Measured, bf16, 16384 x 2048: forwards 42 us
// (268 MB at 6.4 TB/s, calls back to back in a graph), backwards 63 (403 MB at 6.4) and the columns' sums 8.
#include "mixer.cuh"

namespace gdn {
namespace {

// Sums over the CTA; `s` alternates from one call to the next.
template <int NT, int K>
__device__ __forceinline__ void cta_sum(float (&x)[K], float (*s)[32]) {
#pragma unroll
    for (int m = 16; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(~0u, x[k], m);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) s[k][threadIdx.x >> 5] = x[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = 0.f;
#pragma unroll
            for (int i = 0; i < NT / 32; ++i) x[k] += s[k][i];
        }
    }
}

// A thread's columns of a vector of weights, 1 where there is none.
template <int N>
__device__ __forceinline__ void load_weights(const float *w, int i, bool there, float (&x)[N]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        float4 y = make_float4(1.f, 1.f, 1.f, 1.f);
        if (w && there) y = __ldg(reinterpret_cast<const float4 *>(w + i + e));
        x[e] = y.x, x[e + 1] = y.y, x[e + 2] = y.z, x[e + 3] = y.w;
    }
}

// The group whose rows a CTA takes, and which: CTA p of `per` of a group takes its
// rows p, p + per, ..
struct Rows {
    int group;
    long long row, step, end;
};
__device__ __forceinline__ Rows rows_of(const BlockNormArgs &a, int per) {
    const int groups = a.groups ? a.groups : 1;
    const long long each = a.rows / groups;
    const int g = blockIdx.x / per, p = blockIdx.x - g * per;
    return {g, g * each + p, per, (g + 1) * each};
}

template <typename T, int NT, int V>
__global__ void __launch_bounds__(NT) block_kernel(BlockNormArgs a, int per) {
    constexpr int N = kWide<T>;
    using Raw = typename Vec<T, N>::Raw;
    __shared__ float red[2][1][32];
    const Rows k = rows_of(a, per);
    const int nv = a.C / N;
    Raw nx[V], nr[V];
    auto fetch = [&](long long row) {
        const Raw *x = reinterpret_cast<const Raw *>(static_cast<const T *>(a.x) + row * a.C);
        const Raw *r = reinterpret_cast<const Raw *>(static_cast<const T *>(a.res) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + threadIdx.x;
            nx[j] = nr[j] = Raw{};
            if (row < k.end && i < nv) nx[j] = __ldcs(x + i), nr[j] = __ldcs(r + i);
        }
    };
    fetch(k.row);
    float m[V][N], w2[V][N];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + threadIdx.x;
        float s[N];
        load_weights<N>(a.w1, i * N, i < nv, m[j]);
        load_weights<N>(a.w2, i * N, i < nv, w2[j]);
        load_weights<N>(a.s ? a.s + (size_t)k.group * a.C : nullptr, i * N, i < nv, s);
#pragma unroll
        for (int e = 0; e < N; ++e) m[j][e] *= s[e];
    }
    for (long long row = k.row; row < k.end; row += k.step) {
        float x[V][N], h[V][N], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Vec<T, N>::unpack(nx[j], x[j]);
            Vec<T, N>::unpack(nr[j], h[j]);
#pragma unroll
            for (int e = 0; e < N; ++e) ss[0] = fmaf(x[j][e], x[j][e], ss[0]);
        }
        fetch(row + k.step);
        cta_sum<NT, 1>(ss, red[0]);
        const float r1 = rsqrtf(ss[0] / a.C + a.eps);
        ss[0] = 0.f;
        Raw *ho = reinterpret_cast<Raw *>(static_cast<T *>(a.h) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const bool there = j * NT + threadIdx.x < nv;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                h[j][e] = fmaf(x[j][e] * r1, m[j][e], h[j][e]);
                ss[0] = fmaf(h[j][e], h[j][e], ss[0]);
            }
            if (there) __stcs(ho + j * NT + threadIdx.x, Vec<T, N>::pack(h[j]));
        }
        cta_sum<NT, 1>(ss, red[1]);
        const float r2 = rsqrtf(ss[0] / a.C + a.eps);
        Raw *y = reinterpret_cast<Raw *>(static_cast<T *>(a.y) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int e = 0; e < N; ++e) h[j][e] *= r2 * w2[j][e];
            if (j * NT + threadIdx.x < nv) __stcs(y + j * NT + threadIdx.x, Vec<T, N>::pack(h[j]));
        }
    }
}

// part: [CTA][2][C], the sums of dy h r2 and of dres x r1.
template <typename T, int NT, int V>
__global__ void __launch_bounds__(NT) block_bwd_kernel(BlockNormArgs a, int per, float *part) {
    mx::let_follow();
    constexpr int N = kWide<T>;
    using Raw = typename Vec<T, N>::Raw;
    __shared__ float red[2][3][32];
    const Rows k = rows_of(a, per);
    const int nv = a.C / N;
    Raw nx[V], nh[V], nd[V], ng[V];
    auto fetch = [&](long long row) {
        const size_t at = (size_t)row * a.C;
        const Raw *x = reinterpret_cast<const Raw *>(static_cast<const T *>(a.x) + at);
        const Raw *h = reinterpret_cast<const Raw *>(static_cast<const T *>(a.h) + at);
        const Raw *d = reinterpret_cast<const Raw *>(static_cast<const T *>(a.dy) + at);
        const Raw *g = reinterpret_cast<const Raw *>(static_cast<const T *>(a.dh) + at);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int i = j * NT + threadIdx.x;
            nx[j] = nh[j] = nd[j] = ng[j] = Raw{};
            if (row < k.end && i < nv) {
                nx[j] = __ldcs(x + i), nh[j] = __ldcs(h + i), nd[j] = __ldcs(d + i);
                if (a.dh) ng[j] = __ldcs(g + i);
            }
        }
    };
    fetch(k.row);
    float m[V][N], w2[V][N], sum1[V][N], sum2[V][N];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + threadIdx.x;
        float s[N];
        load_weights<N>(a.w1, i * N, i < nv, m[j]);
        load_weights<N>(a.w2, i * N, i < nv, w2[j]);
        load_weights<N>(a.s ? a.s + (size_t)k.group * a.C : nullptr, i * N, i < nv, s);
#pragma unroll
        for (int e = 0; e < N; ++e) m[j][e] *= s[e], sum1[j][e] = sum2[j][e] = 0.f;
    }
    for (long long row = k.row; row < k.end; row += k.step) {
        Raw px[V], ph[V], pd[V], pg[V];
#pragma unroll
        for (int j = 0; j < V; ++j) px[j] = nx[j], ph[j] = nh[j], pd[j] = nd[j], pg[j] = ng[j];
        fetch(row + k.step);
        float sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[N], h[N], d[N];
            Vec<T, N>::unpack(px[j], x);
            Vec<T, N>::unpack(ph[j], h);
            Vec<T, N>::unpack(pd[j], d);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                sums[0] = fmaf(x[e], x[e], sums[0]);
                sums[1] = fmaf(h[e], h[e], sums[1]);
                sums[2] = fmaf(h[e], d[e] * w2[j][e], sums[2]);
            }
        }
        cta_sum<NT, 3>(sums, red[0]);
        const float r1 = rsqrtf(sums[0] / a.C + a.eps), r2 = rsqrtf(sums[1] / a.C + a.eps), m2 = r2 * r2 * (sums[2] / a.C);
        float g[V][N], p[1] = {0.f};
        Raw *dres = reinterpret_cast<Raw *>(static_cast<T *>(a.dres) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[N], h[N], d[N];
            Vec<T, N>::unpack(px[j], x);
            Vec<T, N>::unpack(ph[j], h);
            Vec<T, N>::unpack(pd[j], d);
            Vec<T, N>::unpack(pg[j], g[j]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                g[j][e] = fmaf(r2, fmaf(d[e], w2[j][e], -h[e] * m2), g[j][e]);
                sum2[j][e] = fmaf(d[e], h[e] * r2, sum2[j][e]);
                sum1[j][e] = fmaf(g[j][e], x[e] * r1, sum1[j][e]);
                p[0] = fmaf(x[e], g[j][e] * m[j][e], p[0]);
            }
            if (j * NT + threadIdx.x < nv) __stcs(dres + j * NT + threadIdx.x, Vec<T, N>::pack(g[j]));
        }
        cta_sum<NT, 1>(p, red[1]);
        const float m1 = r1 * r1 * (p[0] / a.C);
        Raw *dx = reinterpret_cast<Raw *>(static_cast<T *>(a.dx) + row * a.C);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[N];
            Vec<T, N>::unpack(px[j], x);
#pragma unroll
            for (int e = 0; e < N; ++e) g[j][e] = r1 * fmaf(g[j][e], m[j][e], -x[e] * m1);
            if (j * NT + threadIdx.x < nv) __stcs(dx + j * NT + threadIdx.x, Vec<T, N>::pack(g[j]));
        }
    }
    float *to = part + (size_t)blockIdx.x * 2 * a.C;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int i = j * NT + threadIdx.x;
        if (i < nv)
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                *reinterpret_cast<float4 *>(to + i * N + e) = make_float4(sum2[j][e], sum2[j][e + 1], sum2[j][e + 2], sum2[j][e + 3]);
                *reinterpret_cast<float4 *>(to + a.C + i * N + e) = make_float4(sum1[j][e], sum1[j][e + 1], sum1[j][e + 2], sum1[j][e + 3]);
            }
    }
}

// The three gradients of columns, from the CTAs' sums, in order: 32 columns a CTA,
// 32 strands of shares or of groups.
__global__ void __launch_bounds__(1024) block_sum_kernel(BlockNormArgs a, const float *part, int groups, int per) {
    mx::follow_on();
    __shared__ float s[2][32][33];
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float dw1 = 0.f, dw2 = 0.f;
    auto take = [&](int g, float x, float y) {  // a group's sums
        dw2 += x;
        dw1 = fmaf(a.s ? a.s[(size_t)g * a.C + c] : 1.f, y, dw1);
        if (a.ds) a.ds[(size_t)g * a.C + c] = y * (a.w1 ? a.w1[c] : 1.f);
    };
    auto add = [&](int g, int first, int step, float &x, float &y) {
#pragma unroll 8
        for (int i = first; i < per; i += step) {
            const float *p = part + ((size_t)g * per + i) * 2 * a.C + c;
            x += p[0], y += p[a.C];
        }
    };
    if (groups < 32) {  // a group's CTAs by strands
        for (int g = 0; g < groups; ++g) {
            float x = 0.f, y = 0.f;
            if (c < a.C) add(g, strand, 32, x, y);
            s[0][strand][lane] = x, s[1][strand][lane] = y;
            __syncthreads();
            if (strand == 0 && c < a.C) {
                x = y = 0.f;
#pragma unroll
                for (int j = 0; j < 32; ++j) x += s[0][j][lane], y += s[1][j][lane];
                take(g, x, y);
            }
            __syncthreads();
        }
    } else {  // groups by strands
        if (c < a.C)
            for (int g = strand; g < groups; g += 32) {
                float x = 0.f, y = 0.f;
                add(g, 0, 1, x, y);
                take(g, x, y);
            }
        s[0][strand][lane] = dw1, s[1][strand][lane] = dw2;
        __syncthreads();
        if (strand == 0) {
            dw1 = dw2 = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) dw1 += s[0][j][lane], dw2 += s[1][j][lane];
        }
    }
    if (strand == 0 && c < a.C) {
        if (a.dw1) a.dw1[c] = dw1;
        if (a.dw2) a.dw2[c] = dw2;
    }
}

// CTAs of a group, where `most` are wanted in all.
int per_group(long long rows, int groups, int most) {
    const int g = groups ? groups : 1;
    const long long each = rows / g, per = most / g;
    return (int)(per < 1 ? 1 : per < each ? per : each);
}
// CTAs of a backward, whose workspace holds their sums: narrow rows have few threads
// a CTA (30230 x 88: 38 us with four CTAs an SM, 33 so).
int most_bwd(int C) { return 152 * (C <= 512 ? 12 : C <= 1024 ? 8 : 4); }

template <typename T, int NT, int V, bool BACK>
int go(const BlockNormArgs &a, cudaStream_t stream) {
    const int groups = a.groups ? a.groups : 1;
    if constexpr (!BACK) {
        const int per = per_group(a.rows, a.groups, mx::resident_ctas<block_kernel<T, NT, V>, NT>());
        block_kernel<T, NT, V><<<groups * per, NT, 0, stream>>>(a, per);
        return mx::launched();
    } else {
        const int fit = mx::resident_ctas<block_bwd_kernel<T, NT, V>, NT>();
        const int most = most_bwd(a.C), per = per_group(a.rows, a.groups, fit < most ? fit : most);
        float *part = static_cast<float *>(a.ws);
        block_bwd_kernel<T, NT, V><<<groups * per, NT, 0, stream>>>(a, per, part);
        const int st = mx::launched();
        if (st != GDN_OK) return st;
        mx::follow(block_sum_kernel, (a.C + 31) / 32, 1024, 0, stream, a, part, groups, per);
        return mx::launched();
    }
}

// Two vectors a thread as in the other norms, more from 512 vectors a row on.
template <typename T, bool BACK>
int launch(const BlockNormArgs &a, cudaStream_t stream) {
    const int nv = a.C / kWide<T>;
    if (nv <= 32) return go<T, 32, 1, BACK>(a, stream);
    if (nv <= 64) return go<T, 32, 2, BACK>(a, stream);
    if (nv <= 128) return go<T, 64, 2, BACK>(a, stream);
    if (nv <= 256) return go<T, 128, 2, BACK>(a, stream);
    if (nv <= 512) return go<T, 256, 2, BACK>(a, stream);
    if (sizeof(T) == 2 || nv <= 1024) return go<T, 512, 2, BACK>(a, stream);
    return go<T, 512, sizeof(T) == 2 ? 2 : 4, BACK>(a, stream);
}

}  // namespace

int launch_block_norm(const BlockNormArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16, false>(a, stream) : launch<float, false>(a, stream);
}
size_t block_norm_bwd_workspace(long long rows, int C, int groups) {
    return sizeof(float) * 2 * C * (size_t)(groups ? groups : 1) * per_group(rows, groups, most_bwd(C));
}
int launch_block_norm_bwd(const BlockNormArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch<__nv_bfloat16, true>(a, stream) : launch<float, true>(a, stream);
}

}  // namespace gdn
