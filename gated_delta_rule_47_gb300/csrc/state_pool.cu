// state_pool.cu -- pages of a pool of recurrent states, [layers][n_slots][page]:
// copies, forks (with the choice of free pages), frees and compaction.
//
// A page moves as it is; what bounds every call is its bytes, read once and
// written once.  The choice of pages is made on the device by one CTA (a scan
// over the live marks), so that no call waits for the host.
#include <stdint.h>

#include "gdn_internal.h"
#include "layer_ops.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                        // 16-byte words in flight per thread
constexpr int kPiece = kThreads * kUnroll;        // words of one piece
constexpr int kPlanThreads = 1024;

// Copies page src[i] to page dst[i] of every layer, i < *count (or n where
// count is null); src -1 writes zeros.  Entries out of range are skipped.
// A CTA takes pieces of 16 KB in turn, four 16-byte words a thread in flight.
// Bound by the bytes: 190 of 400 slots closed up in 6 layers of 1 MB pages, 1.25
// GB, 190 to 206 us, 6.1 to 6.6 TB/s; one page copied 2.1 us.
__global__ void __launch_bounds__(kThreads) move_kernel(PoolArgs p, const int *src, const int *dst, int n,
                                                        const int *count) {
    if (count) n = min(n, *count);
    const long long words = p.page_bytes / 16;
    const long long pieces = (words + kPiece - 1) / kPiece;
    const long long total = pieces * p.layers * n;
    uint4 *pool = static_cast<uint4 *>(p.pool);
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int i = (int)(w / (pieces * p.layers));
        const long long rest = w - (long long)i * pieces * p.layers;
        const int layer = (int)(rest / pieces);
        const long long at = (rest - layer * pieces) * kPiece + threadIdx.x;
        const int s = src[i], d = dst[i];
        if (d < 0 || d >= p.n_slots || s < -1 || s >= p.n_slots || s == d) continue;
        uint4 *to = pool + ((long long)layer * p.n_slots + d) * words;
        const uint4 *from = pool + ((long long)layer * p.n_slots + (s < 0 ? d : s)) * words;
        uint4 x[kUnroll];
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            x[j] = make_uint4(0, 0, 0, 0);
            if (s >= 0 && at + j * kThreads < words) x[j] = __ldcs(from + at + j * kThreads);
        }
#pragma unroll
        for (int j = 0; j < kUnroll; ++j)
            if (at + j * kThreads < words) __stcs(to + at + j * kThreads, x[j]);
    }
}

// Exclusive prefix of x over the CTA's threads; *total gets the sum.
__device__ int block_scan(int x, int *total) {
    __shared__ int sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int t = __shfl_up_sync(~0u, y, m);
        if (lane >= m) y += t;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    if (warp == 0) {
        int z = sums[lane];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int t = __shfl_up_sync(~0u, z, m);
            if (lane >= m) z += t;
        }
        sums[lane] = z;
    }
    __syncthreads();
    *total = sums[31];
    return y - x + (warp ? sums[warp - 1] : 0);
}

// The i-th valid parent gets the i-th free page, lowest first; where none is
// left, and for an invalid parent, the child is -1.  2.8 us for 64 slots: one
// CTA's barriers and scans, as in compact_plan_kernel (3.1 us for 400).
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(unsigned char *live, int n_slots, const int *parents,
                                                                 int *children, int n, int *src, int *dst,
                                                                 int *free_slots) {
    int n_free = 0, total;
    for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        const int is = s < n_slots && live[s] == 0;
        const int at = block_scan(is, &total);
        if (is) free_slots[n_free + at] = s;
        n_free += total;
    }
    __syncthreads();
    int used = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int parent = i < n ? parents[i] : -2;
        const int ok = parent == -1 || (parent >= 0 && parent < n_slots && live[parent] != 0);
        const int at = used + block_scan(ok, &total);
        used += total;
        if (i < n) {
            const int child = ok && at < n_free ? free_slots[at] : -1;
            children[i] = child;
            src[i] = parent;
            dst[i] = child;
        }
    }
    __syncthreads();  // every parent has been looked at before a child is marked
    for (int i = threadIdx.x; i < n; i += kPlanThreads)
        if (dst[i] >= 0) live[dst[i]] = 1;
}

// The live pages past the first n_live move, in order, into the free ones
// before them.  remap[s]: page s's new place, -1 where it is not live.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(unsigned char *live, int n_slots, int *remap,
                                                                    int *n_live_out, int *src, int *dst, int *moves) {
    int n_live = 0, total;
    for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        block_scan(s < n_slots && live[s] != 0, &total);
        n_live += total;
    }
    int holes = 0, movers = 0;
    for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        const int alive = s < n_slots && live[s] != 0;
        const int hole = s < n_live && !alive, mover = s >= n_live && alive;
        const int ah = holes + block_scan(hole, &total);
        holes += total;
        const int am = movers + block_scan(mover, &total);
        movers += total;
        if (hole) dst[ah] = s;
        if (mover) src[am] = s;
        if (s < n_slots) remap[s] = alive && s < n_live ? s : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += kPlanThreads) remap[src[i]] = dst[i];
    for (int s = threadIdx.x; s < n_slots; s += kPlanThreads) live[s] = s < n_live;
    if (threadIdx.x == 0) {
        *n_live_out = n_live;
        *moves = movers;
    }
}

__global__ void free_kernel(unsigned char *live, int n_slots, const int *slots, int n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n && slots[i] >= 0 && slots[i] < n_slots) live[slots[i]] = 0;
}

int launch_moves(const PoolArgs &p, const int *src, const int *dst, int most, const int *count, cudaStream_t stream) {
    const long long pieces = (p.page_bytes / 16 + kPiece - 1) / kPiece * p.layers * most;
    if (pieces == 0) return GDN_OK;  // a pool without bytes: its marks alone
    const long long full = 8LL * device_sm_count();  // 2,048 threads an SM
    move_kernel<<<(unsigned)(pieces < full ? pieces : full), kThreads, 0, stream>>>(p, src, dst, most, count);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

}  // namespace

int launch_pool_copy(const PoolArgs &p, const int *src, const int *dst, int n, cudaStream_t stream) {
    return launch_moves(p, src, dst, n, nullptr, stream);
}

size_t pool_fork_workspace(int n_slots, int n) { return 4 * ((size_t)n_slots + 2 * (size_t)n); }

int launch_pool_fork(const PoolArgs &p, unsigned char *live, const int *parents, int *children, int n, void *ws,
                     cudaStream_t stream) {
    int *src = static_cast<int *>(ws), *dst = src + n, *free_slots = dst + n;
    fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(live, p.n_slots, parents, children, n, src, dst, free_slots);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return launch_moves(p, src, dst, n, nullptr, stream);
}

int launch_pool_free(unsigned char *live, int n_slots, const int *slots, int n, cudaStream_t stream) {
    free_kernel<<<(n + 255) / 256, 256, 0, stream>>>(live, n_slots, slots, n);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    return GDN_OK;
}

size_t pool_compact_workspace(int n_slots) { return 4 * (2 * (size_t)n_slots + 1); }

int launch_pool_compact(const PoolArgs &p, unsigned char *live, int *remap, int *n_live, void *ws,
                        cudaStream_t stream) {
    int *src = static_cast<int *>(ws), *dst = src + p.n_slots, *moves = dst + p.n_slots;
    compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(live, p.n_slots, remap, n_live, src, dst, moves);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    note_launch();
    // at most half of the pages can be past the live ones' count and live
    const int most = p.n_slots / 2;
    return most ? launch_moves(p, src, dst, most, moves, stream) : GDN_OK;
}

}  // namespace gdn
