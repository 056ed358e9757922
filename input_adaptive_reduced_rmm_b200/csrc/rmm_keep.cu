// rmm_keep.cu -- the accepted nodes of a draft tree kept in the caches: for each
// sequence, cache slot len + path[i] moves to slot len + i (i < count), in every
// cache given, and the lengths grow by the counts.  The path is ascending, so
// path[i] >= i: what a sequence keeps only moves forward, inside the tree's own
// T <= 64 slots.
//
// Eight warps per (KV head, sequence, cache), each with 16 dim rows of K^T and a
// 32-byte column of V of its own.  A warp reads what moves within a row or a column
// into registers before it writes any of it, so the move is in place whatever the
// overlap, and no warp waits for another; elements already in place are not
// touched.  Bound by DRAM sectors, since 2-byte elements of K^T move in 32-byte
// sectors: 16 caches of 16 sequences and 8 heads, 64-node trees, take 16.7 us alone and
// 22 in a row of calls on changing caches (with one CTA-wide read before one CTA-wide
// write 33 where this took 15.5).
#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;
constexpr int kKeepThreads = 256;

// K^T rows row0 .. row0 + kRows - 1 of a warp: lane i moves nodes i and, with kWide, i + 32.
template <int kRows, bool kWide>
__device__ __forceinline__ void move_keys(uint16_t* Kt, int64_t ldL, int lane, int p0, int p1, bool m0, bool m1) {
    uint16_t a[kRows], b[kWide ? kRows : 1];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (m0) a[r] = Kt[r * ldL + p0];
        if (kWide && m1) b[r] = Kt[r * ldL + p1];
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (m0) Kt[r * ldL + lane] = a[r];
        if (kWide && m1) Kt[r * ldL + lane + 32] = b[r];
    }
}

__global__ void __launch_bounds__(kKeepThreads)
    cache_keep_kernel(const __grid_constant__ CacheList caches, int Hkv, int64_t ldL, const int32_t* lens,
                      const int32_t* path, const int32_t* count, int T, int32_t* lens_out) {
    const int g = blockIdx.x, b = blockIdx.y, layer = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int len = lens[b], n = count[b];
    const int p0 = lane < T ? path[(size_t)b * T + lane] : -1;
    const int p1 = lane + 32 < T ? path[(size_t)b * T + lane + 32] : -1;
    // ascending and inside the tree, as far as the count goes
    int before0 = __shfl_up_sync(0xffffffffu, p0, 1), before1 = __shfl_up_sync(0xffffffffu, p1, 1);
    const int mid = __shfl_sync(0xffffffffu, p0, 31);
    if (lane == 0) before0 = -1, before1 = mid;
    bool ok = n >= 1 && n <= T && len >= 0 && len <= ldL - T;
    if (ok && lane < n) ok = p0 > before0 && p0 >= 0 && p0 < T;
    if (ok && lane + 32 < n) ok = p1 > before1 && p1 < T;
    ok = __all_sync(0xffffffffu, ok);
    if (lens_out && g == 0 && layer == 0 && threadIdx.x == 0) lens_out[b] = ok ? len + n : len;
    if (!ok) return;  // an empty slot of the batch, or no path: the caches stay as they are
    const bool m0 = lane < n && p0 != lane, m1 = lane + 32 < n && p1 != lane + 32;
    if (!__any_sync(0xffffffffu, m0 || m1)) return;  // the path is in place

    const size_t head = ((size_t)b * Hkv + g) * D * (size_t)ldL;
    uint16_t* Kt = caches.Kt[layer] + head + (int64_t)(warp * 16) * ldL + len;
    uint16_t* V = caches.V[layer] + head + (size_t)len * D + warp * 16 + (lane & 1) * 8;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = (lane >> 1) + 16 * j;
        const int p = __shfl_sync(0xffffffffu, j < 2 ? p0 : p1, i & 31);
        if (i < n && p != i) v[j] = *reinterpret_cast<const uint4*>(V + (size_t)p * D);
    }
    if (n <= 32) {
        move_keys<16, false>(Kt, ldL, lane, p0, p1, m0, m1);
    } else {
        move_keys<8, true>(Kt, ldL, lane, p0, p1, m0, m1);
        move_keys<8, true>(Kt + 8 * ldL, ldL, lane, p0, p1, m0, m1);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = (lane >> 1) + 16 * j;
        const int p = __shfl_sync(0xffffffffu, j < 2 ? p0 : p1, i & 31);
        if (i < n && p != i) *reinterpret_cast<uint4*>(V + (size_t)i * D) = v[j];
    }
}

// The lengths alone, after the move, when they are updated in place: the CTAs of
// the move all read the old ones.
__global__ void grow_lens_kernel(int B, int T, int ldL, int32_t* lens, const int32_t* path,
                                 const int32_t* count) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b >= B) return;
    const int len = lens[b], n = count[b];
    bool ok = n >= 1 && n <= T && len >= 0 && len <= ldL - T;
    for (int i = 0; ok && i < n; ++i) {
        const int p = path[(size_t)b * T + i];
        ok = p >= 0 && p < T && (i == 0 || p > path[(size_t)b * T + i - 1]);
    }
    if (ok) lens[b] = len + n;
}

}  // namespace

cudaError_t launch_cache_keep(const CacheList& caches, int ncaches, int B, int Hkv, int ldL, const int32_t* lens,
                              const int32_t* path, const int32_t* count, int T, int32_t* lens_out,
                              cudaStream_t stream) {
    if (B > 65535 || ncaches > kMaxCaches) return cudaErrorInvalidValue;
    const bool in_place = lens_out == lens;
    cudaError_t e = launch_pdl(cache_keep_kernel, dim3(Hkv, B, ncaches), dim3(kKeepThreads), 0, stream, caches, Hkv,
                               (int64_t)ldL, lens, path, count, T, in_place ? (int32_t*)nullptr : lens_out);
    if (e != cudaSuccess || !in_place) return e;
    return launch_pdl(grow_lens_kernel, dim3((B + 127) / 128), dim3(128), 0, stream, B, T, ldL, lens_out, path, count);
}

}  // namespace rmm
