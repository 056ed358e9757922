// rmm_keep.cu -- the accepted nodes of a draft tree kept in the caches: for each
// sequence, cache slot len + path[i] moves to slot len + i (i < count), in every
// cache given, and the lengths grow by the counts.  The path is ascending, so
// path[i] >= i: what a sequence keeps only moves forward, inside the tree's own
// T <= 64 slots.
//
// One CTA per (KV head, sequence, cache) reads every moved element into
// registers before it writes the first, so the move is in place whatever the
// overlap; elements already in place are not touched.  Latency bound: a head's
// window is 128 rows of at most 128 bytes of K^T and 64 rows of 256 bytes of V.
#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;
constexpr int kKeepThreads = 256;

__global__ void __launch_bounds__(kKeepThreads)
    cache_keep_kernel(const __grid_constant__ CacheList caches, int Hkv, int ldL, const int32_t* lens,
                      const int32_t* path, const int32_t* count, int T, int32_t* lens_out) {
    __shared__ int from[kTreeMax];
    const int g = blockIdx.x, b = blockIdx.y, layer = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int len = lens[b], n = count[b];
    bool ok = n >= 1 && n <= T && len >= 0 && len <= ldL - T;
    if (tid < T) {
        const int p = path[(size_t)b * T + tid];
        from[tid] = p;
        // ascending and inside the tree, as far as the count goes
        if (ok && tid < n) ok = p >= 0 && p < T && (tid == 0 || p > path[(size_t)b * T + tid - 1]);
    }
    ok = __syncthreads_and(ok);
    if (lens_out && g == 0 && layer == 0 && tid == 0) lens_out[b] = ok ? len + n : len;
    if (!ok) return;  // an empty slot of the batch, or no path: the caches stay as they are

    uint16_t* Kt = caches.Kt[layer] + ((size_t)b * Hkv + g) * D * (size_t)ldL + len;
    uint16_t* V = caches.V[layer] + (((size_t)b * Hkv + g) * (size_t)ldL + len) * D;
    // V: 16 pieces of 16 bytes per row, up to 1024 of them over 256 threads
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = (tid >> 4) + 16 * j;
        if (i < n && from[i] != i) v[j] = *reinterpret_cast<const uint4*>(V + (size_t)from[i] * D + (tid & 15) * 8);
    }
    // K^T: 16 dim rows per warp, lane i holds kept nodes i and i + 32
    uint16_t k[16][2];
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = lane + 32 * j;
            if (i < n && from[i] != i) k[r][j] = Kt[(size_t)(warp * 16 + r) * ldL + from[i]];
        }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = (tid >> 4) + 16 * j;
        if (i < n && from[i] != i) *reinterpret_cast<uint4*>(V + (size_t)i * D + (tid & 15) * 8) = v[j];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = lane + 32 * j;
            if (i < n && from[i] != i) Kt[(size_t)(warp * 16 + r) * ldL + i] = k[r][j];
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
                               ldL, lens, path, count, T, in_place ? (int32_t*)nullptr : lens_out);
    if (e != cudaSuccess || !in_place) return e;
    return launch_pdl(grow_lens_kernel, dim3((B + 127) / 128), dim3(128), 0, stream, B, T, ldL, lens_out, path, count);
}

}  // namespace rmm
