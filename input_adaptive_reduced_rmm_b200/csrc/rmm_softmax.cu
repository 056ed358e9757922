// rmm_softmax.cu -- rows of logits as probabilities at a temperature:
//   y_i = e^((x_i - M) / t) / sum_j e^((x_j - M) / t),   M = max_j x_j
// bf16 in, fp32 out; at temperature 0 the limit, 1 at the lowest index of M.
//
// Memory bound by its data, 2 bytes read and 4 written per element; two kernels
// form the maximum and the sum relative to it with one exchange between the CTAs of
// a row, as pairs that merge exactly like a running maximum and sum.
//   softmax_kernel       a row in the registers of a cluster of 1, 2, 4 or 8 CTAs,
//                        read once: the shortest way for one row, but every CTA of
//                        the SM loads, exchanges and stores at the same time
//   softmax_rows_kernel  a row in parts over 4 or 8 small CTAs of 128 threads, each part
//                        copied to shared memory at once and read there twice: six CTAs
//                        per SM in different phases
// Measured, us for (rows, V), registers against parts:
//   (8, 16384) 3.2 3.3    (8, 131072) 6.2 6.3     (16, 16384) 3.3 3.3
//   (16, 32000) 5.2 4.2   (16, 131072) 8.8 8.0    (64, 8192) 3.9 4.2
//   (64, 32000) 12.5 6.0  (512, 16384) 25.9 16.0  (512, 131072) 126 75
// and for rows that start at any element (registers one element at a time)
//   (1, 2051) 2.2 2.4     (1, 4099) 4.5 2.7       (512, 2051) 7.3 9.5
//   (1, 50257) 8.1 4.6    (512, 8195) 40 12       (512, 131069) 444 73
// so parts are taken from 16 rows of 16384 logits on where rows start on 16-byte
// boundaries, and above 4096 logits where they do not but logits and outputs start
// alike, the up to 7 elements at either end one by one.  Temperature 0, and logits and
// outputs that start unlike, keep to the registers with one store per element, which
// long rows feel: (512, 131072) at temperature 0 402 us, (512, 131069) out of 131072
// columns 395, (1, 32000) at temperature 0 5.4.
// (512, 131072) moves its 403 MB at 5.2 TB/s; the two exponentials per
// element take 35 us beside that.  Slower at 512 x 131072 were a second read from L2
// instead of shared memory (80), two 16-byte stores instead of one of 32 (99) and a
// wave of resident clusters over many rows (169).
#include <math.h>

#include "rmm_common.cuh"
#include "rmm_internal.h"

namespace rmm {

namespace {

constexpr int kThreads = 512;
// softmax_rows_kernel: when it is taken, its threads, CTAs per SM and vectors of a thread
// at a time, and the length from which a row has 8 parts instead of 4 (us, 4 against 8 parts:
// 23.6 and 28.1 at 512 x 32000, 80.8 and 75.5 at 512 x 131072; 256 threads 28.5 and 79.8).
constexpr int kManyRows = 16, kLongRow = 16384, kRaggedRow = 4097;
constexpr int kRowThreads = 128, kRowCtas = 6, kRowFly = 4;
constexpr int kEightParts = 65536;
constexpr float kLog2e = 1.4426950408889634f;

// The cluster's barrier wants whole warps: lanes that a condition has parted meet first.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    cluster_sync();
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// 2^x, -inf gives 0 (about 2 ulp)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// what the logits are taken relative to; nothing but -inf (or NaN) has no maximum
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.0f : m; }

// Merge (m, s): the maximum of two parts, the sum relative to it.  Parts of nothing
// but -inf have m = -inf and s = 0; NaN, which no maximum shows, and +inf, which is no
// reference, make s NaN.
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, float c) {
    const float mm = fmaxf(m, m2);
    const float a = m == mm ? s : s * ex2((m - mm) * c);
    const float b = m2 == mm ? s2 : s2 * ex2((m2 - mm) * c);
    m = mm;
    s = a + b;
}

// Eight outputs as one 32-byte store: two of 16 bytes leave every sector half written twice, which
// cost a quarter of the time (512 x 131072: 99 us, 80 with whole sectors).
__device__ __forceinline__ void store8(float* d, const float (&p)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "f"(p[0]), "f"(p[1]),
                     "f"(p[2]), "f"(p[3]), "f"(p[4]), "f"(p[5]), "f"(p[6]), "f"(p[7])
                     : "memory");
    } else {
        reinterpret_cast<float4*>(d)[0] = make_float4(p[0], p[1], p[2], p[3]);
        reinterpret_cast<float4*>(d)[1] = make_float4(p[4], p[5], p[6], p[7]);
    }
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait_but() {  // all but the last n groups
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// NV: 16-byte vectors (8 logits) per thread.  wide: rows of X start on 16-byte
// boundaries; wide_y: rows of Y do (2: on 32-byte boundaries).
template <int NV>
__global__ void __launch_bounds__(kThreads)
    softmax_kernel(const uint16_t* X, int V, int64_t ldx, float c, int one_hot, float* Y,
                   int64_t ldy, int nc, int wide, int wide_y) {
    __shared__ float red_m[kThreads / 32], red_s[kThreads / 32];
    __shared__ int red_i[kThreads / 32];
    __shared__ float part[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / nc;
    const int rank = blockIdx.x % nc;
    const uint16_t* x = X + row * ldx;
    const int v0 = rank * (NV * kThreads);  // first vector of this CTA
    pdl_wait();
    pdl_launch_dependents();
    uint4 r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e0 = (v0 + i * kThreads + tid) * 8;
        if (wide && e0 + 8 <= V) {
            r[i] = ld_nc_v4(x + e0);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // -inf past the row's end
                const uint32_t lo = e0 + 2 * e < V ? x[e0 + 2 * e] : 0xFF80u;
                const uint32_t hi = e0 + 2 * e + 1 < V ? x[e0 + 2 * e + 1] : 0xFF80u;
                w[e] = lo | (hi << 16);
            }
            r[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    auto at = [&](int i, int e) -> float {
        const uint32_t w = e < 2 ? r[i].x : e < 4 ? r[i].y : e < 6 ? r[i].z : r[i].w;
        return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
    };
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, at(i, e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) red_m[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red_m[w]);

    if (one_hot) {
        // the lowest index that holds the CTA's maximum, then the row's
        int best = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 7; e >= 0; --e)
                if (at(i, e) == m) best = min(best, (v0 + i * kThreads + tid) * 8 + e);
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0) red_i[warp] = best;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) best = min(best, red_i[w]);
        if (nc > 1) {
            if (tid == 0) part[0] = m, part[1] = __int_as_float(best);
            cluster_meet();
            float M = -INFINITY;
            for (int j = 0; j < nc; ++j) M = fmaxf(M, ld_shared_cluster_f32(mapa_shared(smem_addr(&part[0]), j)));
            best = 0x7FFFFFFF;
            for (int j = 0; j < nc; ++j)
                if (ld_shared_cluster_f32(mapa_shared(smem_addr(&part[0]), j)) == M)
                    best = min(best, __float_as_int(ld_shared_cluster_f32(mapa_shared(smem_addr(&part[1]), j))));
            m = M;
            cluster_meet();
        }
        if (m == -INFINITY) best = -1;  // nothing but -inf: no probability anywhere
        float* y = Y + row * ldy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e0 = (v0 + i * kThreads + tid) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < V) y[e0 + e] = e0 + e == best ? 1.0f : 0.0f;
        }
        return;
    }

    float s = 0.f;
    const float ref = reference(m);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += ex2((at(i, e) - ref) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) red_s[warp] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red_s[w];
    if (nc > 1) {
        if (tid == 0) part[0] = m, part[1] = s;
        cluster_meet();
        m = -INFINITY, s = 0.f;
        for (int j = 0; j < nc; ++j)
            merge(m, s, ld_shared_cluster_f32(mapa_shared(smem_addr(&part[0]), j)),
                  ld_shared_cluster_f32(mapa_shared(smem_addr(&part[1]), j)), c);
        cluster_meet();  // no CTA leaves while another still reads its pair
    }
    const float inv = s == 0.0f ? 0.0f : 1.0f / s, ref_row = reference(m);
    float* y = Y + row * ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e0 = (v0 + i * kThreads + tid) * 8;
        if (e0 >= V) continue;
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = ex2((at(i, e) - ref_row) * c) * inv;
        if (wide_y && e0 + 8 <= V) {
            store8(y + e0, p, wide_y > 1);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < V) y[e0 + e] = p[e];
        }
    }
}

__device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }

// A part of a row per CTA (a cluster of kParts), all of it on its way to shared memory at
// once: the maximum and the sum as the groups of copies land, the probabilities from there.
// A thread reads only what it copied.
template <int kParts>
__global__ void __launch_bounds__(kRowThreads, kRowCtas)
    softmax_rows_kernel(const uint16_t* X, int V, int64_t ldx, float c, float* Y, int64_t ldy, int per, bool whole) {
    extern __shared__ uint4 held[];
    __shared__ float red_m[kRowThreads / 32], red_s[kRowThreads / 32];
    __shared__ float part[2];
    constexpr int kGroups = 4, kStep = kRowFly * kRowThreads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / kParts;
    const int rank = blockIdx.x % kParts;
    // elements before the row's first 16-byte boundary, whole vectors, elements after the last
    const uint16_t* xr = X + row * ldx;
    float* yr = Y + row * ldy;
    const int head = (int)((16 - (reinterpret_cast<uintptr_t>(xr) & 15)) & 15) / 2;
    const int vecs = (V - head) / 8, lo = rank * per, n = min(vecs - lo, per);  // this CTA's vectors
    const int end = head + vecs * 8;
    const int extra = rank == 0 && tid < head ? tid : rank == kParts - 1 && end + tid < V ? end + tid : -1;
    const uint16_t* x = xr + head + (int64_t)lo * 8;
    float* y = yr + head + (int64_t)lo * 8;
    const int group = (per + kGroups * kStep - 1) / (kGroups * kStep) * kStep;
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        for (int i = g * group + tid; i < min(n, (g + 1) * group); i += kRowThreads)
            cp_async_16(smem_addr(held + i), x + (int64_t)i * 8, 16);
        cp_async_commit();
    }
    auto at = [](const uint4& r, int e) -> float {
        const uint32_t w = e < 2 ? r.x : e < 4 ? r.y : e < 6 ? r.z : r.w;
        return __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
    };
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        if (g == 0) cp_async_wait_but<3>();
        if (g == 1) cp_async_wait_but<2>();
        if (g == 2) cp_async_wait_but<1>();
        if (g == 3) cp_async_wait_but<0>();
        for (int i0 = g * group + tid; i0 < min(n, (g + 1) * group); i0 += kStep) {
            uint4 r[kRowFly];
#pragma unroll
            for (int i = 0; i < kRowFly; ++i)
                r[i] = i0 + i * kRowThreads < n ? held[i0 + i * kRowThreads]
                                                : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
            // the maximum in pairs, as bf16 (exact)
            __nv_bfloat162 top = pair(r[0].x);
#pragma unroll
            for (int i = 0; i < kRowFly; ++i) {
                top = __hmax2(top, __hmax2(pair(r[i].x), pair(r[i].y)));
                top = __hmax2(top, __hmax2(pair(r[i].z), pair(r[i].w)));
            }
            const float mm = fmaxf(m, fmaxf(__low2float(top), __high2float(top)));
            if (mm > m) {
                s *= ex2((m - mm) * c);
                m = mm;
            }
            const float ref = reference(m);
#pragma unroll
            for (int i = 0; i < kRowFly; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += ex2((at(r[i], e) - ref) * c);
        }
    }
    if (extra >= 0) {
        const float v = __uint_as_float((uint32_t)xr[extra] << 16);
        merge(m, s, fmaxf(v, -INFINITY), ex2((v - reference(v)) * c), c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        merge(m, s, m2, s2, c);
    }
    if (lane == 0) red_m[warp] = m, red_s[warp] = s;
    __syncthreads();
    m = red_m[lane & (kRowThreads / 32 - 1)], s = red_s[lane & (kRowThreads / 32 - 1)];
#pragma unroll
    for (int o = kRowThreads / 64; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
        merge(m, s, m2, s2, c);
    }
    if (tid == 0) part[0] = m, part[1] = s;
    cluster_meet();
    m = -INFINITY, s = 0.f;
#pragma unroll
    for (int j = 0; j < kParts; ++j)
        merge(m, s, ld_shared_cluster_f32(mapa_shared(smem_addr(&part[0]), j)),
              ld_shared_cluster_f32(mapa_shared(smem_addr(&part[1]), j)), c);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s, ref = reference(m);
    for (int i0 = tid; i0 < n; i0 += kStep) {
        uint4 r[kRowFly];
#pragma unroll
        for (int i = 0; i < kRowFly; ++i)
            if (i0 + i * kRowThreads < n) r[i] = held[i0 + i * kRowThreads];
#pragma unroll
        for (int i = 0; i < kRowFly; ++i) {
            if (i0 + i * kRowThreads >= n) break;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = ex2((at(r[i], e) - ref) * c) * inv;
            store8(y + (int64_t)(i0 + i * kRowThreads) * 8, p, whole);
        }
    }
    if (extra >= 0) {
        const float v = __uint_as_float((uint32_t)xr[extra] << 16);
        yr[extra] = ex2((v - ref) * c) * inv;
    }
    cluster_meet();  // no CTA leaves while another still reads its pair
}

template <int NV>
cudaError_t launch(const uint16_t* X, int rows, int V, int64_t ldx, float temperature, float* Y, int64_t ldy, int nc,
                   cudaStream_t stream) {
    const int wide = (reinterpret_cast<uintptr_t>(X) & 15) == 0 && ldx % 8 == 0;
    const int wide_y = (reinterpret_cast<uintptr_t>(Y) & 31) == 0 && ldy % 8 == 0   ? 2
                       : (reinterpret_cast<uintptr_t>(Y) & 15) == 0 && ldy % 4 == 0 ? 1
                                                                                    : 0;
    const int one_hot = temperature == 0.0f;
    const float c = one_hot ? 0.0f : kLog2e / temperature;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * nc);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = nc;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, softmax_kernel<NV>, X, V, ldx, c, one_hot, Y, ldy, nc, wide, wide_y);
}

// Whether an element that starts 16 bytes of a row of X starts 32 bytes of the row of Y, in every row.
bool alike(const uint16_t* X, int64_t ldx, const float* Y, int64_t ldy) {
    return (reinterpret_cast<uintptr_t>(X) / 2 - reinterpret_cast<uintptr_t>(Y) / 4) % 8 == 0 && (ldx - ldy) % 8 == 0;
}

template <int kParts>
cudaError_t launch_rows(const uint16_t* X, int rows, int V, int64_t ldx, float temperature, float* Y, int64_t ldy,
                        cudaStream_t stream) {
    const int per = (V / 8 / kParts + 32) & ~31;  // vectors of a part, the last one's fewer
    const bool whole = alike(X, ldx, Y, ldy);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * kParts);
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = (size_t)per * 16;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kParts;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = ensure_smem_limit(softmax_rows_kernel<kParts>, cfg.dynamicSmemBytes);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, softmax_rows_kernel<kParts>, X, V, ldx, kLog2e / temperature, Y, ldy, per, whole);
}

}  // namespace

cudaError_t launch_softmax(const uint16_t* X, int rows, int V, int64_t ldx, float temperature, float* Y, int64_t ldy,
                           cudaStream_t stream) {
    const int vecs = (V + 7) / 8;
    const bool aligned = (reinterpret_cast<uintptr_t>(X) & 15) == 0 && ldx % 8 == 0 &&
                         (reinterpret_cast<uintptr_t>(Y) & 15) == 0 && ldy % 4 == 0;
    const bool ragged = !aligned && alike(X, ldx, Y, ldy);  // rows that start anywhere
    if (temperature != 0.0f && ((aligned && rows >= kManyRows && V >= kLongRow) || (ragged && V >= kRaggedRow)))
        return V >= kEightParts ? launch_rows<8>(X, rows, V, ldx, temperature, Y, ldy, stream)
                                : launch_rows<4>(X, rows, V, ldx, temperature, Y, ldy, stream);
    int nc = 1;
    while (nc < 8 && vecs > nc * kThreads) nc *= 2;
    const int nv = (vecs + nc * kThreads - 1) / (nc * kThreads);
    if (nv <= 1) return launch<1>(X, rows, V, ldx, temperature, Y, ldy, nc, stream);
    if (nv <= 2) return launch<2>(X, rows, V, ldx, temperature, Y, ldy, nc, stream);
    if (nv <= 4) return launch<4>(X, rows, V, ldx, temperature, Y, ldy, nc, stream);
    if (nv <= 8) return launch<8>(X, rows, V, ldx, temperature, Y, ldy, nc, stream);
    return cudaErrorInvalidValue;
}

}  // namespace rmm
