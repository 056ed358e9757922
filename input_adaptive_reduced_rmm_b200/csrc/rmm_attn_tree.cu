// rmm_attn_tree.cu -- reduced attention of a draft tree over the cache.
//
// Sequence b has len_b cached keys and T <= 64 tree nodes whose keys sit at the
// slots len_b .. len_b + T - 1.  For KV head g with its G query heads q:
//   S     = the k dims with the largest max over q and the present t of |Q[q,t,j]|
//   x_l   = scale * sum_{j in S} Q[q,t,j] K[l,j]   for l < len_b and for the slots
//           of node t and its ancestors
//   O     = softmax(x) V, zero where the row sees no key
// One CTA per (sequence, query head, node): 128 keys at a time, a thread per key
// for the logits, a thread per dim for P.V, with the running maximum and sum.
#include <math.h>

#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;

__global__ void __launch_bounds__(D)
    tree_dims_kernel(const uint16_t* __restrict__ Q, int Hq, int Hkv, int T, int ldL, int k,
                     const int32_t* __restrict__ lens, const int32_t* __restrict__ parents, int32_t* __restrict__ idx) {
    __shared__ int32_t par[kTreeMax];
    __shared__ uint32_t sv[D];
    __shared__ int warp_cnt[D / 32];
    const int b = blockIdx.x / Hkv, g = blockIdx.x % Hkv, G = Hq / Hkv, j = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (lens[b] < 0 || lens[b] > ldL - T) return;
    if (parents && j < T) par[j] = parents[(size_t)b * T + j];
    __syncthreads();
    uint32_t m = 0;
    for (int t = 0; t < T; ++t) {
        if (parents && tree_way(par, t) == 0) continue;
        for (int q = 0; q < G; ++q) m = max(m, (uint32_t)(Q[(((size_t)b * Hq + g * G + q) * T + t) * D + j] & 0x7FFF));
    }
    sv[j] = m;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < D; ++i) rank += sv[i] > m || (sv[i] == m && i < j);
    const bool keep = rank < k;
    const unsigned ball = __ballot_sync(0xffffffffu, keep);
    if ((j & 31) == 0) warp_cnt[j >> 5] = __popc(ball);
    __syncthreads();
    int pos = __popc(ball & ((1u << (j & 31)) - 1u));
    for (int i = 0; i < (j >> 5); ++i) pos += warp_cnt[i];
    if (keep) idx[(size_t)blockIdx.x * k + pos] = j;
}

__global__ void __launch_bounds__(D)
    attn_tree_kernel(const uint16_t* __restrict__ Q, const uint16_t* __restrict__ Kt, const uint16_t* __restrict__ V,
                     int Hq, int Hkv, int T, int ldL, int k, float scale, const int32_t* __restrict__ lens,
                     const int32_t* __restrict__ parents, const int32_t* __restrict__ idx, uint16_t* __restrict__ O,
                     int* status) {
    __shared__ int32_t par[kTreeMax];
    __shared__ float qs[D], p_s[D];
    __shared__ int sidx[D];
    __shared__ float red[4];
    const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int g = h / (Hq / Hkv);
    pdl_wait();
    pdl_launch_dependents();
    const size_t row = ((size_t)b * Hq + h) * T + t;
    const int len = lens[b];
    if (len > ldL - T && t == 0 && h == 0 && tid == 0) record_status(status, RMM_ERR_INVALID_ARG);
    if (parents && tid < T) par[tid] = parents[(size_t)b * T + tid];
    __syncthreads();
    const uint64_t way = len < 0 || len > ldL - T ? 0 : parents ? tree_way(par, t) : chain_way(t);
    float acc = 0.f, m = -INFINITY, l = 0.f;
    if (way) {
        if (tid < k) {
            sidx[tid] = idx[((size_t)b * Hkv + g) * k + tid];
            qs[tid] = bf16_bits_to_float(Q[row * D + sidx[tid]]) * scale;
        }
        __syncthreads();
        const uint16_t* Kg = Kt + ((size_t)b * Hkv + g) * D * (size_t)ldL;
        const uint16_t* Vg = V + ((size_t)b * Hkv + g) * (size_t)ldL * D;
        for (int l0 = 0; l0 < len + T; l0 += D) {
            const int key = l0 + tid;
            float x = -INFINITY;
            if (key < len || (key < len + T && ((way >> (key - len)) & 1))) {
                x = 0.f;
                for (int j = 0; j < k; ++j) x = fmaf(qs[j], bf16_bits_to_float(Kg[(size_t)sidx[j] * ldL + key]), x);
            }
            float mx = x;
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if ((tid & 31) == 0) red[tid >> 5] = mx;
            __syncthreads();
            const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
            const float p = x == -INFINITY ? 0.f : expf(x - m_new);
            const float alpha = m == -INFINITY ? 0.f : expf(m - m_new);
            p_s[tid] = p;
            __syncthreads();
            acc *= alpha;
            l *= alpha;
            m = m_new;
            const int n = min(D, len + T - l0);
            for (int i = 0; i < n; ++i) {
                if (p_s[i] == 0.f) continue;
                l += p_s[i];
                acc = fmaf(p_s[i], bf16_bits_to_float(Vg[(size_t)(l0 + i) * D + tid]), acc);
            }
            __syncthreads();
        }
    }
    O[row * D + tid] = float_to_bf16_bits(l > 0.f ? acc / l : 0.f);
}

}  // namespace

size_t attn_tree_partial_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_attn_tree(const uint16_t* Q, const uint16_t* Kt, const uint16_t* V, int B, int Hq, int Hkv, int T,
                             int ldL, int k, float scale, const int32_t* lens, const int32_t* parents, uint16_t* O,
                             int32_t* idx, float* partials, int* status, int num_sms, cudaStream_t stream) {
    cudaError_t e = launch_pdl(tree_dims_kernel, dim3(B * Hkv), dim3(D), 0, stream, Q, Hq, Hkv, T, ldL, k, lens,
                               parents, idx);
    if (e != cudaSuccess) return e;
    return launch_pdl(attn_tree_kernel, dim3(T, Hq, B), dim3(D), 0, stream, Q, Kt, V, Hq, Hkv, T, ldL, k, scale, lens,
                      parents, (const int32_t*)idx, O, status);
}

}  // namespace rmm
