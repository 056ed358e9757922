// rmm_rope.cu -- the q/k/v projections of a batch of sequences into attention
// heads, with per-head RMS norms of q and k and the position rotation in the
// same pass, and the append of keys and values at each sequence's own length.
//
//   x'  = x / sqrt(mean_j x_j^2 + eps) * w                 (q and k, each head)
//   (x'_i, x'_j) -> (x'_i c - x'_j s, x'_j c + x'_i s)     c + is = e^(i pos f_i)
// for the rot/2 pairs (i, j) = (i, i + rot/2), or (2i, 2i+1) when interleaved.
// Everything between the bf16 input and the one rounding to bf16 is fp32; the
// angle pos * f_i is formed and reduced to a fraction of a turn in fp64 (an
// fp32 angle is off by 0.004 rad at position 10^5), its sine and cosine in
// fp32.
//
// Memory bound: each element is read once and written once.  A half-warp holds
// one (token, head) row of 128 dims, 8 per lane, so the norm and the partner of
// a rotated pair are shuffles; it keeps a token's sines and cosines in registers
// over the CTA's heads and has four heads' rows in flight.  With fewer than 16
// tokens the half-warps share them and take different heads.  Keys go through a
// shared tile to the d-major cache, written in 16-byte pieces of 8 slots where
// all 8 belong to the call.
#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;
constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 32;   // tokens per CTA
constexpr int kRopeHeads = 16;    // heads per CTA (q and v): the angles of a token serve them all
constexpr int kRopeKeyHeads = 4;  // heads per CTA (k): one shared tile each
constexpr int kFly = 4;           // heads' rows in flight
constexpr int kTilePitch = kRopeTokens + 1;  // u16 per dim row of a key tile

struct RopeArgs {
    const uint16_t *Yq, *Yk, *Yv, *qn, *kn;
    const float* inv_freq;
    const int32_t *lens, *parents;
    uint16_t *Q, *Kt, *V;
    int T, Hq, Hkv, rot, interleaved, ldL, L0, tiles;
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// cos and sin of pos * f; the product of a 31-bit position and a 24-bit
// frequency is exact in fp64
__device__ __forceinline__ void turn(int pos, float f, float& c, float& s) {
    const double t = (double)pos * (double)f * 0.15915494309189533577;  // turns
    sincospif(2.0f * (float)(t - rint(t)), &s, &c);
}

__global__ void __launch_bounds__(kRopeThreads) qkv_rope_kernel(const RopeArgs a) {
    __shared__ int32_t par[kTreeMax];
    __shared__ int pos_s[kRopeTokens];
    __shared__ uint16_t tile[kRopeKeyHeads][D * kTilePitch];
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.tiles, t0 = (blockIdx.x % a.tiles) * kRopeTokens;
    const int nt = min(kRopeTokens, a.T - t0);
    // head groups of q, then of k, then of v
    const int gq = (a.Hq + kRopeHeads - 1) / kRopeHeads, gk = (a.Hkv + kRopeKeyHeads - 1) / kRopeKeyHeads;
    const int kind = (int)blockIdx.y < gq ? 0 : (int)blockIdx.y < gq + gk ? 1 : 2;
    const int per = kind == 1 ? kRopeKeyHeads : kRopeHeads;
    const int h0 = ((int)blockIdx.y - (kind == 0 ? 0 : kind == 1 ? gq : gq + gk)) * per;
    const int H = kind == 0 ? a.Hq : a.Hkv;
    const int nh = min(per, H - h0);
    pdl_wait();
    pdl_launch_dependents();
    const int start = a.lens ? a.lens[b] : a.L0;
    if (start < 0 || start > a.ldL - a.T) return;  // an empty slot of the batch, or no room: nothing is written
    if (a.parents) {
        if (tid < a.T) par[tid] = a.parents[(size_t)b * a.T + tid];
        __syncthreads();
    }
    if (tid < nt) {
        int p = t0 + tid;
        if (a.parents) p = __popcll(tree_way(par, p)) - 1;  // depth; -1 when absent
        pos_s[tid] = p < 0 ? -1 : start + p;
    }
    __syncthreads();

    const int l = tid & 15, hw = tid >> 4;  // dims 8l .. 8l+7 of the half-warp's row
    const unsigned mask = 0xFFFFu << (tid & 16);
    // half-warps over tokens, the rest over heads
    const int tpar = nt >= 16 ? 16 : nt > 8 ? 16 : nt > 4 ? 8 : nt > 2 ? 4 : nt;
    const int hpar = 16 / tpar, ho = hw / tpar;
    const int half = a.rot >> 4;            // lanes of one half of the rotated dims
    const bool turns = kind != 2 && a.inv_freq;
    const bool turned = turns && 8 * l < a.rot;
    const int partner = a.interleaved ? l : (l < half ? l + half : l < 2 * half ? l - half : l);
    const bool hi = l >= half;
    const uint16_t* Y = kind == 0 ? a.Yq : kind == 1 ? a.Yk : a.Yv;
    const uint16_t* wn = kind == 0 ? a.qn : kind == 1 ? a.kn : nullptr;
    float w[8];
    if (wn) unpack8(ld_nc_v4(wn + 8 * l), w);

    // lanes of a half-warp agree on everything but l, so shuffles stay inside it
    for (int tl = hw % tpar; tl < nt; tl += tpar) {
        const int pos = pos_s[tl];
        if (pos < 0) continue;
        const size_t row = (size_t)b * a.T + t0 + tl;
        const uint16_t* src = Y + (row * H + h0) * D + 8 * l;
        float c[8], s[8];
        if (turns) {
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    c[e] = 1.f, s[e] = 0.f;
                    if (turned) turn(pos, __ldg(a.inv_freq + 4 * l + e), c[e], s[e]);
                }
            } else {
                // the two lanes of a pair of chunks share 8 angles: each forms four
                float mc[4], ms[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mc[e] = 1.f, ms[e] = 0.f;
                    if (turned) turn(pos, __ldg(a.inv_freq + 8 * (hi ? l - half : l) + (hi ? 4 : 0) + e), mc[e], ms[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float oc = __shfl_sync(mask, mc[e], partner, 16);
                    const float os = __shfl_sync(mask, ms[e], partner, 16);
                    c[e] = hi ? oc : mc[e];
                    s[e] = hi ? os : ms[e];
                    c[4 + e] = hi ? mc[e] : oc;
                    s[4 + e] = hi ? ms[e] : os;
                }
            }
        }
        for (int hb = ho; hb < nh; hb += hpar * kFly) {
            uint4 raw[kFly];
#pragma unroll
            for (int i = 0; i < kFly; ++i)
                if (hb + i * hpar < nh) raw[i] = ld_nc_v4(src + (size_t)(hb + i * hpar) * D);
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const int h = hb + i * hpar;
                if (h >= nh) break;
                if (wn || turns) {
                    float x[8];
                    unpack8(raw[i], x);
                    if (wn) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, 16);
                        const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * w[e];
                    }
                    if (turns) {
                        if (a.interleaved) {
                            if (turned) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float u = x[2 * e], v = x[2 * e + 1];
                                    x[2 * e] = u * c[e] - v * s[e];
                                    x[2 * e + 1] = v * c[e] + u * s[e];
                                }
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float y = __shfl_sync(mask, x[e], partner, 16);
                                if (turned) x[e] = x[e] * c[e] + (hi ? y : -y) * s[e];
                            }
                        }
                    }
                    raw[i] = pack8(x);
                }
                if (kind == 0) {
                    *reinterpret_cast<uint4*>(a.Q + (((size_t)b * a.Hq + h0 + h) * a.T + t0 + tl) * D + 8 * l) = raw[i];
                } else if (kind == 2) {
                    *reinterpret_cast<uint4*>(a.V + (((size_t)b * a.Hkv + h0 + h) * a.ldL + start + t0 + tl) * D + 8 * l) =
                        raw[i];
                } else {
                    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tile[h][(8 * l + e) * kTilePitch + tl] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    }
    if (kind != 1) return;
    __syncthreads();
    // head h, dim row j, slots 8p .. 8p+7 of the cache
    const int s0 = start + t0;
    const int p0 = s0 >> 3, np = ((s0 + nt - 1) >> 3) - p0 + 1;
    uint16_t* Kg = a.Kt + ((size_t)b * a.Hkv + h0) * D * (size_t)a.ldL;
    for (int i = tid; i < nh * D * np; i += kRopeThreads) {
        const int hj = i / np, p = p0 + i % np;  // hj: head * D + dim, a row of the cache
        const uint16_t* t = tile[hj >> 7] + (hj & (D - 1)) * kTilePitch;
        uint16_t v[8];
        bool all = true, ok[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int tl = 8 * p + e - s0;
            ok[e] = tl >= 0 && tl < nt && pos_s[min(max(tl, 0), kRopeTokens - 1)] >= 0;
            all = all && ok[e];
            v[e] = ok[e] ? t[tl] : (uint16_t)0;
        }
        uint16_t* dst = Kg + (size_t)hj * a.ldL + 8 * p;
        if (all) {
            *reinterpret_cast<uint4*>(dst) = make_uint4(v[0] | ((uint32_t)v[1] << 16), v[2] | ((uint32_t)v[3] << 16),
                                                        v[4] | ((uint32_t)v[5] << 16), v[6] | ((uint32_t)v[7] << 16));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (ok[e]) dst[e] = v[e];
        }
    }
}

}  // namespace

cudaError_t launch_qkv_rope(const uint16_t* Yq, const uint16_t* Yk, const uint16_t* Yv, int B, int T, int Hq, int Hkv,
                            const uint16_t* q_norm, const uint16_t* k_norm, float eps, const float* inv_freq, int rot,
                            int interleaved, const int32_t* lens, int L0, const int32_t* parents, uint16_t* Q,
                            uint16_t* Kt, uint16_t* V, int ldL, cudaStream_t stream) {
    RopeArgs a{Yq, Yk, Yv, q_norm, k_norm, inv_freq, lens, parents, Q, Kt, V,
               T,  Hq, Hkv, inv_freq ? rot : 0, interleaved, ldL, L0, (T + kRopeTokens - 1) / kRopeTokens, eps};
    const int gq = (Hq + kRopeHeads - 1) / kRopeHeads, gk = (Hkv + kRopeKeyHeads - 1) / kRopeKeyHeads;
    const int gv = (Hkv + kRopeHeads - 1) / kRopeHeads;
    const long long x = (long long)B * a.tiles;
    if (x > 0x7FFFFFFFll || gq + gk + gv > 65535) return cudaErrorInvalidValue;
    return launch_pdl(qkv_rope_kernel, dim3((unsigned)x, gq + gk + gv), dim3(kRopeThreads), 0, stream, a);
}

}  // namespace rmm
