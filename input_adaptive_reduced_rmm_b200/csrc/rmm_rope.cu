// rmm_rope.cu -- the q/k/v projections of a batch of sequences into attention
// heads, with per-head RMS norms of q and k and the position rotation in the
// same pass, and the append of keys and values at each sequence's own length.
//
//   x'  = x / sqrt(mean_j x_j^2 + eps) * w                 (q and k, each head)
//   (x'_i, x'_j) -> (x'_i c - x'_j s, x'_j c + x'_i s)     c + is = e^(i pos f_i)
// for the rot/2 pairs (i, j) = (i, i + rot/2), or (2i, 2i+1) when interleaved.
// Everything between the bf16 input and the one rounding to bf16 is fp32.  The
// angle is a fraction of a turn in 64-bit fixed point, pos * round(2^64 f / 2 pi)
// modulo 2^64, reduced to half a turn either way before it becomes fp32: off by at
// most 2^-26 of a turn from that rounding, 2^-32 from the bits below it and
// pos f 2^-54 from the frequency's product in fp64 (an angle formed in fp32 is off
// by 0.004 rad at position 10^5).  Sine and cosine are fp32.
//
// Memory bound: each element is read once and written once.  A quarter-warp holds
// one (token, head) row of 128 dims; a lane has 8 dims and the 8 that they are
// rotated with, so only the norm's sum crosses lanes, and 8 angles serve both.  It
// keeps a token's sines and cosines, times the norm's weights, in registers over
// the CTA's heads and has four heads' rows in flight.  With fewer than 32 tokens
// the quarter-warps share them and take different heads.  Keys go through a
// shared tile to the d-major cache, written in 16-byte pieces of 8 slots where
// all 8 belong to the call.
//
// Measured: 4096 tokens of 64 + 8 + 8 heads move their 168 MB (beside what stays in
// L2) in 39 us, 4.3 TB/s counted on the data alone; 64 sequences of one token
// take 6.5 us, trees of 25 nodes of 8 sequences 9.3, of 64 nodes of 16 sequences
// (32 + 8 + 8 heads) 17.8.  Steps at 4096 tokens: a whole warp per row 101 us, half-warps 57,
// quarter-warps with packed arithmetic 43, four rows in flight and 64 tokens per
// CTA 38 (two rows 42, 32 tokens 41).
#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;
constexpr int kRopeThreads = 256;
constexpr int kFly = 4;  // heads' rows in flight
// Tokens per CTA; heads per CTA of q and v (the angles of a token serve them all) and of k
// (each with its shared tile).  A batch of single tokens that would have more CTAs than
// places (two per SM) takes more heads per CTA: 64 sequences of 32 + 8 + 8 heads 192 CTAs
// instead of 448, 6.5 us instead of 7.3, of 64 + 8 + 8 heads 256 instead of 576, 6.5 instead of
// 7.7; 8 sequences, which fit, 4.5 instead of 3.9.
struct RopeTile {
    int tokens, heads, key_heads;
};
constexpr RopeTile kSingleTile{1, 32, 16}, kManyTile{64, 16, 2};

struct RopeArgs {
    const uint16_t *Yq, *Yk, *Yv, *qn, *kn;
    const float* inv_freq;
    const int32_t *lens, *parents;
    uint16_t *Q, *Kt, *V;
    int T, Hq, Hkv, rot, interleaved, ldL, L0, tiles;
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4& w, F2 (&f)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = F2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        f[e].get(lo, hi);
        u[e] = pack2(lo, hi);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// cos and sin of pos * f, with `turns` = 2^64 f / 2 pi modulo 2^64
__device__ __forceinline__ void turn(int pos, uint64_t turns, float& c, float& s) {
    const int32_t half = (int32_t)(((uint64_t)(uint32_t)pos * turns) >> 32);  // in units of 2^-31 half turns
    sincospif((float)half * 4.656612873077393e-10f, &s, &c);
}

template <bool kInterleaved, bool kSingle>
__global__ void __launch_bounds__(kRopeThreads, 2) qkv_rope_kernel(const RopeArgs a) {
    constexpr RopeTile kTile = kSingle ? kSingleTile : kManyTile;
    constexpr int kRopeTokens = kTile.tokens, kRopeHeads = kTile.heads, kRopeKeyHeads = kTile.key_heads;
    constexpr int kTilePitch = kRopeTokens + 1;  // u16 per dim row of a key tile
    __shared__ int32_t par[kTreeMax];
    __shared__ int pos_s[kRopeTokens];
    __shared__ uint64_t freq[D / 2];  // 2^64 f / 2 pi modulo 2^64
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
    if (tid >= 64 && tid < 64 + a.rot / 2) {
        double t = (double)a.inv_freq[tid - 64] * 0.15915494309189533577;  // turns per position
        t -= floor(t);
        freq[tid - 64] = __double2ull_rn(t * 18446744073709551616.0);
    }
    if (tid < nt) {
        int p = t0 + tid;
        if (a.parents) p = __popcll(tree_way(par, p)) - 1;  // depth; -1 when absent
        pos_s[tid] = p < 0 ? -1 : start + p;
    }
    const bool holes = __syncthreads_or(tid < nt && pos_s[tid] < 0);  // absent nodes: their slots stay

    const int l = tid & 7, qw = tid >> 3;
    const unsigned mask = 0xFFu << (tid & 24);
    // quarter-warps over tokens, the rest over heads
    const int tpar = nt > 16 ? 32 : nt > 8 ? 16 : nt > 4 ? 8 : nt > 2 ? 4 : nt;
    const int hpar = 32 / tpar, ho = qw / tpar;
    const bool turns = kind != 2 && a.inv_freq;
    // the lane's dims A .. A+7 and B .. B+7: pairs (A + e, B + e), or neighbours when interleaved;
    // a quarter-warp's loads and stores are 128 bytes in a row wherever the pairs allow it
    const int half = a.rot / 2;
    int A = 8 * l, B = 64 + 8 * l;
    bool turned = turns && A < a.rot, turned_b = turns && B < a.rot;
    if (turns && !kInterleaved) {
        turned = turned_b = 8 * l < half;
        A = turned ? 8 * l : a.rot + 2 * (8 * l - half);
        B = turned ? 8 * l + half : A + 8;
    }
    const uint16_t* Y = kind == 0 ? a.Yq : kind == 1 ? a.Yk : a.Yv;
    const uint16_t* wn = kind == 0 ? a.qn : kind == 1 ? a.kn : nullptr;

    // lanes of a quarter-warp agree on everything but l, so shuffles stay inside it
    for (int tl = qw % tpar; tl < nt; tl += tpar) {
        const int pos = pos_s[tl];
        if (pos < 0) continue;
        const size_t row = (size_t)b * a.T + t0 + tl;
        const uint16_t* src = Y + (row * H + h0) * D;
        uint4 na[kFly], nb[kFly];  // the next heads' rows
        auto fetch = [&](int hb) {
#pragma unroll
            for (int i = 0; i < kFly; ++i)
                if (hb + i * hpar < nh) {
                    na[i] = ld_nc_v4(src + (size_t)(hb + i * hpar) * D + A);
                    nb[i] = ld_nc_v4(src + (size_t)(hb + i * hpar) * D + B);
                }
        };
        fetch(ho);
        // x = (a, b): a' = a ca + b sa, b' = b cb + a sb, where the angle's parts hold the norm's
        // weights too: for pairs across a and b the factors are c w_a, -s w_b, c w_b, s w_a
        F2 ca[4], sa[4], cb[4], sb[4];
        {
            F2 one[4] = {F2(1.f, 1.f), F2(1.f, 1.f), F2(1.f, 1.f), F2(1.f, 1.f)};
            F2 wa[4], wb[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) wa[e] = wb[e] = one[e];
            if (wn) {
                unpack8(ld_nc_v4(wn + A), wa);
                unpack8(ld_nc_v4(wn + B), wb);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float c0 = 1.f, s0 = 0.f, c1 = 1.f, s1 = 0.f;
                // of pairs across a and b, 8 angles for both; of neighbours, 4 of a's and 4 of b's
                const int at = !kInterleaved ? 8 * l + 2 * e : e < 2 ? 4 * l + 2 * e : 32 + 4 * l + 2 * (e - 2);
                if (e < 2 ? turned : turned_b) {
                    turn(pos, freq[at], c0, s0);
                    turn(pos, freq[at + 1], c1, s1);
                }
                if (kInterleaved) {
                    // the angles belong to the neighbours of two words: of a for e < 2, of b above; their (c, c) and (-s, s), weights of the partner in the second
                    F2* cx = e < 2 ? ca : cb;
                    F2* sx = e < 2 ? sa : sb;
                    const F2* wx = e < 2 ? wa : wb;
                    const int k = 2 * (e & 1);
                    float u, v;
                    wx[k].get(u, v);
                    cx[k] = F2(u * c0, v * c0);
                    sx[k] = F2(-v * s0, u * s0);
                    wx[k + 1].get(u, v);
                    cx[k + 1] = F2(u * c1, v * c1);
                    sx[k + 1] = F2(-v * s1, u * s1);
                } else {
                    ca[e] = mul2(wa[e], F2(c0, c1));
                    cb[e] = mul2(wb[e], F2(c0, c1));
                    sa[e] = mul2(wb[e], F2(-s0, -s1));
                    sb[e] = mul2(wa[e], F2(s0, s1));
                }
            }
        }
        for (int hb = ho; hb < nh; hb += hpar * kFly) {
            uint4 ra[kFly], rb[kFly];
#pragma unroll
            for (int i = 0; i < kFly; ++i) ra[i] = na[i], rb[i] = nb[i];
            fetch(hb + hpar * kFly);
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                const int h = hb + i * hpar;
                if (h >= nh) break;
                if (wn || turns) {
                    F2 x[4], y[4];
                    unpack8(ra[i], x);
                    unpack8(rb[i], y);
                    float inv = 1.0f;
                    if (wn) {
                        F2 s2 = mul2(x[0], x[0]);
#pragma unroll
                        for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s2 = fma2(y[e], y[e], s2);
                        float s0, s1;
                        s2.get(s0, s1);
                        float ss = s0 + s1;
#pragma unroll
                        for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o, 8);
                        inv = rsqrtf(ss * (1.0f / D) + a.eps);
                    }
                    const F2 i2(inv, inv);
                    F2 p[4], q[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        F2 xs = y[e], ys = x[e];
                        if (kInterleaved) {  // a neighbour's partner is the other half of its word
                            float u, v;
                            x[e].get(u, v);
                            xs = F2(v, u);
                            y[e].get(u, v);
                            ys = F2(v, u);
                        }
                        p[e] = mul2(fma2(x[e], ca[e], mul2(xs, sa[e])), i2);
                        q[e] = mul2(fma2(y[e], cb[e], mul2(ys, sb[e])), i2);
                    }
                    ra[i] = pack8(p);
                    rb[i] = pack8(q);
                }
                if (kind == 1) {
                    uint16_t* ta = tile[h] + A * kTilePitch + tl;
                    uint16_t* tb = tile[h] + B * kTilePitch + tl;
                    const uint32_t ua[4] = {ra[i].x, ra[i].y, ra[i].z, ra[i].w};
                    const uint32_t ub[4] = {rb[i].x, rb[i].y, rb[i].z, rb[i].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        ta[e * kTilePitch] = (uint16_t)(ua[e >> 1] >> (16 * (e & 1)));
                        tb[e * kTilePitch] = (uint16_t)(ub[e >> 1] >> (16 * (e & 1)));
                    }
                } else {
                    uint16_t* dst = kind == 0 ? a.Q + (((size_t)b * a.Hq + h0 + h) * a.T + t0 + tl) * D
                                              : a.V + (((size_t)b * a.Hkv + h0 + h) * a.ldL + start + t0 + tl) * D;
                    *reinterpret_cast<uint4*>(dst + A) = ra[i];
                    *reinterpret_cast<uint4*>(dst + B) = rb[i];
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
        const int tl = 8 * p - s0;
        const uint16_t* t = tile[hj >> 7] + (hj & (D - 1)) * kTilePitch + tl;
        uint16_t* dst = Kg + (size_t)hj * a.ldL + 8 * p;
        if (tl >= 0 && tl + 8 <= nt && !holes) {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = t[2 * e] | ((uint32_t)t[2 * e + 1] << 16);
            *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
        } else {
            for (int e = max(0, -tl); e < 8 && tl + e < nt; ++e)
                if (pos_s[tl + e] >= 0) dst[e] = t[e];
        }
    }
}

}  // namespace

cudaError_t launch_qkv_rope(const uint16_t* Yq, const uint16_t* Yk, const uint16_t* Yv, int B, int T, int Hq, int Hkv,
                            const uint16_t* q_norm, const uint16_t* k_norm, float eps, const float* inv_freq, int rot,
                            int interleaved, const int32_t* lens, int L0, const int32_t* parents, uint16_t* Q,
                            uint16_t* Kt, uint16_t* V, int ldL, int num_sms, cudaStream_t stream) {
    auto groups = [&](const RopeTile& t) {
        return (Hq + t.heads - 1) / t.heads + (Hkv + t.key_heads - 1) / t.key_heads + (Hkv + t.heads - 1) / t.heads;
    };
    const bool single = T == 1 && (long long)B * groups(kManyTile) > 2 * num_sms;
    const RopeTile& tile = single ? kSingleTile : kManyTile;
    RopeArgs a{Yq, Yk, Yv, q_norm, k_norm, inv_freq, lens, parents, Q, Kt, V,
               T,  Hq, Hkv, inv_freq ? rot : 0, interleaved, ldL, L0, (T + tile.tokens - 1) / tile.tokens,
               eps};
    const long long x = (long long)B * a.tiles;
    if (x > 0x7FFFFFFFll || groups(tile) > 65535) return cudaErrorInvalidValue;
    auto* kern = single ? interleaved ? qkv_rope_kernel<true, true> : qkv_rope_kernel<false, true>
                        : interleaved ? qkv_rope_kernel<true, false> : qkv_rope_kernel<false, false>;
    return launch_pdl(kern, dim3((unsigned)x, groups(tile)), dim3(kRopeThreads), 0, stream, a);
}

}  // namespace rmm
