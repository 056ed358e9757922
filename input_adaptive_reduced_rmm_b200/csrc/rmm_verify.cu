// rmm_verify.cu -- drafted tokens checked against the target's probabilities
// with given random numbers, on a chain or a tree, and the next token.
//
// From the root the walk goes to the first child it accepts.  With R the part
// of the target's row still to be covered (mass Z, at first the row itself with
// Z = 1), a child that holds token x, drawn from the draft's row Q, is
//   accepted  if  u Q(x) Z < R(x)        (with probability min(1, R(x) / (Z Q(x))))
//   rejected  otherwise, and R becomes max(R - Z Q, 0), Z its sum,
// which keeps the emitted tokens distributed as the target has them for any
// draft.  Without draft rows the drafts count as certain picks: Q(x) = 1 at the
// child's own token.  The next token is the first index at which the running
// sum of R passes u_0 times its sum.
//
// R and every sum are fp64: a token changes where a sum passes a random number,
// and 1e-16 of the mass keeps that border where the definition has it.
//
// One cluster of 8 CTAs per sequence; each of its 128 warps has a contiguous range
// of the vocabulary.  The tests need one probability each, fetched up front for all
// nodes; the rows themselves are read only at a node where a child is rejected, and
// at the last node, once: R (fp64) and the draft's row then stay in registers for
// the node's further rejections and the search of the next token (above 65536 tokens,
// at eight steps a warp, 128 registers do not hold all of both: the compiler keeps 360
// bytes of a thread's in local memory).  A vocabulary above 131072 does not fit there;
// its passes read the rows again and repeat the rejections so far.  A pass sends every warp's sum to all 8 CTAs, so one barrier of
// the cluster gives each of them the total and, for the next token, the place.
// Latency bound: a node's rows take one exposed read, a rejection one barrier of the
// cluster.  16 trees of 32 nodes over 131072 tokens take 25 us, with certain picks 21
// (57 us when every pass read its rows again and the search walked 32 indices at a
// time), one chain of 8 over 32000 tokens 5.6 us (18 us).
#include <math.h>

#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;
constexpr int kAll = kCtas * kWarps;  // warps of a sequence
constexpr int kStep = 128;            // indices a warp takes at once, 4 per lane

// The cluster's barrier wants whole warps: lanes that a condition has parted meet first.
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    cluster_sync();
}

__device__ __forceinline__ void st_shared_cluster_f64(uint32_t addr, double v) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// a probability as the walk reads it: NaN and negative values count as 0
__device__ __forceinline__ double prob(float p) { return p > 0.0f ? (double)p : 0.0; }

// the inclusive sum over the lanes up to this one
__device__ __forceinline__ double warp_prefix(double v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Rejections at the current node: the mass before each (mass[0] is 1) and its token.
struct Rejections {
    double mass[kTreeMax];
    int token[kTreeMax];
};

// R at one index of token x after n rejections, from the rows' values there.
__device__ __forceinline__ double remaining(double r, double q, int x, bool drawn, int n, const Rejections& w) {
    if (drawn) {
        for (int j = 0; j < n; ++j) r = fmax(r - w.mass[j] * q, 0.0);
    } else {
        for (int j = 0; j < n; ++j)
            if (w.token[j] == x) r = 0.0;
    }
    return r;
}

// NV steps of a warp's range, as a lane holds them: 4 indices of each.
template <int NV>
struct Tile {
    double r[NV][4];
    alignas(16) float q[NV][4];

    __device__ __forceinline__ void load(const float* p, const float* dq, int first, int hi, bool wide) {
        wide = wide && first + (NV - 1) * kStep + 4 <= hi;
        if (dq) {
            if (wide) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    *reinterpret_cast<float4*>(q[i]) = *reinterpret_cast<const float4*>(dq + first + i * kStep);
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) fetch(q[i], dq, first + i * kStep, hi);
            }
        }
        constexpr int kFly = NV < 4 ? NV : 4;
#pragma unroll
        for (int h = 0; h < NV; h += kFly) {
            alignas(16) float a[kFly][4];
#pragma unroll
            for (int i = 0; i < kFly; ++i) {
                if (wide)
                    *reinterpret_cast<float4*>(a[i]) = *reinterpret_cast<const float4*>(p + first + (h + i) * kStep);
                else
                    fetch(a[i], p, first + (h + i) * kStep, hi);
            }
#pragma unroll
            for (int i = 0; i < kFly; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) r[h + i][e] = prob(a[i][e]);
        }
    }
    static __device__ __forceinline__ void fetch(float (&d)[4], const float* s, int x, int hi) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = x + e < hi ? s[x + e] : 0.0f;
    }
    __device__ __forceinline__ void reject(bool drawn, double mass, int token, int first) {
        if (drawn) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) r[i][e] = fmax(r[i][e] - mass * prob(q[i][e]), 0.0);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (first + i * kStep + e == token) r[i][e] = 0.0;
        }
    }
    __device__ __forceinline__ double step_sum(int i) const {
        return (r[i][0] + r[i][1]) + (r[i][2] + r[i][3]);
    }
    __device__ __forceinline__ double sum() const {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i) s += step_sum(i);
        return s;
    }
};

// The place of the first of the lanes' values at which the running sum, from base on,
// passes goal; the last one with mass if none does; -1 without any.  base becomes the
// sum before that place.
__device__ __forceinline__ int place(double v, double goal, int lane, double& base) {
    const double inc = warp_prefix(v, lane);
    const unsigned has = __ballot_sync(0xffffffffu, v > 0.0);
    const unsigned over = __ballot_sync(0xffffffffu, v > 0.0 && base + inc > goal);
    if (!has) return -1;
    const int at = over ? __ffs(over) - 1 : 31 - __clz(has);
    const double upto = __shfl_sync(0xffffffffu, inc, at > 0 ? at - 1 : 0);
    if (at > 0) base += upto;
    return at;
}

// kResident: a warp's range is one tile, kept from pass to pass.
template <int NV, bool kResident>
__global__ void __launch_bounds__(kThreads)
    tree_verify_kernel(const float* P, int64_t ldp, const float* Qd, int64_t ldq, int V, int T, const int32_t* tokens,
                       const int32_t* parents, const float* u, int32_t* path, int32_t* emitted, int32_t* count,
                       int per_warp, bool wide) {
    __shared__ int par[kTreeMax], tok[kTreeMax], way[kTreeMax];
    __shared__ double pv[kTreeMax], qv[kTreeMax], uv[kTreeMax];
    __shared__ Rejections w;
    __shared__ double part[2][kAll];  // [pass parity]: the sums of all warps of the sequence
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;
    const bool drawn = Qd != nullptr;
    const size_t node0 = (size_t)b * T;
    pdl_wait();
    pdl_launch_dependents();
    if (tid < T) {
        const int p = parents[node0 + tid], x = tokens[node0 + tid];
        const bool ok = tid > 0 && p >= 0 && p < tid && x >= 0 && x < V;
        par[tid] = tid == 0 ? p : ok ? p : -1;  // a node that cannot be tested hangs nowhere
        tok[tid] = x;
        pv[tid] = ok ? prob(P[(node0 + p) * ldp + x]) : 0.0;
        qv[tid] = ok && drawn ? prob(Qd[(node0 + p) * ldq + x]) : 1.0;
        uv[tid] = (double)u[node0 + tid];
    }
    if (tid == 0) way[0] = 0, w.mass[0] = 1.0;
    cluster_meet();  // every CTA of the cluster runs, its shared memory can be written
    if (par[0] != -1) {  // an empty slot of the batch
        if (rank == 0) {
            if (tid < T) path[node0 + tid] = emitted[node0 + tid] = -1;
            if (tid == 0) count[b] = 0;
        }
        return;  // all 8 CTAs of the cluster
    }

    const int me = rank * kWarps + warp;
    // this warp's indices; ranges past the end are empty (V <= 2^24, so the product fits)
    const int lo = me * per_warp, hi = min(V, lo + per_warp), first = lo + lane * 4;
    Tile<NV> tile;
    int v = 0, n = 0, found = 1, passes = 0;
    double total = 0.0;
    bool loaded = false;  // the tile holds R of node v after n rejections
    bool summed = false;  // part and total hold the sums of the current R

    auto fill = [&](int start, int n_rej) {
        const float* p = P + (node0 + v) * ldp;
        const float* q = drawn ? Qd + (node0 + v) * ldq : nullptr;
        tile.load(p, q, start, hi, wide);
        for (int j = 0; j < n_rej; ++j) tile.reject(drawn, w.mass[j], w.token[j], start);
    };
    // the sum of R over the vocabulary, rejections 0 .. n_rej-1 applied
    auto pass = [&](int n_rej) -> double {
        double acc = 0.0;
        if (kResident) {
            if (!loaded) {
                fill(first, n_rej);
            } else if (n_rej > n) {
                tile.reject(drawn, w.mass[n], w.token[n], first);
            }
            loaded = true;
            acc = tile.sum();
        } else {
            for (int s = first; s - lane * 4 < hi; s += NV * kStep) {
                fill(s, n_rej);
                acc += tile.sum();
            }
        }
        acc = warp_sum(acc);
        double* const slot = part[passes & 1];  // the other one may still be read by a slower CTA
        if (lane < kCtas) st_shared_cluster_f64(mapa_shared(smem_addr(&slot[me]), lane), acc);
        cluster_meet();
        double t = 0.0;
#pragma unroll
        for (int i = 0; i < kAll / 32; ++i) t += slot[lane * (kAll / 32) + i];
        ++passes;
        return warp_sum(t);
    };

    // children after their parents and in order: one sweep over the nodes walks the tree;
    // every thread of the cluster takes the same steps on the same values.  c = T: the sums
    // of the last node, where its rejections have not left them.
    for (int c = 1; c <= T; ++c) {
        if (c < T) {
            if (par[c] != v) continue;
            const double r = remaining(pv[c], qv[c], tok[c], drawn, n, w);
            if (uv[c] * qv[c] * w.mass[n] < r) {
                if (tid == 0) way[found] = c;
                v = c;
                ++found;
                n = 0;
                loaded = summed = false;
                continue;
            }
            __syncthreads();  // the tests that read the list are done
            if (tid == 0) w.token[n] = tok[c];
            __syncthreads();
        } else if (summed) {
            break;
        }
        const double t = pass(c < T ? n + 1 : n);
        if (c == T) {
            total = t;
        } else if (t > 0.0) {
            ++n;
            total = t;
            summed = true;
            if (tid == 0 && n < kTreeMax) w.mass[n] = t;
            __syncthreads();
        } else {
            loaded = summed = false;  // the draft covered all that was left: the rejection takes nothing away
        }
    }

    // the next token: the warp, then its step, lane and index where the running sum passes u_0
    const double goal = (uv[0] > 0.0 ? uv[0] : 0.0) * total;
    const double* slot = part[(passes - 1) & 1];
    double base = 0.0, mine = 0.0;
#pragma unroll
    for (int i = 0; i < kAll / 32; ++i) mine += slot[lane * (kAll / 32) + i];
    int owner = place(mine, goal, lane, base);
    if (owner >= 0) {
        int pick = -1;
        double upto = base, before = base;
        for (int i = 0; i < kAll / 32; ++i) {
            const double s = slot[owner * (kAll / 32) + i];
            if (s > 0.0 && !(pick >= 0 && upto > goal)) pick = i, before = upto;  // the last one with mass if none passes
            upto += s;
        }
        owner = owner * (kAll / 32) + pick;
        base = before;
    }
    __syncthreads();  // way is written
    if (rank == 0) {
        if (tid < T) {
            path[node0 + tid] = tid < found ? way[tid] : -1;
            if (tid < found - 1)
                emitted[node0 + tid] = tok[way[tid + 1]];
            else if (tid >= found || owner < 0)
                emitted[node0 + tid] = -1;
        }
        if (tid == 0) count[b] = found;
    }
    if (me != owner) return;

    int start = first;
    if (!kResident) {  // the tile, the last one with mass if none passes
        double run = base, before = base;
        int held = -1;
        bool over = false;
        for (int s = first; !over && s - lane * 4 < hi; s += NV * kStep) {
            fill(s, n);
            const double t = warp_sum(tile.sum());
            if (t > 0.0) start = held = s, before = run;
            run += t;
            over = t > 0.0 && run > goal;
        }
        base = before;
        if (!over && held >= 0) fill(held, n);
    }
    double sums[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) sums[i] = warp_sum(tile.step_sum(i));
    double run = base, x[4] = {0.0, 0.0, 0.0, 0.0};
    int step = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (sums[i] > 0.0 && !(step >= 0 && run > goal)) {
            step = i, base = run;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = tile.r[i][e];
        }
        run += sums[i];
    }
    const int at = place((x[0] + x[1]) + (x[2] + x[3]), goal, lane, base);
    if (lane == at) {
        int pick = 0;
        run = base;
        bool over = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            run += x[e];
            if (x[e] > 0.0 && !over) pick = e, over = run > goal;
        }
        emitted[node0 + found - 1] = start + step * kStep + pick;
    }
}

template <int NV, bool kResident>
cudaError_t launch(cudaLaunchConfig_t& cfg, const float* P, int64_t ldp, const float* Qd, int64_t ldq, int V, int T,
                   const int32_t* tokens, const int32_t* parents, const float* u, int32_t* path, int32_t* emitted,
                   int32_t* count, int per_warp, bool wide) {
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel<NV, kResident>, P, ldp, Qd, ldq, V, T, tokens, parents, u, path, emitted,
                              count, per_warp, wide);
}

}  // namespace

cudaError_t launch_tree_verify(const float* P, int64_t ldp, const float* Qd, int64_t ldq, int B, int T, int V,
                               const int32_t* tokens, const int32_t* parents, const float* u, int32_t* path,
                               int32_t* emitted, int32_t* count, cudaStream_t stream) {
    const bool wide = (reinterpret_cast<uintptr_t>(P) & 15) == 0 && ldp % 4 == 0 &&
                     (!Qd || ((reinterpret_cast<uintptr_t>(Qd) & 15) == 0 && ldq % 4 == 0));
    // whole steps per warp, so that a warp's range starts on a 16-byte boundary
    const int per_warp = ((V + kAll - 1) / kAll + kStep - 1) / kStep * kStep;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)B * kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const auto run = per_warp <= kStep       ? launch<1, true>
                     : per_warp <= 2 * kStep ? launch<2, true>
                     : per_warp <= 4 * kStep ? launch<4, true>
                     : per_warp <= 8 * kStep ? launch<8, true>
                                             : launch<4, false>;
    return run(cfg, P, ldp, Qd, ldq, V, T, tokens, parents, u, path, emitted, count, per_warp, wide);
}

}  // namespace rmm
