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
// One cluster of 8 CTAs per sequence.  The tests need one probability each,
// fetched up front for all nodes; a pass over the vocabulary runs only for a
// rejection, and for the next token where the walk ends on an accepted node.
// R is never stored: a pass forms it again from the rows and the masses of the
// rejections before it.  Each pass leaves the sum of every warp's own range of
// indices, so the next token is found by walking the 8 CTAs' sums, 16 warps'
// sums and one warp's range.
#include <math.h>

#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;

__device__ __forceinline__ double ld_shared_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// a probability as the walk reads it: NaN and negative values count as 0
__device__ __forceinline__ double prob(float p) { return p > 0.0f ? (double)p : 0.0; }

struct Walk {
    double mass[kTreeMax + 1];  // Z before each rejection at the current node, then the current Z
    int rejected[kTreeMax];     // their tokens
};

// R at index i, given the rows' values there and the rejections so far.
__device__ __forceinline__ double remaining(double r, double q, int i, bool drawn, int n, const Walk& w) {
    if (drawn) {
        for (int j = 0; j < n; ++j) r = fmax(r - w.mass[j] * q, 0.0);
    } else {
        for (int j = 0; j < n; ++j)
            if (w.rejected[j] == i) r = 0.0;
    }
    return r;
}

__global__ void __launch_bounds__(kThreads)
    tree_verify_kernel(const float* P, int64_t ldp, const float* Qd, int64_t ldq, int V,
                       int T, const int32_t* tokens, const int32_t* parents,
                       const float* u, int32_t* path, int32_t* emitted,
                       int32_t* count, int per_warp, int wide) {
    __shared__ int par[kTreeMax], tok[kTreeMax], way[kTreeMax];
    __shared__ double pv[kTreeMax], qv[kTreeMax], uv[kTreeMax];
    __shared__ Walk w;
    __shared__ double warp_part[kWarps];
    __shared__ double cta_part[2];
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
    __syncthreads();
    if (par[0] != -1) {  // an empty slot of the batch
        if (rank == 0) {
            if (tid < T) path[node0 + tid] = emitted[node0 + tid] = -1;
            if (tid == 0) count[b] = 0;
        }
        return;  // all 8 CTAs of the cluster
    }

    const int lo = (rank * kWarps + warp) * per_warp, hi = min(V, lo + per_warp);  // this warp's indices
    int v = 0, n = 0, found = 1, passes = 0;
    double total = 0.0;
    bool summed = false;  // warp_part and total hold the sums of the current R

    // the sum of R over the vocabulary, rejections 0 .. n-1 applied
    auto pass = [&](int n_rej) -> double {
        const float* p = P + (node0 + v) * ldp;
        const float* q = drawn ? Qd + (node0 + v) * ldq : p;
        double acc = 0.0;
        if (wide) {
            for (int i = lo + lane * 4; i < hi; i += 128) {
                if (i + 4 <= hi) {
                    const float4 a = *reinterpret_cast<const float4*>(p + i);
                    const float4 c = drawn ? *reinterpret_cast<const float4*>(q + i) : a;
                    acc += remaining(prob(a.x), prob(c.x), i, drawn, n_rej, w);
                    acc += remaining(prob(a.y), prob(c.y), i + 1, drawn, n_rej, w);
                    acc += remaining(prob(a.z), prob(c.z), i + 2, drawn, n_rej, w);
                    acc += remaining(prob(a.w), prob(c.w), i + 3, drawn, n_rej, w);
                } else {
                    for (int e = i; e < hi; ++e) acc += remaining(prob(p[e]), prob(q[e]), e, drawn, n_rej, w);
                }
            }
        } else {
            for (int i = lo + lane; i < hi; i += 32) acc += remaining(prob(p[i]), prob(q[i]), i, drawn, n_rej, w);
        }
        acc = warp_sum(acc);
        __syncthreads();  // the sums of the pass before have been read
        if (lane == 0) warp_part[warp] = acc;
        __syncthreads();
        double s = 0.0;
        for (int i = 0; i < kWarps; ++i) s += warp_part[i];
        double* slot = &cta_part[passes & 1];  // read by the cluster until its next barrier
        if (tid == 0) *slot = s;
        cluster_sync();
        double t = 0.0;
        for (int j = 0; j < kCtas; ++j) t += ld_shared_cluster_f64(mapa_shared(smem_addr(slot), j));
        ++passes;
        return t;
    };

    if (tid == 0) {
        way[0] = 0;
        w.mass[0] = 1.0;
    }
    __syncthreads();
    // children after their parents and in order: one sweep over the nodes walks the tree;
    // every thread of the cluster takes the same steps on the same values
    for (int c = 1; c < T; ++c) {
        if (par[c] != v) continue;
        const double r = remaining(pv[c], qv[c], tok[c], drawn, n, w);
        if (uv[c] * qv[c] * w.mass[n] < r) {
            v = c;
            n = 0;
            summed = false;
            __syncthreads();
            if (tid == 0) {
                way[found] = c;
                w.mass[0] = 1.0;
            }
            ++found;
            __syncthreads();
        } else {
            __syncthreads();
            if (tid == 0) w.rejected[n] = tok[c];
            __syncthreads();
            const double t = pass(n + 1);
            if (t > 0.0) {
                ++n;
                total = t;
                summed = true;
                if (tid == 0) w.mass[n] = t;
                __syncthreads();
            } else {
                summed = false;  // the draft covered all that was left: the rejection takes nothing away
            }
        }
    }
    if (!summed) total = pass(n);

    // the next token: the CTA, then the warp, then the index where the running sum passes u_0
    double goal = (uv[0] > 0.0 ? uv[0] : 0.0) * total;
    const uint32_t my_slot = smem_addr(&cta_part[(passes - 1) & 1]);
    int owner = -1;
    double before = 0.0, run = 0.0;
    for (int j = 0; j < kCtas; ++j) {
        const double s = ld_shared_cluster_f64(mapa_shared(my_slot, j));
        if (s > 0.0 && !(owner >= 0 && run > goal)) owner = j, before = run;  // the last one with mass if none passes
        run += s;
    }
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
    if (rank == owner) {
        int ow = -1;
        double wb = before, wr = before;
        for (int i = 0; i < kWarps; ++i) {
            const double s = warp_part[i];
            if (s > 0.0 && !(ow >= 0 && wr > goal)) ow = i, wb = wr;
            wr += s;
        }
        if (warp == ow) {
            const float* p = P + (node0 + v) * ldp;
            const float* q = drawn ? Qd + (node0 + v) * ldq : p;
            double base = wb;
            int last = -1;
            bool done = false;
            for (int i0 = lo; i0 < hi && !done; i0 += 32) {
                const int i = i0 + lane;
                const double x = i < hi ? remaining(prob(p[i]), prob(q[i]), i, drawn, n, w) : 0.0;
                double inc = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned has = __ballot_sync(0xffffffffu, x > 0.0);
                const unsigned over = __ballot_sync(0xffffffffu, x > 0.0 && base + inc > goal);
                if (over) {
                    last = i0 + __ffs(over) - 1;
                    done = true;
                } else if (has) {
                    last = i0 + 31 - __clz(has);
                }
                base += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) emitted[node0 + found - 1] = last;
        }
    }
    cluster_sync();  // no CTA leaves while another still reads its sums
}

}  // namespace

cudaError_t launch_tree_verify(const float* P, int64_t ldp, const float* Qd, int64_t ldq, int B, int T, int V,
                               const int32_t* tokens, const int32_t* parents, const float* u, int32_t* path,
                               int32_t* emitted, int32_t* count, cudaStream_t stream) {
    const int wide = (reinterpret_cast<uintptr_t>(P) & 15) == 0 && ldp % 4 == 0 &&
                     (!Qd || ((reinterpret_cast<uintptr_t>(Qd) & 15) == 0 && ldq % 4 == 0));
    // whole 128-index steps per warp, so that a warp's range starts on a 16-byte boundary
    const int per_warp = ((V + kCtas * kWarps - 1) / (kCtas * kWarps) + 127) / 128 * 128;
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
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel, P, ldp, Qd, ldq, V, T, tokens, parents, u, path, emitted,
                              count, per_warp, wide);
}

}  // namespace rmm
