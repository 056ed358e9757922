// rmm_attn_tree.cu -- reduced attention of draft trees over the caches of a
// batch of sequences with their own lengths, on the tensor cores.
//
// Sequence b has len_b cached keys and T <= 64 tree nodes whose keys sit at the
// slots len_b .. len_b + T - 1.  For KV head g, its G query heads and T nodes
// stack into R = G T rows that share every key and value:
//   S   = the k dims with the largest max over the present rows of |Q[row,j]|
//   x_l = scale * sum_{j in S} Q[row,j] K[l,j]     for l < len_b and for the slots
//         of the row's node and its ancestors
//   O   = softmax(x) V, zero where the row sees no key
//
// What bounds it: K^T (its kept rows) and V are read once per (sequence, KV
// head), 2 (k + 128) bytes a key, against 2 R (k + 128) products a key: memory
// up to about R = 250 rows, the tensor cores and the softmax beyond.  So the rows
// are stacked, up to 256 to a CTA, and the keys are split.
//
// Work: a unit is (sequence, KV head, pair of 128-row tiles); its keys come in
// blocks of 64.  All units, in order, are cut into shares of equal cost, one per
// CTA (one CTA per SM), wherever the cuts fall: ragged batches balance and few
// units still fill the GPU.  A unit costs its blocks and a constant for its start
// and end.  A unit inside one share is finished there; one that was cut leaves
// fp32 partials (maximum, sum, unnormalised output), at most two per CTA, which a
// second kernel joins.  Lengths are read on the device only, so a captured call
// serves any lengths.
//
// Two softmax groups of four warps (a thread per row) alternate on the tensor
// cores: with two row tiles each group has its own tile and both use every key
// block; with one, the groups take alternate key blocks of the same rows, each
// with its own maximum, sum and output, joined at the end of the unit.
//
//   warps 0-7  softmax: S from TMEM, mask, running maximum, P (bf16) over S's own
//              columns, O rescaled only when the maximum grew by more than 2^8;
//              the query operand at the start of a unit, its output at the end
//   warps 8, 9 MMA, a warp for each group: S = Q_S K_S^T for the group's next step
//              as soon as its P.V is done, P.V (A from TMEM) as soon as its P is written
//   warp 10    key and value blocks by tile copies through two rings, running ahead
//              over units
//   12-15      (fewer dims kept) the kept rows of K^T gathered from the d-major cache
//
// Operands in shared memory are 128-byte swizzled: K and V MN-major as the
// caches lay them out, Q K-major (a tile copy) or, gathered, MN-major.  TMEM
// holds S0, S1, O0, O1 (128 columns each).  Value rows past a sequence's slots
// are zeroed in shared memory before P.V: 0 times what they hold could be NaN.
// A row that sees no key has the sum 0 and the output 0; a NaN sum (a NaN or +inf logit)
// is the row's answer, in whatever piece it arose.
// Every wait is bounded: on expiry the kernel records RMM_ERR_TIMEOUT, all roles
// leave their loops, copies and MMAs in flight drain, TMEM is freed.
//
// Measured (whole calls in long rows, on changing inputs): 32 sequences x 8k keys, one
// node, every dim 115 us, 5.1 TB/s of the keys and values (104 and 5.7 in a row of 60);
// 8 x 16k, 25 nodes, half of the dims 70 us (5.7 TB/s in the main loop); 4 x 32k, 64
// nodes of 8 heads per KV head, every dim 311 us, 845 TFLOP/s, the tensor cores 50 %
// busy and the clock at 1.5 GHz; 1 x 2k, 16 nodes 22 us, three kernels' latency.
// Fewer dims save bytes of K^T but bring the selection and the gather: 25 nodes at a
// quarter, a half, three quarters, all of the dims 64, 69, 74, 68 us, one node of
// 32 x 8k 103, 102, 102, 104.
// Of a step of two groups the products take 1261 cycles alone, whatever the softmax
// does beside them, and 2000 with it.
#include <math.h>

#include "rmm_common.cuh"
#include "rmm_internal.h"
#include "rmm_tree.cuh"

namespace rmm {

namespace {

constexpr int D = 128;
constexpr int BM = 128;  // rows per tile (= TMEM lanes)
constexpr int BK = 64;   // keys per block: the step of S, softmax and P.V
constexpr int kMaxStages = 8;
constexpr int kSoftmaxThreads = 256;
constexpr int kMmaWarp = 8, kTmaWarp = 10;  // MMA warps 8 and 9: one per group
constexpr int kGatherWarp = 12, kGatherWarps = 4;  // key rows, when not every dim is kept
constexpr int tree_threads(bool all) { return 32 * (all ? kGatherWarp : kGatherWarp + kGatherWarps); }
constexpr int V_CHUNK = BK * 128;  // 64 dims of a value block (bytes)
constexpr int V_BYTES = 2 * V_CHUNK;
constexpr uint32_t TM_O = 256;  // S of group a at 128 a (two buffers), O of group a at 256 + 128 a
constexpr float kRescaleLog2 = 8.0f;
// Blocks that the start and the end of a unit's piece take the time of, in the share of work that
// a CTA gets (every dim kept, us for 32 x 8k decode: 112 without, 104 at 3, 103 at 6, 104 at 10;
// fewer kept, tree of 25 over 8 x 16k: 79 without, 73.5 at 3, 71.5 at 6, 70 at 10).
__host__ __device__ constexpr int piece_cost(bool all) { return all ? 6 : 10; }
constexpr int kMaxSide = 8;
constexpr int kSmemMax = 232448;  // 227 KB

struct __align__(8) TreeBars {
    uint64_t q_full, o_full, drain;
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t v_full[kMaxStages], v_empty[kMaxStages];
    uint64_t s_full[2][2], p_full[2][2];  // [group][buffer]
    uint64_t pv_done[2];
    uint64_t meet;  // all softmax warps
    uint64_t never;  // watchdog self-test: nothing ever arrives here
    int seg_b, seg_u, seg_x, cost, piece;  // the CTA's share: where it starts, and how much it is
    uint32_t tmem_base;
    int abort_flag;
};

struct TreeArgs {
    const uint16_t *Q, *Kt;
    const int32_t *lens, *parents;
    int32_t* idx;  // kept sets [B * Hkv * k]
    uint16_t* O;
    float* partials;
    long long* cum;  // [B + 1]: cost of the sequences before b; then how many shares, and the cost of a piece
    int* status;
    int B, Hkv, G, T, ldL, R, nrt, nrp, k, kp, nk, nv, slot_rows;
    int side, U;  // row pairs that CTAs of their own take side by side (or 1), units of a sequence then
    int identity;    // every dim kept
    int debug_timeout;
    float scale_log2;
};

__device__ __forceinline__ int blocks_of(const TreeArgs& a, int b) {
    const int len = a.lens[b];
    return len < 0 || len > a.ldL - a.T ? 0 : (len + a.T + BK - 1) / BK;
}

// KV head and row pair of unit u of a sequence.
__device__ __forceinline__ int head_of(const TreeArgs& a, int u) { return a.side > 1 ? u : u / a.nrp; }
__device__ __forceinline__ int pair_of(const TreeArgs& a, int u) { return a.side > 1 ? blockIdx.x % a.side : u % a.nrp; }

// A CTA's share as its roles walk it, one piece of a unit at a time.  A unit of nb blocks
// costs nb + piece: the places [0, piece) stand for the start and end of its pieces, place
// piece + i for block i.
struct Share {
    // blk, n: the piece's first block and how many, nb: of the whole unit
    int b = 0, u = 0, x = 0, left = 0, cost = 0, blk = 0, n = 0, nb = 0;
    __device__ __forceinline__ bool next(const TreeArgs& a, const TreeBars* s, bool first) {
        if (first) {
            b = s->seg_b, u = s->seg_u, x = s->seg_x, left = s->cost;
            if (left <= 0) return false;
            nb = blocks_of(a, b);
        } else {
            left -= cost;
            if (left <= 0) return false;
            x = 0;
            if (++u == a.U) {
                u = 0;
                do nb = blocks_of(a, ++b);
                while (nb == 0);  // left > 0: a later sequence has blocks
            }
        }
        cost = min(nb + s->piece - x, left);
        blk = max(x - s->piece, 0);
        n = x + cost - s->piece - blk;
        return n > 0;  // a share may end before a unit's first block
    }
};

// A place in a ring of stages: its slot and the parity of its round (attn_tree_rings says what
// depths the parity allows).
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int by, int n) {  // by <= n
        slot += by;
        if (slot >= n) slot -= n, phase ^= 1u;
    }
};

// floats of one partial: O in pieces of four dims [32][rows][4], then maxima, then sums
__host__ __device__ constexpr size_t slot_floats(int rows) { return (size_t)rows * (D + 2); }

// what the row of a node sees of the 32 keys from `key0` on, as a bit mask
__device__ __forceinline__ uint32_t sees32(uint64_t way, int key0, int len) {
    const int at = key0 - len;  // slot of the first of them in the tree
    if (at <= -32) return way ? 0xFFFFFFFFu : 0u;
    if (at >= 0) return at < 64 ? (uint32_t)(way >> at) : 0u;
    return ((uint32_t)(way << -at)) | (way ? (1u << -at) - 1u : 0u);
}

// -inf for the keys from key0 on that the row does not see
__device__ __forceinline__ void hide(uint32_t (&x)[2][32], uint64_t way, int key0, int len) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint32_t see = sees32(way, key0 + q * 32, len);
#pragma unroll
        for (int c = 0; c < 32; ++c)
            if (!((see >> c) & 1u)) x[q][c] = 0xFF800000u;
    }
}

// the largest of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The exponentials' instructions in the order written: left to itself the compiler put each
// sum right behind its exponential, and a warp waited 1100 cycles for 64 of them instead of 610.
__device__ __forceinline__ float exp2_here(float x) {
    float y;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ F2 fma2_here(F2 a, F2 b, F2 c) {
    F2 r;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2_here(F2 a, F2 b) {
    F2 r;
    asm volatile("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// p = 2^(x scale - m) for 64 logits of a row, their sum in 32 bits, and P to the 32
// columns at pcol, rounded to bf16, V's type, since a product's operands have one type
// (against 64 bits the outputs are off by 0.0023 of their norm, with P in 32 bits by
// 0.0017, which is their own rounding).  kBatch exponentials are on their way while those before are summed.
__device__ __forceinline__ float exp_block(uint32_t (&x)[2][32], float scale_log2, float neg_m, uint32_t pcol) {
    constexpr int kBatch = 16;
    F2 sum[4] = {F2(0.f, 0.f), F2(0.f, 0.f), F2(0.f, 0.f), F2(0.f, 0.f)};
    const F2 scale(scale_log2, scale_log2), shift(neg_m, neg_m);
    uint32_t pk[2][16];
#pragma unroll
    for (int b = 0; b <= 64; b += kBatch) {
#pragma unroll
        for (int c = b; c < b + kBatch && b < 64; c += 2) {
            uint32_t &u0 = x[c >> 5][c & 31], &u1 = x[c >> 5][(c & 31) + 1];
            float z0, z1;
            fma2_here(F2(__uint_as_float(u0), __uint_as_float(u1)), scale, shift).get(z0, z1);
            u0 = __float_as_uint(z0), u1 = __float_as_uint(z1);
        }
#pragma unroll
        for (int c = b; c < b + kBatch; c += 2) {
            if (b < 64) {
                uint32_t &u0 = x[c >> 5][c & 31], &u1 = x[c >> 5][(c & 31) + 1];
                u0 = __float_as_uint(exp2_here(__uint_as_float(u0)));
                u1 = __float_as_uint(exp2_here(__uint_as_float(u1)));
            }
            if (b > 0) {
                const int d = c - kBatch;
                const float p0 = __uint_as_float(x[d >> 5][d & 31]), p1 = __uint_as_float(x[d >> 5][(d & 31) + 1]);
                sum[(d >> 1) & 3] = add2_here(sum[(d >> 1) & 3], F2(p0, p1));
                pk[d >> 5][(d & 31) >> 1] = pack2(p0, p1);
            }
        }
        if (b == 32) tmem_st_32x32b_x16(pcol, pk[0]);
        if (b == 64) tmem_st_32x32b_x16(pcol + 16, pk[1]);
    }
    float s0, s1;
    add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])).get(s0, s1);
    return s0 + s1;
}

// umma_f16, umma_f16_tmem_a and umma_commit by one thread of a converged warp (the
// same one each time).
__device__ __forceinline__ void umma_f16_elect(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_f16_tmem_a_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                      uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// kAll: every head dimension kept (Q a tile copy, K-major; key blocks tile copies).
template <bool kAll>
__global__ void __launch_bounds__(tree_threads(kAll), 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const TreeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const int kp = kAll ? D : a.kp;
    const int Q_BYTES = kp * 256, K_BYTES = kp * 128;  // a query tile, a key block
    uint8_t* sV = smem;
    uint8_t* sK = sV + a.nv * V_BYTES;
    uint8_t* sQ = sK + a.nk * K_BYTES;
    TreeBars* bars = reinterpret_cast<TreeBars*>(sQ + (a.nrt > 1 ? 2 : 1) * Q_BYTES);
    int32_t* par = reinterpret_cast<int32_t*>(bars + 1);
    volatile int* abort_flag = &bars->abort_flag;
    int* status = a.status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int users = a.nrt > 1 ? 2 : 1;  // groups that release a block
    if (tid == 0) {
        mbar_init(smem_addr(&bars->q_full), kAll ? 1 : kSoftmaxThreads);
        mbar_init(smem_addr(&bars->o_full), 2);
        mbar_init(smem_addr(&bars->drain), 2);
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(smem_addr(&bars->k_full[s]), kAll ? 1 : 32 * kGatherWarps);  // a tile's bytes, or the threads' copies
            mbar_init(smem_addr(&bars->k_empty[s]), users);
            mbar_init(smem_addr(&bars->v_full[s]), 1);
            mbar_init(smem_addr(&bars->v_empty[s]), users);
        }
        for (int s = 0; s < 2; ++s) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(smem_addr(&bars->s_full[s][h]), 1);
                mbar_init(smem_addr(&bars->p_full[s][h]), 4);
            }
            mbar_init(smem_addr(&bars->pv_done[s]), 1);
        }
        mbar_init(smem_addr(&bars->meet), 8);
        mbar_init(smem_addr(&bars->never), 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_addr(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (tid == 32 * kTmaWarp) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        tma_prefetch_desc(&qmap);
    }
    // Lengths, trees, queries and caches come from kernels before this call, the kept sets from the
    // one before.  Nothing is read ahead of this wait: that the kept sets' kernel has waited for the
    // others makes their writes visible to it, not to this grid.
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        // the CTA's share of the whole cost, and where it starts; the last CTA also leaves the
        // running costs for the joining kernel
        const int U = a.U, c = blockIdx.x / a.side;
        const bool last = blockIdx.x == gridDim.x - 1;
        long long blocks = 0, seqs = 0;
        const int mine = lane < a.B ? blocks_of(a, lane) : 0;  // of the first 32 sequences
        for (int b = lane; b < a.B; b += 32) {
            const int nb = b == lane ? mine : blocks_of(a, b);
            blocks += nb;
            seqs += nb > 0;
            if (blockIdx.x == 0 && a.lens[b] > a.ldL - a.T) record_status(status, RMM_ERR_INVALID_ARG);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
            seqs += __shfl_xor_sync(0xffffffffu, seqs, o);
        }
        // shares of more than piece_cost + 1, and never more of them than blocks: none is empty
        const long long C = min((long long)(gridDim.x / a.side), blocks * U);
        const int piece = blocks * U >= C * (2 * piece_cost(kAll)) ? piece_cost(kAll) : 0;
        const long long total = (blocks + seqs * piece) * U;
        const long long p0 = c < C ? total * c / C : total, p1 = c < C ? total * (c + 1) / C : total;
        long long base = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            const int nb = b0 == 0 ? mine : b < a.B ? blocks_of(a, b) : 0;
            const long long n = nb ? (long long)(nb + piece) * U : 0;
            long long end = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += v;
            }
            end += base;
            if (last && b < a.B) {
                a.cum[b + 1] = end;
                if (b == 0) a.cum[0] = 0;
            }
            if (p0 < end && p0 >= end - n) {  // one lane of one round
                const uint32_t in = (uint32_t)(p0 - (end - n));  // below U (ldL / BK + piece_cost) < 2^32
                bars->seg_b = b;
                bars->seg_u = (int)(in / (uint32_t)(nb + piece));
                bars->seg_x = (int)(in % (uint32_t)(nb + piece));
            }
            base = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) {
            bars->cost = (int)(p1 - p0);
            bars->piece = piece;
            if (last) a.cum[a.B + 1] = C, a.cum[a.B + 2] = piece;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    Share w;
    // With the gather warps the block has 512 threads of 128 registers; a softmax thread holds 64
    // logits and wants more.  256 x 184 + 256 x 64 = 63488 of the 65536.
    if (warp < kMmaWarp) {
        if (!kAll) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ------------------------------------------------------------ softmax, query operand, output
        const int grp = warp >> 2, i = tid & 127;  // group, row of the tile = TMEM lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + lane_base + grp * 128, meet = smem_addr(&bars->meet);
        float* xch = reinterpret_cast<float*>(sQ);  // maxima and sums of the two groups (sQ is free by then)
        int piece = 0, meets = 0, queries = 0;
        Ring v0;  // the piece's first block in the value ring
        const uint32_t s_full = smem_addr(&bars->s_full[grp][0]), p_full = smem_addr(&bars->p_full[grp][0]);
        const uint32_t pv_done = smem_addr(&bars->pv_done[grp]);
        uint32_t blocks = 0;  // of this group, over all pieces: a block's buffer is blocks & 1
        // all softmax warps meet (bounded)
        auto together = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(meet);
            return __all_sync(0xffffffffu, mbar_wait(meet, (uint32_t)(meets++) & 1u, status, abort_flag));
        };
        // the tree and the query operand of the piece at `w`
        auto open = [&]() {
            const int rp = pair_of(a, w.u), plane = w.b * a.Hkv + head_of(a, w.u);
            const int tiles = 2 * rp + 1 < a.nrt ? 2 : 1;
            const size_t row0 = (size_t)plane * a.R;
            if (a.parents && tid < a.T) par[tid] = a.parents[(size_t)w.b * a.T + tid];
            if (kAll) {
                if (tid == 0) {
                    const uint32_t qf = smem_addr(&bars->q_full), qb = smem_addr(sQ);
                    mbar_arrive_expect_tx(qf, tiles * BM * 256);
                    for (int t = 0; t < tiles; ++t)
                        for (int h = 0; h < 2; ++h)
                            tma_load_2d(qb + t * Q_BYTES + h * BM * 128, &qmap, qf, h * 64,
                                        (int)(row0 + (2 * rp + t) * BM));
                }
                ++queries;
                if (w.blk == 0 && rp == 0 && a.idx && tid < D) a.idx[(size_t)plane * D + tid] = tid;
            } else {
                // a thread turns 8 rows x 8 dims of each tile and puts the kept dims at their places
                const int c = tid & 15, c16 = tid >> 4;
                uint4 v[2][8];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = (2 * rp + t) * BM + c16 * 8 + e;
                        v[t][e] = t < tiles && r < a.R ? *reinterpret_cast<const uint4*>(a.Q + (row0 + r) * D + c * 8)
                                                       : make_uint4(0, 0, 0, 0);
                    }
                const int32_t* S = a.idx + (size_t)plane * a.k;
                int d[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) d[q] = lane + 32 * q < a.k ? S[lane + 32 * q] : -1;
                uint32_t kept = 0;  // the dims of this thread's 32, and how many come before
                int before = 0;
#pragma unroll
                for (int w4 = 0; w4 < 4; ++w4) {
                    uint32_t m = 0;
#pragma unroll
                    for (int q = 0; q < 4; ++q) m |= (d[q] >> 5) == w4 ? 1u << (d[q] & 31) : 0u;
                    m = __reduce_or_sync(0xffffffffu, m);
                    if (w4 < (c >> 2)) before += __popc(m);
                    if (w4 == (c >> 2)) kept = m;
                }
                before += __popc(kept & ((1u << ((c & 3) * 8)) - 1u));
                kept >>= (c & 3) * 8;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= tiles) break;
                    const uint32_t base = smem_addr(sQ + t * Q_BYTES);
                    int j = before;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
                        uint32_t w[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            w[r] = e < 2 ? v[t][r].x : e < 4 ? v[t][r].y : e < 6 ? v[t][r].z : v[t][r].w;
                        if ((kept >> e) & 1u) {
                            st_shared_v4(base + swz(j, c16, kp * 128),
                                         make_uint4(__byte_perm(w[0], w[1], sel), __byte_perm(w[2], w[3], sel),
                                                    __byte_perm(w[4], w[5], sel), __byte_perm(w[6], w[7], sel)));
                            ++j;
                        }
                    }
                    for (j = a.k + c; j < kp; j += 16) st_shared_v4(base + swz(j, c16, kp * 128), make_uint4(0, 0, 0, 0));
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_addr(&bars->q_full));
            }
        };
        bool ok = true;
        bool more = w.next(a, bars, true);
        if (more) open();
        for (; ok && more; ++piece) {
            const int g = head_of(a, w.u), rp = pair_of(a, w.u);
            const bool two = 2 * rp + 1 < a.nrt;
            const int plane = w.b * a.Hkv + g;
            const int len = a.lens[w.b];
            const int tile = 2 * rp + (two ? grp : 0);
            const int row = tile * BM + i;  // of the unit's G * T rows: query head row / T, node row % T
            const size_t row0 = (size_t)plane * a.R;
            if (!together()) break;  // par; and the outputs of the piece before have been read
            uint64_t way = 0;
            if (row < a.R) way = a.parents ? tree_way(par, row % a.T) : chain_way(row % a.T);
            const bool busy = __any_sync(0xffffffffu, row < a.R);  // the warp has rows

            const int mine = two ? w.n : (w.n + 1 - grp) / 2;  // this group's steps
            float m_use = -INFINITY, l = 0.0f;
            Ring v = v0;
            if (!two && grp == 1) v.next(1, a.nv);
            for (int n = 0; n < mine; ++n, ++blocks) {
                const uint32_t buf = blocks & 1u;
                const int key0 = (w.blk + (two ? n : 2 * n + grp)) * BK;
                if (!__all_sync(0xffffffffu, mbar_wait(s_full + buf * 8, (blocks >> 1) & 1u, status, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (busy) {
                    uint32_t x[2][32];
                    tmem_ld_32x32b_x32(s_col + buf * BK, x[0]);
                    tmem_ld_32x32b_x32(s_col + buf * BK + 32, x[1]);
                    tmem_ld_wait();
                    if (key0 + BK > len) hide(x, way, key0, len);  // the block reaches the tree's slots
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mx[q] = __uint_as_float(x[q >> 1][(q & 1) * 16]);
#pragma unroll
                        for (int c = 1; c < 15; c += 2)
                            mx[q] = max3(mx[q], __uint_as_float(x[q >> 1][(q & 1) * 16 + c]),
                                         __uint_as_float(x[q >> 1][(q & 1) * 16 + c + 1]));
                        mx[q] = fmaxf(mx[q], __uint_as_float(x[q >> 1][(q & 1) * 16 + 15]));
                    }
                    const float m_blk = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                    const bool resc = m_blk > m_use + kRescaleLog2;
                    if (__any_sync(0xffffffffu, resc)) {
                        const float m_new = resc ? m_blk : m_use;
                        const float alpha = resc ? exp2f(m_use - m_new) : 1.0f;
                        m_use = m_new;
                        l *= alpha;
                        if (n > 0) {  // O holds the blocks before once the last P.V is done
                            if (!__all_sync(0xffffffffu, mbar_wait(pv_done, (blocks - 1) & 1u, status, abort_flag))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < 8; ++q) {
                                uint32_t o[16];
                                const uint32_t oc = tmem + lane_base + TM_O + grp * D + q * 16;
                                tmem_ld_32x32b_x16(oc, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                                tmem_st_32x32b_x16(oc, o);
                            }
                        }
                    }
                    // P lies over this block's S, whose every column has been read
                    l += exp_block(x, a.scale_log2, m_use == -INFINITY ? 0.0f : -m_use, s_col + buf * BK);
                    tmem_st_wait();
                }
                if (key0 + BK > len) {
                    // slots that no node holds may contain anything: their values become zeros, two
                    // threads per key (with two tiles both groups write the same zeros)
                    const int slot = key0 + (i & 63) - len;
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait(smem_addr(&bars->v_full[v.slot]), v.phase, status, abort_flag))) {
                        ok = false;
                        break;
                    }
                    if (slot >= a.T || (slot >= 0 && a.parents && tree_way(par, slot) == 0)) {
                        const uint32_t vrow = smem_addr(sV + v.slot * V_BYTES) + (i >> 6) * V_CHUNK + (i & 63) * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e) st_shared_v4(vrow + ((e + lane) & 7) * 16, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + buf * 8);
                v.next(two ? 1 : 2, a.nv);
            }
            if (!ok) break;
            for (int j = 0; j < w.n; ++j) v0.next(1, a.nv);
            if (!__all_sync(0xffffffffu,
                            mbar_wait(smem_addr(&bars->o_full), (uint32_t)piece & 1u, status, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (way == 0) m_use = -INFINITY, l = 0.0f;  // an absent node sees nothing
            const bool whole = w.n == w.nb;
            float* slot = a.partials + (size_t)(2 * blockIdx.x + (w.left == bars->cost ? 0 : 1)) * slot_floats(a.slot_rows);
            const bool second = w.n > 1;  // with one tile: group 1 had a block, O1 holds this unit's data
            float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
            if (!two) {  // both groups hold a part of the same rows
                xch[grp * BM + i] = m_use;
                xch[2 * BM + grp * BM + i] = l;
                if (!together()) break;
                m0 = xch[i], m1 = xch[BM + i], l0 = xch[2 * BM + i], l1 = xch[3 * BM + i];
            }
            // the query operand (every S is done), the tree and the exchange are free: the next
            // piece's products start under this one's output
            fence_proxy_async_smem();
            tc_fence_before();
            if (!together()) break;
            tc_fence_after();
            more = w.next(a, bars, false);
            if (more) open();
            if (two) {
                const float inv = 1.0f / l;
                const int sr = grp * BM + i;
                if (!whole && row < a.R) {
                    slot[D * a.slot_rows + sr] = m_use;
                    slot[(D + 1) * a.slot_rows + sr] = l;
                }
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(tmem + lane_base + TM_O + grp * D + q * 32, o);
                    tmem_ld_wait();
                    if (row >= a.R) continue;
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(a.O + (row0 + row) * D + q * 32);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = l == 0.0f ? 0.0f : __uint_as_float(o[v * 8 + e]) * inv;
                            dst[v] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<uint4*>(slot + ((size_t)(q * 8 + v) * a.slot_rows + sr) * 4) =
                                make_uint4(o[v * 4], o[v * 4 + 1], o[v * 4 + 2], o[v * 4 + 3]);
                    }
                }
            } else {
                // join the groups' parts, 64 dims each
                const float M = fmaxf(m0, m1);
                const float w0 = m0 == -INFINITY ? 0.0f : exp2f(m0 - M), w1 = m1 == -INFINITY ? 0.0f : exp2f(m1 - M);
                const float L = w0 * l0 + w1 * l1;
                const float inv = whole ? (L == 0.0f ? 0.0f : 1.0f / L) : 1.0f;
                if (!whole && row < a.R && grp == 0) {
                    slot[D * a.slot_rows + i] = M;
                    slot[(D + 1) * a.slot_rows + i] = L;
                }
#pragma unroll 1
                for (int q = 0; q < 2 && busy; ++q) {
                    uint32_t o0[32], o1[32];
                    const uint32_t oc = tmem + lane_base + TM_O + grp * 64 + q * 32;
                    __syncwarp();
                    tmem_ld_32x32b_x32(oc, o0);
                    if (second) tmem_ld_32x32b_x32(oc + D, o1);
                    tmem_ld_wait();
                    if (row >= a.R) continue;
                    float f[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        // an output that no key went into (weight 0) may hold anything
                        const float u0 = w0 > 0.0f ? __uint_as_float(o0[c]) * w0 : 0.0f;
                        const float u1 = second && w1 > 0.0f ? __uint_as_float(o1[c]) * w1 : 0.0f;
                        f[c] = (u0 + u1) * inv;
                    }
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(a.O + (row0 + row) * D + grp * 64 + q * 32);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            dst[v] = make_uint4(pack_bf16x2(f[v * 8], f[v * 8 + 1]), pack_bf16x2(f[v * 8 + 2], f[v * 8 + 3]),
                                                pack_bf16x2(f[v * 8 + 4], f[v * 8 + 5]), pack_bf16x2(f[v * 8 + 6], f[v * 8 + 7]));
                    } else {
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            *reinterpret_cast<float4*>(slot + ((size_t)(grp * 16 + q * 8 + v) * a.slot_rows + i) * 4) =
                                make_float4(f[v * 4], f[v * 4 + 1], f[v * 4 + 2], f[v * 4 + 3]);
                    }
                }
            }
            tc_fence_before();
        }
        // no query copy may still be landing when the CTA leaves (after an abort)
        if (tid == 0 && queries > 0) {
            volatile int no_abort = 0;
            mbar_wait(smem_addr(&bars->q_full), (uint32_t)(queries - 1) & 1u, status, &no_abort);
        }
        __syncwarp();
    } else if (warp < kGatherWarp) {
        if (!kAll) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kTmaWarp) {
            // ------------------------------------------------------------ value blocks (and key blocks, every dim kept)
            if (lane == 0) {
                int c = 0, c_keys = 0;  // blocks issued, and key blocks (one more after an abort)
                Ring k, v;
                bool ok = true;
                for (bool more = w.next(a, bars, true); ok && more; more = w.next(a, bars, false)) {
                    const int plane = w.b * a.Hkv + head_of(a, w.u);
                    for (int j = 0; j < w.n; ++j, ++c) {
                        const int key0 = (w.blk + j) * BK;
                        if (kAll) {
                            ok = mbar_wait(smem_addr(&bars->k_empty[k.slot]), k.phase ^ 1u, status, abort_flag);
                            if (!ok) break;
                            const uint32_t kf = smem_addr(&bars->k_full[k.slot]);
                            mbar_arrive_expect_tx(kf, K_BYTES);
                            tma_load_3d(smem_addr(sK + k.slot * K_BYTES), &kmap, kf, key0, 0, plane);
                            ++c_keys;
                            k.next(1, a.nk);
                        }
                        ok = mbar_wait(smem_addr(&bars->v_empty[v.slot]), v.phase ^ 1u, status, abort_flag);
                        if (!ok) break;
                        const uint32_t vb = smem_addr(sV + v.slot * V_BYTES), vf = smem_addr(&bars->v_full[v.slot]);
                        mbar_arrive_expect_tx(vf, V_BYTES);
                        tma_load_3d(vb, &vmap, vf, 0, key0, plane);
                        tma_load_3d(vb + V_CHUNK, &vmap, vf, 64, key0, plane);
                        v.next(1, a.nv);
                    }
                }
                // no copy may still be landing when the CTA leaves (after an abort; else all were consumed)
                volatile int no_abort = 0;
                for (int j = max(0, c_keys - a.nk); j < c_keys; ++j)
                    mbar_wait(smem_addr(&bars->k_full[j % a.nk]), (uint32_t)(j / a.nk) & 1u, status, &no_abort);
                for (int j = max(0, c - a.nv); j < c; ++j)
                    mbar_wait(smem_addr(&bars->v_full[j % a.nv]), (uint32_t)(j / a.nv) & 1u, status, &no_abort);
            }
            __syncwarp();
        } else if (warp < kTmaWarp) {
            // ------------------------------------------------------------ MMA issuers: a warp per group
            // The warp stays together and every instruction elects its thread, so that descriptors
            // are computed once for the warp: issued from a branch of one thread, a product took
            // about 110 cycles whatever its size.
            const int g = warp - kMmaWarp;
            const uint32_t idesc_s = idesc_bf16_f32(BM, BK, kAll ? 0 : 1, 1);
            const uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
            const uint64_t qd0 = smem_desc_sw128(smem_addr(sQ), kAll ? 16 : kp * 128, 1024);
            const uint64_t kd0 = smem_desc_sw128(smem_addr(sK), K_BYTES, 1024);
            const uint64_t vd0 = smem_desc_sw128(smem_addr(sV), V_CHUNK, 1024);
            const uint32_t s_tm = tmem + g * 128, o_tm = tmem + TM_O + g * D;
            const uint32_t s_full = smem_addr(&bars->s_full[g][0]), p_full = smem_addr(&bars->p_full[g][0]);
            const uint32_t pv_done = smem_addr(&bars->pv_done[g]);
            const int k_steps = kp / 16;
            auto wait = [&](uint32_t bar, uint32_t phase) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(bar, phase, status, abort_flag));
            };
            Ring k0, v0;              // the piece's first block
            uint32_t pv = 0;          // P.V products issued: block pv of the group is in buffer pv & 1
            int piece = 0;
            bool ok = true;
            // the self-test's wait runs out after the debug limit, and every role leaves
            if (a.debug_timeout && g == 0)
                ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&bars->never), 0, status, abort_flag, kDebugWaitLimitNs));
            for (bool more = w.next(a, bars, true); ok && more; more = w.next(a, bars, false), ++piece) {
                // with two row tiles every block is this group's, with one every second
                const bool two = 2 * pair_of(a, w.u) + 1 < a.nrt;
                const int by = two ? 1 : 2, steps = two ? w.n : (w.n + 1 - g) / 2;
                const int releases = two ? 1 : users;  // the group alone releases a block of one tile
                const uint64_t qd = qd0 + (uint64_t)((two ? g : 0) * (Q_BYTES / 16));  // descriptors count 16 bytes
                Ring k = k0, v = v0;
                if (!two && g == 1) k.next(1, a.nk), v.next(1, a.nv);
                ok = wait(smem_addr(&bars->q_full), (uint32_t)piece & 1u);
                fence_proxy_async_smem();  // a gathered query operand, written by the softmax warps
                // P.V of a block, then S of the block after next in the same buffer, while the softmax
                // works on the block between
                for (int n = -2; ok && n < steps; ++n) {
                    const uint32_t buf = (pv + (n < 0 ? n : 0)) & 1u;  // of blocks n and n + 2
                    if (n >= 0) {
                        ok = wait(smem_addr(&bars->v_full[v.slot]), v.phase) && wait(p_full + buf * 8, (pv >> 1) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = vd0 + (uint64_t)(v.slot * (V_BYTES / 16));
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            umma_f16_tmem_a_elect(o_tm, s_tm + buf * BK + kk * 8, vd + kk * 128, idesc_pv,
                                                  kk > 0 || n > 0 ? 1u : 0u);
                        umma_commit_elect(pv_done);
                        for (int r = 0; r < releases; ++r) umma_commit_elect(smem_addr(&bars->v_empty[v.slot]));
                        v.next(by, a.nv);
                        ++pv;
                    }
                    if (n + 2 < steps) {
                        ok = wait(smem_addr(&bars->k_full[k.slot]), k.phase);
                        // the P.V just issued reads P, which lies over this buffer's S
                        if (ok && n >= 0) ok = wait(pv_done, (pv - 1) & 1u);
                        if (!ok) break;
                        if (!kAll) fence_proxy_async_smem();  // copied keys, read by the tensor cores
                        tc_fence_after();
                        const uint64_t kd = kd0 + (uint64_t)(k.slot * (K_BYTES / 16));
                        if (kAll) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                umma_f16_elect(s_tm + buf * BK, qd + (kk >> 2) * (BM * 8) + (kk & 3) * 2, kd + kk * 128,
                                               idesc_s, kk > 0 ? 1u : 0u);
                        } else {
                            uint64_t q1 = qd, k1 = kd;
#pragma unroll 1
                            for (int kk = 0; kk < k_steps; ++kk, q1 += 128, k1 += 128)
                                umma_f16_elect(s_tm + buf * BK, q1, k1, idesc_s, kk > 0 ? 1u : 0u);
                        }
                        umma_commit_elect(s_full + buf * 8);
                        for (int r = 0; r < releases; ++r) umma_commit_elect(smem_addr(&bars->k_empty[k.slot]));
                        k.next(by, a.nk);
                    }
                }
                if (ok) umma_commit_elect(smem_addr(&bars->o_full));
                for (int j = 0; j < w.n; ++j) k0.next(1, a.nk), v0.next(1, a.nv);
            }
            __syncwarp();
            umma_commit_elect(smem_addr(&bars->drain));
            // issued MMAs finish on their own; TMEM is not freed under them
            volatile int no_abort = 0;
            mbar_wait(smem_addr(&bars->drain), 0, status, &no_abort);
            __syncwarp();
        }
    } else if (!kAll) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // ------------------------------------------------------------ kept rows of K^T, 16 bytes a copy
        // Quarter-warps take every sixteenth kept row, a lane 8 keys of it.  A warp's copy
        // instruction takes about 110 cycles to leave, so that two warps of them bounded the
        // kernel (1750 cycles a block at 64 kept dims, where its bytes take 1000).
        const int c16 = lane & 7, row = (warp - kGatherWarp) * 4 + (lane >> 3);
        Ring k;
        bool ok = true;
        for (bool more = w.next(a, bars, true); ok && more; more = w.next(a, bars, false)) {
            const int plane = w.b * a.Hkv + head_of(a, w.u);
            uint32_t at[8];  // the rows' places in the d-major cache; the padding repeats a kept row
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (16 * i < kp) at[i] = (uint32_t)a.idx[(size_t)plane * a.k + (16 * i + row < a.k ? 16 * i + row : 0)] * a.ldL;
            const uint16_t* Kg = a.Kt + (size_t)plane * D * a.ldL + c16 * 8;
            for (int j = 0; j < w.n; ++j) {
                const int key0 = (w.blk + j) * BK;
                if (!__all_sync(0xffffffffu,
                                mbar_wait(smem_addr(&bars->k_empty[k.slot]), k.phase ^ 1u, status, abort_flag))) {
                    ok = false;
                    break;
                }
                // row 16 i + row lies at 2048 i + 128 row, its 16-byte pieces permuted by row mod 8
                const uint32_t dst = smem_addr(sK + k.slot * K_BYTES) + row * 128 + ((c16 ^ (row & 7)) << 4);
                const uint32_t bytes = key0 + c16 * 8 < a.ldL ? 16u : 0u;
                const uint16_t* src = bytes ? Kg + key0 : Kg;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (16 * i < kp) cp_async_16(dst + 2048 * i, src + at[i], bytes);
                cp_async_arrive_noinc(smem_addr(&bars->k_full[k.slot]));
                k.next(1, a.nk);
            }
        }
        cp_async_wait_all();  // no copy may still be landing when the CTA leaves
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The partials of a unit that was cut, joined; also the zeros of empty slots.
// kLanes threads take four dims of a row, each every kLanes-th piece with four of
// them in flight and a running maximum.  Bound by the latency of two dependent reads
// from L2 and, with many rows, by the partials' bytes.
constexpr int kJoinThreads = 256;

template <int kLanes>
__global__ void __launch_bounds__(kJoinThreads) attn_tree_join_kernel(const TreeArgs a) {
    constexpr int kRows = kJoinThreads / 32 / kLanes, kFly = 4;
    const int U = a.U, z = threadIdx.x % kLanes, tid = threadIdx.x / kLanes;
    const int plane = blockIdx.x / a.nrp, rp = blockIdx.x % a.nrp, b = plane / a.Hkv, g = plane % a.Hkv;
    const int u = a.side > 1 ? g : g * a.nrp + rp;
    const int r = blockIdx.y * kRows + tid % kRows, c4 = tid / kRows;
    pdl_wait();
    pdl_launch_dependents();
    const long long lo = a.cum[b], hi = a.cum[b + 1], total = a.cum[a.B], C = a.cum[a.B + 1], piece = a.cum[a.B + 2];
    const long long cost = (hi - lo) / U, nb = cost ? cost - piece : 0;
    const long long p0 = lo + u * cost;  // where the unit starts, its blocks `piece` later
    // share c is [total c / C, total (c + 1) / C): the shares of the unit's first and last block
    const int c0 = nb ? (int)(((p0 + piece + 1) * C - 1) / total) : 0, c1 = nb ? (int)(((p0 + cost) * C - 1) / total) : 0;
    if (nb && c0 == c1) return;
    const int n = nb ? c1 - c0 + 1 : 0;
    const int rows = min(2 * BM, a.R - rp * 2 * BM), row = min(r, rows - 1);
    const size_t sf = slot_floats(a.slot_rows);
    // the first share may have begun with another unit: its piece is then its second
    const int skip = nb && total * c0 / C < p0 ? 1 : 0;
    const float* base = a.partials + (size_t)(2 * (c0 * a.side + (a.side > 1 ? rp : 0))) * sf;
    const size_t at = ((size_t)c4 * a.slot_rows + row) * 4;
    float M = -INFINITY, L = 0.f, nan = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = z; i0 < n; i0 += kFly * kLanes) {
        float m[kFly], l[kFly];
        float4 v[kFly];
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const int j = i0 + i * kLanes;
            m[i] = -INFINITY, l[i] = 0.f;
            if (j < n) {
                const float* p = base + (size_t)(2 * j * a.side + (j == 0 ? skip : 0)) * sf;
                m[i] = p[D * a.slot_rows + row];
                l[i] = p[(D + 1) * a.slot_rows + row];
                v[i] = *reinterpret_cast<const float4*>(p + at);
            }
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            top = fmaxf(top, m[i]);
            if (isnan(l[i])) nan = l[i];  // the row's, whatever its piece weighs
        }
        if (top == -INFINITY) continue;  // the row has seen no key
        const float keep = exp2f(M - top);
        M = top;
        L *= keep;
        o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
        for (int i = 0; i < kFly; ++i) {
            const float w = exp2f(m[i] - M);
            if (w > 0.f) {  // a piece in which the row saw nothing may hold anything
                L = fmaf(w, l[i], L);
                o.x = fmaf(w, v[i].x, o.x);
                o.y = fmaf(w, v[i].y, o.y);
                o.z = fmaf(w, v[i].z, o.z);
                o.w = fmaf(w, v[i].w, o.w);
            }
        }
    }
    L += nan;
#pragma unroll
    for (int d = 1; d < kLanes; d *= 2) {
        const float top = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float w = M > -INFINITY ? exp2f(M - top) : 0.f;
        M = top;
        L *= w;
        o.x *= w, o.y *= w, o.z *= w, o.w *= w;
        L += __shfl_xor_sync(0xffffffffu, L, d);
        o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
    }
    if (z > 0 || r >= rows) return;
    const float inv = L == 0.f ? 0.f : 1.0f / L;
    *reinterpret_cast<uint2*>(a.O + (((size_t)b * a.Hkv + g) * a.R + rp * 2 * BM + r) * D + c4 * 4) =
        make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
}

// The kept dims of one (sequence, KV head): the column maximum of |Q| over the
// present rows, 16 row lanes x 16 pieces of 8 dims, then the exact rank of each
// dim under (score desc, index asc).
__global__ void __launch_bounds__(256) tree_dims_kernel(const TreeArgs a) {
    __shared__ int32_t par[kTreeMax];
    __shared__ uint64_t there_s;
    __shared__ uint32_t red[16][D];
    __shared__ __align__(16) uint32_t sv[D];
    __shared__ int warp_cnt[D / 32];
    const int plane = blockIdx.x, b = plane / a.Hkv, tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const int c16 = tid & 15, rl = tid >> 4;
    uint32_t m[4] = {0, 0, 0, 0};  // two dims each, magnitudes of 15 bits
    const uint16_t* q = a.Q + (size_t)plane * a.R * D + c16 * 8;
    uint4 v[8];  // eight rows in flight, the first while the length and the tree arrive
    auto fetch = [&](int r0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = r0 + 16 * i < a.R ? ld_nc_v4(q + (size_t)(r0 + 16 * i) * D) : make_uint4(0, 0, 0, 0);
    };
    fetch(rl);
    if (blocks_of(a, b) == 0) return;
    uint64_t there = ~0ull;
    if (a.parents) {
        if (tid == 0) there_s = 0;
        if (tid < a.T) par[tid] = a.parents[(size_t)b * a.T + tid];
        __syncthreads();
        if (tid < a.T && tree_way(par, tid))
            atomicOr(reinterpret_cast<unsigned long long*>(&there_s), 1ull << tid);
        __syncthreads();
        there = there_s;
    }
    for (int r0 = rl; r0 < a.R; r0 += 128) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t keep = (there >> ((r0 + 16 * i) % a.T)) & 1 ? 0x7FFF7FFFu : 0u;  // absent nodes do not count
            m[0] = __vmaxu2(m[0], v[i].x & keep);
            m[1] = __vmaxu2(m[1], v[i].y & keep);
            m[2] = __vmaxu2(m[2], v[i].z & keep);
            m[3] = __vmaxu2(m[3], v[i].w & keep);
        }
        if (r0 + 128 < a.R) fetch(r0 + 128);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        red[rl][c16 * 8 + 2 * e] = m[e] & 0xFFFFu;
        red[rl][c16 * 8 + 2 * e + 1] = m[e] >> 16;
    }
    __syncthreads();
    // score and, below it, the order of equal ones: no two are the same
    uint32_t key = 0;
    if (tid < D) {
#pragma unroll
        for (int i = 0; i < 16; ++i) key = max(key, red[i][tid]);
        key = key << 7 | (D - 1 - tid);
        sv[tid] = key;
    }
    __syncthreads();
    bool keep = false;
    if (tid < D) {
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < D / 4; ++i) {
            const uint4 o = reinterpret_cast<const uint4*>(sv)[i];
            rank += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
        }
        keep = rank < a.k;
    }
    const unsigned ball = __ballot_sync(0xffffffffu, keep);
    if (tid < D && (tid & 31) == 0) warp_cnt[tid >> 5] = __popc(ball);
    __syncthreads();
    if (keep) {
        int pos = __popc(ball & ((1u << (tid & 31)) - 1u));
        for (int i = 0; i < (tid >> 5); ++i) pos += warp_cnt[i];
        a.idx[(size_t)plane * a.k + pos] = tid;
    }
}

struct TreePlan {
    int R, nrt, nrp, slot_rows, ctas;
};

TreePlan tree_plan(int B, int Hq, int Hkv, int T, int ldL, int num_sms) {
    TreePlan p;
    p.R = Hq / Hkv * T;
    p.nrt = (p.R + BM - 1) / BM;
    p.nrp = (p.nrt + 1) / 2;
    p.slot_rows = p.R < 2 * BM ? (p.R + 3) / 4 * 4 : 2 * BM;
    const long long most = (long long)B * Hkv * p.nrp * ((ldL + BK - 1) / BK);
    p.ctas = most < num_sms ? (int)most : num_sms;
    return p;
}

size_t cum_bytes(int B) { return ((size_t)(B + 3) * sizeof(long long) + 255) / 256 * 256; }

}  // namespace

// Two stages each, then more values and keys by turns while they fit.
// A wait for a full barrier tells a round of its slot by parity, so it also passes two rounds
// early, while the copy of the round before is still on its way.  Whoever waits for a block
// therefore has to know that the one before it in its slot has landed.  A group that takes every
// block waits for that one itself; with one row tile (the last of an odd number) it takes every
// second block, and only an even depth brings it back to the slots it has waited for.  (A wait
// for the blocks between would not do: their slots may have been filled again by then.)  The
// softmax warps, which wait for values only near a sequence's end, know that the products of
// the block two before in their group are done: four stages with one row tile, which every
// size gives.  At a piece's start all blocks of the pieces before have been used.
TreeRings attn_tree_rings(int nrt, int kp) {
    const int kb = kp * 128, by = nrt % 2 ? 2 : 1;
    const int fixed = 1024 + (nrt > 1 ? 2 : 1) * kp * 256 + (int)sizeof(TreeBars) + kTreeMax * 4;
    TreeRings r{2, 2, 0};
    for (bool grew = true; grew;) {
        grew = false;
        if (r.nv < kMaxStages && fixed + (r.nv + by) * V_BYTES + r.nk * kb <= kSmemMax) r.nv += by, grew = true;
        if (r.nk < kMaxStages && r.nk < r.nv && fixed + r.nv * V_BYTES + (r.nk + by) * kb <= kSmemMax) r.nk += by, grew = true;
    }
    r.smem = fixed + r.nv * V_BYTES + r.nk * kb;
    return r;
}

size_t attn_tree_partial_bytes(int B, int Hq, int Hkv, int T, int ldL, int num_sms) {
    const TreePlan p = tree_plan(B, Hq, Hkv, T, ldL, num_sms);
    return cum_bytes(B) + (size_t)p.ctas * 2 * slot_floats(p.slot_rows) * sizeof(float);
}

cudaError_t launch_attn_tree(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                             const uint16_t* Q, const uint16_t* Kt, int B, int Hq, int Hkv, int T, int ldL, int k, float scale,
                             const int32_t* lens, const int32_t* parents, uint16_t* O, int32_t* idx, int want_idx,
                             void* partials, int* status, int debug_timeout, int num_sms, cudaStream_t stream) {
    const TreePlan p = tree_plan(B, Hq, Hkv, T, ldL, num_sms);
    TreeArgs a{};
    a.Q = Q;
    a.Kt = Kt;
    a.lens = lens;
    a.parents = parents;
    a.identity = k == D;
    a.idx = a.identity && !want_idx ? nullptr : idx;
    a.O = O;
    a.cum = static_cast<long long*>(partials);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(partials) + cum_bytes(B));
    a.status = status;
    a.debug_timeout = debug_timeout;
    a.B = B, a.Hkv = Hkv, a.G = Hq / Hkv, a.T = T, a.ldL = ldL;
    a.R = p.R, a.nrt = p.nrt, a.nrp = p.nrp, a.slot_rows = p.slot_rows;
    // Row pairs of a head that CTAs take side by side read its keys and values at the same time, so
    // that L2 serves all but the first (64 nodes of 8 heads over 32k keys, 262 us against 279 with
    // the pairs one after the other); a head with more pairs than this has enough work of its own.
    a.side = p.nrp <= kMaxSide && p.nrp <= p.ctas ? p.nrp : 1;
    a.U = Hkv * p.nrp / a.side;
    a.k = k;
    a.kp = (k + 15) / 16 * 16;
    a.scale_log2 = scale * 1.4426950408889634f;
    const TreeRings rings = attn_tree_rings(p.nrt, a.kp);
    a.nk = rings.nk, a.nv = rings.nv;
    const size_t smem = rings.smem;
    auto* kern = a.identity ? attn_tree_kernel<true> : attn_tree_kernel<false>;
    cudaError_t e = ensure_smem_limit(kern, smem);
    if (e != cudaSuccess) return e;
    if (!a.identity) {
        e = launch_pdl(tree_dims_kernel, dim3(B * Hkv), dim3(256), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(kern, dim3(p.ctas), dim3(tree_threads(a.identity)), smem, stream, qmap, kmap, vmap, a);
    if (e != cudaSuccess) return e;
    // With few units a unit is cut into many pieces, which four threads then share (us of a call, one
    // thread against four: 16 nodes of one sequence, 18 pieces a unit, 22.3 and 21.2; 25 nodes of 8
    // sequences, 2 or 3 pieces, 65 and 74).
    const int units = B * Hkv * p.nrp, lanes = p.ctas > 4 * units ? 4 : 1, rows = kJoinThreads / 32 / lanes;
    const int most_rows = p.R < 2 * BM ? p.R : 2 * BM;
    return launch_pdl(lanes == 4 ? attn_tree_join_kernel<4> : attn_tree_join_kernel<1>,
                      dim3(units, (most_rows + rows - 1) / rows), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace rmm
