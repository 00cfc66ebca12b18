// grouped_mm.cu -- products grouped by expert with ragged sizes, and their
// gradients, on the 5th-generation tensor cores (tcgen05, accumulators in
// TMEM, operands staged by TMA).
//
// Rows [offsets[e], offsets[e+1]) of the row matrices belong to expert e:
//   forward          y[r, n]     = sum_c x[r, c]  * w[e, n, c]
//   input gradient   dx[r, c]    = sum_n dy[r, n] * w[e, n, c]
//   weight gradient  dw[e, n, c] = base[e, n, c] + sum_{r of e} dy[r, n] * x[r, c]
//
// One kernel serves the three, two CTAs of a cluster on one 256 x 256 tile
// (cta_group::2): each holds 128 columns of the A operand and half of the B
// operand, and 128 x 256 of the accumulator.  The A operand (MMA M) is the
// side that is contiguous in the output, the B operand (MMA N) the other, so that the 32 lanes of an epilogue warp always hold 32
// neighbouring output columns:
//   forward          A = w[e]  (reduction contiguous: "K-major")   B = x rows  (K-major)
//   input gradient   A = w[e]  (output side contiguous: "MN-major") B = dy rows (K-major)
//   weight gradient  A = x     (MN-major)                           B = dy      (MN-major)
// With the routed rows on N, tiles of a ragged expert round up to 16 rows,
// not 128.  Reads outside a matrix are zero-filled by TMA (the weights are a
// 3-D tensor, so an expert's edge is an edge too); the one edge TMA does not
// know is the end of an expert's rows inside the reduction of the weight
// gradient: the rows behind it in the last 16-row step are overwritten with
// zeros in shared memory, on both operands, before the MMA reads them (a
// zero on one side alone would let a neighbour's infinity through as NaN).
//
// Persistent: one CTA per SM, the pairs walk the tile list, which every CTA
// derives from the offsets on the device.  Warp roles: 0 TMA producer of the
// CTA's own operands (both CTAs' copies complete on the leading CTA's
// barrier); 1 in the leading CTA MMA issue for the pair, in the other idle
// but for a ragged end, which each CTA zeroes in its own operands before the
// other CTA's warp tells the leader; 2-9 epilogue (two warps per TMEM lane
// quarter, alternating 32 columns).
#include "common.cuh"
#include "gemm_common.cuh"
#include "internal.h"

#include <algorithm>

namespace moe {

namespace {

enum Op : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kBK = 64;                        // reduction elements per stage = one 128-byte swizzle row
constexpr int kTM = 256;                       // A-side width of a pair's tile
constexpr int kBN = 256;                       // B-side width of a pair's tile
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kABytes = kBM * 128;
constexpr int kBBytes = kBN / 2 * 128;         // a CTA holds half of B
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kRingBytes = kStages * kStageBytes;
constexpr int kOutStage = kEpiWarps * 32 * 32 * 2;
constexpr int kChunkBytes = 64 * 128;          // MN-major: 64 elements x 64 reduction rows

size_t smem_bytes(int E) { return 1024 + kRingBytes + 1024 + kOutStage + align_up(12 * (size_t)(E + 1), 16); }

struct MmArgs {
    const int32_t *offsets;   // [E+1]
    int rows;                 // rows of the row matrices
    int E, M, N;              // experts; A-side extent; B-side extent (weight gradient)
    int red;                  // reduction extent (forward, input gradient)
    int box_rows;             // rows per TMA box of a K-major B
    void *out;
    const float *base;        // weight gradient: added to the product (may be out itself), or null
    int32_t *status;
};

// One tile: expert, first A-side column, first B-side row (of the row matrix,
// or of the expert's output features for the weight gradient), rows used,
// and the reduction's first row and length.
struct MmTile {
    int e, m0, row0, nrows, red0, red;
};

// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle:
// 64 elements of the M/N side per 128-byte row, one row per reduction index,
// 8-row atoms 1024 bytes apart (stride offset), the next 64 elements
// kChunkBytes further (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kChunkBytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// ---- the pair: cluster barriers, remote arrivals, cta_group::2 tcgen05 -----
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// True in one lane of a converged warp (the same on every call).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// The address of the leading CTA's barrier at the same place as `bar`.
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
    return a;
}
// Arrive on the leading CTA's barrier; the cluster-scope release (about 2000
// cycles: every block of a product taking it ran at half the speed) is for
// shared-memory writes of this thread that the leader's MMAs read.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_leader_release(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(bar)) : "memory");
}
// TMA tile loads into this CTA's shared memory that complete on a barrier of
// either CTA of the pair (no multicast).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::"
        "cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::"
        "cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
// mbar_wait for arrivals from the other CTA (cluster scope).
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint32_t a = smem_u32(bar);
    long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(a), "r"(parity)
            : "memory");
        if (ok) return true;
        if (it == 0) t0 = clock64();
        if ((it & 255u) == 255u) {
            if (*abort) return false;
            if (clock64() - t0 > kWaitLimitCycles) return false;
        }
    }
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` in both CTAs when every MMA issued so far is done.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// The same on this CTA's `bar` alone.
__device__ __forceinline__ void mma_commit_leader(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

template <int OP>
__device__ __forceinline__ MmTile mm_tile(int w, const MmArgs &a, const int32_t *s_beg, const int32_t *s_end,
                                          const int32_t *s_tiles, int MT, int NT) {
    MmTile t;
    if (OP == kWgrad) {
        t.e = w / (MT * NT);
        const int local = w - t.e * MT * NT;
        const int n = local / MT;
        t.m0 = (local - n * MT) * kTM;
        t.row0 = n * kBN;
        t.nrows = min(kBN, a.N - t.row0);
        t.red0 = s_beg[t.e];
        t.red = s_end[t.e] - t.red0;
    } else {
        int lo = 0, hi = a.E;   // s_tiles[lo]*MT <= w < s_tiles[hi]*MT
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_tiles[mid] * MT <= w) lo = mid; else hi = mid;
        }
        t.e = lo;
        const int nt = s_tiles[lo + 1] - s_tiles[lo];
        const int local = w - s_tiles[lo] * MT;
        const int m = local / nt, n = local - m * nt;
        const int n_e = s_end[lo] - s_beg[lo];
        const int rpt = min(kBN, ((n_e + nt - 1) / nt + 15) & ~15);
        t.m0 = m * kTM;
        t.row0 = s_beg[lo] + n * rpt;
        t.nrows = max(0, min(rpt, n_e - n * rpt));
        t.red0 = 0;
        t.red = a.red;
    }
    return t;
}

// Whether k-block kb ends inside a 16-row step with the next expert's rows in it.
template <int OP>
__device__ __forceinline__ bool ragged_end(const MmTile &t, int kb) {
    const int left = t.red - kb * kBK;
    return OP == kWgrad && left < kBK && (left & 15);
}

template <int OP, bool OUT_BF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_mm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const MmArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem;
    // full: the leader's counts both CTAs' copies, but for a ragged end, where
    // each CTA's own barrier counts its own and `relay` follows
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kRingBytes);
    uint64_t *empty = full + kStages;
    uint64_t *tfull = empty + kStages;
    uint64_t *tempty = tfull + 2;              // the leader's, for both CTAs' epilogues
    uint64_t *relay = tempty + 2;              // the leader's: the other CTA's ragged end is zeroed
    uint64_t *drained = relay + kStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *s_part = reinterpret_cast<int32_t *>(tmem_slot + 2);          // [kThreads / 32]
    __nv_bfloat16 *s_out = reinterpret_cast<__nv_bfloat16 *>(smem + kRingBytes + 1024);
    int32_t *s_beg = reinterpret_cast<int32_t *>(smem + kRingBytes + 1024 + kOutStage);
    int32_t *s_end = s_beg + args.E;
    int32_t *s_tiles = s_end + args.E;                                      // [E+1]

    const int warp = threadIdx.x >> 5, lane = lane_id();
    const int rank = (int)cluster_rank();      // 0: the leader
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&relay[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull[a], 1);
            mbar_init(&tempty[a], 2 * kEpiWarps);
        }
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    pdl_wait();
    // Row ranges of the experts, clamped into the matrices whatever the
    // offsets hold, and the prefix sum of their row tiles: each thread sums a
    // run of experts, then warps and block are scanned.
    const int per = (args.E + kThreads - 1) / kThreads;
    const int e0 = min(args.E, (int)threadIdx.x * per), e1 = min(args.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
        const int b = min(max(__ldg(args.offsets + e), 0), args.rows);
        const int n = min(max(__ldg(args.offsets + e + 1), b), args.rows);
        s_beg[e] = b;
        s_end[e] = n;
        sum += (n - b + kBN - 1) / kBN;
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    int before = incl - sum;
    for (int i = 0; i < warp; ++i) before += s_part[i];
    for (int e = e0; e < e1; ++e) {
        s_tiles[e] = before;
        before += (s_end[e] - s_beg[e] + kBN - 1) / kBN;
    }
    if (threadIdx.x == kThreads - 1) s_tiles[args.E] = before;
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();                            // both CTAs' barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int MT = (args.M + kTM - 1) / kTM;
    const int NT = (args.N + kBN - 1) / kBN;
    const int total = OP == kWgrad ? args.E * MT * NT : s_tiles[args.E] * MT;
    pdl_launch_dependents();

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ----
        if (lane == 0) {
            const uint64_t pol = policy_evict_last();
            int stage = 0;
            uint32_t phase = 0;
            int armed[kStages];
#pragma unroll
            for (int s = 0; s < kStages; ++s) armed[s] = -1;
            bool ok = true;
            for (int w = pair; w < total && ok; w += pairs) {
                const MmTile t = mm_tile<OP>(w, args, s_beg, s_end, s_tiles, MT, NT);
                if (t.nrows == 0) continue;
                const int KB = (t.red + kBK - 1) / kBK;
                const int half = ((t.nrows + 15) & ~15) / 2;         // B rows of each CTA
                const int m0 = t.m0 + rank * kBM, row0 = t.row0 + rank * half;
                const int nbox = OP == kWgrad ? (half + 63) / 64 : (half + args.box_rows - 1) / args.box_rows;
                const int box_bytes = OP == kWgrad ? kChunkBytes : args.box_rows * 128;
                const uint32_t bytes = kABytes + nbox * box_bytes;
                for (int kb = 0; kb < KB; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) { ok = false; break; }
                    uint8_t *sA = ring + stage * kStageBytes;
                    uint8_t *sB = sA + kABytes;
                    const bool ragged = ragged_end<OP>(t, kb);
                    if (rank == 0 || ragged) mbar_arrive_expect_tx(&full[stage], ragged ? bytes : 2 * bytes);
                    if (rank == 0) armed[stage] = (int)phase;
                    const uint32_t bar = ragged ? smem_u32(&full[stage]) : leader_addr(&full[stage]);
                    const int k0 = t.red0 + kb * kBK;
                    if (OP == kFwd) {
                        tma_load_3d_pair(sA, &tmA, bar, k0, m0, t.e, pol);
                    } else {
                        for (int c = 0; c < kBM / 64; ++c) {
                            if (OP == kDgrad)
                                tma_load_3d_pair(sA + c * kChunkBytes, &tmA, bar, m0 + 64 * c, k0, t.e, pol);
                            else
                                tma_load_2d_pair(sA + c * kChunkBytes, &tmA, bar, m0 + 64 * c, k0, pol);
                        }
                    }
                    for (int b = 0; b < nbox; ++b) {
                        if (OP == kWgrad)
                            tma_load_2d_pair(sB + b * kChunkBytes, &tmB, bar, row0 + 64 * b, k0, pol);
                        else
                            tma_load_2d_pair(sB + b * box_bytes, &tmB, bar, k0, row0 + b * args.box_rows, pol);
                    }
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                }
            }
            // Nothing may be in flight towards this CTA when it ends: on success
            // every stage has been consumed (the leader's arrivals on `empty`
            // included), otherwise every armed stage must have landed (the
            // leader's barriers count for both; the pair ends together).
            volatile int never = 0;
            for (int s = 0; s < kStages && ok; ++s) {
                ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag);
                if (++stage == kStages) { stage = 0; phase ^= 1; }
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(args.status, DEV_TIMEOUT);
                for (int s = 0; s < kStages; ++s)
                    if (armed[s] >= 0 && !mbar_wait(&full[s], (uint32_t)armed[s], &never))
                        atomicOr(args.status, DEV_TIMEOUT);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------ MMA issuer / relay ------
        constexpr uint32_t kMajor = (OP == kFwd ? 0u : 1u << 15) | (OP == kWgrad ? 1u << 16 : 0u);
        constexpr int kStepA = OP == kFwd ? 2 : 128, kStepB = OP == kWgrad ? 128 : 2;   // 16-byte units per 16 k
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0, ragged_turn = 0;
        const bool issuer = elect_one();
        bool ok = true;
        for (int w = pair; w < total && ok; w += pairs) {
            const MmTile t = mm_tile<OP>(w, args, s_beg, s_end, s_tiles, MT, NT);
            if (t.nrows == 0 || t.red == 0) continue;
            const int KB = (t.red + kBK - 1) / kBK;
            const int bn = (t.nrows + 15) & ~15;
            const uint32_t idesc = idesc_bf16(kTM, bn) | kMajor;
            if (rank == 0 && !mbar_wait_cluster(&tempty[acc], acc_phase ^ 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d = tmem_base + acc * kBN;
            for (int kb = 0; kb < KB; ++kb) {
                uint8_t *sA = ring + stage * kStageBytes;
                const int left = t.red - kb * kBK;
                const int steps = left >= kBK ? kBK / 16 : (left + 15) / 16;
                const bool ragged = ragged_end<OP>(t, kb);
                const uint32_t turn = (ragged_turn >> stage) & 1u;      // phase of this stage's ragged ends
                if (rank == 0 || ragged) {
                    if (!mbar_wait(&full[stage], rank == 0 ? phase : turn, abort_flag)) { ok = false; break; }
                }
                if (ragged) {
                    // rows [left, steps*16) belong to the next expert: zero
                    // them in every 64-column chunk of both operands
                    const int z = steps * 16 - left;
                    const int chunks = kBM / 64 + (bn / 2 + 63) / 64;
                    for (int i = lane; i < chunks * z * 8; i += 32) {
                        const int c = i / (z * 8), b = i - c * z * 8;
                        *reinterpret_cast<uint4 *>(sA + c * kChunkBytes + left * 128 + b * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    ragged_turn ^= 1u << stage;
                    if (rank != 0) {
                        if (lane == 0) mbar_arrive_leader_release(&relay[stage]);
                    } else if (!mbar_wait_cluster(&relay[stage], turn, abort_flag)) {
                        ok = false;
                        break;
                    }
                }
                if (rank != 0) {
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                    continue;
                }
                if (issuer) {
                    tc_fence_after();
                    const uint32_t sa = smem_u32(sA);
                    const uint64_t da = OP == kFwd ? sdesc_sw128(sa) : sdesc_mn(sa);
                    const uint64_t db = OP == kWgrad ? sdesc_mn(sa + kABytes) : sdesc_sw128(sa + kABytes);
                    if (steps == kBK / 16) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            mma_bf16_pair(d, da + kStepA * k, db + kStepB * k, idesc, (kb | k) != 0);
                    } else {
                        for (int k = 0; k < steps; ++k)
                            mma_bf16_pair(d, da + kStepA * k, db + kStepB * k, idesc, (kb | k) != 0);
                    }
                    mma_commit_pair(&empty[stage]);
                }
                __syncwarp();
                if (++stage == kStages) { stage = 0; phase ^= 1; }
            }
            if (!ok) break;
            if (rank == 0 && issuer) mma_commit_pair(&tfull[acc]);
            __syncwarp();
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
        if (issuer) {
            if (!ok) {
                *abort_flag = 1;
                atomicOr(args.status, DEV_TIMEOUT);
            }
            // no MMA may be reading either CTA's shared memory when they end
            if (rank == 0) {
                volatile int never = 0;
                mma_commit_leader(drained);
                if (!mbar_wait(drained, 0, &never)) atomicOr(args.status, DEV_TIMEOUT);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue --------
        const int ew = warp - 2;                // 0 .. kEpiWarps-1
        const int eg = warp & 3;                // TMEM lanes [32*eg, 32*eg+32)
        const int half = ew >> 2;               // which 32-column chunks
        __nv_bfloat16 *stg = s_out + ew * 32 * 32;   // [32 rows][32 columns]
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int w = pair; w < total; w += pairs) {
            const MmTile t = mm_tile<OP>(w, args, s_beg, s_end, s_tiles, MT, NT);
            if (t.nrows == 0) continue;
            const bool none = OP == kWgrad && t.red == 0;     // an expert without rows: the sum is zero
            if (none && args.base == args.out && args.base != nullptr) continue;
            if (!none) {
                if (!mbar_wait(&tfull[acc], acc_phase, abort_flag)) {
                    *abort_flag = 1;
                    atomicOr(args.status, DEV_TIMEOUT);
                    break;
                }
                tc_fence_after();
            }
            const uint32_t tb = tmem_base + ((uint32_t)(eg * 32) << 16) + acc * kBN;
            const size_t orow = OP == kWgrad ? (size_t)t.e * args.N + t.row0 : (size_t)t.row0;
            const int mw = t.m0 + rank * kBM + eg * 32;      // first output column of this warp
            for (int c0 = half * 32; c0 < t.nrows; c0 += 64) {
                uint32_t g[32];
                if (none) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) g[j] = 0;
                } else {
                    tmem_ld32(tb + c0, g);
                    tmem_ld_wait();
                }
                if (OUT_BF16) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) stg[j * 32 + lane] = __float2bfloat16_rn(__uint_as_float(g[j]));
                    __syncwarp();
                    // 32 rows x 64 bytes: four lanes per row, 16 bytes each
                    const int q = lane & 3;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (lane >> 2) + 8 * i;
                        if (c0 + r < t.nrows && mw + q * 8 < args.M) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(stg + r * 32 + q * 8);
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(args.out) +
                                                       (orow + c0 + r) * args.M + mw + q * 8) = v;
                        }
                    }
                    __syncwarp();
                } else if (mw + lane < args.M) {
                    const size_t at = (orow + c0) * args.M + mw + lane;
                    if (OP == kWgrad && args.base) {     // all reads first: base may be out itself
                        float b[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) b[j] = c0 + j < t.nrows ? args.base[at + (size_t)j * args.M] : 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) g[j] = __float_as_uint(__uint_as_float(g[j]) + b[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c0 + j < t.nrows) static_cast<float *>(args.out)[at + (size_t)j * args.M] = __uint_as_float(g[j]);
                }
            }
            if (none) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_leader(&tempty[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// Row-major [depth][rows][cols] bf16 as a 3-D tensor map, 128-byte swizzle,
// box of box_rows x 64 columns.
bool make_tmap_3d(CUtensorMap *m, const void *ptr, uint64_t depth, uint64_t rows, uint64_t cols, uint32_t box_rows) {
    auto enc = tmap_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {cols, rows, depth};
    cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
    cuuint32_t box[3] = {64, box_rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OP, bool OUT_BF16>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const MmArgs &args, cudaStream_t st) {
    static std::atomic<int> attr_done[64];
    const cudaError_t e = enable_max_dyn_smem((const void *)grouped_mm<OP, OUT_BF16>, attr_done);
    if (e != cudaSuccess) return e;
    return launch_k(grouped_mm<OP, OUT_BF16>, dim3(num_sms() & ~1), dim3(kThreads), smem_bytes(args.E), st, true, a, b, args);
}

}  // namespace

cudaError_t launch_grouped_mm(const void *x, const void *w, const int32_t *offsets, int rows, int N, int C, int E,
                              bool transpose, bool out_bf16, void *out, int32_t *status, cudaStream_t st) {
    const int red = transpose ? N : C;
    MmArgs a = {};
    a.offsets = offsets;
    a.rows = rows;
    a.E = E;
    a.M = transpose ? C : N;
    a.N = kBN;
    a.red = red;
    a.box_rows = rows >= (int64_t)64 * E ? 128 : 32;
    a.out = out;
    a.status = status;
    CUtensorMap ta, tb;
    if (!make_tmap_3d(&ta, w, E, N, C, transpose ? kBK : kBM) ||
        !make_tmap(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, rows, red, a.box_rows))
        return cudaErrorInvalidValue;
    if (transpose)
        return out_bf16 ? launch<kDgrad, true>(ta, tb, a, st) : launch<kDgrad, false>(ta, tb, a, st);
    return out_bf16 ? launch<kFwd, true>(ta, tb, a, st) : launch<kFwd, false>(ta, tb, a, st);
}

cudaError_t launch_grouped_wgrad(const void *dy, const void *x, const int32_t *offsets, int rows, int N, int C, int E,
                                 bool out_bf16, const float *base, void *dw, int32_t *status, cudaStream_t st) {
    MmArgs a = {};
    a.offsets = offsets;
    a.rows = rows;
    a.E = E;
    a.M = C;
    a.N = N;
    a.out = dw;
    a.base = base;
    a.status = status;
    CUtensorMap ta, tb;
    if (!make_tmap(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, rows, C, kBK) ||
        !make_tmap(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy, rows, N, kBK))
        return cudaErrorInvalidValue;
    return out_bf16 ? launch<kWgrad, true>(ta, tb, a, st) : launch<kWgrad, false>(ta, tb, a, st);
}

}  // namespace moe
