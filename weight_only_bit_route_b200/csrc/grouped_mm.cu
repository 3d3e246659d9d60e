// Matrix products grouped by expert, in 16 bits and in 8-bit integers, on the 5th-generation tensor cores.
//
// Rows offsets[e] to offsets[e+1] belong to expert e.  With W_e = w[e] stored [out, in]:
//     forward   y[r, n]  = sum_k x[r, k] w[e, n, k]                     (K = in)
//     gradient  dx[r, k] = sum_n dy[r, n] w[e, n, k]                    (K = out)
//     int8      y[r, n]  = t s_r s_n sum_k q[r, k] w[e, n, k]           (s: row and channel scales; s_r holds the routing weight t)
//     int8 gate/up       h[r, f] = silu(g) u, g and u as above with two banks
//
// One kernel computes them all as D = A B with A the weights (M = 128 of their output features, 256 for a CTA
// pair) and B the rows (N up to NT of one expert): an expert holds few rows more often than few features, and N
// can be any multiple of 16, so little of a tile is padding.  The gradient reads the same stored weights along
// the other axis: A's shared-memory tile is then stored along M (rows of 64 input features, one per output
// feature) and the MMA descriptor says so; nothing is transposed.
//
// A tile is (expert, 128 * CG features, up to NT rows).  A persistent CTA (or pair) takes a fixed sequence of
// them; every role computes it from a table of the experts' first tiles in shared memory, so nothing is handed out
// through the workspace.  Warp roles:
//   warps 0, 3 TMA producers of A and B.  A stage is SL slices of K = 128 bytes (64 elements of 16 bits, 128 of 8)
//              of A and B, 128-byte swizzled; rows past the tensors' ends arrive as zeros, and so does K past its
//              end on both sides.
//   warp 1     issues the MMAs (in a pair: the first CTA's warp, for both) and commits each stage.
//   warps 4-11 epilogue from tensor memory: lane = feature, column = row.  Two accumulator buffers, so that the
//              epilogue of a tile overlaps the next tile's products.
// B's rows behind the tile's last are other experts' rows: their columns are computed and never stored.
//
// The tensor core's fp32 sums are cut off rather than rounded, an error that grows with the contraction.  So in 16 bits
// only kMmChunk = 1024 terms are summed in tensor memory at a time, and the epilogue adds those partial sums in fp32
// registers, rounded to nearest.  Of the bf16 results over K = 4096, 0.7 in a thousand then differ from those of plain
// fp32 sums; 2.3 with one sum, 0.5 with chunks of 512.  Time in a loop, one sum / 1024 / 512 (44 experts, 65,536 rows):
// K = 4096 723 / 727 / 740 us, K = 1536 722 / 736 / 757 (chunks of 1536: 730); 8 tokens over 352 experts 118.7 / 119.4 / 119.8.
//
// Bound by the weight stream up to some hundred rows per expert (352 experts of 4096 x 1536: 8 tokens 117 us in bf16,
// 114 us for int8 gate and up, 6.3 and 6.5 TB/s; 2048 tokens 694 us, 6.6 TB/s), by the tensor pipe and the power cap
// above (65,536 rows over 44 experts: 1340 TFLOP/s in a burst, 1130 sustained at 1.1 to 1.2 GHz, the pipe 80 % active).
//
// Every wait is bounded (moe_set_wait_limit).  On expiry the kernel records MOE_ERR_TIMEOUT, stops issuing work,
// waits (bounded) for its copies and MMAs in flight, frees its tensor memory and returns.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "grouped_mm.cuh"
#include "mm_ptx.cuh"

namespace moe {

constexpr int MM_THREADS = 384;
constexpr int MM_EPI_WARPS = 8;
constexpr int MM_BOXES = 4;
// 16 bits: terms summed in tensor memory at a time (integer sums are exact)
constexpr int kMmChunk = 1024;

// Tile shape of one instantiation.  NT: rows per tile; CG: CTAs per tile; SL: 128-byte slices of K per stage; SPLIT:
// a cluster shares a tile's K.
template <bool I8, bool AMN, bool GU, int NT, int CG, int SL, bool SPLIT>
struct MmCfg {
    static constexpr int kMat = GU ? 2 : 1;
    static constexpr int kBK = (I8 ? 128 : 64) * SL;              // K per stage
    static constexpr int kMmaK = I8 ? 32 : 16;                    // K per MMA
    static constexpr int kABytes = SL * 128 * 128;                // per matrix
    static constexpr int kBBytes = SL * NT / CG * 128;
    static constexpr int kStage = kMat * kABytes + kBBytes;
    // split K: partial sums from the other CTAs, 8 KB per block of 16 rows and matrix
    static constexpr int kMaxSplit = GU ? 4 : 8;
    static constexpr int kRedBytes = SPLIT ? (kMaxSplit - 1) * kMat * 8192 : 0;      // (z - 1) ceil(NT / 16 / z) <= kMaxSplit - 1
    static constexpr int kRingBytes = 200 * 1024 - kRedBytes;     // beside them: the tile table (16 bytes per expert)
    static constexpr int kStages = kRingBytes / kStage < 12 ? kRingBytes / kStage : 12;
    static constexpr int kBlocks = NT / 16;
    static constexpr int kAccCols = kMat * NT;                    // one accumulator buffer
    // Accumulators take tensor memory in two halves, in turn; a tile of more than kHalfRows rows takes both.
    static constexpr int kHalfRows = 2 * kAccCols <= 512 ? NT : NT / 2;
    static constexpr int kHalfCols = kMat * kHalfRows;
    static constexpr int kTmemCols = 2 * kHalfCols;
    static constexpr int kTmem = kTmemCols <= 32 ? 32 : (kTmemCols <= 64 ? 64 : (kTmemCols <= 128 ? 128 : (kTmemCols <= 256 ? 256 : 512)));
    static constexpr int kChunk = I8 ? 1 << 30 : kMmChunk / kBK;  // stages summed in tensor memory at a time
    static constexpr int kSums = I8 ? 1 : (NT + 31) / 32 * 16;    // of one epilogue thread
    static constexpr int kStep = 16 * CG;                         // a tile's N is a multiple of this
    static_assert(kAccCols <= 512 && NT % kStep == 0 && kStages >= 2, "tile shape");
    static_assert(!SPLIT || (CG == 1 && NT <= 64), "split K: the partial sums fit");
    static_assert(NT / CG <= (16 << (MM_BOXES - 1)), "the largest box holds a tile's rows");
};

// The halves' use, kept alike by the issuer and the epilogue
struct MmHalves {
    uint32_t u0 = 0, u1 = 0, next = 0;                            // uses so far, the half whose turn it is
    __device__ __forceinline__ uint32_t uses(uint32_t h) const { return h ? u1 : u0; }
    __device__ __forceinline__ void take(uint32_t h, bool both) {
        if (both || h == 0) u0++;
        if (both || h == 1) u1++;
        next = both ? 0 : h ^ 1u;
    }
};

struct MmTile { int e, m0, n0, nval, bn; };                       // n0: first row (of all rows)

struct MmArgs {
    CUtensorMap a0, a1;                  // weights [E][out][in]; a1: up (gate/up)
    CUtensorMap b[MM_BOXES];             // rows, boxes of 16, 32, 64 and 128
    const int32_t* offsets;
    const float* act_scale;              // int8: [rows]
    const float* s0; const float* s1;    // int8: channel scales [E][out]
    uint16_t* out;                       // [rows][ldo]
    int32_t* status;
    uint32_t mt_inv;                     // mm_inverse(feature tiles)
    int E, mdim, kdim, rows;             // mdim: output features (A's M), kdim: contraction length
    int f16;                             // 16-bit elements are fp16 (else bf16)
    int chunked;                         // bit 0: a0 and a1, bit 1: b see K (gradient: A's features) in 128-byte chunks
    int split_tiles;                     // split K: clusters to launch, if they fit
    int split;                           // CTAs that share a tile's K (1: none)
    int meet;                            // see MmSequence
    int early;                           // the kernel before is this product's own row pass
};

template <int CG>
__device__ __forceinline__ void mm_copy2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if (CG == 2) g_tma2d_pair(dst, map, x, y, bar); else g_tma2d(dst, map, x, y, bar);
}
template <int CG>
__device__ __forceinline__ void mm_copy3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if (CG == 2) g_tma3d_pair(dst, map, x, y, z, bar); else g_tma3d(dst, map, x, y, z, bar);
}
template <int CG>
__device__ __forceinline__ void mm_copy4(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t bar) {
    if (CG == 2) g_tma4d_pair(dst, map, x, y, z, w, bar); else g_tma4d(dst, map, x, y, z, w, bar);
}

// The sum of a lane's 16 columns over the z CTAs that share a tile's K, in the order of the CTAs (own: v)
template <bool I8>
__device__ __forceinline__ void mm_join(uint32_t (&v)[16], const uint8_t* red, int stride, int z, uint32_t krank, int row) {
    uint32_t sum[16];
#pragma unroll
    for (int j = 0; j < 16; j++) sum[j] = 0;                       // (0 is zero in both types)
    for (int r = 0; r < z; r++) {
        const bool own = r == int(krank);
        const uint8_t* p = red + (r < int(krank) ? r : r - 1) * stride + row * 16;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            uint4 o = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            if (!own) o = *reinterpret_cast<const uint4*>(p + j * 2048);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int i = 0; i < 4; i++)
                sum[4 * j + i] = I8 ? sum[4 * j + i] + w[i]
                                    : __float_as_uint(__uint_as_float(sum[4 * j + i]) + __uint_as_float(w[i]));
        }
    }
#pragma unroll
    for (int j = 0; j < 16; j++) v[j] = sum[j];
}

template <bool I8, bool AMN, bool GU, int NT, int CG, int SL, bool SPLIT>
__global__ void __launch_bounds__(MM_THREADS, 1) mm_kernel(const __grid_constant__ MmArgs a) {
    using C = MmCfg<I8, AMN, GU, NT, CG, SL, SPLIT>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[S], empty[S], acc_full[2], acc_empty[2], drain, hold_bar, red_full, red_done, red_free;
    __shared__ uint32_t s_tmem;
    __shared__ uint32_t s_issued[2];                 // stages this CTA's two producers have issued
    __shared__ int s_wsum[MM_THREADS / 32], s_wt[MM_THREADS / 32], s_nact, s_total, s_hold;
    __shared__ volatile GAbort s_ab;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? g_cta_rank() : 0u;
    const int MT = (a.mdim + 128 * CG - 1) / (128 * CG);
    const int KS = (a.kdim + C::kBK - 1) / C::kBK;
    const int z = SPLIT ? a.split : 1;
    const uint32_t krank = SPLIT ? g_cta_rank() : 0u;
    const int kper = (KS + z - 1) / z, ks0 = int(krank) * kper, ks1 = min(KS, ks0 + kper);      // this CTA's stages of K

    if (warp == 4 && lane < 2) g_prefetch_map(lane ? &a.b[0] : &a.a0);
    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&full[s])), "r"(2 * CG));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&empty[s])));
        }
        for (int s = 0; s < 2; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&acc_full[s])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&acc_empty[s])), "r"(MM_EPI_WARPS * CG));
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&drain)));
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&hold_bar)));
        if (SPLIT) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&red_full)));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&red_done)), "r"(MM_EPI_WARPS));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&red_free)), "r"(z));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_ab.flag = 0;
        s_issued[0] = s_issued[1] = 0;
    }
    if (warp == 2) g_tmem_alloc<CG>(g_smem(&s_tmem), C::kTmem);
    if (CG == 2 || SPLIT) {                          // the other CTAs' barriers exist before anything arrives there
        __syncthreads();
        g_cluster_sync();
    }
    if (!a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == MM_THREADS - 1) {                     // (a thread with few offsets or none to wait for)
        s_ab.limit_ns = g_limit_from(a.status);
        s_hold = g_hold_from(a.status);
    }

    uint8_t* ring = smem + ((1024u - (g_smem(smem) & 1023u)) & 1023u);
    uint8_t* red = ring + S * C::kStage;             // split K: [other CTA][own block][matrix][4][128 lanes] of 16 bytes
    int4* tbl = reinterpret_cast<int4*>(red + C::kRedBytes);        // active experts: {expert | rows per tile << 16, first tile, first row, rows}
    constexpr bool kSort = CG == 2;                  // large batches: the experts' tiles from the most rows to the fewest
    constexpr int PER = (kMaxE + MM_THREADS - 1) / MM_THREADS;
    // (8 bits: rows from offsets[E] on have no codes)
    const int rows = I8 ? min(a.rows, max(a.offsets[a.E], 0)) : a.rows;
    if constexpr (kSort) {
        int* rows_of = reinterpret_cast<int*>(ring);                 // scratch until the copies start
        const int pad = (a.E + 3) & ~3;
        bool good = true;
        for (int e = tid; e < pad; e += MM_THREADS) {
            int base = 0, n = 0;
            if (e < a.E) good &= mm_expert_rows(a.offsets, e, rows, base, n);
            rows_of[e] = n;
        }
        const bool clip = __syncthreads_or(!good);
        if (clip) {
            if (tid == 0) set_status(a.status, MOE_ERR_DEVICE_INDEX);
            for (int e = tid; e < a.E; e += MM_THREADS) rows_of[e] = mm_clipped_rows(a.offsets, e, rows).y;
            __syncthreads();
        }
        for (int e = tid; e < a.E; e += MM_THREADS)
            tbl[mm_rank(rows_of, a.E, e)] =
                make_int4(e, 0, clip ? mm_clipped_rows(a.offsets, e, rows).x : a.offsets[e], rows_of[e]);
        g_fence_proxy_async();                                       // before the copies write the scratch
        __syncthreads();
    }
    {
        int ex[PER], eb[PER], ne[PER], nt[PER], local = 0, ltiles = 0;
        bool good = true;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int e = tid * PER + i;
            ex[i] = e;
            eb[i] = 0;
            ne[i] = 0;
            if (e < a.E) {
                if constexpr (kSort) {
                    const int4 te = tbl[e];
                    ex[i] = te.x;
                    eb[i] = te.z;
                    ne[i] = te.w;
                } else {
                    good &= mm_expert_rows(a.offsets, e, rows, eb[i], ne[i]);
                }
            }
        }
        if (!kSort && __syncthreads_or(!good)) {
            if (tid == 0) set_status(a.status, MOE_ERR_DEVICE_INDEX);
#pragma unroll
            for (int i = 0; i < PER; i++) {
                if (ex[i] >= a.E) continue;
                const int2 r = mm_clipped_rows(a.offsets, ex[i], rows);
                eb[i] = r.x;
                ne[i] = r.y;
            }
        }
#pragma unroll
        for (int i = 0; i < PER; i++) {
            nt[i] = ((ne[i] + NT - 1) / NT) * MT;
            local += ne[i] > 0;
            ltiles += nt[i];
        }
        int v = local, w = ltiles;
        for (int o = 1; o < 32; o <<= 1) {
            const int n1 = __shfl_up_sync(0xffffffffu, v, o), n2 = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) { v += n1; w += n2; }
        }
        if (lane == 31) { s_wsum[warp] = v; s_wt[warp] = w; }
        __syncthreads();
        int base = 0, tbase = 0, tot = 0, ttot = 0;
        for (int q = 0; q * 32 * PER < a.E; q++) {                   // (the warps that hold experts)
            if (q < warp) { base += s_wsum[q]; tbase += s_wt[q]; }
            tot += s_wsum[q];
            ttot += s_wt[q];
        }
        int pos = base + v - local, tpos = tbase + w - ltiles;
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (ne[i] > 0) {
                const int row_tiles = (ne[i] + NT - 1) / NT, per = (ne[i] + row_tiles - 1) / row_tiles;
                tbl[pos] = make_int4(ex[i] | (per << 16), tpos, eb[i], ne[i]);
                pos++;
                tpos += nt[i];
            }
        if (tid == 0) { s_nact = tot; s_total = ttot; }
    }
    g_fence_before();
    __syncthreads();
    g_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (they wait for this kernel's end themselves)

    const uint32_t tmem = s_tmem;
    const int nact = s_nact;
    const MmSequence seq(int(blockIdx.x) / (CG * z), int(gridDim.x) / (CG * z), s_total, kSort, a.meet != 0);
    // (by whole warps, once per tile and role: with short contractions a tile takes no more than some thousand cycles,
    // so the expert is found by two votes and nothing is divided)
    auto tile_of = [&](int tile) {
        int lo = 0;
        if (nact > 32) lo = 32 * (__popc(__ballot_sync(0xffffffffu, 32 * lane < nact && tbl[min(32 * lane, nact - 1)].y <= tile)) - 1);
        lo += __popc(__ballot_sync(0xffffffffu, lo + lane < nact && tbl[min(lo + lane, nact - 1)].y <= tile)) - 1;
        const int4 te = tbl[lo];
        MmTile t;
        t.e = te.x & 0xffff;
        const int local = tile - te.y, n_e = te.w, per = te.x >> 16;   // balanced rows per tile
        // the features of a row block run fastest: the CTAs of a wave share the rows, and the expert's
        // weights stay in L2 from one row block to the next
        const int n = mm_div(local, MT, a.mt_inv);
        t.m0 = (local - n * MT) * (128 * CG);
        t.nval = min(per, n_e - n * per);
        t.n0 = te.z + n * per;
        t.bn = (t.nval + C::kStep - 1) / C::kStep * C::kStep;
        return t;
    };
    auto fail = [&]() {
        set_status(a.status, MOE_ERR_TIMEOUT);
        s_ab.flag = 1;
    };

    if (warp == 0 || warp == 3) {
        // ---------------- producers of A (warp 0) and B (warp 3); one lane issues ----------------
        // Two warps, since a copy costs its issuer about 80 cycles and each stage some 100 more.
        const bool isb = warp == 3;
        if (isb && a.early) asm volatile("griddepcontrol.wait;" ::: "memory");      // the row pass's output
        uint32_t it = 0;
        bool ok = true;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const MmTile T = tile_of(seq.tile(i));
            const int half = T.bn / CG;                            // rows of B this CTA stages
            // the smallest box that holds them (the rows too many are never multiplied)
            const int bx = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
            const uint32_t slice = uint32_t(16 << bx) * 128u;
            const uint32_t bytes = isb ? SL * slice : uint32_t(C::kMat * C::kABytes);
            const int r0 = T.n0 + int(rank) * half, m0 = T.m0 + int(rank) * 128;
            for (int ks = ks0; ks < ks1; ks++, it++) {
                const int s = it % S;
                if (it >= uint32_t(S) && !g_wait_long(g_smem(&empty[s]), ((it / S) - 1) & 1, &s_ab)) {
                    ok = false;
                    break;
                }
                uint32_t bar = g_smem(&full[s]);
                if (CG == 2) bar = g_mapa(bar, 0);                 // the pair's stages complete in its first CTA
                const uint32_t sa = g_smem(ring + s * C::kStage), sb = sa + C::kMat * C::kABytes;
                if (g_elect()) {
                    if (CG == 2) g_expect_remote(bar, bytes); else g_expect(bar, bytes);
                    if (isb) {
                        if (SL == 1) {
                            mm_copy2<CG>(sb, &a.b[bx], ks * C::kBK, r0, bar);
                        } else if (a.chunked & 2) {
                            mm_copy4<CG>(sb, &a.b[bx], 0, r0, ks * SL, 0, bar);
                        } else {
                            for (int l = 0; l < SL; l++)
                                mm_copy2<CG>(sb + l * slice, &a.b[bx], ks * C::kBK + l * (C::kBK / SL), r0, bar);
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < C::kMat; m++) {
                            const CUtensorMap* am = m ? &a.a1 : &a.a0;
                            const uint32_t d = sa + m * C::kABytes;
                            if constexpr (AMN) {                   // two halves of 64 features, SL * 64 rows each
                                if (a.chunked & 1) {
                                    mm_copy4<CG>(d, am, 0, ks * C::kBK, m0 / 64, T.e, bar);
                                } else {
                                    for (int h = 0; h < 2; h++)
                                        mm_copy3<CG>(d + h * (SL * 8192), am, m0 + h * 64, ks * C::kBK, T.e, bar);
                                }
                            } else if (SL == 1) {
                                mm_copy3<CG>(d, am, ks * C::kBK, m0, T.e, bar);
                            } else if (a.chunked & 1) {
                                mm_copy4<CG>(d, am, 0, m0, ks * SL, T.e, bar);
                            } else {
                                for (int l = 0; l < SL; l++)
                                    mm_copy3<CG>(d + l * 16384, am, ks * C::kBK + l * (C::kBK / SL), m0, T.e, bar);
                            }
                        }
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) fail();
        if (lane == 0) {
            s_issued[isb] = it;
            // the commits' arrivals here have landed before the CTA exits (the copies: see the end of the kernel)
            if (CG == 2 && !isb && !s_ab.flag)
                for (uint32_t n = it > uint32_t(S) ? it - S : 0; n < it; n++)
                    if (!g_wait(g_smem(&empty[n % S]), (n / S) & 1, &s_ab)) { fail(); break; }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (whole warp, one lane issues) ----------------
        // failure testing (moe_set_wait_hold): wait for a barrier that nothing completes
        if (s_hold && !g_wait_long(g_smem(&hold_bar), 0, &s_ab)) fail();
        uint32_t it = 0;
        MmHalves acc;
        bool ok = true;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const MmTile T = tile_of(seq.tile(i));
            const uint32_t idesc = I8 ? g_idesc_s8(T.bn, 128 * CG)
                                      : (g_idesc(T.bn, a.f16 != 0, 128 * CG) | (AMN ? G_IDESC_A_MN : 0u));
            const bool both = T.bn > C::kHalfRows;
            const uint32_t up = both ? NT : C::kHalfRows;
            const int half = T.bn / CG;
            const uint32_t slice = (half <= 16 ? 16u : half <= 32 ? 32u : half <= 64 ? 64u : 128u) * 128u;
            for (int kc = ks0; kc < ks1 && ok; kc += C::kChunk) {
                const int kend = min(ks1, kc + C::kChunk);
                const uint32_t h = both ? 0 : acc.next, d = tmem + h * C::kHalfCols;
                if ((acc.uses(h) && !g_wait_long(g_smem(&acc_empty[h]), (acc.uses(h) - 1) & 1, &s_ab)) ||
                    (both && acc.u1 && !g_wait_long(g_smem(&acc_empty[1]), (acc.u1 - 1) & 1, &s_ab))) {
                    ok = false;
                    break;
                }
                acc.take(h, both);
                g_fence_after();
                for (int ks = kc; ks < kend; ks++, it++) {
                    const int s = it % S;
                    if (!g_wait_long(g_smem(&full[s]), (it / S) & 1, &s_ab)) {
                        ok = false;
                        break;
                    }
                    g_fence_after();
                    const uint32_t sa = g_smem(ring + s * C::kStage), sb = sa + C::kMat * C::kABytes;
                    const int steps = min(4 * SL, (a.kdim - ks * C::kBK + C::kMmaK - 1) / C::kMmaK);
                    if (g_elect()) {
#pragma unroll
                        for (int k = 0; k < 4 * SL; k++) {
                            if (k >= steps) break;                 // K ends here
                            const uint64_t bd = g_desc(sb + (k / 4) * slice + (k % 4) * 32);
                            const uint32_t add = (k > 0 || ks > kc) ? 1u : 0u;
#pragma unroll
                            for (int m = 0; m < C::kMat; m++) {
                                const uint32_t am = sa + m * C::kABytes;
                                const uint64_t ad = AMN ? g_desc_mn(am + k * 2048, SL * 8192)
                                                        : g_desc(am + (k / 4) * 16384 + (k % 4) * 32);
                                if (I8) g_mma_s8<CG>(d + m * up, ad, bd, idesc, add);
                                else g_mma_f16<CG>(d + m * up, ad, bd, idesc, add);
                            }
                        }
                        g_commit_cg<CG>(g_smem(&empty[s]));
                        if (ks == kend - 1) {
                            g_commit_cg<CG>(g_smem(&acc_full[h]));
                            if (both) g_commit_cg<CG>(g_smem(&acc_full[1]));
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) fail();
        if (g_aborted(&s_ab)) {
            // the MMAs issued so far have finished reading shared memory before the CTA exits
            if (g_elect()) g_commit_own<CG>(g_smem(&drain));
            __syncwarp();
            if (lane == 0) g_drain_wait(g_smem(&drain), 0);
            __syncwarp();
        }
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");      // the row pass's scales
        // Two warps per lane quarter, taking alternate blocks of 16 rows.  Lanes exchange halves of a pair of rows, so
        // that each stores two features (4 bytes) of one row.
        const int q = warp & 3, hsel = (warp - 4) >> 2, odd = lane & 1;
        const uint32_t lane_addr = uint32_t(q * 32) << 16;
        constexpr int kScaleRegs = I8 ? (NT + 63) / 64 : 1;
        MmHalves use;
        bool ok = true;
        // A tile's coordinates and scales, on their way while the tile before is written
        struct Pre {
            MmTile T;
            float w0, w1, rs[kScaleRegs];                                     // my feature's scales, my blocks' rows'
        };
        auto fetch = [&](int ti) {
            Pre p;
            p.T = tile_of(seq.tile(ti));
            const int m = p.T.m0 + int(rank) * 128 + q * 32 + lane;
            p.w0 = p.w1 = 0.f;
            if (I8) {
                if (m < a.mdim) {
                    p.w0 = a.s0[size_t(p.T.e) * a.mdim + m];
                    if (GU) p.w1 = a.s1[size_t(p.T.e) * a.mdim + m];
                }
#pragma unroll
                for (int i = 0; i < kScaleRegs; i++) {
                    const int c = (4 * i + 2 * (lane >> 4) + hsel) * 16 + (lane & 15);   // lanes 0-15: block 2i, 16-31: 2i + 1
                    p.rs[i] = c < p.T.nval ? a.act_scale[p.T.n0 + c] : 0.f;
                }
            }
            return p;
        };
        auto release = [&](uint32_t half) {                                   // this warp has read the accumulator
            g_fence_before();
            __syncwarp();
            if (lane == 0) {
                const uint32_t bar = g_smem(&acc_empty[half]);
                if (CG == 2) g_arrive_remote_relaxed(g_mapa(bar, 0)); else g_arrive(bar);
            }
        };
        Pre next;
        if (seq.count > 0) next = fetch(0);
        for (int ti = 0; ti < seq.count && !g_aborted(&s_ab); ti++) {
            const Pre cur = next;
            const MmTile& T = cur.T;
            const int m = T.m0 + int(rank) * 128 + q * 32 + lane;            // my feature
            const bool mine = m < a.mdim;
            const float w0 = cur.w0, w1 = cur.w1;
            const float (&rs)[kScaleRegs] = cur.rs;
            // 16 bits: the partial sums of all chunks of K but the last
            float sum[C::kSums];
#pragma unroll
            for (int j = 0; j < C::kSums; j++) sum[j] = 0.f;
            if constexpr (!I8) {
                for (int left = ks1 - ks0; left > C::kChunk; left -= C::kChunk) {
                    const uint32_t part = use.next;
                    if (!g_wait_long(g_smem(&acc_full[part]), use.uses(part) & 1, &s_ab)) {
                        ok = false;
                        break;
                    }
                    g_fence_after();
#pragma unroll
                    for (int i = 0; i < C::kSums / 16; i++) {
                        const int c = (2 * i + hsel) * 16;
                        if (c >= T.nval) break;
                        uint32_t v[16];
                        g_ld16(tmem + lane_addr + part * C::kHalfCols + c, v);
                        g_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; j++) sum[16 * i + j] += __uint_as_float(v[j]);
                    }
                    release(part);
                    use.take(part, false);
                }
                if (!ok) break;
            }
            const bool both = T.bn > C::kHalfRows;
            const uint32_t h = both ? 0 : use.next;
            if (!g_wait_long(g_smem(&acc_full[h]), use.uses(h) & 1, &s_ab) ||
                (both && !g_wait_long(g_smem(&acc_full[1]), use.u1 & 1, &s_ab))) {
                ok = false;
                break;
            }
            g_fence_after();
            if (ti + 1 < seq.count) next = fetch(ti + 1);
            const uint32_t acc = tmem + lane_addr + h * C::kHalfCols, up = both ? NT : C::kHalfRows;
            // block i of this warp's, 16 columns, as bits (i is a constant after unrolling)
            auto block = [&](int i, uint32_t (&v)[16], uint32_t (&u)[16]) {
                g_ld16(acc + (2 * i + hsel) * 16, v);
                if constexpr (GU) g_ld16(acc + up + (2 * i + hsel) * 16, u);
                g_ld_wait();
                if constexpr (!I8)
#pragma unroll
                    for (int j = 0; j < 16; j++) v[j] = __float_as_uint(sum[16 * i + j] + __uint_as_float(v[j]));
            };
            uint16_t* dst = a.out + size_t(T.n0 + odd) * a.mdim + (m - odd);
            if constexpr (SPLIT) {
                // Block b of 16 rows is summed by CTA b mod z: hand it the others' partial sums, then wait for theirs.
                // A tile's partial sums go out once every CTA, this one among them, is through with the tile before
                // (red_free): a warp with nothing to send or to sum can then neither be lapped nor run ahead.
                if (ti > 0 && !g_wait_long(g_smem(&red_free), (ti - 1) & 1, &s_ab)) {
                    ok = false;
                    break;
                }
                const int nblk = (T.nval + 15) / 16, nown = (nblk - int(krank) + z - 1) / z;      // blocks; mine of them
                constexpr uint32_t kPart = C::kMat * 8192;                                        // a block's partial sums
                const uint32_t per = uint32_t(C::kBlocks / z + (C::kBlocks < z)) * kPart;         // room for one CTA's
                if (warp == 4 && lane == 0) g_expect(g_smem(&red_full), uint32_t(nown * (z - 1)) * kPart);
#pragma unroll
                for (int i = 0; i < (NT + 31) / 32; i++) {
                    const int b = 2 * i + hsel;
                    if (b >= nblk) break;
                    const uint32_t own = uint32_t(b) & (z - 1);
                    if (own == krank) continue;
                    const uint32_t to = g_mapa(g_smem(red), own) + (krank < own ? krank : krank - 1) * per +
                                        uint32_t(b / z) * kPart + uint32_t(q * 32 + lane) * 16;
                    const uint32_t bar = g_mapa(g_smem(&red_full), own);
                    uint32_t v[16], u[16];
                    block(i, v, u);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        g_st_async4(to + j * 2048, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], bar);
                        if constexpr (GU) g_st_async4(to + 8192 + j * 2048, u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3], bar);
                    }
                }
                if (!g_wait_long(g_smem(&red_full), ti & 1, &s_ab)) {
                    ok = false;
                    break;
                }
            }
#pragma unroll
            for (int i = 0; i < (NT + 31) / 32; i++) {
                const int c = (2 * i + hsel) * 16;
                if (c >= T.nval) break;
                if (SPLIT && (uint32_t(c / 16) & (z - 1)) != krank) continue;
                uint32_t v[16], u[16];
                block(i, v, u);
                if constexpr (SPLIT) {
                    mm_join<I8>(v, red + (c / 16 / z) * (C::kMat * 8192), C::kMat * 8192 * (C::kBlocks / z + (C::kBlocks < z)),
                                z, krank, q * 32 + lane);
                    if constexpr (GU)
                        mm_join<I8>(u, red + (c / 16 / z) * (C::kMat * 8192) + 8192,
                                    C::kMat * 8192 * (C::kBlocks / z + (C::kBlocks < z)), z, krank, q * 32 + lane);
                }
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; j++) {
                    if constexpr (I8) {
                        // the 32-bit sum is rounded to fp32 once (2^-24), then scaled
                        const float f = __shfl_sync(0xffffffffu, rs[i / 2], (i & 1) * 16 + j);
                        y[j] = float(int32_t(v[j])) * (f * w0);
                        // (silu with the approximate exponential and division: a relative error below
                        // (1 + |g|) 2^-21, beside the 2^-9 of the bf16 result; an exponential that overflows gives 0)
                        if constexpr (GU) y[j] = __fdividef(y[j], 1.0f + __expf(-y[j])) * (float(int32_t(u[j])) * (f * w1));
                    } else {
                        y[j] = __uint_as_float(v[j]);
                    }
                }
                uint16_t* row = dst + size_t(c) * a.mdim;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float r = __shfl_xor_sync(0xffffffffu, odd ? y[j] : y[j + 1], 1);
                    const float lo = odd ? r : y[j], hi = odd ? y[j + 1] : r;    // features m - odd, m - odd + 1
                    uint32_t p;
                    if (!I8 && a.f16) {
                        const __half2 h = __floats2half2_rn(lo, hi);
                        p = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                        p = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    if (mine && c + j + odd < T.nval) *reinterpret_cast<uint32_t*>(row + size_t(j) * a.mdim) = p;
                }
            }
            release(h);
            if (both) release(1);
            use.take(h, both);
            if (SPLIT && ti + 1 < seq.count) {
                if (lane == 0) g_arrive(g_smem(&red_done));
                __syncwarp();
                if (warp == 4) {                                              // for the CTA's epilogue warps
                    if (!g_wait_long(g_smem(&red_done), ti & 1, &s_ab)) {
                        ok = false;
                        break;
                    }
                    if (lane < z) g_arrive_remote(g_mapa(g_smem(&red_free), lane));
                }
            }
        }
        if (!ok) fail();
    }

    g_fence_before();
    __syncthreads();
    if (CG == 2) g_cluster_sync();
    if (SPLIT) {
        // A CTA that has seen all its partial sums has nothing more coming in; after an expired wait some may still
        // be on their way (and the barrier that counts them may never complete): let them land.
        g_cluster_sync_relaxed();
        if (tid == 0 && s_ab.flag)
            for (const unsigned long long t0 = g_timer(); g_timer() - t0 < 1000000ull;) __nanosleep(1000);
    }
    // after an expired wait, copies may be in flight for a stage that only some producers had issued: stand in for
    // the others' arrivals, then wait (bounded) for the last stages
    if (rank == 0 && tid == 0 && (CG == 2 || s_ab.flag)) {
        uint32_t n_[2 * CG], hi = 0;
        for (int i = 0; i < 2 * CG; i++) {
            n_[i] = i < 2 ? s_issued[i] : g_ld_cluster(g_mapa(g_smem(&s_issued[i & 1]), 1));
            hi = max(hi, n_[i]);
        }
        for (uint32_t n = hi > uint32_t(S) ? hi - S : 0; n < hi; n++)
            for (int i = 0; i < 2 * CG; i++)
                if (n >= n_[i]) g_arrive(g_smem(&full[n % S]));
        for (uint32_t n = hi > uint32_t(S) ? hi - S : 0; n < hi; n++) g_drain_wait(g_smem(&full[n % S]), (n / S) & 1);
    }
    g_fence_after();
    if (warp == 2) g_tmem_free<CG>(tmem, C::kTmem);
    if (CG == 2) {
        __syncwarp();
        g_cluster_sync();
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <bool I8, bool AMN, bool GU, int NT, int CG, int SL, bool SPLIT>
static int mm_launch(const MmArgs& a, cudaStream_t s) {
    using C = MmCfg<I8, AMN, GU, NT, CG, SL, SPLIT>;
    auto k = mm_kernel<I8, AMN, GU, NT, CG, SL, SPLIT>;
    constexpr int kFixed = C::kStages * C::kStage + C::kRedBytes + 1024;
    constexpr int kSmem = kFixed + 16 * kMaxE;
    int sms = 0;
    const int rc = mm_kernel_ready(reinterpret_cast<const void*>(k), kSmem, &sms);
    if (rc != MOE_OK) return rc;
    // (split K: as many clusters as there are tiles, if they fit)
    const int cl = SPLIT ? a.split : CG, grid = SPLIT ? std::max(1, std::min(a.split_tiles, sms / cl)) * cl : sms / cl * cl;
    return mm_launch_cfg(k, dim3(grid), dim3(MM_THREADS), kFixed + 16 * a.E, cl, s, a);
}

static int mm_mdim(const MmProblem& p) { return p.grad ? p.in_dim : p.out_dim; }
// About how many (expert, row block) pairs there are with blocks of nt rows
static int64_t mm_row_blocks(const MmProblem& p, int nt) {
    return std::max(int64_t(std::min(p.E, p.rows)), (int64_t(p.rows) + nt - 1) / nt);
}

// Tiles of 256 rows x 256 features on CTA pairs when the experts hold more than 64 rows on average (int8: 32, whose
// MMAs take half the time) and half the pairs get a tile; else 64 rows x 128 features on single CTAs.  Measured (4096
// -> 1536, us, single / pair): 352 experts of 47 rows 696 / 763 in bf16 (Zipf load 782 / 780), int8 gate/up 721 / 711
// (775 / 728), int8 down 368 / 375 (442 / 403); 44 experts of 1490 rows 1150 / 583; one expert of 300 rows
// 16 / 25, of 1000 rows (24 pair tiles) 29 / 29, of 3000 61 / 31; four of 150 rows (24 pair tiles, K 2048) 12 / 15.
// (Tiles of 16 rows were never faster than those of 64: 8 tokens over 352 experts 121 us against 117.)  The counts here and
// in mm_split are those of the whole part, 148 SMs; with fewer the launches adapt, the choice stays, at a cost in time alone.
static bool mm_pair(const MmProblem& p) {
    return p.rows > (p.i8 ? 32 : 64) * int64_t(p.E) && mm_row_blocks(p, 256) * ((mm_mdim(p) + 255) / 256) >= 37;
}
// 128-byte slices of K per stage: two; gate/up, with two weight matrices in a stage, one.  Stages in the ring: 4 (gate/up
// 5) on single CTAs, 3 in split tiles, 3 (gate/up 4) on pairs.
static int mm_slices(const MmProblem& p) { return p.w1 ? 1 : 2; }
// Few tiles leave SMs idle: then clusters of 2, 4 or 8 CTAs (gate/up: 4 at most) share each tile's K, as many as
// 148, 132 or 120 SMs hold at once, while each CTA still has two stages of K (one expert, 4096 -> 1536: 8 rows 18 us
// without, 8 with; int8 gate/up of 61 rows 18 / 12).  Pairs of CTAs also turn two rounds of long tiles, the second at
// most half full, into one and a half (two tokens that reach 16 of 352 experts of 4096 -> 1536, bf16: 43 us / 37; one
// expert of 1000 rows 30 / 26; but clusters of 4 over several rounds lose: one token, int8 gate/up, 19 / 32, and so do short
// tiles, 16 experts of 1536 -> 4096 in int8 19 / 26, and gate/up, 28 / 33).
static int mm_split(const MmProblem& p, int* tiles) {
    const int kdim = p.grad ? p.out_dim : p.in_dim;
    const int64_t t = mm_row_blocks(p, 64) * ((mm_mdim(p) + 127) / 128);
    const int bk = (p.i8 ? 128 : 64) * mm_slices(p), ks = (kdim + bk - 1) / bk;
    const int most[] = {148, 148, 132, 120};
    int z = 1;
    for (int i = 1; z < (p.w1 ? 4 : 8) && t * 2 * z <= most[i] && ks >= 4 * z &&
                    int64_t(2 * z - 1) * ((ks + 2 * z - 1) / (2 * z)) < ks; i++)
        z *= 2;
    // (of the experts, rows that spread evenly reach E (1 - exp(-rows / E)))
    const double reached = std::max(p.E * (1.0 - std::exp(-double(p.rows) / p.E)), double(p.rows) / 64);
    const double likely = reached * ((mm_mdim(p) + 127) / 128);
    if (!p.w1 && likely > 148 && likely <= 222 && ks >= 16) z = 2;
    *tiles = int(std::min<int64_t>(t, 1 << 20));
    return z;
}

static CUtensorMapDataType mm_type(bool i8, bool f16) {
    return i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : (f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16);
}

int launch_grouped_mm(const MmProblem& p, cudaStream_t s) {
    if (p.rows <= 0) return MOE_OK;
    const int ge = g_encoder();
    if (ge != MOE_OK) return ge;
    MmArgs a;
    memset(&a, 0, sizeof(a));
    const int el = p.i8 ? 1 : 2, bk = 128 / el;
    const CUtensorMapDataType ty = mm_type(p.i8, p.f16);
    // Tensor maps.  A row of 128-byte chunks, [chunks][rows][128 bytes], lets one copy bring both slices of a stage
    // (gradient: both halves of A's features); it needs rows of whole chunks, else each slice is a copy.
    const int sl = mm_slices(p);
    const uint64_t pitch = uint64_t(p.in_dim) * el, zp = pitch * p.out_dim;
    const int kdim = p.grad ? p.out_dim : p.in_dim;
    const bool ca = p.in_dim % bk == 0 && (p.grad || sl == 2), cb = kdim % bk == 0 && sl == 2;
    a.chunked = (ca ? 1 : 0) | (cb ? 2 : 0);
    const uint32_t bi = p.grad ? 64 : bk, br = p.grad ? 64 * sl : 128;       // box: elements of a row, rows
    int rc = MOE_OK;
    for (int m = 0; m < 2 && rc == MOE_OK; m++) {
        const void* w = m ? p.w1 : p.w0;
        CUtensorMap* map = m ? &a.a1 : &a.a0;
        if (!w) continue;
        rc = ca ? g_map4(map, ty, w, bi, p.out_dim, p.in_dim / bk, p.E, pitch, zp, br)
                : g_map3(map, ty, w, p.in_dim, p.out_dim, p.E, pitch, zp, bi, br);
    }
    const bool pair = mm_pair(p);
    const int boxes = pair ? MM_BOXES : 3;                // those a tile of this shape can ask for
    for (int i = 0; i < boxes && rc == MOE_OK; i++)
        rc = cb ? g_map4(&a.b[i], ty, p.act, bk, p.rows, kdim / bk, 1, uint64_t(kdim) * el, uint64_t(kdim) * el * p.rows,
                         16u << i)
                : g_map(&a.b[i], !p.i8, p.act, kdim, p.rows, uint64_t(kdim) * el, bk, 16u << i, true);
    if (rc != MOE_OK) return rc;
    a.offsets = p.offsets;
    a.act_scale = p.act_scale;
    a.s0 = p.s0;
    a.s1 = p.s1;
    a.out = p.out;
    a.status = p.status;
    a.E = p.E;
    a.mdim = p.grad ? p.in_dim : p.out_dim;
    a.kdim = kdim;
    a.rows = p.rows;
    a.f16 = p.f16;
    a.early = p.i8;
    a.mt_inv = mm_inverse(uint32_t(a.mdim + (pair ? 255 : 127)) / (pair ? 256u : 128u));
    if (pair) {
        // Experts of some hundred rows or fewer on average: the small ones' tiles wait for memory beside the large
        // ones' (65,536 rows, Zipf over 352 experts, int8 gate/up: 1096 us against 1171; over 44 experts the weights
        // read twice cost power: forward 774 against 723 us sustained).
        a.meet = p.rows <= 512 * int64_t(p.E);
        if (p.i8) return p.w1 ? mm_launch<true, false, true, 256, 2, 1, false>(a, s) : mm_launch<true, false, false, 256, 2, 2, false>(a, s);
        return p.grad ? mm_launch<false, true, false, 256, 2, 2, false>(a, s) : mm_launch<false, false, false, 256, 2, 2, false>(a, s);
    }
    a.split = mm_split(p, &a.split_tiles);
    if (a.split > 1) {
        if (p.i8) return p.w1 ? mm_launch<true, false, true, 64, 1, 1, true>(a, s) : mm_launch<true, false, false, 64, 1, 2, true>(a, s);
        return p.grad ? mm_launch<false, true, false, 64, 1, 2, true>(a, s) : mm_launch<false, false, false, 64, 1, 2, true>(a, s);
    }
    if (p.i8) return p.w1 ? mm_launch<true, false, true, 64, 1, 1, false>(a, s) : mm_launch<true, false, false, 64, 1, 2, false>(a, s);
    return p.grad ? mm_launch<false, true, false, 64, 1, 2, false>(a, s) : mm_launch<false, false, false, 64, 1, 2, false>(a, s);
}

}  // namespace moe
