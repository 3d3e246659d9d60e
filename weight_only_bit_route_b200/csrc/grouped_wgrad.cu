// Gradient of the expert products by the weights, on the 5th-generation tensor cores:
//     dw[e, n, k] = sum over the rows r of expert e of dy[r, n] x[r, k]
// (0 for an expert without rows; with `accumulate` the sum is added to dw).
//
// The contraction runs along the rows, and both operands are stored row by row, so both enter the MMA stored
// along M (dy: 128 output features per CTA) and N (x: 256 input features): 128-byte rows of 64 features, one per
// row r, as TMA lays them down.  Nothing is transposed in memory.
//
// A K block is 64 rows.  The expert's last block also brings rows of the next expert: the MMAs stop at the 16-row
// step that holds the last row, and the rows between it and the step's end are overwritten with zeros in shared
// memory, in both operands (a zero in one alone would still meet an infinity or a NaN in the other).
//
// A tile is (expert, 128 * CG output features, 256 input features); a persistent CTA (or pair) takes a fixed
// sequence of them.  Warp roles: 0 and 3 TMA producers of dy and x, 1 MMA issuer (in a pair: the first CTA's), 2 zeroes the last block's
// rows, 4-11 epilogue: tensor memory -> registers -> shared memory -> tile store (or fp32 reduction), which
// clips at the tensor's edges.  The tensor core's fp32 sums are cut off rather than rounded, an error that grows with
// the number of rows; so only 512 rows are summed in tensor memory at a time, and the epilogue adds those partial
// sums in fp32 registers, rounded to nearest (a 65,536-row batch over 44 experts: 4.4e-6 of the result in one sum).
//
// Bound by the writes when experts hold few rows: 352 experts of 47 rows, 4096 x 1536, bf16, take 840 us in a burst and
// 977 in a loop, where the power cap counts; the stores alone (the same call without rows) 820 and 833, 5.4 TB/s.  With
// many rows by the operands' latency and the power cap: 65,536 rows over 44 experts, fp32, 760 us in a burst, 1085 TFLOP/s,
// the tensor pipe 68 % active, and 835 in a loop.  (128 sums a thread: ptxas keeps 7 to 13 words of the rest in local memory.)
#include <algorithm>
#include <cstring>

#include "grouped_mm.cuh"
#include "mm_ptx.cuh"

namespace moe {

constexpr int WG_THREADS = 384;
constexpr int WG_EPI_WARPS = 8;
constexpr int WG_NT = 256;                  // input features per tile
// CG: CTAs per tile; Z: CTAs that share a tile's rows

template <int CG, int Z>
struct WgCfg {
    static constexpr int kBoxesB = WG_NT / CG / 64;               // 64-feature boxes of x this CTA stages
    static constexpr int kBox = 64 * 128;
    static constexpr int kStage = (2 + kBoxesB) * kBox;
    // per epilogue warp: 32-row x 128-byte buffers; a pair's tiles are long, and the room serves the operands better
    static constexpr int kOutBufs = CG == 2 ? 1 : 2;
    static constexpr int kOutBytes = WG_EPI_WARPS * kOutBufs * 4096;
    static constexpr int kMaxStages = 6, kMinStages = (208 * 1024 - kOutBytes) / kStage;      // (with the largest table)
    static constexpr int kFixed = kOutBytes + 1024;               // beside the stages and 16 bytes per expert
    static constexpr int kHalf = WG_NT / 2;                       // columns of one epilogue warp
    static constexpr int kChunk = 8;                              // K blocks summed in tensor memory at a time
    static constexpr int kTmem = 2 * WG_NT;
    static_assert(Z == 1 || (CG == 1 && (Z - 1) * (kHalf / Z) * 4 * 32 * WG_EPI_WARPS <= kMinStages * kStage),
                  "split rows: the partial sums fit the ring");
    static_assert(kBoxesB % 2 == 0, "one copy brings two boxes");
    static_assert(kTmem <= 512 && kMinStages >= 3 && kMinStages <= kMaxStages, "tile shape");
};

struct WgArgs {
    CUtensorMap a, b;                    // dy [rows][out], x [rows][in]: boxes of 64 features x 64 rows
    CUtensorMap d;                       // dw [E][out][in]: boxes of 128 bytes x 32 rows
    const int32_t* offsets;
    int32_t* status;
    void* dw;
    int E, out_dim, in_dim, rows;
    int f16, out_f32, accumulate;
    int stages;                          // of the ring: as many as shared memory holds
    int chunked;                         // a and b are the views [1][features / 64][rows][64] (multiples of 64)
};

// Two fp32 values to 16 bits, low half first
__device__ __forceinline__ uint32_t wg_pair(float lo, float hi, int f16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return f16 ? *reinterpret_cast<const uint32_t*>(&h) : *reinterpret_cast<const uint32_t*>(&b);
}
// All threads of the cluster, each once per step, from wherever its role ends
__device__ __forceinline__ void wg_cluster_step() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
template <int W, int N>
__device__ __forceinline__ float4 wg_pick(const float (&sum)[N], int r, int j) {      // r and j are constants after unrolling
    return make_float4(sum[r * W + 4 * j], sum[r * W + 4 * j + 1], sum[r * W + 4 * j + 2], sum[r * W + 4 * j + 3]);
}

template <int CG, int Z>
__global__ void __launch_bounds__(WG_THREADS, 1) wgrad_kernel(const __grid_constant__ WgArgs a) {
    using C = WgCfg<CG, Z>;
    constexpr int SM = C::kMaxStages;
    const uint32_t S = uint32_t(a.stages);
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[SM], empty[SM], tail[SM], acc_full[2], acc_empty[2], drain, hold_bar;
    __shared__ uint32_t s_tmem, s_issued[2], s_tail[2], s_tphase[2];      // of the producers of A and of B
    __shared__ int s_hold;
    __shared__ volatile GAbort s_ab;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? g_cta_rank() : 0u;
    const uint32_t zr = Z > 1 ? g_cta_rank() : 0u;          // this CTA's share of a tile's rows
    const int MT = (a.out_dim + 128 * CG - 1) / (128 * CG), NTN = (a.in_dim + WG_NT - 1) / WG_NT;

    if (warp == 4 && (lane == 2 || (lane < 2 && a.rows > 0))) g_prefetch_map(lane == 0 ? &a.a : lane == 1 ? &a.b : &a.d);
    if (tid == 0) {
        for (int s = 0; s < SM; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&full[s])), "r"(2 * CG));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&empty[s])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 2;" ::"r"(g_smem(&tail[s])));
        }
        for (int s = 0; s < 2; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&acc_full[s])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&acc_empty[s])), "r"(WG_EPI_WARPS * CG));
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&drain)));
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&hold_bar)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_ab.flag = 0;
        for (int i = 0; i < 2; i++) s_issued[i] = s_tail[i] = s_tphase[i] = 0;
    }
    if (warp == 2) g_tmem_alloc<CG>(g_smem(&s_tmem), C::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == WG_THREADS - 1) {
        s_ab.limit_ns = g_limit_from(a.status);
        s_hold = g_hold_from(a.status);
    }
    uint8_t* ring = smem + ((1024u - (g_smem(smem) & 1023u)) & 1023u);
    uint8_t* outb = ring + S * C::kStage;
    int4* span = reinterpret_cast<int4*>(outb + C::kOutBytes);       // {expert, first row, rows} of every expert
    constexpr bool kSort = CG == 2;                                   // many rows: from the most to the fewest
    {
        int* rows_of = reinterpret_cast<int*>(ring);                 // scratch until the copies start
        const int pad = (a.E + 3) & ~3;
        bool good = true;
        for (int e = tid; e < pad; e += WG_THREADS) {
            int base = 0, n = 0;
            if (e < a.E) good &= mm_expert_rows(a.offsets, e, a.rows, base, n);
            if (kSort) rows_of[e] = n;
            else if (e < a.E) span[e] = make_int4(e, base, n, 0);
        }
        const bool clip = __syncthreads_or(!good);
        if (clip) {
            if (tid == 0) set_status(a.status, MOE_ERR_DEVICE_INDEX);
            for (int e = tid; e < a.E; e += WG_THREADS) {
                const int2 r = mm_clipped_rows(a.offsets, e, a.rows);
                if (kSort) rows_of[e] = r.y;
                else span[e] = make_int4(e, r.x, r.y, 0);
            }
            __syncthreads();
        }
        if (kSort) {
            for (int e = tid; e < a.E; e += WG_THREADS)
                span[mm_rank(rows_of, a.E, e)] =
                    make_int4(e, clip ? mm_clipped_rows(a.offsets, e, a.rows).x : a.offsets[e], rows_of[e], 0);
            g_fence_proxy_async();                                   // before the copies write the scratch
        }
    }
    g_fence_before();
    __syncthreads();
    if (CG == 2) g_cluster_sync();
    g_fence_after();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // (they wait for this kernel's end themselves)

    const uint32_t tmem = s_tmem;
    const int per_e = MT * NTN;
    const MmSequence seq(int(blockIdx.x) / (CG * Z), int(gridDim.x) / (CG * Z), a.E * per_e, kSort, false);
    struct Tile { int e, base, n, m0, n0; };                // base, n: the rows this CTA sums
    auto tile_of = [&](int tile) {
        Tile t;
        const int rank = tile / per_e, local = tile - rank * per_e;
        const int4 sp = span[rank];
        t.e = sp.x;
        t.base = sp.y;
        t.n = sp.z;
        if (Z > 1) {                                        // whole blocks of 64 rows to each
            const int per = (t.n + 64 * Z - 1) / (64 * Z) * 64, first = min(int(zr) * per, t.n);
            t.base += first;
            t.n = min(per, t.n - first);
        }
        t.m0 = (local % MT) * (128 * CG);
        t.n0 = (local / MT) * WG_NT;
        return t;
    };
    auto fail = [&]() {
        set_status(a.status, MOE_ERR_TIMEOUT);
        s_ab.flag = 1;
    };

    if (warp == 0 || warp == 3) {
        // ---------------- producers of A (warp 0) and B (warp 3); one lane issues ----------------
        constexpr int kMaxBoxes = C::kBoxesB > 2 ? C::kBoxesB : 2;
        const bool isb = warp == 3;
        const CUtensorMap* map = isb ? &a.b : &a.a;
        const int boxes = isb ? C::kBoxesB : 2;
        const uint32_t bytes = uint32_t(boxes) * C::kBox;
        uint32_t it = 0, s = 0, ph = 0;               // stages issued; the next one and the parity of its round
        uint32_t tails = 0, tphase = 0;               // per stage: last fill was a tail; phase of its tail barrier
        bool ok = true;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const Tile T = tile_of(seq.tile(i));
            const int KB = (T.n + 63) / 64;
            const int x0 = isb ? T.n0 + int(rank) * (WG_NT / CG) : T.m0 + int(rank) * 128;
            for (int kb = 0; kb < KB; kb++, it++) {
                if (!g_wait_long(g_smem(&empty[s]), ph ^ 1, &s_ab)) {      // (a new barrier's phase before the first is over)
                    ok = false;
                    break;
                }
                // a block whose rows need zeros completes on this CTA's own tail barrier; warp 2 passes it on
                const bool tl = kb == KB - 1 && (T.n & 15);
                uint32_t bar;
                if (tl) {
                    bar = g_smem(&tail[s]);
                    tails |= 1u << s;
                    tphase ^= 1u << s;
                } else {
                    bar = g_smem(&full[s]);
                    if (CG == 2) bar = g_mapa(bar, 0);
                    tails &= ~(1u << s);
                }
                const uint32_t d = g_smem(ring + s * C::kStage) + (isb ? 2 * C::kBox : 0);
                const int r = T.base + kb * 64;
                if (g_elect()) {
                    if (CG == 2 && !tl) g_expect_remote(bar, bytes); else g_expect(bar, bytes);
#pragma unroll
                    for (int h = 0; h < kMaxBoxes; h++) {
                        if (h >= boxes) break;
                        if (a.chunked) {                           // two boxes of 64 features in one copy
                            if (h & 1) continue;
                            if (CG == 2) g_tma4d_pair(d + h * C::kBox, map, 0, r, x0 / 64 + h, 0, bar);
                            else g_tma4d(d + h * C::kBox, map, 0, r, x0 / 64 + h, 0, bar);
                        } else {
                            if (CG == 2) g_tma2d_pair(d + h * C::kBox, map, x0 + h * 64, r, bar);
                            else g_tma2d(d + h * C::kBox, map, x0 + h * 64, r, bar);
                        }
                    }
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) fail();
        if (lane == 0) {
            s_issued[isb] = it;
            s_tail[isb] = tails;
            s_tphase[isb] = tphase;
            // the commits' arrivals here have landed before the CTA exits (the copies: see the end of the kernel)
            if (CG == 2 && !isb && !s_ab.flag)
                for (uint32_t n = it > S ? it - S : 0; n < it; n++)
                    if (!g_wait(g_smem(&empty[n % S]), (n / S) & 1, &s_ab)) { fail(); break; }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (whole warp, one lane issues) ----------------
        if (s_hold && !g_wait_long(g_smem(&hold_bar), 0, &s_ab)) fail();
        const uint32_t idesc = g_idesc(WG_NT, a.f16 != 0, 128 * CG) | G_IDESC_A_MN | G_IDESC_B_MN;
        uint32_t s = 0, ph = 0;
        int t = 0;
        bool ok = true;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const Tile T = tile_of(seq.tile(i));
            if (T.n == 0) continue;
            const int KB = (T.n + 63) / 64;
            for (int kb = 0; kb < KB && ok; kb++) {
                const int kc = kb % C::kChunk;
                const uint32_t d = tmem + (t & 1) * WG_NT;
                if (kc == 0) {
                    if (t >= 2 && !g_wait_long(g_smem(&acc_empty[t & 1]), ((t >> 1) - 1) & 1, &s_ab)) {
                        ok = false;
                        break;
                    }
                    g_fence_after();
                }
                if (!g_wait_long(g_smem(&full[s]), ph, &s_ab)) {
                    ok = false;
                    break;
                }
                g_fence_after();
                const uint32_t sa = g_smem(ring + s * C::kStage), sb = sa + 2 * C::kBox;
                const int steps = min(4, (T.n - kb * 64 + 15) / 16);
                const bool last = kc == C::kChunk - 1 || kb == KB - 1;
                if (g_elect()) {
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (k < steps) g_mma_f16<CG>(d, g_desc_mn(sa + k * 2048, C::kBox), g_desc_mn(sb + k * 2048, C::kBox), idesc,
                                      (k > 0 || kc > 0) ? 1u : 0u);
                    g_commit_cg<CG>(g_smem(&empty[s]));
                    if (last) g_commit_cg<CG>(g_smem(&acc_full[t & 1]));
                }
                __syncwarp();
                if (last) t++;
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        if (!ok) fail();
        if (g_aborted(&s_ab)) {
            if (g_elect()) g_commit_own<CG>(g_smem(&drain));
            __syncwarp();
            if (lane == 0) g_drain_wait(g_smem(&drain), 0);
            __syncwarp();
        }
    } else if (warp == 2) {
        // ---------------- zeros behind an expert's last row ----------------
        uint32_t it = 0, tphase = 0;
        bool ok = true;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const Tile T = tile_of(seq.tile(i));
            const int KB = (T.n + 63) / 64;
            it += KB;
            if (!(T.n & 15)) continue;
            const uint32_t s = (it - 1) % S;
            if (!g_wait_long(g_smem(&tail[s]), (tphase >> s) & 1, &s_ab)) {
                ok = false;
                break;
            }
            tphase ^= 1u << s;
            const int v = T.n - (KB - 1) * 64, end = (v + 15) & ~15;
            // rows v to end of each box: contiguous 128-byte rows (the swizzle moves bytes within a row only)
            for (int j = lane; j < (end - v) * 8 * (2 + C::kBoxesB); j += 32) {
                const int box = j / ((end - v) * 8), c = j - box * ((end - v) * 8);
                *reinterpret_cast<uint4*>(ring + s * C::kStage + box * C::kBox + v * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            g_fence_proxy_async();
            __syncwarp();
            if (lane < 2) {                            // for both producers
                if (CG == 2) g_arrive_remote(g_mapa(g_smem(&full[s]), 0)); else g_arrive(g_smem(&full[s]));
            }
            __syncwarp();
        }
        if (!ok) fail();
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        const int q = warp & 3, c0 = (warp - 4) / 4 * C::kHalf;      // my lanes and columns
        const uint32_t lane_addr = uint32_t(q * 32) << 16;
        uint8_t* buf = outb + (warp - 4) * (C::kOutBufs * 4096);
        int t = 0, nst = 0;
        bool ok = true, finished = false;
        for (int i = 0; i < seq.count && ok && !g_aborted(&s_ab); i++) {
            const Tile T = tile_of(seq.tile(i));
            if (Z == 1 && T.n == 0 && a.accumulate) continue;
            const int m0 = T.m0 + int(rank) * 128 + q * 32, x0 = T.n0 + c0;
            float sum[C::kHalf];
#pragma unroll
            for (int i = 0; i < C::kHalf; i++) sum[i] = 0.f;
            const int chunks = ((T.n + 63) / 64 + C::kChunk - 1) / C::kChunk;
            for (int ch = 0; ch < chunks; ch++, t++) {
                if (!g_wait_long(g_smem(&acc_full[t & 1]), (t >> 1) & 1, &s_ab)) {
                    ok = false;
                    break;
                }
                g_fence_after();
                const uint32_t acc = tmem + lane_addr + (t & 1) * WG_NT + c0;
#pragma unroll
                for (int c = 0; c < C::kHalf; c += 16) {
                    uint32_t v[16];
                    g_ld16(acc + c, v);
                    g_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i++) sum[c + i] += __uint_as_float(v[i]);
                }
                g_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = g_smem(&acc_empty[t & 1]);
                    if (CG == 2) g_arrive_remote_relaxed(g_mapa(bar, 0)); else g_arrive(bar);
                }
            }
            if (!ok) break;
            if constexpr (Z > 1) {
                // (one tile per CTA at most.)  Each CTA of the cluster finishes a Z-th of every warp's columns.
                constexpr int W = C::kHalf / Z;
                wg_cluster_step();                          // every CTA's MMAs are done: the rings are free
#pragma unroll
                for (int r = 0; r < Z; r++) {
                    if (r == int(zr)) continue;
                    const uint32_t to = g_mapa(g_smem(ring), r) +
                                        ((zr < uint32_t(r) ? zr : zr - 1) * WG_EPI_WARPS + (warp - 4)) * (W * 128) + lane * 16;
#pragma unroll
                    for (int j = 0; j < W / 4; j++)
                        g_st_cluster4(to + j * 512, __float_as_uint(sum[r * W + 4 * j]), __float_as_uint(sum[r * W + 4 * j + 1]),
                                      __float_as_uint(sum[r * W + 4 * j + 2]), __float_as_uint(sum[r * W + 4 * j + 3]));
                }
                wg_cluster_step();
                float mine[W];
#pragma unroll
                for (int j = 0; j < W; j++) mine[j] = 0.f;
#pragma unroll
                for (int r = 0; r < Z; r++) {               // in the order of the CTAs
                    const uint8_t* p = ring + ((zr > uint32_t(r) ? r : r - 1) * WG_EPI_WARPS + (warp - 4)) * (W * 128) + lane * 16;
#pragma unroll
                    for (int j = 0; j < W / 4; j++) {
                        float4 v;
                        if (r == int(zr)) v = wg_pick<W>(sum, r, j);
                        else v = *reinterpret_cast<const float4*>(p + j * 512);
                        mine[4 * j] += v.x;
                        mine[4 * j + 1] += v.y;
                        mine[4 * j + 2] += v.z;
                        mine[4 * j + 3] += v.w;
                    }
                }
                const int row = m0 + lane, x = x0 + int(zr) * W;
                if (row < a.out_dim) {
                    const size_t at = (size_t(T.e) * a.out_dim + row) * a.in_dim + x;
#pragma unroll
                    for (int j = 0; j < W; j += 8) {        // (in_dim is a multiple of 8)
                        if (x + j >= a.in_dim) break;
                        if (a.out_f32) {
                            float* d = static_cast<float*>(a.dw) + at + j;
#pragma unroll
                            for (int i = 0; i < 8; i += 4) {
                                float4 o = make_float4(mine[j + i], mine[j + i + 1], mine[j + i + 2], mine[j + i + 3]);
                                if (a.accumulate) {
                                    const float4 b = *reinterpret_cast<const float4*>(d + i);
                                    o = make_float4(o.x + b.x, o.y + b.y, o.z + b.z, o.w + b.w);
                                }
                                *reinterpret_cast<float4*>(d + i) = o;
                            }
                        } else {
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dw) + at + j) =
                                make_uint4(wg_pair(mine[j], mine[j + 1], a.f16), wg_pair(mine[j + 2], mine[j + 3], a.f16),
                                           wg_pair(mine[j + 4], mine[j + 5], a.f16), wg_pair(mine[j + 6], mine[j + 7], a.f16));
                        }
                    }
                }
                finished = true;
                continue;
            }
            // 128 bytes of 32 rows at a time; nothing of the tile is stored past the tensor's edge
            auto put = [&](int x, auto piece) {
                if (m0 >= a.out_dim || x >= a.in_dim) return;
                uint8_t* st = buf + (nst % C::kOutBufs) * 4096;
                if (lane == 0) g_store_wait_read<C::kOutBufs - 1>();   // the buffer's last store has read it
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; i++) *reinterpret_cast<uint4*>(st + g_swz(lane, i)) = piece(i);
                g_fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    g_store3d(&a.d, x, m0, T.e, g_smem(st), a.accumulate != 0);
                    g_store_commit();
                }
                nst++;
            };
            if (a.out_f32) {
#pragma unroll
                for (int c = 0; c < C::kHalf; c += 32)
                    put(x0 + c, [&](int i) {
                        return make_uint4(__float_as_uint(sum[c + 4 * i]), __float_as_uint(sum[c + 4 * i + 1]),
                                          __float_as_uint(sum[c + 4 * i + 2]), __float_as_uint(sum[c + 4 * i + 3]));
                    });
            } else {
#pragma unroll
                for (int c = 0; c < C::kHalf; c += 64)
                    put(x0 + c, [&](int i) {
                        const float* p = sum + c + 8 * i;
                        return make_uint4(wg_pair(p[0], p[1], a.f16), wg_pair(p[2], p[3], a.f16), wg_pair(p[4], p[5], a.f16),
                                          wg_pair(p[6], p[7], a.f16));
                    });
            }
        }
        if (!ok) fail();
        if (lane == 0) g_store_wait();
        __syncwarp();
        if (Z > 1 && !finished) {                           // no tile, or an expired wait: the other CTAs still count on it
            wg_cluster_step();
            wg_cluster_step();
        }
    }
    if (Z > 1 && warp < 4) {
        __syncwarp();
        wg_cluster_step();
        wg_cluster_step();
    }

    g_fence_before();
    __syncthreads();
    // After an expired wait copies may be in flight, for a stage that only some producers had issued: stand in for the
    // others' arrivals, then wait (bounded) for the last stages.  First what completes on this CTA's tail barriers ...
    if (tid == 0 && s_ab.flag) {
        const int big = s_issued[1] > s_issued[0];
        const uint32_t hi = s_issued[big], tl = s_tail[big], ph = s_tphase[big];
        for (uint32_t n = hi > S ? hi - S : 0; n < hi; n++) {
            const uint32_t s = n % S;
            if (!((tl >> s) & 1)) continue;
            if (n >= s_issued[!big]) g_arrive(g_smem(&tail[s]));
            g_drain_wait(g_smem(&tail[s]), ((ph >> s) & 1) ^ 1);
        }
    }
    if (CG == 2) {
        __syncthreads();
        g_cluster_sync();
    }
    // ... then what completes on the full barriers (a pair's: the first CTA's)
    if (rank == 0 && tid == 0) {
        bool aborted = s_ab.flag;
        if (CG == 2) aborted |= g_ld_cluster(g_mapa(g_smem(const_cast<int*>(&s_ab.flag)), 1)) != 0;
        if (aborted) {
            uint32_t n_[2 * CG], hi = 0, tl = 0;
            for (int i = 0; i < 2 * CG; i++) {
                n_[i] = i < 2 ? s_issued[i] : g_ld_cluster(g_mapa(g_smem(&s_issued[i & 1]), 1));
                if (n_[i] >= hi) {
                    hi = n_[i];
                    tl = i < 2 ? s_tail[i] : g_ld_cluster(g_mapa(g_smem(&s_tail[i & 1]), 1));
                }
            }
            for (uint32_t n = hi > S ? hi - S : 0; n < hi; n++) {
                if ((tl >> (n % S)) & 1) continue;
                for (int i = 0; i < 2 * CG; i++)
                    if (n >= n_[i]) g_arrive(g_smem(&full[n % S]));
                g_drain_wait(g_smem(&full[n % S]), (n / S) & 1);
            }
        }
    }
    g_fence_after();
    if (warp == 2) g_tmem_free<CG>(tmem, C::kTmem);
    if (CG == 2) {
        __syncwarp();
        g_cluster_sync();
    }
}

template <int CG, int Z>
static int wg_launch(const WgArgs& a, cudaStream_t s) {
    using C = WgCfg<CG, Z>;
    auto k = wgrad_kernel<CG, Z>;
    // Dynamic shared memory: what a block may have beside the kernel's static 1 KB.
    constexpr int kRoom = 227 * 1024 - 1024;
    static_assert(C::kMinStages * C::kStage + C::kFixed + 16 * kMaxE <= kRoom, "the largest table fits");
    int sms = 0;
    const int rc = mm_kernel_ready(reinterpret_cast<const void*>(k), kRoom, &sms);
    if (rc != MOE_OK) return rc;
    WgArgs args = a;
    args.stages = std::min(C::kMaxStages, (kRoom - C::kFixed - 16 * a.E) / C::kStage);
    const int smem = args.stages * C::kStage + C::kFixed + 16 * a.E;
    const int tiles = a.E * ((a.out_dim + 128 * CG - 1) / (128 * CG)) * ((a.in_dim + WG_NT - 1) / WG_NT);
    return mm_launch_cfg(k, dim3(Z > 1 ? tiles * Z : sms / CG * CG), dim3(WG_THREADS), smem, CG * Z, s, args);
}

int launch_grouped_wgrad(const WgradProblem& p, cudaStream_t s) {
    const int ge = g_encoder();
    if (ge != MOE_OK) return ge;
    WgArgs a;
    memset(&a, 0, sizeof(a));
    const CUtensorMapDataType ty = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = MOE_OK;
    a.chunked = p.out_dim % 64 == 0 && p.in_dim % 64 == 0;
    if (p.rows > 0 && a.chunked) {
        rc = g_map4(&a.a, ty, p.dy, 64, p.rows, p.out_dim / 64, 1, uint64_t(p.out_dim) * 2, uint64_t(p.out_dim) * 2 * p.rows, 64);
        if (rc == MOE_OK)
            rc = g_map4(&a.b, ty, p.x, 64, p.rows, p.in_dim / 64, 1, uint64_t(p.in_dim) * 2, uint64_t(p.in_dim) * 2 * p.rows, 64);
    } else if (p.rows > 0) {
        rc = g_map(&a.a, true, p.dy, p.out_dim, p.rows, uint64_t(p.out_dim) * 2, 64, 64, true);
        if (rc == MOE_OK) rc = g_map(&a.b, true, p.x, p.in_dim, p.rows, uint64_t(p.in_dim) * 2, 64, 64, true);
    }
    const uint64_t pitch = uint64_t(p.in_dim) * (p.out_f32 ? 4 : 2);
    if (rc == MOE_OK)
        rc = g_map3(&a.d, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : ty, p.dw, p.in_dim, p.out_dim, p.E, pitch,
                    pitch * p.out_dim, p.out_f32 ? 32 : 64, 32);
    if (rc != MOE_OK) return rc;
    // tile numbers are 32-bit
    if (int64_t(p.E) * ((p.out_dim + 127) / 128) * ((p.in_dim + 127) / 128) > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    a.offsets = p.offsets;
    a.status = p.status;
    a.dw = p.dw;
    a.E = p.E;
    a.out_dim = p.out_dim;
    a.in_dim = p.in_dim;
    a.rows = p.rows;
    a.f16 = p.f16;
    a.out_f32 = p.out_f32;
    a.accumulate = p.accumulate;
    // (The counts below are those of the whole part, 148 SMs.)
    // Few tiles (33 clusters of four run at once) and many rows: clusters of four share a tile's rows (one expert of
    // 8192 rows, 1000 x 264: 29 us).
    const int64_t tiles = int64_t(p.E) * ((a.out_dim + 127) / 128) * ((a.in_dim + 255) / 256);
    if (tiles * 4 <= 132 && p.rows >= 512 * int64_t(p.E)) return wg_launch<1, 4>(a, s);
    // Up to 128 rows per expert the tiles are short and the writes bound them: single CTAs keep more of them in flight;
    // above, a pair loads a quarter less per tile.  Measured (4096 x 1536, bf16, us, single / pair): 352 experts of 47
    // rows 836 / 1044; 44 of 93 rows 138 / 162, of 186 182 / 166, of 372 281 / 236, of 1490 852 / 686.
    const int64_t pairs = int64_t(p.E) * ((a.out_dim + 255) / 256) * ((a.in_dim + 255) / 256);
    return p.rows > 128 * int64_t(p.E) && pairs >= 37 ? wg_launch<2, 1>(a, s) : wg_launch<1, 1>(a, s);
}

}  // namespace moe
