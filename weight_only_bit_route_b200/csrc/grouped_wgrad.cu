// Gradient of the expert products by the weights, on the 5th-generation tensor cores:
//     dw[e, n, k] = sum over the rows r of expert e of dy[r, n] x[r, k]
// (0 for an expert without rows; with `accumulate` the sum is added to dw).
//
// The contraction runs along the rows, and both operands are stored row by row, so both enter the MMA stored
// along M (dy: 128 output features per CTA) and N (x: NT input features): 128-byte rows of 64 features, one per
// row r, as TMA lays them down.  Nothing is transposed in memory.
//
// A K block is 64 rows.  The expert's last block also brings rows of the next expert: the MMAs stop at the 16-row
// step that holds the last row, and the rows between it and the step's end are overwritten with zeros in shared
// memory, in both operands (a zero in one alone would still meet an infinity or a NaN in the other).
//
// A tile is (expert, 128 * CG output features, NT input features); a persistent CTA (or pair) takes every
// grid-th tile.  Warp roles: 0 TMA producer, 1 MMA issuer (in a pair: the first CTA's), 2 zeroes the last block's
// rows, 4-7 epilogue: tensor memory -> registers -> shared memory -> tile store (or fp32 reduction), which
// clips at the tensor's edges.  Sums are fp32 in tensor memory; one rounding to the output type.
#include <cstring>

#include "grouped_mm.cuh"
#include "mm_ptx.cuh"

namespace moe {

constexpr int WG_THREADS = 256;

template <int NT, int CG>
struct WgCfg {
    static constexpr int kBoxesB = NT / CG / 64;                  // 64-feature boxes of x this CTA stages
    static constexpr int kBox = 64 * 128;
    static constexpr int kStage = (2 + kBoxesB) * kBox;
    static constexpr int kOutBytes = 4 * 2 * 4096;                // per epilogue warp: two 32-row x 128-byte buffers
    static constexpr int kStages = (200 * 1024 - kOutBytes) / kStage;
    static constexpr int kTmem = 2 * NT;
    static_assert(kTmem <= 512 && kStages >= 3 && kStages <= 16, "tile shape");
};

struct WgArgs {
    CUtensorMap a, b;                    // dy [rows][out], x [rows][in]: boxes of 64 features x 64 rows
    CUtensorMap d;                       // dw [E][out][in]: boxes of 128 bytes x 32 rows
    const int32_t* offsets;
    int32_t* status;
    int E, out_dim, in_dim, rows;
    int f16, out_f32, accumulate;
};

template <int NT, int CG>
__global__ void __launch_bounds__(WG_THREADS, 1) wgrad_kernel(const __grid_constant__ WgArgs a) {
    using C = WgCfg<NT, CG>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[S], empty[S], tail[S], acc_full[2], acc_empty[2], drain, hold_bar;
    __shared__ uint32_t s_tmem, s_issued, s_tail;
    __shared__ int s_hold;
    __shared__ volatile GAbort s_ab;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? g_cta_rank() : 0u;
    const int MT = (a.out_dim + 128 * CG - 1) / (128 * CG), NTN = (a.in_dim + NT - 1) / NT;

    if (tid == 0) {
        for (int s = 0; s < S; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&full[s])), "r"(CG));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&empty[s])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&tail[s])));
        }
        for (int s = 0; s < 2; s++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&acc_full[s])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(g_smem(&acc_empty[s])), "r"(4 * CG));
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&drain)));
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(g_smem(&hold_bar)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_ab.flag = 0;
        s_issued = 0;
        s_tail = 0;
    }
    if (warp == 2) g_tmem_alloc<CG>(g_smem(&s_tmem), C::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        s_ab.limit_ns = g_limit_from(a.status);
        s_hold = g_hold_from(a.status);
    }
    uint8_t* ring = smem + ((1024u - (g_smem(smem) & 1023u)) & 1023u);
    uint8_t* outb = ring + S * C::kStage;
    int2* span = reinterpret_cast<int2*>(outb + C::kOutBytes);       // {first row, rows} of every expert
    for (int e = tid; e < a.E; e += WG_THREADS) {
        int base, n;
        mm_expert_rows(a.offsets, e, a.rows, a.status, base, n);
        span[e] = make_int2(base, n);
    }
    g_fence_before();
    __syncthreads();
    if (CG == 2) g_cluster_sync();
    g_fence_after();

    const uint32_t tmem = s_tmem;
    const int per_e = MT * NTN;
    const long long ntiles = (long long)a.E * per_e;
    const long long tile0 = blockIdx.x / CG, tstep = gridDim.x / CG;
    struct Tile { int e, base, n, m0, n0; };
    auto tile_of = [&](long long tile) {
        Tile t;
        t.e = int(tile / per_e);
        const int local = int(tile - (long long)t.e * per_e);
        const int2 sp = span[t.e];
        t.base = sp.x;
        t.n = sp.y;
        t.m0 = (local % MT) * (128 * CG);
        t.n0 = (local / MT) * NT;
        return t;
    };
    auto fail = [&]() {
        set_status(a.status, MOE_ERR_TIMEOUT);
        s_ab.flag = 1;
    };

    if (warp == 0) {
        // ---------------- producer (whole warp, one lane issues) ----------------
        uint32_t it = 0, tails = 0, tphase = 0;       // per stage: last fill was a tail; phase of its tail barrier
        bool ok = true;
        for (long long tile = tile0; tile < ntiles && ok && !g_aborted(&s_ab); tile += tstep) {
            const Tile T = tile_of(tile);
            const int KB = (T.n + 63) / 64;
            for (int kb = 0; kb < KB; kb++, it++) {
                const int s = it % S;
                if (it >= uint32_t(S) && !g_wait_w(g_smem(&empty[s]), ((it / S) - 1) & 1, &s_ab, 32)) {
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
                if (g_elect()) {
                    if (CG == 2 && !tl) g_expect_remote(bar, C::kStage); else g_expect(bar, C::kStage);
                    const uint32_t sa = g_smem(ring + s * C::kStage);
                    const int r = T.base + kb * 64, m0 = T.m0 + int(rank) * 128, n0 = T.n0 + int(rank) * (NT / CG);
#pragma unroll
                    for (int h = 0; h < 2 + C::kBoxesB; h++) {
                        const CUtensorMap* map = h < 2 ? &a.a : &a.b;
                        const int x = h < 2 ? m0 + h * 64 : n0 + (h - 2) * 64;
                        if (CG == 2) g_tma2d_pair(sa + h * C::kBox, map, x, r, bar);
                        else g_tma2d(sa + h * C::kBox, map, x, r, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) fail();
        if (lane == 0) {
            const uint32_t first = it > uint32_t(S) ? it - S : 0;
            if (s_ab.flag) {
                // copies that complete here have landed before the CTA exits (a pair's other copies: below)
                for (uint32_t n = first; n < it; n++) {
                    const uint32_t s = n % S;
                    if ((tails >> s) & 1) g_drain_wait(g_smem(&tail[s]), ((tphase >> s) & 1) ^ 1);
                    else if (CG == 1) g_drain_wait(g_smem(&full[s]), (n / S) & 1);
                }
            } else if (CG == 2) {
                // and so have the commits' arrivals
                for (uint32_t n = first; n < it; n++)
                    if (!g_wait(g_smem(&empty[n % S]), (n / S) & 1, &s_ab)) { fail(); break; }
            }
            s_issued = it;
            s_tail = tails;
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        // ---------------- MMA issuer (whole warp, one lane issues) ----------------
        if (s_hold && !g_wait_w(g_smem(&hold_bar), 0, &s_ab)) fail();
        const uint32_t idesc = g_idesc(NT, a.f16 != 0, 128 * CG) | G_IDESC_A_MN | G_IDESC_B_MN;
        uint32_t it = 0;
        int t = 0;
        bool ok = true;
        for (long long tile = tile0; tile < ntiles && ok && !g_aborted(&s_ab); tile += tstep) {
            const Tile T = tile_of(tile);
            if (T.n == 0) continue;
            const int KB = (T.n + 63) / 64;
            const uint32_t d = tmem + (t & 1) * NT;
            if (t >= 2 && !g_wait_w(g_smem(&acc_empty[t & 1]), ((t >> 1) - 1) & 1, &s_ab)) {
                ok = false;
                break;
            }
            g_fence_after();
            for (int kb = 0; kb < KB; kb++, it++) {
                const int s = it % S;
                if (!g_wait_w(g_smem(&full[s]), (it / S) & 1, &s_ab)) {
                    ok = false;
                    break;
                }
                g_fence_after();
                const uint32_t sa = g_smem(ring + s * C::kStage), sb = sa + 2 * C::kBox;
                const int steps = min(4, (T.n - kb * 64 + 15) / 16);
                if (g_elect()) {
                    for (int k = 0; k < steps; k++)
                        g_mma_f16<CG>(d, g_desc_mn(sa + k * 2048, C::kBox), g_desc_mn(sb + k * 2048, C::kBox), idesc,
                                      (k > 0 || kb > 0) ? 1u : 0u);
                    g_commit_cg<CG>(g_smem(&empty[s]));
                    if (kb == KB - 1) g_commit_cg<CG>(g_smem(&acc_full[t & 1]));
                }
                __syncwarp();
            }
            t++;
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
        for (long long tile = tile0; tile < ntiles && ok && !g_aborted(&s_ab); tile += tstep) {
            const Tile T = tile_of(tile);
            const int KB = (T.n + 63) / 64;
            it += KB;
            if (!(T.n & 15)) continue;
            const uint32_t s = (it - 1) % S;
            if (!g_wait_w(g_smem(&tail[s]), (tphase >> s) & 1, &s_ab, 32)) {
                ok = false;
                break;
            }
            tphase ^= 1u << s;
            const int v = T.n - (KB - 1) * 64, end = (v + 15) & ~15;
            // rows v to end of each box: contiguous 128-byte rows (the swizzle moves bytes within a row only)
            for (int i = lane; i < (end - v) * 8 * (2 + C::kBoxesB); i += 32) {
                const int box = i / ((end - v) * 8), c = i - box * ((end - v) * 8);
                *reinterpret_cast<uint4*>(ring + s * C::kStage + box * C::kBox + v * 128 + c * 16) = make_uint4(0, 0, 0, 0);
            }
            g_fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) g_arrive_remote(g_mapa(g_smem(&full[s]), 0)); else g_arrive(g_smem(&full[s]));
            }
            __syncwarp();
        }
        if (!ok) fail();
    } else if (warp >= 4) {
        // ---------------- epilogue ----------------
        const int q = warp & 3;
        const uint32_t lane_addr = uint32_t(q * 32) << 16;
        uint8_t* buf = outb + q * 8192;
        const int cols = a.out_f32 ? 32 : 64;                     // 128 bytes of a row
        int t = 0, nst = 0;
        bool ok = true;
        for (long long tile = tile0; tile < ntiles && !g_aborted(&s_ab); tile += tstep) {
            const Tile T = tile_of(tile);
            if (T.n == 0 && a.accumulate) continue;
            if (T.n > 0 && !g_wait_w(g_smem(&acc_full[t & 1]), (t >> 1) & 1, &s_ab, 32)) {
                ok = false;
                break;
            }
            g_fence_after();
            const uint32_t acc = tmem + lane_addr + (t & 1) * NT;
            const int m0 = T.m0 + int(rank) * 128 + q * 32;
            for (int c = 0; c < NT; c += cols) {
                const int x = T.n0 + c;
                if (m0 >= a.out_dim || x >= a.in_dim) break;       // nothing of this tile past the tensor's edge
                uint8_t* st = buf + (nst & 1) * 4096;
                if (lane == 0) g_store_wait_read<1>();              // the buffer's store before last has read it
                __syncwarp();
                uint4 o[8];
                if (T.n == 0) {
#pragma unroll
                    for (int i = 0; i < 8; i++) o[i] = make_uint4(0, 0, 0, 0);
                } else if (a.out_f32) {
                    uint32_t v[2][16];
                    g_ld16(acc + c, v[0]);
                    g_ld16(acc + c + 16, v[1]);
                    g_ld_wait();
#pragma unroll
                    for (int i = 0; i < 8; i++)
                        o[i] = make_uint4(v[i / 4][4 * (i % 4)], v[i / 4][4 * (i % 4) + 1], v[i / 4][4 * (i % 4) + 2],
                                          v[i / 4][4 * (i % 4) + 3]);
                } else {
                    uint32_t v[4][16];
#pragma unroll
                    for (int i = 0; i < 4; i++) g_ld16(acc + c + 16 * i, v[i]);
                    g_ld_wait();
                    uint32_t p[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const float lo = __uint_as_float(v[i / 8][2 * (i % 8)]), hi = __uint_as_float(v[i / 8][2 * (i % 8) + 1]);
                        if (a.f16) {
                            const __half2 h = __floats2half2_rn(lo, hi);
                            p[i] = *reinterpret_cast<const uint32_t*>(&h);
                        } else {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                            p[i] = *reinterpret_cast<const uint32_t*>(&h);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++) o[i] = make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
                }
#pragma unroll
                for (int i = 0; i < 8; i++) *reinterpret_cast<uint4*>(st + g_swz(lane, i)) = o[i];
                g_fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    g_store3d(&a.d, x, m0, T.e, g_smem(st), a.accumulate != 0);
                    g_store_commit();
                }
                nst++;
            }
            if (T.n > 0) {
                g_fence_before();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = g_smem(&acc_empty[t & 1]);
                    if (CG == 2) g_arrive_remote(g_mapa(bar, 0)); else g_arrive(bar);
                }
                t++;
            }
        }
        if (!ok) fail();
        if (lane == 0) g_store_wait();
        __syncwarp();
    }

    g_fence_before();
    __syncthreads();
    if (CG == 2) {
        g_cluster_sync();
        // after an expired wait: the pair's copies that complete on the first CTA's barriers (a stage that only
        // one CTA had issued gets the other's arrival from here)
        if (rank == 0 && tid == 0) {
            const uint32_t p0 = s_issued, p1 = g_ld_cluster(g_mapa(g_smem(&s_issued), 1));
            const uint32_t t1 = g_ld_cluster(g_mapa(g_smem(&s_tail), 1));
            const uint32_t lo = min(p0, p1), hi = max(p0, p1), tl = p0 >= p1 ? s_tail : t1;
            const bool aborted = s_ab.flag || g_ld_cluster(g_mapa(g_smem(const_cast<int*>(&s_ab.flag)), 1));
            if (aborted) {
                for (uint32_t n = hi > uint32_t(S) ? hi - S : 0; n < hi; n++) {
                    if ((tl >> (n % S)) & 1) continue;
                    if (n >= lo) g_arrive(g_smem(&full[n % S]));
                    g_drain_wait(g_smem(&full[n % S]), (n / S) & 1);
                }
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

template <int NT, int CG>
static int wg_launch(const WgArgs& a, cudaStream_t s) {
    using C = WgCfg<NT, CG>;
    auto k = wgrad_kernel<NT, CG>;
    constexpr int kFixed = C::kStages * C::kStage + C::kOutBytes + 1024;
    int sms = 0;
    const int rc = mm_kernel_ready(reinterpret_cast<const void*>(k), kFixed + 8 * kMaxE, &sms);
    if (rc != MOE_OK) return rc;
    return mm_launch_cfg(k, dim3(sms / CG * CG), dim3(WG_THREADS), kFixed + 8 * a.E, CG, s, a);
}

int launch_grouped_wgrad(const WgradProblem& p, cudaStream_t s) {
    const int ge = g_encoder();
    if (ge != MOE_OK) return ge;
    WgArgs a;
    memset(&a, 0, sizeof(a));
    const CUtensorMapDataType ty = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = MOE_OK;
    if (p.rows > 0) {
        rc = g_map(&a.a, true, p.dy, p.out_dim, p.rows, uint64_t(p.out_dim) * 2, 64, 64, true);
        if (rc == MOE_OK) rc = g_map(&a.b, true, p.x, p.in_dim, p.rows, uint64_t(p.in_dim) * 2, 64, 64, true);
    }
    const uint64_t pitch = uint64_t(p.in_dim) * (p.out_f32 ? 4 : 2);
    if (rc == MOE_OK)
        rc = g_map3(&a.d, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : ty, p.dw, p.in_dim, p.out_dim, p.E, pitch,
                    pitch * p.out_dim, p.out_f32 ? 32 : 64, 32);
    if (rc != MOE_OK) return rc;
    a.offsets = p.offsets;
    a.status = p.status;
    a.E = p.E;
    a.out_dim = p.out_dim;
    a.in_dim = p.in_dim;
    a.rows = p.rows;
    a.f16 = p.f16;
    a.out_f32 = p.out_f32;
    a.accumulate = p.accumulate;
    return wg_launch<128, 1>(a, s);
}

}  // namespace moe
