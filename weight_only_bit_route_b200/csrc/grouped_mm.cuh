// Internal declarations of the expert products in 16 and 8 bits (grouped_mm.cu, grouped_wgrad.cu, quant_int8.cu).
#pragma once

#include "moe_internal.cuh"

namespace moe {

constexpr int kMmMaxRows = INT32_MAX - 1024;     // a tile's row numbers stay 32-bit

// The rows of expert e: [base, base + n).  False if its offsets leave [0, rows] or decrease: then every expert's rows are
// those of mm_clipped_rows.
__device__ __forceinline__ bool mm_expert_rows(const int32_t* offsets, int e, int rows, int& base, int& n) {
    base = offsets[e];
    const int end = offsets[e + 1];
    n = end - base;
    return base >= 0 && end >= base && end <= rows;
}
// The same with every offset raised to the largest before it and clipped to [0, rows]: no index derived from them leaves
// the rows, and no two experts share one (the tiles of all of them then stay within 32 bits, and none is written twice).
__device__ __forceinline__ int2 mm_clipped_rows(const int32_t* offsets, int e, int rows) {
    int base = 0;
    for (int i = 0; i <= e; i++) base = max(base, min(offsets[i], rows));
    return make_int2(base, max(base, min(offsets[e + 1], rows)) - base);
}

// The tiles of worker p of P, as a sequence: tile p of each round of P, in snake order (every second round runs
// backwards) where the tiles are listed from the largest to the smallest, so that the workers' sums stay within
// about one small tile of each other.  meet: the upper half of the workers starts from the small end, so that
// compute-bound and memory-bound tiles run at the same time (at the price of reading a large expert's weights twice).
struct MmSequence {
    int p, P, count;
    bool snake, back;
    __device__ __forceinline__ MmSequence(int p_, int P_, int ntiles, bool snake_, bool meet)
        : p(p_), P(P_), snake(snake_), back(meet && p_ >= P_ / 2) {
        const int full = ntiles / P, rem = ntiles - full * P;
        count = full + (at(full) < rem ? 1 : 0);
    }
    __device__ __forceinline__ int at(int round) const { return snake && (round & 1) ? P - 1 - p : p; }
    __device__ __forceinline__ int tile(int i) const {
        const int round = back ? count - 1 - i : i;
        return round * P + at(round);
    }
};

// n / d for 0 <= n, with inv = mm_inverse(d): a division costs some hundred cycles, and every role would make one per tile
__device__ __forceinline__ int mm_div(int n, int d, uint32_t inv) {
    const int q = int(__umulhi(uint32_t(n), inv));                   // n / d, or one less
    return q + ((q + 1) * d <= n ? 1 : 0);
}
inline uint32_t mm_inverse(uint32_t d) { return d > 1 ? uint32_t((uint64_t(1) << 32) / d) : 0xffffffffu; }

// Position of expert e among the experts by rows, most first (n: rows of the E experts in shared memory, zeros up to
// the next multiple of 4).
__device__ __forceinline__ int mm_rank(const int* n, int E, int e) {
    const int mine = n[e];
    int r = 0;
    for (int i = 0; i < E; i += 4) {
        const int4 v = *reinterpret_cast<const int4*>(n + i);
        r += (v.x > mine || (v.x == mine && i < e)) + (v.y > mine || (v.y == mine && i + 1 < e)) +
             (v.z > mine || (v.z == mine && i + 2 < e)) + (v.w > mine || (v.w == mine && i + 3 < e));
    }
    return r;
}

struct MmProblem {
    const void* act;             // rows of the contraction: x or codes [rows, in], dy [rows, out] (grad)
    const void* w0; const void* w1;      // weights [E, out, in]; w1: up (int8 gate/up), else null
    const float* s0; const float* s1;    // int8: channel scales [E, out]
    const float* act_scale;              // int8: row scales [rows], times the routing weight
    const int32_t* offsets;              // [E + 1]
    uint16_t* out;                       // [rows, out], [rows, in] (grad)
    int32_t* status;
    int E, out_dim, in_dim, rows;
    bool i8, f16, grad;
};
int launch_grouped_mm(const MmProblem& p, cudaStream_t s);

struct WgradProblem {
    const void* dy; const void* x;       // [rows, out], [rows, in]
    const int32_t* offsets;
    void* dw;                            // [E, out, in], 16 bits or fp32
    int32_t* status;
    int E, out_dim, in_dim, rows;
    bool f16, out_f32, accumulate;
};
int launch_grouped_wgrad(const WgradProblem& p, cudaStream_t s);

// Rows to 8 bits: codes [rows, cols], scales [rows].  With row_slot and top_k, row r reads row row_slot[r] / top_k of
// the nsrc rows of x; with row_slot and row_w (one or the other), the scale is multiplied by row_w[row_slot[r]], slots
// below rows.  With offsets (device), rows outside [offsets[0], offsets[E]) are left alone.  status nullable.
int launch_quant_int8(const void* x, bool f16, int64_t rows, int64_t cols, const int32_t* row_slot, int top_k,
                      int64_t nsrc, const float* row_w, const int32_t* offsets, int E, int8_t* codes, float* scales,
                      int32_t* status, cudaStream_t s);
// Rows of codes and their scales by slot, as above, from the nsrc rows src, src_scales.  A row of scale NaN is recorded
// as MOE_ERR_NONFINITE.
int launch_gather_int8(const int8_t* src, const float* src_scales, int rows, int cols, const int32_t* row_slot, int top_k,
                       int nsrc, const int32_t* offsets, int E, int8_t* codes, float* scales, int32_t* status,
                       cudaStream_t s);

// One-time set-up of a kernel on the current device: its shared-memory attribute; *sms: the device's SM count.
int mm_kernel_ready(const void* kernel, int smem_bytes, int* sms);

// Launch with programmatic dependent launch allowed, in clusters of `cluster` CTAs.
template <typename K, typename... Args>
inline int mm_launch_cfg(K kern, dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return MOE_ERR_CUDA;
    count_launch();
    return MOE_OK;
}

}  // namespace moe
