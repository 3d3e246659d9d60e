// Rows to 8-bit integers with a scale for each row:
//     s = max|x| / 127 (fp32),  q = rint(127 x / max|x|), ties to even, in [-127, 127]
// A zero row gets s = 0 and zero codes.  A row that holds an infinity or a NaN gets s = NaN and zero codes, so
// that every product of the row is NaN.
//
// The codes are those of the real quotient: with x = X 2^a and max|x| = M 2^b, X and M below 2^11, a quotient that is
// no tie lies at least 1 / (254 * 2^11) > 2^-19 of its size away from one, further than fp32 rounds; the division in
// fp32 (IEEE; 127 x is exact) then rounds to the same side, and a tie is exact.  The kernel multiplies by 127 / max|x| first (within 2^-16 of
// the quotient) and divides only where one of eight neighbours lands within 2^-12 of a tie.
//
// A block (or a warp) per row, the row's first 4096 (2048) elements kept in registers between the two passes.  Bound
// by the row's bytes, 2 read and 1 written per element, and by about 8 instructions an element (8192 rows of 4096: 20 us,
// 5 TB/s; 16,384 of 1536: 18 us); the copy of 65,536 rows of codes takes 73 us, bound by the writes.
#include <mutex>

#include "grouped_mm.cuh"

namespace moe {

constexpr int Q8_THREADS = 128;
// Rows of up to 2048 elements, many of them: a warp per row (16,384 rows of 1536: 8 us less than with a block)
constexpr int64_t Q8_WARP_ROWS = 2048, Q8_WARP_COLS = 2048;

// max of the 16-bit magnitudes (sign dropped): as unsigned numbers they order like the values, infinity and NaN last
__device__ __forceinline__ uint32_t q8_max2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t q8_max8(uint32_t m, const uint4& v) {
    return q8_max2(q8_max2(q8_max2(q8_max2(m, v.x), v.y), v.z), v.w);
}

// rint(t) for |t| < 2^22 as a float sum: t + 1.5 2^23 has the whole number in its low bits (ties to even), without
// the conversion instructions, which run at a quarter of the rate
constexpr float Q8_MAGIC = 12582912.f;

// The code by division: near a tie, or in a row so small that 127 / amax overflows.  Powers of two keep 127 x in range.
__device__ __forceinline__ uint32_t q8_divide(float x, float amax) {
    const float c = amax > 0x1p100f ? 0x1p-16f : (amax < 0x1p-90f ? 0x1p64f : 1.f);
    return __float_as_uint(rintf(__fdiv_rn(127.f * (x * c), amax * c)) + Q8_MAGIC);
}

// The token of a slot, or -1
__device__ __forceinline__ long long q8_source(int slot, int top_k, long long nsrc) {
    const int t = slot / top_k;
    return slot >= 0 && t < nsrc ? t : -1;
}

template <bool F16, int TPR>           // TPR threads per row: 32 or the block
__global__ void __launch_bounds__(Q8_THREADS) quant_int8_kernel(const uint16_t* __restrict__ x, long long cols,
                                                               const int32_t* __restrict__ row_slot, int top_k,
                                                               long long nsrc, const float* __restrict__ row_w,
                                                               const int32_t* __restrict__ offsets, int E,
                                                               int8_t* __restrict__ codes, float* __restrict__ scales,
                                                               int32_t* status, long long rows) {
    constexpr int kKeep = TPR == 32 ? 8 : 4;                          // 16-byte chunks per thread kept in registers
    const int tid = int(threadIdx.x) % TPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the product's weights need nothing from here
    const long long row = (long long)blockIdx.x * (Q8_THREADS / TPR) + threadIdx.x / TPR;
    if (row >= rows || (offsets && (row < offsets[0] || row >= offsets[E]))) return;  // a row of no expert
    const long long n = cols / 8;
    uint2* dst = reinterpret_cast<uint2*>(codes + row * cols);
    long long src = row;
    float weight = 1.f;
    if (row_w) {
        const int slot = row_slot[row];
        if (slot >= 0 && slot < rows) weight = row_w[slot];
        else src = -1;
    } else if (row_slot) {
        src = q8_source(row_slot[row], top_k, nsrc);
    }
    if (src < 0) {                                                    // a slot out of range: a zero row
        if (tid == 0) {
            scales[row] = 0.f;
            if (status) set_status(status, MOE_ERR_DEVICE_INDEX);
        }
        for (long long i = tid; i < n; i += TPR) dst[i] = make_uint2(0, 0);
        return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(x + src * cols);
    uint4 keep[kKeep];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kKeep; j++) {
        const long long i = tid + j * TPR;
        keep[j] = i < n ? p[i] : make_uint4(0, 0, 0, 0);
        m = q8_max8(m, keep[j]);
    }
    for (long long i = tid + kKeep * TPR; i < n; i += TPR) m = q8_max8(m, p[i]);
    for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if constexpr (TPR > 32) {
        __shared__ uint32_t sm[TPR / 32];
        if ((tid & 31) == 0) sm[tid >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; w++) m = __vmaxu2(m, sm[w]);
    }
    m = max(m & 0xffffu, m >> 16);
    const bool bad = m >= (F16 ? 0x7c00u : 0x7f80u);
    const float amax = act_lo<F16>(m);
    if (tid == 0) {
        scales[row] = bad ? __int_as_float(0x7fffffff) : __fdiv_rn(amax, 127.f) * weight;
        if (bad && status) set_status(status, MOE_ERR_NONFINITE);
    }
    const bool zero = bad || m == 0;
    const float r = __fdiv_rn(127.f, amax);
    const bool slow = amax < 0x1p-90f && !zero;
    auto put = [&](long long i, const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t c[8];
        float far = 0.f;                                              // largest distance from the whole number
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float t = ((j & 1) ? act_hi<F16>(w[j >> 1]) : act_lo<F16>(w[j >> 1])) * r;
            const float k = t + Q8_MAGIC;
            far = fmaxf(far, fabsf(t - (k - Q8_MAGIC)));
            c[j] = __float_as_uint(k);
        }
        if (slow || far > 0.5f - 0x1p-12f)
#pragma unroll
            for (int j = 0; j < 8; j++) c[j] = q8_divide((j & 1) ? act_hi<F16>(w[j >> 1]) : act_lo<F16>(w[j >> 1]), amax);
        uint2 o = make_uint2(0, 0);
        if (!zero)
            o = make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                           __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
        dst[i] = o;
    };
#pragma unroll
    for (int j = 0; j < kKeep; j++) {
        const long long i = tid + j * TPR;
        if (i < n) put(i, keep[j]);
    }
    for (long long i = tid + kKeep * TPR; i < n; i += TPR) put(i, p[i]);
}

int launch_quant_int8(const void* x, bool f16, int64_t rows, int64_t cols, const int32_t* row_slot, int top_k,
                      int64_t nsrc, const float* row_w, const int32_t* offsets, int E, int8_t* codes, float* scales,
                      int32_t* status, cudaStream_t s) {
    if (rows <= 0) return MOE_OK;
    const bool warp = rows >= Q8_WARP_ROWS && cols <= Q8_WARP_COLS;
    auto k = warp ? (f16 ? quant_int8_kernel<true, 32> : quant_int8_kernel<false, 32>)
                  : (f16 ? quant_int8_kernel<true, Q8_THREADS> : quant_int8_kernel<false, Q8_THREADS>);
    const int64_t blocks = warp ? (rows + Q8_THREADS / 32 - 1) / (Q8_THREADS / 32) : rows;
    return mm_launch_cfg(k, dim3(unsigned(blocks)), dim3(Q8_THREADS), 0, 1, s, static_cast<const uint16_t*>(x),
                         (long long)cols, row_slot, top_k, (long long)nsrc, row_w, offsets, E, codes, scales, status, (long long)rows);
}

// One block per row, 16 bytes per thread and step.
__global__ void __launch_bounds__(Q8_THREADS) gather_int8_kernel(const int8_t* __restrict__ src,
                                                                 const float* __restrict__ src_scales, int cols,
                                                                 const int32_t* __restrict__ row_slot, int top_k, int nsrc,
                                                                 const int32_t* __restrict__ offsets, int E,
                                                                 int8_t* __restrict__ codes, float* __restrict__ scales,
                                                                 int32_t* status) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int row = blockIdx.x;
    if (row < offsets[0] || row >= offsets[E]) return;
    const long long t = q8_source(row_slot[row], top_k, nsrc);
    if (threadIdx.x == 0) {
        const float scale = t < 0 ? 0.f : src_scales[t];
        scales[row] = scale;
        if (t < 0) set_status(status, MOE_ERR_DEVICE_INDEX);
        else if (isnan(scale)) set_status(status, MOE_ERR_NONFINITE);     // (of a row, not of a token that none refers to)
    }
    const uint4* p = reinterpret_cast<const uint4*>(src + (t < 0 ? 0 : t) * cols);
    uint4* d = reinterpret_cast<uint4*>(codes + size_t(row) * cols);
    for (int i = threadIdx.x; i < cols / 16; i += Q8_THREADS) __stcs(d + i, t < 0 ? make_uint4(0, 0, 0, 0) : p[i]);
}

int launch_gather_int8(const int8_t* src, const float* src_scales, int rows, int cols, const int32_t* row_slot, int top_k,
                       int nsrc, const int32_t* offsets, int E, int8_t* codes, float* scales, int32_t* status,
                       cudaStream_t s) {
    return mm_launch_cfg(gather_int8_kernel, dim3(unsigned(rows)), dim3(Q8_THREADS), 0, 1, s, src, src_scales, cols,
                         row_slot, top_k, nsrc, offsets, E, codes, scales, status);
}

// Per device and kernel: the shared-memory attribute, set once under a lock.
int mm_kernel_ready(const void* kernel, int smem_bytes, int* sms) {
    struct Dev { int sms = 0; int n = 0; const void* ready[32] = {}; };
    static std::mutex mu;
    static Dev devs[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
    std::lock_guard<std::mutex> lock(mu);
    Dev& d = devs[dev];
    if (!d.sms && cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        d.sms = 0;
        return MOE_ERR_CUDA;
    }
    *sms = d.sms;
    for (int i = 0; i < d.n; i++)
        if (d.ready[i] == kernel) return MOE_OK;
    if (d.n == 32 || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes) != cudaSuccess)
        return MOE_ERR_CUDA;
    d.ready[d.n++] = kernel;
    return MOE_OK;
}

}  // namespace moe
