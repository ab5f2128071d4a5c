// wq_quant_tokens.cu -- dynamic per-token INT8 quantisation of activations,
// the left operand of the INT8 W8A8 matmul.
//
// "Quantization Methods Compared: INT8, GPTQ, AWQ, FP8, FP4 and KV-Cache
// Quantization", section "What quantisation does": symmetric absmax INT8,
// s = max|x| / 127 and q = round(x / s), here with one binary32 scale per row
// of activations (a token) formed while the row is in registers.
// Arithmetic, binary32 with round to nearest even:
//   s = RN(max|x| / 127); 1 where that is 0
//   q = clip(rint(RN(x / s)), -127, 127)
//
// The quotients are formed from r = RN(1 / s).  bf16 rows: max|x| is a bf16
// value, so s takes 128 significands and x 128 more, and one correction step
// gives the correctly rounded quotient for all of them (checked exhaustively
// by the test suite).  binary32 rows: after one correction the quotient is
// within one unit in the last place, and Markstein's theorem (see
// wq_quotient.cuh) makes the second exact.  Rows whose scale leaves
// [2^-100, 2^100] use the IEEE division.
//
// The pass reads 2 or 4 bytes and writes 1 per value, so it is bound by HBM:
// the row crosses it once, kept in registers between the maximum and the
// codes.  A row of up to 2,048 values (1,024 in binary32) belongs to one warp
// (no barrier), a longer one to a CTA of 256 or 512 threads, 8 values per thread
// and chunk; rows beyond 32,768 values (8,192) are read twice (the second time
// from L2).
// Measured: 8,192 x 28,672 bf16 115 us (6.1 TB/s, 93% of a copy); one row of
// 8,192 4.7 us, which is what the host needs to make the calls (1.9 in a graph);
// binary32 4,096 x 8,192 32.6 us (5.1 TB/s), 4,096 x 14,336 68.5 us (4.3 TB/s).
#include "wq_internal.h"
#include "wq_prompt.cuh"
#include "wq_quotient.cuh"

namespace wq {

namespace {

// Eight consecutive values as loaded.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw(const T *p)
{
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < (int)(sizeof(T) / 2); ++j) r.w[j] = ld_written_v4(p + j * (16 / sizeof(T)));
    return r;
}

template <typename T>
__device__ __forceinline__ Raw8<T> zero_raw()
{
    Raw8<T> r;
#pragma unroll
    for (int j = 0; j < (int)(sizeof(T) / 2); ++j) r.w[j] = make_uint4(0u, 0u, 0u, 0u);
    return r;
}

// Pair i (values 2i and 2i + 1) of eight, widened to binary32.
template <typename T>
__device__ __forceinline__ uint64_t pair_of(const Raw8<T> &r, int i)
{
    if (sizeof(T) == 2) {
        const uint32_t w = word_of(r.w[0], i);
        return ((uint64_t)(w & 0xffff0000u) << 32) | (uint64_t)(w << 16);
    }
    const uint4 &v = r.w[(sizeof(T) / 2 - 1) & (i >> 1)];
    return (i & 1) ? ((uint64_t)v.w << 32) | v.z : ((uint64_t)v.y << 32) | v.x;
}

// Largest magnitude of eight values: for bf16 as the larger half of a packed pair.
template <typename T>
__device__ __forceinline__ float amax8(const Raw8<T> &r, float amax)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t m = bf16x2_max(bf16x2_max(r.w[0].x & 0x7FFF7FFFu, r.w[0].y & 0x7FFF7FFFu),
                                      bf16x2_max(r.w[0].z & 0x7FFF7FFFu, r.w[0].w & 0x7FFF7FFFu));
        return fmaxf(amax, fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t p = pair_of<T>(r, i);
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float((uint32_t)p)), fabsf(__uint_as_float((uint32_t)(p >> 32)))));
        }
        return amax;
    }
}

// s = RN(amax / 127), 1 for a row of zeros.
__device__ __forceinline__ float token_scale(float amax)
{
    const float s = __fdiv_rn(amax, 127.0f);
    return s == 0.0f ? 1.0f : s;
}

// Codes of eight values against the scale s (r = RN(1 / s)), little-endian bytes.
template <typename T>
__device__ __forceinline__ uint2 encode8(const Raw8<T> &v, float s, float r, bool by_reciprocal)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t x = pair_of<T>(v, i);
        uint64_t q;
        if (by_reciprocal) {
            const uint64_t r2 = f32x2_bits(r, r), ns2 = f32x2_bits(-s, -s);
            q = f32x2_mul(x, r2);
            q = f32x2_fma(f32x2_fma(q, ns2, x), r2, q);
            if (sizeof(T) == 4) q = f32x2_fma(f32x2_fma(q, ns2, x), r2, q);
            // |q| <= 127 (1 + 2^-23) here, so rint stays within +-127: no clip
        } else {
            const float a = __fdiv_rn(__uint_as_float((uint32_t)x), s);
            const float b = __fdiv_rn(__uint_as_float((uint32_t)(x >> 32)), s);
            q = f32x2_bits(fminf(fmaxf(a, -127.0f), 127.0f), fminf(fmaxf(b, -127.0f), 127.0f));
        }
        const uint64_t t = f32x2_add(q, f32x2_bits(0x1.8p23f, 0x1.8p23f));  // rounds; the code is the low byte
        w[i] = __byte_perm((uint32_t)t, (uint32_t)(t >> 32), 0x0040);
    }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

constexpr int kWarpRows = 8;  // rows (warps) per CTA of the short-row form

// Rows of up to 256 CH values: one warp per row.
template <typename T, int CH>
__global__ void __launch_bounds__(kWarpRows * 32)
quant_tokens_warp_kernel(const T *x, int64_t M, int64_t K, int64_t ldx, int8_t *__restrict__ q,
                         float *__restrict__ scales)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t m = (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5);
    if (m >= M) return;
    Raw8<T> v[CH];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * 32 + lane) * 8;
        v[i] = k < K ? load_raw<T>(x + m * ldx + k) : zero_raw<T>();
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) amax = amax8<T>(v[i], amax);
    const float s = token_scale(warp_max(amax));
    const bool fast = s >= 0x1p-100f && s <= 0x1p100f;
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * 32 + lane) * 8;
        if (k < K) *reinterpret_cast<uint2 *>(q + m * K + k) = encode8<T>(v[i], s, r, fast);
    }
    if (lane == 0) scales[m] = s;
}

template <int THREADS>
__device__ __forceinline__ float cta_max(float v)
{
    __shared__ float part[THREADS / 32];
    v = warp_max(v);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[threadIdx.x & (THREADS / 32 - 1)];
#pragma unroll
    for (int o = THREADS / 64; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Rows of up to 8 THREADS CH values: one CTA per row, the row in registers.
template <typename T, int THREADS, int CH>
__global__ void __launch_bounds__(THREADS)
quant_tokens_row_kernel(const T *x, int64_t K, int64_t ldx, int8_t *__restrict__ q,
                        float *__restrict__ scales)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t m = blockIdx.x;
    const T *row = x + m * ldx;
    Raw8<T> v[CH];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * THREADS + threadIdx.x) * 8;
        v[i] = k < K ? load_raw<T>(row + k) : zero_raw<T>();
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) amax = amax8<T>(v[i], amax);
    const float s = token_scale(cta_max<THREADS>(amax));
    const bool fast = s >= 0x1p-100f && s <= 0x1p100f;
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * THREADS + threadIdx.x) * 8;
        if (k < K) *reinterpret_cast<uint2 *>(q + m * K + k) = encode8<T>(v[i], s, r, fast);
    }
    if (threadIdx.x == 0) scales[m] = s;
}

// Longer rows: the maximum, then a second pass over the row.
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS)
quant_tokens_long_kernel(const T *x, int64_t K, int64_t ldx, int8_t *__restrict__ q,
                         float *__restrict__ scales)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t m = blockIdx.x;
    const T *row = x + m * ldx;
    float amax = 0.0f;
#pragma unroll 4
    for (int64_t k = (int64_t)threadIdx.x * 8; k < K; k += THREADS * 8) amax = amax8<T>(load_raw<T>(row + k), amax);
    const float s = token_scale(cta_max<THREADS>(amax));
    const bool fast = s >= 0x1p-100f && s <= 0x1p100f;
    const float r = __frcp_rn(s);
#pragma unroll 4
    for (int64_t k = (int64_t)threadIdx.x * 8; k < K; k += THREADS * 8)
        *reinterpret_cast<uint2 *>(q + m * K + k) = encode8<T>(load_raw<T>(row + k), s, r, fast);
    if (threadIdx.x == 0) scales[m] = s;
}

template <typename T>
void dispatch(const T *x, int64_t M, int64_t K, int64_t ldx, int8_t *q, float *s, cudaStream_t st)
{
    const unsigned rows = (unsigned)M, warps = (unsigned)((M + kWarpRows - 1) / kWarpRows);
    const auto per_warp = [&](auto kernel) { launch_behind(kernel, warps, kWarpRows * 32, 0, st, x, M, K, ldx, q, s); };
    const auto per_cta = [&](auto kernel, unsigned threads) { launch_behind(kernel, rows, threads, 0, st, x, K, ldx, q, s); };
    if (K <= 512) per_warp(quant_tokens_warp_kernel<T, 2>);
    else if (K <= 1024) per_warp(quant_tokens_warp_kernel<T, 4>);
    else if (sizeof(T) == 4) {
        // binary32: at most 16 values in a thread's registers, so that the SM holds enough rows (32 values: 8,192 x 2,048 30.5
        // us, 4,096 x 8,192 36.4, 4,096 x 14,336 80.0); beyond 8,192 the second read costs less than one row per SM
        if (K <= 2048) per_cta(quant_tokens_row_kernel<T, 256, 1>, 256);
        else if (K <= 4096) per_cta(quant_tokens_row_kernel<T, 256, 2>, 256);
        else if (K <= 8192) per_cta(quant_tokens_row_kernel<T, 512, 2>, 512);
        else per_cta(quant_tokens_long_kernel<T, 1024>, 1024);
    } else if (K <= 2048) per_warp(quant_tokens_warp_kernel<T, 8>);
    else if (K <= 4096) per_cta(quant_tokens_row_kernel<T, 256, 2>, 256);
    else if (K <= 8192) per_cta(quant_tokens_row_kernel<T, 256, 4>, 256);
    else if (K <= 16384) per_cta(quant_tokens_row_kernel<T, 512, 4>, 512);
    else if (K <= 32768) per_cta(quant_tokens_row_kernel<T, 512, 8>, 512);
    else per_cta(quant_tokens_long_kernel<T, 512>, 512);
}

}  // namespace

void launch_quantize_int8_tokens(const void *x, int xtype, int64_t M, int64_t K, int64_t ldx, int8_t *q, float *s,
                                 cudaStream_t st)
{
    if (xtype == WQ_F32) dispatch(static_cast<const float *>(x), M, K, ldx, q, s, st);
    else dispatch(static_cast<const __nv_bfloat16 *>(x), M, K, ldx, q, s, st);
}

}  // namespace wq
