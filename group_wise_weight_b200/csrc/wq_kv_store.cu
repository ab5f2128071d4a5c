// wq_kv_store.cu -- new tokens' keys and values written into a quantised KV
// cache at their places, the cache that the decode attention of
// wq_kv_attn.cu reads.
//
// "Quantization for LLM inference: FP8, INT4 (GPTQ, AWQ) and GGUF", section
// "KV cache quantization": caches in fp8, or in int4 with blocks of 128.  One
// vector (token, head) of D = 128 values is one block:
//   int4  s, z and the codes exactly as wq_quantize_int4 with g = 128
//         (s = bf16(RN((max - min) / 15)), z = bf16(rint(RN(-min / s)) + 0),
//         q = clip(rint(RN(w / s) + z), 0, 15));
//   fp8   the E4M3 value nearest to RN(w / scale) for the tensor's given
//         binary32 scale, saturated at +-448, as wq_quantize_fp8_tensor
//         encodes against its scale.
// Token m goes to row slots[m] of the cache viewed as [B T][H] vectors; a
// slot outside [0, B T) leaves the token out.
//
// Each value is read once (2 bytes) and written once (0.53 or 1 byte): an HBM
// stream, if the instructions stay few.  8 lanes take a vector, 16 values
// each, so the block's parameters are formed once per 16 values; the int4
// minimum and maximum travel as one bf16 pair (min, -max) through three
// shuffles.  Quotients come from a reciprocal, two per instruction
// (wq_quotient.cuh): one correction step for the bf16 scales of int4, two for
// the arbitrary binary32 scale of fp8; blocks outside the proven range use
// the IEEE division.
// Measured, 16,000 tokens of 8 heads, back to back: fp8 19.2 us (5.1 TB/s; 20.6
// without the launch while the previous kernel ends), int4 23.1 us (3.6 TB/s);
// the schedulers issue 69 and 75% of the time, so the instructions bind.  The
// blocks of a lane are left to other warps (one vector per group of lanes):
// several in turn per warp took 22.8 us.
#include <algorithm>

#include "wq_internal.h"
#include "wq_prompt.cuh"
#include "wq_quotient.cuh"

namespace wq {

namespace {

constexpr int kD = 128;
constexpr int kLanes = kD / 16;  // lanes per vector
constexpr int kThreads = 256;
constexpr int kGroups = kThreads / kLanes;

struct StoreArgs {
    const uint16_t *k, *v;
    int64_t ldk, ldv;
    const int64_t *slots;
    int64_t M, S;
    int H;
    uint8_t *kc, *vc;
    uint16_t *ks, *kz, *vs, *vz;  // int4
    const float *k8s, *v8s;       // fp8
};

// Pair i of a lane's 16 values, widened to binary32.
__device__ __forceinline__ uint64_t pair_of(const uint4 raw[2], int i)
{
    const uint32_t w = word_of(raw[i >> 2], i & 3);
    return ((uint64_t)(w & 0xffff0000u) << 32) | (uint64_t)(w << 16);
}
__device__ __forceinline__ float lo_of(uint64_t p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float hi_of(uint64_t p) { return __uint_as_float((uint32_t)(p >> 32)); }

// The vector's int4 block: this lane's 16 codes, and s and z.
__device__ __forceinline__ uint2 int4_block(const uint4 raw[2], float &s, float &z)
{
    uint32_t lo = raw[0].x, hi = raw[0].x;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = bf16x2_min(lo, word_of(raw[i >> 2], i & 3));
        hi = bf16x2_max(hi, word_of(raw[i >> 2], i & 3));
    }
    hi ^= 0x80008000u;
    uint32_t pk = bf16x2_min(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) pk = bf16x2_min(pk, __shfl_xor_sync(0xffffffffu, pk, o));
    const float mn = __uint_as_float(pk << 16), mx = __uint_as_float((pk & 0xffff0000u) ^ 0x80000000u);
    s = int4_scale(mn, mx);
    const float maxabs = fmaxf(fabsf(mn), fabsf(mx));
    uint32_t code[2];
    if (quotients_by_reciprocal(s, maxabs) && maxabs <= s * 8192.0f) {
        const float r = __frcp_rn(s);
        z = round_bf16(__fadd_rn(rintf(quotient_rn(-mn, s, r)), 0.0f));
        // |w / s + z| < 2^15: the integer rounded by 1.5 * 2^23 is the low half-word of its pattern
        const uint64_t r2 = f32x2_bits(r, r), ns2 = f32x2_bits(-s, -s), z2 = f32x2_bits(z, z);
        const uint64_t m2 = f32x2_bits(0x1.8p23f, 0x1.8p23f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t w = pair_of(raw, 4 * j + i), q0 = f32x2_mul(w, r2);
                const uint64_t q = f32x2_fma(f32x2_fma(q0, ns2, w), r2, q0);
                const uint64_t t = f32x2_add(f32x2_add(q, z2), m2);
                uint32_t p2 = __byte_perm((uint32_t)t, (uint32_t)(t >> 32), 0x5410);
                p2 = __vmins2(__vmaxs2(p2, 0u), 0x000F000Fu);
                b[i] = p2 | (p2 >> 12);  // byte 0: the pair's first code | second << 4
            }
            code[j] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        }
    } else {
        z = round_bf16(__fadd_rn(rintf(__fdiv_rn(-mn, s)), 0.0f));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            code[j] = 0u - kRintBase * 0x11111111u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t p = pair_of(raw, 4 * j + (i >> 1));
                const float t = __fadd_rn(__fdiv_rn((i & 1) ? hi_of(p) : lo_of(p), s), z);
                code[j] += rint_bits(fminf(fmaxf(t, 0.0f), 15.0f)) << (4 * i);
            }
        }
    }
    return make_uint2(code[0], code[1]);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    return h;
}

// This lane's 16 E4M3 codes against the tensor's scale s.
__device__ __forceinline__ uint4 fp8_codes(const uint4 raw[2], float s)
{
    uint32_t m2 = raw[0].x & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m2 = bf16x2_max(m2, word_of(raw[i >> 2], i & 3) & 0x7FFF7FFFu);
    const float maxabs = fmaxf(__uint_as_float(m2 << 16), __uint_as_float(m2 & 0xffff0000u));
    uint32_t c[8];
    if (quotients_by_reciprocal(s, maxabs)) {
        const float r = __frcp_rn(s);
        const uint64_t r2 = f32x2_bits(r, r), ns2 = f32x2_bits(-s, -s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t w = pair_of(raw, i);
            uint64_t q = f32x2_mul(w, r2);
            q = f32x2_fma(f32x2_fma(q, ns2, w), r2, q);
            q = f32x2_fma(f32x2_fma(q, ns2, w), r2, q);
            c[i] = e4m3x2(lo_of(q), hi_of(q));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t w = pair_of(raw, i);
            c[i] = e4m3x2(__fdiv_rn(lo_of(w), s), __fdiv_rn(hi_of(w), s));
        }
    }
    uint32_t word[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a code's sign is its value's (s > 0; the corrections turn -0 into +0)
        const uint32_t sign = __byte_perm(word_of(raw[i >> 1], (2 * i) & 3), word_of(raw[i >> 1], (2 * i + 1) & 3), 0x7531);
        word[i] = __byte_perm(c[2 * i], c[2 * i + 1], 0x5410) | (sign & 0x80808080u);
    }
    return make_uint4(word[0], word[1], word[2], word[3]);
}

// Vector index j runs over (token, K or V, head): a token's heads are adjacent, so are their groups of lanes.  One
// vector per group and CTA (two in flight per lane measured 10% slower at 16,000 tokens of 8 heads, four 25%).
template <bool FP8>
__global__ void __launch_bounds__(kThreads)
kv_store_kernel(const StoreArgs p)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned l = threadIdx.x % kLanes, H = (unsigned)p.H, j = blockIdx.x * kGroups + threadIdx.x / kLanes;
    int64_t slot = -1, row = 0;
    uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    bool is_v = false;
    if (j < (unsigned)p.M * 2u * H) {
        const unsigned m = j / (2u * H), rest = j - m * 2u * H;
        is_v = rest >= H;
        const unsigned h = is_v ? rest - H : rest;
        slot = p.slots[m];
        if (slot >= p.S) slot = -1;
        const uint16_t *src = (is_v ? p.v + m * p.ldv : p.k + m * p.ldk) + h * kD + l * 16;
        raw[0] = ld_written_v4(src);
        raw[1] = ld_written_v4(src + 8);
        row = slot * H + h;
    }
    if (FP8) {
        const uint4 c = fp8_codes(raw, *(is_v ? p.v8s : p.k8s));
        if (slot >= 0) *reinterpret_cast<uint4 *>((is_v ? p.vc : p.kc) + row * kD + l * 16) = c;
    } else {
        float s, z;
        const uint2 c = int4_block(raw, s, z);
        if (slot >= 0) {
            *reinterpret_cast<uint2 *>((is_v ? p.vc : p.kc) + row * (kD / 2) + l * 8) = c;
            if (l == 0) {
                (is_v ? p.vs : p.ks)[row] = f32_to_bf16(s);
                (is_v ? p.vz : p.kz)[row] = f32_to_bf16(z);
            }
        }
    }
}

}  // namespace

void launch_kv_store(bool fp8, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, const int64_t *slots,
                     int64_t M, int64_t S, int64_t H, uint8_t *kc, uint16_t *ks, uint16_t *kz, const float *k8s,
                     uint8_t *vc, uint16_t *vs, uint16_t *vz, const float *v8s, cudaStream_t st)
{
    const StoreArgs a{k, v, ldk, ldv, slots, M, S, (int)H, kc, vc, ks, kz, vs, vz, k8s, v8s};
    const unsigned grid = (unsigned)((M * 2 * H + kGroups - 1) / kGroups);
    if (fp8) launch_behind(kv_store_kernel<true>, grid, kThreads, 0, st, a);
    else launch_behind(kv_store_kernel<false>, grid, kThreads, 0, st, a);
}

}  // namespace wq
