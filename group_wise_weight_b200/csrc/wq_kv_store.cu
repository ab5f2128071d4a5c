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
// stream.  16 lanes take a vector, 8 values each; the int4 minimum and
// maximum travel as one bf16 pair (min, -max) through four shuffles.
// Quotients come from a reciprocal (wq_quotient.cuh): one correction step for
// the bf16 scales of int4, two for the arbitrary binary32 scale of fp8.
#include <algorithm>

#include "wq_internal.h"
#include "wq_quotient.cuh"

namespace wq {

namespace {

constexpr int kD = 128;
constexpr int kLanes = kD / 8;   // lanes per vector
constexpr int kThreads = 256;
constexpr int kUnroll = 4;       // vectors in flight per group of 16 lanes

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

// The vector's int4 block: this lane's 8 codes as one word, and s and z.
__device__ __forceinline__ uint32_t int4_block(const uint4 &raw, float &s, float &z)
{
    const uint32_t lo = bf16x2_min(bf16x2_min(raw.x, raw.y), bf16x2_min(raw.z, raw.w));
    const uint32_t hi = bf16x2_max(bf16x2_max(raw.x, raw.y), bf16x2_max(raw.z, raw.w)) ^ 0x80008000u;
    uint32_t pk = bf16x2_min(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) pk = bf16x2_min(pk, __shfl_xor_sync(0xffffffffu, pk, o));
    const float mn = __uint_as_float(pk << 16), mx = __uint_as_float((pk & 0xffff0000u) ^ 0x80000000u);
    s = int4_scale(mn, mx);
    const bool fast = quotients_by_reciprocal(s, fmaxf(fabsf(mn), fabsf(mx)));
    const float r = __frcp_rn(s);
    const float zq = fast ? quotient_rn(-mn, s, r) : __fdiv_rn(-mn, s);
    z = round_bf16(__fadd_rn(rintf(zq), 0.0f));
    uint32_t packed = 0u - kRintBase * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t word = word_of(raw, i >> 1);
        const float w = __uint_as_float((i & 1) ? (word & 0xffff0000u) : (word << 16));
        const float t = __fadd_rn(fast ? quotient_rn(w, s, r) : __fdiv_rn(w, s), z);
        packed += rint_bits(fminf(fmaxf(t, 0.0f), 15.0f)) << (4 * i);
    }
    return packed;
}

// This lane's 8 E4M3 codes against the tensor's scale s (r = RN(1 / s) when `fast`).
__device__ __forceinline__ uint2 fp8_codes(const uint4 &raw, float s, float r, bool fast)
{
    uint32_t c[4];
    const float top = __fmul_rn(s, 1024.0f);  // |w / s| >= 1024 saturates all the same
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t word = word_of(raw, i);
        float q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float w = __uint_as_float(e ? (word & 0xffff0000u) : (word << 16));
            if (fast) {
                const float wc = fminf(fmaxf(w, -top), top);
                float t = __fmul_rn(wc, r);
                t = __fmaf_rn(__fmaf_rn(-t, s, wc), r, t);
                t = __fmaf_rn(__fmaf_rn(-t, s, wc), r, t);
                q[e] = copysignf(t, w);  // the corrections turn -0 into +0
            } else {
                q[e] = __fdiv_rn(w, s);
            }
        }
        uint16_t h;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(q[1]), "f"(q[0]));
        c[i] = h;
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Vector index j runs over (token, K or V, head): a token's heads are adjacent, so are their 16-lane groups.
template <bool FP8>
__global__ void __launch_bounds__(kThreads)
kv_store_kernel(const StoreArgs p)
{
    constexpr int kGroups = kThreads / kLanes;
    const int l = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
    const int64_t vectors = p.M * 2 * p.H;
    float s8[2] = {0.0f, 0.0f}, r8[2] = {0.0f, 0.0f};
    bool fast8[2] = {false, false};
    if (FP8) {
        s8[0] = *p.k8s;
        s8[1] = *p.v8s;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            fast8[e] = s8[e] >= 0x1p-100f && s8[e] <= 0x1p100f;
            r8[e] = __frcp_rn(s8[e]);
        }
    }
    const int64_t j0 = (int64_t)blockIdx.x * (kGroups * kUnroll) + g;
    uint4 raw[kUnroll];
    int64_t slot[kUnroll], row[kUnroll];
    bool is_v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t j = j0 + u * kGroups;
        slot[u] = -1;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        row[u] = 0;
        is_v[u] = false;
        if (j < vectors) {
            const int64_t m = j / (2 * p.H);
            const int rest = (int)(j - m * 2 * p.H);
            is_v[u] = rest >= p.H;
            const int h = is_v[u] ? rest - p.H : rest;
            slot[u] = p.slots[m];
            if (slot[u] >= p.S) slot[u] = -1;
            raw[u] = ld_stream_v4((is_v[u] ? p.v + m * p.ldv : p.k + m * p.ldk) + h * kD + l * 8);
            row[u] = slot[u] * p.H + h;
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (FP8) {
            const uint2 c = is_v[u] ? fp8_codes(raw[u], s8[1], r8[1], fast8[1]) : fp8_codes(raw[u], s8[0], r8[0], fast8[0]);
            if (slot[u] >= 0) *reinterpret_cast<uint2 *>((is_v[u] ? p.vc : p.kc) + row[u] * kD + l * 8) = c;
        } else {
            float s, z;
            const uint32_t c = int4_block(raw[u], s, z);
            if (slot[u] >= 0) {
                *reinterpret_cast<uint32_t *>((is_v[u] ? p.vc : p.kc) + row[u] * (kD / 2) + l * 4) = c;
                if (l == 0) {
                    (is_v[u] ? p.vs : p.ks)[row[u]] = f32_to_bf16(s);
                    (is_v[u] ? p.vz : p.kz)[row[u]] = f32_to_bf16(z);
                }
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
    const int64_t per = (int64_t)(kThreads / kLanes) * kUnroll;
    const unsigned grid = (unsigned)((M * 2 * H + per - 1) / per);
    if (fp8) kv_store_kernel<true><<<grid, kThreads, 0, st>>>(a);
    else kv_store_kernel<false><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace wq
