// wq_prompt_attn.cu -- causal attention over whole prompts packed one after
// another, with grouped query heads.
//
// Scaled dot-product attention (Vaswani et al. 2017, section 3.2.1) of token
// t of a sequence, query head j, over the tokens u <= t of the same sequence
// and KV head j / (Hq / H):
//   score_u = (q_tj . k_u) / sqrt(D),  p = softmax(score),  o_tj = sum_u p_u v_u.
// Sequence b owns rows starts[b] .. starts[b + 1] of q, k, v and o; rows of
// no sequence are left as they were.
//
// One pass over the keys with the running maximum m and sum l of the softmax
// (Milakov and Gimelshein 2018): when m grows, l and the output accumulator
// are scaled by e^(m_old - m_new).  Scores, m, l and the accumulator are
// binary32; p is rounded to bf16 as the second product's operand (a rounding
// of at most 2^-8 of each term), while l sums the
// unrounded p.
//
// The r = Hq / H query heads of a KV head share its keys and values: a tile's
// rows are (token, head) pairs, token-major, so a tile of 64 rows covers
// 64 / r tokens and reads each key once for all r heads.
#include <algorithm>

#include "wq_common.cuh"
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int kRows = 64;   // (token, head) rows per CTA, 16 per warp
constexpr int kKeys = 64;   // keys per step
constexpr int kThreads = 128;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv, ldo, M;
    const int32_t *starts;
    int B, H, r, tpt;  // tokens per tile
    float scale_log2;  // log2(e) / sqrt(D)
    uint16_t *o;
};

// Tile `t` of the packed batch: its sequence's first row and length, and the tile's first token in it.  Whole
// warp; false when there is no such tile.  Bounds outside [0, M] are clamped, a sequence that ends before it
// begins is empty.
__device__ __forceinline__ bool locate_tile(const PromptArgs &p, int64_t t, int64_t &row0, int &len, int &tok0)
{
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int64_t s = 0, e = 0;
        if (b < p.B) {
            s = std::min<int64_t>(std::max<int64_t>(p.starts[b], 0), p.M);
            e = std::min<int64_t>(std::max<int64_t>(p.starts[b + 1], s), p.M);
        }
        const int64_t n = (e - s + p.tpt - 1) / p.tpt;
        int64_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > t);
        if (hit) {
            const int src = __ffs(hit) - 1;
            row0 = __shfl_sync(0xffffffffu, s, src);
            len = (int)__shfl_sync(0xffffffffu, e - s, src);
            tok0 = (int)(t - before - __shfl_sync(0xffffffffu, upto - n, src)) * p.tpt;
            return true;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

__device__ __forceinline__ void mma_bf16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kThreads)
prompt_attn_kernel(const PromptArgs p)
{
    constexpr int kPitch = D + 8;  // halves; the pad keeps fragment loads off one bank
    extern __shared__ __align__(16) uint16_t sm[];
    uint16_t *ks = sm, *vs = sm + kKeys * kPitch;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, gr = lane >> 2, gc = lane & 3;
    const int h = blockIdx.y;
    int64_t row0;
    int len, tok0;
    if (!locate_tile(p, blockIdx.x, row0, len, tok0)) return;

    // this lane's two rows: tile rows 16 wid + gr and + 8
    int tok[2], head[2];
    bool live[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int i = wid * 16 + gr + 8 * e;
        tok[e] = tok0 + i / p.r;
        head[e] = h * p.r + i % p.r;
        live[e] = i < p.tpt * p.r && tok[e] < len;
        const uint16_t *src = p.q + (row0 + (live[e] ? tok[e] : 0)) * p.ldq + head[e] * D;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
            qf[c][e] = *reinterpret_cast<const uint32_t *>(src + c * 16 + gc * 2);
            qf[c][e + 2] = *reinterpret_cast<const uint32_t *>(src + c * 16 + 8 + gc * 2);
        }
    }
    float o[D / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

    const int last = std::min(len, tok0 + p.tpt);  // keys 0 .. last - 1 are seen by some row
    for (int u0 = 0; u0 < last; u0 += kKeys) {
        __syncthreads();
        for (int i = tid; i < kKeys * (D / 8); i += kThreads) {
            const int u = i / (D / 8), c = i % (D / 8) * 8;
            uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
            if (u0 + u < last) {
                kv = *reinterpret_cast<const uint4 *>(p.k + (row0 + u0 + u) * p.ldk + h * D + c);
                vv = *reinterpret_cast<const uint4 *>(p.v + (row0 + u0 + u) * p.ldv + h * D + c);
            }
            *reinterpret_cast<uint4 *>(ks + u * kPitch + c) = kv;
            *reinterpret_cast<uint4 *>(vs + u * kPitch + c) = vv;
        }
        __syncthreads();
        float s[kKeys / 8][4];
#pragma unroll
        for (int n = 0; n < kKeys / 8; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const uint16_t *b = ks + (n * 8 + gr) * kPitch + c * 16 + gc * 2;
                mma_bf16(s[n], qf[c], *reinterpret_cast<const uint32_t *>(b), *reinterpret_cast<const uint32_t *>(b + 8));
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float top = mx[e];
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int u = u0 + n * 8 + gc * 2 + x;
                    float &v = s[n][2 * e + x];
                    v = u <= tok[e] && u < last ? v : -INFINITY;
                    top = fmaxf(top, v);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float base = top == -INFINITY ? 0.0f : top;
            const float keep = exp2f((mx[e] - base) * p.scale_log2);
            mx[e] = top;
            float add = 0.0f;
#pragma unroll
            for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float &v = s[n][2 * e + x];
                    v = exp2f((v - base) * p.scale_log2);
                    add += v;
                }
            sum[e] = sum[e] * keep + add;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][2 * e] *= keep;
                o[i][2 * e + 1] *= keep;
            }
        }
#pragma unroll
        for (int c = 0; c < kKeys / 16; ++c) {
            const uint32_t a[4] = {pack_bf16x2(s[2 * c][0], s[2 * c][1]), pack_bf16x2(s[2 * c][2], s[2 * c][3]),
                                   pack_bf16x2(s[2 * c + 1][0], s[2 * c + 1][1]),
                                   pack_bf16x2(s[2 * c + 1][2], s[2 * c + 1][3])};
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint16_t *b = vs + (c * 16 + gc * 2) * kPitch + i * 8 + gr;
                mma_bf16(o[i], a, (uint32_t)b[0] | ((uint32_t)b[kPitch] << 16),
                         (uint32_t)b[8 * kPitch] | ((uint32_t)b[9 * kPitch] << 16));
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float l = sum[e];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (!live[e]) continue;
        const float inv = 1.0f / l;
        uint16_t *dst = p.o + (row0 + tok[e]) * p.ldo + head[e] * D + gc * 2;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t *>(dst + i * 8) = pack_bf16x2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
    }
}

}  // namespace

int launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                            int64_t ldv, const int32_t *starts, int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D,
                            uint16_t *o, int64_t ldo, int *status, cudaStream_t st)
{
    (void)status;
    PromptArgs a{q, k, v, ldq, ldk, ldv, ldo, M, starts, (int)B, (int)H, (int)(Hq / H), 0, 0.0f, o};
    a.tpt = kRows / a.r;
    a.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
    const dim3 grid((unsigned)(M / a.tpt + B), (unsigned)H);
    const int smem = 2 * kKeys * (int)(D + 8) * 2;
    if (D == 128) prompt_attn_kernel<128><<<grid, kThreads, smem, st>>>(a);
    else prompt_attn_kernel<64><<<grid, kThreads, smem, st>>>(a);
    return 0;
}

}  // namespace wq
