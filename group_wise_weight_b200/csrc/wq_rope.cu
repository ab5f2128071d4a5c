// wq_rope.cu -- per-head RMS norms of queries and keys and their rotary
// positions, in one pass over the projection's output.
//
// For each token m and head vector x of D values (queries and keys alike):
//   n_i = x_i / sqrt(mean(x^2) + eps) * w_i      (left out without weights)
//   the first `rot` values turn in pairs (a, b) by the angle p_m f_i:
//     (a cos - b sin, b cos + a sin)
//   pairs are (i, i + rot/2), or (2i, 2i + 1) when interleaved; the other
//   D - rot values pass through.
// Sums, norms and rotations are binary32, rounded to bf16 once.  The angle is
// the product of the position and the binary32 frequency in binary64 (31 + 24
// bits against 53: off by at most 2^-53 of itself), reduced to a fraction of
// a turn in binary64 before the binary32 sine and cosine, so far positions
// keep their phase.
//
// The pass reads and writes 2 bytes per value and is bound by HBM.  D / 8
// lanes hold a vector (16-byte loads and stores; the sum of squares is a
// shuffle over them, the pair's other half of the split form one more), a CTA
// takes one token or a few, and its sines and cosines are formed once for all
// heads while the first loads are in flight.
#include <algorithm>

#include "wq_common.cuh"
#include "wq_internal.h"

namespace wq {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;      // vectors in flight per lane group
constexpr int kMaxTokens = 16;  // tokens per CTA
constexpr int kMaxHalf = 64;    // rotated pairs

struct RopeArgs {
    const uint16_t *q, *k, *qw, *kw;
    int64_t ldq, ldk, ldqo, ldko, M;
    const int32_t *positions;
    const float *inv_freq;
    float eps;
    int half, Hq, H, tokens;  // tokens per CTA
    uint16_t *qo, *ko;
};

template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads)
qk_norm_rope_kernel(const RopeArgs p)
{
    constexpr int L = D / 8;  // lanes per vector
    __shared__ __align__(16) float cs[kMaxTokens * kMaxHalf], sn[kMaxTokens * kMaxHalf];
    const int tid = threadIdx.x, l = tid % L;
    const int64_t m0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)std::min<int64_t>(p.tokens, p.M - m0);
    const int vecs = p.Hq + p.H, total = nt * vecs * L;

    for (int base = 0; base < total; base += kThreads * kUnroll) {
        uint4 raw[kUnroll];
        int tok[kUnroll], head[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int idx = base + u * kThreads + tid;
            const int vec = idx / L;
            tok[u] = vec / vecs;
            head[u] = vec - tok[u] * vecs;
            raw[u] = make_uint4(0u, 0u, 0u, 0u);
            if (idx < total) {
                const int64_t m = m0 + tok[u];
                const uint16_t *src = head[u] < p.Hq ? p.q + m * p.ldq + head[u] * D : p.k + m * p.ldk + (head[u] - p.Hq) * D;
                raw[u] = *reinterpret_cast<const uint4 *>(src + l * 8);
            }
        }
        if (base == 0) {
            for (int i = tid; i < nt * p.half; i += kThreads) {
                const int t = i / p.half, f = i - t * p.half;
                const double turns = (double)p.positions[m0 + t] * (double)p.inv_freq[f] * 0.15915494309189535;  // / 2 pi
                const float part = (float)(2.0 * (turns - rint(turns)));
                sincospif(part, &sn[t * kMaxHalf + f], &cs[t * kMaxHalf + f]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int idx = base + u * kThreads + tid;
            const bool is_q = head[u] < p.Hq;
            float x[8];
            const uint32_t w4[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w4[i] << 16);
                x[2 * i + 1] = __uint_as_float(w4[i] & 0xffff0000u);
            }
            if (NORM) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
                const uint4 wv = __ldg(reinterpret_cast<const uint4 *>((is_q ? p.qw : p.kw) + l * 8));
                const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = x[2 * i] * inv * __uint_as_float(ww[i] << 16);
                    x[2 * i + 1] = x[2 * i + 1] * inv * __uint_as_float(ww[i] & 0xffff0000u);
                }
            }
            // lanes past `total` hold tok up to a CTA's worth too far: keep their table reads inside it
            const int t = idx < total ? tok[u] : 0;
            float y[8];
            if (INTERLEAVED) {
                const bool turned = l * 4 < p.half;
                const int f = turned ? l * 4 : 0;
                const float4 c = *reinterpret_cast<const float4 *>(&cs[t * kMaxHalf + f]);
                const float4 s = *reinterpret_cast<const float4 *>(&sn[t * kMaxHalf + f]);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[2 * i] = turned ? x[2 * i] * cc[i] - x[2 * i + 1] * ss[i] : x[2 * i];
                    y[2 * i + 1] = turned ? x[2 * i + 1] * cc[i] + x[2 * i] * ss[i] : x[2 * i + 1];
                }
            } else {
                const int hl = p.half / 8;  // lanes per half
                const bool turned = l < 2 * hl, second = turned && l >= hl;
                const int lane = tid & 31;
                const int other = turned ? (second ? lane - hl : lane + hl) : lane;
                const int f = turned ? (second ? l - hl : l) * 8 : 0;
                const float4 c0 = *reinterpret_cast<const float4 *>(&cs[t * kMaxHalf + f]);
                const float4 c1 = *reinterpret_cast<const float4 *>(&cs[t * kMaxHalf + f + 4]);
                const float4 s0 = *reinterpret_cast<const float4 *>(&sn[t * kMaxHalf + f]);
                const float4 s1 = *reinterpret_cast<const float4 *>(&sn[t * kMaxHalf + f + 4]);
                const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float o = __shfl_sync(0xffffffffu, x[i], other);
                    // first half: a cos - b sin with b the other lane's; second: b cos + a sin
                    y[i] = turned ? fmaf(x[i], cc[i], (second ? o : -o) * ss[i]) : x[i];
                }
            }
            if (idx < total) {
                const int64_t m = m0 + tok[u];
                uint16_t *dst = is_q ? p.qo + m * p.ldqo + head[u] * D : p.ko + m * p.ldko + (head[u] - p.Hq) * D;
                *reinterpret_cast<uint4 *>(dst + l * 8) =
                    make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            }
        }
    }
}

template <int D, bool INTERLEAVED>
void run(const RopeArgs &a, unsigned grid, cudaStream_t st)
{
    if (a.qw) qk_norm_rope_kernel<D, INTERLEAVED, true><<<grid, kThreads, 0, st>>>(a);
    else qk_norm_rope_kernel<D, INTERLEAVED, false><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace

void launch_qk_norm_rope(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *qw,
                         const uint16_t *kw, float eps, const int32_t *positions, const float *inv_freq, int64_t rot,
                         int interleaved, int64_t M, int64_t Hq, int64_t H, int64_t D, uint16_t *qo, int64_t ldqo,
                         uint16_t *ko, int64_t ldko, cudaStream_t st)
{
    RopeArgs a{q, k, qw, kw, ldq, ldk, ldqo, ldko, M, positions, inv_freq, eps, (int)(rot / 2), (int)Hq, (int)H, 1, qo, ko};
    // a few tokens per CTA where a token is small, as long as every SM keeps a few CTAs
    const int64_t lanes = (Hq + H) * (D / 8);
    a.tokens = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxTokens, kThreads * kUnroll / lanes, M / 592}));
    const unsigned grid = (unsigned)((M + a.tokens - 1) / a.tokens);
    if (D == 128) {
        if (interleaved) run<128, true>(a, grid, st);
        else run<128, false>(a, grid, st);
    } else {
        if (interleaved) run<64, true>(a, grid, st);
        else run<64, false>(a, grid, st);
    }
}

}  // namespace wq
