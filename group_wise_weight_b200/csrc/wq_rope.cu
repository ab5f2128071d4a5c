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
// The pass reads and writes 2 bytes per value and should be bound by HBM; the
// first form (a lane's pair partner in another lane, tables in shared memory)
// was bound by its instructions instead.  Here a lane holds both members of
// its four pairs -- 4 values of each half, or 8 adjacent ones when interleaved
// -- so no value crosses lanes but the sum of squares, and the products of
// weights, cosines and sines that its values meet stay in registers for all
// heads of a token:
//   y_a = inv (a (w_a cos) - b (w_b sin)),  y_b = inv (b (w_b cos) + a (w_a sin)).
// A warp takes 256 / D heads of one token at a time, kUnroll loads in flight;
// where tokens are few a token's heads are shared out to several warps, its
// queries and keys apart.  The first heads' loads are under way while the
// sines and cosines are formed, and the kernel starts while the previous one
// ends (without the two 128 tokens took 7.3 us, 16,384 104).
// Measured: 16,384 tokens, 64 + 8 heads of 128 with norms, 102 us (5.9 TB/s,
// 90% of a copy); 128 tokens 5.1 us, 3.7 in a graph: launch and load latency.
#include <algorithm>

#include "wq_internal.h"
#include "wq_prompt.cuh"

namespace wq {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;   // loads in flight per lane
constexpr int kMaxHalf = 64; // rotated pairs

struct RopeArgs {
    const uint16_t *q, *k, *qw, *kw;
    int64_t ldq, ldk, ldqo, ldko, M;
    const int32_t *positions;
    const float *inv_freq;
    float eps;
    int half, Hq, H, split, qsplit;  // warps per token; with more than one, those of the queries (the others have the keys)
    uint16_t *qo, *ko;
};

struct Pairs {
    f32x2 a[2], b[2];  // the first and second members of four pairs
};

template <bool INTERLEAVED>
__device__ __forceinline__ Pairs unpack(const uint2 &u, const uint2 &v)
{
    const float x0 = __uint_as_float(u.x << 16), x1 = __uint_as_float(u.x & 0xffff0000u);
    const float x2 = __uint_as_float(u.y << 16), x3 = __uint_as_float(u.y & 0xffff0000u);
    const float x4 = __uint_as_float(v.x << 16), x5 = __uint_as_float(v.x & 0xffff0000u);
    const float x6 = __uint_as_float(v.y << 16), x7 = __uint_as_float(v.y & 0xffff0000u);
    return INTERLEAVED ? Pairs{{{x0, x2}, {x4, x6}}, {{x1, x3}, {x5, x7}}} : Pairs{{{x0, x1}, {x2, x3}}, {{x4, x5}, {x6, x7}}};
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// What a lane has in flight: its values of kUnroll heads.
struct Batch {
    uint2 u[kUnroll], v[kUnroll];
};

// The heads base + g, base + g + step, ... below `heads` of one token's queries (or keys), g the lane's group in the
// warp: src and dst at the token's row; o1, o2 the places of this lane's two groups of 4 values in a head.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void load_heads(Batch &x, const uint16_t *src, int base, int g, int step, int heads, int o1, int o2)
{
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
        const int h = base + g + e * step;
        x.u[e] = x.v[e] = make_uint2(0u, 0u);
        if (h < heads) {
            if (INTERLEAVED) {
                const uint4 r = *reinterpret_cast<const uint4 *>(src + h * D + o1);
                x.u[e] = make_uint2(r.x, r.y);
                x.v[e] = make_uint2(r.z, r.w);
            } else {
                x.u[e] = *reinterpret_cast<const uint2 *>(src + h * D + o1);
                x.v[e] = *reinterpret_cast<const uint2 *>(src + h * D + o2);
            }
        }
    }
}

// Turns them (or lets them pass, where the lane is not `turned`), `first` and the lane's weights w1, w2 being loaded already.
template <int D, bool INTERLEAVED, bool NORM>
__device__ __forceinline__ void turn_heads(Batch &first, const uint16_t *src, uint16_t *dst, int base, int g, int step, int heads,
                                           int o1, int o2, uint2 w1, uint2 w2, const float c[4], const float s[4], bool turned,
                                           float eps)
{
    constexpr int L = D / 8;  // lanes per head
    float wa[4], wb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) wa[i] = wb[i] = 1.0f;
    if (NORM) {
        const Pairs w = unpack<INTERLEAVED>(w1, w2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            wa[2 * i] = w.a[i].x; wa[2 * i + 1] = w.a[i].y;
            wb[2 * i] = w.b[i].x; wb[2 * i + 1] = w.b[i].y;
        }
    }
    f32x2 ac[2], as[2], bc[2], bs[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        ac[i] = f32x2{wa[2 * i] * c[2 * i], wa[2 * i + 1] * c[2 * i + 1]};
        as[i] = f32x2{wa[2 * i] * s[2 * i], wa[2 * i + 1] * s[2 * i + 1]};
        bc[i] = f32x2{wb[2 * i] * c[2 * i], wb[2 * i + 1] * c[2 * i + 1]};
        bs[i] = f32x2{-wb[2 * i] * s[2 * i], -wb[2 * i + 1] * s[2 * i + 1]};
    }
    while (base < heads) {
#pragma unroll
        for (int e = 0; e < kUnroll; ++e) {
            const int h = base + g + e * step;
            const Pairs x = unpack<INTERLEAVED>(first.u[e], first.v[e]);
            f32x2 ya[2], yb[2];
            float inv = 1.0f;
            if (NORM) {
                f32x2 ss = mul2(x.a[0], x.a[0]);
                ss = fma2_pairs(x.a[1], x.a[1], ss);
                ss = fma2_pairs(x.b[0], x.b[0], ss);
                ss = fma2_pairs(x.b[1], x.b[1], ss);
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                inv = rsqrtf(fmaf(sum, 1.0f / D, eps));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ya[i] = mul2(x.a[i], ac[i]);
                yb[i] = mul2(x.b[i], bc[i]);
                if (turned) {  // values that pass meet no other (an infinity times sin 0 would be NaN, -0 + 0 lose its sign)
                    ya[i] = fma2_pairs(x.b[i], bs[i], ya[i]);
                    yb[i] = fma2_pairs(x.a[i], as[i], yb[i]);
                }
                if (NORM) {
                    ya[i] = mul2(ya[i], f32x2{inv, inv});
                    yb[i] = mul2(yb[i], f32x2{inv, inv});
                }
            }
            if (h < heads) {
                if (INTERLEAVED) {
                    *reinterpret_cast<uint4 *>(dst + h * D + o1) =
                        make_uint4(pack2_bf16(ya[0].x, yb[0].x), pack2_bf16(ya[0].y, yb[0].y),
                                   pack2_bf16(ya[1].x, yb[1].x), pack2_bf16(ya[1].y, yb[1].y));
                } else {
                    *reinterpret_cast<uint2 *>(dst + h * D + o1) = make_uint2(pack2_bf16(ya[0].x, ya[0].y), pack2_bf16(ya[1].x, ya[1].y));
                    *reinterpret_cast<uint2 *>(dst + h * D + o2) = make_uint2(pack2_bf16(yb[0].x, yb[0].y), pack2_bf16(yb[1].x, yb[1].y));
                }
            }
        }
        base += step * kUnroll;
        if (base < heads) load_heads<D, INTERLEAVED>(first, src, base, g, step, heads, o1, o2);
    }
}

// 64 registers, so that an SM holds 32 warps (with 74 and 24 of them: 128 tokens of 72 heads 4.4 us, now 3.7; 8,192 of 40 heads
// of 64 17.9, 16.4; 16,384 of 72 100.5, 101.5).
template <int D, bool INTERLEAVED, bool NORM>
__global__ void __launch_bounds__(kThreads, 4)
qk_norm_rope_kernel(const RopeArgs p)
{
    constexpr int L = D / 8, kHeads = 32 / L;  // heads per warp at a time
    __shared__ __align__(16) float table[kWarps][2][kMaxHalf];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, g = lane / L;
    const int64_t task = (int64_t)blockIdx.x * kWarps + wid;
    const int64_t m = task / p.split;
    const int part = (int)(task - m * p.split);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (m >= p.M) return;
    // lane l holds the pairs 4 l .. 4 l + 3; past the rotated ones, 8 values that do not turn
    const bool turned = 4 * l < p.half;
    const int o1 = INTERLEAVED ? 8 * l : turned ? 4 * l : 8 * l;
    const int o2 = INTERLEAVED ? 8 * l + 4 : turned ? p.half + 4 * l : 8 * l + 4;
    // the first heads and their weights are on their way while the sines and cosines are formed
    const bool keys = p.split > 1 && part >= p.qsplit;
    const uint16_t *src = keys ? p.k + m * p.ldk : p.q + m * p.ldq, *weight = keys ? p.kw : p.qw;
    const int base = (keys ? part - p.qsplit : part) * kHeads, step = (p.split == 1 ? 1 : keys ? p.split - p.qsplit : p.qsplit) * kHeads;
    const int heads = keys ? p.H : p.Hq;
    Batch first;
    load_heads<D, INTERLEAVED>(first, src, base, g, step, heads, o1, o2);
    uint2 w1 = make_uint2(0u, 0u), w2 = w1;
    if (NORM) {
        w1 = *reinterpret_cast<const uint2 *>(weight + o1);
        w2 = *reinterpret_cast<const uint2 *>(weight + o2);
    }
    const double pos = (double)p.positions[m];
    for (int f = lane; f < p.half; f += 32) {
        const double turns = pos * (double)p.inv_freq[f] * 0.15915494309189535;  // / 2 pi
        sincospif((float)(2.0 * (turns - rint(turns))), &table[wid][1][f], &table[wid][0][f]);
    }
    __syncwarp();
    float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (turned) {
        const float4 cv = *reinterpret_cast<const float4 *>(&table[wid][0][4 * l]);
        const float4 sv = *reinterpret_cast<const float4 *>(&table[wid][1][4 * l]);
        c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
        s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
    }
    uint16_t *dst = keys ? p.ko + m * p.ldko : p.qo + m * p.ldqo;
    turn_heads<D, INTERLEAVED, NORM>(first, src, dst, base, g, step, heads, o1, o2, w1, w2, c, s, turned, p.eps);
    if (p.split > 1) return;
    src = p.k + m * p.ldk;
    load_heads<D, INTERLEAVED>(first, src, 0, g, kHeads, p.H, o1, o2);
    if (NORM) {
        w1 = *reinterpret_cast<const uint2 *>(p.kw + o1);
        w2 = *reinterpret_cast<const uint2 *>(p.kw + o2);
    }
    turn_heads<D, INTERLEAVED, NORM>(first, src, p.ko + m * p.ldko, 0, g, kHeads, p.H, o1, o2, w1, w2, c, s, turned, p.eps);
}

template <int D, bool INTERLEAVED>
void run(const RopeArgs &a, unsigned grid, cudaStream_t st)
{
    if (a.qw) launch_behind(qk_norm_rope_kernel<D, INTERLEAVED, true>, grid, kThreads, 0, st, a);
    else launch_behind(qk_norm_rope_kernel<D, INTERLEAVED, false>, grid, kThreads, 0, st, a);
}

}  // namespace

void launch_qk_norm_rope(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *qw,
                         const uint16_t *kw, float eps, const int32_t *positions, const float *inv_freq, int64_t rot,
                         int interleaved, int64_t M, int64_t Hq, int64_t H, int64_t D, uint16_t *qo, int64_t ldqo,
                         uint16_t *ko, int64_t ldko, cudaStream_t st)
{
    RopeArgs a{q, k, qw, kw, ldq, ldk, ldqo, ldko, M, positions, inv_freq, eps, (int)(rot / 2), (int)Hq, (int)H, 1, 1, qo, ko};
    // one warp per token once that fills the device (148 SMs x 32 warps), else a token's heads over more of them, queries
    // and keys apart
    const int64_t at_once = 256 / D, room = 148 * 32 / M, qturns = (Hq + at_once - 1) / at_once, kturns = (H + at_once - 1) / at_once;
    if (room >= 2) {
        const int64_t kwarps = std::max<int64_t>(1, std::min(kturns, room * H / (Hq + H)));
        a.qsplit = (int)std::min(qturns, room - kwarps);
        a.split = a.qsplit + (int)kwarps;
    }
    const unsigned grid = (unsigned)((M * a.split + kWarps - 1) / kWarps);
    if (D == 128) {
        if (interleaved) run<128, true>(a, grid, st);
        else run<128, false>(a, grid, st);
    } else {
        if (interleaved) run<64, true>(a, grid, st);
        else run<64, false>(a, grid, st);
    }
}

}  // namespace wq
