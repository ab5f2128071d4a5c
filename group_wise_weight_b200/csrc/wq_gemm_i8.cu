// wq_gemm_i8.cu -- INT8 W8A8 matmul on the 5th-generation tensor cores
// (sm_100a, tcgen05.mma kind::i8).
//
//   y[m][n] = bf16( float(sum_k xq[m][k] wq[n][k]) * (sx[m] * sw[n]) ),
// sums exact 32-bit integers ("Quantization Methods Compared: INT8, GPTQ,
// AWQ, FP8, FP4 and KV-Cache Quantization", section "What quantisation does":
// the product of the codes, scaled; here a scale per token and per channel).
//
// Three kernels, all persistent, all fed by TMA with the 128-byte swizzle in
// stages of 128 bytes of K (past K's end a copy fills in zeros, which add
// nothing), accumulators double-buffered in tensor memory, every barrier wait
// bounded (but a pair's two cluster barriers and the epilogue warps' named ones, which
// every thread reaches whatever has run out).
//
// Few and middling rows (gemm_i8_rows_kernel): the weights bound the call, so
// their rows are shared out evenly, rounded up to 8: up to 128 tokens N / 148 of
// them to an SM (in rounds of at most 128), beyond that tiles of up to 128
// tokens, the ones on the same weights next to one another; no sum is split.
// A pair of CTAs computes 128 tokens by twice that many weight rows: each loads
// its weight rows and half of the tokens, which halves what the tokens take of
// an SM's intake, and the pair's MMA (128 x up to 256) reads both halves.
// Stages hold several pieces of 128 bytes of K, as many as leave 5 stages in
// the ring: a weight row's bytes then come in runs of up to 1 KB, which DRAM
// gives faster (M = 1, 8192 x 28672: pieces singly 52.3 us, two 39.5, four
// 38.6; N = 1000: 50.2, 32, 21).  Measured: M = 1, 10240 x 8192 17.5 us (4.8
// TB/s), 8192 x 28672 38.3 (6.1 TB/s); M = 100, the same 42.6 us; M = 384, 2048
// x 8192 11.7 us.  With the other two kernels: 18.9, 39.8, 51.5, 20.9.
//
// Few weight rows and a deep K, or few rows and a shallow one
// (gemm_i8_stream_kernel): tiles of 128 weight rows (the MMA's M, so a token
// costs one of its N columns) by 16 to 128 tokens, whole ones to a CTA or a
// tile's K in equal parts to several.  A CTA with a part leaves its integer sums
// in the workspace and adds its stages to the tile's counter, waits for the
// counter (bounded, and the launch is cooperative: CTAs that wait for one
// another all run) and does a share of the columns, exact in any order.  The
// ring takes 200 KB: what an SM has in flight sets the rate (M = 1, N = 57344,
// K = 8192: 6 stages of 18 KB 81.6 us, 11 stages 72.8 us, 6.45 TB/s).
//
// All start while the previous kernel ends (0.4 us of a call; asking L2 for
// the first weights then gained nothing) and read and write nothing before
// that has completed.
//
// Many rows (gemm_i8_pair_kernel): the tensor cores bound the product, provided
// the operands reach them: at 8,192 int8 multiply-adds per cycle an SM that
// computes a 128 x 256 tile alone takes in 96 bytes per cycle, more than L2
// gives every SM at once.  A pair of CTAs computes 256 x 256: each holds the
// accumulators of its 128 rows of activations and loads those and half of the
// tile's 256 weight rows; the pair's MMA reads both halves, so an SM takes in
// 64 bytes per cycle.  The tile's weight rows are fewer, in steps of 32, where
// that fills the last round (M = 700, 8192 x 8192: 45.3 -> 38.9 us; M = 256,
// 10240 x 8192: 27.9 -> 24.3).  Warp 0 of each CTA copies, its completions counted by
// the leader CTA's barrier; in the leader, one thread of warp 1 issues the
// pair's MMAs and their commits, which reach both CTAs; warps 2-9 turn one of
// two accumulators into bf16 while the MMAs fill the other.  Tiles are taken
// round-robin in an order that walks the weight columns within a band of
// activation rows small enough to stay in L2.  Measured: M = 8,190, N = 57,344,
// K = 8,192 in 2.23 to 2.26 ms, 3,410 to 3,457 TOPS with the tensor pipe 89% busy
// (2.49 to 2.76 ms once the power cap lowers the clock); 2,048 x 8,192 x 8,192 86 us.
#include <algorithm>
#include <atomic>

#include "wq_internal.h"
#include "wq_prompt.cuh"

namespace wq {

namespace {

constexpr int kTile = 256;                    // rows of activations and of weights per pair
constexpr int kHalf = 128;                    // of each per CTA
constexpr int kRowBytes = 128;                // bytes of K per row and stage
constexpr int kOperand = kHalf * kRowBytes;   // 16 KB
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kOutWarps = 8;                  // epilogue warps: two per quarter of tensor memory, on alternate 32 columns
constexpr int kThreads = 64 + 32 * kOutWarps;
constexpr int kOutBytes = 32 * 64;            // per epilogue warp: 32 rows of 32 bf16
constexpr int kOutOff = kStages * kStageBytes;
constexpr int kScaleOff = kOutOff + kOutWarps * kOutBytes;
constexpr int kBarOff = kScaleOff + kTile * 4;
constexpr int kSmem = kBarOff + 256;
constexpr int64_t kBandBytes = 32 << 20;      // activation rows of a band: a quarter of L2

struct Bars {
    uint64_t full[kStages], empty[kStages], d_full[2], d_empty[2], done;
    int abort;
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 256, "the barrier area");

struct Args {
    int64_t M, N, K;
    const float *xs;
    const uint16_t *ws;
    uint16_t *y;
    int *status;
    int mt, nt, band, each;  // tiles of rows and columns, row tiles per band, weight rows per CTA and tile (a multiple of 16)
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The leader CTA's shared address of what lies at `p` here.
__device__ __forceinline__ uint32_t at_leader(const void *p)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

__device__ __forceinline__ void arrive_at(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// A tile into this CTA's shared memory, counted by the barrier at cluster address `bar`.
__device__ __forceinline__ void load_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
                 ::"r"(smem_u32(dst)), "l"(map), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}

// D (+)= A B^T over the pair, signed bytes, 32 of K.
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Arrive on this barrier in both CTAs when the MMAs issued so far have completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

// Instruction descriptor, kind::i8: signed A and B (format code 1), both K-major, s32 D (format code 2).
__host__ __device__ constexpr uint32_t idesc_s8_s32(int m, int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Tile t in order: bands of row tiles; within one, column by column.
__device__ __forceinline__ void tile_at(const Args &p, int t, int &mi, int &ni)
{
    const int per_band = p.band * p.nt, b = t / per_band, rest = t - b * per_band;
    const int rows = min(p.band, p.mt - b * p.band);
    ni = rest / rows;
    mi = b * p.band + rest - ni * rows;
}

// The widest store, in bytes, that every row of y allows (y is 16-byte aligned, a tile's columns begin at a multiple of 8).
__device__ __forceinline__ int store_width(int64_t N) { return N % 8 == 0 ? 16 : N % 4 == 0 ? 8 : N % 2 == 0 ? 4 : 2; }

// A warp's 32 rows of 32 bf16 from `out` to `to`, a lane a T at a time, so that a store instruction writes 64 adjacent bytes of
// sizeof(T) / 2 rows.
template <typename T>
__device__ __forceinline__ void copy_rows(const uint8_t *out, uint16_t *to, int64_t N, int rows, int cols)
{
    constexpr int kBytes = sizeof(T), kLanes = 64 / kBytes, kAtOnce = 32 / kLanes;
    const int lane = threadIdx.x & 31, at = lane % kLanes * kBytes;
#pragma unroll 8
    for (int i = 0; i < 32 / kAtOnce; ++i) {
        const int r = kAtOnce * i + lane / kLanes;
        const T g = *reinterpret_cast<const T *>(out + r * 64 + ((at >> 4) ^ ((r >> 1) & 3)) * 16 + (at & 15));
        if (r < rows && at < 2 * cols) *reinterpret_cast<T *>(to + r * N + at / 2) = g;
    }
}

// 32 sums of this lane's row, scaled, to `to` (row 0's place; rows N apart): `rows` rows and `cols` columns of them, `width`
// bytes at a time (1821 tokens, K = 128, about 17,120 weight rows: 2 bytes 60.5 us, 4 44.0, 8 32.9, 16 29.2).
__device__ __forceinline__ void write_rows(const uint32_t v[32], float sx, const float *sw, uint8_t *out, uint16_t *to, int64_t N,
                                           int rows, int cols, int width)
{
    const int lane = threadIdx.x & 31;
    // 16-byte pieces at piece ^ (row / 2) % 4 of the row's 64 bytes: no bank conflicts either way
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 8 * e + 2 * i;
            g[i] = pack2_bf16(__fmul_rn((float)(int)v[j], __fmul_rn(sx, sw[j])),
                              __fmul_rn((float)(int)v[j + 1], __fmul_rn(sx, sw[j + 1])));
        }
        *reinterpret_cast<uint4 *>(out + lane * 64 + (e ^ ((lane >> 1) & 3)) * 16) = make_uint4(g[0], g[1], g[2], g[3]);
    }
    __syncwarp();
    if (width == 16) copy_rows<uint4>(out, to, N, rows, cols);
    else if (width == 8) copy_rows<uint2>(out, to, N, rows, cols);
    else if (width == 4) copy_rows<uint32_t>(out, to, N, rows, cols);
    else copy_rows<uint16_t>(out, to, N, rows, cols);
    __syncwarp();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const Args p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Bars &b = *reinterpret_cast<Bars *>(smem + kBarOff);
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int tiles = p.mt * p.nt, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int stages = (int)((p.K + kRowBytes - 1) / kRowBytes);
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, p.status, &b.abort); };

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&b.full[i], 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.d_full[i], 1);
            mbar_init(&b.d_empty[i], 2 * kOutWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(&b.done, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (wid == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (wid == 0) {
        // ------------------------------ copies ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                int mi, ni;
                tile_at(p, t, mi, ni);
                const int m = mi * kTile + (int)rank * kHalf, n = (2 * ni + (int)rank) * p.each;
                for (int s = 0; s < stages; ++s) {
                    if (issued >= (uint32_t)kStages && !wait(&b.empty[slot], phase ^ 1u)) { ok = false; break; }
                    uint8_t *st = smem + slot * kStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&b.full[slot], 2 * (kOperand + p.each * kRowBytes));  // both CTAs' bytes
                    const uint32_t bar = at_leader(&b.full[slot]);
                    load_pair(st, &xmap, bar, s * kRowBytes, m);
                    load_pair(st + kOperand, &wmap, bar, s * kRowBytes, n);
                    ++issued;
                    if (++slot == (uint32_t)kStages) { slot = 0; phase ^= 1u; }
                }
            }
            // the leader sees every copy of the pair land before either CTA may exit (bounded, ignoring abort)
            if (rank == 0) {
                for (uint32_t j = issued > (uint32_t)kStages ? issued - kStages : 0; j < issued; ++j) {
                    const uint64_t t0 = global_ns();
                    while (!mbar_try_wait(&b.full[j % kStages], (j / kStages) & 1u))
                        if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.status); break; }
                }
            }
        }
        __syncwarp();
    } else if (wid == 1) {
        // ------------------------------ MMAs: one thread of the leader ------------------------------
        if (rank == 0 && elect_one()) {
            uint32_t slot = 0, phase = 0, n = 0;
            const uint32_t base = smem_u32(smem);
            const uint32_t idesc = idesc_s8_s32(kTile, 2 * p.each);
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs, ++n) {
                const uint32_t buf = n & 1u;
                if (n >= 2 && !wait(&b.d_empty[buf], ((n >> 1) - 1) & 1u)) break;
                tc_fence_after();
                for (int s = 0; s < stages; ++s) {
                    if (!wait(&b.full[slot], phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a = base + slot * kStageBytes, w = a + kOperand;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma_pair(tmem + buf * 256u, smem_desc(a + 32u * e, 16, 1024, 2), smem_desc(w + 32u * e, 16, 1024, 2), idesc,
                                 (s > 0 || e > 0) ? 1u : 0u);
                    commit_pair(&b.empty[slot]);
                    if (++slot == (uint32_t)kStages) { slot = 0; phase ^= 1u; }
                }
                if (ok) commit_pair(&b.d_full[buf]);
            }
            commit_pair(&b.done);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&b.done, 0))  // every MMA must complete before tensor memory is released
                if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.status); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue: one row per thread ------------------------------
        const int quarter = wid & 3, et = tid - 64;
        const uint32_t lane_bits = (uint32_t)(quarter * 32) << 16;
        uint8_t *out = smem + kOutOff + (wid - 2) * kOutBytes;
        float *sw = reinterpret_cast<float *>(smem + kScaleOff);
        const uint32_t d_empty[2] = {at_leader(&b.d_empty[0]), at_leader(&b.d_empty[1])};
        const int width = store_width(p.N);
        uint32_t n = 0;
        bool ok = true;  // a warp whose wait has run out still meets the others at the barriers of the tiles that are left
        for (int t = pair; t < tiles; t += pairs, ++n) {
            int mi, ni;
            tile_at(p, t, mi, ni);
            const int64_t m0 = (int64_t)mi * kTile + rank * kHalf + quarter * 32, n0 = (int64_t)ni * 2 * p.each;
            named_bar_sync(1, 32 * kOutWarps);  // the scales of the tile before have been read
            for (int i = et; i < 2 * p.each; i += 32 * kOutWarps) sw[i] = n0 + i < p.N ? bf16_to_f32(p.ws[n0 + i]) : 0.0f;
            named_bar_sync(1, 32 * kOutWarps);
            const float sx = m0 + lane < p.M ? p.xs[m0 + lane] : 0.0f;
            const uint32_t buf = n & 1u;
            ok = ok && warp_wait(&b.d_full[buf], (n >> 1) & 1u, p.status, &b.abort);
            if (!ok) continue;
            tc_fence_after();
            const int rows = (int)min((int64_t)32, p.M - m0), cols = (int)min((int64_t)2 * p.each, p.N - n0);
#pragma unroll 1
            for (int c = (wid - 2) / 4 * 32; c < cols && rows > 0; c += 8 * kOutWarps) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_bits + buf * 256u + (uint32_t)c, v);
                tmem_wait_ld();
                write_rows(v, sx, sw + c, out, p.y + m0 * p.N + n0 + c, p.N, rows, cols - c, width);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(d_empty[buf]);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's MMAs have read this CTA's shared memory, its arrivals have landed
    tc_fence_after();
    if (wid == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ------------------------------------------------------------------------------------------------------------
// The weights' rows shared out
// ------------------------------------------------------------------------------------------------------------

constexpr int kRowsStages = 24;               // at most
constexpr int kRowsRing = 200 * 1024;
constexpr int kLeastStages = 5;  // in the ring, before a stage takes more pieces of K
constexpr int kRowsOut = kRowsRing + 8192;    // (the MMA reads 64 rows of tokens, stale ones behind the last stage's too)
constexpr int kRowsScale = kRowsOut + kOutWarps * kOutBytes;
constexpr int kRowsBar = kRowsScale + 256 * 4;
constexpr int kRowsSmem = kRowsBar + 512;

struct RowsBars {
    uint64_t full[kRowsStages], empty[kRowsStages], d_full[2], d_empty[2], done;
    int abort;
    uint32_t tmem;
};
static_assert(sizeof(RowsBars) <= 512, "the barrier area");

struct RowsArgs {
    Args g;
    int tiles, mt;       // of 2 `each` weight rows by 2 `tokens` tokens; tiles of tokens, which vary first
    int each, tokens;    // weight rows and tokens per CTA of a pair and tile
    int token_bytes, weight_bytes, stage_bytes, stages;  // of 128 of K; PIECES of them to a stage
};

template <int PIECES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_i8_rows_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const RowsArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    RowsBars &b = *reinterpret_cast<RowsBars *>(smem + kRowsBar);
    const Args &p = a.g;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank(), S = (uint32_t)a.stages;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    constexpr int kStep = PIECES * kRowBytes;  // of K
    const int steps = (int)((p.K + kStep - 1) / kStep);
    const bool other = a.tokens < p.M;  // the second CTA has tokens too (all but M = 1)
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, p.status, &b.abort); };

    if (tid == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(&b.full[i], 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.d_full[i], 1);
            mbar_init(&b.d_empty[i], 2 * kOutWarps);  // the epilogue warps of both CTAs
        }
        mbar_init(&b.done, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (wid == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)), "r"(256u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (wid == 0) {
        // ------------------------------ copies ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, phase = 0, issued = 0;
            const uint32_t bytes = (uint32_t)(2 * a.each + (other ? 2 : 1) * a.tokens) * kStep;  // both CTAs'
            bool ok = true;
            for (int t = pair; ok && t < a.tiles; t += pairs) {
                const int n = (2 * (t / a.mt) + (int)rank) * a.each, m = (2 * (t % a.mt) + (int)rank) * a.tokens;
                for (int s = 0; s < steps; ++s) {
                    if (issued >= S && !wait(&b.empty[slot], phase ^ 1u)) { ok = false; break; }
                    uint8_t *st = smem + slot * a.stage_bytes;
                    if (rank == 0) mbar_arrive_expect_tx(&b.full[slot], bytes);
                    const uint32_t bar = at_leader(&b.full[slot]);
#pragma unroll
                    for (int h = 0; h < PIECES; ++h) load_pair(st + PIECES * a.token_bytes + h * a.weight_bytes, &wmap, bar, s * kStep + h * kRowBytes, n);
                    if (rank == 0 || other) {
#pragma unroll
                        for (int h = 0; h < PIECES; ++h) load_pair(st + h * a.token_bytes, &xmap, bar, s * kStep + h * kRowBytes, m);
                    }
                    ++issued;
                    if (++slot == S) { slot = 0; phase ^= 1u; }
                }
            }
            // the leader sees every copy of the pair land before either CTA may exit (bounded, ignoring abort)
            if (rank == 0) {
                for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j) {
                    const uint64_t t0 = global_ns();
                    while (!mbar_try_wait(&b.full[j % S], (j / S) & 1u))
                        if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.status); break; }
                }
            }
        }
        __syncwarp();
    } else if (wid == 1) {
        // ------------------------------ MMAs: one thread of the leader ------------------------------
        if (rank == 0 && elect_one()) {
            uint32_t slot = 0, phase = 0, n = 0;
            const uint32_t base = smem_u32(smem);
            const uint32_t idesc = idesc_s8_s32(128, 2 * ((a.each + 15) & ~15));
            bool ok = true;
            for (int t = pair; ok && t < a.tiles; t += pairs, ++n) {
                const uint32_t buf = n & 1u;
                if (n >= 2 && !wait(&b.d_empty[buf], ((n >> 1) - 1) & 1u)) break;
                tc_fence_after();
                for (int s = 0; s < steps; ++s) {
                    if (!wait(&b.full[slot], phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t x = base + slot * a.stage_bytes, w = x + PIECES * a.token_bytes;
#pragma unroll
                    for (int e = 0; e < 4 * PIECES; ++e)
                        mma_pair(tmem + buf * 128u, smem_desc(x + e / 4 * a.token_bytes + 32u * (e % 4), 16, 1024, 2),
                                 smem_desc(w + e / 4 * a.weight_bytes + 32u * (e % 4), 16, 1024, 2), idesc, (s > 0 || e > 0) ? 1u : 0u);
                    commit_pair(&b.empty[slot]);
                    if (++slot == S) { slot = 0; phase ^= 1u; }
                }
                if (ok) commit_pair(&b.d_full[buf]);
            }
            commit_pair(&b.done);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&b.done, 0))  // every MMA must complete before tensor memory is released
                if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.status); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue: one token per thread ------------------------------
        // Tensor memory holds the CTA's 64 tokens twice: lanes 0-63 with the first CTA's weight rows, 64-127 with the second's.
        const int quarter = wid & 3, half = quarter >> 1, et = tid - 64;
        const uint32_t lane_bits = (uint32_t)(quarter * 32) << 16;
        uint8_t *out = smem + kRowsOut + (wid - 2) * kOutBytes;
        float *sw = reinterpret_cast<float *>(smem + kRowsScale);
        const uint32_t d_empty[2] = {at_leader(&b.d_empty[0]), at_leader(&b.d_empty[1])};
        const int width = store_width(p.N);
        const int row = (quarter & 1) * 32;
        uint32_t n = 0;
        bool ok = true;  // a warp whose wait has run out still meets the others at the barriers of the tiles that are left
        for (int t = pair; t < a.tiles; t += pairs, ++n) {
            const int64_t first = 2 * (int64_t)(t / a.mt) * a.each, m0 = (int64_t)(2 * (t % a.mt) + (int)rank) * a.tokens + row;
            const int rows = (int)min((int64_t)min(32, a.tokens - row), p.M - m0);
            const float sx = lane < rows ? p.xs[m0 + lane] : 0.0f;
            named_bar_sync(1, 32 * kOutWarps);  // the scales of the tile before have been read
            for (int i = et; i < 2 * a.each; i += 32 * kOutWarps)
                sw[i < a.each ? i : 128 + i - a.each] = first + i < p.N ? bf16_to_f32(p.ws[first + i]) : 0.0f;
            named_bar_sync(1, 32 * kOutWarps);
            const uint32_t buf = n & 1u;
            ok = ok && warp_wait(&b.d_full[buf], (n >> 1) & 1u, p.status, &b.abort);
            if (!ok) continue;
            tc_fence_after();
            const int64_t n0 = first + half * a.each;
            const int cols = (int)min((int64_t)a.each, p.N - n0);
#pragma unroll 1
            for (int c = (wid - 2) / 4 * 32; c < cols && rows > 0; c += 8 * kOutWarps) {
                uint32_t v[32];
                tmem_ld32(tmem + lane_bits + buf * 128u + (uint32_t)c, v);
                tmem_wait_ld();
                write_rows(v, sx, sw + 128 * half + c, out, p.y + m0 * p.N + n0 + c, p.N, rows, cols - c, width);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(d_empty[buf]);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the peer's MMAs have read this CTA's shared memory, its arrivals have landed
    tc_fence_after();
    if (wid == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256u) : "memory");
}

// ------------------------------------------------------------------------------------------------------------
// Few rows
// ------------------------------------------------------------------------------------------------------------

// D (+)= A B^T on one CTA, signed bytes, 32 of K.
__device__ __forceinline__ void mma_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// BN tokens by 128 weight rows.
template <int BN>
struct Stream {
    static constexpr int kStage = kOperand + BN * kRowBytes;
    static constexpr int kStages = 200 * 1024 / kStage;  // 11, 10, 8, 6
    static constexpr int kBarOff = kStages * kStage;
    static constexpr int kSmem = kBarOff + 1024;
    static constexpr uint32_t kCols = 2 * BN;  // two accumulators
};

constexpr int kStreamThreads = 192;
constexpr int kReader = 1 << 20;  // a counter's unit for CTAs that have read their share (the stages stay below it)
constexpr int kColumns = 4;       // columns in flight per warp of the shared sum

// Device-scope load with acquire semantics: later reads see what was written before the matching add.
__device__ __forceinline__ int ld_acquire(const int *p)
{
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

struct StreamBars {
    uint64_t full[11], empty[11], d_full[2], d_empty[2], done;
    int abort, complete;
    uint32_t tmem;
    float sx[128];
};
static_assert(sizeof(StreamBars) <= 1024, "the barrier area");

// Units (tile, stage) in tile order, `per` to a CTA: the stages of whole tiles where split = 1; else a tile's stages go to
// `split` CTAs (the last takes what is left), so that a CTA has one part of one tile.
struct Plan {
    int64_t tiles;
    int nt, stages, grid, split, per;
    __host__ __device__ int64_t begin_of(int b) const
    {
        return split > 1 ? (int64_t)(b / split) * stages + b % split * per : (int64_t)b * per;
    }
    __host__ __device__ int64_t end_of(int b) const
    {
        const int64_t end = begin_of(b) + per, last = split > 1 ? (int64_t)(b / split + 1) * stages : tiles * stages;
        return end < last ? end : last;
    }
};

struct StreamArgs {
    Args g;
    Plan plan;
    int *counters, *part;
};

template <int BN>
__global__ void __launch_bounds__(kStreamThreads)
gemm_i8_stream_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap, const StreamArgs p)
{
    using C = Stream<BN>;
    constexpr uint32_t S = (uint32_t)C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    StreamBars &b = *reinterpret_cast<StreamBars *>(smem + C::kBarOff);
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, stages = p.plan.stages, nt = p.plan.nt;
    const int64_t beg = p.plan.begin_of(blockIdx.x), end = p.plan.end_of(blockIdx.x);
    const int count = p.plan.split, mine = (int)blockIdx.x % count;  // parts of a tile, this CTA's
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, p.g.status, &b.abort); };

    if (tid == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(&b.full[i], 1);
            mbar_init(&b.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.d_full[i], 1);
            mbar_init(&b.d_empty[i], 4);
        }
        mbar_init(&b.done, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (wid == 1) tmem_alloc(&b.tmem, C::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    // not earlier: a next kernel that reads its weights before its own wait counts on all but this one being complete
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (wid == 0) {
        // ------------------------------ copies ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, phase = 0, issued = 0;
            int64_t tile = beg / stages;
            int s = (int)(beg - tile * stages);
            for (int64_t u = beg; u < end; ++u) {
                if (issued >= S && !wait(&b.empty[slot], phase ^ 1u)) break;
                uint8_t *st = smem + slot * C::kStage;
                const int n = (int)(tile % nt) * 128, m = (int)(tile / nt) * BN;
                mbar_arrive_expect_tx(&b.full[slot], C::kStage);
                tma_load_2d(st, &wmap, &b.full[slot], s * kRowBytes, n);
                tma_load_2d(st + kOperand, &xmap, &b.full[slot], s * kRowBytes, m);
                ++issued;
                if (++slot == S) { slot = 0; phase ^= 1u; }
                if (++s == stages) { s = 0; ++tile; }
            }
            // every issued copy must land before the CTA may exit (bounded, ignoring abort)
            for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j) {
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(&b.full[j % S], (j / S) & 1u))
                    if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.g.status); break; }
            }
        }
        __syncwarp();
    } else if (wid == 1) {
        // ------------------------------ MMAs: one thread ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, phase = 0, n = 0;
            const uint32_t base = smem_u32(smem);
            constexpr uint32_t idesc = idesc_s8_s32(128, BN);
            bool ok = true;
            for (int64_t u = beg; ok && u < end; ++n) {
                const int s0 = (int)(u % stages), s1 = (int)std::min<int64_t>(stages, s0 + (end - u));
                const uint32_t d = tmem + (n & 1u) * (uint32_t)BN;
                if (n >= 2 && !wait(&b.d_empty[n & 1u], ((n >> 1) - 1) & 1u)) break;
                tc_fence_after();
                for (int s = s0; s < s1; ++s) {
                    if (!wait(&b.full[slot], phase)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t w = base + slot * C::kStage, x = w + kOperand;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mma_one(d, smem_desc(w + 32u * e, 16, 1024, 2), smem_desc(x + 32u * e, 16, 1024, 2), idesc,
                                (s > s0 || e > 0) ? 1u : 0u);
                    tc_commit(&b.empty[slot]);
                    if (++slot == S) { slot = 0; phase ^= 1u; }
                }
                if (ok) tc_commit(&b.d_full[n & 1u]);
                u += s1 - s0;
            }
            tc_commit(&b.done);
            const uint64_t t0 = global_ns();
            while (!mbar_try_wait(&b.done, 0))  // every MMA must complete before tensor memory is released
                if (global_ns() - t0 > kWaitLimitNs) { record_timeout(p.g.status); break; }
        }
        __syncwarp();
    } else {
        // ------------------------------ epilogue: one weight row per thread ------------------------------
        const int quarter = wid & 3, r = quarter * 32 + lane;
        const uint32_t lane_bits = (uint32_t)(quarter * 32) << 16;
        const int64_t M = p.g.M, N = p.g.N;
        uint32_t n = 0;
        int64_t sx_at = -1;
        bool ok = true;  // a warp whose wait has run out still meets the others at the barriers that are left
        for (int64_t u = beg, next; u < end; u = next, ++n) {
            const int64_t tile = u / stages;
            const int s0 = (int)(u - tile * stages), s1 = (int)std::min<int64_t>(stages, s0 + (end - u));
            next = u + (s1 - s0);
            const int64_t nr = tile % nt * 128 + r, m0 = tile / nt * BN;
            const int cols = (int)std::min<int64_t>(BN, M - m0);
            const float sw = nr < N ? bf16_to_f32(p.g.ws[nr]) : 0.0f;
            if (m0 != sx_at) {  // the tokens' scales, while the MMAs run
                named_bar_sync(1, 128);
                if (r < cols) b.sx[r] = p.g.xs[m0 + r];
                named_bar_sync(1, 128);
                sx_at = m0;
            }
            ok = ok && warp_wait(&b.d_full[n & 1u], (n >> 1) & 1u, p.g.status, &b.abort);
            tc_fence_after();
            const uint32_t d = tmem + lane_bits + (n & 1u) * (uint32_t)BN;
            if (count > 1) {  // the sums to the tile's parts: [part][column][row]
                int *part = p.part + (tile * count + mine) * (BN * 128) + r;
#pragma unroll 1
                for (int c = 0; c < cols && ok; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(d + (uint32_t)c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c + e < cols) part[(c + e) * 128] = (int)v[e];
                }
                __threadfence();
                ok = named_bar_and(1, 128, ok);  // one answer for the four warps, which join the tile's sums together
                if (ok && tid == 64) atomicAdd(p.counters + tile, s1 - s0);
            } else if (ok) {
#pragma unroll 1
                for (int c = 0; c < cols; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(d + (uint32_t)c, v);
                    tmem_wait_ld();
                    if (nr < N) {
                        uint16_t *to = p.g.y + (m0 + c) * N + nr;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            if (c + e < cols) *to = f32_to_bf16(__fmul_rn((float)(int)v[e], __fmul_rn(b.sx[c + e], sw)));
                            to += N;
                        }
                    }
                }
            }
            if (!ok) continue;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.d_empty[n & 1u]);
        }
        if (count > 1 && ok) {
            // this CTA's share of its tile's columns
            const int64_t tile = beg / stages;
            if (tid == 64) {
                int there = 1;
                const uint64_t since = global_ns();
                while ((ld_acquire(p.counters + tile) & (kReader - 1)) != stages) {
                    if (b.abort) { there = 0; break; }
                    if (global_ns() - since > kWaitLimitNs) {
                        record_timeout(p.g.status);
                        b.abort = 1;
                        there = 0;
                        break;
                    }
                }
                b.complete = there;
            }
            named_bar_sync(1, 128);
            if (*(volatile int *)&b.complete != 0) {
                __threadfence();
                const int64_t nr = tile % nt * 128 + 4 * lane, m0 = tile / nt * BN;
                const int cols = (int)std::min<int64_t>(BN, M - m0), c0 = cols * mine / count, c1 = cols * (mine + 1) / count;
                const int *parts = p.part + tile * count * (BN * 128) + 4 * lane;
                float sw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sw[i] = nr + i < N ? bf16_to_f32(p.g.ws[nr + i]) : 0.0f;
                // a warp adds up one column of 128 rows at a time, 4 rows per lane
                for (int c = c0 + quarter; c < c1; c += 4 * kColumns) {
                    int4 v[kColumns];
#pragma unroll
                    for (int i = 0; i < kColumns; ++i) v[i] = make_int4(0, 0, 0, 0);
                    for (int o = 0; o < count; ++o) {
#pragma unroll
                        for (int i = 0; i < kColumns; ++i) {
                            if (c + 4 * i < c1) {
                                const int4 w = __ldcg(reinterpret_cast<const int4 *>(parts + ((int64_t)o * BN + c + 4 * i) * 128));
                                v[i].x += w.x; v[i].y += w.y; v[i].z += w.z; v[i].w += w.w;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kColumns; ++i) {
                        if (c + 4 * i >= c1) continue;
                        const int64_t m = m0 + c + 4 * i;
                        const float sx = p.g.xs[m];
                        const float y0 = __fmul_rn((float)v[i].x, __fmul_rn(sx, sw[0])), y1 = __fmul_rn((float)v[i].y, __fmul_rn(sx, sw[1]));
                        const float y2 = __fmul_rn((float)v[i].z, __fmul_rn(sx, sw[2])), y3 = __fmul_rn((float)v[i].w, __fmul_rn(sx, sw[3]));
                        uint16_t *to = p.g.y + m * N + nr;
                        if (N % 4 == 0) {
                            if (nr < N) *reinterpret_cast<uint2 *>(to) = make_uint2(pack2_bf16(y0, y1), pack2_bf16(y2, y3));
                        } else {
                            if (nr < N) to[0] = f32_to_bf16(y0);
                            if (nr + 1 < N) to[1] = f32_to_bf16(y1);
                            if (nr + 2 < N) to[2] = f32_to_bf16(y2);
                            if (nr + 3 < N) to[3] = f32_to_bf16(y3);
                        }
                    }
                }
                // the last of the tile's readers leaves its counter zero
                named_bar_sync(1, 128);
                if (tid == 64 && atomicAdd(p.counters + tile, kReader) / kReader == count - 1) p.counters[tile] = 0;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == 1) tmem_dealloc(tmem, C::kCols);
}

// SMs of the current device; the kernels' shared-memory limits are raised on their first use there.
int sms_of_device()
{
    static std::atomic<int> sms_of[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    int sms = sms_of[dev].load(std::memory_order_acquire);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        const cudaFuncAttribute limit = cudaFuncAttributeMaxDynamicSharedMemorySize;
        cudaFuncSetAttribute(gemm_i8_pair_kernel, limit, kSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_rows_kernel<1>, limit, kRowsSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_rows_kernel<2>, limit, kRowsSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_rows_kernel<4>, limit, kRowsSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_rows_kernel<8>, limit, kRowsSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_stream_kernel<16>, limit, Stream<16>::kSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_stream_kernel<32>, limit, Stream<32>::kSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_stream_kernel<64>, limit, Stream<64>::kSmem + 1024);
        cudaFuncSetAttribute(gemm_i8_stream_kernel<128>, limit, Stream<128>::kSmem + 1024);
        sms_of[dev].store(sms, std::memory_order_release);
    }
    return sms;
}

int stream_bn(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// Tiles of the rows kernel: the fewest rounds in which a CTA has at most 128 weight rows.
struct RowsPlan {
    int mt, tokens, each, tiles, rounds;  // tiles of tokens; tokens and weight rows per CTA
    int token_bytes, weight_bytes, pieces;
};

RowsPlan plan_rows(int64_t M, int64_t N, int sms)
{
    RowsPlan p;
    const int64_t pairs = sms / 2, mt = (M + 127) / 128;
    p.mt = (int)mt;
    p.tokens = (int)((M + 2 * mt - 1) / (2 * mt));
    int64_t each = 0;
    for (int64_t rounds = std::max<int64_t>(1, mt * N / (256 * pairs)); each == 0 || each > 128; ++rounds) {
        const int64_t nt = std::max<int64_t>(1, rounds * pairs / mt);
        each = ((N + 2 * nt - 1) / (2 * nt) + 7) / 8 * 8;
    }
    p.each = (int)each;
    p.tiles = (int)((N + 2 * each - 1) / (2 * each) * mt);
    p.rounds = (int)((p.tiles + pairs - 1) / pairs);
    p.token_bytes = (p.tokens + 7) / 8 * 1024;
    p.weight_bytes = (p.each + 15) / 16 * 2048;
    p.pieces = 8;
    while (p.pieces > 1 && kRowsRing / (p.pieces * (p.token_bytes + p.weight_bytes)) < kLeastStages) p.pieces /= 2;
    return p;
}

// Tiles of the pair kernel: 256 tokens by the weight rows that fill the fewest rounds evenly.
struct PairPlan {
    int mt, nt, each, rounds;  // tiles of tokens and of weight rows; weight rows per CTA
};

PairPlan plan_pairs(int64_t M, int64_t N, int sms)
{
    PairPlan p;
    const int64_t pairs = sms / 2, mt = (M + kTile - 1) / kTile;
    int64_t each = 0;
    for (int64_t rounds = std::max<int64_t>(1, mt * N / (kTile * pairs)); each == 0 || each > kHalf; ++rounds) {
        const int64_t nt = std::max<int64_t>(1, rounds * pairs / mt);
        each = ((N + 2 * nt - 1) / (2 * nt) + 15) / 16 * 16;
    }
    p.mt = (int)mt;
    p.each = (int)each;
    p.nt = (int)((N + 2 * each - 1) / (2 * each));
    p.rounds = (int)((mt * p.nt + pairs - 1) / pairs);
    return p;
}

// Which kernel, by the time that this model gives (microseconds beyond a launch; a stage or piece is 128 of K):
//   rows: the rounds' pieces, each the greatest of what a step takes however small (by the pieces in it), what HBM takes
//     for the weights, and what an SM takes in
//   pairs: the rounds' stages, each kPair in proportion to the tile's weight rows, or what HBM or an SM takes as above
//   stream, whole tiles: a CTA takes ceil(tiles / SMs) of them; a stage takes 0.25 where few CTAs run, and what HBM gives
//     it with every SM at work; a token's stores 0.025
//   stream, split: the same number of CTAs for every tile, 8 stages at least to each, and the adding up
// The rows' and pairs' stores are not in it, which decide where K is small (1821 x 17124 x 128: 33.6 us, its bytes 9.9): there
// it compares main loops only.  Fitted to 250 shapes of 1 to 2000 tokens; over the same shapes what it takes is within 5%
// of the best but for 17 (within 14%).  No others were held back to check it.  Measured, taken (not taken): M = 16, 8192 x 8192: rows 14.7 (split 17.1); M = 100, 57344 x 8192: rows 82
// (whole 89); M = 128, 2048 x 8192: rows 8.7 (split 13.7); M = 256, 8192 x 8192: rows 19.0 (whole 22.7); M = 512, the same:
// pairs 26.9 (rows 31.7); M = 1, 14336 x 4096: whole 11.9 (rows 13.2); M = 1, 1000 x 28672: split 15.3 (rows 18.4).
constexpr double kUnit = 0.25, kUnitAll = 0.36, kPair = 0.33;
constexpr int kLeastUnits = 8;

struct Choice {
    enum { kRows, kPairs, kStream } kernel;
    RowsPlan rows;
    PairPlan pairs;
    Plan plan;  // of the stream
};

Choice choose(int64_t M, int64_t N, int64_t K, int sms)
{
    Choice c;
    const int bn = stream_bn(M);
    Plan &p = c.plan;
    p.nt = (int)((N + 127) / 128);
    p.tiles = (M + bn - 1) / bn * p.nt;
    p.stages = (int)((K + kRowBytes - 1) / kRowBytes);
    const auto unit = [&](int64_t grid) { return std::max(kUnit, kUnitAll * (double)grid / sms); };
    const int64_t rounds = (p.tiles + sms - 1) / sms, whole_grid = (p.tiles + rounds - 1) / rounds;
    const double whole = (double)(rounds * p.stages) * unit(whole_grid) + 0.025 * (double)(rounds * std::min<int64_t>(M, 128));
    const int most = (int)std::min<int64_t>(sms / p.tiles, p.stages / kLeastUnits);
    double split = 1e30;
    if (most > 1) {
        p.per = (p.stages + most - 1) / most;
        p.split = (p.stages + p.per - 1) / p.per;
        p.grid = (int)(p.split * p.tiles);
        split = p.per * unit(p.grid) + 2 + 0.25 * p.split + bn / 32.0;
    }
    if (whole <= split) {
        p.split = 1;
        p.grid = (int)whole_grid;
        p.per = (int)(rounds * p.stages);
    }
    const double stream = std::min(whole, split);
    const int64_t pair_tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
    double pairs = 1e30;
    if (M > 128 && pair_tiles < (1 << 30)) {
        c.pairs = plan_pairs(M, N, sms);
        const double each = c.pairs.each, share = each / c.pairs.mt;
        pairs = (double)c.pairs.rounds * p.stages * std::max({kPair * each / kHalf, 0.00278 * share, 0.0009 * (each + kHalf) + 0.0014 * share}) + 1;
    }
    double rows = 1e30;
    if (N < (1 << 30) && M < (1 << 30) && pair_tiles < (1 << 28)) {
        c.rows = plan_rows(M, N, sms);
        const RowsPlan &r = c.rows;
        const double per = std::min((double)r.each, (double)N * r.mt / (double)(sms / 2 * 2 * (int64_t)r.rounds)), share = per / r.mt;
        const double step = r.pieces == 8 ? 0.062 : r.pieces == 4 ? 0.07 : r.pieces == 2 ? 0.105 : 0.2;
        rows = (double)r.rounds * p.stages * std::max({step, 0.00278 * share, 0.0009 * (per + r.tokens) + 0.0014 * share}) + 1.7;
    }
    c.kernel = rows <= std::min(pairs, stream) ? Choice::kRows : pairs <= stream ? Choice::kPairs : Choice::kStream;
    return c;
}

template <int BN>
int run_stream(const int8_t *xq, const int8_t *wq, const Args &g, const Plan &plan, void *workspace, cudaStream_t st)
{
    using C = Stream<BN>;
    CUtensorMap xmap, wmap;
    if (!encode_tmap_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, kRowBytes, BN,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, kRowBytes, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    StreamArgs a{g, plan, nullptr, nullptr};
    uint8_t *w8 = static_cast<uint8_t *>(workspace);
    a.counters = reinterpret_cast<int *>(w8);
    a.part = reinterpret_cast<int *>(w8 + counter_region_bytes(a.plan.tiles));
    if (plan.split > 1 && clear_extra_counters(workspace, plan.tiles, st) != cudaSuccess) return -2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.plan.grid);
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = C::kSmem + 1024;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    // CTAs that wait for one another start together or not at all, whatever else holds SMs (no time lost: M = 100, 8192 x
    // 28672 52.4 us, 52.7 without)
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan.split > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, gemm_i8_stream_kernel<BN>, xmap, wmap, a);  // a failure is the caller's last error
    return 0;
}

int run_pairs(const int8_t *xq, const int8_t *wq, Args a, const PairPlan &r, int sms, cudaStream_t st)
{
    CUtensorMap xmap, wmap;
    if (!encode_tmap_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)a.K, kRowBytes, kHalf,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.K, kRowBytes, (uint32_t)r.each,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    a.mt = r.mt;
    a.nt = r.nt;
    a.each = r.each;
    a.band = (int)std::max<int64_t>(1, std::min<int64_t>(a.mt, kBandBytes / (kTile * a.K)));
    const int64_t pairs = std::min<int64_t>((int64_t)a.mt * a.nt, sms / 2);
    launch_behind(gemm_i8_pair_kernel, (unsigned)(2 * pairs), kThreads, kSmem + 1024, st, xmap, wmap, a);
    return 0;
}

int run_rows(const int8_t *xq, const int8_t *wq, const Args &g, const RowsPlan &r, int sms, cudaStream_t st)
{
    const int stage_bytes = r.pieces * (r.token_bytes + r.weight_bytes);
    const RowsArgs a{g, r.tiles, r.mt, r.each, r.tokens, r.token_bytes, r.weight_bytes, stage_bytes, std::min(kRowsStages, kRowsRing / stage_bytes)};
    CUtensorMap xmap, wmap;
    if (!encode_tmap_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)g.K, (uint64_t)g.M, (uint64_t)g.K, kRowBytes,
                        (uint32_t)r.tokens, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, (uint64_t)g.K, (uint64_t)g.N, (uint64_t)g.K, kRowBytes,
                        (uint32_t)r.each, CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    const int pairs = std::min(r.tiles, sms / 2);
    const auto kernel = r.pieces == 8   ? gemm_i8_rows_kernel<8>
                        : r.pieces == 4 ? gemm_i8_rows_kernel<4>
                        : r.pieces == 2 ? gemm_i8_rows_kernel<2>
                                        : gemm_i8_rows_kernel<1>;
    launch_behind(kernel, (unsigned)(2 * pairs), kThreads, kRowsSmem + 1024, st, xmap, wmap, a);
    return 0;
}

}  // namespace

size_t gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || N <= 0 || K <= 0 || K % 32 != 0) return 0;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const Choice c = choose(M, N, K, sms);
    if (c.kernel != Choice::kStream || c.plan.split == 1) return 0;  // no tile is split
    return counter_region_bytes(c.plan.tiles) +
           ((size_t)c.plan.tiles * c.plan.split * stream_bn(M) * 128 * sizeof(int) + 255) / 256 * 256;
}

int launch_gemm_w8a8_int8(const int8_t *xq, const float *xscales, int64_t M, int64_t N, int64_t K, const int8_t *wq,
                          const uint16_t *wscales, uint16_t *y, void *workspace, int *status, cudaStream_t st)
{
    const int sms = sms_of_device();
    if (sms < 2) return -2;
    const Args g{M, N, K, xscales, wscales, y, status, 0, 0, 0, 0};
    const Choice c = choose(M, N, K, sms);
    if (c.kernel == Choice::kRows) return run_rows(xq, wq, g, c.rows, sms, st);
    if (c.kernel == Choice::kPairs) return run_pairs(xq, wq, g, c.pairs, sms, st);
    switch (stream_bn(M)) {
    case 16: return run_stream<16>(xq, wq, g, c.plan, workspace, st);
    case 32: return run_stream<32>(xq, wq, g, c.plan, workspace, st);
    case 64: return run_stream<64>(xq, wq, g, c.plan, workspace, st);
    default: return run_stream<128>(xq, wq, g, c.plan, workspace, st);
    }
}

}  // namespace wq
