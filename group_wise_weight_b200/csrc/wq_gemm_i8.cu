// wq_gemm_i8.cu -- INT8 W8A8 matmul for many rows of activations, on pairs
// of SMs (sm_100a, tcgen05.mma kind::i8 with cta_group::2).
//
//   y[m][n] = bf16( float(sum_k xq[m][k] wq[n][k]) * (sx[m] * sw[n]) ),
// sums exact 32-bit integers ("Quantization Methods Compared: INT8, GPTQ,
// AWQ, FP8, FP4 and KV-Cache Quantization", section "What quantisation does":
// the product of the codes, scaled; here a scale per token and per channel).
//
// With many rows the tensor cores bound the product, provided the operands
// reach them: at 8,192 int8 multiply-adds per cycle an SM that computes a
// 128 x 256 tile alone takes in 96 bytes per cycle, more than L2 gives every SM
// at once.  A pair of CTAs computes 256 x 256: each holds the accumulators of
// its 128 rows of activations and loads those and half of the tile's 256
// weight rows; the pair's MMA reads both halves, so an SM takes in 64 bytes
// per cycle.
//
// Per CTA (192 threads): warp 0 copies stages of 128 bytes of K by TMA (128-byte
// swizzle) into a ring, its completions counted by the leader CTA's barrier;
// in the leader, one thread of warp 1 issues the pair's MMAs and their commits,
// which reach both CTAs; warps 2-5 turn one of two accumulators in tensor
// memory into bf16 while the MMAs fill the other.  Tiles are taken round-robin
// in an order that walks the weight columns within a band of activation rows
// small enough to stay in L2.  Every barrier wait is bounded (but the two
// cluster barriers, which every thread reaches).
#include <algorithm>
#include <atomic>

#include "wq_internal.h"
#include "wq_sm100.cuh"

namespace wq {

namespace {

constexpr int kTile = 256;                    // rows of activations and of weights per pair
constexpr int kHalf = 128;                    // of each per CTA
constexpr int kRowBytes = 128;                // bytes of K per row and stage
constexpr int kOperand = kHalf * kRowBytes;   // 16 KB
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kThreads = 192;
constexpr int kOutBytes = 32 * 64;            // per epilogue warp: 32 rows of 32 bf16
constexpr int kOutOff = kStages * kStageBytes;
constexpr int kScaleOff = kOutOff + 4 * kOutBytes;
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
    int mt, nt, band;  // tiles of rows and columns, row tiles per band
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

// D (+)= A B^T over the pair: 256 x 256, signed bytes, 32 of K.
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

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// Tile t in order: bands of row tiles; within one, column by column.
__device__ __forceinline__ void tile_at(const Args &p, int t, int &mi, int &ni)
{
    const int per_band = p.band * p.nt, b = t / per_band, rest = t - b * per_band;
    const int rows = min(p.band, p.mt - b * p.band);
    ni = rest / rows;
    mi = b * p.band + rest - ni * rows;
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
            mbar_init(&b.d_empty[i], 8);  // 4 epilogue warps of each CTA
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

    if (wid == 0) {
        // ------------------------------ copies ------------------------------
        if (elect_one()) {
            uint32_t slot = 0, phase = 0, issued = 0;
            bool ok = true;
            for (int t = pair; ok && t < tiles; t += pairs) {
                int mi, ni;
                tile_at(p, t, mi, ni);
                const int m = mi * kTile + (int)rank * kHalf, n = ni * kTile + (int)rank * kHalf;
                for (int s = 0; s < stages; ++s) {
                    if (issued >= (uint32_t)kStages && !wait(&b.empty[slot], phase ^ 1u)) { ok = false; break; }
                    uint8_t *st = smem + slot * kStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&b.full[slot], 2 * kStageBytes);  // both CTAs' bytes
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
            constexpr uint32_t idesc = idesc_s8_s32(kTile, kTile);
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
        const int quarter = wid & 3, row = quarter * 32 + lane, et = tid - 64;
        const uint32_t lane_bits = (uint32_t)(quarter * 32) << 16;
        uint8_t *out = smem + kOutOff + (wid - 2) * kOutBytes;
        float *sw = reinterpret_cast<float *>(smem + kScaleOff);
        const uint32_t d_empty[2] = {at_leader(&b.d_empty[0]), at_leader(&b.d_empty[1])};
        const bool vectors = p.N % 8 == 0;
        uint32_t n = 0;
        for (int t = pair; t < tiles; t += pairs, ++n) {
            int mi, ni;
            tile_at(p, t, mi, ni);
            const int64_t m0 = (int64_t)mi * kTile + rank * kHalf + quarter * 32, n0 = (int64_t)ni * kTile;
            named_bar_sync(1, 128);  // the scales of the tile before have been read
            for (int i = et; i < kTile; i += 128) sw[i] = n0 + i < p.N ? bf16_to_f32(ld_nc_u16(p.ws + n0 + i)) : 0.0f;
            named_bar_sync(1, 128);
            const float sx = m0 + lane < p.M ? __ldg(p.xs + m0 + lane) : 0.0f;
            const uint32_t buf = n & 1u;
            if (!wait(&b.d_full[buf], (n >> 1) & 1u)) break;
            tc_fence_after();
            const int rows = (int)min((int64_t)32, p.M - m0), cols = (int)min((int64_t)kTile, p.N - n0);
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
                if (c >= cols || rows <= 0) break;
                uint32_t v[32];
                tmem_ld32(tmem + lane_bits + buf * 256u + (uint32_t)c, v);
                tmem_wait_ld();
                // 16-byte pieces at piece ^ (row / 2) % 4 of the row's 64 bytes: no bank conflicts either way
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t g[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = 8 * e + 2 * i;
                        g[i] = pack_bf16x2(__fmul_rn((float)(int)v[j], __fmul_rn(sx, sw[c + j])),
                                           __fmul_rn((float)(int)v[j + 1], __fmul_rn(sx, sw[c + j + 1])));
                    }
                    *reinterpret_cast<uint4 *>(out + lane * 64 + (e ^ ((lane >> 1) & 3)) * 16) = make_uint4(g[0], g[1], g[2], g[3]);
                }
                __syncwarp();
                if (vectors) {
                    const int piece = lane & 3;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2);
                        const uint4 g = *reinterpret_cast<const uint4 *>(out + r * 64 + (piece ^ ((r >> 1) & 3)) * 16);
                        if (r < rows && c + 8 * piece < cols)
                            *reinterpret_cast<uint4 *>(p.y + (m0 + r) * p.N + n0 + c + 8 * piece) = g;
                    }
                } else {  // rows of y begin at any even address: one value per lane
                    for (int r = 0; r < rows; ++r) {
                        const int piece = (lane >> 3) ^ ((r >> 1) & 3);
                        const uint16_t h = *reinterpret_cast<const uint16_t *>(out + r * 64 + piece * 16 + (lane & 7) * 2);
                        if (c + lane < cols) p.y[(m0 + r) * p.N + n0 + c + lane] = h;
                    }
                }
                __syncwarp();
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

// SMs of the current device; the kernel's shared-memory limit is raised on its first use there.
int sms_of_device()
{
    static std::atomic<int> sms_of[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    int sms = sms_of[dev].load(std::memory_order_acquire);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cudaFuncSetAttribute(gemm_i8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem + 1024);
        sms_of[dev].store(sms, std::memory_order_release);
    }
    return sms;
}

}  // namespace

bool gemm_i8_pair_eligible(int64_t M, int64_t N, int64_t K)
{
    return M > 128 && N > 128;
}

int launch_gemm_i8_pair(const int8_t *xq, const float *xscales, int64_t M, int64_t N, int64_t K, const int8_t *wq,
                        const uint16_t *wscales, uint16_t *y, int *status, cudaStream_t st)
{
    CUtensorMap xmap, wmap;
    if (!encode_tmap_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, xq, (uint64_t)K, (uint64_t)M, (uint64_t)K, kRowBytes, kHalf,
                        CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tmap_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, wq, (uint64_t)K, (uint64_t)N, (uint64_t)K, kRowBytes, kHalf,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    const int sms = sms_of_device();
    if (sms < 2) return -2;
    Args a{M, N, K, xscales, wscales, y, status, (int)((M + kTile - 1) / kTile), (int)((N + kTile - 1) / kTile), 0};
    a.band = (int)std::max<int64_t>(1, std::min<int64_t>(a.mt, kBandBytes / (kTile * K)));
    const int64_t pairs = std::min<int64_t>((int64_t)a.mt * a.nt, sms / 2);
    gemm_i8_pair_kernel<<<(unsigned)(2 * pairs), kThreads, kSmem + 1024, st>>>(xmap, wmap, a);
    return 0;
}

}  // namespace wq
