// wq_prompt_attn.cu -- causal attention over whole prompts packed one after
// another, with grouped query heads, on the 5th-generation tensor cores.
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
// are scaled by e^(m_old - m_new).  Scaling is put off until m would grow by
// more than a factor of 2^8 in p (p, l and the accumulator then carry the old
// m, exactly; binary32 has room for 2^8 L), which leaves it to the first few
// blocks of most rows; putting it off is a published refinement of that method
// too.  Each row decides by its own scores.  Scores, m, l and the accumulator are binary32; p is
// rounded to bf16 as the second product's operand (at most 2^-8 of each
// term), while l sums the unrounded p.
//
// The r = Hq / H query heads of a KV head share its keys and values: a tile's
// 128 rows are (token, head) pairs, token-major, so it covers 128 / r tokens
// and short sequences still fill it.  A work item is two such tiles of one KV
// head (consecutive tokens), or one.  The grid has a CTA per item; one that
// runs claims further ones before they are launched (cluster launch control)
// and does their items too, so an SM keeps its pipeline filled across items of
// any length.
//
// Per block of 128 keys and tile: S = Q K^T (both operands K-major in shared
// memory, loaded by TMA with the 128-byte swizzle) into 128 columns of tensor
// memory; a warpgroup, one row per thread, turns S into P in place (bf16,
// the first 64 columns); O += P V with P from tensor memory and V from shared
// memory as it lies there (key rows, so the operand is MN-major).  The two
// tiles are half a period apart: while one's warpgroup is in its softmax the
// tensor core works on the other.  The block's two products take 1,024 cycles
// of the tensor core per tile and its 16,384 exponentials as many of the
// special-function units, so both are at their limits together (heads of 64:
// half the products, the exponentials alone).  Measured, causal halves only:
// one sequence of 16,384 tokens, 64 query and 8 KV heads of 128, 3.32 to 3.43 ms
// (1,282 to 1,325 TFLOP/s; 3.96 ms once the power cap lowers the clock); 32 query
// heads of 64, 1.35 ms (812).  Short prompts lose the ends: 48 of 1 to 331 tokens,
// 64 query heads, 78 us (76 with waits answered lane by lane and a warp's rows
// moving m together, which is wrong: see warp_wait and move_max).  A block of 64 keys with two S tiles, a polynomial for
// part of the exponentials, softmax warpgroups that take turns and key blocks
// asked into L2 ahead each gained nothing.
//
// Roles (512 threads): warps 0-3 and 4-7 the two softmax warpgroups, warp 8 the
// items and a ring of K and V blocks, one thread of warp 9 the MMAs, warps 10
// and 11 a tile's Q each (the next item's as soon as the tile is free), warps
// 12-15 the outputs: O / l in bf16 while the tile's warpgroup is at the next
// item.  Registers: 512 threads of 128 at launch, split 184 to a softmax thread
// and 72 to another.
// Keys past a tile's last visible one are left out of both products in steps
// of 16; inside the step their p is 0, and the copy warp zeroes the V rows past
// the sequence's end, so what lies behind a sequence never enters a sum.
// Every barrier wait is bounded, with one answer for a warp that waits as a whole.
#include <algorithm>
#include <atomic>

#include "wq_internal.h"
#include "wq_prompt.cuh"

namespace wq {

namespace {

constexpr int kRows = 128;      // (token, head) rows per tile
constexpr int kKeys = 128;      // keys per block
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kQueryWarp = 10, kOutWarp = 12;
constexpr int kSoftmaxRegs = 184, kOtherRegs = 72;  // 256 threads each, of 128 at launch
constexpr int kPart = 64, kParts = kKeys / kPart;  // keys of P that are handed to the tensor core at a time
constexpr int kMisses = 4096;  // claims in a row that brought no item
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.0f;  // log2 of the growth of p that is let pass before m moves

// ONE: items of one tile.
template <int D, bool ONE>
struct Cfg {
    static constexpr int kCols = D / 64;               // 128-byte column blocks of a row
    static constexpr int kBlkBytes = kRows * 128;      // one column block of 128 rows
    static constexpr int kTileBytes = kCols * kBlkBytes;
    // columns of tensor memory: S of tile x at 128 x, O at 256 + D x, P over S, or (where O leaves room) behind O, so
    // that S can be overwritten as soon as it is in registers (one prompt of 8,000 tokens, one head of 128: 81.8 us, with
    // P over S 106.8)
    static constexpr bool kOwnP = D == 64 || ONE;
    static constexpr uint32_t kPCol = kOwnP ? 384 : 0, kPStride = kOwnP ? 64 : 128;
    static constexpr int kStages = D == 128 ? 4 : 8;   // K and V blocks in the ring
    static constexpr int kRing = 2 * kTileBytes;       // after the two Q tiles
    static constexpr int kOutOff = kRing + kStages * kTileBytes;  // 32 rows of 32 output values per output warp
    static constexpr int kScaleOff = kOutOff + 4 * 32 * 64;        // 1 / l of two items' rows, per tile
    static constexpr int kBarOff = kScaleOff + 4 * kRows * 4;
    static constexpr int kBytes = kBarOff + 640;
};

struct PromptArgs {
    const int32_t *starts;
    int64_t M, ldo;
    int B, H, r, tpt, tiles;  // tokens per tile, tiles per item
    float scale_log2;  // log2(e) / sqrt(D)
    uint16_t *o;
    int *status;
};

// One work item: the tiles at tokens tok0 and, before `end`, tok0 + tpt of the sequence at row0, KV head h.
struct Item {
    int64_t row0;
    int len, tok0, end, h, valid;
    // keys seen by some row of tile x, and its blocks (0: no such tile)
    __device__ __forceinline__ int last(int x, int tpt) const { return std::min(len, tok0 + (x + 1) * tpt); }
    __device__ __forceinline__ int blocks(int x, int tpt) const
    {
        return tok0 + x * tpt < end ? (last(x, tpt) + kKeys - 1) / kKeys : 0;
    }
    // block j holds the sequence's end within a step of 16 keys: its first row past the end, or 0
    __device__ __forceinline__ int tail(int j) const
    {
        const int rows = len - j * kKeys;
        return rows < kKeys && (rows & 15) ? rows : 0;
    }
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8], q_full[2], q_empty[2], s_full[2], p_full[2][kParts], pv_done[2], item_full[2],
        item_empty[2], landed[8], done, claim,
        l_full[2][2], o_free[2], s_free[2];
    __align__(16) uint8_t claimed[16];
    Item items[2];
    int abort, pad;
    uint32_t tmem;
};
static_assert(sizeof(Bars) <= 640, "the barrier area");

// The pairs of tiles of the packed batch: 32 sequences at a time, among those the pairs latest in their sequence (so
// with the most keys) first, which leaves the shortest work to the end.  A warp that asks for pairs in ascending order
// reads `starts` once.  Bounds outside [0, M] are
// clamped, a sequence that ends before it begins is empty.
struct Finder {
    int next = 0;             // first sequence of the next chunk
    int64_t before = 0;       // pairs before the chunk
    int64_t s = 0, e = 0;     // this lane's sequence
    int n = 0, all = 0;       // its pairs, and those of the chunk

    __device__ __forceinline__ bool find(const PromptArgs &p, int64_t t, Item &it)
    {
        const int lane = threadIdx.x & 31, span = p.tiles * p.tpt;
        if (t < before) *this = Finder();
        for (;;) {
            if (t < before + all) break;
            if (next >= p.B) return false;
            before += all;
            const int b = next + lane;
            next += 32;
            s = e = 0;
            if (b < p.B) {
                s = std::min<int64_t>(std::max<int64_t>(p.starts[b], 0), p.M);
                e = std::min<int64_t>(std::max<int64_t>(p.starts[b + 1], s), p.M);
            }
            // (no batch that fits memory comes near the bound; it keeps the sums of overlapping sequences in 32 bits)
            n = (int)std::min<int64_t>((e - s + span - 1) / span, 1 << 25);
            all = __reduce_add_sync(0xffffffffu, n);
        }
        // the largest place l in a sequence with more than u pairs at or behind it; u's rank among the sequences there
        const int u = (int)(t - before);
        int l = 0, none = __reduce_max_sync(0xffffffffu, n);
        while (none - l > 1) {
            const int mid = (l + none) / 2, pairs = __reduce_add_sync(0xffffffffu, max(0, n - mid));
            if (pairs > u) l = mid;
            else none = mid;
        }
        const int behind = __reduce_add_sync(0xffffffffu, max(0, n - l - 1));
        const int src = (int)__fns(__ballot_sync(0xffffffffu, n > l), 0, u - behind + 1);
        it.row0 = __shfl_sync(0xffffffffu, s, src);
        it.len = (int)__shfl_sync(0xffffffffu, e - s, src);
        it.tok0 = l * span;
        it.end = std::min(it.len, it.tok0 + span);
        return true;
    }
};

// 2^x, the hardware's approximation (denormal results flushed).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ f32x2 add2_pairs(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

template <int N>
__device__ __forceinline__ void registers_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Asks the hardware for a CTA of the grid that has not been launched, to do its items here (the answer arrives on `bar`).
__device__ __forceinline__ void claim_cta(uint8_t *answer, uint64_t *bar)
{
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(smem_u32(answer)), "r"(smem_u32(bar))
                 : "memory");
}

// The claimed CTA's blockIdx.x, or -1 when none was left.
__device__ __forceinline__ int claimed_cta(const uint8_t *answer)
{
    uint32_t x, got;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 r;\n\tld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %1, 1, 0, p;\n\tmov.u32 %0, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}"
                 : "=r"(x), "=r"(got)
                 : "r"(smem_u32(answer))
                 : "memory");
    return got ? (int)x : -1;
}

// Waits whatever `abort` says: for copies and MMAs that must be over before the CTA may end.
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity, int *status)
{
    const uint64_t since = global_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_ns() - since > kWaitLimitNs) { record_timeout(status); return; }
}

// For one thread, and for a whole warp (one answer for all its lanes).
struct Wait {
    int *status;
    volatile int *abort;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const
    {
        return mbar_wait(bar, parity, status, abort);
    }
};

struct WarpWait {
    int *status;
    volatile int *abort;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const
    {
        return warp_wait(bar, parity, status, abort);
    }
};

// Instruction descriptor: bf16 operands, f32 accumulator; PV reads V with its keys along K in rows of D (MN-major).
__device__ __forceinline__ uint32_t idesc_qk(int n) { return idesc_bf16_f32(kRows, n); }
__host__ __device__ constexpr uint32_t idesc_pv(int d) { return idesc_bf16_f32(kRows, d) | (1u << 16); }

template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap, const PromptArgs p)
{
    using C = Cfg<D, ONE>;
    constexpr uint32_t S = (uint32_t)C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Bars &b = *reinterpret_cast<Bars *>(smem + C::kBarOff);
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
    const WarpWait wait{p.status, &b.abort};

    if (tid == 0) {
        for (uint32_t i = 0; i < S; ++i) {
            mbar_init(&b.kv_full[i], 1);
            mbar_init(&b.kv_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.q_full[i], 1);
            mbar_init(&b.q_empty[i], 1);
            mbar_init(&b.s_full[i], 1);
            for (int c = 0; c < kParts; ++c) mbar_init(&b.p_full[i][c], 4);
            mbar_init(&b.pv_done[i], 1);
            mbar_init(&b.item_full[i], 1);
            mbar_init(&b.item_empty[i], 15);  // 8 softmax, 4 output and 2 Q warps, the MMA thread
            mbar_init(&b.s_free[i], 4);
            for (int c = 0; c < 2; ++c) mbar_init(&b.l_full[i][c], 4);
            mbar_init(&b.o_free[i], 4);
        }
        mbar_init(&b.done, 1);
        mbar_init(&b.claim, 1);
        for (uint32_t i = 0; i < S; ++i) mbar_init(&b.landed[i], 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (wid == kMmaWarp) tmem_alloc(&b.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what came before on the stream is complete from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (wid == kLoadWarp) {
        // ------------------------------ items and copies ------------------------------
        registers_dec<kOtherRegs>();
        Item it{};
        Finder finder;
        uint32_t slot = 0, phase = 0, loads = 0, nitem = 0;
        bool ok = true;
        uint32_t claims = 0;
        int cta = blockIdx.x, misses = 0;
        bool claiming = true;  // an answer is under way or unread
        if (lane == 0) claim_cta(b.claimed, &b.claim);
        bool found = finder.find(p, cta / p.H, it);
        for (;;) {
            // this CTA's item, then those of CTAs claimed from the grid (the claim for the next is under way meanwhile)
            while (!found && claiming) {
                if (!wait(&b.claim, claims & 1u)) { ok = false; break; }
                ++claims;
                const int next = claimed_cta(b.claimed);
                __syncwarp();
                // The grid has up to a pair per sequence too many: a long run of those ends the CTA before the waits of
                // its other warps run out.
                claiming = next >= 0 && ++misses < kMisses;
                if (next < 0) break;
                cta = next;
                if (lane == 0 && claiming) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the answer was read before the next is written
                    claim_cta(b.claimed, &b.claim);
                }
                found = finder.find(p, cta / p.H, it);
            }
            if (!ok) break;
            const uint32_t s = nitem & 1u;
            if (nitem >= 2 && !wait(&b.item_empty[s], ((nitem >> 1) - 1) & 1u)) { ok = false; break; }
            it.valid = found;
            misses = 0;
            it.h = cta % p.H;
            if (lane == 0) {
                b.items[s] = it;
                mbar_arrive(&b.item_full[s]);
            }
            __syncwarp();
            ++nitem;
            if (!found) break;
            found = false;
            const int n = std::max(it.blocks(0, p.tpt), it.blocks(1, p.tpt));
            auto load_kv = [&](const CUtensorMap *map, int j) {
                if (loads >= S && !wait(&b.kv_empty[slot], phase ^ 1u)) return false;
                uint8_t *dst = smem + C::kRing + slot * C::kTileBytes;
                // a V block that ends inside a step of 16 keys goes to warp 11 first
                uint64_t *bar = map == &vmap && it.tail(j) ? &b.landed[slot] : &b.kv_full[slot];
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, (uint32_t)C::kTileBytes);
                    for (int c = 0; c < C::kCols; ++c)
                        tma_load_3d(dst + c * C::kBlkBytes, map, bar, c * 64, it.h, (int)it.row0 + j * kKeys);
                }
                ++loads;
                if (++slot == S) { slot = 0; phase ^= 1u; }
                return true;
            };
            for (int j = 0; ok && j < n; ++j) ok = load_kv(&kmap, j) && load_kv(&vmap, j);
            if (!ok) break;
        }
        if (lane == 0) {
            // every issued copy (and answer) must land before the CTA may exit (bounded, ignoring abort)
            if (claiming) drain(&b.claim, claims & 1u, p.status);
            for (uint32_t j = loads > S ? loads - S : 0; j < loads; ++j) drain(&b.kv_full[j % S], (j / S) & 1u, p.status);
        }
    } else if (wid == kMmaWarp) {
        // ------------------------------ MMAs: one thread ------------------------------
        registers_dec<kOtherRegs>();
        if (elect_one()) {
            const Wait wait{p.status, &b.abort};
            uint32_t slot = 0, phase = 0, nitem = 0;
            struct Tile {
                uint32_t sn, pn, qn, on;  // S and P V issued, items begun by S and by P V
                uint32_t parts;           // bit c: the next parity of part c of P
            };
            struct Blocks {
                int last0, last1, nb0, nb1, n;  // per tile: keys and blocks; blocks of the item, 0 at the end
            };
            Tile t0{0, 0, 0, 0, 0}, t1 = t0;
            const uint32_t base = smem_u32(smem);
            bool ok = true;
            auto next_slot = [&]() {
                if (++slot == S) { slot = 0; phase ^= 1u; }
            };
            auto ring = [&](uint32_t s) { return base + C::kRing + s * C::kTileBytes; };
            auto next_item = [&](Blocks &it) {
                const uint32_t is = nitem & 1u;
                if (!wait(&b.item_full[is], (nitem >> 1) & 1u)) return false;
                const Item i = b.items[is];
                mbar_arrive(&b.item_empty[is]);
                ++nitem;
                it.last0 = i.last(0, p.tpt);
                it.last1 = i.last(1, p.tpt);
                it.nb0 = i.blocks(0, p.tpt);
                it.nb1 = i.blocks(1, p.tpt);
                it.n = i.valid ? std::max(it.nb0, it.nb1) : 0;
                return true;
            };
            // S of tile x for `keys` keys, their K at k.  The softmax has taken the S before; where P lies over S, the
            // product with V has read P as well.
            auto scores = [&](Tile &t, int x, bool first, bool final, int keys, uint32_t k) {
                if (first && !wait(&b.q_full[x], t.qn++ & 1u)) return false;
                if (t.sn > 0 && !(C::kOwnP ? wait(&b.s_free[x], (t.sn - 1) & 1u) : wait(&b.pv_done[x], (t.pn - 1) & 1u)))
                    return false;
                tc_fence_after();
                const uint32_t idesc = idesc_qk((min(kKeys, keys) + 15) & ~15);
                const uint32_t q = base + x * C::kTileBytes;
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    const uint32_t off = (uint32_t)(e / 4 * C::kBlkBytes + e % 4 * 32);
                    tc_mma_ss(tmem + 128u * x, smem_desc(q + off, 16, 1024, 2), smem_desc(k + off, 16, 1024, 2), idesc, e > 0);
                }
                tc_commit(&b.s_full[x]);
                if (final) tc_commit(&b.q_empty[x]);
                ++t.sn;
                return true;
            };
            // O += P V of tile x, part by part as P comes
            auto product = [&](Tile &t, int x, bool first, int keys, uint32_t v) {
                // the item before's output has been read
                if (first && t.on++ > 0 && !wait(&b.o_free[x], t.on & 1u)) return false;
#pragma unroll
                for (int c = 0; c < kParts; ++c) {
                    if (c * kPart < keys) {
                        if (!wait(&b.p_full[x][c], (t.parts >> c) & 1u)) return false;
                        t.parts ^= 1u << c;
                        tc_fence_after();
#pragma unroll
                        for (int e = c * (kPart / 16); e < (c + 1) * (kPart / 16); ++e)
                            if (e * 16 < keys)
                                tc_mma_ts(tmem + 256u + (uint32_t)D * x, tmem + C::kPCol + C::kPStride * x + 8u * e,
                                          smem_desc(v + 2048u * e, C::kBlkBytes, 1024, 2), idesc_pv(D), (!first || e > 0) ? 1u : 0u);
                    }
                }
                tc_commit(&b.pv_done[x]);
                ++t.pn;
                return true;
            };
            Blocks it{}, nx{};
            ok = next_item(it);
            if (ok && it.n > 0) {
                ok = wait(&b.kv_full[slot], phase) && scores(t0, 0, true, it.nb0 == 1, it.last0, ring(slot)) &&
                     (it.nb1 == 0 || scores(t1, 1, true, it.nb1 == 1, it.last1, ring(slot)));
                tc_commit(&b.kv_empty[slot]);
                next_slot();
            }
            // Per block: tile 0's product and its next S (of the next item after its last block), then tile 1's; the strict
            // order keeps the tiles half a period apart.  Where S does not wait for the product, both S come first.
            while (ok && it.n > 0) {
                for (int j = 0; ok && j < it.n; ++j) {
                    const uint32_t vs = slot;
                    ok = wait(&b.kv_full[vs], phase);
                    next_slot();
                    const bool end = j + 1 == it.n;
                    if (ok && end) ok = next_item(nx);
                    const int jn = end ? 0 : j + 1, first = end;  // the next S: block jn
                    const int nb0 = end ? nx.nb0 : it.nb0, nb1 = end ? nx.nb1 : it.nb1;
                    const int left0 = (end ? nx.last0 : it.last0) - jn * kKeys, left1 = (end ? nx.last1 : it.last1) - jn * kKeys;
                    const bool more = !end || nx.n > 0, s0 = more && jn < nb0, s1 = more && jn < nb1;
                    const bool o0 = j < it.nb0, o1 = j < it.nb1;
                    const uint32_t v = ring(vs), k = ring(slot);
                    if (C::kOwnP) {
                        ok = ok && (!more || wait(&b.kv_full[slot], phase));
                        if (ok && s0) ok = scores(t0, 0, first, jn + 1 == nb0, left0, k);
                        if (ok && s1) ok = scores(t1, 1, first, jn + 1 == nb1, left1, k);
                        if (more) tc_commit(&b.kv_empty[slot]);
                        if (ok && o0) ok = product(t0, 0, j == 0, it.last0 - j * kKeys, v);
                        if (ok && o1) ok = product(t1, 1, j == 0, it.last1 - j * kKeys, v);
                        tc_commit(&b.kv_empty[vs]);
                    } else {
                        if (ok && o0) ok = product(t0, 0, j == 0, it.last0 - j * kKeys, v);
                        ok = ok && (!more || wait(&b.kv_full[slot], phase));
                        if (ok && s0) ok = scores(t0, 0, first, jn + 1 == nb0, left0, k);
                        if (ok && o1) ok = product(t1, 1, j == 0, it.last1 - j * kKeys, v);
                        tc_commit(&b.kv_empty[vs]);
                        if (ok && s1) ok = scores(t1, 1, first, jn + 1 == nb1, left1, k);
                        if (more) tc_commit(&b.kv_empty[slot]);
                    }
                    if (more) next_slot();
                }
                it = nx;
            }
            tc_commit(&b.done);
            drain(&b.done, 0, p.status);  // every MMA must complete before tensor memory is released
        }
        __syncwarp();
    } else if (wid < 8) {
        // ------------------------------ softmax, one row per thread ------------------------------
        registers_inc<kSoftmaxRegs>();
        const int x = wid >> 2, row = tid & 127;
        const uint32_t lane_bits = (uint32_t)((wid & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_bits + 128u * x, p_addr = tmem + lane_bits + C::kPCol + C::kPStride * x, o_addr = tmem + lane_bits + 256u + (uint32_t)D * x;
        const int row_tok = row / p.r;
        uint32_t nitem = 0, blocks_done = 0, tiles_done = 0;
        bool ok = true;
        while (ok) {
            const uint32_t is = nitem & 1u;
            if (!wait(&b.item_full[is], (nitem >> 1) & 1u)) break;
            const Item it = b.items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.item_empty[is]);
            ++nitem;
            if (!it.valid) break;
            const int nb = it.blocks(x, p.tpt), last = it.last(x, p.tpt), tile_tok = it.tok0 + x * p.tpt;
            const int tok = tile_tok + row_tok;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < nb; ++j) {
                if (!wait(&b.s_full[x], blocks_done & 1u)) { ok = false; break; }
                tc_fence_after();
                const int u0 = j * kKeys, keys = min(kKeys, last - u0);
                // m follows the block's maximum `top` of the row once p would grow by more than 2^kSlack.  The vote only skips
                // the pass over O: which m a row carries is its own affair, or the rows around it (later tokens, the next
                // sequence's, what shared memory held) would decide how its p is rounded.
                auto move_max = [&](float top) {
                    const bool grow = (top - m) * p.scale_log2 > kSlack;
                    if (!__any_sync(0xffffffffu, grow)) return;
                    const float keep = grow ? ex2((m - top) * p.scale_log2) : 1.0f;
                    m = grow ? top : m;
                    l *= keep;
                    if (j == 0) return;
                    // the product of the block before has completed: S was issued after it, or it was waited for
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t w[16];
                        tmem_ld16(o_addr + (uint32_t)c, w);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * keep);
                        tmem_st16(o_addr + (uint32_t)c, w);
                    }
                };
                // P and its sum for 32 keys of the row
                f32x2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                auto exponentials = [&](const uint32_t v[32], int c) {
                    const float shift = -m * p.scale_log2;
                    const f32x2 sc{p.scale_log2, p.scale_log2}, sh{shift, shift};
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const f32x2 s2{__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])};
                        const f32x2 y = fma2_pairs(s2, sc, sh);
                        const f32x2 q{ex2(y.x), ex2(y.y)};
                        sum[e & 1] = add2_pairs(sum[e & 1], q);
                        w[e] = pack2_bf16(q.x, q.y);
                    }
                    tmem_st16(p_addr + 16u * c, w);
                };
                auto hand_over = [&](int part) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.p_full[x][part]);
                };
                // S is in registers: the next one may come; then P's columns and O, free once the product before is done
                auto taken = [&]() {
                    if (!C::kOwnP) return true;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.s_free[x]);
                    if (blocks_done > 0 && !wait(&b.pv_done[x], (blocks_done - 1) & 1u)) return false;
                    tc_fence_after();  // what follows touches O and P, which that product wrote and read
                    return true;
                };
                if (u0 + kKeys <= tile_tok + 1) {  // every row sees every key of the block
                    uint32_t v[kKeys / 32][32];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(s_addr + 32u * c, v[c]);
                    tmem_wait_ld();
                    if (!taken()) { ok = false; break; }
                    float tops[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            tops[(e / 2) & 3] = max3(tops[(e / 2) & 3], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                    move_max(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        exponentials(v[c], c);
                        if ((c + 1) * 32 % kPart == 0) hand_over((c + 1) * 32 / kPart - 1);
                    }
                } else {
                    // a last block: masked where a row does not see a key, P for the pieces of 32 keys that some row sees
                    uint32_t v[kKeys / 32][32];
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(s_addr + 32u * c, v[c]);
                    tmem_wait_ld();
                    if (!taken()) { ok = false; break; }
                    const int seen = min(keys, tok - u0 + 1);
                    float tops[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        if (u0 + 32 * c + 32 > tile_tok + 1) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[c][e] = 32 * c + e >= seen ? 0xff800000u : v[c][e];
                        }
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            tops[(e / 2) & 3] = max3(tops[(e / 2) & 3], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                    }
                    move_max(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])));
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        if (c * 32 < keys) {
                            exponentials(v[c], c);
                            if ((c + 1) * 32 % kPart == 0 || (c + 1) * 32 >= keys) hand_over(c * 32 / kPart);
                        }
                    }
                }
                const f32x2 both = add2_pairs(sum[0], sum[1]);
                l += both.x + both.y;
                ++blocks_done;
            }
            if (!ok) break;
            if (nb == 0) continue;
            const uint32_t buf = tiles_done++ & 1u;
            reinterpret_cast<float *>(smem + C::kScaleOff)[(2 * x + buf) * kRows + row] = 1.0f / l;
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.l_full[x][buf]);
        }
    } else if (wid >= kOutWarp) {
        // ------------------------------ output, both tiles in turn ------------------------------
        registers_dec<kOtherRegs>();
        const int row = tid & 127;
        const uint32_t lane_bits = (uint32_t)((wid & 3) * 32) << 16;
        const int row_tok = row / p.r, row_head = row - row_tok * p.r;
        uint8_t *out = smem + C::kOutOff + (wid & 3) * (32 * 64);
        const int piece = lane & 3;
        uint32_t nitem = 0, blocks[2] = {0, 0}, tiles[2] = {0, 0};
        bool ok = true;
        while (ok) {
            const uint32_t is = nitem & 1u;
            if (!wait(&b.item_full[is], (nitem >> 1) & 1u)) break;
            const Item it = b.items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.item_empty[is]);
            ++nitem;
            if (!it.valid) break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int nb = it.blocks(x, p.tpt), tok = it.tok0 + x * p.tpt + row_tok;
                if (nb == 0 || !ok) continue;
                blocks[x] += nb;
                const uint32_t buf = tiles[x] & 1u;
                ok = wait(&b.l_full[x][buf], (tiles[x] >> 1) & 1u) && wait(&b.pv_done[x], (blocks[x] - 1) & 1u);
                if (!ok) continue;
                ++tiles[x];
                tc_fence_after();
                const uint32_t o_addr = tmem + lane_bits + 256u + (uint32_t)D * x;
                const float inv = reinterpret_cast<const float *>(smem + C::kScaleOff)[(2 * x + buf) * kRows + row];
                const bool live = row < p.tpt * p.r && tok < it.len;
                // 32 output values of a row at a time, through shared memory (16-byte pieces at piece ^ (row / 2) % 4
                // of the row's 64 bytes: no bank conflicts either way), so that a store instruction writes 8 rows' 64
                // adjacent bytes and not 32 rows' 16
                const uint64_t dst = reinterpret_cast<uint64_t>(p.o + (it.row0 + tok) * p.ldo + (it.h * p.r + row_head) * D);
                const uint32_t alive = __ballot_sync(0xffffffffu, live);
                uint64_t to[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) to[i] = __shfl_sync(0xffffffffu, dst, 8 * i + (lane >> 2)) + 16u * piece;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t w[32];
                    tmem_ld32(o_addr + (uint32_t)c, w);
                    tmem_wait_ld();
                    if (c + 32 == D) {  // the tile's next product may write
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b.o_free[x]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t g[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            g[i] = pack2_bf16(__uint_as_float(w[8 * e + 2 * i]) * inv, __uint_as_float(w[8 * e + 2 * i + 1]) * inv);
                        *reinterpret_cast<uint4 *>(out + lane * 64 + (e ^ ((lane >> 1) & 3)) * 16) = make_uint4(g[0], g[1], g[2], g[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 8 * i + (lane >> 2);
                        const uint4 g = *reinterpret_cast<const uint4 *>(out + r * 64 + (piece ^ ((r >> 1) & 3)) * 16);
                        if ((alive >> r) & 1u) *reinterpret_cast<uint4 *>(to[i] + 2u * c) = g;
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ------------------------------ Q of tile x, apart from K and V, which must not wait for a tile; V's tails ------------------------------
        registers_dec<kOtherRegs>();
        const int x = wid - kQueryWarp;
        uint32_t nitem = 0, qn = 0, slot = 0, landed = 0;  // slot: the item's first K; landed: bit s the next parity of slot s
        for (;;) {
            const uint32_t is = nitem & 1u;
            if (!wait(&b.item_full[is], (nitem >> 1) & 1u)) break;
            const Item it = b.items[is];
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.item_empty[is]);
            ++nitem;
            if (!it.valid) break;
            if (it.blocks(x, p.tpt) > 0) {
                if (qn > 0 && !wait(&b.q_empty[x], (qn - 1) & 1u)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&b.q_full[x], (uint32_t)(C::kCols * p.r * p.tpt * 128));
                    for (int c = 0; c < C::kCols; ++c)
                        tma_load_3d(smem + x * C::kTileBytes + c * C::kBlkBytes, &qmap, &b.q_full[x], c * 64, it.h * p.r,
                                    (int)it.row0 + it.tok0 + x * p.tpt);
                }
                __syncwarp();
                ++qn;
            }
            if (x == 1) {
                // V rows past the sequence's end within a step of 16 keys become 0 (the products leave later steps out)
                const int n = std::max(it.blocks(0, p.tpt), it.blocks(1, p.tpt)), rows = it.tail(n - 1);
                const uint32_t vs = (slot + 2 * n - 1) % S;
                slot = (slot + 2 * n) % S;
                if (rows > 0) {
                    if (!wait(&b.landed[vs], (landed >> vs) & 1u)) break;
                    landed ^= 1u << vs;
                    uint8_t *v = smem + C::kRing + vs * C::kTileBytes;
                    const int chunks = (16 - (rows & 15)) * 8;  // of 16 bytes, per column block
                    for (int i = lane; i < chunks * C::kCols; i += 32)
                        *reinterpret_cast<uint4 *>(v + i / chunks * C::kBlkBytes + rows * 128 + i % chunks * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.kv_full[vs]);
                }
            }
        }
        if (lane == 0 && qn > 0) drain(&b.q_full[x], (qn - 1) & 1u, p.status);
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (wid == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// SMs of the current device, 0 on failure; the kernels' shared-memory limits are raised on their first use there.
int sms_of_device()
{
    static std::atomic<int> sms_of[128] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return 0;
    int sms = sms_of[dev].load(std::memory_order_acquire);
    if (sms == 0) {
        const cudaFuncAttribute limit = cudaFuncAttributeMaxDynamicSharedMemorySize;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(prompt_attn_kernel<64, false>, limit, Cfg<64, false>::kBytes + 1024) != cudaSuccess ||
            cudaFuncSetAttribute(prompt_attn_kernel<64, true>, limit, Cfg<64, true>::kBytes + 1024) != cudaSuccess ||
            cudaFuncSetAttribute(prompt_attn_kernel<128, false>, limit, Cfg<128, false>::kBytes + 1024) != cudaSuccess ||
            cudaFuncSetAttribute(prompt_attn_kernel<128, true>, limit, Cfg<128, true>::kBytes + 1024) != cudaSuccess)
            return 0;
        sms_of[dev].store(sms, std::memory_order_release);
    }
    return sms;
}

// Items of at most `tiles` tiles: at most ceil(len / span) of a sequence and KV head.
int64_t items(int64_t M, int64_t B, int64_t tpt, int64_t H, int tiles) { return (M / (tiles * tpt) + B) * H; }

template <int D>
int run(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv, int64_t Hq, PromptArgs a,
        cudaStream_t st)
{
    CUtensorMap qm, km, vm;
    const auto encode = [&](CUtensorMap *map, const uint16_t *base, int64_t heads, int64_t ld, int box_heads, int box_tokens) {
        return encode_tmap_3d(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, D, (uint64_t)heads, (uint64_t)a.M, D * 2,
                              (uint64_t)ld * 2, 64, (uint32_t)box_heads, (uint32_t)box_tokens, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!encode(&qm, q, Hq, ldq, a.r, a.tpt) || !encode(&km, k, a.H, ldk, 1, kKeys) || !encode(&vm, v, a.H, ldv, 1, kKeys))
        return -1;
    const int sms = sms_of_device();
    if (sms == 0) return -2;
    // Two tiles share a CTA's K and V and fill each other's waits; one to a CTA while that leaves SMs over (2,000 tokens, 4
    // heads of 64: 23.2 us with one, 30.8 with two; 1,000 tokens, 16 / 2 heads of 128: 15.7 and 19.8)
    a.tiles = (a.M / a.tpt + a.B / 2) * a.H <= sms ? 1 : 2;
    const unsigned grid = (unsigned)items(a.M, a.B, a.tpt, a.H, a.tiles);
    if (a.tiles == 1) launch_behind(prompt_attn_kernel<D, true>, grid, kThreads, Cfg<D, true>::kBytes + 1024, st, qm, km, vm, a);
    else launch_behind(prompt_attn_kernel<D, false>, grid, kThreads, Cfg<D, false>::kBytes + 1024, st, qm, km, vm, a);
    return 0;
}

}  // namespace

int64_t prompt_attention_items(int64_t M, int64_t B, int64_t Hq, int64_t H)
{
    return items(M, B, kRows / (Hq / H), H, 1);
}

int launch_prompt_attention(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v,
                            int64_t ldv, const int32_t *starts, int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D,
                            uint16_t *o, int64_t ldo, int *status, cudaStream_t st)
{
    const int r = (int)(Hq / H);
    const PromptArgs a{starts, M, ldo, (int)B, (int)H, r, kRows / r, 2, 1.4426950408889634f / sqrtf((float)D), o, status};
    return D == 128 ? run<128>(q, ldq, k, ldk, v, ldv, Hq, a, st) : run<64>(q, ldq, k, ldk, v, ldv, Hq, a, st);
}

}  // namespace wq
