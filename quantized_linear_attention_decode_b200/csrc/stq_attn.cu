// stq_attn.cu -- causal softmax attention over packed prompts with grouped heads (sm_100a).
//
//   y_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j <= i + (Lk - Lq)
//
// of the query's sequence (its queries are its last Lq positions).  Bound by the
// tensor cores, 4 x 128 operations a visible pair and head, and as much by the
// exponentials: a 128 x 128 tile is 1024 cycles of either.
//
// A CTA takes 256 query rows of one key head as two tiles of 128 and walks over the
// keys in tiles of 128.  A row is a (token, query head) pair: `pack` query heads of
// the key head, a power of two, stand side by side, so that one key tile serves all
// of them and a short prompt fills its tiles.  Tensor memory holds, for each query
// tile, S = Q K^T (128 columns; its first 64 become P in 16 bits, the other operand of
// O += P V straight from there) and O (128 columns): all 512 columns.  Warps 0-3 and
// 4-7 do the softmax of one tile each, a thread a row: no thread needs another for
// its maximum and sum.  Warp 8 loads (TMA, 128-byte swizzle, two stages each of K and
// V), one lane of warp 9 issues the products: while one tile's warps take
// exponentials, the tensor core works for the other.
//
// Items (256 rows of one key head) come from the grid: a CTA that has issued its
// item's last load asks for a block that has not begun and runs it in that block's place,
// so that the next loads and scores stand behind this item's last weights and its output.
// Blocks are ordered by tokens from a sequence's end, then heads: the longest first.
// A key tile of which 64 keys are seen at most is half a tile for all three.
// When this was chosen, 24 prompts to 2000 tokens took 319 us with a CTA an item, 283 with the
// heads outermost (8192 tokens 534), 274 so (520); 582 for the 8192 tokens where a CTA asked as
// soon as it began an item, and kept the next one waiting.
//
// The running maximum that P is taken against moves only when a score lies more than
// 2^8 above it (P then stays below 2^8, within fp16's range), so O is rescaled in
// tensor memory a few times a row and not in every tile.  P is rounded to the type of
// v (2^-9 of a weight in bf16, as the output itself); all else is fp32.  In fp16 P and
// its sum are lifted by 2^7, as far as that range allows: weights down to 2^-21 of the
// largest keep their bits, and what is lost of smaller ones is 2^-32 of it.
//
// A tile's products take 1090 cycles (S reads both operands from shared memory, 72
// cycles a step of 16 against 64 of arithmetic), and the next scores wait 300 more for
// the product that still reads P in their place; a softmax takes 1460 and is hidden
// behind the other tile.  So taking a part of the exponentials on the fp32 pipe instead
// (a polynomial for 1, 2 or 3 of 8) cost 1, 3 and 7 %, and two warps that issue one
// tile's products each, interleaved in the tensor core, 4 %.
// 32 query and 8 key heads, bf16: 8192 tokens 536 us, 1025 TFLOP/s; 24 prompts to 2000
// tokens 278 us, 730 TFLOP/s of visible pairs.
#include <algorithm>
#include <cmath>

#include "stq_host.h"
#include "stq_map.h"
#include "stq_tc.h"

namespace stq {
namespace {

constexpr int kRows = 128;               // of a query tile, and keys of a key tile
constexpr int kTileBytes = kRows * kD * 2;
constexpr int kHalfTile = kTileBytes / 2;  // 64 of the 128 dims: rows of 128 bytes
constexpr int kStages = 2;
constexpr int kThreads = 384;  // three warpgroups; warp 10 finds the items, warp 11 only hands its registers over
// registers a thread: 168 at launch, then 208 in the softmax warpgroups and 88 in the third (2 * 208 + 88 = 3 * 168)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;

template <bool BF16>
constexpr float kLift = BF16 ? 0.0f : 7.0f;  // log2 of what P is multiplied by

struct PromptAttn {
    const int32_t *q_start, *k_start;
    int n, heads, group, pack, total_q, total_k;
    float scale_log2;  // |scale| log2(e)
    bool negative;     // scale < 0
    void *y;
    int32_t *err;
    Waits waits;
};

struct __align__(1024) AttnSmem {
    uint8_t q[2][kTileBytes];
    uint8_t k[kStages][kTileBytes], v[kStages][kTileBytes];
    unsigned long long q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    unsigned long long s_full[2], p_full[2][2], o_full[2];  // p_full: of either half of the keys
    unsigned long long item_full[2], item_empty[2], wanted, asked, drained;
    uint4 answer;
    uint32_t tmem;
    // sequence's first query row (-1: no more items), its queries, first key row, keys, the item's first token, block of heads
    int item[2][8];
};

// Queries and keys of sequence i; false where a range is none.
__device__ __forceinline__ bool sequence(const PromptAttn &a, int i, int *lq, int *lk)
{
    const int q0 = a.q_start[i], q1 = a.q_start[i + 1], k0 = a.k_start[i], k1 = a.k_start[i + 1];
    *lq = q1 - q0;
    *lk = k1 - k0;
    return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k;
}

// Sequence and tokens of a tile: tiles of all sequences in order, within a sequence from its end, where
// a tile sees most keys.  One warp; false when there is no such tile.
// `from` and `base`: where the last search began to find its tile, and the tiles before there; blocks mostly come in order.
__device__ __forceinline__ bool find_item(const PromptAttn &a, int tile, int *from, long long *base, int *seq, int *token)
{
    const int lane = threadIdx.x & 31, tokens = 2 * kRows / a.pack;
    if (tile < *base) *from = *base = 0;
    for (; *from < a.n; *from += 32) {
        int lq = 0, lk, mine = 0;
        if (*from + lane < a.n && sequence(a, *from + lane, &lq, &lk)) mine = (lq + tokens - 1) / tokens;
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, *base + upto > tile);
        if (past) {
            const int who = __ffs(past) - 1;
            const long long end = *base + __shfl_sync(0xffffffffu, upto, who);
            *seq = *from + who;
            *token = static_cast<int>(end - 1 - tile) * tokens;
            return true;
        }
        *base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float f_of(uint32_t u) { return __uint_as_float(u); }

// Two values in the 16-bit type of v.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (BF16) {
        const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&w);
    }
    const __half2 w = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&w);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map, const PromptAttn a)
{
    extern __shared__ uint8_t raw_smem[];
    AttnSmem &sm = *reinterpret_cast<AttnSmem *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (warp == 8 && lane == 0) {
        const auto init = [](unsigned long long &b, uint32_t count) { barrier_init(smem_addr(&b), count); };
        init(sm.q_full, 1);
        init(sm.q_empty, 1);
        for (int s = 0; s < kStages; ++s) {
            init(sm.k_full[s], 1);
            init(sm.k_empty[s], 1);
            init(sm.v_full[s], 1);
            init(sm.v_empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            init(sm.s_full[i], 1);
            init(sm.p_full[i][0], kRows);
            init(sm.p_full[i][1], kRows);
            init(sm.o_full[i], 1);
            init(sm.item_full[i], 1);
            init(sm.item_empty[i], 2 + 8);
        }
        init(sm.wanted, 1);
        init(sm.asked, 1);
        init(sm.drained, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(smem_addr(&sm.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    const int per_tile = kRows / a.pack;  // tokens of a query tile
    bool ok = true;

    const auto wait = [&](unsigned long long &b, uint32_t parity) { return barrier_wait(smem_addr(&b), parity, a.waits.wait_ns); };
    // Item n of this CTA, a value a lane; false: no more.  The whole warp calls these.
    int entry = 0;
    const auto take = [&](int n) {
        ok = __all_sync(0xffffffffu, wait(sm.item_full[n & 1], n >> 1 & 1));
        if (ok) entry = sm.item[n & 1][lane & 7];
        return ok && __shfl_sync(0xffffffffu, entry, 0) >= 0;
    };
    const auto taken = [&](int n) {
        __syncwarp();
        if (lane == 0) barrier_arrive(smem_addr(&sm.item_empty[n & 1]));
    };
    const auto value = [&](int i) { return __shfl_sync(0xffffffffu, entry, i); };
    // keys that query tile i takes: up to what its last token sees
    const auto keys_of = [&](int i) {
        const int lq = value(1), lk = value(3), first = value(4) + i * per_tile, last = min(first + per_tile, lq) - 1;
        return first < lq ? max(0, min(lk, last + lk - lq + 1)) : 0;
    };
    const auto tiles_of = [](int keys) { return (keys + kRows - 1) / kRows; };
    // whether the key tile at j of `keys` ends in its first half
    const auto is_short = [](int keys, int j) { return keys - j * kRows <= kRows / 2; };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 10) {
            // ------------------------------------------------ the items: this block's, then others that have not begun
            const uint32_t blocks = a.heads / a.pack;
            uint32_t x = blockIdx.x;
            int from = 0;
            long long base = 0;
            for (int n = 0, asked = 0; ok;) {
                if (x == 0 && a.err != nullptr)
                    for (int i = lane; i < a.n; i += 32) {
                        int lq, lk;
                        if (!sequence(a, i, &lq, &lk)) *a.err = STQ_ERR_INDEX;
                    }
                int seq = 0, token = 0;
                if (find_item(a, static_cast<int>(x / blocks), &from, &base, &seq, &token)) {
                    if (lane == 0) {
                        int *item = sm.item[n & 1];
                        item[0] = a.q_start[seq];
                        item[1] = a.q_start[seq + 1] - a.q_start[seq];
                        item[2] = a.k_start[seq];
                        item[3] = a.k_start[seq + 1] - a.k_start[seq];
                        item[4] = token;
                        item[5] = static_cast<int>(x % blocks);
                        barrier_arrive(smem_addr(&sm.item_full[n & 1]));
                    }
                    __syncwarp();
                    ++n;
                    // not before this one's loads are under way, so that no CTA keeps an item waiting that another could run
                    ok = wait(sm.wanted, (n - 1) & 1) &&
                         (n < 2 || wait(sm.item_empty[n & 1], (n >> 1 & 1) ^ 1));
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                }
                if (lane == 0) {
                    barrier_expect(smem_addr(&sm.asked), 16);
                    next_block(smem_addr(&sm.answer), smem_addr(&sm.asked));
                }
                __syncwarp();
                ok = __all_sync(0xffffffffu, wait(sm.asked, asked & 1));
                if (!ok) break;
                ++asked;
                const bool more = next_block_is(smem_addr(&sm.answer), &x);
                fence_async_smem();  // the next answer is written over this one
                __syncwarp();
                if (!more) {
                    if (lane == 0) {
                        sm.item[n & 1][0] = -1;
                        barrier_arrive(smem_addr(&sm.item_full[n & 1]));
                    }
                    break;
                }
            }
        }
        if (warp == 8) {
            // ------------------------------------------------ loads
            int queries = 0, tile = 0, values = 0;  // loads of queries, key tiles and their values so far
            for (int n = 0; take(n); ++n) {
                const int tiles[2] = {tiles_of(keys_of(0)), tiles_of(keys_of(1))}, all = max(tiles[0], tiles[1]);
                const int q_row = value(0) + value(4), k_row = value(2), block = value(5), kv_head = block / (a.group / a.pack);
                if (lane == 0 && all > 0) {
                    const uint32_t qf = smem_addr(&sm.q_full);
                    ok = queries == 0 || wait(sm.q_empty, (queries & 1) ^ 1);
                    if (ok) {
                        barrier_expect(qf, (tiles[0] > 0 ? kTileBytes : 0) + (tiles[1] > 0 ? kTileBytes : 0));
                        for (int i = 0; i < 2; ++i)
                            for (int half = 0; half < 2 && tiles[i] > 0; ++half)
                                tma_load3(smem_addr(sm.q[i]) + half * kHalfTile, &q_map, qf, 64 * half, block * a.pack, q_row + i * per_tile);
                        ++queries;
                    }
                    for (int j = 0; j < all && ok; ++j) {
                        const int s = tile % kStages;
                        const uint32_t parity = (tile / kStages & 1) ^ 1;
                        const uint32_t kf = smem_addr(&sm.k_full[s]), vf = smem_addr(&sm.v_full[s]);
                        ok = tile < kStages || wait(sm.k_empty[s], parity);
                        if (!ok) break;
                        barrier_expect(kf, kTileBytes + (tile == 0 && blockIdx.x == 0 ? a.waits.stall_tx : 0));
                        for (int half = 0; half < 2; ++half)
                            tma_load3(smem_addr(sm.k[s]) + half * kHalfTile, &k_map, kf, 64 * half, kv_head, k_row + j * kRows);
                        ++tile;
                        ok = values < kStages || wait(sm.v_empty[s], parity);
                        if (!ok) break;
                        barrier_expect(vf, kTileBytes);
                        for (int half = 0; half < 2; ++half)
                            tma_load3(smem_addr(sm.v[s]) + half * kHalfTile, &v_map, vf, 64 * half, kv_head, k_row + j * kRows);
                        ++values;
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) barrier_arrive(smem_addr(&sm.wanted));
                taken(n);
            }
            if (lane == 0) {  // the loads land before the memory is given back, whatever became of those who wanted them
                if (queries > 0) wait(sm.q_full, (queries - 1) & 1);
                for (int j = max(0, tile - kStages); j < tile; ++j) wait(sm.k_full[j % kStages], j / kStages & 1);
                for (int j = max(0, values - kStages); j < values; ++j) wait(sm.v_full[j % kStages], j / kStages & 1);
            }
            __syncwarp();
        }
        if (warp == 9) {
            // ------------------------------------------------ products
            constexpr uint32_t type = BF16 ? 1 : 0;
            const uint32_t negate = a.negative ? 1u << 13 : 0u;
            const uint32_t qk = tc_idesc(type, kRows, kRows, false, false) | negate, qk_short = tc_idesc(type, kRows, kRows / 2, false, false) | negate;
            constexpr uint32_t pv = tc_idesc(type, kRows, kD, true);
            int queries = 0, tile = 0, done[2] = {0, 0};  // key tiles so far: of K and V, and of each query tile
            int keys[2] = {0, 0};
            // elect.sync wants the whole warp, so lanes leave only by a verdict that all share: one for each tile of keys, behind its
            // products (a vote for every wait, or products under a condition that lanes could differ in, cost 4 to 9 %).  After a
            // wait that gave up, products go on until then, of whatever is there; no stage is handed back to the loads.
            const auto scores = [&](int i, int j) {  // S_i = Q_i K_j^T
                if (elect_one()) {
                    uint32_t qa = smem_addr(sm.q[i]), ka = smem_addr(sm.k[(tile + j) % kStages]);
                    const uint32_t desc = is_short(keys[i], j) ? qk_short : qk;
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t off = (s >> 2) * kHalfTile + (s & 3) * 32;
                        tc_mma_ss(tmem + 128 * i, tc_desc(qa + off, 16, 1024), tc_desc(ka + off, 16, 1024), desc, s > 0);
                    }
                    tc_commit(smem_addr(&sm.s_full[i]));
                }
                __syncwarp();
            };
            // S_i may be written over: the product that reads P in its place is done
            const auto free_scores = [&](int i) { return done[i] == 0 || wait(sm.o_full[i], (done[i] - 1) & 1); };
            for (int n = 0; take(n); ++n) {
                taken(n);
                keys[0] = keys_of(0);
                keys[1] = keys_of(1);
                const int tiles[2] = {tiles_of(keys[0]), tiles_of(keys[1])}, all = max(tiles[0], tiles[1]), lk = value(3);
                if (all == 0) continue;
                ok = wait(sm.q_full, queries++ & 1) && wait(sm.k_full[tile % kStages], tile / kStages & 1);
                for (int i = 0; i < 2; ++i) {
                    if (tiles[i] == 0) continue;
                    ok = ok && free_scores(i);
                    tc_fence_after();
                    scores(i, 0);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (elect_one()) tc_commit(smem_addr(&sm.k_empty[tile % kStages]));
                __syncwarp();
                for (int j = 0; j < all; ++j) {
                    const int s = (tile + j) % kStages, next = tile + j + 1;
                    ok = ok && wait(sm.v_full[s], (tile + j) / kStages & 1) &&
                         (j + 1 == all || wait(sm.k_full[next % kStages], next / kStages & 1));
                    if (j + 1 == all) {  // no more scores of these queries
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (elect_one()) tc_commit(smem_addr(&sm.q_empty));
                        __syncwarp();
                    }
                    const int valid = lk - j * kRows;
                    if (valid < kRows) {
                        // rows behind the sequence's last key are another sequence's or nobody's: their weights are zero,
                        // but zero times an infinity is not
                        for (int e = lane; e < (kRows - valid) * 8; e += 32)
                            for (int half = 0; half < 2; ++half)
                                *reinterpret_cast<uint4 *>(sm.v[s] + half * kHalfTile + valid * 128 + e * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                    for (int i = 0; i < 2; ++i) {
                        if (j >= tiles[i]) continue;
                        const bool first_half = is_short(keys[i], j);
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && wait(sm.p_full[i][half], done[i] & 1);
                            tc_fence_after();
                            if (elect_one()) {
                                uint32_t va = smem_addr(sm.v[s]);
                                if (half == 0 || !first_half) {
#pragma unroll
                                    for (int t = 4 * half; t < 4 * half + 4; ++t)
                                        tc_mma_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * t, tc_desc(va + t * 2048, kHalfTile, 1024), pv, j > 0 || t > 0);
                                }
                                if (half == 1) tc_commit(smem_addr(&sm.o_full[i]));
                            }
                            __syncwarp();
                        }
                        ++done[i];
                        if (j + 1 < tiles[i]) {  // the next scores go where P is
                            ok = ok && free_scores(i);
                            tc_fence_after();
                            scores(i, j + 1);
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (elect_one()) {
                        tc_commit(smem_addr(&sm.v_empty[s]));
                        if (j + 1 < all) tc_commit(smem_addr(&sm.k_empty[next % kStages]));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                tile += all;
            }
            if (!ok && elect_one()) {  // products in flight end (bounded) before the memory is given back
                tc_commit(smem_addr(&sm.drained));
                wait(sm.drained, 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int i = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + 128 * i + lanes, to = tmem + 256 + 128 * i + lanes;
        const float c = a.scale_log2;
        int done = 0;  // key tiles so far
        for (int n = 0; take(n); ++n) {
            const int keys = keys_of(i), tiles = tiles_of(keys);
            const int sees = min(value(3), value(4) + i * per_tile + row / a.pack + value(3) - value(1) + 1);  // keys that this row sees (none: <= 0)
            const int least = min(value(3), value(4) + i * per_tile + value(3) - value(1) + 1);  // that the tile's first row sees
            float top = -INFINITY, sum = 0.0f;  // in units of log 2: P = exp2(c s - top + kLift)
            for (int j = 0; j < tiles && ok; ++j, ++done) {
                ok = __all_sync(0xffffffffu, wait(sm.s_full[i], done & 1));
                if (!ok) break;
                tc_fence_after();
                const bool first_half = is_short(keys, j);
                uint32_t x[4][32];
                tmem_load32(ts, x[0]);
                tmem_load32(ts + 32, x[1]);
                if (!first_half) {
                    tmem_load32(ts + 64, x[2]);
                    tmem_load32(ts + 96, x[3]);
                }
                tmem_wait_load();
                if ((j + 1) * kRows > least) {  // some row of the tile does not see all of these keys
                    const int limit = sees - j * kRows;
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * b + e >= limit) x[b][e] = 0xff800000u;
                }
                float ms[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    ms[b] = fmaxf(f_of(x[b][0]), f_of(x[b][1]));
#pragma unroll
                    for (int e = 2; e < 32; e += 2) ms[b] = max3(ms[b], f_of(x[b][e]), f_of(x[b][e + 1]));
                }
                const float m = max3(fmaxf(ms[0], ms[1]), ms[2], ms[3]) * c;
                const bool moves = m > top + 8.0f;
                if (__any_sync(0xffffffffu, moves)) {
                    const float now = moves ? m : top;
                    const float f = top == -INFINITY ? 0.0f : exp2_approx(top - now);
                    top = now;
                    sum *= f;
                    if (j > 0) {
#pragma unroll 1  // (unrolled, it spills registers)
                        for (int b = 0; b < 4; ++b) {
                            uint32_t o[32];
                            tmem_load32(to + 32 * b, o);
                            tmem_wait_load();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(f_of(o[e]) * f);
                            tmem_store32(to + 32 * b, o);
                        }
                    }
                }
                const float off = top == -INFINITY ? 0.0f : kLift<BF16> - top;
                float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half == 0 || !first_half) {
                        uint32_t w[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const uint32_t *s = &x[2 * half + (e >> 4)][2 * (e & 15)];
                            float2 z = __ffma2_rn(make_float2(f_of(s[0]), f_of(s[1])), make_float2(c, c), make_float2(off, off));
                            z = make_float2(exp2_approx(z.x), exp2_approx(z.y));
                            part[e & 1] = __fadd2_rn(part[e & 1], z);
                            w[e] = pack2<BF16>(z.x, z.y);
                        }
                        tmem_store32(ts + 32 * half, w);
                        tmem_wait_store();
                        tc_fence_before();
                    }
                    barrier_arrive(smem_addr(&sm.p_full[i][half]));
                }
                sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
            }
            if (ok && tiles > 0) ok = wait(sm.o_full[i], (done - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float f = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that sees no key is zero
            const int token = value(4) + i * per_tile + row / a.pack, lq = value(1);
            uint16_t *y = static_cast<uint16_t *>(a.y) + (static_cast<int64_t>(value(0) + token) * a.heads + value(5) * a.pack + row % a.pack) * kD;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                uint32_t o[32];
                if (tiles > 0) {
                    tmem_load32(to + 32 * b, o);
                    tmem_wait_load();
                }
                if (token < lq) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            w[d] = f == 0.0f ? 0u : pack2<BF16>(f_of(o[8 * e + 2 * d]) * f, f_of(o[8 * e + 2 * d + 1]) * f);
                        *reinterpret_cast<uint4 *>(y + 32 * b + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();  // the next products go over what was read here
            taken(n);
        }
    }
    if (!ok && a.err != nullptr) *a.err = STQ_ERR_TIMEOUT;
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

stq_status check_rows(const stq_rows *r, const char *name, int32_t dtype, int32_t heads, int32_t tokens)
{
    if (r == nullptr) return fail_status(STQ_ERR_ARG, "%s is NULL", name);
    if (tokens > 0 && r->data == nullptr) return fail_status(STQ_ERR_ARG, "%s.data is NULL", name);
    if (!rows_aligned(r, dtype)) return fail_status(STQ_ERR_ARG, "%s: rows must start on 16-byte boundaries", name);
    if (!rows_mappable(*r, heads, tokens))
        return fail_status(STQ_ERR_UNSUPPORTED, "%s: strides must be positive (and below 2^38)", name);
    return STQ_OK;
}

}  // namespace
}  // namespace stq

using stq::fail_status;

extern "C" stq_status stq_attn_prompt(const int32_t *q_start, const int32_t *k_start, int32_t n, int32_t num_heads,
                                      int32_t num_kv_heads, int32_t total_q, int32_t total_k, int32_t dtype,
                                      const stq_rows *q, const stq_rows *k, const stq_rows *v, float scale, void *y,
                                      int32_t *err, void *stream)
{
    if (n < 0 || total_q < 0 || total_k < 0) return fail_status(STQ_ERR_ARG, "n = %d, total_q = %d, total_k = %d", n, total_q, total_k);
    if (num_kv_heads < 1 || num_heads < 1 || num_heads % num_kv_heads != 0)
        return fail_status(STQ_ERR_ARG, "num_heads=%d is no multiple of num_kv_heads=%d", num_heads, num_kv_heads);
    if (stq::dtype_bytes(dtype) == 0) return fail_status(STQ_ERR_ARG, "dtype %d", dtype);
    if (dtype == STQ_F32) return fail_status(STQ_ERR_UNSUPPORTED, "prompt attention takes 16-bit types");
    if (!std::isfinite(scale)) return fail_status(STQ_ERR_ARG, "scale is not finite");
    stq_status st = stq::check_rows(q, "q", dtype, num_heads, total_q);
    if (st == STQ_OK) st = stq::check_rows(k, "k", dtype, num_kv_heads, total_k);
    if (st == STQ_OK) st = stq::check_rows(v, "v", dtype, num_kv_heads, total_k);
    if (st != STQ_OK) return st;
    if (n > 0 && (q_start == nullptr || k_start == nullptr)) return fail_status(STQ_ERR_ARG, "q_start or k_start is NULL");
    if (n > 0 && total_q > 0 && y == nullptr) return fail_status(STQ_ERR_ARG, "y is NULL");
    if (reinterpret_cast<uintptr_t>(y) % 16 != 0) return fail_status(STQ_ERR_ARG, "y must be 16-byte aligned");
    const int group = num_heads / num_kv_heads;
    int pack = 1;  // the largest power of two that divides the group, up to a tile's rows
    while (pack < stq::kRows && group % (2 * pack) == 0) pack *= 2;
    const long long tiles = (static_cast<long long>(total_q) * pack + 2 * stq::kRows - 1) / (2 * stq::kRows) + n;
    if (tiles * (num_heads / pack) > 0x7FFFFFFFll) return fail_status(STQ_ERR_ARG, "too many query tiles or heads");
    if (n == 0 || total_q == 0) return STQ_OK;
    if (stq::fault("launch")) return fail_status(STQ_ERR_CUDA, "injected launch failure (STQ_FAULT=launch)");
    cudaPointerAttributes where;
    cudaError_t e = cudaPointerGetAttributes(&where, y);
    if (e != cudaSuccess) return stq::cuda_fail(e, "device of y");
    if (where.type != cudaMemoryTypeDevice && where.type != cudaMemoryTypeManaged) return fail_status(STQ_ERR_ARG, "y is no device memory");
    stq::DeviceGuard g(where.device);
    stq::NvtxRange nvtx("stq_attn_prompt");
    if (!g.ok) return fail_status(STQ_ERR_CUDA, "cannot select device %d", where.device);
    CUtensorMap qm, km, vm;
    // without any key the maps of k and v are not used: q's stand in
    const stq_rows *kr = total_k > 0 ? k : q, *vr = total_k > 0 ? v : q;
    const int kt = total_k > 0 ? total_k : total_q, kh = total_k > 0 ? num_kv_heads : num_heads;
    if (!stq::make_map(&qm, *q, dtype, total_q, num_heads, pack, stq::kRows / pack) ||
        !stq::make_map(&km, *kr, dtype, kt, kh, 1, stq::kRows) || !stq::make_map(&vm, *vr, dtype, kt, kh, 1, stq::kRows))
        return fail_status(STQ_ERR_CUDA, "tensor map");
    stq::PromptAttn a;
    a.q_start = q_start;
    a.k_start = k_start;
    a.n = n;
    a.heads = num_heads;
    a.group = group;
    a.pack = pack;
    a.total_q = total_q;
    a.total_k = total_k;
    // at least 2^-100, so that a hidden score of -inf stays one
    a.scale_log2 = static_cast<float>(std::max(std::fabs(static_cast<double>(scale)) * 1.4426950408889634, 0x1p-100));
    a.negative = scale < 0.0f;
    a.y = y;
    a.err = err;
    a.waits = stq::waits();
    const auto kernel = dtype == STQ_BF16 ? stq::attn_prompt_kernel<true> : stq::attn_prompt_kernel<false>;
    const int smem = static_cast<int>(sizeof(stq::AttnSmem)) + 1024;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return stq::cuda_fail(e, "prompt attention attribute");
    const unsigned grid = static_cast<unsigned>(tiles * (num_heads / pack));
    kernel<<<grid, stq::kThreads, smem, static_cast<cudaStream_t>(stream)>>>(qm, km, vm, a);
    stq::count_launch();
    e = cudaGetLastError();
    return e == cudaSuccess ? STQ_OK : stq::cuda_fail(e, "prompt attention launch");
}
