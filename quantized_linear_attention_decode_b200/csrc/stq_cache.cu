// stq_cache.cu -- keys and values held in 4 bits, and attention of single tokens over them (sm_100a).
//
// A page of 64 tokens of one key head is one 9216-byte block: 64 bytes of codes
// and four binary16 scales for each token's key, and the same for its value
// (layout: include/stq.h).  The block is laid out for the reader: one bulk copy
// brings it into shared memory, and one 16-byte read gives a thread exactly the
// codes that its matrix fragments need.
//
// Codes are kept in sign and magnitude.  A word rotated right by 4 j and masked
// with 0x80078007 is a pair of binary16 subnormals, z 2^-24 each: the tensor core
// takes them as they are, so a pair of codes costs two integer instructions and
// no conversion, and the 2^24 goes into a factor that is applied anyway.
#include <cmath>
#include <new>

#include "stq_host.h"
#include "stq_ptx.h"

struct stq_cache {
    int pages = 0, heads = 0, device = 0, sms = 0;
    uint8_t *d_data = nullptr;
    uint32_t *d_err = nullptr;
};

namespace stq {
namespace {

constexpr int kPage = STQ_CACHE_PAGE, kBlock = STQ_CACHE_BLOCK;
constexpr int kKeyScales = 4096, kValues = 4608, kValueScales = 8704;  // offsets inside a block
constexpr uint32_t kCodes = 0x80078007u;  // sign and magnitude of one low and one high code
constexpr uint32_t kLow = 0x0888F777u;    // bits of the four low codes of a word

static_assert(kValueScales + 512 == kBlock && kD == 128, "block layout");

struct CacheView {
    uint8_t *data;
    int pages, heads;
    uint32_t *err;
    __device__ uint8_t *block(int page, int h) const { return data + (static_cast<size_t>(page) * heads + h) * kBlock; }
};

struct Rows {
    const void *data;
    long long token_stride, head_stride;
};

// ---------------------------------------------------------------- append and read
//
// A warp takes one token of one key head: lanes 0-15 its key, 16-31 its value,
// 8 dims a lane, so that a group of 32 values is four lanes.  Bound by memory
// (the rows in, 144 bytes out); not tuned further.

// The word of eight codes z[0..3] (low) and z[4..7] (high).
__device__ __forceinline__ uint32_t low_codes(const int (&z)[4])
{
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t m = static_cast<uint32_t>(abs(z[j]));
        w |= m << (4 * j) | (z[j] < 0 ? 1u : 0u) << (4 * j + 15);
    }
    return w;
}

__device__ __forceinline__ void word_codes(uint32_t w, float (&z)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t p = __funnelshift_r(w, w, 4 * j) & kCodes;
        const float lo = static_cast<float>(p & 7u), hi = static_cast<float>(p >> 16 & 7u);
        z[j] = p & 0x8000u ? -lo : lo;
        z[4 + j] = p & 0x80000000u ? -hi : hi;
    }
}

__global__ void __launch_bounds__(256) append_kernel(CacheView c, const long long *slot, int n, int dtype, Rows k, Rows v)
{
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(n) * c.heads) return;
    const int i = static_cast<int>(item / c.heads), h = static_cast<int>(item - static_cast<long long>(i) * c.heads);
    const int lane = threadIdx.x & 31, l = lane & 15;
    const bool key = lane < 16;
    const long long at = slot[i];
    if (at < 0) return;
    if (at >= static_cast<long long>(c.pages) * kPage) {
        if (lane == 0) atomicOr(c.err, kErrIndex);
        return;
    }
    const Rows &r = key ? k : v;
    float x[8];
    load8(r.data, i * r.token_stride + h * r.head_stride + 8 * l, dtype, x);
    float a = 0.0f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        a = fmaxf(a, fabsf(x[j]));
        bad |= !isfinite(x[j]);
    }
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t mine = __ballot_sync(0xffffffffu, bad);
    __half s = __float2half_rn(__fdiv_rn(a, 7.0f));
    float sf = __half2float(s);
    if ((mine >> (lane & ~3) & 15u) != 0 || !isfinite(sf)) {
        s = __float2half_rn(0.0f);
        sf = 0.0f;
        if ((lane & 3) == 0) atomicOr(c.err, kErrNonFinite);
    }
    int lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float z = sf > 0.0f ? rintf(__fdiv_rn(x[j], sf)) : 0.0f;
        z = fminf(fmaxf(z, -7.0f), 7.0f);
        (j < 4 ? lo : hi)[j & 3] = static_cast<int>(z);
    }
    const int o = static_cast<int>(at & (kPage - 1)), g = l >> 2, t = l & 3;
    uint8_t *b = c.block(static_cast<int>(at / kPage), h);
    if (key) {
        const uint32_t w0 = low_codes(lo), w1 = low_codes(hi);
        *reinterpret_cast<uint32_t *>(b + 64 * o + 16 * t + 4 * g) = w0 | __funnelshift_l(w1, w1, 16);
        if (t == 0) *reinterpret_cast<__half *>(b + kKeyScales + 8 * o + 2 * g) = s;
    } else {
        // a value word holds two tokens: each append changes its own token's bits
        // only, with an AND and an OR, so tokens of one pair may come in one call
        const int p = o >> 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w = half ? low_codes(hi) : low_codes(lo), others = ~kLow;
            if (o & 1) {
                w = __funnelshift_l(w, w, 16);
                others = kLow;
            }
            uint32_t *to = reinterpret_cast<uint32_t *>(b + kValues + 128 * p + 16 * ((2 * t + half + 2 * p) & 7) + 4 * g);
            atomicAnd(to, w | others);
            atomicOr(to, w);
        }
        if (t == 0) *reinterpret_cast<__half *>(b + kValueScales + 16 * p + 4 * g + 2 * (o & 1)) = s;
    }
}

__global__ void __launch_bounds__(256) read_kernel(CacheView c, const long long *slot, int n, float *k, float *v)
{
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(n) * c.heads) return;
    const int i = static_cast<int>(item / c.heads), h = static_cast<int>(item - static_cast<long long>(i) * c.heads);
    const int lane = threadIdx.x & 31, l = lane & 15;
    const bool key = lane < 16;
    const long long at = slot[i];
    if (at < 0) return;
    if (at >= static_cast<long long>(c.pages) * kPage) {
        if (lane == 0) atomicOr(c.err, kErrIndex);
        return;
    }
    const int o = static_cast<int>(at & (kPage - 1)), g = l >> 2, t = l & 3, p = o >> 1;
    const uint8_t *b = c.block(static_cast<int>(at / kPage), h);
    float z[8], s;
    if (key) {
        word_codes(*reinterpret_cast<const uint32_t *>(b + 64 * o + 16 * t + 4 * g), z);
        s = __half2float(*reinterpret_cast<const __half *>(b + kKeyScales + 8 * o + 2 * g));
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w = *reinterpret_cast<const uint32_t *>(b + kValues + 128 * p + 16 * ((2 * t + half + 2 * p) & 7) + 4 * g);
            if (o & 1) w = __funnelshift_l(w, w, 16);
            float y[8];
            word_codes(w, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * half + j] = y[j];
        }
        s = __half2float(*reinterpret_cast<const __half *>(b + kValueScales + 16 * p + 4 * g + 2 * (o & 1)));
    }
    float4 *to = reinterpret_cast<float4 *>((key ? k : v) + static_cast<size_t>(item) * kD + 8 * l);
    to[0] = make_float4(s * z[0], s * z[1], s * z[2], s * z[3]);
    to[1] = make_float4(s * z[4], s * z[5], s * z[6], s * z[7]);
}

// ---------------------------------------------------------------- attention of one token a sequence
//
// Bound by reading the cache: 144 bytes a token and key head, 256 codes of it to
// unpack.  The units of work are (sequence, key head and block of query heads,
// page) in that order; every CTA takes an equal contiguous share of all units, so
// a few long sequences and many ragged ones fill the machine alike.  A share
// falls into segments, the runs of pages of one (sequence, head block).  The
// segments that a CTA does not finish alone leave an unnormalised partial sum,
// and join_kernel adds those in the order of the CTAs.
//
// Within a CTA each warp takes every kWarps-th page of the segment with its own
// two-stage ring, softmax statistics and accumulators, and the warps are joined at
// the segment's end.  Per page and block of eight heads, with mma.sync (the
// matrices have 8 columns, far below a tcgen05 tile's 128 rows):
//   S = K q^T      16 tokens x 8 heads a tile.  A group of 32 dims is two steps of
//                  16, so its binary16 scale multiplies the fp32 sums, 4 products
//                  a token in place of 32 conversions.
//   O^T += V^T P^T 16 dims x 8 heads a tile; a value's scale goes into P.  P is
//                  rounded to binary16, and so is its product with the scale: 2^-11 of a
//                  weight each, below the output's own rounding in bf16.
// P is 2^15 exp2(x - R) with R at least the running maximum of x + max(0, log2 of the
// page's largest value scale), so that P times a scale stays below 2^15 while small
// weights keep their bits: what falls below binary16's subnormals is 2^-39 of the
// largest weight.  Sums are fp32.

constexpr int kWarps = 4;
constexpr int kStagesW = 2;

struct AttnArgs {
    CacheView c;
    const int32_t *table;
    const int32_t *seq_len;
    int max_pages, n, heads, group, blocks;  // blocks: of 8 NT query heads, for each key head
    int dtype;
    Rows q;
    float scale_log2;  // scale log2(e)
    void *y;
    float *part;
};

// Floats of one partial: sums [8 NT][128], then R and the sum of weights of each head.
__host__ __device__ constexpr int part_floats(int nt) { return 8 * nt * (kD + 2); }

// Pages of sequence i; 0 where its length is out of range.
__device__ __forceinline__ int pages_of(const AttnArgs &a, int i)
{
    const int len = a.seq_len[i];
    return len < 0 || len > static_cast<long long>(a.max_pages) * kPage ? 0 : (len + kPage - 1) / kPage;
}

// All pages of the sequences before `upto` (the whole warp calls it).
__device__ __forceinline__ long long pages_before(const AttnArgs &a, int upto)
{
    long long sum = 0;
    for (int i = threadIdx.x & 31; i < upto; i += 32) sum += pages_of(a, i);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    return sum;
}

// Where a walk over the units stands: page `page` of sequence seq, head block sub.
struct Walk {
    int seq, pages, sub, page;
};

// The place of unit u of all (u below their number); the whole warp calls it.
__device__ __forceinline__ Walk place_of(const AttnArgs &a, long long u, int subs)
{
    const int lane = threadIdx.x & 31;
    Walk w{0, 0, 0, 0};
    long long base = 0;
    for (int first = 0; first < a.n; first += 32) {
        const int i = first + lane;
        const int p = i < a.n ? pages_of(a, i) : 0;
        long long upto = static_cast<long long>(p) * subs;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + upto > u);
        if (past) {
            const int who = __ffs(past) - 1;
            const long long end = __shfl_sync(0xffffffffu, base + upto, who);
            w.seq = first + who;
            w.pages = __shfl_sync(0xffffffffu, p, who);
            const long long in = u - (end - static_cast<long long>(w.pages) * subs);
            w.sub = static_cast<int>(in / w.pages);
            w.page = static_cast<int>(in - static_cast<long long>(w.sub) * w.pages);
            return w;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return w;
}

// The next head block, or the next sequence that has pages.
__device__ __forceinline__ void next_segment(const AttnArgs &a, Walk &w, int subs)
{
    w.page = 0;
    if (++w.sub < subs) return;
    w.sub = 0;
    do {
        ++w.seq;
        w.pages = w.seq < a.n ? pages_of(a, w.seq) : 0;
    } while (w.seq < a.n && w.pages == 0);
}

// A warp's pages in the order it takes them, running ahead of the arithmetic: the
// page numbers of 32 pages at a time are held one in each lane.
struct Feed {
    Walk w;
    long long left;  // units from the segment's first page in the share to the share's end
    int page, end;   // this warp's next page in the segment, and the segment's end in the share
    int ids, first;  // ids: lane j has the page number of page first + j * kWarps
};

__device__ __forceinline__ void feed_segment(const AttnArgs &a, Feed &f, int warp)
{
    const long long room = f.w.page + f.left;
    f.end = room < f.w.pages ? static_cast<int>(room) : f.w.pages;
    f.page = f.w.page + warp;
    f.first = f.page - 32 * kWarps;
}

// The page number of the warp's next page (-1: none left; -2: outside the cache).
__device__ __forceinline__ int feed_next(const AttnArgs &a, Feed &f, int warp, int subs, int *head)
{
    while (f.page >= f.end) {
        f.left -= f.end - f.w.page;
        if (f.left <= 0) return -1;
        next_segment(a, f.w, subs);
        feed_segment(a, f, warp);
    }
    if (f.page >= f.first + 32 * kWarps) {
        f.first = f.page;
        const int p = f.first + (threadIdx.x & 31) * kWarps;
        f.ids = p < f.end ? a.table[static_cast<size_t>(f.w.seq) * a.max_pages + p] : 0;
    }
    const int id = __shfl_sync(0xffffffffu, f.ids, (f.page - f.first) / kWarps);
    f.page += kWarps;
    *head = f.w.sub / a.blocks;
    return id < 0 || id >= a.c.pages ? -2 : id;
}

template <int NT>
struct __align__(128) AttnSmem {
    uint8_t stage[kWarps][kStagesW][kBlock];
    float sum[8 * NT][kD + 4];
    float top[kWarps][8 * NT], weight[kWarps][8 * NT];
    unsigned long long full[kWarps][kStagesW];
};

__device__ __forceinline__ uint32_t pair_of(uint32_t w, int j) { return __funnelshift_r(w, w, 4 * j) & kCodes; }

template <int NT>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_decode_kernel(const AttnArgs a)
{
    extern __shared__ uint8_t raw_smem[];
    AttnSmem<NT> &sm = *reinterpret_cast<AttnSmem<NT> *>((reinterpret_cast<uintptr_t>(raw_smem) + 127) & ~uintptr_t(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    launch_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
            const int len = a.seq_len[i];
            if (len < 0 || len > static_cast<long long>(a.max_pages) * kPage) atomicOr(a.c.err, kErrIndex);
        }
    const int subs = a.c.heads * a.blocks;
    const long long units = pages_before(a, a.n) * subs;
    const long long lo = units * blockIdx.x / gridDim.x, hi = units * (blockIdx.x + 1) / gridDim.x;
    if (lo >= hi) return;
    const uint32_t bar0 = smem_addr(&sm.full[warp][0]), st0 = smem_addr(&sm.stage[warp][0][0]);
    if (lane == 0) {
        for (int s = 0; s < kStagesW; ++s) barrier_init(bar0 + 8 * s, 1);
        fence_barrier_init();
    }
    __syncwarp();

    Feed feed;
    feed.w = place_of(a, lo, subs);
    feed.left = hi - lo;
    feed.ids = 0;
    feed_segment(a, feed, warp);
    Walk w = feed.w;
    long long left = hi - lo;
    int issued = 0, taken = 0;        // pages of this warp, by number
    uint32_t absent = 0;              // bit s: stage s stands for a page outside the cache
    bool dead = false;                // a copy did not arrive
    const auto issue = [&]() {
        int head = 0;
        const int id = feed_next(a, feed, warp, subs, &head);
        if (id == -1) return;
        const int s = issued % kStagesW;
        if (id >= 0) {
            absent &= ~(1u << s);
            if (lane == 0) {
                barrier_expect(bar0 + 8 * s, kBlock);
                bulk_copy(st0 + s * kBlock, a.c.block(id, head), kBlock, bar0 + 8 * s);
            }
        } else {
            absent |= 1u << s;
            if (lane == 0) {
                atomicOr(a.c.err, kErrIndex);
                barrier_arrive(bar0 + 8 * s);
            }
        }
        ++issued;
    };
    for (int s = 0; s < kStagesW; ++s) issue();

    bool first = true;
    while (left > 0) {
        const int p0 = w.page, p1 = static_cast<int>(p0 + left < w.pages ? p0 + left : w.pages);
        const int len = a.seq_len[w.seq];
        const int kvh = w.sub / a.blocks, hb = w.sub - kvh * a.blocks;
        const int h0 = kvh * a.group + hb * 8 * NT, nh = min(8 * NT, a.group - hb * 8 * NT);

        // q as B fragments: step (group gi, j) takes dims 32 gi + 8 t + j and + 4 + j of head g, scaled by
        // a power of two so that every row lies in binary16's range (the largest value in [1, 2))
        uint32_t qf[NT][4][4];
        float fac[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float x[4][8], top = 0.0f;
            const int h = nt * 8 + g;
#pragma unroll
            for (int gi = 0; gi < 4; ++gi) {
                if (h < nh) load8(a.q.data, w.seq * a.q.token_stride + (h0 + h) * a.q.head_stride + 32 * gi + 8 * t, a.dtype, x[gi]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (h >= nh) x[gi][j] = 0.0f;
                    top = fmaxf(top, fabsf(x[gi][j]));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = top > 0.0f && top < INFINITY ? ilogbf(top) : 0;
#pragma unroll
            for (int gi = 0; gi < 4; ++gi)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 v = __floats2half2_rn(ldexpf(x[gi][j], -e), ldexpf(x[gi][4 + j], -e));
                    qf[nt][gi][j] = *reinterpret_cast<const uint32_t *>(&v);
                }
            // this head's factor is wanted where its scores are: columns 2t, 2t + 1 of every lane
            const float f = ldexpf(a.scale_log2, e + 24);
            fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
            fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        }

        float o[8][NT][4], top[NT][2], weight[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt][0] = top[nt][1] = -INFINITY;
            weight[nt][0] = weight[nt][1] = 0.0f;
#pragma unroll
            for (int m = 0; m < 8; ++m) o[m][nt][0] = o[m][nt][1] = o[m][nt][2] = o[m][nt][3] = 0.0f;
        }

        for (int p = p0 + warp; p < p1 && !dead; p += kWarps) {
            const int s = taken % kStagesW;
            if (!__all_sync(0xffffffffu, barrier_wait(bar0 + 8 * s, taken / kStagesW & 1))) {
                if (lane == 0) atomicOr(a.c.err, kErrTimeout);
                dead = true;
                break;
            }
            if (!(absent >> s & 1)) {
                const uint8_t *b = sm.stage[warp][s];
                float x[4][NT][4];
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const int r0 = mt * 16 + g, r1 = r0 + 8;
                    const uint4 ka = *reinterpret_cast<const uint4 *>(b + 64 * r0 + 16 * t);
                    const uint4 kb = *reinterpret_cast<const uint4 *>(b + 64 * r1 + 16 * t);
                    const uint2 sa = *reinterpret_cast<const uint2 *>(b + kKeyScales + 8 * r0);
                    const uint2 sb = *reinterpret_cast<const uint2 *>(b + kKeyScales + 8 * r1);
                    const float2 sa0 = __half22float2(*reinterpret_cast<const __half2 *>(&sa.x)), sa1 = __half22float2(*reinterpret_cast<const __half2 *>(&sa.y));
                    const float2 sb0 = __half22float2(*reinterpret_cast<const __half2 *>(&sb.x)), sb1 = __half22float2(*reinterpret_cast<const __half2 *>(&sb.y));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
                    const float fa[4] = {sa0.x, sa0.y, sa1.x, sa1.y}, fb[4] = {sb0.x, sb0.y, sb1.x, sb1.y};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) x[mt][nt][0] = x[mt][nt][1] = x[mt][nt][2] = x[mt][nt][3] = 0.0f;
#pragma unroll
                    for (int gi = 0; gi < 4; ++gi) {
                        uint32_t pa[4], pb[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            pa[j] = pair_of(wa[gi], j);
                            pb[j] = pair_of(wb[gi], j);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(c, pa[0], pb[0], pa[1], pb[1], qf[nt][gi][0], qf[nt][gi][1]);
                            mma_f16(c, pa[2], pb[2], pa[3], pb[3], qf[nt][gi][2], qf[nt][gi][3]);
                            x[mt][nt][0] = fmaf(fa[gi], c[0], x[mt][nt][0]);
                            x[mt][nt][1] = fmaf(fa[gi], c[1], x[mt][nt][1]);
                            x[mt][nt][2] = fmaf(fb[gi], c[2], x[mt][nt][2]);
                            x[mt][nt][3] = fmaf(fb[gi], c[3], x[mt][nt][3]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[mt][nt][j] *= fac[nt][j & 1];
                }
                const int valid = len - p * kPage;  // tokens of this page
                if (valid < kPage) {
#pragma unroll
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (mt * 16 + g + (j >> 1) * 8 >= valid) x[mt][nt][j] = -INFINITY;
                }
                // the page's largest value scale (positive binary16 values order as integers), as a power of two >= 1
                const uint4 vs = *reinterpret_cast<const uint4 *>(b + kValueScales + 16 * lane);
                const __half2 m2 = __hmax2(__hmax2(*reinterpret_cast<const __half2 *>(&vs.x), *reinterpret_cast<const __half2 *>(&vs.y)),
                                           __hmax2(*reinterpret_cast<const __half2 *>(&vs.z), *reinterpret_cast<const __half2 *>(&vs.w)));
                const uint32_t mu = *reinterpret_cast<const uint32_t *>(&m2);
                const uint32_t biggest = __reduce_max_sync(0xffffffffu, max(mu & 0xffffu, mu >> 16));
                const float up = static_cast<float>(max(0, static_cast<int>(biggest >> 10) - 14));
                bool moved = false;
                float old[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = -INFINITY;
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt) m = fmaxf(m, fmaxf(x[mt][nt][j], x[mt][nt][2 + j]));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16)) + up;
                        old[nt][j] = top[nt][j];
                        moved |= m > top[nt][j];
                        top[nt][j] = fmaxf(top[nt][j], m);
                    }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float f0 = exp2_approx(old[nt][0] - top[nt][0]), f1 = exp2_approx(old[nt][1] - top[nt][1]);
                        weight[nt][0] *= f0;
                        weight[nt][1] *= f1;
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            o[m][nt][0] *= f0;
                            o[m][nt][1] *= f1;
                            o[m][nt][2] *= f0;
                            o[m][nt][3] *= f1;
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    const int pr = mt * 8 + t;  // pairs pr and pr + 4; both lie rotated by 2 t
                    const int pos = (g + 2 * t & 7) * 16;
                    const uint4 va = *reinterpret_cast<const uint4 *>(b + kValues + 128 * pr + pos);
                    const uint4 vb = *reinterpret_cast<const uint4 *>(b + kValues + 128 * (pr + 4) + pos);
                    const uint4 ua = *reinterpret_cast<const uint4 *>(b + kValueScales + 16 * pr);
                    const uint4 ub = *reinterpret_cast<const uint4 *>(b + kValueScales + 16 * (pr + 4));
                    const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
                    const uint32_t fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w};
                    __half2 b0[NT], b1[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float e[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) e[j] = exp2_approx(x[mt][nt][j] - top[nt][j & 1] + 15.0f);
                        weight[nt][0] += e[0] + e[2];
                        weight[nt][1] += e[1] + e[3];
                        const __half2 c0 = __floats2half2_rn(e[0], e[1]), c1 = __floats2half2_rn(e[2], e[3]);
                        const uint32_t d0 = transpose8(*reinterpret_cast<const uint32_t *>(&c0));
                        const uint32_t d1 = transpose8(*reinterpret_cast<const uint32_t *>(&c1));
                        b0[nt] = *reinterpret_cast<const __half2 *>(&d0);
                        b1[nt] = *reinterpret_cast<const __half2 *>(&d1);
                    }
#pragma unroll
                    for (int gi = 0; gi < 4; ++gi) {
                        uint32_t pa[4], pb[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            pa[j] = pair_of(wa[gi], j);
                            pb[j] = pair_of(wb[gi], j);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const __half2 e0 = __hmul2(b0[nt], *reinterpret_cast<const __half2 *>(&fa[gi]));
                            const __half2 e1 = __hmul2(b1[nt], *reinterpret_cast<const __half2 *>(&fb[gi]));
                            const uint32_t u0 = *reinterpret_cast<const uint32_t *>(&e0), u1 = *reinterpret_cast<const uint32_t *>(&e1);
                            mma_f16(o[2 * gi][nt], pa[0], pa[1], pb[0], pb[1], u0, u1);
                            mma_f16(o[2 * gi + 1][nt], pa[2], pa[3], pb[2], pb[3], u0, u1);
                        }
                    }
                }
            }
            __syncwarp();
            ++taken;
            issue();
        }

        // join the warps in order
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = weight[nt][j];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    sm.top[warp][nt * 8 + 2 * t + j] = top[nt][j];
                    sm.weight[warp][nt * 8 + 2 * t + j] = l;
                }
            }
        __syncthreads();
        float f[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float all = -INFINITY;
                for (int v = 0; v < kWarps; ++v) all = fmaxf(all, sm.top[v][nt * 8 + 2 * t + j]);
                f[nt][j] = top[nt][j] == -INFINITY ? 0.0f : exp2_approx(top[nt][j] - all);
            }
        for (int v = 0; v < kWarps; ++v) {
            if (warp == v) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int m = 0; m < 8; ++m)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int dim = 32 * (m >> 1) + 4 * g + 2 * (m & 1) + (j >> 1);
                            float *to = &sm.sum[nt * 8 + 2 * t + (j & 1)][dim];
                            const float y = o[m][nt][j] * f[nt][j & 1];
                            *to = v == 0 ? y : *to + y;
                        }
            }
            __syncthreads();
        }
        const bool whole = p0 == 0 && p1 == w.pages;
        float *part = a.part + (static_cast<size_t>(blockIdx.x) * 2 + (first ? 0 : 1)) * part_floats(NT);
        for (int e = threadIdx.x; e < nh * kD; e += blockDim.x) {
            const int h = e / kD, d = e - h * kD;
            if (whole) {
                float all = -INFINITY, l = 0.0f;
                for (int v = 0; v < kWarps; ++v) all = fmaxf(all, sm.top[v][h]);
                for (int v = 0; v < kWarps; ++v)
                    if (sm.top[v][h] != -INFINITY) l += sm.weight[v][h] * exp2_approx(sm.top[v][h] - all);
                const float y = l > 0.0f || l != l ? sm.sum[h][d] * 16777216.0f / l : 0.0f;
                store_from_float(a.y, (static_cast<int64_t>(w.seq) * a.heads + h0 + h) * kD + d, a.dtype, y);
            } else {
                part[h * kD + d] = sm.sum[h][d];
                if (d == 0) {
                    float all = -INFINITY, l = 0.0f;
                    for (int v = 0; v < kWarps; ++v) all = fmaxf(all, sm.top[v][h]);
                    for (int v = 0; v < kWarps; ++v)
                        if (sm.top[v][h] != -INFINITY) l += sm.weight[v][h] * exp2_approx(sm.top[v][h] - all);
                    part[8 * NT * kD + 2 * h] = all;
                    part[8 * NT * kD + 2 * h + 1] = l;
                }
            }
        }
        __syncthreads();  // the sums are read before the next segment's are written
        first = false;
        left -= p1 - p0;
        next_segment(a, w, subs);
    }
    // after a wait that gave up, let the copies in flight land (bounded) before the memory is given back
    if (dead)
        for (; taken < issued; ++taken) barrier_wait(bar0 + 8 * (taken % kStagesW), taken / kStagesW & 1);
}

// Joins the partial sums of one (sequence, query head) in the order of the CTAs
// that left them, and writes the zeros of sequences without tokens.  One CTA of
// eight warps: each takes every eighth partial, a lane four dims.
template <int NT>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a, int ctas)
{
    __shared__ float acc[8][kD];
    __shared__ float tops[8], weights[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int seq = blockIdx.x / a.heads, head = blockIdx.x - seq * a.heads;
    const int kvh = head / a.group, in = head - kvh * a.group, hb = in / (8 * NT), h = in - hb * 8 * NT;
    const int subs = a.c.heads * a.blocks, sub = kvh * a.blocks + hb;
    const int len = a.seq_len[seq];
    const int pages = pages_of(a, seq);
    const long long units = pages_before(a, a.n) * subs;
    const long long u0 = pages_before(a, seq) * subs + static_cast<long long>(sub) * pages, u1 = u0 + pages - 1;
    wait_previous_grid();  // in every CTA, so that the end of this grid is the end of both
    if (len < 0 || len > static_cast<long long>(a.max_pages) * kPage) return;
    const int64_t at = (static_cast<int64_t>(seq) * a.heads + head) * kD;
    if (len == 0) {
        if (threadIdx.x < kD) store_from_float(a.y, at + threadIdx.x, a.dtype, 0.0f);
        return;
    }
    // CTA b has units [units b / ctas, units (b + 1) / ctas)
    const int b0 = static_cast<int>(((u0 + 1) * ctas - 1) / units), b1 = static_cast<int>(((u1 + 1) * ctas - 1) / units);
    if (b0 == b1) return;  // finished by one CTA
    const auto part_of = [&](int b) {  // a segment that a CTA begins in is its first
        const bool begins = units * b / ctas >= u0;
        return a.part + (static_cast<size_t>(b) * 2 + (begins ? 0 : 1)) * part_floats(NT);
    };
    float top = -INFINITY, weight = 0.0f;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int b = b0 + warp; b <= b1; b += 8) {
        if (units * b / ctas == units * (b + 1) / ctas) continue;  // a CTA without units
        const float *p = part_of(b);
        const float r = p[8 * NT * kD + 2 * h], l = p[8 * NT * kD + 2 * h + 1];
        const float4 v = *reinterpret_cast<const float4 *>(p + h * kD + 4 * lane);
        if (r == -INFINITY) continue;
        const float m = fmaxf(top, r), f0 = exp2_approx(top - m), f1 = exp2_approx(r - m);
        y = make_float4(y.x * f0 + v.x * f1, y.y * f0 + v.y * f1, y.z * f0 + v.z * f1, y.w * f0 + v.w * f1);
        weight = weight * f0 + l * f1;
        top = m;
    }
    *reinterpret_cast<float4 *>(&acc[warp][4 * lane]) = y;
    if (lane == 0) {
        tops[warp] = top;
        weights[warp] = weight;
    }
    __syncthreads();
    if (threadIdx.x < kD) {
        float all = -INFINITY, l = 0.0f, s = 0.0f;
        for (int v = 0; v < 8; ++v) all = fmaxf(all, tops[v]);
        for (int v = 0; v < 8; ++v)
            if (tops[v] != -INFINITY) {
                const float f = exp2_approx(tops[v] - all);
                l += weights[v] * f;
                s += acc[v][threadIdx.x] * f;
            }
        store_from_float(a.y, at + threadIdx.x, a.dtype, l > 0.0f || l != l ? s * 16777216.0f / l : 0.0f);
    }
}

CacheView view(const stq_cache *c) { return CacheView{c->d_data, c->pages, c->heads, c->d_err}; }

Rows rows(const stq_rows *r) { return Rows{r->data, r->token_stride, r->head_stride}; }

// CTAs of one attn_decode launch: two on every SM.
int attn_ctas(const stq_cache *c) { return 2 * c->sms; }

// Blocks of 16 query heads where a key head has more than 8, else of 8.
int attn_nt(int group) { return group > 8 ? 2 : 1; }

template <int NT>
cudaError_t launch_attn(const AttnArgs &a, int ctas, cudaStream_t s)
{
    const int smem = static_cast<int>(sizeof(AttnSmem<NT>)) + 128;
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attn_decode_kernel<NT><<<ctas, kWarps * 32, smem, s>>>(a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // the join's prologue may run while the last CTAs finish
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n) * a.heads);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_kernel<NT>, a, ctas);
    count_launch();
    return e;
}

stq_status check_rows(const stq_rows *r, const char *name, int32_t dtype, int32_t n)
{
    if (r == nullptr) return fail_status(STQ_ERR_ARG, "%s is NULL", name);
    if (n > 0 && r->data == nullptr) return fail_status(STQ_ERR_ARG, "%s.data is NULL", name);
    if (!rows_aligned(r, dtype)) return fail_status(STQ_ERR_ARG, "%s: rows must start on 16-byte boundaries", name);
    return STQ_OK;
}

}  // namespace
}  // namespace stq

using stq::fail_status;

extern "C" {

stq_status stq_cache_create(int32_t num_pages, int32_t num_kv_heads, int32_t head_dim, stq_cache **out)
{
    if (out == nullptr) return fail_status(STQ_ERR_ARG, "out is NULL");
    *out = nullptr;
    if (num_pages < 1 || num_kv_heads < 1)
        return fail_status(STQ_ERR_ARG, "sizes pages=%d heads=%d must be >= 1", num_pages, num_kv_heads);
    if (head_dim != stq::kD) return fail_status(STQ_ERR_UNSUPPORTED, "head_dim=%d: only 128", head_dim);
    if (static_cast<double>(num_pages) * num_kv_heads * stq::kBlock > 9.0e18)
        return fail_status(STQ_ERR_ARG, "cache size overflows");
    if (stq::fault("alloc")) return fail_status(STQ_ERR_OOM, "injected allocation failure (STQ_FAULT=alloc)");
    stq_cache *c = new (std::nothrow) stq_cache();
    if (c == nullptr) return fail_status(STQ_ERR_OOM, "host allocation");
    c->pages = num_pages;
    c->heads = num_kv_heads;
    const size_t bytes = static_cast<size_t>(num_pages) * num_kv_heads * stq::kBlock;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&c->sms, cudaDevAttrMultiProcessorCount, c->device);
    if (e == cudaSuccess) e = cudaMalloc(&c->d_data, bytes);
    if (e == cudaSuccess) e = cudaMalloc(&c->d_err, 256);
    if (e == cudaSuccess) e = cudaMemset(c->d_data, 0, bytes);
    if (e == cudaSuccess) e = cudaMemset(c->d_err, 0, 256);
    // the zeros are there before any stream's first append
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        const stq_status r = stq::cuda_fail(e, "cache allocation");
        cudaFree(c->d_data);
        cudaFree(c->d_err);
        cudaGetLastError();
        delete c;
        return r;
    }
    *out = c;
    return STQ_OK;
}

stq_status stq_cache_destroy(stq_cache *c)
{
    if (c == nullptr) return STQ_OK;
    stq::DeviceGuard g(c->device);
    cudaFree(c->d_data);
    cudaFree(c->d_err);
    delete c;
    return STQ_OK;
}

stq_status stq_cache_bytes(const stq_cache *c, size_t *bytes)
{
    if (c == nullptr || bytes == nullptr) return fail_status(STQ_ERR_ARG, "NULL argument");
    *bytes = static_cast<size_t>(c->pages) * c->heads * stq::kBlock;
    return STQ_OK;
}

stq_status stq_cache_append(stq_cache *c, const int64_t *slot, int32_t n, int32_t dtype, const stq_rows *k,
                            const stq_rows *v, void *stream)
{
    if (c == nullptr) return fail_status(STQ_ERR_ARG, "cache is NULL");
    if (n < 0) return fail_status(STQ_ERR_ARG, "n = %d", n);
    if (stq::dtype_bytes(dtype) == 0) return fail_status(STQ_ERR_ARG, "dtype %d", dtype);
    stq_status st = stq::check_rows(k, "k", dtype, n);
    if (st == STQ_OK) st = stq::check_rows(v, "v", dtype, n);
    if (st != STQ_OK) return st;
    if (n > 0 && slot == nullptr) return fail_status(STQ_ERR_ARG, "slot is NULL");
    if (static_cast<long long>(n) * c->heads > 0x7FFFFFFFll) return fail_status(STQ_ERR_ARG, "n * heads too large");
    if (n == 0) return STQ_OK;
    if (stq::fault("launch")) return fail_status(STQ_ERR_CUDA, "injected launch failure (STQ_FAULT=launch)");
    stq::DeviceGuard g(c->device);
    stq::NvtxRange nvtx("stq_cache_append");
    if (!g.ok) return fail_status(STQ_ERR_CUDA, "cannot select device %d", c->device);
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(n) * c->heads + 7) / 8);
    stq::append_kernel<<<ctas, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        stq::view(c), reinterpret_cast<const long long *>(slot), n, dtype, stq::rows(k), stq::rows(v));
    stq::count_launch();
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? STQ_OK : stq::cuda_fail(e, "append launch");
}

stq_status stq_cache_read(stq_cache *c, const int64_t *slot, int32_t n, float *k_out, float *v_out, void *stream)
{
    if (c == nullptr) return fail_status(STQ_ERR_ARG, "cache is NULL");
    if (n < 0) return fail_status(STQ_ERR_ARG, "n = %d", n);
    if (n > 0 && (slot == nullptr || k_out == nullptr || v_out == nullptr))
        return fail_status(STQ_ERR_ARG, "a slot/k_out/v_out pointer is NULL");
    if ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) % 16 != 0)
        return fail_status(STQ_ERR_ARG, "k_out and v_out must be 16-byte aligned");
    if (static_cast<long long>(n) * c->heads > 0x7FFFFFFFll) return fail_status(STQ_ERR_ARG, "n * heads too large");
    if (n == 0) return STQ_OK;
    if (stq::fault("launch")) return fail_status(STQ_ERR_CUDA, "injected launch failure (STQ_FAULT=launch)");
    stq::DeviceGuard g(c->device);
    stq::NvtxRange nvtx("stq_cache_read");
    if (!g.ok) return fail_status(STQ_ERR_CUDA, "cannot select device %d", c->device);
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(n) * c->heads + 7) / 8);
    stq::read_kernel<<<ctas, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        stq::view(c), reinterpret_cast<const long long *>(slot), n, k_out, v_out);
    stq::count_launch();
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? STQ_OK : stq::cuda_fail(e, "read launch");
}

stq_status stq_attn_decode_workspace(const stq_cache *c, int32_t n, int32_t num_heads, size_t *bytes)
{
    if (c == nullptr || bytes == nullptr) return fail_status(STQ_ERR_ARG, "NULL argument");
    if (n < 0) return fail_status(STQ_ERR_ARG, "n = %d", n);
    if (num_heads < 1 || num_heads % c->heads != 0)
        return fail_status(STQ_ERR_ARG, "num_heads=%d is no multiple of the cache's %d heads", num_heads, c->heads);
    *bytes = static_cast<size_t>(stq::attn_ctas(c)) * 2 * stq::part_floats(stq::attn_nt(num_heads / c->heads)) * sizeof(float);
    return STQ_OK;
}

stq_status stq_attn_decode(stq_cache *c, const int32_t *page_table, int32_t max_pages, const int32_t *seq_len,
                           int32_t n, int32_t num_heads, int32_t dtype, const stq_rows *q, float scale, void *y,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    size_t need = 0;
    stq_status st = stq_attn_decode_workspace(c, n, num_heads, &need);
    if (st != STQ_OK) return st;
    if (stq::dtype_bytes(dtype) == 0) return fail_status(STQ_ERR_ARG, "dtype %d", dtype);
    if (max_pages < 0) return fail_status(STQ_ERR_ARG, "max_pages = %d", max_pages);
    if (!std::isfinite(scale)) return fail_status(STQ_ERR_ARG, "scale is not finite");
    st = stq::check_rows(q, "q", dtype, n);
    if (st != STQ_OK) return st;
    if (n > 0 && ((page_table == nullptr && max_pages > 0) || seq_len == nullptr || y == nullptr || workspace == nullptr))
        return fail_status(STQ_ERR_ARG, "a page_table/seq_len/y/workspace pointer is NULL");
    if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(workspace)) % 16 != 0)
        return fail_status(STQ_ERR_ARG, "y and workspace must be 16-byte aligned");
    if (n > 0 && workspace_bytes < need)
        return fail_status(STQ_ERR_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (static_cast<long long>(n) * num_heads > 0x7FFFFFFFll) return fail_status(STQ_ERR_ARG, "n * num_heads too large");
    if (n == 0) return STQ_OK;
    if (stq::fault("launch")) return fail_status(STQ_ERR_CUDA, "injected launch failure (STQ_FAULT=launch)");
    stq::DeviceGuard g(c->device);
    stq::NvtxRange nvtx("stq_attn_decode");
    if (!g.ok) return fail_status(STQ_ERR_CUDA, "cannot select device %d", c->device);
    stq::AttnArgs a;
    a.c = stq::view(c);
    a.table = page_table;
    a.seq_len = seq_len;
    a.max_pages = max_pages;
    a.n = n;
    a.heads = num_heads;
    a.group = num_heads / c->heads;
    const int nt = stq::attn_nt(a.group);
    a.blocks = (a.group + 8 * nt - 1) / (8 * nt);
    a.dtype = dtype;
    a.q = stq::rows(q);
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.y = y;
    a.part = static_cast<float *>(workspace);
    const int ctas = stq::attn_ctas(c);
    const cudaError_t e = nt == 2 ? stq::launch_attn<2>(a, ctas, static_cast<cudaStream_t>(stream))
                                  : stq::launch_attn<1>(a, ctas, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? STQ_OK : stq::cuda_fail(e, "attention launch");
}

stq_status stq_cache_check(stq_cache *c, void *stream)
{
    if (c == nullptr) return fail_status(STQ_ERR_ARG, "cache is NULL");
    stq::DeviceGuard g(c->device);
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    uint32_t word = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&word, c->d_err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(c->d_err, 0, 4);
    if (e != cudaSuccess) return stq::cuda_fail(e, "error word");
    if (word & stq::kErrTimeout) return fail_status(STQ_ERR_TIMEOUT, "a device-side wait timed out");
    if (word & stq::kErrIndex) return fail_status(STQ_ERR_INDEX, "token slot, page or length out of range");
    if (word & stq::kErrNonFinite) return fail_status(STQ_ERR_NONFINITE, "non-finite value appended");
    return STQ_OK;
}

}  // extern "C"
