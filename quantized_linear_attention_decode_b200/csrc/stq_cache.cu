// stq_cache.cu -- keys and values held in 4 bits, and attention of single tokens over them (sm_100a).
//
// A page of 64 tokens of one key head is one 9216-byte block of two halves of 32
// tokens: 64 bytes of codes and four binary16 scales for each token's key, and the
// same for its value (layout: include/stq.h).  A half is laid out for the reader: one
// bulk copy brings it into shared memory, and one 16-byte read gives a thread exactly
// the codes that its matrix fragments need.
//
// A code z is kept as u = z + 8 in four bits.  (w & 0x000f000f) | 0x64006400 is a pair of
// binary16 values 1024 + u, and with 0x00f000f0 one of 1024 + 16 u; a packed subtraction
// makes z and 16 z of them, exactly, and the 16 goes into the other operand.  Eight codes
// cost a shift, four logic operations and four packed additions.  (Taken without the
// subtraction, as binary16 subnormals u 2^-24 with the offset removed from the sums, the
// arithmetic was 12 % fewer instructions and no faster, and the sums lost up to 10 bits: the
// tensor core lines products up by their operands' nominal exponents.)
#include <algorithm>
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
constexpr int kHalf = kPage / 2, kHalfBlock = kBlock / 2;              // tokens and bytes of a half
constexpr int kKeyScales = 2048, kValues = 2304, kValueScales = 4352;  // offsets inside it
static_assert(kValueScales + 8 * kHalf == kHalfBlock && kD == 128, "block layout");

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
// An item is one token of one key head.  To read, a warp takes one: lanes 0-15 its key,
// 16-31 its value, 8 dims a lane.  To append, a warp takes two, 16 dims a lane, so that a
// group of 32 values is two lanes: bound by instructions (a warp with one item took 300, and
// 17.5 us for 6600 tokens of 8 heads; two 16 us).

// Four codes as 16 bits of the word, from numbers kCode + z: their bits are those of kCode plus z, and so are sums of them.
constexpr float kCode = 0x1.8p23f + 8.0f;
__device__ __forceinline__ uint32_t pack4(const float *t)
{
    constexpr uint32_t kBits = 0x4b400000u;  // of kCode - 8
    return __float_as_uint(t[0]) + (__float_as_uint(t[1]) << 4) + (__float_as_uint(t[2]) << 8) + (__float_as_uint(t[3]) << 12) - kBits * 0x1111u;
}

// ... and back.
__device__ __forceinline__ void unpack4(uint32_t w, float *z)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = static_cast<float>(static_cast<int>(w >> (4 * j) & 15u) - 8);
}

__global__ void __launch_bounds__(256) append_kernel(CacheView c, const long long *slot, int n, int dtype, Rows k, Rows v)
{
    const int lane = threadIdx.x & 31, l = lane & 7;
    const uint32_t item = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 2 + (lane >> 4);
    const bool key = !(lane & 8);
    const int i = static_cast<int>(item / c.heads), h = static_cast<int>(item - i * static_cast<uint32_t>(c.heads));
    const bool there = item < static_cast<uint32_t>(n) * c.heads;
    const long long at = there ? slot[i] : -1;
    if (there && at >= static_cast<long long>(c.pages) * kPage && l == 0 && key) atomicOr(c.err, kErrIndex);
    const bool held = at >= 0 && at < static_cast<long long>(c.pages) * kPage;
    const Rows &r = key ? k : v;
    float x[16];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        float y[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (held) load8(r.data, i * r.token_stride + h * r.head_stride + 16 * l + 8 * part, dtype, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[8 * part + j] = y[j];
    }
    // the largest size, by its bits: an infinity or a NaN is above all
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if (!held) return;
    __half s = __float2half_rn(__fdiv_rn(__uint_as_float(top), 7.0f));
    float sf = __half2float(s);
    if (top >= 0x7f800000u || !isfinite(sf)) {
        s = __float2half_rn(0.0f);
        sf = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = 0.0f;
        if ((lane & 1) == 0) atomicOr(c.err, kErrNonFinite);
    }
    // kCode + rint(x / s): x times the reciprocal and the quotient are each within 7.01 * 2^-24 of x / s, which decides unless
    // they lie within 2^-20 of a tie; the division is made only then.  A normal s is within 2^-11 of max / 7, so that no quotient is above 7.01; a
    // subnormal one's are clipped.
    float z[16], off = 0.0f;
    const float inv = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        z[j] = fmaf(x[j], inv, kCode);
        off = fmaxf(off, fabsf(fmaf(x[j], inv, kCode - z[j])));
    }
    if (off > 0.499998f || (sf < 0x1p-14f && sf > 0.0f))
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = kCode + fminf(fmaxf(rintf(__fdiv_rn(x[j], sf)), -7.0f), 7.0f);
    // dims 32 g + 16 u and on
    const int o = static_cast<int>(at & (kHalf - 1)), g = l >> 1, u = l & 1;
    uint8_t *b = c.block(static_cast<int>(at / kPage), h) + (at & kHalf ? kHalfBlock : 0) + 4 * g;
    if (key) {
#pragma unroll
        for (int w = 0; w < 2; ++w) *reinterpret_cast<uint32_t *>(b + 64 * o + 16 * (2 * u + w)) = pack4(z + 8 * w) | pack4(z + 8 * w + 4) << 16;
        if (u == 0) *reinterpret_cast<__half *>(b - 2 * g + kKeyScales + 8 * o) = s;
    } else {
        const int p = o >> 1;
#pragma unroll
        for (int w = 0; w < 4; ++w)
            *reinterpret_cast<uint16_t *>(b + kValues + 128 * p + 16 * ((4 * u + w + 2 * p) & 7) + 2 * (o & 1)) = static_cast<uint16_t>(pack4(z + 4 * w));
        if (u == 0) *reinterpret_cast<__half *>(b + kValueScales + 16 * p + 2 * (o & 1)) = s;
    }
}

__global__ void __launch_bounds__(256) read_kernel(CacheView c, const long long *slot, int n, float *k, float *v)
{
    const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= static_cast<uint32_t>(n) * c.heads) return;
    const int i = static_cast<int>(item / c.heads), h = static_cast<int>(item - i * static_cast<uint32_t>(c.heads));
    const int lane = threadIdx.x & 31, l = lane & 15;
    const bool key = lane < 16;
    const long long at = slot[i];
    if (at < 0) return;
    if (at >= static_cast<long long>(c.pages) * kPage) {
        if (lane == 0) atomicOr(c.err, kErrIndex);
        return;
    }
    const int o = static_cast<int>(at & (kHalf - 1)), g = l >> 2, t = l & 3, p = o >> 1;
    const uint8_t *b = c.block(static_cast<int>(at / kPage), h) + (at & kHalf ? kHalfBlock : 0);
    float z[8], s;
    if (key) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(b + 64 * o + 16 * t + 4 * g);
        unpack4(w, z);
        unpack4(w >> 16, z + 4);
        s = __half2float(*reinterpret_cast<const __half *>(b + kKeyScales + 8 * o + 2 * g));
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half)
            unpack4(*reinterpret_cast<const uint16_t *>(b + kValues + 128 * p + 16 * ((2 * t + half + 2 * p) & 7) + 4 * g + 2 * (o & 1)), z + 4 * half);
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
// half page) in that order; every warp takes an equal contiguous share of all units, so
// a few long sequences and many ragged ones fill the machine alike.  A share
// falls into segments, the runs of units of one (sequence, head block).  The
// segments that a warp does not finish alone leave an unnormalised partial sum,
// and join_kernel adds those in the order of the warps.  (Shares a CTA at a time,
// its warps joined at the end of every segment, took 218 us on 64 ragged sequences
// up to 8192 tokens: the joins of short segments stand in a row.)  Where there are
// fewer halves than half of the warps, a unit is a quarter of a page.
//
// A warp has its own ring of halves in shared memory, filled by bulk copies that run
// ahead over the segments.  Per half and block of eight heads, with mma.sync (the
// matrices have 8 columns, far below a tcgen05 tile's 128 rows):
//   S = K q^T      16 tokens x 8 heads a tile.  A group of 32 dims is two steps of
//                  16, so its binary16 scale multiplies the fp32 sums, 4 products
//                  a token in place of 32 conversions.
//   O^T += V^T P^T 16 dims x 8 heads a tile; a value's scale goes into P.  P is
//                  rounded to binary16, and so is its product with the scale: 2^-11 of a
//                  weight each, below the output's own rounding in bf16.
// P is 2^11 exp2(x - R) with R at least the running maximum, less 4, of x + max(0, log2 of the
// unit's largest value scale), so that P times a scale stays below 2^15 while small
// weights keep their bits: what falls below binary16's subnormals is 2^-36 of the
// largest weight.  Sums are fp32.
//
// For fp16 and fp32 rows P, and P's product with a scale, are two binary16 values each
// (TERMS_P), the second what rounding to the first left, and both meet the codes: 2^-22 of a
// weight stays behind, for twice the products.  So is q for fp32 rows (TERMS_Q; of 16 bits it
// is exact in one).  64 sequences to 8192 tokens, 32/8 heads: 77 us in bf16, 86 in fp16 (with
// one value 75, and 1.6 times the error of the output's own rounding), 93 in fp32.

constexpr int kWarps = 4;   // of a CTA; they share nothing but its memory
constexpr int kStagesW = 2;  // units in a warp's ring
constexpr int kUnitBytes = STQ_CACHE_BLOCK;  // a page of a head; quarters of one take a half

constexpr float kSlack = 4.0f;           // how far a score may lie above R

// Pages of a table's row: a length, rounded up to a page, stays within 31 bits.
constexpr int kMostPages = (0x7FFFFFFF - (kPage - 1)) / kPage;

struct AttnArgs {
    CacheView c;
    const int32_t *table;
    const int32_t *seq_len;
    int max_pages, n, heads, group, blocks;  // blocks: of 8 NT query heads, for each key head
    int warps;                               // of the launch
    int dtype;
    Rows q;
    float scale_log2;  // scale log2(e)
    void *y;
    float *part;
    Waits waits;
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

// How all units are shared out: `warps` shares (no more than there are units) of q or q + 1 units,
// the longer ones first.
struct Shares {
    int subs, shift;  // segments of a sequence; 2^shift units of a page (1 or 4)
    long long units, q;
    int warps, longer;
    __device__ long long begin(int w) const { return q * w + min(w, longer); }
    __device__ int owner(long long u) const
    {
        const long long past = u - (q + 1) * longer;
        return static_cast<int>(past < 0 ? u / (q + 1) : longer + past / q);
    }
};

__device__ __forceinline__ Shares shares_of(const AttnArgs &a)
{
    Shares s;
    s.subs = a.c.heads * a.blocks;
    s.units = pages_before(a, a.n) * s.subs;
    s.shift = s.units * 4 <= a.warps ? 2 : 0;
    s.units <<= s.shift;
    s.warps = static_cast<int>(min(static_cast<long long>(a.warps), max(s.units, 1ll)));
    s.q = s.units / s.warps;
    s.longer = static_cast<int>(s.units - s.q * s.warps);
    return s;
}

// Where a walk over the units stands: unit `unit` of the `units` of sequence seq, segment sub.
struct Walk {
    int seq, sub, unit, units;
};

// The place of unit u of all (u below their number); the whole warp calls it.
__device__ __forceinline__ Walk place_of(const AttnArgs &a, const Shares &s, long long u)
{
    const int lane = threadIdx.x & 31;
    Walk w{0, 0, 0, 1};
    long long base = 0;
    for (int first = 0; first < a.n; first += 32) {
        const int i = first + lane;
        const int mine = i < a.n ? pages_of(a, i) << s.shift : 0;
        long long upto = static_cast<long long>(mine) * s.subs;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + upto > u);
        if (past) {
            const int who = __ffs(past) - 1;
            w.seq = first + who;
            w.units = __shfl_sync(0xffffffffu, mine, who);
            const long long in = u - (base + __shfl_sync(0xffffffffu, upto, who) - static_cast<long long>(w.units) * s.subs);
            w.sub = static_cast<int>(in / w.units);
            w.unit = static_cast<int>(in - static_cast<long long>(w.sub) * w.units);
            return w;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return w;
}

// The next segment, of this sequence or of the next one that has pages.
__device__ __forceinline__ void next_segment(const AttnArgs &a, const Shares &s, Walk &w)
{
    w.unit = 0;
    if (++w.sub < s.subs) return;
    w.sub = 0;
    do {
        ++w.seq;
        w.units = w.seq < a.n ? pages_of(a, w.seq) << s.shift : 0;
    } while (w.seq < a.n && w.units == 0);
}

// A share's units in their order, running ahead of the arithmetic: the page numbers
// of 32 units at a time are held one in each lane.
struct Feed {
    Walk w;
    int left;        // units of the share that are still to come
    int first, end;  // lane j has the page number of unit first + j of the segment, up to `end`
    int ids;
};

// The page number of the next unit (-1: none left; -2: outside the cache) its key head and the half.
__device__ __forceinline__ int feed_next(const AttnArgs &a, const Shares &s, Feed &f, int *head, int *half)
{
    if (f.left == 0) return -1;
    if (f.w.unit == f.w.units) {
        next_segment(a, s, f.w);
        f.end = 0;
    }
    if (f.w.unit >= f.end) {
        f.first = f.w.unit;
        f.end = min(f.first + 32, f.w.units);
        const int u = f.first + static_cast<int>(threadIdx.x & 31);
        f.ids = u < f.end ? a.table[static_cast<size_t>(f.w.seq) * a.max_pages + (u >> s.shift)] : 0;
    }
    const int id = __shfl_sync(0xffffffffu, f.ids, f.w.unit - f.first);
    *head = f.w.sub / a.blocks;
    *half = s.shift == 2 ? f.w.unit >> 1 & 1 : 0;
    ++f.w.unit;
    --f.left;
    return id < 0 || id >= a.c.pages ? -2 : id;
}

struct __align__(128) AttnSmem {
    uint8_t stage[kWarps][kStagesW][kUnitBytes];
    unsigned long long full[kWarps][kStagesW];
};

__device__ __forceinline__ __half2 halves(uint32_t h) { return *reinterpret_cast<const __half2 *>(&h); }

// What rounding x to `h` left, in binary16 again.
__device__ __forceinline__ uint32_t rest_of(float2 x, __half2 h)
{
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x.x - f.x, x.y - f.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float2 floats_of(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// The running state of one segment: lane (g, t) has columns 2t, 2t + 1 of each block of eight heads.
template <int NT, int TERMS_Q>
struct Segment {
    uint32_t qf[TERMS_Q][NT][4][4];  // q as B fragments
    float fac[NT][2];       // from products of codes to scores in units of log 2
    float o[8][NT][4], top[NT][2], weight[NT][2];
};

// q: step (group gi, j) takes dims 32 gi + 8 t + j and + 4 + j of head g, scaled by a power of two
// so that every row lies high in binary16's range (the largest value in [2^13, 2^14): a 16-bit q is
// exact down to 2^-20 of it), and by 1 / 16 where the codes come as 16 u.
template <int NT, int TERMS_Q>
__device__ __forceinline__ void begin_segment(const AttnArgs &a, Segment<NT, TERMS_Q> &sg, int seq, int h0, int nh)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float x[4][8], big = 0.0f;
        const int h = nt * 8 + g;
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
            if (h < nh) load8(a.q.data, seq * a.q.token_stride + (h0 + h) * a.q.head_stride + 32 * gi + 8 * t, a.dtype, x[gi]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (h >= nh) x[gi][j] = 0.0f;
                big = fmaxf(big, fabsf(x[gi][j]));
            }
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^e <= big < 2^(e + 1), within what both 2^e and 2^-e can be; the scale's sign goes into q, so that
        // the largest product gives the largest score
        const int e = min(max(static_cast<int>(__float_as_uint(big) >> 23) - 127, -100), 100);
        const float down = copysignf(__uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23), a.scale_log2);
        // (at least 2^-100, so that a hidden token's -inf stays one; sums of products are below 2^40, scores below 2^-60 then)
        const float f = fmaxf(fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23), 0x1p-100f);
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float fold = j & 1 ? 0.0625f * down : down;
                const float2 f = make_float2(x[gi][j] * fold, x[gi][4 + j] * fold);
                const __half2 v = __floats2half2_rn(f.x, f.y);
                sg.qf[0][nt][gi][j] = *reinterpret_cast<const uint32_t *>(&v);
                if (TERMS_Q == 2) sg.qf[TERMS_Q - 1][nt][gi][j] = rest_of(f, v);
            }
        }
        sg.fac[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t);
        sg.fac[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        sg.top[nt][0] = sg.top[nt][1] = -INFINITY;
        sg.weight[nt][0] = sg.weight[nt][1] = 0.0f;
#pragma unroll
        for (int m = 0; m < 8; ++m) sg.o[m][nt][0] = sg.o[m][nt][1] = sg.o[m][nt][2] = sg.o[m][nt][3] = 0.0f;
    }
}

// (a & b) | c in one instruction (two constants, which the compiler would take in two steps).
__device__ __forceinline__ uint32_t select_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Four pairs of codes of a word as binary16: z, 16 z, z, 16 z.  u in the mantissa of 2^10, or 16 u,
// less what the offset makes of it: exact.
__device__ __forceinline__ void pairs_of(uint32_t w, uint32_t (&p)[4])
{
    const uint32_t v = w >> 8;
    p[0] = select_or(w, 0x000f000fu, 0x64006400u);
    p[1] = select_or(w, 0x00f000f0u, 0x64006400u);
    p[2] = select_or(v, 0x000f000fu, 0x64006400u);
    p[3] = select_or(v, 0x00f000f0u, 0x64006400u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 z = __hadd2(*reinterpret_cast<const __half2 *>(&p[j]), __float2half2_rn(j & 1 ? -1152.0f : -1032.0f));
        p[j] = *reinterpret_cast<const uint32_t *>(&z);
    }
}

// MT tiles of 16 tokens in shared memory, from tile m0 on; `valid` of the tokens there are the
// sequence's, at least one of them in these tiles.
template <int NT, int TERMS_Q, int TERMS_P, int MT>
__device__ __forceinline__ void take_unit(Segment<NT, TERMS_Q> &sg, const uint8_t *b, int valid, int m0)
{
    constexpr int kLast = TERMS_Q - 1, kLastP = TERMS_P - 1;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float x[MT][NT][4];  // scores in units of fac
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const uint8_t *bh = b + (mt >> 1) * kHalfBlock;
        const int r0 = (m0 + (mt & 1)) * 16 + g, r1 = r0 + 8;
        const uint4 ka = *reinterpret_cast<const uint4 *>(bh + 64 * r0 + 16 * t);
        const uint4 kb = *reinterpret_cast<const uint4 *>(bh + 64 * r1 + 16 * t);
        const uint2 sa = *reinterpret_cast<const uint2 *>(bh + kKeyScales + 8 * r0);
        const uint2 sb = *reinterpret_cast<const uint2 *>(bh + kKeyScales + 8 * r1);
        const float2 sa0 = floats_of(sa.x), sa1 = floats_of(sa.y), sb0 = floats_of(sb.x), sb1 = floats_of(sb.y);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
        const float fa[4] = {sa0.x, sa0.y, sa1.x, sa1.y}, fb[4] = {sb0.x, sb0.y, sb1.x, sb1.y};
        float c[4][NT][4];
        uint32_t pa[4][4], pb[4][4];
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
            pairs_of(wa[gi], pa[gi]);
            pairs_of(wb[gi], pb[gi]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_f16_from(c[gi][nt], 0.0f, 0.0f, 0.0f, 0.0f, pa[gi][0], pb[gi][0], pa[gi][1], pb[gi][1], sg.qf[kLast][nt][gi][0], sg.qf[kLast][nt][gi][1]);
            }
        }
#pragma unroll
        for (int term = kLast; term >= 0; --term)  // the smaller products first
#pragma unroll
            for (int gi = 0; gi < 4; ++gi)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (term < kLast) mma_f16(c[gi][nt], pa[gi][0], pb[gi][0], pa[gi][1], pb[gi][1], sg.qf[term][nt][gi][0], sg.qf[term][nt][gi][1]);
                    mma_f16(c[gi][nt], pa[gi][2], pb[gi][2], pa[gi][3], pb[gi][3], sg.qf[term][nt][gi][2], sg.qf[term][nt][gi][3]);
                }
#pragma unroll
        for (int gi = 0; gi < 4; ++gi)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float f = j < 2 ? fa[gi] : fb[gi];
                    x[mt][nt][j] = gi == 0 ? f * c[gi][nt][j] : fmaf(f, c[gi][nt][j], x[mt][nt][j]);
                }
    }
    if (valid < MT * 16 + m0 * 16) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((m0 + mt) * 16 + g + (j >> 1) * 8 >= valid) x[mt][nt][j] = -INFINITY;
    }
    // the largest value scale of the sequence's tokens (positive binary16 values order as integers), as a power of two >= 1
    uint32_t mu = 0;
#pragma unroll
    for (int half = 0; half < (MT + 1) / 2; ++half) {
        const uint2 vs = *reinterpret_cast<const uint2 *>(b + half * kHalfBlock + kValueScales + 8 * lane);
        const int there = valid - half * kHalf - (lane & 30);  // of this lane's two tokens: what a page's last user left says nothing
        mu = __vmaxu2(mu, __vmaxu2(vs.x, vs.y) & (there >= 2 ? 0xffffffffu : there == 1 ? 0xffffu : 0u));
    }
    const uint32_t biggest = __reduce_max_sync(0xffffffffu, max(mu & 0xffffu, mu >> 16));
    const float up = static_cast<float>(max(0, static_cast<int>(biggest >> 10) - 14));
    // R moves only when a score is 2^4 above it, so that the lanes seldom have to agree on a new one
    bool moves = false;
    float m[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float y = fmaxf(x[0][nt][j], x[0][nt][2 + j]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) y = fmaxf(y, fmaxf(x[mt][nt][j], x[mt][nt][2 + j]));
            m[nt][j] = fmaf(y, sg.fac[nt][j], up);
            moves |= m[nt][j] > sg.top[nt][j] + kSlack;
        }
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y = m[nt][j];
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                y = fmaxf(y, sg.top[nt][j]);
                f[j] = exp2_approx(sg.top[nt][j] - y);
                sg.top[nt][j] = y;
                sg.weight[nt][j] *= f[j];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sg.o[k][nt][0] *= f[0];
                sg.o[k][nt][1] *= f[1];
                sg.o[k][nt][2] *= f[0];
                sg.o[k][nt][3] *= f[1];
            }
        }
    }
    float base[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) base[nt][j] = 15.0f - kSlack - sg.top[nt][j];
    const int pos = ((g + 2 * t) & 7) * 16;  // a tile's pairs t and t + 4 lie rotated by 2 t
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const uint8_t *bh = b + (mt >> 1) * kHalfBlock;
        const int pr = (m0 + (mt & 1)) * 8 + t;
        const uint4 va = *reinterpret_cast<const uint4 *>(bh + kValues + 128 * pr + pos);
        const uint4 vb = *reinterpret_cast<const uint4 *>(bh + kValues + 128 * (pr + 4) + pos);
        const uint4 ua = *reinterpret_cast<const uint4 *>(bh + kValueScales + 16 * pr);
        const uint4 ub = *reinterpret_cast<const uint4 *>(bh + kValueScales + 16 * (pr + 4));
        const uint32_t wa[4] = {va.x, va.y, va.z, va.w}, wb[4] = {vb.x, vb.y, vb.z, vb.w};
        const uint32_t fa[4] = {ua.x, ua.y, ua.z, ua.w}, fb[4] = {ub.x, ub.y, ub.z, ub.w};
        __half2 b0[TERMS_P][NT], b1[TERMS_P][NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float e[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) e[j] = exp2_approx(fmaf(x[mt][nt][j], sg.fac[nt][j & 1], base[nt][j & 1]));
            sg.weight[nt][0] += e[0] + e[2];
            sg.weight[nt][1] += e[1] + e[3];
            const __half2 c0 = __floats2half2_rn(e[0], e[1]), c1 = __floats2half2_rn(e[2], e[3]);
            b0[0][nt] = halves(transpose8(*reinterpret_cast<const uint32_t *>(&c0)));
            b1[0][nt] = halves(transpose8(*reinterpret_cast<const uint32_t *>(&c1)));
            if (TERMS_P == 2) {
                b0[kLastP][nt] = halves(transpose8(rest_of(make_float2(e[0], e[1]), c0)));
                b1[kLastP][nt] = halves(transpose8(rest_of(make_float2(e[2], e[3]), c1)));
            }
        }
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
            uint32_t pa[4], pb[4];
            pairs_of(wa[gi], pa);
            pairs_of(wb[gi], pb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const __half2 s0 = halves(fa[gi]), s1 = halves(fb[gi]);
                const __half2 e0 = __hmul2(b0[0][nt], s0), e1 = __hmul2(b1[0][nt], s1);
                if (TERMS_P == 2) {  // what the product's rounding left (a fused multiply-add has it), and the second value's product
                    const __half2 r0 = __hfma2(b0[kLastP][nt], s0, __hfma2(b0[0][nt], s0, __hneg2(e0)));
                    const __half2 r1 = __hfma2(b1[kLastP][nt], s1, __hfma2(b1[0][nt], s1, __hneg2(e1)));
                    const uint32_t v0 = *reinterpret_cast<const uint32_t *>(&r0), v1 = *reinterpret_cast<const uint32_t *>(&r1);
                    mma_f16(sg.o[2 * gi][nt], pa[0], pa[1], pb[0], pb[1], v0, v1);
                    mma_f16(sg.o[2 * gi + 1][nt], pa[2], pa[3], pb[2], pb[3], v0, v1);
                }
                const uint32_t u0 = *reinterpret_cast<const uint32_t *>(&e0), u1 = *reinterpret_cast<const uint32_t *>(&e1);
                mma_f16(sg.o[2 * gi][nt], pa[0], pa[1], pb[0], pb[1], u0, u1);
                mma_f16(sg.o[2 * gi + 1][nt], pa[2], pa[3], pb[2], pb[3], u0, u1);
            }
        }
    }
}

// Four consecutive values of a row of y, rounded once.
__device__ __forceinline__ void store4(void *y, int64_t at, int dtype, const float (&v)[4])
{
    if (dtype == STQ_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + at) = make_float4(v[0], v[1], v[2], v[3]);
        return;
    }
    uint2 w;
    if (dtype == STQ_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + at) = w;
}

// The segment's result: y itself where the warp had all of it (part == nullptr), else a partial.
template <int NT, int TERMS_Q>
__device__ __forceinline__ void end_segment(const AttnArgs &a, Segment<NT, TERMS_Q> &sg, int seq, int h0, int nh, float *part)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float l = sg.weight[nt][j];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int h = nt * 8 + 2 * t + j;
            if (h >= nh) continue;
            const float f = part ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;  // no weight at all: every page absent
#pragma unroll
            for (int gi = 0; gi < 4; ++gi) {
                // rows 8 to 15 of a tile are sums of 16 z
                const float v[4] = {sg.o[2 * gi][nt][j] * f, sg.o[2 * gi][nt][2 + j] * (0.0625f * f),
                                    sg.o[2 * gi + 1][nt][j] * f, sg.o[2 * gi + 1][nt][2 + j] * (0.0625f * f)};
                if (part) *reinterpret_cast<float4 *>(part + h * kD + 32 * gi + 4 * g) = make_float4(v[0], v[1], v[2], v[3]);
                else store4(a.y, (static_cast<int64_t>(seq) * a.heads + h0 + h) * kD + 32 * gi + 4 * g, a.dtype, v);
            }
            if (part && g == 0) *reinterpret_cast<float2 *>(part + 8 * NT * kD + 2 * h) = make_float2(sg.top[nt][j], l);
        }
}

constexpr int attn_ctas(int nt, bool wide) { return nt == 1 && !wide ? 3 : 2; }  // CTAs on an SM: what their registers allow (168, or 255)

template <int NT, int TERMS_Q, int TERMS_P>
__global__ void __launch_bounds__(kWarps * 32, attn_ctas(NT, TERMS_Q == 2)) attn_decode_kernel(const AttnArgs a)
{
    extern __shared__ __align__(128) uint8_t raw_smem[];
    AttnSmem &sm = *reinterpret_cast<AttnSmem *>(raw_smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    launch_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
            const int len = a.seq_len[i];
            if (len < 0 || len > static_cast<long long>(a.max_pages) * kPage) atomicOr(a.c.err, kErrIndex);
        }
    const Shares s = shares_of(a);
    // neighbouring shares go to different SMs, so that a launch with few units spreads
    const int me = warp * gridDim.x + blockIdx.x;
    if (me >= s.warps || s.units == 0) return;
    const long long lo = s.begin(me), hi = s.begin(me + 1);
    const uint32_t bar0 = smem_addr(&sm.full[warp][0]), st0 = smem_addr(&sm.stage[warp][0][0]);
    if (lane == 0) {
        for (int k = 0; k < kStagesW; ++k) barrier_init(bar0 + 8 * k, 1);
        fence_barrier_init();
    }
    __syncwarp();

    Walk w = place_of(a, s, lo);
    Feed feed;
    feed.w = w;
    feed.left = static_cast<int>(hi - lo);
    feed.first = feed.end = 0;
    feed.ids = 0;
    int issued = 0, taken = 0;  // units of this warp, by number
    uint32_t absent = 0;        // bit k: stage k stands for a half outside the cache
    const auto issue = [&]() {
        int head = 0, half = 0;
        const int id = feed_next(a, s, feed, &head, &half);
        if (id == -1) return;
        const int k = issued % kStagesW;
        if (id >= 0) {
            absent &= ~(1u << k);
            if (lane == 0) {
                const uint32_t bytes = s.shift == 2 ? kHalfBlock : kUnitBytes;
                barrier_expect(bar0 + 8 * k, bytes + (me == 0 && issued == 0 ? a.waits.stall_tx : 0));
                bulk_copy(st0 + k * kUnitBytes, a.c.block(id, head) + half * kHalfBlock, bytes, bar0 + 8 * k);
            }
        } else {
            absent |= 1u << k;
            if (lane == 0) {
                atomicOr(a.c.err, kErrIndex);
                barrier_arrive(bar0 + 8 * k);
            }
        }
        ++issued;
    };
    for (int k = 0; k < kStagesW; ++k) issue();

    bool dead = false;  // a copy did not arrive
    int left = static_cast<int>(hi - lo);
    for (bool first = true; left > 0 && !dead; first = false) {
        const int u0 = w.unit, u1 = left < w.units - u0 ? u0 + left : w.units;
        const int len = a.seq_len[w.seq];
        const int kvh = w.sub / a.blocks, hb = w.sub - kvh * a.blocks;
        const int h0 = kvh * a.group + hb * 8 * NT, nh = min(8 * NT, a.group - hb * 8 * NT);
        Segment<NT, TERMS_Q> sg;
        begin_segment(a, sg, w.seq, h0, nh);
        for (int u = u0; u < u1; ++u) {
            const int k = taken % kStagesW;
            if (!__all_sync(0xffffffffu, barrier_wait(bar0 + 8 * k, taken / kStagesW & 1, a.waits.wait_ns))) {
                if (lane == 0) atomicOr(a.c.err, kErrTimeout);
                dead = true;
                break;
            }
            if (!(absent >> k & 1)) {
                const uint8_t *page = sm.stage[warp][k];
                if (s.shift == 2) {
                    if (u * 16 < len) take_unit<NT, TERMS_Q, TERMS_P, 1>(sg, page, len - (u >> 1) * kHalf, u & 1);
                } else if (u * kPage < len) {
                    take_unit<NT, TERMS_Q, TERMS_P, 4>(sg, page, len - u * kPage, 0);
                }
            }
            __syncwarp();
            ++taken;
            issue();
        }
        if (dead) break;
        const bool whole = u0 == 0 && u1 == w.units;
        end_segment(a, sg, w.seq, h0, nh, whole ? nullptr : a.part + (static_cast<size_t>(me) * 2 + (first ? 0 : 1)) * part_floats(NT));
        left -= u1 - u0;
        next_segment(a, s, w);
    }
    // after a wait that gave up, let the copies in flight land (bounded) before the memory is given back
    if (dead)
        for (; taken < issued; ++taken) barrier_wait(bar0 + 8 * (taken % kStagesW), taken / kStagesW & 1, a.waits.wait_ns);
}

// Joins the partial sums of one (sequence, query head) in the order of the warps
// that left them, and writes the zeros of sequences without tokens.  First the
// factor of every partial, one a thread at a time, then the sums: a warp takes every
// so many-th partial, a lane four dims, and the warps are added in order.
constexpr int kMostJoinWarps = 16;
constexpr int join_floats(int join_warps, int warps) { return join_warps * (kD + 2) + warps; }

template <int NT>
__global__ void join_kernel(const AttnArgs a)
{
    extern __shared__ __align__(16) float join_smem[];  // join_floats of them
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float *acc = join_smem, *red = acc + warps * kD, *red2 = red + warps, *factor = red2 + warps;
    const int seq = blockIdx.x / a.heads, head = blockIdx.x - seq * a.heads;
    const int kvh = head / a.group, in = head - kvh * a.group, hb = in / (8 * NT), h = in - hb * 8 * NT;
    const Shares s = shares_of(a);
    const int len = a.seq_len[seq];
    const long long units = static_cast<long long>(pages_of(a, seq)) << s.shift;
    const long long u0 = (pages_before(a, seq) * s.subs << s.shift) + (kvh * a.blocks + hb) * units, u1 = u0 + units - 1;
    wait_previous_grid();  // in every CTA, so that the end of this grid is the end of both
    if (len < 0 || len > static_cast<long long>(a.max_pages) * kPage) return;
    const int64_t at = (static_cast<int64_t>(seq) * a.heads + head) * kD;
    if (len == 0) {
        for (int d = threadIdx.x; d < kD; d += blockDim.x) store_from_float(a.y, at + d, a.dtype, 0.0f);
        return;
    }
    const int w0 = s.owner(u0), count = s.owner(u1) - w0 + 1;
    if (count == 1) return;  // one warp had all of it
    // the segment is the last of its first warp's share unless that share begins in it, and the first of the others'
    const int slot0 = s.begin(w0) >= u0 ? 0 : 1;
    const auto part = [&](int i) { return a.part + (static_cast<size_t>(w0 + i) * 2 + (i == 0 ? slot0 : 0)) * part_floats(NT); };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        const float r = part(i)[8 * NT * kD + 2 * h];
        factor[i] = r;
        top = fmaxf(top, r);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) red[warp] = top;
    __syncthreads();
    for (int v = 0; v < warps; ++v) top = fmaxf(top, red[v]);
    float l = 0.0f;
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        const float f = factor[i] == -INFINITY ? 0.0f : exp2_approx(factor[i] - top);  // -inf: every page of it absent
        factor[i] = f;
        l += f * part(i)[8 * NT * kD + 2 * h + 1];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    if (lane == 0) red2[warp] = l;
    __syncthreads();
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int i = warp; i < count; i += warps) {
        const float4 v = *reinterpret_cast<const float4 *>(part(i) + h * kD + 4 * lane);
        const float f = factor[i];
        y = make_float4(fmaf(v.x, f, y.x), fmaf(v.y, f, y.y), fmaf(v.z, f, y.z), fmaf(v.w, f, y.w));
    }
    *reinterpret_cast<float4 *>(acc + warp * kD + 4 * lane) = y;
    __syncthreads();
    l = 0.0f;
    for (int v = 0; v < warps; ++v) l += red2[v];
    for (int d = threadIdx.x; d < kD; d += blockDim.x) {
        float sum = 0.0f;
        for (int v = 0; v < warps; ++v) sum += acc[v * kD + d];
        store_from_float(a.y, at + d, a.dtype, l == 0.0f ? 0.0f : sum / l);
    }
}

CacheView view(const stq_cache *c) { return CacheView{c->d_data, c->pages, c->heads, c->d_err}; }

Rows rows(const stq_rows *r) { return Rows{r->data, r->token_stride, r->head_stride}; }

// Blocks of 16 query heads where a key head has more than 8, else of 8 (and of fp32 rows, whose second values take the registers).
int attn_nt(int group, bool wide) { return group > 8 && !wide ? 2 : 1; }

// Warps of one attn_decode launch: all that the SMs hold.
int attn_warps(const stq_cache *c, int nt, bool wide) { return c->sms * kWarps * attn_ctas(nt, wide); }

template <int NT, int TERMS_Q, int TERMS_P>
cudaError_t launch_attn(const AttnArgs &a, cudaStream_t s)
{
    const int smem = static_cast<int>(sizeof(AttnSmem));
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<NT, TERMS_Q, TERMS_P>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attn_decode_kernel<NT, TERMS_Q, TERMS_P><<<a.warps / kWarps, kWarps * 32, smem, s>>>(a);
    count_launch();
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // a warp of the join for every four partials that an even batch leaves a segment
    const long long partials = a.warps / std::max(1ll, static_cast<long long>(a.n) * a.c.heads * a.blocks);
    int join_warps = 2;
    while (join_warps < kMostJoinWarps && join_warps * 4 < partials) join_warps *= 2;
    const int join_smem = static_cast<int>(join_floats(join_warps, a.warps) * sizeof(float));
    return launch_behind(join_kernel<NT>, dim3(static_cast<unsigned>(a.n) * a.heads), join_warps * 32, join_smem, s, a);
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
    const unsigned ctas = static_cast<unsigned>((static_cast<long long>(n) * c->heads + 15) / 16);
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
    // (fp32 rows take no more than this: fewer warps, or smaller partials)
    const int nt = stq::attn_nt(num_heads / c->heads, false);
    *bytes = static_cast<size_t>(stq::attn_warps(c, nt, false)) * 2 * stq::part_floats(nt) * sizeof(float);
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
    if (max_pages < 0 || max_pages > stq::kMostPages) return fail_status(STQ_ERR_ARG, "max_pages = %d", max_pages);
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
    const bool wide = dtype == STQ_F32;
    const int nt = stq::attn_nt(a.group, wide);
    a.blocks = (a.group + 8 * nt - 1) / (8 * nt);
    a.dtype = dtype;
    a.q = stq::rows(q);
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    a.y = y;
    a.part = static_cast<float *>(workspace);
    a.waits = stq::waits();
    a.warps = stq::attn_warps(c, nt, wide);
    const auto launch = wide                 ? stq::launch_attn<1, 2, 2>
                        : dtype == STQ_F16 ? (nt == 2 ? stq::launch_attn<2, 1, 2> : stq::launch_attn<1, 1, 2>)
                                           : (nt == 2 ? stq::launch_attn<2, 1, 1> : stq::launch_attn<1, 1, 1>);
    const cudaError_t e = launch(a, static_cast<cudaStream_t>(stream));
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
