// stq_chunk.cu -- the gated delta rule over whole prompts in chunks of 64 tokens (sm_100a).
//
// Within a chunk that starts from the state X_0, with R_ti the product of the decays
// behind token i up to t (R_t the product from the chunk's start, D_i = R_63,i) and
//   u_t = b_t (v_t - a_t X_{t-1}^T k_t),   X_t = R_t X_0 + sum_{i <= t} R_ti k_i u_i^T,
// the rows u solve a triangular system, and all that remains is products:
//   U   = T diag(b) (V - diag(R) K X_0),   T = (I + A)^-1,  A_ti = b_t R_ti k_t.k_i  (i < t)
//   Y   = diag(R) Q X_0 + P U,             P_ti = R_ti q_t.k_i                        (i <= t)
//   X_C = R_63 X_0 + K^T diag(D) U.
// T and P do not depend on the state: prepare_kernel computes them for all chunks and
// heads at once.  chunk_kernel then walks over a prompt's chunks, one CTA a head.
//
// Precision.  The state has to come out as the recurrence in fp32 gives it.  k is a
// 16-bit value, exact in tf32 (11 bits); X_0, V - K X_0, T and D U are fp32 values
// and enter the tensor core as two tf32 terms, x = hi + lo, 2^-21 of x left: 2 products
// against k, 3 of the 4 for T times a vector.  Y is rounded to 16 bits: in bf16 one term each
// of R Q, X_0, P and U, rounded to nearest (2^-11), is below that.  In fp16 it would make the
// error 1.8 times that of the output's own rounding, nearly all of it by P and U, which enter as
// two terms (670 us in place of 624 on two prompts of 8192 tokens; what is left is 1.1 times).
// Sums are fp32.
//
// What is no number stays none.  A NaN in q is one in its row of P; one in X_0, v or the decays is one in a whole column of
// V - diag(R) K X_0 (products with zeros keep it), so of U, Y and X_C; one in k or b in rows of T, so in U.  So P and U
// alone take care to keep it (where they are two terms, the second does).  Y has it from the chunk's first token on, since P's
// zeros above the diagonal meet U's rows.
#include <cmath>

#include "stq_host.h"
#include "stq_map.h"
#include "stq_tc.h"

namespace stq {
namespace {

constexpr int kC = kPromptChunk;  // tokens of a chunk

// What prepare_kernel leaves for one (chunk, head): T diag(b) and P, the ten 16 x 16 blocks on and
// below the diagonal each (block (i, j) at i (i + 1) / 2 + j), then R_t and D_t.
constexpr int kBlockFloats = 256, kTriangle = 10 * kBlockFloats;
struct Prepared {
    float t[kTriangle], p[kTriangle], r[kC], d[kC];
};
static_assert(sizeof(Prepared) == kPreparedBytes, "workspace size");

// Chunks are numbered through all entries in their order, whatever rows these have: there are no more than
// prompt_chunks(n, total) where ranges do not overlap.
__device__ __forceinline__ int chunks_of(const PromptIO &io, int e)
{
    const int len = io.span.length(e);
    return len > 0 ? (len + kC - 1) / kC : 0;
}

__device__ __forceinline__ Prepared *prepared(const PromptIO &io, int H, long long chunk, int h)
{
    return reinterpret_cast<Prepared *>(io.workspace) + chunk * H + h;
}

__device__ __forceinline__ int block_of(int i, int j) { return (i * (i + 1) / 2 + j) * kBlockFloats; }

// x rounded to tf32, to nearest; what is left of it.  Arithmetic's NaN, 0x7fffffff, is carried over into minus zero: it lives on in
// the rest, so where no rest follows something else has to keep it.
__device__ __forceinline__ float tf32_hi(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

// ... and a NaN kept (by cvt.rna.tf32 the walk took 8 % longer, at half as many places).
__device__ __forceinline__ float tf32_hi_or_nan(float x) { return isnan(x) ? x : tf32_hi(x); }

// The same by cutting, for a first term whose rest follows: what the tensor core cuts off the rest is 2^-21 of x.
__device__ __forceinline__ float tf32_cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

// Whether P and U enter Y as two terms.
template <bool BF16>
constexpr bool kTwoTerms = !BF16;

// Two neighbouring registers of a row as a pair, for packed arithmetic.
__device__ __forceinline__ float2 pair_at(const uint32_t *x) { return make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])); }
__device__ __forceinline__ void put_pair(uint32_t *x, float2 y)
{
    x[0] = __float_as_uint(y.x);
    x[1] = __float_as_uint(y.y);
}
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.0f, -1.0f), a); }

// ---------------------------------------------------------------- T and P of every chunk

constexpr int kPrepThreads = 128;
constexpr int kPrepRow = kD + 8;  // 16-bit values of a row in shared memory: eight rows on eight different banks

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
}

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// 16 bytes to shared memory, asynchronously; zeros where `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct PrepSmem {
    union {
        struct {
            uint16_t k[kC][kPrepRow], q[kC][kPrepRow];
        } in;
        struct {
            float a[kC][kC + 4], t[kC][kC + 4];
        } m;
    };
    float w[3][16][20];
    float near[8][8][8];         // R_ti within group b: [b][t][i]
    float mid[8][8];             // products of the groups strictly between two
    float pre[kC], suf[kC];      // products from the token's group's start through it, and behind it to the group's end
    float alpha[kC], beta[kC];
    int item[3];
};

// The entry and the chunk of it that `chunk` of all is; the whole warp calls it.  False: there are not so many.
__device__ __forceinline__ bool find_chunk(const PromptIO &io, int chunk, int *entry, int *at)
{
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int first = 0; first < io.n; first += 32) {
        const int mine = first + lane < io.n ? chunks_of(io, first + lane) : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + upto > chunk);
        if (past) {
            const int who = __ffs(past) - 1;
            *entry = first + who;
            *at = static_cast<int>(chunk - base) - __shfl_sync(0xffffffffu, upto - mine, who);
            return true;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], float b0, float b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])), "r"(__float_as_uint(a[3])),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// d += a b of fp32 16 x 16 and 16 x 8 blocks (rows of `pitch` floats), each factor in two tf32 terms, three products.
__device__ __forceinline__ void block_product(float (&d)[4], const float *a, const float *b, int pitch_a, int pitch_b)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int k = 0; k < 16; k += 8) {
        float x[4], xh[4], xl[4], y[2], yh[2], yl[2];
        x[0] = a[g * pitch_a + k + t4];
        x[1] = a[(g + 8) * pitch_a + k + t4];
        x[2] = a[g * pitch_a + k + t4 + 4];
        x[3] = a[(g + 8) * pitch_a + k + t4 + 4];
        y[0] = b[(k + t4) * pitch_b + g];
        y[1] = b[(k + t4 + 4) * pitch_b + g];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xh[i] = tf32_hi(x[i]);
            xl[i] = x[i] - xh[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            yh[i] = tf32_hi(y[i]);
            yl[i] = y[i] - yh[i];
        }
        mma_tf32(d, xl, yh[0], yh[1]);
        mma_tf32(d, xh, yl[0], yl[1]);
        mma_tf32(d, xh, yh[0], yh[1]);
    }
}

// The blocks of T at distance D below the diagonal, T_ij = -T_ii sum_{j <= k < i} A_ik T_kj, in halves of
// eight columns dealt to the warps.
template <int D>
__device__ __forceinline__ void below(PrepSmem &s)
{
    constexpr int kPitch = kC + 4, kPitchW = 20;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int x = 0; x < 2 * (4 - D); x += 4) {
        const int j = (x + warp) >> 1, c = (x + warp & 1) * 8, i = j + D;
        if (j >= 4 - D) continue;
        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < D; ++k) block_product(w, &s.m.a[16 * i][16 * (j + k)], &s.m.t[16 * (j + k)][16 * j + c], kPitch, kPitch);
        *reinterpret_cast<float2 *>(&s.w[j][g][c + 2 * t4]) = make_float2(w[0], w[1]);
        *reinterpret_cast<float2 *>(&s.w[j][g + 8][c + 2 * t4]) = make_float2(w[2], w[3]);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2 * (4 - D); x += 4) {
        const int j = (x + warp) >> 1, c = (x + warp & 1) * 8, i = j + D;
        if (j >= 4 - D) continue;
        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        block_product(w, &s.m.t[16 * i][16 * i], &s.w[j][0][c], kPitch, kPitchW);
        *reinterpret_cast<float2 *>(&s.m.t[16 * i + g][16 * j + c + 2 * t4]) = make_float2(-w[0], -w[1]);
        *reinterpret_cast<float2 *>(&s.m.t[16 * i + g + 8][16 * j + c + 2 * t4]) = make_float2(-w[2], -w[3]);
    }
    __syncthreads();
}

// Bound by the latencies of its steps, five CTAs on an SM hiding each other's, and by
// shared-memory accesses.  The inverse: its diagonal blocks of 16 by substitution, a thread a
// column, the others by block products in three tf32 terms (in fp32 on the other pipe they
// took four times the accesses).  R_ti is put together from products within groups of eight
// tokens and of whole groups between them.  8832 chunks and heads: 143 us, 42 % of the issue
// slots, 35 % of DRAM.
template <bool BF16>
__global__ void __launch_bounds__(kPrepThreads, 5) prepare_kernel(PromptIO io, int H)
{
    extern __shared__ __align__(16) uint8_t raw_smem[];
    PrepSmem &s = *reinterpret_cast<PrepSmem *>(raw_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int h = blockIdx.y;
    launch_dependents();
    if (warp == 0) {
        int e = 0, at = 0;
        const bool found = find_chunk(io, blockIdx.x, &e, &at);
        if (lane == 0) {
            s.item[0] = found ? e : -1;
            s.item[1] = at;
        }
    }
    __syncthreads();
    const int e = s.item[0];
    if (e < 0) {
        wait_previous_grid();
        return;
    }
    const long long row0 = io.span.seq_start[e] + static_cast<long long>(s.item[1]) * kC;
    const int m = min(kC, io.span.length(e) - s.item[1] * kC);
    Prepared *out = prepared(io, H, blockIdx.x, h);
#pragma unroll
    for (int i = 0; i < kC * kD / 8 / kPrepThreads; ++i) {  // 16 threads a row
        const int t = tid / 16 + 8 * i, d = tid % 16 * 8;
        const long long row = row0 + min(t, m - 1);
        copy16(smem_addr(&s.in.k[t][d]), static_cast<const uint16_t *>(io.k.data) + row * io.k.token_stride + h * io.k.head_stride + d, t < m);
        copy16(smem_addr(&s.in.q[t][d]), static_cast<const uint16_t *>(io.q.data) + row * io.q.token_stride + h * io.q.head_stride + d, t < m);
    }
    if (tid < kC) {
        s.alpha[tid] = 1.0f;
        s.beta[tid] = 0.0f;
        if (tid < m) {
            copy4(smem_addr(&s.alpha[tid]), io.alpha + (row0 + tid) * H + h);
            copy4(smem_addr(&s.beta[tid]), io.beta + (row0 + tid) * H + h);
        }
    }
    copies_wait();
    __syncthreads();
    // products of decays, never quotients: a decay may be zero
    if (tid < kC) {
        const int b = tid >> 3, i = tid & 7;
        float r = 1.0f;
#pragma unroll
        for (int t = 0; t < 8; ++t) {  // column i of the group
            r = t > i ? r * s.alpha[8 * b + t] : t == i ? 1.0f : 0.0f;
            s.near[b][t][i] = r;
        }
        s.suf[tid] = r;
        r = 1.0f;
#pragma unroll
        for (int t = 0; t < 8; ++t) r = t <= i ? r * s.alpha[8 * b + t] : r;
        s.pre[tid] = r;
    }
    __syncthreads();
    if (tid < 64) {
        const int hi = tid >> 3, lo = tid & 7;
        float r = 1.0f, before = 1.0f, behind = 1.0f;
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const float all = s.pre[8 * b + 7];
            if (b > lo && b < hi) r *= all;
            if (b < hi) before *= all;   // of this thread's token, whose group is hi
            if (b > hi) behind *= all;
        }
        s.mid[hi][lo] = r;
        out->r[tid] = before * s.pre[tid];
        out->d[tid] = s.suf[tid] * behind;
    }
    // k k^T and q k^T, rows 16 warp .. + 15, columns up to the diagonal
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[nt][j] = qk[nt][j] = 0.0f;
    const uint32_t k0 = smem_addr(&s.in.k[0][0]), q0 = smem_addr(&s.in.q[0][0]);
    const uint32_t arow = (16 * warp + (lane & 15)) * (kPrepRow * 2) + (lane >> 4) * 16;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
        uint32_t ka[4], qa[4];
        load_matrices(ka, k0 + arow + ks * 32);
        load_matrices(qa, q0 + arow + ks * 32);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            if (np > warp) continue;
            uint32_t b[4];  // rows 16 np .. + 7 and + 8 .. + 15, both halves of the step
            load_matrices(b, k0 + (16 * np + (lane & 7) + (lane >> 4) * 8) * (kPrepRow * 2) + ks * 32 + (lane >> 3 & 1) * 16);
            mma16<BF16>(kk[2 * np], ka, b[0], b[1]);
            mma16<BF16>(kk[2 * np + 1], ka, b[2], b[3]);
            mma16<BF16>(qk[2 * np], qa, b[0], b[1]);
            mma16<BF16>(qk[2 * np + 1], qa, b[2], b[3]);
        }
    }
    __syncthreads();  // k and q are read, R's parts are there
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        if (nt / 2 > warp) continue;
        const float2 suf = *reinterpret_cast<const float2 *>(&s.suf[8 * nt + 2 * t4]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = 16 * warp + g + 8 * half, i = 8 * nt + 2 * t4, b = 2 * warp + half;
            float2 r = make_float2(0.0f, 0.0f);
            if (b == nt) {
                r = *reinterpret_cast<const float2 *>(&s.near[b][g][2 * t4]);
            } else if (b > nt) {
                const float through = s.mid[b][nt] * s.pre[t];
                r = make_float2(suf.x * through, suf.y * through);
            }
            const float beta = s.beta[t];
            const float2 a = make_float2(i < t ? beta * (r.x * kk[nt][2 * half]) : 0.0f, i + 1 < t ? beta * (r.y * kk[nt][2 * half + 1]) : 0.0f);
            float2 p = make_float2(i <= t ? r.x * qk[nt][2 * half] : 0.0f, i + 1 <= t ? r.y * qk[nt][2 * half + 1] : 0.0f);
            if (!kTwoTerms<BF16>) p = make_float2(tf32_hi_or_nan(p.x), tf32_hi_or_nan(p.y));
            *reinterpret_cast<float2 *>(&s.m.a[t][i]) = a;
            *reinterpret_cast<float2 *>(out->p + block_of(warp, nt / 2) + (t & 15) * 16 + (i & 15)) = p;
        }
    }
    __syncthreads();
    // the inverses of the diagonal blocks
    if (tid < kC) {
        const int b = tid >> 4, c = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = i == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) y = fmaf(-s.m.a[16 * b + i][16 * b + j], x[j], y);
            x[i] = y;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) s.m.t[16 * b + i][16 * b + c] = x[i];
    }
    __syncthreads();
    below<1>(s);
    below<2>(s);
    below<3>(s);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) {
            const int t = 16 * i + (tid >> 3), col = 16 * j + (tid & 7) * 2;
            const float2 y = *reinterpret_cast<const float2 *>(&s.m.t[t][col]);
            *reinterpret_cast<float2 *>(out->t + block_of(i, j) + 2 * tid) = make_float2(y.x * s.beta[col], y.y * s.beta[col + 1]);
        }
    wait_previous_grid();  // nothing here needs the states that it unpacks, but what comes behind this grid does
}

// ---------------------------------------------------------------- the walk over the chunks
//
// Transposed throughout: lane j of tensor memory is column j of the state (and of V, U
// and Y), so X_0^T, (V - K X_0)^T, U^T are the products' A operands straight from
// tensor memory, and what threads do between the products is their own row's.  B operands
// (K, Q, K^T, T, P, as fp32 in 128-byte swizzled rows) are written to shared memory by six
// warps that run ahead.  Columns of tensor memory:
//     0  X^T, the sum that the chunk's update goes onto, scaled by R_63 beforehand
//   128  X_0^T hi; then (T (V - R K X_0))^T in two parts; then (D U)^T hi | lo
//   256  X_0^T lo; then (V - R K X_0)^T hi | lo; then U^T lo where it is needed
//   384  (K X_0)^T; then U^T hi
//   448  (diag(R) Q X_0)^T, then Y^T
// A product of 8 deep takes about 64 cycles at 128 columns and 45 at 64, for its A operand's
// sake, so K and Q stand under each other for the hi term, and T's two terms for R's.
// Bound by the chain of all but Y's with what stands between them: 3.8 us a chunk in bf16, 4.2 in
// fp16 (2 prompts of 8192 tokens with 32 heads 540 us); 24 prompts to 1500 tokens in bf16 285 us,
// tensor pipe 45 % busy.

constexpr int kGroupThreads = 256;  // warps 0-7: two for each quarter of the lanes, half of the columns each
constexpr int kFeedThreads = 128;   // warps 8-11; warp 12 issues the products
constexpr int kSideThreads = 64;    // warps 13 and 14
constexpr int kChunkThreads = 512;  // four warpgroups; warp 15 only hands its registers over
// registers a thread: 128 at launch and in warps 8-11, then 152 in warps 0-7 and 80 in the last four
// (2 * 152 + 128 + 80 = 4 * 128); where a branch spills instead, the walk takes up to twice as long
constexpr int kGroupRegs = 152, kOtherRegs = 80;
constexpr uint32_t kColX = 0, kColHi = 128, kColLo = 256, kColK = 384, kColY = 448;
// U's second term, of tokens 32 half .. + 31: the parts of X_0^T lo that are written last
constexpr __device__ uint32_t rest_column(int half) { return kColLo + 64 * half + 32; }

// P's second term, on and below the diagonal: 64 rows of the first 32 tokens, the last 32 rows of the others.
constexpr int kRestBlock = kC * 128, kRestBytes = kRestBlock + kC / 2 * 128;
template <bool TWO_TERMS>
struct __align__(1024) Rest {
    uint8_t p_rest[kRestBytes];
};
template <>
struct __align__(1024) Rest<false> {
    static constexpr uint8_t *p_rest = nullptr;
};

template <bool BF16>
struct __align__(1024) ChunkSmem : Rest<kTwoTerms<BF16>> {
    uint8_t kq[2 * kC * kD * 4];  // 4 blocks of 32 dims: 128 rows of 128 bytes, K's and Q's
    uint8_t kt[kC * kD * 4];      // 2 blocks of 32 tokens: 128 rows
    uint8_t t[2 * kC * kC * 4];   // 2 blocks of 32 tokens: 128 rows, T's hi and lo
    uint8_t p[kC * kC * 4];       // 2 blocks of 32 tokens: 64 rows
    uint8_t raw_k[2][kC * 128], raw_q[2][kC * 128], v[2][kC * 128];  // as they come: 64 dims, 128-byte swizzled rows
    float tp_raw[2 * kTriangle];
    struct {
        float r[kC], d[kC];
    } rd[2];
    unsigned long long kq_raw, kq_full, kq_empty, kt_full, kt_empty, tp_raw_full, t_full, t_empty, p_full, p_empty, v_full, v_empty;
    unsigned long long x_full[2], k_done, r_full, u_done, u_full, y_done, x_done, drained;
    unsigned long long before;  // chunks of the entries before this one
    uint32_t tmem;
    int item;
};
static_assert(sizeof(ChunkSmem<false>) + 1024 <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void tc_mma_tf32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

// Byte of element (row, col) of a B operand with `rows` rows: blocks of 32 columns, 16-byte pieces exchanged by row.
__device__ __forceinline__ uint32_t swizzled(int rows, int row, int col)
{
    return static_cast<uint32_t>((col >> 5) * rows * 128 + row * 128 + (((col >> 2 & 7) ^ (row & 7)) << 4) + (col & 3) * 4);
}

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w)
{
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <bool BF16>
__device__ __forceinline__ float widen1(uint16_t w)
{
    if (BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
    return __half2float(*reinterpret_cast<const __half *>(&w));
}

template <bool BF16>
__device__ __forceinline__ uint16_t narrow1(float x)
{
    if (BF16) {
        const __nv_bfloat16 h = __float2bfloat16_rn(x);
        return *reinterpret_cast<const uint16_t *>(&h);
    }
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t *>(&h);
}

template <bool BF16>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                                                              const __grid_constant__ CUtensorMap v_map, PoolView pool, PromptIO io)
{
    extern __shared__ uint8_t raw_smem[];
    ChunkSmem<BF16> &sm = *reinterpret_cast<ChunkSmem<BF16> *>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, tid = threadIdx.x;
    const int H = pool.H, h = blockIdx.x % H;
    // long prompts first: the entry of this rank by length (all CTAs agree on the order); in their order where
    // there are too many to rank
    if (io.n <= kFeedThreads) {
        if (tid < io.n) {
            const int len = io.span.length(tid);
            int rank = 0;
            for (int i = 0; i < io.n; ++i) {
                const int other = io.span.length(i);
                rank += other > len || (other == len && i < tid);
            }
            if (rank == static_cast<int>(blockIdx.x) / H) sm.item = tid;
        }
    } else if (tid == 0) {
        sm.item = blockIdx.x / H;
    }
    if (tid == kFeedThreads) sm.before = 0;
    __syncthreads();
    launch_dependents();
    const int e = __shfl_sync(0xffffffffu, sm.item, 0);
    const int req = io.req_idx[e], slot = io.slot_idx[e];
    if (req < 0 || req >= pool.R || slot < 0 || slot >= pool.S) {
        wait_previous_grid();
        if (tid == 0) atomicOr(pool.err, kErrIndex);
        return;
    }
    int len = io.span.length(e);
    if (len < 0) {
        if (tid == 0) atomicOr(pool.err, kErrIndex);
        len = 0;
    }
    const bool fresh = io.span.is_fresh(e);
    float *state = io.state + (static_cast<size_t>(e) * H + h) * kD * kD;
    if (len == 0) {
        wait_previous_grid();
        if (fresh)
            for (int i = tid; i < kD * kD / 4; i += kChunkThreads) reinterpret_cast<float4 *>(state)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        return;
    }
    const int chunks = (len + kC - 1) / kC;
    {
        unsigned long long before = 0;
        for (int i = tid; i < e; i += kChunkThreads) before += chunks_of(io, i);
        if (before > 0) atomicAdd(&sm.before, before);
    }
    const long long first = io.span.seq_start[e];
    if (warp == 12) {
        if (lane == 0) {
            const auto init = [](unsigned long long &b, uint32_t count) { barrier_init(smem_addr(&b), count); };
            init(sm.kq_full, kFeedThreads);
            init(sm.kq_empty, 1);
            init(sm.kt_full, kFeedThreads);
            init(sm.kt_empty, 1);
            init(sm.t_full, kSideThreads);
            init(sm.t_empty, 1);
            init(sm.p_full, kSideThreads);
            init(sm.p_empty, 1);
            init(sm.kq_raw, 1);
            init(sm.tp_raw_full, 1);
            init(sm.v_full, 1);
            init(sm.v_empty, kGroupThreads);
            init(sm.x_full[0], kGroupThreads);
            init(sm.x_full[1], kGroupThreads);
            init(sm.k_done, 1);
            init(sm.r_full, kGroupThreads);
            init(sm.u_done, 1);
            init(sm.u_full, kGroupThreads);
            init(sm.y_done, 1);
            init(sm.x_done, 1);
            init(sm.drained, 1);
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_addr(&sm.tmem), 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    wait_previous_grid();  // T and P, and the states that are there already
    // (ranges that overlap may name more chunks than there is workspace for: their results are undefined, but in bounds)
    const long long at = static_cast<long long>(sm.before);
    const Prepared *prep = prepared(io, H, at + chunks <= prompt_chunks(io.n, io.span.total) ? at : 0, h);
    bool ok = true;
    const auto wait = [&](unsigned long long &b, uint32_t parity) { return barrier_wait(smem_addr(&b), parity, pool.wait_ns); };
    // after a wait that gave up: loads in flight land before the memory is given back (no more than one phase each is)
    const auto drain = [&] {
        if (tid == kGroupThreads || tid == kGroupThreads + kFeedThreads + 32)
            for (auto *bar : {&sm.kq_raw, &sm.tp_raw_full, &sm.v_full}) {
                wait(*bar, 0);
                wait(*bar, 1);
            }
    };

    if (warp >= 8 && warp < 12) {
        // ------------------------------------------------ K, Q and K^T of the chunks
        const int ft = tid - kGroupThreads, fw = warp - 8;
        const auto fetch = [&](int c) {  // as they are, by one thread
            const uint32_t bar = smem_addr(&sm.kq_raw);
            barrier_expect(bar, 4 * kC * 128 + (c == 0 && blockIdx.x == 0 ? pool.stall_tx : 0));
            for (int half = 0; half < 2; ++half) {
                tma_load3(smem_addr(sm.raw_k[half]), &k_map, bar, 64 * half, h, static_cast<int>(first) + c * kC);
                tma_load3(smem_addr(sm.raw_q[half]), &q_map, bar, 64 * half, h, static_cast<int>(first) + c * kC);
            }
        };
        if (ft == 0) fetch(0);
        for (int c = 0; c < chunks && ok; ++c) {
            const int m = min(kC, len - c * kC);
            float rt[2];
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) rt[pass] = prep[static_cast<size_t>(c) * H].r[32 * pass + lane];
            ok = wait(sm.kq_raw, c & 1) && (c == 0 || wait(sm.kq_empty, (c & 1) ^ 1));
            // a lane's two tokens, 32 dims of each a warp; rows behind the prompt's last are not its own
            const uint8_t *rk = sm.raw_k[fw >> 1], *rq = sm.raw_q[fw >> 1];
#pragma unroll
            for (int pass = 0; pass < 2 && ok; ++pass) {
                const int t = 32 * pass + lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 128 * t + ((((fw & 1) * 4 + i) ^ (t & 7)) << 4);
                    uint4 k = *reinterpret_cast<const uint4 *>(rk + at), q = *reinterpret_cast<const uint4 *>(rq + at);
                    if (t >= m) k = q = make_uint4(0, 0, 0, 0);
                    const uint32_t to0 = swizzled(2 * kC, t, 32 * fw + 8 * i), to1 = swizzled(2 * kC, t, 32 * fw + 8 * i + 4);
                    const float2 k0 = widen<BF16>(k.x), k1 = widen<BF16>(k.y), k2 = widen<BF16>(k.z), k3 = widen<BF16>(k.w);
                    *reinterpret_cast<float4 *>(sm.kq + to0) = make_float4(k0.x, k0.y, k1.x, k1.y);
                    *reinterpret_cast<float4 *>(sm.kq + to1) = make_float4(k2.x, k2.y, k3.x, k3.y);
                    const float2 q0 = widen<BF16>(q.x), q1 = widen<BF16>(q.y), q2 = widen<BF16>(q.z), q3 = widen<BF16>(q.w);
                    const float r = rt[pass];
                    *reinterpret_cast<float4 *>(sm.kq + kC * 128 + to0) = make_float4(tf32_hi(q0.x * r), tf32_hi(q0.y * r), tf32_hi(q1.x * r), tf32_hi(q1.y * r));
                    *reinterpret_cast<float4 *>(sm.kq + kC * 128 + to1) = make_float4(tf32_hi(q2.x * r), tf32_hi(q2.y * r), tf32_hi(q3.x * r), tf32_hi(q3.y * r));
                }
            }
            if (ok) {
                fence_async_smem();
                barrier_arrive(smem_addr(&sm.kq_full));
                // K^T from the same
                if (c > 0) ok = wait(sm.kt_empty, (c & 1) ^ 1);
            }
#pragma unroll
            for (int pass = 0; pass < 2 && ok; ++pass) {
                const int t = 32 * pass + lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 k = *reinterpret_cast<const uint4 *>(rk + 128 * t + ((((fw & 1) * 4 + i) ^ (t & 7)) << 4));
                    if (t >= m) k = make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const float2 a = widen<BF16>(w[d]);
                        *reinterpret_cast<float *>(sm.kt + swizzled(kD, 32 * fw + 8 * i + 2 * d, t)) = a.x;
                        *reinterpret_cast<float *>(sm.kt + swizzled(kD, 32 * fw + 8 * i + 2 * d + 1, t)) = a.y;
                    }
                }
            }
            if (ok) {
                fence_async_smem();
                barrier_arrive(smem_addr(&sm.kt_full));
            }
            ok = all_agree<2, kFeedThreads>(ok);  // all have read what comes next over it
            if (ok && ft == 0 && c + 1 < chunks) fetch(c + 1);
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 13 || warp == 14) {
            // ------------------------------------------------ T, P, and V, R and D of the chunks
            const int ft = tid - kGroupThreads - kFeedThreads - 32;
            for (int i = ft; i < kC * kC / 4; i += kSideThreads) {  // above the diagonal they stay zero
                reinterpret_cast<uint4 *>(sm.t)[i] = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4 *>(sm.t)[i + kC * kC / 4] = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4 *>(sm.p)[i] = make_uint4(0, 0, 0, 0);
                if (kTwoTerms<BF16> && i < kRestBytes / 16) reinterpret_cast<uint4 *>(sm.p_rest)[i] = make_uint4(0, 0, 0, 0);
            }
            const auto fetch_tp = [&](int c) {
                const uint32_t bar = smem_addr(&sm.tp_raw_full);
                barrier_expect(bar, 2 * kTriangle * 4);
                bulk_copy(smem_addr(sm.tp_raw), prep[static_cast<size_t>(c) * H].t, 2 * kTriangle * 4, bar);
            };
            const auto fetch_v = [&](int c) {
                const uint32_t bar = smem_addr(&sm.v_full);
                barrier_expect(bar, 2 * kC * 128 + 2 * kC * 4);
                for (int half = 0; half < 2; ++half) tma_load3(smem_addr(sm.v[half]), &v_map, bar, 64 * half, h, static_cast<int>(first) + c * kC);
                bulk_copy(smem_addr(&sm.rd[c & 1]), prep[static_cast<size_t>(c) * H].r, 2 * kC * 4, bar);
            };
            if (ft == 0) {
                fetch_v(0);
                fetch_tp(0);
            }
            all_agree<1, kSideThreads>(true);
            for (int c = 0; c < chunks; ++c) {
                // ten blocks each of T and P, ten vectors a thread; T's place is free before P's
                const auto place = [&](int i, int *row, int *col) {
                    const int x = ft + kSideThreads * i, blk = x / (kBlockFloats / 4), in = x % (kBlockFloats / 4) * 4;
                    const int bi = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, bj = blk - bi * (bi + 1) / 2;
                    *row = 16 * bi + in / 16;
                    *col = 16 * bj + in % 16;
                    return 4 * x;
                };
                // (ok may be false in the thread that fetches: the others learn it below)
                ok = ok && wait(sm.tp_raw_full, c & 1) && (c == 0 || wait(sm.t_empty, (c & 1) ^ 1));
#pragma unroll
                for (int i = 0; i < 10 && ok; ++i) {
                    int row, col;
                    const float4 tv = *reinterpret_cast<const float4 *>(sm.tp_raw + place(i, &row, &col));
                    const float4 hi = make_float4(tf32_hi(tv.x), tf32_hi(tv.y), tf32_hi(tv.z), tf32_hi(tv.w));
                    const uint32_t at = swizzled(2 * kC, row, col);
                    *reinterpret_cast<float4 *>(sm.t + at) = hi;
                    *reinterpret_cast<float4 *>(sm.t + kC * 128 + at) = make_float4(tv.x - hi.x, tv.y - hi.y, tv.z - hi.z, tv.w - hi.w);
                }
                if (ok) {
                    fence_async_smem();
                    barrier_arrive(smem_addr(&sm.t_full));
                    ok = c == 0 || wait(sm.p_empty, (c & 1) ^ 1);
                }
#pragma unroll (kTwoTerms<BF16> ? 5 : 10)  // (all ten spill there, which costs the walk 8 %)
                for (int i = 0; i < 10 && ok; ++i) {
                    int row, col;
                    float4 pv = *reinterpret_cast<const float4 *>(sm.tp_raw + kTriangle + place(i, &row, &col));
                    if (kTwoTerms<BF16>) {
                        const float4 first = make_float4(tf32_hi(pv.x), tf32_hi(pv.y), tf32_hi(pv.z), tf32_hi(pv.w));
                        // (rows below 32 have no columns from 32 on; a row's place in its group of eight is the same in both)
                        const uint32_t to = col < 32 ? swizzled(kC, row, col) : kRestBlock + swizzled(kC / 2, row - 32, col - 32);
                        *reinterpret_cast<float4 *>(sm.p_rest + to) = make_float4(pv.x - first.x, pv.y - first.y, pv.z - first.z, pv.w - first.w);
                        pv = first;
                    }
                    *reinterpret_cast<float4 *>(sm.p + swizzled(kC, row, col)) = pv;
                }
                if (ok) {
                    fence_async_smem();
                    barrier_arrive(smem_addr(&sm.p_full));
                }
                ok = all_agree<1, kSideThreads>(ok);  // all have read what comes next over it
                if (!ok) break;
                if (ft == 0 && c + 1 < chunks) {
                    fetch_tp(c + 1);
                    ok = wait(sm.v_empty, c & 1);
                    if (ok) fetch_v(c + 1);
                }
            }
            if (ok && ft == 0) wait(sm.v_full, (chunks - 1) & 1);  // lands, whatever became of those who wanted it
        } else if (warp == 12) {
            // ------------------------------------------------ products
            constexpr uint32_t n32 = tc_idesc(2, 128, 32, false), n64 = tc_idesc(2, 128, 64, false), n128 = tc_idesc(2, 128, 128, false);
            const uint32_t kq = smem_addr(sm.kq), kt = smem_addr(sm.kt), tt = smem_addr(sm.t), p = smem_addr(sm.p);
            // step s of 8 in an operand of blocks of 32 columns and `rows` rows
            const auto step = [](uint32_t base, int rows, int s) { return tc_desc(base + (s >> 2) * rows * 128 + (s & 3) * 32, 16, 1024); };
            // (after a wait that gave up, products go on, of whatever is there, until all lanes have agreed on it, once a chunk:
            // elect.sync wants the whole warp)
            for (int c = 0; c < chunks && ok; ++c) {
                const uint32_t phase = c & 1;
                // key rows 0-31 and 64-95 of X_0 come first
                ok = wait(sm.kq_full, phase);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    ok = ok && wait(sm.x_full[b], phase);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int s = 4 * b + (i >> 2) * 8 + (i & 3);
                            tc_mma_tf32(tmem + kColK, tmem + kColHi + 8 * s, step(kq, 128, s), n128, b > 0 || i > 0);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int s = 4 * b + (i >> 2) * 8 + (i & 3);
                            tc_mma_tf32(tmem + kColK, tmem + kColLo + 8 * s, step(kq, 128, s), n64, true);
                        }
                        if (b == 1) {
                            tc_commit(smem_addr(&sm.k_done));
                            tc_commit(smem_addr(&sm.kq_empty));
                        }
                    }
                    __syncwarp();
                }
                ok = ok && wait(sm.t_full, phase) && wait(sm.r_full, phase);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 8; ++s) tc_mma_tf32(tmem + kColHi, tmem + kColLo + 8 * s, step(tt, 128, s), n128, s > 0);
#pragma unroll
                    for (int s = 0; s < 8; ++s) tc_mma_tf32(tmem + kColHi, tmem + kColLo + 64 + 8 * s, step(tt, 128, s), n64, true);
                    tc_commit(smem_addr(&sm.u_done));
                    tc_commit(smem_addr(&sm.t_empty));
                }
                __syncwarp();
                ok = ok && wait(sm.kt_full, phase) && wait(sm.u_full, phase);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 16; ++s) tc_mma_tf32(tmem + kColX, tmem + kColHi + 8 * s, step(kt, 128, s & 7), n128, true);
                    tc_commit(smem_addr(&sm.x_done));
                    tc_commit(smem_addr(&sm.kt_empty));
                }
                __syncwarp();
                ok = ok && wait(sm.p_full, phase);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 8; ++s) tc_mma_tf32(tmem + kColY, tmem + kColK + 8 * s, step(p, 64, s), n64, true);
                    if (kTwoTerms<BF16>) {
                        const uint32_t rest = smem_addr(sm.p_rest);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tc_mma_tf32(tmem + kColY, tmem + rest_column(0) + 8 * s, step(p, 64, s), n64, true);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tc_mma_tf32(tmem + kColY + 32, tmem + rest_column(1) + 8 * s, step(p + kC * 128 + 32 * 128, 64, s), n32, true);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tc_mma_tf32(tmem + kColY, tmem + kColK + 8 * s, step(rest, 64, s), n64, true);
#pragma unroll
                        for (int s = 0; s < 4; ++s) tc_mma_tf32(tmem + kColY + 32, tmem + kColK + 32 + 8 * s, step(rest + kRestBlock, 32, s), n32, true);
                    }
                    tc_commit(smem_addr(&sm.y_done));
                    tc_commit(smem_addr(&sm.p_empty));
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok && elect_one()) {  // products in flight end (bounded) before the memory is given back
                tc_commit(smem_addr(&sm.drained));
                wait(sm.drained, 0);
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------ between the products: a lane is a column of the state
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGroupRegs));
        const int half = warp >> 2, j = (warp & 3) * 32 + lane;
        const uint32_t base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint8_t *v = sm.v[j >> 6] + (j & 7) * 2;
        // X_0 and its terms, 32 key rows at a time; x_next: R_63 of the chunk that starts
        const auto put = [&](int col, uint32_t (&x)[32], float x_next) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(tf32_hi(__uint_as_float(x[i])));
            tmem_store32(base + kColHi + col, w);
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(w + i, minus(pair_at(x + i), pair_at(w + i)));
            tmem_store32(base + kColLo + col, w);
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(x + i, __fmul2_rn(pair_at(x + i), make_float2(x_next, x_next)));
            tmem_store32(base + kColX + col, x);
        };
        ok = wait(sm.v_full, 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            const float x_next = sm.rd[0].r[kC - 1];
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int col = 64 * half + 32 * b;
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = fresh ? 0u : __float_as_uint(state[static_cast<size_t>(col + i) * kD + j]);
                put(col, x, x_next);
                tmem_wait_store();
                tc_fence_before();
                barrier_arrive(smem_addr(&sm.x_full[b]));
            }
        }
        uint32_t ys[16];  // the last chunk's Y, two tokens a register, until there is time to store it
        const auto store_y = [&](int c) {
            const int left = len - c * kC - 32 * half;
            // two exchanges between lanes give each 4 columns of 8 tokens: 8-byte stores, and a quarter as many
            const bool odd = lane & 1, two = lane & 2;
            uint32_t pairs[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t mine = odd ? ys[8 + i] : ys[i], other = __shfl_xor_sync(0xffffffffu, odd ? ys[i] : ys[8 + i], 1);
                const uint32_t a = odd ? other : mine, b = odd ? mine : other;
                pairs[2 * i] = __byte_perm(a, b, 0x5410);
                pairs[2 * i + 1] = __byte_perm(a, b, 0x7632);
            }
            const int t0 = (odd ? 16 : 0) + (two ? 8 : 0);
            uint16_t *y = static_cast<uint16_t *>(io.y) + ((first + static_cast<long long>(c) * kC + 32 * half + t0) * H + h) * kD + (j & ~3);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t mine = two ? pairs[8 + i] : pairs[i], other = __shfl_xor_sync(0xffffffffu, two ? pairs[i] : pairs[8 + i], 2);
                if (t0 + i < left) *reinterpret_cast<uint2 *>(y + static_cast<size_t>(i) * H * kD) = two ? make_uint2(other, mine) : make_uint2(mine, other);
            }
        };
        for (int c = 0; c < chunks && ok; ++c) {
            const uint32_t phase = c & 1;
            const auto &rd = sm.rd[c & 1];
            const int left = len - c * kC - 32 * half;  // of this thread's tokens
            uint32_t x[32], w[32];
            // V - diag(R) K X_0
            float vs[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int t = 32 * half + i;
                vs[i] = widen1<BF16>(*reinterpret_cast<const uint16_t *>(v + 128 * t + (((j >> 3 & 7) ^ (t & 7)) << 4)));
            }
            barrier_arrive(smem_addr(&sm.v_empty));
            ok = __all_sync(0xffffffffu, wait(sm.k_done, phase));
            if (!ok) break;
            tc_fence_after();
            tmem_load32(base + kColK + 32 * half, x);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 r = *reinterpret_cast<const float2 *>(&rd.r[32 * half + i]);
                const float2 y = __ffma2_rn(make_float2(-r.x, -r.y), pair_at(x + i), make_float2(vs[i], vs[i + 1]));
                vs[i] = y.x;
                vs[i + 1] = y.y;
            }
            if (left < 32) {  // rows behind the prompt's last are not its own
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i >= left) vs[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(tf32_cut(vs[i]));
            tmem_store32(base + kColLo + 32 * half, w);
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(x + i, minus(make_float2(vs[i], vs[i + 1]), pair_at(w + i)));
            tmem_store32(base + kColLo + 64 + 32 * half, x);
            tmem_wait_store();
            tc_fence_before();
            barrier_arrive(smem_addr(&sm.r_full));
            // U, and D U
            ok = __all_sync(0xffffffffu, wait(sm.u_done, phase));
            if (!ok) break;
            tc_fence_after();
            tmem_load32(base + kColHi + 32 * half, x);
            tmem_load32(base + kColHi + 64 + 32 * half, w);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(x + i, __fadd2_rn(pair_at(x + i), pair_at(w + i)));
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(tf32_hi(__uint_as_float(x[i])));
            if (!kTwoTerms<BF16>) {
                // One NaN in a column of U makes its whole column of Y one, as it should be (top of the file): zero times U is added to an element.
                float2 none[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < 32; i += 2) none[i >> 1 & 1] = __ffma2_rn(pair_at(x + i), make_float2(0.0f, 0.0f), none[i >> 1 & 1]);
                w[0] = __float_as_uint(__uint_as_float(w[0]) + ((none[0].x + none[0].y) + (none[1].x + none[1].y)));
            }
            tmem_store32(base + kColK + 32 * half, w);
            if (kTwoTerms<BF16>) {  // where the next chunk's X_0 has not come yet
#pragma unroll
                for (int i = 0; i < 32; i += 2) put_pair(w + i, minus(pair_at(x + i), pair_at(w + i)));
                tmem_store32(base + rest_column(half), w);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(x + i, __fmul2_rn(pair_at(x + i), *reinterpret_cast<const float2 *>(&rd.d[32 * half + i])));
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(tf32_cut(__uint_as_float(x[i])));
            tmem_store32(base + kColHi + 32 * half, w);
#pragma unroll
            for (int i = 0; i < 32; i += 2) put_pair(x + i, minus(pair_at(x + i), pair_at(w + i)));
            tmem_store32(base + kColHi + 64 + 32 * half, x);
            tmem_wait_store();
            tc_fence_before();
            barrier_arrive(smem_addr(&sm.u_full));
            if (c > 0) store_y(c - 1);
            // the state after the chunk
            float x_next = 0.0f;
            if (c + 1 < chunks) {
                ok = __all_sync(0xffffffffu, wait(sm.v_full, phase ^ 1));
                if (!ok) break;
                x_next = sm.rd[phase ^ 1].r[kC - 1];
            }
            ok = __all_sync(0xffffffffu, wait(sm.x_done, phase));
            if (!ok) break;
            tc_fence_after();
            // the first half of this thread's rows, then Y (whose products come behind the state's; the next chunk's
            // go where it is), and those products may begin
            const auto update = [&](int b) {
                const int col = 64 * half + 32 * b;
                tmem_load32(base + kColX + col, x);
                tmem_wait_load();
                if (c + 1 < chunks) {
                    put(col, x, x_next);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) state[static_cast<size_t>(col + i) * kD + j] = __uint_as_float(x[i]);
                }
            };
            update(0);
            ok = __all_sync(0xffffffffu, wait(sm.y_done, phase));
            if (!ok) break;
            tc_fence_after();
            tmem_load32(base + kColY + 32 * half, x);
            tmem_wait_load();
            tmem_wait_store();
            tc_fence_before();
            barrier_arrive(smem_addr(&sm.x_full[0]));
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ys[i] = narrow1<BF16>(__uint_as_float(x[2 * i])) | static_cast<uint32_t>(narrow1<BF16>(__uint_as_float(x[2 * i + 1]))) << 16;
            update(1);
            tmem_wait_store();
            tc_fence_before();
            barrier_arrive(smem_addr(&sm.x_full[1]));
        }
        if (ok) store_y(chunks - 1);
    }
    if (!ok) {
        if (lane == 0) atomicOr(pool.err, kErrTimeout);
        drain();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

template <bool BF16>
cudaError_t launch(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    CUtensorMap q, k, v;
    if (!make_map(&q, io.q, io.dtype, io.span.total, p.H, 1, kC) || !make_map(&k, io.k, io.dtype, io.span.total, p.H, 1, kC) ||
        !make_map(&v, io.v, io.dtype, io.span.total, p.H, 1, kC))
        return cudaErrorInvalidValue;
    const int prep = static_cast<int>(sizeof(PrepSmem)), smem = static_cast<int>(sizeof(ChunkSmem<BF16>)) + 1024;
    cudaError_t e = cudaFuncSetAttribute(prepare_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, prep);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(chunk_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // each begins while the one before it ends
    const dim3 prepared(static_cast<unsigned>(prompt_chunks(io.n, io.span.total)), static_cast<unsigned>(p.H));
    e = launch_behind(prepare_kernel<BF16>, prepared, kPrepThreads, prep, stream, io, p.H);
    if (e != cudaSuccess) return e;
    return launch_behind(chunk_kernel<BF16>, dim3(static_cast<unsigned>(io.n) * p.H), kChunkThreads, smem, stream, q, k, v, p, io);
}

}  // namespace

cudaError_t launch_prompt_chunks(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    return io.dtype == STQ_BF16 ? launch<true>(p, io, stream) : launch<false>(p, io, stream);
}

}  // namespace stq
