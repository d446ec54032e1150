// stq_prompt.cu -- the gated delta rule over whole prompts (sm_100a).
//
// For every head of every prompt, with the state held in fp32 from the first token
// to the last,
//   X_t = a_t X_{t-1} + b_t k_t (v_t - a_t X_{t-1}^T k_t)^T,   y_t = X_t^T q_t.
#include <cmath>

#include "stq_host.h"
#include "stq_map.h"
#include "stq_ptx.h"

namespace stq {
namespace {

// ---------------------------------------------------------------- in fp32, four tokens at a time
//
// Columns of X do not depend on each other, so a warp owns some of them for the
// whole prompt, in registers, and no warp waits for another but for the staged
// tokens.  Lane (c, r) has kCols columns c and the rows that r takes of them:
// blocks of four rows, r, r + RP, ... of the 32 blocks.  Tokens are taken four at a
// time, from the state X before them: with A_j = a_0 ... a_j and D_ij = a_{i+1} ... a_j,
//   u_j = b_j (v_j - A_j X^T k_j - sum_{i<j} D_ij (k_i . k_j) u_i)
//   y_j = A_j X^T q_j + sum_{i<=j} D_ij (k_i . q_j) u_i
//   X <- A_3 X + sum_i D_i3 k_i u_i^T,
// all fp32: three multiply-adds an element and token, and one sum over a column's
// lanes, one chain of dependent sums and one broadcast in place of four.
// Bound by the fp32 pipe (49152 multiply-adds a token and head) and by reads and exchanges
// through shared memory when there are prompts and heads enough, else by the latency of
// four tokens; more lanes on a column (RP) shorten the latter.  768 units of 100 tokens take
// 292 us (26 TFLOP/s: half of the issue slots, two warps a scheduler do not hide each other's
// sums and loads), one unit 0.2 us a token.

constexpr int kThreads = 128;
constexpr int kBlock = 4;                          // tokens taken at a time
constexpr int kTokens = kThreads / 32 * kBlock;    // staged at a time: a block a warp
constexpr int kCols = 4;                           // columns of a lane
constexpr int kKk = 0, kKq = 6, kSums = 16;        // of a block's coefficients: 6 and 10 inner products with their decays,
constexpr int kDecay = 16, kGate = 20, kLast = 24; // then A_j, b_j and D_j3

template <int RP>
constexpr int kCtaCols = kThreads / RP * kCols;  // columns of a CTA

template <int RP>
struct __align__(16) Staged {
    float k[kTokens][kD], q[kTokens][kD];
    float v[kTokens][kCtaCols<RP>];
    float coef[kTokens / kBlock][28];
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float dot4(float4 a, float4 b) { return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w))); }

// Halves the values that a lane holds: it keeps the lower or (with the lane's bit `o` set) the upper half,
// summed with those of the lane across that bit.
template <int N>
__device__ __forceinline__ void fold(float (&x)[N], float (&to)[N / 2], int o)
{
    const bool upper = threadIdx.x & o;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = upper ? x[i + N / 2] : x[i], give = upper ? x[i] : x[i + N / 2];
        to[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
}

// Four consecutive elements as they lie in memory, and as numbers.
template <int TYPE>
struct Four {
    uint2 w;
    __device__ __forceinline__ float4 wide() const
    {
        if (TYPE == STQ_BF16)
            return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
};
template <>
struct Four<STQ_F32> {
    float4 w;
    __device__ __forceinline__ float4 wide() const { return w; }
};
template <int TYPE>
__device__ __forceinline__ Four<TYPE> load4(const void *p, int64_t i)
{
    return *reinterpret_cast<const Four<TYPE> *>(static_cast<const uint8_t *>(p) + i * static_cast<int>(sizeof(Four<TYPE>) / 4));
}

// The head's rows of tokens [t0, t0 + m), as they come (zeros behind them, with decay 1 and gate 0), in the registers of all threads:
// warp w has block w...
template <int RP, int TYPE>
struct Incoming {
    static constexpr int kVecV = kTokens * kCtaCols<RP> / 4 / kThreads;
    Four<TYPE> k[kBlock], q[kBlock], v[kVecV];
    float a, b;  // of token lane of the block

    __device__ __forceinline__ void load(const PromptIO &io, int H, int h, int col0, long long t0, int m)
    {
        const int tid = threadIdx.x, lane = tid & 31, mine = tid / 32 * kBlock;
        const Four<TYPE> zero = {};
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            const bool there = mine + i < m;
            k[i] = there ? load4<TYPE>(io.k.data, (t0 + mine + i) * io.k.token_stride + h * io.k.head_stride + 4 * lane) : zero;
            q[i] = there ? load4<TYPE>(io.q.data, (t0 + mine + i) * io.q.token_stride + h * io.q.head_stride + 4 * lane) : zero;
        }
#pragma unroll
        for (int i = 0; i < kVecV; ++i) {
            const int e = tid + i * kThreads, t = e / (kCtaCols<RP> / 4), d = e % (kCtaCols<RP> / 4) * 4;
            v[i] = t < m ? load4<TYPE>(io.v.data, (t0 + t) * io.v.token_stride + h * io.v.head_stride + col0 + d) : zero;
        }
        const bool there = lane < kBlock && mine + lane < m;
        a = there ? io.alpha[(t0 + mine + lane) * H + h] : 1.0f;
        b = there ? io.beta[(t0 + mine + lane) * H + h] : 0.0f;
    }

    // ... and from there to shared memory, with the block's coefficients.
    __device__ __forceinline__ void store(Staged<RP> &s) const
    {
        const int tid = threadIdx.x, lane = tid & 31, block = tid / 32;
        float4 kw[kBlock], qw[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            *reinterpret_cast<float4 *>(&s.k[block * kBlock + i][4 * lane]) = kw[i] = k[i].wide();
            *reinterpret_cast<float4 *>(&s.q[block * kBlock + i][4 * lane]) = qw[i] = q[i].wide();
        }
#pragma unroll
        for (int i = 0; i < kVecV; ++i) {
            const int e = tid + i * kThreads, t = e / (kCtaCols<RP> / 4), d = e % (kCtaCols<RP> / 4) * 4;
            *reinterpret_cast<float4 *>(&s.v[t][d]) = v[i].wide();
        }
        float x[kSums], x8[8], x4[4], x2[2], x1[1];
        {
            int to = 0;
#pragma unroll
            for (int i = 0; i < kBlock; ++i)
#pragma unroll
                for (int j = i + 1; j < kBlock; ++j) x[to++] = dot4(kw[i], kw[j]);
#pragma unroll
            for (int i = 0; i < kBlock; ++i)
#pragma unroll
                for (int j = i; j < kBlock; ++j) x[to++] = dot4(kw[i], qw[j]);
        }
        fold(x, x8, 16);
        fold(x8, x4, 8);
        fold(x4, x2, 4);
        fold(x2, x1, 2);  // lanes 2n and 2n + 1 have sum n
        const float sum = x1[0] + __shfl_xor_sync(0xffffffffu, x1[0], 1);
        // D_ij of sum n; its i and j (two bits each), in the order above
        constexpr uint32_t kOfI = 0xe9500940u, kOfJ = 0xfb9e4fb9u;
        const int n = lane >> 1, i = kOfI >> (2 * n) & 3, j = kOfJ >> (2 * n) & 3;
        float decay = 1.0f, before = 1.0f, after = 1.0f;
#pragma unroll
        for (int m = 0; m < kBlock; ++m) {
            const float am = __shfl_sync(0xffffffffu, a, m);
            if (i < m && m <= j) decay *= am;
            if (m <= lane) before *= am;
            if (m > lane) after *= am;
        }
        float *c = s.coef[block];
        if (!(lane & 1)) c[n] = decay * sum;
        if (lane < kBlock) {
            c[kDecay + lane] = before;
            c[kGate + lane] = b;
            c[kLast + lane] = after;
        }
    }
};

template <int RP, int TYPE>
__global__ void __launch_bounds__(kThreads, RP == 8 ? 2 : 3) prompt_tokens_kernel(PoolView p, PromptIO io)
{
    __shared__ Staged<RP> st[2];
    __shared__ float4 solved[2][kThreads / RP][kCols];  // u of a column's four tokens, of this block and of the last
    constexpr int kSlices = kD / kCtaCols<RP>;
    constexpr int kBlocks = 32 / RP;  // blocks of four rows of a lane
    const int unit = blockIdx.x / kSlices, slice = blockIdx.x % kSlices;
    const int e = unit / p.H, h = unit - e * p.H;
    const int req = io.req_idx[e], slot = io.slot_idx[e];
    if (req < 0 || req >= p.R || slot < 0 || slot >= p.S) {
        wait_previous_grid();
        if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
        return;
    }
    launch_dependents();
    int len = io.span.length(e);
    if (len < 0) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
        len = 0;
    }
    const bool fresh = io.span.is_fresh(e);
    if (len == 0 && !fresh) {
        wait_previous_grid();
        return;
    }
    const long long first = io.span.seq_start[e];
    const int lane = threadIdx.x & 31, r = lane % RP;
    const int col = threadIdx.x / RP * kCols;  // of the CTA's
    const int col0 = slice * kCtaCols<RP>;
    float *S = io.state + static_cast<size_t>(unit) * kD * kD + col0 + col;

    Incoming<RP, TYPE> in;
    in.load(io, p.H, h, col0, first, min(len, kTokens));
    in.store(st[0]);
    wait_previous_grid();  // the states that are there already

    // x[b][c][0..1]: rows 4 (r + RP b) + {0, 1} and {2, 3} of column c
    float2 x[kBlocks][kCols][2];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = fresh ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *reinterpret_cast<const float4 *>(S + static_cast<size_t>(4 * (r + RP * b) + i) * kD);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[b][0][i] = make_float2(w[2 * i].x, w[2 * i + 1].x);
            x[b][1][i] = make_float2(w[2 * i].y, w[2 * i + 1].y);
            x[b][2][i] = make_float2(w[2 * i].z, w[2 * i + 1].z);
            x[b][3][i] = make_float2(w[2 * i].w, w[2 * i + 1].w);
        }
    }
    // X^T times the block's rows of k or q, summed over the lanes with the same lane & 3 of a column: column (lane & 3)'s
    const auto products = [&](const float (*rows)[kD], float (&to)[kBlock]) {
        float2 acc[kCols][kBlock];
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int t = 0; t < kBlock; ++t) acc[j][t] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int t = 0; t < kBlock; ++t) {
                const float4 w = *reinterpret_cast<const float4 *>(&rows[t][4 * (r + RP * b)]);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    acc[j][t] = fma2(x[b][j][0], make_float2(w.x, w.y), acc[j][t]);
                    acc[j][t] = fma2(x[b][j][1], make_float2(w.z, w.w), acc[j][t]);
                }
            }
        float all[kCols * kBlock], half[2 * kBlock];
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
            for (int t = 0; t < kBlock; ++t) all[j * kBlock + t] = acc[j][t].x + acc[j][t].y;
        fold(all, half, 2);
        fold(half, to, 1);
    };

    __syncthreads();
    for (int t0 = 0; t0 < len; t0 += kTokens) {
        const Staged<RP> &s = st[t0 / kTokens & 1];
        const int coming = min(len - t0 - kTokens, kTokens);  // tokens after these
        if (coming > 0) in.load(io, p.H, h, col0, first + t0 + kTokens, coming);
        const int m = min(len - t0, kTokens);
        for (int t1 = 0; t1 < m; t1 += kBlock) {
            float sum[kBlock];
            {
                float both[2 * kBlock], part[kBlock];
                products(&s.k[t1], part);
#pragma unroll
                for (int t = 0; t < kBlock; ++t) both[t] = part[t];
                products(&s.q[t1], part);
#pragma unroll
                for (int t = 0; t < kBlock; ++t) both[kBlock + t] = part[t];
                fold(both, sum, 4);  // lanes with bit 2 clear have X^T k, the others X^T q
            }
#pragma unroll
            for (int o = 8; o < RP; o *= 2)
#pragma unroll
                for (int t = 0; t < kBlock; ++t) sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], o);
            float c[28];
#pragma unroll
            for (int i = 0; i < 28; i += 4) {
                const float4 w = *reinterpret_cast<const float4 *>(&s.coef[t1 / kBlock][i]);
                c[i] = w.x; c[i + 1] = w.y; c[i + 2] = w.z; c[i + 3] = w.w;
            }
            const int own = col + (r & 3);
            // (in the lanes of X^T q, a value that nobody reads)
            const float u0 = c[kGate] * fmaf(-c[kDecay], sum[0], s.v[t1][own]);
            const float u1 = c[kGate + 1] * fmaf(-c[kKk], u0, fmaf(-c[kDecay + 1], sum[1], s.v[t1 + 1][own]));
            const float u2 = c[kGate + 2] * fmaf(-c[kKk + 3], u1, fmaf(-c[kKk + 1], u0, fmaf(-c[kDecay + 2], sum[2], s.v[t1 + 2][own])));
            const float u3 = c[kGate + 3] * fmaf(-c[kKk + 5], u2, fmaf(-c[kKk + 4], u1, fmaf(-c[kKk + 2], u0, fmaf(-c[kDecay + 3], sum[3], s.v[t1 + 3][own]))));
            float4 *us = solved[t1 / kBlock & 1][threadIdx.x / RP];
            if (r < kCols) us[r] = make_float4(u0, u1, u2, u3);
            __syncwarp();
            {
                const float4 w4 = us[r & 3];
                const float w[kBlock] = {w4.x, w4.y, w4.z, w4.w};
                const float y[kBlock] = {fmaf(c[kKq], w[0], c[kDecay] * sum[0]),
                                         fmaf(c[kKq + 4], w[1], fmaf(c[kKq + 1], w[0], c[kDecay + 1] * sum[1])),
                                         fmaf(c[kKq + 7], w[2], fmaf(c[kKq + 5], w[1], fmaf(c[kKq + 2], w[0], c[kDecay + 2] * sum[2]))),
                                         fmaf(c[kKq + 9], w[3], fmaf(c[kKq + 8], w[2], fmaf(c[kKq + 6], w[1], fmaf(c[kKq + 3], w[0], c[kDecay + 3] * sum[3]))))};
                if ((r & ~3) == 4) {
#pragma unroll
                    for (int t = 0; t < kBlock; ++t)
                        if (t1 + t < m) store_from_float(io.y, ((first + t0 + t1 + t) * p.H + h) * kD + col0 + own, TYPE, y[t]);
                }
            }
            const float2 all = make_float2(c[kDecay + 3], c[kDecay + 3]), none = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int j = 0; j < kCols; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) x[b][j][i] = fma2(x[b][j][i], all, none);
            float u[kCols][kBlock];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                const float4 w = us[j];
                u[j][0] = c[kLast] * w.x;
                u[j][1] = c[kLast + 1] * w.y;
                u[j][2] = c[kLast + 2] * w.z;
                u[j][3] = c[kLast + 3] * w.w;
            }
#pragma unroll
            for (int t = 0; t < kBlock; ++t)
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const float4 w = *reinterpret_cast<const float4 *>(&s.k[t1 + t][4 * (r + RP * b)]);
#pragma unroll
                    for (int j = 0; j < kCols; ++j) {
                        x[b][j][0] = fma2(make_float2(w.x, w.y), make_float2(u[j][t], u[j][t]), x[b][j][0]);
                        x[b][j][1] = fma2(make_float2(w.z, w.w), make_float2(u[j][t], u[j][t]), x[b][j][1]);
                    }
                }
        }
        if (coming > 0) in.store(st[(t0 / kTokens & 1) ^ 1]);
        __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float *to = S + static_cast<size_t>(4 * (r + RP * b) + 2 * i) * kD;
            *reinterpret_cast<float4 *>(to) = make_float4(x[b][0][i].x, x[b][1][i].x, x[b][2][i].x, x[b][3][i].x);
            *reinterpret_cast<float4 *>(to + kD) = make_float4(x[b][0][i].y, x[b][1][i].y, x[b][2][i].y, x[b][3][i].y);
        }
}

template <int RP, int TYPE>
cudaError_t launch_tokens(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    const unsigned ctas = static_cast<unsigned>(io.n) * p.H * (kD / kCtaCols<RP>);
    // begun while the states are unpacked, few CTAs save 1 to 2 us (16 of them: 21 against 22 us); many then crowd on some
    // SMs (128: 47 against 39 us)
    if (ctas <= 64) return launch_behind(prompt_tokens_kernel<RP, TYPE>, dim3(ctas), kThreads, 0, stream, p, io);
    prompt_tokens_kernel<RP, TYPE><<<ctas, kThreads, 0, stream>>>(p, io);
    count_launch();
    return cudaGetLastError();
}

template <int RP>
cudaError_t launch_tokens(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    if (io.dtype == STQ_F32) return launch_tokens<RP, STQ_F32>(p, io, stream);
    return io.dtype == STQ_BF16 ? launch_tokens<RP, STQ_BF16>(p, io, stream) : launch_tokens<RP, STQ_F16>(p, io, stream);
}

}  // namespace

cudaError_t launch_prompt(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    // 16-bit rows (that a tensor map can describe) go in chunks of 64 tokens, which take as long for one token as for 64.  Four at a
    // time is faster up to 64 tokens where entries are few (one entry on 32 heads: 10 against 23 us for one token, 23 both for
    // 64, 31 against 27 for 96), up to 24 where they are many (64 on 32 heads: 166 against 269 us for one token each, 278 against
    // 275 for 24, 508 against 284 for 64).  The host knows only their sum, of which one entry may have nearly all (60 of one
    // token and 4 of 1000: 605 against 359 us): so below 64 and two for each further entry, where even then the longest is
    // short.
    const int total = io.span.total;
    if (io.dtype != STQ_F32 && p.H <= 65535 && total >= kPromptChunk + 2ll * (io.n - 1) && rows_mappable(io.q, p.H, total) &&
        rows_mappable(io.k, p.H, total) && rows_mappable(io.v, p.H, total))
        return launch_prompt_chunks(p, io, stream);
    const long long units = static_cast<long long>(io.n) * p.H;
    // more lanes a column shorten a block's latency and cost each warp more loads and exchanges a column: 16 against
    // 8 lanes take 54 against 66 us on 32 units of 200 tokens, 314 against 324 us on 96 of 700, but 139 against
    // 108 us on 128 of 200
    return units >= 128 ? launch_tokens<8>(p, io, stream) : launch_tokens<16>(p, io, stream);
}

}  // namespace stq
