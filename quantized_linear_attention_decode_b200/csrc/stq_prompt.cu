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

// ---------------------------------------------------------------- token by token
//
// Columns of X do not depend on each other, so a warp owns some of them for the
// whole prompt, in registers, and no warp waits for another but for the staged
// tokens.  Lane (c, r) has kCols columns c and the rows that r takes of them:
// blocks of four rows, r, r + RP, ... of the 32 blocks.  A token costs three
// multiply-adds an element, all fp32: the two column sums X^T k and X^T q of the
// state before the token (y follows as a X^T q + u (k . q)), then X += k u^T.
// The decay is not multiplied in: X = c X~ with the product c of the decays, and
// X~ is rescaled when c leaves [2^-20, 2^20], so that an element costs three packed
// instructions a token pair in place of four.
// Bound by the fp32 pipe (98304 multiply-adds a token and head) when there are
// prompts and heads enough, else by a token's latency; more lanes on a column (RP)
// then shorten the latter.

constexpr int kThreads = 128;
constexpr int kTokens = 16;  // staged at a time
constexpr int kCols = 4;     // columns of a lane

template <int RP>
constexpr int kCtaCols = kThreads / RP * kCols;  // columns of a CTA

template <int RP>
struct __align__(16) Staged {
    float k[kTokens][kD], q[kTokens][kD];
    float v[kTokens][kCtaCols<RP>];
    // before the token X~ is multiplied by `rescale` (1: left alone); then X = c X~ with its decay, and 1 / c
    float4 scale[kTokens];  // rescale, c, 1 / c, gate
    float kq[kTokens];
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The head's rows of tokens [t0, t0 + m), as they come (zeros behind them), in the registers of all threads...
template <int RP>
struct Incoming {
    static constexpr int kVec = kTokens * kD / 8 / kThreads, kVecV = (kTokens * kCtaCols<RP> / 8 + kThreads - 1) / kThreads;
    float k[kVec][8], q[kVec][8], v[kVecV][8], a, b;

    __device__ __forceinline__ void load(const PromptIO &io, int H, int h, int col0, long long t0, int m)
    {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int t = (tid + i * kThreads) / (kD / 8), d = tid % (kD / 8) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) k[i][j] = q[i][j] = 0.0f;
            if (t < m) {
                load8(io.k.data, (t0 + t) * io.k.token_stride + h * io.k.head_stride + d, io.dtype, k[i]);
                load8(io.q.data, (t0 + t) * io.q.token_stride + h * io.q.head_stride + d, io.dtype, q[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kVecV; ++i) {
            const int e = tid + i * kThreads, t = e / (kCtaCols<RP> / 8), d = e % (kCtaCols<RP> / 8) * 8;
            if (t < m) load8(io.v.data, (t0 + t) * io.v.token_stride + h * io.v.head_stride + col0 + d, io.dtype, v[i]);
        }
        a = tid < m ? io.alpha[(t0 + tid) * H + h] : 1.0f;
        b = tid < m ? io.beta[(t0 + tid) * H + h] : 0.0f;
    }

    // ... and from there to shared memory.  c: the product of decays that X~ stands under, kept by the first warp.
    __device__ __forceinline__ void store(Staged<RP> &s, int m, float &c) const
    {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int t = (tid + i * kThreads) / (kD / 8), d = tid % (kD / 8) * 8;
            *reinterpret_cast<float4 *>(&s.k[t][d]) = make_float4(k[i][0], k[i][1], k[i][2], k[i][3]);
            *reinterpret_cast<float4 *>(&s.k[t][d + 4]) = make_float4(k[i][4], k[i][5], k[i][6], k[i][7]);
            *reinterpret_cast<float4 *>(&s.q[t][d]) = make_float4(q[i][0], q[i][1], q[i][2], q[i][3]);
            *reinterpret_cast<float4 *>(&s.q[t][d + 4]) = make_float4(q[i][4], q[i][5], q[i][6], q[i][7]);
            float kq = 0.0f;  // 16 lanes hold a token
#pragma unroll
            for (int j = 0; j < 8; ++j) kq = fmaf(k[i][j], q[i][j], kq);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
            if (tid % 16 == 0) s.kq[t] = kq;
        }
#pragma unroll
        for (int i = 0; i < kVecV; ++i) {
            const int e = tid + i * kThreads, t = e / (kCtaCols<RP> / 8), d = e % (kCtaCols<RP> / 8) * 8;
            if (t < m) {
                *reinterpret_cast<float4 *>(&s.v[t][d]) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                *reinterpret_cast<float4 *>(&s.v[t][d + 4]) = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
            }
        }
        if (tid < 32) {
            float rescale = 1.0f, mine = 1.0f;
#pragma unroll
            for (int t = 0; t < kTokens; ++t) {
                const float next = c * __shfl_sync(0xffffffffu, a, t);
                const bool out = !(fabsf(next) >= 0x1p-20f && fabsf(next) <= 0x1p20f);
                if (tid == t) {
                    rescale = out ? next : 1.0f;
                    mine = out ? 1.0f : next;
                }
                c = out ? 1.0f : next;
            }
            if (tid < kTokens) s.scale[tid] = make_float4(rescale, mine, 1.0f / mine, b);
        }
    }
};

template <int RP>
__global__ void __launch_bounds__(kThreads, RP == 4 ? 2 : RP == 8 ? 3 : 4) prompt_tokens_kernel(PoolView p, PromptIO io)
{
    extern __shared__ __align__(16) uint8_t raw_smem[];
    Staged<RP> *st = reinterpret_cast<Staged<RP> *>(raw_smem);  // two of them
    constexpr int kSlices = kD / kCtaCols<RP>;
    constexpr int kBlocks = 32 / RP;  // blocks of four rows of a lane
    const int unit = blockIdx.x / kSlices, slice = blockIdx.x % kSlices;
    const int e = unit / p.H, h = unit - e * p.H;
    const int req = io.req_idx[e], slot = io.slot_idx[e];
    if (req < 0 || req >= p.R || slot < 0 || slot >= p.S) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
        return;
    }
    int len = io.span.length(e);
    if (len < 0) {
        if (threadIdx.x == 0) atomicOr(p.err, kErrIndex);
        len = 0;
    }
    const bool fresh = io.span.is_fresh(e);
    if (len == 0 && !fresh) return;
    const long long first = io.span.seq_start[e];
    const int lane = threadIdx.x & 31, r = lane % RP;
    const int col = threadIdx.x / RP * kCols;  // of the CTA's
    const int col0 = slice * kCtaCols<RP>;
    float *S = io.state + static_cast<size_t>(unit) * kD * kD + col0 + col;

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
    float c = 1.0f, last = 1.0f;  // X = last x; c runs ahead in the first warp
    Incoming<RP> in;
    in.load(io, p.H, h, col0, first, min(len, kTokens));
    in.store(st[0], min(len, kTokens), c);
    __syncthreads();
    for (int t0 = 0; t0 < len; t0 += kTokens) {
        const Staged<RP> &s = st[t0 / kTokens & 1];
        const int coming = min(len - t0 - kTokens, kTokens);  // tokens after these
        if (coming > 0) in.load(io, p.H, h, col0, first + t0 + kTokens, coming);
        const int m = min(len - t0, kTokens);
        for (int t = 0; t < m; ++t) {
            float2 sk[kCols], sq[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) sk[j] = sq[j] = make_float2(0.0f, 0.0f);
            float4 k4[kBlocks];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                k4[b] = *reinterpret_cast<const float4 *>(&s.k[t][4 * (r + RP * b)]);
                const float4 q4 = *reinterpret_cast<const float4 *>(&s.q[t][4 * (r + RP * b)]);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    sk[j] = fma2(x[b][j][0], make_float2(k4[b].x, k4[b].y), sk[j]);
                    sk[j] = fma2(x[b][j][1], make_float2(k4[b].z, k4[b].w), sk[j]);
                    sq[j] = fma2(x[b][j][0], make_float2(q4.x, q4.y), sq[j]);
                    sq[j] = fma2(x[b][j][1], make_float2(q4.z, q4.w), sq[j]);
                }
            }
            const float4 scale = s.scale[t];
            const float kq = s.kq[t];
            // the sums over the lanes of a column: each exchange halves the columns that a lane is left with, until
            // lane r has column r mod 4's two
            float vk, vq;
            const float v = s.v[t][col + (r & 3)];
            {
                const bool odd = r & 1, two = r & 2;
                float k2[2], q2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float ke = sk[2 * j].x + sk[2 * j].y, ko = sk[2 * j + 1].x + sk[2 * j + 1].y;
                    const float qe = sq[2 * j].x + sq[2 * j].y, qo = sq[2 * j + 1].x + sq[2 * j + 1].y;
                    k2[j] = (odd ? ko : ke) + __shfl_xor_sync(0xffffffffu, odd ? ke : ko, 1);
                    q2[j] = (odd ? qo : qe) + __shfl_xor_sync(0xffffffffu, odd ? qe : qo, 1);
                }
                vk = (two ? k2[1] : k2[0]) + __shfl_xor_sync(0xffffffffu, two ? k2[0] : k2[1], 2);
                vq = (two ? q2[1] : q2[0]) + __shfl_xor_sync(0xffffffffu, two ? q2[0] : q2[1], 2);
            }
#pragma unroll
            for (int o = 4; o < RP; o *= 2) {
                vk += __shfl_xor_sync(0xffffffffu, vk, o);
                vq += __shfl_xor_sync(0xffffffffu, vq, o);
            }
            if (scale.x != 1.0f) {  // the same for every thread of the head
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) x[b][j][i] = make_float2(x[b][j][i].x * scale.x, x[b][j][i].y * scale.x);
                vk *= scale.x;
                vq *= scale.x;
            }
            last = scale.y;
            float own = scale.w * fmaf(-scale.y, vk, v);
            const float y = fmaf(scale.y, vq, own * kq);
            own *= scale.z;
            float u[kCols];
            {
                const bool odd = r & 1, two = r & 2;
                const float beside = __shfl_xor_sync(0xffffffffu, own, 1);
                const float even = odd ? beside : own, uneven = odd ? own : beside;
                const float even2 = __shfl_xor_sync(0xffffffffu, even, 2), uneven2 = __shfl_xor_sync(0xffffffffu, uneven, 2);
                u[0] = two ? even2 : even;
                u[1] = two ? uneven2 : uneven;
                u[2] = two ? even : even2;
                u[3] = two ? uneven : uneven2;
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const float2 uu = make_float2(u[j], u[j]);
                    x[b][j][0] = fma2(make_float2(k4[b].x, k4[b].y), uu, x[b][j][0]);
                    x[b][j][1] = fma2(make_float2(k4[b].z, k4[b].w), uu, x[b][j][1]);
                }
            if (r < 4) store_from_float(io.y, ((first + t0 + t) * p.H + h) * kD + col0 + col + r, io.dtype, y);
        }
        if (coming > 0) in.store(st[(t0 / kTokens & 1) ^ 1], coming, c);
        __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float *to = S + static_cast<size_t>(4 * (r + RP * b) + 2 * i) * kD;
            *reinterpret_cast<float4 *>(to) = make_float4(last * x[b][0][i].x, last * x[b][1][i].x, last * x[b][2][i].x, last * x[b][3][i].x);
            *reinterpret_cast<float4 *>(to + kD) = make_float4(last * x[b][0][i].y, last * x[b][1][i].y, last * x[b][2][i].y, last * x[b][3][i].y);
        }
}

template <int RP>
cudaError_t launch_tokens(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    const int smem = 2 * static_cast<int>(sizeof(Staged<RP>));
    cudaError_t e = cudaFuncSetAttribute(prompt_tokens_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned ctas = static_cast<unsigned>(io.n) * p.H * (kD / kCtaCols<RP>);
    prompt_tokens_kernel<RP><<<ctas, kThreads, smem, stream>>>(p, io);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PoolView &p, const PromptIO &io, cudaStream_t stream)
{
    // 16-bit rows go in chunks (of rows that a tensor map can describe), unless the prompts are so short that
    // most of a chunk would be empty
    const int total = io.span.total;
    if (io.dtype != STQ_F32 && p.H <= 65535 && total >= 16ll * io.n && rows_mappable(io.q, p.H, total) &&
        rows_mappable(io.k, p.H, total) && rows_mappable(io.v, p.H, total))
        return launch_prompt_chunks(p, io, stream);
    const long long units = static_cast<long long>(io.n) * p.H;
    // more lanes a column shorten a token (16: 880 cycles at three warps on a scheduler) and cost a fixed part of
    // each warp's instructions; enough warps to fill the schedulers once decide
    if (units >= 256) return launch_tokens<4>(p, io, stream);
    return units >= 128 ? launch_tokens<8>(p, io, stream) : launch_tokens<16>(p, io, stream);
}

}  // namespace stq
