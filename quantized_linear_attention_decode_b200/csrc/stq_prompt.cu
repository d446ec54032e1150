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
    float a[kTokens], b[kTokens], kq[kTokens];
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// The head's rows of tokens [t0, t0 + m) into shared memory, as fp32; tokens behind them as zeros.
template <int RP>
__device__ __forceinline__ void stage(Staged<RP> &s, const PromptIO &io, int H, int h, int col0, long long t0, int m)
{
    const int tid = threadIdx.x;
    for (int e = tid; e < kTokens * kD / 8; e += kThreads) {
        const int t = e / (kD / 8), d = e % (kD / 8) * 8;
        float x[8], z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = z[j] = 0.0f;
        if (t < m) {
            load8(io.k.data, (t0 + t) * io.k.token_stride + h * io.k.head_stride + d, io.dtype, x);
            load8(io.q.data, (t0 + t) * io.q.token_stride + h * io.q.head_stride + d, io.dtype, z);
        }
        *reinterpret_cast<float4 *>(&s.k[t][d]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(&s.k[t][d + 4]) = make_float4(x[4], x[5], x[6], x[7]);
        *reinterpret_cast<float4 *>(&s.q[t][d]) = make_float4(z[0], z[1], z[2], z[3]);
        *reinterpret_cast<float4 *>(&s.q[t][d + 4]) = make_float4(z[4], z[5], z[6], z[7]);
        float kq = 0.0f;  // 16 lanes hold a token
#pragma unroll
        for (int j = 0; j < 8; ++j) kq = fmaf(x[j], z[j], kq);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, o);
        if (tid % 16 == 0) s.kq[t] = kq;
    }
    for (int e = tid; e < kTokens * kCtaCols<RP> / 8; e += kThreads) {
        const int t = e / (kCtaCols<RP> / 8), d = e % (kCtaCols<RP> / 8) * 8;
        if (t < m) {
            float x[8];
            load8(io.v.data, (t0 + t) * io.v.token_stride + h * io.v.head_stride + col0 + d, io.dtype, x);
            *reinterpret_cast<float4 *>(&s.v[t][d]) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(&s.v[t][d + 4]) = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
    if (tid < m) {
        s.a[tid] = io.alpha[(t0 + tid) * H + h];
        s.b[tid] = io.beta[(t0 + tid) * H + h];
    }
}

template <int RP>
__global__ void __launch_bounds__(kThreads, RP == 4 ? 2 : 4) prompt_tokens_kernel(PoolView p, PromptIO io)
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
    float c = 1.0f;  // X = c x
    stage<RP>(st[0], io, p.H, h, col0, first, min(len, kTokens));
    __syncthreads();
    for (int t0 = 0; t0 < len; t0 += kTokens) {
        const Staged<RP> &s = st[t0 / kTokens & 1];
        if (t0 + kTokens < len) stage<RP>(st[(t0 / kTokens & 1) ^ 1], io, p.H, h, col0, first + t0 + kTokens, min(len - t0 - kTokens, kTokens));
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
            float vk[kCols], vq[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                vk[j] = sk[j].x + sk[j].y;
                vq[j] = sq[j].x + sq[j].y;
            }
#pragma unroll
            for (int o = RP / 2; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    vk[j] += __shfl_xor_sync(0xffffffffu, vk[j], o);
                    vq[j] += __shfl_xor_sync(0xffffffffu, vq[j], o);
                }
            const float a = s.a[t], beta = s.b[t], kq = s.kq[t];
            c *= a;
            if (!(fabsf(c) >= 0x1p-20f && fabsf(c) <= 0x1p20f)) {  // the same for every thread of the head
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) x[b][j][i] = make_float2(x[b][j][i].x * c, x[b][j][i].y * c);
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    vk[j] *= c;
                    vq[j] *= c;
                }
                c = 1.0f;
            }
            const float inv = __frcp_rn(c);
            const float4 v4 = *reinterpret_cast<const float4 *>(&s.v[t][col]);
            const float v[kCols] = {v4.x, v4.y, v4.z, v4.w};
            float u[kCols], y[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
                u[j] = beta * fmaf(-c, vk[j], v[j]);
                y[j] = fmaf(c, vq[j], u[j] * kq);
                u[j] *= inv;
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int j = 0; j < kCols; ++j) {
                    const float2 uu = make_float2(u[j], u[j]);
                    x[b][j][0] = fma2(make_float2(k4[b].x, k4[b].y), uu, x[b][j][0]);
                    x[b][j][1] = fma2(make_float2(k4[b].z, k4[b].w), uu, x[b][j][1]);
                }
            if (r == 0) {
                const int64_t at = ((first + t0 + t) * p.H + h) * kD + col0 + col;
                if (io.dtype == STQ_F32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(io.y) + at) = make_float4(y[0], y[1], y[2], y[3]);
                } else {
                    uint2 w;
                    if (io.dtype == STQ_BF16) {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
                        w = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                    } else {
                        const __half2 lo = __floats2half2_rn(y[0], y[1]), hi = __floats2half2_rn(y[2], y[3]);
                        w = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                    }
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(io.y) + at) = w;
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float *to = S + static_cast<size_t>(4 * (r + RP * b) + 2 * i) * kD;
            *reinterpret_cast<float4 *>(to) = make_float4(c * x[b][0][i].x, c * x[b][1][i].x, c * x[b][2][i].x, c * x[b][3][i].x);
            *reinterpret_cast<float4 *>(to + kD) = make_float4(c * x[b][0][i].y, c * x[b][1][i].y, c * x[b][2][i].y, c * x[b][3][i].y);
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
    if (units >= 256) return launch_tokens<4>(p, io, stream);
    return units >= 128 ? launch_tokens<8>(p, io, stream) : launch_tokens<16>(p, io, stream);
}

}  // namespace stq
