// Group norm with an activation, channels last, and its gradients, fp32
// arithmetic. x is [N, S, C]; group g of sample n is its S rows' channels
// [g C/G, (g+1) C/G), M = S C/G values:
//   mean = sum x / M,  rstd = (sum (x - mean)^2 / M + eps)^-1/2,
//   z = (x - mean) rstd w_c + b_c,  y = act(z).
// Gradients, with h = (x - mean) rstd, d = dy act'(z), u = d w_c:
//   dx = rstd (u - mean_group(u) - h mean_group(u h)),
//   dw_c = sum_{n,s} d h,  db_c = sum_{n,s} d.
#include "group_norm.h"

namespace dp {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ld(const float *p, size_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p, size_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void st(float *p, size_t i, float x) { p[i] = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, size_t i, float x) { p[i] = __float2bfloat16_rn(x); }

__device__ __forceinline__ float act_fwd(float z, int act)
{
    return act == DP_ACT_SILU ? z / (1.f + expf(-z)) : z;
}
// act'(z); SiLU: p (1 + z (1 - p)) with p = sigmoid(z)
__device__ __forceinline__ float act_grad(float z, int act)
{
    if (act != DP_ACT_SILU) return 1.f;
    const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
    const float p = z >= 0.f ? r : e * r, m = z >= 0.f ? e * r : r;   // sigmoid(z), 1 - sigmoid(z)
    return p * (1.f + z * m);
}

// sums over the CTA, the same in every thread
__device__ __forceinline__ float2 block_sum(float a, float b)
{
    __shared__ float2 red[kThreads / 32];
    __syncthreads();
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, m);
        b += __shfl_xor_sync(0xffffffffu, b, m);
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
        a += red[i].x;
        b += red[i].y;
    }
    return make_float2(a, b);
}

// One CTA per (sample, group): the mean, the squared distances from it, the
// outputs, each in a walk over the group's values.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gn_forward_kernel(GroupNorm p)
{
    const T *x = (const T *)p.x, *w = (const T *)p.weight, *b = (const T *)p.bias;
    T *y = (T *)p.y;
    const int W = p.C / p.G, g = blockIdx.x % p.G, n = blockIdx.x / p.G;
    const size_t base = (size_t)n * p.S * p.C + (size_t)g * W, m = (size_t)p.S * W;
    const auto at = [&](size_t i) { return base + (i / W) * p.C + i % W; };
    float sum = 0.f;
    for (size_t i = threadIdx.x; i < m; i += kThreads) sum += ld(x, at(i));
    const float mean = block_sum(sum, 0.f).x / (float)m;
    float sq = 0.f;
    for (size_t i = threadIdx.x; i < m; i += kThreads) {
        const float d = ld(x, at(i)) - mean;
        sq = fmaf(d, d, sq);
    }
    const float rstd = 1.f / sqrtf(block_sum(sq, 0.f).x / (float)m + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[blockIdx.x] = mean;
        if (p.rstd) p.rstd[blockIdx.x] = rstd;
    }
    for (size_t i = threadIdx.x; i < m; i += kThreads) {
        const int c = g * W + (int)(i % W);
        float z = (ld(x, at(i)) - mean) * rstd;
        if (w) z *= ld(w, c);
        if (b) z += ld(b, c);
        st(y, at(i), act_fwd(z, p.act));
    }
}

template <typename T>
__device__ __forceinline__ float2 grad_of(const GroupNorm &p, size_t i, int c, float mean, float rstd)
{
    const float h = (ld((const T *)p.x, i) - mean) * rstd;
    float z = h;
    if (p.weight) z *= ld((const T *)p.weight, c);
    if (p.bias) z += ld((const T *)p.bias, c);
    return make_float2(ld((const T *)p.dy, i) * act_grad(z, p.act), h);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
gn_backward_kernel(GroupNorm p)
{
    const int W = p.C / p.G, g = blockIdx.x % p.G, n = blockIdx.x / p.G;
    const size_t base = (size_t)n * p.S * p.C + (size_t)g * W, m = (size_t)p.S * W;
    const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
    const auto at = [&](size_t i) { return base + (i / W) * p.C + i % W; };
    const auto u_of = [&](size_t i, float &h) {
        const int c = g * W + (int)(i % W);
        const float2 dh = grad_of<T>(p, at(i), c, mean, rstd);
        h = dh.y;
        return p.weight ? dh.x * ld((const T *)p.weight, c) : dh.x;
    };
    float su = 0.f, suh = 0.f, h;
    for (size_t i = threadIdx.x; i < m; i += kThreads) {
        const float u = u_of(i, h);
        su += u;
        suh = fmaf(u, h, suh);
    }
    const float2 s = block_sum(su, suh);
    const float mu = s.x / (float)m, muh = s.y / (float)m;
    for (size_t i = threadIdx.x; i < m; i += kThreads) {
        const float u = u_of(i, h);
        st((T *)p.dx, at(i), rstd * (u - mu - h * muh));
    }
}

// Channel sums in two steps without atomics: CTA (slice, 32 channels) adds
// its rows, then one thread per channel adds the slices in order.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gn_channel_partial_kernel(GroupNorm p, int slices, float *part)
{
    __shared__ float red[2][kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.y * 32 + lane;
    const long long rows = (long long)p.N * p.S, per = (rows + slices - 1) / slices;
    const long long r0 = blockIdx.x * per, r1 = r0 + per < rows ? r0 + per : rows;
    float dw = 0.f, db = 0.f;
    if (c < p.C) {
        const int g = c / (p.C / p.G);
        for (long long r = r0 + warp; r < r1; r += kThreads / 32) {
            const size_t ng = (size_t)(r / p.S) * p.G + g;
            const float2 dh = grad_of<T>(p, (size_t)r * p.C + c, c, p.mean[ng], p.rstd[ng]);
            dw = fmaf(dh.x, dh.y, dw);
            db += dh.x;
        }
    }
    red[0][warp][lane] = dw;
    red[1][warp][lane] = db;
    __syncthreads();
    if (warp < 2 && c < p.C) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) s += red[warp][i][lane];
        part[((size_t)blockIdx.x * 2 + warp) * p.C + c] = s;
    }
}

__global__ void gn_channel_sum_kernel(GroupNorm p, int slices, const float *part)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= 2 * p.C) return;
    const int which = i / p.C, c = i - which * p.C;
    float s = 0.f;
    for (int k = 0; k < slices; ++k) s += part[((size_t)k * 2 + which) * p.C + c];
    float *dst = which ? p.dbias : p.dweight;
    if (dst) dst[c] = s;
}

int channel_slices(const GroupNorm &p)
{
    const long long rows = (long long)p.N * p.S;
    return (int)(rows < 64 ? 1 : rows / 64 < 256 ? rows / 64 : 256);
}

template <typename T>
cudaError_t forward_typed(const GroupNorm &p)
{
    gn_forward_kernel<T><<<(unsigned)(p.N * p.G), kThreads, 0, p.stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward_typed(const GroupNorm &p)
{
    gn_backward_kernel<T><<<(unsigned)(p.N * p.G), kThreads, 0, p.stream>>>(p);
    if (p.dweight || p.dbias) {
        const int k = channel_slices(p);
        gn_channel_partial_kernel<T><<<dim3(k, (p.C + 31) / 32), kThreads, 0, p.stream>>>(p, k, p.scratch);
        gn_channel_sum_kernel<<<(2 * p.C + 255) / 256, 256, 0, p.stream>>>(p, k, p.scratch);
    }
    return cudaGetLastError();
}

}  // namespace

size_t gn_forward_scratch_bytes(const GroupNorm &) { return 0; }

size_t gn_backward_scratch_bytes(const GroupNorm &p) { return (size_t)channel_slices(p) * 2 * p.C * sizeof(float); }

cudaError_t launch_gn_forward(const GroupNorm &p)
{
    return p.dtype == DP_F32 ? forward_typed<float>(p) : forward_typed<__nv_bfloat16>(p);
}

cudaError_t launch_gn_backward(const GroupNorm &p)
{
    return p.dtype == DP_F32 ? backward_typed<float>(p) : backward_typed<__nv_bfloat16>(p);
}

}  // namespace dp
