// Linear attention with a decay for each head: declarations shared by its
// translation units.
//
// Everything the operator computes is one recurrence over a sequence's rows,
// a "pass" (gamma = exp(log_decay[h])):
//   forward   S_t = gamma S_{t-1} + y_t z_t^T         out_t = S_t^T x_t
//   reverse   G_t = y_t z_t^T + gamma G_{t+1}         out_t = G_t^T x_t
// with S_{-1} = init, and gamma G_T := init (a gradient that reaches the
// final state reaches the last token undecayed). `fin` is S_{T-1}, or
// gamma G_0. The outputs are x, y, z = q, k, v forward; the gradients are
//   dq: d_o, v, k forward from h0^T;  dv: k, q, d_o reverse from dh_final
//   (fin: dh0);  dk: v, d_o, q reverse from dh_final^T.
//
// In chunks of C rows, with E the state entering the chunk and r' = r
// forward, C-1-r reverse:
//   out_r = sum_{s on the seen side} gamma^|r-s| (x_r . y_s) z_s
//           + gamma^(r' + o) E^T x_r                       o = 1 forward, 0 reverse
//   E_next = gamma^R E + sum_r gamma^(R-1-r' + 1-o) y_r z_r^T   (R live rows)
#pragma once

#include "internal.h"

namespace dp {

struct LaPass {
    int N, T, H;               // sequences, rows of the time axis, heads
    int Dx, Dz;                // state rows (x, y) and columns (z, out)
    int dtype;                 // dp_dtype of x, y, z, out
    const void *x, *y, *z;
    void *out;
    const float *log_decay;    // [H]
    const float *init;         // [N,H,Dx,Dz], or [N,H,Dz,Dx] with state_t; NULL: zeros
    float *fin;                // as init; NULL: not written
    bool state_t;              // init and fin hold the transposed state
    bool reverse;
    const int *cu;             // packed sequences (NULL: dense)
    int max_T;                 // longest sequence
    int P;                     // segments of a sequence, one CTA each
    float *part;               // states of the segments (P > 1): N H P la_part_cells(..) values
    int shares;                // P == 1: `part` holds kLaShareFlags words and as many states instead
    uint32_t *status;
    cudaStream_t stream;
};

constexpr int kLaMaxCluster = 8, kLaMaxSegments = 32;
constexpr int kLaShareFlags = 1024, kLaMaxShares = kLaShareFlags - 1;

// fp32 values of one segment's state in the workspace (the tensor-core kernel
// pads the state to 128 rows and at least 64 columns, in either orientation)
inline size_t la_part_cells(int Dk, int Dv)
{
    const int d = Dk > Dv ? Dk : Dv;
    return (size_t)128 * (d < 64 ? 64 : d);
}

// CUDA-core kernel: any supported size and type, fp32 arithmetic; a sequence's
// segments are one cluster.
int la_simt_cluster(int N, int H, int max_T);
cudaError_t launch_la_simt(const LaPass &p);

// Tensor-core kernel: bf16, any supported size.
bool la_tc_supported(int dtype);
int la_tc_segments(int N, int H, int T, int max_T, bool packed, int passes, int sms);
cudaError_t launch_la_tc(const LaPass &p);
// The gradients: the passes of dq, dk and dv, each with its own `part`.
// `apart`: dv's final state may lie over dk's initial one, so dv runs after.
cudaError_t launch_la_grad_tc(const LaPass (&p)[3], bool apart);

// One token: state <- gamma state + k v^T, o = state^T q.
struct LaStep {
    int B, H, Dk, Dv, dtype;
    const void *q, *k, *v;
    const float *log_decay;
    float *state;
    void *o;
    cudaStream_t stream;
};
cudaError_t launch_la_step(const LaStep &p);

// ---- the part of a sequence that one CTA runs: rows
// [begin, end) of the sequence, in segments of whole chunks
struct LaSegment {
    int n, h;            // sequence, head
    int rank;            // segment of the sequence
    size_t row0;         // first row of the sequence in the [rows, H, D] layout
    int len, seg;        // rows of the sequence, of a segment
    int begin, end;
    bool ok;
};

__device__ __forceinline__ LaSegment la_segment(const int *cu, int N, int T, int H, int max_T, int P, int chunk,
                                                unsigned block)
{
    LaSegment g;
    const unsigned nh = block / P;
    g.rank = (int)(block - nh * P);
    g.n = (int)(nh / H);
    g.h = (int)(nh - (unsigned)g.n * H);
    const SeqRange sq = seq_range(cu, g.n, N, T, max_T);
    g.ok = sq.ok;
    g.row0 = (size_t)sq.b_map * T + sq.t0;
    g.len = sq.len;
    const int chunks = (g.len + chunk - 1) / chunk;
    g.seg = (chunks + P - 1) / P * chunk;
    g.begin = g.rank * g.seg < g.len ? g.rank * g.seg : g.len;
    g.end = g.begin + g.seg < g.len ? g.begin + g.seg : g.len;
    return g;
}

// gamma^n for a log decay; n = 0 gives 1 for every decay (a decay of 0 included).
__device__ __forceinline__ float la_power(float log_decay, int n)
{
    return n == 0 ? 1.f : expf((float)n * log_decay);
}

// gamma^n as the sum of two fp32 values, to about 2^-28 of it. The state is
// multiplied by the same power once per chunk, so an error of that power
// grows with the number of chunks that a head remembers. In pairs of fp32
// (the 64-bit unit would take microseconds): n log gamma = k ln 2 + r exactly
// enough, exp(r / 8) by its series, squared three times, times 2^k.
__device__ __forceinline__ float2 la_power2(float log_decay, int n)
{
    if (n == 0) return make_float2(1.f, 0.f);
    const float m = (float)n, xh = m * log_decay;
    if (!(xh > -104.f && xh < 88.f)) return make_float2(expf(xh), 0.f);   // 0, overflow, NaN
    const float xl = fmaf(m, log_decay, -xh);
    const float k = rintf(xh * 1.44269504f);
    // ln 2 in two parts; k times the first (16 bits) is exact
    const float a = fmaf(k, -0.693145751953125f, xh), t = k * 1.42860682e-6f;
    const float rh = a - t, rl = ((a - rh) - t) + xl - fmaf(k, 1.42860682e-6f, -t);
    const float u = 0.125f * rh, v = 0.125f * rl;
    // exp(u + v) = 1 + u + (v + u v + u^2/2 + ..): |u| < 0.044, |v| < 2^-20
    float q = fmaf(u, 1.f / 720.f, 1.f / 120.f);
    q = fmaf(u, q, 1.f / 24.f);
    q = fmaf(u, q, 1.f / 6.f);
    q = fmaf(u, q, 0.5f);
    q = fmaf(u * u, q, fmaf(u, v, v));
    float h = 1.f + u, l = (u - (h - 1.f)) + q;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const float p = h * h;
        l = fmaf(2.f * h, l, fmaf(l, l, fmaf(h, h, -p)));
        h = p;
    }
    const float s = h + l;
    l -= s - h;
    return make_float2(ldexpf(s, (int)k), ldexpf(l, (int)k));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace dp
