// Linear attention with a decay for each head on the tensor cores (tcgen05,
// TMEM, TMA): bf16 rows, fp32 sums and states, chunks of 128 rows.
// linear_attn.h states the recurrence and its chunked form.
//
// Per chunk (X, Y, Z: its 128 rows; E: the state entering it, fp32 in
// registers, its bf16 copy in shared memory):
//   A  = X Y^T                 MMA, then gamma^|r-s| and the causal mask in
//                              fp32, rounded to bf16 into TMEM
//   O  = X E                   MMA, its rows scaled by gamma^(r'+o) in TMEM
//   O += A Z                   MMA (A from TMEM), rounded to bf16, TMA store
//   B  = (w Y)^T Z             MMA (w Y from TMEM)
//   E  = gamma^R E + B         registers
// B does not depend on E, so the chunks' MMAs do not wait for one another;
// the one recurrence is the last line.
//
// Roundings. A and the copy of E that the readout uses are rounded to bf16
// (2^-9 of each term, as much as the inputs carry). The state itself is an
// fp32 result that runs on over the whole sequence, so w Y is not rounded:
// the fp32 product is cut into three bf16 terms (8 bits each, exact), and B
// is the sum of three MMAs, the small terms first. The MMAs only add within
// a chunk; the sum over chunks is an fp32 multiply-add in registers.
//
// One CTA runs one segment of one (sequence, head). With P > 1 a cluster of P
// CTAs holds the segments of one sequence: each first runs B and E alone over
// its rows, the segments' states go through global memory, and each CTA then
// starts from the decayed sum of those before it.
#include "linear_attn.h"
#include "sm100.cuh"
#include "tensor_map.h"

namespace dp {
namespace {

using namespace sm100;

constexpr int kC = 128;
constexpr int kThreads = 512;
// warps 0-3 scores and output, 4-11 weighted keys and state, then one each:
constexpr int kStateWarp = 4, kLoadWarp = 12, kOutMmaWarp = 13, kStateMmaWarp = 14, kStoreWarp = 15;
constexpr int kOutWarps = 4, kStateWarps = 8;
constexpr uint32_t kTries = 1u << 22;
constexpr uint32_t kSub = 16384;    // one [128 rows][64 columns] bf16 tile, 128-byte swizzle

// TMEM columns (fp32 lanes = rows of the chunk, or of the state)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColA = 0;       // A, fp32; its bf16 form overwrites the first half
constexpr uint32_t kColY = 128;     // w Y of 64 rows: three terms of 32 columns
constexpr uint32_t kColB = 224;
constexpr uint32_t kColO = 352;

enum {
    bFullX, bFullY = bFullX + 2, bFullZ = bFullY + 2, bEmptyX = bFullZ + 2, bEmptyY = bEmptyX + 2,
    bEmptyZ = bEmptyY + 2, bAFull = bEmptyZ + 2, bAReady, bInterFull, bOutFull, bOutFree, bStaged, bStored,
    bYReady, bYFree, bBFull, bStateReady, bZReady, bFinOut, bFinState, kBars
};

template <int DXP, int DZP> struct Layout {
    static constexpr int nx = DXP / 64, nz = DZP / 64;
    static constexpr bool own_stage = DZP > DXP;           // else the output tile goes over X's
    static constexpr uint32_t stage = (2 * nx + nz) * kSub;
    static constexpr uint32_t off_y = nx * kSub, off_z = 2 * nx * kSub;
    static constexpr uint32_t off_e = 2 * stage;           // bf16 state [DXP][DZP]
    static constexpr uint32_t e_sub = DXP * 128;
    static constexpr uint32_t off_out = off_e + nz * e_sub;
    static constexpr uint32_t off_aux = off_out + (own_stage ? nz * kSub : 0);
    static constexpr uint32_t aux = 2048;
    static constexpr uint32_t bytes = off_aux + aux + 1024;
};

struct Params {
    int N, T, H, Dx, Dz, max_T, P;
    const float *log_decay, *init;
    float *fin, *part;
    const int *cu;
    uint32_t *status;
    int state_t;
};

struct Cta {
    uint8_t *base;
    uint64_t *bar;
    float *pw;                    // gamma^0 .. gamma^128
    float2 *pc;                   // gamma^128, gamma^(rows of the ragged chunk), as two fp32 each
    volatile uint32_t *abort;
    uint32_t *status;
    uint32_t tmem;
    LaSegment g;
    int chunks;                   // of this segment
    int own_chunks;               // chunks of the first phase (the segment's own state), 0 or `chunks`
    bool has0;                    // a state enters the segment
    bool packed;
    int updates;                  // chunks of the second phase that update the state

    __device__ __forceinline__ bool wait(int b, uint32_t parity) const
    {
        if (mbar_wait(&bar[b], parity, kTries, abort)) return true;
        *abort = 1;
        if (status) atomicCAS(status, 0u, (uint32_t)kDevTimeout);
        return false;
    }
    // the same for a whole warp, which agrees on the answer
    __device__ __forceinline__ bool wait_warp(int b, uint32_t parity) const
    {
        return __all_sync(0xffffffffu, wait(b, parity));
    }
    // chunk i of a phase in processing order: its first row, live rows
    template <bool REV> __device__ __forceinline__ int row(int i) const
    {
        return g.begin + (REV ? chunks - 1 - i : i) * kC;
    }
    template <bool REV> __device__ __forceinline__ int live(int i) const
    {
        const int n = g.end - row<REV>(i);
        return n < kC ? n : kC;
    }
};

// D[tmem] (+)= A[tmem, bf16 pairs] * B[smem desc]; issued by one thread
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16 lanes x 16 columns: register 2j holds lane t/4, column 4j + t%4,
// register 2j+1 the lane 8 above it
__device__ __forceinline__ void tmem_st_16x16(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, const void *src, int c0, int c1, int c2, int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

__device__ __forceinline__ void arrive_warp(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ------------------------------------------------------------------ loads
template <int DXP, int DZP, bool REV>
__device__ void load_role(const Cta &c, const CUtensorMap *mx, const CUtensorMap *my, const CUtensorMap *mz)
{
    using L = Layout<DXP, DZP>;
    const int b = c.packed ? 0 : c.g.n;
    const int t0 = c.packed ? (int)c.g.row0 : 0;
    const int total = c.own_chunks + c.chunks;
    bool ok = true;
    int i = 0;
    for (; i < total && ok; ++i) {
        const int st = i & 1, use = i >> 1;
        const bool second = i >= c.own_chunks;
        const int j = second ? i - c.own_chunks : i;
        const int t = t0 + c.row<REV>(j);
        uint8_t *s = c.base + st * L::stage;
        if (second) {
            if (j >= 2) ok = c.wait(bEmptyX + st, ((j >> 1) - 1) & 1);
            if (!ok) break;
            mbar_arrive_expect_tx(&c.bar[bFullX + st], L::nx * kSub);
            for (int u = 0; u < L::nx; ++u) tma_load_4d(s + u * kSub, mx, &c.bar[bFullX + st], 64 * u, c.g.h, t, b);
        }
        if (use >= 1 && !(ok = c.wait(bEmptyY + st, (use - 1) & 1))) break;
        mbar_arrive_expect_tx(&c.bar[bFullY + st], L::nx * kSub);
        for (int u = 0; u < L::nx; ++u)
            tma_load_4d(s + L::off_y + u * kSub, my, &c.bar[bFullY + st], 64 * u, c.g.h, t, b);
        if (use >= 1 && !(ok = c.wait(bEmptyZ + st, (use - 1) & 1))) {
            ++i;   // X and Y of this chunk are on their way
            break;
        }
        mbar_arrive_expect_tx(&c.bar[bFullZ + st], L::nz * kSub);
        for (int u = 0; u < L::nz; ++u)
            tma_load_4d(s + L::off_z + u * kSub, mz, &c.bar[bFullZ + st], 64 * u, c.g.h, t, b);
    }
    if (ok) return;
    // A wait ran out: let the copies in flight land (bounded) before the
    // shared memory goes away. Stage st was last loaded at chunk k.
    uint32_t none = 0;
    for (int k = i > 2 ? i - 2 : 0; k < i + 1 && k < total; ++k) {
        const int st = k & 1, use = k >> 1, j = k - c.own_chunks;
        if (j >= 0) mbar_wait(&c.bar[bFullX + st], (j >> 1) & 1, 1u << 14, &none);
        mbar_wait(&c.bar[bFullY + st], use & 1, 1u << 14, &none);
        mbar_wait(&c.bar[bFullZ + st], use & 1, 1u << 14, &none);
    }
}

// ------------------------------------------------------------------ MMAs of scores and output
template <int DXP, int DZP, bool REV>
__device__ void out_mma_role(const Cta &c)
{
    using L = Layout<DXP, DZP>;
    const uint32_t base = smem_addr(c.base), dA = c.tmem + kColA, dO = c.tmem + kColO;
    int inter = 0;
    for (int j = 0; j < c.chunks; ++j) {
        const int i = c.own_chunks + j, st = i & 1, live = c.live<REV>(j);
        const uint32_t sx = base + st * L::stage, sy = sx + L::off_y, sz = sx + L::off_z;
        if (!c.wait(bFullX + st, (j >> 1) & 1) || !c.wait(bFullY + st, (i >> 1) & 1)) break;
        // A's columns are free once the last chunk's A Z has completed
        if (j > 0 && !c.wait(bOutFull, (j - 1) & 1)) break;
        tc_fence_after();
        for (int k = 0; k < DXP / 16; ++k)
            mma_ss(dA, sdesc_sw128(sx + (k >> 2) * kSub + (k & 3) * 32, 0, 1024),
                   sdesc_sw128(sy + (k >> 2) * kSub + (k & 3) * 32, 0, 1024), idesc_bf16(kC, kC, false, false), k > 0);
        mma_commit(&c.bar[bAFull]);
        mma_commit(&c.bar[bEmptyY + st]);
        const bool state = c.has0 || j > 0;
        if (j > 0 && !c.wait(bOutFree, (j - 1) & 1)) break;
        if (state) {
            if (!c.wait(bStateReady, inter & 1)) break;
            tc_fence_after();
            for (int k = 0; k < DXP / 16; ++k)
                mma_ss(dO, sdesc_sw128(sx + (k >> 2) * kSub + (k & 3) * 32, 0, 1024),
                       sdesc_sw128(base + L::off_e + k * 2048, L::e_sub, 1024), idesc_bf16(kC, DZP, false, true), k > 0);
            mma_commit(&c.bar[bInterFull]);
            ++inter;
        }
        if (!c.wait(bFullZ + st, (i >> 1) & 1)) break;
        if (c.packed && live < kC && !c.wait(bZReady, 0)) break;
        if (!c.wait(bAReady, j & 1)) break;
        tc_fence_after();
        for (int k = 0; k < (live + 15) / 16; ++k)
            mma_ts(dO, dA + k * 8, sdesc_sw128(sz + k * 2048, kSub, 1024), idesc_bf16(kC, DZP, false, true),
                   state || k > 0);
        mma_commit(&c.bar[bOutFull]);
        mma_commit(&c.bar[bEmptyZ + st]);
    }
    mma_commit(&c.bar[bFinOut]);
    uint32_t none = 0;
    mbar_wait(&c.bar[bFinOut], 0, kTries, &none);
}

// ------------------------------------------------------------------ MMAs of the state
template <int DXP, int DZP, bool REV>
__device__ void state_mma_role(const Cta &c)
{
    using L = Layout<DXP, DZP>;
    const uint32_t base = smem_addr(c.base), dB = c.tmem + kColB, aY = c.tmem + kColY;
    int half = 0;
    for (int i = 0; i < c.own_chunks + c.updates; ++i) {
        const bool second = i >= c.own_chunks;
        const int st = i & 1, live = c.live<REV>(second ? i - c.own_chunks : i);
        const uint32_t sz = base + st * L::stage + L::off_z;
        if (!c.wait(bFullZ + st, (i >> 1) & 1)) break;
        bool ok = true;
        for (int hh = 0; hh < 2; ++hh, ++half) {
            if (!(ok = c.wait(bYReady, half & 1))) break;
            tc_fence_after();
            const int rows = live - 64 * hh < 64 ? live - 64 * hh : 64;
            for (int term = 2; term >= 0; --term)
                for (int k = 0; k < (rows + 15) / 16; ++k)
                    mma_ts(dB, aY + term * 32 + k * 8, sdesc_sw128(sz + (4 * hh + k) * 2048, kSub, 1024),
                           idesc_bf16(kC, DZP, false, true), hh > 0 || term < 2 || k > 0);
            mma_commit(&c.bar[bYFree]);
        }
        if (!ok) break;
        mma_commit(&c.bar[bBFull]);
        mma_commit(&c.bar[bEmptyZ + st]);
        if (!second) mbar_arrive(&c.bar[bEmptyZ + st]);   // the first phase has no A Z
    }
    mma_commit(&c.bar[bFinState]);
    uint32_t none = 0;
    mbar_wait(&c.bar[bFinState], 0, kTries, &none);
}

// ------------------------------------------------------------------ scores and output (lane = row of the chunk)
template <int DXP, int DZP, bool REV>
__device__ void out_role(const Cta &c, __nv_bfloat16 *out, int H, int Dz)
{
    using L = Layout<DXP, DZP>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = 32 * warp + lane;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t tA = c.tmem + lanes + kColA, tO = c.tmem + lanes + kColO;
    int inter = 0;
    for (int j = 0; j < c.chunks; ++j) {
        const int live = c.live<REV>(j), st = (c.own_chunks + j) & 1;
        const bool state = c.has0 || j > 0;
        if (!c.wait_warp(bAFull, j & 1)) return;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {   // columns 32b .. 32b+31
            uint32_t u[32], w[16];
            if (REV ? b < warp : b > warp) {
#pragma unroll
                for (int q = 0; q < 16; ++q) w[q] = 0;
            } else {
                tmem_ld32(tA + 32 * b, u);
                tmem_wait_ld();
                float f[32];
                if (b == warp) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const int far = REV ? q - lane : lane - q;
                        f[q] = far >= 0 ? __uint_as_float(u[q]) * c.pw[far >= 0 ? far : 0] : 0.f;
                    }
                } else {
                    // |r - s| = [distance to the near edge of the column block] + [column within it]
                    const float wr = c.pw[REV ? 32 * (b - warp) - lane : 32 * (warp - b) + lane - 31];
#pragma unroll
                    for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(u[q]) * (wr * c.pw[REV ? q : 31 - q]);
                }
                if (REV && live < kC) {   // columns past the sequence are on the seen side here
#pragma unroll
                    for (int q = 0; q < 32; ++q) f[q] = 32 * b + q < live ? f[q] : 0.f;
                }
#pragma unroll
                for (int q = 0; q < 16; ++q) w[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
            }
            // the fp32 columns that this overwrites (of blocks <= b) have been read
            tmem_st16(tA + 16 * b, w);
        }
        if (state) {
            if (!c.wait_warp(bInterFull, inter++ & 1)) return;
            tc_fence_after();
            const int e = REV ? live - 1 - r : r + 1;
            const float wr = e >= 0 ? c.pw[e] : 0.f;
#pragma unroll 1
            for (int b = 0; b < DZP / 32; ++b) {
                uint32_t u[32];
                tmem_ld32(tO + 32 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q) u[q] = __float_as_uint(wr * __uint_as_float(u[q]));
                tmem_st32(tO + 32 * b, u);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&c.bar[bAReady]);
        if (!c.wait_warp(bOutFull, j & 1)) return;
        tc_fence_after();
        if (L::own_stage && j > 0 && !c.wait_warp(bStored, (j - 1) & 1)) return;
        uint8_t *tile = c.base + (L::own_stage ? L::off_out : st * L::stage);
#pragma unroll 1
        for (int b = 0; b < DZP / 32; ++b) {
            uint32_t u[32];
            tmem_ld32(tO + 32 * b, u);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 v;
                v.x = pack_bf16x2(__uint_as_float(u[8 * q]), __uint_as_float(u[8 * q + 1]));
                v.y = pack_bf16x2(__uint_as_float(u[8 * q + 2]), __uint_as_float(u[8 * q + 3]));
                v.z = pack_bf16x2(__uint_as_float(u[8 * q + 4]), __uint_as_float(u[8 * q + 5]));
                v.w = pack_bf16x2(__uint_as_float(u[8 * q + 6]), __uint_as_float(u[8 * q + 7]));
                *(uint4 *)(tile + (b >> 1) * kSub + sw128_offset(r, (b & 1) * 4 + q)) = v;
            }
        }
        tc_fence_before();
        arrive_warp(&c.bar[bOutFree]);
        if (c.packed && live < kC) {
            // the last rows of a packed sequence: no TMA store, which would
            // run on into the next sequence; each warp writes its own rows
            __syncwarp();
            const int per = Dz / 8;
            for (int q = lane; q < 32 * per; q += 32) {
                const int rr = 32 * warp + q / per, ch = q % per;
                if (rr < live)
                    *(uint4 *)(out + ((c.g.row0 + c.row<REV>(j) + rr) * H + c.g.h) * Dz + ch * 8) =
                        *(const uint4 *)(tile + (ch >> 3) * kSub + sw128_offset(rr, ch & 7));
            }
        }
        fence_proxy_async_smem();
        arrive_warp(&c.bar[bStaged]);
    }
}

template <int DXP, int DZP, bool REV>
__device__ void store_role(const Cta &c, const CUtensorMap *mo)
{
    using L = Layout<DXP, DZP>;
    const int b = c.packed ? 0 : c.g.n, t0 = c.packed ? (int)c.g.row0 : 0;
    for (int j = 0; j < c.chunks; ++j) {
        const int st = (c.own_chunks + j) & 1;
        if (!c.wait(bStaged, j & 1)) break;
        const uint8_t *tile = c.base + (L::own_stage ? L::off_out : st * L::stage);
        if (!(c.packed && c.live<REV>(j) < kC)) {
            for (int u = 0; u < L::nz; ++u) tma_store_4d(mo, tile + u * kSub, 64 * u, c.g.h, t0 + c.row<REV>(j), b);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        mbar_arrive(&c.bar[bEmptyX + st]);
        mbar_arrive(&c.bar[bStored]);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ------------------------------------------------------------------ weighted keys and state (lane = row of the state)
template <int DXP, int DZP, bool REV>
struct StateRole {
    using L = Layout<DXP, DZP>;
    static constexpr int kN = DZP / 2;       // state columns of a thread
    const Cta &c;
    const Params &p;
    int warp, lane, quarter, side, dx, dz0;
    bool live_rows;                          // this warp's rows are within DXP
    size_t head;
    float s[kN];
    int half = 0;                            // halves of chunks sent so far

    __device__ __forceinline__ StateRole(const Cta &c_, const Params &p_) : c(c_), p(p_)
    {
        warp = (threadIdx.x >> 5) - kStateWarp;
        lane = threadIdx.x & 31;
        quarter = warp & 3;
        side = warp >> 2;
        dx = 32 * quarter + lane;
        dz0 = side * kN;
        live_rows = 32 * quarter < DXP;
        head = (size_t)c.g.n * p.H + c.g.h;
    }

    // element (dx, dz0 + q) of an [N,H,..] state; every state in global
    // memory is read and written once per segment
    __device__ __forceinline__ void load_scaled(const float *src, float w, bool transposed)
    {
        if (dx >= p.Dx || dz0 >= p.Dz) return;
        if (transposed) {
#pragma unroll
            for (int q = 0; q < kN; ++q)
                if (dz0 + q < p.Dz) s[q] = fmaf(w, __ldcg(src + (size_t)(dz0 + q) * p.Dx + dx), s[q]);
        } else {
#pragma unroll
            for (int q = 0; q < kN; q += 4)
                if (dz0 + q < p.Dz) {
                    const float4 v = __ldcg((const float4 *)(src + (size_t)dx * p.Dz + dz0 + q));
                    s[q] = fmaf(w, v.x, s[q]);
                    s[q + 1] = fmaf(w, v.y, s[q + 1]);
                    s[q + 2] = fmaf(w, v.z, s[q + 2]);
                    s[q + 3] = fmaf(w, v.w, s[q + 3]);
                }
        }
    }
    __device__ __forceinline__ void store(float *dst, bool transposed) const
    {
        if (dx >= p.Dx || dz0 >= p.Dz) return;
        if (transposed) {
#pragma unroll
            for (int q = 0; q < kN; ++q)
                if (dz0 + q < p.Dz) dst[(size_t)(dz0 + q) * p.Dx + dx] = s[q];
        } else {
#pragma unroll
            for (int q = 0; q < kN; q += 4)
                if (dz0 + q < p.Dz)
                    *(float4 *)(dst + (size_t)dx * p.Dz + dz0 + q) = make_float4(s[q], s[q + 1], s[q + 2], s[q + 3]);
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int q = 0; q < kN; ++q) s[q] = 0.f;
    }

    // rows 64 hh + 32 side .. +31 of w Y, transposed into TMEM as three bf16 terms
    __device__ __forceinline__ void send_keys(uint32_t sy, int hh, int live)
    {
        const int r0 = 64 * hh + 32 * side;
        float w[8];
        uint32_t keep[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            keep[q] = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 8 * q + 2 * (lane & 3) + e, n = REV ? r + 1 : live - 1 - r;
                const bool in = r < live;
                w[2 * q + e] = in ? c.pw[n >= 0 ? n : 0] : 0.f;
                keep[q] |= in ? 0xffffu << (16 * e) : 0u;   // rows past the sequence count as zeros
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {    // 16 state rows each
            const int d = 32 * quarter + 16 * x;
            const uint32_t sub = sy + (d >> 6) * kSub;
            const uint32_t chunk = ((d & 63) >> 3) + ((lane >> 3) & 1);
            uint32_t hi[8], mid[8], lo[8];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                ldmatrix_x4_trans(sub + sw128_offset(r0 + 16 * q + 8 * (lane >> 4) + (lane & 7), chunk), hi[4 * q],
                                  hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t pair = hi[q] & keep[q >> 1];
                const float a = __uint_as_float(pair << 16) * w[2 * (q >> 1)];
                const float b = __uint_as_float(pair & 0xffff0000u) * w[2 * (q >> 1) + 1];
                // the top 8 bits of what is left, three times: 24 in all
                const float a1 = a - __uint_as_float(__float_as_uint(a) & 0xffff0000u);
                const float b1 = b - __uint_as_float(__float_as_uint(b) & 0xffff0000u);
                const float a2 = a1 - __uint_as_float(__float_as_uint(a1) & 0xffff0000u);
                const float b2 = b1 - __uint_as_float(__float_as_uint(b1) & 0xffff0000u);
                hi[q] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                mid[q] = __byte_perm(__float_as_uint(a1), __float_as_uint(b1), 0x7632);
                lo[q] = __byte_perm(__float_as_uint(a2), __float_as_uint(b2), 0x7632);
            }
            const uint32_t t = c.tmem + ((uint32_t)d << 16) + kColY + 16 * side;
            tmem_st_16x16(t, hi);
            tmem_st_16x16(t + 32, mid);
            tmem_st_16x16(t + 64, lo);
        }
    }

    // one chunk: w Y out, B in, E <- gamma^R E + B. Chunk i of all, j of its phase.
    __device__ __forceinline__ bool chunk(int i, int j, bool first_phase)
    {
        const int st = i & 1, live = c.live<REV>(j);
        if (!c.wait_warp(bFullY + st, (i >> 1) & 1)) return false;
        if (c.packed && live < kC && !clear_tail(i, live)) return false;
        for (int hh = 0; hh < 2; ++hh, ++half) {
            if (half > 0 && !c.wait_warp(bYFree, (half - 1) & 1)) return false;
            tc_fence_after();
            if (live_rows) send_keys(smem_addr(c.base + st * L::stage + L::off_y), hh, live);
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&c.bar[bYReady]);
        }
        arrive_warp(&c.bar[bEmptyY + st]);
        if (first_phase && warp == 0 && lane == 0) mbar_arrive(&c.bar[bEmptyY + st]);   // there is no X Y^T
        if (!c.wait_warp(bBFull, i & 1)) return false;
        tc_fence_after();
        if (live_rows) {
            const float2 w = live == kC ? c.pc[0] : c.pc[1];
#pragma unroll
            for (int b = 0; b < kN / 32; ++b) {
                uint32_t u[32];
                tmem_ld32(c.tmem + ((uint32_t)(32 * quarter) << 16) + kColB + dz0 + 32 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    s[32 * b + q] = fmaf(s[32 * b + q], w.x, fmaf(s[32 * b + q], w.y, __uint_as_float(u[q])));
            }
        }
        tc_fence_before();
        return true;
    }

    // The rows of Z past the end of a packed sequence belong to the next one:
    // they count as zeros (A and w Y are zero there, but zero times NaN is not).
    __device__ __forceinline__ bool clear_tail(int i, int live)
    {
        const int st = i & 1;
        if (!c.wait_warp(bFullZ + st, (i >> 1) & 1)) return false;
        uint8_t *z = c.base + st * L::stage + L::off_z;
        for (int q = warp * 32 + lane; q < (kC - live) * 8 * L::nz; q += kStateWarps * 32) {
            const int u = q / ((kC - live) * 8), e = q - u * (kC - live) * 8;
            *(uint4 *)(z + u * kSub + (live + (e >> 3)) * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        return true;
    }

    // the bf16 copy that the readout multiplies by
    __device__ __forceinline__ void publish()
    {
        if (live_rows) {
            uint8_t *e = c.base + L::off_e + (DZP == 128 ? side * L::e_sub : 0);
#pragma unroll
            for (int q = 0; q < kN / 8; ++q) {
                uint4 v;
                v.x = pack_bf16x2(s[8 * q], s[8 * q + 1]);
                v.y = pack_bf16x2(s[8 * q + 2], s[8 * q + 3]);
                v.z = pack_bf16x2(s[8 * q + 4], s[8 * q + 5]);
                v.w = pack_bf16x2(s[8 * q + 6], s[8 * q + 7]);
                *(uint4 *)(e + sw128_offset(dx, (DZP == 128 ? 0 : 4 * side) + q)) = v;
            }
        }
        fence_proxy_async_smem();
        arrive_warp(&c.bar[bStateReady]);
    }

    __device__ __forceinline__ void run()
    {
        const size_t cells = (size_t)p.Dx * p.Dz;
        const int last_rank = c.g.len > 0 ? (c.g.len - 1) / c.g.seg : 0;
        bool ok = true;
        clear();
        for (int i = 0; i < c.own_chunks && ok; ++i) ok = chunk(i, i, true);
        if (p.P > 1) {
            if (c.own_chunks > 0) store(p.part + (head * p.P + c.g.rank) * cells, false);
            __threadfence();
            cluster_arrive();
            cluster_wait();
            clear();
        }
        if (!ok) return;
        const float ld = p.log_decay[c.g.h];
        if (p.init)
            load_scaled(p.init + head * cells, la_power(ld, REV ? c.g.len - c.g.end : c.g.begin), p.state_t);
        if (c.g.rank <= last_rank) {
            const int from = REV ? c.g.rank + 1 : 0, to = REV ? last_rank + 1 : c.g.rank;
            for (int q = from; q < to; ++q)
                load_scaled(p.part + (head * p.P + q) * cells,
                            la_power(ld, REV ? q * c.g.seg - c.g.end : c.g.begin - (q + 1) * c.g.seg), false);
        }
        if (c.has0 && c.chunks > 0) publish();
        int inter = 0;
        for (int j = 0; j < c.chunks; ++j) {
            const int i = c.own_chunks + j, live = c.live<REV>(j);
            if (j >= c.updates) {
                // nothing reads the state after this chunk
                if (c.packed && live < kC) {
                    if (!clear_tail(i, live)) return;
                    arrive_warp(&c.bar[bZReady]);
                }
                break;
            }
            if (!chunk(i, j, false)) return;
            if (c.packed && live < kC) arrive_warp(&c.bar[bZReady]);
            if ((c.has0 || j > 0) && !c.wait_warp(bInterFull, inter++ & 1)) return;   // the last copy has been read
            if (j + 1 < c.chunks) publish();
        }
        if (p.fin && c.g.rank == (REV ? 0 : last_rank)) store(p.fin + head * cells, p.state_t);
    }
};

template <int DXP, int DZP, bool REV>
__global__ void __launch_bounds__(kThreads, 1)
la_tc_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
             const __grid_constant__ CUtensorMap mz, const __grid_constant__ CUtensorMap mo, const Params p,
             __nv_bfloat16 *out)
{
    using L = Layout<DXP, DZP>;
    extern __shared__ uint8_t smem_raw[];
    Cta c;
    c.g = la_segment(p.cu, p.N, p.T, p.H, p.max_T, p.P, kC, blockIdx.x);
    if (!c.g.ok) {   // the whole cluster sees the same offsets and leaves together
        if (threadIdx.x == 0 && c.g.h == 0 && c.g.rank == 0) report_bad_sequence(p.status);
        return;
    }
    c.base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    c.bar = (uint64_t *)(c.base + L::off_aux);
    c.pc = (float2 *)(c.bar + kBars);
    c.pw = (float *)(c.pc + 2);
    uint32_t *slot = (uint32_t *)(c.pw + kC + 1);
    c.abort = slot + 1;
    c.status = p.status;
    c.packed = p.cu != nullptr;
    c.chunks = (c.g.end - c.g.begin + kC - 1) / kC;
    const int last_rank = c.g.len > 0 ? (c.g.len - 1) / c.g.seg : 0;
    c.own_chunks = p.P > 1 && (REV ? c.g.rank > 0 : c.g.rank < last_rank) ? c.chunks : 0;
    c.has0 = p.init != nullptr || (REV ? c.g.rank < last_rank : c.g.rank > 0);
    const bool write_fin = p.fin && c.g.rank == (REV ? 0 : last_rank);
    c.updates = write_fin || c.chunks == 0 ? c.chunks : c.chunks - 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float ld = p.log_decay[c.g.h];
    if (threadIdx.x <= kC) c.pw[threadIdx.x] = la_power(ld, threadIdx.x);
    if (threadIdx.x == 160) c.pc[0] = la_power2(ld, kC);
    if (threadIdx.x == 192) c.pc[1] = la_power2(ld, c.g.len % kC);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int n = i == bAReady || i == bOutFree || i == bStaged ? kOutWarps
                          : i == bYReady || i == bStateReady || i == bZReady ? kStateWarps
                          : i == bEmptyY || i == bEmptyY + 1 ? kStateWarps + 1
                          : i == bEmptyZ || i == bEmptyZ + 1 ? 2
                                                             : 1;
            mbar_init(&c.bar[i], n);
        }
        *c.abort = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0 && c.chunks > 0) {
        tma_prefetch_desc(&mx);
        tma_prefetch_desc(&my);
        tma_prefetch_desc(&mz);
        tma_prefetch_desc(&mo);
    }
    if (warp == 0) tmem_alloc(slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = *slot;

    if (warp >= kStateWarp && warp < kLoadWarp) {
        StateRole<DXP, DZP, REV> role(c, p);
        role.run();
    } else {
        if (p.P > 1) cluster_arrive();
        if (warp < kStateWarp) {
            out_role<DXP, DZP, REV>(c, out, p.H, p.Dz);
        } else if (lane == 0) {
            if (warp == kLoadWarp) load_role<DXP, DZP, REV>(c, &mx, &my, &mz);
            else if (warp == kOutMmaWarp) out_mma_role<DXP, DZP, REV>(c);
            else if (warp == kStateMmaWarp) state_mma_role<DXP, DZP, REV>(c);
            else store_role<DXP, DZP, REV>(c, &mo);
        }
        __syncwarp();
        if (p.P > 1) cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(c.tmem, kTmemCols);
}

bool rows_map(CUtensorMap *map, const void *base, int D, const LaPass &p)
{
    const cuuint64_t B = p.cu ? 1 : p.N, T = p.T, H = p.H;
    const cuuint64_t dims[4] = {(cuuint64_t)D, H, T, B};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, H * D * 2, T * H * D * 2};
    const cuuint32_t box[4] = {64, 1, kC, 1};
    return encode(map, base, 4, dims, strides, box);
}

template <int DXP, int DZP, bool REV>
cudaError_t launch_sized(const LaPass &p, const CUtensorMap (&m)[4])
{
    auto kernel = la_tc_kernel<DXP, DZP, REV>;
    constexpr int smem = (int)Layout<DXP, DZP>::bytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const Params pr{p.N, p.T, p.H, p.Dx, p.Dz, p.max_T, p.P, p.log_decay, p.init, p.fin, p.part, p.cu, p.status,
                    p.state_t ? 1 : 0};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((size_t)p.N * p.H * p.P));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = p.stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.P;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], pr, (__nv_bfloat16 *)p.out);
}

template <int DXP, int DZP>
cudaError_t launch_dir(const LaPass &p, const CUtensorMap (&m)[4])
{
    return p.reverse ? launch_sized<DXP, DZP, true>(p, m) : launch_sized<DXP, DZP, false>(p, m);
}

}  // namespace

bool la_tc_supported(int dtype) { return dtype == DP_BF16 && tensor_map_encoder() != nullptr; }

int la_tc_cluster(int N, int H, int max_T)
{
    int P = 1;
    while (P < kLaMaxCluster && (long long)N * H * P * 2 <= 152 && max_T >= 2 * P * kC) P *= 2;
    return P;
}

cudaError_t launch_la_tc(const LaPass &p)
{
    if ((size_t)p.N * p.H == 0) return cudaSuccess;
    CUtensorMap m[4] = {};
    // without rows there is nothing to load: the maps are not used
    if (p.T > 0 && (!rows_map(&m[0], p.x, p.Dx, p) || !rows_map(&m[1], p.y, p.Dx, p) ||
                    !rows_map(&m[2], p.z, p.Dz, p) || !rows_map(&m[3], p.out, p.Dz, p)))
        return cudaErrorInvalidValue;
    if (p.Dx == 128) return p.Dz == 128 ? launch_dir<128, 128>(p, m) : launch_dir<128, 64>(p, m);
    return p.Dz == 128 ? launch_dir<64, 128>(p, m) : launch_dir<64, 64>(p, m);
}

}  // namespace dp
