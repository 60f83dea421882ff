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
constexpr int kThreads = 640;
// warps 0-3 scores, 4-7 output, 8-15 weighted keys and state, then one each:
constexpr int kOutWarp = 4, kStateWarp = 8, kLoadWarp = 16, kOutMmaWarp = 17, kStateMmaWarp = 18, kStoreWarp = 19;
constexpr int kOutWarps = 4, kStateWarps = 8;
// registers after the move: two warpgroups of 128 a thread, three of 72, out
// of the 640 x 96 that the kernel is launched with
constexpr int kMovedRegs = 2 * 128 * 128 + 3 * 128 * 72;
constexpr uint32_t kTries = 1u << 22;
constexpr uint32_t kSub = 16384;    // one [128 rows][64 columns] bf16 tile, 128-byte swizzle

// TMEM columns (fp32 lanes = rows of the chunk, or of the state)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColA = 0;       // A, fp32; its bf16 form overwrites the first half
constexpr uint32_t kColY = 128;     // w Y of 32 rows, two buffers: three terms of 16 columns each
constexpr uint32_t kColB = 224;
constexpr uint32_t kColO = 352;

enum {
    bFullX, bFullY = bFullX + 2, bFullZ = bFullY + 2, bEmptyX = bFullZ + 2, bEmptyY = bEmptyX + 2,
    bEmptyZ = bEmptyY + 2, bAFull = bEmptyZ + 2, bAReady, bInterFull, bInterReady, bOutFull, bOutFree, bStaged, bStored,
    bYReady, bYFree = bYReady + 2, bBFull = bYFree + 2, bBFree, bStateReady, bZReady, bFinOut, bFinState, kBars
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
    uint32_t pw;                  // shared: gamma^0 .. gamma^128
    uint32_t pr;                  // shared: gamma^31 .. gamma^0
    uint32_t pc;                  // shared: gamma^128, gamma^(rows of the ragged chunk), as two fp32 each
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

// 16 lanes x 8 columns: register 2j holds lane t/4, column 4j + t%4,
// register 2j+1 the lane 8 above it
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ float lds(uint32_t a)
{
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a));
    return f;
}
__device__ __forceinline__ float4 lds4(uint32_t a)
{
    float4 f;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(a));
    return f;
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
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
// The issuing thread's own instructions are on the MMAs' path (an MMA takes
// about 68 cycles): descriptors are built once and advanced by an addition
// to their address field, and the loops over a whole chunk are unrolled.
template <int DXP, int DZP, bool REV>
__device__ void out_mma_role(const Cta &c)
{
    using L = Layout<DXP, DZP>;
    const uint32_t base = smem_addr(c.base), dA = c.tmem + kColA, dO = c.tmem + kColO;
    const uint64_t kmajor = sdesc_sw128(base, 0, 1024), zmajor = sdesc_sw128(base + L::off_z, kSub, 1024);
    const uint64_t emajor = sdesc_sw128(base + L::off_e, L::e_sub, 1024);
    int inter = 0;
    for (int j = 0; j < c.chunks; ++j) {
        const int i = c.own_chunks + j, st = i & 1, live = c.live<REV>(j);
        const uint32_t stage = (uint32_t)st * (L::stage >> 4);
        const uint64_t x = kmajor + stage, y = x + (L::off_y >> 4), z = zmajor + stage;
        if (!c.wait(bFullX + st, (j >> 1) & 1) || !c.wait(bFullY + st, (i >> 1) & 1)) break;
        // A's columns are free once the last chunk's A Z has completed
        if (j > 0 && !c.wait(bOutFull, (j - 1) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < DXP / 16; ++k)
            mma_ss(dA, x + ((k >> 2) * (kSub >> 4) + (k & 3) * 2), y + ((k >> 2) * (kSub >> 4) + (k & 3) * 2),
                   idesc_bf16(kC, kC, false, false), k > 0);
        mma_commit(&c.bar[bAFull]);
        mma_commit(&c.bar[bEmptyY + st]);
        const bool state = c.has0 || j > 0;
        if (j > 0 && !c.wait(bOutFree, (j - 1) & 1)) break;
        if (state) {
            if (!c.wait(bStateReady, inter & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DXP / 16; ++k)
                mma_ss(dO, x + ((k >> 2) * (kSub >> 4) + (k & 3) * 2), emajor + k * 128,
                       idesc_bf16(kC, DZP, false, true), k > 0);
            mma_commit(&c.bar[bInterFull]);
        }
        if (!c.wait(bFullZ + st, (i >> 1) & 1)) break;
        if (c.packed && live < kC && !c.wait(bZReady, 0)) break;
        if (state && !c.wait(bInterReady, inter++ & 1)) break;
        if (!c.wait(bAReady, j & 1)) break;
        tc_fence_after();
        if (live > kC - 16) {
#pragma unroll
            for (int k = 0; k < kC / 16; ++k)
                mma_ts(dO, dA + k * 8, z + k * 128, idesc_bf16(kC, DZP, false, true), state || k > 0);
        } else {
            for (int k = 0; k < (live + 15) / 16; ++k)
                mma_ts(dO, dA + k * 8, z + k * 128, idesc_bf16(kC, DZP, false, true), state || k > 0);
        }
        mma_commit(&c.bar[bOutFull]);
        mma_commit(&c.bar[bEmptyZ + st]);
    }
    mma_commit(&c.bar[bFinOut]);
    uint32_t none = 0;
    mbar_wait(&c.bar[bFinOut], 0, kTries, &none);
}

// ------------------------------------------------------------------ MMAs of the state
// B of a chunk in four quarters of 32 rows, which go through two TMEM buffers.
template <int DXP, int DZP, bool REV>
__device__ void state_mma_role(const Cta &c)
{
    using L = Layout<DXP, DZP>;
    const uint32_t dB = c.tmem + kColB, aY = c.tmem + kColY;
    const uint64_t zmajor = sdesc_sw128(smem_addr(c.base) + L::off_z, kSub, 1024);
    for (int i = 0; i < c.own_chunks + c.updates; ++i) {
        const bool second = i >= c.own_chunks;
        const int st = i & 1, live = c.live<REV>(second ? i - c.own_chunks : i);
        const uint64_t z = zmajor + (uint32_t)st * (L::stage >> 4);
        if (!c.wait(bFullZ + st, (i >> 1) & 1)) break;
        bool ok = true;
#pragma unroll
        for (int qd = 0; qd < 4; ++qd) {
            // buffer qd & 1 in its (2 i + qd / 2)-th use
            if (!(ok = c.wait(bYReady + (qd & 1), (qd >> 1) & 1))) break;
            if (qd == 0 && i > 0 && !(ok = c.wait(bBFree, (i - 1) & 1))) break;
            tc_fence_after();
            const int rows = live - 32 * qd;
#pragma unroll
            for (int term = 2; term >= 0; --term)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (rows > 16 * k)
                        mma_ts(dB, aY + (qd & 1) * 48 + term * 16 + k * 8, z + (2 * qd + k) * 128,
                               idesc_bf16(kC, DZP, false, true), qd > 0 || term < 2 || k > 0);
            mma_commit(&c.bar[bYFree + (qd & 1)]);
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

// ------------------------------------------------------------------ scores (lane = row of the chunk)
template <int DXP, int DZP, bool REV>
__device__ void score_role(const Cta &c)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t tA = c.tmem + ((uint32_t)(32 * warp) << 16) + kColA;
    for (int j = 0; j < c.chunks; ++j) {
        const int live = c.live<REV>(j);
        if (!c.wait_warp(bAFull, j & 1)) return;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {   // columns 32b .. 32b+31
            uint32_t u[32];
            if (REV ? b < warp : b > warp) {
#pragma unroll
                for (int q = 0; q < 16; ++q) u[q] = 0;
            } else {
                tmem_ld32(tA + 32 * b, u);
                // |r - s| = [distance to the near edge of the column block] + [column within it]
                float4 pq[2];
                const float wr =
                    b == warp ? 1.f : lds(c.pw + 4 * (REV ? 32 * (b - warp) - lane : 32 * (warp - b) + lane - 31));
                tmem_wait_ld();
                if (b == warp) {
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const int far = REV ? q - lane : lane - q;
                        const float w = lds(c.pw + 4 * (far >= 0 ? far : 0));
                        u[q] = far >= 0 ? __float_as_uint(__uint_as_float(u[q]) * w) : 0u;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 32; q += 8) {
                        pq[0] = lds4((REV ? c.pw : c.pr) + 4 * q);
                        pq[1] = lds4((REV ? c.pw : c.pr) + 4 * q + 16);
                        const float w[8] = {pq[0].x, pq[0].y, pq[0].z, pq[0].w, pq[1].x, pq[1].y, pq[1].z, pq[1].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[q + e] = __float_as_uint(__uint_as_float(u[q + e]) * (wr * w[e]));
                    }
                }
                if (REV && live < kC) {   // columns past the sequence are on the seen side here
#pragma unroll
                    for (int q = 0; q < 32; ++q) u[q] = 32 * b + q < live ? u[q] : 0u;
                }
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    u[q] = pack_bf16x2(__uint_as_float(u[2 * q]), __uint_as_float(u[2 * q + 1]));
            }
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q] = u[q];
            // the fp32 columns that this overwrites (of blocks <= b) have been read
            tmem_st16(tA + 16 * b, w);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&c.bar[bAReady]);
    }
}

// ------------------------------------------------------------------ output (lane = row of the chunk)
template <int DXP, int DZP, bool REV>
__device__ void out_role(const Cta &c, __nv_bfloat16 *out, int H, int Dz)
{
    using L = Layout<DXP, DZP>;
    const int warp = (threadIdx.x >> 5) - kOutWarp, lane = threadIdx.x & 31, r = 32 * warp + lane;
    const uint32_t tO = c.tmem + ((uint32_t)(32 * warp) << 16) + kColO;
    int inter = 0;
    for (int j = 0; j < c.chunks; ++j) {
        const int live = c.live<REV>(j), st = (c.own_chunks + j) & 1;
        if (c.has0 || j > 0) {
            if (!c.wait_warp(bInterFull, inter++ & 1)) return;
            tc_fence_after();
            const int e = REV ? live - 1 - r : r + 1;
            const float wr = e >= 0 ? lds(c.pw + 4 * e) : 0.f;
#pragma unroll 1
            for (int b = 0; b < DZP / 32; ++b) {
                uint32_t u[32];
                tmem_ld32(tO + 32 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 32; ++q) u[q] = __float_as_uint(wr * __uint_as_float(u[q]));
                tmem_st32(tO + 32 * b, u);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&c.bar[bInterReady]);
        }
        if (!c.wait_warp(bOutFull, j & 1)) return;
        tc_fence_after();
        if (L::own_stage && j > 0 && !c.wait_warp(bStored, (j - 1) & 1)) return;
        const uint32_t tile = smem_addr(c.base) + (L::own_stage ? L::off_out : st * L::stage);
#pragma unroll 1
        for (int b = 0; b < DZP / 32; ++b) {
            uint32_t u[32];
            tmem_ld32(tO + 32 * b, u);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = pack_bf16x2(__uint_as_float(u[8 * q + 2 * e]), __uint_as_float(u[8 * q + 2 * e + 1]));
                sts4(tile + (b >> 1) * kSub + sw128_offset(r, (b & 1) * 4 + q), v[0], v[1], v[2], v[3]);
            }
        }
        tc_fence_before();
        arrive_warp(&c.bar[bOutFree]);
        if (c.packed && live < kC) {
            // the last rows of a packed sequence: no TMA store, which would
            // run on into the next sequence; each warp writes its own rows
            const uint8_t *t = c.base + (L::own_stage ? L::off_out : st * L::stage);
            const int per = Dz / 8;
            for (int q = lane; q < 32 * per; q += 32) {
                const int rr = 32 * warp + q / per, ch = q % per;
                if (rr < live)
                    *(uint4 *)(out + ((c.g.row0 + c.row<REV>(j) + rr) * H + c.g.h) * Dz + ch * 8) =
                        *(const uint4 *)(t + (ch >> 3) * kSub + sw128_offset(rr, ch & 7));
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

    // the segment's own state, in an order of the threads' own
    __device__ __forceinline__ void store_part(float *dst) const
    {
        float4 *d = (float4 *)dst + warp * 32 + lane;
#pragma unroll
        for (int q = 0; q < kN; q += 4)
            d[(q / 4) * (kStateWarps * 32)] = make_float4(s[q], s[q + 1], s[q + 2], s[q + 3]);
    }
    __device__ __forceinline__ void add_part(const float *src, float w)
    {
        const float4 *d = (const float4 *)src + warp * 32 + lane;
#pragma unroll
        for (int b = 0; b < kN; b += 32) {
            float4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __ldcg(d + (b / 4 + q) * (kStateWarps * 32));
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                s[b + 4 * q] = fmaf(w, v[q].x, s[b + 4 * q]);
                s[b + 4 * q + 1] = fmaf(w, v[q].y, s[b + 4 * q + 1]);
                s[b + 4 * q + 2] = fmaf(w, v[q].z, s[b + 4 * q + 2]);
                s[b + 4 * q + 3] = fmaf(w, v[q].w, s[b + 4 * q + 3]);
            }
        }
    }

    // quarter qd of w Y (rows 32 qd .. +31; this warp: 16 of them, 32 state
    // rows), transposed into TMEM buffer qd & 1 as three bf16 terms
    __device__ __forceinline__ void send_keys(uint32_t sy, int qd, int live)
    {
        const int r0 = 32 * qd + 16 * side;
        float w[4];
        uint32_t keep[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int r = r0 + 8 * q + 2 * (lane & 3);
            if (r + 1 < live) {
                w[2 * q] = lds(c.pw + 4 * (REV ? r + 1 : live - 1 - r));
                w[2 * q + 1] = lds(c.pw + 4 * (REV ? r + 2 : live - 2 - r));
                keep[q] = 0xffffffffu;
            } else {   // rows past the sequence count as zeros
                w[2 * q] = lds(c.pw + (REV && r < live ? 4 * (r + 1) : 0));
                w[2 * q + 1] = 0.f;
                keep[q] = r < live ? 0xffffu : 0u;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {    // 16 state rows each
            const int d = 32 * quarter + 16 * x;
            const uint32_t chunk = ((d & 63) >> 3) + ((lane >> 3) & 1);
            uint32_t hi[4], mid[4], lo[4];
            ldmatrix_x4_trans(sy + (d >> 6) * kSub + sw128_offset(r0 + 8 * (lane >> 4) + (lane & 7), chunk), hi[0],
                              hi[1], hi[2], hi[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
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
            const uint32_t t = c.tmem + ((uint32_t)d << 16) + kColY + (qd & 1) * 48 + 8 * side;
            tmem_st_16x8(t, hi);
            tmem_st_16x8(t + 16, mid);
            tmem_st_16x8(t + 32, lo);
        }
    }

    // Quarter qd of chunk i (chunk j of its phase) into its buffer, once the
    // MMAs of the buffer's last use have completed. The first quarter also
    // waits for the chunk's rows.
    __device__ __forceinline__ bool send(int i, int j, int qd)
    {
        const int st = i & 1, live = c.live<REV>(j);
        if (qd == 0) {
            if (!c.wait_warp(bFullY + st, (i >> 1) & 1)) return false;
            if (c.packed && live < kC && !clear_tail(i, live)) return false;
        }
        // the buffer's use before this one: 2 i + qd / 2 - 1
        if ((i > 0 || qd > 1) && !c.wait_warp(bYFree + (qd & 1), (qd >> 1) ^ 1)) return false;
        tc_fence_after();
        if (live_rows) send_keys(smem_addr(c.base + st * L::stage + L::off_y), qd, live);
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(&c.bar[bYReady + (qd & 1)]);
        return true;
    }

    // Chunk i: its quarters, the next chunk's first quarter (next_j >= 0; it
    // covers the wait for this one's MMAs), then E <- gamma^R E + B.
    __device__ __forceinline__ bool chunk(int i, int j, bool first_phase, int next_j)
    {
        if (i == 0 && !send(i, j, 0)) return false;
#pragma unroll 1
        for (int qd = 1; qd < 4; ++qd)
            if (!send(i, j, qd)) return false;
        arrive_warp(&c.bar[bEmptyY + (i & 1)]);
        if (first_phase && warp == 0 && lane == 0) mbar_arrive(&c.bar[bEmptyY + (i & 1)]);   // there is no X Y^T
        if (next_j >= 0 && !send(i + 1, next_j, 0)) return false;
        if (!c.wait_warp(bBFull, i & 1)) return false;
        tc_fence_after();
        if (live_rows) {
            const uint32_t pc = c.pc + (c.live<REV>(j) == kC ? 0 : 8);
            const float wx = lds(pc), wy = lds(pc + 4);
#pragma unroll
            for (int b = 0; b < kN / 16; ++b) {
                uint32_t u[16];
                tmem_ld16(c.tmem + ((uint32_t)(32 * quarter) << 16) + kColB + dz0 + 16 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    s[16 * b + q] = fmaf(s[16 * b + q], wx, fmaf(s[16 * b + q], wy, __uint_as_float(u[q])));
            }
        }
        tc_fence_before();
        arrive_warp(&c.bar[bBFree]);
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
        if (i >= c.own_chunks) arrive_warp(&c.bar[bZReady]);   // for A Z; w Y's own signal follows
        return true;
    }

    // the bf16 copy that the readout multiplies by
    __device__ __forceinline__ void publish()
    {
        if (live_rows) {
            const uint32_t e = smem_addr(c.base) + L::off_e + (DZP == 128 ? side * L::e_sub : 0);
#pragma unroll
            for (int q = 0; q < kN / 8; ++q)
                sts4(e + sw128_offset(dx, (DZP == 128 ? 0 : 4 * side) + q), pack_bf16x2(s[8 * q], s[8 * q + 1]),
                     pack_bf16x2(s[8 * q + 2], s[8 * q + 3]), pack_bf16x2(s[8 * q + 4], s[8 * q + 5]),
                     pack_bf16x2(s[8 * q + 6], s[8 * q + 7]));
        }
        fence_proxy_async_smem();
        arrive_warp(&c.bar[bStateReady]);
    }

    __device__ __forceinline__ void run()
    {
        const size_t cells = (size_t)p.Dx * p.Dz, pad = (size_t)kN * kStateWarps * 32;
        const int last_rank = c.g.len > 0 ? (c.g.len - 1) / c.g.seg : 0;
        bool ok = true;
        clear();
        for (int i = 0; i < c.own_chunks && ok; ++i)
            ok = chunk(i, i, true, i + 1 < c.own_chunks ? i + 1 : c.updates > 0 ? 0 : -1);
        if (p.P > 1) {
            if (c.own_chunks > 0) store_part(p.part + (head * p.P + c.g.rank) * pad);
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
                add_part(p.part + (head * p.P + q) * pad,
                         la_power(ld, REV ? q * c.g.seg - c.g.end : c.g.begin - (q + 1) * c.g.seg));
        }
        if (c.has0 && c.chunks > 0) publish();
        int inter = 0;
        for (int j = 0; j < c.chunks; ++j) {
            const int i = c.own_chunks + j, live = c.live<REV>(j);
            if (j >= c.updates) {
                // nothing reads the state after this chunk
                if (c.packed && live < kC && !clear_tail(i, live)) return;
                break;
            }
            if (!chunk(i, j, false, j + 1 < c.updates ? j + 1 : -1)) return;
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
    float *pw = (float *)(c.base + L::off_aux + 512), *pr = pw + 132;
    float2 *pc = (float2 *)(pr + 32);
    uint32_t *slot = (uint32_t *)(pc + 2);
    c.pw = smem_addr(pw);
    c.pr = smem_addr(pr);
    c.pc = smem_addr(pc);
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
    if (threadIdx.x <= kC) pw[threadIdx.x] = la_power(ld, threadIdx.x);
    else if (threadIdx.x >= 160 && threadIdx.x < 192) pr[threadIdx.x - 160] = la_power(ld, 191 - threadIdx.x);
    else if (threadIdx.x == 192) pc[0] = la_power2(ld, kC);
    else if (threadIdx.x == 224) pc[1] = la_power2(ld, c.g.len % kC);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kBars; ++i) {
            const int n = i == bAReady || i == bInterReady || i == bOutFree || i == bStaged ? kOutWarps
                          : i == bYReady || i == bYReady + 1 || i == bBFree || i == bStateReady || i == bZReady
                              ? kStateWarps
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

    // registers move to the warps that hold the state (kMovedRegs)
    if (warp >= kStateWarp && warp < kLoadWarp) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp >= kStateWarp && warp < kLoadWarp) {
        StateRole<DXP, DZP, REV> role(c, p);
        role.run();
    } else {
        if (p.P > 1) cluster_arrive();
        if (warp < kOutWarp) {
            score_role<DXP, DZP, REV>(c);
        } else if (warp < kStateWarp) {
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
    // the register moves inside the kernel draw on what the launch allots
    static const bool fits = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs * kThreads >= kMovedRegs;
    }();
    if (!fits) return cudaErrorLaunchOutOfResources;
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
