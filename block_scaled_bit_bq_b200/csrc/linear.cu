// linear.cu -- the products of a linear layer over block-scaled data (bq_linear and its two
// gradients): out[j, i] = sum_c X(j, c) Q(i, c), X bf16, Q block-scaled codes, the roles of
// the stored matrices as LinearArgs says.
//
// Every code times its block scale is a bf16 value (widen.cuh), so the codes are widened on the
// way to the tensor cores and the products with X are exact; sums are fp32.
//
// Two kernels:
//  - k_linear_mma, on the fifth-generation tensor cores: out's transpose in tiles of 128
//    (i, from Q) x up to 256 (j, from X);
//  - k_linear_rows, for the forward product of a few tokens, where the weight's bytes are all
//    that counts: the codes go straight from global memory to mma.sync fragments.
#include "internal.h"
#include "tc.cuh"
#include "widen.cuh"

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

namespace bq {

__device__ unsigned int g_linear_wait_timeouts = 0;

namespace {

// ---------------------------------------------------------------------------
// Shared pieces
// ---------------------------------------------------------------------------

// Byte offset of block scale (row, blk) in either scale layout. Scales of an even block and
// the one after it are adjacent in both.
__device__ __forceinline__ size_t scale_offset(const LinearArgs& a, uint32_t row, uint32_t blk)
{
    return a.gemm_layout ? (size_t)gemm_scale_offset(row, blk, a.nb) : (size_t)row * a.nb + blk;
}

// Scale loads as volatile asm: they stay where they are issued, ahead of the codes' use (as
// plain loads the compiler moves them down to it, and each one's latency shows).
__device__ __forceinline__ uint32_t ldg_u8(const uint8_t* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ldg_u16(const uint8_t* p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t ldg_u32(const uint8_t* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// The scale bytes of two 32-code groups of a row (one MX byte or two NV bytes each), at p: of an
// even group and of the one after it, the second where it exists. In one load where a row's
// scales start on a multiple of its size (wide). The loaded words are taken apart only where
// they are used (pair_scale): doing so here would wait for them.
template <bool NV>
__device__ __forceinline__ void load_scale_pair(const uint8_t* p, bool wide, bool second, uint32_t (&s)[2])
{
    if (wide) {
        s[0] = NV ? ldg_u32(p) : ldg_u16(p);
    } else {
        s[0] = NV ? ldg_u16(p) : ldg_u8(p);
        if (second) s[1] = NV ? ldg_u16(p + 2) : ldg_u8(p + 1);
    }
}

template <bool NV>
__device__ __forceinline__ uint32_t pair_scale(const uint32_t (&s)[2], bool wide, int which)
{
    if (which == 0) return NV ? s[0] & 0xFFFFu : s[0] & 0xFFu;
    return wide ? (NV ? s[0] >> 16 : s[0] >> 8) : s[1];
}

template <bool NV>
__device__ __forceinline__ float out_scale(const LinearArgs& a) { return NV ? __fmul_rn(__ldg(a.tensor_scale), NV_OUT) : 1.0f; }

__device__ __forceinline__ void store_out(const LinearArgs& a, size_t o, float v)
{
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(a.out)[o] = v;
}

// n (at most 32) rows of out from row j on, 32 columns (i0 + lane) by a warp, lane l holding
// column i0 + l: v[e] is row j + e. Times sc, rounded to out's type. As bf16 with rows of whole
// groups of four columns, lanes swap 4 x 4 blocks first and store 8 bytes of four rows at a
// time (a quarter of the stores).
__device__ __forceinline__ void store_rows(const LinearArgs& a, uint32_t j, uint32_t i0, uint32_t lane, uint32_t n,
                                           const uint32_t (&v)[32], float sc)
{
    const uint32_t i = i0 + lane;
    if (!a.out_bf16) {
        float* p = reinterpret_cast<float*>(a.out) + (size_t)j * a.ni + i;
#pragma unroll
        for (uint32_t e = 0; e < 32; ++e, p += a.ni)
            if (e < n && i < a.ni) *p = __fmul_rn(__uint_as_float(v[e]), sc);
    } else if (a.ni % 4u != 0) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)j * a.ni + i;
#pragma unroll
        for (uint32_t e = 0; e < 32; ++e, p += a.ni)
            if (e < n && i < a.ni) *p = __float2bfloat16_rn(__fmul_rn(__uint_as_float(v[e]), sc));
    } else {
        const uint32_t i4 = i & ~3u, dr = ((lane & 2u) ? 2u : 0u) + (lane & 1u);     // this lane's row of four
        const uint32_t sel = (lane & 1u) ? 0x3276u : 0x5410u;
        const bool up = (lane & 2u) != 0u;
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(a.out) + (size_t)(j + dr) * a.ni + i4;
#pragma unroll
        for (uint32_t e = 0; e < 32; e += 4, p += (size_t)4 * a.ni) {
            uint32_t r[2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) {       // rows e + 2 h and + 1: a pair of columns per lane, of one row
                const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(__uint_as_float(v[e + 2 * h]), sc),
                                                               __fmul_rn(__uint_as_float(v[e + 2 * h + 1]), sc));
                const uint32_t own = *reinterpret_cast<const uint32_t*>(&b);
                r[h] = __byte_perm(own, __shfl_xor_sync(0xFFFFFFFFu, own, 1), sel);
            }
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? r[0] : r[1], 2);
            const uint32_t w[2] = {up ? got : r[0], up ? r[1] : got};
            if (e + dr < n && i4 < a.ni) st_v2(p, w);
        }
    }
}

// ---------------------------------------------------------------------------
// Few tokens: y[t, n] for t < 8 MT.
//
// A CTA of 8 warps takes 16 R weight rows; the warps share out the columns in pieces of 128
// (64 bytes of codes), piece after piece in turn, so that together they read runs of 512
// bytes of a row. A lane (g = lane / 4, q = lane % 4) loads the 32 codes q of rows g and g +
// 8 of each 16 (16 bytes each) and the 32 values q of token g, and takes the columns in the
// order in which widening leaves them: an mma.sync adds up 16 columns in any order as long as
// both operands use the same one. The warps' sums meet in shared memory, in warp order.
//
// The weight's bytes set the floor; widening them (half the ALU's rate) with few warps to hide
// the loads behind is what bounds it above that: 8 tokens x 28672 x 8192 under NV in 46-50 us,
// 2.7-2.9 TB/s of 133 MB (the same loads alone: 29 us).
// ---------------------------------------------------------------------------

constexpr int ROWS_WARPS = 8;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_x(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

template <bool NV, int R, int MT>
__global__ void __launch_bounds__(32 * ROWS_WARPS, R * MT == 1 ? 3 : 2) k_linear_rows(const LinearArgs a)
{
    using W = Widen<BQ_FP4_E2M1, NV>;
    constexpr uint32_t TS = 16 * R + 4;              // floats from token to token: conflict-free
    __shared__ float part[ROWS_WARPS][8 * MT * TS];
    pdl_wait();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, g = lane >> 2, q = lane & 3u;
    const uint32_t row0 = blockIdx.x * (16u * R);
    const uint32_t groups = a.k / 32u;
    float acc[R][MT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[r][t][e] = 0.0f;

    // Rows past the last and columns past the end read the last ones instead: those rows are not
    // stored, and those columns meet zeros of x.
    constexpr uint32_t GB = NV ? 2u : 1u;                        // scale bytes of 32 codes
    const uint8_t *code[2 * R], *scale[2 * R];
#pragma unroll
    for (int h = 0; h < 2 * R; ++h) {
        const uint32_t row = min(row0 + 8u * h + g, a.ni - 1u);
        code[h] = a.codes + (size_t)row * (a.k / 2);
        scale[h] = a.scales + scale_offset(a, row, 0u);
    }
    const uint16_t* xr[MT];
    bool tok[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const uint32_t j = 8u * t + g;
        tok[t] = j < a.nj;
        xr[t] = reinterpret_cast<const uint16_t*>(a.x) + (tok[t] ? j : 0u) * a.ldx;
    }

    // a piece's loads; other warps (three CTAs an SM, two with 32 rows or 16 tokens) work meanwhile
    uint32_t w[2 * R][4], s[2 * R];
    uint4 x[MT][4];
    auto fetch = [&](uint32_t next) {
        const bool in = next < groups;
        const uint32_t grp = min(next, groups - 1u);
        // block grp * GB of a row: in the tiled layout four to a tile of 512 bytes
        const uint32_t so = a.gemm_layout ? ((grp * GB) >> 2) * 512u + ((grp * GB) & 3u) : grp * GB;
#pragma unroll
        for (int h = 0; h < 2 * R; ++h) {
            ld_nc_v4(code[h] + (size_t)grp * 16u, w[h]);
            s[h] = NV ? ldg_u16(scale[h] + so) : ldg_u8(scale[h] + so);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[t][i] = in && tok[t] ? ldg_x(xr[t] + grp * 32u + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
    };
    const uint32_t g0 = 4u * warp + q;
    if (4u * warp < groups) fetch(g0);
    for (uint32_t grp = g0; grp - q < groups; grp += 4u * ROWS_WARPS) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t p0[16], p1[16];
            const bool one = NV || __all_sync(0xFFFFFFFFu, W::fits(s[2 * r]) && W::fits(s[2 * r + 1]));
            W::pairs(w[2 * r], s[2 * r], one, p0);
            W::pairs(w[2 * r + 1], s[2 * r + 1], one, p1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const uint4 v = x[t][i];                     // (e0 e1) (e2 e3) (e4 e5) (e6 e7)
                    mma_16816(acc[r][t], p0[4 * i], p1[4 * i], p0[4 * i + 1], p1[4 * i + 1],
                              __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632));
                    mma_16816(acc[r][t], p0[4 * i + 2], p1[4 * i + 2], p0[4 * i + 3], p1[4 * i + 3],
                              __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                }
            }
        }
        if (grp - q + 4u * ROWS_WARPS < groups) fetch(grp + 4u * ROWS_WARPS);
    }

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)              // d[e]: row g + 8 (e / 2), token 2 q + e % 2
                part[warp][(8 * t + 2 * q + (e & 1)) * TS + 16 * r + g + 8 * (e >> 1)] = acc[r][t][e];
    __syncthreads();
    const float sc = out_scale<NV>(a);
    for (uint32_t o = threadIdx.x; o < 8u * MT * 16u * R; o += 32u * ROWS_WARPS) {
        const uint32_t t = o / (16u * R), i = o % (16u * R);
        if (t >= a.nj || row0 + i >= a.ni) continue;
        float v = part[0][t * TS + i];
#pragma unroll
        for (int k = 1; k < ROWS_WARPS; ++k) v = __fadd_rn(v, part[k][t * TS + i]);
        store_out(a, (size_t)t * a.ni + row0 + i, __fmul_rn(v, sc));
    }
}

// ---------------------------------------------------------------------------
// Tensor cores. out^T in tiles of 128 (i) x bt (j), the contraction in parts of 64 steps, one
// or two to a stage of the ring:
//   A: Q widened to bf16, 128 i x 64 c (16 KB), by the widening warps: four groups of four
//      warps take the parts (64 steps) in turn, a thread 64 codes of one stored row. The codes
//      come through a ring of their own, 16 KB chunks of four parts (two of 8-bit codes) by
//      tensor-map copies, and what lies outside the matrix as zeros; the scales by plain loads,
//      two of the thread's parts ahead;
//   B: X by a tensor-map copy, bt j x 64 c.
// Both with the 128-byte swizzle. Where the stored rows run along the contraction (LIN_FORWARD
// for both operands, LIN_GRAD_INPUT for X) an operand is K-major: rows of 128 bytes, groups of
// 8 rows 1024 bytes apart. Where the rows are the contraction (Q of both gradients, X of
// LIN_GRAD_WEIGHT) it is MN-major: chunks of 64 i (or j) x 64 c, a row of 128 bytes per c, and
// the tensor cores transpose it. Either way a thread's 64 values are one row of 128 bytes.
//
// Warp 0 issues the copies of X, warp 26 those of the codes, warp 1 the MMAs (4 of 16 steps a
// part, fp32 accumulator in tensor memory, two of them so that a tile's epilogue overlaps the
// next tile), warps 2-17 widen, warps 18-25 write the accumulator out. A CTA per SM, persistent
// over the tiles. Large products run on pairs of CTAs (PAIR): a tile is 256 i x 256 j, each CTA
// of a pair widens its own 128 i and copies its own 128 j, and the first one issues MMAs that
// read both (half the shared memory and copies of X per MMA of a lone CTA). With fewer tiles
// than SMs, a cluster of 2, 4 or 8 CTAs shares a tile's contraction and adds up its parts
// through distributed shared memory, in rank order: no workspace, and the same sums every time.
// Waits give up after a second as in the block-scaled GEMM (counted in g_linear_wait_timeouts), the
// epilogue's for an accumulator after a second in which no stage was done. A pair's stage is whole
// on the first CTA's barrier: both CTAs' copies complete there, and the second CTA's codes are handed
// over there. tests/linear_ring_model.py is a model of all this.
//
// 4096 tokens x 11008 x 4096: 270 us forward (NV), 289-340 input gradient (MX), 303-330 weight
// gradient (E4M3), as the power cap's clock has it (1.1-1.37 PFLOP/s; tensor pipe active 61-74 %,
// the widening warps' ALU 45-49 %); dequantizing to bf16 and a library product take 248-284. With few
// tokens the hand-over of a part (about 0.35 us whatever the tile's width) bounds it.
// ---------------------------------------------------------------------------

constexpr uint32_t WIDEN_GROUPS = 4, GROUP_WARPS = 4, GROUP_THREADS = 32 * GROUP_WARPS;
constexpr uint32_t WIDEN_WARPS = WIDEN_GROUPS * GROUP_WARPS;
constexpr uint32_t EPI_WARP = 2 + WIDEN_WARPS, EPI_WARPS = 8, CODES_WARP = EPI_WARP + EPI_WARPS;
constexpr int MMA_THREADS = 32 * (CODES_WARP + 1);
constexpr int MAX_STAGES = 8, MAX_CHUNKS = 8;
constexpr uint32_t CHUNK_BYTES = 16384;
constexpr uint32_t A_BYTES = 128u * 128u;
constexpr uint32_t SMEM_MAX = 232448u;
constexpr uint32_t ACC_COLS = 256;
constexpr uint32_t SMEM_ROOM = SMEM_MAX - 2048u;       // less alignment slack and static shared memory
static_assert(SMEM_ROOM - 2u * CHUNK_BYTES >= WIDEN_GROUPS * (A_BYTES + 256u * 128u), "a stage ring of as many parts as groups");

struct MmaPlan {
    uint32_t bt;            // tile width in j: a multiple of 16 (of 64 for LIN_GRAD_WEIGHT), at most 256
    uint32_t subs;          // 64-step parts of a stage: 1 or 2
    uint32_t stages;        // of the ring
    uint32_t chunks;        // of the code ring
    uint32_t tiles_i, tiles;    // tiles of i, and in all (i by i)
    uint32_t blocks;        // of the contraction: 256 steps, four parts, each
    uint32_t split;         // CTAs per tile (a cluster): 1, 2, 4 or 8
    uint32_t pair;          // 1: tiles of 256 x 256 on pairs of CTAs (bt 128 each)
    uint32_t skip_cta;      // fault injection for tests: this CTA issues no copies of X for its first stage
};

// Instruction descriptor of the bf16 MMA: fp32 accumulator (bits 4-5), bf16 operands (7-9,
// 10-12), MN-major flags of A and B (15, 16), N / 8 (17-22), M / 16 (24-28).
template <int OP>
__device__ __forceinline__ uint32_t mma_desc(uint32_t m, uint32_t n)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((OP == LIN_FORWARD ? 0u : 1u) << 15) |
           ((OP == LIN_GRAD_WEIGHT ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// MN-major operand: chunks of 64 x 64 (8 KB) side by side, 8 steps 1024 bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) { return smem_desc(addr, 8192u, 1024u, 2u); }

template <bool PAIR>
__device__ __forceinline__ void tc_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (PAIR)
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void load_x(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    if constexpr (PAIR) tma_load_2d_pair(dst, map, bar, x, y);
    else tma_load_2d(dst, map, bar, x, y);
}

// Commit of the MMAs so far: an arrival on bar, in a pair on that barrier of both CTAs.
template <bool PAIR>
__device__ __forceinline__ void tc_commit_all(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(bar), "h"((uint16_t)3) : "memory");
    else
        tc_commit(bar);
}

// Arrivals on the first CTA's barrier (bar: its address in this CTA), for its thread that waits
// there to let MMAs go that read, or write over, what this CTA holds. Of shared memory written
// before (its waits: ACQ_SHARED); a release of everything, global memory too, takes about 900
// cycles, and 4096 tokens x 11008 x 4096 forward 316 us with it.
__device__ __forceinline__ void mbar_arrive_first_shared(uint32_t bar)
{
    fence_release_shared();
    asm volatile("{\n.reg .b32 p;\nmapa.shared::cluster.u32 p, %0, 0;\n"
                 "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [p];\n}" :: "r"(bar) : "memory");
}

// Of everything before, accumulator reads among it (its waits: ACQ_CLUSTER): once a tile.
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar)
{
    asm volatile("{\n.reg .b32 p;\nmapa.shared::cluster.u32 p, %0, 0;\n"
                 "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [p];\n}" :: "r"(bar) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xFFFFFFFF;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0u;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four floats of another CTA's shared memory (addr: the same variable's address in this CTA).
__device__ __forceinline__ float4 ld_cluster(uint32_t addr, uint32_t rank)
{
    float4 v;
    asm volatile("{\n.reg .b32 p;\nmapa.shared::cluster.u32 p, %4, %5;\nld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [p];\n}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank));
    return v;
}

// The sum over S ranks, in order, of four floats at the same place in each; all loads are under
// way before the first is used (one after the other, they took most of a small product's time).
template <int S>
__device__ __forceinline__ float4 sum_cluster(uint32_t addr)
{
    float4 p[S];
#pragma unroll
    for (int r = 0; r < S; ++r) p[r] = ld_cluster(addr, (uint32_t)r);
    float4 v = p[0];
#pragma unroll
    for (int r = 1; r < S; ++r) {
        v.x = __fadd_rn(v.x, p[r].x);
        v.y = __fadd_rn(v.y, p[r].y);
        v.z = __fadd_rn(v.z, p[r].z);
        v.w = __fadd_rn(v.w, p[r].w);
    }
    return v;
}

template <int OP, int FMT, bool NV, bool PAIR>
__global__ void __launch_bounds__(MMA_THREADS, 1) k_linear_mma(const __grid_constant__ CUtensorMap xmap,
                                                             const __grid_constant__ CUtensorMap qmap,
                                                             const LinearArgs a, const MmaPlan pl)
{
    using W = Widen<FMT, NV>;
    constexpr uint32_t CP = Fmt<FMT>::four ? 4u : 2u;     // parts of a chunk of codes
    constexpr std::integral_constant<int, ACQ_CTA> acq_cta{};
    constexpr std::integral_constant<int, PAIR ? ACQ_SHARED : ACQ_CTA> acq_stage{};     // a stage is full
    constexpr std::integral_constant<int, PAIR ? ACQ_CLUSTER : ACQ_CTA> acq_acc{};      // an accumulator is full, empty
    extern __shared__ uint8_t linear_smem[];
    __shared__ __align__(8) uint64_t full[MAX_STAGES], empty[MAX_STAGES], code_full[MAX_CHUNKS],
        code_empty[MAX_CHUNKS], acc_full[2], acc_empty[2], done_bar;
    __shared__ uint32_t tmem_holder;
    __shared__ volatile int abort_flag;
    __shared__ volatile uint32_t stages_done;        // of the MMA warp (of a pair's second CTA: handed over)
    // (from lane 0, so that the compiler sees the warps' roles as uniform branches)
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31u;
    const uint32_t base = (smem_addr(linear_smem) + 1023u) & ~1023u;
    // bt: the j that this CTA copies; a pair's tile has twice as many
    const uint32_t bt = pl.bt, subs = pl.subs, NS = pl.stages;
    const uint32_t tile_j = PAIR ? 2u * bt : bt;
    const uint32_t b_bytes = bt * 128u, sub_bytes = A_BYTES + b_bytes, stage_bytes = subs * sub_bytes;
    const uint32_t code_base = base + NS * stage_bytes;
    const uint32_t rank = PAIR || pl.split > 1 ? cluster_rank() : 0u;
    // this CTA's (pair's) tiles and its part of the contraction
    const uint32_t share = PAIR ? 2u : pl.split;
    const uint32_t first = share > 1 ? blockIdx.x / share : blockIdx.x;
    const uint32_t step = PAIR ? gridDim.x / 2u : (pl.split > 1 ? pl.tiles : gridDim.x);
    const uint32_t krank = PAIR ? 0u : rank;
    const uint32_t p0 = 4u * (uint32_t)((uint64_t)pl.blocks * krank / pl.split);          // first part
    const uint32_t kts = 4u * (uint32_t)((uint64_t)pl.blocks * (krank + 1) / pl.split) - p0;   // parts
    const uint32_t tile_stages = kts / subs, tile_chunks = kts / CP;
    // parts past the contraction's end fill up its last block: they take part in every hand-over,
    // but nothing is copied, widened or multiplied for them
    auto live = [&](uint32_t part) { return (uint64_t)part * 64u < a.nc; };
    // A warp's wait, and whether some warp has given up: the same answer for all lanes, since what
    // follows (barriers of whole warps, tcgen05) wants them together
    auto get = [](auto acq, uint64_t& bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait_ring<decltype(acq)::value>(smem_addr(&bar), parity)) != 0;
    };
    auto stopped = [&]() { return __any_sync(0xFFFFFFFFu, abort_flag) != 0; };
    // first i of a tile for this CTA, and first j of the tile
    auto tile_i0 = [&](uint32_t t) { return t % pl.tiles_i * (PAIR ? 256u : 128u) + (PAIR ? rank * 128u : 0u); };
    auto tile_j0 = [&](uint32_t t) { return t / pl.tiles_i * tile_j; };

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < NS; ++s) {
            // the widening warps and the warp that issues the copies; in a pair the first CTA's
            // barrier is the stage's: both CTAs' copies complete on it, and the second CTA arrives
            // there once its own is complete
            mbar_init(smem_addr(&full[s]), subs * GROUP_WARPS + 1u + (PAIR && rank == 0 ? 1u : 0u));
            mbar_init(smem_addr(&empty[s]), 1);
        }
        for (uint32_t c = 0; c < pl.chunks; ++c) {
            mbar_init(smem_addr(&code_full[c]), 1);
            mbar_init(smem_addr(&code_empty[c]), CP * GROUP_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&acc_full[b]), 1);
            mbar_init(smem_addr(&acc_empty[b]), PAIR ? 2u * EPI_WARPS : EPI_WARPS);
        }
        mbar_init(smem_addr(&done_bar), 1);
        abort_flag = 0;
        stages_done = 0;
        fence_mbar_init();
    }
    __syncwarp();
    if (PAIR) cluster_sync();                        // the other CTA is there, its barriers are set
    if (warp == 1) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_addr(&tmem_holder)), "r"(2u * ACC_COLS) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         :: "r"(smem_addr(&tmem_holder)), "r"(2u * ACC_COLS) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (PAIR) cluster_sync();                        // the first CTA's MMAs use both accumulators
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_holder;
    pdl_wait();

    if (warp == 0) {
        // ---- X tiles ----
        const bool leader = elect_one();
        uint32_t s = 0, round = 0;                   // slot of the ring, and how often it wrapped
        bool go = true;
        for (uint32_t t = first; t < pl.tiles && go; t += step) {
            const int j0 = (int)(tile_j0(t) + (PAIR ? rank * bt : 0u));
            for (uint32_t kk = 0; kk < tile_stages; ++kk) {
                go = (round == 0 || get(acq_cta, empty[s], (round - 1) & 1u)) && !stopped();
                if (!go) break;
                if (leader) {
                    const uint32_t fb = smem_addr(&full[s]);
                    uint32_t dst = base + s * stage_bytes + A_BYTES, part = p0 + kk * subs;
                    const uint32_t n_live = live(part) ? (subs == 2 && live(part + 1) ? 2u : 1u) : 0u;
                    // a pair's MMAs read both CTAs' X on either SM: both CTAs' bytes are awaited on the
                    // first one's barrier (this slot's earlier use is over there too: its MMAs freed the
                    // slot here). The second CTA's warp arrives on its own all the same, so that it
                    // cannot fall behind by a use of a slot, which a wait by parity would not tell
                    if (PAIR && rank != 0) mbar_arrive(fb);
                    else mbar_arrive_expect_tx(fb, (PAIR ? 2u : 1u) * n_live * b_bytes);
                    const bool skip = blockIdx.x == pl.skip_cta && t == first && kk == 0;     // tests only
                    for (uint32_t u = 0; u < n_live && !skip; ++u, ++part, dst += sub_bytes) {
                        const int c = (int)(part * 64u);
                        if (OP == LIN_GRAD_WEIGHT) {
                            for (uint32_t x = 0; x < bt / 64u; ++x)
                                load_x<PAIR>(dst + x * 8192u, &xmap, fb, j0 + (int)(64u * x), c);
                        } else {
                            load_x<PAIR>(dst, &xmap, fb, c, j0);
                        }
                    }
                }
                __syncwarp();
                if (++s == NS) { s = 0; ++round; }
            }
        }
        if (!go) abort_flag = 1;
    } else if (warp == 1) {
        // ---- MMAs: 16 steps are 32 bytes along a K-major row, 16 rows (2 KB) of an MN-major
        // chunk. The whole warp runs the loop, so that descriptors stay in uniform registers ----
        constexpr uint32_t ka = OP == LIN_FORWARD ? 2u : 128u, kb = OP == LIN_GRAD_WEIGHT ? 128u : 2u;
        const bool leader = elect_one();
        const uint32_t idesc = mma_desc<OP>(PAIR ? 256u : 128u, tile_j);
        const uint64_t ad0 = OP == LIN_FORWARD ? operand_desc(base) : mn_desc(base);
        const uint64_t bd0 = OP == LIN_GRAD_WEIGHT ? mn_desc(base + A_BYTES) : operand_desc(base + A_BYTES);
        uint32_t s = 0, par = 0, i = 0, stage = 0;
        bool go = true;
        if (PAIR && rank != 0) {
            // the second CTA of a pair only says when its codes of a stage are widened
            for (uint32_t t = first; t < pl.tiles && go; t += step) {
                for (uint32_t kk = 0; kk < tile_stages; ++kk) {
                    go = get(acq_cta, full[s], par) && !stopped();
                    if (!go) break;
                    if (leader) {
                        mbar_arrive_first_shared(smem_addr(&full[s]));
                        stages_done = ++stage;
                    }
                    __syncwarp();
                    if (++s == NS) { s = 0; par ^= 1u; }
                }
            }
        } else {
            for (uint32_t t = first; t < pl.tiles && go; t += step, ++i) {
                const uint32_t b = i & 1u;
                go = (i < 2 || get(acq_acc, acc_empty[b], (i / 2 - 1) & 1u)) && !stopped();
                if (!go) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + b * ACC_COLS;
                uint32_t acc = 0;
                for (uint32_t kk = 0; kk < tile_stages; ++kk) {
                    go = get(acq_stage, full[s], par);
                    if (!go) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    for (uint32_t u = 0; u < subs; ++u) {
                        const uint64_t so = (s * stage_bytes + u * sub_bytes) >> 4, ad = ad0 + so, bd = bd0 + so;
                        if (leader && live(p0 + kk * subs + u)) {
#pragma unroll
                            for (uint32_t k = 0; k < 4; ++k)
                                tc_mma_bf16<PAIR>(d, ad + ka * k, bd + kb * k, idesc, k ? 1u : acc);
                        }
                        acc = 1;
                    }
                    if (leader) {
                        tc_commit_all<PAIR>(smem_addr(&empty[s]));
                        stages_done = ++stage;
                    }
                    __syncwarp();
                    if (++s == NS) { s = 0; par ^= 1u; }
                }
                if (!go) break;
                if (leader) tc_commit_all<PAIR>(smem_addr(&acc_full[b]));
                __syncwarp();
            }
            // every MMA issued so far completes before done_bar's phase does
            if (leader) tc_commit_all<PAIR>(smem_addr(&done_bar));
            __syncwarp();
        }
        if (!mbar_wait(smem_addr(&done_bar), 0u) || !go) abort_flag = 1;
    } else if (warp < 2 + WIDEN_WARPS) {
        // ---- Q tiles: a thread takes 64 codes of one stored row: forward, row r of the tile and
        // the part's columns; gradients, row r of the part and half h of the tile's columns.
        // Group g takes parts g, g + 4, ... (a tile has a multiple of four): it comes by every fourth
        // part of the stage ring and every chunk of codes (of 8-bit codes, every second), so its
        // waits by parity never look back further than one use of a slot: the stage ring holds four
        // parts or more, the code ring two chunks or more (of 8-bit codes, an even number) ----
        const uint32_t g = (warp - 2u) / GROUP_WARPS, tid = (threadIdx.x - 64u) % GROUP_THREADS;
        const uint32_t r = OP == LIN_FORWARD ? tid : tid & 63u, h = OP == LIN_FORWARD ? 0u : tid >> 6;
        // where its codes lie in a chunk: row cr of 128 (or 64) bytes, 16-byte units from cu on (a
        // multiple of their number, so that unit e is at the first one's address xor 16 e)
        const uint32_t cr = OP == LIN_FORWARD ? r : (g % CP) * 64u + r;
        const uint32_t cu = OP == LIN_FORWARD ? 2u * g : (Fmt<FMT>::four ? 2u * h : 4u * h);
        const uint32_t src_off = cr * (OP == LIN_GRAD_INPUT ? 64u : 128u) +
                                 ((cu ^ (OP == LIN_GRAD_INPUT ? (cr >> 1) & 3u : cr & 7u)) << 4);
        // where its values go: a row of 128 bytes, unit e at e ^ (r % 8)
        const uint32_t dst_off = (g % subs) * sub_bytes + h * 8192u + r * 128u + ((r & 7u) << 4);
        const uint32_t groups = a.k / 32u;
        const bool wide = a.gemm_layout || (NV ? a.nb % 4u == 0 : a.nb % 2u == 0);
        // the scales, two of this group's parts ahead: of row ld_row, 32-code groups ld_grp and + 1.
        // From part to part the pointer goes by a fixed step: 8 groups along a row, or 256 rows
        constexpr uint32_t GB = NV ? 2u : 1u;                 // bytes of a group
        const size_t ld_step = OP == LIN_FORWARD ? (a.gemm_layout ? 2u * GB * 512u : 8u * GB)
                                                 : (a.gemm_layout ? (size_t)2u * (a.nb / 4u) * 512u : (size_t)256u * a.nb);
        uint32_t ld_tile = first, ld_pk = g, ld_row = 0, ld_grp = 0;
        const uint8_t* ld_p = nullptr;
        auto start_tile = [&]() {
            if (ld_tile >= pl.tiles) return;
            const uint32_t i0 = tile_i0(ld_tile), kk = p0 + g;
            ld_row = OP == LIN_FORWARD ? i0 + r : kk * 64u + r;
            ld_grp = OP == LIN_FORWARD ? kk * 2u : i0 / 32u + 2u * h;
            ld_p = a.scales + scale_offset(a, ld_row, GB * ld_grp);
        };
        start_tile();
        uint32_t sc[2][2];
        auto fetch = [&](uint32_t (&cs)[2]) {
            cs[0] = cs[1] = 0u;
            if (ld_tile < pl.tiles && ld_row < a.q_rows && ld_grp < groups) load_scale_pair<NV>(ld_p, wide, ld_grp + 1u < groups, cs);
            ld_p += ld_step;
            if (OP == LIN_FORWARD) ld_grp += 8u;
            else ld_row += 256u;
            ld_pk += WIDEN_GROUPS;
            if (ld_pk >= kts) {
                ld_pk = g;
                ld_tile += step;
                start_tile();
            }
        };
        fetch(sc[0]);
        fetch(sc[1]);
        uint32_t s = g / subs, round = 0, c = g / CP, c_par = 0;      // slots of the two rings
        bool ok = true;
        for (uint32_t t = first; t < pl.tiles && ok; t += step) {
            for (uint32_t pk = g; pk < kts && ok; pk += WIDEN_GROUPS) {
                ok = mbar_wait_ring(smem_addr(&code_full[c]), c_par);
                const uint32_t src = code_base + c * CHUNK_BYTES + src_off;
                uint32_t o[2][16], w[2][W::WORDS];
#pragma unroll
                for (uint32_t x = 0; x < 2; ++x)
#pragma unroll
                    for (uint32_t e = 0; e < W::WORDS / 4; ++e)
                        lds_v4(src ^ ((x * (W::WORDS / 4) + e) << 4), w[x][4 * e], w[x][4 * e + 1], w[x][4 * e + 2],
                               w[x][4 * e + 3]);
                const uint32_t s0 = pair_scale<NV>(sc[0], wide, 0), s1 = pair_scale<NV>(sc[0], wide, 1);
                sc[0][0] = sc[1][0];
                sc[0][1] = sc[1][1];
                const bool one = __all_sync(0xFFFFFFFFu, W::fits(s0) && W::fits(s1) && W::numbers(w[0]) && W::numbers(w[1]));
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t v[W::WORDS * W::RAW];
                    W::pairs(w[x], x ? s1 : s0, one, v);
                    W::in_order(v, o[x]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&code_empty[c]));
                fetch(sc[1]);
                if (ok && round > 0) ok = mbar_wait_ring(smem_addr(&empty[s]), (round - 1) & 1u);
                ok = __all_sync(0xFFFFFFFFu, ok && !abort_flag) != 0;
                if (!ok) { abort_flag = 1; break; }
                if (live(p0 + pk)) {
                    const uint32_t dst = base + s * stage_bytes + dst_off;
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e)
                        sts_v4(dst ^ (e << 4), o[e >> 2][4 * (e & 3)], o[e >> 2][4 * (e & 3) + 1], o[e >> 2][4 * (e & 3) + 2],
                               o[e >> 2][4 * (e & 3) + 3]);
                    fence_proxy_async();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&full[s]));
                s += WIDEN_GROUPS / subs;
                while (s >= NS) { s -= NS; ++round; }
                c += WIDEN_GROUPS / CP;
                while (c >= pl.chunks) { c -= pl.chunks; c_par ^= 1u; }
            }
        }
    } else if (warp == CODES_WARP) {
        // ---- codes: forward, boxes of 128 rows x 256 columns along the tile's rows; gradients,
        // boxes of 256 (128) rows of the contraction x the tile's 128 columns ----
        const bool leader = elect_one();
        uint32_t c = 0, round = 0;
        bool go = true;
        for (uint32_t t = first; t < pl.tiles && go; t += step) {
            const uint32_t i0 = tile_i0(t);
            for (uint32_t n = 0; n < tile_chunks; ++n) {
                go = (round == 0 || get(acq_cta, code_empty[c], (round - 1) & 1u)) && !stopped();
                if (!go) break;
                if (leader) {
                    const uint32_t part = p0 + n * CP, fb = smem_addr(&code_full[c]);
                    mbar_arrive_expect_tx(fb, CHUNK_BYTES);
                    if (OP == LIN_FORWARD) tma_load_2d(code_base + c * CHUNK_BYTES, &qmap, fb, (int)(part * 32u), (int)i0);
                    else tma_load_2d(code_base + c * CHUNK_BYTES, &qmap, fb, (int)(Fmt<FMT>::four ? i0 / 2u : i0), (int)(part * 64u));
                }
                __syncwarp();
                if (++c == pl.chunks) { c = 0; ++round; }
            }
        }
        if (!go) abort_flag = 1;
    } else {
        // ---- epilogue: warp w reads lanes 32 (w % 4) .. + 31 of the accumulator, i.e. 32 i, and
        // every second 32 columns ----
        const uint32_t q = warp & 3u, il = q * 32u + lane, half = (warp - EPI_WARP) >> 2;
        const float sc = out_scale<NV>(a);
        uint32_t n = 0;
        for (uint32_t t = first; t < pl.tiles; t += step, ++n) {
            const uint32_t b = n & 1u;
            // a tile's whole contraction may lie before this: the wait goes on as long as stages do
            bool ok = false;
            for (uint32_t seen = stages_done, now;; seen = now) {
                ok = mbar_wait_ring<acq_acc.value>(smem_addr(&acc_full[b]), (n / 2) & 1u);
                now = stages_done;
                if (ok || abort_flag || now == seen) break;
            }
            ok = __all_sync(0xFFFFFFFFu, ok && !abort_flag) != 0;
            if (!ok) { abort_flag = 1; break; }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t i0 = tile_i0(t) + q * 32u, j0 = tile_j0(t);
            const uint32_t cols = min(tile_j, a.nj - j0);
            for (uint32_t c0 = half * 32u; c0 < cols; c0 += 64u) {
                uint32_t v[32];
                tmem_ld32(tmem + b * ACC_COLS + ((q * 32u) << 16) + c0, v);
                if (pl.split > 1) {
                    // this CTA's part of the sums, [j][i], over the stages (all consumed)
#pragma unroll
                    for (uint32_t e = 0; e < 32; ++e)
                        if (c0 + e < bt)
                            asm volatile("st.shared.b32 [%0], %1;" :: "r"(base + ((c0 + e) * 128u + il) * 4u), "r"(v[e]) : "memory");
                } else {
                    store_rows(a, j0 + c0, i0, lane, min(32u, cols - c0), v, sc);
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_first(smem_addr(&acc_empty[b]));
                else mbar_arrive(smem_addr(&acc_empty[b]));
            }
        }
    }
    __syncwarp();
    __syncthreads();                                 // no warp issues anything any more
    // Every copy that was waited for has landed. A CTA that gave up may have issued others: it
    // keeps its shared memory for another second
    if (abort_flag) linger();
    if (PAIR) cluster_sync();                        // neither CTA leaves while the other's MMAs or arrivals may use it
    if (!PAIR && pl.split > 1) {
        cluster_sync();
        // every CTA of the cluster adds up the parts of its share of the columns
        const uint32_t i = tile_i0(first), j0 = tile_j0(first);
        const uint32_t from = bt * rank / pl.split, to = min(bt * (rank + 1) / pl.split, a.nj - j0);
        const float sc = out_scale<NV>(a);
        for (uint32_t o = from * 128u + threadIdx.x * 4u; o < to * 128u; o += MMA_THREADS * 4u) {
            const uint32_t ii = i + (o & 127u), at = base + o * 4u;
            if (ii >= a.ni) continue;
            const float4 v = pl.split == 2 ? sum_cluster<2>(at) : pl.split == 4 ? sum_cluster<4>(at) : sum_cluster<8>(at);
            const float e[4] = {v.x, v.y, v.z, v.w};
            const size_t oo = (size_t)(j0 + (o >> 7)) * a.ni + ii;
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
                if (ii + c < a.ni) store_out(a, oo + c, NV ? __fmul_rn(e[c], sc) : e[c]);
        }
        cluster_sync();                              // no CTA leaves while its parts are being read
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0 && abort_flag) atomicAdd(&g_linear_wait_timeouts, 1u);
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(2u * ACC_COLS) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(2u * ACC_COLS) : "memory");
    }
}

// The codes as stored: boxes of CHUNK_BYTES (see the codes warp).
cudaError_t codes_map(int op, bool four, const LinearArgs& a, CUtensorMap* map)
{
    *map = CUtensorMap{};
    const EncodeTiled enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const uint32_t row_bytes = four ? a.k / 2u : a.k, width = op == LIN_GRAD_INPUT ? 64u : 128u;
    const cuuint64_t dims[2] = {row_bytes, a.q_rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {width, CHUNK_BYTES / width};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.codes), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           op == LIN_GRAD_INPUT ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// x as stored, boxes of 64 columns (128 bytes) x box_rows rows, 128-byte swizzle; what lies
// outside the matrix arrives as zeros.
cudaError_t x_map(const LinearArgs& a, uint32_t box_rows, CUtensorMap* map)
{
    *map = CUtensorMap{};
    const EncodeTiled enc = encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {a.x_cols, a.x_rows};
    const cuuint64_t strides[1] = {a.ldx * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.x), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Test hook (bq_debug_skip_linear_copy), consumed by the next launch.
constexpr uint32_t NO_CTA = 0xFFFFFFFFu;
std::atomic<uint32_t> g_skip_cta{NO_CTA};

uint32_t ceil_div(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

uint32_t plan_stage_bytes(const MmaPlan& p) { return p.subs * (A_BYTES + p.bt * 128u); }

// The tile width that takes the fewest rounds of tiles over the SMs, weighed by a round's
// length (a stage costs bt, and no less than the 128 that widening its codes takes); then a
// split of the contraction while tiles leave SMs idle and every CTA keeps a block of it.
MmaPlan make_mma_plan(int op, const LinearArgs& a, uint32_t sms)
{
    MmaPlan p;
    const uint32_t unit = op == LIN_GRAD_WEIGHT ? 64u : 16u;
    p.tiles_i = ceil_div(a.ni, 128u);
    const uint32_t most = std::min(256u, ceil_div(a.nj, unit) * unit);
    uint64_t best = ~0ull;
    p.bt = most;
    for (uint32_t bt = most; bt >= unit && (bt >= 128u || bt == most); bt -= unit) {
        const uint64_t tiles = (uint64_t)p.tiles_i * ceil_div(a.nj, bt);
        const uint64_t cost = ((tiles + sms - 1) / sms) * std::max(bt, 128u);
        if (cost < best) { best = cost; p.bt = bt; }
    }
    // pairs of CTAs (a part of a tile costs them no more than a lone CTA's, see above) where they
    // take no more rounds: a little more from one tile for each pair of SMs on, no more from two
    // thirds of that
    const uint64_t pair_tiles = (uint64_t)ceil_div(a.ni, 256u) * ceil_div(a.nj, 256u);
    const uint64_t pair_cost = ((pair_tiles + sms / 2 - 1) / (sms / 2)) * 256u;
    p.pair = pair_tiles * 3 >= sms && pair_cost * 4 <= best * (pair_tiles >= sms / 2 ? 5u : 4u) ? 1u : 0u;
    if (p.pair) {
        p.bt = 128;
        p.tiles_i = ceil_div(a.ni, 256u);
    }
    p.tiles = p.tiles_i * ceil_div(a.nj, p.pair ? 256u : p.bt);
    p.subs = p.bt > 128u ? 1u : 2u;
    p.blocks = ceil_div(a.nc, 256u);
    p.split = 1;
    while (!p.pair && p.split < 8 && p.tiles * p.split * 2 <= sms && p.blocks >= p.split * 2) p.split *= 2;
    // two chunks of codes at least, up to four stages, then more chunks: with narrow tiles the
    // codes are most of what is read, and their ring keeps the memory busy
    const uint32_t room = SMEM_ROOM, stage = plan_stage_bytes(p);
    p.stages = std::min(4u, (room - 2u * CHUNK_BYTES) / stage);          // four parts or more
    p.skip_cta = g_skip_cta.exchange(NO_CTA, std::memory_order_acq_rel);
    p.chunks = std::min<uint32_t>(MAX_CHUNKS, (room - p.stages * stage) / CHUNK_BYTES) & ~1u;
    return p;
}

// Lets kern use up to bytes of dynamic shared memory on the current device (once per device).
template <typename K>
cudaError_t allow_smem(K kern, uint32_t bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0u;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <int OP, int FMT, bool NV, bool PAIR>
cudaError_t run_plan(const LinearArgs& a, const MmaPlan& pl, uint32_t sms, cudaStream_t st)
{
    constexpr auto kern = k_linear_mma<OP, FMT, NV, PAIR>;
    static std::atomic<uint64_t> attr_set{0};        // a bit per device
    cudaError_t e = allow_smem(kern, SMEM_MAX - 1024u, attr_set);
    if (e != cudaSuccess) return e;
    CUtensorMap xm, qm;
    e = x_map(a, OP == LIN_GRAD_WEIGHT ? 64u : pl.bt, &xm);
    if (e != cudaSuccess) return e;
    e = codes_map(OP, Fmt<FMT>::four, a, &qm);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(PAIR ? 2u * std::min(pl.tiles, sms / 2u) : pl.split > 1 ? pl.tiles * pl.split : std::min(pl.tiles, sms));
    cfg.blockDim = dim3(MMA_THREADS);
    cfg.dynamicSmemBytes = pl.stages * plan_stage_bytes(pl) + pl.chunks * CHUNK_BYTES + 1024u;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = PAIR ? 2u : pl.split;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR || pl.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, xm, qm, a, pl);
}

template <int OP, int FMT, bool NV>
cudaError_t run_mma(const LinearArgs& a, cudaStream_t st)
{
    const uint32_t sms = (uint32_t)device_sm_count();
    const MmaPlan pl = make_mma_plan(OP, a, sms);
    return pl.pair ? run_plan<OP, FMT, NV, true>(a, pl, sms, st) : run_plan<OP, FMT, NV, false>(a, pl, sms, st);
}

template <bool NV, int R, int MT>
cudaError_t run_rows(const LinearArgs& a, cudaStream_t st)
{
    return launch_pdl(k_linear_rows<NV, R, MT>, ceil_div(a.ni, 16u * R), 32 * ROWS_WARPS, 0, st, a);
}

template <bool NV>
cudaError_t run_forward(const LinearArgs& a, cudaStream_t st)
{
    if (a.nj > 16) return run_mma<LIN_FORWARD, BQ_FP4_E2M1, NV>(a, st);
    // 32 rows share each read of x, 16 have more loads under way: 32 for more than 4 tokens
    // where that leaves two CTAs per SM (11008 x 4096, us: 1 token 10.0 with 16 rows, 11.5 with
    // 32; 8 tokens 13.8 and 12.0)
    const bool two = a.nj > 4 && ceil_div(a.ni, 32u) >= 2u * (uint32_t)device_sm_count();
    if (a.nj <= 8) return two ? run_rows<NV, 2, 1>(a, st) : run_rows<NV, 1, 1>(a, st);
    return run_rows<NV, 1, 2>(a, st);
}

}  // namespace

cudaError_t launch_linear(int op, int fmt, bool nv, const LinearArgs& a, cudaStream_t st)
{
    if (op == LIN_FORWARD) return nv ? run_forward<true>(a, st) : run_forward<false>(a, st);
    if (op == LIN_GRAD_INPUT)
        return nv ? run_mma<LIN_GRAD_INPUT, BQ_FP4_E2M1, true>(a, st) : run_mma<LIN_GRAD_INPUT, BQ_FP4_E2M1, false>(a, st);
    if (fmt == BQ_FP8_E4M3) return run_mma<LIN_GRAD_WEIGHT, BQ_FP8_E4M3, false>(a, st);
    if (fmt == BQ_FP8_E5M2) return run_mma<LIN_GRAD_WEIGHT, BQ_FP8_E5M2, false>(a, st);
    if (fmt == BQ_INT8_SYM) return run_mma<LIN_GRAD_WEIGHT, BQ_INT8_SYM, false>(a, st);
    return cudaErrorInvalidValue;
}

void linear_skip_copy(uint32_t cta) { g_skip_cta.store(cta, std::memory_order_release); }

cudaError_t linear_wait_timeouts(unsigned int* count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_linear_wait_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0u;
        e = cudaMemcpyToSymbol(g_linear_wait_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace bq
