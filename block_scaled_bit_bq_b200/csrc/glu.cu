// glu.cu -- the gated activation h = a(g) u with the 8-bit copies of g and u that its
// backward pass reads, and that backward pass: du = dh a(G), dg = dh U a'(G).
//
// a(g) = g s(v), s(v) = 1 / (1 + exp(-v)). With v = g (SiLU) or v = 2 sqrt(2 / pi) (g +
// 0.044715 g^3) (GELU's tanh form: (1 + tanh z) / 2 = s(2 z)), both have
// a'(g) = s (1 + g (1 - s) v').
//
// Both passes stream: every input byte is read once, every output byte written once, and
// HBM bounds them (forward 4 + 2 + 2 (1 + 1/32) bytes per element, backward 2 (1 + 1/32) +
// 2 + 4). A thread takes 16 consecutive elements (32-byte loads and stores); two adjacent
// lanes hold one 32-element block and join its largest magnitude by a shuffle.
#include "dequant_ops.cuh"
#include "internal.h"

namespace bq {

namespace {

constexpr int GLU_THREADS = 256;

__device__ __forceinline__ float ex2_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x cut to [-12, 12]; NaN stays NaN (fminf and fmaxf would give a bound).
__device__ __forceinline__ float cut12(float x)
{
    float r;
    asm("{\nmax.NaN.f32 %0, %1, 0fC1400000;\nmin.NaN.f32 %0, %0, 0f41400000;\n}" : "=f"(r) : "f"(x));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f;
constexpr float GELU_2C = 1.5957691216057308f;                      // 2 sqrt(2 / pi)
constexpr float GELU_K = 0.044715f;

// s(v) of a(g) = g s(v), and (when SLOPE) g v' (1 - s) to form a'. The approximations are good
// to about 2^-22 plus |v| 2^-24 from exp's argument; results are rounded to bf16 (2^-9). An s below
// 2^-126 comes out as 0 (v < -87.3; the approximations flush). GELU's argument is cut at |g| = 12, where s is 0 or 1 in fp32 already: beyond it g^3 would overflow.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float logistic(float g, float& slope)
{
    if constexpr (ACT == BQ_ACT_SILU) {
        const float s = rcp_approx(__fadd_rn(1.0f, ex2_approx(__fmul_rn(g, -LOG2E))));
        if constexpr (SLOPE) slope = __fmaf_rn(__fmul_rn(g, s), __fadd_rn(1.0f, -s), s);
        return s;
    } else {
        const float c = cut12(g), c2 = __fmul_rn(c, c);
        const float v = __fmul_rn(c, __fmaf_rn(GELU_2C * GELU_K, c2, GELU_2C));
        const float s = rcp_approx(__fadd_rn(1.0f, ex2_approx(__fmul_rn(v, -LOG2E))));
        if constexpr (SLOPE) {
            const float cv = __fmul_rn(c, __fmaf_rn(3.0f * GELU_2C * GELU_K, c2, GELU_2C));
            slope = __fmaf_rn(__fmul_rn(cv, s), __fadd_rn(1.0f, -s), s);
        }
        return s;
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// Codes of a chunk under its block's scale, and the scale's exponent: e from the largest
// magnitude of the two lanes' chunks, codes of x 2^-e (exact, or below the smallest code's
// half when it underflows).
template <int FMT>
__device__ __forceinline__ int quant_chunk(const uint32_t (&w)[8], uint32_t (&code)[4])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = bf2_absmax(m, w[i]);
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const uint32_t am = max(m & 0xFFFFu, m >> 16);
    const int e = ue8m0_exponent<FMT>(__uint_as_float(am << 16));
    const float inv = exp2i(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = mul2(make_float2(bf_lo(w[2 * i]), bf_hi(w[2 * i])), splat(inv));
        const float2 b = mul2(make_float2(bf_lo(w[2 * i + 1]), bf_hi(w[2 * i + 1])), splat(inv));
        if constexpr (FMT == BQ_INT8_SYM) {
            // |x 2^-e| <= 127: MAGIC's sum holds the rounded integer in its low byte
            const float2 p = add2(a, splat(MAGIC)), q = add2(b, splat(MAGIC));
            const uint32_t lo = __byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x0040u);
            const uint32_t hi = __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040u);
            code[i] = __byte_perm(lo, hi, 0x5410u);
        } else {
            code[i] = cvt_pair<FMT>(a.y, a.x) | (cvt_pair<FMT>(b.y, b.x) << 16);
        }
    }
    return e;
}

// FMT < 0: h alone.
template <int FMT, int ACT>
__global__ void __launch_bounds__(GLU_THREADS) k_glu(const GluArgs a)
{
    pdl_wait();
    // n_chunks is even (a row holds whole blocks): the two lanes of a block run alike. Lanes
    // past the end work on the last chunk and store nothing
    const uint64_t c64 = (uint64_t)blockIdx.x * GLU_THREADS + threadIdx.x;
    const bool live = c64 < a.n_chunks;
    const uint32_t c = live ? (uint32_t)c64 : a.n_chunks - 1u;
    const uint32_t row = fast_div(c, a.cpr), col = (c - row * a.cpr.d) * 16u;
    uint32_t g[8], u[8];
    ld_nc_v8(reinterpret_cast<const __nv_bfloat16*>(a.x0) + row * a.ldx0 + col, g);
    ld_nc_v8(reinterpret_cast<const __nv_bfloat16*>(a.x1) + row * a.ldx1 + col, u);
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g0 = bf_lo(g[i]), g1 = bf_hi(g[i]);
        float unused;
        const float s0 = logistic<ACT, false>(g0, unused), s1 = logistic<ACT, false>(g1, unused);
        const float2 r = mul2(mul2(make_float2(g0, g1), make_float2(s0, s1)), make_float2(bf_lo(u[i]), bf_hi(u[i])));
        h[i] = bf16_pair(r.x, r.y);
    }
    if (live) st_v8(reinterpret_cast<__nv_bfloat16*>(a.y0) + (size_t)c * 16u, h);
    if constexpr (FMT >= 0) {
        uint32_t gc[4], uc[4];
        const int ge = quant_chunk<FMT>(g, gc), ue = quant_chunk<FMT>(u, uc);
        if (live) {
            st_v4(a.codes0 + (size_t)c * 16u, gc);
            st_v4(a.codes1 + (size_t)c * 16u, uc);
            if ((c & 1u) == 0) {
                a.scales0[c >> 1] = (uint8_t)(ge + 127);
                a.scales1[c >> 1] = (uint8_t)(ue + 127);
            }
        }
    }
}

template <int FMT>
__device__ __forceinline__ void chunk_floats(const uint32_t (&w)[4], uint32_t scale, float2 (&v)[8])
{
    float2 raw[8];
    chunk_values<FMT, 1>(w, 0, raw);
    const UnitScale us{exp2i((int)scale - 127), 0.0f};
    dequant_chunk<FMT, SK_UE8M0>(us, raw, v);
}

// dg of a chunk once more, for products dh u that overflow: the slope may bring them back (it may be
// as small as 2^-126, or 0) and goes first there: u a' is a normal number then (|u| >= 1, |a'| <
// 1.14), and dg finite where the true value is. Four elements at a time, which keeps its registers
// below the pass's own.
template <int FMT, int ACT>
__device__ __forceinline__ void dgate_again(const GluArgs& a, uint32_t c, uint32_t row, uint32_t col)
{
    constexpr float largest = 3.402823466e38f;
    const uint32_t gs = __ldg(a.scales0 + (c >> 1)), us = __ldg(a.scales1 + (c >> 1));
#pragma unroll 1
    for (uint32_t q = 0; q < 4; ++q) {
        const uint2 dw = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.x0) + row * a.ldx0 + col) + q);
        const uint32_t gw[4] = {__ldg(reinterpret_cast<const uint32_t*>(a.codes0) + (size_t)c * 4u + q), 0u, 0u, 0u};
        const uint32_t uw[4] = {__ldg(reinterpret_cast<const uint32_t*>(a.codes1) + (size_t)c * 4u + q), 0u, 0u, 0u};
        float2 g[8], u[8];
        chunk_floats<FMT>(gw, gs, g);
        chunk_floats<FMT>(uw, us, u);
        uint32_t r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = i ? dw.y : dw.x;
            const float2 d = make_float2(bf_lo(w), bf_hi(w)), p = mul2(d, u[i]);
            float t0, t1;
            (void)logistic<ACT, true>(g[i].x, t0);
            (void)logistic<ACT, true>(g[i].y, t1);
            r[i] = bf16_pair(fabsf(p.x) <= largest ? __fmul_rn(p.x, t0) : __fmul_rn(d.x, __fmul_rn(u[i].x, t0)),
                             fabsf(p.y) <= largest ? __fmul_rn(p.y, t1) : __fmul_rn(d.y, __fmul_rn(u[i].y, t1)));
        }
        st_v2(reinterpret_cast<__nv_bfloat16*>(a.y0) + row * a.ldy0 + col + 4u * q, r);
    }
}

// The look for such a product (the largest |dh u| of a chunk) shows under GELU, whose arithmetic is
// next to HBM's time (8192 x 4096 E5M2: 42.5 -> 43.3 us); chosen for each element it took 43.7, and
// SiLU's passes 1.3 % more. INT8 takes 54-56 registers by itself, four CTAs an SM: five are 4 %
// faster at 4096 x 11008 under GELU (57.8 -> 56.2 us).
template <int FMT, int ACT>
__global__ void __launch_bounds__(GLU_THREADS, FMT == BQ_INT8_SYM ? 5 : 0) k_glu_backward(const GluArgs a)
{
    pdl_wait();
    const uint64_t c64 = (uint64_t)blockIdx.x * GLU_THREADS + threadIdx.x;
    if (c64 < a.n_chunks) {
        const uint32_t c = (uint32_t)c64;
        const uint32_t row = fast_div(c, a.cpr), col = (c - row * a.cpr.d) * 16u;
        uint32_t dh[8], gc[4], uc[4];
        ld_nc_v8(reinterpret_cast<const __nv_bfloat16*>(a.x0) + row * a.ldx0 + col, dh);
        ld_nc_v4(a.codes0 + (size_t)c * 16u, gc);
        ld_nc_v4(a.codes1 + (size_t)c * 16u, uc);
        const uint32_t gs = __ldg(a.scales0 + (c >> 1)), us = __ldg(a.scales1 + (c >> 1));
        float2 g[8], u[8];
        chunk_floats<FMT>(gc, gs, g);
        chunk_floats<FMT>(uc, us, u);
        uint32_t dg[8], du[8];
        float most = 0.0f;                           // of |dh u|
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t0, t1;
            const float s0 = logistic<ACT, true>(g[i].x, t0), s1 = logistic<ACT, true>(g[i].y, t1);
            const float2 d = make_float2(bf_lo(dh[i]), bf_hi(dh[i]));
            const float2 ru = mul2(d, mul2(g[i], make_float2(s0, s1)));
            const float2 p = mul2(d, u[i]), rg = mul2(p, make_float2(t0, t1));
            du[i] = bf16_pair(ru.x, ru.y);
            dg[i] = bf16_pair(rg.x, rg.y);
            most = fmaxf(most, fmaxf(fabsf(p.x), fabsf(p.y)));
        }
        // (dh is read again before anything is written)
        if (most > 3.402823466e38f) dgate_again<FMT, ACT>(a, c, row, col);
        else st_v8(reinterpret_cast<__nv_bfloat16*>(a.y0) + row * a.ldy0 + col, dg);
        st_v8(reinterpret_cast<__nv_bfloat16*>(a.y1) + row * a.ldy1 + col, du);
    }
}

// A thread per chunk: CTAs that come and go keep more loads under way than CTAs that loop over
// their share (8 per SM: 66 + 63 us for 4096 x 11008 forward and backward; one chunk a thread:
// 61 + 56 us, 96 % of the copy peak, with inputs from HBM; forward and backward of one step 110 us, as
// L2 serves some of the copies).
unsigned glu_grid(uint32_t n_chunks) { return (unsigned)(((uint64_t)n_chunks + GLU_THREADS - 1) / GLU_THREADS); }

template <int FMT>
cudaError_t run_glu(int act, const GluArgs& a, cudaStream_t st)
{
    return act == BQ_ACT_SILU ? launch_pdl(k_glu<FMT, BQ_ACT_SILU>, glu_grid(a.n_chunks), GLU_THREADS, 0, st, a)
                              : launch_pdl(k_glu<FMT, BQ_ACT_GELU_TANH>, glu_grid(a.n_chunks), GLU_THREADS, 0, st, a);
}

template <int FMT>
cudaError_t run_glu_backward(int act, const GluArgs& a, cudaStream_t st)
{
    return act == BQ_ACT_SILU
               ? launch_pdl(k_glu_backward<FMT, BQ_ACT_SILU>, glu_grid(a.n_chunks), GLU_THREADS, 0, st, a)
               : launch_pdl(k_glu_backward<FMT, BQ_ACT_GELU_TANH>, glu_grid(a.n_chunks), GLU_THREADS, 0, st, a);
}

}  // namespace

cudaError_t launch_glu(int fmt, int act, const GluArgs& a, cudaStream_t st)
{
    switch (fmt) {
    case -1: return run_glu<-1>(act, a, st);
    case BQ_FP8_E4M3: return run_glu<BQ_FP8_E4M3>(act, a, st);
    case BQ_FP8_E5M2: return run_glu<BQ_FP8_E5M2>(act, a, st);
    case BQ_INT8_SYM: return run_glu<BQ_INT8_SYM>(act, a, st);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_glu_backward(int fmt, int act, const GluArgs& a, cudaStream_t st)
{
    switch (fmt) {
    case BQ_FP8_E4M3: return run_glu_backward<BQ_FP8_E4M3>(act, a, st);
    case BQ_FP8_E5M2: return run_glu_backward<BQ_FP8_E5M2>(act, a, st);
    case BQ_INT8_SYM: return run_glu_backward<BQ_INT8_SYM>(act, a, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bq
