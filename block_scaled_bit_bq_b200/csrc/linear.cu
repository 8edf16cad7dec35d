// linear.cu -- the products of a linear layer over block-scaled data (bq_linear and its two
// gradients): out[j, i] = sum_c X(j, c) Q(i, c), X bf16, Q block-scaled codes, each role of
// the stored matrices as LinearArgs says.
#include "internal.h"

namespace bq {

namespace {

// One code's value times its block's scale (without NV's tensor scale).
template <int FMT, bool NV>
__device__ __forceinline__ float code_value(const LinearArgs& a, uint32_t row, uint32_t col)
{
    float v;
    if constexpr (FMT == BQ_FP4_E2M1) {
        const uint32_t b = a.codes[(size_t)row * (a.k / 2) + col / 2];
        v = dec_pair<FMT>((b >> (4 * (col & 1))) & 0xFu).x;
    } else {
        const uint32_t b = a.codes[(size_t)row * a.k + col];
        v = FMT == BQ_INT8_SYM ? (float)(int8_t)b : dec_pair<FMT == BQ_INT8_SYM ? BQ_FP8_E4M3 : FMT>(b).x;
    }
    const uint32_t blk = col / (NV ? 16u : 32u);
    const size_t so = a.gemm_layout ? gemm_scale_offset(row, blk, a.nb) : (size_t)row * a.nb + blk;
    const uint32_t sc = a.scales[so];
    return __fmul_rn(v, NV ? e4m3_value(sc) : exp2i((int)sc - 127));
}

constexpr int T = 32;

// A CTA per 32 x 32 tile of the output, 32 steps of the contraction at a time through shared
// memory; thread (x, y) sums out[j0 + y + 8 r, i0 + x], r = 0..3.
template <int OP, int FMT, bool NV>
__global__ void __launch_bounds__(256) k_linear_tile(const LinearArgs a)
{
    __shared__ float xs[T][T + 1], qs[T][T + 1];     // [j][c], [i][c]
    const uint32_t tx = threadIdx.x & 31u, ty = threadIdx.x >> 5;
    const uint32_t tiles_i = (a.ni + T - 1) / T;
    const uint32_t i0 = (blockIdx.x % tiles_i) * T, j0 = (blockIdx.x / tiles_i) * T;
    const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (uint32_t c0 = 0; c0 < a.nc; c0 += T) {
        for (uint32_t r = ty; r < T; r += 8) {
            if (OP == LIN_GRAD_WEIGHT) {             // rows are the contraction
                const uint32_t c = c0 + r, j = j0 + tx, i = i0 + tx;
                xs[tx][r] = c < a.nc && j < a.nj ? __bfloat162float(x[c * a.ldx + j]) : 0.f;
                qs[tx][r] = c < a.nc && i < a.ni ? code_value<FMT, NV>(a, c, i) : 0.f;
            } else {
                const uint32_t c = c0 + tx, j = j0 + r;
                xs[r][tx] = c < a.nc && j < a.nj ? __bfloat162float(x[j * a.ldx + c]) : 0.f;
                if (OP == LIN_FORWARD) {
                    const uint32_t i = i0 + r;
                    qs[r][tx] = c < a.nc && i < a.ni ? code_value<FMT, NV>(a, i, c) : 0.f;
                } else {
                    const uint32_t cc = c0 + r, i = i0 + tx;
                    qs[tx][r] = cc < a.nc && i < a.ni ? code_value<FMT, NV>(a, cc, i) : 0.f;
                }
            }
        }
        __syncthreads();
        for (int c = 0; c < T; ++c)
            for (int r = 0; r < 4; ++r) acc[r] = __fmaf_rn(xs[ty + 8 * r][c], qs[tx][c], acc[r]);
        __syncthreads();
    }
    const float sc = a.tensor_scale ? *a.tensor_scale : 1.0f;
    const uint32_t i = i0 + tx;
    for (int r = 0; r < 4; ++r) {
        const uint32_t j = j0 + ty + 8 * r;
        if (i >= a.ni || j >= a.nj) continue;
        const float v = __fmul_rn(acc[r], sc);
        const size_t o = (size_t)j * a.ni + i;
        if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
        else reinterpret_cast<float*>(a.out)[o] = v;
    }
}

template <int OP, int FMT, bool NV>
cudaError_t run_tile(const LinearArgs& a, cudaStream_t st)
{
    const uint64_t tiles = (uint64_t)((a.ni + T - 1) / T) * ((a.nj + T - 1) / T);
    k_linear_tile<OP, FMT, NV><<<(unsigned)tiles, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear(int op, int fmt, bool nv, const LinearArgs& a, cudaStream_t st)
{
    if (op == LIN_FORWARD)
        return nv ? run_tile<LIN_FORWARD, BQ_FP4_E2M1, true>(a, st) : run_tile<LIN_FORWARD, BQ_FP4_E2M1, false>(a, st);
    if (op == LIN_GRAD_INPUT)
        return nv ? run_tile<LIN_GRAD_INPUT, BQ_FP4_E2M1, true>(a, st)
                  : run_tile<LIN_GRAD_INPUT, BQ_FP4_E2M1, false>(a, st);
    if (fmt == BQ_FP8_E4M3) return run_tile<LIN_GRAD_WEIGHT, BQ_FP8_E4M3, false>(a, st);
    if (fmt == BQ_FP8_E5M2) return run_tile<LIN_GRAD_WEIGHT, BQ_FP8_E5M2, false>(a, st);
    if (fmt == BQ_INT8_SYM) return run_tile<LIN_GRAD_WEIGHT, BQ_INT8_SYM, false>(a, st);
    return cudaErrorInvalidValue;
}

cudaError_t linear_wait_timeouts(unsigned int* count, bool)
{
    *count = 0;
    return cudaSuccess;
}

}  // namespace bq
