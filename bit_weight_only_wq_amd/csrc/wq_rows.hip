// Rows of activations (or weights) to 8 bits with one scale a row, and the
// root-mean-square norm with the residual's addition in front of it (gfx950).
//
// With t a row's values before any scaling (the norm: t = h w, h = x + residual
// rounded to the input's type, w the norm's weight; else t = x, or x silu(gate)):
//     code = round-half-even(127 t / max|t|),   value = code * scale
// The norm's factor r = 1 / sqrt(mean h^2 + eps) cancels in 127 t / max|t|, so
// codes do not depend on how the squares were summed; it enters the scale only.
// h and w have at most 11 significant bits each, so t is exact in fp32.  A code
// is 127 / max times t in fp32, off by less than 2^-15 (two roundings of a
// number up to 127), and wherever that lies near a border between two codes the
// quotient is formed in fp64.  Without a gate one that is not on the border lies
// 2^-24 from it at least.  Gated values are off by some 2^-52 in fp64; they have
// exact ties too (a value whose gate is that of the row's largest), so what lies
// within 2^-40 of a border counts as on it.
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ float to_float(uint16_t b, bool bf16) {
    return bf16 ? __builtin_bit_cast(float, (uint32_t)b << 16) : half_bits_to_float(b);
}
__device__ __forceinline__ uint16_t from_float(float f, bool bf16) {
    return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : float_to_half_bits_rne(f);
}

// Largest of a block's bit patterns and sum of its doubles, in every thread.
__device__ __forceinline__ void block_join(uint32_t& top, double& sum) {
    __shared__ uint32_t tops[kThreads / kWave];
    __shared__ double sums[kThreads / kWave];
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t t = __shfl_xor(top, o, kWave);
        top = t > top ? t : top;
        sum += __shfl_xor(sum, o, kWave);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        tops[threadIdx.x >> 6] = top;
        sums[threadIdx.x >> 6] = sum;
    }
    __syncthreads();
    top = 0;
    sum = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        top = tops[w] > top ? tops[w] : top;
        sum += sums[w];
    }
}

// round-half-even(127 t / top), ties as above.
__device__ __forceinline__ int exact_code(double t, double top) {
    const double q = 127.0 * t / top;
    const double half = 0.5 * __builtin_rint(2.0 * q);
    return (int)__builtin_rint(__builtin_fabs(q - half) < 0x1p-40 ? half : q);
}

__device__ __forceinline__ double silu64(double g) { return g / (1.0 + exp(-g)); }

// One workgroup a row, one value at a time; any size, stride and alignment.
__global__ __launch_bounds__(kThreads) void norm_any_kernel(const NormCall A) {
    const int64_t row = blockIdx.x;
    const uint16_t* x = static_cast<const uint16_t*>(A.x) + row * A.x_stride;
    const uint16_t* res = A.residual ? static_cast<const uint16_t*>(A.residual) + row * A.residual_stride : nullptr;
    uint16_t* total = A.total ? static_cast<uint16_t*>(A.total) + row * A.total_stride : nullptr;
    const uint16_t* w = static_cast<const uint16_t*>(A.weight);
    const uint16_t* h = total ? total : x;
    uint32_t top = 0;
    double sum = 0.0;
    for (int64_t k = threadIdx.x; k < A.K; k += kThreads) {
        uint16_t b = x[k];
        if (res) b = from_float(to_float(b, A.bf16) + to_float(res[k], A.bf16), A.bf16);
        if (total) total[k] = b;
        const float v = to_float(b, A.bf16);
        const uint32_t u = __builtin_bit_cast(uint32_t, v * to_float(w[k], A.bf16)) & 0x7FFFFFFFu;
        top = u > top ? u : top;
        sum += (double)v * (double)v;
    }
    block_join(top, sum);
    const double r = 1.0 / sqrt(sum / (double)A.K + (double)A.eps);
    const double t64 = (double)__builtin_bit_cast(float, top);
    const bool fine = top < kInfBits && sum < __builtin_inf();
    for (int64_t k = threadIdx.x; k < A.K; k += kThreads) {
        const float t = to_float(h[k], A.bf16) * to_float(w[k], A.bf16);
        if (A.out)
            static_cast<uint16_t*>(A.out)[row * A.out_stride + k] = from_float(t * (float)r, A.bf16);
        else
            static_cast<int8_t*>(A.codes)[row * A.codes_stride + k] =
                fine && top ? (int8_t)exact_code((double)t, t64) : (int8_t)0;
    }
    if (A.codes && threadIdx.x == 0)
        A.scales[row] = !fine ? __builtin_nanf("") : top ? (float)(r * t64 / 127.0) : 1.0f;
}

__global__ __launch_bounds__(kThreads) void rows_any_kernel(const RowsCall A) {
    const int64_t row = blockIdx.x;
    const uint16_t* x = static_cast<const uint16_t*>(A.x) + row * A.x_stride;
    const uint16_t* g = A.gate ? static_cast<const uint16_t*>(A.gate) + row * A.gate_stride : nullptr;
    int8_t* codes = static_cast<int8_t*>(A.codes) + row * A.codes_stride;
    const auto value = [&](int64_t k) {
        double v = (double)to_float(x[k], A.bf16);
        if (g) v *= silu64((double)to_float(g[k], A.bf16));
        return v;
    };
    double most = 0.0;
    bool bad = false;
    for (int64_t k = threadIdx.x; k < A.K; k += kThreads) {
        const double v = __builtin_fabs(value(k));
        bad |= !(v <= 3.4028234663852886e38);
        most = v > most ? v : most;
    }
    __shared__ double mosts[kThreads];
    __shared__ int bads;
    if (threadIdx.x == 0) bads = 0;
    mosts[threadIdx.x] = most;
    __syncthreads();
    if (bad) bads = 1;
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o && mosts[threadIdx.x + o] > mosts[threadIdx.x]) mosts[threadIdx.x] = mosts[threadIdx.x + o];
        __syncthreads();
    }
    most = mosts[0];
    const float scale = (float)(most / 127.0);
    for (int64_t k = threadIdx.x; k < A.K; k += kThreads)
        codes[k] = bads || scale == 0.0f ? (int8_t)0 : (int8_t)exact_code(value(k), most);
    if (threadIdx.x == 0) A.scales[row] = bads ? __builtin_nanf("") : scale == 0.0f ? 1.0f : scale;
}

}  // namespace

hipError_t launch_norm(const NormCall& c, hipStream_t stream) {
    norm_any_kernel<<<dim3((unsigned)c.rows), dim3(kThreads), 0, stream>>>(c);
    return hipGetLastError();
}

hipError_t launch_rows(const RowsCall& c, hipStream_t stream) {
    rows_any_kernel<<<dim3((unsigned)c.rows), dim3(kThreads), 0, stream>>>(c);
    return hipGetLastError();
}

}  // namespace wq
