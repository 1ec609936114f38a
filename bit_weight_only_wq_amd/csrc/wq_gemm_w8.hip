// Product of 8-bit activations and 8-bit weights (gfx950):
//     Y[b, n] = a_scales[b] w_scales[n] sum_k A[b, k] W[n, k] + bias[n]
// The sum is exact (int32; K < 2^17), so however it is split it comes out the
// same: results do not depend on the kernel, the batch or the split.
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

typedef int i4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint16_t w8_round(float f, bool bf16) {
    return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : float_to_half_bits_rne(f);
}

// acc a w + bias, every step rounded by itself (no fused multiply-add), so that
// all kernels give the same bits.
__device__ __forceinline__ uint16_t w8_value(int acc, float as, float ws, bool has_bias, uint16_t bias, bool bf16) {
#pragma clang fp contract(off)
    float y = (float)acc * as;
    y = y * ws;
    if (has_bias) y = y + (bf16 ? __builtin_bit_cast(float, (uint32_t)bias << 16) : half_bits_to_float(bias));
    return w8_round(y, bf16);
}

// 64 x 64 tiles, 64 k a step through LDS.
__global__ __launch_bounds__(256) void w8_tile_kernel(const W8Call C) {
    __shared__ __align__(16) int8_t as[64][80], ws[64][80];
    const int64_t n0 = (int64_t)blockIdx.x * 64, b0 = (int64_t)blockIdx.y * 64;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int r = tid >> 2, kc = (tid & 3) * 16;
    const int8_t* a = static_cast<const int8_t*>(C.A);
    const int8_t* w = static_cast<const int8_t*>(C.W);
    i4_t acc[4] = {};
    for (int64_t k = 0; k < C.K; k += 64) {
        uint4 va = make_uint4(0, 0, 0, 0), vw = va;
        if (k + kc < C.K && b0 + r < C.B) va = *reinterpret_cast<const uint4*>(a + (b0 + r) * C.a_stride + k + kc);
        if (k + kc < C.K && n0 + r < C.N) vw = *reinterpret_cast<const uint4*>(w + (n0 + r) * C.w_stride + k + kc);
        __syncthreads();
        *reinterpret_cast<uint4*>(&as[r][kc]) = va;
        *reinterpret_cast<uint4*>(&ws[r][kc]) = vw;
        __syncthreads();
        const i4_t fw = *reinterpret_cast<const i4_t*>(&ws[wave * 16 + (lane & 15)][(lane >> 4) * 16]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const i4_t fa = *reinterpret_cast<const i4_t*>(&as[j * 16 + (lane & 15)][(lane >> 4) * 16]);
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, fa, acc[j], 0, 0, 0);
        }
    }
    const uint16_t* bias = static_cast<const uint16_t*>(C.bias);
    uint16_t* Y = static_cast<uint16_t*>(C.Y);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + wave * 16 + (lane >> 4) * 4 + i, b = b0 + j * 16 + (lane & 15);
            if (n >= C.N || b >= C.B) continue;
            Y[b * C.y_stride + n] =
                w8_value(acc[j][i], C.a_scales[b], C.w_scales[n], bias != nullptr, bias ? bias[n] : (uint16_t)0, C.bf16);
        }
}

}  // namespace

hipError_t launch_gemm_w8(const W8Call& c, int num_cus, const Scratch& ws, hipStream_t stream) {
    if (ws.sizing()) return hipSuccess;
    w8_tile_kernel<<<dim3((unsigned)((c.N + 63) / 64), (unsigned)((c.B + 63) / 64)), dim3(256), 0, stream>>>(c);
    return hipGetLastError();
}

}  // namespace wq
