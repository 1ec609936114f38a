// Decode attention over a paged int4 KV cache (gfx950): one new token per
// sequence, out = softmax(scale K q) V over the sequence's pages and window.
//
// Plain form: a workgroup of 128 threads per (entry, query head) walks the
// blocks with a running maximum and sum.  Thread t scores token t of a block
// and then owns channel t of the output.
#include "wq_paged.h"

namespace wq {

using namespace paged;

namespace {

struct AttnArgs {
    PagedArgs c;
    const uint16_t* q;
    uint16_t* out;
    const int32_t* lens;
    const int32_t* seqs;
    int64_t q_stride, out_stride, window;
    int q_heads, group;
    float scale;       // times log2(e)
};

__device__ __forceinline__ float block_max2(float v, float* red) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return __builtin_fmaxf(red[0], red[1]);
}

__global__ __launch_bounds__(128) void paged_attn_kernel(const AttnArgs A) {
    __shared__ float qf[kD], p[kG], red[2];
    const int64_t entry = blockIdx.x;
    const int g = blockIdx.y, head = g / A.group, tid = threadIdx.x;
    const int64_t slot = slot_of(A.c, A.seqs, entry);
    const int64_t len = slot < 0 ? 0 : clamped_len(A.c, A.lens, slot);
    const int64_t left = A.window > 0 && len > A.window ? len - A.window : 0;
    qf[tid] = half_bits_to_float(A.q[entry * A.q_stride + (int64_t)g * kD + tid]);
    float M = -__builtin_huge_valf(), L = 0.0f, o = 0.0f;
    for (int64_t b = left / kG; b * kG < len; ++b) {
        const bool whole = (b + 1) * kG <= len;
        const int64_t at = b * kG + tid;
        int64_t page = whole ? A.c.table[slot * A.c.max_pages + b] : 0;
        const bool bad = page < 0 || page >= A.c.num_pages;
        const uint8_t* rec = record(A.c, bad ? 0 : page, head);
        const uint16_t* ks = reinterpret_cast<const uint16_t*>(rec + kKScales);
        __syncthreads();
        float s = -__builtin_huge_valf();
        if (at >= left && at < len) {
            s = 0.0f;
            if (whole)
                for (int d = 0; d < kD; ++d) {
                    const float c = (float)((rec[tid * kRow + (d >> 1)] >> (4 * (d & 1))) & 15);
                    s += qf[d] * ((c - half_bits_to_float(ks[kD + d])) * half_bits_to_float(ks[d]));
                }
            else
                for (int d = 0; d < kD; ++d)
                    s += qf[d] * half_bits_to_float(window_of(A.c, slot, head, 0)[tid * kD + d]);
            s *= A.scale;
            if (bad) s = __builtin_nanf("");
        }
        const float Mn = __builtin_fmaxf(M, block_max2(s, red));
        const float alpha = __builtin_amdgcn_exp2f(M - Mn);
        M = Mn;
        p[tid] = at >= left && at < len ? __builtin_amdgcn_exp2f(s - M) : 0.0f;
        __syncthreads();
        o *= alpha;
        L *= alpha;
        for (int t = 0; t < kG; ++t) {
            L += p[t];
            if (b * kG + t < left || b * kG + t >= len) continue;
            float v;
            if (whole) {
                const float c = (float)((rec[kVCodes + tid * kRow + (t >> 1)] >> (4 * (t & 1))) & 15);
                v = (c - half_bits_to_float(ks[3 * kD + t])) * half_bits_to_float(ks[2 * kD + t]);
            } else {
                v = half_bits_to_float(window_of(A.c, slot, head, 1)[t * kD + tid]);
            }
            o += p[t] * v;
        }
    }
    A.out[entry * A.out_stride + (int64_t)g * kD + tid] = float_to_half_bits_rne(len > 0 ? o / L : 0.0f);
}

}  // namespace

hipError_t launch_paged_attention(const void* q, int64_t q_stride, int64_t q_heads, const PagedArgs& c,
                                  const int32_t* lens, const int32_t* seqs, int64_t count, int64_t window,
                                  float scale, void* out, int64_t out_stride, int num_cus, const Scratch& ws,
                                  hipStream_t stream) {
    if (ws.sizing()) return hipSuccess;
    const AttnArgs A{c, static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), lens, seqs, q_stride,
                     out_stride, window, (int)q_heads, (int)(q_heads / c.heads), scale * 1.4426950408889634f};
    paged_attn_kernel<<<dim3((unsigned)count, (unsigned)q_heads), dim3(128), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace wq
