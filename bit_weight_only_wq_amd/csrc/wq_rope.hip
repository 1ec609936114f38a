// Rotary positions (gfx950): pair j of a head turns by positions[t] * freqs[j].
//
// One pass over x: what bounds it is HBM (2 bytes in, 2 out per channel).  A
// token's cosines and sines serve all its heads, so a workgroup takes whole
// tokens (or a run of one token's heads), forms the angles once into LDS and
// then streams the heads through registers.
//
// The angle p f is formed in fp64 and reduced to a fraction of a turn there:
// at position 10^6 an fp32 product would already be off by 0.06 radians.  What
// is left, in [-1/2, 1/2] turns, is exact enough in fp32 (2^-25 of a turn), and
// so are its sine and cosine for an fp16 result.
#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 512;   // dim <= 1024

struct RopeArgs {
    const uint16_t* x;
    uint16_t* out;
    const int32_t* pos;
    const double* freqs;
    int64_t tokens, xt, xh, ot, oh;   // strides in elements
    int heads, dim, rot;
    int tokens_per_block, heads_per_block;
    float scale;
    bool copy_rest;                   // channels past rot (not in place)
};

// cos and sin of the block's tokens, tokens_per_block x rot / 2, into LDS.
__device__ __forceinline__ void fill_angles(const RopeArgs& A, int64_t t0, int nt, float2* cs) {
    const int half = A.rot >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        const double turns = (double)A.pos[t0 + t] * A.freqs[j] * 0.15915494309189535;   // 1 / (2 pi)
        const float f = (float)(turns - __builtin_rint(turns));
        float s, c;
        sincospif(2.0f * f, &s, &c);
        cs[i] = make_float2(c * A.scale, s * A.scale);
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return (uint32_t)float_to_half_bits_rne(a) | ((uint32_t)float_to_half_bits_rne(b) << 16);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return half_bits_to_float((uint16_t)u); }
__device__ __forceinline__ float hi_f(uint32_t u) { return half_bits_to_float((uint16_t)(u >> 16)); }

// 16-byte form.  A head is `per_head` chunks: half layout, rot / 16 chunk
// pairs (8 channels at j and 8 at j + rot / 2); interleaved, rot / 8 chunks;
// then the chunks past rot.  A thread keeps one chunk place and walks heads
// (and tokens), so its cosines change only with the token.  8192 tokens of 72
// heads of 128, all turned: 51 us, 5.9 TB/s, what HBM gives a copy.  Heads asked
// for before the angles are formed took 52 to 57 us there, and 7.6 instead of
// 8.5 us for 1777 tokens of 40 heads, half of each turned.
template <bool HALF>
__global__ __launch_bounds__(kThreads) void rope_vec_kernel(const RopeArgs A) {
    __shared__ __align__(16) float2 cs[2 * kMaxPairs];
    const int64_t t0 = (int64_t)blockIdx.x * A.tokens_per_block;
    const int nt = (int)(A.tokens - t0 < A.tokens_per_block ? A.tokens - t0 : A.tokens_per_block);
    const int h0 = blockIdx.y * A.heads_per_block;
    const int nh = A.heads - h0 < A.heads_per_block ? A.heads - h0 : A.heads_per_block;
    fill_angles(A, t0, nt, cs);

    const int turned = HALF ? A.rot >> 4 : A.rot >> 3;
    const int per_head = turned + (A.copy_rest ? (A.dim - A.rot) >> 3 : 0);
    const int step = kThreads / per_head;          // heads a sweep covers (per_head <= 128: dim <= 1024)
    const int c = threadIdx.x % per_head, r = threadIdx.x / per_head;
    if (r >= step) return;
    const int half = A.rot >> 1;
    int t = r / nh, h = r - t * nh;
    const int dt = step / nh, dh = step - dt * nh;
    while (t < nt) {
        const uint16_t* x = A.x + (t0 + t) * A.xt + (int64_t)(h0 + h) * A.xh;
        uint16_t* o = A.out + (t0 + t) * A.ot + (int64_t)(h0 + h) * A.oh;
        if (c >= turned) {
            const int at = A.rot + 8 * (c - turned);
            *reinterpret_cast<uint4*>(o + at) = *reinterpret_cast<const uint4*>(x + at);
        } else if (HALF) {
            const uint4 ua = *reinterpret_cast<const uint4*>(x + 8 * c);
            const uint4 ub = *reinterpret_cast<const uint4*>(x + half + 8 * c);
            const uint32_t a[4] = {ua.x, ua.y, ua.z, ua.w}, b[4] = {ub.x, ub.y, ub.z, ub.w};
            const float4* w = reinterpret_cast<const float4*>(cs + t * half + 8 * c);
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = w[i];             // cos, sin of channels 2i and 2i + 1
                ya[i] = pack2(lo_f(a[i]) * v.x - lo_f(b[i]) * v.y, hi_f(a[i]) * v.z - hi_f(b[i]) * v.w);
                yb[i] = pack2(lo_f(a[i]) * v.y + lo_f(b[i]) * v.x, hi_f(a[i]) * v.w + hi_f(b[i]) * v.z);
            }
            *reinterpret_cast<uint4*>(o + 8 * c) = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            *reinterpret_cast<uint4*>(o + half + 8 * c) = make_uint4(yb[0], yb[1], yb[2], yb[3]);
        } else {
            const uint4 u = *reinterpret_cast<const uint4*>(x + 8 * c);
            const uint32_t a[4] = {u.x, u.y, u.z, u.w};
            const float4* w = reinterpret_cast<const float4*>(cs + t * half + 4 * c);
            const float4 v0 = w[0], v1 = w[1];
            const float co[4] = {v0.x, v0.z, v1.x, v1.z}, si[4] = {v0.y, v0.w, v1.y, v1.w};
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = pack2(lo_f(a[i]) * co[i] - hi_f(a[i]) * si[i], lo_f(a[i]) * si[i] + hi_f(a[i]) * co[i]);
            *reinterpret_cast<uint4*>(o + 8 * c) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        t += dt;
        h += dh;
        if (h >= nh) {
            h -= nh;
            ++t;
        }
    }
}

// Any strides and sizes: one pair, or one channel past rot, at a time.
__global__ __launch_bounds__(kThreads) void rope_any_kernel(const RopeArgs A, bool half_layout) {
    __shared__ __align__(16) float2 cs[2 * kMaxPairs];
    const int64_t t0 = (int64_t)blockIdx.x * A.tokens_per_block;
    const int nt = (int)(A.tokens - t0 < A.tokens_per_block ? A.tokens - t0 : A.tokens_per_block);
    const int h0 = blockIdx.y * A.heads_per_block;
    const int nh = A.heads - h0 < A.heads_per_block ? A.heads - h0 : A.heads_per_block;
    fill_angles(A, t0, nt, cs);
    const int half = A.rot >> 1;
    const int per_head = half + (A.copy_rest ? A.dim - A.rot : 0);
    for (int i = threadIdx.x; i < nt * nh * per_head; i += kThreads) {
        const int row = i / per_head, c = i - row * per_head;
        const int t = row / nh, h = row - t * nh;
        const uint16_t* x = A.x + (t0 + t) * A.xt + (int64_t)(h0 + h) * A.xh;
        uint16_t* o = A.out + (t0 + t) * A.ot + (int64_t)(h0 + h) * A.oh;
        if (c >= half) {
            o[A.rot + c - half] = x[A.rot + c - half];
            continue;
        }
        const int i0 = half_layout ? c : 2 * c, i1 = half_layout ? c + half : 2 * c + 1;
        const float a = half_bits_to_float(x[i0]), b = half_bits_to_float(x[i1]);
        const float2 v = cs[t * half + c];
        o[i0] = float_to_half_bits_rne(a * v.x - b * v.y);
        o[i1] = float_to_half_bits_rne(a * v.y + b * v.x);
    }
}

}  // namespace

hipError_t launch_rope(const RopeCall& c, int num_cus, hipStream_t stream) {
    RopeArgs A;
    A.x = static_cast<const uint16_t*>(c.x);
    A.out = static_cast<uint16_t*>(c.out);
    A.pos = c.positions;
    A.freqs = c.freqs;
    A.tokens = c.tokens;
    A.xt = c.xt;
    A.xh = c.xh;
    A.ot = c.ot;
    A.oh = c.oh;
    A.heads = (int)c.heads;
    A.dim = (int)c.dim;
    A.rot = (int)c.rot;
    A.scale = c.scale;
    A.copy_rest = c.x != c.out && c.rot < c.dim;
    if (c.rot == 0 && !A.copy_rest) return hipSuccess;
    const auto by8 = [](int64_t v) { return v % 8 == 0; };
    const bool aligned = reinterpret_cast<uintptr_t>(c.x) % 16 == 0 && reinterpret_cast<uintptr_t>(c.out) % 16 == 0 &&
                         by8(c.xt) && by8(c.xh) && by8(c.ot) && by8(c.oh) && by8(c.dim) &&
                         c.rot % (c.half_layout ? 16 : 8) == 0;
    // Heads one sweep of a block covers.  Blocks of up to eight sweeps, at most as
    // many blocks as are resident at once (8 a compute unit): 1777 tokens of 40
    // heads take one block a token, 8.5 us; split in two at 32 heads, 9.1.
    const int64_t units = aligned ? c.rot / (c.half_layout ? 16 : 8) + (A.copy_rest ? (c.dim - c.rot) / 8 : 0)
                                  : c.rot / 2 + (A.copy_rest ? c.dim - c.rot : 0);
    const int64_t sweep = kThreads / units > 1 ? kThreads / units : 1;
    int64_t sweeps = (c.tokens * c.heads + sweep * 8 * num_cus - 1) / (sweep * 8 * num_cus);
    sweeps = sweeps < 1 ? 1 : (sweeps > 8 ? 8 : sweeps);
    const int64_t rows = sweep * sweeps;
    const int64_t most = c.rot > 0 ? 4 * kMaxPairs / c.rot : rows;        // tokens whose angles fit in LDS
    int64_t tpb = rows / c.heads;
    tpb = tpb > most ? most : tpb;
    A.tokens_per_block = (int)(tpb < 1 ? 1 : tpb);
    A.heads_per_block = (int)(tpb >= 1 || rows >= c.heads ? c.heads : rows);
    const dim3 grid((unsigned)((c.tokens + A.tokens_per_block - 1) / A.tokens_per_block),
                    (unsigned)((c.heads + A.heads_per_block - 1) / A.heads_per_block));
    if (!aligned)
        rope_any_kernel<<<grid, dim3(kThreads), 0, stream>>>(A, c.half_layout);
    else if (c.half_layout)
        rope_vec_kernel<true><<<grid, dim3(kThreads), 0, stream>>>(A);
    else
        rope_vec_kernel<false><<<grid, dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace wq
