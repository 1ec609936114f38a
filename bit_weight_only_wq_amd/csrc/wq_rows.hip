// Rows of activations (or weights) to 8 bits with one scale a row, and the
// root-mean-square norm with the residual's addition in front of it (gfx950).
//
// With t a row's values before any scaling (the norm: t = h w, h = x + residual
// rounded to the input's type, w the norm's weight; else t = x, or x silu(gate)):
//     code = round-half-even(127 t / max|t|),   value = code * scale
// The norm's factor r = 1 / sqrt(mean h^2 + eps) cancels in 127 t / max|t|, so
// codes do not depend on how the squares were summed; it enters the scale only.
// h and w have at most 11 significant bits each, so t is exact in fp32 (two bf16
// values' below 2^-133 is not: rows whose max is below 2^-100 take their products in
// fp64, and in other rows such a t has code 0).  A code is 127 / max times t in fp32, off by less than 2^-15 (two roundings of a
// number up to 127), and wherever that lies near a border between two codes the
// quotient is formed in fp64.  Without a gate one that is not on the border lies
// 2^-24 from it at least.  Gated values are off by some 2^-52 in fp64; they have
// exact ties too (a value whose gate is that of the row's largest), so what lies
// within 2^-40 of a border counts as on it.
#include <type_traits>

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

// Largest of a row's TPR threads' values, none below 0, in each of them.
template <int TPR>
__device__ __forceinline__ double row_most(double v, double* mosts) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const double t = __shfl_xor(v, o, kWave);
        v = t > v ? t : v;
    }
    if constexpr (TPR > kWave) {
        if ((threadIdx.x & 63) == 0) mosts[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int w = 0; w < TPR / kWave; ++w) v = mosts[w] > v ? mosts[w] : v;
    }
    return v;
}

// round-half-even(127 t / top), ties as above.
__device__ __forceinline__ int exact_code(double t, double top) {
    const double q = 127.0 * t / top;
    const double half = 0.5 * __builtin_rint(2.0 * q);
    return (int)__builtin_rint(__builtin_fabs(q - half) < 0x1p-40 ? half : q);
}

// 1 / sqrt(mean h^2 + eps).  The mean is in 64 bits: bf16's squares may leave fp32's
// range, and sums in another order then give the same factor (but once in 2^28 rows).
__device__ __forceinline__ float norm_factor(const NormCall& A, double sum) {
    const double mean = sum * A.per_value + (double)A.eps;
    return mean > 0x1p-100 && mean < 0x1p100 ? 1.0f / __builtin_sqrtf((float)mean) : (float)(1.0 / sqrt(mean));
}

__device__ __forceinline__ double norm_factor64(const NormCall& A, double sum) {
    return 1.0 / sqrt(sum * A.per_value + (double)A.eps);
}

// The norm's value t r, t = h w.  Two bf16 values' product may be past fp32's largest,
// or lose bits below its smallest normal number, while t r is a bf16 number: then all
// of it is formed in 64 bits.  A product that is 0 is one of a 0, or less than 2^-149:
// then t r is 0 in bf16 too unless r is 2^16 at least.
__device__ __forceinline__ bool past_fp32(float t) { return __builtin_amdgcn_classf(t, 0x294); }   // subnormal or infinite
__device__ __forceinline__ float norm_value64(uint16_t h, uint16_t w, double r) {
    return (float)((double)to_float(h, true) * (double)to_float(w, true) * r);
}

// A row whose largest |t| is below 2^-100, not all of its h being 0: what fp32 says of
// its products may be off.
__device__ __forceinline__ bool small_row(bool bf16, uint32_t top, double sum) { return bf16 && top < 0x0D800000u && sum > 0.0; }
// The scale of a row's codes, most its largest |t|.  (r most may be past fp32, with a bf16
// weight past 2^118, where a 127th of it is not.)
__device__ __forceinline__ float norm_scale(const NormCall& A, bool bf16, double sum, float r, double most, bool small) {
    if (most == 0.0) return 1.0f;
    const float y = r * (float)most;
    return small || (bf16 && y == __builtin_inff()) ? (float)(norm_factor64(A, sum) * most / 127.0) : y / 127.0f;
}

__device__ __forceinline__ double silu64(double g) { return g / (1.0 + exp(-g)); }

// Rows past what registers hold: one workgroup a row, one value at a time, each read
// twice.  2048 rows of 53248: 440 us with a residual (1.7 TB/s), 280 without norm, 619
// gated (exp in 64 bits, twice); 64 such rows, on as many compute units, 149, 81 and 154.
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
    const float r = norm_factor(A, sum);
    const bool fine = top < kInfBits && sum < __builtin_inf(), small = small_row(A.bf16, top, sum);
    double most = (double)__builtin_bit_cast(float, top);
    if (small && A.codes) {
        double m = 0.0;
        for (int64_t k = threadIdx.x; k < A.K; k += kThreads) {
            const double t = __builtin_fabs((double)to_float(h[k], true) * (double)to_float(w[k], true));
            m = t > m ? t : m;
        }
        __shared__ double mosts[kThreads / kWave];
        most = row_most<kThreads>(m, mosts);
    }
    for (int64_t k = threadIdx.x; k < A.K; k += kThreads) {
        const float t = to_float(h[k], A.bf16) * to_float(w[k], A.bf16);
        if (A.out) {
            float y = t * r;
            if (A.bf16 && (past_fp32(t) || t == 0.0f)) y = norm_value64(h[k], w[k], norm_factor64(A, sum));
            static_cast<uint16_t*>(A.out)[row * A.out_stride + k] = from_float(y, A.bf16);
        } else {
            static_cast<int8_t*>(A.codes)[row * A.codes_stride + k] =
                fine && most > 0.0 ? (int8_t)exact_code((double)to_float(h[k], A.bf16) * (double)to_float(w[k], A.bf16), most) : (int8_t)0;
        }
    }
    if (A.codes && threadIdx.x == 0) A.scales[row] = fine ? norm_scale(A, A.bf16, sum, r, most, small) : __builtin_nanf("");
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

// ---- rows in registers ----------------------------------------------------------
//
// TPR threads take a row of up to 8 TPR VPT values, kept in registers from the one
// load to the codes; a wave takes a row by itself where it is short (no meeting),
// a workgroup where it is longer.

enum { MODE_NORM_CODES, MODE_NORM_VALUES, MODE_ROWS, MODE_GATED };

typedef unsigned int u4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u2_t __attribute__((ext_vector_type(2)));
// Global memory takes wide accesses at any address: 8192 rows with a residual, of 8192
// values 88 us, of 8191 130, one value at a time 255; gated, of 11008 91, of 11007 147.
typedef u4_t u4_any __attribute__((aligned(2)));
typedef u2_t u2_any __attribute__((aligned(1)));

// Eight values at p, of which the first n exist; `tail`: whether rows end inside
// eight (the same for all threads, so that other rows skip it at once).
__device__ __forceinline__ u4_t load8(const uint16_t* p, int n, bool tail) {
    u4_t v = {0, 0, 0, 0};
    if (n >= 8) v = *reinterpret_cast<const u4_any*>(p);
    if (tail && n > 0 && n < 8) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) v[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
    return v;
}
__device__ __forceinline__ void store8(uint16_t* p, u4_t v, int n, bool tail) {
    if (n >= 8) *reinterpret_cast<u4_any*>(p) = v;
    if (tail && n > 0 && n < 8) {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
}

template <bool BF16>
__device__ __forceinline__ float part(u4_t v, int e) {
    const uint32_t w = v[e >> 1];
    if (BF16) return __builtin_bit_cast(float, e & 1 ? w & 0xFFFF0000u : w << 16);
    return half_bits_to_float((uint16_t)(e & 1 ? w >> 16 : w));
}

template <bool BF16>
__device__ __forceinline__ u4_t pack8(const float (&f)[8]) {
    u4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (uint32_t)from_float(f[2 * i], BF16) | ((uint32_t)from_float(f[2 * i + 1], BF16) << 16);
    return v;
}

// Largest bit pattern and sum over a row's TPR threads, in each of them.
template <int TPR>
__device__ __forceinline__ void row_join(uint32_t& top, double& sum, uint32_t* tops, double* sums) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t t = __shfl_xor(top, o, kWave);
        top = t > top ? t : top;
        sum += __shfl_xor(sum, o, kWave);
    }
    if constexpr (TPR > kWave) {
        if ((threadIdx.x & 63) == 0) {
            tops[threadIdx.x >> 6] = top;
            sums[threadIdx.x >> 6] = sum;
        }
        __syncthreads();
        top = 0;
        sum = 0.0;
#pragma unroll
        for (int w = 0; w < TPR / kWave; ++w) {
            top = tops[w] > top ? tops[w] : top;
            sum += sums[w];
        }
    }
}

// x silu(g), off by at most 2^-21 of it for g >= -80 (two instructions of one step of
// 2^-23, four roundings of 2^-24): exp(-g) as 2^hi (1 + lo ln 2), hi + lo = -g / ln 2
// in two parts.  Past 100 it is below fp32's half step next to 1.
__device__ __forceinline__ float gated32(float x, float g) {
    const float c = __builtin_fminf(g, 100.0f), hi = c * -1.44269502f;
    const float lo = __builtin_fmaf(c, -1.92596299e-8f, __builtin_fmaf(c, -1.44269502f, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return x * (g * __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e * lo, 0.693147182f, e)));
}

// Codes of eight values t, given 127 / top, and a bit for each that lies within
// `win` of a border between two codes.
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float inv, float win, uint32_t& close) {
    uint32_t z[8];
    float off[8], far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = __builtin_fmaf(t[i], inv, 12582912.0f);     // 1.5 * 2^23: the sum's low bits are the code
        z[i] = __builtin_bit_cast(uint32_t, r);
        off[i] = __builtin_fmaf(t[i], inv, 12582912.0f - r);
        far = __builtin_fmaxf(far, __builtin_fabsf(off[i]));
    }
    close = 0;
    if (!(far <= 0.5f - win))
#pragma unroll
        for (int i = 0; i < 8; ++i) close |= !(__builtin_fabsf(off[i]) <= 0.5f - win) ? 1u << i : 0u;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __builtin_amdgcn_perm(z[4 * i + 1], z[4 * i], 0x0C0C0400u) |
               __builtin_amdgcn_perm(z[4 * i + 3], z[4 * i + 2], 0x04000C0Cu);
    return make_uint2(w[0], w[1]);
}

// The codes of a thread's vectors.  The few next to a border are decided in 64
// bits after all are written, one after another from memory (value(k): the value
// at place k of the row): vector by vector their waits add up (64 rows of 28672
// gated values 12.7 instead of 11.6 us).
template <int TPR, int VPT, class F>
__device__ __forceinline__ void write_codes(const float (&t)[VPT][8], int8_t* codes, int K, bool none, float top, double most,
                                            float win, F value) {
    static_assert(VPT <= 4, "a bit for each value");
    const int tid = threadIdx.x % TPR;
    // (127 / top may be infinite: all in 64 bits then)
    const float inv = 127.0f / top;
    win = top < 0x1p-100f ? 1.0f : win;
    uint32_t close = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = 8 * (i * TPR + tid), n = K - k;
        if (n <= 0) continue;
        uint32_t near = 0;
        uint2 c = make_uint2(0, 0);
        if (!none) c = codes8(t[i], inv, win, near);
        if (n >= 8) *reinterpret_cast<u2_any*>(codes + k) = u2_t{c.x, c.y};
        if ((K & 7) != 0 && n < 8) {
            near &= (1u << n) - 1;
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) codes[k + e] = (int8_t)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
        }
        close |= near << (8 * i);
    }
    while (close) {
        const int bit = __builtin_ctz(close);
        close &= close - 1;
        const int k = ((bit >> 3) * TPR + tid) * 8 + (bit & 7);
        codes[k] = (int8_t)exact_code(value(k), most);
    }
}

// (WAVES: 1024 threads of three vectors, bf16 values, at 64 registers, so that a compute
// unit holds two workgroups.)
template <int MODE, bool BF16, int TPR, int VPT, int WAVES = (MODE == MODE_NORM_VALUES && BF16 && TPR == 1024 && VPT == 3 ? 8 : 1)>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, WAVES) void norm_vec_kernel(const NormCall A) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    __shared__ uint32_t tops[TPR / kWave];
    __shared__ double sums[TPR / kWave], mosts[TPR / kWave];
    const int64_t row = (int64_t)blockIdx.x * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
    if (RPB > 1 && row >= A.rows) return;                           // (a whole wave)
    const int tid = threadIdx.x % TPR, K = (int)A.K;
    const bool tail = (K & 7) != 0;
    const uint16_t* x = static_cast<const uint16_t*>(A.x) + row * A.x_stride;
    const uint16_t* res = static_cast<const uint16_t*>(A.residual) + row * A.residual_stride;
    const uint16_t* wt = static_cast<const uint16_t*>(A.weight);
    uint16_t* total = static_cast<uint16_t*>(A.total) + row * A.total_stride;
    const bool add = A.residual != nullptr;
    u4_t h[VPT], b[VPT], w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = 8 * (i * TPR + tid), n = K - k;
        b[i] = u4_t{0, 0, 0, 0};
        h[i] = load8(x + k, n, tail);
        if (add) b[i] = load8(res + k, n, tail);
        w[i] = load8(wt + k, n, tail);
    }
    float t[VPT][8];
    uint32_t top = 0;
    bool past = false;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = 8 * (i * TPR + tid), n = K - k;
        if (add) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = part<BF16>(h[i], e) + part<BF16>(b[i], e);
            h[i] = pack8<BF16>(f);
            store8(total + k, h[i], n, tail);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float f = part<BF16>(h[i], e);
            t[i][e] = f * part<BF16>(w[i], e);
            const uint32_t u = __builtin_bit_cast(uint32_t, t[i][e]) & 0x7FFFFFFFu;
            top = u > top ? u : top;
            if (MODE == MODE_NORM_VALUES && BF16) past |= past_fp32(t[i][e]);
            sum = __builtin_fma((double)f, (double)f, sum);
        }
    }
    row_join<TPR>(top, sum, tops, sums);
    const float r = norm_factor(A, sum);
    const uint16_t* from = add ? total : x;
    if constexpr (MODE == MODE_NORM_VALUES) {
        uint16_t* out = static_cast<uint16_t*>(A.out) + row * A.out_stride;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = 8 * (i * TPR + tid), n = K - k;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = t[i][e] * r;
            store8(out + k, pack8<BF16>(f), n, tail);
        }
        // What fp32's product does not hold, once all is written (the thread's values one
        // after another from memory: seldom, and few registers).
        if (BF16 && (past || r >= 0x1p16f) && sum > 0.0) {
            const double r64 = norm_factor64(A, sum);
#pragma clang loop unroll(disable)
            for (int v = 0; v < 8 * VPT; ++v) {
                const int k = 8 * ((v >> 3) * TPR + tid) + (v & 7);
                if (k >= K) break;
                const uint16_t hk = from[k], wk = wt[k];
                const float p = to_float(hk, BF16) * to_float(wk, BF16);
                if (past_fp32(p) || p == 0.0f) out[k] = from_float(norm_value64(hk, wk, r64), BF16);
            }
        }
        return;
    }
    const bool fine = top < kInfBits && sum < __builtin_inf(), small = small_row(BF16, top, sum);
    const auto value64 = [&](int k) { return (double)to_float(from[k], BF16) * (double)to_float(wt[k], BF16); };
    double most = (double)__builtin_bit_cast(float, top);
    if (small) {
        double m = 0.0;
#pragma clang loop unroll(disable)
        for (int v = 0; v < 8 * VPT; ++v) {
            const int k = 8 * ((v >> 3) * TPR + tid) + (v & 7);
            if (k >= K) break;
            const double a = __builtin_fabs(value64(k));
            m = a > m ? a : m;
        }
        most = row_most<TPR>(m, mosts);
    }
    write_codes<TPR>(t, static_cast<int8_t*>(A.codes) + row * A.codes_stride, K, !fine || most == 0.0,
                     __builtin_bit_cast(float, top), most, 0x1p-14f, value64);
    if (tid == 0) A.scales[row] = fine ? norm_scale(A, BF16, sum, r, most, small) : __builtin_nanf("");
}

// (WAVES: gated rows of 512 threads are held to registers for another workgroup a
// compute unit: 8192 x 11008 111 -> 95 us, 4096 x 14336 69 -> 63, 8192 x 8192 74 -> 72;
// the other widths lose by it, 8192 x 4096 36 -> 38.)
template <int MODE, bool BF16, int TPR, int VPT, int WAVES = (MODE != MODE_GATED || TPR != 512 ? 1 : VPT == 2 ? 8 : 6)>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, WAVES) void rows_vec_kernel(const RowsCall A) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    constexpr bool GATED = MODE == MODE_GATED;
    __shared__ uint32_t tops[TPR / kWave];
    __shared__ double sums[TPR / kWave], mosts[TPR / kWave];
    const int64_t row = (int64_t)blockIdx.x * RPB + (RPB > 1 ? threadIdx.x / TPR : 0);
    if (RPB > 1 && row >= A.rows) return;                           // (a whole wave)
    const int tid = threadIdx.x % TPR, K = (int)A.K;
    const bool tail = (K & 7) != 0;
    const uint16_t* x = static_cast<const uint16_t*>(A.x) + row * A.x_stride;
    const uint16_t* g = static_cast<const uint16_t*>(A.gate) + row * A.gate_stride;
    u4_t xv[VPT], gv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int k = 8 * (i * TPR + tid), n = K - k;
        xv[i] = load8(x + k, n, tail);
        gv[i] = GATED ? load8(g + k, n, tail) : u4_t{0, 0, 0, 0};
    }
    // A value in 64 bits, from memory again where it is needed (seldom).
    const auto value64 = [&](int k) {
        double y = (double)to_float(x[k], BF16);
        if (GATED) y *= silu64((double)to_float(g[k], BF16));
        return y;
    };
    float t[VPT][8], least = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[i][e] = part<BF16>(xv[i], e);
            if (GATED) {
                const float gate = part<BF16>(gv[i], e);
                t[i][e] = gated32(t[i][e], gate);
                least = __builtin_fminf(least, gate);
            }
            const uint32_t u = __builtin_bit_cast(uint32_t, t[i][e]) & 0x7FFFFFFFu;
            top = u > top ? u : top;
        }
    const float mine = __builtin_bit_cast(float, top);
    // (exp(-gate) may leave fp32's range: the row goes in 64 bits.  So does one whose products
    // are all small, rows of zeros among them.  8192 x 11008: 91 to 107 us, one such gate in
    // every row 431, rows of zeros 212.)
    if (GATED && least < -80.0f) top = 0x80000000u;
    double none = 0.0;
    row_join<TPR>(top, none, tops, sums);
    double most = (double)__builtin_bit_cast(float, top);
    bool bad = top >= kInfBits;
    const bool slow = GATED && (top >= 0x80000000u || top < 0x21800000u);   // 2^-60
    if (GATED) {
        // The largest magnitude in 64 bits: of the values near the largest in 32 (of
        // all of the row's in the slow case).
        double m = 0.0;
        if (slow) {
            bad = false;
            for (int k = tid; k < K; k += TPR) {
                const double y = __builtin_fabs(value64(k));
                m = !(y <= 3.4028234663852886e38) ? __builtin_inf() : y > m ? y : m;
            }
        } else if (!bad && mine >= __builtin_bit_cast(float, top) * (1.0f - 0x1p-18f)) {
            const float near = __builtin_bit_cast(float, top) * (1.0f - 0x1p-18f);
            uint32_t close = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) close |= __builtin_fabsf(t[i][e]) >= near ? 1u << (8 * i + e) : 0u;
            while (close) {
                const int bit = __builtin_ctz(close);
                close &= close - 1;
                const double y = __builtin_fabs(value64(((bit >> 3) * TPR + tid) * 8 + (bit & 7)));
                m = y > m ? y : m;
            }
        }
        most = row_most<TPR>(m, mosts);
        bad |= !(most <= 3.4028234663852886e38);
    }
    const bool zero = most <= 127 * 0x1p-150;                       // most / 127 rounds to 0
    // (gated32 is off by 2^-21 at most, a quotient by 2^-14; in the slow case every code is decided in 64 bits)
    write_codes<TPR>(t, static_cast<int8_t*>(A.codes) + row * A.codes_stride, K, bad || zero, slow ? 0.0f : (float)most, most,
                     GATED ? 0x1p-13f : 0x1p-14f, value64);
    if (tid == 0) A.scales[row] = bad ? __builtin_nanf("") : zero ? 1.0f : (float)(most / 127.0);
}

// Runs f with the row's threads and vectors a thread as constants: two vectors a
// thread, so that several workgroups a compute unit wait for memory by turns.  (Times
// that are compared were taken together; a long burst's are 5 to 10 % lower than those
// of its first hundred calls, as the clock rises.)
// 8192 rows of 8192 with a residual: 512 threads of two 86 us (5.4 TB/s), 256 of four
// 94, 1024 of one 95; of 4864: 256 of three 61 us, 512 of two 69; of 11008, gated: 512
// of three 90 us (5.0 TB/s), 1024 of two 129, 256 of six 315 (they spill); of 4096: 256
// of two 46 us, 512 of one 48, a wave of eight 121; 2048 rows of 20480 without norm:
// 1024 of three 26 us, of four 33; 28672 rows of 8192 117 us, 6.0 TB/s.  What bounds the
// norm and the plain rows is HBM, the gated ones the vector units as well (some 30
// instructions a value).
template <class F>
void with_width(int64_t K, F f) {
    using std::integral_constant;
    if (K <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (K <= 1024) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (K <= 2048) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (K <= 4096) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (K <= 6144) f(integral_constant<int, 256>{}, integral_constant<int, 3>{});
    else if (K <= 8192) f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else if (K <= 12288) f(integral_constant<int, 512>{}, integral_constant<int, 3>{});
    else if (K <= 16384) f(integral_constant<int, 512>{}, integral_constant<int, 4>{});
    else if (K <= 24576) f(integral_constant<int, 1024>{}, integral_constant<int, 3>{});
    else f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <int MODE, bool BF16>
void run_norm_vec(const NormCall& c, hipStream_t stream) {
    with_width(c.K, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value, RPB = TPR < 256 ? 256 / TPR : 1;
        norm_vec_kernel<MODE, BF16, TPR, VPT><<<dim3((unsigned)((c.rows + RPB - 1) / RPB)), dim3(TPR * RPB), 0, stream>>>(c);
    });
}

template <int MODE, bool BF16>
void run_rows_vec(const RowsCall& c, hipStream_t stream) {
    with_width(c.K, [&](auto tpr, auto vpt) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value, RPB = TPR < 256 ? 256 / TPR : 1;
        rows_vec_kernel<MODE, BF16, TPR, VPT><<<dim3((unsigned)((c.rows + RPB - 1) / RPB)), dim3(TPR * RPB), 0, stream>>>(c);
    });
}

}  // namespace

constexpr int64_t kWidest = 32768;          // values of a row that 1024 threads hold
constexpr int64_t kRows = (int64_t)1 << 20;   // of a launch: a grid holds fewer than 2^32 threads

static const void* after(const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; }
static void* after(void* p, int64_t bytes) { return p ? static_cast<char*>(p) + bytes : nullptr; }

hipError_t launch_norm(const NormCall& all, hipStream_t stream) {
    for (int64_t r = 0; r < all.rows; r += kRows) {
        NormCall c = all;
        c.rows = all.rows - r < kRows ? all.rows - r : kRows;
        c.x = after(all.x, 2 * r * all.x_stride);
        c.residual = after(all.residual, 2 * r * all.residual_stride);
        c.total = after(all.total, 2 * r * all.total_stride);
        c.codes = after(all.codes, r * all.codes_stride);
        c.out = after(all.out, 2 * r * all.out_stride);
        c.scales = all.scales ? all.scales + r : nullptr;
        if (c.K > kWidest) norm_any_kernel<<<dim3((unsigned)c.rows), dim3(kThreads), 0, stream>>>(c);
        else if (c.codes && c.bf16) run_norm_vec<MODE_NORM_CODES, true>(c, stream);
        else if (c.codes) run_norm_vec<MODE_NORM_CODES, false>(c, stream);
        else if (c.bf16) run_norm_vec<MODE_NORM_VALUES, true>(c, stream);
        else run_norm_vec<MODE_NORM_VALUES, false>(c, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_rows(const RowsCall& all, hipStream_t stream) {
    for (int64_t r = 0; r < all.rows; r += kRows) {
        RowsCall c = all;
        c.rows = all.rows - r < kRows ? all.rows - r : kRows;
        c.x = after(all.x, 2 * r * all.x_stride);
        c.gate = after(all.gate, 2 * r * all.gate_stride);
        c.codes = after(all.codes, r * all.codes_stride);
        c.scales = all.scales + r;
        if (c.K > kWidest) rows_any_kernel<<<dim3((unsigned)c.rows), dim3(kThreads), 0, stream>>>(c);
        else if (c.gate && c.bf16) run_rows_vec<MODE_GATED, true>(c, stream);
        else if (c.gate) run_rows_vec<MODE_GATED, false>(c, stream);
        else if (c.bf16) run_rows_vec<MODE_ROWS, true>(c, stream);
        else run_rows_vec<MODE_ROWS, false>(c, stream);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace wq
