// Product of 8-bit activations and 8-bit weights (gfx950):
//     Y[b, n] = a_scales[b] w_scales[n] sum_k A[b, k] W[n, k] + bias[n]
// The sum is exact (int32; K < 2^17), so however it is split it comes out the
// same: results do not depend on the kernel, the batch or the split.
//
// Two kernels, both on the int8 matrix instructions, both fed through LDS by
// loads that write it directly, in pieces of 128 bytes of a row (pieces of 64
// come at half the rate: 17 instead of 33 TB/s from the caches, 4.6 instead of
// 8.5 from the memory-side one).  Chunk c (16 bytes) of a slot's row p lies at
// place c ^ (p / 2 & 7), so that 16 lanes that read one chunk of 16 rows touch
// all 64 banks (by p & 7 instead, half of all LDS cycles were conflicts).
//   w8_wide_kernel  256 x 256 or 128 x 128 tiles, two slots, 32x32x32 products;
//                   compute-bound sizes.  Workgroups stay and take tile after
//                   tile, the next one's loads running while the last one's
//                   results are stored.
//   w8_ring_kernel  smaller tiles, four or eight slots, 16x16x64 products, K
//                   split over workgroups where there are few tiles; what is
//                   bound by reading W.
// Rows past B or N and k past K are read as zeros: offsets past a buffer's end.
#include <type_traits>

#include "wq_device.h"
#include "wq_launch.h"

namespace wq {

namespace {

typedef int i4_t __attribute__((ext_vector_type(4)));
typedef int i16_t __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void w8_lds_t;

constexpr int kStep = 128;               // k (bytes) of a step
constexpr uint32_t kFar = 0x80000000u;   // an offset past every buffer (strides are at most 2^22, tiles 256 rows)

__device__ __forceinline__ __amdgpu_buffer_rsrc_t w8_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}

// s_waitcnt: vmcnt(n) and lgkmcnt(0).
constexpr int w8_wait(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// All waves meet; what they wrote to or read from LDS before is done.
__device__ __forceinline__ void w8_meet() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ float w8_bias(uint16_t b, bool bf16) {
    return bf16 ? __builtin_bit_cast(float, (uint32_t)b << 16) : half_bits_to_float(b);
}

// acc a w + bias, every step rounded by itself (no fused multiply-add), so that
// all kernels give the same bits.
__device__ __forceinline__ uint16_t w8_value(int acc, float as, float ws, bool has_bias, float bias, bool bf16) {
#pragma clang fp contract(off)
    float y = (float)acc * as;
    y = y * ws;
    if (has_bias) y = y + bias;
    return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : float_to_half_bits_rne(y);
}

// Instruction order of NM products, ND shared-memory reads and NV loads: after
// each product one read and one load, as long as there are any.
template <int NM, int ND, int NV, int I = 0>
struct Spread {
    static __device__ __forceinline__ void go() {
        if constexpr (I < NM) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            constexpr int v = (I + 1) * NV * 2 / NM - I * NV * 2 / NM, d = (I + 1) * ND * 4 / 3 / NM - I * ND * 4 / 3 / NM;
            if constexpr (I * NV * 2 / NM < NV && v > 0) __builtin_amdgcn_sched_group_barrier(0x20, v, 0);
            if constexpr (I * ND * 4 / 3 / NM < ND && d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
            Spread<NM, ND, NV, I + 1>::go();
        }
    }
};

// Scales a wave's sums and stores them.  A lane holds, of every 32 x 32 block
// (i, j), rows 8 (e / 4) + 4 (lane / 32) + e % 4 of A and column NF (lane % 32) + j
// of the wave's W rows, so it has NF neighbouring values of a row of Y.  Y goes
// through a buffer that ends with the last row: rows past it are dropped.  The
// stores are marked as streamed (the 2), so that Y does not push A and W out of the
// caches: 8192 x 4096 x 22016 656 -> 618 us, 2048 x 4096 x 12288 122 -> 116.
template <int MF, int NF, bool BF16>
__device__ __forceinline__ bool w8_store(const W8Call& C, const i16_t (&acc)[MF][NF], int64_t b0, int64_t n0,
                                         const float* sal, const float* swl) {
#pragma clang fp contract(off)
    const int r32 = threadIdx.x & 31, g2 = (threadIdx.x >> 5) & 1;
    const int rows = (int)(C.B - b0 < 32 * MF ? C.B - b0 : 32 * MF);
    if (rows <= 0) return false;
    uint32_t stride = 2u * (uint32_t)C.y_stride;
    asm volatile("" : "+s"(stride));    // the rows' offsets are formed here, not kept through the products
    const auto ry = w8_rsrc(static_cast<uint16_t*>(C.Y) + b0 * C.y_stride, (uint32_t)(rows - 1) * stride + 2u * (uint32_t)C.N);
    const uint32_t n = (uint32_t)n0 + r32 * NF, N = (uint32_t)C.N;
    const bool wide = N % NF == 0 && C.y_stride % NF == 0 && reinterpret_cast<uintptr_t>(C.Y) % (2 * NF) == 0;
    float sw[NF], bs[NF];
#pragma unroll
    for (int j = 0; j < NF; ++j) sw[j] = swl[r32 * NF + j];
    if (C.bias)
#pragma unroll
        for (int j = 0; j < NF; ++j) bs[j] = w8_bias(static_cast<const uint16_t*>(C.bias)[n + j < N ? n + j : N - 1], BF16);
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 s4 = *reinterpret_cast<const float4*>(sal + i * 32 + q * 8 + g2 * 4);
            const float sa[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float y[NF];
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    y[j] = (float)acc[i][j][4 * q + r] * sa[r];
                    y[j] = y[j] * sw[j];
                }
                if (C.bias)
#pragma unroll
                    for (int j = 0; j < NF; ++j) y[j] = y[j] + bs[j];
                uint16_t o[NF];
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    o[j] = BF16 ? __builtin_bit_cast(uint16_t, (__bf16)y[j]) : float_to_half_bits_rne(y[j]);
                const uint32_t at = (uint32_t)(i * 32 + q * 8 + r + g2 * 4) * stride + 2 * n;
                if (wide) {
                    const int to = (int)(n < N ? at : kFar);
                    if constexpr (NF == 4) {
                        typedef unsigned int v2_t __attribute__((ext_vector_type(2)));
                        __builtin_amdgcn_raw_buffer_store_b64(v2_t{o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16}, ry, to, 0, 2);
                    } else {
                        __builtin_amdgcn_raw_buffer_store_b32(o[0] | (uint32_t)o[1] << 16, ry, to, 0, 2);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < NF; ++j)
                        __builtin_amdgcn_raw_buffer_store_b16((short)o[j], ry, (int)(n + j < N ? at + 2 * j : kFar), 0, 0);
                }
            }
        }
    return true;
}

// A tile's place and its operands.
struct W8Tile {
    const uint8_t *a, *w;
    uint32_t abytes, wbytes, K;    // K = 0: no tile, nothing is read
    int64_t b0, n0;
};

// Two slots of 128 k.  In the first half of a step's products (two of its four
// pieces of 32 k) the other half's operands are read from LDS; then the waves
// meet, the slot is free and the other one has landed; in the second half the
// slot is loaded anew and the next step's first operands are read.  So one meeting
// a step, with products waiting on both sides of it.  8192 x 8192 x 28672: 1.51 ms,
// 2550 TOP/s; the products' own time is 73 % of the cycles, and the clock then
// stands at 1.7 GHz, held there by power (operands of zeros: 1.37 ms).  Measured
// besides: steps of 64 k in four slots 1.61 ms (twice the meetings, pieces of 64
// bytes); four waves of 128 x 128 1.59 ms; workgroups that end with their tile
// 1.61 ms.
template <int BM, int BN, int WM, int WN, int THREADS = (BM / WM) * (BN / WN) * 64>
__global__ __launch_bounds__(THREADS, 1) void w8_wide_kernel(const W8Call C, int tiles_m, int tiles_n) {
    constexpr int WAVES = THREADS / 64, MF = WM / 32, NF = WN / 32;
    constexpr int LA = BM / 8 / WAVES, LW = BN / 8 / WAVES;         // 1 KB loads of a wave a step
    static_assert(BM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0 && WAVES % 2 == 0, "loads divide evenly");
    __shared__ __align__(1024) uint4 as0[BM * 8], as1[BM * 8], ws0[BN * 8], ws1[BN * 8];
    __shared__ __align__(256) float sal[BM], swl[BN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const uint32_t K = (uint32_t)C.K;

    // Workgroups are dealt to the eight XCDs in turn.  Each XCD takes a run of the
    // tile order, which walks eight tiles of A before the next tile of W, and its
    // workgroups take that run's tiles in turn.
    const int total = tiles_m * tiles_n, xcd = blockIdx.x % 8;
    const int per = total / 8, rest = total % 8;
    int id = xcd * per + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    const int end = (xcd + 1) * per + (xcd + 1 < rest ? xcd + 1 : rest);
    const int hop = (gridDim.x + 7 - xcd) / 8;
    const auto place = [&](int id) {
        W8Tile T;
        T.K = id < end ? K : 0u;
        id = id < end ? id : 0;
        const int group = id / (8 * tiles_n), gm = tiles_m - group * 8 < 8 ? tiles_m - group * 8 : 8;
        const int in = id - group * 8 * tiles_n;
        T.b0 = (int64_t)(group * 8 + in % gm) * BM;
        T.n0 = (int64_t)(in / gm) * BN;
        const int rows_a = (int)(C.B - T.b0 < BM ? C.B - T.b0 : BM), rows_w = (int)(C.N - T.n0 < BN ? C.N - T.n0 : BN);
        T.a = static_cast<const uint8_t*>(C.A) + T.b0 * C.a_stride;
        T.w = static_cast<const uint8_t*>(C.W) + T.n0 * C.w_stride;
        T.abytes = (uint32_t)(rows_a - 1) * (uint32_t)C.a_stride + K;
        T.wbytes = (uint32_t)(rows_w - 1) * (uint32_t)C.w_stride + K;
        return T;
    };

    // Row p of a wave's WN rows in LDS is its row NF (p % 32) + p / 32 of W, so that
    // a lane's columns of Y are neighbours.
    uint32_t aoff[LA], woff[LW];
    const int row = 8 * wave + (lane >> 3);                         // (8 WAVES rows on, the chunk is the same)
    const uint32_t chunk = 16u * ((lane & 7) ^ ((row >> 1) & 7));
#pragma unroll
    for (int q = 0; q < LA; ++q) aoff[q] = (uint32_t)(8 * WAVES * q + row) * (uint32_t)C.a_stride + chunk;
#pragma unroll
    for (int q = 0; q < LW; ++q) {
        const int p = 8 * WAVES * q + row, pw = p % WN;
        woff[q] = (uint32_t)(p - pw + (pw % 32) * NF + pw / 32) * (uint32_t)C.w_stride + chunk;
    }
    const auto load = [&](const W8Tile& T, uint32_t k, uint4* as, uint4* ws) {
        const bool in = k + chunk < T.K;
        const int base = (int)(k < T.K ? k : 0u);                   // (never past a buffer's end)
        const auto ra = w8_rsrc(T.a, T.abytes), rw = w8_rsrc(T.w, T.wbytes);
#pragma unroll
        for (int q = 0; q < LA; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (w8_lds_t*)(as + 64 * (WAVES * q + wave)), 16,
                                                     (int)(in ? aoff[q] : kFar), base, 0, 0);
#pragma unroll
        for (int q = 0; q < LW; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w8_lds_t*)(ws + 64 * (WAVES * q + wave)), 16,
                                                     (int)(in ? woff[q] : kFar), base, 0, 0);
    };
    // A tile's scales; rows past the end get zeros.
    const auto load_scales = [&](const W8Tile& T) {
        const auto ra = w8_rsrc(C.a_scales + T.b0, 4u * (uint32_t)(C.B - T.b0 < BM ? C.B - T.b0 : BM));
        const auto rw = w8_rsrc(C.w_scales + T.n0, 4u * (uint32_t)(C.N - T.n0 < BN ? C.N - T.n0 : BN));
#pragma unroll
        for (int q = 0; q < (BM + BN) / 64; q += WAVES) {
            const int at = q + wave;
            if (at < BM / 64)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (w8_lds_t*)(sal + 64 * at), 4, (64 * at + lane) * 4, 0, 0, 0);
            else if (at < (BM + BN) / 64)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w8_lds_t*)(swl + 64 * (at - BM / 64)), 4,
                                                         (64 * (at - BM / 64) + lane) * 4, 0, 0, 0);
        }
    };

    i16_t acc[MF][NF];
    const auto clear = [&] {
#pragma unroll
        for (int i = 0; i < MF; ++i)
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    };
    clear();
    const int r32 = lane & 31, g2 = lane >> 5;
    const int arow = (wm * WM + r32) * 8, wrow = (wn * WN + r32) * 8, key = (r32 >> 1) & 7;
    int at[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) at[s] = (2 * s + g2) ^ key;
    struct Frags {
        i4_t a[2][MF], w[2][NF];
    };
    const auto read = [&](Frags& f, const uint4* as, const uint4* ws, int h) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < MF; ++i) f.a[s][i] = __builtin_bit_cast(i4_t, as[arow + at[2 * h + s] + i * 256]);
#pragma unroll
            for (int j = 0; j < NF; ++j) f.w[s][j] = __builtin_bit_cast(i4_t, ws[wrow + at[2 * h + s] + j * 256]);
        }
    };
    constexpr int NM = 2 * MF * NF, ND = 2 * (MF + NF);
    constexpr std::integral_constant<int, 0> none{};
    constexpr std::integral_constant<int, LA + LW> some{};
    const auto mm = [&](const Frags& f, auto loads) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < MF; ++i)
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[s][i], f.w[s][j], acc[i][j], 0, 0, 0);
        Spread<NM, ND, decltype(loads)::value>::go();
        __builtin_amdgcn_sched_barrier(0);
    };
    // The other slot has landed, and all waves have read this one.  A tile begins
    // with both slots landed, so its first meeting waits for no load (nor for the
    // stores of the tile before).
    const auto landed = [&](bool fresh) {
        if (fresh) __builtin_amdgcn_s_waitcnt(w8_wait(63));
        else __builtin_amdgcn_s_waitcnt(0);
        w8_meet();
    };

    const uint32_t span = (K + 2 * kStep - 1) / (2 * kStep) * (2 * kStep);   // k of a tile, in pairs of steps
    Frags f0, f1;
    W8Tile T = place(id);
    load(T, 0, as0, ws0);
    load(T, kStep, as1, ws1);
    __builtin_amdgcn_s_waitcnt(0);
    w8_meet();
    for (;;) {
        read(f0, as0, ws0, 0);
        id += hop;
        const W8Tile next = place(id);
        for (uint32_t k = 0; k < span; k += 2 * kStep) {
            const bool last = k + 2 * kStep >= span;
            const uint32_t k2 = last ? 0 : k + 2 * kStep;
            W8Tile L = T;
            if (last) L = next;
            read(f1, as0, ws0, 1);
            mm(f0, none);
            landed(k == 0);
            if (k == 0) load_scales(T);
            load(L, k2, as0, ws0);
            read(f0, as1, ws1, 0);
            mm(f1, some);
            read(f1, as1, ws1, 1);
            mm(f0, none);
            landed(false);
            load(L, k2 + kStep, as1, ws1);
            read(f0, as0, ws0, 0);
            mm(f1, some);
        }
        const int64_t b0 = T.b0 + wm * WM, nw = T.n0 + wn * WN;
        const bool stored = C.bf16 ? w8_store<MF, NF, true>(C, acc, b0, nw, sal + wm * WM, swl + wn * WN)
                                   : w8_store<MF, NF, false>(C, acc, b0, nw, sal + wm * WM, swl + wn * WN);
        if (id >= end) break;
        clear();
        T = next;
        // The next tile's loads came before this one's stores, which are 16 MF at least.
        if (stored) __builtin_amdgcn_s_waitcnt(w8_wait(16 * MF));
        else __builtin_amdgcn_s_waitcnt(w8_wait(0));
        w8_meet();
    }
    __builtin_amdgcn_s_waitcnt(0);
}

// A workgroup's tile of BM rows of A and BN rows of W through a ring of S slots of
// 128 k, loaded S - 1 steps ahead; a wave takes WM by WN of it.  KG groups of waves
// take parts of K, each with a ring of its own, and meet at the end: where there is
// one workgroup a compute unit, a step's own latency (meeting, reads from LDS,
// products one after another) is what counts, and KG steps then run at once.  With splits, part z
// of K goes to plane z of the partial sums.  28672 x 8192: 42 us at one row, 43 at
// 16 (5.5 TB/s; a kernel that only reads gets 6.5), 47 at 64, 59 at 128.  W straight
// to registers instead, K split over a workgroup's waves, took 49 us at one row and
// 72 at 16 (pieces of 64 bytes, A read by every wave); lines of W asked for into the
// cache further ahead made it slower (42 -> 65 us), and so did no shift of the walks
// (45 -> 49 us at one row).
template <int BM, int BN, int WM, int WN, int S, int KG, int THREADS = KG * (BM / WM) * (BN / WN) * 64>
__global__ __launch_bounds__(THREADS) void w8_ring_kernel(const W8Call C, int* part, int splits, int split_steps) {
    constexpr int WAVES = THREADS / 64 / KG, MF = WM / 16, NF = WN / 16;   // (waves of a group)
    constexpr int RM = BM < 8 * WAVES ? 8 * WAVES : BM;             // rows of a slot: whole loads for every wave
    constexpr int LA = RM / 8 / WAVES, LW = BN / 8 / WAVES;
    static_assert(RM % (8 * WAVES) == 0 && BN % (8 * WAVES) == 0, "loads divide evenly");
    constexpr int SLOT = (RM + BN) * 8;
    __shared__ __align__(1024) uint4 s0[KG * SLOT], s1[KG * SLOT], s2[KG * SLOT], s3[KG * SLOT];
    constexpr int MORE = S == 8 ? KG * SLOT : 1;
    __shared__ __align__(1024) uint4 s4[MORE], s5[MORE], s6[MORE], s7[MORE];
    static_assert(S == 4 || S == 8, "the walk below");
    const int lane = threadIdx.x & 63, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = any_wave % WAVES, group = any_wave / WAVES;
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const int r16 = lane & 15, g4 = lane >> 4;
    // The eight XCDs take runs of the order rows of A, then of W, then splits of K:
    // tiles that share W rows run on one XCD, whose cache then reads them once.
    const int tiles_n = (int)((C.N + BN - 1) / BN), tiles_m = (int)((C.B + BM - 1) / BM);
    const int xcd = blockIdx.x % 8, rest = gridDim.x % 8;
    const int id = xcd * (gridDim.x / 8) + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    const int tn = id / tiles_m % tiles_n, z = id / tiles_m / tiles_n;
    const int64_t n0 = (int64_t)tn * BN, b0 = (int64_t)(id % tiles_m) * BM;
    const int rows_a = (int)(C.B - b0 < BM ? C.B - b0 : BM), rows_w = (int)(C.N - n0 < BN ? C.N - n0 : BN);
    const uint8_t* const a = static_cast<const uint8_t*>(C.A) + b0 * C.a_stride;
    const uint8_t* const w = static_cast<const uint8_t*>(C.W) + n0 * C.w_stride;
    const uint32_t K = (uint32_t)C.K;
    // This workgroup's part of K, and this group's part of that (which may be empty).
    const int all = (int)((K + kStep - 1) / kStep) - z * split_steps, part_steps = all < split_steps ? all : split_steps;
    const int turns = (part_steps + KG - 1) / KG, first = z * split_steps + group * turns;
    const int left = part_steps - group * turns, steps = left < turns ? (left > 0 ? left : 0) : turns;
    // Workgroups start their walks over K at different steps (and wrap): rows lie
    // K apart, and the same columns of many rows fall on the same memory channels.
    const int shift = steps > 0 ? (id / tiles_m) * 5 % steps : 0;
    const uint32_t abytes = (uint32_t)(rows_a - 1) * (uint32_t)C.a_stride + K;
    const uint32_t wbytes = (uint32_t)(rows_w - 1) * (uint32_t)C.w_stride + K;
    // Chunk c of row p lies at c ^ (p / 2 & 7).
    uint32_t aoff[LA], woff[LW];
    const int row = 8 * wave + (lane >> 3);                        // (8 WAVES rows on, the chunk is the same)
    const uint32_t chunk = 16u * ((lane & 7) ^ ((row >> 1) & 7));
    static_assert(WAVES % 2 == 0, "4 WAVES is a multiple of 8");
#pragma unroll
    for (int q = 0; q < LA; ++q) aoff[q] = (uint32_t)(8 * WAVES * q + row) * (uint32_t)C.a_stride + chunk;
#pragma unroll
    for (int q = 0; q < LW; ++q) woff[q] = (uint32_t)(8 * WAVES * q + row) * (uint32_t)C.w_stride + chunk;
    const auto ra = w8_rsrc(a, abytes), rw = w8_rsrc(w, wbytes);
    // Step `step` of this part of K; past its end, and past K, nothing is read and
    // zeros are written.
    const auto load = [&](int step, uint4* s) {
        const int at = step + shift < steps ? step + shift : step + shift - steps;
        const uint32_t k = step < steps ? (uint32_t)(first + at) * kStep : 0u;   // (never past a buffer's end)
        const bool in = k + chunk < (step < steps ? K : 0u);
#pragma unroll
        for (int q = 0; q < LW; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (w8_lds_t*)(s + group * SLOT + 64 * (WAVES * q + wave)), 16,
                                                     (int)(in ? woff[q] : kFar), (int)k, 0, 0);
#pragma unroll
        for (int q = 0; q < LA; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (w8_lds_t*)(s + group * SLOT + BN * 8 + 64 * (WAVES * q + wave)), 16,
                                                     (int)(in ? aoff[q] : kFar), (int)k, 0, 0);
    };
    i4_t acc[MF][NF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[m][j] = i4_t{0, 0, 0, 0};
    const int key = (r16 >> 1) & 7;
    struct Frags {
        i4_t a[2][MF], w[2][NF];
    };
    const int c0 = g4 ^ key, c1 = (4 + g4) ^ key;
    const int wrow = group * SLOT + (wn * WN + r16) * 8, arow = group * SLOT + BN * 8 + (wm * WM + r16) * 8;
    const auto read = [&](Frags& f, const uint4* s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < NF; ++j) f.w[h][j] = __builtin_bit_cast(i4_t, s[wrow + j * 128 + (h ? c1 : c0)]);
#pragma unroll
            for (int m = 0; m < MF; ++m) f.a[h][m] = __builtin_bit_cast(i4_t, s[arow + m * 128 + (h ? c1 : c0)]);
        }
    };
    const auto mm = [&](const Frags& f) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int j = 0; j < NF; ++j) acc[m][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[h][j], f.a[h][m], acc[m][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto turn = [&] {
        __builtin_amdgcn_s_waitcnt(w8_wait((S - 2) * (LA + LW)));
        w8_meet();
    };
    load(0, s0);
    load(1, s1);
    load(2, s2);
    load(3, s3);
    if constexpr (S == 8) load(4, s4), load(5, s5), load(6, s6), load(7, s7);
    Frags f0, f1;
    __builtin_amdgcn_s_waitcnt(w8_wait((S - 1) * (LA + LW)));
    w8_meet();
    read(f0, s0);
    // Step u: slot `at` is free (its values are in f), the next step's has landed.
    const auto one = [&](int u, uint4* at, const uint4* next, const Frags& f, Frags& g) {
        turn();
        load(u + S, at);
        read(g, next);
        mm(f);
    };
    for (int u = 0; u < turns; u += S) {
        one(u, s0, s1, f0, f1);
        one(u + 1, s1, s2, f1, f0);
        one(u + 2, s2, s3, f0, f1);
        if constexpr (S == 4) one(u + 3, s3, s0, f1, f0);
        if constexpr (S == 8) {
            one(u + 3, s3, s4, f1, f0);
            if (u + 4 >= turns) break;
            one(u + 4, s4, s5, f0, f1);
            one(u + 5, s5, s6, f1, f0);
            one(u + 6, s6, s7, f0, f1);
            one(u + 7, s7, s0, f1, f0);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    if constexpr (KG > 1) {
        // The groups' sums meet in the first group's registers.
        constexpr int EACH = MF * NF * 64 * WAVES;
        static_assert((KG - 1) * EACH <= KG * SLOT, "the sums fit a slot");
        i4_t* const sums = reinterpret_cast<i4_t*>(s0);
        w8_meet();
        if (group > 0)
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int j = 0; j < NF; ++j) sums[(group - 1) * EACH + ((m * NF + j) * WAVES + wave) * 64 + lane] = acc[m][j];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g)
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int j = 0; j < NF; ++j) acc[m][j] += sums[g * EACH + ((m * NF + j) * WAVES + wave) * 64 + lane];
    }

    // A lane holds four neighbouring columns of row r16 of each block.
    const uint16_t* bias = static_cast<const uint16_t*>(C.bias);
    uint16_t* Y = static_cast<uint16_t*>(C.Y);
    const bool wide = C.N % 4 == 0 && C.y_stride % 4 == 0 && reinterpret_cast<uintptr_t>(Y) % 8 == 0;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const int64_t n = n0 + wn * WN + j * 16 + g4 * 4;
        if (n >= C.N) continue;
        float sw[4], bs[4];
        if (splits == 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t ni = n + i < C.N ? n + i : C.N - 1;
                sw[i] = C.w_scales[ni];
                bs[i] = bias ? w8_bias(bias[ni], C.bf16) : 0.0f;
            }
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int64_t b = b0 + wm * WM + m * 16 + r16;
            if (b >= C.B) continue;
            if (splits > 1) {
                *reinterpret_cast<i4_t*>(part + ((int64_t)z * C.B + b) * ((C.N + 3) / 4 * 4) + n) = acc[m][j];
                continue;
            }
            const float sa = C.a_scales[b];
            uint16_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = w8_value(acc[m][j][i], sa, sw[i], bias != nullptr, bs[i], C.bf16);
            uint16_t* y = Y + b * C.y_stride + n;
            if (wide)
                *reinterpret_cast<uint2*>(y) = make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < C.N) y[i] = o[i];
        }
    }
}

// Sums of the splits of K, scaled: four columns a thread, eight planes asked for at
// a time (333 x 4096 in two planes: 4.8 us; one plane after another 5.7).
__global__ __launch_bounds__(256) void w8_join_kernel(const W8Call C, const int* part, int splits) {
    const int64_t quads = (C.N + 3) / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads * C.B) return;
    const int64_t b = (uint32_t)i / (uint32_t)quads, n = (i - b * quads) * 4, plane = C.B * quads * 4;
    const float sa = C.a_scales[b];
    float sw[4], bs[4];
    const uint16_t* bias = static_cast<const uint16_t*>(C.bias);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t nj = n + j < C.N ? n + j : C.N - 1;
        sw[j] = C.w_scales[nj];
        bs[j] = bias ? w8_bias(bias[nj], C.bf16) : 0.0f;
    }
    i4_t sum = i4_t{0, 0, 0, 0};
    for (int z = 0; z < splits; z += 8) {
        i4_t p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            p[u] = i4_t{0, 0, 0, 0};
            if (z + u < splits) p[u] = *reinterpret_cast<const i4_t*>(part + (z + u) * plane + i * 4);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += p[u];
    }
    uint16_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = w8_value(sum[j], sa, sw[j], bias != nullptr, bs[j], C.bf16);
    uint16_t* y = static_cast<uint16_t*>(C.Y) + b * C.y_stride + n;
    if (C.N % 4 == 0 && C.y_stride % 4 == 0 && reinterpret_cast<uintptr_t>(C.Y) % 8 == 0)
        *reinterpret_cast<uint2*>(y) = make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
    else
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < C.N) y[j] = o[j];
}

// ---- which kernel ------------------------------------------------------------------

enum W8Shape { R16x32, R32x32, R32x64, R32x128, R64x32, R64x64, R64x128, R128x64, R128x128, W128, W256 };

struct W8Plan {
    W8Shape shape;
    int splits;
};

// Sizes of a variant, workgroups a compute unit holds, and what it costs in us:
// first, and for each step with that many (1, 2, 3) workgroups on every compute
// unit.  Fitted to B = 48 .. 2048 on nine matrices, 512 x 512 to 28672 x 8192.  What it
// takes now for K = 4096: N = 4096, B = 100, 200, 500, 1000: 9.6, 14, 18, 26 us; N = 12288:
// 18, 24, 40, 57; N = 22016: 31, 43, 61, 121.
struct W8Cost {
    W8Shape shape;
    int bm, bn, fit;
    double first, step[3];
};
constexpr W8Cost kCosts[] = {
    {R64x32, 64, 32, 3, 3.9, {0.20, 0.42, 0.60}},  {R64x64, 64, 64, 2, 4.2, {0.34, 0.56, 0}},
    {R128x64, 128, 64, 1, 4.5, {0.45, 0, 0}},       {R128x128, 128, 128, 1, 6.0, {0.63, 0, 0}},
    {W128, 128, 128, 2, 4.2, {0.87, 1.12, 0}},      {W256, 256, 256, 1, 4.5, {1.75, 0, 0}},
};

int64_t w8_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Up to 64 rows what counts is that all of the GPU reads W: the narrowest tile that
// needs no more than one workgroup a compute unit, the widest where all need more.  One
// row, N = 4096, K = 4096: 32 rows of W a workgroup 7 us, 64: 8.5, 128: 11.  One row, N =
// 28672, K = 8192: 128 rows 42 us, 64: 44, 32: 46.  Right past a tile's last size half of
// the compute units are idle: one row, K = 8192: N = 8192 takes 15 us (256 workgroups),
// 8224 22 (129), 10240 25 (160), 16384 28 (256), 16448 33 (129), 20480 35 (160).  K is split
// where that leaves compute units idle, into parts of 16 steps at least (but for tiles of
// 128 rows of W, and those of 64 up to 32 rows): N = 1024, K = 8192 in four parts 7.7 us,
// in one 11; N = 4096, K = 4096 in two 7.9, in one 6.9.  Past 64 rows the least of the costs above: B = 333, K =
// 11008, N = 4096 takes 128 x 128 in two parts, 33 us (128 x 64 in one: 35; 64 x 64: 39;
// 256 x 256: 108).
W8Plan w8_plan(int64_t B, int64_t K, int64_t N, int cus, bool scratch) {
    const int64_t steps = w8_ceil(K, kStep);
    const auto parts = [&](int64_t tiles, int64_t room) {
        const int64_t most = steps / 16, idle = room / tiles, s = most < idle ? most : idle;
        return (int)(scratch && s > 1 ? s : 1);
    };
    const int64_t t32 = w8_ceil(N, 32), t64 = w8_ceil(N, 64);
    if (B <= 32) {
        if (t64 > cus) return {R32x128, 1};
        if (t32 > cus) return {R32x64, 1};
        if (w8_ceil(B, 16) * t32 <= cus) return {R16x32, parts(w8_ceil(B, 16) * t32, cus - 1)};
        return {R32x32, 1};
    }
    if (B <= 64) {
        if (t64 > cus) return {R64x128, 1};
        if (8 * t32 > 5 * (int64_t)cus) return {R64x64, parts(t64, cus)};
        return {R32x32, parts(2 * t32, cus - 1)};
    }
    W8Plan best{W256, 1};
    double least = 1e30;
    for (const W8Cost& c : kCosts) {
        const int64_t tiles = w8_ceil(B, c.bm) * w8_ceil(N, c.bn);
        const bool stays = c.shape == W128 || c.shape == W256;
        if (!stays && tiles >= (int64_t)1 << 22) continue;          // (a grid holds fewer than 2^32 threads)
        for (int s = 1; s <= 8; s *= 2) {
            if (s > 1 && (stays || !scratch || steps / s < 16 || tiles * s > cus * c.fit)) break;
            const int64_t full = tiles * s / ((int64_t)cus * c.fit), left = tiles * s - full * cus * c.fit;
            const double each = (double)w8_ceil(steps, s);
            double cost = c.first + (double)full * (each * c.step[c.fit - 1] + 1.0);
            if (left > 0) cost += each * c.step[w8_ceil(left, cus) - 1];
            if (s > 1) cost += 1.5 + 8.0 * (double)B * (double)N * s / 4e6;   // partial sums, 4 TB/s
            if (cost < least) {
                least = cost;
                best = {c.shape, s};
            }
        }
    }
    return best;
}

template <int BM, int BN, int WM, int WN, int S, int KG = 1>
hipError_t run_ring(const W8Call& c, int splits, const Scratch& ws, hipStream_t stream) {
    const int64_t steps = w8_ceil(c.K, kStep);
    const int each = (int)(w8_ceil(w8_ceil(steps, splits), S) * S);
    splits = (int)w8_ceil(steps, each);
    const int64_t quads = w8_ceil(c.N, 4);
    ws.want(splits > 1 ? (size_t)(16 * quads * c.B * splits) : 0);
    if (ws.sizing()) return hipSuccess;
    const int64_t tiles = w8_ceil(c.N, BN) * w8_ceil(c.B, BM);
    w8_ring_kernel<BM, BN, WM, WN, S, KG><<<dim3((unsigned)(tiles * splits)), dim3(KG * (BM / WM) * (BN / WN) * 64), 0, stream>>>(
        c, static_cast<int*>(ws.ptr), splits, each);
    if (splits > 1)
        w8_join_kernel<<<dim3((unsigned)w8_ceil(quads * c.B, 256)), dim3(256), 0, stream>>>(c, static_cast<const int*>(ws.ptr),
                                                                                             splits);
    return hipGetLastError();
}

// Two groups of waves where there is about one workgroup a compute unit and each has
// 16 steps or more: 1 x 4096 x 4096 7.1 -> 6.4 us, 1 x 11008 x 4096 15.4 -> 12.9,
// 128 x 4096 x 4096 9.9 -> 9.1; with four steps (512 x 512) one group takes 3.9,
// two 4.3, and with more workgroups than compute units neither gains.
template <int BM, int BN, int WM, int WN, int S1, int S2>
hipError_t run_ring_groups(const W8Call& c, int splits, int num_cus, const Scratch& ws, hipStream_t stream) {
    const int64_t tiles = w8_ceil(c.N, BN) * w8_ceil(c.B, BM);
    if (4 * tiles * splits <= 5 * (int64_t)num_cus && w8_ceil(c.K, kStep) >= 16 * (int64_t)splits)
        return run_ring<BM, BN, WM, WN, S2, 2>(c, splits, ws, stream);
    return run_ring<BM, BN, WM, WN, S1>(c, splits, ws, stream);
}

template <int BM, int BN, int WM, int WN>
hipError_t run_wide(const W8Call& c, int num_cus, const Scratch& ws, hipStream_t stream) {
    if (ws.sizing()) return hipSuccess;
    const int tm = (int)w8_ceil(c.B, BM), tn = (int)w8_ceil(c.N, BN);
    constexpr int lds = (BM + BN) * (2 * kStep + 4), fit = 160 * 1024 / lds;   // workgroups a compute unit holds
    const int most = num_cus * (fit < 2 ? 1 : 2), blocks = tm * tn < most ? tm * tn : most;
    w8_wide_kernel<BM, BN, WM, WN><<<dim3((unsigned)blocks), dim3((BM / WM) * (BN / WN) * 64), 0, stream>>>(c, tm, tn);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w8(const W8Call& c, int num_cus, const Scratch& ws, hipStream_t stream) {
    const W8Plan p = w8_plan(c.B, c.K, c.N, num_cus, ws.sizing() || ws.ptr);
    switch (p.shape) {
        case R16x32: return run_ring_groups<16, 32, 16, 16, 8, 8>(c, p.splits, num_cus, ws, stream);
        case R32x32: return run_ring_groups<32, 32, 16, 16, 8, 4>(c, p.splits, num_cus, ws, stream);
        case R32x64: return run_ring<32, 64, 32, 16, 4>(c, p.splits, ws, stream);
        case R32x128: return run_ring<32, 128, 32, 16, 4>(c, p.splits, ws, stream);
        case R64x32: return run_ring_groups<64, 32, 32, 16, 4, 4>(c, p.splits, num_cus, ws, stream);
        case R64x64: return run_ring_groups<64, 64, 32, 32, 4, 4>(c, p.splits, num_cus, ws, stream);
        case R64x128: return run_ring<64, 128, 32, 32, 4>(c, p.splits, ws, stream);
        case R128x64: return run_ring<128, 64, 32, 32, 4>(c, p.splits, ws, stream);
        case R128x128: return run_ring<128, 128, 64, 32, 4>(c, p.splits, ws, stream);
        case W128: return run_wide<128, 128, 64, 64>(c, num_cus, ws, stream);
        default: return run_wide<256, 256, 64, 128>(c, num_cus, ws, stream);
    }
}

}  // namespace wq
