// Paged int4 KV cache (gfx950): append of new tokens, and copying, forking and
// compacting pages.
//
// Append quantizes whole blocks with the group-wise asymmetric codec ("What
// actually happens when you quantize a KV cache", §3-§4: s = (max - min) / 15,
// z = round(-min / s), c = clamp(round(x / s) + z)), K per channel and V per
// token (§7 "axis choice"), deciding every rounding as exact arithmetic would.
#include "wq_paged.h"

namespace wq {

using namespace paged;

namespace {

constexpr int kThreads = 256;

// ---- append ------------------------------------------------------------------

struct AppendArgs {
    PagedArgs c;
    const uint16_t* k;
    const uint16_t* v;
    int64_t tokens, k_stride, v_stride;
    const int32_t* lens;
    const int32_t* seqs;
    const int32_t* cu;
    int64_t count;
};

// Codes of eight fp16 values of groups with header h[i] (s, 1/s, z, tie
// threshold): the fp32 estimate round(x / s), or the exact decision where a
// lane of the wave is too near a tie.
__device__ __forceinline__ void encode8(const uint4& u, const float4 (&h)[8], uint32_t (&q)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[8], k[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = half_bits_to_float((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
        const float t = x[i] * h[i].y;
        k[i] = __builtin_rintf(t);
        near |= __builtin_fabsf(t - k[i]) > h[i].w;
    }
    if (__builtin_amdgcn_ballot_w64(near) != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = rne_div_exact(x[i], h[i].x, h[i].y, -h[i].z - 2.0f, 17.0f - h[i].z);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = (uint32_t)__builtin_amdgcn_fmed3f(k[i] + h[i].z, 0.0f, 15.0f);
}

__device__ __forceinline__ float4 header4(const GroupHeader& g) { return make_float4(g.s, g.rcp, g.Z, g.thr); }

__device__ __forceinline__ uint32_t pk_min(uint32_t a, uint32_t b) {
    return as_u32(__builtin_elementwise_min(as_h2(a), as_h2(b)));
}
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return as_u32(__builtin_elementwise_max(as_h2(a), as_h2(b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// One side of one block by the 256 threads: thread (c8, r) = (tid % 16, tid / 16)
// holds channels 8 c8 .. + 7 of eight tokens, 16 bytes each, so a load
// instruction of a wave reads whole 256-byte token rows.  Minima and maxima are
// taken on pairs of fp16 values, as they lie.
//
// K (a group is a channel): tokens r + 16 i.  The channel's minimum and maximum
// over the thread's tokens, then over r (lanes 16 and 32 apart, and the four
// waves through LDS); 128 threads make the headers; eight codes are four bytes
// of a token's code row, stored as they are.
__device__ __forceinline__ void quantize_k(uint8_t* rec, const uint4 (&u)[8], float4* hdr, uint32_t (*mnx)[2][kD / 2]) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int c8 = tid & 15, r = tid >> 4;
    uint32_t mn[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, mx[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            mn[e] = pk_min(mn[e], w[e]);
            mx[e] = pk_max(mx[e], w[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = 16; o < 64; o <<= 1) {
            mn[e] = pk_min(mn[e], (uint32_t)__shfl_xor((int)mn[e], o, 64));
            mx[e] = pk_max(mx[e], (uint32_t)__shfl_xor((int)mx[e], o, 64));
        }
    }
    if (lane < 16) {
        *reinterpret_cast<uint4*>(&mnx[wv][0][4 * c8]) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
        *reinterpret_cast<uint4*>(&mnx[wv][1][4 * c8]) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
    }
    __syncthreads();
    if (tid < kD) {
        uint32_t lo = mnx[0][0][tid >> 1], hi = mnx[0][1][tid >> 1];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            lo = pk_min(lo, mnx[w][0][tid >> 1]);
            hi = pk_max(hi, mnx[w][1][tid >> 1]);
        }
        const int at = 16 * (tid & 1);
        const GroupHeader g = make_header(half_bits_to_float((uint16_t)(lo >> at)), half_bits_to_float((uint16_t)(hi >> at)), 15);
        hdr[tid] = header4(g);
        reinterpret_cast<uint16_t*>(rec + kKScales)[tid] = g.sbits;
        reinterpret_cast<uint16_t*>(rec + kKZeros)[tid] = g.zbits;
    }
    __syncthreads();
    float4 h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = hdr[8 * c8 + e];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t q[8], w = 0;
        encode8(u[i], h, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= q[e] << (4 * e);
        *reinterpret_cast<uint32_t*>(rec + (r + 16 * i) * kRow + 4 * c8) = w;
    }
}

// V (a group is a token): tokens 8 r .. 8 r + 7.  The token's minimum and
// maximum over its 16 lanes; lanes 0..7 of the 16 make the eight headers; the
// eight codes of one channel are four bytes of that channel's code row, turned
// through an LDS tile so that rows are stored 16 bytes at a time.
__device__ __forceinline__ void quantize_v(uint8_t* rec, const uint4 (&u)[8], float4* hdr, uint32_t* tile) {
    const int tid = threadIdx.x;
    const int c8 = tid & 15, r = tid >> 4;
    uint32_t own = 0;                      // minimum and maximum of the lane's token (c8 < 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t mn = pk_min(pk_min(w[0], w[1]), pk_min(w[2], w[3]));
        uint32_t mx = pk_max(pk_max(w[0], w[1]), pk_max(w[2], w[3]));
        // The halves against each other, then the 16 lanes: (min, max) in one word.
        mn = pk_min(mn, __builtin_amdgcn_alignbit(mn, mn, 16));
        mx = pk_max(mx, __builtin_amdgcn_alignbit(mx, mx, 16));
        mn = pk_min(mn, dpp_u<0xB1>(mn));
        mx = pk_max(mx, dpp_u<0xB1>(mx));
        mn = pk_min(mn, dpp_u<0x4E>(mn));
        mx = pk_max(mx, dpp_u<0x4E>(mx));
        mn = pk_min(mn, dpp_u<0x141>(mn));
        mx = pk_max(mx, dpp_u<0x141>(mx));
        mn = pk_min(mn, dpp_u<0x140>(mn));
        mx = pk_max(mx, dpp_u<0x140>(mx));
        if (c8 == i) own = (mn & 0xFFFFu) | (mx << 16);
    }
    if (c8 < 8) {
        const GroupHeader g = make_header(half_bits_to_float((uint16_t)own), half_bits_to_float((uint16_t)(own >> 16)), 15);
        hdr[8 * r + c8] = header4(g);
        reinterpret_cast<uint16_t*>(rec + kVScales)[8 * r + c8] = g.sbits;
        reinterpret_cast<uint16_t*>(rec + kVZeros)[8 * r + c8] = g.zbits;
    }
    __syncthreads();
    uint32_t w[8] = {};                    // channel e of the thread: tokens 8 r + i in nibble i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 ht = hdr[8 * r + i];
        const float4 h[8] = {ht, ht, ht, ht, ht, ht, ht, ht};
        uint32_t q[8];
        encode8(u[i], h, q);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] |= q[e] << (4 * i);
    }
    // Row stride of 17 words: the 16 rows a store instruction meets fall on
    // different banks.
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[(8 * c8 + e) * 17 + r] = w[e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = tid + kThreads * i, d = at >> 2, q4 = (at & 3) * 4;
        const uint32_t* s = tile + d * 17 + q4;
        *reinterpret_cast<uint4*>(rec + kVCodes + d * kRow + 4 * q4) = make_uint4(s[0], s[1], s[2], s[3]);
    }
}

// Grid (tasks, heads, sides).  A task is one block of one entry; entry i has
// the tasks from cu[i] / 128 + 2 i on, which leaves room for every block it
// can touch (n tokens touch at most n / 128 + 2), so a task finds its entry by
// counting, without a running sum.  The task of an entry's first block also
// writes the window's new rows, after it has read the old ones; so no other
// workgroup writes what it reads.
__global__ __launch_bounds__(kThreads) void paged_append_kernel(const AppendArgs A) {
    __shared__ float4 hdr[kG];
    __shared__ __align__(16) uint32_t buf[kD * 17];
    __shared__ int found[4];
    static_assert(4 * 2 * (kD / 2) <= kD * 17, "minima and maxima fit in the tile");

    const int tid = threadIdx.x;
    const int64_t task = blockIdx.x, head = blockIdx.y;
    const int side = blockIdx.z;
    int64_t entry = task, cu0 = task, cu1 = task + 1, first_task = task;
    if (A.cu) {
        int before = 0;                    // entries whose tasks start at or before this one
        for (int64_t i = tid; i < A.count; i += kThreads) before += (int64_t)(A.cu[i] >> 7) + 2 * i <= task;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) before += __shfl_xor(before, o, 64);
        if ((tid & 63) == 0) found[tid >> 6] = before;
        __syncthreads();
        entry = found[0] + found[1] + found[2] + found[3] - 1;
        if (entry < 0) return;
        cu0 = A.cu[entry];
        cu1 = A.cu[entry + 1];
        first_task = (cu0 >> 7) + 2 * entry;
        if (task < first_task || cu0 < 0 || cu1 < cu0 || cu1 > A.tokens) return;
    }
    const int64_t n = cu1 - cu0, slot = slot_of(A.c, A.seqs, entry);
    if (n == 0 || slot < 0) return;
    const int64_t len = A.lens[slot];
    if (len < n || len > capacity(A.c)) return;
    const int64_t start = len - n;
    const int64_t block = start / kG + (task - first_task);
    if (block * kG >= len) return;
    const bool first = task == first_task, whole = (block + 1) * kG <= len;
    if (!whole && !first) return;          // the first block's task writes the rows of the last
    const uint16_t* in = side == 0 ? A.k : A.v;
    const int64_t stride = side == 0 ? A.k_stride : A.v_stride;
    uint16_t* win = window_of(A.c, slot, head, side);
    // What is needed from memory is asked for at once: the block's rows, its page
    // and the slots named before.
    uint4 u[8];
    int64_t page = -1;
    if (whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = tid >> 4;
            const int64_t p = block * kG + (side == 0 ? r + 16 * i : 8 * r + i);
            u[i] = *reinterpret_cast<const uint4*>((p < start ? win + p % kG * kD : in + (cu0 + p - start) * stride + head * kD) +
                                                   8 * (tid & 15));
        }
        page = A.c.table[slot * A.c.max_pages + block];
    }
    if (A.seqs) {                          // a slot named twice: its first entry counts
        int again = 0;
        for (int64_t i = tid; i < entry; i += kThreads) again |= A.seqs[i] == slot;
        if (__syncthreads_or(again)) return;
    }
    if (page >= 0 && page < A.c.num_pages) {
        uint8_t* rec = record(A.c, page, head);
        if (side == 0) quantize_k(rec, u, hdr, reinterpret_cast<uint32_t(*)[2][kD / 2]>(buf));
        else quantize_v(rec, u, hdr, buf);
    }
    if (!first || len % kG == 0) return;
    // Rows of the last, unfinished block.  No thread overwrites a row that
    // another has yet to read: a block quantized above has passed a barrier
    // after its rows were used, and one without a page needs none of them.
    const int64_t tail = len / kG * kG, from = start > tail ? start : tail;
    for (int64_t i = tid; i < (len - from) * 16; i += kThreads) {
        const int64_t p = from + (i >> 4);
        const int c = (int)(i & 15) * 8;
        *reinterpret_cast<uint4*>(win + (p - tail) * kD + c) =
            *reinterpret_cast<const uint4*>(in + (cu0 + p - start) * stride + head * kD + c);
    }
}

// ---- copy and fork -------------------------------------------------------------

struct Pairs {
    int2 p[kPairsPerLaunch];               // (source, destination)
};

constexpr int kVecsPerThread = 4;          // 16-byte vectors a thread moves

// Page bytes are contiguous over the heads: workgroup (x, y) moves 16 KB.
__global__ __launch_bounds__(kThreads) void paged_copy_kernel(const PagedArgs c, const Pairs pairs) {
    const int2 p = pairs.p[blockIdx.y];
    const int64_t vecs = c.heads * (kRecord / 16);
    const uint4* src = static_cast<const uint4*>(c.pages) + p.x * vecs;
    uint4* dst = static_cast<uint4*>(c.pages) + p.y * vecs;
    const int64_t at = (int64_t)blockIdx.x * (kThreads * kVecsPerThread) + threadIdx.x;
    uint4 u[kVecsPerThread];
#pragma unroll
    for (int i = 0; i < kVecsPerThread; ++i)
        if (at + i * kThreads < vecs) u[i] = src[at + i * kThreads];
#pragma unroll
    for (int i = 0; i < kVecsPerThread; ++i)
        if (at + i * kThreads < vecs) dst[at + i * kThreads] = u[i];
}

// Workgroup (2 head + side, pair): the live rows of one side of one head's
// window; the first also the table row and the length.
__global__ __launch_bounds__(kThreads) void paged_fork_kernel(const PagedArgs c, int32_t* table, int32_t* lens,
                                                              const Pairs pairs) {
    const int2 p = pairs.p[blockIdx.y];
    const int head = blockIdx.x >> 1, side = blockIdx.x & 1, tid = threadIdx.x;
    const int64_t len = clamped_len(c, lens, p.x);
    const uint4* src = reinterpret_cast<const uint4*>(window_of(c, p.x, head, side));
    uint4* dst = reinterpret_cast<uint4*>(window_of(c, p.y, head, side));
    const int vecs = (int)(len % kG) * (kD / 8);
    for (int i = tid; i < vecs; i += kThreads) dst[i] = src[i];
    if (blockIdx.x == 0) {
        for (int64_t b = tid; b < len / kG; b += kThreads)
            table[p.y * c.max_pages + b] = table[p.x * c.max_pages + b];
        if (tid == 0) lens[p.y] = (int32_t)len;
    }
}

// ---- compact -------------------------------------------------------------------
// Scratch: int32 moves, pad[3], hole[num_pages], mover[num_pages], rank[num_pages].
// hole[i] and mover[i] are the i-th free id below `used` and the i-th page in
// use from `used` on, both ascending (there are equally many); rank[page] is a
// mover's i.

constexpr int kPlanThreads = 1024;
constexpr int kRangeWords = 8192;          // pages a bit each, 262144 at a time
constexpr int kRangePages = kRangeWords * 32;

// Marks the pages of [lo, lo + 262144) that the table names as whole blocks: a
// wave takes a slot at a time.
__device__ __forceinline__ void mark_range(const PagedArgs& c, const int32_t* lens, int64_t lo, uint32_t* bits) {
    for (int i = threadIdx.x; i < kRangeWords; i += kPlanThreads) bits[i] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 63;
    for (int64_t s = threadIdx.x >> 6; s < c.slots; s += kPlanThreads / 64) {
        const int64_t blocks = clamped_len(c, lens, s) / kG;
        for (int64_t b = lane; b < blocks; b += 64) {
            const int64_t p = c.table[s * c.max_pages + b];
            if (p >= lo && p < lo + kRangePages && p < c.num_pages)
                atomicOr(bits + ((p - lo) >> 5), 1u << ((p - lo) & 31));
        }
    }
    __syncthreads();
}

// Sum of v over the threads before this one, and over all of them.
__device__ __forceinline__ int64_t scan_before(int64_t v, int64_t* wave_sum, int64_t& total) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int64_t inc = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t up = __shfl_up(inc, o, 64);
        if (lane >= o) inc += up;
    }
    __syncthreads();
    if (lane == 63) wave_sum[wv] = inc;
    __syncthreads();
    int64_t before = inc - v;
    total = 0;
    for (int w = 0; w < kPlanThreads / 64; ++w) {
        if (w < wv) before += wave_sum[w];
        total += wave_sum[w];
    }
    return before;
}

// One workgroup: the pages in use as bits in LDS (ids past 262144 in further
// ranges), their count, then the ranks of free and moving ids by a running sum.
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(const PagedArgs c, const int32_t* lens,
                                                                    int32_t* used, int32_t* ws) {
    __shared__ uint32_t bits[kRangeWords];
    __shared__ int64_t wave_sum[kPlanThreads / 64];
    constexpr int per = kRangeWords / kPlanThreads;   // consecutive words of a thread
    const int tid = threadIdx.x;
    int32_t* hole = ws + 4;
    int32_t* mover = hole + c.num_pages;
    int32_t* rank = mover + c.num_pages;

    int64_t live = 0;
    for (int64_t lo = 0; lo < c.num_pages; lo += kRangePages) {
        mark_range(c, lens, lo, bits);
        int64_t mine = 0, total;
        for (int i = 0; i < per; ++i) mine += __builtin_popcount(bits[tid * per + i]);
        scan_before(mine, wave_sum, total);
        live += total;
        __syncthreads();
    }
    int64_t holes = 0, movers = 0;
    for (int64_t lo = 0; lo < c.num_pages; lo += kRangePages) {
        if (c.num_pages > kRangePages) mark_range(c, lens, lo, bits);
        // Free ids below `live` and used ids from it on, among this thread's words.
        const int64_t at = lo + (int64_t)tid * per * 32;
        int64_t h = 0, m = 0;
        for (int i = 0; i < per; ++i) {
            const uint32_t w = bits[tid * per + i];
            const int64_t base = at + 32 * i, below = live - base;
            const uint32_t low = below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
            h += __builtin_popcount(~w & low);
            m += __builtin_popcount(w & ~low);
        }
        int64_t ht, mt;
        int64_t hb = holes + scan_before(h, wave_sum, ht), mb = movers + scan_before(m, wave_sum, mt);
        for (int i = 0; i < per; ++i) {
            const uint32_t w = bits[tid * per + i];
            const int64_t base = at + 32 * i, below = live - base;
            const uint32_t low = below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
            for (uint32_t x = ~w & low; x; x &= x - 1) hole[hb++] = (int32_t)(base + __builtin_ctz(x));
            for (uint32_t x = w & ~low; x; x &= x - 1) {
                const int64_t p = base + __builtin_ctz(x);
                rank[p] = (int32_t)mb;
                mover[mb++] = (int32_t)p;
            }
        }
        holes += ht;
        movers += mt;
        __syncthreads();
    }
    if (tid == 0) {
        ws[0] = (int32_t)movers;
        *used = (int32_t)live;
    }
}

// Moves the pages of the plan, 16 KB a step, and writes the new table.
__global__ __launch_bounds__(kThreads) void compact_move_kernel(const PagedArgs c, const int32_t* lens,
                                                                int32_t* table_out, const int32_t* used,
                                                                const int32_t* ws) {
    const int32_t* hole = ws + 4;
    const int32_t* mover = hole + c.num_pages;
    const int32_t* rank = mover + c.num_pages;
    const int64_t vecs = c.heads * (kRecord / 16);
    constexpr int kStep = kThreads * kVecsPerThread;
    const int64_t steps = (vecs + kStep - 1) / kStep, all = ws[0] * steps;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int64_t m = i / steps, at = (i - m * steps) * kStep + threadIdx.x;
        const uint4* src = static_cast<const uint4*>(c.pages) + mover[m] * vecs;
        uint4* dst = static_cast<uint4*>(c.pages) + hole[m] * vecs;
        uint4 u[kVecsPerThread];
#pragma unroll
        for (int k = 0; k < kVecsPerThread; ++k)
            if (at + k * kThreads < vecs) u[k] = src[at + k * kThreads];
#pragma unroll
        for (int k = 0; k < kVecsPerThread; ++k)
            if (at + k * kThreads < vecs) dst[at + k * kThreads] = u[k];
    }
    const int32_t live = *used;
    const int64_t entries = c.slots * c.max_pages;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < entries; i += (int64_t)gridDim.x * kThreads) {
        const int64_t s = i / c.max_pages, b = i - s * c.max_pages;
        int32_t to = -1;
        if (b < clamped_len(c, lens, s) / kG) {
            const int32_t p = c.table[i];
            if (p >= 0 && p < c.num_pages) to = p < live ? p : hole[rank[p]];
        }
        table_out[i] = to;
    }
}

}  // namespace

hipError_t launch_paged_append(const void* k, const void* v, int64_t tokens, int64_t k_stride, int64_t v_stride,
                               const PagedArgs& c, const int32_t* lens, const int32_t* seqs, const int32_t* cu,
                               int64_t count, hipStream_t stream) {
    const AppendArgs A{c, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), tokens, k_stride,
                       v_stride, lens, seqs, cu, count};
    const int64_t tasks = cu ? tokens / kG + 2 * count : count;
    paged_append_kernel<<<dim3((unsigned)tasks, (unsigned)c.heads, 2), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

hipError_t launch_paged_copy(const PagedArgs& c, const int32_t* pairs, int64_t count, hipStream_t stream) {
    const int64_t vecs = c.heads * (kRecord / 16), step = kThreads * kVecsPerThread;
    for (int64_t at = 0; at < count; at += kPairsPerLaunch) {
        Pairs p;
        const int64_t n = count - at < kPairsPerLaunch ? count - at : kPairsPerLaunch;
        for (int64_t i = 0; i < n; ++i) p.p[i] = make_int2(pairs[2 * (at + i)], pairs[2 * (at + i) + 1]);
        paged_copy_kernel<<<dim3((unsigned)((vecs + step - 1) / step), (unsigned)n), dim3(kThreads), 0, stream>>>(c, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_paged_fork(const PagedArgs& c, int32_t* lens, const int32_t* pairs, int64_t count,
                             hipStream_t stream) {
    for (int64_t at = 0; at < count; at += kPairsPerLaunch) {
        Pairs p;
        const int64_t n = count - at < kPairsPerLaunch ? count - at : kPairsPerLaunch;
        for (int64_t i = 0; i < n; ++i) p.p[i] = make_int2(pairs[2 * (at + i)], pairs[2 * (at + i) + 1]);
        paged_fork_kernel<<<dim3((unsigned)(2 * c.heads), (unsigned)n), dim3(kThreads), 0, stream>>>(
            c, const_cast<int32_t*>(c.table), lens, p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

size_t paged_compact_bytes(const PagedArgs& c) { return (size_t)(4 + 3 * c.num_pages) * sizeof(int32_t); }

hipError_t launch_paged_compact(const PagedArgs& c, const int32_t* lens, int32_t* table_out, int32_t* used,
                                void* scratch, int num_cus, hipStream_t stream) {
    int32_t* ws = static_cast<int32_t*>(scratch);
    compact_plan_kernel<<<dim3(1), dim3(kPlanThreads), 0, stream>>>(c, lens, used, ws);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    compact_move_kernel<<<dim3((unsigned)(8 * num_cus)), dim3(kThreads), 0, stream>>>(c, lens, table_out, used, ws);
    return hipGetLastError();
}

}  // namespace wq
