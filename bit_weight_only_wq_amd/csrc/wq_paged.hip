// Paged int4 KV cache (gfx950): append of new tokens, and copying, forking and
// compacting pages.
//
// Append quantizes whole blocks with the group-wise asymmetric codec ("What
// actually happens when you quantize a KV cache", §3-§4: s = (max - min) / 15,
// z = round(-min / s), c = clamp(round(x / s) + z)), K per channel and V per
// token (§7 "axis choice"), deciding every rounding as exact arithmetic would.
//
// What bounds it: a call with many blocks, vector instructions and waiting (64
// prompts of 4096 tokens with 8 heads, 1.36 GB: 414 us, 3.3 TB/s; by counters 61 % of
// the SIMDs' cycles are vector instructions, 18 a value, of which the encoding is
// six; codes leave in 32-byte pieces, half a row each, though no byte twice; 16
// prompts, 31 MB: 14 us); a decode step, the chain
// of dependent reads of lens, window and table (64 sequences, one of which
// completes a block, 8 heads: 6.5 us, 3.2 where none does).  Whole blocks are
// therefore quantized in quarters of 256 threads, which start within the time
// that the single tokens take.
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

// What encoding needs of a group: 1 / s, kRound + Z, s and s / 2.  Adding kRound
// = 1.5 * 2^23 to a number of small magnitude rounds it to the nearest integer,
// ties to even, and leaves that in the low bits.
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ float4 header4(const GroupHeader& g) { return make_float4(g.rcp, kRound + g.Z, g.s, 0.5f * g.s); }

// Eight 4-bit codes, of consecutive fp16 values in u whose groups' headers are
// h(e), as the nibbles 0 .. 7 of a word.  Six instructions a value:
// y = x / s + Z + kRound by one fma from fp16 x, which is k + Z + kRound with k
// the nearest integer to x / s but for the reciprocal's error; r = x - k s, which
// is exact, and |r| < s / 2 says that k is right; the clamp to 0 .. 15; and a
// shift-and-add that leaves the constant part of each y in the word (kRound's
// bits, 0x4B400000 at nibble e: their sum is taken off at the end, modulo 2^32).
// Where a lane of the wave has |r| >= s / 2 (ties mostly: x = s / 2 is one value
// in some thousands), k moves towards r unless it is a tie and k is even.
template <class Head>
__device__ __forceinline__ uint32_t encode8(const uint4& u, const Head& h) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float y[8], r[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float4 he = h(e);
        const float x = (float)as_h2(w[e >> 1])[e & 1];
        y[e] = __builtin_fmaf(x, he.x, he.y);
        r[e] = __builtin_fmaf(he.y - y[e], he.z, x);
        near |= __builtin_fabsf(r[e]) >= he.w;
    }
    if (__builtin_amdgcn_ballot_w64(near) != 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 he = h(e);
            const float k = y[e] - he.y, a = __builtin_fabsf(r[e]);
            const bool odd = __builtin_bit_cast(uint32_t, k + kRound) & 1u;
            if (a > he.w || (a == he.w && odd)) y[e] += __builtin_copysignf(1.0f, r[e]);
        }
    }
    uint32_t q = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e)
        q = (q << 4) + __builtin_bit_cast(uint32_t, __builtin_amdgcn_fmed3f(y[e], kRound, kRound + 15.0f));
    // 0x4B400000 * (1 + 16 + 16^2 + ..), modulo 2^32.
    return q - 0x4B400000u * 0x11111111u;
}

// (As instructions: the compiler would first quiet NaNs, which do not occur.)
__device__ __forceinline__ uint32_t pk_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("v_pk_min_f16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("v_pk_max_f16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// A quarter of one block of one head by 256 threads: part 0 and 1 are channels 0
// .. 63 and 64 .. 127 of K, part 2 and 3 tokens 0 .. 63 and 64 .. 127 of V.  A
// thread holds 16-byte pieces (eight channels) of four tokens.  Minima and
// maxima are taken on pairs of fp16 values, as they lie.
//
// K (a group is a channel): thread (c8, r) = (tid % 8, tid / 8) has tokens r +
// 32 i.  The channel's minimum and maximum over the thread's tokens, then over r
// (lanes 8, 16 and 32 apart, and the four waves through LDS); 64 threads make
// the headers; eight codes are four bytes of a token's code row.
// V (a group is a token): thread (c8, r) = (tid % 16, tid / 16) has tokens 4 r ..
// 4 r + 3.  The token's minimum and maximum over its 16 lanes, of which four
// make the headers; the four codes of one channel are two bytes of that
// channel's code row, turned through an LDS tile so that rows are stored 16
// bytes at a time.
constexpr int kRows = 4;                   // tokens of a thread
constexpr int kHalf = 64;                  // channels (K) or tokens (V) of a part
constexpr int kTileRow = 9;                // words of a tile row: 32 bytes of codes, and one to spread the banks

// Barrier for what the workgroup shares in LDS: it does not wait for loads and
// stores of memory, as __syncthreads does.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct PartLds {
    float4 hdr[kHalf];
    uint32_t mnx[kThreads / 64][2][kHalf / 2];
    uint32_t tile[kD * kTileRow];
};

// Token (of the block) and byte (of its 256) of the thread's piece i.
__device__ __forceinline__ int part_token(int part, int i) {
    const int tid = threadIdx.x;
    return part < 2 ? (tid >> 3) + 32 * i : kHalf * (part & 1) + kRows * (tid >> 4) + i;
}
__device__ __forceinline__ int part_channel(int part) {
    const int tid = threadIdx.x;
    return part < 2 ? kHalf * part + 8 * (tid & 7) : 8 * (tid & 15);
}

__device__ __forceinline__ void quantize_part(uint8_t* rec, int part, const uint4 (&u)[kRows], PartLds& s) {
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, half = part & 1;
    if (part < 2) {
        const int c8 = tid & 7, r = tid >> 3;
        uint32_t mn[4] = {u[0].x, u[0].y, u[0].z, u[0].w}, mx[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 1; i < kRows; ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mn[e] = pk_min(mn[e], w[e]);
                mx[e] = pk_max(mx[e], w[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            mn[e] = pk_min(mn[e], dpp_u<0x128>(mn[e]));       // row_ror 8
            mx[e] = pk_max(mx[e], dpp_u<0x128>(mx[e]));
#pragma unroll
            for (int o = 16; o < 64; o <<= 1) {
                mn[e] = pk_min(mn[e], (uint32_t)__shfl_xor((int)mn[e], o, 64));
                mx[e] = pk_max(mx[e], (uint32_t)__shfl_xor((int)mx[e], o, 64));
            }
        }
        if (lane < 8) {
            *reinterpret_cast<uint4*>(&s.mnx[wv][0][4 * c8]) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
            *reinterpret_cast<uint4*>(&s.mnx[wv][1][4 * c8]) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
        }
        lds_barrier();
        GroupHeader g;
        if (tid < kHalf) {
            uint32_t lo = s.mnx[0][0][tid >> 1], hi = s.mnx[0][1][tid >> 1];
#pragma unroll
            for (int w = 1; w < kThreads / 64; ++w) {
                lo = pk_min(lo, s.mnx[w][0][tid >> 1]);
                hi = pk_max(hi, s.mnx[w][1][tid >> 1]);
            }
            const int at = 16 * (tid & 1);
            g = make_header(half_bits_to_float((uint16_t)(lo >> at)), half_bits_to_float((uint16_t)(hi >> at)), 15);
            s.hdr[tid] = header4(g);
        }
        lds_barrier();
        float4 h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = s.hdr[8 * c8 + e];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            *reinterpret_cast<uint32_t*>(rec + (r + 32 * i) * kRow + half * (kRow / 2) + 4 * c8) =
                encode8(u[i], [&](int e) { return h[e]; });
        if (tid < kHalf) {
            reinterpret_cast<uint16_t*>(rec + kKScales)[kHalf * half + tid] = g.sbits;
            reinterpret_cast<uint16_t*>(rec + kKZeros)[kHalf * half + tid] = g.zbits;
        }
        return;
    }
    const int c8 = tid & 15, r = tid >> 4;
    uint32_t own = 0;                      // minimum and maximum of the lane's token (c8 < 4)
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        uint32_t mn = pk_min(pk_min(u[i].x, u[i].y), pk_min(u[i].z, u[i].w));
        uint32_t mx = pk_max(pk_max(u[i].x, u[i].y), pk_max(u[i].z, u[i].w));
        mn = pk_min(mn, __builtin_amdgcn_alignbit(mn, mn, 16));   // the halves against each other, then the lanes
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
    GroupHeader g;
    if (c8 < kRows) {
        g = make_header(half_bits_to_float((uint16_t)own), half_bits_to_float((uint16_t)(own >> 16)), 15);
        s.hdr[kRows * r + c8] = header4(g);
    }
    lds_barrier();
    uint32_t q[kRows];                     // token 4 r + i: the thread's eight channels in the nibbles
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const float4 h = s.hdr[kRows * r + i];
        q[i] = encode8(u[i], [&](int) { return h; });
    }
    uint16_t* to = reinterpret_cast<uint16_t*>(s.tile);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t w = 0;                    // channel e: tokens 4 r + i in nibble i
#pragma unroll
        for (int i = 0; i < kRows; ++i) w |= ((q[i] >> (4 * e)) & 15u) << (4 * i);
        to[(8 * c8 + e) * (2 * kTileRow) + r] = (uint16_t)w;
    }
    lds_barrier();
    const int d = tid >> 1, q4 = (tid & 1) * 4;
    const uint32_t* w = s.tile + d * kTileRow + q4;
    *reinterpret_cast<uint4*>(rec + kVCodes + d * kRow + half * (kRow / 2) + 4 * q4) = make_uint4(w[0], w[1], w[2], w[3]);
    if (c8 < kRows) {
        reinterpret_cast<uint16_t*>(rec + kVScales)[kHalf * half + kRows * r + c8] = g.sbits;
        reinterpret_cast<uint16_t*>(rec + kVZeros)[kHalf * half + kRows * r + c8] = g.zbits;
    }
}

// Grid (tasks, heads, parts).  A task is one block of one entry; entry i has the
// tasks from cu[i] / 128 + 2 i on, which leaves room for every block it can
// touch (n tokens touch at most n / 128 + 2), so a task finds its entry by
// counting, without a running sum.  The task of an entry's first block also
// writes the window's new rows (each part the channels or, of V, the rows it
// reads of an old window: part p of a side its 64 channels), after it has read
// the old ones; so no other workgroup writes what it reads.
__global__ __launch_bounds__(kThreads) void paged_append_kernel(const AppendArgs A) {
    __shared__ __align__(16) PartLds s;
    __shared__ int found[4];
    read_arguments(A);

    const int tid = threadIdx.x;
    const int64_t task = blockIdx.x;
    const int part = blockIdx.z, side = part >> 1;
    const int head = blockIdx.y;
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
    const int old = start > block * kG ? (int)(start - block * kG) : 0;        // rows of the block that the window holds
    const uint16_t* block_in = in + (cu0 + block * kG - start) * stride;       // its row 0's place among the new ones
    uint16_t* win = window_of(A.c, slot, head, side);
    // What is needed from memory is asked for at once: the block's rows, its page
    // and the slots named before.
    uint4 u[kRows];
    int64_t page = -1;
    if (whole) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int t = part_token(part, i);
            u[i] = *reinterpret_cast<const uint4*>((t < old ? win + t * kD : block_in + t * stride + head * kD) +
                                                   part_channel(part));
        }
        page = A.c.table[slot * A.c.max_pages + block];
    }
    if (A.seqs) {                          // a slot named twice: its first entry counts
        int again = 0;
        for (int64_t i = tid; i < entry; i += kThreads) again |= A.seqs[i] == slot;
        if (__syncthreads_or(again)) return;
    }
    if (page >= 0 && page < A.c.num_pages) quantize_part(record(A.c, page, head), part, u, s);
    if (!first || len % kG == 0) return;
    // The new rows of the last, unfinished block: a part writes what it alone
    // reads of an old window (K: its channels, V: its rows), which it has read:
    // a block quantized above has passed a barrier after its rows were used, and
    // one without a page needs none of them.
    const int64_t tail = len / kG * kG, from = start > tail ? start : tail;
    const int lo = part < 2 ? 0 : kHalf * (part & 1), hi = part < 2 ? kG : lo + kHalf;
    const int r0 = (int)(from - tail) > lo ? (int)(from - tail) : lo, r1 = (int)(len - tail) < hi ? (int)(len - tail) : hi;
    const int pieces = part < 2 ? 8 : 16, c0 = part < 2 ? kHalf * part : 0;
    const uint16_t* tail_in = in + (cu0 + tail - start) * stride;
    for (int i = tid; i < (r1 - r0) * pieces; i += kThreads) {
        const int r = r0 + i / pieces, c = c0 + i % pieces * 8;
        *reinterpret_cast<uint4*>(win + r * kD + c) = *reinterpret_cast<const uint4*>(tail_in + r * stride + head * kD + c);
    }
}

// One token per entry, up to kMaxOnes entries: a few workgroups share out what
// there is to do, since in most steps few entries fill a block, and the time of
// a call is the time to start workgroups and to find those out.  Every workgroup
// reads all slots and lengths; the parts of the blocks to quantize go round the
// workgroups, and the rows to copy round the waves.
constexpr int kMaxOnes = 1024;
constexpr int kCopyHeads = 8;              // heads of a copying task

__global__ __launch_bounds__(kThreads) void paged_append_ones_kernel(const AppendArgs A) {
    __shared__ __align__(16) PartLds s;
    __shared__ int slots[kMaxOnes], lens[kMaxOnes];   // of good entries; slot -1 otherwise
    read_arguments(A);
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, count = (int)A.count;
    for (int i = tid; i < (count + 63) / 64 * 64; i += kThreads) {
        const int64_t slot = i < count ? slot_of(A.c, A.seqs, i) : -1;
        const int64_t len = slot >= 0 ? A.lens[slot] : 0;
        slots[i] = (int)slot;
        lens[i] = len >= 1 && len <= capacity(A.c) ? (int)len : 0;
    }
    __syncthreads();
    // A slot named twice: its first entry counts (whole wave; uniform).
    const auto repeated = [&](int entry) {
        const int slot = slots[entry];
        bool again = false;
        for (int i = lane; i < entry; i += 64) again |= slots[i] == slot;
        return A.seqs && __builtin_amdgcn_ballot_w64(again) != 0;
    };

    // Blocks that become whole: quantizing tasks (which, head, part) in order.
    const int per_block = (int)A.c.heads * 4;
    int seen = 0;                          // whole blocks in the entries before
    int64_t task = blockIdx.x;
    for (int base = 0; base < count; base += 64) {
        uint64_t whole = __builtin_amdgcn_ballot_w64(lens[base + lane] > 0 && lens[base + lane] % kG == 0);
        const int here = __builtin_popcountll(whole);
        for (; task < (int64_t)(seen + here) * per_block; task += gridDim.x) {
            int k = (int)(task / per_block) - seen;
            const int hp = (int)(task % per_block), head = hp >> 2, part = hp & 3, side = part >> 1;
            uint64_t m = whole;
            for (; k > 0; --k) m &= m - 1;
            const int entry = base + __builtin_ctzll(m);
            const int64_t slot = slots[entry], block = lens[entry] / kG - 1;
            const uint16_t* win = window_of(A.c, slot, head, side);
            const uint16_t* fresh = side == 0 ? A.k + entry * A.k_stride + head * kD : A.v + entry * A.v_stride + head * kD;
            uint4 u[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int t = part_token(part, i);
                u[i] = *reinterpret_cast<const uint4*>((t < kG - 1 ? win + t * kD : fresh) + part_channel(part));
            }
            const int64_t page = A.c.table[slot * A.c.max_pages + block];
            if (repeated(entry) || page < 0 || page >= A.c.num_pages) continue;
            quantize_part(record(A.c, page, head), part, u, s);
            lds_barrier();                 // the next task's use of s
        }
        seen += here;
    }

    // Rows that go to a window: tasks (entry, eight heads).
    const int groups = ((int)A.c.heads + kCopyHeads - 1) / kCopyHeads;
    const int waves = gridDim.x * (kThreads / 64);
    for (int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + wv; t < (int64_t)count * groups; t += waves) {
        const int entry = (int)(t / groups), h0 = (int)(t % groups) * kCopyHeads;
        const int len = lens[entry];
        if (len == 0 || len % kG == 0 || repeated(entry)) continue;
        const int nh = (int)A.c.heads - h0 < kCopyHeads ? (int)A.c.heads - h0 : kCopyHeads;
        const int64_t slot = slots[entry];
#pragma unroll
        for (int i = 0; i < kCopyHeads * 2 * 16 / 64; ++i) {
            const int at = lane + 64 * i, c = at % 16 * 8, side = at / 16 % 2, h = at / 32;
            if (h < nh)
                *reinterpret_cast<uint4*>(window_of(A.c, slot, h0 + h, side) + (len % kG - 1) * kD + c) =
                    *reinterpret_cast<const uint4*>((side == 0 ? A.k + entry * A.k_stride : A.v + entry * A.v_stride) +
                                                    (h0 + h) * kD + c);
        }
    }
}

// ---- copy and fork -------------------------------------------------------------

struct Pairs {
    int2 p[kPairsPerLaunch];               // (source, destination)
};

// Page bytes are contiguous over the heads: thread by thread one 16-byte vector,
// loaded past the caches and stored through them.  400 pages of 139264 bytes take
// 20.6 us (median; 19.0 the least), 5.4 TB/s.  (When this was chosen: 18.2, against
// 26.3 with both sides cached and 20.2 with four vectors a thread.)
__global__ __launch_bounds__(kThreads) void paged_copy_kernel(const PagedArgs c, const Pairs pairs) {
    const int2 p = pairs.p[blockIdx.y];
    const int64_t vecs = c.heads * (kRecord / 16), at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= vecs) return;
    static_cast<uint4*>(c.pages)[p.y * vecs + at] = load_stream(static_cast<const uint4*>(c.pages) + p.x * vecs + at);
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
constexpr int kRangeWords = 4096;          // pages a bit each, 131072 at a time
constexpr int kRangePages = kRangeWords * 32;
constexpr int kPlanSlots = 1024;           // slots whose lengths are looked up at a time

struct PlanLds {
    uint32_t bits[kRangeWords];            // page in use
    int hole[kRangeWords], mover[kRangeWords];   // free ids below `live`, and used ids from it on, before each word
    int blocks[kPlanSlots];
    int2 wave_sum[kPlanThreads / 64];
};

// Marks the pages of [lo, lo + kRangePages) that the table names as whole blocks.
__device__ __forceinline__ void mark_range(const PagedArgs& c, const int32_t* lens, int64_t lo, PlanLds& s) {
    for (int i = threadIdx.x; i < kRangeWords; i += kPlanThreads) s.bits[i] = 0;
    for (int64_t s0 = 0; s0 < c.slots; s0 += kPlanSlots) {
        const int n = c.slots - s0 < kPlanSlots ? (int)(c.slots - s0) : kPlanSlots;
        __syncthreads();
        if ((int)threadIdx.x < n) s.blocks[threadIdx.x] = (int)(clamped_len(c, lens, s0 + threadIdx.x) / kG);
        __syncthreads();
        // Four entries of a thread at a time, so that their loads overlap.
        const int64_t entries = n * c.max_pages;
        for (int64_t e0 = threadIdx.x; e0 < entries; e0 += 4 * kPlanThreads) {
            int64_t p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t e = e0 + k * kPlanThreads, sl = e < entries ? e / c.max_pages : 0;
                p[k] = e < entries && e - sl * c.max_pages < s.blocks[sl] ? c.table[s0 * c.max_pages + e] : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (p[k] >= lo && p[k] < lo + kRangePages && p[k] < c.num_pages)
                    atomicOr(s.bits + ((p[k] - lo) >> 5), 1u << ((p[k] - lo) & 31));
        }
    }
    __syncthreads();
}

// Sums of v over the threads before this one, and over all of them.
__device__ __forceinline__ int2 scan_before(int2 v, int2* wave_sum, int2& total) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int2 inc = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(inc.x, o, 64), y = __shfl_up(inc.y, o, 64);
        if (lane >= o) inc = make_int2(inc.x + x, inc.y + y);
    }
    __syncthreads();
    if (lane == 63) wave_sum[wv] = inc;
    __syncthreads();
    int2 w = lane < kPlanThreads / 64 ? wave_sum[lane] : make_int2(0, 0), upto = w;
#pragma unroll
    for (int o = 1; o < kPlanThreads / 64; o <<= 1) {
        const int x = __shfl_up(upto.x, o, 64), y = __shfl_up(upto.y, o, 64);
        if (lane >= o) upto = make_int2(upto.x + x, upto.y + y);
    }
    constexpr int last = kPlanThreads / 64 - 1;
    total = make_int2(__shfl(upto.x, last, 64), __shfl(upto.y, last, 64));
    return make_int2(inc.x - v.x + __shfl(upto.x - w.x, wv, 64), inc.y - v.y + __shfl(upto.y - w.y, wv, 64));
}

// The ids of word i below `live`.
__device__ __forceinline__ uint32_t low_mask(int64_t first, int64_t live) {
    const int64_t below = live - first;
    return below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
}

// A pool of 4096 pages, half of them in use by 96 slots: 9.4 us, and 44 to 46 for
// the pages moved after it (227 MB read and written, 5.0 TB/s, a copy's rate).
// One workgroup: the pages in use as bits in LDS (ids past 131072 in further
// ranges), their count, the running counts of free and moving ids word by word,
// and from those every page's place.
__global__ __launch_bounds__(kPlanThreads) void compact_plan_kernel(const PagedArgs c, const int32_t* lens,
                                                                    int32_t* used, int32_t* ws) {
    __shared__ PlanLds s;
    constexpr int per = kRangeWords / kPlanThreads;   // consecutive words of a thread
    const int tid = threadIdx.x;
    int32_t* hole = ws + 4;
    int32_t* mover = hole + c.num_pages;
    int32_t* rank = mover + c.num_pages;

    int64_t live = 0;
    for (int64_t lo = 0; lo < c.num_pages; lo += kRangePages) {
        mark_range(c, lens, lo, s);
        int2 mine = make_int2(0, 0), total;
#pragma unroll
        for (int i = 0; i < per; ++i) mine.x += __builtin_popcount(s.bits[tid * per + i]);
        scan_before(mine, s.wave_sum, total);
        live += total.x;
        __syncthreads();
    }
    int64_t holes = 0, movers = 0;
    for (int64_t lo = 0; lo < c.num_pages; lo += kRangePages) {
        if (c.num_pages > kRangePages) mark_range(c, lens, lo, s);
        int2 mine = make_int2(0, 0), total;
        int2 at[per];
#pragma unroll
        for (int i = 0; i < per; ++i) {
            const int word = tid * per + i;
            const uint32_t w = s.bits[word], low = low_mask(lo + 32 * (int64_t)word, live);
            at[i] = mine;
            mine.x += __builtin_popcount(~w & low);
            mine.y += __builtin_popcount(w & ~low);
        }
        const int2 before = scan_before(mine, s.wave_sum, total);
#pragma unroll
        for (int i = 0; i < per; ++i) {
            s.hole[tid * per + i] = before.x + at[i].x;
            s.mover[tid * per + i] = before.y + at[i].y;
        }
        __syncthreads();
        const int n = c.num_pages - lo < kRangePages ? (int)(c.num_pages - lo) : kRangePages;
        for (int i = tid; i < n; i += kPlanThreads) {
            const int word = i >> 5;
            const uint32_t w = s.bits[word], low = low_mask(lo + 32 * (int64_t)word, live), bit = 1u << (i & 31);
            if (~w & low & bit) hole[holes + s.hole[word] + __builtin_popcount(~w & low & (bit - 1))] = (int32_t)(lo + i);
            if (w & ~low & bit) {
                const int64_t r = movers + s.mover[word] + __builtin_popcount(w & ~low & (bit - 1));
                mover[r] = (int32_t)(lo + i);
                rank[lo + i] = (int32_t)r;
            }
        }
        holes += total.x;
        movers += total.y;
        __syncthreads();
    }
    if (tid == 0) {
        ws[0] = (int32_t)movers;
        *used = (int32_t)live;
    }
}

// Moves the pages of the plan, two vectors a thread at a time, and writes the new
// table.
constexpr int kMoveVecs = 2;

__global__ __launch_bounds__(kThreads) void compact_move_kernel(const PagedArgs c, const int32_t* lens,
                                                                int32_t* table_out, const int32_t* used,
                                                                const int32_t* ws) {
    const int32_t* hole = ws + 4;
    const int32_t* mover = hole + c.num_pages;
    const int32_t* rank = mover + c.num_pages;
    const int64_t vecs = c.heads * (kRecord / 16);
    constexpr int kStep = kThreads * kMoveVecs;
    const int64_t steps = (vecs + kStep - 1) / kStep, all = ws[0] * steps;
    for (int64_t i = blockIdx.x; i < all; i += gridDim.x) {
        const int64_t m = i / steps, at = (i - m * steps) * kStep + threadIdx.x;
        const uint4* src = static_cast<const uint4*>(c.pages) + mover[m] * vecs;
        uint4* dst = static_cast<uint4*>(c.pages) + hole[m] * vecs;
        uint4 u[kMoveVecs];
#pragma unroll
        for (int k = 0; k < kMoveVecs; ++k)
            if (at + k * kThreads < vecs) u[k] = load_stream(src + at + k * kThreads);
#pragma unroll
        for (int k = 0; k < kMoveVecs; ++k)
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
                               int64_t count, int num_cus, hipStream_t stream) {
    const AppendArgs A{c, static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), tokens, k_stride,
                       v_stride, lens, seqs, cu, count};
    if (!cu && count <= kMaxOnes) {
        // As many workgroups as there can be tasks, up to two per compute unit.
        const int64_t wgs = 4 * c.heads * count, most = 2 * (int64_t)num_cus;
        paged_append_ones_kernel<<<dim3((unsigned)(wgs < most ? wgs : most)), dim3(kThreads), 0, stream>>>(A);
        return hipGetLastError();
    }
    const int64_t tasks = cu ? tokens / kG + 2 * count : count;
    paged_append_kernel<<<dim3((unsigned)tasks, (unsigned)c.heads, 4), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

hipError_t launch_paged_copy(const PagedArgs& c, const int32_t* pairs, int64_t count, hipStream_t stream) {
    const int64_t vecs = c.heads * (kRecord / 16), step = kThreads;
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
    compact_move_kernel<<<dim3((unsigned)(16 * num_cus)), dim3(kThreads), 0, stream>>>(c, lens, table_out, used, ws);
    return hipGetLastError();
}

}  // namespace wq
