// Decode attention over a paged int4 KV cache (gfx950): one new token per
// sequence, out = softmax(scale K q) V over the sequence's pages and window
// ("What actually happens when you quantize a KV cache", §2 the decode step,
// §3-§4 the codec, §7 "axis choice").
//
// What bounds it: HBM for groups of up to 4 query heads; from there on start and
// join, and the vector instructions of the softmax and of the factors' halves.  A
// token of a KV head is 136 bytes and is read once for up to 16 query heads of its
// group (larger groups are several rows, and each reads it), so both products run
// on the matrix cores, with those heads as the 16 columns of
// v_mfma_f32_16x16x32_f16.
//
// Work is cut into units of about 17 KB: one page record (128 tokens of one KV
// head), or 32 tokens of a window.  The units of all entries stand in one line
// (entry, KV head and chunk of up to 16 query heads, unit); the workgroups of
// the grid (one per compute unit) each take an equal run of it, whatever the
// lengths are, and their eight waves equal parts of that: every wave forms the
// running sum of the units itself from lens.  A wave keeps a running maximum,
// sum and output per head.  Where its part covers a whole row (entry, head,
// chunk) it writes the result; else the waves' fp32 sums are joined in LDS, in
// order, and where a row goes past the workgroup, the workgroups' sums by a
// second kernel.  No atomics: a result depends on the batch, not on timing.
//
// One unit of a page, per wave, with lane = 16 g + m:
//   scores   A = a_d = q_d s_d of 16 slots, B = codes of 16 tokens x 32 channels
//            (a lane's 16 bytes are channels 32 g .. 32 g + 31 of one token,
//            four k-steps).  The result's rows 4 g + i are slots, its columns m
//            tokens, so a lane holds its eight tokens' scores for up to four
//            slots, and the softmax costs no more than the heads there are.
//   values   A = codes of 16 channels x 32 tokens (a lane's 16 bytes are tokens
//            32 g .. of one channel), B = w_t = p_t s_t of 16 slots, turned
//            through LDS.
// a and w are fp16 pairs hi + lo (22 bits: hi is the rounded product, lo the
// rounded rest), so their rounding stays far below that of the fp16 result.
// Up to 8 heads a row, hi and lo are neighbouring slots, and every product is
// issued once; past 8 all slots are heads, and it is issued for hi and for lo.
// Slot 4 g + i is head g + 4 u, u = i / 2 or i: the kernel is built for NH = 1,
// 2 or 4 heads a lane (rows of up to 4, 8 and 16).
//
// A code needs no conversion: its bits alone, in the low byte of an fp16, are a
// subnormal number, and the matrix cores take those exactly.  Scores: c 2^-24
// at even positions and 16 c 2^-24 at odd ones (a shift and four ANDs for a
// word of eight codes), with q's odd channels 16 times smaller.  Values:
// 16 c 2^-24 everywhere (two more shifts): the hardware adds products of c
// 2^-24 to a sum with less of their lower bits (measured over 64 products of
// positive numbers: 4e-6 off, all one way, against 2.4e-7 for 16 c 2^-24 and
// for normal numbers), which a long sum of positive weights does not bear.  A score
// is a sum of 128 and softmax takes differences of scores: equal scores, in
// blocks with and without zero points and in the window, came out less than 1e-6 of
// the sum of their terms' magnitudes apart.
// The zero points enter as sum a_d z_d (a product with the zeros as B, once per
// unit) and sum w_t z_t (in fp32, per lane): any fp16 value, as a scale may be.
//
// Ranges: q is scaled by a power of two per head so that its largest channel is
// 2^6 .. 2^7, and a block's key scales so that the largest is 2^7 .. 2^8 (as far as
// a factor of 2^15 takes it), hence |a| < 2^15; both powers are taken out of the
// score.  fp16 ends at 2^-24, so a channel's a keeps its 22 bits down to 2^-15 of
// the product of those two (2^-11 in the odd channels), and what a smaller one
// loses is below 2^-38 (2^-34) of it.  (Without the scales' power, keys of 2^-10
// left relative errors of 2e-3 in the output, and of 2e-2 where they lie ten
// deviations off zero.)  w is kept below 2^14 by the reference R of the running
// exponent, R = max over tokens of (score + exponent of its scale - 14): what is
// rounded is the weight times the scale, and the largest of those products stays
// near 2^13, whatever the scales beside it (2^13 / 2^x where that scale is 2^-x of
// 1/4).  One below it by 2^-15 keeps its 22 bits, and a smaller one is off by 2^-38
// of the largest.
//
// Measured, kernel and join together: 32 sequences of 4096 tokens with 32 heads
// of their own (571 MB) 101 us, 5.7 TB/s; one of 131149 tokens with 64 query
// heads on 8 (143 MB) 40 us, 3.6 TB/s; 64 of lengths from 0 to 16384 with the
// same heads (142 MB) 46 us; one of 500 tokens with 32 heads 10.8 us, which is a
// launch and one workgroup's chain of dependent reads.  32 sequences of 8192
// tokens and 8 KV heads (287 to 294 MB) with groups of 12 heads 72 us, 16 74, 24
// 126 (two rows), 64 239 (four rows).
#include "wq_paged.h"

namespace wq {

using namespace paged;

namespace {

typedef unsigned short us2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxRow = 16;               // query heads of a row (columns of a product)
constexpr int kQuarter = 32;              // window tokens of a unit
constexpr int kVHalf = kD / 2;            // channels of a window unit's V in LDS at a time
constexpr int kVRow = kVHalf + 8;         // fp16 elements of such a row
constexpr int kPart = kD + 4;             // floats of one head's partial sums in LDS: 128 O, R, L, zeros
constexpr int kMaxCount = 65536;          // entries of a call (the C entry point takes fewer)
constexpr int kJoin = 256;                // threads of the joining kernel
constexpr int kBufWord3 = 0x00020000;     // raw, unswizzled gfx9 buffer

struct AttnArgs {
    PagedArgs c;
    const uint16_t* q;
    uint16_t* out;
    const int32_t* lens;
    const int32_t* seqs;
    int64_t q_stride, out_stride, window;
    int count;
    int group;                            // query heads per KV head
    int chunks, per_chunk;                // rows per KV head, query heads of each (the last may have fewer)
    int groups;                           // workgroups that share the line; 0: one workgroup per row
    float scale;                          // times log2(e)
    int4* cross;                          // [groups] the row that begins in a run and goes past it: row (or -1),
                                          // end of its units, which partial; [groups].w is the number of units
    float2* part_ml;                      // [groups][2][per_chunk] R and sum
    float* part_o;                        // [groups][2][per_chunk][128]
};

// What of a sequence is read: blocks b0 .. nb - 1 and window quarters w0 ..
// w1 - 1; `left` is the first position that counts.
struct Span {
    int len, left, b0, nb, w0, w1;
    __device__ __forceinline__ int units() const { return nb - b0 + w1 - w0; }
};

__device__ __forceinline__ Span span_of(int len, int64_t window) {
    Span s;
    s.len = len;
    s.left = window > 0 && window < len ? len - (int)window : 0;
    s.nb = len / kG;
    s.b0 = s.left / kG < s.nb ? s.left / kG : s.nb;
    const int tail = s.nb * kG;
    s.w0 = s.left > tail ? (s.left - tail) / kQuarter : 0;
    s.w1 = (len - tail + kQuarter - 1) / kQuarter;
    return s;
}

// v, taken anew: what is computed from it is not kept in registers from
// elsewhere (the loop over units needs nearly all of them).
__device__ __forceinline__ int anew(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// a b, rounded: what follows does not take the product into an fma.
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ uint32_t pk_mul(uint32_t a, uint32_t b) { return as_u32(as_h2(a) * as_h2(b)); }
__device__ __forceinline__ uint32_t pk_rest(uint32_t a, uint32_t b, uint32_t hi) {
    return as_u32(__builtin_elementwise_fma(as_h2(a), as_h2(b), -as_h2(hi)));
}

// Eight consecutive halves (0 1)(2 3)(4 5)(6 7) in the order the codes of a
// word unpack to: (0 4)(1 5)(2 6)(3 7).
__device__ __forceinline__ uint4 code_order(const uint4& d) {
    return make_uint4(__builtin_amdgcn_perm(d.z, d.x, 0x05040100u), __builtin_amdgcn_perm(d.z, d.x, 0x07060302u),
                      __builtin_amdgcn_perm(d.w, d.y, 0x05040100u), __builtin_amdgcn_perm(d.w, d.y, 0x07060302u));
}

__device__ __forceinline__ h8_t as_h8(const uint4& u) { return __builtin_bit_cast(h8_t, u); }

// The eight 4-bit codes of a word, in code order, as fp16.
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
// c 2^-24 at even positions, 16 c 2^-24 at odd ones.
__device__ __forceinline__ h8_t unpack_k(uint32_t w) {
    const uint32_t s = w >> 8;
    return as_h8(make_uint4(w & kLow, w & kHigh, s & kLow, s & kHigh));
}
// 16 c 2^-24.
__device__ __forceinline__ h8_t unpack_v(uint32_t w) {
    return as_h8(make_uint4((w << 4) & kHigh, w & kHigh, (w >> 4) & kHigh, (w >> 8) & kHigh));
}
// Exponents of a head's largest |q| and of a block's largest key scale, as
// multiplied: their products stay below 2^15, and kQTop + 24 is the most that two
// fp16 factors reach.
constexpr int kQTop = 6, kSTop = 7;
constexpr float kVUnit = 0x1p20f;         // what scales the values' sums back (the scores' 2^24 is in k_unit)
constexpr float kZUnit = 0x1p-20f;        // of the zeros' sum, in the scores' sums
// fp16 pairs: 1, 1 / 16 and 16, 1 / 16 beside 1, and 1024 (which an exponent field
// is taken to) + 28.
constexpr uint32_t kOnes = 0x3C003C00u, kSixteenth = 0x2C002C00u, kSixteen = 0x4C004C00u, kEvenSixteenth = 0x3C002C00u;
constexpr uint32_t kHalf1052 = 0x641C641Cu;

__device__ __forceinline__ f4_t mfma(const h8_t& a, const h8_t& b, const f4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t half_pair(float a, float b) {
    return as_u32(h2_t{(_Float16)a, (_Float16)b});
}

// Largest value over the four lanes of an m.
__device__ __forceinline__ float column_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16, 64));
    return __builtin_fmaxf(v, __shfl_xor(v, 32, 64));
}
// Largest value over the 16 lanes of a g.
__device__ __forceinline__ float row_max(float v) {
    v = __builtin_fmaxf(v, dpp_f<0xB1>(v));
    v = __builtin_fmaxf(v, dpp_f<0x4E>(v));
    v = __builtin_fmaxf(v, dpp_f<0x141>(v));
    return __builtin_fmaxf(v, dpp_f<0x140>(v));
}

// n units shared by k takers: the first n % k take one more.
struct Share {
    int q, r;
    __device__ __forceinline__ Share(int n, int k) : q(n / k), r(n - n / k * k) {}
    __device__ __forceinline__ int begin(int i) const { return i * q + (i < r ? i : r); }
    __device__ __forceinline__ int of(int f) const {     // whose unit f is (q > 0 or f < r)
        const int at = r * (q + 1);
        return f < at ? f / (q + 1) : r + (f - at) / q;
    }
};

// 64 entries' slots and lengths, one per lane.
struct Chunk {
    int base, slot, len;
    __device__ __forceinline__ void load(const AttnArgs& A, int at, int lane) {
        base = at;
        slot = -1;
        len = 0;
        if (at + lane < A.count) {
            slot = (int)slot_of(A.c, A.seqs, at + lane);
            if (slot >= 0) len = (int)clamped_len(A.c, A.lens, slot);
        }
    }
};

// A place in the line of units.
struct Cursor {
    int entry, row, unit;                 // row of the entry, unit of the row
    int head, first;                      // the row's KV head and first query head of its group
    int slot, units;
    Span s;
    int64_t page;                         // of this unit, if it is a block
    __device__ __forceinline__ bool block() const { return unit < s.nb - s.b0; }
};

// Bytes of a wave in LDS: a record's headers, the row's queries (64 a lane), and
// the weights on their way from the scores' lanes to the values' (a window
// unit's share of them beside 64 channels of its V).
constexpr int kPRow = kG + 8;             // fp16 elements of a slot's weights
constexpr int kPWindow = kQuarter + 8;
constexpr int kTurn = 16 * kPWindow * 2 + kQuarter * kVRow * 2;
constexpr int kWaveLds = 1024 + 4096 + kTurn;
static_assert(kTurn >= 16 * kPRow * 2, "a block's weights fit");
static_assert(kWaveLds >= kMaxRow * kPart * 4, "a wave's last partial sums fit in its place");

template <int NH>
__global__ __launch_bounds__(kThreads, 2) void paged_attn_kernel(const AttnArgs A) {
    constexpr bool kSplit = NH <= 2;      // hi and lo in slots of their own
    // [kWaves][kWaveLds], then [kWaves][per_chunk][kPart] first partial sums.
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ int chunk_units[kMaxCount / 64];
    __shared__ int seg_row[2 * kWaves], seg_begin[2 * kWaves], seg_end[2 * kWaves];   // (2 wave + 0 first, 1 last)
    read_arguments(A);
    const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, m = lane & 15;
    const int rows = (int)A.c.heads * A.chunks;                          // of an entry
    uint16_t* head_lds = reinterpret_cast<uint16_t*>(lds + wv * kWaveLds);
    const auto q_lds = [&](int j) { return reinterpret_cast<uint4*>(lds + wv * kWaveLds + 1024) + anew(lane) + 64 * j; };
    uint16_t* p_lds = head_lds + (1024 + 4096) / 2;
    uint16_t* v_lds = p_lds + 16 * kPWindow;
    const bool m_lo = kSplit && (m & 1);  // slot m holds lo halves
    if (lane < 2) seg_row[2 * wv + lane] = -1;

    // ---- this wave's run [f0, f1) of the line, and where it begins.
    Chunk ch;
    Cursor cu;
    int f0, f1;
    cu.unit = 0;
    int run0 = 0, run1 = 0;               // the workgroup's run
    if (A.groups == 0) {                  // one workgroup per row
        cu.entry = (int)blockIdx.x / rows;
        cu.row = (int)blockIdx.x - cu.entry * rows;
        ch.load(A, cu.entry & ~63, lane);
        run1 = span_of(__builtin_amdgcn_readlane(ch.len, cu.entry & 63), A.window).units();
        if (run1 == 0) {                  // nothing to see: zeros
            const int h = cu.row / A.chunks, first = (cu.row - h * A.chunks) * A.per_chunk;
            const int n = A.group - first < A.per_chunk ? A.group - first : A.per_chunk;
            uint32_t* o = reinterpret_cast<uint32_t*>(A.out + cu.entry * A.out_stride + (int64_t)(h * A.group + first) * kD);
            for (int i = threadIdx.x; i < n * (kD / 2); i += kThreads) o[i] = 0;
            return;
        }
        f0 = cu.unit = run1 * wv / kWaves;
        f1 = run1 * (wv + 1) / kWaves;
    } else {
        int total = 0, u = 0, inc = 0;
        const auto scan = [&](int at) {   // units of 64 entries, and their running sum
            ch.load(A, at, lane);
            u = inc = span_of(ch.len, A.window).units() * rows;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(inc, o, 64);
                if (lane >= o) inc += up;
            }
        };
        // More than 64 entries: the waves share them, and each takes the sums of
        // 64 from LDS.
        const int chunks = (A.count + 63) / 64;
        if (chunks == 1) {
            scan(0);
            total = __builtin_amdgcn_readlane(inc, 63);
        } else {
            for (int c = wv; c < chunks; c += kWaves) {
                scan(64 * c);
                if (lane == 63) chunk_units[c] = inc;
            }
            __syncthreads();
            for (int c = lane; c < chunks; c += 64) total += chunk_units[c];
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o, 64);
            total = uniform(total);
        }
        const int used = A.groups < total ? A.groups : total;
        if (blockIdx.x == 0 && threadIdx.x == 0) A.cross[A.groups] = make_int4(0, 0, 0, total);
        if ((int)blockIdx.x >= used) {
            if (threadIdx.x == 0) A.cross[blockIdx.x] = make_int4(-1, 0, 0, 0);
            return;
        }
        const Share share(total, used);
        run0 = share.begin(blockIdx.x);
        run1 = share.begin(blockIdx.x + 1);
        const int n = run1 - run0;
        f0 = run0 + (int)((int64_t)n * wv / kWaves);
        f1 = run0 + (int)((int64_t)n * (wv + 1) / kWaves);
        const int find = f0 < f1 ? f0 : run0;            // (a wave without units looks at any)
        int before = 0, at = 0;
        if (chunks > 1) {
            for (int c0 = 0;; c0 += 64) {                // ends: find < total
                int sum = c0 + lane < chunks ? chunk_units[c0 + lane] : 0, upto = sum;
#pragma unroll
                for (int o = 1; o < 64; o <<= 1) {
                    const int up = __shfl_up(upto, o, 64);
                    if (lane >= o) upto += up;
                }
                const uint64_t past = __builtin_amdgcn_ballot_w64(before + upto > find);
                if (past != 0) {
                    const int i = __builtin_ctzll(past);
                    before += __builtin_amdgcn_readlane(upto - sum, i);
                    at = 64 * (c0 + i);
                    break;
                }
                before += __builtin_amdgcn_readlane(upto, 63);
            }
            scan(at);
        }
        const int i = __builtin_ctzll(__builtin_amdgcn_ballot_w64(before + inc > find));
        before += __builtin_amdgcn_readlane(inc - u, i);
        cu.entry = at + i;
        cu.unit = find - before;          // in the entry, for now
    }
    cu.entry = uniform(cu.entry);
    cu.slot = __builtin_amdgcn_readlane(ch.slot, cu.entry & 63);
    cu.s = span_of(__builtin_amdgcn_readlane(ch.len, cu.entry & 63), A.window);
    cu.units = cu.s.units();
    if (A.groups != 0) {
        cu.row = cu.unit / cu.units;
        cu.unit -= cu.row * cu.units;
    }
    cu.head = cu.row / A.chunks;
    cu.first = (cu.row - cu.head * A.chunks) * A.per_chunk;

    const auto fetch_page = [&](Cursor& c) {
        c.page = c.block() ? (int64_t)A.c.table[c.slot * A.c.max_pages + c.s.b0 + c.unit] : 0;
    };
    const auto advance = [&](Cursor& c) {   // to the next unit of the line (there is one)
        if (++c.unit < c.units) return;
        c.unit = 0;
        c.first += A.per_chunk;
        if (c.first >= A.group) {
            c.first = 0;
            ++c.head;
        }
        if (++c.row < rows) return;
        c.row = 0;
        c.head = 0;
        do {
            if ((++c.entry & 63) == 0) ch.load(A, c.entry, lane);
            c.slot = __builtin_amdgcn_readlane(ch.slot, c.entry & 63);
            c.s = span_of(__builtin_amdgcn_readlane(ch.len, c.entry & 63), A.window);
            c.units = c.s.units();
        } while (c.units == 0);
    };

    // ---- loads of a block's record: through a buffer of its bytes, or of none
    // where there is no such block, so that the loads are always issued.
    const uint32_t k_off = (uint32_t)((8 * m) * kRow + 16 * g);                     // + 64 per token of the lane's eight
    const uint32_t v_off = (uint32_t)(kVCodes + m * kRow + 16 * g);                 // + 1024 per 16 channels
    const uint32_t h_off = (uint32_t)(kKScales + 16 * lane);
    const auto buffer = [&](const Cursor& c, bool valid) {
        const int64_t page = c.page >= 0 && c.page < A.c.num_pages ? c.page : 0;
        const uint8_t* rec = record(A.c, page, c.head);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(rec), (short)0, valid && c.block() ? kRecord : 0,
                                                 kBufWord3);
    };
    const auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2));   // 2: streamed
    };
    // (Offsets taken anew, so that the constants stay in the instructions.)
    const auto load_k = [&](__amdgpu_buffer_rsrc_t r, uint4 (&K)[8], uint4& H) {
        const uint32_t ko = (uint32_t)anew((int)k_off);
#pragma unroll
        for (int i = 0; i < 8; ++i) K[i] = load16(r, ko + kRow * (i / 2 + 4 * (i & 1)));
        H = load16(r, (uint32_t)anew((int)h_off));
    };
    const auto load_v = [&](__amdgpu_buffer_rsrc_t r, uint4 (&V)[8]) {
        const uint32_t vo = (uint32_t)anew((int)v_off);
#pragma unroll
        for (int i = 0; i < 8; ++i) V[i] = load16(r, vo + 1024 * i);
    };

    const float zero = __builtin_bit_cast(float, vgpr_const(0));

    // A row's queries as they lie, 4 NH heads of 256 bytes: 16-byte piece lane +
    // 64 k of them.
    const auto load_q = [&](const Cursor& c, uint4 (&piece)[NH]) {
        const int n = A.group - c.first < A.per_chunk ? A.group - c.first : A.per_chunk;
        const int lq = anew(lane);
        const uint4* src = reinterpret_cast<const uint4*>(A.q + c.entry * A.q_stride + (int64_t)(c.head * A.group + c.first) * kD);
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            piece[k] = make_uint4(0, 0, 0, 0);
            if ((lq >> 4) + 4 * k < n) piece[k] = src[lq + 64 * k];
        }
    };

    uint4 K[8], V[8], H, piece0[NH];
    load_q(cu, piece0);
    fetch_page(cu);
    {
        const auto r = buffer(cu, f0 < f1);
        load_k(r, K, H);
        load_v(r, V);
    }
    Cursor nx = cu;
    if (f1 - f0 > 1) {
        advance(nx);
        fetch_page(nx);
    }

    // ---- the row's state.
    // Of the lane's heads g + 4 u, alike in the lanes of a g (L and cz: in
    // their sum): score units (log2, >= 0), reference, sum of weights, zeros.
    float cn[NH], R[NH], L[NH], cz[NH];
    f4_t O[8] = {};                       // / 2^20 while the row is in its blocks
    bool bad = false, in_blocks = false;
    int heads_here = 0;                   // query heads of the row

    const auto turned = [&]() {               // the wave's LDS writes before its reads that follow
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    // A new row, from its queries: turned through LDS to the slots' lanes, |q| <
    // 2^(kQTop + 1) by a power of two that cn undoes.
    const auto start_row = [&](const Cursor& c, const uint4 (&piece)[NH]) {
        bad = false;
        in_blocks = true;
        heads_here = A.group - c.first < A.per_chunk ? A.group - c.first : A.per_chunk;
#pragma unroll
        for (int u = 0; u < NH; ++u) {
            R[u] = -__builtin_huge_valf();
            L[u] = cz[u] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) O[i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
        uint4* q_raw = reinterpret_cast<uint4*>(p_lds);
#pragma unroll
        for (int k = 0; k < NH; ++k) q_raw[anew(lane) + 64 * k] = piece[k];
        turned();
        const int mq = anew(m), hq = (mq >> 2) + 4 * (kSplit ? (mq & 3) >> 1 : mq & 3);
        const bool none = NH == 1 && (mq & 3) >= 2;
        uint4 raw[4];
        us2_t top2 = us2_t{0, 0};             // (magnitudes order as their bits do)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            raw[j] = none ? make_uint4(0, 0, 0, 0) : q_raw[16 * (none ? 0 : hq) + 4 * anew(g) + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top2 = __builtin_elementwise_max(top2, __builtin_bit_cast(us2_t, word(raw[j], i) & 0x7FFF7FFFu));
        }
        turned();                             // (read before the weights come to the same place)
        const float top = column_max(half_bits_to_float(top2.x > top2.y ? top2.x : top2.y));
        const int e = (top > 0.0f ? __builtin_amdgcn_frexp_expf(top) - 1 : 0) - kQTop;   // top * 2^-e in 2^kQTop * [1, 2)
        // (Within 2^-90 .. 2^80: no product with an infinity is 0 * inf.)
        const float unit = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(__builtin_fabsf(A.scale), e), 0x1p-90f, 0x1p80f);
#pragma unroll
        for (int u = 0; u < NH; ++u) cn[u] = __shfl(unit, 4 * anew(g) + (kSplit ? 2 * u : u), 64);   // from the head's slot
        // 2^-e in two factors that fp16 holds, the second with scale's sign.
        const int e1 = -e / 2, e2 = -e - e1;
        const _Float16 f1_ = (_Float16)__builtin_amdgcn_ldexpf(1.0f, e1);
        const _Float16 f2_ = (_Float16)__builtin_amdgcn_ldexpf(A.scale < 0.0f ? -1.0f : 1.0f, e2);
        const uint32_t f1 = as_u32(h2_t{f1_, f1_}), f2 = as_u32(h2_t{f2_, f2_}), f2s = pk_mul(f2, kSixteenth);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // To LDS (16 registers), in code order, the odd channels / 16.
            const uint4 c4 = code_order(raw[j]);
            *q_lds(j) = make_uint4(pk_mul(pk_mul(c4.x, f1), f2), pk_mul(pk_mul(c4.y, f1), f2s),
                                       pk_mul(pk_mul(c4.z, f1), f2), pk_mul(pk_mul(c4.w, f1), f2s));
        }
    };
    start_row(cu, piece0);

    // What the lanes of head g + 4 u hold, for the lanes of a slot m of it.
    const auto to_slot = [&](const float (&v)[NH]) {
        const int mt = anew(m), from = 16 * (mt >> 2), u_of = kSplit ? (mt & 3) >> 1 : mt & 3;
        float r = __shfl(v[0], from, 64);
#pragma unroll
        for (int u = 1; u < NH; ++u) {
            const float w = __shfl(v[u], from, 64);
            r = u_of == u ? w : r;
        }
        return r;
    };
    // The head (of the row) that this lane writes sums of, or -1.
    const auto my_head = [&]() {
        const int mt = anew(m), h = (mt >> 2) + 4 * (kSplit ? (mt & 3) >> 1 : mt & 3);
        return h < heads_here && !(kSplit && (mt & 1)) && (NH > 1 || (mt & 3) < 2) ? h : -1;
    };
    // A slot's two halves together (in both slots).
    const auto both = [&](float v) { return kSplit ? v + dpp_f<0xB1>(v) : v; };
    const auto total_l = [&](int u) { return bad ? __builtin_nanf("") : group_sum<16>(L[u]); };
    const auto keep = [&](float* part) {      // partial sums to LDS
        const float k = in_blocks ? kVUnit : 1.0f;
        const int h = my_head(), gp = anew(g);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const f4_t o = {both(O[t][0]) * k, both(O[t][1]) * k, both(O[t][2]) * k, both(O[t][3]) * k};
            if (h >= 0) *reinterpret_cast<f4_t*>(part + h * kPart + 16 * t + 4 * gp) = o;
        }
#pragma unroll
        for (int u = 0; u < NH; ++u) {
            const f4_t s = {R[u], total_l(u), group_sum<16>(cz[u]), 0.0f};
            if (anew(m) == 0 && gp + 4 * u < heads_here) *reinterpret_cast<f4_t*>(part + (gp + 4 * u) * kPart + kD) = s;
        }
    };
    const auto note_segment = [&](int at, int f) {
        if (lane == 0) {
            seg_row[at] = cu.entry * rows + cu.row;
            seg_begin[at] = f - cu.unit;
            seg_end[at] = f - cu.unit + cu.units;
        }
    };
    bool open = false;                    // a row left unfinished (or finished, but begun before) at the end

    for (int f = f0; f < f1; ++f) {
        const bool more = f + 1 < f1;
        // The next row's queries, ahead of the next unit's codes (past 8 heads
        // there are no registers for them: they are loaded where it starts).
        uint4 piece[NH];
        if (kSplit && more && nx.unit == 0) load_q(nx, piece);
        const auto nbuf = buffer(nx, more);

        // New reference for the running exponent, and what is held with the old one.
        // Past 2^24 a score and its reference are rounded by more than they are
        // apart (at most 15, see x2).  So the reference goes up by two steps of fp32,
        // but not by 16: then, at any size, no weight leaves fp16 at the top, and the
        // largest does not vanish.  (A step of 16: -15 .. 0 is rounded to -16 or 0, and
        // 16 is added; of 32 and more: both are rounded away.)
        const auto rebase = [&](const float (&cand)[NH]) {
            float alpha[NH];
            bool grows = false;
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                const float c = row_max(cand[u]);
                const float r = __builtin_fmaxf(R[u], c + __builtin_fminf(__builtin_fabsf(c) * 0x1p-23f, 15.9f));
                grows |= r > R[u];
                alpha[u] = R[u] - r;
                R[u] = r;
            }
            if (__builtin_amdgcn_ballot_w64(grows) != 0) {
#pragma unroll
                for (int u = 0; u < NH; ++u) {
                    alpha[u] = exp2_hw(alpha[u]);
                    L[u] *= alpha[u];
                    cz[u] *= alpha[u];
                }
                const float a = to_slot(alpha);
#pragma unroll
                for (int i = 0; i < 8; ++i) O[i] *= a;
            }
        };
        // Weights hi + lo of head u into their slots' rows.
        const auto halves = [](float w0, float w1, uint32_t& hi, uint32_t& lo) {
            const h2_t h = h2_t{(_Float16)w0, (_Float16)w1};
            hi = as_u32(h);
            lo = as_u32(h2_t{(_Float16)(w0 - (float)h.x), (_Float16)(w1 - (float)h.y)});
        };
        if (cu.block()) {
            bad |= cu.page < 0 || cu.page >= A.c.num_pages;
            // Headers to LDS: 16 bytes a lane in, the lane's 64 bytes of each out.
            // K's scales (lanes 0 .. 15) go there times the power of two 2^up that
            // brings the largest to 2^kSTop, as far as fp16 holds it; K's zeros (lanes
            // 16 .. 31) those of the even channels / 16, as the queries of the odd ones.
            us2_t s2 = us2_t{0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s2 = __builtin_elementwise_max(s2, __builtin_bit_cast(us2_t, word(H, i) & 0x7FFF7FFFu));
            const float s_top = row_max(half_bits_to_float(s2.x > s2.y ? s2.x : s2.y));
            const int s_exp = (uniform(__builtin_bit_cast(int, s_top)) >> 23) - 127;
            const int up = kSTop - s_exp < -14 ? -14 : (kSTop - s_exp > 15 ? 15 : kSTop - s_exp);   // (scales are below 2^16)
            {
                const int hl = anew(lane);
                const uint32_t f = hl < 16 ? (uint32_t)(up + 15) * 0x04000400u : (hl < 32 ? kEvenSixteenth : kOnes);
                *reinterpret_cast<uint4*>(head_lds + 8 * hl) =
                    make_uint4(pk_mul(H.x, f), pk_mul(H.y, f), pk_mul(H.z, f), pk_mul(H.w, f));
            }
            const float k_unit = __builtin_bit_cast(float, (127 + 24 - up) << 23);   // 2^24 / 2^up
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const uint4* hd = reinterpret_cast<const uint4*>(head_lds) + 4 * g;   // + 16 per header array
            uint4 a0[4], a1[4];               // hi or lo (a0); hi and lo past 8 heads
            f4_t z4 = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 s = code_order(hd[j]), z = code_order(hd[16 + j]), qj = *q_lds(j);
                a0[j] = make_uint4(pk_mul(qj.x, s.x), pk_mul(qj.y, s.y), pk_mul(qj.z, s.z), pk_mul(qj.w, s.w));
                a1[j] = make_uint4(pk_rest(qj.x, s.x, a0[j].x), pk_rest(qj.y, s.y, a0[j].y),
                                   pk_rest(qj.z, s.z, a0[j].z), pk_rest(qj.w, s.w, a0[j].w));
                if (kSplit)
                    a0[j] = make_uint4(m_lo ? a1[j].x : a0[j].x, m_lo ? a1[j].y : a0[j].y, m_lo ? a1[j].z : a0[j].z,
                                       m_lo ? a1[j].w : a0[j].w);
                z4 = mfma(as_h8(a0[j]), as_h8(z), z4);
                if (!kSplit) z4 = mfma(as_h8(a1[j]), as_h8(z), z4);
            }
            z4 *= -kZUnit;
            f4_t S[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) S[r] = z4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const h8_t b = unpack_k(word(K[r], j));
                    S[r] = mfma(as_h8(a0[j]), b, S[r]);
                    if (!kSplit) S[r] = mfma(as_h8(a1[j]), b, S[r]);
                }
            load_k(nbuf, K, H);

            // Scores of the lane's tokens 8 m + place(r) for its heads, times cc in log2.
            float sc[NH][8], cc[NH];
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                cc[u] = cn[u] * k_unit;
#pragma unroll
                for (int r = 0; r < 8; ++r) sc[u][r] = kSplit ? S[r][(2 * u) & 3] + S[r][(2 * u + 1) & 3] : S[r][u];
            }
            // Tokens left of the window do not count, whatever they hold.
            const int skip = cu.s.left - (cu.s.b0 + cu.unit) * kG;
            if (skip > 0) {
                const int ms = anew(m), two = 2 * anew(lane);
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int u = 0; u < NH; ++u)
                        if (8 * ms + r / 2 + 4 * (r & 1) < skip) sc[u][r] = -__builtin_huge_valf();
                uint32_t* v = reinterpret_cast<uint32_t*>(head_lds) + 128 + two / 2;   // this lane's two tokens
                const uint32_t kept = two < skip ? (two + 1 < skip ? 0u : 0xFFFF0000u) : ~0u;
                v[0] &= kept;
                v[64] &= kept;
                turned();
            }
            const uint4 vs = reinterpret_cast<const uint4*>(head_lds)[32 + m];
            const uint4 vz = reinterpret_cast<const uint4*>(head_lds)[48 + m];
            // The tokens' scales lie below 2^(x + 14), x the exponent field - 28 of each,
            // but no less than -15.
            uint32_t x2[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const us2_t field = __builtin_elementwise_max(__builtin_bit_cast(us2_t, (word(vs, i) >> 10) & 0x001F001Fu),
                                                              us2_t{13, 13});
                x2[i] = as_u32(as_h2(__builtin_bit_cast(uint32_t, field) | 0x64006400u) - as_h2(kHalf1052));
            }
            float cand[NH];
            const auto candidates = [&]() {
                float far = 0.0f;
#pragma unroll
                for (int u = 0; u < NH; ++u) {
                    cand[u] = -__builtin_huge_valf();
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int e = r / 2 + 4 * (r & 1);
                        cand[u] = __builtin_fmaxf(cand[u], __builtin_fmaf(sc[u][r], cc[u], (float)as_h2(x2[e >> 1])[e & 1]));
                    }
                    far = __builtin_fmaxf(far, __builtin_fabsf(cand[u]));
                }
                return far;
            };
            // Far scores are rounded first: then the exponents below take one number
            // from itself, and not from another that is rounded by more than 1.
            if (__builtin_amdgcn_ballot_w64(candidates() >= 0x1p20f) != 0) {
#pragma unroll
                for (int u = 0; u < NH; ++u) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) sc[u][r] = rounded_product(sc[u][r], cc[u]);
                    cc[u] = 1.0f;
                }
                candidates();
            }
            rebase(cand);
            uint4 low[NH];
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                float w[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const int e = r / 2 + 4 * (r & 1);
                    const float p = exp2_hw(__builtin_fmaf(sc[u][r], cc[u], -R[u]));
                    L[u] += p;
                    w[r] = __builtin_fmaf(p, (float)as_h2(word(vs, e >> 1))[e & 1], zero);   // (one v_fma_mix)
                    cz[u] = __builtin_fmaf(w[r], (float)as_h2(word(vz, e >> 1))[e & 1], cz[u]);
                }
                uint4 high;
                halves(w[0], w[1], high.x, low[u].x);
                halves(w[2], w[3], high.y, low[u].y);
                halves(w[4], w[5], high.z, low[u].z);
                halves(w[6], w[7], high.w, low[u].w);
                uint4* to = reinterpret_cast<uint4*>(p_lds + (4 * g + (kSplit ? 2 * u : u)) * kPRow + 8 * m);
                *to = high;
                if (kSplit) *reinterpret_cast<uint4*>(p_lds + (4 * g + 2 * u + 1) * kPRow + 8 * m) = low[u];
            }
            turned();
            uint4 b0[4], b1[4];
            const uint4* pr = reinterpret_cast<const uint4*>(p_lds + m * kPRow + 32 * g);
#pragma unroll
            for (int j = 0; j < 4; ++j) b0[j] = pr[j];
            if (!kSplit) {                    // the lo halves through the same rows
                turned();
#pragma unroll
                for (int u = 0; u < NH; ++u)
                    *reinterpret_cast<uint4*>(p_lds + (4 * g + u) * kPRow + 8 * m) = low[u];
                turned();
#pragma unroll
                for (int j = 0; j < 4; ++j) b1[j] = pr[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const h8_t c = unpack_v(word(V[t], j));
                    O[t] = mfma(c, as_h8(b0[j]), O[t]);
                    if (!kSplit) O[t] = mfma(c, as_h8(b1[j]), O[t]);
                }
            __builtin_amdgcn_wave_barrier();   // what is in LDS is read before the next unit's goes in
        } else {
            // ---- 32 tokens of the window, fp16.
            const int gw = anew(g), mw = anew(m);
            const int t0 = kQuarter * (cu.s.w0 + cu.unit - (cu.s.nb - cu.s.b0));
            const int end = cu.s.len - cu.s.nb * kG, begin = cu.s.left - cu.s.nb * kG;   // rows that count
            const uint16_t* wk = window_of(A.c, cu.slot, cu.head, 0) + t0 * kD;
            const uint16_t* wvp = window_of(A.c, cu.slot, cu.head, 1) + t0 * kD;
            uint4 kx[2][4], vx[8];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    kx[r][j] = *reinterpret_cast<const uint4*>(wk + (16 * r + mw) * kD + 32 * gw + 8 * j);
#pragma unroll
            for (int i = 0; i < 8; ++i) vx[i] = *reinterpret_cast<const uint4*>(wvp + (4 * i + gw) * kD + 8 * mw);
            if (in_blocks) {
                in_blocks = false;
#pragma unroll
                for (int t = 0; t < 8; ++t) O[t] *= kVUnit;
            }
            f4_t S[2] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 c4 = *q_lds(j);    // (exact: the lo slots hold nothing)
                const uint4 qw = m_lo ? make_uint4(0, 0, 0, 0)
                                      : make_uint4(c4.x, pk_mul(c4.y, kSixteen), c4.z, pk_mul(c4.w, kSixteen));
#pragma unroll
                for (int r = 0; r < 2; ++r) S[r] = mfma(as_h8(qw), as_h8(code_order(kx[r][j])), S[r]);
            }
            float sc[NH][2], cand[NH];
#pragma unroll
            for (int u = 0; u < NH; ++u) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int t = t0 + 16 * r + mw;
                    sc[u][r] = t >= begin && t < end ? rounded_product(S[r][kSplit ? (2 * u) & 3 : u], cn[u]) : -__builtin_huge_valf();
                }
                cand[u] = __builtin_fmaxf(sc[u][0], sc[u][1]) + (float)(1 - 14);   // (as a scale of 1)
            }
            rebase(cand);
            uint32_t low[NH];
#pragma unroll
            for (int u = 0; u < NH; ++u) {
                const float p0 = exp2_hw(sc[u][0] - R[u]), p1 = exp2_hw(sc[u][1] - R[u]);
                L[u] += p0 + p1;
                uint32_t high;
                halves(p0, p1, high, low[u]);
                uint16_t* to = p_lds + (4 * gw + (kSplit ? 2 * u : u)) * kPWindow + mw;
                to[0] = (uint16_t)high;
                to[16] = (uint16_t)(high >> 16);
                if (kSplit) {
                    to[kPWindow] = (uint16_t)low[u];
                    to[kPWindow + 16] = (uint16_t)(low[u] >> 16);
                }
            }
            turned();
            const uint4* pr = reinterpret_cast<const uint4*>(p_lds + mw * kPWindow + 8 * gw);
            const h8_t b0 = as_h8(*pr);
            h8_t b1 = b0;
            if (!kSplit) {
                turned();
#pragma unroll
                for (int u = 0; u < NH; ++u) {
                    uint16_t* to = p_lds + (4 * gw + u) * kPWindow + mw;
                    to[0] = (uint16_t)low[u];
                    to[16] = (uint16_t)(low[u] >> 16);
                }
                turned();
                b1 = as_h8(*pr);
            }
            // V rows through LDS, 64 channels at a time, to be read by channel
            // (zeros where a row does not count: it may hold anything).
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int t = t0 + 4 * i + gw;
                    const bool in = t >= begin && t < end;
                    if ((mw >> 3) == half)
                        *reinterpret_cast<uint4*>(v_lds + (4 * i + gw) * kVRow + 8 * (mw & 7)) =
                            in ? vx[i] : make_uint4(0, 0, 0, 0);
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    uint32_t u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint16_t* at = v_lds + (8 * gw + 2 * i) * kVRow + 16 * t + mw;
                        u[i] = (uint32_t)at[0] | ((uint32_t)at[kVRow] << 16);
                    }
                    const h8_t a = as_h8(make_uint4(u[0], u[1], u[2], u[3]));
                    O[4 * half + t] = mfma(a, b0, O[4 * half + t]);
                    if (!kSplit) O[4 * half + t] = mfma(a, b1, O[4 * half + t]);
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            }
            __builtin_amdgcn_wave_barrier();
            load_k(nbuf, K, H);
        }
        load_v(nbuf, V);

        // ---- the end of the row, or of this wave's part of it.
        if (!more || cu.unit + 1 == cu.units) {
            if (cu.unit <= f - f0 && cu.unit + 1 == cu.units) {   // all of the row was here
                float inv_u[NH], z_u[NH];
#pragma unroll
                for (int u = 0; u < NH; ++u) {
                    inv_u[u] = 1.0f / total_l(u);
                    z_u[u] = group_sum<16>(cz[u]) * inv_u[u];
                }
                const float inv = to_slot(inv_u), z = to_slot(z_u), k = in_blocks ? inv * kVUnit : inv;
                const int mo = my_head();
                uint16_t* o = A.out + cu.entry * A.out_stride + (int64_t)(cu.head * A.group + cu.first + mo) * kD + 4 * anew(g);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(both(O[t][i]), k, -z);
                    if (mo >= 0) *reinterpret_cast<uint2*>(o + 16 * t) = make_uint2(half_pair(v[0], v[1]), half_pair(v[2], v[3]));
                }
            } else if (more) {                                    // the end of a row begun before: first partial sums
                keep(reinterpret_cast<float*>(lds + kWaves * kWaveLds) + wv * A.per_chunk * kPart);
                note_segment(2 * wv, f);
            } else {
                open = true;
                note_segment(2 * wv + 1, f);
            }
            if (!kSplit && more) load_q(nx, piece);
            if (more) start_row(nx, piece);
        }
        if (!more) break;
        cu = nx;
        if (f + 2 < f1) {
            advance(nx);
            fetch_page(nx);
        }
    }
    // ---- the workgroup's partial sums, joined row by row.
    __syncthreads();                      // no wave needs its headers and window rows any more
    if (open) keep(reinterpret_cast<float*>(lds + wv * kWaveLds));
    __syncthreads();
    // Segment 2 w + k: wave w's first (k = 0) or last row.  Their rows ascend, so
    // a row's segments are the lanes that hold its number.  Lane k takes the
    // k-th row's description; then the waves share the rows' (head, channel)
    // places, 64 at a time.
    const int mine = lane < 2 * kWaves ? seg_row[lane] : -1;
    const int from = lane < 2 * kWaves ? seg_begin[lane] : 0, to = lane < 2 * kWaves ? seg_end[lane] : 0;
    uint32_t left = (uint32_t)__builtin_amdgcn_ballot_w64(mine >= 0);
    int joins = 0, k_row = 0, k_begin = 0, k_end = 0;
    uint32_t k_in = 0;
    for (; left != 0; ++joins) {
        const int s0 = __builtin_ctz(left);
        const int row = __builtin_amdgcn_readlane(mine, s0);
        const uint32_t in = (uint32_t)__builtin_amdgcn_ballot_w64(mine == row);
        left &= ~in;
        const int begin = __builtin_amdgcn_readlane(from, s0), end = __builtin_amdgcn_readlane(to, s0);
        if (lane == joins) {
            k_row = row;
            k_begin = begin;
            k_end = end;
            k_in = in;
        }
    }
    if (A.groups != 0 && wv == 0) {       // the last one may go on in the next run
        const int k = joins > 0 ? joins - 1 : 0;
        const int begin = __builtin_amdgcn_readlane(k_begin, k), end = __builtin_amdgcn_readlane(k_end, k);
        const int row = joins > 0 && begin >= run0 && end > run1 ? __builtin_amdgcn_readlane(k_row, k) : -1;
        if (lane == 0) A.cross[blockIdx.x] = make_int4(row, end, begin <= run0 ? 0 : 1, 0);
    }
    const int tasks = (A.per_chunk * (kD / 4) + 63) / 64;            // of a row
    for (int task = wv; task < joins * tasks; task += kWaves) {
        const int k = task / tasks;
        const int row = __builtin_amdgcn_readlane(k_row, k), begin = __builtin_amdgcn_readlane(k_begin, k);
        const int end = __builtin_amdgcn_readlane(k_end, k);
        const uint32_t in = (uint32_t)__builtin_amdgcn_readlane((int)k_in, k);
        const int entry = row / rows, in_entry = row - entry * rows;
        const int h = in_entry / A.chunks, first = (in_entry - h * A.chunks) * A.per_chunk;
        const int n = A.group - first < A.per_chunk ? A.group - first : A.per_chunk;
        const bool whole = begin >= run0 && end <= run1;
        const int64_t at = ((int64_t)blockIdx.x * 2 + (begin <= run0 ? 0 : 1)) * A.per_chunk;
        const int i = (task - k * tasks) * 64 + lane;
        if (i < n * (kD / 4)) {
            const int q_head = i / (kD / 4), c = i % (kD / 4) * 4;
            // A wave has one segment of the row at most.  All are read at once; what
            // lies in the places of the others (anything) does not count.
            f4_t o[kWaves], st[kWaves];
            float top = -__builtin_huge_valf(), l = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const bool is_first = (in >> (2 * w)) & 1, has = (in >> (2 * w)) & 3;
                const float* part = reinterpret_cast<const float*>(lds + (is_first ? kWaves * kWaveLds + w * A.per_chunk * kPart * 4
                                                                                   : w * kWaveLds)) + q_head * kPart;
                st[w] = *reinterpret_cast<const f4_t*>(part + kD);
                o[w] = *reinterpret_cast<const f4_t*>(part + c);
                if (!has) {
                    st[w] = f4_t{-__builtin_huge_valf(), 0.0f, 0.0f, 0.0f};
                    o[w] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
                }
                top = __builtin_fmaxf(top, st[w][0]);
            }
            f4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = exp2_hw(st[w][0] - top);
                l = __builtin_fmaf(f, st[w][1], l);
                sum += (o[w] - st[w][2]) * f;
            }
            if (whole) {
                const float inv = 1.0f / l;
                *reinterpret_cast<uint2*>(A.out + entry * A.out_stride + (int64_t)(h * A.group + first + q_head) * kD + c) =
                    make_uint2(half_pair(sum[0] * inv, sum[1] * inv), half_pair(sum[2] * inv, sum[3] * inv));
            } else {
                *reinterpret_cast<f4_t*>(A.part_o + (at + q_head) * kD + c) = sum;
                if (c == 0) A.part_ml[at + q_head] = make_float2(top, l);
            }
        }
    }
}

// Workgroup (b < groups - 1, query head of the row): the row that begins in run b
// and goes past it, from the partial sums of the runs that share it,
//     out = sum_p 2^(R_p - R) O_p / sum_p 2^(R_p - R) L_p:
// thread (j, c) takes channels 4 c .. of the partial sums j, j + 8, .., then the
// eight j's are added in order.  The other workgroups, one per entry: zeros
// where there is nothing to see.
__global__ __launch_bounds__(kJoin) void paged_join_kernel(const AttnArgs A) {
    constexpr int kWide = kJoin / (kD / 4);
    __shared__ f4_t acc[kWide][kD / 4];
    __shared__ float2 acc_rl[kWide];
    read_arguments(A);
    const int rows = (int)A.c.heads * A.chunks, tid = threadIdx.x;
    if ((int)blockIdx.x >= A.groups - 1) {
        if (blockIdx.y != 0) return;
        const int entry = (int)blockIdx.x - (A.groups - 1);
        const int64_t slot = slot_of(A.c, A.seqs, entry);
        if (slot >= 0 && clamped_len(A.c, A.lens, slot) > 0) return;
        uint2* out = reinterpret_cast<uint2*>(A.out + entry * A.out_stride);
        for (int i = tid; i < (int)A.c.heads * A.group * (kD / 4); i += kJoin) out[i] = make_uint2(0, 0);
        return;
    }
    const int4 x = A.cross[blockIdx.x];
    if (x.x < 0) return;
    const int entry = x.x / rows, row = x.x - entry * rows, q_head = blockIdx.y;
    const int h = row / A.chunks, first = (row - h * A.chunks) * A.per_chunk;
    if (first + q_head >= A.group) return;
    const int total = A.cross[A.groups].w;
    const Share share(total, A.groups < total ? A.groups : total);
    const int w0 = blockIdx.x, w1 = share.of(x.y - 1);
    const int j = tid / (kD / 4), c = tid % (kD / 4);
    float R = -__builtin_huge_valf(), l = 0.0f;
    f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = w0 + j; w <= w1; w += 4 * kWide) {      // four at a time
        float2 ml[4];
        f4_t v[4];
        float top = R;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = w + k * kWide <= w1 ? w + k * kWide : w1;
            const int64_t at = ((int64_t)p * 2 + (p == w0 ? x.z : 0)) * A.per_chunk + q_head;
            ml[k] = A.part_ml[at];
            v[k] = *reinterpret_cast<const f4_t*>(A.part_o + at * kD + 4 * c);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (w + k * kWide > w1) ml[k] = make_float2(-__builtin_huge_valf(), 0.0f);
            top = __builtin_fmaxf(top, ml[k].x);
        }
        const float f0 = exp2_hw(R - top);
        l *= f0;
        o *= f0;
        R = top;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = exp2_hw(ml[k].x - top);
            l = __builtin_fmaf(f, ml[k].y, l);
            o += v[k] * f;
        }
    }
    acc[j][c] = o;
    if (c == 0) acc_rl[j] = make_float2(R, l);
    __syncthreads();
    if (j != 0) return;
    float top = R;
    for (int k = 1; k < kWide; ++k) top = __builtin_fmaxf(top, acc_rl[k].x);
    f4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
    float ls = 0.0f;
#pragma unroll
    for (int k = 0; k < kWide; ++k) {
        const float f = exp2_hw(acc_rl[k].x - top);
        ls = __builtin_fmaf(f, acc_rl[k].y, ls);
        sum += acc[k][c] * f;
    }
    const float inv = 1.0f / ls;
    uint16_t* out = A.out + entry * A.out_stride + (int64_t)(h * A.group + first + q_head) * kD + 4 * c;
    *reinterpret_cast<uint2*>(out) = make_uint2(half_pair(sum[0] * inv, sum[1] * inv), half_pair(sum[2] * inv, sum[3] * inv));
}

}  // namespace

bool paged_attention_rows_fit(const PagedArgs& c, int64_t q_heads, int64_t count) {
    const int64_t chunks = (q_heads / c.heads + kMaxRow - 1) / kMaxRow;
    return count * c.heads * chunks * kThreads < ((int64_t)1 << 32);
}

hipError_t launch_paged_attention(const void* q, int64_t q_stride, int64_t q_heads, const PagedArgs& c,
                                  const int32_t* lens, const int32_t* seqs, int64_t count, int64_t window,
                                  float scale, void* out, int64_t out_stride, int num_cus, const Scratch& ws,
                                  hipStream_t stream) {
    AttnArgs A;
    A.c = c;
    A.q = static_cast<const uint16_t*>(q);
    A.out = static_cast<uint16_t*>(out);
    A.lens = lens;
    A.seqs = seqs;
    A.q_stride = q_stride;
    A.out_stride = out_stride;
    A.window = window;
    A.count = (int)count;
    A.group = (int)(q_heads / c.heads);
    A.chunks = (A.group + kMaxRow - 1) / kMaxRow;
    A.per_chunk = (A.group + A.chunks - 1) / A.chunks;
    A.chunks = (A.group + A.per_chunk - 1) / A.per_chunk;
    A.scale = scale * 1.4426950408889634f;
    // One workgroup of eight waves per compute unit (two waves fill a SIMD's
    // registers), but no more than there can be units.
    const int64_t rows = count * c.heads * A.chunks, most = rows * (c.max_pages + 4);
    const int64_t groups = num_cus < most ? num_cus : most;
    // A few rows of at most 16 units: one workgroup each, two units a wave, and
    // no second kernel (32 rows of 7 units 10.7 us instead of 13.0; with more
    // rows than compute units the equal runs win, 4096 rows of 2 units 80 us
    // instead of 152).  The lengths lie on the device, so the rule takes the most
    // that the table's width lets them be: short sequences in a cache made for long
    // ones have the runs and the join.
    const bool short_rows = c.max_pages + 4 <= 16 && rows <= num_cus;
    const size_t cross_bytes = (size_t)(groups + 1) * sizeof(int4);
    const size_t parts = (size_t)groups * 2 * A.per_chunk;
    if (ws.sizing()) {
        if (short_rows) return hipSuccess;
        ws.want(cross_bytes + (parts * sizeof(float2) + 15) / 16 * 16 + parts * kD * sizeof(float));
        return hipSuccess;
    }
    uint8_t* at = short_rows ? nullptr : static_cast<uint8_t*>(ws.ptr);
    A.groups = at ? (int)groups : 0;
    A.cross = reinterpret_cast<int4*>(at);
    A.part_ml = reinterpret_cast<float2*>(at + cross_bytes);
    A.part_o = reinterpret_cast<float*>(at + cross_bytes + (parts * sizeof(float2) + 15) / 16 * 16);
    const int64_t grid = at ? groups : rows;
    const size_t lds = kWaves * (kWaveLds + (size_t)A.per_chunk * kPart * sizeof(float));
    const auto kernel = A.per_chunk <= 4 ? paged_attn_kernel<1> : A.per_chunk <= 8 ? paged_attn_kernel<2> : paged_attn_kernel<4>;
    kernel<<<dim3((unsigned)grid), dim3(kThreads), lds, stream>>>(A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !at) return e;
    paged_join_kernel<<<dim3((unsigned)(groups - 1 + count), (unsigned)A.per_chunk), dim3(kJoin), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace wq
