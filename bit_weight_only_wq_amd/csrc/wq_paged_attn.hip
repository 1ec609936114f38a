// Decode attention over a paged int4 KV cache (gfx950): one new token per
// sequence, out = softmax(scale K q) V over the sequence's pages and window
// ("What actually happens when you quantize a KV cache", §2 the decode step,
// §3-§4 the codec, §7 "axis choice").
//
// What bounds it: HBM.  A token of a KV head is 136 bytes and is read once for
// all the query heads of its group, so both products run on the matrix cores,
// with the group's heads as the 16 columns of v_mfma_f32_16x16x32_f16.
//
// Work is cut into units of about 17 KB: one page record (128 tokens of one KV
// head), or 32 tokens of a window.  The units of all entries stand in one line
// (entry, KV head and chunk of up to 16 query heads, unit) and the wavefronts
// of the grid each take an equal run of it, whatever the lengths are: every
// wave forms the running sum of the units itself from lens.  A wave keeps a
// running maximum, sum and output per head; where its run covers a whole row
// (entry, head, chunk) it writes the result, else fp32 partial sums, which a
// second kernel joins in order.  No atomics: a result depends on the batch,
// not on timing.
//
// One unit of a page, per wave, with lane = 16 g + m:
//   scores   A = codes of 16 tokens x 32 channels, B = a_d = q_d s_d.  A lane's
//            16 bytes are channels 32 g .. 32 g + 31 of one token, four
//            k-steps; row m of token group r is token 32 (m / 4) + 4 r + m % 4,
//            so that the result's rows 4 g + i of lane (g, head) are tokens
//            32 g + 4 r + i: what the lane needs as B of the second product.
//   values   A = codes of 16 channels x 32 tokens (a lane's 16 bytes are tokens
//            32 g .. of one channel), B = w_t = p_t s_t.
// Codes become exact fp16 integers (0x6400 | c is 1024 + c, 0x5400 | 16 c is
// 64 + c; minus that).  a and w are held as fp16 pairs hi + lo (22 bits: hi is
// the rounded product, lo the rounded rest), two products each, so their
// rounding stays far below that of the fp16 result.  The zero points enter as
// sum a_d z_d (a product with the zeros as A, once per unit) and sum w_t z_t
// (in fp32, per lane).
//
// Ranges: q is scaled by a power of two per head so that |q| < 2, hence
// |a| < 2 * 8736.  w is kept below 2^14 by the reference R of the running
// exponent, R = max over units of (largest score + exponent of the largest
// scale - 14), which also keeps the weights of tokens with small scales (and
// those next to one that takes most of the weight but has small values) far
// above fp16's smallest numbers.
#include "wq_paged.h"

namespace wq {

using namespace paged;

namespace {

typedef unsigned short us2_t __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxRow = 16;               // query heads of a row (columns of a product)
constexpr int kQuarter = 32;              // window tokens of a unit
constexpr int kVRow = kD + 8;             // fp16 elements of a window row in LDS
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
    int workers;                          // waves that share the line; 0: one per row
    float scale;                          // times log2(e)
    int32_t* prefix;                      // [count + 1] units before each entry
    float2* part_ml;                      // [workers][2][per_chunk] R and sum
    float* part_o;                        // [workers][2][per_chunk][128]
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

// The eight 4-bit codes of a word as fp16 integers, in code order.
struct Masks {
    uint32_t lo, hi;
};
// (1024 + c, 64 + c as they come out of the two masks.)
__device__ __forceinline__ h8_t unpack_raised(uint32_t w, const Masks& k) {
    const uint32_t s = w >> 8;
    return as_h8(make_uint4((w & k.lo) | 0x64006400u, (w & k.hi) | 0x54005400u, (s & k.lo) | 0x64006400u,
                            (s & k.hi) | 0x54005400u));
}
__device__ __forceinline__ h8_t unpack(uint32_t w, const Masks& k) {
    const h2_t e = {(_Float16)-1024.0f, (_Float16)-1024.0f}, o = {(_Float16)-64.0f, (_Float16)-64.0f};
    const uint32_t s = w >> 8;
    uint4 u;
    u.x = as_u32(as_h2((w & k.lo) | 0x64006400u) + e);
    u.y = as_u32(as_h2((w & k.hi) | 0x54005400u) + o);
    u.z = as_u32(as_h2((s & k.lo) | 0x64006400u) + e);
    u.w = as_u32(as_h2((s & k.hi) | 0x54005400u) + o);
    return as_h8(u);
}

__device__ __forceinline__ f4_t mfma(const h8_t& a, const h8_t& b, const f4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t word(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Largest value over the four lanes that share a column.
__device__ __forceinline__ float column_max(float v) {
    v = __builtin_fmaxf(v, __shfl_xor(v, 16, 64));
    return __builtin_fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float column_sum(float v) {
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

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
    int slot, units;
    Span s;
    int64_t page;                         // of this unit, if it is a block
    __device__ __forceinline__ bool block() const { return unit < s.nb - s.b0; }
};

__global__ __launch_bounds__(kThreads, 2) void paged_attn_kernel(const AttnArgs A) {
    __shared__ __align__(16) uint16_t lds_head[kWaves][512];             // a record's K and V headers
    __shared__ __align__(16) uint16_t lds_v[kWaves][kQuarter * kVRow];   // a window unit's V
    const int lane = threadIdx.x & 63, wv = uniform(threadIdx.x >> 6);
    const int g = lane >> 4, m = lane & 15;
    const int me = (int)blockIdx.x * kWaves + wv;
    const int rows = (int)A.c.heads * A.chunks;                          // of an entry
    uint16_t* head_lds = lds_head[wv];
    uint16_t* v_lds = lds_v[wv];

    // ---- this wave's run [f0, f1) of the line, and where it begins.
    Chunk ch;
    Cursor cu;
    int f0, f1;
    cu.unit = 0;
    if (A.workers == 0) {                 // one wave per row
        if (me >= A.count * rows) return;
        cu.entry = me / rows;
        cu.row = me - cu.entry * rows;
        ch.load(A, cu.entry & ~63, lane);
        f0 = 0;
        f1 = span_of(__builtin_amdgcn_readlane(ch.len, cu.entry & 63), A.window).units();
        if (f1 == 0) {                    // nothing to see: zeros
            const int h = cu.row / A.chunks, first = (cu.row - h * A.chunks) * A.per_chunk;
            const int n = A.group - first < A.per_chunk ? A.group - first : A.per_chunk;
            uint32_t* o = reinterpret_cast<uint32_t*>(A.out + cu.entry * A.out_stride + (int64_t)(h * A.group + first) * kD);
            for (int i = lane; i < n * (kD / 2); i += 64) o[i] = 0;
            return;
        }
    } else {
        int total = 0;
        for (int at = 0; at < A.count; at += 64) {
            ch.load(A, at, lane);
            int u = span_of(ch.len, A.window).units() * rows, inc = u;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(inc, o, 64);
                if (lane >= o) inc += up;
            }
            if (me == 0 && at + lane < A.count) A.prefix[at + lane] = total + inc - u;
            total += __builtin_amdgcn_readlane(inc, 63);
        }
        if (me == 0 && lane == 0) A.prefix[A.count] = total;
        const int W = A.workers < total ? A.workers : total;
        if (me >= W) return;
        f0 = (int)((int64_t)me * total / W);
        f1 = (int)((int64_t)(me + 1) * total / W);
        int before = 0;
        for (int at = 0;; at += 64) {     // ends: f0 < total
            if (A.count > 64) ch.load(A, at, lane);
            int u = span_of(ch.len, A.window).units() * rows, inc = u;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(inc, o, 64);
                if (lane >= o) inc += up;
            }
            const uint64_t past = __builtin_amdgcn_ballot_w64(before + inc > f0);
            if (past != 0) {
                const int i = __builtin_ctzll(past);
                before += __builtin_amdgcn_readlane(inc - u, i);
                cu.entry = at + i;
                break;
            }
            before += __builtin_amdgcn_readlane(inc, 63);
        }
        cu.unit = f0 - before;            // in the entry, for now
    }
    cu.entry = uniform(cu.entry);
    cu.slot = __builtin_amdgcn_readlane(ch.slot, cu.entry & 63);
    cu.s = span_of(__builtin_amdgcn_readlane(ch.len, cu.entry & 63), A.window);
    cu.units = cu.s.units();
    if (A.workers != 0) {
        cu.row = cu.unit / cu.units;
        cu.unit -= cu.row * cu.units;
    }

    const auto fetch_page = [&](Cursor& c) {
        c.page = c.block() ? (int64_t)A.c.table[c.slot * A.c.max_pages + c.s.b0 + c.unit] : 0;
    };
    const auto advance = [&](Cursor& c) {   // to the next unit of the line (there is one)
        if (++c.unit < c.units) return;
        c.unit = 0;
        if (++c.row < rows) return;
        c.row = 0;
        do {
            if ((++c.entry & 63) == 0) ch.load(A, c.entry, lane);
            c.slot = __builtin_amdgcn_readlane(ch.slot, c.entry & 63);
            c.s = span_of(__builtin_amdgcn_readlane(ch.len, c.entry & 63), A.window);
            c.units = c.s.units();
        } while (c.units == 0);
    };

    // ---- loads of a block's record: through a buffer of its bytes, or of none
    // where there is no such block, so that the loads are always issued.
    const uint32_t k_off = (uint32_t)((32 * (m >> 2) + (m & 3)) * kRow + 16 * g);   // + 256 per token group
    const uint32_t v_off = (uint32_t)(kVCodes + m * kRow + 16 * g);                 // + 1024 per 16 channels
    const uint32_t h_off = (uint32_t)(kKScales + 16 * lane);
    const auto buffer = [&](const Cursor& c, bool valid) {
        const int64_t page = c.page >= 0 && c.page < A.c.num_pages ? c.page : 0;
        const uint8_t* rec = record(A.c, page, c.row / A.chunks);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(rec), (short)0, valid && c.block() ? kRecord : 0,
                                                 kBufWord3);
    };
    const auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 2));   // 2: streamed
    };

    Masks mk;
    mk.lo = vgpr_const(0x000F000Fu);
    mk.hi = vgpr_const(0x00F000F0u);

    uint4 K[8], V[8], H;
    fetch_page(cu);
    {
        const auto r = buffer(cu, true);
#pragma unroll
        for (int i = 0; i < 8; ++i) K[i] = load16(r, k_off + 256 * i);
        H = load16(r, h_off);
#pragma unroll
        for (int i = 0; i < 8; ++i) V[i] = load16(r, v_off + 1024 * i);
    }
    Cursor nx = cu;
    if (f1 - f0 > 1) {
        advance(nx);
        fetch_page(nx);
    }

    // ---- the row's state.
    uint4 q[4];                           // fp16, in code order
    float cn = 0.0f;                      // score units (log2) of this lane's column, >= 0
    float R = 0.0f, L = 0.0f, cz = 0.0f;
    f4_t O[8];
    bool begun = false, bad = false;
    int heads_here = 0;                   // query heads of the row

    for (int f = f0; f < f1; ++f) {
        const int h = cu.row / A.chunks, first = (cu.row - h * A.chunks) * A.per_chunk;
        if (!begun) {
            begun = true;
            bad = false;
            heads_here = A.group - first < A.per_chunk ? A.group - first : A.per_chunk;
            R = -__builtin_huge_valf();
            L = 0.0f;
            cz = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) O[i] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            uint4 raw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[j] = make_uint4(0, 0, 0, 0);
            if (m < heads_here) {
                const uint4* src = reinterpret_cast<const uint4*>(A.q + cu.entry * A.q_stride +
                                                                  (int64_t)(h * A.group + first + m) * kD + 32 * g);
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[j] = src[j];
            }
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h2_t v = as_h2(word(raw[j], i));
                    top = __builtin_fmaxf(top, __builtin_fmaxf(__builtin_fabsf((float)v.x), __builtin_fabsf((float)v.y)));
                }
            top = column_max(top);
            const int e = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) - 1 : 0;   // top * 2^-e in [1, 2)
            // (Within 2^-120 .. 2^100: no product with an infinity is 0 * inf.)
            cn = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(__builtin_fabsf(A.scale), e), 0x1p-120f, 0x1p100f);
            const float sign = A.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h2_t v = as_h2(word(raw[j], i));
                    w[i] = as_u32(h2_t{(_Float16)__builtin_amdgcn_ldexpf(sign * (float)v.x, -e),
                                       (_Float16)__builtin_amdgcn_ldexpf(sign * (float)v.y, -e)});
                }
                q[j] = code_order(make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
        const bool more = f + 1 < f1;
        const auto nbuf = buffer(nx, more);

        // New reference for the running exponent, and what is held with the old one.
        const auto rebase = [&](float cand) {
            const float Rn = __builtin_fmaxf(R, column_max(cand));
            if (__builtin_amdgcn_ballot_w64(Rn > R) != 0) {
                const float alpha = exp2_hw(R - Rn);
                L *= alpha;
                cz *= alpha;
#pragma unroll
                for (int i = 0; i < 8; ++i) O[i] *= alpha;
                R = Rn;
            }
        };

        if (cu.block()) {
            bad |= cu.page < 0 || cu.page >= A.c.num_pages;
            // Headers to LDS: 16 bytes a lane in, the lane's 64 bytes of each out.
            *reinterpret_cast<uint4*>(head_lds + 8 * lane) = H;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const uint4* hd = reinterpret_cast<const uint4*>(head_lds) + 4 * g;   // + 16 per header array
            uint4 bh[4], bl[4];
            const h8_t raised = as_h8(make_uint4(0x64006400u, 0x54005400u, 0x64006400u, 0x54005400u));
            f4_t z4 = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 s = code_order(hd[j]), z = code_order(hd[16 + j]);
                bh[j] = make_uint4(pk_mul(q[j].x, s.x), pk_mul(q[j].y, s.y), pk_mul(q[j].z, s.z), pk_mul(q[j].w, s.w));
                bl[j] = make_uint4(pk_rest(q[j].x, s.x, bh[j].x), pk_rest(q[j].y, s.y, bh[j].y),
                                   pk_rest(q[j].z, s.z, bh[j].z), pk_rest(q[j].w, s.w, bh[j].w));
                z4 = mfma(as_h8(z), as_h8(bh[j]), z4);
                z4 = mfma(as_h8(z), as_h8(bl[j]), z4);
                z4 = mfma(raised, as_h8(bh[j]), z4);
                z4 = mfma(raised, as_h8(bl[j]), z4);
            }
            f4_t S[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                S[r] = -z4;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const h8_t a = unpack_raised(word(K[r], j), mk);
                    S[r] = mfma(a, as_h8(bh[j]), S[r]);
                    S[r] = mfma(a, as_h8(bl[j]), S[r]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) K[i] = load16(nbuf, k_off + 256 * i);
            H = load16(nbuf, h_off);

            uint4 vs[4], vz[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                vs[j] = hd[32 + j];
                vz[j] = hd[48 + j];
            }
            // Tokens left of the window do not count, whatever they hold.
            const int skip = cu.s.left - (cu.s.b0 + cu.unit) * kG;
            if (skip > 0) {
                asm volatile("" ::: "memory");   // (a branch, not selects in every unit)
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (32 * g + 4 * r + i < skip) S[r][i] = -__builtin_huge_valf();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const auto keep = [&](uint32_t u, int i) {
                        const int at = 32 * g + 8 * j + 2 * i;
                        return u & (at < skip ? (at + 1 < skip ? 0u : 0xFFFF0000u) : ~0u);
                    };
                    vs[j] = make_uint4(keep(vs[j].x, 0), keep(vs[j].y, 1), keep(vs[j].z, 2), keep(vs[j].w, 3));
                    vz[j] = make_uint4(keep(vz[j].x, 0), keep(vz[j].y, 1), keep(vz[j].z, 2), keep(vz[j].w, 3));
                }
            }
            float top = S[0][0];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                top = __builtin_fmaxf(top, __builtin_fmaxf(__builtin_fmaxf(S[r][0], S[r][1]),
                                                           __builtin_fmaxf(S[r][2], S[r][3])));
            us2_t big = us2_t{0, 0};          // scales are positive: they order as their bits do
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = __builtin_elementwise_max(big, __builtin_bit_cast(us2_t, word(vs[j], i)));
            const float sm = half_bits_to_float(big.x > big.y ? big.x : big.y);
            rebase(top * cn + (float)(__builtin_amdgcn_frexp_expf(sm) - 14));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // Tokens 32 g + 8 j + 4 e + i.
                float w[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = exp2_hw(__builtin_fmaf(S[2 * j + e][i], cn, -R));
                        const h2_t s = as_h2(word(vs[j], 2 * e + (i >> 1))), z = as_h2(word(vz[j], 2 * e + (i >> 1)));
                        L += p;
                        w[e][i] = p * (float)s[i & 1];
                        cz = __builtin_fmaf(w[e][i], (float)z[i & 1], cz);
                    }
                uint32_t wh[4], wl[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h2_t hi = h2_t{(_Float16)w[0][i], (_Float16)w[1][i]};
                    wh[i] = as_u32(hi);
                    wl[i] = as_u32(h2_t{(_Float16)(w[0][i] - (float)hi.x), (_Float16)(w[1][i] - (float)hi.y)});
                }
                const h8_t b0 = as_h8(make_uint4(wh[0], wh[1], wh[2], wh[3]));
                const h8_t b1 = as_h8(make_uint4(wl[0], wl[1], wl[2], wl[3]));
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const h8_t a = unpack(word(V[t], j), mk);
                    O[t] = mfma(a, b0, O[t]);
                    O[t] = mfma(a, b1, O[t]);
                }
            }
            __builtin_amdgcn_wave_barrier();   // the headers are read before the next unit's go in
        } else {
            // ---- 32 tokens of the window, fp16.
            const int t0 = kQuarter * (cu.s.w0 + cu.unit - (cu.s.nb - cu.s.b0));
            const int end = cu.s.len - cu.s.nb * kG, begin = cu.s.left - cu.s.nb * kG;   // rows that count
            const uint16_t* wk = window_of(A.c, cu.slot, h, 0) + t0 * kD;
            const uint16_t* wvp = window_of(A.c, cu.slot, h, 1) + t0 * kD;
            uint4 kx[2][4], vx[8];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    kx[r][j] = *reinterpret_cast<const uint4*>(wk + (8 * (m >> 2) + 4 * r + (m & 3)) * kD + 32 * g + 8 * j);
#pragma unroll
            for (int i = 0; i < 8; ++i) vx[i] = *reinterpret_cast<const uint4*>(wvp + (4 * i + g) * kD + 8 * m);
            f4_t S[2];
            float top = -__builtin_huge_valf();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                S[r] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < 4; ++j) S[r] = mfma(as_h8(code_order(kx[r][j])), as_h8(q[j]), S[r]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = t0 + 8 * g + 4 * r + i;
                    S[r][i] = t >= begin && t < end ? S[r][i] * cn : -__builtin_huge_valf();
                    top = __builtin_fmaxf(top, S[r][i]);
                }
            }
            // V rows to LDS (zeros where a row does not count: it may hold
            // anything), to be read by channel.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int t = t0 + 4 * i + g;
                const bool in = t >= begin && t < end;
                *reinterpret_cast<uint4*>(v_lds + (4 * i + g) * kVRow + 8 * m) =
                    in ? vx[i] : make_uint4(0, 0, 0, 0);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            rebase(top + (float)(1 - 14));
            uint32_t wh[4], wl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p0 = exp2_hw(S[i >> 1][2 * (i & 1)] - R), p1 = exp2_hw(S[i >> 1][2 * (i & 1) + 1] - R);
                L += p0 + p1;
                const h2_t hi = h2_t{(_Float16)p0, (_Float16)p1};
                wh[i] = as_u32(hi);
                wl[i] = as_u32(h2_t{(_Float16)(p0 - (float)hi.x), (_Float16)(p1 - (float)hi.y)});
            }
            const h8_t b0 = as_h8(make_uint4(wh[0], wh[1], wh[2], wh[3]));
            const h8_t b1 = as_h8(make_uint4(wl[0], wl[1], wl[2], wl[3]));
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint16_t* at = v_lds + (8 * g + 2 * i) * kVRow + 16 * t + m;
                    u[i] = (uint32_t)at[0] | ((uint32_t)at[kVRow] << 16);
                }
                const h8_t a = as_h8(make_uint4(u[0], u[1], u[2], u[3]));
                O[t] = mfma(a, b0, O[t]);
                O[t] = mfma(a, b1, O[t]);
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 8; ++i) K[i] = load16(nbuf, k_off + 256 * i);
            H = load16(nbuf, h_off);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) V[i] = load16(nbuf, v_off + 1024 * i);

        // ---- the end of the row, or of this wave's part of it.
        if (!more || cu.unit + 1 == cu.units) {
            begun = false;
            const int from = cu.unit - (f - f0);           // the row's unit at f0 (below 0: it began later)
            const bool whole = from <= 0 && cu.unit + 1 == cu.units;
            const float l = bad ? __builtin_nanf("") : column_sum(L), z = column_sum(cz);
            if (whole) {
                const float inv = 1.0f / l;
                uint16_t* o = A.out + cu.entry * A.out_stride + (int64_t)(h * A.group + first + m) * kD + 4 * g;
                if (m < heads_here) {
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        uint2 y;
                        y.x = (uint32_t)float_to_half_bits_rne((O[t][0] - z) * inv) |
                              ((uint32_t)float_to_half_bits_rne((O[t][1] - z) * inv) << 16);
                        y.y = (uint32_t)float_to_half_bits_rne((O[t][2] - z) * inv) |
                              ((uint32_t)float_to_half_bits_rne((O[t][3] - z) * inv) << 16);
                        *reinterpret_cast<uint2*>(o + 16 * t) = y;
                    }
                }
            } else if (m < heads_here) {
                // Partial 0 of this worker: the row that holds f0; 1: a later one.
                const int64_t at = ((int64_t)me * 2 + (from >= 0 ? 0 : 1)) * A.per_chunk + m;
                if (g == 0) A.part_ml[at] = make_float2(R, l);
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    *reinterpret_cast<f4_t*>(A.part_o + at * kD + 16 * t + 4 * g) = O[t] - z;
            }
        }
        cu = nx;
        if (f + 2 < f1) {
            advance(nx);
            fetch_page(nx);
        }
    }
}

// One workgroup per (row of the line, query head of the row): the partial sums
// of the workers whose runs share the row, in their order,
//     out = sum_p 2^(R_p - R) O_p / sum_p 2^(R_p - R) L_p,
// and zeros for a row without units.
__global__ __launch_bounds__(kThreads) void paged_join_kernel(const AttnArgs A) {
    __shared__ float acc[kWaves][kD];
    const int rows = (int)A.c.heads * A.chunks;
    const int entry = blockIdx.x / rows, row = blockIdx.x - entry * rows;
    const int h = row / A.chunks, first = (row - h * A.chunks) * A.per_chunk, n = blockIdx.y;
    if (first + n >= A.group) return;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    uint16_t* out = A.out + entry * A.out_stride + (int64_t)(h * A.group + first + n) * kD;
    const int total = A.prefix[A.count], begin = A.prefix[entry], units = (A.prefix[entry + 1] - begin) / rows;
    if (units == 0) {
        if (threadIdx.x < kD / 2) reinterpret_cast<uint32_t*>(out)[threadIdx.x] = 0;
        return;
    }
    // Worker of unit f: the last w with w * total / W <= f.
    const int W = A.workers < total ? A.workers : total;
    const int64_t a = begin + (int64_t)row * units, b = a + units;
    const int w0 = (int)(((a + 1) * W - 1) / total), w1 = (int)((b * W - 1) / total);
    if (w0 == w1) return;                                    // written by its wave
    const int head0 = (int64_t)w0 * total / W == a ? 0 : 1;  // where the first worker's part is
    const auto part = [&](int w) { return ((int64_t)w * 2 + (w == w0 ? head0 : 0)) * A.per_chunk + n; };
    float R = -__builtin_huge_valf();
    for (int w = w0 + lane; w <= w1; w += 64) R = __builtin_fmaxf(R, A.part_ml[part(w)].x);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) R = __builtin_fmaxf(R, __shfl_xor(R, o, 64));
    float l = 0.0f;
    for (int w = w0 + lane; w <= w1; w += 64) {
        const float2 ml = A.part_ml[part(w)];
        l += ml.y * exp2_hw(ml.x - R);
    }
    l = group_sum<64>(l);
    float2 o = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int w = w0 + wv; w <= w1; w += kWaves) {
        const int64_t at = part(w);
        const float f = exp2_hw(A.part_ml[at].x - R);
        const float2 v = *reinterpret_cast<const float2*>(A.part_o + at * kD + 2 * lane);
        o.x = __builtin_fmaf(f, v.x, o.x);
        o.y = __builtin_fmaf(f, v.y, o.y);
    }
    acc[wv][2 * lane] = o.x;
    acc[wv][2 * lane + 1] = o.y;
    __syncthreads();
    if (threadIdx.x < kD) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) v += acc[k][threadIdx.x];
        out[threadIdx.x] = float_to_half_bits_rne(v / l);
    }
}

}  // namespace

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
    // Two waves per SIMD (the registers of a wave leave room for two), but no
    // more than there can be units.
    const int64_t rows = count * c.heads * A.chunks, most = rows * (c.max_pages + 4);
    const int64_t workers = 8 * (int64_t)num_cus < most ? 8 * (int64_t)num_cus : most;
    const size_t prefix_bytes = ((size_t)(count + 1) * 4 + 15) / 16 * 16;
    const size_t parts = (size_t)workers * 2 * A.per_chunk;
    if (ws.sizing()) {
        ws.want(prefix_bytes + (parts * sizeof(float2) + 15) / 16 * 16 + parts * kD * sizeof(float));
        return hipSuccess;
    }
    uint8_t* at = static_cast<uint8_t*>(ws.ptr);
    A.workers = at ? (int)workers : 0;
    A.prefix = reinterpret_cast<int32_t*>(at);
    A.part_ml = reinterpret_cast<float2*>(at + prefix_bytes);
    A.part_o = reinterpret_cast<float*>(at + prefix_bytes + (parts * sizeof(float2) + 15) / 16 * 16);
    const int64_t waves = at ? workers : rows;
    paged_attn_kernel<<<dim3((unsigned)((waves + kWaves - 1) / kWaves)), dim3(kThreads), 0, stream>>>(A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !at) return e;
    paged_join_kernel<<<dim3((unsigned)rows, (unsigned)A.per_chunk), dim3(kThreads), 0, stream>>>(A);
    return hipGetLastError();
}

}  // namespace wq
