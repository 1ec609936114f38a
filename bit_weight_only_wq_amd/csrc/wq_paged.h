// Layout of the paged int4 KV cache, shared by its kernels (wq_kv_paged in
// wq.h), and the checks on ids that come from device memory.
#pragma once

#include "wq_device.h"
#include "wq_launch.h"

namespace wq {
namespace paged {

constexpr int kD = 128;             // head dimension
constexpr int kG = 128;             // tokens per block
constexpr int kRow = 64;            // bytes of a code row
constexpr int kRecord = 17408;      // bytes of one page's record of one head
constexpr int kVCodes = 8192, kKScales = 16384, kKZeros = 16640, kVScales = 16896, kVZeros = 17152;
constexpr int kSide = kG * kD;      // fp16 elements of one side of a window

// Asks for all of a kernel's arguments at its start.  They lie in host memory,
// 64 bytes a line; left to the compiler each line is read where its first value
// is used, and every such read is a trip of a microsecond or two on the path of
// a short kernel.
template <class T>
__device__ __forceinline__ void read_arguments(const T& a) {
    static_assert(sizeof(T) <= 4 * 64, "four lines");
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&a);
    constexpr int n = sizeof(T) / 4;
    asm volatile("" ::"s"(w[0]), "s"(w[n > 16 ? 16 : 0]), "s"(w[n > 32 ? 32 : 0]), "s"(w[n > 48 ? 48 : 0]), "s"(w[n - 1]));
}

// Slot of entry i, or -1 for padding.
__device__ __forceinline__ int64_t slot_of(const PagedArgs& c, const int32_t* seqs, int64_t i) {
    const int64_t s = seqs ? seqs[i] : i;
    return s >= 0 && s < c.slots ? s : -1;
}

// The most tokens a slot can hold.
__device__ __forceinline__ int64_t capacity(const PagedArgs& c) { return c.max_pages * kG + (kG - 1); }

__device__ __forceinline__ int64_t clamped_len(const PagedArgs& c, const int32_t* lens, int64_t slot) {
    const int64_t n = lens[slot], cap = capacity(c);
    return n < 0 ? 0 : (n > cap ? cap : n);
}

__device__ __forceinline__ uint8_t* record(const PagedArgs& c, int64_t page, int64_t head) {
    return static_cast<uint8_t*>(c.pages) + (page * c.heads + head) * kRecord;
}

// Side 0 (K) or 1 (V) of a slot's window, [128 tokens][128].
__device__ __forceinline__ uint16_t* window_of(const PagedArgs& c, int64_t slot, int64_t head, int side) {
    return static_cast<uint16_t*>(c.windows) + ((slot * c.heads + head) * 2 + side) * kSide;
}

}  // namespace paged
}  // namespace wq
