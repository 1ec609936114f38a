// C ABI of the weight-only group-quantized decode GEMM (declared in include/wq.h).
// Validation happens here, synchronously, before anything is enqueued; the
// kernels are then launched on the caller's stream without synchronizing.
// The library allocates no device memory: scratch (split partials, the
// per-tensor maximum) comes from a caller-owned workspace sized by the
// wq_*_workspace_size queries, and calls without one take plans that need
// none.
#include <float.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <mutex>
#include <new>

#include "wq.h"
#include "wq_launch.h"

namespace {

thread_local char g_last_error[256] = "";

wq_status fail(wq_status st, const char* fmt, long long a = 0, long long b = 0) {
    snprintf(g_last_error, sizeof(g_last_error), fmt, a, b);
    return st;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Compute units of the current device, cached per device (the one lazily
// cached device property).
int num_cus() {
    static int cached[64] = {0};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cached[dev] == 0) {
        int v = 0;
        if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0)
            v = 256;
        cached[dev] = v;
    }
    return cached[dev];
}

wq_status check_hip(hipError_t e, const char* what) {
    if (e == hipSuccess) return WQ_OK;
    snprintf(g_last_error, sizeof(g_last_error), "%s: %s", what, hipGetErrorString(e));
    return WQ_ERR_HIP;
}

// A caller's workspace against the bytes the call needs.  Null with size 0
// means none: the call then takes a plan that needs none.  Otherwise it must
// be 16-byte aligned and hold at least `need` bytes.
wq_status check_workspace(const char* who, const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) {
        if (ws_bytes == 0) return WQ_OK;
        snprintf(g_last_error, sizeof(g_last_error), "%s: null workspace with workspace_bytes=%llu", who,
                 (unsigned long long)ws_bytes);
        return WQ_ERR_INVALID_ARG;
    }
    if (!aligned(ws, 16)) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: workspace needs 16-byte alignment", who);
        return WQ_ERR_MISALIGNED;
    }
    if (ws_bytes < need) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: workspace of %llu bytes, the call needs %llu", who,
                 (unsigned long long)ws_bytes, (unsigned long long)need);
        return WQ_ERR_INVALID_ARG;
    }
    return WQ_OK;
}

// Runs fn(paths) with a host array of count path slots.
template <class F>
wq_status with_paths(int32_t count, F fn) {
    int32_t paths_small[64];
    int32_t* paths = count <= 64 ? paths_small : new (std::nothrow) int32_t[count];
    if (!paths) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_grouped: out of host memory (count=%lld)", count);
    const wq_status st = fn(paths);
    if (paths != paths_small) delete[] paths;
    return st;
}

}  // namespace

// ---- the static scratch of wq_gemm_static -------------------------------------
// For callers that cannot allocate (code under graph capture, tight serving
// loops, harnesses that forbid it): split partials live in this fixed device
// array instead of a caller workspace.  Each GPU the library runs on holds its
// own copy until the process ends.  In host code `scratch` names a host-side
// stand-in, so its device address is looked up once per device
// (hipGetSymbolAddress, with that device current) and only that address is
// ever passed to kernels.
constexpr size_t kStaticScratchBytes = (size_t)16 << 20;
static __device__ __align__(256) unsigned char scratch[kStaticScratchBytes];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

// Device address of the current device's copy of `scratch`.
wq_status static_scratch(void** out) {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return check_hip(e, "wq_gemm_static: hipGetDevice");
    if (dev < 0 || dev >= kMaxDevices)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_static: device %lld beyond the %lld the library tracks", dev,
                    kMaxDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return check_hip(e, "wq_gemm_static: hipGetSymbolAddress(scratch)");
        if (!p) return fail(WQ_ERR_HIP, "wq_gemm_static: null address for the static scratch");
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return WQ_OK;
}

}  // namespace

extern "C" {

int32_t wq_version(void) { return WQ_VERSION; }

const char* wq_status_string(wq_status s) {
    switch (s) {
        case WQ_OK: return "ok";
        case WQ_ERR_INVALID_ARG: return "invalid argument";
        case WQ_ERR_UNSUPPORTED: return "unsupported shape or layout";
        case WQ_ERR_MISALIGNED: return "misaligned pointer or stride";
        case WQ_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char* wq_last_error(void) { return g_last_error; }

size_t wq_codes_bytes(int64_t N, int64_t K, int32_t bits) {
    if (N < 0 || K < 0 || bits < 1 || bits > 8 || (K * bits) % 8 != 0) return 0;
    return (size_t)(N * K * bits / 8);
}

int64_t wq_num_groups(int64_t N, int64_t K, int32_t group) {
    if (N < 0 || K < 0 || group < 1 || K % group != 0) return -1;
    return N * (K / group);
}

// Measured crossover on MI355X: the GEMV path wins at B <= 2, the matrix-core
// kernels from B = 3 on.
int32_t wq_gemv_max_batch(void) { return 1; }

// ---- quantize/pack -----------------------------------------------------------

// Shape and scheme checks of a quantize call (no pointers).
static wq_status check_quant_shape(int64_t N, int64_t K, int32_t group, int32_t bits, int32_t scheme) {
    if (N < 0 || K < 1 || group < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: need N >= 0, K >= 1, group >= 1 (N=%lld K=%lld)", N, K);
    if (K % group != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: K=%lld is not a multiple of group=%lld", K, group);
    if (bits < 1 || bits > 8)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: bits=%lld out of range", bits);
    if (scheme < WQ_SCHEME_ASYM || scheme > WQ_SCHEME_OFFSET)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: unknown scheme %lld", scheme);
    if (scheme == WQ_SCHEME_NF4 && bits != 4)
        return fail(WQ_ERR_UNSUPPORTED, "wq_quantize_pack: NF4 codes are 4 bits (got %lld)", bits);
    if (bits < 2)
        return fail(WQ_ERR_UNSUPPORTED, "wq_quantize_pack: the codec takes bits 2..8 (got %lld)", bits);
    if (group % 8 != 0)
        return fail(WQ_ERR_UNSUPPORTED, "wq_quantize_pack: group=%lld must be a multiple of 8", group);
    return WQ_OK;
}

wq_status wq_quantize_workspace_size(int64_t N, int64_t K, int32_t group, int32_t bits, int32_t scheme,
                                     size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_quantize_workspace_size: null bytes");
    *bytes = 0;
    const wq_status st = check_quant_shape(N, K, group, bits, scheme);
    if (st != WQ_OK) return st;
    *bytes = N == 0 ? 0 : wq::quantize_scratch_bytes(scheme);
    return WQ_OK;
}

wq_status wq_quantize_pack_ex(const void* W, int64_t N, int64_t K, int32_t group, int32_t bits,
                              int32_t scheme, void* codes, void* scales, void* zeros, void* workspace,
                              size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    wq_status st = check_quant_shape(N, K, group, bits, scheme);
    if (st != WQ_OK) return st;
    const size_t need = wq::quantize_scratch_bytes(scheme);
    st = check_workspace("wq_quantize_pack", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    if (N == 0) return WQ_OK;
    if (!W || !codes || !scales || !zeros)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: null pointer");
    if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(zeros, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_quantize_pack: W and codes need 16-byte alignment");
    if (need > 0 && !workspace)
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_pack: the per-tensor scheme needs a workspace of %lld bytes",
                    (long long)need);
    return check_hip(wq::launch_quantize_pack(W, N, K, group, bits, scheme, codes, scales, zeros, workspace,
                                              static_cast<hipStream_t>(stream)),
                     "wq_quantize_pack launch");
}

wq_status wq_quantize_pack(const void* W, int64_t N, int64_t K, int32_t group, int32_t bits,
                           void* codes, void* scales, void* zeros, void* stream) {
    return wq_quantize_pack_ex(W, N, K, group, bits, WQ_SCHEME_ASYM, codes, scales, zeros, nullptr, 0,
                               stream);
}

wq_status wq_dequantize(const void* codes, const void* scales, const void* zeros, int64_t N,
                        int64_t K, int32_t group, int32_t bits, int32_t scheme, void* W,
                        void* stream) {
    g_last_error[0] = '\0';
    if (N < 0 || K < 1 || group < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_dequantize: need N >= 0, K >= 1, group >= 1 (N=%lld K=%lld)", N, K);
    if (K % group != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_dequantize: K=%lld is not a multiple of group=%lld", K, group);
    if (scheme < WQ_SCHEME_ASYM || scheme > WQ_SCHEME_OFFSET)
        return fail(WQ_ERR_INVALID_ARG, "wq_dequantize: unknown scheme %lld", scheme);
    if (bits < 2 || bits > 8)
        return fail(WQ_ERR_UNSUPPORTED, "wq_dequantize: the codec takes bits 2..8 (got %lld)", bits);
    if (scheme == WQ_SCHEME_NF4 && bits != 4)
        return fail(WQ_ERR_UNSUPPORTED, "wq_dequantize: NF4 codes are 4 bits (got %lld)", bits);
    if (group % 8 != 0)
        return fail(WQ_ERR_UNSUPPORTED, "wq_dequantize: group=%lld must be a multiple of 8", group);
    if (N == 0) return WQ_OK;
    if (!codes || !scales || !zeros || !W) return fail(WQ_ERR_INVALID_ARG, "wq_dequantize: null pointer");
    if (!aligned(W, 16) || !aligned(scales, 2) || !aligned(zeros, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_dequantize: W needs 16-byte alignment");
    return check_hip(wq::launch_dequantize(codes, scales, zeros, W, N, K, group, bits, scheme,
                                           static_cast<hipStream_t>(stream)),
                     "wq_dequantize launch");
}

// ---- products ----------------------------------------------------------------

// Validates the shape of one product and picks its kernel family (path on
// return); checks no pointer.  A no-op product (B == 0 or N == 0) returns
// WQ_OK with path = -1.
// The header pointers (null for a size query: taken as aligned) decide
// between kernels that need aligned header arrays and those that do not.
static wq_status check_gemm_shape(int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                                  const void* scales, const void* zeros, int32_t& path) {
    if (B < 0 || N < 0 || K < 1 || group < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm: need B >= 0, N >= 0, K >= 1, group >= 1 (B=%lld K=%lld)", B, K);
    if (K % group != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm: K=%lld is not a multiple of group=%lld", K, group);
    if (bits < 1 || bits > 8)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm: bits=%lld out of range", bits);
    if (bits != 2 && bits != 3 && bits != 4 && bits != 8)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: bits=%lld (GPU kernels take 2, 3, 4 or 8)", bits);
    if (path < WQ_PATH_AUTO || path > WQ_PATH_MFMA)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm: unknown path %lld", path);
    const bool low = bits == 2 || bits == 3;
    if (low) {
        // 32-code chunks inside one group; rows of whole 16-byte loads.
        const int unit = bits == 2 ? 64 : 128;
        if (K % unit != 0 || group % 32 != 0)
            return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: bits 2/3 need K %% (64 or 128) == 0 and group %% 32 == 0 "
                        "(K=%lld group=%lld)", K, group);
    } else {
        const int vals = 128 / bits;  // codes per 16-byte chunk
        if (K % vals != 0 || group % vals != 0)
            return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: K=%lld and group=%lld must be multiples of the 16-byte chunk",
                        K, group);
    }
    if (low && !wq::gemv_lowbit_supports(K, group, bits))
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: the 2/3-bit GEMV does not take K=%lld at bits=%lld", K, bits);
    if (B == 0 || N == 0) {
        path = -1;
        return WQ_OK;
    }
    if (low) {
        // The K-split-wave matrix-core kernel where it takes the shape and
        // the header arrays (X's alignment is checked with the pointers),
        // the bit-stream GEMV otherwise.
        const bool kw = wq::kw_takes(B, K, N, group, bits, false, nullptr, scales, zeros, num_cus());
        if (path == WQ_PATH_MFMA && !kw)
            return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: bits=%lld takes the MFMA path only for 2 <= B <= 32, "
                        "group 128, K = 2048, 4096 or 8192, at least 1.8 16-row tiles per compute unit and "
                        "16-byte aligned header arrays", bits);
        path = (path == WQ_PATH_GEMV || !kw) ? WQ_PATH_GEMV : WQ_PATH_MFMA;
        return WQ_OK;
    }
    const bool gemv_ok = wq::gemv_supports(K, bits);
    const bool mfma_ok = wq::mfma_path_takes(B, K, N, group, bits, scales, zeros);
    int use = path;
    if (use == WQ_PATH_AUTO) {
        if (mfma_ok && (B > wq_gemv_max_batch() || !gemv_ok)) use = WQ_PATH_MFMA;
        else use = WQ_PATH_GEMV;
    }
    if (use == WQ_PATH_GEMV && !gemv_ok)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm: GEMV path does not take K=%lld at bits=%lld", K, bits);
    if (use == WQ_PATH_MFMA && !mfma_ok)
        return fail(WQ_ERR_UNSUPPORTED,
                    "wq_gemm: MFMA path needs group %% %lld == 0 (group=%lld), or B <= 4 with aligned header arrays",
                    bits == 4 ? 128 : 64, group);
    path = use;
    return WQ_OK;
}

// Shape, then pointers.
static wq_status check_gemm(const void* X, const void* codes, const void* scales,
                            const void* zeros, const void* Y, int64_t B, int64_t K, int64_t N,
                            int32_t group, int32_t bits, int32_t& path) {
    const wq_status st = check_gemm_shape(B, K, N, group, bits, scales, zeros, path);
    if (st != WQ_OK || path < 0) return st;
    if (!X || !codes || !scales || !zeros || !Y)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm: null pointer");
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(zeros, 2) || !aligned(Y, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_gemm: X and codes need 16-byte alignment");
    return WQ_OK;
}

// Sizes (ws.need set) or launches one validated product on its kernel family.
static wq_status run_gemm(const void* X, const void* codes, const void* scales, const void* zeros,
                          void* Y, int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                          int32_t use, const wq::Scratch& ws, hipStream_t st) {
    if (use == WQ_PATH_MFMA)
        return check_hip(wq::launch_gemm_mfma(X, codes, scales, zeros, Y, B, K, N, group, bits,
                                              num_cus(), ws, st),
                         "wq_gemm (mfma) launch");
    if (ws.sizing()) return WQ_OK;   // the GEMVs use no scratch
    if (bits == 2 || bits == 3)
        return check_hip(wq::launch_gemv_lowbit(X, codes, scales, zeros, Y, B, K, N, group, bits, 0,
                                                num_cus(), st),
                         "wq_gemm (2/3-bit gemv) launch");
    return check_hip(wq::launch_gemv(X, codes, scales, zeros, Y, B, K, N, group, bits, num_cus(), st),
                     "wq_gemm (gemv) launch");
}

wq_status wq_gemm_workspace_size(int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                                 int32_t path, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_workspace_size: null bytes");
    *bytes = 0;
    int32_t use = path;
    const wq_status st = check_gemm_shape(B, K, N, group, bits, nullptr, nullptr, use);
    if (st != WQ_OK || use < 0) return st;
    size_t need = 0;
    wq::Scratch ws;
    ws.need = &need;
    // Sizing launches nothing; the pointers are never read.
    const wq_status s2 = run_gemm(nullptr, nullptr, nullptr, nullptr, nullptr, B, K, N, group, bits, use, ws,
                                  nullptr);
    if (s2 != WQ_OK) return s2;
    *bytes = need;
    return WQ_OK;
}

wq_status wq_gemm_ex(const void* X, const void* codes, const void* scales, const void* zeros,
                     void* Y, int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                     int32_t path, void* workspace, size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    int32_t use = path;
    wq_status st = check_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use);
    if (st != WQ_OK) return st;
    if (use < 0) return check_workspace("wq_gemm", workspace, workspace_bytes, 0);
    size_t need = 0;
    if (workspace) {
        wq::Scratch sz;
        sz.need = &need;
        st = run_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use, sz, nullptr);
        if (st != WQ_OK) return st;
    }
    st = check_workspace("wq_gemm", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    wq::Scratch ws;
    ws.ptr = need > 0 ? workspace : nullptr;
    return run_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use, ws, static_cast<hipStream_t>(stream));
}

wq_status wq_gemm(const void* X, const void* codes, const void* scales, const void* zeros,
                  void* Y, int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                  void* stream) {
    return wq_gemm_ex(X, codes, scales, zeros, Y, B, K, N, group, bits, WQ_PATH_AUTO, nullptr, 0, stream);
}

wq_status wq_gemm_static(const void* X, const void* codes, const void* scales, const void* zeros,
                         void* Y, int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                         int32_t path, void* stream) {
    g_last_error[0] = '\0';
    int32_t use = path;
    wq_status st = check_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use);
    if (st != WQ_OK || use < 0) return st;
    // The plan wq_gemm_ex takes with a workspace, sized first.
    size_t need = 0;
    wq::Scratch sz;
    sz.need = &need;
    st = run_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use, sz, nullptr);
    if (st != WQ_OK) return st;
    if (need > kStaticScratchBytes)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_static: the call needs %lld bytes of scratch, the static array "
                    "holds %lld (use wq_gemm_ex with a workspace)", (long long)need, (long long)kStaticScratchBytes);
    wq::Scratch ws;
    if (need > 0) {
        st = static_scratch(&ws.ptr);
        if (st != WQ_OK) return st;
    }
    return run_gemm(X, codes, scales, zeros, Y, B, K, N, group, bits, use, ws, static_cast<hipStream_t>(stream));
}

// Validates every item (paths[i] receives its kernel family, -1 for a no-op).
static wq_status check_items(const wq_gemm_item* items, int32_t count, int32_t* paths) {
    for (int32_t i = 0; i < count; ++i) {
        const wq_gemm_item& it = items[i];
        paths[i] = WQ_PATH_AUTO;
        const wq_status st = check_gemm(it.X, it.codes, it.scales, it.zeros, it.Y, it.B, it.K, it.N,
                                        it.group, it.bits, paths[i]);
        if (st != WQ_OK) {
            char msg[sizeof(g_last_error)];
            snprintf(msg, sizeof(msg), "%s", g_last_error);
            snprintf(g_last_error, sizeof(g_last_error), "item %d: %s", (int)i, msg);
            return st;
        }
    }
    return WQ_OK;
}

// Sizes or launches a validated item list: X-resident products of one
// (B, bits) go out together, in item order; every other product is one
// wq_gemm.  Launches follow one another on the stream, so they share the
// scratch (its size is the largest any of them needs).
static wq_status run_items(const wq_gemm_item* items, int32_t count, int32_t* paths, const wq::Scratch& ws,
                           hipStream_t st) {
    wq::XrProduct group_buf[64];
    for (int32_t i = 0; i < count; ++i) {
        const wq_gemm_item& it = items[i];
        if (paths[i] < 0) continue;
        const bool xr = paths[i] == WQ_PATH_MFMA && wq::xr_groupable(it.B, it.K, it.group, it.bits);
        if (!xr) {
            const wq_status s2 = run_gemm(it.X, it.codes, it.scales, it.zeros, it.Y, it.B, it.K, it.N,
                                          it.group, it.bits, paths[i], ws, st);
            if (s2 != WQ_OK) return s2;
            continue;
        }
        // Collect the not yet issued X-resident items of this (B, bits).
        int n = 0;
        for (int32_t j = i; j < count && n < 64; ++j) {
            const wq_gemm_item& o = items[j];
            if (paths[j] != WQ_PATH_MFMA || o.B != it.B || o.bits != it.bits ||
                !wq::xr_groupable(o.B, o.K, o.group, o.bits))
                continue;
            group_buf[n++] = wq::XrProduct{o.X, o.codes, o.scales, o.zeros, o.Y, o.K, o.N, o.group};
            paths[j] = -1;  // issued
        }
        // (A product left alone in a launch keeps the single-call kernel.)
        const wq_status s2 = check_hip(wq::launch_gemm_xr_many(group_buf, n, it.B, it.bits, num_cus(), ws, st),
                                       "wq_gemm_grouped (x-resident) launch");
        if (s2 != WQ_OK) return s2;
    }
    return WQ_OK;
}

wq_status wq_gemm_grouped_workspace_size(const wq_gemm_item* items, int32_t count, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_grouped_workspace_size: null bytes");
    *bytes = 0;
    if (count < 0 || (count > 0 && !items))
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_grouped: count=%lld, items=%lld (null)", count,
                    (long long)(items != nullptr));
    return with_paths(count, [&](int32_t* paths) {
        wq_status st = check_items(items, count, paths);
        if (st != WQ_OK) return st;
        size_t need = 0;
        wq::Scratch ws;
        ws.need = &need;
        st = run_items(items, count, paths, ws, nullptr);
        if (st == WQ_OK) *bytes = need;
        return st;
    });
}

wq_status wq_gemm_grouped(const wq_gemm_item* items, int32_t count, void* workspace, size_t workspace_bytes,
                          void* stream) {
    g_last_error[0] = '\0';
    if (count < 0 || (count > 0 && !items))
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_grouped: count=%lld, items=%lld (null)", count,
                    (long long)(items != nullptr));
    return with_paths(count, [&](int32_t* paths) {
        // Validate everything (and size the scratch) before enqueuing anything.
        wq_status st = check_items(items, count, paths);
        if (st != WQ_OK) return st;
        size_t need = 0;
        if (workspace) {
            // Sizing marks issued items in paths; run it on a copy.
            int32_t copy_small[64];
            int32_t* copy = count <= 64 ? copy_small : new (std::nothrow) int32_t[count];
            if (!copy) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_grouped: out of host memory (count=%lld)", count);
            memcpy(copy, paths, sizeof(int32_t) * (size_t)count);
            wq::Scratch sz;
            sz.need = &need;
            st = run_items(items, count, copy, sz, nullptr);
            if (copy != copy_small) delete[] copy;
            if (st != WQ_OK) return st;
        }
        st = check_workspace("wq_gemm_grouped", workspace, workspace_bytes, need);
        if (st != WQ_OK) return st;
        wq::Scratch ws;
        ws.ptr = need > 0 ? workspace : nullptr;
        return run_items(items, count, paths, ws, static_cast<hipStream_t>(stream));
    });
}

// ---- KV cache ------------------------------------------------------------------

// Validates a cache descriptor (not its contents) and copies it into `a`;
// buffers are checked only when `buffers` is set.
static wq_status check_kv_cache(const wq_kv_cache* c, wq::KvCacheArgs& a, bool buffers = true) {
    if (!c) return fail(WQ_ERR_INVALID_ARG, "kv cache: null descriptor");
    if (c->heads < 0 || c->max_blocks < 1 || c->heads > ((int64_t)1 << 31) - 1 ||
        c->max_blocks > ((int64_t)1 << 24))
        return fail(WQ_ERR_INVALID_ARG, "kv cache: need heads >= 0, 1 <= max_blocks <= 2^24 (heads=%lld max_blocks=%lld)",
                    c->heads, c->max_blocks);
    if (buffers && c->heads > 0) {
        if (!c->kcodes || !c->kscales || !c->kzeros || !c->vcodes || !c->vscales || !c->vzeros || !c->kres ||
            !c->vres)
            return fail(WQ_ERR_INVALID_ARG, "kv cache: null buffer");
        if (!aligned(c->kcodes, 16) || !aligned(c->vcodes, 16) || !aligned(c->kres, 16) || !aligned(c->vres, 16) ||
            !aligned(c->kscales, 2) || !aligned(c->kzeros, 2) || !aligned(c->vscales, 2) || !aligned(c->vzeros, 2))
            return fail(WQ_ERR_MISALIGNED, "kv cache: code and residual buffers need 16-byte alignment");
    }
    a = wq::KvCacheArgs{c->kcodes, c->kscales, c->kzeros, c->vcodes, c->vscales, c->vzeros,
                        c->kres,   c->vres,    c->heads,  c->max_blocks};
    return WQ_OK;
}

wq_status wq_kv_quantize_block(const void* K, const void* V, const wq_kv_cache* cache, int64_t block,
                               void* stream) {
    g_last_error[0] = '\0';
    wq::KvCacheArgs a;
    const wq_status st = check_kv_cache(cache, a);
    if (st != WQ_OK) return st;
    if (block < 0 || block >= a.max_blocks)
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_quantize_block: block=%lld outside [0, %lld)", block, a.max_blocks);
    if (a.heads == 0) return WQ_OK;
    if (!K || !V) return fail(WQ_ERR_INVALID_ARG, "wq_kv_quantize_block: null K or V");
    if (!aligned(K, 16) || !aligned(V, 16))
        return fail(WQ_ERR_MISALIGNED, "wq_kv_quantize_block: K and V need 16-byte alignment");
    return check_hip(wq::launch_kv_quantize(K, V, a, block, static_cast<hipStream_t>(stream)),
                     "wq_kv_quantize_block launch");
}

wq_status wq_kv_workspace_size(const wq_kv_cache* cache, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_kv_workspace_size: null bytes");
    *bytes = 0;
    wq::KvCacheArgs a;
    const wq_status st = check_kv_cache(cache, a, false);
    if (st != WQ_OK || a.heads == 0) return st;
    size_t need = 0;
    wq::Scratch ws;
    ws.need = &need;
    const wq_status s2 = check_hip(wq::launch_kv_attention(nullptr, a, nullptr, nullptr, num_cus(), ws, nullptr),
                                   "wq_kv_workspace_size");
    if (s2 == WQ_OK) *bytes = need;
    return s2;
}

wq_status wq_kv_attention(const void* q, const wq_kv_cache* cache, const int32_t* lens, void* out,
                          void* workspace, size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    wq::KvCacheArgs a;
    wq_status st = check_kv_cache(cache, a);
    if (st != WQ_OK) return st;
    size_t need = 0;
    if (workspace && a.heads > 0) {
        wq::Scratch sz;
        sz.need = &need;
        st = check_hip(wq::launch_kv_attention(nullptr, a, nullptr, nullptr, num_cus(), sz, nullptr),
                       "wq_kv_attention sizing");
        if (st != WQ_OK) return st;
    }
    st = check_workspace("wq_kv_attention", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    if (a.heads == 0) return WQ_OK;
    if (!q || !lens || !out) return fail(WQ_ERR_INVALID_ARG, "wq_kv_attention: null q, lens or out");
    if (!aligned(q, 2) || !aligned(out, 2) || !aligned(lens, 4))
        return fail(WQ_ERR_MISALIGNED, "wq_kv_attention: q/out need 2-byte and lens 4-byte alignment");
    wq::Scratch ws;
    ws.ptr = need > 0 ? workspace : nullptr;
    return check_hip(wq::launch_kv_attention(q, a, lens, out, num_cus(), ws, static_cast<hipStream_t>(stream)),
                     "wq_kv_attention launch");
}

// ---- rotary positions ------------------------------------------------------------

// Whether rows of `dim` elements at t * ts + h * hs never overlap.
static bool rows_apart(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
    if (heads > 1 && hs < dim) return false;
    if (tokens <= 1) return true;
    return ts >= (heads - 1) * hs + dim || (ts >= dim && (heads <= 1 || hs >= (tokens - 1) * ts + dim));
}

wq_status wq_rope(const void* x, int64_t tokens, int64_t heads, int64_t dim, int64_t x_token_stride,
                  int64_t x_head_stride, const int32_t* positions, const double* freqs, int64_t rot,
                  int32_t layout, float scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                  void* stream) {
    g_last_error[0] = '\0';
    if (tokens < 0 || heads < 0 || dim < 1 || rot < 0 || rot > dim || rot % 2 != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_rope: need tokens, heads >= 0, dim >= 1, even rot in [0, dim] (dim=%lld "
                    "rot=%lld)", dim, rot);
    if (layout != WQ_ROPE_HALF && layout != WQ_ROPE_INTERLEAVED)
        return fail(WQ_ERR_INVALID_ARG, "wq_rope: unknown layout %lld", layout);
    if (dim > 1024 || tokens >= ((int64_t)1 << 24) || heads > 65535)
        return fail(WQ_ERR_UNSUPPORTED, "wq_rope: dim <= 1024, tokens < 2^24, heads <= 65535 (tokens=%lld heads=%lld)",
                    tokens, heads);
    const int64_t far = (int64_t)1 << 37;    // offsets stay far inside 64 bits
    if (x_token_stride < 0 || x_head_stride < 0 || x_token_stride > far || x_head_stride > far ||
        out_token_stride < 0 || out_head_stride < 0 || out_token_stride > far || out_head_stride > far)
        return fail(WQ_ERR_INVALID_ARG, "wq_rope: strides must be in [0, 2^37]");
    if (tokens == 0 || heads == 0) return WQ_OK;
    if (!rows_apart(tokens, heads, dim, out_token_stride, out_head_stride))
        return fail(WQ_ERR_INVALID_ARG, "wq_rope: output strides (%lld, %lld) make heads overlap", out_token_stride,
                    out_head_stride);
    if (x == out && ((tokens > 1 && x_token_stride != out_token_stride) || (heads > 1 && x_head_stride != out_head_stride)))
        return fail(WQ_ERR_INVALID_ARG, "wq_rope: in place needs equal strides");
    if (!x || !out || (rot > 0 && (!positions || !freqs))) return fail(WQ_ERR_INVALID_ARG, "wq_rope: null pointer");
    if (!aligned(x, 2) || !aligned(out, 2) || !aligned(positions, 4) || !aligned(freqs, 8))
        return fail(WQ_ERR_MISALIGNED, "wq_rope: x and out need 2-byte, positions 4-byte, freqs 8-byte alignment");
    const wq::RopeCall c{x, out, positions, freqs, tokens, heads, dim, rot, x_token_stride, x_head_stride,
                         out_token_stride, out_head_stride, layout == WQ_ROPE_HALF, scale};
    return check_hip(wq::launch_rope(c, num_cus(), static_cast<hipStream_t>(stream)), "wq_rope launch");
}

// ---- 8-bit path ------------------------------------------------------------------

// Rows of K values `stride` elements apart; an output's rows may not overlap.
static bool row_strides_ok(int64_t rows, int64_t K, int64_t stride, bool output) {
    return stride >= 0 && stride <= (int64_t)1 << 37 && (!output || rows <= 1 || stride >= K);
}

static wq_status check_rows_shape(const char* who, int64_t rows, int64_t K, int32_t dtype) {
    if (rows < 0 || K < 1 || (dtype != WQ_FP16 && dtype != WQ_BF16)) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: need rows >= 0, K >= 1 and a known dtype (rows=%lld K=%lld "
                 "dtype=%d)", who, (long long)rows, (long long)K, (int)dtype);
        return WQ_ERR_INVALID_ARG;
    }
    if (rows >= (int64_t)1 << 24 || K > (int64_t)1 << 20) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: rows < 2^24 and K <= 2^20 (rows=%lld K=%lld)", who,
                 (long long)rows, (long long)K);
        return WQ_ERR_UNSUPPORTED;
    }
    return WQ_OK;
}

static wq_status run_norm(const char* who, const wq::NormCall& c, int32_t dtype, void* stream) {
    g_last_error[0] = '\0';
    const wq_status st = check_rows_shape(who, c.rows, c.K, dtype);
    if (st != WQ_OK) return st;
    if (!(c.eps >= FLT_MIN && c.eps <= FLT_MAX))
        return fail(WQ_ERR_INVALID_ARG, "rmsnorm: eps must be finite and at least 2^-126");
    if (!row_strides_ok(c.rows, c.K, c.x_stride, false) || !row_strides_ok(c.rows, c.K, c.residual_stride, false) ||
        !row_strides_ok(c.rows, c.K, c.total_stride, c.total) || !row_strides_ok(c.rows, c.K, c.codes_stride, c.codes) ||
        !row_strides_ok(c.rows, c.K, c.out_stride, c.out))
        return fail(WQ_ERR_INVALID_ARG, "rmsnorm: strides must be in [0, 2^37], an output's at least K=%lld", c.K);
    if (c.rows == 0) return WQ_OK;
    if (!c.x || !c.weight || !(c.codes ? (const void*)c.scales : c.out)) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: null pointer", who);
        return WQ_ERR_INVALID_ARG;
    }
    if (!c.residual != !c.total)
        return fail(WQ_ERR_INVALID_ARG, "rmsnorm: residual and total go together");
    if (c.total && c.rows > 1 && ((c.total == c.x && c.total_stride != c.x_stride) ||
                                  (c.total == c.residual && c.total_stride != c.residual_stride)))
        return fail(WQ_ERR_INVALID_ARG, "rmsnorm: in place needs equal strides");
    if (!aligned(c.x, 2) || !aligned(c.residual, 2) || !aligned(c.weight, 2) || !aligned(c.total, 2) ||
        !aligned(c.out, 2) || !aligned(c.scales, 4))
        return fail(WQ_ERR_MISALIGNED, "rmsnorm: 16-bit arrays need 2-byte, scales 4-byte alignment");
    return check_hip(wq::launch_norm(c, static_cast<hipStream_t>(stream)), "rmsnorm launch");
}

wq_status wq_rmsnorm_quantize(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                              const void* weight, int64_t rows, int64_t K, int32_t dtype, float eps, void* total,
                              int64_t total_stride, void* codes, int64_t codes_stride, float* scales, void* stream) {
    // (a null codes must not pass for a call of wq_rmsnorm)
    if (!codes && rows > 0) return fail(WQ_ERR_INVALID_ARG, "wq_rmsnorm_quantize: null pointer");
    const wq::NormCall c{x, residual, weight, total, codes, scales, nullptr, rows, K, x_stride, residual_stride,
                         total_stride, codes_stride, 0, K > 0 ? 1.0 / (double)K : 0.0, eps, dtype == WQ_BF16};
    return run_norm("wq_rmsnorm_quantize", c, dtype, stream);
}

wq_status wq_rmsnorm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                     const void* weight, int64_t rows, int64_t K, int32_t dtype, float eps, void* total,
                     int64_t total_stride, void* out, int64_t out_stride, void* stream) {
    const wq::NormCall c{x, residual, weight, total, nullptr, nullptr, out, rows, K, x_stride, residual_stride,
                         total_stride, 0, out_stride, K > 0 ? 1.0 / (double)K : 0.0, eps, dtype == WQ_BF16};
    return run_norm("wq_rmsnorm", c, dtype, stream);
}

wq_status wq_quantize_rows(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, int64_t rows,
                           int64_t K, int32_t dtype, void* codes, int64_t codes_stride, float* scales, void* stream) {
    g_last_error[0] = '\0';
    const wq_status st = check_rows_shape("wq_quantize_rows", rows, K, dtype);
    if (st != WQ_OK) return st;
    if (!row_strides_ok(rows, K, x_stride, false) || !row_strides_ok(rows, K, gate_stride, false) ||
        !row_strides_ok(rows, K, codes_stride, true))
        return fail(WQ_ERR_INVALID_ARG, "wq_quantize_rows: strides must be in [0, 2^37], that of codes at least K=%lld", K);
    if (rows == 0) return WQ_OK;
    if (!x || !codes || !scales) return fail(WQ_ERR_INVALID_ARG, "wq_quantize_rows: null pointer");
    if (!aligned(x, 2) || !aligned(gate, 2) || !aligned(scales, 4))
        return fail(WQ_ERR_MISALIGNED, "wq_quantize_rows: x and gate need 2-byte, scales 4-byte alignment");
    const wq::RowsCall c{x, gate, codes, scales, rows, K, x_stride, gate_stride, codes_stride, dtype == WQ_BF16};
    return check_hip(wq::launch_rows(c, static_cast<hipStream_t>(stream)), "wq_quantize_rows launch");
}

static wq_status check_w8_shape(int64_t B, int64_t K, int64_t N) {
    if (B < 0 || N < 0 || K < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8: need B, N >= 0 and K >= 1 (B=%lld K=%lld)", B, K);
    if (K % 16 != 0 || K >= (int64_t)1 << 17)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_w8a8: K must be a multiple of 16 below 2^17 (K=%lld)", K);
    if (B > (int64_t)1 << 20 || N > (int64_t)1 << 22)
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_w8a8: B <= 2^20 and N <= 2^22 (B=%lld N=%lld)", B, N);
    return WQ_OK;
}

// Whether two runs of bytes meet.
static bool bytes_meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return b && pa < pb + (uintptr_t)b_bytes && pb < pa + (uintptr_t)a_bytes;
}

wq_status wq_gemm_w8a8_workspace_size(int64_t B, int64_t K, int64_t N, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8_workspace_size: null bytes");
    *bytes = 0;
    const wq_status st = check_w8_shape(B, K, N);
    if (st != WQ_OK || B == 0 || N == 0) return st;
    wq::W8Call c{};
    c.B = B;
    c.K = K;
    c.N = N;
    size_t need = 0;
    wq::Scratch ws;
    ws.need = &need;
    const hipError_t e = wq::launch_gemm_w8(c, num_cus(), ws, nullptr);
    if (e != hipSuccess) return check_hip(e, "wq_gemm_w8a8_workspace_size");
    *bytes = need;
    return WQ_OK;
}

wq_status wq_gemm_w8a8(const void* A, int64_t a_stride, const float* a_scales, const void* W, int64_t w_stride,
                       const float* w_scales, const void* bias, void* Y, int64_t y_stride, int64_t B, int64_t K,
                       int64_t N, int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    size_t need = 0;
    wq_status st = wq_gemm_w8a8_workspace_size(B, K, N, &need);
    if (st != WQ_OK) return st;
    if (dtype != WQ_FP16 && dtype != WQ_BF16)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8: unknown dtype %lld", dtype);
    const int64_t far = (int64_t)1 << 22;
    if ((B > 1 && (a_stride < K || y_stride < N)) || (N > 1 && w_stride < K) || a_stride < 0 || w_stride < 0 ||
        y_stride < 0 || a_stride > far || w_stride > far || y_stride > far)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8: a_stride and w_stride must be in [K, 2^22], y_stride in [N, 2^22] "
                    "(K=%lld N=%lld)", K, N);
    if (B == 0 || N == 0) return WQ_OK;
    if (!A || !a_scales || !W || !w_scales || !Y) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8: null pointer");
    if (!aligned(A, 16) || !aligned(W, 16) || a_stride % 16 != 0 || w_stride % 16 != 0 || !aligned(a_scales, 4) ||
        !aligned(w_scales, 4) || !aligned(bias, 2) || !aligned(Y, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_gemm_w8a8: A, W and their strides need 16-byte, scales 4-byte, bias and Y "
                    "2-byte alignment");
    st = check_workspace("wq_gemm_w8a8", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    // (one row has no stride: the kernels' buffers end by it)
    const wq::W8Call c{A, a_scales, W, w_scales, bias, Y, B, K, N, B > 1 ? a_stride : K, N > 1 ? w_stride : K,
                       B > 1 ? y_stride : N, dtype == WQ_BF16};
    // The first kernel writes partial sums while others of its workgroups still read.
    if (workspace && need > 0) {
        const int64_t n = (int64_t)need;
        if (bytes_meet(workspace, n, A, (B - 1) * c.a_stride + K) || bytes_meet(workspace, n, W, (N - 1) * c.w_stride + K) ||
            bytes_meet(workspace, n, Y, 2 * ((B - 1) * c.y_stride + N)) || bytes_meet(workspace, n, a_scales, 4 * B) ||
            bytes_meet(workspace, n, w_scales, 4 * N) || bytes_meet(workspace, n, bias, 2 * N))
            return fail(WQ_ERR_INVALID_ARG, "wq_gemm_w8a8: the workspace overlaps an operand or Y");
    }
    wq::Scratch ws;
    ws.ptr = workspace;
    return check_hip(wq::launch_gemm_w8(c, num_cus(), ws, static_cast<hipStream_t>(stream)), "wq_gemm_w8a8 launch");
}

// ---- paged KV cache --------------------------------------------------------------

// Validates a descriptor's sizes, and the buffers named in `need` (1 pages,
// 2 windows, 4 table), and copies it into `a`.
static wq_status check_paged(const wq_kv_paged* c, wq::PagedArgs& a, int need) {
    if (!c) return fail(WQ_ERR_INVALID_ARG, "paged kv cache: null descriptor");
    const int64_t top = ((int64_t)1 << 31) - 1;
    if (c->heads < 1 || c->heads > 32767 || c->num_pages < 1 || c->num_pages > top || c->slots < 1 ||
        c->slots > top)
        return fail(WQ_ERR_INVALID_ARG, "paged kv cache: need 1 <= heads <= 32767 and 1 <= num_pages, slots < 2^31 "
                    "(heads=%lld num_pages=%lld)", c->heads, c->num_pages);
    if (c->max_pages < 1 || c->max_pages > ((int64_t)1 << 24) - 1)
        return fail(WQ_ERR_INVALID_ARG, "paged kv cache: need 1 <= max_pages < 2^24 (max_pages=%lld)", c->max_pages);
    if (((need & 1) && !c->pages) || ((need & 2) && !c->windows) || ((need & 4) && !c->table))
        return fail(WQ_ERR_INVALID_ARG, "paged kv cache: null buffer");
    if (((need & 1) && !aligned(c->pages, 16)) || ((need & 2) && !aligned(c->windows, 16)) ||
        ((need & 4) && !aligned(c->table, 4)))
        return fail(WQ_ERR_MISALIGNED, "paged kv cache: pages and windows need 16-byte, table 4-byte alignment");
    a = wq::PagedArgs{c->pages, c->windows, static_cast<const int32_t*>(c->table), c->heads, c->num_pages, c->slots,
                      c->max_pages};
    return WQ_OK;
}

// Entries of a call's batch.
static wq_status check_batch(const char* who, const wq::PagedArgs& a, const int32_t* lens, const int32_t* seqs,
                             int64_t count) {
    if (count < 0 || count > 65535 || (!seqs && count > a.slots)) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: count=%lld outside [0, 65535], or past the %lld slots", who,
                 (long long)count, (long long)a.slots);
        return WQ_ERR_INVALID_ARG;
    }
    if (count > 0 && (!lens || !aligned(lens, 4) || !aligned(seqs, 4))) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: null or misaligned lens or seqs", who);
        return lens ? WQ_ERR_MISALIGNED : WQ_ERR_INVALID_ARG;
    }
    return WQ_OK;
}

wq_status wq_kv_paged_append(const void* k, const void* v, int64_t tokens, int64_t k_stride, int64_t v_stride,
                             const wq_kv_paged* cache, const int32_t* lens, const int32_t* seqs, const int32_t* cu,
                             int64_t count, void* stream) {
    g_last_error[0] = '\0';
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 7);
    if (st != WQ_OK) return st;
    st = check_batch("wq_kv_paged_append", a, lens, seqs, count);
    if (st != WQ_OK) return st;
    if (tokens < 0 || tokens > ((int64_t)1 << 30) || (!cu && tokens != count))
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_append: tokens=%lld for %lld entries (without cu: one each)", tokens,
                    count);
    if (count == 0 || tokens == 0) return WQ_OK;
    const int64_t row = a.heads * 128;
    if (k_stride < row || v_stride < row || k_stride > ((int64_t)1 << 31) || v_stride > ((int64_t)1 << 31))
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_append: k_stride=%lld and v_stride=%lld must hold a token's heads",
                    k_stride, v_stride);
    if (!k || !v) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_append: null k or v");
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 || !aligned(cu, 4))
        return fail(WQ_ERR_MISALIGNED, "wq_kv_paged_append: k, v and their strides need 16-byte, cu 4-byte alignment");
    return check_hip(wq::launch_paged_append(k, v, tokens, k_stride, v_stride, a, lens, seqs, cu, count,
                                             num_cus(), static_cast<hipStream_t>(stream)),
                     "wq_kv_paged_append launch");
}

// Shape checks of an attention call (no pointers but the descriptor).
static wq_status check_paged_attention(const wq::PagedArgs& a, int64_t count, int64_t q_heads) {
    if (count < 0 || count > 65535 || q_heads < a.heads || q_heads % a.heads != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_attention: need 0 <= count <= 65535 and q_heads a multiple of the "
                    "cache's heads (count=%lld q_heads=%lld)", count, q_heads);
    if (count * q_heads >= ((int64_t)1 << 24) || count * q_heads > (((int64_t)1 << 31) - 1) / (a.max_pages + 4))
        return fail(WQ_ERR_UNSUPPORTED, "wq_kv_paged_attention: count * q_heads must be below 2^24, and times "
                    "(max_pages + 4) below 2^31 (count=%lld q_heads=%lld)", count, q_heads);
    return WQ_OK;
}

wq_status wq_kv_paged_workspace_size(const wq_kv_paged* cache, int64_t count, int64_t q_heads, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_workspace_size: null bytes");
    *bytes = 0;
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 0);
    if (st == WQ_OK) st = check_paged_attention(a, count, q_heads);
    if (st != WQ_OK || count == 0) return st;
    size_t need = 0;
    wq::Scratch ws;
    ws.need = &need;
    st = check_hip(wq::launch_paged_attention(nullptr, 0, q_heads, a, nullptr, nullptr, count, 0, 1.0f, nullptr, 0,
                                              num_cus(), ws, nullptr),
                   "wq_kv_paged_workspace_size");
    if (st == WQ_OK) *bytes = need;
    return st;
}

wq_status wq_kv_paged_attention(const void* q, int64_t q_stride, int64_t q_heads, const wq_kv_paged* cache,
                                const int32_t* lens, const int32_t* seqs, int64_t count, int64_t window, float scale,
                                void* out, int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 7);
    if (st == WQ_OK) st = check_paged_attention(a, count, q_heads);
    if (st == WQ_OK) st = check_batch("wq_kv_paged_attention", a, lens, seqs, count);
    if (st != WQ_OK) return st;
    const int64_t far = (int64_t)1 << 31, row = q_heads * 128;
    if (window < 0 || !(scale - scale == 0.0f))
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_attention: window=%lld must be >= 0, and scale finite", window);
    if (count > 0 && (q_stride < row || out_stride < row || q_stride > far || out_stride > far))
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_attention: q_stride=%lld and out_stride=%lld must hold an entry's "
                    "heads", q_stride, out_stride);
    size_t need = 0;
    if (workspace && count > 0) {
        wq::Scratch sz;
        sz.need = &need;
        st = check_hip(wq::launch_paged_attention(nullptr, 0, q_heads, a, nullptr, nullptr, count, 0, scale, nullptr, 0,
                                                  num_cus(), sz, nullptr),
                       "wq_kv_paged_attention sizing");
        if (st != WQ_OK) return st;
    }
    st = check_workspace("wq_kv_paged_attention", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    if (count == 0) return WQ_OK;
    if (!q || !out) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_attention: null q or out");
    if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 8) || out_stride % 4 != 0)
        return fail(WQ_ERR_MISALIGNED, "wq_kv_paged_attention: q and its stride need 16-byte, out and its stride 8-byte "
                    "alignment");
    if (need == 0 && !wq::paged_attention_rows_fit(a, q_heads, count))
        return fail(WQ_ERR_UNSUPPORTED, "wq_kv_paged_attention: too many rows without a workspace (count=%lld "
                    "q_heads=%lld)", count, q_heads);
    wq::Scratch ws;
    ws.ptr = need > 0 ? workspace : nullptr;
    return check_hip(wq::launch_paged_attention(q, q_stride, q_heads, a, lens, seqs, count, window, scale, out, out_stride,
                                                num_cus(), ws, static_cast<hipStream_t>(stream)),
                     "wq_kv_paged_attention launch");
}

// Pairs of ids below `limit`: in range, no destination twice, none a source.
static wq_status check_pairs(const char* who, const int32_t* pairs, int64_t count, int64_t limit) {
    if (count < 0 || (count > 0 && !pairs)) {
        snprintf(g_last_error, sizeof(g_last_error), "%s: null pairs or count=%lld", who, (long long)count);
        return WQ_ERR_INVALID_ARG;
    }
    if (count == 0) return WQ_OK;
    int32_t* ids = new (std::nothrow) int32_t[2 * (size_t)count];
    if (!ids) return fail(WQ_ERR_INVALID_ARG, "paged kv cache: out of host memory (count=%lld)", count);
    int32_t* dst = ids + count;
    int64_t bad = -1;
    for (int64_t i = 0; i < count && bad < 0; ++i) {
        ids[i] = pairs[2 * i];
        dst[i] = pairs[2 * i + 1];
        if (ids[i] < 0 || dst[i] < 0 || ids[i] >= limit || dst[i] >= limit) bad = i;
    }
    const char* what = "an id out of range";
    if (bad < 0) {
        std::sort(ids, ids + count);
        std::sort(dst, dst + count);
        for (int64_t i = 0; i < count && bad < 0; ++i) {
            if (i > 0 && dst[i] == dst[i - 1]) {
                bad = dst[i];
                what = "a destination twice:";
            } else if (std::binary_search(ids, ids + count, dst[i])) {
                bad = dst[i];
                what = "a destination that is a source:";
            }
        }
    }
    delete[] ids;
    if (bad < 0) return WQ_OK;
    snprintf(g_last_error, sizeof(g_last_error), "%s: %s %lld", who, what, (long long)bad);
    return WQ_ERR_INVALID_ARG;
}

wq_status wq_kv_paged_copy(const wq_kv_paged* cache, const int32_t* pairs, int64_t count, void* stream) {
    g_last_error[0] = '\0';
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 1);
    if (st == WQ_OK) st = check_pairs("wq_kv_paged_copy", pairs, count, a.num_pages);
    if (st != WQ_OK || count == 0) return st;
    return check_hip(wq::launch_paged_copy(a, pairs, count, static_cast<hipStream_t>(stream)), "wq_kv_paged_copy launch");
}

wq_status wq_kv_paged_fork(const wq_kv_paged* cache, int32_t* lens, const int32_t* pairs, int64_t count, void* stream) {
    g_last_error[0] = '\0';
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 6);
    if (st == WQ_OK) st = check_pairs("wq_kv_paged_fork", pairs, count, a.slots);
    if (st != WQ_OK || count == 0) return st;
    if (!lens) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_fork: null lens");
    if (!aligned(lens, 4)) return fail(WQ_ERR_MISALIGNED, "wq_kv_paged_fork: lens need 4-byte alignment");
    return check_hip(wq::launch_paged_fork(a, lens, pairs, count, static_cast<hipStream_t>(stream)),
                     "wq_kv_paged_fork launch");
}

wq_status wq_kv_paged_compact_workspace_size(const wq_kv_paged* cache, size_t* bytes) {
    g_last_error[0] = '\0';
    if (!bytes) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_compact_workspace_size: null bytes");
    *bytes = 0;
    wq::PagedArgs a;
    const wq_status st = check_paged(cache, a, 0);
    if (st == WQ_OK) *bytes = wq::paged_compact_bytes(a);
    return st;
}

wq_status wq_kv_paged_compact(const wq_kv_paged* cache, const int32_t* lens, void* table_out, int32_t* used,
                              void* workspace, size_t workspace_bytes, void* stream) {
    g_last_error[0] = '\0';
    wq::PagedArgs a;
    wq_status st = check_paged(cache, a, 5);
    if (st != WQ_OK) return st;
    const size_t need = wq::paged_compact_bytes(a);
    st = check_workspace("wq_kv_paged_compact", workspace, workspace_bytes, need);
    if (st != WQ_OK) return st;
    if (!workspace)
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_compact: needs a workspace of %lld bytes", (long long)need);
    if (!lens || !table_out || !used) return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_compact: null pointer");
    if (!aligned(lens, 4) || !aligned(table_out, 4) || !aligned(used, 4))
        return fail(WQ_ERR_MISALIGNED, "wq_kv_paged_compact: lens, table_out and used need 4-byte alignment");
    const uintptr_t from = reinterpret_cast<uintptr_t>(cache->table), to = reinterpret_cast<uintptr_t>(table_out);
    if ((from < to ? to - from : from - to) / sizeof(int32_t) < (uintptr_t)(a.slots * a.max_pages))
        return fail(WQ_ERR_INVALID_ARG, "wq_kv_paged_compact: table_out must not overlap the cache's table");
    return check_hip(wq::launch_paged_compact(a, lens, static_cast<int32_t*>(table_out), used, workspace, num_cus(),
                                              static_cast<hipStream_t>(stream)),
                     "wq_kv_paged_compact launch");
}

// ---- other weight formats ------------------------------------------------------

wq_status wq_gemm_offset(const void* X, const void* codes, const void* scales, const void* mins,
                         void* Y, int64_t B, int64_t K, int64_t N, int32_t group, int32_t bits,
                         void* stream) {
    g_last_error[0] = '\0';
    if (B < 0 || N < 0 || K < 1 || group < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_offset: need B >= 0, N >= 0, K >= 1, group >= 1 (B=%lld K=%lld)", B, K);
    if (K % group != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_offset: K=%lld is not a multiple of group=%lld", K, group);
    if (bits < 1 || bits > 8) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_offset: bits=%lld out of range", bits);
    if (!wq::gemv_lowbit_supports(K, group, bits))
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_offset: bits 2, 3, 4 or 8, group %% 32 == 0 and K a multiple of "
                    "the load unit (K=%lld bits=%lld)", K, bits);
    if (B == 0 || N == 0) return WQ_OK;
    if (!X || !codes || !scales || !mins || !Y) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_offset: null pointer");
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(mins, 2) || !aligned(Y, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_gemm_offset: X and codes need 16-byte alignment");
    if (wq::kw_takes(B, K, N, group, bits, true, X, scales, mins, num_cus()))
        return check_hip(wq::launch_gemm_kw(X, codes, scales, mins, Y, B, K, N, group, bits, true, num_cus(),
                                            static_cast<hipStream_t>(stream)),
                         "wq_gemm_offset (mfma) launch");
    return check_hip(wq::launch_gemv_lowbit(X, codes, scales, mins, Y, B, K, N, group, bits, 1, num_cus(),
                                            static_cast<hipStream_t>(stream)),
                     "wq_gemm_offset launch");
}

wq_status wq_gemm_nf4(const void* X, const void* codes, const void* scales, void* Y, int64_t B,
                      int64_t K, int64_t N, int32_t group, void* stream) {
    g_last_error[0] = '\0';
    if (B < 0 || N < 0 || K < 1 || group < 1)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_nf4: need B >= 0, N >= 0, K >= 1, group >= 1 (B=%lld K=%lld)", B, K);
    if (K % group != 0)
        return fail(WQ_ERR_INVALID_ARG, "wq_gemm_nf4: K=%lld is not a multiple of group=%lld", K, group);
    if (!wq::gemv_nf4_supports(K, group))
        return fail(WQ_ERR_UNSUPPORTED, "wq_gemm_nf4: needs K %% 32 == 0, group %% 32 == 0, K <= 16384 (K=%lld group=%lld)",
                    K, group);
    if (B == 0 || N == 0) return WQ_OK;
    if (!X || !codes || !scales || !Y) return fail(WQ_ERR_INVALID_ARG, "wq_gemm_nf4: null pointer");
    if (!aligned(X, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(Y, 2))
        return fail(WQ_ERR_MISALIGNED, "wq_gemm_nf4: X and codes need 16-byte alignment");
    if (wq::kw_nf4_takes(B, K, N, group, X, scales, num_cus()))
        return check_hip(wq::launch_gemm_kw_nf4(X, codes, scales, Y, B, K, N, group, num_cus(),
                                                static_cast<hipStream_t>(stream)),
                         "wq_gemm_nf4 (mfma) launch");
    return check_hip(wq::launch_gemv_nf4(X, codes, scales, Y, B, K, N, group, num_cus(),
                                         static_cast<hipStream_t>(stream)),
                     "wq_gemm_nf4 launch");
}

}  // extern "C"
