// Argument checks that the operators around the layer share (block_api.hip,
// dense_api.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "host.h"
#include "mega_moe.h"

namespace mega_moe {

constexpr int32_t MAX_TOKENS = 1 << 21;     // one workgroup of up to 1024 threads per token
constexpr int64_t MAX_X_STRIDE = 1 << 22;       // a tile's rows within 32-bit byte offsets
constexpr int MAX_DEVICES = 64;

inline int bad(const char* what) { return fail(MEGA_MOE_ERR_INVALID_ARG, "%s", what); }

inline int check_tokens(int32_t n) {
    if (n < 0 || n > MAX_TOKENS)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "num_tokens must be in [0, %d], got %d", MAX_TOKENS, n);
    return MEGA_MOE_OK;
}

inline bool type_ok(int32_t t) { return t == MEGA_MOE_BF16 || t == MEGA_MOE_F32; }
inline int64_t type_bytes(int32_t t) { return t == MEGA_MOE_F32 ? 4 : 2; }

// Whether [p, p + n) and [q, q + m) meet.
inline bool meet(const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return p && q && n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

// The tensors of one call, for the checks that are alike for all of them.
struct Tensors {
    struct One {
        const char* name;
        const void* p;
        int64_t bytes;      // from its first to its last element
        int64_t row, pitch; // bytes of a row and from row to row; pitch 0: dense
        bool out;
        int64_t part = 0, part_pitch = 0;   // of parts that make up every row at one distance, rows too; 0: whole rows
    };
    One list[24];
    int n = 0;

    // rows x cols elements of `size` bytes, `stride` elements from row to row
    void add(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size, bool out) {
        const int64_t bytes = rows > 0 && cols > 0 ? ((rows - 1) * stride + cols) * size : 0;
        list[n++] = One{name, p, p ? bytes : 0, cols * size, stride == cols || rows <= 1 ? 0 : stride * size, out};
    }

    // rows of `parts` parts of `cols` elements each, `part_stride` elements apart
    void add_parts(const char* name, const void* p, int64_t rows, int64_t parts, int64_t cols, int64_t part_stride, int64_t stride, int64_t size, bool out) {
        add(name, p, rows, (parts - 1) * part_stride + cols, stride, size, out);
        if (parts > 1 && (rows <= 1 || stride % part_stride == 0)) {
            list[n - 1].part = cols * size;
            list[n - 1].part_pitch = part_stride * size;
        }
    }

    // Whether pieces of `row` bytes, `pitch` apart, from p on meet those of `other` bytes from q on.
    static bool between(const void* p, int64_t row, const void* q, int64_t other, int64_t pitch) {
        const int64_t d = (int64_t)(((uintptr_t)q - (uintptr_t)p) % (uintptr_t)pitch);
        const int64_t gap = (uintptr_t)q >= (uintptr_t)p ? d : (pitch - (int64_t)(((uintptr_t)p - (uintptr_t)q) % (uintptr_t)pitch)) % pitch;
        return gap < row || gap + other > pitch;
    }

    // An output and another tensor share an element?  Two views with the same
    // pitch may lie between each other's rows (columns of one wider array), or
    // between each other's parts (heads of q, k and v in turn).
    static bool share(const One& a, const One& b) {
        if (!meet(a.p, a.bytes, b.p, b.bytes)) return false;
        if (a.part_pitch && a.part_pitch == b.part_pitch && !between(a.p, a.part, b.p, b.part, a.part_pitch)) return false;
        if (a.pitch == 0 || a.pitch != b.pitch) return true;
        return between(a.p, a.row, b.p, b.row, a.pitch);
    }

    // `may`: outputs that may be exactly the input `same`
    int check(const char* may = "", const char* same = "", const char* may2 = "", const char* same2 = "") const {
        for (int i = 0; i < n; ++i) {
            if (!list[i].out || !list[i].p) continue;
            for (int j = 0; j < n; ++j) {
                if (i == j || (list[j].out && j < i) || !list[j].p) continue;
                const bool named = (!std::strcmp(list[i].name, may) && !std::strcmp(list[j].name, same)) ||
                                   (!std::strcmp(list[i].name, may2) && !std::strcmp(list[j].name, same2));
                if (named && list[i].p == list[j].p && list[i].pitch == list[j].pitch && list[i].row == list[j].row) continue;
                if (share(list[i], list[j]))
                    return fail(MEGA_MOE_ERR_INVALID_ARG, "%s overlaps %s", list[i].name, list[j].name);
            }
        }
        return MEGA_MOE_OK;
    }
};

// A row stride as given (0: dense), or -1 if it cannot be used: 2^21 rows of the
// widest stride stay within 63 bits of bytes.
inline int64_t stride_of(int64_t given, int64_t cols, int64_t unit) {
    if (given == 0) return cols;
    return given >= cols && given % unit == 0 && given <= ((int64_t)1 << 38) ? given : -1;
}

// The current device can run the kernels and holds the stream and the first
// tensor.  Device kinds are looked up once each.
inline int check_device(const void* tensor, void* stream) {
    static std::atomic<int> kind[MAX_DEVICES];     // 0 not asked, 1 gfx950, 2 another
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(MEGA_MOE_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= MAX_DEVICES)
        return fail(MEGA_MOE_ERR_UNSUPPORTED, "device %d: at most %d devices", dev, MAX_DEVICES);
    int k = kind[dev].load(std::memory_order_relaxed);
    if (k == 0) {
        hipDeviceProp_t prop;
        e = hipGetDeviceProperties(&prop, dev);
        if (e != hipSuccess)
            return fail(MEGA_MOE_ERR_HIP, "hipGetDeviceProperties: %s", hipGetErrorString(e));
        k = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
        kind[dev].store(k, std::memory_order_relaxed);
    }
    if (k != 1)
        return fail(MEGA_MOE_ERR_UNSUPPORTED, "device %d is not gfx950, which this library is built for", dev);
    if (stream) {
        hipDevice_t sd = dev;
        e = hipStreamGetDevice((hipStream_t)stream, &sd);
        if (e != hipSuccess) return fail(MEGA_MOE_ERR_HIP, "hipStreamGetDevice: %s", hipGetErrorString(e));
        if (sd != dev)
            return fail(MEGA_MOE_ERR_INVALID_ARG, "the stream is of device %d, the current device is %d", sd, dev);
    }
    hipPointerAttribute_t at;
    e = hipPointerGetAttributes(&at, tensor);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        return bad("a tensor is not in memory that the device knows");
    }
    // the runtime has an answer for ordinary host memory too
    if (at.type == hipMemoryTypeUnregistered) return bad("the tensors are in host memory that the device does not know");
    if (at.type == hipMemoryTypeDevice && at.device != dev)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "the tensors are on device %d, the current device is %d", at.device, dev);
    return MEGA_MOE_OK;
}

inline int launched() {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(MEGA_MOE_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return ok();
}

inline int check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need == 0) return MEGA_MOE_OK;
    if (!ws || have < need)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "the workspace has %lld bytes, the call needs %lld",
                    (long long)(ws ? have : 0), (long long)need);
    if (!aligned(ws, 16)) return bad("workspace must be 16-byte aligned");
    return MEGA_MOE_OK;
}

inline bool words_aligned(std::initializer_list<const void*> list) {
    for (const void* p : list)
        if (!aligned(p, 4)) return false;
    return true;
}

inline bool lines_aligned(std::initializer_list<const void*> list) {
    for (const void* p : list)
        if (!aligned(p, 16)) return false;
    return true;
}

}  // namespace mega_moe
