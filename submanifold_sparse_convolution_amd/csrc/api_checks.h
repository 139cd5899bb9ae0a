// Argument checks shared by the row operators' C entries.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "smc_internal.h"
#include "smconv.h"

namespace smc {

constexpr int64_t kMaxDim = 1 << 21;           // channels and row distances: tile offsets fit 31 bits
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1024;   // row numbers are 32-bit
constexpr size_t kAlign = 256;

inline int bad(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int bad(int status, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(status, buf);
}

inline int hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return SMC_OK;
    return bad(SMC_ERR_HIP, "%s failed: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }
inline bool words16(const void* p, int64_t ld) { return aligned16(p) && (ld & 7) == 0; }   // 16-bit rows
inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// A [rows, cols] tensor: present where it has elements, row distance in range.
inline int check_rows(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (!p && rows > 0) return bad(SMC_ERR_ARG, "%s is NULL", name);
    if (ld < cols || ld > kMaxDim)
        return bad(SMC_ERR_ARG, "row distance of %s is %lld, outside [%lld, 2^21]", name, (long long)ld,
                   (long long)cols);
    if (((uintptr_t)p & 1) != 0) return bad(SMC_ERR_ARG, "%s is not aligned to its elements", name);
    return SMC_OK;
}

// Do the tensors at p and q (rows of cols elements of es bytes, ld elements from
// row to row) share memory? Columns of one buffer, whose ranges overlap with equal
// row distances in bytes, are told apart; other overlapping ranges count as shared.
inline bool share_memory(const void* p, int64_t ldp, int esp, const void* q, int64_t ldq, int esq, int64_t rows,
                  int64_t colsp, int64_t colsq) {
    if (!p || !q || rows <= 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    const uint64_t pitch = (uint64_t)ldp * esp, wp = (uint64_t)colsp * esp, wq = (uint64_t)colsq * esq;
    if (a + (uint64_t)(rows - 1) * pitch + wp <= b || b + (uint64_t)(rows - 1) * ldq * esq + wq <= a) return false;
    if (pitch != (uint64_t)ldq * esq) return true;
    const uint64_t apart = a > b ? (pitch - (a - b) % pitch) % pitch : (b - a) % pitch;    // q's columns after p's
    return apart < wp || apart + wq > pitch;
}

// Do the `bytes` bytes at v lie over the tensor at p (16-bit rows of cols elements, ld elements apart)?
inline bool over_rows(const void* v, size_t bytes, const void* p, int64_t ld, int64_t rows, int64_t cols) {
    if (!v || !p || rows <= 0 || bytes == 0) return false;
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)v;
    const uint64_t pitch = (uint64_t)ld * 2, width = (uint64_t)cols * 2;
    if (b + bytes <= a || b >= a + (uint64_t)(rows - 1) * pitch + width) return false;
    if (b < a) return true;
    const uint64_t into = (b - a) % pitch;             // bytes of b's row that lie before it
    return into < width || into + bytes > pitch;        // (b lies before the last row's end, so another row follows)
}

// Do the bytes at v lie over those at w?
inline bool over_bytes(const void* v, size_t bytes, const void* w, size_t others) {
    const uintptr_t a = (uintptr_t)v, b = (uintptr_t)w;
    return v && w && bytes > 0 && others > 0 && a < b + others && b < a + bytes;
}

inline int check_common(int64_t n, int64_t c, const char* cname, int dtype) {
    if (n < 0 || n > kMaxRows) return bad(SMC_ERR_ARG, "n = %lld", (long long)n);
    if (c < 1 || c > kMaxDim) return bad(SMC_ERR_ARG, "%s = %lld outside [1, 2^21]", cname, (long long)c);
    if (dtype != SMC_DTYPE_BF16 && dtype != SMC_DTYPE_F16)
        return bad(SMC_ERR_ARG, "dtype %d (SMC_DTYPE_BF16 or SMC_DTYPE_F16)", dtype);
    return SMC_OK;
}

#define CHECK(call)              \
    do {                         \
        const int rc_ = (call);  \
        if (rc_) return rc_;     \
    } while (0)

}  // namespace smc
