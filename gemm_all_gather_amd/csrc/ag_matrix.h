// Host-side checks shared by the entry points that take matrices in device memory: sizes, alignment, strides, overlaps
// and workspaces, and the device's CU count.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "ag.h"
#include "ag_status.h"

namespace ag {
constexpr int64_t kMaxDim = int64_t{1} << 31;    // rows (M)
constexpr int64_t kMaxRow = int64_t{1} << 20;    // row length and stride: a tile's rows stay within 32-bit offsets

inline uint64_t up256(uint64_t v) { return (v + 255) & ~uint64_t{255}; }

// A matrix (or vector: rows = 1) in device memory.
struct Mat {
    const char* name;
    uint64_t at;
    int64_t rows, cols, ld;
    int esize;
    bool empty() const { return at == 0 || rows == 0 || cols == 0; }
    uint64_t extent() const { return (static_cast<uint64_t>(rows - 1) * ld + cols) * esize; }
};

// Whether two matrices share a byte.  Matrices of one row pitch whose columns lie side by side do not.
inline bool share(const Mat& a, const Mat& b)
{
    if (a.empty() || b.empty()) return false;
    if (a.at >= b.at + b.extent() || b.at >= a.at + a.extent()) return false;
    const uint64_t pitch = static_cast<uint64_t>(a.ld) * a.esize;
    if (a.rows > 1 && b.rows > 1 && pitch == static_cast<uint64_t>(b.ld) * b.esize) {
        const uint64_t d = (b.at >= a.at ? (b.at - a.at) : pitch - (a.at - b.at) % pitch) % pitch;
        const uint64_t ca = static_cast<uint64_t>(a.cols) * a.esize, cb = static_cast<uint64_t>(b.cols) * b.esize;
        if (d >= ca && d + cb <= pitch) return false;
    }
    return true;
}

inline ag_status_t check_mat(const Mat& m, bool needed)
{
    if (m.rows == 0 || m.cols == 0) return AG_OK;
    if (m.at == 0) return needed ? fail(AG_ERR_INVALID_ARG, "%s is NULL", m.name) : AG_OK;
    if (m.at % m.esize != 0) return fail(AG_ERR_INVALID_ARG, "%s is not aligned to its %d-byte elements", m.name, m.esize);
    if (m.ld < m.cols)
        return fail(AG_ERR_INVALID_ARG, "row stride %lld of %s is below its %lld columns", static_cast<long long>(m.ld),
                    m.name, static_cast<long long>(m.cols));
    if (m.rows > 1 && m.ld > kMaxRow)
        return fail(AG_ERR_UNSUPPORTED, "row stride %lld of %s is above %lld", static_cast<long long>(m.ld), m.name,
                    static_cast<long long>(kMaxRow));
    return AG_OK;
}

inline ag_status_t check_overlaps(std::initializer_list<Mat> ins, std::initializer_list<Mat> outs)
{
    for (const Mat* o = outs.begin(); o != outs.end(); ++o) {
        for (const Mat& i : ins)
            if (share(*o, i)) return fail(AG_ERR_INVALID_ARG, "%s overlaps %s", o->name, i.name);
        for (const Mat* q = outs.begin(); q != o; ++q)
            if (share(*o, *q)) return fail(AG_ERR_INVALID_ARG, "%s overlaps %s", o->name, q->name);
    }
    return AG_OK;
}

inline ag_status_t current_cus(int* cus)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail_hip(e, "hipGetDevice");
    e = hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return fail_hip(e, "hipDeviceGetAttribute(multiProcessorCount)");
    return AG_OK;
}

inline ag_status_t check_workspace(const void* workspace, size_t have, uint64_t need, std::initializer_list<Mat> mats)
{
    if (need == 0) return AG_OK;
    if (workspace == nullptr || reinterpret_cast<uint64_t>(workspace) % 256 != 0)
        return fail(AG_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (have < need)
        return fail(AG_ERR_INVALID_ARG, "workspace of %zu bytes, %llu needed", have, static_cast<unsigned long long>(need));
    const Mat w{"workspace", reinterpret_cast<uint64_t>(workspace), 1, static_cast<int64_t>(need), static_cast<int64_t>(need), 1};
    for (const Mat& m : mats)
        if (share(w, m)) return fail(AG_ERR_INVALID_ARG, "the workspace overlaps %s", m.name);
    return AG_OK;
}

inline uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

}  // namespace ag
