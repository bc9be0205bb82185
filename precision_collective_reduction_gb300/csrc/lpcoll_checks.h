// lpcoll_checks.h -- host-side argument checks shared by the entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "lpcoll.h"

namespace lpc {

// Keeps e for lpcoll_last_cuda_error.
void record_cuda_error(cudaError_t e);

inline bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

inline bool bad_dtype(int dtype) { return dtype != LPCOLL_F32 && dtype != LPCOLL_BF16; }

inline int check_ptr(const void *p)
{
    if (p == nullptr)
        return LPCOLL_ERR_ARG;
    return misaligned(p) ? LPCOLL_ERR_ALIGN : LPCOLL_OK;
}

inline int finish(cudaError_t e)
{
    if (e == cudaSuccess)
        return LPCOLL_OK;
    record_cuda_error(e);
    return LPCOLL_ERR_CUDA;
}

// First non-OK status of a list of checks (NULL before alignment is kept by
// the order in which callers list them).
inline int first_error(std::initializer_list<int> sts)
{
    int align = LPCOLL_OK;
    for (int s : sts) {
        if (s == LPCOLL_ERR_ALIGN) {
            if (align == LPCOLL_OK)
                align = s;
        } else if (s != LPCOLL_OK) {
            return s;
        }
    }
    return align;
}

inline size_t elem_bytes(int dtype) { return dtype == LPCOLL_F32 ? 4 : 2; }

inline size_t blocks_of(size_t n, int block) { return (n + block - 1) / block; }

// NULL / alignment check of one per-rank pointer array.
template <class P>
int check_rank_array(P const *arr, int nranks)
{
    if (arr == nullptr)
        return LPCOLL_ERR_ARG;
    for (int r = 0; r < nranks; ++r)
        if (arr[r] == nullptr)
            return LPCOLL_ERR_RANK;
    for (int r = 0; r < nranks; ++r)
        if (misaligned(arr[r]))
            return LPCOLL_ERR_ALIGN;
    return LPCOLL_OK;
}

}  // namespace lpc
