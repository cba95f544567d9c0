// The names of the HIP runtime's interface that the library's headers use.
#pragma once

#include <stddef.h>
#include <string.h>

typedef void *hipStream_t;
typedef int hipError_t;
enum { hipSuccess = 0, hipErrorInvalidConfiguration = 9 };

inline hipError_t hipGetLastError() { return hipSuccess; }
inline hipError_t hipMemsetAsync(void *p, int v, size_t n, hipStream_t)
{
    memset(p, v, n);
    return hipSuccess;
}
