// Rows read straight from memory into matrix-core operands, for products of few
// tokens: a lane's operand of one instruction is eight consecutive columns of a row.
#pragma once

#include "vq_ffn.h"

namespace vq {
namespace {

template <class T>
__device__ inline typename T::V8 chunk(const typename T::E* row, int64_t col)
{
    typename T::V8 v;
    __builtin_memcpy(&v, row + col, 16);
    return v;
}

// The same as it is loaded ahead.  ODD: rows may begin at an odd element (8192 x 4096
// with rows of 4097, one token: 15.6 us by words, 28.7 us by chunks; of 4098, 13.0).
template <class T, bool ODD>
struct Ahead {
    typename T::V8 v;
    __device__ __forceinline__ void load(const typename T::E* row, int64_t col) { v = chunk<T>(row, col); }
    __device__ __forceinline__ typename T::V8 get(const typename T::E*) const { return v; }
};
template <class T>
struct Ahead<T, true> {
    Words w;
    __device__ __forceinline__ void load(const typename T::E* row, int64_t col) { w.load(row + col); }
    __device__ __forceinline__ typename T::V8 get(const typename T::E* row) const
    {
        const uint4 u = w.get(row);                              // columns are multiples of eight
        return __builtin_bit_cast(typename T::V8, u);
    }
};

// A chunk with columns at or past K as zeros.
template <class T>
__device__ inline typename T::V8 chunk_tail(const typename T::E* row, int64_t col, int64_t K)
{
    typename T::V8 v = {};
    if (col + 8 <= K) {
        v = chunk<T>(row, col);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < K) v[i] = row[col + i];
    }
    return v;
}

}  // namespace
}  // namespace vq
