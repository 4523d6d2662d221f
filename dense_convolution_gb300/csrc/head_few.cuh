// Products of a few tokens' values with rows of a matrix that is read in place,
// whatever its type, row stride and alignment: vectors of the rows, and where the
// tokens' values for their elements lie in shared memory.
#pragma once

#include <stdint.h>

#include "head_device.cuh"

namespace conv2d_gb300 {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T> __host__ __device__ constexpr int shift_bits() { return sizeof(T) == 4 ? 2 : 3; }

// A token's values in shared memory: for each element of a vector one block of `pitch` slots, a
// zero slot on both sides.  Two tokens' words lie side by side, for the packed
// multiply-adds (kPair = 2; a single token has none to share with).
template <int NT> constexpr int kPair = NT > 1 ? 2 : 1;
template <int P> struct Word;
template <> struct Word<1> { using T = float; };
template <> struct Word<2> { using T = f32x2; };
__device__ __forceinline__ float fma_words(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f32x2 fma_words(f32x2 a, f32x2 b, f32x2 c) { return fma2(a, b, c); }
template <int P> __device__ __forceinline__ typename Word<P>::T spread(float a) {
    if constexpr (P == 2) return both(a);
    else return a;
}
template <typename T> __host__ __device__ int few_pitch(int hidden) {
    return ((hidden + 16 / (int)sizeof(T) - 1) >> shift_bits<T>()) + 3;
}

template <typename T> __device__ __forceinline__ int phase_of(const T* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// Offsets of the V elements of slot 0 in the words of a token (or pair), for rows that start
// `shift` elements after a boundary: element i of slot s is h's element
// s V + i - shift.
template <typename T> __device__ __forceinline__ void word_offsets(int shift, int pitch, int (&off)[kVec<T>]) {
    constexpr int V = kVec<T>;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = i - shift;                           // -(V-1) .. V-1
        off[i] = (e & (V - 1)) * pitch + (e >> shift_bits<T>()) + 1;
    }
}

}  // namespace conv2d_gb300
