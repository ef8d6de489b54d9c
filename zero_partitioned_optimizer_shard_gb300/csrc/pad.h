/*
 * pad.h -- 8 neighbouring 16-bit elements of a row that may start in the middle of a 32-bit word, from
 * loads of whole words where both halves belong to the row, and of a half alone at the row's ends:
 * what lies beside the row is not the caller's row, and is not read.  Plain arithmetic, for the host
 * too: the tests run it on the CPU.
 */
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ZERO_BOTH __host__ __device__ __forceinline__
#else
#define ZERO_BOTH inline
#endif

namespace zero {

/* How many of elements [8c, 8c + 8) a row of dim has. */
ZERO_BOTH uint32_t pad_left(uint32_t c, uint32_t dim)
{
    return 8 * c + 8 <= dim ? 8 : 8 * c < dim ? dim - 8 * c : 0;
}

/* The words that hold at least one of chunk c's elements.  odd: the row starts in a word's upper
 * half.  word(e) loads elements e and e + 1, an aligned word; half(e) element e alone.  (Chunks inside a
 * row on a path of their own, whole words only: 159 us for the loss of 100 x 1,601 by 50,257, 138 so.) */
template <class Word, class Half>
ZERO_BOTH void pad_load(uint32_t (&w)[5], uint32_t c, uint32_t dim, uint32_t odd, Word word, Half half)
{
    const uint32_t left = pad_left(c, dim);
#ifdef __CUDACC__
#pragma unroll
#endif
    for (uint32_t j = 0; j < 5; ++j) {
        const int64_t e = (int64_t)(8 * c + 2 * j) - odd;
        const bool low = e >= 0, high = e + 1 < dim;
        w[j] = 0;
        if (left && 2 * j < left + odd)
            w[j] = low && high ? word(e) : low ? half(e) : (uint32_t)half(e + 1) << 16;
    }
}

/* The chunk's elements from those words, 0 behind the row's end, in w[0] to w[3]. */
ZERO_BOTH void pad_shift(uint32_t (&w)[5], uint32_t c, uint32_t dim, uint32_t odd)
{
    const uint32_t left = pad_left(c, dim);
#ifdef __CUDACC__
#pragma unroll
#endif
    for (uint32_t j = 0; j < 4; ++j) {
        w[j] = odd ? w[j] >> 16 | w[j + 1] << 16 : w[j];
        w[j] = 2 * j + 1 < left ? w[j] : 2 * j < left ? w[j] & 0xffff : 0;
    }
}

}  // namespace zero
