// row_piece.h -- sixteen bytes of a row whose neighbours are not to be read. No CUDA
// here but the qualifier: the CPU tests run the same code.
#pragma once

#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define MOE_ROW_PIECE __device__ __forceinline__
#else
#define MOE_ROW_PIECE inline
#endif

namespace moe {

// Elements first, first + 1, .. of a row of n (2 or 4 bytes each, first may be
// negative) as four words, 0 for those that are not the row's. The words are put
// together from values: an array of elements need not lie as 16-byte words have to.
template <class T>
MOE_ROW_PIECE void row_piece(uint32_t (&w)[4], const T* row, int first, int n) {
    constexpr int kOfWord = 4 / sizeof(T);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t word = 0;
#pragma unroll
        for (int k = 0; k < kOfWord; ++k) {
            const int at = first + e * kOfWord + k;
            if (at >= 0 && at < n) {
                const T v = row[at];
                uint32_t bits = 0;
                std::memcpy(&bits, &v, sizeof(T));  // (of a value: no access to memory)
                word |= bits << (8 * (int)sizeof(T) * k);
            }
        }
        w[e] = word;
    }
}

}  // namespace moe
