// Drives row_piece.h: for rows of 1 to 40 elements in arrays of just their size, each
// piece that touches them or lies a piece beside them, against the bytes that it should
// have. Built with the address and undefined-behaviour sanitizers. Prints the number of pieces.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "row_piece.h"

template <class T>
static long check() {
    constexpr int kPer = 16 / sizeof(T);
    long pieces = 0;
    for (int n = 1; n <= 40; ++n) {
        T* row = (T*)std::malloc(n * sizeof(T));
        for (int i = 0; i < n; ++i) row[i] = (T)(1000 + 7 * i + n);
        for (int first = -2 * kPer; first < n + 2 * kPer; ++first, ++pieces) {
            T want[kPer];
            for (int e = 0; e < kPer; ++e) want[e] = first + e >= 0 && first + e < n ? row[first + e] : T(0);
            uint32_t w[4];
            moe::row_piece(w, row, first, n);
            if (std::memcmp(w, want, 16) != 0) {
                std::printf("%zu-byte row of %d from %d\n", sizeof(T), n, first);
                std::exit(1);
            }
        }
        std::free(row);
    }
    return pieces;
}

int main() {
    std::printf("%ld %ld\n", check<uint16_t>(), check<float>());
    return 0;
}
