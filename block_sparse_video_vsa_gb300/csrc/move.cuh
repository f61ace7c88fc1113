// Moving cached tokens: the codes and scales of one kv head's tokens from their
// pages into registers, and out to other places.
#pragma once

#include "cache.cuh"

namespace vsa {

constexpr int kMaxTree = 1024;  // nodes of a drafted tree

#if defined(__CUDACC__)

constexpr int kMoveThreads = 128;  // two a token of a page

// A thread's half of a token: the K or the V of it, half the threads each, so
// that a warp reads and writes neighbouring rows: codes in 16-byte pieces, four
// (D = 128) or two neighbouring lanes a row, scales in one piece a row.
template <int kD>
struct MovedToken {
    static constexpr int kPieces = kD / 32;                              // of 16 code bytes, a row
    static constexpr int kRows = kMoveThreads / kPieces;                 // rows of K or V a turn
    static constexpr int kTurns = 2 * kPageTokens / kRows;               // of 64 tokens, K and V
    uint4 codes;
    uint32_t scales;  // kD / 4 of the row's bits: the lane's share of its scale bytes (two channels groups a piece)
};

// Where the row of K (side 0) or V of a sequence's token is; null: its page is out of range.
template <int kD>
__device__ __forceinline__ unsigned char* token_page(const CacheView& c, const int32_t* table, int width, int b, int h,
                                                     int token) {
    const int id = table[(size_t)b * width + token / kPageTokens];
    if (id < 0 || id >= c.pages) {
        atomicOr(c.err, VSA_DEVERR_INDEX);
        return nullptr;
    }
    return c.pool + ((size_t)id * c.kv_heads + h) * PageLayout<kD>::kBytes;
}

// Reads tokens source[0 .. size) (places in the sequence; -1: none) of kv head h
// (kMoveThreads threads call it, `thread` is a thread's number among them; `source` is shared memory).
template <int kD>
__device__ __forceinline__ void take_tokens(const CacheView& c, const int32_t* table, int width, int b, int h,
                                            const int* source, int size, unsigned thread,
                                            MovedToken<kD> (&x)[MovedToken<kD>::kTurns]) {
    using L = PageLayout<kD>;
    using M = MovedToken<kD>;
    const int piece = thread % M::kPieces;
#pragma unroll
    for (int i = 0; i < M::kTurns; ++i) {
        const int row = i * M::kRows + thread / M::kPieces;  // K rows, then V rows
        const int side = row / kPageTokens, t = row % kPageTokens;
        const int token = t < size ? source[t] : -1;
        const unsigned char* page = token >= 0 ? token_page<kD>(c, table, width, b, h, token) : nullptr;
        x[i].codes = make_uint4(0, 0, 0, 0);
        x[i].scales = 0xFFFFFFFFu;  // two bytes are in use: all ones says that there is none
        if (page) {
            const int slot = token % kPageTokens;
            x[i].codes = *reinterpret_cast<const uint4*>(page + side * L::kV + slot * L::kRow + piece * 16);
            x[i].scales = *reinterpret_cast<const uint16_t*>(page + (side ? L::kVScale : L::kKScale) +
                                                             slot * L::kGroups + piece * 2);
        }
    }
}

// Writes what take_tokens read to the places first .. first + size - 1 of a table's sequence.
template <int kD>
__device__ __forceinline__ void put_tokens(const CacheView& c, const int32_t* table, int width, int b, int h, int first,
                                           int size, unsigned thread, const MovedToken<kD> (&x)[MovedToken<kD>::kTurns]) {
    using L = PageLayout<kD>;
    using M = MovedToken<kD>;
    const int piece = thread % M::kPieces;
#pragma unroll
    for (int i = 0; i < M::kTurns; ++i) {
        const int row = i * M::kRows + thread / M::kPieces;
        const int side = row / kPageTokens, t = row % kPageTokens;
        if (t >= size || x[i].scales == 0xFFFFFFFFu) continue;
        unsigned char* page = token_page<kD>(c, table, width, b, h, first + t);
        if (!page) continue;
        const int slot = (first + t) % kPageTokens;
        *reinterpret_cast<uint4*>(page + side * L::kV + slot * L::kRow + piece * 16) = x[i].codes;
        *reinterpret_cast<uint16_t*>(page + (side ? L::kVScale : L::kKScale) + slot * L::kGroups + piece * 2) =
            (uint16_t)x[i].scales;
    }
}

#endif  // __CUDACC__

}  // namespace vsa
