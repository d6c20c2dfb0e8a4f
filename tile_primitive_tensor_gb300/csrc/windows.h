// Which 16 bytes a row that starts anywhere is copied in. Plain host and device
// code, so that what is read can be checked without a GPU.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TPG_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TPG_HOST_DEVICE inline
#endif

namespace tpg {

// A copy's source, an aligned address, and how many of its 16 bytes are read: those
// before the row's end (0: none, and the address is that of the row's first 16).
struct CopyWindow {
    uintptr_t at;
    uint32_t bytes;
};

// The aligned 16 bytes that begin `offset` bytes (a multiple of 16) behind the ones in
// which the row at `row`, of `bytes` bytes, starts.
TPG_HOST_DEVICE CopyWindow copy_window(uintptr_t row, uint64_t bytes, uint64_t offset) {
    const uintptr_t end = row + bytes, start = row & ~uintptr_t(15), at = start + offset;
    if (at >= end) return {start, 0};
    return {at, uint32_t(end - at < 16 ? end - at : 16)};
}

// Whether a row's first copy has to leave bytes out: those before the matrix, which
// begins at `base`. (A copy reads its window from the beginning on. Before other rows
// lie the rows before them, or what is between the two.)
TPG_HOST_DEVICE bool begins_apart(uintptr_t row, uintptr_t base, uint64_t offset) {
    return offset == 0 && (row & ~uintptr_t(15)) < base;
}

}  // namespace tpg
