// Products that walk K in 128-byte pieces (8-bit integer, block-scaled fp8): operand loads, the
// swizzle of their LDS stages and the order of their tiles.
#pragma once

#include "qpl_gemm.h"

namespace qpl {

namespace {

// Four outputs stored at 2-byte alignment: rows of y may start at any element.
struct __attribute__((packed, aligned(2))) Segment4 {
  u32x2 v;
};

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, (int)kRawBufferWord3);
}

// Byte of chunk c of stage row r: two rows fill the 64 banks, so the 16 lanes that read 16 bytes each in a
// cycle, 16 rows apart by one, hit each bank once.
__device__ __forceinline__ int chunk_at(int r, int c) { return r * PR_ROW + ((c ^ ((r >> 1) & 7)) << 4); }

// Tile (row tile, column tile) at position s of the walk: groups of four row tiles,
// column by column, so that workgroups of one XCD share operand rows in its L2.
// Tiles number below 2^31: y has at most 2^40 elements and a tile 2^12 of them, and the
// grouped weights' columns, E N <= 2^36, bound the tiles of experts with few rows.
__device__ __forceinline__ void walk(int s, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per_group = GROUP_M * tiles_n;
  const int g = s / per_group;
  const int gm = min(tiles_m - g * GROUP_M, GROUP_M);
  const int r = s - g * per_group;
  tm = g * GROUP_M + r % gm;
  tn = r / gm;
}

}  // namespace

}  // namespace qpl
