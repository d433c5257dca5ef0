// Global -> LDS transfers whose lanes hold the whole offset (buffer_load ... lds without a scalar offset).
//
// Whether a lane reads memory or gets zeros has to follow from its own offset and the descriptor's size: documents
// differ on whether the scalar offset counts in that comparison, and on what happens where it exceeds the size.  The
// forms with a scalar offset (qpl_dma.h) may therefore only move a lane along its own row by it, and a lane whose row
// or columns are not there has kOutOfRange in its own offset.  Here nothing rests on it.
#pragma once

#include "qpl_dma.h"

namespace qpl {

// 16 bytes per lane: lane l writes LDS bytes [lds_addr + 16 l, + 16); an offset past the descriptor's size writes zeros.
__device__ __forceinline__ void dma16(uint32_t lds_addr, uint32_t voff, u32x4 desc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(desc)
               : "memory");
}

// 4 bytes per lane: lane l writes LDS bytes [lds_addr + 4 l, + 4).
__device__ __forceinline__ void dma4(uint32_t lds_addr, uint32_t voff, u32x4 desc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(desc)
               : "memory");
}

}  // namespace qpl
