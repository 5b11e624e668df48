// engram_layers_device.h -- device helpers shared by the layers around the gate:
// memory through buffer descriptors, and straight into LDS (gfx950).
#pragma once

#include "engram_device.h"

namespace engram {

// Memory through a buffer descriptor: a base that all lanes share and a 32-bit
// offset each, below 2 GB; loads from kBeyond give zero and stores to it are
// dropped.
constexpr uint32_t kBeyond = 0xf0000000u;
__device__ __forceinline__ u32x4 buffer_words(const void* p) {
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  return u32x4{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, 0x80000000u, 0x00020000u};
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)0x80000000u, 0x00020000);
}

// 16 bytes a lane from src + off into LDS, lane l's at to + 16 l (`to` shared by
// the wave).  Written in assembly because the compiler, for the builtin, waits
// for every load on its way before a transposing LDS read (the linear layer's
// dx at 8192^3: 1.19 ms instead of 0.84 ms); there is no result register, and
// whoever calls it waits (vmcnt) and meets the other waves before LDS is read.
__device__ __forceinline__ void load_to_lds(uint32_t to, u32x4 src, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(to), "v"(off), "s"(src)
               : "memory");  // m0 is reserved: the compiler itself sets it anew wherever it uses it
}

}  // namespace engram
