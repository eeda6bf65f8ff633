// Helpers of the tcgen05 kernels: TMA tile loads, bounded mbarrier waits, commits and
// shared-memory matrix descriptors.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace dfssm {

constexpr long long kTcSpinLimit = 1LL << 24;

// Shared-memory matrix descriptor, K-major, 128-byte swizzle: start address, leading
// byte offset 16 (unused by this layout), stride byte offset 1024, version 1.
DFSSM_DEV uint64_t umma_desc_sw128(uint32_t saddr) {
  return uint64_t((saddr >> 4) & 0x3fffu) | (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// One lane of a converged warp.
DFSSM_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

DFSSM_DEV void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}

// Bounded wait; one that gives up sets `bit` in *status and *fail, which ends the block's
// other waits.
DFSSM_DEV bool tc_wait(uint64_t* bar, unsigned parity, unsigned* status, int* fail, unsigned bit = 65536u) {
  long long spins = 0;
  while (!mbar_try_wait(bar, parity)) {
    if (++spins > kTcSpinLimit || *reinterpret_cast<volatile int*>(fail)) {
      if (spins > kTcSpinLimit && status) atomicOr(status, bit);
      *reinterpret_cast<volatile int*>(fail) = 1;
      return false;
    }
  }
  return true;
}

DFSSM_DEV void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(smem_u32(bar)) : "memory");
}

}  // namespace dfssm
