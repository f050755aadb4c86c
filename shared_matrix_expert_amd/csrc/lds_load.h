// Direct global -> LDS loads that the compiler does not count (gfx950).
//
// global_load_lds takes its LDS address from m0: lane l's bytes go to m0 + 16 l
// (or 4 l).  The builtin is not used because the compiler, which cannot tell the
// stages of a ring of LDS buffers apart, waits for every such load of its own
// before the next LDS read; the kernels that use these count them themselves (a
// counted s_waitcnt and a barrier).  They have no register output.
//
// m0 is a register that the compiler keeps for itself and an asm statement may not
// name as clobbered, so each load puts back what it held: two scalar moves, which
// cost nothing that shows (16384 x 8192 x 4096 in FP8 472 us a pass with and without
// them, the router's products of 16384 x 512 x 4096 317 and 318 us).
#pragma once

#include "common.h"

namespace em {

// 16 bytes from each lane's own address.
EM_DEV void lds_load16(const void* src, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(src), "s"(dst) : "memory");
}
// 16 (4) bytes from `off` past an address that is the same for the wave.
EM_DEV void lds_load16(const void* base, uint32_t off, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(off), "s"(base), "s"(dst) : "memory");
}
EM_DEV void lds_load4(const void* base, uint32_t off, uint32_t dst) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0) : "v"(off), "s"(base), "s"(dst) : "memory");
}

}  // namespace em
