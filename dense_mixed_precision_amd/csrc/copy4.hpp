// copy4.hpp -- direct copies of 4 bytes a lane into LDS, beside kernels.hpp's of
// 16.  Included in its namespace, after it.
#ifndef MPGEMM_COPY4_HPP
#define MPGEMM_COPY4_HPP

// One wave instruction: lane l copies 4 bytes from rsrc at voff into LDS at
// byte address lds_addr + 4*l (see dma16).
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds_addr, uint32_t voff)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 ::"s"(lds_addr), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}

#endif  // MPGEMM_COPY4_HPP
