// sbl_b8_device.cuh -- device-side building blocks of the 8-bit block kernels
// beside those of sbl_device.cuh.
#pragma once

#include "sbl_device.cuh"

namespace sbl {

// Bit of the device error word (the others: sbl_device.cuh).
constexpr uint32_t kErrB8Gemm = 1u << 6;

// mbar_wait that reads the clock only after some tries: a read of the global
// timer takes longer than most waits of the issuing warp.
__device__ __forceinline__ bool mbar_wait_spin(uint32_t bar, uint32_t parity, uint32_t *err, uint32_t code)
{
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity, err, code);
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Programmatic dependent launch.  Kernels that use this let their dependents
// start only after their own wait, so when a kernel follows one of them,
// everything before that predecessor is complete when it starts.  One that
// needs nothing from its predecessor may therefore work at once and wait at its
// end instead (`late`), where the wait keeps that promise for the kernel after
// it.  It must read global memory past L1 (TMA, ld.cg).
__device__ __forceinline__ void grid_wait_and_release()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace sbl
