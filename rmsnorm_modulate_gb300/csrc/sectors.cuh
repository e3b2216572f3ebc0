// Loads and stores of 32 bytes.
#pragma once

#include "device_common.cuh"

namespace rmsmod {

// 32 bytes (a whole sector) at once where rows start on 32 bytes, else 16 and 16.
__device__ __forceinline__ void load_pair(const uint4* p, bool both, bool wide, uint4* v)
{
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                       "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
    } else {
        v[0] = ld_stream(p);
        if (both)
            v[1] = ld_stream(p + 1);
    }
}

__device__ __forceinline__ void store_pair(uint4* p, bool both, bool wide, const uint4 (&v)[2])
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0].x),
                     "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
                     "r"(v[1].w)
                     : "memory");
    } else {
        st_stream(p, v[0]);
        if (both)
            st_stream(p + 1, v[1]);
    }
}

}  // namespace rmsmod
