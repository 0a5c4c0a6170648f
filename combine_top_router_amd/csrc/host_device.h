// For rules that kernels and host compilers without HIP share.
#pragma once

#ifdef __HIP__
#define MOE_HOST_DEVICE __host__ __device__
#else
#define MOE_HOST_DEVICE
#endif
