// tmap.h — tensor maps for the kernels' TMA copies (encoded in gemm_tc.cu).
#pragma once

#include "common.cuh"

namespace moe {

namespace tc {

// dims/strides innermost first (strides in bytes, rank-1 of them).
bool make_map(CUtensorMap* m, CUtensorMapDataType dt, const void* base, int rank, const uint64_t* dims,
              const uint64_t* strides_bytes, const uint32_t* box, CUtensorMapSwizzle swz);

}  // namespace tc

}  // namespace moe
