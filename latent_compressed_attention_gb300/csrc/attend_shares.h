// What attend_paged.cu's kernels hand each other through the workspace, numbered: plain functions, which a test runs on the
// host as well.
#pragma once

#ifdef __CUDACC__
#define MLA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MLA_HOST_DEVICE inline
#endif

namespace mla {

// A share has at most two parts of tiles that are cut: one of a tile that started before it, one of a tile that starts in it.
MLA_HOST_DEVICE long long part_number(int share, bool starts) { return 2ll * share + (starts ? 1 : 0); }

// Whether a tile's first and last share, as they stand in the workspace, are two that there are, in this order.  Where a wait
// of the kernel before ran out they were never written, and the workspace holds anything.
MLA_HOST_DEVICE bool shares_written(int first, int last, int shares) { return 0 <= first && first <= last && last < shares; }

}  // namespace mla
