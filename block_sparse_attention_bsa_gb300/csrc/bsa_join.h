// Where the join of the paged attention finds a segment's partial results.
// Plain C++, so that a host test can compile it.
#pragma once

#ifdef __CUDACC__
#define BSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BSA_HOST_DEVICE inline
#endif

namespace bsa {

// Partial results of one row of a segment: n of them, `step` rows apart from
// `at` on.
struct Parts {
  int n, at, step;
};

// `first` and `last` are the CTAs that have the segment's first and last tile, as
// the main kernel wrote them to the workspace.  Where a bounded wait of it gave
// up they may not have been written and be any bytes: a pair that no schedule
// makes has no partial results.  `two`: each CTA left two rows (one of each
// softmax group), else one in `half` of its two.
BSA_HOST_DEVICE Parts segment_parts(int first, int last, int ctas, int segment, bool two, int half, int slot_rows,
                                    int row) {
  if (first < 0 || last < first || last >= ctas) return Parts{0, 0, 0};
  return Parts{(last - first + 1) << (two ? 1 : 0), ((segment + first) * 2 + half) * slot_rows + row,
               (two ? 1 : 2) * slot_rows};
}

}  // namespace bsa
