// ssm_sequences.h -- which sequences of a packed call run, and how many segments
// they come to.  Plain C++ for host and device: the workspace is sized by the one
// and addressed by the other, whatever cu_seqlens holds.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define SSM_HD __host__ __device__ __forceinline__
#else
#define SSM_HD inline
#endif

namespace ssm {

// A sequence [t0, t1) runs if it lies within the tokens and cu_seqlens does not go back at
// it or before it.  (Each by itself would not do: after a step back sequences may lie over
// earlier ones, and come to more segments and outputs than there are tokens.)
SSM_HD bool goes_back(int t0, int t1) { return t1 < t0; }
SSM_HD bool within(int t0, int t1, int64_t tokens) { return t0 >= 0 && t1 >= t0 && t1 <= tokens; }

// Segments of `seg` tokens that a sequence is cut into, one at least.
SSM_HD uint32_t segments_of(uint32_t len, uint32_t seg) { return len <= seg ? 1u : (len + seg - 1u) / seg; }

// No call comes to more: each sequence has at most its whole segments and one, and the
// whole segments of disjoint sequences fit into the tokens.
SSM_HD int64_t segments_at_most(int64_t tokens, uint32_t seg, int num_seqs) { return tokens / seg + num_seqs; }

}  // namespace ssm
