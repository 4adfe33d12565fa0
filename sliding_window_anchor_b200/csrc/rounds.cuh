// rounds.cuh — rounds of a group of warps that meet at a barrier without a time limit.
// Plain C++: the host compiles it too.
#pragma once

#ifdef __CUDACC__
#define ER_ROUNDS_FN __device__ __forceinline__
#else
#define ER_ROUNDS_FN inline
#endif

namespace er {

// Behind rounds 0 .. n of one member, each with one meeting in front of everything that can
// make the member give up: c is the round that it gave up in, or n + 1.  It meets the others
// in the rounds that it leaves out: members can give up apart from one another (a wait that
// one of them does not make, or that ends just behind its limit), and a barrier waits for
// all of them.
template <class Meet>
ER_ROUNDS_FN void meet_rest(int c, int n, Meet&& meet) {
#pragma unroll 1
  for (++c; c <= n; ++c) meet();
}

}  // namespace er
