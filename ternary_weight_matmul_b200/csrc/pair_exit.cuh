// pair_exit.cuh -- how the two producers of a CTA pair agree on what was issued when a wait has given up.
//
// Each producer numbers its stages (iteration j fills slot j % stages) and may give up at an iteration of
// its own. Stage j's barrier, in the pair's first CTA, is armed by that CTA's producer with both CTAs'
// bytes, so it completes when both have issued j. After both have stopped, each issues what only the other
// one did ([from, to): at most `stages` iterations, and their slots are free, as the other producer saw the
// MMAs that read them complete), and then every barrier of [drain, to) completes: everything older was
// consumed before its slot was filled again.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MMF_HD __host__ __device__ __forceinline__
#else
#define MMF_HD inline
#endif

namespace mmf {

struct PairExit {
  uint32_t from, to;  // iterations this CTA's producer still has to issue
  uint32_t drain;     // first iteration whose barrier is waited for (up to `to`)
};

MMF_HD PairExit pair_exit(uint32_t mine, uint32_t other, uint32_t stages) {
  PairExit e;
  e.from = mine;
  e.to = mine > other ? mine : other;
  e.drain = e.to > stages ? e.to - stages : 0u;
  return e;
}

}  // namespace mmf
