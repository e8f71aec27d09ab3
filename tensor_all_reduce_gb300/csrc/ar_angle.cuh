// Angles of the rotation by position (how exact they are: ar_rope.cu).
#pragma once

#include <stdint.h>

namespace ar {

// Fraction of a turn a position, in units of 2^-64 turns (modulo 1).
__device__ __forceinline__ unsigned long long turn_of(float inv_freq) {
  double t = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= floor(t);
  return (unsigned long long)(t * 18446744073709549568.0);  // t < 1; 2^64 less one ulp keeps it in range
}

__device__ __forceinline__ void angle(unsigned long long turn, int pos, float* s, float* c) {
  const unsigned long long a = turn * (unsigned long long)(long long)pos;
  const int top = (int)(unsigned)((a + 0x80000000ull) >> 32);  // [-0.5, 0.5) turns in units of 2^-32
  sincospif((float)top * 0x1p-31f, s, c);                      // 2 pi turns = pi * (2 turns)
}

// The position axis of frequency i (P: axes, sections and dealt of a call).
template <class P>
__device__ __forceinline__ int axis_of(const P& p, int i) {
  if (p.axes == 1) return 0;
  if (!p.dealt) {
    int a = 0;
    for (int end = p.sections[0]; a < p.axes - 1 && i >= end;) end += p.sections[++a];
    return a;
  }
  // round k deals one frequency to each axis whose section is longer than k; all rounds up to the
  // end of the shortest section left at once
  int left = i, done = 0;
  for (int phase = 0; phase < p.axes; ++phase) {
    int shortest = 0x7fffffff, open = 0;
    for (int a = 0; a < p.axes; ++a)
      if (p.sections[a] > done) {
        ++open;
        shortest = min(shortest, p.sections[a]);
      }
    if (open == 0) break;
    if (left < (shortest - done) * open) {
      int nth = left % open;
      for (int a = 0; a < p.axes; ++a)
        if (p.sections[a] > done && nth-- == 0) return a;
    }
    left -= (shortest - done) * open;
    done = shortest;
  }
  return 0;
}

}  // namespace ar
