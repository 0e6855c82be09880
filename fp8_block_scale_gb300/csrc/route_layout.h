// How routing by scores lays a token's experts out over a warp (route_scores.cu): plain
// arithmetic without CUDA, so that the host can check every size.
#pragma once

#include <math.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

struct RouteLayout {
  int E, groups, group_size;
  int lanes;        // lanes per group, a power of two: lane = group * lanes + part
  int per;          // experts per lane, in runs of 1 << run
  int run;
};

// bytes: of a logit.  wide: rows and bias start on 16 bytes.
inline RouteLayout route_layout(int E, int groups, int bytes, bool wide) {
  RouteLayout p;
  p.E = E;
  p.groups = groups;
  p.group_size = E / groups;
  p.lanes = 32;
  while (p.lanes * groups > 32) p.lanes /= 2;
  p.run = 0;
  p.per = (p.group_size + p.lanes - 1) / p.lanes;
  // runs of 16 bytes where every group starts on them and they waste no more than a quarter of the places
  const int run = 16 / bytes, padded = (p.group_size + p.lanes * run - 1) / (p.lanes * run) * run;
  if (wide && p.group_size % run == 0 && 4 * padded <= 5 * p.per) {
    p.run = bytes == 4 ? 2 : 3;
    p.per = padded;
  }
  return p;
}

// The places a lane of the kernel that is taken.  In runs: 4, 8, 12, 16, 32, 64 and 128 hold whole runs of four,
// all but 4 and 12 of eight.  More than 64 are needed where a number of groups that is no power of two leaves
// lanes idle: up to 120, for 17 groups of 120 experts.
inline int route_places(const RouteLayout& p) {
  return p.per <= 2 && p.run == 0   ? 2
         : p.per <= 4 && p.run < 3  ? 4
         : p.per <= 8               ? 8
         : p.per <= 9 && p.run == 0 ? 9
         : p.per <= 12 && p.run < 3 ? 12
         : p.per <= 16              ? 16
         : p.per <= 32              ? 32
         : p.per <= 64              ? 64
                                    : 128;
}

// The expert of a lane's i-th place, or -1: a group's lanes take runs of 1 << run experts in turn.
MOE_HOST_DEVICE int route_expert_at(const RouteLayout& p, int i, int lane) {
  const int off = ((((i >> p.run) * p.lanes + lane % p.lanes) << p.run) | (i & ((1 << p.run) - 1))), g = lane / p.lanes;
  return g < p.groups && off < p.group_size ? g * p.group_size + off : -1;
}

// How far a softmax score may be off, in units of 2^-23 of 1 / total (the score of the largest logit), where a
// lane of `places` adds its experts' exponentials.  With x the distance to the largest logit an exponential is off by 2 +
// 1.7 x units of itself (2 + 1.173 x by the hardware's, x / 2 from the rounding of x), and so is a score,
// most at x = 0.  Below it stand the total's errors: its terms', 2 + 1.7 times the average of x over the softmax;
// half a unit for each of places + 5 additions; the reciprocal's 1 and the product's half.  That average is at most
// W((E - 1) / e), of E - 1 experts at one distance (W: Lambert's, W(y) <= ln((y + e^3) / 4)).  One unit to spare.
inline float route_softmax_units(int E, int places) {
  const double average = log((static_cast<double>(E) / 2.718281828459045 + 20.085536923187668) / 4.0);
  return static_cast<float>(2.0 + (2.0 + 1.7 * average) + 0.5 * (places + 5) + 1.5 + 1.0);
}

}  // namespace moe
