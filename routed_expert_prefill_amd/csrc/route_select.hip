// Selection of experts from the scores of a router: sigmoid or softmax scores
// over all experts, a bias that only chooses, groups of experts of which the
// best are kept, the k largest choices and their gates.
//
//   s = sigmoid(z) or softmax(z),  c = s + bias  (s = 0, c = -inf where z = -inf)
//   a group's value: the sum of its group_top largest c (a c of -inf adds nothing)
//   c = -inf outside the top_groups groups of largest value
//   ids: the k largest c, descending;  gates: s of the chosen, over their sum, times scale
//
// Equal values go to the lower index, NaN comes before every number.  All of it
// is taken in fp64, so that neighbours in the order stand in the order of the
// formulas; a gate is rounded once.
//
// One wave per token: lane l holds experts l, l + 64, l + 128, l + 192.
#include <math.h>

#include "kernels.h"

namespace moe {

constexpr int kSelThreads = 256;
constexpr int kSelWaves = kSelThreads / kWave;
constexpr int kSelPerLane = 4;  // 64 lanes x 4 >= 256 experts

// v as a number that orders as the choice does: NaN first.  Above 0.
__device__ __forceinline__ unsigned long long sel_key(double v) {
  if (v != v) return ~0ull;
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

__device__ __forceinline__ double sel_wave_sum(double v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__global__ __launch_bounds__(kSelThreads) void route_select_kernel(SelectArgs a) {
  __shared__ double choice[kSelWaves][kSelPerLane * kWave];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int per = a.E / a.groups;
  const long long nwaves = (long long)gridDim.x * kSelWaves;
  for (long long t = (long long)blockIdx.x * kSelWaves + wave; t < a.T; t += nwaves) {
    double s[kSelPerLane], c[kSelPerLane];
    double top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kSelPerLane; ++i) {
      const int e = lane + kWave * i;
      s[i] = -INFINITY;  // no expert, as one out of service
      if (e < a.E) {
        const size_t at = (size_t)t * a.E + e;
        s[i] = a.f32 ? (double)static_cast<const float *>(a.logits)[at]
                     : (double)bf16_bits_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
      }
      top = fmax(top, s[i]);
    }
    if (a.softmax) {
#pragma unroll
      for (int m = kWave / 2; m > 0; m >>= 1) top = fmax(top, __shfl_xor(top, m));
    }
    double sum = 0.0;
    bool gone[kSelPerLane];
#pragma unroll
    for (int i = 0; i < kSelPerLane; ++i) {
      gone[i] = s[i] == -INFINITY;
      if (gone[i])
        s[i] = 0.0;
      else
        s[i] = a.softmax ? exp(s[i] - top) : 1.0 / (1.0 + exp(-s[i]));
      sum += s[i];
    }
    if (a.softmax) {
      sum = sel_wave_sum(sum);
#pragma unroll
      for (int i = 0; i < kSelPerLane; ++i)
        if (!gone[i]) s[i] /= sum;
    }
#pragma unroll
    for (int i = 0; i < kSelPerLane; ++i) {
      const int e = lane + kWave * i;
      c[i] = gone[i] ? -INFINITY : s[i] + (a.bias ? (double)a.bias[e] : 0.0);
    }
    if (a.groups > 1) {
#pragma unroll
      for (int i = 0; i < kSelPerLane; ++i) choice[wave][lane + kWave * i] = c[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // lane g: the value of group g, its two largest choices in order of keys
      double v = 0.0;
      if (lane < a.groups) {
        double one = -INFINITY, two = -INFINITY;
        for (int i = 0; i < per; ++i) {
          const double x = choice[wave][lane * per + i];
          if (sel_key(x) > sel_key(one)) {
            two = one;
            one = x;
          } else if (sel_key(x) > sel_key(two)) {
            two = x;
          }
        }
        v = a.group_top == 1 || two == -INFINITY ? one : one + two;
      }
      const unsigned long long mine = sel_key(v);
      int ahead = 0;
      for (int g = 0; g < a.groups; ++g) {
        const unsigned long long other = __shfl(mine, g);
        ahead += other > mine || (other == mine && g < lane);
      }
      const unsigned long long kept = __ballot(lane < a.groups && ahead < a.top_groups);
#pragma unroll
      for (int i = 0; i < kSelPerLane; ++i) {
        const int e = lane + kWave * i;
        if (e < a.E && !((kept >> (e / per)) & 1)) c[i] = -INFINITY;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // read before the next token's
    }
    unsigned long long key[kSelPerLane];
#pragma unroll
    for (int i = 0; i < kSelPerLane; ++i) key[i] = lane + kWave * i < a.E ? sel_key(c[i]) : 0;
    double gate = 0.0;  // lane j keeps the j-th
    for (int j = 0; j < a.k; ++j) {
      unsigned long long bk = 0;
      int bi = 0x7fffffff;
      double bs = 0.0;
#pragma unroll
      for (int i = 0; i < kSelPerLane; ++i) {
        if (key[i] > bk) {
          bk = key[i];
          bi = lane + kWave * i;
          bs = c[i] == -INFINITY ? 0.0 : s[i];
        }
      }
#pragma unroll
      for (int m = 1; m < kWave; m <<= 1) {
        const unsigned long long ok = __shfl_xor(bk, m);
        const int oi = __shfl_xor(bi, m);
        const double os = __shfl_xor(bs, m);
        if (ok > bk || (ok == bk && oi < bi)) {
          bk = ok;
          bi = oi;
          bs = os;
        }
      }
#pragma unroll
      for (int i = 0; i < kSelPerLane; ++i)
        if (lane + kWave * i == bi) key[i] = 0;
      if (lane == j) gate = bs;
      if (lane == 0) a.ids[(size_t)t * a.k + j] = bi;
    }
    if (a.renormalise) {
      double total = 0.0;
      for (int j = 0; j < a.k; ++j) total += __shfl(gate, j);
      gate = total == 0.0 ? 0.0 : gate / total;
    }
    if (lane < a.k) a.gates[(size_t)t * a.k + lane] = (float)(gate * (double)a.scale);
  }
}

hipError_t launch_route_select(const SelectArgs &a, int grid_cap, hipStream_t stream) {
  const long long want = ((long long)a.T + kSelWaves - 1) / kSelWaves;
  const int grid = (int)(want < grid_cap ? want : grid_cap);
  return launch(route_select_kernel, dim3(grid), dim3(kSelThreads), stream, a);
}

}  // namespace moe
