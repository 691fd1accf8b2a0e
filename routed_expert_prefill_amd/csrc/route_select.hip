// Selection of experts from the scores of a router: sigmoid or softmax scores
// over all experts, a bias that only chooses, groups of experts of which the
// best are kept, the k largest choices and their gates.
//
//   s = sigmoid(z) or softmax(z),  c = s + bias  (s = 0, c = -inf where z = -inf)
//   a group's value: the sum of its group_top largest c (a c of -inf adds nothing)
//   c = -inf outside the top_groups groups of largest value
//   ids: the k largest c, descending;  gates: s of the chosen, over their sum, times scale
//
// Equal values go to the lower index, NaN comes before every number.  The order is
// that of choices in fp64, a gate is formed in fp64 and rounded once.
//
// One wave per token.  Choices are first taken in fp32, with a bound on how far they
// may be off; where every pair of neighbours that decides something (the chosen ones,
// the first one left out, the last group kept and the first one dropped) is further
// apart than that, the order is the one of fp64.  Otherwise, for about one token in two
// thousand of ordinary logits and for ties, the wave does the token again in fp64; and
// for infinities, NaN and too few experts in service a third time, with those cases'
// rules.  (A kernel waits for its slowest wave: with the third form for every such
// token 8192 tokens of 256 experts in groups took 21.0 us.)
//
// Bound by instructions, about 450 to a token: 8192 tokens of 256 experts in groups
// take 10.2 us on MI355X, calls one after another (the kernel 9.6 at the least in a
// trace), of which the 8.4 MB that they read are 1.4 at 6.2 TB/s; one token 4.2 in a
// graph, an empty launch 2.2.  Choices in fp64 only took 35 and 12.8; maxima through
// __shfl_xor, where lanes now move inside the vector instruction, 12.5 (11.4 at the time).  Two and four tokens to a wave, one after the other or in step:
// 13.9 and 17.
#include <math.h>

#include "kernels.h"

namespace moe {

constexpr int kSelThreads = 256;
constexpr int kSelWaves = kSelThreads / kWave;
// Workgroups in x: a grid takes fewer than 2^32 threads in each dimension.
constexpr unsigned kSelLine = 1u << 22;
constexpr int kSelPerLane = 4;  // 64 lanes x 4 >= 256 experts

// v as a number that orders as the choice does: NaN first.  Above 0.
__device__ __forceinline__ unsigned long long sel_key(double v) {
  if (v != v) return ~0ull;
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : b | (1ull << 63);
}

// From -709.8 on down exp(-z) overflows, where the score is a subnormal number still,
// down to -745: there it is exp(z), which is less than a step off from -37 on.  (Not
// from there, where fp32 logits lie so near that the two formulas' roundings could turn
// their order; at -700 neighbours are 6e-5 of a score apart.)
__device__ __forceinline__ double sel_sigmoid(double z) {
  const bool far = z <= -700.0;
  const double e = exp(far ? z : -z);
  return far ? e : 1.0 / (1.0 + e);
}

__device__ __forceinline__ double sel_wave_sum(double v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Any token, in fp64: lane l holds experts l, l + 64, l + 128, l + 192.
__device__ __forceinline__ void select_any(const SelectArgs &a, long long t, double *choice) {
  const int lane = lane_id();
  const int per = a.E / a.groups;
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
      s[i] = a.softmax ? exp(s[i] - top) : sel_sigmoid(s[i]);
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
    for (int i = 0; i < kSelPerLane; ++i) choice[lane + kWave * i] = c[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // lane g: the value of group g, its two largest choices in order of keys
    double v = 0.0;
    if (lane < a.groups) {
      double one = -INFINITY, two = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double x = choice[lane * per + i];
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

// v as the lane that CTRL names has it; lanes of rows outside ROWS keep their own.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float sel_dpp(float v) {
  const int b = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(b, b, CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double sel_dpp(double v) {
  const int lo = __double2loint(v), hi = __double2hiint(v);
  return __hiloint2double(__builtin_amdgcn_update_dpp(hi, hi, CTRL, ROWS, 0xf, false),
                          __builtin_amdgcn_update_dpp(lo, lo, CTRL, ROWS, 0xf, false));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;  // within 16 lanes
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;  // lane 15 (31) to the 16 (32) lanes behind

__device__ __forceinline__ float sel_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double sel_lane(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ double sel_max(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double sel_min(double a, double b) { return fmin(a, b); }
// (in fp32 the instruction itself: fmaxf and fminf quiet each operand first, and a
// lane move of theirs is one more)
__device__ __forceinline__ float sel_max(float a, float b) {
  asm("v_max_f32 %0, %0, %1" : "+v"(a) : "v"(b));
  return a;
}

// The largest of the wave's values, in scalar registers.
__device__ __forceinline__ double sel_wave_max(double v) {
  v = sel_max(v, sel_dpp<kXor1>(v));
  v = sel_max(v, sel_dpp<kXor2>(v));
  v = sel_max(v, sel_dpp<kHalfMirror>(v));
  v = sel_max(v, sel_dpp<kMirror>(v));
  v = sel_max(v, sel_dpp<kBcast15, 0xa>(v));
  v = sel_max(v, sel_dpp<kBcast31, 0xc>(v));
  return sel_lane(v, kWave - 1);
}
// (s_nop 1: two wait states between a vector instruction and a lane move of its result)
#define MOE_DPP_ALL " row_mask:0xf bank_mask:0xf\n\ts_nop 1\n\t"
__device__ __forceinline__ float sel_wave_max(float v) {
  asm("s_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 quad_perm:[1,0,3,2]" MOE_DPP_ALL
      "v_max_f32_dpp %0, %0, %0 quad_perm:[2,3,0,1]" MOE_DPP_ALL
      "v_max_f32_dpp %0, %0, %0 row_half_mirror" MOE_DPP_ALL
      "v_max_f32_dpp %0, %0, %0 row_mirror" MOE_DPP_ALL
      "v_max_f32_dpp %0, %0, %0 row_bcast:15 row_mask:0xa bank_mask:0xf\n\ts_nop 1\n\t"
      "v_max_f32_dpp %0, %0, %0 row_bcast:31 row_mask:0xc bank_mask:0xf\n\ts_nop 1"
      : "+v"(v));
  return sel_lane(v, kWave - 1);
}

__device__ __forceinline__ float sel_wave_sum(float v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// The two largest of 2 * 2 values in descending pairs.
__device__ __forceinline__ void sel_merge(double &one, double &two, double o1, double o2) {
  two = sel_max(sel_min(one, o1), sel_max(two, o2));
  one = sel_max(one, o1);
}
__device__ __forceinline__ void sel_merge(float &one, float &two, float o1, float o2) {
  float low = one;
  asm("v_min_f32 %0, %0, %1" : "+v"(low) : "v"(o1));
  two = sel_max(low, sel_max(two, o2));
  one = sel_max(one, o1);
}
// The same with the pair of the lane that CTRL names.
#define MOE_SEL_MERGE(NAME, CTRL, HOW)                                                 \
  __device__ __forceinline__ void NAME(double &one, double &two) {                     \
    sel_merge(one, two, sel_dpp<CTRL>(one), sel_dpp<CTRL>(two));                       \
  }                                                                                    \
  __device__ __forceinline__ void NAME(float &one, float &two) {                       \
    float low;                                                                         \
    asm("s_nop 1\n\t"                                                                  \
        "v_min_f32_dpp %2, %0, %0 " HOW " row_mask:0xf bank_mask:0xf\n\t"              \
        "v_max_f32_dpp %1, %1, %1 " HOW " row_mask:0xf bank_mask:0xf\n\t"              \
        "v_max_f32_dpp %0, %0, %0 " HOW " row_mask:0xf bank_mask:0xf\n\t"              \
        "v_max_f32 %1, %1, %2"                                                         \
        : "+v"(one), "+v"(two), "=&v"(low));                                           \
  }
MOE_SEL_MERGE(sel_merge_xor1, kXor1, "quad_perm:[1,0,3,2]")
MOE_SEL_MERGE(sel_merge_xor2, kXor2, "quad_perm:[2,3,0,1]")
MOE_SEL_MERGE(sel_merge_half, kHalfMirror, "row_half_mirror")
MOE_SEL_MERGE(sel_merge_row, kMirror, "row_mirror")
#undef MOE_SEL_MERGE

// A token with choices in fp32 or fp64: lane l holds experts 4 l .. 4 l + 3.  False,
// and nothing written, where fp32 does not tell the order of fp64, and for NaN,
// infinities and a token with too few experts in service.
//
// How far an fp32 score may be off, with an exponential and 1 / x of a step (2^-23)
// each and the argument's, 0.61 |z| of them (the product with log2 e, and that
// constant's own): a sigmoid by 2^-23 (s (1 - s)
// (0.61 |z| + 1) + 1.5 s), below 1.57 x 2^-23; a softmax score by 27 x 2^-24 of the largest
// (its argument s |d| / top <= 0.37, the sum of 256 with its own arguments' 5.5), below
// 2^-19.  The bias' addition rounds once more.
template <bool SOFTMAX, typename R>
__device__ __forceinline__ bool select_fast(const SelectArgs &a, long long t, R *choice) {
  constexpr bool F64 = sizeof(R) == 8;
  constexpr R kNone = -INFINITY;
  const int lane = lane_id();
  float z[4];
  const size_t row = (size_t)t * a.E;
  const int e0 = lane * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = -INFINITY;
  if (a.E % 4 == 0) {
    if (e0 < a.E) {
      if (a.f32) {
        const float *from = static_cast<const float *>(a.logits) + row + e0;
        const f32x4 v = *reinterpret_cast<const f32x4 *>(from);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = v[i];
      } else {
        const uint16_t *from = static_cast<const uint16_t *>(a.logits) + row + e0;
        const uint2 v = *reinterpret_cast<const uint2 *>(from);
        z[0] = __uint_as_float(v.x << 16);
        z[1] = __uint_as_float(v.x & 0xffff0000u);
        z[2] = __uint_as_float(v.y << 16);
        z[3] = __uint_as_float(v.y & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < a.E)
        z[i] = a.f32 ? static_cast<const float *>(a.logits)[row + e0 + i]
                     : bf16_bits_to_f32(static_cast<const uint16_t *>(a.logits)[row + e0 + i]);
  }
  R x[4];
  float top = 0.f, off = 0x1.ap-23f, most = 1.f;
  double sum = 0.0;  // fp64 softmax
  if (SOFTMAX) {
    top = sel_wave_max(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
    R part = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F64)
        x[i] = exp((double)z[i] - (double)top);
      else
        x[i] = __expf(z[i] - top);  // 0 for -inf
      part += x[i];
    }
    if constexpr (F64) {
      sum = sel_wave_sum(part);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] /= sum;
    } else {
      most = __builtin_amdgcn_rcpf(sel_wave_sum(part));
      off = most * 0x1p-19f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= most;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F64)
        x[i] = sel_sigmoid(z[i]);
      else
        x[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-z[i]));
    }
  }
  if (a.bias) {
    float large = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e0 + i < a.E) x[i] += (R)a.bias[e0 + i];
      if (!F64 && z[i] != -INFINITY) large = fmaxf(large, fabsf((float)x[i]));
    }
    if (!F64) most = sel_wave_max(large);
  }
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    odd = odd || !(z[i] < INFINITY) || !(x[i] < (R)INFINITY);
    if (z[i] == -INFINITY) x[i] = kNone;
  }
  if (__any(odd)) return false;
  const R apart = F64 ? 0 : 2.0f * off + most * 0x1p-23f;

  // this lane's choices in descending order, equal ones with the lower index first;
  // their places among the four packed alike
  uint32_t place = 0x03020100u;
  auto sort2 = [&](int i, int j) {
    const uint32_t pi = place >> (8 * i) & 0xff, pj = place >> (8 * j) & 0xff;
    const bool swap = x[j] > x[i] || (F64 && x[j] == x[i] && pj < pi);
    const R hi = swap ? x[j] : x[i], lo = swap ? x[i] : x[j];
    x[i] = hi;
    x[j] = lo;
    place ^= swap ? (pi ^ pj) << (8 * i) | (pi ^ pj) << (8 * j) : 0u;
  };
  auto sort4 = [&]() {
    sort2(0, 1);
    sort2(2, 3);
    sort2(0, 2);
    sort2(1, 3);
    sort2(1, 2);
  };
  sort4();

  if (a.groups > 1) {
    const int per = a.E / a.groups, lanes = per / 4;
    const bool runs = per % 4 == 0 && (lanes & (lanes - 1)) == 0;  // of 1, 2, 4 .. 32 lanes
    R one = x[0], two = x[1];
    const int group = runs ? lane / lanes : lane;  // that this lane has the value of
    if (runs) {
      if (lanes >= 2) sel_merge_xor1(one, two);
      if (lanes >= 4) sel_merge_xor2(one, two);
      if (lanes >= 8) sel_merge_half(one, two);
      if (lanes >= 16) sel_merge_row(one, two);
      if (lanes >= 32) sel_merge(one, two, (R)__shfl_xor(one, 16), (R)__shfl_xor(two, 16));
    } else {
      // lane g looks through group g
#pragma unroll
      for (int i = 0; i < 4; ++i) choice[e0 + (place >> (8 * i) & 0xff)] = x[i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      one = two = kNone;
      if (lane < a.groups)
        for (int i = 0; i < per; ++i) sel_merge(one, two, choice[lane * per + i], kNone);
    }
    const R value = a.group_top == 1 || two == kNone ? one : one + two;
    int ahead = 0;
    for (int g = 0; g < a.groups; ++g) {
      const R other = sel_lane(value, runs ? g * lanes : g);
      ahead += other > value || (other == value && g < group);
    }
    const bool is = group < a.groups, keep = is && ahead < a.top_groups;
    if (!F64 && a.top_groups < a.groups) {
      const R low = -sel_wave_max(keep ? -value : kNone);
      const R high = sel_wave_max(is && !keep ? value : kNone);
      // (each of two values: two choices' errors and the rounding of their sum, twice a
      // choice's size)
      if (!(low - high > 2 * apart + most * 0x1p-22f)) return false;
    }
    if (runs) {
      if (!keep) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = kNone;
      }
    } else {
      const unsigned long long kept = __ballot(keep);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = e0 + (int)(place >> (8 * i) & 0xff);
        if (e >= a.E || !((kept >> (e / per)) & 1)) x[i] = kNone;
      }
      sort4();
    }
  }

  bool sure = true;
  R before = INFINITY;
  int id = 0;  // lane j keeps the j-th
  for (int j = 0; j <= a.k; ++j) {
    if (F64 && j == a.k) break;
    const R best = sel_wave_max(x[0]);
    sure = sure && (F64 ? best != kNone : before - best > apart);
    before = best;
    if (j == a.k) break;
    const int from = __ffsll(__ballot(x[0] == best)) - 1;
    const int e = from * 4 + (__builtin_amdgcn_readlane((int)place, from) & 0xff);
    if (lane == j) id = e;
    if (lane == from) {
      x[0] = x[1];
      x[1] = x[2];
      x[2] = x[3];
      x[3] = kNone;
      place >>= 8;
    }
  }
  if (!sure) return false;

  // gates, in fp64 from the logits of the chosen
  double gate = 0.0;
  if (lane < a.k) {
    const size_t at = row + id;
    const double v = a.f32 ? static_cast<const float *>(a.logits)[at]
                           : bf16_bits_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
    gate = SOFTMAX ? exp(v - (double)top) : sel_sigmoid(v);
  }
  if (a.renormalise) {  // at most 16: the first 16 lanes
    double total = gate;
    total += sel_dpp<kXor1>(total);
    total += sel_dpp<kXor2>(total);
    total += sel_dpp<kHalfMirror>(total);
    total += sel_dpp<kMirror>(total);
    gate = total == 0.0 ? 0.0 : gate / total;
  } else if (SOFTMAX) {
    if (!F64) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += exp((double)z[i] - (double)top);
      sum = sel_wave_sum(sum);
    }
    gate /= sum;
  }
  if (lane < a.k) {
    a.ids[(size_t)t * a.k + lane] = id;
    a.gates[(size_t)t * a.k + lane] = (float)(gate * (double)a.scale);
  }
  return true;
}

// (No loop over tokens: the constants of the fp64 exponentials would be kept across
// it, in more scalar registers than there are.)
template <bool SOFTMAX>
__global__ __launch_bounds__(kSelThreads) void route_select_kernel(SelectArgs a) {
  __shared__ double choice[kSelWaves][kSelPerLane * kWave];
  const int wave = threadIdx.x / kWave;
  // the last line of workgroups may end past the tokens
  const long long t = ((long long)blockIdx.y * kSelLine + blockIdx.x) * kSelWaves + wave;
  if (t >= a.T) return;
  if (select_fast<SOFTMAX, float>(a, t, reinterpret_cast<float *>(choice[wave]))) return;
  if (select_fast<SOFTMAX, double>(a, t, choice[wave])) return;
  select_any(a, t, choice[wave]);
}

hipError_t launch_route_select(const SelectArgs &a, hipStream_t stream) {
  const unsigned blocks = ((unsigned)a.T + kSelWaves - 1) / kSelWaves;
  const dim3 grid(blocks < kSelLine ? blocks : kSelLine, (blocks + kSelLine - 1) / kSelLine),
      block(kSelThreads);
  if (a.softmax) return launch(route_select_kernel<true>, grid, block, stream, a);
  return launch(route_select_kernel<false>, grid, block, stream, a);
}

}  // namespace moe
