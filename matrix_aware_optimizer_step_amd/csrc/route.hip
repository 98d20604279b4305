// Routing of tokens to experts (include/muon355.h has the definition).
//
//   s = softmax(z) or sigmoid(z);  chosen = the k largest of s + bias among the
//   best groups;  w_j = scale * s_j, over the chosen ones' sum if renormalised
//
// and the order of the (token, expert) pairs by expert.
//
// A token is 16 lanes with V logits each, so that four tokens share a wave and
// every reduction is four rotations inside a row of lanes; or 32 lanes, with one
// exchange of two rows more (launch_route has the rule).  The k best are
// taken one after the other: the largest key of all lanes, then the lowest
// expert that has it.
//
// Equal inputs to the comparison give equal answers whatever the arithmetic:
// where the keys are the logits themselves (no bias, one group or groups by
// their best) they are compared as they are.  Where they are scores, rounded
// to fp32, keys that lie within the rounding of each other and decide something
// are computed again in fp64: the few experts in question, one a lane, put in
// order among themselves; or the whole token, where it is a border between
// groups, or more than 16 experts.  That is a token in a thousand where scores
// and biases are spread, and most of them where many keys are equal or next to
// each other: 5003 tokens of 128 experts take 8 to 9 us with random biases, 8 to
// 14 with multiples of 1e-3 (as the bias's steps make them), and 18 where biases
// are equal and most scores vanish (logits of +-16); of 256 in groups 14 to 15,
// 15 to 31 and 31.
//
// Measured: 65536 tokens, 8 of 128, softmax 30 us for the choice under the profiler
// (each of the eight costs 69 instructions for four tokens; the logits' 34 MB are
// 5 us), 11 for the order, 10 for the gradient (14 where it is not renormalised and
// reads the logits).  5003 tokens, 8 of
// 256 in groups by biased sigmoid scores: 15 and 10.  One token: 5.4.
//
// The order by expert needs no sort and no atomics on global memory: a token
// chooses an expert at most once, so 64 tokens are one 64-bit mask for each
// expert, and a pair's place among them is the number of bits below its own.

#include <type_traits>

#include "block_internal.h"

namespace muon {
namespace {

constexpr int kLanes = 16;
constexpr int kMaxCandidates = 16;
constexpr int kPlanTokens = 256;  // tokens of a workgroup of the second kernel

// Keys of fp32 scores that are further apart than this are in the right order.
// A score is off by 2^-22 of itself (the exponential by an ulp, a sum and a
// quotient by half an ulp each), a softmax also by 0.37 * 2^-24 (its argument's
// rounding, e^-x x <= 0.37), and by its sum's rounding, the same factor for all
// scores of a token: 36 additions at most, 2^-23 * 18, which shifts two keys by
// that times the difference of their biases.  The addition of the bias is off by
// half an ulp of the key.  Twice all that:
__device__ __forceinline__ float margin(float key, float widest) {
  return 6.6e-7f * fabsf(key) + 9.5e-6f * widest + 6e-8f;
}

__device__ __forceinline__ float inf() { return __builtin_inff(); }

template <int CTRL>
__device__ __forceinline__ int rotated(int x) {
  return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float rotated(float x) {
  return __builtin_bit_cast(float, rotated<CTRL>(__builtin_bit_cast(int, x)));
}
template <int CTRL>
__device__ __forceinline__ double rotated(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = rotated<CTRL>(static_cast<int>(u)), hi = rotated<CTRL>(static_cast<int>(u >> 32));
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// x of two neighbouring rows of 16 lanes, in both: a the lower row's, b the upper
// one's.
__device__ __forceinline__ void pair_rows(int x, int& a, int& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void pair_rows(float x, float& a, float& b) {
  int p, q;
  pair_rows(__builtin_bit_cast(int, x), p, q);
  a = __builtin_bit_cast(float, p);
  b = __builtin_bit_cast(float, q);
}
__device__ __forceinline__ void pair_rows(double x, double& a, double& b) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  int p[2], q[2];
  pair_rows(static_cast<int>(u), p[0], q[0]);
  pair_rows(static_cast<int>(u >> 32), p[1], q[1]);
  __builtin_memcpy(&a, p, 8);
  __builtin_memcpy(&b, q, 8);
}
// The larger one (no operand is a NaN: tokens that hold one are set apart).
__device__ __forceinline__ float larger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ int larger(int a, int b) { return max(a, b); }
// f over a row of 16 lanes, or over two of them, in every lane.
template <int LANES, typename T, typename F>
__device__ __forceinline__ T over_lanes(T x, F f) {
  x = f(x, rotated<0x128>(x));
  x = f(x, rotated<0x124>(x));
  x = f(x, rotated<0x122>(x));
  x = f(x, rotated<0x121>(x));
  if (LANES == 16) return x;
  T a, b;
  pair_rows(x, a, b);
  return f(a, b);
}
template <int LANES = kLanes, typename T>
__device__ __forceinline__ T row_max(T x) {
  return over_lanes<LANES>(x, [](T a, T b) { return larger(a, b); });
}
template <int LANES>
__device__ __forceinline__ int row_min(int x) {
  return over_lanes<LANES>(x, [](int a, int b) { return min(a, b); });
}
template <int LANES>
__device__ __forceinline__ uint32_t row_or(uint32_t x) {
  return static_cast<uint32_t>(over_lanes<LANES>(static_cast<int>(x), [](int a, int b) { return a | b; }));
}
template <int LANES = kLanes, typename T>
__device__ __forceinline__ T row_sum(T x) {
  return over_lanes<LANES>(x, [](T a, T b) { return a + b; });
}

__device__ __forceinline__ float exponential(float x) { return expf(x); }
__device__ __forceinline__ double exponential(double x) { return exp(x); }
template <typename T>
__device__ __forceinline__ T sigmoid(T z) {
  const T e = exponential(z < 0 ? z : -z);
  return (z < 0 ? e : T(1)) / (T(1) + e);
}

// V logits of a token from expert first on; -inf behind the last.
template <int V>
__device__ __forceinline__ void load(float* z, const char* row, int dtype, int first, int experts) {
  if (dtype) {
    uint32_t w[V / 2];
    if (first + V <= experts) {
      __builtin_memcpy(w, row + 2 * first, sizeof(w));
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = __builtin_bit_cast(float, v % 2 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        z[v] = first + v < experts
                   ? __builtin_bit_cast(float, static_cast<uint32_t>(
                                                   reinterpret_cast<const uint16_t*>(row)[first + v]) << 16)
                   : -inf();
    }
  } else if (first + V <= experts) {
    __builtin_memcpy(z, row + 4 * first, 4 * V);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) z[v] = first + v < experts ? reinterpret_cast<const float*>(row)[first + v] : -inf();
  }
}

__device__ __forceinline__ float logit(const char* row, int dtype, int e) {
  return dtype ? __builtin_bit_cast(float, static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[e]) << 16)
               : reinterpret_cast<const float*>(row)[e];
}

// fp64 exponentials are not computed side by side: the registers.
template <typename T>
__device__ __forceinline__ void one_by_one() {
  if (sizeof(T) == 8) __builtin_amdgcn_sched_barrier(0);
}

// What a token's lanes found: lane j has the j-th best.
struct Choice {
  int expert;    // -1: none
  float z, bias; // its logit and bias
  int found;     // lanes that hold a candidate: k, or more where some are as near as the k-th
  bool near;     // candidates are close to each other: their order, or who is among the k, needs fp64
  bool again;    // the whole token does
};

// The k best of a token.  T: type of the keys; SCORES: the keys are scores
// (plus bias, `bias` in LDS, `widest` its largest magnitude), else the logits.
// `row`: the token's logits in memory.  `shared`: LDS of this token's own
// (kMaxExpertGroups + 2 * LANES of T).
template <typename T, int V, int LANES, bool SCORES>
__device__ __forceinline__ Choice choose(const RouteArgs& a, const float* z, const float* bias, float widest,
                                         const char* row, int lane, T* shared) {
  const int first = lane * V;
  T key[V];
  if (SCORES) {
    if (a.sigmoid) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        key[v] = sigmoid(T(z[v]));
        one_by_one<T>();
      }
    } else {
      float m = z[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = larger(m, z[v]);
      const T top = row_max<LANES>(m);
      T sum = T(0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        key[v] = exponential(T(z[v]) - top);
        sum += key[v];
        one_by_one<T>();
      }
      const T scale = T(1) / row_sum<LANES>(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] *= scale;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] += T(bias[first + v]);  // (zeros where there is none)
      if (z[v] == -inf()) key[v] = -T(inf());
      one_by_one<T>();
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = T(z[v]);
  }
  bool near = false, again = false;
  if (a.groups > 1) {
    const int size = a.experts / a.groups;
    const int g0 = first / size, in0 = first - g0 * size;  // group of the lane's first expert, and its place there
    if (size % V == 0) {
      // every lane's experts are of one group, a group is size / V lanes: each
      // lane's two best go to LDS, and lane g joins those of group g
      T b1 = key[0], b2 = -T(inf());
#pragma unroll
      for (int v = 1; v < V; ++v) {
        b2 = larger(b2, key[v] < b1 ? key[v] : b1);
        b1 = larger(b1, key[v]);
      }
      T* two = shared + kMaxExpertGroups;
      two[2 * lane] = b1;
      two[2 * lane + 1] = b2;
      __builtin_amdgcn_wave_barrier();
      if (lane < a.groups) {  // (no more groups than lanes)
        const int lanes = size / V;
        b1 = b2 = -T(inf());
        for (int l = lane * lanes; l < (lane + 1) * lanes; ++l) {
          const T x = two[2 * l], y = two[2 * l + 1];
          b2 = larger(larger(b2, y), x < b1 ? x : b1);
          b1 = larger(b1, x);
        }
        shared[lane] = a.group_best > 1 && b2 > -T(inf()) ? b1 + b2 : b1;
      }
    } else {
      // runs of experts that cross group borders: every lane offers its two
      // best of each group
      for (int g = 0; g < a.groups; ++g) {
        T b1 = -T(inf()), b2 = -T(inf());
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int in = first + v - g * size;
          const T x = in >= 0 && in < size ? key[v] : -T(inf());
          b2 = larger(b2, x < b1 ? x : b1);
          b1 = larger(b1, x);
        }
        const T m1 = row_max<LANES>(b1);
        T score = m1;
        if (a.group_best > 1) {
          const int who = row_min<LANES>(b1 == m1 ? lane : LANES);  // the lane whose best is the group's
          const T m2 = row_max<LANES>(lane == who ? b2 : b1);
          if (m2 > -T(inf())) score = m1 + m2;
        }
        shared[g] = score;  // every lane writes the same value
      }
    }
    __builtin_amdgcn_wave_barrier();
    // a group stays if fewer than top_groups are better (or equal and before it);
    // a lane looks at one group or two (all lanes at all groups: 5003 tokens, 8
    // groups of 32, 25 us against 18)
    uint32_t kept = 0;
    T low = T(inf()), high = -T(inf());  // worst kept, best dropped
    for (int g = lane; g < a.groups; g += LANES) {
      const T mark = shared[g];
      int ahead = 0;
#pragma unroll 4
      for (int o = 0; o < a.groups; ++o) {
        const T x = shared[o];
        ahead += x > mark || (x == mark && o < g);
      }
      if (ahead < a.top_groups) {
        kept |= 1u << g;
        low = mark < low ? mark : low;
      } else {
        high = mark > high ? mark : high;
      }
    }
    kept = row_or<LANES>(kept);
    low = -row_max<LANES>(-low);
    high = row_max<LANES>(high);
    if (SCORES && high > -T(inf()) && low - high <= T(2 * margin(static_cast<float>(low), 2 * widest))) again = true;
    int g = g0, in = in0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(kept >> (g & 31) & 1u) || first + v >= a.experts) key[v] = -T(inf());  // (g: a group up to the last expert)
      if (++in == size) {
        in = 0;
        ++g;
      }
    }
  }
  Choice c;
  c.expert = -1;
  T before = T(0);
  int j = 0;
  for (;; ++j) {
    T best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = larger(best, key[v]);
    best = row_max<LANES>(best);
    if (!(best > -T(inf()))) break;  // the same in all lanes
    const bool close = SCORES && sizeof(T) == 4 && j > 0 && before - best <= T(margin(static_cast<float>(best), widest));
    if (j >= a.k && !close) break;
    if (j == kMaxCandidates) {
      again = true;
      break;
    }
    near = near || close;
    int at = V;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) at = key[v] == best ? v : at;
    const int expert = row_min<LANES>(at < V ? first + at : 1 << 30);
    const int taken = first + at == expert ? at : V;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = v == taken ? -T(inf()) : key[v];
    before = best;
    if (lane == j) c.expert = expert;
  }
  c.z = c.bias = 0.0f;
  if (c.expert >= 0) {
    c.z = logit(row, a.dtype, c.expert);
    if (SCORES) c.bias = bias[c.expert];
  }
  c.found = j;
  c.near = near;
  c.again = again;
  return c;
}

// The candidates' order by their keys in fp64, one a lane.
template <int V, int LANES>
__device__ __forceinline__ void put_in_order(const RouteArgs& a, const float* z, Choice& c, int lane, double* shared) {
  double key = -inf();
  if (a.sigmoid) {
    if (lane < c.found) key = sigmoid(static_cast<double>(c.z));
  } else {
    float m = z[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = larger(m, z[v]);
    m = row_max<LANES>(m);
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      sum += exponential(static_cast<double>(z[v]) - m);
      one_by_one<double>();
    }
    sum = row_sum<LANES>(sum);
    if (lane < c.found) key = exponential(static_cast<double>(c.z) - m) / sum;
  }
  key += c.bias;
  int rank = 0;
  shared[lane] = key;
  int* experts = reinterpret_cast<int*>(shared + LANES);
  experts[lane] = c.expert;
  __builtin_amdgcn_wave_barrier();
  for (int o = 0; o < c.found; ++o) {
    const double x = shared[o];
    rank += x > key || (x == key && experts[o] < c.expert);
  }
  __builtin_amdgcn_wave_barrier();
  float* logits = reinterpret_cast<float*>(shared);
  if (lane < c.found) {
    experts[rank] = c.expert;
    logits[rank] = c.z;
  }
  __builtin_amdgcn_wave_barrier();
  if (lane < c.found) {
    c.expert = experts[lane];
    c.z = logits[lane];
  }
}

// Exclusive sums of the experts' rows, each rounded up to `align`, by one
// wave: base[e], and base[experts] behind the last.
__device__ __forceinline__ void scan_rows(const int* total, int* base, int experts, int align) {
  const int lane = threadIdx.x & 63;
  constexpr int kPer = kMaxExperts / 64;
  int own[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    const int n = e < experts ? total[e] : 0;
    own[i] = sum;
    sum += (n + align - 1) / align * align;
  }
  int upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(upto, d);
    if (lane >= d) upto += x;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e < experts) base[e] = upto - sum + own[i];
  }
  if (lane == 63) base[experts] = upto;
}

// What every workgroup of a launch of `blocks` writes of the order besides its
// own pairs: the rows between an expert's last pair and the next expert's
// first, the rows behind the last expert, and (the first one) the offsets and
// the loads.
__device__ __forceinline__ void write_rest(const RouteArgs& a, const int* total, const int* base, int block,
                                           int blocks) {
  const int threads = blockDim.x;
  if (a.pairs) {
    if (a.align > 1) {  // a wave for an expert
      const int waves = threads / 64;
      for (int e = block * waves + (threadIdx.x >> 6); e < a.experts; e += blocks * waves)
        for (int r = base[e] + total[e] + (threadIdx.x & 63); r < base[e + 1]; r += 64) a.pairs[r] = -1;
    }
    for (int64_t r = base[a.experts] + static_cast<int64_t>(block) * threads + threadIdx.x; r < a.capacity;
         r += static_cast<int64_t>(blocks) * threads)
      a.pairs[r] = -1;
  }
  if (block == 0) {
    for (int e = threadIdx.x; e <= a.experts; e += threads) {
      if (a.offsets) a.offsets[e] = base[e];
      if (a.loads && e < a.experts) a.loads[e] += total[e];
    }
  }
}

// TOKENS tokens in a workgroup, of LANES lanes each; 64 tokens of 32 lanes in
// passes of 16 (the registers).
template <int LANES, int TOKENS>
constexpr int kThreadsOf = LANES * (LANES == 16 ? TOKENS : 16);

template <int V, int LANES, int TOKENS, bool SCORES>
__global__ __launch_bounds__((kThreadsOf<LANES, TOKENS>)) void route_kernel(const RouteArgs a) {
  constexpr int kThreads = kThreadsOf<LANES, TOKENS>;
  __shared__ uint64_t mask[kMaxExperts];
  __shared__ int total[kMaxExperts], base[kMaxExperts + 1];
  __shared__ int16_t found[TOKENS][kMaxChosen];
  using Mark = std::conditional_t<SCORES, double, float>;
  __shared__ Mark marks[kThreads / LANES][kMaxExpertGroups + 2 * LANES];
  __shared__ float bias[SCORES ? LANES * V : 1];
  const int lane = threadIdx.x & (LANES - 1);
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * TOKENS;
  const bool plan = a.slots || a.loads;
  for (int e = threadIdx.x; e < a.experts; e += kThreads) mask[e] = 0;
  __syncthreads();
  float widest = 0.0f;
  bool bad_bias = false;
  if (SCORES) {
    for (int e = threadIdx.x; e < LANES * V; e += kThreads) bias[e] = a.bias && e < a.experts ? a.bias[e] : 0.0f;
    __syncthreads();
    for (int v = 0; v < V; ++v) {
      const float b = bias[lane * V + v];
      bad_bias = bad_bias || b != b;
      widest = fmaxf(widest, fabsf(b));
    }
    widest = row_max<LANES>(widest);
  }
#pragma unroll 1
  for (int local = threadIdx.x / LANES; local < TOKENS; local += kThreads / LANES) {
    const int64_t token = token0 + local;
    if (token >= a.tokens) break;
    const bool there = !a.mask || a.mask[token];
    const char* row = a.logits + token * a.ld * (a.dtype ? 2 : 4);
    float z[V];
    bool bad = false;
    if (there) {
      load<V>(z, row, a.dtype, lane * V, a.experts);
#pragma unroll
      for (int v = 0; v < V; ++v) bad = bad || z[v] != z[v] || (!a.sigmoid && z[v] == inf());
      bad = row_max<LANES>(bad || bad_bias ? 1 : 0) != 0;
    }
    if (!there || bad) {  // nothing is chosen (and the weights are NaN where something is not a number)
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = -inf();
    }
    Choice c;
    Mark* own = marks[threadIdx.x / LANES];
    c = choose<float, V, LANES, SCORES>(a, z, bias, widest, row, lane, reinterpret_cast<float*>(own));
    if constexpr (SCORES) {
      if (c.near && !c.again) put_in_order<V, LANES>(a, z, c, lane, own);
      if (c.again) {
        c = choose<double, V, LANES, true>(a, z, bias, widest, row, lane, own);
        load<V>(z, row, a.dtype, lane * V, a.experts);  // (not kept meanwhile: the registers)
      }
    }
    if (lane >= a.k) c.expert = -1;
    // the weights, lane j those of the j-th
    const bool some = c.expert >= 0;
    float s = 0.0f;
    if (a.sigmoid) {
      if (some) s = sigmoid(c.z);
    } else {
      // over the chosen ones' largest logit where they are renormalised: the
      // row's sum falls out
      float m = some ? c.z : -inf(), sum = 1.0f;
      if (!a.renormalize) {
        m = z[0];
#pragma unroll
        for (int v = 1; v < V; ++v) m = larger(m, z[v]);
      }
      m = row_max<LANES>(m);
      if (!a.renormalize && m > -inf()) {
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += exponential(z[v] - m);
        sum = row_sum<LANES>(sum);
      }
      if (some) s = exponential(c.z - m) / sum;
    }
    float w = a.scale * s;
    if (a.renormalize) {
      const float sum = row_sum<LANES>(s);
      w = sum > 0.0f ? a.scale * (s / sum) : 0.0f;
    }
    if (bad) w = __builtin_nanf("");
    if (lane < a.k) {
      a.chosen[token * a.k + lane] = c.expert;
      a.weights[token * a.k + lane] = w;
    }
    if (lane < kMaxChosen) found[local][lane] = static_cast<int16_t>(c.expert);
    if (plan && some) atomicOr(reinterpret_cast<uint32_t*>(&mask[c.expert]) + (local >> 5), 1u << (local & 31));
  }
  if (!plan) return;
  __syncthreads();
  if (gridDim.x > 1) {  // the counts, for the second kernel
    const int wide = (a.experts + 15) & ~15;
    for (int e = threadIdx.x; e < wide; e += kThreads)
      a.counts[static_cast<int64_t>(blockIdx.x) * wide + e] =
          e < a.experts ? static_cast<uint8_t>(__builtin_popcountll(mask[e])) : uint8_t{0};
    return;
  }
  for (int e = threadIdx.x; e < a.experts; e += kThreads) total[e] = __builtin_popcountll(mask[e]);
  __syncthreads();
  if (threadIdx.x < 64) scan_rows(total, base, a.experts, a.align);
  __syncthreads();
  if (a.slots && lane < a.k) {
    for (int local = threadIdx.x / LANES; local < a.tokens; local += kThreads / LANES) {
      const int e = found[local][lane], p = local * a.k + lane;
      int slot = -1;
      if (e >= 0) {
        slot = base[e] + __builtin_popcountll(mask[e] & ((uint64_t{1} << local) - 1));
        a.pairs[slot] = p;
      }
      a.slots[p] = slot;
    }
  }
  write_rest(a, total, base, 0, 1);
}

// The pairs' order from the counts of every a.group tokens and the chosen experts.
// Each workgroup sums all counts by itself (they are few and in L2), eight
// experts a lane.  That is quadratic in the tokens, and why the ABI layer refuses
// more than 2^22 of them.
__global__ __launch_bounds__(1024) void plan_kernel(const RouteArgs a) {
  constexpr int kParts = kPlanTokens / 64;
  __shared__ uint64_t mask[kParts][kMaxExperts];
  __shared__ int total[kMaxExperts], before[kMaxExperts], base[kMaxExperts + 1];
  __shared__ int sums[2][16][kMaxExperts];  // of each wave's rows, all and those before; expert e at (e % 8) * 64 + e / 8
  const int tid = threadIdx.x;
  const int wide = (a.experts + 15) & ~15, words = wide / 8;  // 2 .. 64 words of 8 experts
  const int rows = (a.tokens + a.group - 1) / a.group;
  const int own = blockIdx.x * (kPlanTokens / a.group);  // rows before this workgroup's tokens
  // this workgroup's pairs, kept from here to the end
  constexpr int kPairs = kPlanTokens * kMaxChosen / 1024;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanTokens * a.k;
  const int count = static_cast<int>(min(static_cast<int64_t>(kPlanTokens), a.tokens - static_cast<int64_t>(blockIdx.x) * kPlanTokens)) * a.k;
  int mine[kPairs], local[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int at = tid + i * 1024;
    mine[i] = a.slots && at < count ? a.chosen[first + at] : -1;
    local[i] = at / a.k;
  }
  for (int e = tid; e < kMaxExperts; e += 1024) {
#pragma unroll
    for (int q = 0; q < kParts; ++q) mask[q][e] = 0;
  }
  __syncthreads();
  {
    // A wave takes 64 / lanes rows at a time, a lane a word of each; sums are
    // 16-bit counters, two to a register, joined over the rows of a wave by
    // lane exchanges before a counter can overflow.  (LDS atomics here took
    // half of the kernel's time.)
    int lanes = 2;
    while (lanes < words) lanes *= 2;
    const int lane = tid & 63, wave = tid >> 6, word = lane & (lanes - 1);
    const int step = 16 * (64 / lanes), most = 16 * lanes - 1;  // rows of a pass; passes that fit 16 bits
    int all[8], low[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) all[i] = low[i] = 0;
    for (int start = 0; start < rows; start += step * most) {
      uint32_t x[4] = {0, 0, 0, 0}, y[4] = {0, 0, 0, 0};
      const int end = min(rows, start + step * most);
      // eight loads are in flight together: none depends on a branch
      for (int r = start + wave * (64 / lanes) + lane / lanes; r < end; r += 8 * step) {
        uint2 u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          u[q] = *reinterpret_cast<const uint2*>(a.counts + static_cast<int64_t>(min(r + q * step, rows - 1)) * wide +
                                                 min(word, words - 1) * 8);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t here = r + q * step < end ? 0x00ff00ffu : 0, keep = r + q * step < own ? here : 0;
          const uint32_t w[4] = {u[q].x, u[q].x >> 8, u[q].y, u[q].y >> 8};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] += w[i] & here;
            y[i] += w[i] & keep;
          }
        }
      }
      for (int d = lanes; d < 64; d *= 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] += __shfl_xor(x[i], d);
          y[i] += __shfl_xor(y[i], d);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = i / 4 * 2 + i % 2, shift = i % 4 / 2 * 16;
        all[i] += x[n] >> shift & 0xffffu;
        low[i] += y[n] >> shift & 0xffffu;
      }
    }
    if (lane < lanes) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[0][wave][i * 64 + word] = all[i];
        sums[1][wave][i * 64 + word] = low[i];
      }
    }
  }
  if (a.slots) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (mine[i] >= 0)
        atomicOr(reinterpret_cast<uint32_t*>(&mask[local[i] / 64][mine[i]]) + (local[i] >> 5 & 1), 1u << (local[i] & 31));
  }
  __syncthreads();
  {
    const int e = tid & (kMaxExperts - 1), half = tid / kMaxExperts;
    int sum = 0;
    if (e < a.experts) {
#pragma unroll
      for (int w = 0; w < 16; ++w) sum += sums[half][w][(e & 7) * 64 + (e >> 3)];
    }
    (half ? before : total)[e] = sum;
  }
  __syncthreads();
  if (tid < 64) scan_rows(total, base, a.experts, a.align);
  __syncthreads();
  if (a.slots) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int at = tid + i * 1024;
      if (at >= count) break;
      const int e = mine[i], t = local[i];
      int slot = -1;
      if (e >= 0) {
        slot = base[e] + before[e];
        const int part = t / 64;
        for (int q = 0; q < part; ++q) slot += __builtin_popcountll(mask[q][e]);
        slot += __builtin_popcountll(mask[part][e] & ((uint64_t{1} << (t % 64)) - 1));
        a.pairs[slot] = static_cast<int32_t>(first + at);
      }
      a.slots[first + at] = slot;
    }
  }
  write_rest(a, total, base, blockIdx.x, gridDim.x);
}

// dL/dz from dL/dw.  With G = sum of g_i w_i / scale where the weights are
// renormalised and 0 where not:
//   sigmoid:              dz_j = (g_j - G) w_j (1 - s_j) for the chosen, else 0
//   softmax renormalised: dz_j = (g_j - G) w_j           for the chosen, else 0
//   softmax:              dz_e = g_e w_e - p_e * sum of g_i w_i
// Only the last needs the whole row of logits.
template <int V>
__global__ __launch_bounds__(256) void backward_kernel(const RouteBackwardArgs a) {
  __shared__ float rows[256 / kLanes][kLanes * V];
  const int lane = threadIdx.x & (kLanes - 1), local = threadIdx.x / kLanes;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + local;
  if (token >= a.tokens) return;
  const char* row = a.logits + token * a.ld * (a.dtype ? 2 : 4);
  const int first = lane * V;
  int e = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < a.k) {
    e = a.chosen[token * a.k + lane];
    w = a.weights[token * a.k + lane];
    if (e >= a.experts) e = -1;
    if (e >= 0) g = a.grad[token * a.k + lane];
  }
  float out[V];
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = 0.0f;
  const float gw = row_sum(e >= 0 ? g * w : w * 0.0f);  // (a NaN weight of a token that went nowhere stays)
  // (the logits of a token that went nowhere may be anything: they are not looked at)
  if (!a.sigmoid && !a.renormalize && row_max(e >= 0 ? 1 : 0)) {
    float z[V];
    load<V>(z, row, a.dtype, first, a.experts);
    float m = z[0], sum = 0.0f;
#pragma unroll
    for (int v = 1; v < V; ++v) m = larger(m, z[v]);
    m = row_max(m);
    if (m > -inf()) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        z[v] = exponential(z[v] - m);
        sum += z[v];
      }
      const float f = -gw / row_sum(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = z[v] * f;
    }
  }
  float d = (g - (a.renormalize && a.scale != 0.0f ? gw / a.scale : 0.0f)) * w;
  if (a.sigmoid && e >= 0) d *= sigmoid(-logit(row, a.dtype, e));
  if (gw != gw) {
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = gw;
  }
  // the chosen ones' terms reach their owners through LDS (one wave's accesses
  // are in order)
#pragma unroll
  for (int v = 0; v < V; ++v) rows[local][first + v] = out[v];
  __builtin_amdgcn_wave_barrier();
  if (e >= 0) rows[local][e] += d;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = rows[local][first + v];
  char* to = a.out + token * a.ld_out * (a.dtype ? 2 : 4);
  if (a.dtype) {
    if (first + V <= a.experts) {
      __bf16 b[V];
#pragma unroll
      for (int v = 0; v < V; ++v) b[v] = static_cast<__bf16>(out[v]);
      __builtin_memcpy(to + 2 * first, b, sizeof(b));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (first + v < a.experts) reinterpret_cast<__bf16*>(to)[first + v] = static_cast<__bf16>(out[v]);
    }
  } else if (first + V <= a.experts) {
    __builtin_memcpy(to + 4 * first, out, sizeof(out));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (first + v < a.experts) reinterpret_cast<float*>(to)[first + v] = out[v];
  }
}

// bias <- bias + rate * sign(mean load - load); the loads start again from zero.
__global__ __launch_bounds__(kMaxExperts) void balance_kernel(const BalanceArgs a) {
  __shared__ int64_t part[kMaxExperts / 64];
  const int e = threadIdx.x;
  const int64_t mine = e < a.experts ? a.loads[e] : 0;
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  if ((e & 63) == 0) part[e >> 6] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kMaxExperts / 64; ++w) sum += part[w];
  if (e >= a.experts) return;
  if (!a.control || !a.control->skip) {
    const int64_t scaled = mine * a.experts;  // against the sum: no rounding decides the sign
    a.bias[e] += scaled < sum ? a.rate : scaled > sum ? -a.rate : 0.0f;
  }
  a.loads[e] = 0;
}

bool by_score(const RouteArgs& a) { return a.bias || (a.groups > 1 && a.group_best > 1); }

template <int V, int LANES, int TOKENS>
void launch_kernel(const RouteArgs& a, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>((a.tokens + TOKENS - 1) / TOKENS);
  if (by_score(a)) {
    route_kernel<V, LANES, TOKENS, true><<<blocks, kThreadsOf<LANES, TOKENS>, 0, s>>>(a);
  } else {
    route_kernel<V, LANES, TOKENS, false><<<blocks, kThreadsOf<LANES, TOKENS>, 0, s>>>(a);
  }
}

// 16 tokens in a workgroup while 64 leave compute units without one (5003 tokens
// of 256 experts: 34 us against 63), 64 where the second kernel would have too
// many counts to sum, and where one workgroup does it all.
template <int V, int LANES>
void launch_tokens(const RouteArgs& a, hipStream_t s) {
  a.group == 16 ? launch_kernel<V, LANES, 16>(a, s) : launch_kernel<V, LANES, 64>(a, s);
}

}  // namespace

// 16 lanes a token up to 256 experts, 32 above (512 experts, 5003 tokens: 11 us
// against 32, with a bias 18 against 47; 65536: 72 against 70, 145 against 186).
// With 256 experts and keys that are scores 32 as long as 16 leave a SIMD with two
// waves or fewer (in groups, 500 tokens: 13 us against 18, 5003: 15 against 18, 16384:
// 25 against 23).  A whole wave for a token was slower from 5003 tokens on at any
// size (256 experts in groups: 22).
hipError_t launch_route(const RouteArgs& args, hipStream_t s) {
  RouteArgs a = args;
  a.group = route_group(a.tokens, a.experts);
  if (a.experts <= 64) {
    launch_tokens<4, 16>(a, s);
  } else if (a.experts <= 128) {
    launch_tokens<8, 16>(a, s);
  } else if (a.experts <= 256) {
    if (by_score(a) && a.group == 16 && a.tokens <= 8192) {
      route_kernel<8, 32, 16, true><<<(a.tokens + 15) / 16, kThreadsOf<32, 16>, 0, s>>>(a);
    } else {
      launch_tokens<16, 16>(a, s);
    }
  } else {
    launch_tokens<16, 32>(a, s);
  }
  if (a.tokens > 64 && (a.slots || a.loads))
    plan_kernel<<<(a.tokens + kPlanTokens - 1) / kPlanTokens, 1024, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>((a.tokens + 15) / 16);
  if (a.experts <= 64) {
    backward_kernel<4><<<blocks, 256, 0, s>>>(a);
  } else if (a.experts <= 128) {
    backward_kernel<8><<<blocks, 256, 0, s>>>(a);
  } else if (a.experts <= 256) {
    backward_kernel<16><<<blocks, 256, 0, s>>>(a);
  } else {
    backward_kernel<32><<<blocks, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t s) {
  balance_kernel<<<1, kMaxExperts, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace muon
