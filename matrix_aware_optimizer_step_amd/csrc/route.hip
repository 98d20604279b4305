// Routing of tokens to experts (include/muon355.h has the definition).
//
//   s = softmax(z) or sigmoid(z);  chosen = the k largest of s + bias among the
//   best groups;  w_j = scale * s_j, over the chosen ones' sum if renormalised
//
// and the order of the (token, expert) pairs by expert.
//
// A token is 16 lanes with V logits each, so that four tokens share a wave and
// every reduction is four rotations inside a row of lanes.  The k best are
// taken one after the other: the largest key of all lanes, then the lowest
// expert that has it.
//
// Equal inputs to the comparison give equal answers whatever the arithmetic:
// where the keys are the logits themselves (no bias, one group or groups by
// their best) they are compared as they are.  Where they are scores, rounded
// to fp32, a token in which two keys that decide something lie within the
// rounding is done again in fp64, one token in a thousand.
//
// The order by expert needs no sort and no atomics on global memory: a token
// chooses an expert at most once, so 64 tokens are one 64-bit mask for each
// expert, and a pair's place among them is the number of bits below its own.

#include "block_internal.h"

namespace muon {
namespace {

constexpr int kLanes = 16;
constexpr int kRouteThreads = kRouteTokens * kLanes;
constexpr int kPlanTokens = 256;  // tokens of a workgroup of the second kernel
constexpr float kNear = 4e-6f;    // of a key's terms: more than two scores' rounding errors

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
// Over a row of 16 lanes, in every one of them.
template <typename T>
__device__ __forceinline__ T row_max(T x) {
  T y;
  y = rotated<0x128>(x); x = x > y ? x : y;
  y = rotated<0x124>(x); x = x > y ? x : y;
  y = rotated<0x122>(x); x = x > y ? x : y;
  y = rotated<0x121>(x); return x > y ? x : y;
}
__device__ __forceinline__ int row_min(int x) {
  x = min(x, rotated<0x128>(x));
  x = min(x, rotated<0x124>(x));
  x = min(x, rotated<0x122>(x));
  return min(x, rotated<0x121>(x));
}
template <typename T>
__device__ __forceinline__ T row_sum(T x) {
  x += rotated<0x128>(x);
  x += rotated<0x124>(x);
  x += rotated<0x122>(x);
  return x + rotated<0x121>(x);
}

__device__ __forceinline__ float exponential(float x) { return expf(x); }
__device__ __forceinline__ double exponential(double x) { return exp(x); }
template <typename T>
__device__ __forceinline__ T sigmoid(T z) {
  const T e = exponential(z < 0 ? z : -z);
  return z < 0 ? e / (T(1) + e) : T(1) / (T(1) + e);
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

// What a token's 16 lanes found: lane j has the j-th best.
struct Choice {
  int expert;   // -1: none
  float z;
  bool near;    // two keys that decide something are too close for their type
};

// The k best of a token.  T: type of the keys; SCORES: the keys are scores
// (plus bias), else the logits.  `shared`: LDS floats of this token's own
// (2 * kMaxExpertGroups of T).
template <typename T, int V, bool SCORES>
__device__ __forceinline__ Choice choose(const RouteArgs& a, const float* z, const float* bias, int lane, T* shared) {
  const int first = lane * V;
  T key[V];
  float widest = 0.0f;  // largest bias
  if (SCORES) {
    T scale = T(1), top = T(0);
    if (!a.sigmoid) {
      float m = z[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = z[v] > m ? z[v] : m;
      top = row_max(m);
      T sum = T(0);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        key[v] = exponential(T(z[v]) - top);
        sum += key[v];
      }
      scale = T(1) / row_sum(sum);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = a.sigmoid ? sigmoid(T(z[v])) : key[v] * scale;
      if (a.bias) {
        key[v] += T(bias[v]);
        widest = fmaxf(widest, fabsf(bias[v]));
      }
      if (z[v] == -inf()) key[v] = -T(inf());
    }
    if (a.bias) widest = row_max(widest);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = T(z[v]);
  }
  bool near = false;
  if (a.groups > 1) {
    // the two best of each group: lanes own runs of experts that may cross
    // group borders, so every lane offers its best two of each group it holds
    const int size = a.experts / a.groups;
    const int g0 = first / size, in0 = first - g0 * size;  // group of the lane's first expert, and its place there
    for (int g = 0; g < a.groups; ++g) {
      T b1 = -T(inf()), b2 = -T(inf());
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int in = first + v - g * size;
        if (in >= 0 && in < size) {
          if (key[v] > b1) {
            b2 = b1;
            b1 = key[v];
          } else if (key[v] > b2) {
            b2 = key[v];
          }
        }
      }
      const T m1 = row_max(b1);
      T score = m1;
      if (a.group_best > 1) {
        const int who = row_min(b1 == m1 ? lane : kLanes);  // the lane whose best is the group's
        const T m2 = row_max(lane == who ? b2 : b1);
        if (m2 > -T(inf())) score = m1 + m2;
      }
      shared[g] = score;  // every lane writes the same value
    }
    __builtin_amdgcn_wave_barrier();
    // a group stays if fewer than top_groups are better (or equal and before it)
    uint32_t kept = 0;
    T low = T(inf()), high = -T(inf());  // worst kept, best dropped
    for (int g = 0; g < a.groups; ++g) {
      const T mark = shared[g];
      int ahead = 0;
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
    if (SCORES && high > -T(inf()) && low - high <= T(2 * kNear) * (fabs(static_cast<float>(low)) + 2 * widest))
      near = true;
    int g = g0, in = in0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!(kept >> g & 1u) || first + v >= a.experts) key[v] = -T(inf());
      if (++in == size) {
        in = 0;
        ++g;
      }
    }
  }
  Choice c;
  c.expert = -1;
  c.z = 0.0f;
  T before = T(0);
  float z_before = 0.0f, b_before = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    T best = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
    best = row_max(best);
    if (!(best > -T(inf()))) break;  // the same in all 16 lanes
    int at = V;
    float zv = 0.0f, bv = 0.0f;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (key[v] == best) {
        at = v;
        zv = z[v];
        if (SCORES && a.bias) bv = bias[v];
      }
    const int expert = row_min(at < V ? first + at : 1 << 30);
    const bool mine = at < V && first + at == expert;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (mine && v == at) key[v] = -T(inf());
    if (SCORES) {
      zv = row_max(mine ? zv : -inf());
      if (a.bias) bv = row_max(mine ? bv : -inf());
      if (j > 0 && before - best <= T(kNear) * (fabs(static_cast<float>(best)) + widest) &&
          !(zv == z_before && bv == b_before))
        near = true;
      before = best;
      z_before = zv;
      b_before = bv;
    } else {
      zv = static_cast<float>(best);
    }
    if (lane == j) {
      c.expert = expert;
      c.z = zv;
    }
  }
  if (SCORES && sizeof(T) == 4) {  // and the last one against everything that is left
    bool close = false;
#pragma unroll
    for (int v = 0; v < V; ++v)
      close = close || (key[v] > -T(inf()) && before - key[v] <= T(kNear) * (fabs(static_cast<float>(before)) + widest) &&
                        !(z[v] == z_before && (!a.bias || bias[v] == b_before)));
    near = near || row_max(close ? 1 : 0);
  }
  c.near = near;
  return c;
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
    if (a.align > 1)
      for (int e = block; e < a.experts; e += blocks)
        for (int r = base[e] + total[e] + threadIdx.x; r < base[e + 1]; r += threads) a.pairs[r] = -1;
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

// 64 tokens in a workgroup of 64 * 16 lanes, or of half as many in two passes
// (V = 32: the registers).
template <int V>
constexpr int kThreadsOf = V > 16 ? kRouteThreads / 2 : kRouteThreads;

template <int V, bool SCORES>
__global__ __launch_bounds__(kThreadsOf<V>) void route_kernel(const RouteArgs a) {
  constexpr int kThreads = kThreadsOf<V>;
  __shared__ uint64_t mask[kMaxExperts];
  __shared__ int total[kMaxExperts], base[kMaxExperts + 1];
  __shared__ int16_t found[kRouteTokens][kMaxChosen];
  __shared__ double marks[kThreads / kLanes][SCORES ? kMaxExpertGroups : kMaxExpertGroups / 2];
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t token0 = static_cast<int64_t>(blockIdx.x) * kRouteTokens;
  const bool plan = a.slots || a.loads;
  for (int e = threadIdx.x; e < a.experts; e += kThreads) mask[e] = 0;
  __syncthreads();
  float bias[V];
  bool bad_bias = false;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = SCORES && a.bias && lane * V + v < a.experts ? a.bias[lane * V + v] : 0.0f;
    bad_bias = bad_bias || bias[v] != bias[v];
  }
#pragma unroll 1
  for (int local = threadIdx.x / kLanes; local < kRouteTokens; local += kThreads / kLanes) {
    const int64_t token = token0 + local;
    if (token >= a.tokens) break;
    const bool there = !a.mask || a.mask[token];
    float z[V];
    bool bad = false;
    if (there) {
      load<V>(z, a.logits + token * a.ld * (a.dtype ? 2 : 4), a.dtype, lane * V, a.experts);
#pragma unroll
      for (int v = 0; v < V; ++v) bad = bad || z[v] != z[v] || (!a.sigmoid && z[v] == inf());
      bad = row_max(bad || bad_bias ? 1 : 0) != 0;
    }
    if (!there || bad) {  // nothing is chosen (and the weights are NaN where something is not a number)
#pragma unroll
      for (int v = 0; v < V; ++v) z[v] = -inf();
    }
    Choice c;
    double* own = marks[threadIdx.x / kLanes];
    c = choose<float, V, SCORES>(a, z, bias, lane, reinterpret_cast<float*>(own));
    if constexpr (SCORES) {
      if (__ballot(c.near)) c = choose<double, V, true>(a, z, bias, lane, own);
    }
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
        for (int v = 1; v < V; ++v) m = z[v] > m ? z[v] : m;
      }
      m = row_max(m);
      if (!a.renormalize && m > -inf()) {
        sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) sum += exponential(z[v] - m);
        sum = row_sum(sum);
      }
      if (some) s = exponential(c.z - m) / sum;
    }
    float w = a.scale * s;
    if (a.renormalize) {
      const float sum = row_sum(s);
      w = sum > 0.0f ? a.scale * (s / sum) : 0.0f;
    }
    if (bad) w = __builtin_nanf("");
    if (lane < a.k) {
      a.chosen[token * a.k + lane] = c.expert;
      a.weights[token * a.k + lane] = w;
    }
    found[local][lane] = static_cast<int16_t>(c.expert);
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
    for (int local = threadIdx.x / kLanes; local < a.tokens; local += kThreads / kLanes) {
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

// The pairs' order from the counts of every 64 tokens and the chosen experts.
// Each workgroup sums all counts by itself (they are few and in L2), 16
// experts for a thread.
__global__ __launch_bounds__(1024) void plan_kernel(const RouteArgs a) {
  constexpr int kParts = kPlanTokens / kRouteTokens;
  __shared__ uint64_t mask[kParts][kMaxExperts];
  __shared__ int total[kMaxExperts], before[kMaxExperts], base[kMaxExperts + 1];
  const int tid = threadIdx.x;
  const int wide = (a.experts + 15) & ~15, chunks = wide / 16;  // 1 .. 32 chunks of 16 experts
  const int rows = (a.tokens + kRouteTokens - 1) / kRouteTokens;
  const int own = blockIdx.x * kParts;  // rows before this workgroup's tokens
  for (int e = tid; e < kMaxExperts; e += 1024) {
    total[e] = before[e] = 0;
#pragma unroll
    for (int q = 0; q < kParts; ++q) mask[q][e] = 0;
  }
  __syncthreads();
  {
    // thread = (row, chunk); the sums of its rows as two 16-bit counters a word
    const int per = 1024 / chunks;
    const int chunk = tid % chunks, row = tid / chunks;
    if (row < per) {
      for (int start = 0; start < rows; start += per * 64) {  // 64 rows of 64 tokens fit 16 bits
        uint32_t all[8], low[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) all[i] = low[i] = 0;
        const int end = min(rows, start + per * 64);
#pragma unroll 4
        for (int r = start + row; r < end; r += per) {
          const uint4 u = *reinterpret_cast<const uint4*>(a.counts + static_cast<int64_t>(r) * wide + chunk * 16);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t even = w[i] & 0x00ff00ffu, odd = (w[i] >> 8) & 0x00ff00ffu;
            all[2 * i] += even;
            all[2 * i + 1] += odd;
            if (r < own) {
              low[2 * i] += even;
              low[2 * i + 1] += odd;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = chunk * 16 + 4 * (i / 2) + i % 2;
          if (all[i] & 0xffffu) atomicAdd(&total[e], static_cast<int>(all[i] & 0xffffu));
          if (all[i] >> 16) atomicAdd(&total[e + 2], static_cast<int>(all[i] >> 16));
          if (low[i] & 0xffffu) atomicAdd(&before[e], static_cast<int>(low[i] & 0xffffu));
          if (low[i] >> 16) atomicAdd(&before[e + 2], static_cast<int>(low[i] >> 16));
        }
      }
    }
  }
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanTokens * a.k;
  const int64_t last = min(first + kPlanTokens * a.k, static_cast<int64_t>(a.tokens) * a.k);
  if (a.slots) {
    for (int64_t p = first + tid; p < last; p += 1024) {
      const int e = a.chosen[p];
      const int t = static_cast<int>(p - first) / a.k;
      if (e >= 0)
        atomicOr(reinterpret_cast<uint32_t*>(&mask[t / kRouteTokens][e]) + (t >> 5 & 1), 1u << (t & 31));
    }
  }
  __syncthreads();
  if (tid < 64) scan_rows(total, base, a.experts, a.align);
  __syncthreads();
  if (a.slots) {
    for (int64_t p = first + tid; p < last; p += 1024) {
      const int e = a.chosen[p];
      const int t = static_cast<int>(p - first) / a.k;
      int slot = -1;
      if (e >= 0) {
        slot = base[e] + before[e];
        const int part = t / kRouteTokens;
        for (int q = 0; q < part; ++q) slot += __builtin_popcountll(mask[q][e]);
        slot += __builtin_popcountll(mask[part][e] & ((uint64_t{1} << (t % kRouteTokens)) - 1));
        a.pairs[slot] = static_cast<int32_t>(p);
      }
      a.slots[p] = slot;
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
  if (!a.sigmoid && !a.renormalize) {
    float z[V];
    load<V>(z, row, a.dtype, first, a.experts);
    float m = z[0], sum = 0.0f;
#pragma unroll
    for (int v = 1; v < V; ++v) m = z[v] > m ? z[v] : m;
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
  if (a.sigmoid && e >= 0) {
    float zj;
    if (a.dtype) {
      zj = __builtin_bit_cast(float, static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[e]) << 16);
    } else {
      zj = reinterpret_cast<const float*>(row)[e];
    }
    d *= sigmoid(-zj);
  }
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

template <int V>
void launch_kernel(const RouteArgs& a, bool scores, uint32_t blocks, hipStream_t s) {
  if (scores) {
    route_kernel<V, true><<<blocks, kThreadsOf<V>, 0, s>>>(a);
  } else {
    route_kernel<V, false><<<blocks, kThreadsOf<V>, 0, s>>>(a);
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>((a.tokens + kRouteTokens - 1) / kRouteTokens);
  const bool scores = a.bias || (a.groups > 1 && a.group_best > 1);
  if (a.experts <= 64) {
    launch_kernel<4>(a, scores, blocks, s);
  } else if (a.experts <= 128) {
    launch_kernel<8>(a, scores, blocks, s);
  } else if (a.experts <= 256) {
    launch_kernel<16>(a, scores, blocks, s);
  } else {
    launch_kernel<32>(a, scores, blocks, s);
  }
  if (blocks > 1 && (a.slots || a.loads))
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
