// Routing from given logits: scores (sigmoid or softmax), a bias for balance,
// groups of experts, top-k, renormalised weights.  One warp takes a token; a
// lane has PER consecutive experts, a group of experts its own lanes.
//
//   c_e = s_e + b_e; each lane sorts its experts by c; groups by their two best
//   c or the best; then k rounds of a warp's largest head, ties to the lower
//   index.
//
// What bounds it: for many tokens the instructions of the scores and the
// rounds, not the bytes of the logits; for few, the launch.
//
// Keys.  The order of a lane's experts is that of unsigned words: c's bits in
// an order-preserving form, the last four replaced by the expert's place in the
// lane, lower places first.  So a compare and exchange of the sort is a minimum
// and a maximum, and a round one warp maximum and one vote.
//
// The order is that of the real numbers.  Without a bias it is the logits'
// own (both scores grow with them), which needs no score; bf16 logits have
// nothing in the four bits.  Otherwise c is off by at most 2^-21 (sigmoid) or
// 2^-17 (softmax: the rounded argument of exp and the sum) of the largest
// score, half a step of its own and the four bits: where two neighbours in the
// order, or the last group kept and the first dropped, are nearer than twice
// that and not of equal logits and biases, the warp makes the token's choice
// again in 64 bits (exact_choice).  Weights are computed from the chosen
// logits, relative to the largest of them, so that they neither vanish nor
// overflow.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

#include "internal.h"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 256;
constexpr uint32_t kAll = 0xffffffffu;

// Classes of experts, in the order of their keys: none (not to be chosen),
// NaN, out (logit -inf), numbers.
enum Class : uint32_t { kNone = 0, kNaN = 1, kOut = 2, kNumber = 3 };
constexpr uint32_t kPlace = 15u;  // the place in the lane, in a key
__device__ __forceinline__ uint32_t number_key(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0u;  // the two zeros tie
  return b & 0x80000000u ? ~b : b | 0x80000000u;  // at least 0x007FFFFF
}
__device__ __forceinline__ float key_number(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
constexpr uint32_t kNaNKey = 16u, kOutKey = 32u;  // below every number's

template <bool F32>
__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t t, int e) {
  const int64_t i = t * a.ld + e;
  float v;
  if constexpr (F32)
    v = __ldg(static_cast<const float*>(a.logits) + i);
  else
    v = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + i)) << 16);
  return v == INFINITY ? FLT_MAX : v;  // +inf as the largest number
}

// The lane's PER logits at `at`, in the widest loads they take (-inf for a lane without any).
template <int PER, bool F32>
__device__ __forceinline__ void load_lane(const RouteArgs& a, int64_t at, bool any, float (&l)[PER]) {
  constexpr int kBytes = PER * (F32 ? 4 : 2), kWord = kBytes < 16 ? kBytes : 16;
  uint32_t u[(kBytes + 3) / 4];
  const char* p = static_cast<const char*>(a.logits) + at * (F32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < (kBytes + 3) / 4; ++i) u[i] = F32 ? 0xFF800000u : 0xFF80FF80u;
  if (any) {
#pragma unroll
    for (int i = 0; i < kBytes / kWord; ++i) {
      if constexpr (kWord == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        u[4 * i] = v.x, u[4 * i + 1] = v.y, u[4 * i + 2] = v.z, u[4 * i + 3] = v.w;
      } else if constexpr (kWord == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + i);
        u[0] = v.x, u[1] = v.y;
      } else if constexpr (kWord == 4) {
        u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      } else {
        u[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float v = __uint_as_float(F32 ? u[i] : i % 2 != 0 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
    l[i] = v == INFINITY ? FLT_MAX : v;  // +inf as the largest number
  }
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Groups kept, as bits, from the value of group `lane` (NaN: none of its
// experts can be chosen): those with fewer than top_groups before them.
template <typename T>
__device__ __forceinline__ uint32_t best_groups(T v, int n_groups, int top_groups, int* rank) {
  const int lane = threadIdx.x % 32;
  int before = 0;
  for (int g = 0; g < n_groups; ++g) {
    const T o = __shfl_sync(kAll, v, g);
    const bool ahead = isnan(v) ? !isnan(o) || g < lane : o > v || (o == v && g < lane);
    before += ahead ? 1 : 0;
  }
  *rank = before;
  return __ballot_sync(kAll, lane < n_groups && before < top_groups);
}

// The value of group `lane` from c in shared memory (NaN: not available).
template <typename T>
__device__ __forceinline__ T group_value(const T* c, const RouteArgs& a) {
  const int lane = threadIdx.x % 32, size = a.n_experts / a.n_groups;
  T best = 0, second = 0;
  int n = 0;
  if (lane < a.n_groups)
    for (int i = 0; i < size; ++i) {
      const T v = c[lane * size + i];
      if (isnan(v)) continue;
      if (n == 0 || v > best) {
        second = best;
        best = v;
      } else if (n == 1 || v > second) {
        second = v;
      }
      ++n;
    }
  if (n == 0) return static_cast<T>(NAN);
  return a.group_max || n == 1 ? best : best + second;
}

// The token's choice in 64 bits: lane s < k gets the s-th expert.
template <bool F32>
__device__ __noinline__ int exact_choice(const RouteArgs& a, int64_t t, double* c_smem) {
  constexpr int PER = kMaxExperts / 32;
  const int lane = threadIdx.x % 32;
  double c[PER];
  uint32_t cls[PER];  // 3: a number
  float m = -INFINITY;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = lane * PER + p;
    const float l = e < a.n_experts ? logit_at<F32>(a, t, e) : -INFINITY;
    c[p] = l;
    cls[p] = e >= a.n_experts ? kNone : isnan(l) ? kNaN : l == -INFINITY ? kOut : kNumber;
    if (cls[p] == kNumber) m = fmaxf(m, l);
  }
  m = warp_max(m);
  double z = 0.0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    if (cls[p] != kNumber) continue;
    if (a.softmax)
      z += c[p] = exp(c[p] - static_cast<double>(m));
    else
      c[p] = 1.0 / (1.0 + exp(-c[p]));
  }
  if (a.softmax) z = warp_sum(z);
  __syncwarp();
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = lane * PER + p;
    if (e >= a.n_experts) continue;
    if (cls[p] == kNumber) {
      if (a.softmax) c[p] /= z;
      if (a.bias != nullptr) c[p] += static_cast<double>(__ldg(a.bias + e));
      if (isnan(c[p])) cls[p] = kNaN;
    } else if (a.bias != nullptr && isnan(__ldg(a.bias + e))) {
      cls[p] = kNaN;
    }
    c_smem[e] = cls[p] == kNumber ? c[p] : NAN;
  }
  __syncwarp();
  uint32_t kept = kAll;
  int rank;
  if (a.n_groups > 1) kept = best_groups(group_value(c_smem, a), a.n_groups, a.top_groups, &rank);
  const int size = a.n_experts / a.n_groups;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = lane * PER + p;
    if (e < a.n_experts && !(kept >> (e / size) & 1u)) cls[p] = kNone;
    if (a.bias == nullptr && cls[p] == kNumber) c[p] = logit_at<F32>(a, t, e);  // scores may have met where these have not
  }
  int mine = -1;
  for (int s = 0; s < a.top_k; ++s) {
    uint32_t bc = kNone;
    double bv = 0.0;
    int be = kMaxExperts;
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (cls[p] > bc || (cls[p] == kNumber && bc == kNumber && c[p] > bv)) {
        bc = cls[p];
        bv = c[p];
        be = lane * PER + p;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint32_t oc = __shfl_xor_sync(kAll, bc, o);
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      const bool same = oc == bc && (oc != kNumber || ov == bv);
      if (oc > bc || (oc == kNumber && bc == kNumber && ov > bv) || (same && oe < be)) {
        bc = oc;
        bv = ov;
        be = oe;
      }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (be == lane * PER + p) cls[p] = kNone;
    if (lane == s) mine = be;
  }
  return mine;
}

// The lane's keys in descending order, by a network of minima and maxima
// (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if ((i + j) / (2 * p) == (i + j + k) / (2 * p) && i + j + k < N) {
            const uint32_t a = key[i + j], b = key[i + j + k];
            key[i + j] = max(a, b);
            key[i + j + k] = min(a, b);
          }
}

// lanes: those of a group (32 without groups: the experts are all one group's).
template <int PER, bool F32>
__global__ void __launch_bounds__(kThreads) route_kernel(const __grid_constant__ RouteArgs a, const int lanes, const int vec) {
  __shared__ double c_smem[kWarps][kMaxExperts];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int size = a.n_experts / a.n_groups, group = lane / lanes, first = group * size + lane % lanes * PER;
  // this lane's experts: first .. first + mine - 1
  const int mine = group < a.n_groups ? min(max(size - lane % lanes * PER, 0), PER) : 0;
  const bool by_logit = a.bias == nullptr;           // the logits' own order is the experts',
  const bool groups_by_logit = by_logit && (a.group_max || size == 1);  // and the groups' too
  const bool scores = !by_logit || (a.n_groups > 1 && !groups_by_logit);
  const bool exact_keys = by_logit && !F32;
  float bias[PER];
#pragma unroll
  for (int p = 0; p < PER; ++p) bias[p] = !by_logit && p < mine ? __ldg(a.bias + first + p) : 0.f;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[PER];
    if (vec) {  // (mine is PER or 0, and whole lanes start on their loads' size)
      load_lane<PER, F32>(a, t * a.ld + first, mine > 0, l);
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p) l[p] = p < mine ? logit_at<F32>(a, t, first + p) : -INFINITY;
    }
    float m = -INFINITY, z = 1.f, top_score = 1.f;
    if (a.softmax && (scores || !a.renormalise)) {
#pragma unroll
      for (int p = 0; p < PER; ++p) m = fmaxf(m, l[p]);  // (NaN is skipped)
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int p = 0; p < PER; ++p)
        if (l[p] > -INFINITY) z += expf(l[p] - m);
      z = warp_sum(z);
      top_score = 1.f / z;
    }
    uint32_t key[PER];     // what is chosen by
    float second = -INFINITY, best = -INFINITY;  // the lane's two best c, which the keys have cut short
    int numbers = 0;
    float far = 0.f;       // the largest |c|
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      float c = l[p];
      if (scores) {
        c = (a.softmax ? expf(l[p] - m) * top_score : __fdividef(1.f, 1.f + expf(-l[p]))) + bias[p];
        far = fmaxf(far, fabsf(c));
      }
      if (l[p] > -INFINITY && !isnan(c)) {
        second = fmaxf(second, fminf(best, c));
        best = fmaxf(best, c);
        ++numbers;
      }
      const float by = by_logit ? l[p] : c;
      uint32_t k = number_key(by);
      if (l[p] == -INFINITY) k = kOutKey;
      if (isnan(l[p]) || isnan(by)) k = kNaNKey;
      key[p] = p < mine ? (k & ~kPlace) | (kPlace - p) : 0u;
    }
    sort_keys(key);
    bool sure = true;
    const float near = scores ? top_score * (a.softmax ? 1.52587890625e-05f : 9.5367431640625e-07f) : 0.f;
    if (a.n_groups > 1) {
      // a group's two best, over its lanes
      for (int j = 1; j < lanes; j *= 2) {
        const float ob = __shfl_down_sync(kAll, best, j), os = __shfl_down_sync(kAll, second, j);
        const int on = __shfl_down_sync(kAll, numbers, j);
        if (lane % lanes + j < lanes) {
          numbers += on;
          second = fmaxf(fmaxf(second, os), fminf(best, ob));
          best = fmaxf(best, ob);
        }
      }
      float v = numbers == 0 ? NAN : a.group_max || numbers == 1 ? best : best + second;
      v = __shfl_sync(kAll, v, min(lane * lanes, 31));  // group `lane`'s
      int rank;
      const uint32_t kept = best_groups(v, a.n_groups, a.top_groups, &rank);
      if (!groups_by_logit && a.top_groups < a.n_groups) {
        const uint32_t in = __ballot_sync(kAll, lane < a.n_groups && rank == a.top_groups - 1);
        const uint32_t out = __ballot_sync(kAll, lane < a.n_groups && rank == a.top_groups);
        const float vi = __shfl_sync(kAll, v, __ffs(in) - 1), vo = __shfl_sync(kAll, v, __ffs(out) - 1);
        far = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(far)));
        sure = isnan(vo) || vi - vo > 2.f * (near + far * 2.384185791015625e-07f);
      }
      if (group >= a.n_groups || !(kept >> group & 1u)) {
#pragma unroll
        for (int p = 0; p < PER; ++p) key[p] = 0u;
      }
    }
    int id = -1;
    uint32_t mine_key = 0u;
    const int rounds = a.top_k + (exact_keys ? 0 : 1);  // one more, to be sure of the last
    for (int s = 0; s < rounds; ++s) {
      const uint32_t head = key[0] & ~kPlace;
      const uint32_t top = __reduce_max_sync(kAll, head);
      const int owner = __ffs(__ballot_sync(kAll, head == top)) - 1;
      const int e = __shfl_sync(kAll, first + static_cast<int>(kPlace - (key[0] & kPlace)), owner);
      if (lane == owner) {
#pragma unroll
        for (int p = 0; p + 1 < PER; ++p) key[p] = key[p + 1];
        key[PER - 1] = 0u;
      }
      if (lane == s) {
        id = e;
        mine_key = top;
      }
    }
    if (!exact_keys) {  // each of the k beside the one that follows it
      const uint32_t next_key = __shfl_down_sync(kAll, mine_key, 1);
      const int next = __shfl_down_sync(kAll, id, 1);
      const float c = key_number(mine_key), d = key_number(next_key);
      // 2^-18: four bits of each
      bool fine = lane >= a.top_k || next_key <= kOutKey || c - d > near + fmaxf(fabsf(c), fabsf(d)) * 3.814697265625e-06f;
      if (!fine)
        fine = logit_at<F32>(a, t, id) == logit_at<F32>(a, t, next) &&
               (by_logit || __ldg(a.bias + id) == __ldg(a.bias + next));
      sure = __all_sync(kAll, fine) && sure;
    }
    if (!sure) id = exact_choice<F32>(a, t, c_smem[warp]);
    // the weights
    const bool on = lane < a.top_k;
    const float x = on ? logit_at<F32>(a, t, id) : -INFINITY;
    float w;
    if (a.renormalise) {
      const float lm = warp_max(isnan(x) ? -INFINITY : x);
      // far below 0 the sigmoid is the exponential
      const bool exponential = a.softmax || lm < -60.f;
      w = x == -INFINITY ? 0.f : exponential ? expf(x - lm) : 1.f / (1.f + expf(-x));
      const float sum = warp_sum(w);
      w = sum == 0.f ? 0.f : w / sum;
    } else {
      w = x == -INFINITY ? 0.f : a.softmax ? expf(x - m) * top_score : 1.f / (1.f + expf(-x));
    }
    if (on) {
      a.ids[t * a.top_k + lane] = id;
      a.w[t * a.top_k + lane] = w * a.scale;
    }
  }
}

template <bool F32>
cudaError_t launch(const RouteArgs& a, int num_sms, cudaStream_t s) {
  const int64_t need = (static_cast<int64_t>(a.n_tokens) + kWarps - 1) / kWarps, most = static_cast<int64_t>(num_sms) * 8;
  const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(kThreads);
  // the fewest experts to a lane that leave every group lanes of its own
  const int size = a.n_experts / a.n_groups;
  auto lanes = [&](int per) { return a.n_groups > 1 ? (size + per - 1) / per : 32; };
  auto fits = [&](int per) { return a.n_groups > 1 ? a.n_groups * lanes(per) <= 32 : a.n_experts <= 32 * per; };
  const int bytes = F32 ? 4 : 2;
  auto vec = [&](int per) {  // a lane's experts are one load, or two of 16 bytes
    return size % per == 0 && a.ld % per == 0 &&
                   (reinterpret_cast<uintptr_t>(a.logits) & static_cast<uintptr_t>(std::min(per * bytes, 16) - 1)) == 0
               ? 1
               : 0;
  };
  if (fits(1)) return launch_kernel(route_kernel<1, F32>, grid, block, 0, s, a, lanes(1), vec(1));
  if (fits(2)) return launch_kernel(route_kernel<2, F32>, grid, block, 0, s, a, lanes(2), vec(2));
  if (fits(4)) return launch_kernel(route_kernel<4, F32>, grid, block, 0, s, a, lanes(4), vec(4));
  if (fits(8)) return launch_kernel(route_kernel<8, F32>, grid, block, 0, s, a, lanes(8), vec(8));
  return launch_kernel(route_kernel<16, F32>, grid, block, 0, s, a, lanes(16), vec(16));
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}

}  // namespace cbmoe
