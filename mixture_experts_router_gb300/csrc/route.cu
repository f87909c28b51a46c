// Routing from given logits: scores (sigmoid or softmax), a bias for balance,
// groups of experts, top-k, renormalised weights.  One warp takes a token; a
// lane has PER consecutive experts, a group of experts its own lanes.
//
//   c_e = s_e + b_e; each lane sorts its experts by c; groups by their two best
//   c or the best; then k rounds of a warp's largest head, ties to the lower
//   index.
//
// What bounds it: for many tokens the instructions of the scores and the
// rounds (16384 x 256 sigmoid, 4 of 8 groups, 8 chosen: 18.6 us with some 770
// instructions a token and warp; 8192 x 128 softmax, 4 chosen: 5.5), not the
// bytes of the logits; for few, the launch (3.5 us for one).
//
// Keys.  The order of a lane's experts is that of unsigned words: c's bits in
// an order-preserving form, the last four replaced by the expert's place in the
// lane, lower places first.  So a compare and exchange of the sort is a minimum
// and a maximum, and a round one warp maximum and one vote.
//
// The order is that of the real numbers.  Without a bias it is the logits'
// own (both scores grow with them), and needs no score but of the groups' two
// best; bf16 logits have nothing in the four bits.  Otherwise c is off by at
// most 2^-21 (sigmoid) or 2^-20 of the largest score (softmax), half a step of
// its own and the four bits.  Where two neighbours in the order are nearer than
// twice that and not of equal logits and biases, or the last one chosen and any
// that is left, those experts are put in order in 64 bits (exact_order); where
// the last group kept and the first dropped are near, the groups near them get
// their values in 64 bits.  Weights are computed
// from the chosen logits, relative to the largest of them, so that they neither
// vanish nor overflow.
//
// (The rounded product in exp(-l) = 2^(-l log2 e) moves a sigmoid by at most
// s (1 - s) |l| 2^-24 < 2^-26, a softmax score by e^-x x 2^-24 of the largest.)
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "internal.h"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 256;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kScratch = 320;                 // 8-byte words of a warp's shared memory,
constexpr int kPicks = kScratch - 32;         //   of which the last are for the chosen ones
static_assert(kPicks * 2 >= 18 * 32 && kScratch >= kMaxExperts, "room for 16 keys of each lane, and all c");

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

// The experts of lanes 0 .. n - 1, whose c are numbers, in the order of these
// in 64 bits: lane s gets the s-th, the lanes from n on keep theirs.  m: the
// largest logit, for the softmax.
template <bool F32>
__device__ __noinline__ int exact_order(const RouteArgs& a, int64_t t, int id, int n, float m, double* smem) {
  const int lane = threadIdx.x % 32;
  double c = 0.0, z = 1.0;
  if (a.softmax && a.bias != nullptr) {
    z = 0.0;
    for (int e = lane; e < a.n_experts; e += 32) {
      const float l = logit_at<F32>(a, t, e);
      if (l > -INFINITY) z += exp(static_cast<double>(l) - static_cast<double>(m));
    }
    z = warp_sum(z);
  }
  if (lane < n) {
    c = logit_at<F32>(a, t, id);
    if (a.bias != nullptr)
      c = (a.softmax ? exp(c - static_cast<double>(m)) / z : 1.0 / (1.0 + exp(-c))) + static_cast<double>(__ldg(a.bias + id));
  }
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kAll, c, j);
    const int e = __shfl_sync(kAll, id, j);
    rank += o > c || (o == c && e < id) ? 1 : 0;
  }
  int* order = reinterpret_cast<int*>(smem);
  __syncwarp();
  if (lane < n) order[rank] = id;
  __syncwarp();
  const int mine = lane < n ? order[lane] : id;
  __syncwarp();
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

// Blocks of an SM, all of them resident: registers are worth more than warps
// (16384 x 256 in groups: 20.5 us with 4 blocks, 18.9 with 3; 65536 x 128 in
// groups: 52.7 with 5, 50.3 with 4).
template <int PER>
constexpr int kBlocks = PER > 8 ? 2 : PER == 8 ? 3 : 4;

enum Mode { kByLogit = 0, kSigmoid = 1, kSoftmax = 2 };  // what c is: the logit, or a score and its bias

// The groups kept, the values of those in `who` taken again in 64 bits: of their
// experts with keys not below `low` (a lane's own group's).  v: lane g's group's;
// keys: the lanes' sorted ones, [place][lane].
template <int PER, bool F32, int MODE>
__device__ __noinline__ uint32_t exact_groups(const RouteArgs& a, int64_t t, const uint32_t* keys, uint32_t who, float v,
                                              float low, int first, int lanes, float m, bool one) {
  const int lane = threadIdx.x % 32, group = lane / lanes;
  double z = 1.0;
  if constexpr (MODE == kSoftmax) {
    z = 0.0;
    for (int e = lane; e < a.n_experts; e += 32) {
      const float l = logit_at<F32>(a, t, e);
      if (l > -INFINITY) z += exp(static_cast<double>(l) - static_cast<double>(m));
    }
    z = warp_sum(z);
  }
  double best = 0.0, second = 0.0;
  int n = 0;
  auto add = [&](double c) {
    if (n == 0 || c > best) {
      second = best;
      best = c;
    } else if (n == 1 || c > second) {
      second = c;
    }
    n = min(n + 1, 2);
  };
  for (int p = 0; p < PER; ++p) {
    const uint32_t key = keys[p * 32 + lane];
    const bool go = (who >> group & 1u) && key > (kOutKey | kPlace) && !(key_number(key & ~kPlace) < low);
    if (!__any_sync(kAll, go)) break;
    if (!go) continue;
    const int e = first + static_cast<int>(kPlace - (key & kPlace));
    double c = logit_at<F32>(a, t, e);
    if (MODE != kByLogit || !one) {
      c = a.softmax ? exp(c - static_cast<double>(m)) / z : 1.0 / (1.0 + exp(-c));
      if (MODE != kByLogit) c += static_cast<double>(__ldg(a.bias + e));
    }
    add(c);
  }
  for (int j = 1; j < lanes; j *= 2) {
    const double ob = __shfl_down_sync(kAll, best, j), os = __shfl_down_sync(kAll, second, j);
    const int on = __shfl_down_sync(kAll, n, j);
    if (lane % lanes + j < lanes) {
      if (on > 0) add(ob);
      if (on > 1) add(os);
    }
  }
  const double value = one || n == 1 ? best : best + second;
  const double exact = __shfl_sync(kAll, value, min(lane * lanes, 31));
  int rank;
  return best_groups(who >> lane & 1u ? exact : static_cast<double>(v), a.n_groups, a.top_groups, &rank);
}

__device__ __forceinline__ float exp_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}

__device__ __forceinline__ float sigmoid_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp_fast(-v)));
  return r;
}

// lanes: those of a group (32 without groups: the experts are all one group's).
template <int PER, bool F32, int MODE>
__global__ void __launch_bounds__(kThreads, kBlocks<PER>)
    route_kernel(const __grid_constant__ RouteArgs a, const int lanes, const int vec) {
  // a warp's sorted keys ([place][lane], and one 0 behind them) and picks; or c in 64 bits
  __shared__ double c_smem[kWarps][kScratch];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int size = a.n_experts / a.n_groups, group = lane / lanes, place = lane % lanes, first = group * size + place * PER;
  // this lane's experts: first .. first + mine - 1
  const int mine = group < a.n_groups ? min(max(size - place * PER, 0), PER) : 0;
  constexpr bool kExactKeys = MODE == kByLogit && !F32;
  constexpr float kCut = 3.814697265625e-06f;  // 2^-18: the four bits, twice
  const bool one = a.group_max || size == 1;   // a group's value is its best c
  float bias[PER], far = 1.f;                  // far: no |c| is larger
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    bias[p] = MODE != kByLogit && p < mine ? __ldg(a.bias + first + p) : 0.f;
    far = fmaxf(far, 1.f + fabsf(bias[p]));
  }
  if (MODE != kByLogit) far = warp_max(far);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    float l[PER];
    if (vec) {  // (mine is PER or 0, and whole lanes start on their loads' size)
      load_lane<PER, F32>(a, t * a.ld + first, mine > 0, l);
    } else {
#pragma unroll
      for (int p = 0; p < PER; ++p) l[p] = p < mine ? logit_at<F32>(a, t, first + p) : -INFINITY;
    }
    float m = -INFINITY, top_score = 1.f;
    if (a.softmax) {
#pragma unroll
      for (int p = 0; p < PER; ++p) m = fmaxf(m, l[p]);  // (NaN is skipped)
      m = warp_max(m);
      if (MODE == kSoftmax || !a.renormalise) {
        float z = 0.f;
#pragma unroll
        for (int p = 0; p < PER; ++p)
          if (l[p] > -INFINITY) z += expf(l[p] - m);
        top_score = 1.f / warp_sum(z);
      }
    }
    // the keys; classes beside numbers only where one of the lanes has any
    float c[PER];
    float odd = 0.f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      c[p] = MODE == kByLogit   ? l[p] + 0.f  // (the two zeros tie)
             : MODE == kSigmoid ? sigmoid_fast(l[p]) + bias[p]
                                : exp_fast(l[p] - m) * top_score + bias[p];
      odd = fmaf(MODE == kByLogit ? c[p] : c[p] + l[p], 0.f, odd);  // NaN after a NaN or an infinity
    }
    uint32_t key[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const uint32_t u = __float_as_uint(c[p]);
      key[p] = ((u ^ ((static_cast<int32_t>(u) >> 31) | 0x80000000u)) & ~kPlace) | (kPlace - p);
    }
    if (__any_sync(kAll, isnan(odd) && mine > 0)) {
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        uint32_t k = number_key(fminf(fmaxf(c[p], -FLT_MAX), FLT_MAX));  // (of -inf the four bits would leave a NaN)
        if (l[p] == -INFINITY) k = kOutKey;
        if (isnan(l[p]) || isnan(bias[p])) k = kNaNKey;
        key[p] = (k & ~kPlace) | (kPlace - p);
      }
    }
    if (mine < PER) {
#pragma unroll
      for (int p = 0; p < PER; ++p)
        if (p >= mine) key[p] = 0u;
    }
    sort_keys(key);
    uint32_t* keys = reinterpret_cast<uint32_t*>(c_smem[warp]) + lane;
    __syncwarp();
#pragma unroll
    for (int p = 0; p < PER; ++p) keys[p * 32] = key[p];
    keys[PER * 32] = 0u;
    uint32_t head = key[0];
    const float near = MODE == kByLogit ? 0.f : top_score * (MODE == kSigmoid ? 9.5367431640625e-07f : 1.9073486328125e-06f);
    if (a.n_groups > 1) {
      // a group's two best, over its lanes
      const uint32_t k0 = key[0] & ~kPlace, k1 = PER > 1 ? key[PER > 1 ? 1 : 0] & ~kPlace : 0u;
      float best = k0 > kOutKey ? key_number(k0) : -INFINITY, second = k1 > kOutKey ? key_number(k1) : -INFINITY;
      int numbers = (k0 > kOutKey) + (k1 > kOutKey);
      for (int j = 1; j < lanes; j *= 2) {
        const float ob = __shfl_down_sync(kAll, best, j), os = __shfl_down_sync(kAll, second, j);
        const int on = __shfl_down_sync(kAll, numbers, j);
        if (place + j < lanes) {
          numbers += on;
          second = fmaxf(fmaxf(second, os), fminf(best, ob));
          best = fmaxf(best, ob);
        }
      }
      // to lane g group g's value; of its two best scores without a bias (softmax: in units of the largest)
      const int from = min(lane * lanes, 31);
      const float gb = __shfl_sync(kAll, best, from), gs = __shfl_sync(kAll, second, from);
      const int gn = __shfl_sync(kAll, numbers, from);
      auto score = [&](float x) { return a.softmax ? exp_fast(x - m) : sigmoid_fast(x); };
      float v = NAN;
      // (finite, so that what is near the cut can be told: infinite biases are looked at again in 64 bits)
      if (gn > 0) v = one || gn == 1 ? gb : MODE == kByLogit ? score(gb) + score(gs) : fminf(fmaxf(gb + gs, -FLT_MAX), FLT_MAX);
      if (MODE == kByLogit && !one && gn == 1) v = score(gb);
      uint32_t kept = 0u, left = lane < a.n_groups && !isnan(v) ? number_key(v) : 0u, last = 0u;
      uint32_t in_play = lane < a.n_groups ? 1u : 0u;
      for (int s = 0; s < a.top_groups; ++s) {
        last = __reduce_max_sync(kAll, left);
        const uint32_t who = __ballot_sync(kAll, left == last && in_play != 0u);
        const uint32_t lowest = who & (0u - who);
        kept |= lowest;
        if (lowest >> lane & 1u) left = in_play = 0u;
      }
      const uint32_t next = __reduce_max_sync(kAll, left);
      // near the cut?
      float slack = 0.f;
      if (MODE != kByLogit)
        slack = 2.f * (near + far * kCut);
      else if (!one)
        slack = a.softmax ? 4.f * kCut * (1.f + fabsf(m)) : 4.f * kCut;
      else if (F32)
        slack = kCut * fmaxf(fabsf(key_number(last)), fabsf(key_number(next)));
      if (next != 0u && !(kExactKeys && one) && !(key_number(last) - key_number(next) > slack)) {
        // all groups that may lie on either side of it, their experts that may be among the two best
        const bool play = !isnan(v) && v <= key_number(last) + slack && v >= key_number(next) - slack;
        const uint32_t who = __ballot_sync(kAll, lane < a.n_groups && play);
        const float low = __shfl_sync(kAll, one || gn < 2 ? gb : gs, min(group, 31));
        kept = exact_groups<PER, F32, MODE>(a, t, keys - lane, who, v, low - (near + fabsf(low) * kCut), first, lanes, m, one);
      }
      if (group >= a.n_groups || !(kept >> group & 1u)) head = 0u;
    }
    uint2* picks = reinterpret_cast<uint2*>(c_smem[warp] + kPicks);  // the chosen ones' keys and indexes, in order
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t* at = keys;
    auto pick = [&](int s) {
      const uint32_t top = __reduce_max_sync(kAll, head & ~kPlace);
      const bool mine_too = (head & ~kPlace) == top;
      const uint32_t who = __ballot_sync(kAll, mine_too);
      if (mine_too && (who & below) == 0u) {
        picks[s] = make_uint2(top, first + static_cast<int>(kPlace - (head & kPlace)));
        at += 32;
        head = *at;
      }
    };
    __syncwarp();
    for (int s = 0; s < a.top_k + (kExactKeys ? 0 : 1); ++s) pick(s);  // one more, to be sure of the last
    __syncwarp();
    uint2 own = lane <= a.top_k ? picks[lane] : make_uint2(0u, 0u);
    int id = static_cast<int>(own.y);
    const bool on = lane < a.top_k;
    float x = on ? logit_at<F32>(a, t, id) : -INFINITY;
    if constexpr (!kExactKeys) {  // each of the k beside the one that follows it
      auto apart = [&](uint32_t k, uint32_t following) {
        const float u = key_number(k), v = key_number(following);
        return following <= kOutKey || u - v > near + fmaxf(fabsf(u), fabsf(v)) * kCut;
      };
      auto same = [&](float of, int e, int other) {  // equal logits and biases: a tie, which the index decides
        return of == logit_at<F32>(a, t, other) && (MODE == kByLogit || __ldg(a.bias + e) == __ldg(a.bias + other));
      };
      const uint32_t next_key = __shfl_down_sync(kAll, own.x, 1);
      const int next = __shfl_down_sync(kAll, id, 1);
      bool fine = !on || apart(own.x, next_key);
      if (!__all_sync(kAll, fine)) {
        if (!fine) fine = same(x, id, next);
        // the last one beside all that are left, each lane's
        const uint2 last = picks[a.top_k - 1];
        const int last_id = static_cast<int>(last.y);
        if (!apart(last.x, picks[a.top_k].x) && head != 0u) {
          const float lx = logit_at<F32>(a, t, last_id);
          for (const uint32_t* q = at; fine && !apart(last.x, *q & ~kPlace); q += 32)
            fine = same(lx, last_id, first + static_cast<int>(kPlace - (*q & kPlace)));
        }
        if (!__all_sync(kAll, fine)) {
          // all that may belong before the k-th, and one that does not; then these in 64 bits
          int n = a.top_k;
          while (n < 31 && !apart(picks[n - 1].x, picks[n].x)) {
            __syncwarp();
            pick(++n);
            __syncwarp();
          }
          if (lane <= n) id = static_cast<int>(picks[lane].y);
          // numbers come first; what is none stands in its place already, and compares with nothing
          const int numbers = __popc(__ballot_sync(kAll, lane < n && picks[lane].x > kOutKey));
          __syncwarp();
          id = n < 31 ? exact_order<F32>(a, t, id, numbers, m, c_smem[warp]) : exact_choice<F32>(a, t, c_smem[warp]);
          x = on ? logit_at<F32>(a, t, id) : -INFINITY;
        }
      }
    }
    // the weights
    float w = x == -INFINITY ? 0.f : a.softmax ? expf(x - m) : 1.f / (1.f + expf(-x));
    if (a.renormalise) {
      if (a.softmax || __any_sync(kAll, on && x < -60.f)) {  // relative to the largest of them
        float lm = isnan(x) ? -INFINITY : x;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) lm = fmaxf(lm, __shfl_xor_sync(kAll, lm, o));
        if (a.softmax) {
          w = x == -INFINITY ? 0.f : expf(x - lm);
        } else if (x > -INFINITY) {
          // s(x) = e^min(x, 0) / (1 + e^-|x|); the difference with what its rounding leaves, exactly: |from| >= |to|
          const float from = fminf(x, 0.f), to = fminf(lm, 0.f), d = from - to, e = expf(d);
          w = fmaf(e, (from - d) - to, e) / (1.f + expf(-fabsf(x)));
        }
      }
      float sum = w;  // of the first 16 lanes
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      w = sum == 0.f ? 0.f : w / sum;
    } else if (a.softmax) {
      w = x == -INFINITY ? 0.f : w * top_score;
    }
    if (on) {
      a.ids[t * a.top_k + lane] = id;
      a.w[t * a.top_k + lane] = w * a.scale;
    }
  }
}

template <bool F32>
cudaError_t launch(const RouteArgs& a, int num_sms, cudaStream_t s) {
  const int need = (a.n_tokens - 1) / kWarps + 1;
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
  auto run = [&](auto per) {
    constexpr int PER = decltype(per)::value;
    const dim3 grid(std::min(need, num_sms * kBlocks<PER>));
    auto go = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kThreads), 0, s, a, lanes(PER), vec(PER)); };
    return a.bias == nullptr ? go(route_kernel<PER, F32, kByLogit>)
           : a.softmax       ? go(route_kernel<PER, F32, kSoftmax>)
                             : go(route_kernel<PER, F32, kSigmoid>);
  };
  if (fits(1)) return run(std::integral_constant<int, 1>{});
  if (fits(2)) return run(std::integral_constant<int, 2>{});
  if (fits(4)) return run(std::integral_constant<int, 4>{});
  if (fits(8)) return run(std::integral_constant<int, 8>{});
  return run(std::integral_constant<int, 16>{});
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}

}  // namespace cbmoe
