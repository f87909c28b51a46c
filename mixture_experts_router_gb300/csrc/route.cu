// Routing from given logits: scores (sigmoid or softmax), a bias for balance,
// groups of experts, top-k, renormalised weights.  One warp takes a token,
// lane l its experts PER l .. PER l + PER - 1.
//
//   c_e = s_e + b_e; groups by their two best c or the best; then k rounds of
//   a warp's largest (two warp reductions each), ties to the lower index.
//
// What bounds it: for many tokens the instructions of the rounds, not the
// bytes of the logits; for few, the launch.
//
// The order is that of the real numbers.  Without a bias it is the logits'
// own (both scores grow with them), which needs no score.  With one, c is off
// by at most 2^-21 (sigmoid) or 2^-17 (softmax: the rounded argument of exp
// and the sum) of the largest score and half a step of its own: where two
// neighbours in the order, or the last group kept and the first dropped, are
// nearer than twice that and not of equal logits and biases, the warp makes
// the token's choice again in 64 bits (exact_choice).  Weights are computed
// from the chosen logits, relative to the largest of them, so that they
// neither vanish nor overflow.
#include <cuda_bf16.h>

#include <cfloat>

#include "internal.h"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxExperts = 256;
constexpr uint32_t kAll = 0xffffffffu;

// Keys of the order: 0 not to be chosen, then NaN, experts that are out, numbers.
constexpr uint32_t kNaN = 1u, kOut = 2u;
__device__ __forceinline__ uint32_t number_key(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0u;  // the two zeros tie
  return b & 0x80000000u ? ~b : b | 0x80000000u;  // at least 0x007FFFFF
}
__device__ __forceinline__ float key_number(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <bool F32>
__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t t, int e) {
  const int64_t i = t * a.ld + e;
  float v;
  if constexpr (F32)
    v = __ldg(static_cast<const float*>(a.logits) + i);
  else
    v = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.logits) + i)) << 16);
  return fminf(v, FLT_MAX) == v || isnan(v) ? v : FLT_MAX;  // +inf as the largest number
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
template <int PER, bool F32>
__device__ __noinline__ int exact_choice(const RouteArgs& a, int64_t t, double* c_smem) {
  const int lane = threadIdx.x % 32;
  double c[PER];
  uint32_t cls[PER];  // 3: a number
  float m = -INFINITY;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = lane * PER + p;
    const float l = e < a.n_experts ? logit_at<F32>(a, t, e) : -INFINITY;
    c[p] = l;
    cls[p] = e >= a.n_experts ? 0u : isnan(l) ? kNaN : l == -INFINITY ? kOut : 3u;
    if (cls[p] == 3u) m = fmaxf(m, l);
  }
  m = warp_max(m);
  double z = 0.0;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    if (cls[p] != 3u) continue;
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
    if (cls[p] == 3u) {
      if (a.softmax) c[p] /= z;
      if (a.bias != nullptr) c[p] += static_cast<double>(__ldg(a.bias + e));
      if (isnan(c[p])) cls[p] = kNaN;
    } else if (a.bias != nullptr && isnan(__ldg(a.bias + e))) {
      cls[p] = kNaN;
    }
    c_smem[e] = cls[p] == 3u ? c[p] : NAN;
  }
  __syncwarp();
  uint32_t kept = kAll;
  int rank;
  if (a.n_groups > 1) kept = best_groups(group_value(c_smem, a), a.n_groups, a.top_groups, &rank);
  const int size = a.n_experts / a.n_groups;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    const int e = lane * PER + p;
    if (e < a.n_experts && !(kept >> (e / size) & 1u)) cls[p] = 0u;
    if (a.bias == nullptr && cls[p] == 3u) c[p] = logit_at<F32>(a, t, e);  // scores may have met where these have not
  }
  int mine = -1;
  for (int s = 0; s < a.top_k; ++s) {
    uint32_t bc = 0u;
    double bv = 0.0;
    int be = kMaxExperts;
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (cls[p] > bc || (cls[p] == 3u && bc == 3u && c[p] > bv)) {
        bc = cls[p];
        bv = c[p];
        be = lane * PER + p;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint32_t oc = __shfl_xor_sync(kAll, bc, o);
      const double ov = __shfl_xor_sync(kAll, bv, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      const bool same = oc == bc && (oc != 3u || ov == bv);
      if (oc > bc || (oc == 3u && bc == 3u && ov > bv) || (same && oe < be)) {
        bc = oc;
        bv = ov;
        be = oe;
      }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p)
      if (be == lane * PER + p) cls[p] = 0u;
    if (lane == s) mine = be;
  }
  return mine;
}

template <int PER, bool F32>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  __shared__ double c_smem[kWarps][kMaxExperts];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int size = a.n_experts / a.n_groups;
  // whether the logits' own order is the experts', and the groups' too
  const bool by_logit = a.bias == nullptr;
  const bool groups_by_logit = by_logit && (a.group_max || size == 1);
  const bool scores = !by_logit || (a.n_groups > 1 && !groups_by_logit);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp; t < a.n_tokens;
       t += static_cast<int64_t>(gridDim.x) * kWarps) {
    float c[PER];       // what is chosen by
    uint32_t key[PER];
    float m = -INFINITY;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
      const int e = lane * PER + p;
      c[p] = e < a.n_experts ? logit_at<F32>(a, t, e) : -INFINITY;
      key[p] = e >= a.n_experts ? 0u : isnan(c[p]) ? kNaN : c[p] == -INFINITY ? kOut : number_key(c[p]);
      if (key[p] > kOut) m = fmaxf(m, c[p]);
    }
    float z = 1.f, top_score = 1.f;
    if (a.softmax && (scores || !a.renormalise)) {
      m = warp_max(m);
      z = 0.f;
#pragma unroll
      for (int p = 0; p < PER; ++p)
        if (key[p] > kOut) z += expf(c[p] - m);
      z = warp_sum(z);
      top_score = 1.f / z;
    }
    float far = 0.f;  // the largest |c|
    if (scores) {
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int e = lane * PER + p;
        const float b = by_logit || e >= a.n_experts ? 0.f : __ldg(a.bias + e);
        if (key[p] > kOut) {
          c[p] = a.softmax ? expf(c[p] - m) * top_score : 1.f / (1.f + expf(-c[p]));
          c[p] += b;
          far = fmaxf(far, fabsf(c[p]));
          if (!by_logit) key[p] = isnan(c[p]) ? kNaN : number_key(c[p]);
        } else if (e < a.n_experts && isnan(b)) {
          key[p] = kNaN;
        }
      }
      far = warp_max(far);
    }
    const float near = top_score * (a.softmax ? 1.52587890625e-05f : 9.5367431640625e-07f) + far * 2.384185791015625e-07f;
    bool sure = true;
    if (a.n_groups > 1) {
      float* cs = reinterpret_cast<float*>(c_smem[warp]);
      __syncwarp();
#pragma unroll
      for (int p = 0; p < PER; ++p)
        if (lane * PER + p < a.n_experts) cs[lane * PER + p] = key[p] > kOut ? c[p] : NAN;
      __syncwarp();
      int rank;
      const float v = group_value(cs, a);
      const uint32_t kept = best_groups(v, a.n_groups, a.top_groups, &rank);
      if (!groups_by_logit && a.top_groups < a.n_groups) {
        const uint32_t in = __ballot_sync(kAll, lane < a.n_groups && rank == a.top_groups - 1);
        const uint32_t out = __ballot_sync(kAll, lane < a.n_groups && rank == a.top_groups);
        const float vi = __shfl_sync(kAll, v, __ffs(in) - 1), vo = __shfl_sync(kAll, v, __ffs(out) - 1);
        sure = isnan(vo) || vi - vo > 2.f * near;
      }
#pragma unroll
      for (int p = 0; p < PER; ++p) {
        const int e = lane * PER + p;
        if (e < a.n_experts && !(kept >> (e / size) & 1u)) key[p] = 0u;
      }
    }
    int id = -1;
    uint32_t last_key = 0u;
    int last = -1;
    const int rounds = a.top_k + (by_logit ? 0 : 1);  // one more, to be sure of the last
    for (int s = 0; s < rounds && sure; ++s) {
      uint32_t bk = key[0];
      int bp = 0;
#pragma unroll
      for (int p = 1; p < PER; ++p)
        if (key[p] > bk) {
          bk = key[p];
          bp = p;
        }
      const uint32_t wk = __reduce_max_sync(kAll, bk);
      const int e = static_cast<int>(
          __reduce_min_sync(kAll, bk == wk ? static_cast<uint32_t>(lane * PER + bp) : ~0u));
      if (!by_logit && s > 0 && wk > kOut && !(key_number(last_key) - key_number(wk) > near))
        sure = logit_at<F32>(a, t, last) == logit_at<F32>(a, t, e) && __ldg(a.bias + last) == __ldg(a.bias + e);
#pragma unroll
      for (int p = 0; p < PER; ++p)
        if (e == lane * PER + p) key[p] = 0u;
      if (lane == s && s < a.top_k) id = e;
      last_key = wk;
      last = e;
    }
    if (!sure) id = exact_choice<PER, F32>(a, t, c_smem[warp]);
    // the weights
    const bool on = lane < a.top_k;
    const float l = on ? logit_at<F32>(a, t, id) : -INFINITY;
    float w;
    if (a.renormalise) {
      const float lm = warp_max(isnan(l) ? -INFINITY : l);
      // far below 0 the sigmoid is the exponential
      const bool exponential = a.softmax || lm < -60.f;
      w = l == -INFINITY ? 0.f : exponential ? expf(l - lm) : 1.f / (1.f + expf(-l));
      const float sum = warp_sum(w);
      w = sum == 0.f ? 0.f : w / sum;
    } else {
      w = l == -INFINITY ? 0.f : a.softmax ? expf(l - m) * top_score : 1.f / (1.f + expf(-l));
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
  if (a.n_experts <= 32) return launch_kernel(route_kernel<1, F32>, grid, block, 0, s, a);
  if (a.n_experts <= 64) return launch_kernel(route_kernel<2, F32>, grid, block, 0, s, a);
  if (a.n_experts <= 128) return launch_kernel(route_kernel<4, F32>, grid, block, 0, s, a);
  return launch_kernel(route_kernel<8, F32>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch<true>(a, num_sms, s) : launch<false>(a, num_sms, s);
}

}  // namespace cbmoe
