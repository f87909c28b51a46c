// The whole layer for a few tokens (1 to 16) in one cooperative launch, on
// the weights of an ordinary handle (bf16, int8, int4 or fp8 experts):
//
//   1. logits     l[t][e] = x[t] . Wr[e] + b[e]: one expert at a time per
//                 block, the block's warps splitting d;
//      -- grid barrier --
//   2. gate       every block takes the top-k of all n tokens from the n x E
//                 logits (warp_gate) and lists the experts that any token chose;
//   3. gate/up    H[t k + s][j] = bf16( SiLU(g) * u ), g and u the dot products
//                 of x[t] with feature j's gate and up rows of expert ids[t][s];
//      -- grid barrier --
//   4. down and combine   out[t][c] = sum_s w[t][s] (H[t k + s] . Wd[ids[t][s]][c]).
//
// What bounds it: the chosen experts' weights, read once from HBM; with at most 16
// tokens an expert's 128-row tiles of the large kernels would be nearly all
// padding, so nothing is staged in shared memory: a weight element goes
// straight from global memory into the register fragment of an
// mma.sync m16n8k16 (A: 16 weight rows, B: 8 tokens), in the manner of the
// mma router.  A dot product does not depend on the order of its terms, so a
// thread's k-slots are consecutive elements and every weight load is 16
// bytes.  In step 3 the 16 rows are 8 gate rows and the same 8 features' up
// rows, which puts a feature's g and u into one thread; in step 4 they are
// 16 output columns.
//
// The balance: the active experts' features (step 3) and the output columns
// (step 4) are cut into one contiguous share per block, to the row; a share's
// last tile loads only the rows that it has.  A block's 16 warps split the
// rows' bytes in turns of 64, so that together they read 1 KB runs of each
// row.  Each warp keeps kSlots steps (32 bytes a thread each: 128 KB per SM)
// in flight, across tiles and experts; the first of step 4's are requested
// before the barrier that ends step 3, since they do not depend on it.
//
// Every sum is fp32 in a fixed order (mma accumulators, then the warps'
// partial sums in warp order, experts in ascending order), so results do not
// change from run to run.  H is rounded to bf16 as everywhere in the layer:
// it is the MMA's operand.
#include <cuda_bf16.h>

#include "grid_barrier.cuh"
#include "int8_bf16.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "router_common.cuh"
#include "swiglu.cuh"

namespace cbmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSlots = 8;         // steps in flight per warp
constexpr int kStepBytes = 64;    // bytes of a row per step: 4 threads x 16
constexpr int kMaxTokens = kFewTokens;
constexpr int kMaxExperts = 256;
constexpr int kMaxK = 16;

// Weight formats of the kernel: the quantised ones as in WeightFormat.
constexpr int kBf16 = 3;
template <int WF>
constexpr int kElems = WF == kBf16 ? 8 : WF == kWInt4 ? 32 : 16;  // elements per 16 bytes

struct Smem {
  float red[2][kWarps][16][kMaxTokens];  // partial sums: [buffer][warp][row][token]
  float logit[kMaxTokens * kMaxExperts];
  float w[kMaxTokens * kMaxK];           // gate weight of each (token, slot)
  uint32_t mask[kMaxExperts];            // tokens of each expert
  uint8_t slot[kMaxExperts][kMaxTokens]; // the slot at which a token chose it
  int16_t act[kMaxExperts];              // active experts, ascending
  int n_act;
  int warp_act[kMaxExperts / 32];
  int ok;
};

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 16 bytes of a weight row -> its elements as bf16 pairs, in memory order.
template <int WF>
__device__ __forceinline__ void widen(const uint4& v, uint32_t zz, uint32_t (&o)[kElems<WF> / 2]) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (WF == kBf16) {
      o[i] = in[i];
    } else if constexpr (WF == kWInt4) {
      uint32_t t[4];
      int4x8_minus_zero_to_bf16(in[i], zz, t);
#pragma unroll
      for (int m = 0; m < 4; ++m) o[4 * i + m] = t[m];
    } else if constexpr (WF == kWFp8) {
      fp8x4_to_bf16x4(in[i], o[2 * i], o[2 * i + 1]);
    } else {
      int8x4_to_bf16x4(in[i], o[2 * i], o[2 * i + 1]);
    }
  }
}

// acc += the two rows' elements times NT x 8 tokens' elements.  act[n]: this
// lane's token row (column lane / 4 of n-tile n) at the step's first element,
// or nullptr (reads as zero).
template <int WF, int NT>
__device__ __forceinline__ void step_mma(const uint4& lo, const uint4& hi, uint32_t zlo, uint32_t zhi,
                                         const uint16_t* const (&act)[NT], float (&acc)[NT][4]) {
  constexpr int P = kElems<WF> / 2;  // pairs per thread and row
  uint4 b[NT][P / 4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < P / 4; ++i)
      b[n][i] = act[n] != nullptr ? reinterpret_cast<const uint4*>(act[n])[i] : make_uint4(0, 0, 0, 0);
  uint32_t a0[P], a1[P];
  widen<WF>(lo, zlo, a0);
  widen<WF>(hi, zhi, a1);
#pragma unroll
  for (int i = 0; i < P / 4; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      router_detail::mma_bf16(acc[n], a0[4 * i], a1[4 * i], a0[4 * i + 1], a1[4 * i + 1], b[n][i].x, b[n][i].y);
      router_detail::mma_bf16(acc[n], a0[4 * i + 2], a1[4 * i + 2], a0[4 * i + 3], a1[4 * i + 3], b[n][i].z, b[n][i].w);
    }
}

// ------------------------------------------------------------- 1. logits
__device__ __forceinline__ void few_logits(const FewArgs& p, Smem& s) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int e = blockIdx.x; e < p.E; e += gridDim.x) {
    float sum[kMaxTokens];
#pragma unroll
    for (int t = 0; t < kMaxTokens; ++t) sum[t] = 0.f;
    for (int c = threadIdx.x * 8; c < p.d; c += kThreads * 8) {
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.wr + static_cast<int64_t>(e) * p.d + c));
      const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int t = 0; t < kMaxTokens; ++t) {
        if (t >= p.n) break;
        const uint4 xv = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t) * p.d + c));
        const uint32_t xu[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[t] = fmaf(__uint_as_float(xu[i] << 16), __uint_as_float(wu[i] << 16), sum[t]);
          sum[t] = fmaf(__uint_as_float(xu[i] & 0xFFFF0000u), __uint_as_float(wu[i] & 0xFFFF0000u), sum[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < kMaxTokens; ++t) {
      if (t >= p.n) break;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[t] += __shfl_xor_sync(0xffffffffu, sum[t], o);
      if (lane == 0) s.red[0][warp][0][t] = sum[t];
    }
    __syncthreads();
    if (threadIdx.x < p.n) {
      float v = 0.f;
      for (int i = 0; i < kWarps; ++i) v += s.red[0][i][0][threadIdx.x];
      p.logits[threadIdx.x * p.E + e] = v + (p.bias != nullptr ? p.bias[e] : 0.f);
    }
    __syncthreads();
  }
}

// --------------------------------------------------------------- 2. gate
__device__ __forceinline__ void few_gate(const FewArgs& p, Smem& s) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) s.mask[e] = 0u;
  if (p.ids == nullptr)
    for (int i = threadIdx.x; i < p.n * p.E; i += kThreads) s.logit[i] = __ldcg(p.logits + i);
  __syncthreads();
  if (p.ids == nullptr) {
    if (warp < p.n) {
      int id;
      float w;
      const float* ls = s.logit + warp * p.E;
      if (p.E <= 32)
        router_detail::warp_gate<1>(ls, p.E, p.k, p.raw_weights, id, w);
      else if (p.E <= 128)
        router_detail::warp_gate<4>(ls, p.E, p.k, p.raw_weights, id, w);
      else
        router_detail::warp_gate<8>(ls, p.E, p.k, p.raw_weights, id, w);
      if (lane < p.k) {
        s.w[warp * p.k + lane] = w;
        s.slot[id][warp] = static_cast<uint8_t>(lane);
        atomicOr(&s.mask[id], 1u << warp);
      }
    }
  } else if (threadIdx.x < p.n) {  // the hash router's experts: one per token, weight 1
    const int id = p.ids[threadIdx.x];
    s.w[threadIdx.x] = 1.f;
    s.slot[id][threadIdx.x] = 0;
    atomicOr(&s.mask[id], 1u << threadIdx.x);
  }
  __syncthreads();
  const int e = threadIdx.x;
  const bool on = e < p.E && s.mask[e] != 0u;
  const uint32_t ballot = __ballot_sync(0xffffffffu, on);
  if (e < kMaxExperts && lane == 0) s.warp_act[warp] = __popc(ballot);
  __syncthreads();
  if (e < kMaxExperts) {
    int base = 0;
    for (int i = 0; i < warp; ++i) base += s.warp_act[i];
    if (on) s.act[base + __popc(ballot & ((1u << lane) - 1u))] = static_cast<int16_t>(e);
    if (e == kMaxExperts - 1) s.n_act = base + __popc(ballot);
  }
  __syncthreads();
}

// --------------------------------------------------------- 3. gate and up
// A share's features are cut into tiles of at most 8 of one expert.  A cursor
// walks (tile, step); the loads' runs kSlots steps ahead of the sums'.
struct UpCursor {
  int j, end;    // first feature of the tile and the share's end, in act index x f + feature
  int step, steps;
  int a, feat, rows;  // active expert, feature within it, rows of the tile
  __device__ __forceinline__ void open(int f) {
    if (j < end) {
      a = j / f;
      feat = j - a * f;
      rows = min(8, min(end - j, f - feat));
    } else {
      rows = 0;
    }
  }
  __device__ __forceinline__ bool next(int f) {  // true: a new tile
    if (++step < steps) return false;
    step = 0;
    j += rows;
    open(f);
    return true;
  }
};

template <int WF, int NT>
__device__ __forceinline__ void few_gateup(const FewArgs& p, Smem& s, int64_t row_bytes) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  const int64_t total = static_cast<int64_t>(s.n_act) * p.f;
  const int row_steps = static_cast<int>(row_bytes / kStepBytes);
  UpCursor ld{};
  ld.j = static_cast<int>(total * blockIdx.x / gridDim.x);
  ld.end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  ld.steps = (row_steps + kWarps - 1) / kWarps;
  ld.open(p.f);
  UpCursor use = ld;
  const uint8_t* gate_ptr = nullptr;  // this thread's gate row of the loads' tile, at its warp's first step
  const uint8_t* up_ptr = nullptr;
  auto locate = [&]() {
    gate_ptr = up_ptr = nullptr;
    if (g < ld.rows) {
      const int feat = ld.feat + g;
      const int64_t row = static_cast<int64_t>(s.act[ld.a]) * 2 * p.f + (feat / p.gu_block) * 2 * p.gu_block +
                          feat % p.gu_block;
      gate_ptr = static_cast<const uint8_t*>(p.wgu) + row * row_bytes + warp * kStepBytes + q * 16;
      up_ptr = gate_ptr + p.gu_block * row_bytes;
    }
  };
  locate();
  uint4 lo[kSlots], hi[kSlots];
  auto load = [&](uint4& l, uint4& h) {
    l = h = make_uint4(0, 0, 0, 0);
    if (gate_ptr != nullptr && ld.step * kWarps + warp < row_steps) {
      const int64_t at = static_cast<int64_t>(ld.step) * kWarps * kStepBytes;
      l = load_stream(gate_ptr + at);
      h = load_stream(up_ptr + at);
    }
    if (ld.next(p.f)) locate();
  };
#pragma unroll
  for (int i = 0; i < kSlots; ++i) load(lo[i], hi[i]);

  float acc[NT][4];
  const uint16_t* act[NT];
  uint32_t zlo = 0, zhi = 0;
  auto begin = [&]() {  // of a tile's sums
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      act[n] = nullptr;
    }
    if (use.rows == 0) return;
    const int e = s.act[use.a];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if ((s.mask[e] >> (n * 8 + g)) & 1u)
        act[n] = p.x + static_cast<int64_t>(n * 8 + g) * p.d + (warp * 4 + q) * kElems<WF>;
    if constexpr (WF == kWInt4) {
      const int64_t at = static_cast<int64_t>(e) * p.f + use.feat + min(g, use.rows - 1);
      zlo = (0x4300u | __ldg(p.zg + at)) * 0x00010001u;
      zhi = (0x4300u | __ldg(p.zu + at)) * 0x00010001u;
    }
  };
  begin();
  int buf = 0;
  while (use.rows > 0) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      if (use.rows > 0) {
        const uint16_t* at[NT];
        const bool in = use.step * kWarps + warp < row_steps;
#pragma unroll
        for (int n = 0; n < NT; ++n)
          at[n] = in && act[n] != nullptr ? act[n] + use.step * kWarps * 4 * kElems<WF> : nullptr;
        step_mma<WF, NT>(lo[i], hi[i], zlo, zhi, at, acc);
        load(lo[i], hi[i]);
        const UpCursor done = use;
        if (use.next(p.f)) {  // the tile's sums are complete in the 16 warps
          auto* red = s.red[buf][warp];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2*>(&red[g][n * 8 + 2 * q]) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2*>(&red[g + 8][n * 8 + 2 * q]) = make_float2(acc[n][2], acc[n][3]);
          }
          __syncthreads();
          const int r = threadIdx.x % 8, t = threadIdx.x / 8;
          const int e = s.act[done.a];
          if (t < NT * 8 && r < done.rows && ((s.mask[e] >> t) & 1u)) {
            float gs = 0.f, us = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              gs += s.red[buf][w][r][t];
              us += s.red[buf][w][r + 8][t];
            }
            if constexpr (WF != kBf16) {
              const int64_t at2 = static_cast<int64_t>(e) * p.f + done.feat + r;
              gs *= __ldg(p.sg + at2);
              us *= __ldg(p.su + at2);
            }
            const __nv_bfloat16 h = __float2bfloat16_rn(silu(gs) * us);
            p.h[(static_cast<int64_t>(t) * p.k + s.slot[e][t]) * p.f + done.feat + r] = __bfloat16_as_ushort(h);
          }
          buf ^= 1;  // the other buffer's readers passed this barrier
          begin();
        }
      }
    }
  }
}

// ------------------------------------------------- 4. down and combine
struct DownCursor {
  int c, end;  // first output column of the tile, the share's end
  int a, n_act;
  int step, steps;
  __device__ __forceinline__ int rows() const { return min(16, end - c); }
  // 0: another step; 1: another expert; 2: another tile
  __device__ __forceinline__ int next() {
    if (++step < steps) return 0;
    step = 0;
    if (++a < n_act) return 1;
    a = 0;
    c += 16;
    return 2;
  }
};

template <int WF, int NT>
struct Down {
  const FewArgs& p;
  Smem& s;
  int64_t row_bytes;
  int row_steps;
  DownCursor ld, use;
  const uint8_t* ptr;  // this thread's row g of the loads' tile and expert; row g + 8 is 8 rows on
  bool v0, v1;
  uint4 lo[kSlots], hi[kSlots];

  __device__ __forceinline__ Down(const FewArgs& p_, Smem& s_, int64_t rb) : p(p_), s(s_), row_bytes(rb) {
    row_steps = static_cast<int>(row_bytes / kStepBytes);
    ld.c = static_cast<int>(static_cast<int64_t>(p.d) * blockIdx.x / gridDim.x);
    ld.end = static_cast<int>(static_cast<int64_t>(p.d) * (blockIdx.x + 1) / gridDim.x);
    ld.a = 0;
    ld.n_act = s.n_act;
    ld.step = 0;
    ld.steps = (row_steps + kWarps - 1) / kWarps;
    use = ld;
    locate();
  }
  __device__ __forceinline__ void locate() {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
    v0 = g < ld.rows();
    v1 = g + 8 < ld.rows();
    const int64_t row = static_cast<int64_t>(s.act[ld.a]) * p.d + ld.c + g;
    ptr = static_cast<const uint8_t*>(p.wd) + row * row_bytes + warp * kStepBytes + q * 16;
  }
  __device__ __forceinline__ void load(uint4& l, uint4& h) {
    const int warp = threadIdx.x / 32;
    l = h = make_uint4(0, 0, 0, 0);
    if (ld.step * kWarps + warp < row_steps) {
      const uint8_t* at = ptr + static_cast<int64_t>(ld.step) * kWarps * kStepBytes;
      if (v0) l = load_stream(at);
      if (v1) h = load_stream(at + 8 * row_bytes);
    }
    if (ld.next() != 0) locate();
  }
  __device__ __forceinline__ void prologue() {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) load(lo[i], hi[i]);
  }
  __device__ __forceinline__ void run() {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
    float acc[NT][4], tot[NT][4];
    const uint16_t* act[NT];
    uint32_t zlo = 0, zhi = 0;
    auto clear = [&](float (&v)[NT][4]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n][0] = v[n][1] = v[n][2] = v[n][3] = 0.f;
    };
    auto begin = [&]() {  // of an expert's sums
      clear(acc);
      const int e = s.act[use.a];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int t = n * 8 + g;
        act[n] = (s.mask[e] >> t) & 1u
                     ? p.h + (static_cast<int64_t>(t) * p.k + s.slot[e][t]) * p.f + (warp * 4 + q) * kElems<WF>
                     : nullptr;
      }
      if constexpr (WF == kWInt4) {
        const int64_t at = static_cast<int64_t>(e) * p.d;
        zlo = (0x4300u | __ldg(p.zd + at + min(use.c + g, p.d - 1))) * 0x00010001u;
        zhi = (0x4300u | __ldg(p.zd + at + min(use.c + g + 8, p.d - 1))) * 0x00010001u;
      }
    };
    clear(tot);
    int buf = 0;
    if (use.rows() > 0) begin();
    while (use.rows() > 0) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (use.rows() > 0) {
          const uint16_t* at[NT];
          const bool in = use.step * kWarps + warp < row_steps;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            at[n] = in && act[n] != nullptr ? act[n] + use.step * kWarps * 4 * kElems<WF> : nullptr;
          step_mma<WF, NT>(lo[i], hi[i], zlo, zhi, at, acc);
          load(lo[i], hi[i]);
          const DownCursor done = use;
          const int moved = use.next();
          if (moved != 0) {  // this warp's part of the expert is complete: weigh it
            const int e = s.act[done.a];
            float sc0 = 1.f, sc1 = 1.f;
            if constexpr (WF != kBf16) {
              const int64_t row = static_cast<int64_t>(e) * p.d;
              sc0 = __ldg(p.sd + row + min(done.c + g, p.d - 1));
              sc1 = __ldg(p.sd + row + min(done.c + g + 8, p.d - 1));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int t = n * 8 + 2 * q + u;
                if ((s.mask[e] >> t) & 1u) {  // a token that did not choose e takes nothing from it
                  const float w = s.w[t * p.k + s.slot[e][t]];
                  tot[n][u] = fmaf(w * sc0, acc[n][u], tot[n][u]);
                  tot[n][2 + u] = fmaf(w * sc1, acc[n][2 + u], tot[n][2 + u]);
                }
              }
            if (moved == 2) {
              auto* red = s.red[buf][warp];
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<float2*>(&red[g][n * 8 + 2 * q]) = make_float2(tot[n][0], tot[n][1]);
                *reinterpret_cast<float2*>(&red[g + 8][n * 8 + 2 * q]) = make_float2(tot[n][2], tot[n][3]);
              }
              clear(tot);
              __syncthreads();
              const int r = threadIdx.x % 16, t = threadIdx.x / 16;
              if (t < p.n && r < done.rows()) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += s.red[buf][w][r][t];
                const int64_t o = static_cast<int64_t>(t) * p.d + done.c + r;
                if (p.out_f32)
                  static_cast<float*>(p.out)[o] = v;
                else
                  static_cast<uint16_t*>(p.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
              }
              buf ^= 1;
            }
            if (use.rows() > 0) begin();
          }
        }
      }
    }
  }
};

template <int WF, int NT>
__global__ void __launch_bounds__(kThreads, 1) few_tokens_kernel(const FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  grid_dep_wait();
  const unsigned G = gridDim.x;
  bool ok = true;
  if (p.ids == nullptr) {
    few_logits(p, s);
    ok = grid_barrier_wait(p.bar, G, p.wait_limit_ns, p.err, &s.ok);
    if (threadIdx.x == 0) grid_barrier_depart(p.bar, G);
  }
  const int64_t up_bytes = static_cast<int64_t>(p.d) / kElems<WF> * 16;
  const int64_t down_bytes = static_cast<int64_t>(p.f) / kElems<WF> * 16;
  if (ok) {
    few_gate(p, s);
    few_gateup<WF, NT>(p, s, up_bytes);
    Down<WF, NT> down(p, s, down_bytes);
    down.prologue();
    if (grid_barrier_wait(p.bar + 2, G, p.wait_limit_ns, p.err, &s.ok)) down.run();
  } else {
    // the other blocks still find this one at the second barrier
    grid_barrier_wait(p.bar + 2, G, p.wait_limit_ns, p.err, &s.ok);
  }
  if (threadIdx.x == 0) grid_barrier_depart(p.bar + 2, G);
}

template <typename F>
cudaError_t for_kernel(int wf, int n, F&& f) {
  const bool two = n > 8;
  switch (wf) {
    case kBf16: return two ? f(few_tokens_kernel<kBf16, 2>) : f(few_tokens_kernel<kBf16, 1>);
    case kWInt8: return two ? f(few_tokens_kernel<kWInt8, 2>) : f(few_tokens_kernel<kWInt8, 1>);
    case kWInt4: return two ? f(few_tokens_kernel<kWInt4, 2>) : f(few_tokens_kernel<kWInt4, 1>);
    case kWFp8: return two ? f(few_tokens_kernel<kWFp8, 2>) : f(few_tokens_kernel<kWFp8, 1>);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int few_format(bool quantised, WeightFormat wf) { return quantised ? static_cast<int>(wf) : kBf16; }

cudaError_t few_tokens_prepare(int wf, int* blocks_per_sm) {
  *blocks_per_sm = 0;
  for (int n : {1, kMaxTokens}) {
    const cudaError_t e = for_kernel(wf, n, [&](auto kernel) {
      cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
      int per_sm = 0;
      if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, sizeof(Smem));
      *blocks_per_sm = n == 1 ? per_sm : (per_sm < *blocks_per_sm ? per_sm : *blocks_per_sm);
      return r;
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_few_tokens(int wf, const FewArgs& a, int grid, cudaStream_t s) {
  if (a.n <= 0) return cudaSuccess;
  if (a.n > kMaxTokens || a.E > kMaxExperts || a.k > kMaxK || grid <= 0) return cudaErrorInvalidValue;
  return for_kernel(wf, a.n, [&](auto kernel) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  });
}

}  // namespace cbmoe
