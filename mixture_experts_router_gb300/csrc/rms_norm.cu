// Root-mean-square norm with the residual's addition, written in x's type, as
// e4m3 rows with an fp32 scale per 128 columns, or both:
//
//   h = x + r,  y = h / sqrt(mean h^2 + eps) * g,  s = max|y| / 448,  code = e4m3(y / s).
//
// Bound by memory: every element is read and written once, a row staying in
// registers between its sum of squares and its results (16384 x 4096 bf16 with
// the residual and both results: 95.6 us, 6.3 TB/s; one row of 4096: 2.5 us, the
// launch and two round trips).  R threads share a row
// (a power of two from 32), each holding up to 4 times 8 elements.  Rows that
// start on 16 bytes: a thread's elements are 8 in a row (16 bytes of bf16),
// 16 lanes a scale's 128 columns.  Others: 2 of every 64, or an element of every
// 32 where rows are odd (a warp's loads are whole lines), a warp's first half
// and last half of steps a scale's columns (2915 rows of bf16, both results, 91
// MB: 58 us for 6259 columns one by one, 48 for 6258 in pairs).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace cbmoe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kBlock = 256;  // threads of a block with rows of at most as many

__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Eight elements of one thread: consecutive from p (VEC 8: on 16 bytes), or
// VEC of every 32 VEC from p, of which those below `left` exist.
template <bool F32, int VEC>
__device__ __forceinline__ void load8(const void* base, int64_t at, int left, float (&v)[8]) {
  if constexpr (VEC == 8) {
    if constexpr (F32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 a = q[0], b = q[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
      const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    }
  } else if constexpr (VEC == 2) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      v[i] = v[i + 1] = 0.f;
      if (i * 32 < left) {
        if constexpr (F32) {
          const float2 a = *reinterpret_cast<const float2*>(static_cast<const float*>(base) + at + i * 32);
          v[i] = a.x, v[i + 1] = a.y;
        } else {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + at + i * 32);
          v[i] = __uint_as_float(u << 16), v[i + 1] = __uint_as_float(u & 0xFFFF0000u);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (i * 32 < left) {
        if constexpr (F32)
          v[i] = static_cast<const float*>(base)[at + i * 32];
        else
          v[i] = bf16_to_f32(static_cast<const uint16_t*>(base)[at + i * 32]);
      }
    }
  }
}
template <bool F32, int VEC>
__device__ __forceinline__ void store8(void* base, int64_t at, int left, const float (&v)[8]) {
  if constexpr (VEC == 8) {
    if constexpr (F32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = f32_to_bf16(v[2 * i]) | static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
  } else if constexpr (VEC == 2) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      if (i * 32 < left) {
        if constexpr (F32)
          *reinterpret_cast<float2*>(static_cast<float*>(base) + at + i * 32) = make_float2(v[i], v[i + 1]);
        else
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + at + i * 32) =
              f32_to_bf16(v[i]) | static_cast<uint32_t>(f32_to_bf16(v[i + 1])) << 16;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i * 32 < left) {
        if constexpr (F32)
          static_cast<float*>(base)[at + i * 32] = v[i];
        else
          static_cast<uint16_t*>(base)[at + i * 32] = f32_to_bf16(v[i]);
      }
  }
}
template <int VEC>
__device__ __forceinline__ void load8(bool f32, const void* base, int64_t at, int left, float (&v)[8]) {
  if (f32)
    load8<true, VEC>(base, at, left, v);
  else
    load8<false, VEC>(base, at, left, v);
}

// The scale of a group whose largest magnitude has the bits `top`.
struct GroupScale {
  float scale;
  bool finite;
};
__device__ __forceinline__ GroupScale group_scale(uint32_t top) {
  GroupScale r;
  r.finite = top < 0x7F800000u;
  r.scale = r.finite ? __uint_as_float(top) / 448.f : __int_as_float(0x7FC00000);
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// What a code of a finite group is nearest to.
__device__ __forceinline__ float quotient(float y, float scale) { return scale > 0.f ? y / scale : 0.f; }
// The codes of eight elements.  A product with the reciprocal may lie on the
// other side of a border between two codes; but where products with a little
// less and with a little more than it (2^-21 of it: it, the factors, the
// products and the quotient are rounded, 2^-24 each) give the same codes, so do
// the quotients in between.  Else, in one of some 400 warps, they are divided
// (16384 x 4096 bf16, residual and both results: 95.6 us, with divisions alone
// 110.6).  fp32 rows have the time to divide (8192 x 4096, residual, codes: 70.5
// us, by products 73.5).
template <bool DIVIDE>
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float scale) {
  uint32_t u[2] = {}, v[2] = {};
  if constexpr (!DIVIDE) {
    const bool fine = scale > 1e-30f && scale < 1e30f;  // the reciprocal and the products are normal numbers
    const float inverse = 1.f / scale, less = fine ? inverse * (1.f - 0x1p-21f) : 0.f,
                more = fine ? inverse * (1.f + 0x1p-21f) : INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j / 2] |= e4m3x2(y[2 * j] * less, y[2 * j + 1] * less) << (j % 2 * 16);
      v[j / 2] |= e4m3x2(y[2 * j] * more, y[2 * j + 1] * more) << (j % 2 * 16);
    }
    if (u[0] == v[0] && u[1] == v[1]) return make_uint2(u[0], u[1]);
    u[0] = u[1] = 0u;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j / 2] |= e4m3x2(quotient(y[2 * j], scale), quotient(y[2 * j + 1], scale)) << (j % 2 * 16);
  return make_uint2(u[0], u[1]);
}

template <int STEPS, bool F32, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > kBlock ? 1 : STEPS > 2 ? 3 : STEPS == 2 ? 4 : 6) rms_norm_kernel(const NormArgs a, const int per_row) {
  __shared__ float partial[32];
  const int rows_here = blockDim.x / per_row, tid = threadIdx.x % per_row, lane = threadIdx.x % 32;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_here + threadIdx.x / per_row;
  const bool on = row < a.rows;
  // the first of a step's eight columns of this thread, and how many columns there are from it
  int col[STEPS];
  float h[STEPS][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int chunk = i * per_row + tid;  // of 8 columns
    col[i] = VEC == 8 ? chunk * 8 : chunk / 32 * 256 + lane * VEC;
    const int left = a.cols - col[i];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
    if (on && left > 0) {
      load8<F32, VEC>(a.x, row * a.ld_x + col[i], left, h[i]);
      if (a.residual != nullptr) {
        float r[8];
        load8<F32, VEC>(a.residual, row * a.ld_residual + col[i], left, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] += r[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (per_row > 32) {
    if (lane == 0) partial[threadIdx.x / 32] = sum;
    __syncthreads();
    const int first = threadIdx.x / per_row * (per_row / 32);
    sum = 0.f;
    for (int i = 0; i < per_row / 32; ++i) sum += partial[first + i];
  }
  const float factor = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int left = on ? a.cols - col[i] : 0;
    float y[8] = {};
    if (left > 0) {
      if (a.sum != nullptr) store8<F32, VEC>(a.sum, row * a.ld_sum + col[i], left, h[i]);
      load8<VEC>(a.weight_f32 != 0, a.weight, col[i], left, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= h[i][j] * factor;
      if (a.out != nullptr) {
        if (a.out_f32)
          store8<true, VEC>(a.out, row * a.ld_out + col[i], left, y);
        else
          store8<false, VEC>(a.out, row * a.ld_out + col[i], left, y);
      }
    }
    if (a.codes != nullptr) {  // (the same for all threads)
      const int groups = (a.cols + 127) / 128;
      uint32_t top[VEC == 8 ? 1 : 2] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t& t = top[VEC == 8 ? 0 : j / 4];
        t = max(t, __float_as_uint(y[j]) & 0x7FFFFFFFu);
      }
      if constexpr (VEC == 8) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
        if (left > 0) {
          const GroupScale s = group_scale(top[0]);
          *reinterpret_cast<uint2*>(a.codes + row * a.cols + col[i]) = s.finite ? codes8<F32>(y, s.scale) : make_uint2(0u, 0u);
          if (lane % 16 == 0) a.scales[row * groups + col[i] / 128] = s.scale;
        }
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const GroupScale s = group_scale(__reduce_max_sync(0xffffffffu, top[b]));
          if (b * 128 < left) {
            if (lane == 0) a.scales[row * groups + col[i] / 128 + b] = s.scale;
#pragma unroll
            for (int j = 4 * b; j < 4 * b + 4; j += VEC)
              if (j * 32 < left) {
                uint8_t* const to = a.codes + row * a.cols + col[i] + j * 32;
                const uint32_t u = s.finite ? e4m3x2(quotient(y[j], s.scale), VEC == 2 ? quotient(y[j + 1], s.scale) : 0.f) : 0u;
                if constexpr (VEC == 2)
                  *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(u);
                else
                  *to = static_cast<uint8_t>(u);
              }
          }
        }
      }
    }
  }
}

// Raw loads of 8 elements.
template <bool F32>
struct Raw {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = q[i];
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = __uint_as_float(F32 ? u[i] : i % 2 != 0 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
  }
};

// Many rows of 513 to 8192 columns that start on 16 bytes: blocks that stay,
// a row at a time, whose next row is on its way while this one is written
// (residual and both results, 16384 x 4096: 124 us a block per row, 108 with
// 4 blocks an SM, 95.6 with 3: 6.3 TB/s; 2048 x 4096: 18.6 a block per row, 14.4;
// 512 x 4096: 5.2, 5.8; 512 x 7168: 11.4, 8.6; 304 x 7168: 5.6, 7.3).
template <int THREADS, int STEPS>
constexpr int kRowBlocks = THREADS == kBlock ? (STEPS == 2 ? 3 : 2) : STEPS == 1 ? 8 : 6;  // of an SM

template <int THREADS, int STEPS, bool F32>
__global__ void __launch_bounds__(THREADS, kRowBlocks<THREADS, STEPS>) rms_norm_rows_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float partial[2][THREADS / 32];
  const int tid = threadIdx.x, lane = tid % 32;
  Raw<F32> x[STEPS], r[STEPS];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int col = (i * THREADS + tid) * 8;
      if (col < a.cols) {
        x[i].load(a.x, row * a.ld_x + col);
        if (a.residual != nullptr) r[i].load(a.residual, row * a.ld_residual + col);
      }
    }
  };
  int64_t row = blockIdx.x;
  int turn = 0;
  fetch(row);
  for (; row < a.rows; row += gridDim.x) {
    float h[STEPS][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int col = (i * THREADS + tid) * 8;
      if (col < a.cols) {
        x[i].floats(h[i]);
        if (a.residual != nullptr) {
          float f[8];
          r[i].floats(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[i][j] += f[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
    }
    if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) partial[turn][tid / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) sum += partial[turn][i];
    turn ^= 1;
    const float factor = 1.f / sqrtf(sum / static_cast<float>(a.cols) + a.eps);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int col = (i * THREADS + tid) * 8;
      float y[8] = {};
      if (col < a.cols) {
        if (a.sum != nullptr) store8<F32, 8>(a.sum, row * a.ld_sum + col, 8, h[i]);
        load8<8>(a.weight_f32 != 0, a.weight, col, 8, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= h[i][j] * factor;
        if (a.out != nullptr) {
          if (a.out_f32)
            store8<true, 8>(a.out, row * a.ld_out + col, 8, y);
          else
            store8<false, 8>(a.out, row * a.ld_out + col, 8, y);
        }
      }
      if (a.codes != nullptr) {
        uint32_t top = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(y[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (col < a.cols) {
          const GroupScale s = group_scale(top);
          *reinterpret_cast<uint2*>(a.codes + row * a.cols + col) = s.finite ? codes8<F32>(y, s.scale) : make_uint2(0u, 0u);
          if (lane % 16 == 0) a.scales[row * ((a.cols + 127) / 128) + col / 128] = s.scale;
        }
      }
    }
  }
}

template <int STEPS, bool F32, int VEC>
cudaError_t launch(const NormArgs& a, int per_row, cudaStream_t s) {
  const int threads = per_row < kBlock ? kBlock : per_row, rows_here = threads / per_row;
  const dim3 grid(static_cast<unsigned>((a.rows + rows_here - 1) / rows_here));
  if (threads > kBlock) return launch_kernel(rms_norm_kernel<STEPS, F32, VEC, kMaxThreads>, grid, dim3(threads), 0, s, a, per_row);
  return launch_kernel(rms_norm_kernel<STEPS, F32, VEC, kBlock>, grid, dim3(threads), 0, s, a, per_row);
}
template <bool F32, int VEC>
cudaError_t launch_steps(const NormArgs& a, int num_sms, cudaStream_t s) {
  const int chunks = (a.cols + 255) / 256 * 32;  // of 8 columns; unaligned rows take them by warps
  // Few rows: as many threads as there are chunks, the shortest way through a
  // row.  Many: blocks of 256 threads while 4 steps suffice, more rows in
  // flight (16384 x 4096 that way, with codes by the reciprocal: 146 us with 512
  // threads a row, 126 with 128, 110 with 256).
  int per_row = 32;
  while (per_row < kMaxThreads && per_row < chunks &&
         (per_row < kBlock || a.rows <= 2 * num_sms || 4 * per_row < chunks))
    per_row *= 2;
  if constexpr (VEC == 8) {
    if (a.rows >= (chunks > 512 ? 3 : 4) * num_sms && chunks > 64 && chunks <= 1024) {
      auto rows = [&](auto kernel, int threads, int blocks) {
        // (a block has a row at least: its first is fetched unasked)
        return launch_kernel(kernel, dim3(static_cast<unsigned>(std::min<int64_t>(a.rows, num_sms * blocks))), dim3(threads), 0, s, a);
      };
      if (chunks <= 128) return rows(rms_norm_rows_kernel<128, 1, F32>, 128, kRowBlocks<128, 1>);
      if (chunks <= 256) return rows(rms_norm_rows_kernel<128, 2, F32>, 128, kRowBlocks<128, 2>);
      if (chunks <= 512) return rows(rms_norm_rows_kernel<kBlock, 2, F32>, kBlock, kRowBlocks<kBlock, 2>);
      return rows(rms_norm_rows_kernel<kBlock, 4, F32>, kBlock, kRowBlocks<kBlock, 4>);
    }
  }
  const int steps = (chunks + per_row - 1) / per_row;
  if (steps <= 1) return launch<1, F32, VEC>(a, per_row, s);
  if (steps <= 2) return launch<2, F32, VEC>(a, per_row, s);
  return launch<4, F32, VEC>(a, per_row, s);
}

// Rows that all start on `bytes` bytes.
bool on(const void* p, int64_t ld, int size, unsigned bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * size) & (bytes - 1)) == 0;
}
// Whether the columns, and all rows, are whole pieces of n (8: of 16 bytes at least).
bool in_pieces(const NormArgs& a, int n) {
  const int size = a.f32 ? 4 : 2, out_size = a.out_f32 ? 4 : 2, weight_size = a.weight_f32 ? 4 : 2;
  auto bytes = [&](int of) { return static_cast<unsigned>(n == 8 ? 16 : n * of); };
  return a.cols % n == 0 && on(a.x, a.ld_x, size, bytes(size)) && on(a.residual, a.ld_residual, size, bytes(size)) &&
         on(a.sum, a.ld_sum, size, bytes(size)) && on(a.weight, 0, 1, bytes(weight_size)) &&
         on(a.out, a.ld_out, out_size, bytes(out_size)) && on(a.codes, 0, 1, static_cast<unsigned>(n));
}

template <bool F32>
cudaError_t launch_type(const NormArgs& a, int num_sms, cudaStream_t s) {
  if (in_pieces(a, 8)) return launch_steps<F32, 8>(a, num_sms, s);
  return in_pieces(a, 2) ? launch_steps<F32, 2>(a, num_sms, s) : launch_steps<F32, 1>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t s) {
  return a.f32 ? launch_type<true>(a, num_sms, s) : launch_type<false>(a, num_sms, s);
}

}  // namespace cbmoe
