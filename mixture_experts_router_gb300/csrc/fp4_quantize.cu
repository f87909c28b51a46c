// Quantisation to 4-bit floating point with block scales and its way back.
//
// Bound by memory: 2 or 4 bytes an element in, half a byte and a 16th or 32nd
// out (28672 x 4096 bf16, mx: 55 us, 5.4 TB/s, and 49 us, 6.1 TB/s, back).  NV is
// bound by its arithmetic (two conversions of each element) and, in bf16, by
// the elements next to a border, which are common there: 89 to 234 us by the
// data and g, with L2 flushed before (mx alike: 63), fp32 98 (mx: 94).  A
// block of 256 threads takes a tile of 128 rows x 256 columns, a thread 8
// consecutive elements of 16 rows (16 bytes of bf16, so a warp reads 512-byte
// runs), kBatch rows' loads ahead of their arithmetic.  The largest magnitude
// of a block of 32 or 16 elements is a maximum over 4 or 2 neighbouring lanes,
// taken on the bit patterns (so a NaN or an infinity comes out on top).  The
// scales of the tile are gathered in shared memory in the order of the scale
// array, which makes them whole 512-byte stores with the padding's zeros in
// place.
//
// Exactness.  MX divides by a power of two, which is exact.  For NV the
// quotients a / (6 g) and x / (s g) are computed in fp32, each off by at most
// 2^-22 of itself, and rounded twice, scaled down and up by kNear = 2^-20;
// where the two codes agree they are the exact quotient's.  Where not, the
// quotient lies next to the border b of two codes, and the sign of
// fma(b s, g, -|x|), whose only rounding cannot change its sign, decides; zero
// is a tie, which goes to the even code.  (b s is exact: 3 and 4 significant
// bits.)  Where g is so small or large that fp32 could under- or overflow on
// the way, everything is done in 64 bits.
#include <cuda_bf16.h>

#include <type_traits>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cbmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kTileCols = 256;
constexpr int kTileRows = kScaleTileRows;
constexpr int kRowsAtOnce = kThreads / (kTileCols / 8);
constexpr int kBatch = 4;
constexpr int kTileBatches = kTileRows / kRowsAtOnce / kBatch;  // of 32 rows
constexpr float kNear = 9.5367431640625e-07f;  // 2^-20

template <int FMT>
constexpr int kScaleTiles = kTileCols / (4 * kFp4Block<FMT>);  // 512-byte scale tiles per tile

// Eight elements as floats from a row, `VEC`: it starts on 16 bytes.
template <typename T, bool VEC>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
      T e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = __ldg(p + i);
      memcpy(v, e, sizeof(v));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void floats(float (&f)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4)
        f[i] = __uint_as_float(u[i]);
      else
        f[i] = __uint_as_float((i & 1) ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
    }
  }
};

__device__ __forceinline__ uint32_t e4m3_code(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xFFu;
}

// Border between the magnitudes of codes c and c + 1 (c in 0..6): e2m1's bits
// with a mantissa bit 1 behind them.
__device__ __forceinline__ float border_above(uint32_t c) {
  return __uint_as_float(((2u * c + 1u) << 21)) * __uint_as_float(253u << 23);
}

struct NvScale {
  float g, six_g;
  bool wide;  // fp32 may under- or overflow on the way: 64 bits throughout
};

// Nearest e4m3 code of a / (6 g), a >= 0 finite.
__device__ __forceinline__ uint32_t nv_scale_code(float a, const NvScale& n) {
  const float t = n.wide ? static_cast<float>(static_cast<double>(a) / (6.0 * n.g)) : a / n.six_g;
  const uint32_t lo = e4m3_code(t * (1.f - kNear)), hi = e4m3_code(t * (1.f + kNear));
  if (lo == hi) return lo;
  const double mid = 0.5 * (static_cast<double>(e4m3_value(lo)) + static_cast<double>(e4m3_value(hi)));
  const double border = mid * 6.0 * static_cast<double>(n.g);  // 5 + 2 + 24 significant bits: exact
  if (a > border) return hi;
  if (a < border) return lo;
  return (lo & 1u) ? hi : lo;
}

// Codes of eight elements over s g.
__device__ __forceinline__ uint32_t nv_codes(const float (&x)[8], float s, const NvScale& n) {
  if (s == 0.f) return 0u;
  float lo[8], hi[8];
  if (!n.wide) {
    const float inv = 1.f / (s * n.g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = x[i] * inv * (1.f - kNear);
      hi[i] = x[i] * inv * (1.f + kNear);
    }
  } else {
    const double inv = 1.0 / (static_cast<double>(s) * n.g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = static_cast<float>(x[i] * inv) * (1.f - kNear);
      hi[i] = static_cast<float>(x[i] * inv) * (1.f + kNear);
    }
  }
  uint32_t c = e2m1x8(lo);
  const uint32_t d = c ^ e2m1x8(hi);
  if (d == 0u) return c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (((d >> (4 * i)) & 15u) == 0u) continue;
    const uint32_t m = (c >> (4 * i)) & 7u;  // the lower magnitude; m + 1 is the other
    const float b = border_above(m) * s;
    bool up;
    if (!n.wide) {
      const float r = fmaf(b, n.g, -fabsf(x[i]));
      up = r < 0.f || (r == 0.f && (m & 1u));
    } else {
      const double v = static_cast<double>(b) * n.g, a = fabsf(x[i]);
      up = a > v || (a == v && (m & 1u));
    }
    if (up) c += 1u << (4 * i);
  }
  return c;
}

// PARTS blocks share a tile: 1, or a batch of 32 rows each.
template <int FMT, typename T, bool VEC, int PARTS>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const T* x, int64_t rows, int64_t cols, int64_t ld,
                                                                const float* tensor_scale, uint8_t* codes,
                                                                uint8_t* scales, int64_t col_tiles) {
  constexpr int LANES = kFp4Block<FMT> / 8;  // lanes that share a block
  __shared__ __align__(16) uint8_t tile[kScaleTiles<FMT> * kScaleTileBytes];
  const int at = static_cast<int>(blockIdx.x / PARTS), part = static_cast<int>(blockIdx.x % PARTS);
  const int64_t row0 = (at / col_tiles) * kTileRows;
  const int64_t col0 = (at % col_tiles) * kTileCols;
  const int lane = threadIdx.x % 32;
  const int64_t col = col0 + lane * 8;
  const bool in = col < cols;
  for (int i = threadIdx.x; i < kScaleTiles<FMT> * kScaleTileBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
  grid_dep_wait();
  NvScale nv{};
  if constexpr (FMT == kFp4Nv) {
    // the g of a matrix of zeros is 0: as an infinite one, it leaves every scale and code 0
    const float g = __ldg(tensor_scale);
    nv.g = g > 0.f ? g : __uint_as_float(0x7F800000u);
    nv.six_g = 6.f * nv.g;
    nv.wide = !(nv.g > 0x1p-80f && nv.g < 0x1p+80f);
  }
  __syncthreads();
  const int first = threadIdx.x / 32;
  const int i_first = part * kBatch, i_end = PARTS == 1 ? kTileRows / kRowsAtOnce : i_first + kBatch;
  for (int i0 = i_first; i0 < i_end; i0 += kBatch) {
    if (row0 + i0 * kRowsAtOnce >= rows) break;
    Eight<T, VEC> v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t r = row0 + first + (i0 + i) * kRowsAtOnce;
      if (in && r < rows)
        v[i].load(x + r * ld + col);
      else
        v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int rt = first + (i0 + i) * kRowsAtOnce;
      float f[8];
      v[i].floats(f);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 1; o < LANES; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      uint32_t byte, c;
      if constexpr (FMT == kFp4Mx) {
        // the largest's exponent field less 2 (a subnormal's is below the range: 0)
        byte = static_cast<uint32_t>(max(static_cast<int>(top >> 23) - 2, 0));
        const float up = __uint_as_float((254u - min(byte, 252u)) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= up;
        c = e2m1x8(f);
      } else {
        const bool finite = top < 0x7F800000u;
        byte = nv_scale_code(finite ? __uint_as_float(top) : 0.f, nv);
        c = finite ? nv_codes(f, e4m3_value(byte), nv) : 0u;
      }
      if (top >= 0x7F800000u) {
        byte = FMT == kFp4Mx ? 255u : 0x7Fu;
        c = 0u;
      }
      const int64_t r = row0 + rt;
      if (in && r < rows) {
        *reinterpret_cast<uint32_t*>(codes + r * (cols / 2) + col / 2) = c;
        const int j = lane / LANES;  // block of the tile's columns
        if (lane % LANES == 0) tile[j / 4 * kScaleTileBytes + scale_tile_byte(rt, j % 4)] = static_cast<uint8_t>(byte);
      }
    }
  }
  __syncthreads();
  const int64_t scale_cols = (cols / kFp4Block<FMT> + 3) / 4;  // scale tiles per row tile
  const int64_t t0 = col0 / (4 * kFp4Block<FMT>);
  const int n = static_cast<int>(min(static_cast<int64_t>(kScaleTiles<FMT>), scale_cols - t0)) * (kScaleTileBytes / 16);
  uint4* dst = reinterpret_cast<uint4*>(scales + ((row0 / kTileRows) * scale_cols + t0) * kScaleTileBytes);
  // (16 bytes of the array are a row's 4 scales in each of the tile's batches)
  for (int i = threadIdx.x; i < n; i += kThreads) {
    if constexpr (PARTS == 1)
      dst[i] = reinterpret_cast<const uint4*>(tile)[i];
    else
      reinterpret_cast<uint32_t*>(dst + i)[part] = reinterpret_cast<const uint32_t*>(tile)[i * 4 + part];
  }
}

// The same tiles the other way; a thread turns 4 bytes of codes into 8 values.
template <int FMT, typename T, bool VEC, int PARTS>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                  const float* tensor_scale, int64_t rows,
                                                                  int64_t cols, T* out, int64_t ld,
                                                                  int64_t col_tiles) {
  const int at = static_cast<int>(blockIdx.x / PARTS), part = static_cast<int>(blockIdx.x % PARTS);
  const int64_t row0 = (at / col_tiles) * kTileRows;
  const int64_t col = (at % col_tiles) * kTileCols + threadIdx.x % 32 * 8;
  if (col >= cols) return;
  grid_dep_wait();
  const int64_t scale_cols = (cols / kFp4Block<FMT> + 3) / 4;
  const int64_t j = col / kFp4Block<FMT>;
  const uint8_t* sp = scales + ((row0 / kTileRows) * scale_cols + j / 4) * kScaleTileBytes;
  float g = 1.f;
  if constexpr (FMT == kFp4Nv) g = __ldg(tensor_scale);
  const int first = threadIdx.x / 32;
  const int i_first = part * kBatch, i_end = PARTS == 1 ? kTileRows / kRowsAtOnce : i_first + kBatch;
  for (int i0 = i_first; i0 < i_end; i0 += kBatch) {
    uint32_t c[kBatch], s[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int rt = first + (i0 + i) * kRowsAtOnce;
      c[i] = s[i] = 0u;
      if (row0 + rt < rows) {
        c[i] = __ldg(reinterpret_cast<const uint32_t*>(codes + (row0 + rt) * (cols / 2) + col / 2));
        s[i] = __ldg(sp + scale_tile_byte(rt, static_cast<int>(j % 4)));
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t r = row0 + first + (i0 + i) * kRowsAtOnce;
      if (r >= rows) continue;
      const float sv = scale_value<FMT>(s[i]);
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = e2m1_value(c[i] >> (4 * e)) * sv;
        if constexpr (FMT == kFp4Nv) v[e] *= g;
      }
      T* p = out + r * ld + col;
      if constexpr (sizeof(T) == 4) {
        if constexpr (VEC) {
          reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) reinterpret_cast<float*>(p)[e] = v[e];
        }
      } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if constexpr (VEC) {
          *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
      }
    }
  }
}

bool rows_on_16(const void* p, int64_t ld, int64_t elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * elem % 16 == 0;
}

// Where there are not two tiles for each SM, a tile is shared by a block per
// batch, which has a quarter of the latency to sit through (nv, bf16, 50
// tiles: 4.1 us against 10.3, and 2.3 against 4.1 back; 288 tiles: 8.8 against
// 9.0).
int parts_of(const Fp4Args& a, int num_sms) { return fp4_tiles(a.rows, a.cols) < 2 * num_sms ? kTileBatches : 1; }

template <int FMT, typename T, bool VEC, int PARTS>
cudaError_t quantize(const Fp4Args& a, cudaStream_t s) {
  const int64_t ct = (a.cols + kTileCols - 1) / kTileCols;
  return launch_kernel(fp4_quantize_kernel<FMT, T, VEC, PARTS>, static_cast<unsigned>(fp4_tiles(a.rows, a.cols) * PARTS),
                       kThreads, 0, s, static_cast<const T*>(a.x), a.rows, a.cols, a.ld, a.tensor_scale, a.codes,
                       a.scales, ct);
}

template <int FMT, typename T, bool VEC, int PARTS>
cudaError_t dequantize(const Fp4Args& a, cudaStream_t s) {
  const int64_t ct = (a.cols + kTileCols - 1) / kTileCols;
  return launch_kernel(fp4_dequantize_kernel<FMT, T, VEC, PARTS>,
                       static_cast<unsigned>(fp4_tiles(a.rows, a.cols) * PARTS), kThreads, 0, s,
                       const_cast<const uint8_t*>(a.codes), const_cast<const uint8_t*>(a.scales), a.tensor_scale, a.rows,
                       a.cols, static_cast<T*>(a.x), a.ld, ct);
}

// f(format, a value of the element type, whether rows start on 16 bytes, parts), all as types
template <typename F>
cudaError_t with_types(const Fp4Args& a, int num_sms, F&& f) {
  const auto parts = [&](auto fmt, auto t, auto vec) {
    return parts_of(a, num_sms) == 1 ? f(fmt, t, vec, std::integral_constant<int, 1>{})
                                     : f(fmt, t, vec, std::integral_constant<int, kTileBatches>{});
  };
  const auto rows = [&](auto fmt, auto t) {
    return rows_on_16(a.x, a.ld, sizeof(t)) ? parts(fmt, t, std::true_type{}) : parts(fmt, t, std::false_type{});
  };
  const auto type = [&](auto fmt) { return a.f32 ? rows(fmt, float{}) : rows(fmt, uint16_t{}); };
  return a.format == kFp4Mx ? type(std::integral_constant<int, kFp4Mx>{}) : type(std::integral_constant<int, kFp4Nv>{});
}

}  // namespace

int64_t fp4_tiles(int64_t rows, int64_t cols) {
  return (rows + kTileRows - 1) / kTileRows * ((cols + kTileCols - 1) / kTileCols);
}

cudaError_t launch_fp4_quantize(const Fp4Args& a, int num_sms, cudaStream_t s) {
  return with_types(a, num_sms, [&](auto fmt, auto t, auto vec, auto parts) {
    return quantize<decltype(fmt)::value, decltype(t), decltype(vec)::value, decltype(parts)::value>(a, s);
  });
}

cudaError_t launch_fp4_dequantize(const Fp4Args& a, int num_sms, cudaStream_t s) {
  return with_types(a, num_sms, [&](auto fmt, auto t, auto vec, auto parts) {
    return dequantize<decltype(fmt)::value, decltype(t), decltype(vec)::value, decltype(parts)::value>(a, s);
  });
}

}  // namespace cbmoe
