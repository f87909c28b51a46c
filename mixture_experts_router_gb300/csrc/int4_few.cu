// A few rows (1 to 16) by 4-bit integer weights with a scale and a zero point
// per group of 32, 64 or 128 elements of a row:
//
//   y[t][j] = sum_g s[g][j] sum_{i in g} x[t][i] (q[j][i] - z[g][j]),
//
// one matrix, or one per expert with the experts of each row given; then the
// rows as they are, silu(gate) * up, or the weighted sum over a row's experts.
//
// What bounds it: the weights, read once from HBM (of an expert with more rows
// than a part holds, once per part), and the instructions that widen them.
// A warp takes tiles of 32 weight rows (SwiGLU: 16 features' gate and up
// rows), a stage of 256 elements (128 bytes of a row) at a time, through a ring
// in shared memory of its own that cp.async fills: with no thread but its own
// 32 to wait for, a warp needs no barrier to keep its loads in flight across
// stages, tiles and experts.  A stage brings the tile's codes, scales and zero
// points and the same stretch of its rows of x.  The codes become bf16 (8-bit
// x: fp16) exactly in registers and go through mma.sync m16n8k16 (A: weight
// rows, B: up to 8 rows of x per n-tile); a group's sum is taken from zero and
// joins the tile's sum with its scale, in fp32, so that no weight is rounded.
//
// Layouts.  A dot product does not depend on the order of its terms: within a
// group thread q of a quad owns a quarter of the group's consecutive elements,
// so it reads its codes in one piece of 4, 8 or 16 bytes.  The 16-byte units
// of a row stand at unit ^ key(row), the units of x in the order in which the
// quads read them: no bank conflicts either way.  Row 2g and 2g + 1 of each
// half of a tile are lane group g's, so its scales and zero points are pairs.
//
// Warps: `ks` of a block's eight share a tile, taking its stages in turn, where
// there would be fewer tiles than warps; their sums are joined in order.  The
// weighted sum has one tile per block at a time, all experts' stages going to
// the eight warps in turn.  All sums are in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 32;            // weight rows of a tile: two m16 fragments
constexpr int kMaxPairs = 256;       // (row of x, slot)
constexpr int kMaxExperts = 256;
constexpr int kRedStride = 36;       // floats: the fragments' stores meet no bank twice
constexpr int kMaxTokens = kFewTokens;

// Elements of a row in a stage: with 16 rows of x beside them, half as many.
template <int NT>
constexpr int kStageOf = NT == 1 ? 256 : 128;

// Bytes of a stage for nx rows of x: codes, scales, x, zero points, x scales.
template <int GROUP, int NT, bool F8>
__host__ __device__ constexpr int stage_bytes(int nx) {
  constexpr int K = kStageOf<NT>;
  return (kRows * K / 2 + K / GROUP * kRows * 5 + nx * (F8 ? K + K / 32 : 2 * K) + 127) / 128 * 128;
}

template <int NT>
struct Shared {
  float red[kWarps][NT * 8][kRedStride];  // sums of a tile: [warp][row of x][weight row]
  uint8_t pair[kMaxPairs];      // pairs by expert, then in order
  int16_t act[kMaxPairs];       // parts: their expert,
  int16_t first[kMaxPairs];     //   first entry of `pair`
  uint8_t count[kMaxPairs];     //   and number of them
  uint32_t bad[kMaxPairs / 32]; // pairs whose expert does not exist
  int warp_parts[kWarps];
  int n_parts;
};

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_pending() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes of a word minus their zero point, pairs of elements m and m + 4.
// bf16: a nibble n in a half word under 0x4300 is 128 + n.  fp16: under 0x6400
// 1024 + n, and one bit field further up 1024 + 16 n, so two shifts fewer:
// (1024 + 16 n) / 16 - (64 + z).  All of it is exact.
template <bool F8>
struct Zero {
  uint32_t a, b;
  __device__ __forceinline__ void set(uint32_t z) {
    if constexpr (F8) {
      a = (0x6400u | z) * 0x00010001u;
      b = (0xD400u | z << 4) * 0x00010001u;  // -(64 + z)
    } else {
      a = (0x4300u | z) * 0x00010001u;
    }
  }
};
template <bool F8>
__device__ __forceinline__ void widen(uint32_t v, const Zero<F8>& z, uint32_t (&o)[4]) {
  if constexpr (F8) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t lo, hi;
      asm("lop3.b32 %0, %1, 0x000F000F, 0x64006400, 0xEA;" : "=r"(lo) : "r"(v >> (8 * j)));
      asm("lop3.b32 %0, %1, 0x00F000F0, 0x64006400, 0xEA;" : "=r"(hi) : "r"(v >> (8 * j)));
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * j]) : "r"(lo), "r"(z.a));
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[2 * j + 1]) : "r"(hi), "r"(0x2C002C00u), "r"(z.b));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t n;
      asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(n) : "r"(v >> (4 * j)));
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(n), "r"(z.a));
    }
  }
}

// The lane group's place among the 16-byte units of a row: bits reversed, so
// that neighbouring groups differ first in the widest reads' own bit.
__device__ __forceinline__ int unit_key(int g) { return (g & 1) << 2 | (g & 2) | g >> 2; }

template <int GROUP, int NT, bool F8, int DEPTH>
struct Worker {
  static constexpr int kStageK = kStageOf<NT>;
  static constexpr int kRowBytes = kStageK / 2;
  static constexpr int kGroups = kStageK / GROUP;         // of a stage
  static constexpr int kTokBytes = F8 ? kStageK : 2 * kStageK;  // a row of x in a stage
  static constexpr int kWords = GROUP / 32;               // of a thread, row and group
  const Int4Args& p;
  Shared<NT>& s;
  uint8_t* ring;
  const int warp, lane, g, q;
  const int bytes;      // of a stage
  const int nst;        // stages of a row
  const int tiles;      // of a matrix
  int slot_in = 0, slot_out = 0;

  // Where the loads, or the arithmetic, stand: the tile, its part, the stage.
  struct Place {
    int sub, part, tile, st;
  };
  Place in;
  int end;              // of the tiles to be walked
  int step;

  __device__ __forceinline__ Worker(const Int4Args& p_, Shared<NT>& s_, uint8_t* ring_)
      : p(p_),
        s(s_),
        ring(ring_ + (threadIdx.x / 32) * (DEPTH * stage_bytes<GROUP, NT, F8>(p_.nx))),
        warp(threadIdx.x / 32),
        lane(threadIdx.x % 32),
        g(threadIdx.x % 32 >> 2),
        q(threadIdx.x & 3),
        bytes(stage_bytes<GROUP, NT, F8>(p_.nx)),
        nst((p_.k + kStageK - 1) / kStageK),
        tiles(((p_.swiglu ? p_.n / 2 : p_.n) + tile_out(p_) - 1) / tile_out(p_)) {}
  __device__ __forceinline__ static int tile_out(const Int4Args& p) { return p.swiglu ? kRows / 2 : kRows; }

  // Weight row of row r of a tile; rows past the end are the last one again.
  __device__ __forceinline__ int weight_row(int tile, int r) const {
    if (p.swiglu) {
      const int f = p.n / 2;
      return (r >= kRows / 2 ? f : 0) + min(tile * (kRows / 2) + r % (kRows / 2), f - 1);
    }
    return min(tile * kRows + r, p.n - 1);
  }
  __device__ __forceinline__ int x_row(int pair) const { return p.x_per_slot ? pair : pair / p.top; }

  // ------------------------------------------------------------- the walk
  __device__ __forceinline__ void settle(Place& a) const {  // the weighted sum's stages go on into the next part
    while (a.st >= nst && a.part < s.n_parts) {
      a.st -= nst;
      ++a.part;
    }
    if (a.part >= s.n_parts) {
      a.sub += step;
      a.part = s.n_parts;
    }
  }
  __device__ __forceinline__ void start(Place& a, int sub) const {
    a.sub = sub;
    if (p.w != nullptr) {
      a.tile = sub;
      a.part = 0;
      a.st = warp;
      settle(a);
      // a warp without a stage in one tile has none in any
      if (a.sub != sub) a.sub = end;
    } else {
      a.part = sub / tiles;
      a.tile = sub % tiles;
      a.st = warp % p.ks;
    }
  }
  __device__ __forceinline__ bool any(const Place& a) const { return a.sub < end; }
  __device__ __forceinline__ void next(Place& a) const {
    if (p.w != nullptr) {
      a.st += kWarps;
      const int sub = a.sub;
      settle(a);
      if (a.sub != sub) start(a, a.sub);
    } else {
      a.st += p.ks;
      if (a.st >= nst) start(a, a.sub + step);
    }
  }

  // -------------------------------------------------------------- a stage
  __device__ __forceinline__ void issue() {
    if (any(in)) {
      uint8_t* dst = ring + slot_in * bytes;
      const int e = s.act[in.part], k0 = in.st * kStageK, left = p.k - k0;
      const int64_t row_bytes = p.k / 2;
      const uint8_t* codes = p.codes + static_cast<int64_t>(e) * p.n * row_bytes + k0 / 2;
      constexpr int kPer = kRowBytes / 16;  // units of a row
      const int unit = lane % kPer;
      if (unit * 32 < left) {
#pragma unroll
        for (int i = 0; i < kRows * kPer / 32; ++i) {
          const int r = i * (32 / kPer) + lane / kPer;
          cp_async_16(dst + code_unit(r, unit, r >> 1 & 7), codes + weight_row(in.tile, r) * row_bytes + unit * 16);
        }
      }
      // scales: units of 4 rows; zero points: units of 8
      uint8_t* scales = dst + kRows * kRowBytes;
      uint8_t* x = scales + kGroups * kRows * 4;
      uint8_t* zeros = x + p.nx * kTokBytes;
      const int64_t meta = (static_cast<int64_t>(e) * (p.k / GROUP) + k0 / GROUP) * p.n;
#pragma unroll
      for (int i = 0; i < (kGroups * 8 + 31) / 32; ++i) {
        const int u = i * 32 + lane, gi = u / 8, r = u % 8 * 4;
        if (gi < kGroups && gi * GROUP < left && in_rows(in.tile, r))
          cp_async_16(scales + u * 16, p.scales + meta + static_cast<int64_t>(gi) * p.n + weight_row(in.tile, r));
      }
      if (p.zeros != nullptr) {
        const int gi = lane / 4, r = lane % 4 * 8;
        if (gi < kGroups && gi * GROUP < left && in_rows(in.tile, r))
          cp_async_8(zeros + lane * 8, p.zeros + meta + static_cast<int64_t>(gi) * p.n + weight_row(in.tile, r));
      }
      // x: 8 elements to a lane
      const int count = s.count[in.part], first = s.first[in.part];
      constexpr int kUnits = GROUP / 8, kLanes = kStageK / 8;  // of a group; of a row of x
      const int u = lane % kLanes;
      const int at = u / kUnits * kUnits + u % kWords * 4 + u % kUnits / kWords;
      if (u * 8 < left)
        for (int t = lane / kLanes; t < count; t += 32 / kLanes) {
          const int64_t row = x_row(s.pair[first + t]);
          if constexpr (F8)
            cp_async_8(x + t * kTokBytes + ((at ^ (t & 3) << 2) << 3),
                       static_cast<const uint8_t*>(p.x) + row * p.ld_x + k0 + u * 8);
          else
            cp_async_16(x + t * kTokBytes + ((at ^ (t & 1) << 2) << 4),
                        static_cast<const uint16_t*>(p.x) + row * p.ld_x + k0 + u * 8);
        }
      if constexpr (F8) {
        float* xs = reinterpret_cast<float*>(zeros + kGroups * kRows);
        constexpr int kScales = kStageK / 128;
        const int t = lane / kScales, h = lane % kScales;
        if (t < count && h * 128 < left)
          cp_async_4(xs + lane, p.x_scales + static_cast<int64_t>(x_row(s.pair[first + t])) * ((p.k + 127) / 128) +
                                    k0 / 128 + h);
      }
      next(in);
    }
    cp_async_commit();
    slot_in = slot_in + 1 == DEPTH ? 0 : slot_in + 1;
  }
  // byte of 16-byte unit `unit` of row r, one of lane group g's, in a stage
  __device__ __forceinline__ static int code_unit(int r, int unit, int g) {
    const int u = r * (kRowBytes / 16) + unit;
    return (u ^ unit_key(g)) << 4;
  }
  // whether the rows from r of a tile are the matrix's (all of r's 4 or 8 are, or none is)
  __device__ __forceinline__ bool in_rows(int tile, int r) const {
    return p.swiglu ? tile * (kRows / 2) + r % (kRows / 2) < p.n / 2 : tile * kRows + r < p.n;
  }

  __device__ __forceinline__ void clear(float (&v)[2][NT][4]) const {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) v[m][n][0] = v[m][n][1] = v[m][n][2] = v[m][n][3] = 0.f;
  }

  // acc += the oldest stage in the ring, which is stage st of a part of `count` rows.
  __device__ __forceinline__ void take(int st, int count, float (&acc)[2][NT][4]) {
    cp_async_wait_pending<DEPTH - 2>();
    __syncwarp();
    issue();
    const uint8_t* src = ring + slot_out * bytes;
    slot_out = slot_out + 1 == DEPTH ? 0 : slot_out + 1;
    const uint8_t* scales = src + kRows * kRowBytes;
    const uint8_t* x = scales + kGroups * kRows * 4;
    const uint8_t* zeros = x + p.nx * kTokBytes;
    const float* xs = reinterpret_cast<const float*>(zeros + kGroups * kRows);
    const int groups = min(kGroups, (p.k - st * kStageK) / GROUP);
    int tok[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) tok[n] = min(n * 8 + g, count - 1);
    const bool wide = count > 8;
#pragma unroll
    for (int gi = 0; gi < kGroups; ++gi) {
      if (gi >= groups) break;
      uint32_t v[4][kWords];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (j >> 1) * 16 + 2 * g + (j & 1);
        const int unit = gi * (GROUP / 32) + q * kWords / 4;
        const uint8_t* at = src + code_unit(r, unit, g) + (q * kWords % 4) * 4;
        if constexpr (kWords == 4) {
          const uint4 w = *reinterpret_cast<const uint4*>(at);
          v[j][0] = w.x, v[j][1] = w.y, v[j][2] = w.z, v[j][3] = w.w;
        } else if constexpr (kWords == 2) {
          const uint2 w = *reinterpret_cast<const uint2*>(at);
          v[j][0] = w.x, v[j][1] = w.y;
        } else {
          v[j][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      Zero<F8> zz[4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t z = 0x0808u;
        if (p.zeros != nullptr) z = *reinterpret_cast<const uint16_t*>(zeros + gi * kRows + m * 16 + 2 * g);
        zz[2 * m].set(z & 15u);
        zz[2 * m + 1].set(z >> 8 & 15u);
      }
      float sum[2][NT][4];
      clear(sum);
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n > 0 && !wide) break;
          const int unit = gi * (GROUP / 8) + w * 4 + q;
          if constexpr (F8) {
            const uint2 e = *reinterpret_cast<const uint2*>(x + tok[n] * kTokBytes +
                                                            ((unit ^ (tok[n] & 3) << 2) << 3));
            const uint32_t lo = __byte_perm(e.x, e.y, 0x5140), hi = __byte_perm(e.x, e.y, 0x7362);
            const uint16_t h[4] = {static_cast<uint16_t>(lo), static_cast<uint16_t>(lo >> 16), static_cast<uint16_t>(hi),
                                   static_cast<uint16_t>(hi >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b[n][i]) : "h"(h[i]));
          } else {
            const uint4 e = *reinterpret_cast<const uint4*>(x + tok[n] * kTokBytes +
                                                            ((unit ^ (tok[n] & 1) << 2) << 4));
            b[n][0] = __byte_perm(e.x, e.z, 0x5410);
            b[n][1] = __byte_perm(e.x, e.z, 0x7632);
            b[n][2] = __byte_perm(e.y, e.w, 0x5410);
            b[n][3] = __byte_perm(e.y, e.w, 0x7632);
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a0[4], a1[4];
          widen<F8>(v[2 * m][w], zz[2 * m], a0);
          widen<F8>(v[2 * m + 1][w], zz[2 * m + 1], a1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n > 0 && !wide) break;
            if constexpr (F8) {
              mma_f16(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
              mma_f16(sum[m][n], a0[2], a1[2], a0[3], a1[3], b[n][2], b[n][3]);
            } else {
              router_detail::mma_bf16(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
              router_detail::mma_bf16(sum[m][n], a0[2], a1[2], a0[3], a1[3], b[n][2], b[n][3]);
            }
          }
        }
      }
      const float2 s0 = *reinterpret_cast<const float2*>(scales + (gi * kRows + 2 * g) * 4);
      const float2 s1 = *reinterpret_cast<const float2*>(scales + (gi * kRows + 16 + 2 * g) * 4);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n > 0 && !wide) break;
        float x0 = 1.f, x1 = 1.f;
        if constexpr (F8) {
          x0 = xs[min(n * 8 + 2 * q, count - 1) * (kStageK / 128) + gi * GROUP / 128];
          x1 = xs[min(n * 8 + 2 * q + 1, count - 1) * (kStageK / 128) + gi * GROUP / 128];
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float2 sc = m == 0 ? s0 : s1;
          if constexpr (F8) {  // the row's scale first: either product alone may pass fp32's range no sooner than the result
            acc[m][n][0] = fmaf(sc.x, x0 * sum[m][n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(sc.x, x1 * sum[m][n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(sc.y, x0 * sum[m][n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(sc.y, x1 * sum[m][n][3], acc[m][n][3]);
          } else {
            acc[m][n][0] = fmaf(sc.x, sum[m][n][0], acc[m][n][0]);
            acc[m][n][1] = fmaf(sc.x, sum[m][n][1], acc[m][n][1]);
            acc[m][n][2] = fmaf(sc.y, sum[m][n][2], acc[m][n][2]);
            acc[m][n][3] = fmaf(sc.y, sum[m][n][3], acc[m][n][3]);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put_sums(const float (&acc)[2][NT][4], int count) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n > 0 && count <= 8) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float* to = &s.red[warp][n * 8 + 2 * q][16 * m + 2 * g];
        *reinterpret_cast<float2*>(to) = make_float2(acc[m][n][0], acc[m][n][2]);
        *reinterpret_cast<float2*>(to + kRedStride) = make_float2(acc[m][n][1], acc[m][n][3]);
      }
    }
  }
  __device__ __forceinline__ void store(int64_t row, int col, float v) const {
    if (p.out_f32)
      static_cast<float*>(p.out)[row * p.ld_out + col] = v;
    else
      static_cast<uint16_t*>(p.out)[row * p.ld_out + col] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
  __device__ __forceinline__ void fill() {
    in = Place{};
    start(in, first_sub());
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) issue();
  }
  __device__ __forceinline__ int first_sub() const {
    return p.w != nullptr ? blockIdx.x : blockIdx.x * (kWarps / p.ks) + warp / p.ks;
  }

  // ---------------------------------------------- each pair a row of its own
  __device__ __forceinline__ void rows() {
    const int ks = p.ks, mine = warp % ks, first_warp = warp - mine;
    end = s.n_parts * tiles;
    step = gridDim.x * (kWarps / ks);
    fill();
    auto meet = [&]() {  // the warps that share a tile
      if (ks > 1)
        named_bar_sync(1 + warp / ks, ks * 32);
      else
        __syncwarp();
    };
    for (int sub = first_sub(); sub < end; sub += step) {
      const int part = sub / tiles, tile = sub % tiles;
      const int count = s.count[part], first = s.first[part];
      float acc[2][NT][4];
      clear(acc);
      for (int st = mine; st < nst; st += ks) take(st, count, acc);
      put_sums(acc, count);
      meet();
      for (int i = mine; i < count; i += ks) {
        float v = 0.f;
        for (int w = 0; w < ks; ++w) v += s.red[first_warp + w][i][lane];
        const int64_t row = s.pair[first + i];
        if (p.swiglu) {
          const float up = __shfl_down_sync(0xffffffffu, v, kRows / 2);
          const int col = tile * (kRows / 2) + lane;
          if (lane < kRows / 2 && col < p.n / 2) store(row, col, v / (1.f + expf(-v)) * up);
        } else {
          const int col = tile * kRows + lane;
          if (col < p.n) store(row, col, v);
        }
      }
      meet();
    }
    cp_async_wait_all();
    // rows whose expert does not exist
    const int cols = p.swiglu ? p.n / 2 : p.n;
    for (int i = 0; i < p.pairs; ++i)
      if (s.bad[i / 32] >> (i % 32) & 1u)
        for (int c = blockIdx.x * kThreads + threadIdx.x; c < cols; c += gridDim.x * kThreads)
          store(i, c, __int_as_float(0x7FC00000));
  }

  // ------------------------------------------- the weighted sum of a row's pairs
  __device__ __forceinline__ void weighted(float (*sums)[kRows]) {
    // sums: this warp's [row of x][weight row]
    end = tiles;
    step = gridDim.x;
    fill();
    const int tokens = p.pairs / p.top;
    for (int sub = blockIdx.x; sub < end; sub += step) {
      for (int t = 0; t < tokens; ++t) sums[t][lane] = 0.f;
      Place a{};
      start(a, sub);
      while (a.sub == sub && a.part < s.n_parts) {
        const int part = a.part, count = s.count[part], first = s.first[part];
        float acc[2][NT][4];
        clear(acc);
        for (; a.st < nst; a.st += kWarps) take(a.st, count, acc);
        settle(a);
        put_sums(acc, count);
        __syncwarp();
        for (int i = 0; i < count; ++i) {
          const int pair = s.pair[first + i];
          float& v = sums[pair / p.top][lane];
          v = fmaf(__ldg(p.w + pair), s.red[warp][i][lane], v);
        }
        __syncwarp();
      }
      __syncthreads();
      const int col = sub * kRows + lane;
      for (int t = warp; t < tokens; t += kWarps) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += (sums - warp * kMaxTokens + w * kMaxTokens)[t][lane];
        for (int i = t * p.top; i < (t + 1) * p.top; ++i)
          if (s.bad[i / 32] >> (i % 32) & 1u) v = __int_as_float(0x7FC00000);
        if (col < p.n) store(t, col, v);
      }
      __syncthreads();
    }
    cp_async_wait_all();
  }
};

// The parts: each expert's pairs in order, at most NT x 8 to a part.  masks:
// scratch of kMaxExperts x kMaxPairs bits.
template <int NT>
__device__ __forceinline__ void find_parts(const Int4Args& p, Shared<NT>& s, uint32_t* masks) {
  constexpr int kWordsOf = kMaxPairs / 32;
  const int e = threadIdx.x, lane = e % 32, warp = e / 32;
  if (p.ids == nullptr) {
    if (e < p.pairs) s.pair[e] = static_cast<uint8_t>(e);
    if (e < kWordsOf) s.bad[e] = 0u;
    const int parts = (p.pairs + NT * 8 - 1) / (NT * 8);
    if (e < parts) {
      s.act[e] = 0;
      s.first[e] = static_cast<int16_t>(e * NT * 8);
      s.count[e] = static_cast<uint8_t>(min(NT * 8, p.pairs - e * NT * 8));
    }
    if (e == 0) s.n_parts = parts;
    __syncthreads();
    return;
  }
  for (int i = e; i < kMaxExperts * kWordsOf; i += kThreads) masks[i] = 0u;
  if (e < kWordsOf) s.bad[e] = 0u;
  __syncthreads();
  if (e < p.pairs) {
    const int id = __ldg(p.ids + e);
    const bool ok = id >= 0 && id < p.n_experts;
    atomicOr(ok ? &masks[id * kWordsOf + warp] : &s.bad[warp], 1u << lane);
    if (!ok && blockIdx.x == 0) set_error(p.status, kErrDevice);
  }
  __syncthreads();
  uint32_t mine[kWordsOf];
  int count = 0;
#pragma unroll
  for (int i = 0; i < kWordsOf; ++i) {
    mine[i] = masks[e * kWordsOf + i];
    count += __popc(mine[i]);
  }
  const int parts = (count + NT * 8 - 1) / (NT * 8);
  const int both = parts | count << 16;  // scanned together
  int sum = both;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int below = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += below;
  }
  if (lane == 31) s.warp_parts[warp] = sum;
  __syncthreads();
  int before = sum - both;
  for (int i = 0; i < warp; ++i) before += s.warp_parts[i];
  const int base = before & 0xFFFF;
  int at = before >> 16;
  for (int a = 0; a < parts; ++a) {
    s.act[base + a] = static_cast<int16_t>(e);
    s.first[base + a] = static_cast<int16_t>(at + a * NT * 8);
    s.count[base + a] = static_cast<uint8_t>(min(NT * 8, count - a * NT * 8));
  }
#pragma unroll
  for (int i = 0; i < kWordsOf; ++i)
    for (uint32_t m = mine[i]; m != 0u; m &= m - 1u) s.pair[at++] = static_cast<uint8_t>(i * 32 + __ffs(m) - 1);
  if (e == kMaxExperts - 1) s.n_parts = base + parts;
  __syncthreads();
}

template <int GROUP, int NT, bool F8, int DEPTH>
__global__ void __launch_bounds__(kThreads, 2) int4_few_kernel(const Int4Args p) {
  static_assert(kThreads == kMaxExperts && kThreads == kMaxPairs, "a thread per expert and per pair");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<NT> s;
  // the ring, and before it is filled the masks; behind it the weighted sums
  find_parts<NT>(p, s, reinterpret_cast<uint32_t*>(smem));
  Worker<GROUP, NT, F8, DEPTH> w(p, s, smem);
  if (p.w == nullptr) {
    w.rows();
  } else {
    float(*sums)[kRows] = reinterpret_cast<float(*)[kRows]>(smem + kWarps * DEPTH * w.bytes);
    w.weighted(sums + w.warp * kMaxTokens);
  }
}

constexpr int kSmemOfSm = 227 * 1024;
constexpr int kMaskBytes = kMaxExperts * kMaxPairs / 8;

template <int GROUP, int NT, bool F8, int DEPTH>
cudaError_t launch(const Int4Args& a, int num_sms, cudaStream_t st) {
  auto kernel = int4_few_kernel<GROUP, NT, F8, DEPTH>;
  const int ring = kWarps * DEPTH * stage_bytes<GROUP, NT, F8>(a.nx);
  const int smem = std::max(ring + (a.w != nullptr ? kWarps * kMaxTokens * kRows * 4 : 0), kMaskBytes);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int per_sm = std::max(1, std::min(2, kSmemOfSm / (smem + static_cast<int>(sizeof(Shared<NT>)) + 1024)));
  const int tile_out = a.swiglu ? kRows / 2 : kRows, cols = a.swiglu ? a.n / 2 : a.n;
  const int64_t tiles = (cols + tile_out - 1) / tile_out;
  const int64_t parts = a.ids != nullptr ? std::min(a.pairs, a.n_experts) : 1;  // about
  const int64_t slots = static_cast<int64_t>(per_sm) * num_sms;
  Int4Args b = a;
  b.ks = 1;
  int64_t blocks = tiles;
  if (a.w == nullptr) {
    const int stages = (a.k + kStageOf<NT> - 1) / kStageOf<NT>;
    while (b.ks < kWarps && 2 * b.ks <= stages && parts * tiles * b.ks < slots * kWarps) b.ks *= 2;
    const int64_t most = (a.ids != nullptr ? a.pairs : (a.pairs + NT * 8 - 1) / (NT * 8)) * tiles;
    blocks = (most * b.ks + kWarps - 1) / kWarps;
  }
  const int grid = static_cast<int>(blocks < slots ? blocks : slots);
  return launch_kernel(kernel, dim3(grid), dim3(kThreads), static_cast<size_t>(smem), st, b);
}

// The deepest ring that leaves two blocks on an SM, or else fits one.
template <int GROUP, int NT, bool F8>
cudaError_t launch_depth(const Int4Args& a, int num_sms, cudaStream_t s) {
  const int stage = kWarps * stage_bytes<GROUP, NT, F8>(a.nx);
  const int fixed = static_cast<int>(sizeof(Shared<NT>)) + 1024 + (a.w != nullptr ? kWarps * kMaxTokens * kRows * 4 : 0);
  const int half = kSmemOfSm / 2 - fixed;
  if (4 * stage <= half) return launch<GROUP, NT, F8, 4>(a, num_sms, s);
  if (3 * stage <= half || 4 * stage > kSmemOfSm - fixed) {
    if (3 * stage <= kSmemOfSm - fixed) return launch<GROUP, NT, F8, 3>(a, num_sms, s);
    return launch<GROUP, NT, F8, 2>(a, num_sms, s);
  }
  return launch<GROUP, NT, F8, 4>(a, num_sms, s);
}

template <int GROUP>
cudaError_t launch_group(Int4Args a, int num_sms, cudaStream_t s) {
  const bool f8 = a.x_scales != nullptr;
  const int rows = a.ids != nullptr ? a.pairs / a.top : a.pairs;  // at most, of an expert (once per row of x)
  // parts of up to 16 rows where experts have more than 4 on average; else the few with more than 8 are taken twice
  const bool two = rows > 8 && (a.ids == nullptr || a.pairs > 4 * a.n_experts);
  a.nx = std::min(a.pairs, two ? 16 : 8);
  if (two) return f8 ? launch_depth<GROUP, 2, true>(a, num_sms, s) : launch_depth<GROUP, 2, false>(a, num_sms, s);
  return f8 ? launch_depth<GROUP, 1, true>(a, num_sms, s) : launch_depth<GROUP, 1, false>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_int4_few(int group, const Int4Args& a, int num_sms, cudaStream_t s) {
  switch (group) {
    case 32: return launch_group<32>(a, num_sms, s);
    case 64: return launch_group<64>(a, num_sms, s);
    case 128: return launch_group<128>(a, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cbmoe
