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
#include <climits>

#include "internal.h"
#include "ptx.cuh"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kRows = 32;            // weight rows of a tile: two m16 fragments
constexpr int kMaxPairs = 256;       // (row of x, slot)
constexpr int kMaxExperts = 256;
constexpr int kRedStride = 36;       // floats: the fragments' stores meet no bank twice
constexpr int kMaxTokens = kFewTokens;
constexpr int kWarpsOfSm = 16;       // in blocks of 8, or of 16 for the weighted sum
constexpr int kMaxDepth = 4;

// One of the kernel's forms: groups of GROUP elements, NT n-tiles of 8 rows of
// x to a part, SK elements of a row in a stage, x in 8 bits or not, WARPS to a block.
template <int GROUP_, int NT_, int SK_, bool F8_, int WARPS_>
struct Form {
  static constexpr int kGroup = GROUP_, NT = NT_, SK = SK_, kWarps = WARPS_;
  static constexpr bool F8 = F8_;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRowBytes = SK / 2;
  static constexpr int kGroups = SK / kGroup;            // of a stage
  static constexpr int kWords = kGroup / 32;             // of codes, to a thread, row and group
  // a row of x in a stage; for neighbours' reads to meet no bank twice 8-bit
  // rows are padded, and of 16-bit ones every other has its 64-byte halves swapped
  static constexpr int kTokBytes = F8 ? SK + 32 : 2 * SK;
  static constexpr int kScales = kRows * kRowBytes;      // where the scales, zero points and x stand
  static constexpr int kZeros = kScales + kGroups * kRows * 4;
  static constexpr int kX = kZeros + kGroups * kRows;
  // bytes of a stage with nx rows of x (and 8-bit rows' scales behind them)
  __host__ __device__ static constexpr int stage(int nx) {
    return (kX + nx * (kTokBytes + (F8 ? SK / 32 : 0)) + 127) / 128 * 128;
  }
  static_assert(kX + (NT == 1 ? 1 : 9) * kTokBytes >= NT * 8 * kRedStride * 4, "a tile's sums fit a stage");
};

template <int WARPS>
struct Shared {
  uint8_t pair[kMaxPairs];      // pairs by expert, then in order,
  uint8_t row[kMaxPairs];       //   and their rows of x
  int16_t act[kMaxPairs];       // parts: their expert,
  int16_t first[kMaxPairs];     //   first entry of `pair`
  uint8_t count[kMaxPairs];     //   and number of them
  uint32_t bad[kMaxPairs / 32]; // pairs whose expert does not exist
  int red[WARPS];               // where a warp has its sums of a tile, in the dynamic array
  int warp_parts[kMaxExperts / 32];
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

template <bool F8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (F8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    router_detail::mma_bf16(c, a0, a1, a2, a3, b0, b1);
}
// The same from zero.
template <bool F8>
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Eight codes of a word minus their zero point, pairs of elements m and m + 4.
// bf16: a nibble n in a half word under 0x4300 is 128 + n.  fp16: under 0x6400
// 1024 + n, and one bit field further up 1024 + 16 n, so two shifts fewer:
// (1024 + 16 n) / 16 - (64 + z).  All of it is exact.
template <bool F8>
struct Zero {
  uint32_t a, b;
  // byte `at` of v is the zero point
  __device__ __forceinline__ void set(uint32_t v, int at) {
    a = __byte_perm(v, F8 ? 0x64u : 0x43u, at == 0 ? 0x4040 : 0x4141);
    if constexpr (F8) b = __byte_perm(v << 4, 0xD4u, at == 0 ? 0x4040 : 0x4141);  // -(64 + z)
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

template <class F>
struct Worker {
  static constexpr int NT = F::NT, SK = F::SK, GROUP = F::kGroup, kWords = F::kWords, kWarps = F::kWarps;
  static constexpr bool F8 = F::F8;
  static constexpr int kPer = F::kRowBytes / 16;  // 16-byte units of a row in a stage
  const Int4Args& p;
  Shared<kWarps>& s;
  uint8_t* const dynamic;
  const int warp, lane, g, q;
  const int bytes;        // of a stage
  const int nst;          // stages of a row
  const int tiles;        // of a matrix
  const int row_bytes;
  const int ring;         // this warp's, in the dynamic array
  int slot_in = 0, slot_out = 0;
  int ks = 1;             // warps that share a tile

  // Where the loads stand: the tile, its part, the stage; and this lane's
  // codes, scales and zero points of the tile.
  struct Place {
    int sub, part, tile, st;
    const uint8_t *lo, *hi;     // codes of the tile's rows of the first and the second fragment
    int64_t scales, zeros;      // elements
  };
  Place in;
  int end, step;          // of the walk over the tiles

  __device__ __forceinline__ Worker(const Int4Args& p_, Shared<kWarps>& s_, uint8_t* smem)
      : p(p_),
        s(s_),
        dynamic(smem),
        warp(threadIdx.x / 32),
        lane(threadIdx.x % 32),
        g(threadIdx.x % 32 >> 2),
        q(threadIdx.x & 3),
        bytes(F::stage(p_.nx)),
        nst((p_.k + SK - 1) / SK),
        tiles(((p_.swiglu ? p_.n / 2 : p_.n) + tile_out(p_) - 1) / tile_out(p_)),
        row_bytes(p_.k / 2),
        ring(static_cast<int>(threadIdx.x / 32) * p_.depth * F::stage(p_.nx)) {}
  __device__ __forceinline__ static int tile_out(const Int4Args& p) { return p.swiglu ? kRows / 2 : kRows; }

  // The lane group's place among the 16-byte units of its rows: what differs
  // between neighbours is first the widest reads' own bit.
  __device__ __forceinline__ static int unit_key(int g) {
    return kPer == 8 ? (g & 1) << 2 | (g & 2) | g >> 2 : (g & 2) | g >> 2;
  }

  // ------------------------------------------------------------- the walk
  __device__ __forceinline__ void at_tile(Place& a) const {
    const int e = s.act[a.part];
    const int r0 = p.swiglu ? a.tile * (kRows / 2) : a.tile * kRows, second = p.swiglu ? p.n / 2 : kRows / 2;
    const bool both = p.swiglu || r0 + kRows / 2 < p.n;  // else the second fragment is the first again
    const int64_t matrix = static_cast<int64_t>(e) * p.n;
    a.lo = p.codes + (matrix + r0 + 2 * (lane / kPer)) * row_bytes + lane % kPer * 16;
    a.hi = both ? a.lo + static_cast<int64_t>(second) * row_bytes : a.lo;
    const int64_t meta = static_cast<int64_t>(e) * (p.k / GROUP) * p.n + r0;
    const int up = both ? second : 0;
    a.scales = meta + (lane % 8 >= 4 ? up : 0) + lane % 4 * 4 + static_cast<int64_t>(lane / 8) * p.n;
    a.zeros = meta + (lane % 4 >= 2 ? up : 0) + lane % 2 * 8 + static_cast<int64_t>(lane / 4) * p.n;
  }
  __device__ __forceinline__ bool any(const Place& a) const { return a.sub < end; }
  // rows(): a tile is a part's
  __device__ __forceinline__ void start_row(Place& a, int sub) const {
    a.sub = sub;
    if (sub >= end) return;
    a.part = sub / tiles;
    a.tile = sub - a.part * tiles;
    a.st = warp % ks;
    at_tile(a);
  }
  // weighted(): a tile's parts, `kWarps / ks` warps apart, one after the other
  __device__ __forceinline__ void start_sum(Place& a, int sub) const {
    a.sub = sub;
    a.tile = sub;
    a.part = warp / ks;
    a.st = warp % ks;
    if (a.part >= s.n_parts) a.sub = end;  // (in every tile)
    if (any(a)) at_tile(a);
  }
  __device__ __forceinline__ void next(Place& a) const {
    a.st += ks;
    if (a.st < nst) return;
    if (p.w == nullptr) {
      start_row(a, a.sub + step);
    } else {
      a.st = warp % ks;
      a.part += kWarps / ks;
      if (a.part >= s.n_parts)
        start_sum(a, a.sub + step);
      else
        at_tile(a);
    }
  }

  // -------------------------------------------------------------- a stage
  __device__ __forceinline__ void issue() {
    if (any(in)) {
      uint8_t* dst = dynamic + ring + slot_in * bytes;
      const int k0 = in.st * SK, left = p.k - k0;
      if (lane % kPer * 32 < left) {
        // row j of lane group h stands at row 8 j + h: rows 2 h and 2 h + 1 of each fragment
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int j = kPer == 8 ? i >> 1 : i, h = kPer == 8 ? (i & 1) * 4 + lane / kPer : lane / kPer;
          const int off = (j & 1) * row_bytes + (kPer == 8 ? (i & 1) * 8 * row_bytes : 0);
          cp_async_16(dst + (j * 8 + h) * F::kRowBytes + ((lane % kPer ^ unit_key(h)) << 4),
                      (j < 2 ? in.lo : in.hi) + (k0 / 2 + off));
        }
      }
      // scales: 4 rows to a lane; zero points: 8
      const int64_t before = static_cast<int64_t>(in.st * F::kGroups) * p.n;
#pragma unroll
      for (int i = 0; i < (F::kGroups + 3) / 4; ++i) {
        const int gi = i * 4 + lane / 8;
        if (gi < F::kGroups && gi * GROUP < left)
          cp_async_16(dst + F::kScales + (i * 32 + lane) * 16, p.scales + in.scales + before + static_cast<int64_t>(i * 4) * p.n);
      }
      if (p.zeros != nullptr && lane / 4 < F::kGroups && lane / 4 * GROUP < left)
        cp_async_8(dst + F::kZeros + lane * 8, p.zeros + in.zeros + before);
      // x: 8 elements to a lane, in the order in which the quads read them
      const int count = s.count[in.part], first = s.first[in.part];
      constexpr int kUnits = GROUP / 8, kLanes = SK / 8;  // of a group; of a row of x
      const int u = lane % kLanes;
      const int at = u / kUnits * kUnits + u % kWords * 4 + u % kUnits / kWords;
      uint8_t* x = dst + F::kX;
      if (u * 8 < left)
        for (int t = lane / kLanes; t < count; t += 32 / kLanes) {
          const int64_t from = s.row[first + t] * p.ld_x + k0 + u * 8;
          if constexpr (F8)
            cp_async_8(x + t * F::kTokBytes + at * 8, static_cast<const uint8_t*>(p.x) + from);
          else
            cp_async_16(x + t * F::kTokBytes + ((at ^ (t & 1) << 2) << 4), static_cast<const uint16_t*>(p.x) + from);
        }
      if constexpr (F8) {
        constexpr int kScales = SK / 128;
        const int t = lane / kScales, h = lane % kScales;
        if (t < count && h * 128 < left)
          cp_async_4(x + p.nx * F::kTokBytes + lane * 4,
                     p.x_scales + static_cast<int64_t>(s.row[first + t]) * ((p.k + 127) / 128) + k0 / 128 + h);
      }
      next(in);
    }
    cp_async_commit();
    slot_in = slot_in + 1 == p.depth ? 0 : slot_in + 1;
  }

  __device__ __forceinline__ void clear(float (&v)[2][NT][4]) const {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) v[m][n][0] = v[m][n][1] = v[m][n][2] = v[m][n][3] = 0.f;
  }

  // acc += the oldest stage in the ring, which is stage st of a part of `count` rows.
  __device__ __forceinline__ void take(int st, int count, float (&acc)[2][NT][4]) {
    if (p.depth == 2)
      cp_async_wait_pending<0>();
    else if (p.depth == 3)
      cp_async_wait_pending<1>();
    else
      cp_async_wait_pending<2>();
    __syncwarp();
    issue();
    const uint8_t* src = dynamic + ring + slot_out * bytes;
    slot_out = slot_out + 1 == p.depth ? 0 : slot_out + 1;
    const int groups = (p.k - st * SK) / GROUP;
    const uint8_t* codes = src + g * F::kRowBytes;
    const int unit = ((q * kWords / 4 ^ unit_key(g)) << 4) + q * kWords % 4 * 4;
    const uint8_t* x[NT][2];  // 16-bit rows: for the units in even and in odd halves
    const float* xs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = min(n * 8 + g, count - 1), swap = F8 ? 0 : (t & 1) << 6;
      x[n][0] = src + F::kX + t * F::kTokBytes + q * (F8 ? 8 : 16) + swap;
      x[n][1] = x[n][0] - 2 * swap;
      if constexpr (F8)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xs[n][i] = reinterpret_cast<const float*>(src + F::kX + p.nx * F::kTokBytes) +
                     min(n * 8 + 2 * q + i, count - 1) * (SK / 128);
    }
    const bool wide = count > 8;
#pragma unroll
    for (int gi = 0; gi < F::kGroups; ++gi) {
      if (gi >= groups) break;
      uint32_t v[4][kWords];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* at = codes + (unit ^ gi * GROUP / 2) + j * 8 * F::kRowBytes;
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
        if (p.zeros != nullptr) z = *reinterpret_cast<const uint16_t*>(src + F::kZeros + gi * kRows + m * 16 + 2 * g);
        zz[2 * m].set(z, 0);
        zz[2 * m + 1].set(z, 1);
      }
      float sum[2][NT][4];
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n > 0 && !wide) break;
          const uint8_t* at = x[n][F8 ? 0 : (gi * (GROUP / 32) + w) & 1] + (gi * (GROUP / 8) + w * 4) * (F8 ? 8 : 16);
          if constexpr (F8) {
            const uint2 e = *reinterpret_cast<const uint2*>(at);
            const uint32_t lo = __byte_perm(e.x, e.y, 0x5140), hi = __byte_perm(e.x, e.y, 0x7362);
            const uint16_t h[4] = {static_cast<uint16_t>(lo), static_cast<uint16_t>(lo >> 16), static_cast<uint16_t>(hi),
                                   static_cast<uint16_t>(hi >> 16)};
#pragma unroll
            for (int i = 0; i < 4; ++i) asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b[n][i]) : "h"(h[i]));
          } else {
            const uint4 e = *reinterpret_cast<const uint4*>(at);
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
            if (w == 0)
              mma_first<F8>(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
            else
              mma<F8>(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
            mma<F8>(sum[m][n], a0[2], a1[2], a0[3], a1[3], b[n][2], b[n][3]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float2 sc = *reinterpret_cast<const float2*>(src + F::kScales + (gi * kRows + m * 16 + 2 * g) * 4);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n > 0 && !wide) break;
          float* c = acc[m][n];
          const float* t = sum[m][n];
          if constexpr (F8) {  // x's scale first, then the weights'
            const float x0 = xs[n][0][gi * GROUP / 128], x1 = xs[n][1][gi * GROUP / 128];
            c[0] = fmaf(sc.x, x0 * t[0], c[0]);
            c[1] = fmaf(sc.x, x1 * t[1], c[1]);
            c[2] = fmaf(sc.y, x0 * t[2], c[2]);
            c[3] = fmaf(sc.y, x1 * t[3], c[3]);
          } else {
            c[0] = fmaf(sc.x, t[0], c[0]);
            c[1] = fmaf(sc.x, t[1], c[1]);
            c[2] = fmaf(sc.y, t[2], c[2]);
            c[3] = fmaf(sc.y, t[3], c[3]);
          }
        }
      }
    }
  }

  // The tile's sums of this warp, [row of x][weight row], into the stage that
  // it used last: nothing is loaded there before the next one is taken.
  __device__ __forceinline__ float* put_sums(const float (&acc)[2][NT][4], int count) {
    const int at = ring + (slot_out == 0 ? p.depth - 1 : slot_out - 1) * bytes;
    float* red = reinterpret_cast<float*>(dynamic + at);
    __syncwarp();  // all lanes have read it
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n > 0 && count <= 8) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float* to = red + (n * 8 + 2 * q) * kRedStride + 16 * m + 2 * g;
        *reinterpret_cast<float2*>(to) = make_float2(acc[m][n][0], acc[m][n][2]);
        *reinterpret_cast<float2*>(to + kRedStride) = make_float2(acc[m][n][1], acc[m][n][3]);
      }
    }
    if (lane == 0) s.red[warp] = at;
    return red;
  }
  __device__ __forceinline__ void store(int64_t row, int col, float v) const {
    if (p.out_f32)
      static_cast<float*>(p.out)[row * p.ld_out + col] = v;
    else
      static_cast<uint16_t*>(p.out)[row * p.ld_out + col] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }

  // ---------------------------------------------- each pair a row of its own
  __device__ __forceinline__ void rows() {
    ks = p.ks;
    const int mine = warp % ks, first_warp = warp - mine;
    const int from = blockIdx.x * (kWarps / ks) + warp / ks;
    end = s.n_parts * tiles;
    step = gridDim.x * (kWarps / ks);
    start_row(in, from);
    for (int i = 0; i < p.depth - 1; ++i) issue();
    auto meet = [&]() {  // the warps that share a tile
      if (ks > 1)
        named_bar_sync(1 + warp / ks, ks * 32);
      else
        __syncwarp();
    };
    for (int sub = from; sub < end; sub += step) {
      const int part = sub / tiles, tile = sub - part * tiles;
      const int count = s.count[part], first = s.first[part];
      float acc[2][NT][4];
      clear(acc);
      for (int st = mine; st < nst; st += ks) take(st, count, acc);
      put_sums(acc, count);
      meet();
      for (int i = mine; i < count; i += ks) {
        float v = 0.f;
        for (int w = 0; w < ks; ++w)
          v += reinterpret_cast<const float*>(dynamic + s.red[first_warp + w])[i * kRedStride + lane];
        const int64_t row = s.pair[first + i];
        if (p.swiglu) {
          const float up = __shfl_down_sync(0xffffffffu, v, kRows / 2);
          const int col = tile * (kRows / 2) + lane;
          if (lane < kRows / 2) store(row, col, v / (1.f + expf(-v)) * up);
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
        for (int c = blockIdx.x * F::kThreads + threadIdx.x; c < cols; c += gridDim.x * F::kThreads)
          store(i, c, __int_as_float(0x7FC00000));
  }

  // ------------------------------------------- the weighted sum of a row's pairs
  // The warps take a tile's parts in turn, or `ks` of them a part's stages:
  // whichever leaves the busiest with the least (a part's end costs about a
  // stage).
  __device__ __forceinline__ void weighted() {
    const int tokens = p.pairs / p.top;
    float* all = reinterpret_cast<float*>(dynamic + kWarps * p.depth * bytes);  // [warp][row of x][weight row]
    float* sums = all + warp * tokens * kRows;
    int least = INT_MAX;
    for (int k = 1; k <= kWarps && k <= nst; k *= 2) {
      const int each = kWarps / k, load = (s.n_parts + each - 1) / each * ((nst + k - 1) / k + 1);
      if (load < least) {
        least = load;
        ks = k;
      }
    }
    end = tiles;
    step = gridDim.x;
    start_sum(in, blockIdx.x);
    for (int i = 0; i < p.depth - 1; ++i) issue();
    for (int sub = blockIdx.x; sub < end; sub += step) {
      for (int t = 0; t < tokens; ++t) sums[t * kRows + lane] = 0.f;
      for (int part = warp / ks; part < s.n_parts; part += kWarps / ks) {
        const int count = s.count[part], first = s.first[part];
        float acc[2][NT][4];
        clear(acc);
        for (int st = warp % ks; st < nst; st += ks) take(st, count, acc);
        const float* red = put_sums(acc, count);
        __syncwarp();
        for (int i = 0; i < count; ++i) {
          const int pair = s.pair[first + i];
          float& v = sums[pair / p.top * kRows + lane];
          v = fmaf(__ldg(p.w + pair), red[i * kRedStride + lane], v);
        }
        __syncwarp();
      }
      __syncthreads();
      const int col = sub * kRows + lane;
      for (int t = warp; t < tokens; t += kWarps) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += all[(w * tokens + t) * kRows + lane];
        for (int i = t * p.top; i < (t + 1) * p.top; ++i)
          if (s.bad[i / 32] >> (i % 32) & 1u) v = __int_as_float(0x7FC00000);
        if (col < p.n) store(t, col, v);
      }
      __syncthreads();
    }
    cp_async_wait_all();
  }
};

// The parts: each expert's pairs in order, at most nx to a part.  masks:
// scratch of kMaxExperts x kMaxPairs bits.
template <class F>
__device__ __forceinline__ void find_parts(const Int4Args& p, Shared<F::kWarps>& s, uint32_t* masks) {
  constexpr int kWordsOf = kMaxPairs / 32;
  const int most = p.nx;
  const int e = threadIdx.x, lane = e % 32, warp = e / 32;
  if (p.ids == nullptr) {
    if (e < p.pairs) s.pair[e] = s.row[e] = static_cast<uint8_t>(e);
    if (e < kWordsOf) s.bad[e] = 0u;
    const int parts = (p.pairs + most - 1) / most;
    if (e < parts) {
      s.act[e] = 0;
      s.first[e] = static_cast<int16_t>(e * most);
      s.count[e] = static_cast<uint8_t>(min(most, p.pairs - e * most));
    }
    if (e == 0) s.n_parts = parts;
    __syncthreads();
    return;
  }
  for (int i = e; i < kMaxExperts * kWordsOf; i += F::kThreads) masks[i] = 0u;
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
    mine[i] = e < kMaxExperts ? masks[e * kWordsOf + i] : 0u;
    count += __popc(mine[i]);
  }
  const int parts = (count + most - 1) / most;
  const int both = parts | count << 16;  // scanned together
  int sum = both;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int below = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += below;
  }
  if (e < kMaxExperts && lane == 31) s.warp_parts[warp] = sum;
  __syncthreads();
  if (e < kMaxExperts) {
    int before = sum - both;
    for (int i = 0; i < warp; ++i) before += s.warp_parts[i];
    const int base = before & 0xFFFF;
    int at = before >> 16;
    for (int a = 0; a < parts; ++a) {
      s.act[base + a] = static_cast<int16_t>(e);
      s.first[base + a] = static_cast<int16_t>(at + a * most);
      s.count[base + a] = static_cast<uint8_t>(min(most, count - a * most));
    }
#pragma unroll
    for (int i = 0; i < kWordsOf; ++i)
      for (uint32_t m = mine[i]; m != 0u; m &= m - 1u) {
        const int pair = i * 32 + __ffs(m) - 1;
        s.pair[at] = static_cast<uint8_t>(pair);
        s.row[at++] = static_cast<uint8_t>(p.x_per_slot ? pair : pair / p.top);
      }
    if (e == kMaxExperts - 1) s.n_parts = base + parts;
  }
  __syncthreads();
}

template <class F>
__global__ void __launch_bounds__(F::kThreads, kWarpsOfSm / F::kWarps) int4_few_kernel(const Int4Args p) {
  static_assert(F::kThreads >= kMaxExperts && F::kThreads >= kMaxPairs, "a thread per expert and per pair");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared<F::kWarps> s;
  // the warps' rings, and before they are filled the masks; behind them the weighted sums
  find_parts<F>(p, s, reinterpret_cast<uint32_t*>(smem));
  Worker<F> w(p, s, smem);
  if constexpr (F::kWarps == 8)
    w.rows();
  else
    w.weighted();
}

constexpr int kSmemOfSm = 228 * 1024, kSmemOfBlock = 227 * 1024;
constexpr int kMaskBytes = kMaxExperts * kMaxPairs / 8;

template <class F>
cudaError_t launch(Int4Args a, int num_sms, cudaStream_t st) {
  auto kernel = int4_few_kernel<F>;
  constexpr int kBlocks = kWarpsOfSm / F::kWarps;  // of an SM
  const int stage = F::kWarps * F::stage(a.nx), fixed = static_cast<int>(sizeof(Shared<F::kWarps>)) + 1024;
  const int sums = F::kWarps == 8 ? 0 : F::kWarps * (a.pairs / a.top) * kRows * 4;
  const int most = std::min(kSmemOfSm / kBlocks - fixed, kSmemOfBlock - fixed + 1024);
  a.depth = std::max(2, std::min(kMaxDepth, (most - sums) / stage));
  const int smem = std::max(a.depth * stage + sums, kMaskBytes);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int tile_out = a.swiglu ? kRows / 2 : kRows, cols = a.swiglu ? a.n / 2 : a.n;
  const int64_t tiles = (cols + tile_out - 1) / tile_out;
  const int64_t slots = static_cast<int64_t>(kBlocks) * num_sms;
  a.ks = 1;
  int64_t blocks = tiles;
  if (F::kWarps == 8) {
    const int stages = (a.k + F::SK - 1) / F::SK;
    const int64_t parts = a.ids != nullptr ? std::min(a.pairs, a.n_experts) : 1;  // about
    while (a.ks < F::kWarps && 2 * a.ks <= stages && parts * tiles * a.ks < slots * F::kWarps) a.ks *= 2;
    const int64_t at_most = (a.ids != nullptr ? a.pairs : 1) * tiles;
    blocks = (at_most * a.ks + F::kWarps - 1) / F::kWarps;
  }
  const int grid = static_cast<int>(blocks < slots ? blocks : slots);
  return launch_kernel(kernel, dim3(grid), dim3(F::kThreads), static_cast<size_t>(smem), st, a);
}

template <int GROUP, bool F8>
cudaError_t launch_form(Int4Args a, int num_sms, cudaStream_t s) {
  const int rows = a.pairs / a.top;  // of an expert, unless a row names it twice
  // Parts of up to 16 rows where experts have more than 4 on average; else the few with more than 8 are taken twice.
  // (The weighted sum's blocks have no room for 16 beside their sums.)
  if (a.w == nullptr && rows > 8 && (a.ids == nullptr || a.pairs > 4 * a.n_experts)) {
    a.nx = std::min(rows, 16);
    return launch<Form<GROUP, 2, 128, F8, 8>>(a, num_sms, s);
  }
  a.nx = std::min(rows, 8);
  // twice as long stages while few rows of x stand beside the codes
  if (a.w == nullptr) return a.nx <= 3 ? launch<Form<GROUP, 1, 256, F8, 8>>(a, num_sms, s) : launch<Form<GROUP, 1, 128, F8, 8>>(a, num_sms, s);
  return a.nx <= 3 ? launch<Form<GROUP, 1, 256, F8, 16>>(a, num_sms, s) : launch<Form<GROUP, 1, 128, F8, 16>>(a, num_sms, s);
}

template <int GROUP>
cudaError_t launch_group(const Int4Args& a, int num_sms, cudaStream_t s) {
  const bool f8 = a.x_scales != nullptr;
  return f8 ? launch_form<GROUP, true>(a, num_sms, s) : launch_form<GROUP, false>(a, num_sms, s);
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
