// A few rows (1 to 16) by 4-bit integer weights with a scale and a zero point
// per group of 32, 64 or 128 elements of a row:
//
//   y[t][j] = sum_g s[g][j] ( sum_{i in g} x[t][i] q[j][i]  -  z[g][j] sum_{i in g} x[t][i] ),
//
// one matrix, or one per expert with the experts of each row given; then the
// rows as they are, silu(gate) * up (rows_kernel), or the weighted sum over a
// row's experts (sum_kernel).
//
// What bounds it: the weights, read once from HBM (of an expert with more rows
// than a part holds, once per part), and the instructions that widen them: 270
// a warp and stage in rows_kernel, 480 in sum_kernel with groups of 32 (8 rows
// by two of 8 experts of 28672 x 4096: 67 us, 5.4 TB/s of what is read; 16 rows
// by 6 of 64 of 4096 x 1536 in groups of 32, summed: 43 us, 3.4 TB/s).  Few
// tiles are bound by latency (one row by 14336 x 4096: 10 us, 2.5 of them
// before the first weights arrive); more than 8 rows of one matrix by the
// instructions of two column tiles (16 rows by 4096 x 14336: 21 us).
// Both kernels take tiles of 32 weight rows (SwiGLU: 16 features' gate and up
// rows) in stages of 128 elements, 64 bytes of a row: codes, scales and zero
// points come by cp.async into a ring in shared memory that belongs to one
// warp.  With no thread but its own 32 to wait for, a warp needs no barrier to
// keep its loads in flight across stages, tiles and experts.
//
// Widening.  A bf16 word with bits only in its low byte is that byte times
// 2^-133: its subnormals and its lowest normal numbers have one spacing.  So a
// code is an MMA operand as soon as its neighbours are masked away: n 2^-133 in
// bits 0-3, 16 n 2^-133 in bits 4-7 (for which x is given as x / 16), and after
// one shift by 8 bits the other two of each half word: 5 instructions for 8
// codes and none of them rounds.  (128 + n minus 128 + z, as an ordinary bf16
// number, takes 11.)  x is multiplied by 2^64 to keep the sums in fp32's
// normal range.  8-bit x goes the same way in fp16, whose spacing is 2^-24 and
// which holds every e4m3 number and its sixteenth.  The tensor core takes
// subnormal operands exactly (measured: 256 byte values, both types).
//   The zero points meet a group's sum of x: in rows_kernel it is made with the
// operands (8 rows by two of 8 experts of 28672 x 4096: 75 -> 68 us), in
// sum_kernel it comes from one more MMA per 16 elements, whose weights are all
// 1.  A group's sums are taken from zero and join the tile's with their scale,
// in fp32: no weight is rounded.
//
// Layouts.  A dot product does not depend on the order of its terms: within a
// group thread q of a quad owns a quarter of the group's consecutive elements,
// so it reads its codes in one piece of 4, 8 or 16 bytes.  The 16-byte units
// of a row stand at unit ^ key(row): no bank conflicts.  Rows 2g and 2g + 1 of
// each half of a tile are lane group g's, so its scales and zero points are
// pairs.
//
// rows_kernel keeps a part's rows of x in shared memory, in the order of the
// MMA's operands, and walks its share of the tiles; `ks` of a block's sixteen
// warps share a tile, neighbours in k, so that 64 ks bytes of each row are
// read together.  (x in the ring beside the codes cost as much as the codes:
// all blocks read the same few lines of L2; 8 rows by two of 8 experts of
// 28672 x 4096, loads alone, 113 us against 66 without.)  Where one matrix
// has so long rows that x does not fit, a cluster of blocks splits k: each
// keeps its stretch of x and the sums of a batch of tiles, which are joined
// over distributed shared memory.
//   sum_kernel has one tile per block at a time and all its experts' parts; each
// pair has its own row of x there, which comes through the ring.  Where that
// leaves SMs without a tile, a cluster shares one: its parts' stages, then the
// joining of the sums over distributed shared memory.
//
// All sums are in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "router_common.cuh"

namespace cbmoe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 32;            // weight rows of a tile: two m16 fragments
constexpr int kStageK = 128;         // elements of a row in a stage
constexpr int kRowBytes = kStageK / 2;
constexpr int kMaxPairs = 256;       // (row of x, slot)
constexpr int kMaxDepth = 5;
constexpr int kMaxCluster = 8;
constexpr int kXBytes = 2 * kStageK; // of a row of x in a stage, as MMA operands
constexpr int kKeyBytes = kMaxPairs * 4;

// A stage: codes, scales, zero points (and in sum_kernel rows of x).
constexpr int kScales = kRows * kRowBytes;
template <int GROUP>
constexpr int kGroups = kStageK / GROUP;
template <int GROUP>
constexpr int kZeros = kScales + kGroups<GROUP> * kRows * 4;
template <int GROUP>
constexpr int kStage = (kZeros<GROUP> + kGroups<GROUP> * kRows + 127) / 128 * 128;
// Floats of a row of a warp's sums: with 36 the fragments' stores meet no bank
// twice.  The sums of two column tiles stand in a stage that has been read, where
// the zero points may be the constant ones that no load brings back: with 34
// (some banks twice) all 16 rows end before them.
template <int NT>
constexpr int kRedStride = NT == 1 ? 36 : 34;
// a row of x in sum_kernel's ring; for neighbours' reads to meet no bank twice
// 8-bit rows are padded, and of 16-bit ones every other has its 64-byte halves swapped
template <bool F8>
constexpr int kRingX = F8 ? kStageK + 32 : 2 * kStageK;

struct Shared {
  uint8_t pair[kMaxPairs];      // pairs by expert, then in order,
  uint8_t row[kMaxPairs];       //   their rows of x,
  uint8_t token[kMaxPairs];     //   rows of ids
  float w[kMaxPairs];           //   and weights
  int16_t act[kMaxPairs];       // parts: their expert,
  int16_t first[kMaxPairs];     //   first entry of `pair`
  uint8_t count[kMaxPairs];     //   and number of them
  uint32_t bad[kMaxPairs / 32]; // pairs whose expert does not exist
  int red[kWarps];              // where a warp has its sums of more than 8 rows, floats of the dynamic array
  uint32_t starts[kMaxPairs / 32];  // entries of `pair` that begin a part
  uint32_t n_parts;
  int n_good;                   // pairs whose expert exists
};

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the n newest groups have landed.
__device__ __forceinline__ void cp_async_wait_pending(int n) {
  if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 3;" ::: "memory");
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

// Eight codes as operands, pairs of elements m and m + 4: 0 and 2 in units of
// 2^-133 (fp16: 2^-24), 1 and 3 in sixteenths of it.
__device__ __forceinline__ void widen(uint32_t v, uint32_t (&o)[4]) {
  o[0] = v & 0x000F000Fu;
  o[1] = v & 0x00F000F0u;
  o[2] = v >> 8 & 0x000F000Fu;
  o[3] = v >> 8 & 0x00F000F0u;
}
constexpr uint32_t kOnes = 0x00010001u, kSixteens = 0x00100010u;
// What undoes the operands' units: 2^133 2^-64, or 2^24.
template <bool F8>
constexpr float kUnit = F8 ? 16777216.f : 590295810358705651712.f;

// Eight elements of x as operands to match.
__device__ __forceinline__ void x_bf16(const uint4& e, uint32_t (&b)[4]) {
  const uint32_t p[4] = {__byte_perm(e.x, e.z, 0x5410), __byte_perm(e.x, e.z, 0x7632), __byte_perm(e.y, e.w, 0x5410),
                         __byte_perm(e.y, e.w, 0x7632)};
#pragma unroll
  for (int i = 0; i < 4; ++i)  // times 2^64 or 2^60
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(b[i]) : "r"(p[i]), "r"(i % 2 == 0 ? 0x5F805F80u : 0x5D805D80u));
}
__device__ __forceinline__ void x_e4m3(const uint2& e, uint32_t (&b)[4]) {
  const uint32_t lo = __byte_perm(e.x, e.y, 0x5140), hi = __byte_perm(e.x, e.y, 0x7362);
  const uint16_t h[4] = {static_cast<uint16_t>(lo), static_cast<uint16_t>(lo >> 16), static_cast<uint16_t>(hi),
                         static_cast<uint16_t>(hi >> 16)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b[i]) : "h"(h[i]));
    if (i % 2 == 1) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(b[i]) : "r"(0x2C002C00u));  // a sixteenth
  }
}

// The sum of eight elements that are operands.
template <bool F8>
__device__ __forceinline__ float operand_sum(const uint32_t (&b)[4]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (F8) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b[i]));
      sum = fmaf(v.x + v.y, i % 2 == 0 ? 1.f : 16.f, sum);
    } else {
      const float one = i % 2 == 0 ? 0x1p-64f : 0x1p-60f;
      sum = fmaf(__uint_as_float(b[i] << 16), one, sum);
      sum = fmaf(__uint_as_float(b[i] & 0xFFFF0000u), one, sum);
    }
  }
  return sum;
}

// The lane group's place among the 16-byte units of its rows: what differs
// between neighbours is first the widest reads' own bit.
__device__ __forceinline__ int unit_key(int g) { return (g & 2) | g >> 2; }

template <int NT>
struct Sums {  // m16n8 fragments: [fragment][n-tile]
  float v[2][NT][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) v[m][n][0] = v[m][n][1] = v[m][n][2] = v[m][n][3] = 0.f;
  }
};

// acc += the first `groups` groups of a stage.  fetch(n, i, b): n-tile n's
// operands for this lane's i-th word of codes, of the first NT n-tiles.
// x_scale: of the lane's two columns of each n-tile.  x_sums(n, i): the sums
// of x over group i in these columns, or null: by MMAs of their own.
template <int GROUP, int NT, bool F8, int TILES, typename Fetch, typename XSums>
__device__ __forceinline__ void add_stage(const uint8_t* stage, int groups, Fetch&& fetch, XSums&& x_sums,
                                          const float (&x_scale)[TILES][2], Sums<TILES>& acc) {
  constexpr bool kGiven = !std::is_same_v<std::decay_t<XSums>, std::nullptr_t>;
  constexpr int kWords = GROUP / 32;  // of a thread, row and group
  const int g = threadIdx.x % 32 >> 2, q = threadIdx.x & 3;
  const uint8_t* codes = stage + g * kRowBytes;
  const int unit = ((q * kWords / 4 ^ unit_key(g)) << 4) + q * kWords % 4 * 4;
#pragma unroll
  for (int gi = 0; gi < kGroups<GROUP>; ++gi) {
    if (gi >= groups) break;
    uint32_t v[4][kWords];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* at = codes + (unit ^ gi * GROUP / 2) + j * 8 * kRowBytes;
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
    float sum[2][NT][4], all[NT][4];  // all: x's own sums, in every row
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      uint32_t b[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        fetch(n, gi * kWords + w, b[n]);
        if constexpr (!kGiven) {
          if (w == 0)
            mma_first<F8>(all[n], kOnes, kOnes, kSixteens, kSixteens, b[n][0], b[n][1]);
          else
            mma<F8>(all[n], kOnes, kOnes, kSixteens, kSixteens, b[n][0], b[n][1]);
          mma<F8>(all[n], kOnes, kOnes, kSixteens, kSixteens, b[n][2], b[n][3]);
        }
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t a0[4], a1[4];
        widen(v[2 * m][w], a0);
        widen(v[2 * m + 1][w], a1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (w == 0)
            mma_first<F8>(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
          else
            mma<F8>(sum[m][n], a0[0], a1[0], a0[1], a1[1], b[n][0], b[n][1]);
          mma<F8>(sum[m][n], a0[2], a1[2], a0[3], a1[3], b[n][2], b[n][3]);
        }
      }
    }
    if constexpr (kGiven) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 v = x_sums(n, gi);
        all[n][0] = v.x;
        all[n][1] = v.y;
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float2 sc = *reinterpret_cast<const float2*>(stage + kScales + (gi * kRows + m * 16 + 2 * g) * 4);
      sc.x *= kUnit<F8>;
      sc.y *= kUnit<F8>;
      const uint32_t z = *reinterpret_cast<const uint16_t*>(stage + kZeros<GROUP> + gi * kRows + m * 16 + 2 * g);
      // 2^23 + z as a float's bits, less 2^23
      const float z0 = __uint_as_float(__byte_perm(z, 0x4B000000u, 0x7650)) - 8388608.f;
      const float z1 = __uint_as_float(__byte_perm(z, 0x4B000000u, 0x7651)) - 8388608.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float* c = acc.v[m][n];
        float t[4] = {fmaf(-z0, all[n][0], sum[m][n][0]), fmaf(-z0, all[n][1], sum[m][n][1]),
                      fmaf(-z1, all[n][0], sum[m][n][2]), fmaf(-z1, all[n][1], sum[m][n][3])};
        if constexpr (F8) {
          t[0] *= x_scale[n][0];
          t[1] *= x_scale[n][1];
          t[2] *= x_scale[n][0];
          t[3] *= x_scale[n][1];
        }
        c[0] = fmaf(sc.x, t[0], c[0]);
        c[1] = fmaf(sc.x, t[1], c[1]);
        c[2] = fmaf(sc.y, t[2], c[2]);
        c[3] = fmaf(sc.y, t[3], c[3]);
      }
    }
  }
}

// What both kernels' warps have: their ring and the tile whose codes go into it.
template <int GROUP>
struct Ring {
  const Int4Args& p;
  uint8_t *const base, *const end;  // of this warp
  const int bytes;        // of a stage
  const int lane;
  uint8_t *in, *out;      // the slots to be filled and to be read next

  __device__ __forceinline__ Ring(const Int4Args& p_, uint8_t* base_, int bytes_)
      : p(p_), base(base_), end(base_ + p_.depth * bytes_), bytes(bytes_), lane(threadIdx.x % 32), in(base_), out(base_) {
    if (p.zeros == nullptr)  // 8 everywhere, and nothing loaded over it
      for (uint8_t* slot = base; slot < end; slot += bytes)
        for (int i = lane; i < kGroups<GROUP> * kRows / 4; i += 32)
          *reinterpret_cast<uint32_t*>(slot + kZeros<GROUP> + i * 4) = 0x08080808u;
  }

  // This lane's codes, scales and zero points of a tile's next stage.
  struct Tile {
    const uint8_t* codes[4];
    const float* scales;
    const uint8_t* zeros;
  };
  __device__ __forceinline__ Tile tile(int expert, int index, int st) const {
    const int r0 = p.swiglu ? index * (kRows / 2) : index * kRows, second = p.swiglu ? p.n / 2 : kRows / 2;
    const int up = p.swiglu || r0 + kRows / 2 < p.n ? second : 0;  // without a second fragment: the first again
    const int row_bytes = p.k / 2;
    Tile t;
    t.codes[0] = p.codes + (static_cast<int64_t>(expert) * p.n + r0 + 2 * (lane / 4)) * row_bytes + lane % 4 * 16 + st * kRowBytes;
    t.codes[1] = t.codes[0] + row_bytes;
    t.codes[2] = t.codes[0] + static_cast<int64_t>(up) * row_bytes;
    t.codes[3] = t.codes[2] + row_bytes;
    const int64_t meta = (static_cast<int64_t>(expert) * (p.k / GROUP) + st * kGroups<GROUP>) * p.n + r0;
    t.scales = p.scales + meta + (lane % 8 >= 4 ? up : 0) + lane % 4 * 4 + static_cast<int64_t>(lane / 8) * p.n;
    t.zeros = p.zeros + meta + (lane % 4 >= 2 ? up : 0) + lane % 2 * 8 + static_cast<int64_t>(lane / 4) * p.n;
    return t;
  }
  // A tile's stage into the next slot: `left` elements of a row from it on; t goes on by `step` stages.
  __device__ __forceinline__ void load(Tile& t, int left, int step) {
    // row j of lane group h stands at row 8 j + h: rows 2 h and 2 h + 1 of each fragment
    const int h = lane / 4;
    uint8_t* to = in + h * kRowBytes + ((lane % 4 ^ unit_key(h)) << 4);
    if (lane % 4 * 32 < left) {
#pragma unroll
      for (int j = 0; j < 4; ++j) cp_async_16(to + j * 8 * kRowBytes, t.codes[j]);
    }
    // scales: 4 rows to a lane; zero points: 8
    if (lane < kGroups<GROUP> * 8 && lane / 8 * GROUP < left) cp_async_16(in + kScales + lane * 16, t.scales);
    if (p.zeros != nullptr && lane < kGroups<GROUP> * 4 && lane / 4 * GROUP < left)
      cp_async_8(in + kZeros<GROUP> + lane * 8, t.zeros);
#pragma unroll
    for (int j = 0; j < 4; ++j) t.codes[j] += step * kRowBytes;
    const int64_t meta = static_cast<int64_t>(step * kGroups<GROUP>) * p.n;
    t.scales += meta;
    t.zeros += meta;
  }
  // Ends the loads into a slot (there may be none).
  __device__ __forceinline__ void commit() {
    cp_async_commit();
    in += bytes;
    if (in == end) in = base;
  }
  // The oldest slot, landed for the whole warp, which has also read the one before it.
  __device__ __forceinline__ const uint8_t* wait() {
    cp_async_wait_pending(p.depth - 2);
    __syncwarp();
    const uint8_t* src = out;
    out += bytes;
    if (out == end) out = base;
    return src;
  }
  // The slot that was read last: nothing is loaded there before the next wait.
  __device__ __forceinline__ float* used() const { return reinterpret_cast<float*>((out == base ? end : out) - bytes); }
};

__device__ __forceinline__ void store(const Int4Args& p, int64_t row, int col, float v) {
  if (p.out_f32)
    static_cast<float*>(p.out)[row * p.ld_out + col] = v;
  else
    static_cast<uint16_t*>(p.out)[row * p.ld_out + col] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ bool is_bad(const Shared& s, int pair) { return s.bad[pair / 32] >> (pair % 32) & 1u; }

// The parts: each expert's pairs in order, at most nx to a part.  A pair's
// place is the number of smaller keys (expert, pair), compared one by one.
// keys: scratch of kMaxPairs words.
__device__ __forceinline__ void find_parts(const Int4Args& p, Shared& s, int32_t* keys) {
  constexpr int kWordsOf = kMaxPairs / 32;
  static_assert(kMaxPairs <= kThreads, "a thread per pair");
  const int e = threadIdx.x, lane = e % 32, warp = e / 32, most = p.nx;
  if (p.ids == nullptr) {
    if (e < p.pairs) s.pair[e] = s.row[e] = static_cast<uint8_t>(e);
    const int parts = (p.pairs + most - 1) / most;
    if (e < parts) {
      s.act[e] = 0;
      s.first[e] = static_cast<int16_t>(e * most);
      s.count[e] = static_cast<uint8_t>(min(most, p.pairs - e * most));
    }
    if (e == 0) {
      s.n_parts = parts;
      s.n_good = p.pairs;
    }
    __syncthreads();
    return;
  }
  int32_t key = INT_MAX;  // of the pairs whose expert exists: expert x kMaxPairs + pair
  float w = 0.f;
  if (e < kMaxPairs) {
    const int id = e < p.pairs ? __ldg(p.ids + e) : -1;
    if (p.w != nullptr && e < p.pairs) w = __ldg(p.w + e);
    if (id >= 0 && id < p.n_experts)
      key = id * kMaxPairs + e;
    else if (e < p.pairs && blockIdx.x == 0)
      set_error(p.status, kErrDevice);
    keys[e] = key;
    const uint32_t bad = __ballot_sync(0xffffffffu, e < p.pairs && key == INT_MAX);
    if (lane == 0) {
      s.bad[warp] = bad;
      s.starts[warp] = 0u;
    }
  }
  __syncthreads();
  const bool good = key != INT_MAX;
  bool start = false;
  int at = 0;
  if (good) {
    const int own = key & ~(kMaxPairs - 1);
    int less = 0;
    for (int i = 0; i < p.pairs; i += 4) {
      const int4 k = *reinterpret_cast<const int4*>(keys + i);
      at += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
      less += (k.x < own) + (k.y < own) + (k.z < own) + (k.w < own);
    }
    const int token = e / p.top;
    s.pair[at] = static_cast<uint8_t>(e);
    s.token[at] = static_cast<uint8_t>(token);
    s.row[at] = static_cast<uint8_t>(p.x_per_slot ? e : token);
    s.w[at] = w;
    start = (at - less) % most == 0;
    if (start) atomicOr(&s.starts[at / 32], 1u << at % 32);
  }
  __syncthreads();
  if (e < kMaxPairs) {
    int part = 0, parts = 0, good_ones = p.pairs, next = kMaxPairs;
#pragma unroll
    for (int i = 0; i < kWordsOf; ++i) {
      const uint32_t word = s.starts[i];
      const int d = at - i * 32;  // bits below, and above, this one
      const uint32_t below = d >= 32 ? word : d > 0 ? word & ((1u << d) - 1u) : 0u;
      const uint32_t above = d < 0 ? word : d < 31 ? word >> (d + 1) << (d + 1) : 0u;
      part += __popc(below);
      parts += __popc(word);
      if (above != 0u) next = min(next, i * 32 + __ffs(above) - 1);
      good_ones -= __popc(s.bad[i]);
    }
    if (start) {
      s.act[part] = static_cast<int16_t>(key / kMaxPairs);
      s.first[part] = static_cast<int16_t>(at);
      s.count[part] = static_cast<uint8_t>(min(next, good_ones) - at);
    }
    if (e == 0) {
      s.n_parts = parts;
      s.n_good = good_ones;
    }
  }
  __syncthreads();
}

// A tile's sums, [row of x][weight row].
template <int NT>
__device__ __forceinline__ void put_sums(const Sums<NT>& acc, int count, float* red) {
  const int g = threadIdx.x % 32 >> 2, q = threadIdx.x & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = n * 8 + 2 * q + i;
      if (t >= count) continue;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        *reinterpret_cast<float2*>(red + t * kRedStride<NT> + 16 * m + 2 * g) = make_float2(acc.v[m][n][i], acc.v[m][n][2 + i]);
    }
}

// ------------------------------------------------ each pair a row of its own
// Dynamic shared memory: the rings (and first the keys), the warps' sums of
// two tiles, those of a batch of tiles where a cluster splits k, x, its scales.
template <int NT>
constexpr int kRedRows = NT == 1 ? 2 * kWarps * kRedStride<NT> : 0;  // floats of the warps' sums, for a row of x
constexpr int kBatchBytes = 8 * 1024;                            // of a batch's sums, about

// SPLIT: k is split over the blocks of a cluster.
template <int GROUP, int NT, bool F8, bool SPLIT>
struct RowsWorker {
  static constexpr int kWords = GROUP / 32;
  static_assert(NT == 1 || NT * 8 * kRedStride<NT> * 4 <= kZeros<GROUP>, "sums over the zero points");
  const Int4Args& p;
  Shared& s;
  uint8_t* const block;   // the dynamic array
  Ring<GROUP> ring;
  uint8_t* const x;       // [stage][word of a lane][row of x][quad's lane] x 16 bytes
  float* const x_sums;    // [group][row of x], an even number of them: in the operands' units
  float* const x_scales;  // [stage][row of x]
  float* const sums;      // [tile of the batch][row of x][weight row]
  float* const reds;      // [turn][warp][row of x][weight row]
  const int lane, group, mine, groups;  // groups of ks warps; this warp's place in its own
  const int tiles;        // of a matrix
  int lo, hi;             // this block's (or cluster's) tiles of all parts
  int s0, s1;             // its stages

  // A walk over the group's tiles.  Segments end where the part or the batch does.
  struct Place {
    int sub, seg_end, st, part;
    typename Ring<GROUP>::Tile tile;
  };
  Place in;

  __device__ __forceinline__ RowsWorker(const Int4Args& p_, Shared& s_, uint8_t* smem)
      : p(p_),
        s(s_),
        block(smem),
        ring(p_, smem + threadIdx.x / 32 * p_.depth * kStage<GROUP>, kStage<GROUP>),
        x(smem + kWarps * p_.depth * kStage<GROUP> + (p_.batch * kRows + kRedRows<NT>) * p_.nx * 4),
        x_sums(reinterpret_cast<float*>(x + p_.slice * p_.nx * kXBytes)),
        x_scales(x_sums + p_.slice * kGroups<GROUP> * ((p_.nx + 1) & ~1)),
        sums(reinterpret_cast<float*>(smem + kWarps * p_.depth * kStage<GROUP>)),
        reds(sums + p_.batch * p_.nx * kRows),
        lane(threadIdx.x % 32),
        group(threadIdx.x / 32 >> p_.ks_bits),
        mine(threadIdx.x / 32 & (p_.ks - 1)),
        groups(kWarps >> p_.ks_bits),
        tiles(p_.tiles) {
    const int nst = (p.k + kStageK - 1) / kStageK;
    const int rank = SPLIT ? static_cast<int>(cluster_ctarank()) : 0;
    s0 = min(nst, rank * p.slice);
    s1 = min(nst, s0 + p.slice);
    const uint32_t total = s.n_parts * tiles;  // n is at most 2^24: 2^28
    const uint32_t at = SPLIT ? blockIdx.x / p.cluster : blockIdx.x, of = SPLIT ? gridDim.x / p.cluster : gridDim.x;
    uint32_t each = total / of, more = total - each * of, first = 0, place = at;
    if (!SPLIT && s.n_parts > 1 && of >= s.n_parts) {
      // Blocks of their own for each part, where none has more tiles for it:
      // no block changes its x (one row by 8 of 256 experts of 4096 x 2048: 17 -> 15 us).
      const uint32_t blocks = of / s.n_parts, own = tiles / blocks, rest = tiles - own * blocks;
      if (own + (rest > 0) <= each + (more > 0)) {
        const uint32_t part = at / blocks;
        first = part * tiles;
        place = at - part * blocks;
        each = part < s.n_parts ? own : 0;
        more = part < s.n_parts ? rest : 0;
      }
    }
    lo = static_cast<int>(first + each * place + min(place, more));
    hi = lo + static_cast<int>(each + (place < more));
  }
  __device__ __forceinline__ int segment_end(int from, int part) const {
    int end = min(hi, (part + 1) * tiles);
    if (SPLIT) end = min(end, lo + ((from - lo) / p.batch + 1) * p.batch);
    return end;
  }
  __device__ __forceinline__ void settle(Place& a) const {  // onto a tile of this group, or to the end
    while (a.sub >= a.seg_end && a.seg_end < hi) {
      a.sub = a.seg_end + group;
      if (a.seg_end == (a.part + 1) * tiles) ++a.part;
      a.seg_end = segment_end(a.seg_end, a.part);
    }
    if (a.sub >= a.seg_end || s0 + mine >= s1) {
      a.sub = hi;
      return;
    }
    a.st = s0 + mine;
    a.tile = ring.tile(s.act[a.part], a.sub - a.part * tiles, a.st);
  }
  __device__ __forceinline__ void issue() {
    if (in.sub < hi) {
      ring.load(in.tile, p.k - in.st * kStageK, p.ks);
      in.st += p.ks;
      if (in.st >= s1) {
        in.sub += groups;
        settle(in);
      }
    }
    ring.commit();
  }

  // The rows of x of a part, as operands.
  __device__ __forceinline__ void load_x(int part) {
    const int count = s.count[part], first = s.first[part];
    const int units = min((s1 - s0) * (kStageK / 8), (p.k - s0 * kStageK) / 8);  // of 8 elements
    // a warp takes kBatch x 32 units of a row at a time, their loads together
    constexpr int kBatch = 8;
    using Unit = std::conditional_t<F8, uint2, uint4>;
    const int blocks = (units + kBatch * 32 - 1) / (kBatch * 32);
    for (int i = threadIdx.x / 32; i < blocks * count; i += kWarps) {
      const int t = i / blocks, u0 = (i - t * blocks) * kBatch * 32 + lane;
      const Unit* from = reinterpret_cast<const Unit*>(static_cast<const uint8_t*>(p.x) +
                                                       (s.row[first + t] * p.ld_x + s0 * kStageK) * (F8 ? 1 : 2));
      Unit e[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (u0 + j * 32 < units) e[j] = __ldg(from + u0 + j * 32);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int u = u0 + j * 32;
        if (u - lane >= units) break;
        uint32_t b[4] = {};
        if (u < units) {
          if constexpr (F8)
            x_e4m3(e[j], b);
          else
            x_bf16(e[j], b);
        }
        float sum = operand_sum<F8>(b);
#pragma unroll
        for (int o = GROUP / 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (u >= units) break;
        if (u % (GROUP / 8) == 0) x_sums[u / (GROUP / 8) * ((p.nx + 1) & ~1) + t] = sum / kUnit<F8>;
        const int st = u / 16, r = u % 16 % (GROUP / 8), word = u % 16 / (GROUP / 8) * kWords + r % kWords, quad = r / kWords;
        *reinterpret_cast<uint4*>(x + (((st * 4 + word) * p.nx + t) * 4 + quad) * 16) = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
    if constexpr (F8)
      for (int i = threadIdx.x; i < (s1 - s0) * count; i += kThreads) {
        const int st = i / count, t = i - st * count;
        x_scales[st * p.nx + t] = __ldg(p.x_scales + static_cast<int64_t>(s.row[first + t]) * ((p.k + 127) / 128) + s0 + st);
      }
  }

  // A tile's result for one row of x, from the lanes' sums over k.
  __device__ __forceinline__ void finish(int tile, int pair, float v) const {
    if (p.swiglu) {
      const float up = __shfl_down_sync(0xffffffffu, v, kRows / 2);
      if (lane < kRows / 2) store(p, pair, tile * (kRows / 2) + lane, v / (1.f + expf(-v)) * up);
    } else if (tile * kRows + lane < p.n) {
      store(p, pair, tile * kRows + lane, v);
    }
  }

  __device__ __forceinline__ void take(int st, int count, Sums<NT>& acc) {
    const uint8_t* src = ring.wait();
    issue();
    const int g = lane >> 2, q = lane & 3;
    const uint8_t* xs = x + (st - s0) * p.nx * kXBytes + q * 16;
    const uint8_t* at[NT];
    float scale[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      at[n] = xs + min(n * 8 + g, count - 1) * 64;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        scale[n][i] = F8 ? x_scales[(st - s0) * p.nx + min(n * 8 + 2 * q + i, count - 1)] : 1.f;
    }
    const int word = p.nx * 64, left = (p.k - st * kStageK) / GROUP;
    auto fetch = [&](int n, int i, uint32_t(&b)[4]) {
      const uint4 e = *reinterpret_cast<const uint4*>(at[n] + i * word);
      b[0] = e.x, b[1] = e.y, b[2] = e.z, b[3] = e.w;
    };
    auto sums_of = [&](int n, int i) {
      return *reinterpret_cast<const float2*>(x_sums + ((st - s0) * kGroups<GROUP> + i) * ((p.nx + 1) & ~1) +
                                              min(n * 8 + 2 * q, (count - 1) & ~1));
    };
    if (NT > 1 && count <= 8)
      add_stage<GROUP, 1, F8>(src, left, fetch, sums_of, scale, acc);
    else
      add_stage<GROUP, NT, F8>(src, left, fetch, sums_of, scale, acc);
  }

  // The sums of a batch of tiles over the cluster's blocks; a tile's is finished by one of them.
  __device__ __forceinline__ void join(int from, int to) {
    cluster_sync();
    const int rank = static_cast<int>(cluster_ctarank()), warp = threadIdx.x / 32;
    const int count = s.count[0];  // (one part: its rows are all the matrix meets at once)
    for (int i = warp; i < (to - from) * count; i += kWarps) {
      const int b = i / count, t = i - b * count;
      if (b % p.cluster != rank) continue;
      const uint32_t at = smem_u32(sums + (b * p.nx + t) * kRows + lane);
      float v = 0.f;
      for (int r = 0; r < p.cluster; ++r) {
        float w;
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(mapa_shared(at, r)) : "memory");
        v += w;
      }
      const int part = (from + b) / tiles;
      if (t < s.count[part]) finish(from + b - part * tiles, s.pair[s.first[part] + t], v);
    }
    cluster_sync();
  }

  __device__ __forceinline__ void run() {
    int part = s.n_parts > 1 ? lo / tiles : 0;
    in.sub = lo + group;
    in.part = part;
    in.seg_end = lo < hi ? segment_end(lo, part) : lo;
    settle(in);
    for (int i = 0; i < p.depth - 1; ++i) issue();
    auto meet = [&]() {  // the warps that share a tile
      if (p.ks > 1)
        named_bar_sync(1 + group, p.ks * 32);
      else
        __syncwarp();
    };
    const int first_warp = group * p.ks;
    int turn = 0;
    for (int from = lo; from < hi;) {
      const int to = segment_end(from, part);
      const int count = s.count[part], first = s.first[part];
      if (from == lo || from == part * tiles) load_x(part);
      __syncthreads();
      for (int sub = from + group; sub < to; sub += groups) {
        Sums<NT> acc;
        acc.clear();
        for (int st = s0 + mine; st < s1; st += p.ks) take(st, count, acc);
        // the warps' sums: two sets in turn, so that a tile's are read while the next one's are written
        // (with more than 8 rows in the slot just read, which no one loads into before all have read it)
        float* const set = reds + (turn * kWarps + first_warp) * p.nx * kRedStride<NT>;
        turn ^= 1;
        if constexpr (NT > 1) {
          float* red = ring.used();
          __syncwarp();  // all lanes have read it
          put_sums(acc, count, red);
          if (lane == 0) s.red[threadIdx.x / 32] = static_cast<int>(red - reinterpret_cast<float*>(block));
        } else {
          put_sums(acc, count, set + mine * p.nx * kRedStride<NT>);
        }
        meet();
        // another warp each time, where there are fewer rows than warps
        for (int t = (mine - ((sub - from) >> (4 - p.ks_bits))) & (p.ks - 1); t < count; t += p.ks) {
          float v = 0.f;
          const int at = t * kRedStride<NT> + lane;
#pragma unroll 4
          for (int w = 0; w < p.ks; ++w)
            v += NT > 1 ? reinterpret_cast<const float*>(block)[s.red[first_warp + w] + at] : set[w * p.nx * kRedStride<NT> + at];
          if constexpr (SPLIT)
            sums[((sub - lo) % p.batch * p.nx + t) * kRows + lane] = v;
          else
            finish(sub - part * tiles, s.pair[first + t], v);
        }
        if constexpr (NT > 1) meet();
      }
      __syncthreads();  // x may be replaced
      if constexpr (SPLIT)
        if (to == hi || (to - lo) % p.batch == 0) join(lo + (to - 1 - lo) / p.batch * p.batch, to);
      from = to;
      if (to == (part + 1) * tiles) ++part;
    }
    cp_async_wait_all();
    // rows whose expert does not exist
    const int cols = p.swiglu ? p.n / 2 : p.n;
    if (s.n_good < p.pairs)
      for (int i = 0; i < p.pairs; ++i)
        if (is_bad(s, i))
          for (int c = blockIdx.x * kThreads + threadIdx.x; c < cols; c += gridDim.x * kThreads)
            store(p, i, c, __int_as_float(0x7FC00000));
  }
};

template <int GROUP, int NT, bool F8, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ Int4Args p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared s;
  find_parts(p, s, reinterpret_cast<int32_t*>(smem));
  RowsWorker<GROUP, NT, F8, SPLIT> w(p, s, smem);
  w.run();
}

// --------------------------------------------- the weighted sum of a row's pairs
// Dynamic shared memory: the rings (and first the keys), the warps' sums.
template <int GROUP, bool F8>
struct SumWorker {
  static constexpr int kWords = GROUP / 32;
  static_assert(8 * kRedStride<1> * 4 <= kZeros<GROUP>, "sums over the zero points");
  const Int4Args& p;
  Shared& s;
  Ring<GROUP> ring;
  float* const all;       // [warp][row of out][weight row]
  float* const joined;    // [turn][row of out][weight row], where a cluster shares a tile
  const int lane, warp, tokens, nst;
  const int tiles;
  int lo, hi;             // of the stages of all parts, one after the other: this warp's

  struct Place {
    int tile, part, st;
    int64_t x;
    typename Ring<GROUP>::Tile at;
  };
  Place in;

  __host__ __device__ static constexpr int stage(int nx) {
    return (kStage<GROUP> + nx * (kRingX<F8> + (F8 ? 4 : 0)) + 127) / 128 * 128;
  }
  __device__ __forceinline__ SumWorker(const Int4Args& p_, Shared& s_, uint8_t* smem)
      : p(p_),
        s(s_),
        ring(p_, smem + threadIdx.x / 32 * p_.depth * stage(p_.nx), stage(p_.nx)),
        all(reinterpret_cast<float*>(smem + kWarps * p_.depth * stage(p_.nx))),
        joined(all + kWarps * (p_.pairs / p_.top) * kRows),
        lane(threadIdx.x % 32),
        warp(threadIdx.x / 32),
        tokens(p_.pairs / p_.top),
        nst((p_.k + kStageK - 1) / kStageK),
        tiles((p_.n + kRows - 1) / kRows) {
    const int total = s.n_parts * nst;  // k is at most 49152: 2^17
    const int place = cluster_ctarank() * kWarps + warp, of = p.cluster * kWarps;
    lo = total * place / of;
    hi = total * (place + 1) / of;
  }
  __device__ __forceinline__ void start(Place& a, int tile) const {
    a.tile = lo < hi ? tile : tiles;
    a.part = lo / nst;
    a.st = lo - a.part * nst;
    if (a.tile < tiles) at_part(a);
  }
  __device__ __forceinline__ void at_part(Place& a) const {
    a.at = ring.tile(s.act[a.part], a.tile, a.st);
    a.x = x_of(a.part, lane / 16) + a.st * kStageK;
  }
  // this lane's elements of the first stage of a part's row t, as an index into x
  __device__ __forceinline__ int64_t x_of(int part, int t) const {
    return s.row[s.first[part] + min(t, s.count[part] - 1)] * p.ld_x + lane % 16 * 8;
  }
  __device__ __forceinline__ void issue() {
    if (in.tile < tiles) {
      // x: 8 elements to a lane, in the order in which the quads read them
      uint8_t* x = ring.in + kStage<GROUP>;
      const int count = s.count[in.part], left = p.k - in.st * kStageK;
      const int u = lane % 16, r = u % (GROUP / 8);
      const int at = u / (GROUP / 8) * (GROUP / 8) + r % kWords * 4 + r / kWords;
      int64_t from = in.x;
      if (u * 8 < left)
        for (int t = lane / 16; t < count; t += 2) {
          if (t >= 2) from = x_of(in.part, t) + in.st * kStageK;
          if constexpr (F8)
            cp_async_8(x + t * kRingX<F8> + at * 8, static_cast<const uint8_t*>(p.x) + from);
          else
            cp_async_16(x + t * kRingX<F8> + ((at ^ (t & 1) << 2) << 4), static_cast<const uint16_t*>(p.x) + from);
        }
      if constexpr (F8)
        if (lane < count)
          cp_async_4(x + p.nx * kRingX<F8> + lane * 4,
                     p.x_scales + static_cast<int64_t>(s.row[s.first[in.part] + lane]) * ((p.k + 127) / 128) + in.st);
      ring.load(in.at, left, 1);
      in.x += kStageK;
      ++in.st;
      if (in.part * nst + in.st == hi) {
        start(in, in.tile + gridDim.x / p.cluster);
      } else if (in.st == nst) {
        in.st = 0;
        ++in.part;
        at_part(in);
      }
    }
    ring.commit();
  }
  __device__ __forceinline__ void take(int st, int count, Sums<1>& acc) {
    const uint8_t* src = ring.wait();
    issue();
    const int q = lane & 3, t = min(lane >> 2, count - 1);
    const uint8_t* x = src + kStage<GROUP> + t * kRingX<F8>;
    // 16-bit rows: where the units of even and of odd 64 bytes are
    const uint8_t* at[2] = {x + q * (F8 ? 8 : 16) + (F8 ? 0 : (t & 1) << 6), x + q * (F8 ? 8 : 16) - (F8 ? 0 : (t & 1) << 6)};
    float scale[1][2] = {{1.f, 1.f}};
    if constexpr (F8) {
      const float* xs = reinterpret_cast<const float*>(src + kStage<GROUP> + p.nx * kRingX<F8>);
      scale[0][0] = xs[min(2 * q, count - 1)];
      scale[0][1] = xs[min(2 * q + 1, count - 1)];
    }
    add_stage<GROUP, 1, F8>(
        src, (p.k - st * kStageK) / GROUP,
        [&](int, int i, uint32_t(&b)[4]) {
          if constexpr (F8)
            x_e4m3(*reinterpret_cast<const uint2*>(at[0] + i * 32), b);
          else
            x_bf16(*reinterpret_cast<const uint4*>(at[i & 1] + i * 64), b);
        },
        nullptr, scale, acc);
  }
  __device__ __forceinline__ void finish(int tile, int t, float v) const {
    if (s.n_good < p.pairs)
      for (int i = t * p.top; i < (t + 1) * p.top; ++i)
        if (is_bad(s, i)) v = __int_as_float(0x7FC00000);
    if (tile * kRows + lane < p.n) store(p, t, tile * kRows + lane, v);
  }
  __device__ __forceinline__ void run() {
    float* sums = all + warp * tokens * kRows;
    const int step = gridDim.x / p.cluster, rank = cluster_ctarank();
    start(in, blockIdx.x / p.cluster);
    for (int i = 0; i < p.depth - 1; ++i) issue();
    int turn = 0;
    for (int tile = blockIdx.x / p.cluster; tile < tiles; tile += step) {
      for (int t = 0; t < tokens; ++t) sums[t * kRows + lane] = 0.f;
      for (int at = lo; at < hi;) {
        const int part = at / nst, end = min(hi, (part + 1) * nst);
        const int count = s.count[part], first = s.first[part];
        Sums<1> acc;
        acc.clear();
        for (; at < end; ++at) take(at - part * nst, count, acc);
        float* red = ring.used();
        __syncwarp();  // all lanes have read it
        put_sums(acc, count, red);
        __syncwarp();
        for (int i = 0; i < count; ++i) {
          float& v = sums[s.token[first + i] * kRows + lane];
          v = fmaf(s.w[first + i], red[i * kRedStride<1> + lane], v);
        }
        __syncwarp();
      }
      __syncthreads();
      for (int t = warp; t < tokens; t += kWarps) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += all[(w * tokens + t) * kRows + lane];
        if (p.cluster == 1)
          finish(tile, t, v);
        else
          joined[(turn * tokens + t) * kRows + lane] = v;
      }
      if (p.cluster == 1) {
        __syncthreads();
        continue;
      }
      // the blocks' sums; those of the next tile go elsewhere, and the one after that waits for all blocks
      cluster_sync();
      for (int t = warp * p.cluster + rank; t < tokens; t += kWarps * p.cluster) {
        const uint32_t at = smem_u32(joined + (turn * tokens + t) * kRows + lane);
        float v = 0.f;
        for (int r = 0; r < p.cluster; ++r) {
          float w;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(mapa_shared(at, r)) : "memory");
          v += w;
        }
        finish(tile, t, v);
      }
      turn ^= 1;
    }
    if (p.cluster > 1) cluster_sync();  // a block's shared memory is read until here
    cp_async_wait_all();
  }
};

template <int GROUP, bool F8>
__global__ void __launch_bounds__(kThreads, 1) sum_kernel(const __grid_constant__ Int4Args p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Shared s;
  find_parts(p, s, reinterpret_cast<int32_t*>(smem));
  SumWorker<GROUP, F8> w(p, s, smem);
  w.run();
}

// ------------------------------------------------------------------ launches
constexpr int kSmem = 227 * 1024 - static_cast<int>(sizeof(Shared)) - 128;  // dynamic, of a block

// Allows a kernel its shared memory, once per device (bits of `done`).
template <typename K>
cudaError_t allow_shared(K kernel, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Clusters of `size` blocks that are resident at once (a cluster stays within
// a part of the GPU: 36 of 4, 15 of 8), asked for once per device.
template <typename K>
int64_t resident_clusters(K kernel, int size, int num_sms, std::atomic<int> (&known)[64]) {
  if (size <= 1) return num_sms;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 1;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms / size * size, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 1;
    }
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Of x in rows_kernel: operands, sums, scales.
template <int GROUP, bool F8>
int rows_x_bytes(int stages, int rows) {
  return stages * (rows * kXBytes + kGroups<GROUP> * ((rows + 1) & ~1) * 4 + (F8 ? rows * 4 : 0));
}

template <typename K>
cudaError_t launch_clusters(K kernel, int64_t clusters, const Int4Args& a, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * a.cluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int GROUP, int NT, bool F8, bool SPLIT>
cudaError_t launch_rows(Int4Args a, int num_sms, cudaStream_t st) {
  auto kernel = rows_kernel<GROUP, NT, F8, SPLIT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, done);
  if (e != cudaSuccess) return e;
  const int out_cols = a.swiglu ? kRows / 2 : kRows, cols = a.swiglu ? a.n / 2 : a.n;
  const int64_t tiles = a.tiles = (cols + out_cols - 1) / out_cols;
  const int nst = (a.k + kStageK - 1) / kStageK;
  static std::atomic<int> known[4][64];  // by the logarithm of the size
  const int64_t clusters = resident_clusters(kernel, a.cluster, num_sms, known[a.cluster >= 8 ? 3 : a.cluster >= 4 ? 2 : a.cluster - 1]);
  const int64_t at_most = (a.ids != nullptr ? a.pairs : (a.pairs + a.nx - 1) / a.nx) * tiles;
  const int64_t about = (a.ids != nullptr ? std::min(a.pairs, a.n_experts) : (a.pairs + a.nx - 1) / a.nx) * tiles;
  const int64_t of = std::min(at_most, clusters);
  a.slice = (nst + a.cluster - 1) / a.cluster;
  // Sixteen warps on one tile, or groups of them on several: what leaves the
  // busiest with the least, with 256 bytes of each row read together if there
  // are that many.  A tile's end counts as a stage (one row by 14336 x 4096: 10.4 us,
  // 11.7 where it counts as none; as two or three: the same, here and at 11 other shapes).
  const int64_t share = (about + of - 1) / of;
  int64_t least = INT64_MAX;
  int fewest = 1;
  while (fewest < 4 && 2 * fewest <= a.slice) fewest *= 2;
  for (int ks = fewest; ks == fewest || (ks <= kWarps && ks <= a.slice); ks *= 2) {
    const int64_t load = (share + kWarps / ks - 1) / (kWarps / ks) * ((a.slice + ks - 1) / ks + 1);
    if (load < least) {
      least = load;
      a.ks = ks;
    }
  }
  for (a.ks_bits = 0; 1 << a.ks_bits < a.ks;) ++a.ks_bits;
  const int x_bytes = rows_x_bytes<GROUP, F8>(a.slice, a.nx);
  a.batch = a.cluster > 1 ? static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(share, kBatchBytes / (a.nx * kRows * 4)))) : 0;
  const int rest = kSmem - x_bytes - (a.batch * kRows + kRedRows<NT>) * a.nx * 4;
  a.depth = std::min(kMaxDepth, rest / (kWarps * kStage<GROUP>));
  if (a.depth < 2) return cudaErrorInvalidValue;
  const int smem = std::max(kSmem - rest + a.depth * kWarps * kStage<GROUP>, kKeyBytes);
  return launch_clusters(kernel, of, a, smem, st);
}

template <int GROUP, bool F8>
cudaError_t launch_sum(Int4Args a, int num_sms, cudaStream_t st) {
  auto kernel = sum_kernel<GROUP, F8>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, done);
  if (e != cudaSuccess) return e;
  const int tokens = a.pairs / a.top, tiles = (a.n + kRows - 1) / kRows, nst = (a.k + kStageK - 1) / kStageK;
  static std::atomic<int> known[4][64];  // by the logarithm of the size
  int64_t clusters[4];
  int best = 0;
  // A tile to a block, or to a cluster: what leaves the busiest with the fewest
  // stages, a tile's end counting as 2 and a cluster's as 3 (16 rows by 6 of 64
  // experts of 2048 x 1408, 64 tiles: 34 us by blocks, 23 by pairs; 4096 x 1536: 43 and 48).
  int64_t least = INT64_MAX;
  for (int i = 0; i < 4; ++i) {
    clusters[i] = resident_clusters(kernel, 1 << i, num_sms, known[i]);
    const int64_t stages = (static_cast<int64_t>(std::min(a.pairs, a.n_experts)) * nst + (kWarps << i) - 1) / (kWarps << i);
    const int64_t load = (tiles + clusters[i] - 1) / clusters[i] * (stages + (i == 0 ? 2 : 3));
    if (load < least) {
      least = load;
      best = i;
    }
  }
  a.cluster = 1 << best;
  const int stage = kWarps * SumWorker<GROUP, F8>::stage(a.nx), sums = (kWarps + 2) * tokens * kRows * 4;
  a.depth = std::min(kMaxDepth, (kSmem - sums) / stage);
  if (a.depth < 2) return cudaErrorInvalidValue;
  return launch_clusters(kernel, std::min<int64_t>(tiles, clusters[best]), a, std::max(a.depth * stage + sums, kKeyBytes), st);
}

template <int GROUP, bool F8>
cudaError_t launch_form(Int4Args a, int num_sms, cudaStream_t s) {
  const int rows = a.pairs / a.top;  // of an expert, unless a row names it twice
  a.cluster = 1;
  a.nx = std::min(rows, 8);
  if (a.w != nullptr) return launch_sum<GROUP, F8>(a, num_sms, s);
  // Parts of up to 16 rows where experts have more than 8 on average; else the few with more than 8 are taken twice
  // (28672 x 4096, SwiGLU, 16 rows by top of E experts, parts of 16 and of 8: 8 of 8 143 and 184 us, 3 of 4 77 and 89;
  // 4 of 8 136 and 137, 2 of 4 75 and 72, 3 of 8 136 and 114, 2 of 8 127 and 96).
  if (rows > 8 && (a.ids == nullptr || a.pairs > 8 * a.n_experts)) a.nx = rows;
  // x has to fit: one matrix splits k over a cluster (its blocks walk the same
  // tiles, whatever is in memory), experts take fewer rows at a time
  const int nst = (a.k + kStageK - 1) / kStageK;
  auto fits = [&]() {
    const int x = rows_x_bytes<GROUP, F8>((nst + a.cluster - 1) / a.cluster, a.nx) + 4 * (a.nx > 8 ? kRedRows<2> : kRedRows<1>) * a.nx;
    return x <= kSmem - 2 * kWarps * kStage<GROUP> - kBatchBytes;  // two stages a warp at least
  };
  while (!fits() && a.ids == nullptr && a.cluster < kMaxCluster) a.cluster *= 2;
  while (!fits() && a.nx > 1) a.nx = (a.nx + 1) / 2;
  if (!fits()) return cudaErrorInvalidValue;
  if (a.cluster > 1)
    return a.nx > 8 ? launch_rows<GROUP, 2, F8, true>(a, num_sms, s) : launch_rows<GROUP, 1, F8, true>(a, num_sms, s);
  return a.nx > 8 ? launch_rows<GROUP, 2, F8, false>(a, num_sms, s) : launch_rows<GROUP, 1, F8, false>(a, num_sms, s);
}

template <int GROUP>
cudaError_t launch_group(const Int4Args& a, int num_sms, cudaStream_t s) {
  return a.x_scales != nullptr ? launch_form<GROUP, true>(a, num_sms, s) : launch_form<GROUP, false>(a, num_sms, s);
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
