// Product of two 4-bit block-scaled matrices: out = g_a g_b (A s_a) (B s_b)^T,
// one pair, or one B per expert for A's rows in 128-row tiles.
//
// The block-scaled tcgen05.mma (kind::mxf4: a power-of-two scale per 32
// elements; kind::mxf4nvf4: an e4m3 scale per 16) takes K = 64 codes per
// instruction from shared memory and the scales of both operands from tensor
// memory, and sums in fp32.  Codes arrive by TMA (128-byte swizzled rows of
// K = 256), scales as whole 512-byte tiles of 128 rows x 4 blocks, each of
// which becomes 4 columns of tensor memory, the same for each quarter of the
// lanes.  A row's tail past k is zero codes (TMA's fill); scale words past the
// array are not used, and no instruction runs past k.
//
// The two operands' roles.  The MMA's M side is 128 rows, its N side BN.
//  * more than 128 rows of A, or experts: A's rows are the M side, BN rows of
//    B the N side; in large dense products 256 of A's rows against 256 of B's
//    on a pair of SMs (below);
//  * up to 128 rows of A ("swap"): B's rows (the weights) are the M side and
//    all of A the N side, BN >= m of 16..128, so the 128-row side is never
//    padding and a CTA streams its weight rows once.  What bounds these is
//    the weights' HBM traffic; a cluster of up to 8 CTAs shares a tile along
//    k and adds its partial sums through distributed shared memory, in rank
//    order.
//
// Per CTA: warp 0 TMA producer, warp 1 tensor memory, scale copies and MMAs,
// warps 4.. epilogue.  Stage s of the ring has its own scale columns in tensor
// memory, so a stage's commit frees both.  Every wait on a barrier in memory is
// bounded; the allocation of tensor memory and the clusters' barriers are not
// (they wait for CTAs whose own waits are).
//
// Measured on the GPU alone (inputs larger than L2 in turn or as large as they
// are): 1 x 14336 x 4096 8.0 us, 64 x 4096 x 14336 10.1 us (the weights at 4.1
// and 3.1 TB/s: launch, first loads and the joining are most of both), 64
// experts of 1536 x 4096 in 84 row tiles 53 us (4.6 TB/s), 4096 x 14336 x 4096
// 81 us and 8192^3 164 us (nv) or 157 us (mx): 5.9, 6.7 and 7.0 PFLOP/s.
#include <cuda_bf16.h>

#include <atomic>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace cbmoe {
namespace {

constexpr int BP = 128;            // rows of the M side
constexpr int BK = 256;            // elements per stage: 128 bytes of codes
constexpr int ROW_BYTES = BK / 2;
constexpr int EPI_WARP0 = 4;
// epilogue warps: a quarter of the lanes each, and with two per quarter half
// of the columns
template <bool SWAP>
constexpr int EPI_WARPS = SWAP ? 4 : 8;
template <bool SWAP>
constexpr int THREADS = (EPI_WARP0 + EPI_WARPS<SWAP>) * 32;
constexpr int P_BYTES = BP * ROW_BYTES;

constexpr int pow2_at_least(int v) {
  int p = 32;
  while (p < v) p *= 2;
  return p;
}

template <int FMT, int BN, bool SWAP>
struct Cfg {
  static constexpr int STAGES = SWAP && BN >= 64 ? 3 : 4;  // (two CTAs per SM when swapped)
  static constexpr int W = BK / (4 * kFp4Block<FMT>);   // scale words per stage: 2 (MX) or 4 (NV)
  static constexpr int QT = (BN + 127) / 128;           // scale row tiles of the N side
  static constexpr int Q_BYTES = BN * ROW_BYTES;
  static constexpr int SF_BYTES = W * kScaleTileBytes;  // of one row tile
  static constexpr int STAGE = P_BYTES + Q_BYTES + (1 + QT) * SF_BYTES;
  static constexpr int SF0 = BN < 32 ? 32 : BN;         // first scale column
  static constexpr int SF_COLS = W * 4 * (1 + QT);      // per stage
  static constexpr int TMEM = pow2_at_least(SF0 + STAGES * SF_COLS);
  static constexpr int BYTES = STAGES * STAGE + 1024 + 256;
  static_assert(STAGE % 1024 == 0 && Q_BYTES % 1024 == 0 && BYTES <= 232448 && TMEM <= 512, "layout");
  static_assert(STAGES * STAGE >= BN * BP * 4 || !SWAP, "the ring holds the partial sums");
};

// A tile of the output: M-side rows from p0, N-side rows from q0.
struct Tile {
  int p0, q0, e;
};

template <int BN, bool SWAP>
struct Tiles {
  int pt, total;
  __device__ __forceinline__ explicit Tiles(const Fp4MatmulArgs& a) {
    const int mt = (a.m + BP - 1) / BP;
    if constexpr (SWAP) {
      pt = (a.n + BP - 1) / BP;
      total = pt;
    } else {
      pt = a.tile_offsets != nullptr ? min(max(a.tile_offsets[a.n_groups], 0), mt) : mt;
      total = pt * ((a.n + BN - 1) / BN);
    }
  }
  // consecutive tiles take the row tiles against one column tile, so that
  // the CTAs running together read few rows of B
  __device__ __forceinline__ Tile at(int i, const Fp4MatmulArgs& a) const {
    Tile t{i % pt * BP, i / pt * BN, 0};
    if (!SWAP && a.tile_offsets != nullptr) {  // the expert: the last e with tile_offsets[e] <= row tile
      int lo = 0, hi = a.n_groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (__ldg(a.tile_offsets + mid) <= i % pt)
          lo = mid;
        else
          hi = mid - 1;
      }
      t.e = lo;
    }
    return t;
  }
};

// What launches without a status word of their own ran into.
__device__ int g_error;

__device__ __forceinline__ void timed_out(const Fp4MatmulArgs& a) {
  set_error(a.status != nullptr ? a.status : &g_error, kErrTimeout);
}

// The MMA warp's place in the ring.  The whole warp walks it, so that its
// addresses are uniform values, and an elected lane issues: an MMA or a copy of
// scales then takes 37 cycles to issue, by a lane that walks alone 80 and
// more, which made a stage's copies take longer than its MMAs.
template <int STAGES>
struct Issuer {
  uint64_t* full;
  const Fp4MatmulArgs& a;
  int s = 0;
  uint32_t phase = 0;
  bool ready = false, ok = true;
  const bool leader;
  __device__ __forceinline__ Issuer(uint64_t* full_, const Fp4MatmulArgs& a_)
      : full(full_), a(a_), leader(elect_one()) {}

  // All lanes or none; false once a wait has run out.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_limit_ns));
    if (!ok) timed_out(a);
    return ok;
  }
  __device__ __forceinline__ bool wait_stage() {
    if (!__all_sync(0xffffffffu, ready) && !wait(full + s, phase)) return false;
    tc_fence_after();
    return true;
  }
  __device__ __forceinline__ void next() {
    __syncwarp();
    if (++s == STAGES) {
      s = 0;
      phase ^= 1u;
    }
    ready = mbar_test(full + s, phase);
  }
};

// One warp hands the accumulator back: its loads are done.
__device__ __forceinline__ void release(uint64_t* tempty, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(tempty);
}

// Eight 16-byte chunks (4 registers each) of a lane's row become one chunk of
// each of its 8-lane group's rows: h[4 i ..] of lane l is then chunk l % 8 of
// row i of the group, and the group's 8 lanes store 128 contiguous bytes of a
// row (a lane storing its own row's chunks would write half sectors of 32 rows
// at a time, which took longer than the MMAs of k = 4096).
__device__ __forceinline__ void transpose_chunks(uint32_t* h, int lane) {
#pragma unroll
  for (int b = 1; b < 8; b *= 2) {
    const bool upper = lane & b;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c & b) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        uint32_t& lo = h[4 * c + r];
        uint32_t& hi = h[4 * (c | b) + r];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, b);
        lo = upper ? got : lo;
        hi = upper ? hi : got;
      }
    }
  }
}

// The same word by word: h[i] of lane l becomes word l of row i.
__device__ __forceinline__ void transpose_words(uint32_t* h, int lane) {
#pragma unroll
  for (int b = 1; b < 32; b *= 2) {
    const bool upper = lane & b;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (c & b) continue;
      uint32_t& lo = h[c];
      uint32_t& hi = h[c | b];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, b);
      lo = upper ? got : lo;
      hi = upper ? hi : got;
    }
  }
}

// A warp's 32 rows x 128 bytes, lane = row, h its 32 words: to out (the first
// row's first byte, rows `pitch` bytes apart and on 16 bytes), `rows` of them,
// `elems` elements of ELEM bytes each.
template <int ELEM>
__device__ __forceinline__ void store_rows(uint8_t* out, int64_t pitch, uint32_t* h, int rows, int elems, int lane) {
  constexpr int PER = 16 / ELEM;  // elements of a chunk
  transpose_chunks(h, lane);
  uint8_t* o = out + (lane & 24) * pitch + (lane & 7) * 16;
  const int left = elems - (lane & 7) * PER;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((lane & 24) + i >= rows) continue;
    if (left >= PER) {
      *reinterpret_cast<uint4*>(o + i * pitch) = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
    } else {
#pragma unroll
      for (int u = 0; u < PER - 1; ++u) {
        if (u >= left) break;
        if constexpr (ELEM == 4)
          reinterpret_cast<uint32_t*>(o + i * pitch)[u] = h[4 * i + u];
        else
          reinterpret_cast<uint16_t*>(o + i * pitch)[u] = static_cast<uint16_t>(h[4 * i + u / 2] >> (16 * (u & 1)));
      }
    }
  }
  __syncwarp();
}

// The same for rows that start anywhere, a row's 128 bytes by the whole warp in
// words of 4 bytes.  A row of 2-byte elements that starts between two words
// is moved up by an element first: its words then hold elements 2 l - 1 and
// 2 l, the one before the first from `carry`, the last 128 bytes' last
// element; the ends of the warp's columns (`begin`, `end`) are single elements.
// (Element by element, a lane per row, 4096 x 14331 x 4096 took 542 us.)
template <int ELEM>
__device__ __forceinline__ void store_any_rows(uint8_t* out, int64_t pitch, uint32_t* h, int rows, int elems,
                                               uint32_t& carry, bool begin, bool end, int lane) {
  const auto moved = [&](int row) {
    return ELEM == 2 ? static_cast<int>(reinterpret_cast<uintptr_t>(out + row * pitch) >> 1 & 1) : 0;
  };
  if constexpr (ELEM == 2) {
    const int mine = moved(lane);
    const uint32_t before = carry;
    carry = h[31];
#pragma unroll
    for (int j = 31; j >= 0; --j) h[j] = __funnelshift_rc(j > 0 ? h[j - 1] : before, h[j], 32 - 16 * mine);
    if (end && mine && lane < rows && elems >= 64)
      *reinterpret_cast<uint16_t*>(out + lane * pitch + 126) = static_cast<uint16_t>(carry >> 16);
  }
  transpose_words(h, lane);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i >= rows) break;
    if constexpr (ELEM == 4) {
      if (lane < elems) *reinterpret_cast<uint32_t*>(out + i * pitch + lane * 4) = h[i];
    } else {
      const int up = moved(i), e = 2 * lane - up;  // the word's first element
      uint8_t* o = out + i * pitch + e * 2;
      if (begin && e < 0) {
        if (elems > 0) *reinterpret_cast<uint16_t*>(o + 2) = static_cast<uint16_t>(h[i] >> 16);
      } else if (e + 1 < elems) {
        *reinterpret_cast<uint32_t*>(o) = h[i];
      } else if (e < elems) {
        *reinterpret_cast<uint16_t*>(o) = static_cast<uint16_t>(h[i]);
      }
    }
  }
  __syncwarp();
}

// The two matrices' scales (NV) as factors of the fp32 sums: first, then second.
// second is 1 and first their product, unless that leaves fp32's normal range
// where a result need not: then first has the significant bits with an
// exponent that keeps the sums' products normal (a sum other than 0 lies
// between 2^-20 and 2^60), and second is a power of two.
struct MatrixScale {
  float first = 1.f, second = 1.f;
  __device__ __forceinline__ static MatrixScale of(float ga, float gb) {
    MatrixScale m;
    m.first = ga * gb;
    const float size = fabsf(m.first);
    if (!(size >= 0x1p-126f && size < __uint_as_float(0x7F800000u)) && isfinite(ga) && isfinite(gb)) {
      int ea, eb;
      const float bits = frexpf(ga, &ea) * frexpf(gb, &eb);  // 0, or from 1/4 to 1
      const int e = min(max(ea + eb, -90), 60);
      m.first = ldexpf(bits, e);
      m.second = ldexpf(1.f, min(ea + eb - e, 127));  // (0 and 2^127: results below and past fp32)
    }
    return m;
  }
  // sums[i] as the bits of a float
  template <int N>
  __device__ __forceinline__ void apply(uint32_t (&sums)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i] = __float_as_uint(first * __uint_as_float(sums[i]));
    if (second != 1.f) {
#pragma unroll
      for (int i = 0; i < N; ++i) sums[i] = __float_as_uint(second * __uint_as_float(sums[i]));
    }
  }
};

template <int FMT>
__device__ __forceinline__ MatrixScale matrix_scale(const Fp4MatmulArgs& a, int e) {
  if constexpr (FMT == kFp4Nv) return MatrixScale::of(__ldg(a.a_tensor_scale), __ldg(a.b_tensor_scale + e));
  return MatrixScale{};
}

// Two floats' bits as a pair of bf16.
__device__ __forceinline__ uint32_t bf16_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// An epilogue warp's part of a tile: 32 rows from row0, COLS columns from
// `first`, from tensor memory at `acc`.  done(): the accumulator is read.
template <int FMT, int COLS, typename F>
__device__ __forceinline__ void store_tile(const Fp4MatmulArgs& a, uint32_t acc, int row0, int first, int e, int vec,
                                           int lane, F&& done) {
  const MatrixScale g = matrix_scale<FMT>(a, e);
  const int rows = a.m - row0;  // the warp's rows (all 32 but in the last tiles)
  const int elem = a.out_f32 ? 4 : 2;
  uint8_t* out = static_cast<uint8_t*>(a.out) + (static_cast<int64_t>(row0) * a.ld_out + first) * elem;
  const int64_t pitch = a.ld_out * elem;
  if (a.out_f32 || !vec) {
    // 128 bytes of each row at a time
    const int step = a.out_f32 ? 32 : 64;
    uint32_t carry = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < COLS && first + c0 < a.n; c0 += step) {
      uint32_t v[32];
      tmem_load32(acc + c0, v);
      const bool last = c0 + step >= COLS || first + c0 + step >= a.n;
      if (a.out_f32) {
        if (last) done();
        g.apply(v);
        if (vec)
          store_rows<4>(out + c0 * 4, pitch, v, rows, a.n - first - c0, lane);
        else
          store_any_rows<4>(out + c0 * 4, pitch, v, rows, a.n - first - c0, carry, c0 == 0, last, lane);
      } else {
        uint32_t u[32];
        tmem_load32(acc + c0 + 32, u);
        if (last) done();
        g.apply(v);
        g.apply(u);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = bf16_pair(v[2 * j], v[2 * j + 1]);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[16 + j] = bf16_pair(u[2 * j], u[2 * j + 1]);
        store_any_rows<2>(out + c0 * 2, pitch, v, rows, a.n - first - c0, carry, c0 == 0, last, lane);
      }
    }
    if (first >= a.n) done();
  } else {
    // all columns as bf16 in registers, the accumulator handed on, then the stores
    uint32_t h[COLS / 2];
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += 32) {
      uint32_t v[32];
      tmem_load32(acc + c0, v);
      g.apply(v);
#pragma unroll
      for (int j = 0; j < 16; ++j) h[c0 / 2 + j] = bf16_pair(v[2 * j], v[2 * j + 1]);
    }
    done();
#pragma unroll
    for (int c = 0; c < COLS; c += 64)
      if (first + c < a.n) store_rows<2>(out + c * 2, pitch, h + c / 2, rows, a.n - first - c, lane);
  }
}

template <int FMT, int BN, bool SWAP>
__global__ void __launch_bounds__((THREADS<SWAP>), 1)
    fp4_matmul_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                      const Fp4MatmulArgs a, const int ksplit, const int vec) {
  using C = Cfg<FMT, BN, SWAP>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = SWAP ? static_cast<int>(cluster_ctarank()) : 0;
  const int worker = SWAP ? static_cast<int>(blockIdx.x) / ksplit : static_cast<int>(blockIdx.x);
  const int workers = SWAP ? static_cast<int>(gridDim.x) / ksplit : static_cast<int>(gridDim.x);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1 + a.test_stall);
    mbar_init(tempty, EPI_WARPS<SWAP>);
    fence_barrier_init();
    prefetch_tensormap(&tm_p);
    prefetch_tensormap(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Tiles<BN, SWAP> tiles(a);
  const int stages = (a.k + BK - 1) / BK;
  const int kb0 = SWAP ? rank * stages / ksplit : 0;
  const int kb1 = SWAP ? (rank + 1) * stages / ksplit : stages;
  const int words = (a.k / kFp4Block<FMT> + 3) / 4;  // scale tiles per row tile

  if (warp == 0) {
    if (lane == 0) {
      const uint8_t* ps = SWAP ? a.b_scales : a.a_scales;
      const uint8_t* qs = SWAP ? a.a_scales : a.b_scales;
      const int64_t q_tiles = ((SWAP ? a.m : a.n) + 127) / 128;
      int64_t it = 0;
      bool ok = true;
      for (int i = worker; ok && i < tiles.total; i += workers) {
        const Tile t = tiles.at(i, a);
        const int q_row = t.q0 + (SWAP ? 0 : t.e * a.n);
        const uint8_t* p_sf = ps + static_cast<int64_t>(t.p0 / 128) * words * kScaleTileBytes;
        const uint8_t* q_sf = qs + (t.e * q_tiles + t.q0 / 128) * words * kScaleTileBytes;
        const int nq = min(C::QT, static_cast<int>(q_tiles - t.q0 / 128));
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = static_cast<int>(it % STAGES);
          if (!mbar_wait(&empty[s], static_cast<uint32_t>(((it / STAGES) & 1) ^ 1), a.wait_limit_ns)) {
            timed_out(a);
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          uint8_t* sf = st + P_BYTES + C::Q_BYTES;
          const int nw = min(C::W, words - kb * C::W);
          const uint32_t sf_bytes = static_cast<uint32_t>(nw * kScaleTileBytes);
          mbar_arrive_expect_tx(&full[s], P_BYTES + C::Q_BYTES + (1 + nq) * sf_bytes);
          tma_load_2d(st, &tm_p, &full[s], kb * ROW_BYTES, t.p0);
          tma_load_2d(st + P_BYTES, &tm_q, &full[s], kb * ROW_BYTES, q_row);
          bulk_load(sf, p_sf + static_cast<int64_t>(kb) * C::SF_BYTES, sf_bytes, &full[s]);
          for (int j = 0; j < nq; ++j)
            bulk_load(sf + (1 + j) * C::SF_BYTES,
                      q_sf + (static_cast<int64_t>(j) * words + kb * C::W) * kScaleTileBytes, sf_bytes, &full[s]);
        }
      }
      // no copy may still be in flight into shared memory at exit
      for (int64_t j = (it > STAGES ? it - STAGES : 0); j < it; ++j)
        if (!mbar_wait(&full[j % STAGES], static_cast<uint32_t>((j / STAGES) & 1), a.wait_limit_ns))
          timed_out(a);
    }
  } else if (warp == 1) {
    Issuer<STAGES> is(full, a);
    const uint64_t desc0 = sw128_desc(smem_u32(smem)), sdesc0 = scale_desc(smem_u32(smem + P_BYTES + C::Q_BYTES));
    uint32_t tphase = 0;
    for (int i = worker; is.ok && i < tiles.total; i += workers, tphase ^= 1u) {
      if (!is.wait(tempty, tphase ^ 1u)) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!is.wait_stage()) break;
        const uint64_t pd = desc0 + is.s * (C::STAGE / 16), qd = pd + P_BYTES / 16;
        const uint64_t sd = sdesc0 + is.s * (C::STAGE / 16);
        const uint32_t sfp = tmem + C::SF0 + static_cast<uint32_t>(is.s) * C::SF_COLS;
        const uint32_t sfq = sfp + 4 * C::W;
        if (is.leader) {
          // words past the array are an earlier stage's, which no MMA uses
#pragma unroll
          for (int w = 0; w < C::W; ++w) {
            tc_copy_scales(sfp + 4 * w, sd + w * (kScaleTileBytes / 16));
#pragma unroll
            for (int j = 0; j < C::QT; ++j)
              tc_copy_scales(sfq + 4 * (w * C::QT + j), sd + ((1 + j) * C::SF_BYTES + w * kScaleTileBytes) / 16);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j > 0 && kb * BK + j * 64 >= a.k) break;
            const uint32_t acc = (kb != kb0 || j != 0) ? 1u : 0u;
            if constexpr (FMT == kFp4Mx)
              tc_mma_mx4(tmem, pd + 2 * j, qd + 2 * j, idesc_fp4(BP, BN, true, (j & 1) * 2), sfp + 4 * (j / 2),
                         sfq + 4 * C::QT * (j / 2), acc);
            else
              tc_mma_nv4(tmem, pd + 2 * j, qd + 2 * j, idesc_fp4(BP, BN, false, 0), sfp + 4 * j, sfq + 4 * C::QT * j,
                         acc);
          }
          tc_commit(&empty[is.s]);
        }
        is.next();
      }
      if (is.ok && is.leader) tc_commit(tfull);
      __syncwarp();
    }
  } else if (warp >= EPI_WARP0) {
    const int q = warp & 3;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    constexpr int COLS = SWAP ? BN : BN / (EPI_WARPS<SWAP> / 4);  // of this warp
    const int col0 = SWAP ? 0 : (warp - EPI_WARP0) / 4 * COLS;
    uint32_t tphase = 0;
    for (int i = worker; i < tiles.total; i += workers, tphase ^= 1u) {
      const Tile t = tiles.at(i, a);
      if (!mbar_wait(tfull, tphase, a.wait_limit_ns)) {
        timed_out(a);
        break;
      }
      tc_fence_after();
      if constexpr (SWAP) {
        // partial sums into the ring (its loads and MMAs are done): [token][weight row]
        float* part = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int c0 = 0; c0 < BN; c0 += 16) {
          uint32_t v[16];
          tmem_load16(lanes + c0, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c0 + j) * BP + q * 32 + lane] = __uint_as_float(v[j]);
        }
      } else {
        store_tile<FMT, COLS>(a, lanes + col0, t.p0 + q * 32, t.q0 + col0, t.e, vec, lane, [&]() { release(tempty, lane); });
      }
    }
  }

  if constexpr (SWAP) {
    __syncwarp();
    cluster_sync();  // every rank's partial sums are in its shared memory
    // a token per warp, four output columns per lane; the ranks share the tokens
    const int col = worker * BP + lane * 4;
    const MatrixScale g = matrix_scale<FMT>(a, 0);
    for (int t = rank + ksplit * warp; t < a.m; t += ksplit * (THREADS<SWAP> / 32)) {
      const uint32_t at = smem_u32(reinterpret_cast<float*>(smem) + t * BP + lane * 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int j = 0; j < ksplit; ++j) {
        const float4 x = ld_shared_cluster_f32x4(mapa_shared(at, j));
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
      }
      uint32_t f[4] = {__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)};
      g.apply(f);
      const int64_t o = static_cast<int64_t>(t) * a.ld_out + col;
      if (a.out_f32) {
        uint32_t* out = static_cast<uint32_t*>(a.out) + o;
        if (vec && col + 4 <= a.n) {
          *reinterpret_cast<uint4*>(out) = make_uint4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (col + u < a.n) out[u] = f[u];
        }
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + o;
        const uint2 h = make_uint2(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]));
        if (vec && col + 4 <= a.n) {
          *reinterpret_cast<uint2*>(out) = h;
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (col + u < a.n) out[u] = static_cast<uint16_t>((u < 2 ? h.x : h.y) >> (16 * (u & 1)));
        }
      }
    }
    __syncwarp();
    cluster_sync();  // no rank leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// ------------------------------------------------------------------- CTA pairs
// A cluster of two CTAs takes 256 rows of A (128 each) against 256 rows of B
// with the 2-SM MMA.  Each stages half of B's rows and the tensor cores read
// both halves: 38 KB a stage (NV) against 54.  What bounds it is that feed: a
// stage takes 306 ns, 124 bytes/ns and SM (64 a cycle), its four MMAs about
// 190 (from issuing each twice).  The accumulator is single, scales having the rest of tensor memory;
// handing it over costs 0.7 us a tile, and the output's stores share the feed
// (4096 x 14336 x 4096 without them: 68 us instead of 82).
//
// Barriers: both CTAs' copies complete the even CTA's `full`; the MMA's
// commits arrive on `empty` and `tfull` of both; the epilogue warps of both
// arrive on the even CTA's `tempty`.
template <int FMT>
struct PairCfg {
  static constexpr int STAGES = 5, BN = 256, EPI = 8, THREADS = (EPI_WARP0 + EPI) * 32;
  static constexpr int W = BK / (4 * kFp4Block<FMT>);
  static constexpr int Q_BYTES = BN / 2 * ROW_BYTES;
  static constexpr int SF_BYTES = W * kScaleTileBytes;
  static constexpr int STAGE = P_BYTES + Q_BYTES + 3 * SF_BYTES;
  static constexpr int SF_COLS = W * 4 * 3;  // per stage: own rows of A, two row tiles of B
  static constexpr int TMEM = 512;
  static constexpr int BYTES = STAGES * STAGE + 1024 + 256;
  static_assert(STAGE % 1024 == 0 && BYTES <= 232448 && BN + STAGES * SF_COLS <= TMEM, "layout");
};

template <int FMT>
__global__ void __launch_bounds__(PairCfg<FMT>::THREADS, 1)
    fp4_matmul_pair_kernel(const __grid_constant__ CUtensorMap tm_p, const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_ps, const __grid_constant__ CUtensorMap tm_qs,
                           const Fp4MatmulArgs a, const int vec) {
  using C = PairCfg<FMT>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool even = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1 + a.test_stall);
    mbar_init(tempty, 2 * C::EPI);
    fence_barrier_init();
    prefetch_tensormap(&tm_p);
    prefetch_tensormap(&tm_q);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::TMEM);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int pt = (a.m + 2 * BP - 1) / (2 * BP), total = pt * ((a.n + C::BN - 1) / C::BN);
  const int first = blockIdx.x / 2, step = gridDim.x / 2;
  const int stages = (a.k + BK - 1) / BK;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full_even = mapa_shared(smem_u32(full), 0);
      int64_t it = 0;
      bool ok = true;
      for (int i = first; ok && i < total; i += step) {
        const int p0 = (i % pt * 2 + rank) * BP, q0 = i / pt * C::BN;
        for (int kb = 0; kb < stages; ++kb, ++it) {
          const int s = static_cast<int>(it % STAGES);
          if (!mbar_wait(&empty[s], static_cast<uint32_t>(((it / STAGES) & 1) ^ 1), a.wait_limit_ns)) {
            timed_out(a);
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::STAGE;
          uint8_t* sf = st + P_BYTES + C::Q_BYTES;
          if (even) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE);
          const uint32_t bar = full_even + static_cast<uint32_t>(s * 8);
          tma_load_2d_pair(st, &tm_p, bar, kb * ROW_BYTES, p0);
          tma_load_2d_pair(st + P_BYTES, &tm_q, bar, kb * ROW_BYTES, q0 + rank * BP);
          tma_load_2d_pair(sf, &tm_ps, bar, kb * (C::SF_BYTES / 8), p0 / BP);
          tma_load_2d_pair(sf + C::SF_BYTES, &tm_qs, bar, kb * (C::SF_BYTES / 8), q0 / BP);
        }
      }
      // no copy may still be in flight into shared memory at exit (the even
      // CTA's `full` counts both CTAs' copies)
      for (int64_t j = (it > STAGES ? it - STAGES : 0); even && j < it; ++j)
        if (!mbar_wait(&full[j % STAGES], static_cast<uint32_t>((j / STAGES) & 1), a.wait_limit_ns))
          timed_out(a);
    }
  } else if (warp == 1 && even) {
    Issuer<STAGES> is(full, a);
    const uint64_t desc0 = sw128_desc(smem_u32(smem)), sdesc0 = scale_desc(smem_u32(smem + P_BYTES + C::Q_BYTES));
    uint32_t tphase = 0;
    for (int i = first; is.ok && i < total; i += step, tphase ^= 1u) {
      if (!is.wait(tempty, tphase ^ 1u)) break;
      tc_fence_after();
      for (int kb = 0; kb < stages; ++kb) {
        if (!is.wait_stage()) break;
        const uint64_t pd = desc0 + is.s * (C::STAGE / 16), qd = pd + P_BYTES / 16;
        const uint64_t sd = sdesc0 + is.s * (C::STAGE / 16);
        const uint32_t sfp = tmem + C::BN + static_cast<uint32_t>(is.s) * C::SF_COLS;
        const uint32_t sfq = sfp + 4 * C::W;
        if (is.leader) {
#pragma unroll
          for (int w = 0; w < C::W; ++w) {
            tc_copy_scales_pair(sfp + 4 * w, sd + w * (kScaleTileBytes / 16));
#pragma unroll
            for (int j = 0; j < 2; ++j)
              tc_copy_scales_pair(sfq + 4 * (2 * w + j), sd + ((1 + j) * C::SF_BYTES + w * kScaleTileBytes) / 16);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j > 0 && kb * BK + j * 64 >= a.k) break;
            const uint32_t acc = (kb | j) != 0 ? 1u : 0u;
            if constexpr (FMT == kFp4Mx)
              tc_mma_mx4_pair(tmem, pd + 2 * j, qd + 2 * j, idesc_fp4(2 * BP, C::BN, true, (j & 1) * 2),
                              sfp + 4 * (j / 2), sfq + 8 * (j / 2), acc);
            else
              tc_mma_nv4_pair(tmem, pd + 2 * j, qd + 2 * j, idesc_fp4(2 * BP, C::BN, false, 0), sfp + 4 * j,
                              sfq + 8 * j, acc);
          }
          tc_commit_pair_multicast(&empty[is.s], 3);
        }
        is.next();
      }
      if (is.ok && is.leader) tc_commit_pair_multicast(tfull, 3);
      __syncwarp();
    }
  } else if (warp >= EPI_WARP0) {
    const int q = warp & 3, col0 = (warp - EPI_WARP0) / 4 * 128;
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col0);
    const uint32_t tempty_even = mapa_shared(smem_u32(tempty), 0);
    uint32_t tphase = 0;
    for (int i = first; i < total; i += step, tphase ^= 1u) {
      if (!mbar_wait(tfull, tphase, a.wait_limit_ns)) {
        timed_out(a);
        break;
      }
      tc_fence_after();
      store_tile<FMT, 128>(a, acc, (i % pt * 2 + rank) * BP + q * 32, i / pt * C::BN + col0, 0, vec, lane, [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(tempty_even);
      });
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM);
  }
}

bool map_codes(CUtensorMap* m, const uint8_t* codes, int64_t rows, int k, int box) {
  return make_tmap(m, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, static_cast<uint64_t>(k / 2),
                   static_cast<uint64_t>(rows), ROW_BYTES, static_cast<uint32_t>(box));
}

// Scale tiles as 8-byte elements, rows of one row tile each; a box is a stage's
// words of `box` row tiles.
template <int FMT>
bool map_scales(CUtensorMap* m, const uint8_t* scales, int64_t rows, int k, int box) {
  const uint64_t words = static_cast<uint64_t>((k / kFp4Block<FMT> + 3) / 4);
  return make_tmap(m, scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, words * (kScaleTileBytes / 8),
                   static_cast<uint64_t>((rows + 127) / 128), BK / (4 * kFp4Block<FMT>) * (kScaleTileBytes / 8),
                   static_cast<uint32_t>(box), CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Whether the output's rows start on 16 bytes.
int rows_on_16(const Fp4MatmulArgs& a) {
  return (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && a.ld_out * (a.out_f32 ? 4 : 2) % 16 == 0 ? 1 : 0;
}

// Allows a kernel its shared memory, once per device (bits of `done`).
template <typename K>
cudaError_t allow_shared(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// A launch in clusters of `cluster` CTAs (0: none).  It follows arbitrary work
// of the caller, so it does not begin before that has ended: a kernel that
// let it begin and allocated tensor memory only then could wait for it.
template <typename K, typename... Args>
cudaError_t launch_cluster(K kernel, unsigned grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int FMT, int BN, bool SWAP>
cudaError_t launch(const Fp4MatmulArgs& a, int num_sms, cudaStream_t s) {
  using C = Cfg<FMT, BN, SWAP>;
  auto kernel = fp4_matmul_kernel<FMT, BN, SWAP>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, C::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap tp, tq;
  const int64_t b_rows = static_cast<int64_t>(a.n) * a.n_groups;
  if (!map_codes(&tp, SWAP ? a.b_codes : a.a_codes, SWAP ? b_rows : a.m, a.k, BP) ||
      !map_codes(&tq, SWAP ? a.a_codes : a.b_codes, SWAP ? a.m : b_rows, a.k, BN))
    return cudaErrorInvalidValue;
  const int vec = rows_on_16(a);
  int64_t grid;
  int ksplit = 1;
  if (SWAP) {
    const int tiles = (a.n + BP - 1) / BP, stages = (a.k + BK - 1) / BK;
    // CTAs enough for every SM, or for half of them twice where they keep 4
    // stages each (112 tiles of 16 stages: 9.7 us unsplit, 9.3 in two, 12.4 in
    // four; 32 tiles of 56 stages: 23.8, 15.3, 11.5 in four and 12.3 in eight)
    while (ksplit < 8) {
      const int64_t ctas = 2ll * ksplit * tiles;
      const int each = stages / (2 * ksplit);
      if (each < 2 || ctas > (each >= 4 ? num_sms + num_sms / 2 : num_sms)) break;
      ksplit *= 2;
    }
    grid = static_cast<int64_t>(tiles) * ksplit;
  } else {
    const int64_t tiles = static_cast<int64_t>((a.m + BP - 1) / BP) * ((a.n + BN - 1) / BN);
    grid = tiles < num_sms ? tiles : num_sms;
  }
  return launch_cluster(kernel, static_cast<unsigned>(grid), THREADS<SWAP>, C::BYTES, SWAP ? ksplit : 0, s, tp, tq,
                        a, ksplit, vec);
}

template <int FMT>
cudaError_t launch_pair(const Fp4MatmulArgs& a, int num_sms, cudaStream_t s) {
  using C = PairCfg<FMT>;
  auto kernel = fp4_matmul_pair_kernel<FMT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_shared(kernel, C::BYTES, done);
  if (e != cudaSuccess) return e;
  CUtensorMap tp, tq, tps, tqs;
  if (!map_codes(&tp, a.a_codes, a.m, a.k, BP) || !map_codes(&tq, a.b_codes, a.n, a.k, BP) ||
      !map_scales<FMT>(&tps, a.a_scales, a.m, a.k, 1) || !map_scales<FMT>(&tqs, a.b_scales, a.n, a.k, 2))
    return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>((a.m + 2 * BP - 1) / (2 * BP)) * ((a.n + C::BN - 1) / C::BN);
  const int64_t pairs = num_sms / 2;
  return launch_cluster(kernel, static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)), C::THREADS, C::BYTES, 2, s, tp,
                        tq, tps, tqs, a, rows_on_16(a));
}

template <int FMT>
cudaError_t launch_format(const Fp4MatmulArgs& a, int num_sms, cudaStream_t s) {
  if (a.tile_offsets == nullptr && a.m <= 128) {
    if (a.m <= 16) return launch<FMT, 16, true>(a, num_sms, s);
    if (a.m <= 32) return launch<FMT, 32, true>(a, num_sms, s);
    if (a.m <= 64) return launch<FMT, 64, true>(a, num_sms, s);
    return launch<FMT, 128, true>(a, num_sms, s);
  }
  // 128-column tiles where one for each SM is enough (512 x 4096 x 4096, 128 of
  // them: 9.2 us against 10.8; 768 x 4096 x 4096, 192: 13.9 against 11.1);
  // beyond, pairs for dense products of more than a round of wide tiles that
  // are long enough for their set-up (nv, k = 4096: 1024 x 14336, 25.9 us
  // against 27.8, 4096 x 14336, 82 against 97; k = 512: 2048 x 4096, 8.9
  // against 8.0, 3000 x 14336, 27.4 against 26.6).  Experts keep single CTAs:
  // of an odd number of row tiles a pair wastes half (2.8 row tiles each: 37.9
  // us against 31.8; 10.4: 74.5 against 77.8).
  const int64_t row_tiles = (a.m + BP - 1) / BP;
  if (row_tiles * ((a.n + 127) / 128) <= num_sms) return launch<FMT, 128, false>(a, num_sms, s);
  if (a.tile_offsets == nullptr && a.k >= 1024 && row_tiles * ((a.n + 255) / 256) > num_sms)
    return launch_pair<FMT>(a, num_sms, s);
  return launch<FMT, 256, false>(a, num_sms, s);
}

}  // namespace

cudaError_t take_fp4_error(int* code) {
  const int none = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_error, sizeof(int));
  return e == cudaSuccess && *code != 0 ? cudaMemcpyToSymbol(g_error, &none, sizeof(int)) : e;
}

cudaError_t launch_fp4_matmul(const Fp4MatmulArgs& a, int num_sms, cudaStream_t s) {
  return a.format == kFp4Mx ? launch_format<kFp4Mx>(a, num_sms, s) : launch_format<kFp4Nv>(a, num_sms, s);
}

}  // namespace cbmoe
