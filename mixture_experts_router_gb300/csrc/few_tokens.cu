// The whole layer for a few tokens (1 to 16) in one cooperative launch, on
// the weights of an ordinary handle (bf16, int8, int4 or fp8 experts):
//
//   1. logits     l[t][e] = x[t] . Wr[e] + b[e]: one expert at a time per
//                 block, the block's warps splitting d;
//      -- grid barrier (none with few experts and tokens: every block then
//         takes all the logits) --
//   2. gate       every block takes the top-k of all n tokens from the n x E
//                 logits (warp_gate) and lists the experts that any token chose;
//   3. gate/up    H[t k + s][j] = bf16( SiLU(g) * u ), g and u the dot products
//                 of x[t] with feature j's gate and up rows of expert ids[t][s];
//      -- grid barrier --
//   4. down and combine   out[t][c] = sum_s w[t][s] (H[t k + s] . Wd[ids[t][s]][c]).
//
// What bounds it: the chosen experts' weights, read once from HBM (of an expert
// in two parts, twice: see launch_format); with at most 16 tokens an expert's
// 128-row tiles of the large kernels would be nearly all padding.  So a tile
// here is at most 32 weight rows (in step 3, 16 features' gate and up rows; in
// step 4, 32 output columns), streamed through a ring of stages of 512 (int4
// with 16 tokens: 256) bytes per row, with the same stretch of the chosen
// tokens' activations beside them.
//
// A block is two halves, each with a ring, two feeding warps and 8 users:
//
//   weights (1 thread)  one TMA copy per stage.  The tensor maps split a row
//               into 128-byte chunks as a dimension of its own, so that one
//               copy brings that much of every row of the tile; there is a
//               map for each height.  A copy costs its SM about 55 ns and then
//               2.2 ns per 128 bytes, so several small ones per stage would
//               bound the kernel (a bulk copy per row held it at 2 TB/s).  It
//               runs ahead across tiles, experts and the second barrier: step
//               4's weights do not wait for H.
//   tokens (1 warp)     by cp.async into the stage, in the weights' swizzle.
//   users (8 warps)     a warp owns an eighth of a stage's stretch, reads
//               fragments with wide loads, widens quantised codes to bf16
//               exactly in registers and issues mma.sync m16n8k16 (A: weight
//               rows, B: the expert's own tokens, in their order).  A dot
//               product does not depend on the order of its terms, so a
//               thread's k-slots are consecutive elements.
//
// The halves take a block's step-3 tiles in turn, so that one joins its
// warps' sums while the other streams; in step 4 they take the experts in
// turn (or, of few experts, half of k each).
//
// The balance: the parts' features (step 3) and the output columns
// (step 4) are cut into one contiguous share per block, in steps of 4 (the
// rows of the smallest copy).
//
// Measured on the GPU alone, d x f x experts, bf16 if not said: 1 token of 2 of
// 8 of 4096 x 14336, 112 us and 8 tokens 379 (6.3 and 6.7 TB/s); 3 tokens of 4
// of 128 of 2048 x 768, 33 us (half of it start and barriers); 16 tokens of 6
// of 64 of 4096 x 1536, int8, 196 us (4.9 TB/s: widening) and int4 162; 1 token
// of 2 of 8 of 256 x 512, 12 us (launch and phases).
//
// Every sum is fp32 in a fixed order (mma accumulators, experts in ascending
// order, then the warps in order), so results do not change from run to
// run.  H is rounded to bf16 as everywhere in the layer: it is the MMA's
// operand.  Rows past the tile's end and columns past the expert's tokens
// read the last one again, and their sums are dropped.
#include <cuda_bf16.h>

#include "grid_barrier.cuh"
#include "int8_bf16.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "router_common.cuh"
#include "swiglu.cuh"

namespace cbmoe {
namespace {

constexpr int kUsers = 512;             // threads that use the ring
constexpr int kUserWarps = kUsers / 32;
constexpr int kHalves = 2;
constexpr int kWeightWarp = kUserWarps;             // one per half
constexpr int kTokenWarp = kWeightWarp + kHalves;
constexpr int kThreads = (kTokenWarp + kHalves) * 32;
constexpr int kRows = 32;               // weight rows of a tile: two m16 fragments
constexpr int kAlong = 8;               // warps along a row's stretch: a half's users
constexpr int kFewParts = 8;            // parts below which the halves split k in step 4
constexpr int kShareStep = kFewRowStep; // shares and tiles are multiples of this many rows
constexpr int kMaxTokens = kFewTokens;
constexpr int kMaxExperts = 256;
constexpr int kMaxK = 16;
constexpr int kLogitTokens = 4;
constexpr int kMaxParts = kMaxTokens * kMaxK;
constexpr uint32_t kUserBar = 1;        // named barriers: all users, and each half's
constexpr uint32_t kHalfBar = 2;
constexpr int kSmemLimit = 232448;

// Weight formats of the kernel: the quantised ones as in WeightFormat.
constexpr int kBf16 = 3;
template <int WF>
constexpr int kElems = WF == kBf16 ? 8 : WF == kWInt4 ? 32 : 16;  // elements per 16 bytes

// NT: n-tiles of 8 tokens per part; MT: 8 or 16, at least the tokens of the call.
template <int NT, int MT>
struct Shared {
  union {
    float red[kUserWarps][kRows][MT];     // partial sums: [warp][row][token]
    float logit[kMaxTokens * kMaxExperts];
    float part[kUserWarps][kMaxTokens];   // the logits' partial sums
  };
  float w[kMaxTokens * kMaxK];            // gate weight of each (token, slot)
  uint32_t mask[kMaxExperts];             // tokens of each expert
  uint8_t slot[kMaxExperts][kMaxTokens];  // the slot at which a token chose it
  // parts: an active expert and at most NT x 8 of its tokens (n k at most)
  int16_t act[kMaxParts];                 // the expert, ascending
  uint8_t tok[kMaxParts][NT * 8];
  uint8_t count[kMaxParts];
  int16_t row0[kMaxParts];                // the part's first row of H
  int n_act;
  int warp_parts[kMaxExperts / 32];
  int ok;
};

// Bytes of a row per stage; int4's with 16 tokens, four times as many bytes
// each beside them, are fewer.  (With 8 tokens 256 bytes are slower too: 16
// tokens over 64 experts 170 us against 162.)
template <int WF, int NT>
constexpr int kSeg = WF == kWInt4 && NT == 2 ? 256 : 512;

template <int WF, int NT, int MT>
struct Geo {
  static constexpr int kSeg = cbmoe::kSeg<WF, NT>;
  static constexpr int kRowLines = kSeg / 128;
  static constexpr int kWeightBytes = kRows * kSeg;
  static constexpr int kStep = kSeg / kAlong;             // bytes of a row per warp
  static constexpr int kStepElems = kStep / 64 ? kElems<WF> : kElems<WF> / 2;  // elements per thread and row
  static constexpr int kTokBytes = kSeg / 16 * kElems<WF> * 2;  // a token's stretch in a stage
  static constexpr int kTokLines = kTokBytes / 128;
  static constexpr int kStage = kWeightBytes + NT * 8 * kTokBytes;
  static constexpr int kShared = (static_cast<int>(sizeof(Shared<NT, MT>)) + 256 + 1023) / 1024 * 1024;
  static constexpr int kFit = (kSmemLimit - kShared - 1024) / kStage;
  static constexpr int kStages = (kFit < 12 ? kFit : 12) / kHalves;  // of each half
  static constexpr int kBytes = 1024 + kShared + kHalves * kStages * kStage;
  static_assert(kStages >= 2 && 16 * kHalves * kStages <= 256 && kStage % 1024 == 0, "ring");
};

// Byte of 16-byte unit `unit` of 128-byte line `line` of a swizzled area.
__device__ __forceinline__ int swizzled(int line, int unit) { return line * 128 + ((unit ^ (line & 7)) << 4); }
// The same byte of row `row`, rows being LINES (a power of two) lines: `first`
// is row 0's.
template <int LINES>
__device__ __forceinline__ int in_row(int first, int row) {
  return row * (LINES * 128) + (first ^ (((row * LINES) & 7) << 4));
}

// Elements 8 i .. 8 i + 7 of a thread's 16 bytes of a weight row as four bf16
// pairs, in the order of pair_up: memory order, but for int4 and fp8 the
// pairs that masks take out of a word without moving bytes.
//   int4: elements m and m + 4.  A nibble n in a half word under 0x4300 is
// 128 + n, minus 128 + z exactly n - z (11 instructions for 8 elements; in
// memory order, by bytes, 15).
//   fp8: elements m and m + 2.  Sign and magnitude of an e4m3 byte at bits 15
// and 10-4 are its value times 2^-120 (as in fp8x4_to_bf16x4).
template <int WF>
__device__ __forceinline__ void widen8(const uint4& v, int i, uint32_t zz, uint32_t (&o)[4]) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  if constexpr (WF == kBf16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = in[j];
  } else if constexpr (WF == kWInt4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t n;
      asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(n) : "r"(in[i] >> (4 * j)));
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(n), "r"(zz));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t w = in[2 * i + j];
      if constexpr (WF == kWFp8) {
        uint32_t a, b;
        asm("lop3.b32 %0, %1, 0x80008000, %2, 0xEA;" : "=r"(a) : "r"(w << 8), "r"((w << 4) & 0x07F007F0u));
        asm("lop3.b32 %0, %1, 0x80008000, %2, 0xEA;" : "=r"(b) : "r"(w), "r"((w >> 4) & 0x07F007F0u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * j]) : "r"(a), "r"(0x7B807B80u));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[2 * j + 1]) : "r"(b), "r"(0x7B807B80u));
      } else {
        int8x4_to_bf16x4_fma(w, o[2 * j], o[2 * j + 1]);
      }
    }
  }
}
// Eight elements of a token in the same pairs.
template <int WF>
__device__ __forceinline__ uint4 pair_up(const uint4& t) {
  if constexpr (WF == kWInt4)
    return make_uint4(__byte_perm(t.x, t.z, 0x5410), __byte_perm(t.x, t.z, 0x7632), __byte_perm(t.y, t.w, 0x5410),
                      __byte_perm(t.y, t.w, 0x7632));
  else if constexpr (WF == kWFp8)
    return make_uint4(__byte_perm(t.x, t.y, 0x5410), __byte_perm(t.x, t.y, 0x7632), __byte_perm(t.z, t.w, 0x5410),
                      __byte_perm(t.z, t.w, 0x7632));
  else
    return t;
}

// A stretch of the ring's stages, one after the other.
template <int STAGES>
struct RingPos {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1u;
    }
  }
};

template <int WF, int NT, int MT>
struct Block {
  using G = Geo<WF, NT, MT>;
  static constexpr int kSeg = G::kSeg;
  const FewArgs& p;
  const FewMaps& maps;
  Shared<NT, MT>& s;
  uint64_t* full;
  uint64_t* empty;
  uint8_t* ring;
  RingPos<G::kStages> pos;  // the producer's, or a user's, place in the ring
  bool ok = true;           // no wait of this thread has run out
  int opened = 0;           // the weight thread's last stages, at most the whole ring
  const int warp, lane, half;
  int first_w;
  int first_tok[G::kStepElems / 8];

  __device__ __forceinline__ Block(const FewArgs& p_, const FewMaps& maps_, uint8_t* smem)
      : p(p_),
        maps(maps_),
        s(*reinterpret_cast<Shared<NT, MT>*>(smem)),
        full(reinterpret_cast<uint64_t*>(smem + G::kShared - 256) + half_of_warp() * 2 * G::kStages),
        empty(full + G::kStages),
        ring(smem + G::kShared + half_of_warp() * G::kStages * G::kStage),
        warp(threadIdx.x / 32),
        lane(threadIdx.x % 32),
        half(half_of_warp()) {
    const int along = warp % kAlong, q = lane & 3;
    const int byte = along * G::kStep + q * (G::kStep / 4);  // of a row's stretch
    first_w = swizzled(byte / 128, byte % 128 / 16) + byte % 16;
#pragma unroll
    for (int i = 0; i < G::kStepElems / 8; ++i) {
      const int unit = (along * 4 + q) * (G::kStepElems / 8) + i;
      first_tok[i] = swizzled(unit / 8, unit % 8);
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < kHalves * G::kStages; ++i) {
        uint64_t* bars = full + i / G::kStages * 2 * G::kStages + i % G::kStages;
        mbar_init(bars, 1 + 32);  // full: the weights' announcement, the token warp's lanes
        mbar_init(bars + G::kStages, kAlong);
      }
      fence_barrier_init();
    }
  }
  __device__ __forceinline__ static int half_of_warp() {
    const int warp = threadIdx.x / 32;
    return warp < kUserWarps ? warp / kAlong : (warp - kUserWarps) % kHalves;
  }
  __device__ __forceinline__ bool user() const { return warp < kUserWarps; }

  // A wait that ran out is recorded once; the thread then runs through without
  // waiting (the results are garbage), so that no barrier is left short, and
  // a producer copies nothing more.
  __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_wait(bar, parity, p.wait_limit_ns)) {
      set_error(p.err, kErrTimeout);
      ok = false;
    }
  }

  // ------------------------------------------------------------- 1. logits
  // Four tokens at a time: their loads go out together.
  // sum[i] += x[t0 + i] . Wr[e] over 8 elements from c, for the tokens there are
  __device__ __forceinline__ void add_products(int e, int t0, int c, float (&sum)[kLogitTokens]) const {
    const uint4 wv = __ldg(reinterpret_cast<const uint4*>(p.wr + static_cast<int64_t>(e) * p.d + c));
    uint4 xv[kLogitTokens];
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i)
      xv[i] = __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(min(t0 + i, p.n - 1)) * p.d + c));
    const uint32_t wu[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
      const uint32_t xu[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[i] = fmaf(__uint_as_float(xu[j] << 16), __uint_as_float(wu[j] << 16), sum[i]);
        sum[i] = fmaf(__uint_as_float(xu[j] & 0xFFFF0000u), __uint_as_float(wu[j] & 0xFFFF0000u), sum[i]);
      }
    }
  }
  __device__ __forceinline__ void put_logits(int t0, float (&sum)[kLogitTokens]) {
#pragma unroll
    for (int i = 0; i < kLogitTokens; ++i) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      if (lane == 0) s.part[warp][(t0 + i) % kMaxTokens] = sum[i];
    }
  }
  // Few experts, tokens and elements: every block takes all the logits itself,
  // which is sooner than a barrier; a warp has one expert's share of d.  (Of 8
  // experts x d 256: 2.2 us against 3.3; x d 4096: 5.5 against 3.1, all blocks
  // fetching the same rows.)
  __device__ __forceinline__ static bool logits_here(const FewArgs& p) {
    return p.ids == nullptr && p.E <= kUserWarps && p.n * p.E <= 32 && p.E * p.d <= 8192;
  }
  __device__ __forceinline__ void own_logits() {
    const int per = kUserWarps / p.E, e = warp / per, part = warp % per;  // warps of an expert
    if (user() && e < p.E) {
      for (int t0 = 0; t0 < p.n; t0 += kLogitTokens) {
        float sum[kLogitTokens] = {};
        for (int c = (part * 32 + lane) * 8; c < p.d; c += per * 256) add_products(e, t0, c, sum);
        put_logits(t0, sum);
      }
    }
    __syncthreads();
    float v = 0.f;
    const int i = threadIdx.x, te = i % p.E, t = i / p.E;
    if (i < p.n * p.E) {
      for (int w = 0; w < per; ++w) v += s.part[te * per + w][t];
      v += p.bias != nullptr ? p.bias[te] : 0.f;
    }
    __syncthreads();
    if (i < p.n * p.E) s.logit[i] = v;
  }
  // Otherwise an expert and up to four tokens per block, its warps splitting d.
  __device__ __forceinline__ void logits() {
    const int items = p.E * ((p.n + kLogitTokens - 1) / kLogitTokens);
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      const int e = item % p.E, t0 = item / p.E * kLogitTokens;
      if (user()) {
        float sum[kLogitTokens] = {};
        for (int c = threadIdx.x * 8; c < p.d; c += kUsers * 8) add_products(e, t0, c, sum);
        put_logits(t0, sum);
      }
      __syncthreads();
      const int t = t0 + threadIdx.x;
      if (threadIdx.x < kLogitTokens && t < p.n) {
        float v = 0.f;
        for (int i = 0; i < kUserWarps; ++i) v += s.part[i][t];
        p.logits[t * p.E + e] = v + (p.bias != nullptr ? p.bias[e] : 0.f);
      }
      __syncthreads();
    }
  }

  // --------------------------------------------------------------- 2. gate
  __device__ __forceinline__ void gate() {
    for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) s.mask[e] = 0u;
    if (p.ids == nullptr && !logits_here(p))
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
    } else if (threadIdx.x < p.n) {  // given experts
      const int t = threadIdx.x;
      const uint32_t bit = 1u << t;
      const int32_t* ids = p.ids + t * p.k;
      int good = 0;  // slots in order that are in range and new
      for (; good < p.k; ++good) {
        const int id = ids[good];
        if (id < 0 || id >= p.E || (atomicOr(&s.mask[id], bit) & bit) != 0u) break;
        s.slot[id][t] = static_cast<uint8_t>(good);
        s.w[t * p.k + good] = p.w != nullptr ? p.w[t * p.k + good] : 1.f;
      }
      if (good < p.k) {  // experts 0 .. k - 1 with NaN weights instead
        if (blockIdx.x == 0) set_error(p.err, kErrDevice);
        for (int i = 0; i < good; ++i) atomicAnd(&s.mask[ids[i]], ~bit);
        for (int i = 0; i < p.k; ++i) {
          s.slot[i][t] = static_cast<uint8_t>(i);
          s.w[t * p.k + i] = __int_as_float(0x7FC00000);
          atomicOr(&s.mask[i], bit);
        }
      }
    }
    __syncthreads();
    // the parts: an expert's tokens in order, NT x 8 at most to a part
    const int e = threadIdx.x;
    const uint32_t all = e < p.E ? s.mask[e] : 0u;
    const int parts = (__popc(all) + NT * 8 - 1) / (NT * 8);
    const int mine = parts | __popc(all) << 16;  // parts, and rows of H: scanned together
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int below = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += below;
    }
    if (e < kMaxExperts && lane == 31) s.warp_parts[warp] = sum;
    __syncthreads();
    if (e < kMaxExperts) {
      int before = sum - mine;
      for (int i = 0; i < warp; ++i) before += s.warp_parts[i];
      const int base = before & 0xFFFF;
      int row = before >> 16;
      uint32_t m = all;
      for (int a = base; a < base + parts; ++a) {
        s.act[a] = static_cast<int16_t>(e);
        int c = 0;
        for (; m != 0u && c < NT * 8; m &= m - 1u, ++c) s.tok[a][c] = static_cast<uint8_t>(__ffs(m) - 1);
        s.count[a] = static_cast<uint8_t>(c);
        s.row0[a] = static_cast<int16_t>(row);  // a part's tokens one after the other
        row += c;
      }
      if (e == kMaxExperts - 1) s.n_act = base + parts;
    }
    __syncthreads();
  }

  // ---------------------------------------------------- the second barrier
  // The users' arrival (their H is written) and their wait; the token warp
  // only waits, and the weight warp runs past.
  __device__ __forceinline__ bool poll(unsigned expected) {
    const uint64_t start = globaltimer_ns();
    for (int i = 0; ld_acquire_gpu_u32(p.bar + 2) < expected; ++i)
      if ((i & 63) == 63 && globaltimer_ns() - start > p.wait_limit_ns) {
        set_error(p.err, kErrTimeout);
        return false;
      }
    return true;
  }
  __device__ __forceinline__ bool users_meet(unsigned expected) {
    named_bar_sync(kUserBar, kUsers);
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(p.bar + 2, 1u);
      s.ok = poll(expected) ? 1 : 0;
      __threadfence();
    }
    named_bar_sync(kUserBar, kUsers);
    return s.ok != 0;
  }

  // ------------------------------------------------------------- the ring
  __device__ __forceinline__ uint8_t* stage() const { return ring + pos.stage * G::kStage; }

  // Weight warp, one thread: wait for the stage, announce its bytes.  False:
  // nothing may be copied.
  __device__ __forceinline__ bool open_stage(int rows) {
    wait(&empty[pos.stage], pos.phase ^ 1u);
    if (ok) {
      mbar_arrive_expect_tx(&full[pos.stage], static_cast<uint32_t>(rows * kSeg));
      opened = min(opened + 1, G::kStages);
    }
    return ok;
  }
  // No copy may still be in flight into shared memory at exit.  (The users see
  // the copies land, unless one of their waits ran out.)
  __device__ __forceinline__ void see_copies_land() {
    RingPos<G::kStages> last = pos;
    if ((last.stage -= opened) < 0) {
      last.stage += G::kStages;
      last.phase ^= 1u;
    }
    for (; opened > 0; --opened, last.next())
      if (!mbar_wait(&full[last.stage], last.phase, p.wait_limit_ns)) {
        set_error(p.err, kErrTimeout);
        break;
      }
  }

  // Token warp: the stages of a tile over the weights' bytes [at, end) of a
  // row, for `count` tokens' rows; mine: this lane's (lane < count).
  __device__ __forceinline__ void feed_tokens(int at, int end, int count, const uint16_t* mine) {
    for (; at < end && ok; at += kSeg, pos.next()) {
      wait(&empty[pos.stage], pos.phase ^ 1u);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const int units = min(kSeg, end - at) / 16 * kElems<WF> * 2 / 16;  // of 16 bytes
      const int first = at / 16 * kElems<WF> * 2 + lane * 16;
      uint8_t* dst = stage() + G::kWeightBytes;
#pragma unroll 2
      for (int i = 0; i < count; ++i) {
        const uint8_t* src =
            reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uintptr_t>(mine), i)) + first;
#pragma unroll
        for (int u = 0; u < G::kTokBytes / 16; u += 32)
          if (u + lane < units)
            cp_async_16(dst + in_row<G::kTokLines>(swizzled((u + lane) / 8, lane % 8), i), src + u * 16);
      }
      cp_async_arrive(&full[pos.stage]);
    }
  }

  // Where a user's fragments stand in a stage: rows lo and hi of both m16
  // halves, and the tokens of its columns.  first_w, first_tok: those of the
  // first row and token.
  struct Places {
    int w[4];
    int tok[NT][G::kStepElems / 8];
  };
  __device__ __forceinline__ void place_rows(Places& at, int r0, int r1, int r2, int r3) const {
    at.w[0] = in_row<G::kRowLines>(first_w, r0);
    at.w[1] = in_row<G::kRowLines>(first_w, r1);
    at.w[2] = in_row<G::kRowLines>(first_w, r2);
    at.w[3] = in_row<G::kRowLines>(first_w, r3);
  }
  __device__ __forceinline__ void place_tokens(Places& at, int count) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = min(n * 8 + (lane >> 2), count - 1);
#pragma unroll
      for (int i = 0; i < G::kStepElems / 8; ++i)
        at.tok[n][i] = G::kWeightBytes + in_row<G::kTokLines>(first_tok[i], row);
    }
  }

  // User: acc += its fragments of the tile's stages over the bytes [b, end)
  // of a row, for the first `halves` m16 fragments and n-tiles `tiles`.
  __device__ __forceinline__ void use_stages(int b, int end, int halves, int tiles, const Places& at,
                                             const uint32_t (&zz)[4], float (&acc)[2][NT][4]) {
    for (; b < end; b += kSeg) {
      wait(&full[pos.stage], pos.phase);
      if (warp % kAlong * G::kStep < end - b) {
        const uint8_t* st = stage();
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (G::kStep == 64) {
            v[i] = *reinterpret_cast<const uint4*>(st + at.w[i]);
          } else {
            const uint2 half = *reinterpret_cast<const uint2*>(st + at.w[i]);
            v[i] = make_uint4(half.x, half.y, 0u, 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < G::kStepElems / 8; ++i) {
          uint4 t[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n == 0 || n < tiles) t[n] = pair_up<WF>(*reinterpret_cast<const uint4*>(st + at.tok[n][i]));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (m == 1 && halves < 2) break;
            uint32_t a0[4], a1[4];
            widen8<WF>(v[2 * m], i, zz[2 * m], a0);
            widen8<WF>(v[2 * m + 1], i, zz[2 * m + 1], a1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (n > 0 && n >= tiles) break;
              router_detail::mma_bf16(acc[m][n], a0[0], a1[0], a0[1], a1[1], t[n].x, t[n].y);
              router_detail::mma_bf16(acc[m][n], a0[2], a1[2], a0[3], a1[3], t[n].z, t[n].w);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[pos.stage]);
      pos.next();
    }
  }
  __device__ __forceinline__ void clear(float (&v)[2][NT][4]) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) v[m][n][0] = v[m][n][1] = v[m][n][2] = v[m][n][3] = 0.f;
  }

  // --------------------------------------------------------- 3. gate and up
  // Calls f(part, first feature, features) for each tile of this half of the
  // block's share: at most 16 features of one interleave block of one part,
  // of a size that gives the halves equally many.
  template <typename F>
  __device__ __forceinline__ void up_tiles(F&& f) {
    const int64_t total = static_cast<int64_t>(s.n_act) * p.f / kShareStep;
    int j = static_cast<int>(total * blockIdx.x / gridDim.x) * kShareStep;
    const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x) * kShareStep;
    const int turns = (end - j + 16 * kHalves - 1) / (16 * kHalves);
    const int size = turns > 0 ? (end - j + turns * kHalves * kShareStep - 1) / (turns * kHalves * kShareStep) * kShareStep
                               : 0;
    int a = j / p.f, feat = j - a * p.f;
    for (int i = 0; j < end; i ^= 1) {
      const int rows = min(size, min(end - j, p.gu_block - feat % p.gu_block));
      if (i == half) f(a, feat, rows);
      j += rows;
      feat += rows;
      if (feat == p.f) {
        feat = 0;
        ++a;
      }
    }
  }

  __device__ __forceinline__ void feed_gateup(int row_bytes) {
    up_tiles([&](int a, int feat, int rows) {
      const int blk = s.act[a] * (p.f / p.gu_block) + feat / p.gu_block;
      const CUtensorMap* map = &maps.gate_up[rows / kShareStep - 1];
      for (int at = 0; at < row_bytes && open_stage(2 * rows); at += kSeg, pos.next())
        tma_load_5d(stage(), map, &full[pos.stage], 0, at / 128, feat % p.gu_block, 0, blk);
    });
  }
  __device__ __forceinline__ void feed_x(int row_bytes) {
    up_tiles([&](int a, int, int) {
      const int count = s.count[a];
      feed_tokens(0, row_bytes, count, p.x + (lane < count ? static_cast<int64_t>(s.tok[a][lane]) * p.d : 0));
    });
  }

  __device__ __forceinline__ void gateup(int row_bytes) {
    const int g = lane >> 2, q = lane & 3;
    up_tiles([&](int a, int feat0, int rows) {
      const int e = s.act[a], count = s.count[a];
      const int f0 = min(g, rows - 1), f1 = min(8 + g, rows - 1);  // gate rows; up rows stand `rows` further
      Places at;
      place_rows(at, f0, rows + f0, f1, rows + f1);
      place_tokens(at, count);
      uint32_t zz[4] = {0, 0, 0, 0};
      if constexpr (WF == kWInt4) {
        const int64_t z = static_cast<int64_t>(e) * p.f + feat0;
        zz[0] = (0x4300u | __ldg(p.zg + z + f0)) * 0x00010001u;
        zz[1] = (0x4300u | __ldg(p.zu + z + f0)) * 0x00010001u;
        zz[2] = (0x4300u | __ldg(p.zg + z + f1)) * 0x00010001u;
        zz[3] = (0x4300u | __ldg(p.zu + z + f1)) * 0x00010001u;
      }
      float acc[2][NT][4];
      clear(acc);
      use_stages(0, row_bytes, rows > 8 ? 2 : 1, count > 8 ? 2 : 1, at, zz, acc);
      named_bar_sync(kHalfBar + half, kAlong * 32);  // the last tile's sums are read
      // row 16 m + r of a warp's sums: gate (r < 8) or up of feature 8 m + r % 8
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          *reinterpret_cast<float2*>(&s.red[warp][16 * m + g][n * 8 + 2 * q]) = make_float2(acc[m][n][0], acc[m][n][1]);
          *reinterpret_cast<float2*>(&s.red[warp][16 * m + 8 + g][n * 8 + 2 * q]) =
              make_float2(acc[m][n][2], acc[m][n][3]);
        }
      named_bar_sync(kHalfBar + half, kAlong * 32);
      const int r = threadIdx.x % 16, t = threadIdx.x % (kAlong * 32) / 16;
      if (t < count && r < rows) {
        const int row = (r & 8) * 2 + (r & 7);
        float gs = 0.f, us = 0.f;
#pragma unroll
        for (int w = 0; w < kAlong; ++w) {
          gs += s.red[half * kAlong + w][row][t];
          us += s.red[half * kAlong + w][row + 8][t];
        }
        if constexpr (WF != kBf16) {
          const int64_t sc = static_cast<int64_t>(e) * p.f + feat0 + r;
          gs *= __ldg(p.sg + sc);
          us *= __ldg(p.su + sc);
        }
        const __nv_bfloat16 h = __float2bfloat16_rn(silu(gs) * us);
        p.h[static_cast<int64_t>(s.row0[a] + t) * p.f + feat0 + r] = __bfloat16_as_ushort(h);
      }
    });
  }

  // ------------------------------------------------- 4. down and combine
  // Calls f(first column, columns, part, first and last byte of a row) for
  // this half of the block's share, tiles of at most 32 output columns, and
  // done(first column, columns) after each: the halves take the parts in
  // turn, or half of each row where there are few.
  template <typename F, typename D>
  __device__ __forceinline__ void down_tiles(int row_bytes, F&& f, D&& done) {
    const int64_t total = p.d / kShareStep;
    const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x) * kShareStep;
    const bool split = s.n_act < kFewParts;
    const int mid = (row_bytes + kSeg * kHalves - 1) / (kSeg * kHalves) * kSeg;
    const int from = split && half == 1 ? mid : 0, to = split && half == 0 ? min(mid, row_bytes) : row_bytes;
    for (int c = static_cast<int>(total * blockIdx.x / gridDim.x) * kShareStep; c < end; c += kRows) {
      const int rows = min(kRows, end - c);
      for (int a = split ? 0 : half; a < s.n_act; a += split ? 1 : kHalves)
        if (from < to) f(c, rows, a, from, to);
      done(c, rows);
    }
  }

  __device__ __forceinline__ void feed_down(int row_bytes) {
    down_tiles(
        row_bytes,
        [&](int c, int rows, int a, int from, int to) {
          const CUtensorMap* map = &maps.down[rows / kShareStep - 1];
          const int row = s.act[a] * p.d + c;
          for (int at = from; at < to && open_stage(rows); at += kSeg, pos.next())
            tma_load_3d(stage(), map, &full[pos.stage], 0, at / 128, row);
        },
        [](int, int) {});
  }
  __device__ __forceinline__ void feed_h(int row_bytes) {
    down_tiles(
        row_bytes,
        [&](int, int, int a, int from, int to) {
          const int count = s.count[a];
          feed_tokens(from, to, count, p.h + static_cast<int64_t>(s.row0[a] + min(lane, count - 1)) * p.f);
        },
        [](int, int) {});
  }
  // After a second barrier that was not met: nobody will use the stages that
  // the weight warp opened ahead; see their copies land.
  __device__ __forceinline__ void drop_down(int row_bytes) {
    int left = G::kStages;
    down_tiles(
        row_bytes,
        [&](int, int, int, int from, int to) {
          for (int at = from; at < to && left > 0; at += kSeg, --left, pos.next()) {
            mbar_arrive(&full[pos.stage]);
            mbar_wait(&full[pos.stage], pos.phase, p.wait_limit_ns);
          }
        },
        [](int, int) {});
  }

  __device__ __forceinline__ void down(int row_bytes) {
    const int g = lane >> 2, q = lane & 3;
    auto zero = [&]() {  // the warp's own sums
      float4* r = reinterpret_cast<float4*>(&s.red[warp][0][0]);
      for (int i = lane; i < kRows * MT / 4; i += 32) r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      __syncwarp();
    };
    zero();
    Places at;
    int row[4], placed = 0;
    auto part = [&](int c, int rows, int a, int from, int to) {
      const int e = s.act[a], count = s.count[a];
      if (rows != placed) {
        placed = rows;
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = min(8 * i + g, rows - 1);
        place_rows(at, row[0], row[1], row[2], row[3]);
      }
      place_tokens(at, count);
      const int64_t ch = static_cast<int64_t>(e) * p.d + c;
      uint32_t zz[4] = {0, 0, 0, 0};
      float sc[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (WF == kWInt4) zz[i] = (0x4300u | __ldg(p.zd + ch + row[i])) * 0x00010001u;
        if constexpr (WF != kBf16) sc[i] = __ldg(p.sd + ch + row[i]);
      }
      float acc[2][NT][4];
      clear(acc);
      use_stages(from, to, rows > 16 ? 2 : 1, count > 8 ? 2 : 1, at, zz, acc);
      // the warp's share of the part, weighed and added to its tokens' sums
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (n * 8 + u >= count) break;
          const int i = n * 8 + 2 * q + u;
          if (i >= count) continue;
          const int t = s.tok[a][i];
          const float w = s.w[t * p.k + s.slot[e][t]];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float& sum = s.red[warp][8 * r + g][t];
            sum = fmaf(w * sc[r], acc[r / 2][n][(r & 1) * 2 + u], sum);
          }
        }
      __syncwarp();
    };
    down_tiles(row_bytes, part, [&](int c, int rows) {
      named_bar_sync(kUserBar, kUsers);
      for (int o = threadIdx.x; o < kRows * MT; o += kUsers) {
        const int r = o % kRows, t = o / kRows;
        if (t >= p.n || r >= rows) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kUserWarps; ++w) sum += s.red[w][r][t];
        const int64_t to = static_cast<int64_t>(t) * p.d + c + r;
        if (p.out_f32)
          static_cast<float*>(p.out)[to] = sum;
        else
          static_cast<uint16_t*>(p.out)[to] = __bfloat16_as_ushort(__float2bfloat16_rn(sum));
      }
      named_bar_sync(kUserBar, kUsers);
      zero();
    });
  }
};

template <int WF, int NT, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    few_tokens_kernel(const __grid_constant__ FewMaps maps, const FewArgs p) {
  using G = Geo<WF, NT, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Block<WF, NT, MT> b(p, maps, smem);
  const unsigned blocks = gridDim.x;
  const unsigned expected = blocks + static_cast<unsigned>(p.test_stall);
  bool ok = true;
  if (Block<WF, NT, MT>::logits_here(p)) {
    __syncthreads();
    b.own_logits();
  } else if (p.ids == nullptr) {
    b.logits();
    ok = grid_barrier_wait(p.bar, expected, p.wait_limit_ns, p.err, &b.s.ok);
    if (threadIdx.x == 0) grid_barrier_depart(p.bar, blocks);
  } else {
    __syncthreads();
  }
  const int up_bytes = p.d / kElems<WF> * 16, down_bytes = p.f / kElems<WF> * 16;
  if (ok) b.gate();
  // (a block that timed out above still meets the others at the second barrier)
  if (b.warp >= kWeightWarp && b.warp < kTokenWarp) {
    if (ok && b.lane == 0) {
      b.feed_gateup(up_bytes);
      b.feed_down(down_bytes);
      b.see_copies_land();
    }
  } else if (b.warp >= kTokenWarp) {
    if (ok) {
      b.feed_x(up_bytes);
      bool met = true;
      if (b.lane == 0) {
        met = b.poll(expected);
        __threadfence();
      }
      __syncwarp();  // the other lanes read other blocks' H too (a vote orders no memory)
      if (__all_sync(0xffffffffu, met))
        b.feed_h(down_bytes);
      else
        b.drop_down(down_bytes);
      cp_async_wait_all();
    }
  } else {
    if (ok) b.gateup(up_bytes);
    if (b.users_meet(expected) && ok) b.down(down_bytes);
  }
  __syncthreads();
  if (threadIdx.x == 0) grid_barrier_depart(p.bar + 2, blocks);
}

template <int WF, int NT, int MT>
cudaError_t prepare(int* per_sm) {
  auto kernel = few_tokens_kernel<WF, NT, MT>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<WF, NT, MT>::kBytes);
  if (e != cudaSuccess) return e;
  int n = 0;
  const cudaError_t o = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, Geo<WF, NT, MT>::kBytes);
  *per_sm = n < *per_sm ? n : *per_sm;
  return o;
}

template <int WF, int NT, int MT>
cudaError_t launch(const FewMaps& m, const FewArgs& a, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Geo<WF, NT, MT>::kBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_tokens_kernel<WF, NT, MT>, m, a);
}

}  // namespace

int few_format(bool quantised, WeightFormat wf) { return quantised ? static_cast<int>(wf) : kBf16; }

template <int WF>
static cudaError_t prepare_format(int* blocks_per_sm) {
  cudaError_t e = prepare<WF, 1, 8>(blocks_per_sm);
  if (e == cudaSuccess) e = prepare<WF, 1, 16>(blocks_per_sm);
  return e == cudaSuccess ? prepare<WF, 2, 16>(blocks_per_sm) : e;
}

cudaError_t few_tokens_prepare(int format, int* blocks_per_sm) {
  *blocks_per_sm = 1;
  switch (format) {
    case kBf16: return prepare_format<kBf16>(blocks_per_sm);
    case kWInt8: return prepare_format<kWInt8>(blocks_per_sm);
    case kWInt4: return prepare_format<kWInt4>(blocks_per_sm);
    case kWFp8: return prepare_format<kWFp8>(blocks_per_sm);
  }
  return cudaErrorInvalidValue;
}

template <int NT>
static bool part_maps(int format, const FewArgs& a, FewMaps* m) {
  const uint64_t elems = format == kBf16 ? kElems<kBf16> : format == kWInt4 ? kElems<kWInt4> : kElems<kWInt8>;
  const uint64_t up = a.d / elems * 16, down = a.f / elems * 16, blk = a.gu_block;
  const cuuint32_t lines = (format == kWInt4 ? kSeg<kWInt4, NT> : kSeg<kBf16, NT>) / 128;
  // rows of bytes as (byte of a 128-byte chunk, chunk, row[, gate or up, interleave block])
  const cuuint64_t up_dims[5] = {128, up / 128, blk, 2, static_cast<uint64_t>(a.E) * a.f / blk};
  const cuuint64_t up_strides[4] = {128, up, blk * up, 2 * blk * up};
  const cuuint64_t down_dims[3] = {128, down / 128, static_cast<uint64_t>(a.E) * a.d};
  const cuuint64_t down_strides[2] = {128, down};
  bool ok = true;
  for (int i = 0; i < kRows / 2 / kShareStep; ++i) {
    const cuuint32_t box[5] = {128, lines, static_cast<cuuint32_t>((i + 1) * kShareStep), 2, 1};
    ok = ok && make_tmap_nd(&m->gate_up[i], a.wgu, 5, up_dims, up_strides, box);
  }
  for (int i = 0; i < kRows / kShareStep; ++i) {
    const cuuint32_t box[3] = {128, lines, static_cast<cuuint32_t>((i + 1) * kShareStep)};
    ok = ok && make_tmap_nd(&m->down[i], a.wd, 3, down_dims, down_strides, box);
  }
  return ok;
}

bool few_token_maps(int format, const FewArgs& a, FewMaps (&m)[2]) {
  return part_maps<1>(format, a, &m[0]) && part_maps<2>(format, a, &m[1]);
}

// More than 8 tokens: parts of up to 16 where experts have more than 4 of the
// tokens on average.  Below, the few experts that have more than 8 are taken
// in two parts, their weights read twice; the smaller stages leave half as
// many again of them in flight.
template <int WF>
static cudaError_t launch_format(const FewMaps (&m)[2], const FewArgs& a, int grid, cudaStream_t s) {
  if (a.n <= 8) return launch<WF, 1, 8>(m[0], a, grid, s);
  return a.n * a.k > 4 * a.E ? launch<WF, 2, 16>(m[1], a, grid, s) : launch<WF, 1, 16>(m[0], a, grid, s);
}

cudaError_t launch_few_tokens(int format, const FewMaps (&m)[2], const FewArgs& a, int grid, cudaStream_t s) {
  if (a.n <= 0) return cudaSuccess;
  if (a.n > kMaxTokens || a.E > kMaxExperts || a.k > kMaxK || grid <= 0) return cudaErrorInvalidValue;
  switch (format) {
    case kBf16: return launch_format<kBf16>(m, a, grid, s);
    case kWInt8: return launch_format<kWInt8>(m, a, grid, s);
    case kWInt4: return launch_format<kWInt4>(m, a, grid, s);
    case kWFp8: return launch_format<kWFp8>(m, a, grid, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace cbmoe
