// Host side of the C ABI in cb_fp4.h: argument validation and the launches.
#include <atomic>
#include <cstdlib>
#include <cstring>

#include "cb_fp4.h"
#include "fp4.cuh"
#include "internal.h"

using namespace cbmoe;

namespace {

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Testing only: what CB_MOE_INJECT_FAULT asks for.
enum Fault { kNoFault, kLaunch, kStall };
Fault injected_fault() {
  const char* v = std::getenv("CB_MOE_INJECT_FAULT");
  return v == nullptr ? kNoFault : std::strcmp(v, "launch") == 0 ? kLaunch : std::strcmp(v, "stall") == 0 ? kStall : kNoFault;
}

int64_t scale_bytes(int32_t format, int64_t rows, int64_t cols) {
  const int64_t block = format == CB_FP4_MX ? kFp4Block<kFp4Mx> : kFp4Block<kFp4Nv>;
  return (rows + kScaleTileRows - 1) / kScaleTileRows * ((cols / block + 3) / 4) * kScaleTileBytes;
}

bool known_format(int32_t f) { return f == CB_FP4_MX || f == CB_FP4_NV; }
bool known_type(int32_t t) { return t == CB_T_BF16 || t == CB_T_F32; }

// The current device: this library's kernels are for compute capability 10.3.
// A device's SM count is asked for once (0: not
// yet; negative: a wrong GPU).
cb_status_t check_device(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return CB_ERR_CUDA;
  }
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return CB_ERR_CUDA;
    }
    if (major != 10 || minor != 3) n = -1;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  *sms = n;
  return n > 0 ? CB_OK : CB_ERR_UNSUPPORTED;
}

bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// Arguments of the quantiser and its way back; x is its input or output.
cb_status_t check_matrix(int32_t format, const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld,
                         const float* tensor_scale, const uint8_t* codes, const uint8_t* scales) {
  if (!known_format(format) || !known_type(type) || rows < 0 || cols <= 0 || cols % 32 != 0 || ld < cols)
    return CB_ERR_INVALID_ARG;
  if (rows > 0 && (x == nullptr || codes == nullptr || scales == nullptr)) return CB_ERR_INVALID_ARG;
  if ((tensor_scale != nullptr) != (format == CB_FP4_NV)) return CB_ERR_INVALID_ARG;
  if (!on(codes, 16) || !on(scales, 16) || !on(x, type == CB_T_F32 ? 4 : 2) || !on(tensor_scale, 4))
    return CB_ERR_ALIGNMENT;
  // (the quotients first: a product of both sizes may pass 64 bits)
  if (cols >= (1ll << 31) || rows / kScaleTileRows >= (1ll << 31) || fp4_tiles(rows, cols) >= (1ll << 31) ||
      ld >= (1ll << 62) / (rows + 1))
    return CB_ERR_UNSUPPORTED;
  if (rows > 0) {
    const uint64_t xb = (static_cast<uint64_t>(rows - 1) * ld + cols) * (type == CB_T_F32 ? 4 : 2);
    const uint64_t cb = static_cast<uint64_t>(rows) * cols / 2, sb = static_cast<uint64_t>(scale_bytes(format, rows, cols));
    if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb) || overlap(codes, cb, scales, sb))
      return CB_ERR_INVALID_ARG;
  }
  return CB_OK;
}

}  // namespace

extern "C" {

cb_status_t cb_fp4_scale_bytes(int32_t format, int64_t rows, int64_t cols, uint64_t* bytes) {
  if (bytes == nullptr || !known_format(format) || rows < 0 || cols <= 0 || cols % 32 != 0) return CB_ERR_INVALID_ARG;
  *bytes = static_cast<uint64_t>(scale_bytes(format, rows, cols));
  return CB_OK;
}

cb_status_t cb_fp4_quantize(int32_t format, const void* x, int32_t x_type, int64_t rows, int64_t cols, int64_t ld,
                            const float* tensor_scale, uint8_t* codes, uint8_t* scales, void* stream) {
  cb_status_t st = check_matrix(format, x, x_type, rows, cols, ld, tensor_scale, codes, scales);
  if (st != CB_OK || rows == 0) return st;
  int sms;
  if ((st = check_device(&sms)) != CB_OK) return st;
  if (injected_fault() == kLaunch) return CB_ERR_CUDA;
  const Fp4Args a{format, x_type == CB_T_F32, const_cast<void*>(x), rows, cols, ld, tensor_scale, codes, scales};
  return launch_fp4_quantize(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

cb_status_t cb_fp4_dequantize(int32_t format, const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                              int64_t rows, int64_t cols, void* out, int32_t out_type, int64_t ld, void* stream) {
  cb_status_t st = check_matrix(format, out, out_type, rows, cols, ld, tensor_scale, codes, scales);
  if (st != CB_OK || rows == 0) return st;
  int sms;
  if ((st = check_device(&sms)) != CB_OK) return st;
  if (injected_fault() == kLaunch) return CB_ERR_CUDA;
  const Fp4Args a{format, out_type == CB_T_F32, out, rows, cols, ld, tensor_scale, const_cast<uint8_t*>(codes),
                  const_cast<uint8_t*>(scales)};
  return launch_fp4_dequantize(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

cb_status_t cb_fp4_matmul(const cb_fp4_matmul_t* p, void* stream) {
  if (p == nullptr || !known_format(p->format) || !known_type(p->out_type)) return CB_ERR_INVALID_ARG;
  if (p->m < 0 || p->n < 0 || p->k <= 0 || p->k % 32 != 0 || p->ld_out < p->n || p->n_groups < 1 ||
      (p->n_groups > 1 && p->tile_offsets == nullptr))
    return CB_ERR_INVALID_ARG;
  const bool nv = p->format == CB_FP4_NV;
  if ((p->a_tensor_scale != nullptr) != nv || (p->b_tensor_scale != nullptr) != nv) return CB_ERR_INVALID_ARG;
  const int64_t limit = 1ll << 31;
  if (p->m >= limit - 128 || p->n >= limit - 256 || p->k >= limit - 256 || p->n > (limit - 256) / p->n_groups)
    return CB_ERR_UNSUPPORTED;
  if (p->m == 0 || p->n == 0) return CB_OK;
  if (p->a_codes == nullptr || p->a_scales == nullptr || p->b_codes == nullptr || p->b_scales == nullptr ||
      p->out == nullptr)
    return CB_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(p->a_codes), static_cast<const void*>(p->a_scales),
                        static_cast<const void*>(p->b_codes), static_cast<const void*>(p->b_scales),
                        static_cast<const void*>(p->out)})
    if (!on(q, 16)) return CB_ERR_ALIGNMENT;
  for (const void* q : {static_cast<const void*>(p->a_tensor_scale), static_cast<const void*>(p->b_tensor_scale),
                        static_cast<const void*>(p->tile_offsets), static_cast<const void*>(p->status)})
    if (!on(q, 4)) return CB_ERR_ALIGNMENT;
  // tiles of the output are counted in 32 bits
  if ((p->m + 127) / 128 >= limit / ((p->n + 127) / 128)) return CB_ERR_UNSUPPORTED;
  if (p->ld_out >= (1ll << 62) / p->m) return CB_ERR_UNSUPPORTED;
  const uint64_t out_bytes =
      (static_cast<uint64_t>(p->m - 1) * p->ld_out + p->n) * (p->out_type == CB_T_F32 ? 4 : 2);
  const uint64_t g = static_cast<uint64_t>(p->n_groups);
  if (overlap(p->out, out_bytes, p->a_codes, static_cast<uint64_t>(p->m) * p->k / 2) ||
      overlap(p->out, out_bytes, p->b_codes, g * p->n * p->k / 2) ||
      overlap(p->out, out_bytes, p->a_scales, scale_bytes(p->format, p->m, p->k)) ||
      overlap(p->out, out_bytes, p->b_scales, g * scale_bytes(p->format, p->n, p->k)))
    return CB_ERR_INVALID_ARG;
  int sms = 0;
  const cb_status_t st = check_device(&sms);
  if (st != CB_OK) return st;
  const Fault fault = injected_fault();
  if (fault == kLaunch) return CB_ERR_CUDA;
  Fp4MatmulArgs a{};
  a.format = p->format;
  a.out_f32 = p->out_type == CB_T_F32;
  a.m = static_cast<int32_t>(p->m);
  a.n = static_cast<int32_t>(p->n);
  a.k = static_cast<int32_t>(p->k);
  a.a_codes = p->a_codes;
  a.a_scales = p->a_scales;
  a.a_tensor_scale = p->a_tensor_scale;
  a.b_codes = p->b_codes;
  a.b_scales = p->b_scales;
  a.b_tensor_scale = p->b_tensor_scale;
  a.n_groups = p->n_groups;
  a.tile_offsets = p->tile_offsets;
  a.out = p->out;
  a.ld_out = p->ld_out;
  a.status = p->status;
  a.wait_limit_ns = kWaitLimitNs;
  if (fault == kStall) {
    a.test_stall = 1;
    a.wait_limit_ns = 1000000ull;  // 1 ms
  }
  return launch_fp4_matmul(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

cb_status_t cb_fp4_last_error(void) {
  int sms, code = 0;
  const cb_status_t st = check_device(&sms);
  if (st != CB_OK) return st;
  return take_fp4_error(&code) == cudaSuccess ? static_cast<cb_status_t>(code) : CB_ERR_CUDA;
}

}  // extern "C"
