// group.cu -- 4-bit weights with one step per group of inputs, and their
// product with a few tokens (include/decode.h, w4a4_group_*).
#include <cuda_runtime.h>

#include <cstdint>

#include "decode.cuh"
#include "decode.h"
#include "gelu.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace w4a4 {
namespace {

constexpr int kTileRows = 16;   // rows of a weight tile
constexpr int kBlockK = 128;    // inputs of a weight block: 1024 bytes of codes per tile

struct GroupShape {
  int N, K, group;
  int tiles, blocks;  // ceil(N / 16), ceil(K / 128)
};

// Byte offset of the word that holds inputs 8 i .. 8 i + 7 of row n.
__device__ __forceinline__ int64_t word_offset(const GroupShape &s, int n, int i) {
  const int t = n / kTileRows, h = (n >> 3) & 1, r = n & 7;
  const int b = i >> 4, j = (i >> 2) & 3, c = i & 3;
  return ((static_cast<int64_t>(t) * s.blocks + b) * 2 + h) * 512 + 64 * r + 16 * c + 4 * j;
}

// Element offset of the step of row n, group g.
__device__ __forceinline__ int64_t scale_offset(const GroupShape &s, int n, int g) {
  const int t = n / kTileRows, h = (n >> 3) & 1, r = n & 7;
  const int per = kBlockK / s.group, b = g / per;
  return ((static_cast<int64_t>(t) * s.blocks + b) * 8 + r) * (2 * per) + 2 * (g % per) + h;
}

// Nibble of element e (0..7) in a word: 0, 2, 4, 6, 1, 3, 5, 7 from the lowest up.
__device__ __forceinline__ int nibble_shift(int e) { return 4 * ((e >> 1) + 4 * (e & 1)); }

__device__ __forceinline__ int code_of(uint32_t w, int e) {
  return (static_cast<int>((w >> nibble_shift(e)) & 15u) ^ 8) - 8;
}

// One thread per word; the 4, 8 or 16 threads of a group share its maximum.
// Rows and inputs of the padding get zero codes and steps.
template <typename T>
__global__ void __launch_bounds__(256)
    group_quantize_kernel(const uint16_t *__restrict__ W, GroupShape s, uint8_t *__restrict__ codes,
                          uint16_t *__restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int words = s.blocks * (kBlockK / 8);
  const int64_t total = static_cast<int64_t>(s.tiles) * kTileRows * words;
  const int lanes = s.group / 8;  // threads of a group
  // every thread of a warp takes part in the shuffles: total is a multiple of 32
  for (int64_t at = blockIdx.x * 256ll + threadIdx.x; at < total; at += gridDim.x * 256ll) {
    const int n = static_cast<int>(at / words), i = static_cast<int>(at % words);
    float x[8];
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < s.N && 8 * i < s.K) v = *reinterpret_cast<const uint4 *>(W + static_cast<int64_t>(n) * s.K + 8 * i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = T::lo(u[e]);
      x[2 * e + 1] = T::hi(u[e]);
      m = fmaxf(m, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
    }
    for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint16_t step16 = T::round(__fdiv_rn(m, 7.0f));
    const float step = T::to_f32(step16);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float q = step > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(x[e], step)), -8.0f), 7.0f) : 0.0f;
      w |= (static_cast<uint32_t>(static_cast<int>(q)) & 15u) << nibble_shift(e);
    }
    *reinterpret_cast<uint32_t *>(codes + word_offset(s, n, i)) = w;
    if (i % lanes == 0) scales[scale_offset(s, n, i / lanes)] = step16;
  }
}

__global__ void __launch_bounds__(256)
    group_pack_kernel(const uint8_t *__restrict__ plain, const uint16_t *__restrict__ steps, GroupShape s,
                      uint8_t *__restrict__ codes, uint16_t *__restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const int words = s.blocks * (kBlockK / 8);
  const int64_t total = static_cast<int64_t>(s.tiles) * kTileRows * words;
  const int lanes = s.group / 8;
  for (int64_t at = blockIdx.x * 256ll + threadIdx.x; at < total; at += gridDim.x * 256ll) {
    const int n = static_cast<int>(at / words), i = static_cast<int>(at % words);
    const bool live = n < s.N && 8 * i < s.K;
    uint32_t v = 0, w = 0;
    if (live) v = *reinterpret_cast<const uint32_t *>(plain + static_cast<int64_t>(n) * (s.K / 2) + 4 * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= ((v >> (4 * e)) & 15u) << nibble_shift(e);
    *reinterpret_cast<uint32_t *>(codes + word_offset(s, n, i)) = w;
    if (i % lanes == 0) {
      const int g = i / lanes;
      scales[scale_offset(s, n, g)] = live ? steps[static_cast<int64_t>(n) * (s.K / s.group) + g] : uint16_t(0);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
    group_dequantize_kernel(const uint8_t *__restrict__ codes, const uint16_t *__restrict__ scales, GroupShape s,
                            uint16_t *__restrict__ W) {
  griddep_launch_dependents();
  griddep_wait();
  const int words = s.K / 8;
  const int64_t total = static_cast<int64_t>(s.N) * words;
  for (int64_t at = blockIdx.x * 256ll + threadIdx.x; at < total; at += gridDim.x * 256ll) {
    const int n = static_cast<int>(at / words), i = static_cast<int>(at % words);
    const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + word_offset(s, n, i));
    const float step = T::to_f32(scales[scale_offset(s, n, 8 * i / s.group)]);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = T::pack(static_cast<float>(code_of(w, 2 * e)) * step, static_cast<float>(code_of(w, 2 * e + 1)) * step);
    *reinterpret_cast<uint4 *>(W + static_cast<int64_t>(n) * s.K + 8 * i) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// One warp per row and token: lane l takes words l, l + 32, ... of the row.
template <typename T>
__global__ void __launch_bounds__(256)
    group_gemv_kernel(const uint16_t *__restrict__ X, int M, const uint8_t *__restrict__ codes,
                      const uint16_t *__restrict__ scales, GroupShape s, const uint16_t *__restrict__ bias,
                      uint16_t *__restrict__ Y, bool gelu) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int n = static_cast<int>(unit / M), m = static_cast<int>(unit % M);
  if (n >= s.N) return;
  float sum = 0.0f;
  for (int i = lane; i < s.K / 8; i += 32) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + word_offset(s, n, i));
    const uint4 v = *reinterpret_cast<const uint4 *>(X + static_cast<int64_t>(m) * s.K + 8 * i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float part = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      part = fmaf(T::lo(u[e]), static_cast<float>(code_of(w, 2 * e)), part);
      part = fmaf(T::hi(u[e]), static_cast<float>(code_of(w, 2 * e + 1)), part);
    }
    sum = fmaf(T::to_f32(scales[scale_offset(s, n, 8 * i / s.group)]), part, sum);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    if (bias) sum += T::to_f32(bias[n]);
    uint16_t y = T::round(sum);
    if (gelu) y = static_cast<uint16_t>(gelu_pair_bf16(y) & 0xFFFFu);
    Y[static_cast<int64_t>(m) * s.N + n] = y;
  }
}

constexpr uint32_t kGroupFlags = W4A4_FLAG_FP16;

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }
bool group_shape_ok(int32_t N, int32_t K, int32_t group) {
  return N >= 1 && N <= 0x7FFFFFF0 && K >= group && K % group == 0 && K <= (1 << 20);
}

GroupShape shape_of(int32_t N, int32_t K, int32_t group) {
  return {N, K, group, (N - 1) / kTileRows + 1, (K + kBlockK - 1) / kBlockK};
}

size_t code_bytes(const GroupShape &s) { return static_cast<size_t>(s.tiles) * s.blocks * 1024; }
size_t scale_bytes(const GroupShape &s) {
  return static_cast<size_t>(s.tiles) * s.blocks * (16 * (kBlockK / s.group)) * 2;
}
size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

w4a4_status check_group(const w4a4_group_weights_t *w) {
  if (!w) return W4A4_ERR_ARG;
  if (!group_ok(w->group) || (w->flags & ~kGroupFlags)) return W4A4_ERR_UNSUPPORTED;
  if (!group_shape_ok(w->N, w->K, w->group)) return W4A4_ERR_SHAPE;
  if (!w->codes || !w->scales) return W4A4_ERR_ARG;
  if (!ptr_aligned16(w->codes) || !ptr_aligned16(w->scales)) return W4A4_ERR_ALIGN;
  return W4A4_OK;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), int64_t grid, int threads, size_t smem, void *stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// blocks of 256 threads for n threads' work, at most 16 per SM
int64_t stride_grid(int64_t n) {
  const int64_t need = (n + 255) / 256, most = 16ll * device_sm_count();
  return need < most ? need : most;
}

}  // namespace
}  // namespace w4a4

extern "C" {

size_t w4a4_group_weights_bytes(int32_t N, int32_t K, int32_t group) {
  using namespace w4a4;
  if (!group_ok(group) || !group_shape_ok(N, K, group)) return 0;
  const GroupShape s = shape_of(N, K, group);
  return round256(code_bytes(s)) + scale_bytes(s);
}

w4a4_status w4a4_group_bind(void *base, size_t bytes, int32_t N, int32_t K, int32_t group, uint32_t flags,
                            w4a4_group_weights_t *out) {
  using namespace w4a4;
  if (!base || !out) return W4A4_ERR_ARG;
  if (!group_ok(group) || (flags & ~kGroupFlags)) return W4A4_ERR_UNSUPPORTED;
  if (!ptr_aligned16(base)) return W4A4_ERR_ALIGN;
  if (!group_shape_ok(N, K, group)) return W4A4_ERR_SHAPE;
  if (bytes < w4a4_group_weights_bytes(N, K, group)) return W4A4_ERR_SHAPE;
  uint8_t *b = static_cast<uint8_t *>(base);
  out->N = N;
  out->K = K;
  out->group = group;
  out->flags = flags;
  out->codes = b;
  out->scales = reinterpret_cast<uint16_t *>(b + round256(code_bytes(shape_of(N, K, group))));
  return W4A4_OK;
}

w4a4_status w4a4_group_quantize(const uint16_t *W, const w4a4_group_weights_t *w, void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!W) return W4A4_ERR_ARG;
  if (!ptr_aligned16(W)) return W4A4_ERR_ALIGN;
  const GroupShape s = shape_of(w->N, w->K, w->group);
  const int64_t grid = stride_grid(static_cast<int64_t>(s.tiles) * 16 * s.blocks * 16);
  return launch_status(launch((w->flags & W4A4_FLAG_FP16) ? group_quantize_kernel<Fp16> : group_quantize_kernel<Bf16>,
                              grid, 256, 0, stream, W, s, w->codes, w->scales));
}

w4a4_status w4a4_group_pack(const uint8_t *codes, const uint16_t *scales, const w4a4_group_weights_t *w,
                            void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!codes || !scales) return W4A4_ERR_ARG;
  if (!ptr_aligned16(codes) || !ptr_aligned16(scales)) return W4A4_ERR_ALIGN;
  const GroupShape s = shape_of(w->N, w->K, w->group);
  const int64_t grid = stride_grid(static_cast<int64_t>(s.tiles) * 16 * s.blocks * 16);
  return launch_status(launch(group_pack_kernel, grid, 256, 0, stream, codes, scales, s, w->codes, w->scales));
}

w4a4_status w4a4_group_dequantize(const w4a4_group_weights_t *w, uint16_t *W, void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!W) return W4A4_ERR_ARG;
  if (!ptr_aligned16(W)) return W4A4_ERR_ALIGN;
  const GroupShape s = shape_of(w->N, w->K, w->group);
  const int64_t grid = stride_grid(static_cast<int64_t>(s.N) * (s.K / 8));
  return launch_status(
      launch((w->flags & W4A4_FLAG_FP16) ? group_dequantize_kernel<Fp16> : group_dequantize_kernel<Bf16>, grid, 256, 0,
             stream, w->codes, w->scales, s, W));
}

w4a4_status w4a4_group_gemv(const uint16_t *X, int64_t M, const w4a4_group_weights_t *w, const uint16_t *bias,
                            uint16_t *Y, uint32_t flags, void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  const bool fp16 = (w->flags & W4A4_FLAG_FP16) != 0, gelu = (flags & W4A4_FLAG_GELU_OUT) != 0;
  if ((flags & ~W4A4_FLAG_GELU_OUT) || (gelu && fp16)) return W4A4_ERR_UNSUPPORTED;
  if (M < 0 || M > W4A4_GEMV_MAX_TOKENS) return W4A4_ERR_SHAPE;
  if (M == 0) return W4A4_OK;
  if (!X || !Y) return W4A4_ERR_ARG;
  if (!ptr_aligned16(X) || !ptr_aligned16(Y) || (bias && !ptr_aligned16(bias))) return W4A4_ERR_ALIGN;
  const GroupShape s = shape_of(w->N, w->K, w->group);
  const int64_t grid = (static_cast<int64_t>(s.N) * M + 7) / 8;
  if (grid > 0x7FFFFFFF) return W4A4_ERR_SHAPE;
  return launch_status(launch(fp16 ? group_gemv_kernel<Fp16> : group_gemv_kernel<Bf16>, grid, 256, 0, stream, X,
                              static_cast<int>(M), w->codes, w->scales, s, bias, Y, gelu));
}

}  // extern "C"
