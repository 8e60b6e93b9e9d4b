// kv.cu -- the paged key-value cache (include/decode.h, w4a4_kv_*): new tokens
// rotated and appended, and one new token per sequence attending to what is
// cached.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "decode.cuh"
#include "decode.h"
#include "kernels.h"
#include "ptx.cuh"

namespace w4a4 {
namespace {

struct Cache {
  uint16_t *k, *v;
  int n_pages, page_size, heads;
  int64_t stride_page, stride_token, stride_head;
};

struct Pages {
  const int32_t *table;  // [n_seqs, max_pages]
  int n_seqs, max_pages;
};

struct AppendArgs {
  Cache cache;
  Pages pages;
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t k_stride, v_stride, q_stride;
  int q_heads, head_dim, rot_dim, n_table;
  const int32_t *seq, *pos, *table_pos;
  const float *table;
  bool pairs;
};

// One block per token; thread by thread over its elements.
template <typename T>
__global__ void __launch_bounds__(128) kv_append_kernel(AppendArgs a, unsigned int *__restrict__ status) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int p = a.pos[t];
  if (p < 0) return;
  const int64_t s = a.seq ? a.seq[t] : t;
  const int64_t turn = a.table_pos ? a.table_pos[t] : p;
  const int entry = p / a.cache.page_size;
  int page = -1;
  if (s >= 0 && s < a.pages.n_seqs && entry < a.pages.max_pages) page = a.pages.table[s * a.pages.max_pages + entry];
  if (page < 0 || page >= a.cache.n_pages || (a.rot_dim && (turn < 0 || turn >= a.n_table))) {
    if (threadIdx.x == 0) atomicOr(status, W4A4_DEV_RANGE);
    return;
  }
  const int64_t row = page * a.cache.stride_page + (p % a.cache.page_size) * a.cache.stride_token;
  const int D = a.head_dim, half = a.rot_dim / 2;
  const float *tab = a.table + turn * a.rot_dim;
  for (int u = threadIdx.x; u < a.cache.heads * D; u += 128)
    a.cache.v[row + (u / D) * a.cache.stride_head + u % D] = a.v[t * a.v_stride + u];
  // per head half turned pairs, then what is only copied
  const int units = half + D - a.rot_dim;
  for (int u = threadIdx.x; u < (a.cache.heads + a.q_heads) * units; u += 128) {
    const int head = u / units, i = u % units;
    const bool key = head < a.cache.heads;
    const uint16_t *src = key ? a.k + t * a.k_stride + head * D : a.q + t * a.q_stride + (head - a.cache.heads) * D;
    uint16_t *dst = key ? a.cache.k + row + head * a.cache.stride_head
                        : a.q_out + (t * a.q_heads + (head - a.cache.heads)) * D;
    if (i >= half) {
      dst[i + half] = src[i + half];
      continue;
    }
    const int ia = a.pairs ? 2 * i : i, ib = a.pairs ? 2 * i + 1 : i + half;
    const float x = T::to_f32(src[ia]), y = T::to_f32(src[ib]), c = tab[i], sn = tab[i + half];
    dst[ia] = T::round(x * c - y * sn);
    dst[ib] = T::round(y * c + x * sn);
  }
}

struct AttendArgs {
  Cache cache;
  Pages pages;
  const uint16_t *q;
  int64_t q_stride;
  int q_heads;
  const int32_t *lens;
  float scale;
  int window;
  uint16_t *out;
  float *lse;
};

// One block of 4 warps per sequence and query head: every warp takes each
// fourth token with its own running maximum and sum; joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(128) kv_attend_kernel(AttendArgs a, unsigned int *__restrict__ status) {
  constexpr int V = D / 32;
  __shared__ float part[4][D + 2];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.x / a.q_heads, h = blockIdx.x % a.q_heads;
  const int kvh = h / (a.q_heads / a.cache.heads);
  const int64_t room = static_cast<int64_t>(a.pages.max_pages) * a.cache.page_size;
  int64_t len = a.lens[b];
  if (len > room) {
    len = room;
    if (threadIdx.x == 0) atomicOr(status, W4A4_DEV_RANGE);
  }
  const int64_t first = a.window && len > a.window ? len - a.window : 0;
  float q[V], acc[V], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < V; ++i) {
    q[i] = T::to_f32(a.q[b * a.q_stride + h * D + lane + 32 * i]);
    acc[i] = 0.0f;
  }
  for (int64_t t = first + warp; t < len; t += 4) {
    const int page = a.pages.table[b * static_cast<int64_t>(a.pages.max_pages) + t / a.cache.page_size];
    if (page < 0 || page >= a.cache.n_pages) {
      if (lane == 0) atomicOr(status, W4A4_DEV_RANGE);
      continue;
    }
    const int64_t at = page * a.cache.stride_page + (t % a.cache.page_size) * a.cache.stride_token +
                       kvh * a.cache.stride_head + lane;
    float s = 0.0f;
    for (int i = 0; i < V; ++i) s = fmaf(q[i], T::to_f32(a.cache.k[at + 32 * i]), s);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.0f : mn;
    const float keep = expf(m - base), p = expf(s - base);
    l = l * keep + p;
    for (int i = 0; i < V; ++i) acc[i] = acc[i] * keep + p * T::to_f32(a.cache.v[at + 32 * i]);
    m = mn;
  }
  for (int i = 0; i < V; ++i) part[warp][lane + 32 * i] = acc[i];
  if (lane == 0) {
    part[warp][D] = m;
    part[warp][D + 1] = l;
  }
  __syncthreads();
  float top = -INFINITY, total = 0.0f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, part[w][D]);
  const float base = top == -INFINITY ? 0.0f : top;
  float f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = expf(part[w][D] - base);
    total += f[w] * part[w][D + 1];
  }
  for (int d = threadIdx.x; d < D; d += 128) {
    float o = 0.0f;
    for (int w = 0; w < 4; ++w) o += f[w] * part[w][d];
    a.out[(static_cast<int64_t>(b) * a.q_heads + h) * D + d] = T::round(total == 0.0f ? 0.0f : o / total);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[static_cast<int64_t>(b) * a.q_heads + h] = total == 0.0f ? -INFINITY : base + logf(total);
}

w4a4_status check_cache(const w4a4_kv_cache_t *c, Cache *out) {
  if (!c) return W4A4_ERR_ARG;
  if ((c->flags & ~W4A4_FLAG_FP16) || (c->head_dim != 64 && c->head_dim != 128)) return W4A4_ERR_UNSUPPORTED;
  if (c->n_pages < 0 || c->n_pages >= (int64_t(1) << 31) || c->page_size < 1 || c->n_heads < 1 || c->n_heads > 65535)
    return W4A4_ERR_SHAPE;
  const int64_t strides[3] = {c->stride_page, c->stride_token, c->stride_head};
  for (int64_t s : strides) {
    if (s < 0) return W4A4_ERR_SHAPE;
    if (s % 8) return W4A4_ERR_ALIGN;
  }
  if (c->n_pages && (!c->k || !c->v)) return W4A4_ERR_ARG;
  if (!ptr_aligned16(c->k) || !ptr_aligned16(c->v)) return W4A4_ERR_ALIGN;
  *out = {c->k, c->v, static_cast<int>(c->n_pages), c->page_size, c->n_heads,
          c->stride_page, c->stride_token, c->stride_head};
  return W4A4_OK;
}

w4a4_status check_pages(const int32_t *pages, int32_t n_seqs, int32_t max_pages) {
  if (n_seqs < 0 || max_pages < 0 || static_cast<int64_t>(n_seqs) * max_pages >= (int64_t(1) << 31))
    return W4A4_ERR_SHAPE;
  if (static_cast<int64_t>(n_seqs) * max_pages > 0 && !pages) return W4A4_ERR_ARG;
  return ptr_aligned4(pages) ? W4A4_OK : W4A4_ERR_ALIGN;
}

template <typename A>
w4a4_status launch(void (*kern)(A, unsigned int *), int64_t grid, int threads, const A &args, void *stream) {
  unsigned int *status = nullptr;
  if (status_word(&status) != cudaSuccess) return W4A4_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch_status(cudaLaunchKernelEx(&cfg, kern, args, status));
}

}  // namespace
}  // namespace w4a4

extern "C" {

w4a4_status w4a4_rope_table(int32_t n_pos, int32_t rot_dim, double base, float *table) {
  if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16) return W4A4_ERR_UNSUPPORTED;
  if (n_pos < 0) return W4A4_ERR_SHAPE;
  if (!(base > 0.0) || std::isinf(base)) return W4A4_ERR_ARG;
  if (n_pos && !table) return W4A4_ERR_ARG;
  const int half = rot_dim / 2;
  double freq[64];
  for (int i = 0; i < half; ++i) freq[i] = std::pow(base, -2.0 * i / rot_dim);
  for (int64_t p = 0; p < n_pos; ++p)
    for (int i = 0; i < half; ++i) {
      table[p * rot_dim + i] = static_cast<float>(std::cos(p * freq[i]));
      table[p * rot_dim + half + i] = static_cast<float>(std::sin(p * freq[i]));
    }
  return W4A4_OK;
}

w4a4_status w4a4_kv_append(const w4a4_kv_cache_t *cache, const uint16_t *k, int64_t k_stride, const uint16_t *v,
                           int64_t v_stride, const uint16_t *q, int64_t q_stride, int32_t n_q_heads,
                           uint16_t *q_out, int64_t T, const int32_t *pages, int32_t n_seqs, int32_t max_pages,
                           const int32_t *seq, const int32_t *pos, const float *table, int32_t n_table,
                           int32_t rot_dim, const int32_t *table_pos, uint32_t flags, void *stream) {
  using namespace w4a4;
  AppendArgs a = {};
  w4a4_status st = check_cache(cache, &a.cache);
  if (st != W4A4_OK) return st;
  if (flags & ~W4A4_FLAG_ROPE_PAIRS) return W4A4_ERR_UNSUPPORTED;
  const int D = cache->head_dim;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 16) return W4A4_ERR_UNSUPPORTED;
  if (T < 0 || T >= (int64_t(1) << 31) || n_table < 0 || (q && (n_q_heads < 1 || n_q_heads > 65535)))
    return W4A4_ERR_SHAPE;
  if ((st = check_pages(pages, n_seqs, max_pages)) != W4A4_OK) return st;
  if ((a.cache.n_pages > 1 && a.cache.stride_page == 0) || (a.cache.page_size > 1 && a.cache.stride_token == 0) ||
      (a.cache.heads > 1 && a.cache.stride_head == 0))
    return W4A4_ERR_SHAPE;
  if (T == 0) return W4A4_OK;
  if (!k || !v || !pos || (q && !q_out) || (rot_dim && n_table && !table)) return W4A4_ERR_ARG;
  if (k_stride < static_cast<int64_t>(a.cache.heads) * D || v_stride < static_cast<int64_t>(a.cache.heads) * D ||
      (q && q_stride < static_cast<int64_t>(n_q_heads) * D))
    return W4A4_ERR_SHAPE;
  if (q && q == q_out && q_stride != static_cast<int64_t>(n_q_heads) * D) return W4A4_ERR_ARG;
  if (!ptr_aligned16(k) || !ptr_aligned16(v) || !ptr_aligned16(q) || (q && !ptr_aligned16(q_out)) ||
      !ptr_aligned16(table) || !ptr_aligned4(seq) || !ptr_aligned4(pos) || !ptr_aligned4(table_pos) || k_stride % 8 || v_stride % 8 || (q && q_stride % 8))
    return W4A4_ERR_ALIGN;
  a.pages = {pages, n_seqs, max_pages};
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_heads = q ? n_q_heads : 0;
  a.head_dim = D;
  a.rot_dim = rot_dim;
  a.n_table = n_table;
  a.seq = seq;
  a.pos = pos;
  a.table_pos = table_pos;
  a.table = table;
  a.pairs = (flags & W4A4_FLAG_ROPE_PAIRS) != 0;
  return launch((cache->flags & W4A4_FLAG_FP16) ? kv_append_kernel<Fp16> : kv_append_kernel<Bf16>, T, 128, a, stream);
}

size_t w4a4_kv_attend_workspace_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_seqs < 0 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || (head_dim != 64 && head_dim != 128))
    return 0;
  return 256;
}

w4a4_status w4a4_kv_attend(const uint16_t *q, int64_t q_stride, int32_t n_q_heads, const w4a4_kv_cache_t *cache,
                           const int32_t *pages, int32_t n_seqs, int32_t max_pages, const int32_t *lens,
                           float scale, int32_t window, uint16_t *out, float *lse, void *workspace,
                           size_t workspace_bytes, void *stream) {
  using namespace w4a4;
  AttendArgs a = {};
  w4a4_status st = check_cache(cache, &a.cache);
  if (st != W4A4_OK) return st;
  const int D = cache->head_dim;
  if (n_q_heads < 1 || n_q_heads > 65535 || n_q_heads % a.cache.heads || window < 0) return W4A4_ERR_SHAPE;
  if ((st = check_pages(pages, n_seqs, max_pages)) != W4A4_OK) return st;
  if (!std::isfinite(scale)) return W4A4_ERR_ARG;
  if (n_seqs == 0) return W4A4_OK;
  if (!q || !lens || !out || !workspace) return W4A4_ERR_ARG;
  if (q_stride < static_cast<int64_t>(n_q_heads) * D) return W4A4_ERR_SHAPE;
  if (workspace_bytes < w4a4_kv_attend_workspace_bytes(n_seqs, n_q_heads, a.cache.heads, D)) return W4A4_ERR_SHAPE;
  if (!ptr_aligned16(q) || !ptr_aligned4(lens) || !ptr_aligned16(out) || !ptr_aligned4(lse) ||
      !ptr_aligned16(workspace) || q_stride % 8)
    return W4A4_ERR_ALIGN;
  a.pages = {pages, n_seqs, max_pages};
  a.q = q;
  a.q_stride = q_stride;
  a.q_heads = n_q_heads;
  a.lens = lens;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.lse = lse;
  const bool fp16 = (cache->flags & W4A4_FLAG_FP16) != 0;
  const int64_t grid = static_cast<int64_t>(n_seqs) * n_q_heads;
  if (grid > 0x7FFFFFFF) return W4A4_ERR_SHAPE;
  auto kern = D == 64 ? (fp16 ? kv_attend_kernel<Fp16, 64> : kv_attend_kernel<Bf16, 64>)
                      : (fp16 ? kv_attend_kernel<Fp16, 128> : kv_attend_kernel<Bf16, 128>);
  return launch(kern, grid, 128, a, stream);
}

}  // extern "C"
