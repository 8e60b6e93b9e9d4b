// kv.cu -- the paged key-value cache (include/decode.h, w4a4_kv_*): new tokens
// rotated and appended, and one new token per sequence attending to what is
// cached.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ctxcache.h"
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

// Pairs of elements turned: (a, b) -> (a c - b s, b c + a s).  Halves: elements i of
// two 16-byte pieces, with 8 angles; neighbours: within one piece, with 4.
template <typename T>
__device__ __forceinline__ void turn_halves(uint4 &x, uint4 &y, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = T::lo(a[i]), a1 = T::hi(a[i]), b0 = T::lo(b[i]), b1 = T::hi(b[i]);
    a[i] = T::pack(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
    b[i] = T::pack(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
  y = make_uint4(b[0], b[1], b[2], b[3]);
}
template <typename T, int FIRST>
__device__ __forceinline__ void turn_neighbours(uint4 &x, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = T::lo(a[i]), a1 = T::hi(a[i]);
    a[i] = T::pack(a0 * c[FIRST + i] - a1 * s[FIRST + i], a1 * c[FIRST + i] + a0 * s[FIRST + i]);
  }
  x = make_uint4(a[0], a[1], a[2], a[3]);
}

__device__ __forceinline__ void load4(const float *from, float (&to)[8], int first) {
  const float4 v = *reinterpret_cast<const float4 *>(from);
  to[first] = v.x, to[first + 1] = v.y, to[first + 2] = v.z, to[first + 3] = v.w;
}

// ------------------------------------------------------------------- append
//
// Every byte of the new keys, values and queries is read and written once: bound by
// HBM for prompts, by the chain position -> page -> store for a few tokens.  A warp
// takes a token (or one of `parts` shares of its heads, where tokens are too few to
// fill the GPU).  A lane keeps two 16-byte pieces of the heads for good, where halves
// turn the two that turn together, so the token's cosines and sines are read once into
// registers, and goes over the heads in rounds of four whose loads are all in flight
// before the first store, and before the page is known.  The pieces of
// neighbouring lanes are neighbours in memory: with each lane's two pieces side by side
// every sector was written in two halves, 24.6 us instead of 22 for 5003 tokens of 128
// dims turned in part.  (One block per token, thread by thread over its elements, took 67
// us for 8 frames; now 26, and 94 % of the copy rate on four times as many tokens.)
constexpr int kAppendWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_append_kernel(AppendArgs a, int64_t T_, int parts, unsigned int *__restrict__ status) {
  constexpr int kUnits = D / 16, kHeads = 32 / kUnits, kRound = 4;  // units of a head, heads of a pass
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int64_t t = id / parts;
  if (t >= T_) return;
  const int part = static_cast<int>(id % parts);
  const int u = lane % kUnits, hl = lane / kUnits;
  const int p = a.pos[t];
  if (p < 0) return;
  const int64_t s = a.seq ? a.seq[t] : t;
  const int64_t angle = a.table_pos ? a.table_pos[t] : p;
  const int entry = p / a.cache.page_size;
  int page = -1;
  if (s >= 0 && s < a.pages.n_seqs && entry < a.pages.max_pages) page = a.pages.table[s * a.pages.max_pages + entry];
  const bool in_table = a.rot_dim == 0 || (angle >= 0 && angle < a.n_table);
  // This lane's pieces of a head: elements e0 .. + 7 and e1 .. + 7, and whether they turn.
  const int half = a.rot_dim / 2;
  int e0 = 8 * u, e1 = D / 2 + 8 * u;
  bool turn0, turn1;
  float c[8], sn[8];
  const float *cosines = a.table + angle * a.rot_dim;
  if (a.pairs) {
    turn0 = e0 < a.rot_dim;
    turn1 = e1 < a.rot_dim;
    if (turn0 && in_table) load4(cosines + e0 / 2, c, 0), load4(cosines + half + e0 / 2, sn, 0);
    if (turn1 && in_table) load4(cosines + e1 / 2, c, 4), load4(cosines + half + e1 / 2, sn, 4);
  } else {
    const int units = a.rot_dim / 16;  // lanes u < units turn, the others copy what is left
    turn0 = turn1 = u < units;
    e0 = turn0 ? 8 * u : a.rot_dim + 8 * (u - units);
    e1 = e0 + (turn0 ? half : (D - a.rot_dim) / 2);
    if (turn0 && in_table) {
      load4(cosines + e0, c, 0), load4(cosines + e0 + 4, c, 4);
      load4(cosines + half + e0, sn, 0), load4(cosines + half + e0 + 4, sn, 4);
    }
  }
  // heads in the order keys, queries, values
  const int Hk = a.cache.heads, Hq = a.q_heads, total = 2 * Hk + Hq;
  const int64_t row = page * a.cache.stride_page + (p - entry * a.cache.page_size) * a.cache.stride_token;
  const bool ok = page >= 0 && page < a.cache.n_pages && in_table;
  if (!ok) {
    if (lane == 0) atomicOr(status, W4A4_DEV_RANGE);
    return;
  }
  for (int h0 = part * kHeads * kRound; h0 < total; h0 += parts * kHeads * kRound) {
    uint4 x[kRound], y[kRound];
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const int h = h0 + i * kHeads + hl;
      if (h < total) {
        const bool value = h >= Hk + Hq;
        const uint16_t *src = h < Hk ? a.k + t * a.k_stride + h * D
                              : value ? a.v + t * a.v_stride + (h - Hk - Hq) * D
                                      : a.q + t * a.q_stride + (h - Hk) * D;
        x[i] = *reinterpret_cast<const uint4 *>(src + (value ? 8 * u : e0));
        y[i] = *reinterpret_cast<const uint4 *>(src + (value ? D / 2 + 8 * u : e1));
      }
    }
#pragma unroll
    for (int i = 0; i < kRound; ++i) {
      const int h = h0 + i * kHeads + hl;
      if (h < total) {
        const bool value = h >= Hk + Hq;
        if (!value) {
          if (a.pairs) {
            if (turn0) turn_neighbours<T, 0>(x[i], c, sn);
            if (turn1) turn_neighbours<T, 4>(y[i], c, sn);
          } else if (turn0) {
            turn_halves<T>(x[i], y[i], c, sn);
          }
        }
        uint16_t *dst = h < Hk ? a.cache.k + row + h * a.cache.stride_head
                        : value ? a.cache.v + row + (h - Hk - Hq) * a.cache.stride_head
                                : a.q_out + (t * Hq + (h - Hk)) * D;
        *reinterpret_cast<uint4 *>(dst + (value ? 8 * u : e0)) = x[i];
        *reinterpret_cast<uint4 *>(dst + (value ? D / 2 + 8 * u : e1)) = y[i];
      }
    }
  }
}

// ------------------------------------------------------------------- attend
//
// out[b, h] = sum_t p_t V[t], p = softmax_t(scale q.K[t]).  Every cached token
// is read once, 4 D bytes per cache head, and used for 4 D flops per query head
// that shares it: bound by HBM for any usual number of shared heads, so the
// design is about keeping reads in flight.
//
//  * The work is the concatenation, over sequences, cache heads and chunks of up
//    to 16 of the heads that share one, of tiles of 64 tokens.  The lengths are on
//    the device, so every block of a grid that fills the GPU once adds them up
//    and takes an equal share of that line: a long sequence is split over
//    as many blocks as it needs, short ones share a block.  A block finishes
//    the items that lie inside its share; of an item that it shares with other
//    blocks it leaves maximum, sum and unnormalised output in the workspace
//    (two at most: its first and its last), and kv_join_kernel joins those.
//  * A warp works alone on 16 tokens at a time, through its own ring of
//    stages filled by 16-byte asynchronous copies: no block-wide wait inside an
//    item, and rows are addressed one by one, so pages may have any size.  Rows
//    without a token are filled with zeros by the copy itself.
//  * The products are m16n8k16 tensor-core instructions (a tile has at most 16
//    rows of queries, so tcgen05's 128-row tiles would be nearly empty, and at
//    HBM's pace these take a quarter of the tensor pipe).  Scores: A = queries (heads
//    x dims), B = keys.  Its accumulator holds for head lane / 4 two neighbouring
//    tokens per register pair, which is the B operand (tokens x heads) of the second
//    product with A = V^T (dims x tokens): the weights never leave their lane.
//    The order of dims inside a product is free as long as both operands share it,
//    so a lane's operands are 16-byte pieces of rows as they lie in memory.
//  * Weights enter the second product as two 16-bit terms (hi + lo, 2^-16 or
//    better): one term would put an error of half a bf16 step on every weight,
//    as large as the rounding of the result.

constexpr int kAttendWarps = 4;
constexpr int kTile = 64;            // tokens of a block's tile: 16 per warp
constexpr int kMaxBlocks = 640;      // partial results in the workspace: 2 per block
constexpr int kChunk = 16;           // most query heads of a block's item

constexpr int attend_stages(int D) { return D == 64 ? 5 : 2; }

struct AttendArgs {
  Cache cache;
  Pages pages;
  const uint16_t *q;
  int64_t q_stride;
  int q_heads, group;                // query heads, and how many share a cache head
  int chunks, chunk;                 // chunks of a group, heads of a chunk
  uint32_t div_mul;                  // t / page_size = (t * div_mul) >> div_shift, t < 2^31
  int div_shift;
  const int32_t *lens;
  float scale_log2;                  // scale * log2(e): the softmax runs in powers of two
  int window;
  uint16_t *out;
  float *lse;
  float *part;                       // [blocks][2][chunk][D + 4]: output, maximum, sum
  int4 *joins;                       // [blocks]: item and last block of a shared item, by its first block
};

// Tokens [first, end) of sequence b.
__device__ __forceinline__ void token_range(const AttendArgs &a, int b, int &first, int &end, bool &over) {
  const int room = a.pages.max_pages * a.cache.page_size;  // at most 2^30
  const int len = a.lens[b];
  over = len > room;
  end = over ? room : max(len, 0);
  first = a.window && end > a.window ? end - a.window : 0;
}

__device__ __forceinline__ int tiles_of(const AttendArgs &a, int b) {
  int first, end;
  bool over;
  token_range(a, b, first, end, over);
  return (end - first + kTile - 1) / kTile;
}

// Position of 16-byte piece `piece` of row `row` in a stage: the pieces of a
// row are exchanged so that the 8 lanes of a shared-memory phase hit different
// banks in all three accesses: the copies (one row), the keys (rows 2 i and
// 2 i + 1, pieces 0..3 or 4..7) and the values (every other of 8 rows, pieces 2 i
// and 2 i + 1).
__device__ __forceinline__ int swizzle(int row, int piece) { return piece ^ ((row & 6) ^ ((row & 1) << 2)); }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
  const int bytes = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a / b without the cost of a 64-bit division where 32 bits do
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Four output elements from d on of query head h, and at d = 0 its lse.
template <typename T, int D>
__device__ __forceinline__ void write_out(const AttendArgs &a, int b, int h, int d, float4 o, float base, float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = static_cast<int64_t>(b) * a.q_heads + h;
  *reinterpret_cast<uint2 *>(a.out + at * D + d) = make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
  if (d == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (base + log2f(sum)) * 0.69314718055994531f;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kAttendWarps) kv_attend_kernel(AttendArgs a, unsigned int *__restrict__ status) {
  constexpr int kStages = attend_stages(D);
  constexpr int kRow = 2 * D;                 // bytes of a row
  constexpr int kStage = 2 * 16 * kRow;       // 16 keys, 16 values
  constexpr int kPieces = D / 8;
  constexpr int kRowsPer = 32 / kPieces;      // rows that one copy instruction of a warp covers
  constexpr int kPart = D + 4;                // floats of a partial result
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t live_rows[kAttendWarps][kStages];
  __shared__ int64_t sums[kAttendWarps + 1];
  __shared__ int64_t found[2];                // start of the sequence that the share begins in, its number
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int B = a.pages.n_seqs;
  const int per_seq = a.cache.heads * a.chunks;  // items of a sequence

  // The line of tiles.  Up to 32 sequences every warp adds up for itself, one per lane;
  // of more, every thread of the block adds up a run.
  const bool few = B <= 32;
  const int run = few ? 1 : (B + 127) / 128, run0 = few ? lane : tid * run;
  int64_t mine = 0;
  for (int i = run0; i < min(B, run0 + run); ++i) {
    int first, end;
    bool over;
    token_range(a, i, first, end, over);
    if (over && blockIdx.x == 0) atomicOr(status, W4A4_DEV_RANGE);
    mine += static_cast<int64_t>((end - first + kTile - 1) / kTile) * per_seq;
  }
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  int64_t total = __shfl_sync(0xffffffffu, upto, 31);
  if (!few) {
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kAttendWarps; ++w) {
      if (w < warp) upto += sums[w];
      total += sums[w];
    }
  }
  // Nothing to attend to: zeros, spread over the blocks.
  for (int i = blockIdx.x; i < B; i += gridDim.x)
    if (tiles_of(a, i) == 0) {
      for (int j = tid; j < a.q_heads * D / 8; j += 128)
        reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(i) * a.q_heads * D)[j] = make_uint4(0u, 0u, 0u, 0u);
      if (a.lse)
        for (int j = tid; j < a.q_heads; j += 128) a.lse[static_cast<int64_t>(i) * a.q_heads + j] = -INFINITY;
    }
  const int64_t blocks = total < gridDim.x ? total : gridDim.x;  // no share is empty
  if (blockIdx.x >= blocks) {
    if (tid == 0) a.joins[blockIdx.x].x = -1;
    return;
  }
  // equal shares, the first `more` blocks one tile more
  const int64_t share = div_small(total, blocks), more = total - share * blocks;
  const int64_t begin = blockIdx.x * share + min(static_cast<int64_t>(blockIdx.x), more);
  const int64_t stop = begin + share + (blockIdx.x < more ? 1 : 0);
  // the sequence that the share begins in, and where that begins
  int b;
  int64_t seq_at;
  if (few) {
    b = __ffs(__ballot_sync(0xffffffffu, begin < upto)) - 1;
    seq_at = __shfl_sync(0xffffffffu, upto - mine, b);
  } else {
    if (upto - mine <= begin && begin < upto) {
      int64_t at = upto - mine;
      int i = run0;
      for (;; ++i) {
        const int64_t n = static_cast<int64_t>(tiles_of(a, i)) * per_seq;
        if (begin < at + n) break;
        at += n;
      }
      found[0] = at;
      found[1] = i;
    }
    __syncthreads();
    seq_at = found[0];
    b = static_cast<int>(found[1]);
  }
  bool absent = false;
  int4 join = make_int4(-1, 0, 0, 0);

  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  for (int64_t u = begin; u < stop;) {
    int first, end;
    bool over;
    token_range(a, b, first, end, over);
    const int tiles = (end - first + kTile - 1) / kTile;
    if (u >= seq_at + static_cast<int64_t>(tiles) * per_seq) {  // the next sequence
      seq_at += static_cast<int64_t>(tiles) * per_seq;
      ++b;
      continue;
    }
    const int item = static_cast<int>(div_small(u - seq_at, tiles));
    const int t0 = static_cast<int>(u - seq_at - static_cast<int64_t>(item) * tiles);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + (stop - u)));
    const int kvh = item / a.chunks;
    const int h0 = (item % a.chunks) * a.chunk;            // first head of the chunk, in its group
    const int heads = min(a.chunk, a.group - h0);
    const uint16_t *qrow = a.q + b * a.q_stride + static_cast<int64_t>(kvh * a.group + h0) * D;
    const int from = first + t0 * kTile, to = min(end, first + t1 * kTile);
    const int subs = (to - from + 15) / 16;                // 16-token pieces; this warp: warp, warp + 4, ...

    // The row of token from + 16 i + lane % 16 in the cache, or -1.
    const int32_t *table = a.pages.table + static_cast<int64_t>(b) * a.pages.max_pages;
    auto row_of = [&](int i) -> int64_t {
      const int t = from + 16 * i + (lane & 15);
      if (t >= to || t < from) return -1;
      const int entry = static_cast<int>((static_cast<uint64_t>(t) * a.div_mul) >> a.div_shift);
      const int page = __ldg(table + entry);
      if (page < 0 || page >= a.cache.n_pages) {
        absent = true;
        return -1;
      }
      return page * a.cache.stride_page + (t - entry * a.cache.page_size) * a.cache.stride_token;
    };
    const uint16_t *kbase = a.cache.k + kvh * a.cache.stride_head;
    const uint16_t *vbase = a.cache.v + kvh * a.cache.stride_head;
    auto fill = [&](int stage, int64_t row) {
      const uint32_t dst = ring + stage * kStage;
      const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) live_rows[warp][stage] = live & 0xFFFFu;
#pragma unroll
      for (int i = 0; i < 16 / kRowsPer; ++i) {
        const int rr = i * kRowsPer + lane / kPieces, piece = lane % kPieces;
        const int64_t off = __shfl_sync(0xffffffffu, row, rr);
        const bool ok = off >= 0;
        const int64_t at = off + piece * 8;
        const uint32_t to_ = dst + rr * kRow + swizzle(rr, piece) * 16;
        copy16(to_, ok ? kbase + at : a.q, ok);
        copy16(to_ + 16 * kRow, ok ? vbase + at : a.q, ok);
      }
    };
    int ahead = warp;                                       // next piece to fill
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s) {
      if (ahead < subs) fill(s, row_of(ahead));
      copy_commit();
      ahead += kAttendWarps;
    }
    int64_t next_row = ahead < subs ? row_of(ahead) : -1;

    // queries: pieces c, c + 4, ... of rows r and r + 8, as the keys' lanes read theirs
    uint4 q0[D / 32], q1[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      q0[j] = r < heads ? *reinterpret_cast<const uint4 *>(qrow + r * D + 8 * (c + 4 * j)) : make_uint4(0u, 0u, 0u, 0u);
      q1[j] = NT == 2 && r + 8 < heads ? *reinterpret_cast<const uint4 *>(qrow + (r + 8) * D + 8 * (c + 4 * j))
                                       : make_uint4(0u, 0u, 0u, 0u);
    }
    float acc[NT][D / 16][4];
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n] = -INFINITY;
      l[n] = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.0f;
    }

    int stage = 0;
    for (int sub = warp; sub < subs; sub += kAttendWarps) {
      copy_wait<kStages - 2>();
      __syncwarp();
      // the stage that was read last round takes the piece kStages - 1 ahead
      {
        const int s = stage == 0 ? kStages - 1 : stage - 1;
        if (ahead < subs) fill(s, next_row);
        copy_commit();
        ahead += kAttendWarps;
        next_row = ahead < subs ? row_of(ahead) : -1;
      }
      const uint32_t keys = ring + stage * kStage, values = keys + 16 * kRow;
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
        const int row = 8 * t + r;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 k = lds16(keys + row * kRow + swizzle(row, c + 4 * j) * 16);
          T::mma(s[t], q0[j].x, q1[j].x, q0[j].y, q1[j].y, k.x, k.y);
          T::mma(s[t], q0[j].z, q1[j].z, q0[j].w, q1[j].w, k.z, k.w);
        }
      }
      const uint32_t live = live_rows[warp][stage];
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[4] = {s[0][2 * n] * a.scale_log2, s[0][2 * n + 1] * a.scale_log2, s[1][2 * n] * a.scale_log2,
                      s[1][2 * n + 1] * a.scale_log2};
        if (live != 0xFFFFu) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((live >> (8 * (e >> 1) + 2 * c + (e & 1))) & 1u)) x[e] = -INFINITY;
        }
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[n], top);
        const float base = mn == -INFINITY ? 0.0f : mn;
        if (__any_sync(0xffffffffu, mn != m[n])) {
          const float keep = exp2f(m[n] - base);
          l[n] *= keep;
          // outputs lie by head 2 c, 2 c + 1: their factors are in the lanes of those heads
          const float k0 = __shfl_sync(0xffffffffu, keep, 8 * c), k1 = __shfl_sync(0xffffffffu, keep, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[n][i][0] *= k0;
            acc[n][i][1] *= k1;
            acc[n][i][2] *= k0;
            acc[n][i][3] *= k1;
          }
          m[n] = mn;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = ex2(x[e] - base);
        l[n] += (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          hi[n][t] = T::pack(x[2 * t], x[2 * t + 1]);
          lo[n][t] = T::pack(x[2 * t] - T::lo(hi[n][t]), x[2 * t + 1] - T::hi(hi[n][t]));
        }
      }
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * c + (i & 1) + 8 * (i >> 1);
          v[i] = lds16(values + row * kRow + swizzle(row, r + 8 * j) * 16);
        }
        const uint32_t w[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                  {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows of A: dims 64 j + 8 r + 2 i (lanes' first) and + 1; columns: tokens
          const uint32_t a0 = __byte_perm(w[0][i], w[1][i], 0x5410), a1 = __byte_perm(w[0][i], w[1][i], 0x7632);
          const uint32_t a2 = __byte_perm(w[2][i], w[3][i], 0x5410), a3 = __byte_perm(w[2][i], w[3][i], 0x7632);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            T::mma(acc[n][4 * j + i], a0, a1, a2, a3, hi[n][0], hi[n][1]);
            T::mma(acc[n][4 * j + i], a0, a1, a2, a3, lo[n][0], lo[n][1]);
          }
        }
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();                                        // the rings are free: they take the warps' results
    float *box = reinterpret_cast<float *>(smem);           // [warp][head][kPart]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
      if (c == 0) {
        box[(warp * 8 * NT + 8 * n + r) * kPart + D] = m[n];
        box[(warp * 8 * NT + 8 * n + r) * kPart + D + 1] = l[n];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2 *>(
              &box[(warp * 8 * NT + 8 * n + 2 * c + e) * kPart + 64 * (i / 4) + 8 * r + 2 * (i % 4)]) =
              make_float2(acc[n][i][e], acc[n][i][2 + e]);
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == tiles;
    const int slot = u == begin ? 0 : 1;
    for (int i = tid; i < heads * (D / 4); i += 128) {
      const int h = i / (D / 4), d = 4 * (i % (D / 4));
      float top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, box[(w * 8 * NT + h) * kPart + D]);
      const float base = top == -INFINITY ? 0.0f : top;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        const float *p = &box[(w * 8 * NT + h) * kPart];
        const float f = exp2f(p[D] - base);
        sum = fmaf(f, p[D + 1], sum);
        const float4 v = *reinterpret_cast<const float4 *>(p + d);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      if (whole) {
        write_out<T, D>(a, b, kvh * a.group + h0 + h, d, o, base, sum);
      } else {
        float *p = a.part + ((static_cast<int64_t>(blockIdx.x) * 2 + slot) * a.chunk + h) * kPart;
        *reinterpret_cast<float4 *>(p + d) = o;
        if (d == 0) *reinterpret_cast<float2 *>(p + D) = make_float2(top, sum);
      }
    }
    if (!whole && t0 == 0) {
      // the block that holds the item's last tile
      const int64_t last = u + tiles - 1, wide = more * (share + 1);
      join = make_int4(b, item, slot,
                       static_cast<int>(last < wide ? div_small(last, share + 1) : more + div_small(last - wide, share)));
    }
    __syncthreads();                                        // before the rings are filled again
    u += t1 - t0;
  }
  if (absent) atomicOr(status, W4A4_DEV_RANGE);
  if (tid == 0) a.joins[blockIdx.x] = join;
}

// One block per (block of the main kernel, head): where that block was the first of
// a shared item, the item's parts are joined, those of blocks first..last.  A lane takes 4 dims
// of every kGroups-th part with its own running maximum and sum, 8 parts in flight: after
// the wait three dependent reads remain.  Blocks without an item leave at once; all
// fit on the GPU together.  (A list of the shared items made by each block first, then a
// pass for the weights and one for the outputs, took 11 to 24 us.)
constexpr int kJoinThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(AttendArgs a) {
  constexpr int kPart = D + 4, kLanes = D / 4, kGroups = kJoinThreads / kLanes, kFlight = 8;
  __shared__ float4 box[kGroups][kLanes];
  __shared__ float2 stats[kGroups];
  griddep_launch_dependents();
  griddep_wait();
  const int lead = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int4 j = a.joins[lead];
  if (j.x < 0) return;
  const int kvh = j.y / a.chunks, h0 = (j.y % a.chunks) * a.chunk;
  if (h >= min(a.chunk, a.group - h0)) return;
  const int parts = j.w - lead + 1, g = tid / kLanes, d = 4 * (tid % kLanes);
  // this item's part is its first block's slot j.z, every later block's slot 0
  const float *first = a.part + ((static_cast<int64_t>(lead) * 2 + j.z) * a.chunk + h) * kPart;
  const float *later = a.part + (static_cast<int64_t>(lead) * 2 * a.chunk + h) * kPart;
  float m = -INFINITY, sum = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = g; i0 < parts; i0 += kGroups * kFlight) {
    float4 v[kFlight];
    float2 ml[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + f * kGroups;
      v[f] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      ml[f] = make_float2(-INFINITY, 0.0f);
      if (i < parts) {
        const float *p = i == 0 ? first : later + static_cast<int64_t>(i) * 2 * a.chunk * kPart;
        v[f] = *reinterpret_cast<const float4 *>(p + d);
        ml[f] = *reinterpret_cast<const float2 *>(p + D);
      }
    }
    float top = m;
#pragma unroll
    for (int f = 0; f < kFlight; ++f) top = fmaxf(top, ml[f].x);
    const float base = top == -INFINITY ? 0.0f : top, keep = exp2f(m - base);
    m = top;
    sum *= keep;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const float w = exp2f(ml[f].x - base);
      sum = fmaf(w, ml[f].y, sum);
      o.x = fmaf(w, v[f].x, o.x);
      o.y = fmaf(w, v[f].y, o.y);
      o.z = fmaf(w, v[f].z, o.z);
      o.w = fmaf(w, v[f].w, o.w);
    }
  }
  box[g][tid % kLanes] = o;
  if (tid % kLanes == 0) stats[g] = make_float2(m, sum);
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) m = fmaxf(m, stats[i].x);
  const float base = m == -INFINITY ? 0.0f : m;
  sum = 0.0f;
  o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float w = exp2f(stats[i].x - base);
    const float4 v = box[i][tid];
    sum = fmaf(w, stats[i].y, sum);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  write_out<T, D>(a, j.x, kvh * a.group + h0 + h, d, o, base, sum);
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

cudaLaunchConfig_t launch_config(int64_t grid, int threads, size_t smem, void *stream, cudaLaunchAttribute *attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

size_t part_bytes(int group, int D) {
  const int chunks = (group + kChunk - 1) / kChunk, chunk = (group + chunks - 1) / chunks;
  return static_cast<size_t>(kMaxBlocks) * 2 * chunk * (D + 4) * sizeof(float);
}

template <typename T, int D, int NT>
w4a4_status launch_attend(AttendArgs &a, void *stream) {
  constexpr int kStages = attend_stages(D);
  constexpr int kRing = kAttendWarps * kStages * 2 * 16 * 2 * D, kBox = kAttendWarps * 8 * NT * (D + 4) * 4;
  constexpr int kSmem = kRing > kBox ? kRing : kBox;
  static ContextCache<int> occupancy;  // per context: attribute set, blocks per SM
  int per_sm = 0;
  if (occupancy.get(&per_sm, [](int *v) {
        cudaError_t e = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kSmem);
        if (e == cudaSuccess)
          e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kv_attend_kernel<T, D, NT>, 32 * kAttendWarps, kSmem);
        return e;
      }) != cudaSuccess || per_sm < 1)
    return W4A4_ERR_CUDA;
  unsigned int *status = nullptr;
  if (status_word(&status) != cudaSuccess) return W4A4_ERR_CUDA;
  // blocks: one per place on the GPU, fewer when there cannot be that many tiles
  int64_t grid = static_cast<int64_t>(device_sm_count()) * per_sm;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  const int64_t tiles = (static_cast<int64_t>(a.pages.max_pages) * a.cache.page_size + kTile - 1) / kTile;
  const int64_t items = static_cast<int64_t>(a.pages.n_seqs) * a.cache.heads * a.chunks;
  if (tiles < grid && items < grid && items * tiles < grid) grid = items * tiles > 0 ? items * tiles : 1;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = launch_config(grid, 32 * kAttendWarps, kSmem, stream, &attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attend_kernel<T, D, NT>, a, status);
  // one block, or items of one tile: nothing is shared
  if (e != cudaSuccess || grid == 1 || tiles <= 1) return launch_status(e);
  cfg = launch_config(grid, kJoinThreads, 0, stream, &attr);
  cfg.gridDim.y = static_cast<unsigned>(a.chunk);
  return launch_status(cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D>, a));
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
  unsigned int *status = nullptr;
  if (status_word(&status) != cudaSuccess) return W4A4_ERR_CUDA;
  cudaLaunchAttribute attr;
  // shares of a token's heads (at most one per 4 passes of a warp) until there
  // are 8 warps per SM
  const int heads = 2 * a.cache.heads + a.q_heads, round = 4 * (32 / (D / 16)), most = (heads + round - 1) / round;
  const int64_t want = (8ll * device_sm_count() + T - 1) / T;
  const int parts = static_cast<int>(want < most ? want : most);
  const cudaLaunchConfig_t cfg =
      launch_config((T * parts + kAppendWarps - 1) / kAppendWarps, 32 * kAppendWarps, 0, stream, &attr);
  const bool fp16 = (cache->flags & W4A4_FLAG_FP16) != 0;
  auto kern = D == 64 ? (fp16 ? kv_append_kernel<Fp16, 64> : kv_append_kernel<Bf16, 64>)
                      : (fp16 ? kv_append_kernel<Fp16, 128> : kv_append_kernel<Bf16, 128>);
  return launch_status(cudaLaunchKernelEx(&cfg, kern, a, T, parts, status));
}

size_t w4a4_kv_attend_workspace_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_seqs < 0 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || (head_dim != 64 && head_dim != 128))
    return 0;
  return w4a4::part_bytes(n_q_heads / n_kv_heads, head_dim) + sizeof(int4) * w4a4::kMaxBlocks;
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
  if (static_cast<int64_t>(max_pages) * a.cache.page_size > (int64_t(1) << 30)) return W4A4_ERR_SHAPE;
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
  a.group = n_q_heads / a.cache.heads;
  a.chunks = (a.group + kChunk - 1) / kChunk;
  a.chunk = (a.group + a.chunks - 1) / a.chunks;
  int shift = 0;  // page_size <= 2^shift
  while ((int64_t(1) << shift) < a.cache.page_size) ++shift;
  a.div_shift = 31 + shift;
  a.div_mul = static_cast<uint32_t>((uint64_t(1) << a.div_shift) / a.cache.page_size + 1);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float *>(workspace);
  a.joins = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + part_bytes(a.group, D));
  const bool fp16 = (cache->flags & W4A4_FLAG_FP16) != 0, wide = a.chunk > 8;
  if (D == 64) {
    if (fp16) return wide ? launch_attend<Fp16, 64, 2>(a, stream) : launch_attend<Fp16, 64, 1>(a, stream);
    return wide ? launch_attend<Bf16, 64, 2>(a, stream) : launch_attend<Bf16, 64, 1>(a, stream);
  }
  if (fp16) return wide ? launch_attend<Fp16, 128, 2>(a, stream) : launch_attend<Fp16, 128, 1>(a, stream);
  return wide ? launch_attend<Bf16, 128, 2>(a, stream) : launch_attend<Bf16, 128, 1>(a, stream);
}

}  // extern "C"
