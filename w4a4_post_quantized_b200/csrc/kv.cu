// kv.cu -- the paged key-value cache (include/decode.h, w4a4_kv_*): new tokens
// rotated and appended, and one new token per sequence attending to what is
// cached.
#include <cuda_runtime.h>

#include <algorithm>
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
  int q_heads, rot_dim, n_table;
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
// registers, and goes over the heads in rounds of append_round passes whose loads are all in
// flight before the first store, and before the page is known.  The pieces of
// neighbouring lanes are neighbours in memory: with each lane's two pieces side by side
// every sector was written in two halves, 24.6 us instead of 22 for 5003 tokens of 128
// dims turned in part.  (One block per token, thread by thread over its elements, took 67
// us for 8 frames; now 25.0, 5.5 TB/s, and 77.8, 100 % of a copy's rate, on 40000 tokens.)
constexpr int kAppendWarps = 2;

// Passes of a round.  More are more loads in flight per warp, fewer leave registers for more
// warps: 8 frames (64 dims, 48 heads) 26.8 us with 4, 25.1 with 3, 26.2 with 2; 4000 tokens of
// 128 dims and 48 heads 22.4 with 4, 18.9 with 2.
constexpr int append_round(int D) { return D == 64 ? 3 : 2; }

template <typename T, int D>
__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_append_kernel(AppendArgs a, int64_t T_, int parts, unsigned int *__restrict__ status) {
  constexpr int kUnits = D / 16, kHeads = 32 / kUnits, kRound = append_round(D);  // units of a head, heads of a pass
  griddep_wait();
  griddep_launch_dependents();
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
//  * The warps of a block take neighbouring cache heads (4, 2 or 1, by what divides
//    their number) of the same tokens, so that a token's row is read in one go in whichever
//    order the cache holds tokens and heads; one head where rows are long and there is
//    little to do (w4a4_kv_attend has the rule).
//  * The work of such a team is the concatenation, over sequences, groups of heads and
//    chunks of up to 16 of the query heads that share one, of pieces of 16 tokens (of 32 at
//    64 dims; with 16 there 61.9 us instead of 57.6 for 64 frames).  The lengths are on the
//    device, so every block of a grid that fills the GPU once adds them up and each team
//    takes an equal share of that line: a long sequence is split over as many teams as it
//    needs, short ones share one.  A team finishes the items that lie inside its share; of an
//    item that it shares with others it leaves maximum, sum and unnormalised output in the
//    workspace (two at most: its first and its last), and kv_join_kernel joins those.  A
//    block whose teams all work on one item joins them first.
//  * A warp works alone, through its own ring of stages filled by 16-byte asynchronous
//    copies that run ahead across the ends of items: no block-wide wait anywhere.  A piece
//    that lies in one page is looked up once, one that does not row by row.  Rows
//    without a token are filled with zeros by the copy itself.
//  * Where the table leaves room for little (w4a4_kv_attend's launch has the rule), there is no line:
//    one cluster of up to 8 blocks takes each item, a piece or a few per warp, and its
//    blocks join their parts through distributed shared memory.  One launch instead of two.
//  * The products are m16n8k16 tensor-core instructions (a piece has at most 16
//    rows of queries, so tcgen05's 128-row tiles would be nearly empty, and at
//    HBM's pace these take a quarter of the tensor pipe).  Scores: A = queries (heads
//    x dims), B = keys.  Its accumulator holds for head lane / 4 two neighbouring
//    tokens per register pair, which is the B operand (tokens x heads) of the second
//    product with A = V^T (dims x tokens): the weights never leave their lane.
//    The order of dims inside a product is free as long as both operands share it,
//    so a lane's operands are 16-byte pieces of rows as they lie in memory.
//  * Weights enter the second product as two 16-bit terms, hi + lo, off by at most 2^-16 of the
//    weight: one term would put an error of half a bf16 step on every weight, as large as the
//    rounding of the result.  In fp16 the low term is a multiple of 2^-24, so the reference that is
//    subtracted from the scores lies kTop = 15 below their maximum: the error is then at most
//    2^-40 of the largest weight, which is more than 2^-16 of its own for weights below 2^-24 of the largest.
//    The total adds the weights as they were before.
//
// us, and the share of a copy's rate: 64 frames of one sequence (87936 tokens, 16 heads of 64)
// 57.8, 97 %; 64 sequences of 4160 to 8192 126, 99 %; 23 of 250 to 4001 and none 37.5, 78 %, where the
// wait for the first lengths, pages and rows and the join are what is left; one frame (1374 tokens) 7.2,
// all of it such waits.  In long ones issue slots are 34 %, the tensor pipe 21 % busy.

constexpr int kAttendWarps = 4;
constexpr int kMaxCluster = 8;       // blocks of a cluster (8 is what every launch may ask for)
constexpr int kMaxBlocks = 448;      // partial results in the workspace: two per warp
constexpr int kChunk = 16;           // most query heads of a warp's item (8: 66 us, not 54, for 16 sharing a head)
constexpr float kLog2e = 1.4426950408889634f;

constexpr int attend_piece(int D) { return D == 64 ? 32 : 16; }  // tokens of a stage: 8 KB of keys and values
// Stages of a warp's ring: with two, three blocks fit on an SM.  (Two blocks with three
// stages: 64 frames 62 us instead of 57.6, 64 sequences of 8k 131 instead of 127.)
constexpr int kAttendStages = 2;

struct AttendArgs {
  Cache cache;
  Pages pages;
  const uint16_t *q;
  int64_t q_stride;
  int q_heads, group;                // query heads, and how many share a cache head
  int chunks, chunk;                 // chunks of a group, heads of a chunk
  int team;                          // warps (cache heads) of a team: 4, 2 or 1
  uint32_t div_mul;                  // t / page_size = (t * div_mul) >> div_shift, t < 2^31
  int div_shift;
  const int32_t *lens;
  float scale_log2;                  // scale * log2(e): the softmax runs in powers of two
  int window;
  uint16_t *out;
  float *lse;
  float *part;                       // [teams][2][team][chunk][D + 4]: output, maximum, sum
  int cluster;                       // blocks that share an item, where the clusters' form runs

  // an item's group of heads and chunk
  __device__ __forceinline__ int heads_of(int item) const { return chunks == 1 ? item : item / chunks; }
  __device__ __forceinline__ int chunk_of(int item) const { return chunks == 1 ? 0 : item % chunks; }
};

// Equal shares of the line, the first `more` teams one piece more; none is empty.  (Places in
// the line are below 2^31, checked on the host: a 64-bit division takes half a microsecond.)
struct Shares {
  int teams, share, more;
  __device__ __forceinline__ Shares(int total, int most) {
    teams = min(total, most);
    share = teams ? total / teams : 0;
    more = total - share * teams;
  }
  __device__ __forceinline__ int begin(int team) const { return min(team, teams) * share + min(team, more); }
  // the team that holds a place in the line
  __device__ __forceinline__ int owner(int at) const {
    const int wide = more * (share + 1);
    return at < wide ? at / (share + 1) : more + (at - wide) / share;
  }
};

// The tokens of a sequence, [first, end), and its pieces, [p0, p0 + pieces).  FRESH: read past
// L1, where a kernel that has not waited might find what stood there before.
template <int P, bool FRESH = false>
struct Range {
  int first, end, p0, pieces;
  __device__ __forceinline__ Range(const AttendArgs &a, int b) {
    const int room = a.pages.max_pages * a.cache.page_size;  // at most 2^30
    end = min(max(FRESH ? __ldcg(a.lens + b) : a.lens[b], 0), room);
    first = a.window && end > a.window ? end - a.window : 0;
    p0 = first / P;
    pieces = (end + P - 1) / P - p0;
  }
};

// Position of 16-byte piece `piece` of row `row` in a stage: the pieces of a
// row are exchanged so that the 8 lanes of a shared-memory phase hit different
// banks in all three accesses: the copies (one row), the keys (rows 2 i and
// 2 i + 1, pieces 0..3 or 4..7) and the values (every other of 8 rows, pieces 2 i
// and 2 i + 1).
__device__ __forceinline__ int swizzle(int row, int piece) { return piece ^ ((row & 6) ^ ((row & 1) << 2)); }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {  // zeros unless live
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

// From another block's shared memory.
__device__ __forceinline__ float4 ld_cluster16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster8(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

// The logarithm of a sum of 2^x held as top and sum of 2^(x - top); top is any finite reference.
__device__ __forceinline__ float log_sum(float top, float sum) {
  return sum == 0.0f ? -INFINITY : ((top == -INFINITY ? 0.0f : top) + log2f(sum)) * 0.69314718055994531f;
}

// Four output elements from d on of query head h, and at d = 0 its lse.
template <typename T, int D>
__device__ __forceinline__ void write_out(const AttendArgs &a, int b, int h, int d, float4 o, float top, float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = static_cast<int64_t>(b) * a.q_heads + h;
  *reinterpret_cast<uint2 *>(a.out + at * D + d) = make_uint2(T::pack(o.x * inv, o.y * inv), T::pack(o.z * inv, o.w * inv));
  if (d == 0 && a.lse) a.lse[at] = log_sum(top, sum);
}

// Three blocks on an SM, two with the sums of 16 heads (168 registers a thread do not hold
// those at 128 dims; at 64 three blocks gain nothing, 31.6 us and 31.8).
//
// CLUSTER: an item is shared by the warps of one cluster of blocks, which join their parts
// through shared memory: one launch and no line, for calls with little to do.
template <typename T, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(32 * kAttendWarps, NT == 1 ? 3 : 2)
    kv_attend_kernel(AttendArgs a, unsigned int *__restrict__ status) {
  constexpr int P = attend_piece(D);
  constexpr int kStages = kAttendStages;
  constexpr int kRow = 2 * D;                 // bytes of a row
  constexpr int kStage = 2 * P * kRow;        // keys, then values
  constexpr int kPieces = D / 8;              // 16-byte pieces of a row
  constexpr int kRowsPer = 32 / kPieces;      // rows that one copy instruction of a warp covers
  constexpr int kCopies = P / kRowsPer;
  constexpr int kPart = D + 4;                // floats of a partial result
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t live_rows[kAttendWarps][kStages];
  __shared__ int sums[kAttendWarps];
  __shared__ int found[kAttendWarps][2];  // start of the sequence that a team's share begins in, its number
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int B = a.pages.n_seqs;
  const int per_seq = a.cache.heads / a.team * a.chunks;  // items of a sequence
  const int teams_here = kAttendWarps / a.team;
  const int team = blockIdx.x * teams_here + warp / a.team, member = warp % a.team;

  int b = 0, begin = 0, left = 0;              // the share's first sequence, place in the line, pieces
  int item = 0, piece = 0;                     // of that sequence, of that item: where it begins
  bool merged = false;                         // the block's teams all work on one item, and leave one part
  const int team0 = blockIdx.x * teams_here;
  if constexpr (CLUSTER) {
    const int index = blockIdx.x / a.cluster, w = (blockIdx.x - index * a.cluster) * kAttendWarps + warp;
    b = index / per_seq;
    item = index - b * per_seq;
    const Range<P> v(a, b);
    if (w == 0 && item == 0 && lane == 0 && a.lens[b] > v.end) atomicOr(status, W4A4_DEV_RANGE);
    const int warps = kAttendWarps * a.cluster, each = v.pieces / warps, more = v.pieces - each * warps;
    piece = w * each + min(w, more);
    left = each + (w < more ? 1 : 0);
  } else {
    // The line of pieces.  Up to 32 sequences every warp adds up for itself, one per lane;
    // of more, every thread of the block adds up a run.
    const bool few = B <= 32;
    const int run = few ? 1 : (B + 127) / 128, run0 = few ? lane : tid * run;
    int mine = 0;
    for (int i = run0; i < min(B, run0 + run); ++i) {
      const Range<P> v(a, i);
      if (blockIdx.x == 0 && a.lens[i] > v.end) atomicOr(status, W4A4_DEV_RANGE);
      mine += v.pieces * per_seq;
    }
    int upto = mine;
    for (int o = 1; o < min(B, 32); o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    int total = __shfl_sync(0xffffffffu, upto, min(B, 32) - 1);
    if (!few) {
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      total = 0;
      for (int w = 0; w < kAttendWarps; ++w) {
        if (w < warp) upto += sums[w];
        total += sums[w];
      }
    }
    const Shares shares(total, gridDim.x * teams_here);
    begin = shares.begin(team);
    left = team < shares.teams ? shares.begin(team + 1) - begin : 0;
    // The sequence that the share begins in, and where that begins.
    int off = 0;  // of the share in it
    if (few) {
      if (left) {
        b = __ffs(__ballot_sync(0xffffffffu, begin < upto)) - 1;
        off = begin - __shfl_sync(0xffffffffu, upto - mine, b);
      }
    } else {
      for (int t = 0; t < teams_here; ++t) {
        const int from = shares.begin(blockIdx.x * teams_here + t);
        if (upto - mine <= from && from < upto) {
          int at = upto - mine;
          int i = run0;
          for (;; ++i) {
            const int n = Range<P>(a, i).pieces * per_seq;
            if (from < at + n) break;
            at += n;
          }
          found[t][0] = at;
          found[t][1] = i;
        }
      }
      __syncthreads();
      if (left) {
        off = begin - found[warp / a.team][0];
        b = found[warp / a.team][1];
      }
    }
    // Nothing to attend to: zeros, spread over the warps.
    for (int i = blockIdx.x * kAttendWarps + warp; i < B; i += gridDim.x * kAttendWarps)
      if (Range<P>(a, i).pieces == 0) {
        for (int j = lane; j < a.q_heads * D / 8; j += 32)
          reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(i) * a.q_heads * D)[j] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse)
          for (int j = lane; j < a.q_heads; j += 32) a.lse[static_cast<int64_t>(i) * a.q_heads + j] = -INFINITY;
      }
    if (left == 0) return;
    const int pieces = Range<P>(a, b).pieces;
    item = off / pieces;
    piece = off - item * pieces;
    const int item_at = begin - piece;
    merged = teams_here > 1 && team0 + teams_here <= shares.teams && item_at <= shares.begin(team0) &&
             shares.begin(team0 + teams_here) <= item_at + pieces;
  }

  // ---- the copies' side: the next piece to look up, then its rows
  Range<P> cr(a, b);
  int cb = b, citem = item, cpiece = piece, cleft = left;
  Range<P> range = cr;
  const int64_t values = a.cache.v - a.cache.k;
  const int crow = lane / kPieces, cpos = lane % kPieces;
  bool absent = false, ready = false, one = false;
  // the piece that is looked up: of its first token, where one page holds all of it, or of
  // token lane % P the page, and the place without the page's; a page is not used before the copies, a round later
  int look_t0 = 0, look_lo = 0, look_hi = 0, page = -1;  // tokens look_t0 + look_lo .. look_hi - 1 are there
  int64_t rest = 0;
  auto look_up = [&]() {
    ready = cleft > 0;
    if (!ready) return;
    if (cpiece == cr.pieces) {
      cpiece = 0;
      if (++citem == per_seq) {
        citem = 0;
        do cr = Range<P>(a, ++cb);
        while (cr.pieces == 0);
      }
    }
    look_t0 = (cr.p0 + cpiece) * P;
    int t = look_t0;
    int entry = static_cast<int>((static_cast<uint64_t>(t) * a.div_mul) >> a.div_shift);
    one = t - entry * a.cache.page_size + P <= a.cache.page_size;
    if (!one) {
      t += lane % P;
      entry = static_cast<int>((static_cast<uint64_t>(t) * a.div_mul) >> a.div_shift);
    }
    page = -1;
    if (one || (t >= cr.first && t < cr.end))
      page = a.pages.table[static_cast<int64_t>(cb) * a.pages.max_pages + entry];
    rest = static_cast<int64_t>(a.heads_of(citem) * a.team + member) * a.cache.stride_head +
           (t - entry * a.cache.page_size) * a.cache.stride_token;
    look_lo = max(cr.first - look_t0, 0);
    look_hi = min(cr.end - look_t0, P);
    ++cpiece;
    --cleft;
  };
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  constexpr uint32_t kAll = 0xFFFFFFFFu >> (32 - P);
  auto fill = [&](int stage) {
    if (ready) {
      const uint32_t dst = ring + stage * kStage;
      const bool ok = page >= 0 && page < a.cache.n_pages;
      const int64_t row = rest + page * a.cache.stride_page;
      uint32_t live = (kAll >> (P - look_hi)) & (kAll << look_lo);
      if (one) {
        if (!ok) absent = true, live = 0;
      } else {
        const uint32_t found = __ballot_sync(0xffffffffu, ok);
        if (live & ~found) absent = true;
        live &= found;
      }
      if (lane == 0) live_rows[warp][stage] = live;
      if (one && live == kAll) {
        const uint16_t *k = a.cache.k + row + crow * a.cache.stride_token + 8 * cpos;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int rr = i * kRowsPer + crow;
          const uint32_t to = dst + rr * kRow + swizzle(rr, cpos) * 16;
          copy16(to, k);
          copy16(to + P * kRow, k + values);
          k += kRowsPer * a.cache.stride_token;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
          const int rr = i * kRowsPer + crow;
          const int64_t of = one ? row + rr * a.cache.stride_token : __shfl_sync(0xffffffffu, row, rr);
          const bool there = (live >> rr) & 1u;
          const uint16_t *k = a.cache.k + of + 8 * cpos;
          const uint32_t to = dst + rr * kRow + swizzle(rr, cpos) * 16;
          copy16(to, there ? k : a.q, there);
          copy16(to + P * kRow, there ? k + values : a.q, there);
        }
      }
    }
    copy_commit();
  };
  look_up();
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) {
    fill(s);
    look_up();
  }

  // ---- the products' side
  int stage = 0;
  bool at_begin = true;
  while (left > 0) {
    if (piece == range.pieces) {
      piece = 0;
      if (++item == per_seq) {
        item = 0;
        do range = Range<P>(a, ++b);
        while (range.pieces == 0);
      }
    }
    const int n_here = min(range.pieces - piece, left);
    const int kvh = a.heads_of(item) * a.team + member;
    const int h0 = a.chunk_of(item) * a.chunk;             // first head of the chunk, in its group
    const int heads = min(a.chunk, a.group - h0);
    const int64_t head0 = static_cast<int64_t>(kvh) * a.group + h0;
    const uint16_t *qrow = a.q + b * a.q_stride + head0 * D;

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

    for (int k = 0; k < n_here; ++k) {
      copy_wait<kStages - 2>();
      __syncwarp();
      fill(stage == 0 ? kStages - 1 : stage - 1);           // the stage that was read last
      look_up();
      const uint32_t keys = ring + stage * kStage, vals = keys + P * kRow;
      float s[P / 8][4];
#pragma unroll
      for (int t = 0; t < P / 8; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
        const int rr = 8 * t + r;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = lds16(keys + rr * kRow + swizzle(rr, c + 4 * j) * 16);
          T::mma(s[t], q0[j].x, q1[j].x, q0[j].y, q1[j].y, x.x, x.y);
          T::mma(s[t], q0[j].z, q1[j].z, q0[j].w, q1[j].w, x.z, x.w);
        }
      }
      const uint32_t lv = live_rows[warp][stage];
      uint32_t hi[NT][P / 8], lo[NT][P / 8];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[P / 4];
#pragma unroll
        for (int e = 0; e < P / 4; ++e) x[e] = s[e / 2][2 * n + e % 2] * a.scale_log2;
        if (lv != kAll) {
#pragma unroll
          for (int e = 0; e < P / 4; ++e)
            if (!((lv >> (8 * (e / 2) + 2 * c + e % 2)) & 1u)) x[e] = -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < P / 4; ++e) top = fmaxf(top, x[e]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[n], top - T::kTop);
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
        for (int e = 0; e < P / 4; ++e) {
          x[e] = ex2(x[e] - base);
          l[n] += x[e];
        }
#pragma unroll
        for (int t = 0; t < P / 8; ++t) {
          hi[n][t] = T::pack(x[2 * t], x[2 * t + 1]);
          lo[n][t] = T::pack(x[2 * t] - T::lo(hi[n][t]), x[2 * t + 1] - T::hi(hi[n][t]));
        }
      }
#pragma unroll
      for (int t = 0; t < P / 16; ++t)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 16 * t + 2 * c + (i & 1) + 8 * (i >> 1);
            v[i] = lds16(vals + rr * kRow + swizzle(rr, r + 8 * j) * 16);
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
              T::mma(acc[n][4 * j + i], a0, a1, a2, a3, hi[n][2 * t], hi[n][2 * t + 1]);
              T::mma(acc[n][4 * j + i], a0, a1, a2, a3, lo[n][2 * t], lo[n][2 * t + 1]);
            }
          }
        }
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

    // The item, or this team's part of it, is done.  A lane holds dims 64 j + 8 r .. + 7 of
    // heads 2 c and 2 c + 1 (+ 8 n).
    const bool whole_item = !CLUSTER && !merged && piece == 0 && n_here == range.pieces;
    const int slot = at_begin ? 0 : 1;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * c + e;
        const float sum = __shfl_sync(0xffffffffu, l[n], 8 * c + 4 * e), top = __shfl_sync(0xffffffffu, m[n], 8 * c + 4 * e);
        if (h >= heads) continue;
        if (whole_item) {
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          const int64_t at = static_cast<int64_t>(b) * a.q_heads + head0 + h;
#pragma unroll
          for (int j = 0; j < D / 64; ++j)
            *reinterpret_cast<uint4 *>(a.out + at * D + 64 * j + 8 * r) =
                make_uint4(T::pack(acc[n][4 * j][e] * inv, acc[n][4 * j][2 + e] * inv),
                           T::pack(acc[n][4 * j + 1][e] * inv, acc[n][4 * j + 1][2 + e] * inv),
                           T::pack(acc[n][4 * j + 2][e] * inv, acc[n][4 * j + 2][2 + e] * inv),
                           T::pack(acc[n][4 * j + 3][e] * inv, acc[n][4 * j + 3][2 + e] * inv));
          if (r == 0 && a.lse) a.lse[at] = log_sum(top, sum);
        } else {
          float *p = CLUSTER || merged ? reinterpret_cast<float *>(smem + warp * kStages * kStage) + h * kPart
                            : a.part + (((static_cast<int64_t>(team) * 2 + slot) * a.team + member) * a.chunk + h) * kPart;
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            float4 *o = reinterpret_cast<float4 *>(p + 64 * j + 8 * r);
            o[0] = make_float4(acc[n][4 * j][e], acc[n][4 * j][2 + e], acc[n][4 * j + 1][e], acc[n][4 * j + 1][2 + e]);
            o[1] = make_float4(acc[n][4 * j + 2][e], acc[n][4 * j + 2][2 + e], acc[n][4 * j + 3][e],
                               acc[n][4 * j + 3][2 + e]);
          }
          if (r == 0) *reinterpret_cast<float2 *>(p + D) = make_float2(top, sum);
        }
      }
    }
    at_begin = false;
    left -= n_here;
    piece += n_here;
  }
  if (absent) atomicOr(status, W4A4_DEV_RANGE);
  if constexpr (CLUSTER) {
    const int h0 = a.chunk_of(item) * a.chunk, heads = min(a.chunk, a.group - h0);
    auto part = [&](int t, int h) { return smem + (t % kAttendWarps) * kStages * kStage + h * kPart * 4; };
    if (at_begin && lane < heads)  // no share
      *reinterpret_cast<float2 *>(part(warp, lane) + 4 * D) = make_float2(-INFINITY, 0.0f);
    __syncwarp();
    cluster_sync();
    // Block `rank` writes dims rank * 4 q .. + 4 q - 1 of every head, a warp per head: lane t has the
    // weight of part t, lanes j of q the dims 4 j of every kGroups-th part.
    const int rank = cluster_ctarank(), q = D / 4 / a.cluster, groups = 32 / q;
    const int j = lane % q, g = lane / q, d = 4 * (rank * q + j);
    for (int h = warp; h < heads; h += kAttendWarps) {
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (lane < kAttendWarps * a.cluster) ml = ld_cluster8(cluster_addr(part(lane, h) + 4 * D, lane / kAttendWarps));
      float4 v[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int t = g + i * groups;
        v[i] = ld_cluster16(cluster_addr(part(t, h) + 4 * d, t / kAttendWarps));
      }
      float top = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float f = exp2f(ml.x - (top == -INFINITY ? 0.0f : top));
      float sum = ml.y == 0.0f ? 0.0f : f * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      float4 o4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const int t = g + i * groups;
        const float w = __shfl_sync(0xffffffffu, f, t);
        if (w != 0.0f) {  // what an empty part holds may be anything
          o4.x = fmaf(w, v[i].x, o4.x);
          o4.y = fmaf(w, v[i].y, o4.y);
          o4.z = fmaf(w, v[i].z, o4.z);
          o4.w = fmaf(w, v[i].w, o4.w);
        }
      }
      for (int o = q; o < 32; o <<= 1) {
        o4.x += __shfl_xor_sync(0xffffffffu, o4.x, o);
        o4.y += __shfl_xor_sync(0xffffffffu, o4.y, o);
        o4.z += __shfl_xor_sync(0xffffffffu, o4.z, o);
        o4.w += __shfl_xor_sync(0xffffffffu, o4.w, o);
      }
      if (lane < q) write_out<T, D>(a, b, a.heads_of(item) * a.group + h0 + h, d, o4, top, sum);
    }
    __syncwarp();
    cluster_sync();  // no block leaves while another reads its shared memory
  } else
  if (merged) {  // the same for every warp of the block; the rings hold the teams' parts
    __syncthreads();
    const int first = team - team0;                        // this warp joins heads first, first + teams_here, ...
    const int heads = min(a.chunk, a.group - a.chunk_of(item) * a.chunk);
    for (int h = first; h < heads; h += teams_here) {
      float top = -INFINITY, sum = 0.0f;
      auto part = [&](int t) {
        return reinterpret_cast<const float *>(smem + (t * a.team + member) * kStages * kStage) + h * kPart;
      };
      for (int t = 0; t < teams_here; ++t) top = fmaxf(top, part(t)[D]);
      const float base = top == -INFINITY ? 0.0f : top;
      float o[D / 32] = {};
      for (int t = 0; t < teams_here; ++t) {
        const float f = exp2f(part(t)[D] - base);
        sum = fmaf(f, part(t)[D + 1], sum);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(f, part(t)[lane + 32 * i], o[i]);
      }
      float *p = a.part + ((static_cast<int64_t>(team0) * 2 * a.team + member) * a.chunk + h) * kPart;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) p[lane + 32 * i] = o[i];
      if (lane == 0) *reinterpret_cast<float2 *>(p + D) = make_float2(top, sum);
    }
  }
}

// Joins the parts of every item that teams share, per head: a warp per item and head,
// which leaves at once where one team held all of it; a block where there are more than
// kManyParts (a quarter as many where every block has one job at most).  (Warps only: 100000
// tokens of one head 59 us instead of 23, one frame 9.4 instead of 7.6; blocks above 4 parts:
// 64 sequences of 8192 132 instead of 127.)  Which teams hold parts follows from the line,
// which each block works out while the main kernel still runs.  A lane takes 4 dims of
// every kGroups-th part with its own running maximum and sum, 8 parts in flight: after the
// wait one read remains.  (Lists of the shared items made by every block, or written by
// the main kernel, put two or three more behind the wait; 7 to 11 us in all.)
constexpr int kJoinWarps = 8;
constexpr int kManyParts = 32;

// The parts of an item at [at, end) of the line: those of single teams at its edges, and
// one for every block of teams_here > 1 teams that lies inside it.
struct Parts {
  int first, left, inner, all, block0, teams_here, first_slot;
  Parts() = default;
  __device__ __forceinline__ Parts(const Shares &s, int at, int end, int teams_here_) {
    teams_here = teams_here_;
    first = s.owner(at);
    const int last = s.owner(end - 1);
    first_slot = s.begin(first) < at ? 1 : 0;
    left = all = last - first + 1;
    inner = block0 = 0;
    if (teams_here > 1) {
      const int from = first + first_slot;                                // the first team wholly inside
      const int to = s.begin(last + 1) <= end ? last + 1 : last;          // behind the last one
      block0 = (from + teams_here - 1) / teams_here;
      const int block1 = to / teams_here;
      if (block1 > block0) {
        inner = block1 - block0;
        left = block0 * teams_here - first;
        all = left + inner + last + 1 - block1 * teams_here;
      }
    }
  }
  __device__ __forceinline__ int slot_of(int i) const {  // twice the team, plus 1 for its second slot
    if (i == 0 && left > 0) return 2 * first + first_slot;
    if (i < left) return 2 * (first + i);
    if (i < left + inner) return 2 * (block0 + i - left) * teams_here;
    return 2 * ((block0 + inner) * teams_here + i - left - inner);
  }
};

template <int D>
struct Sum {
  float m = -INFINITY, sum = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

  template <int N>
  __device__ __forceinline__ void add(const float4 (&v)[N], const float2 (&ml)[N]) {
    float top = m;
#pragma unroll
    for (int f = 0; f < N; ++f) top = fmaxf(top, ml[f].x);
    const float base = top == -INFINITY ? 0.0f : top, keep = exp2f(m - base);
    m = top;
    sum *= keep;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int f = 0; f < N; ++f) {
      const float w = exp2f(ml[f].x - base);
      sum = fmaf(w, ml[f].y, sum);
      o.x = fmaf(w, v[f].x, o.x);
      o.y = fmaf(w, v[f].y, o.y);
      o.z = fmaf(w, v[f].z, o.z);
      o.w = fmaf(w, v[f].w, o.w);
    }
  }
  // every stride-th part from g on
  __device__ __forceinline__ void gather(const float *base, int64_t slot_floats, const Parts &parts, int g, int stride,
                                         int d) {
    constexpr int kFlight = 8;
    for (int i0 = g; i0 < parts.all; i0 += stride * kFlight) {
      float4 v[kFlight];
      float2 ml[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int i = i0 + f * stride;
        v[f] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        ml[f] = make_float2(-INFINITY, 0.0f);
        if (i < parts.all) {
          const float *p = base + parts.slot_of(i) * slot_floats;
          v[f] = *reinterpret_cast<const float4 *>(p + d);
          ml[f] = *reinterpret_cast<const float2 *>(p + D);
        }
      }
      add(v, ml);
    }
    if (D == 64) {  // two parts per warp at a time
      const float4 v[1] = {make_float4(__shfl_xor_sync(0xffffffffu, o.x, 16), __shfl_xor_sync(0xffffffffu, o.y, 16),
                                       __shfl_xor_sync(0xffffffffu, o.z, 16), __shfl_xor_sync(0xffffffffu, o.w, 16))};
      const float2 ml[1] = {make_float2(__shfl_xor_sync(0xffffffffu, m, 16), __shfl_xor_sync(0xffffffffu, sum, 16))};
      add(v, ml);  // the lower half's lanes are used
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_join_kernel(AttendArgs a, int most) {
  constexpr int P = attend_piece(D);
  constexpr int kPart = D + 4, kLanes = D / 4, kGroups = 32 / kLanes;
  // a warp's job: its sequence, query head (-1: nothing to do) and parts
  struct Job {
    int b, head, h;
    Parts parts;
  };
  __shared__ float4 box[kJoinWarps][kLanes];
  __shared__ float2 stats[kJoinWarps];
  __shared__ int starts[32 * kJoinWarps];  // of the runs of sequences in the line
  __shared__ int sums[kJoinWarps];
  __shared__ Job large[kJoinWarps];            // the warps' jobs that take the block
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.pages.n_seqs;
  const int per_seq = a.cache.heads / a.team * a.chunks, per_item = a.team * a.chunk, d = 4 * (lane % kLanes);
  const int64_t slot_floats = static_cast<int64_t>(per_item) * kPart;
  const int per_b = per_seq * per_item;
  const int64_t jobs = static_cast<int64_t>(B) * per_b;
  const int many_parts = jobs <= gridDim.x ? kManyParts / 4 : kManyParts;
  const int teams_here = kAttendWarps / a.team;
  // The line again, from the lengths.  The main kernel does not write them, and lets this one start only when
  // what was in front of it is done: they can be read before the wait.
  const int run = (B + 32 * kJoinWarps - 1) / (32 * kJoinWarps);
  int mine = 0;
  for (int i = tid * run; i < min(B, (tid + 1) * run); ++i) mine += Range<P, true>(a, i).pieces * per_seq;
  int upto = mine;
  for (int o = 1; o < min(B, 32); o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == min(B, 32) - 1) sums[warp] = upto;
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) upto += sums[w];
    total += sums[w];
  }
  starts[tid] = upto - mine;
  __syncthreads();
  const Shares shares(total, most);
  bool waited = false;
  for (int64_t job0 = blockIdx.x; job0 < jobs; job0 += static_cast<int64_t>(gridDim.x) * kJoinWarps) {
    const int64_t job = job0 + static_cast<int64_t>(warp) * gridDim.x;
    Job v;
    v.head = -1;
    bool many = false;
    if (job < jobs) {
      v.b = jobs < (int64_t(1) << 31) ? static_cast<int>(job) / per_b : static_cast<int>(job / per_b);
      const int in = static_cast<int>(job - static_cast<int64_t>(v.b) * per_b), item = in / per_item;
      v.h = in - item * per_item;
      const int h0 = a.chunk_of(item) * a.chunk, hm = v.h / a.chunk, hc = v.h - hm * a.chunk;
      const int pieces = Range<P, true>(a, v.b).pieces;
      if (hc < min(a.chunk, a.group - h0) && pieces > 0) {
        const int r = v.b / run;
        int at = starts[r] + item * pieces;
        for (int i = r * run; i < v.b; ++i) at += Range<P, true>(a, i).pieces * per_seq;
        v.parts = Parts(shares, at, at + pieces, teams_here);
        // one team held all of it and has written it, unless its block left it as a part
        if (v.parts.all > 1 || v.parts.inner > 0) v.head = (a.heads_of(item) * a.team + hm) * a.group + h0 + hc;
        many = v.head >= 0 && v.parts.all > many_parts;
      }
    }
    if (!waited) {
      griddep_wait();
      griddep_launch_dependents();
      waited = true;
    }
    if (v.head >= 0 && !many) {
      Sum<D> s;
      s.gather(a.part + v.h * kPart, slot_floats, v.parts, lane / kLanes, kGroups, d);
      if (lane < kLanes) write_out<T, D>(a, v.b, v.head, d, s.o, s.m, s.sum);
    }
    if (lane == 0) {
      if (!many) v.head = -1;
      large[warp] = v;
    }
    if (!__syncthreads_or(many)) continue;
    for (int w = 0; w < kJoinWarps; ++w) {
      if (large[w].head < 0) continue;
      const Job j = large[w];
      Sum<D> s;
      s.gather(a.part + j.h * kPart, slot_floats, j.parts, warp * kGroups + lane / kLanes, kJoinWarps * kGroups, d);
      if (lane < kLanes) box[warp][lane] = s.o;
      if (lane == 0) stats[warp] = make_float2(s.m, s.sum);
      __syncthreads();
      if (tid < kLanes) {
        Sum<D> t;
        float4 v4[kJoinWarps];
        float2 ml[kJoinWarps];
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) v4[i] = box[i][tid], ml[i] = stats[i];
        t.add(v4, ml);
        write_out<T, D>(a, j.b, j.head, d, t.o, t.m, t.sum);
      }
      __syncthreads();
    }
    __syncthreads();
  }
}

constexpr int kMaxSeqs = 1 << 24, kMaxHeads = 65535;

w4a4_status check_cache(const w4a4_kv_cache_t *c, Cache *out) {
  if (!c) return W4A4_ERR_ARG;
  if ((c->flags & ~W4A4_FLAG_FP16) || (c->head_dim != 64 && c->head_dim != 128)) return W4A4_ERR_UNSUPPORTED;
  if (c->n_pages < 0 || c->n_pages >= (int64_t(1) << 31) || c->page_size < 1 || c->n_heads < 1 || c->n_heads > kMaxHeads)
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
  if (n_seqs < 0 || n_seqs > kMaxSeqs || max_pages < 0 || static_cast<int64_t>(n_seqs) * max_pages >= (int64_t(1) << 31))
    return W4A4_ERR_SHAPE;
  if (static_cast<int64_t>(n_seqs) * max_pages > 0 && !pages) return W4A4_ERR_ARG;
  return ptr_aligned4(pages) ? W4A4_OK : W4A4_ERR_ALIGN;
}

// Whether the output takes part of the queries' memory, other than all of it in place.
bool out_in_q(const uint16_t *q, int64_t stride, int64_t rows, int64_t row, const uint16_t *out) {
  return !(q == out && (rows == 1 || stride == row)) && overlap(q, rows, row, stride, out, rows * row);
}

cudaLaunchConfig_t launch_config(int64_t grid, int threads, size_t smem, void *stream, cudaLaunchAttribute *attr,
                                 int cluster = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cfg;
}

size_t part_bytes(int group, int D) {
  const int chunks = (group + kChunk - 1) / kChunk, chunk = (group + chunks - 1) / chunks;
  return static_cast<size_t>(kMaxBlocks) * kAttendWarps * 2 * chunk * (D + 4) * sizeof(float);
}

// Blocks of a kernel per SM, once per context; 0 when it cannot run.
template <typename T, int D, int NT, bool CLUSTER>
int attend_blocks(int smem) {
  static ContextCache<int> occupancy;
  int per_sm = 0;
  const cudaError_t e = occupancy.get(&per_sm, [smem](int *v) {
    cudaError_t r = cudaFuncSetAttribute(kv_attend_kernel<T, D, NT, CLUSTER>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r == cudaSuccess)
      r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kv_attend_kernel<T, D, NT, CLUSTER>, 32 * kAttendWarps, smem);
    return r;
  });
  return e == cudaSuccess ? per_sm : 0;
}

template <typename T, int D, int NT>
w4a4_status launch_attend(AttendArgs &a, void *stream) {
  constexpr int P = attend_piece(D), kSmem = kAttendWarps * kAttendStages * 2 * P * 2 * D;
  unsigned int *status = nullptr;
  if (status_word(&status) != cudaSuccess) return W4A4_ERR_CUDA;
  // most pieces of a sequence: of the table's room, or of a window that begins with a piece's last token
  int64_t pieces = (static_cast<int64_t>(a.pages.max_pages) * a.cache.page_size + P - 1) / P;
  if (a.window) pieces = std::min<int64_t>(pieces, (static_cast<int64_t>(a.window) + P - 2) / P + 1);
  cudaLaunchAttribute attr[2];
  {
    // Clusters of as many blocks for an item as fit on the GPU and have a piece for every warp, where
    // no warp gets many, as far as the host knows: 4; 1 where few items leave most of the GPU to
    // a finer cut; 12 where blocks of long rows fill half of it.  (The host knows the table's width
    // only: short sequences under a wide table take the line.)  us with clusters and with the
    // line: 16 heads of 64, 1 sequence of 128 4.1 and 5.6, 1 of 1374 7.2 and 7.6, 16 of 500 11.6 and 14.1,
    // of 1374 (11 pieces a warp) 25.1 and 22.9; 8 heads of 128: 1 of 500 5.3 and 6.2, 1 of 4096 (8) 12.1 and
    // 11.2, 16 of 1374 (11, half the GPU) 20.6 and 23.1; 1 head of 64 for 8, 1 of 1374 7.4 and 6.8, 8 of 4096
    // (8 items) 11.2 and 9.6.  (A launch as clusters takes 0.8 us more: one block per item goes without.)
    const int per_sm = attend_blocks<T, D, NT, true>(kSmem);
    if (per_sm < 1) return W4A4_ERR_CUDA;
    const int64_t places = static_cast<int64_t>(device_sm_count()) * per_sm;
    const int64_t items = static_cast<int64_t>(a.pages.n_seqs) * a.cache.heads * a.chunks;
    int cluster = kMaxCluster;
    while (cluster > 1 && (items * cluster > places || pieces <= kAttendWarps * (cluster / 2))) cluster /= 2;
    const int most = items < 16 ? 1 : D == 128 && 2 * items * cluster >= places ? 12 : 4;
    if (pieces > 1 && items * cluster <= places && pieces <= most * kAttendWarps * cluster) {
      AttendArgs own = a;
      own.team = 1;
      own.cluster = cluster;
      const cudaLaunchConfig_t cfg =
          launch_config(items * cluster, 32 * kAttendWarps, kSmem, stream, attr, cluster > 1 ? cluster : 0);
      return launch_status(cudaLaunchKernelEx(&cfg, kv_attend_kernel<T, D, NT, true>, own, status));
    }
  }
  const int per_sm = attend_blocks<T, D, NT, false>(kSmem);
  if (per_sm < 1) return W4A4_ERR_CUDA;
  // blocks: one per place on the GPU, fewer when there cannot be that many pieces
  const int teams_here = kAttendWarps / a.team;
  int64_t grid = static_cast<int64_t>(device_sm_count()) * per_sm;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  const int64_t most = grid * teams_here;
  const int64_t items = static_cast<int64_t>(a.pages.n_seqs) * (a.cache.heads / a.team) * a.chunks;
  if (pieces < most && items < most && items * pieces < most) grid = (items * pieces + teams_here - 1) / teams_here;
  if (grid < 1) grid = 1;
  const int teams = static_cast<int>(grid) * teams_here;
  cudaLaunchConfig_t cfg = launch_config(grid, 32 * kAttendWarps, kSmem, stream, attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attend_kernel<T, D, NT, false>, a, status);
  // one team, or items of one piece: nothing is shared
  if (e != cudaSuccess || teams == 1 || pieces <= 1) return launch_status(e);
  cfg = launch_config(2 * device_sm_count(), 32 * kJoinWarps, 0, stream, attr);
  return launch_status(cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D>, a, teams));
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

w4a4_status w4a4_kv_append(const w4a4_kv_cache_t *cache, const w4a4_kv_append_t *tokens, void *stream) {
  using namespace w4a4;
  AppendArgs a = {};
  w4a4_status st = check_cache(cache, &a.cache);
  if (st != W4A4_OK) return st;
  if (!tokens) return W4A4_ERR_ARG;
  const w4a4_kv_append_t &t = *tokens;
  if (t.flags & ~W4A4_FLAG_ROPE_PAIRS) return W4A4_ERR_UNSUPPORTED;
  const int D = cache->head_dim, Hk = a.cache.heads, Hq = t.q ? t.n_q_heads : 0;
  if (t.rot_dim < 0 || t.rot_dim > D || t.rot_dim % 16) return W4A4_ERR_UNSUPPORTED;
  if (t.n_tokens < 0 || t.n_tokens >= (int64_t(1) << 31) || t.n_table < 0 || (t.q && (Hq < 1 || Hq > kMaxHeads)))
    return W4A4_ERR_SHAPE;
  if ((st = check_pages(t.pages, t.n_seqs, t.max_pages)) != W4A4_OK) return st;
  if ((a.cache.n_pages > 1 && a.cache.stride_page < D) || (a.cache.page_size > 1 && a.cache.stride_token < D) ||
      (Hk > 1 && a.cache.stride_head < D))
    return W4A4_ERR_SHAPE;
  if (t.n_tokens == 0) return W4A4_OK;
  if (!t.k || !t.v || !t.pos || (t.q && !t.q_out) || (t.rot_dim && t.n_table && !t.table)) return W4A4_ERR_ARG;
  if (t.k_stride < static_cast<int64_t>(Hk) * D || t.v_stride < static_cast<int64_t>(Hk) * D ||
      (t.q && t.q_stride < static_cast<int64_t>(Hq) * D))
    return W4A4_ERR_SHAPE;
  if (!ptr_aligned16(t.k) || !ptr_aligned16(t.v) || !ptr_aligned16(t.q) || (t.q && !ptr_aligned16(t.q_out)) ||
      !ptr_aligned16(t.table) || !ptr_aligned4(t.seq) || !ptr_aligned4(t.pos) || !ptr_aligned4(t.table_pos) ||
      t.k_stride % 8 || t.v_stride % 8 || (t.q && t.q_stride % 8))
    return W4A4_ERR_ALIGN;
  if (a.cache.n_pages && overlap(a.cache.k, 1, D, 0, a.cache.v, D)) return W4A4_ERR_ARG;
  if (t.q) {  // a token's heads are spread over warps, which read and write in no order
    const int64_t q_row = static_cast<int64_t>(Hq) * D, kv_row = static_cast<int64_t>(Hk) * D;
    if (out_in_q(t.q, t.q_stride, t.n_tokens, q_row, t.q_out) ||
        overlap(t.k, t.n_tokens, kv_row, t.k_stride, t.q_out, t.n_tokens * q_row) ||
        overlap(t.v, t.n_tokens, kv_row, t.v_stride, t.q_out, t.n_tokens * q_row))
      return W4A4_ERR_ARG;
    const size_t per_token = 4 * static_cast<size_t>(t.n_tokens);
    const struct {
      const void *at;
      size_t bytes;
    } read[5] = {{t.pages, 4 * static_cast<size_t>(t.n_seqs) * t.max_pages}, {t.pos, per_token}, {t.seq, per_token},
                 {t.table_pos, per_token}, {t.table, 4 * static_cast<size_t>(t.n_table) * t.rot_dim}};
    for (const auto &r : read)
      if (r.at && r.bytes && overlap_bytes(t.q_out, 2 * static_cast<size_t>(t.n_tokens) * q_row, r.at, r.bytes))
        return W4A4_ERR_ARG;
  }
  a.pages = {t.pages, t.n_seqs, t.max_pages};
  a.k = t.k;
  a.v = t.v;
  a.q = t.q;
  a.q_out = t.q_out;
  a.k_stride = t.k_stride;
  a.v_stride = t.v_stride;
  a.q_stride = t.q_stride;
  a.q_heads = Hq;
  a.rot_dim = t.rot_dim;
  a.n_table = t.n_table;
  a.seq = t.seq;
  a.pos = t.pos;
  a.table_pos = t.table_pos;
  a.table = t.table;
  a.pairs = (t.flags & W4A4_FLAG_ROPE_PAIRS) != 0;
  unsigned int *status = nullptr;
  if (status_word(&status) != cudaSuccess) return W4A4_ERR_CUDA;
  cudaLaunchAttribute attr;
  // shares of a token's heads, at most one per round of a warp, up to about the 24 warps per SM that
  // fit (over the same outputs again): 600 tokens of 128 dims and 48 heads 4.9 us (up to 16 warps 5.5, 4 8.9), 1000
  // 6.4 (6.6, 9.2); 5003 19.4 undivided, 25.0 in as many shares as there are rounds
  const int round = append_round(D) * (32 / (D / 16)), most = (2 * Hk + Hq + round - 1) / round;
  const int64_t want = (24ll * device_sm_count() + t.n_tokens - 1) / t.n_tokens;
  const int parts = static_cast<int>(want < most ? want : most);
  const cudaLaunchConfig_t cfg =
      launch_config((t.n_tokens * parts + kAppendWarps - 1) / kAppendWarps, 32 * kAppendWarps, 0, stream, &attr);
  const bool fp16 = (cache->flags & W4A4_FLAG_FP16) != 0;
  auto kern = D == 64 ? (fp16 ? kv_append_kernel<Fp16, 64> : kv_append_kernel<Bf16, 64>)
                      : (fp16 ? kv_append_kernel<Fp16, 128> : kv_append_kernel<Bf16, 128>);
  return launch_status(cudaLaunchKernelEx(&cfg, kern, a, t.n_tokens, parts, status));
}

size_t w4a4_kv_attend_workspace_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  using namespace w4a4;
  if (n_seqs < 0 || n_seqs > kMaxSeqs || n_q_heads < 1 || n_q_heads > kMaxHeads || n_kv_heads < 1 ||
      n_q_heads % n_kv_heads || (head_dim != 64 && head_dim != 128))
    return 0;
  return part_bytes(n_q_heads / n_kv_heads, head_dim);
}

w4a4_status w4a4_kv_attend(const w4a4_kv_cache_t *cache, const w4a4_kv_attend_t *tokens, void *stream) {
  using namespace w4a4;
  AttendArgs a = {};
  w4a4_status st = check_cache(cache, &a.cache);
  if (st != W4A4_OK) return st;
  if (!tokens) return W4A4_ERR_ARG;
  const w4a4_kv_attend_t &t = *tokens;
  const int D = cache->head_dim, Hk = a.cache.heads, Hq = t.n_q_heads;
  if (Hq < 1 || Hq > kMaxHeads || Hq % Hk || t.window < 0) return W4A4_ERR_SHAPE;
  if ((st = check_pages(t.pages, t.n_seqs, t.max_pages)) != W4A4_OK) return st;
  if (static_cast<int64_t>(t.max_pages) * a.cache.page_size > (int64_t(1) << 30)) return W4A4_ERR_SHAPE;
  if (!std::isfinite(t.scale * kLog2e)) return W4A4_ERR_ARG;
  if (t.n_seqs == 0) return W4A4_OK;
  if (!t.q || !t.lens || !t.out || !t.workspace) return W4A4_ERR_ARG;
  if (t.q_stride < static_cast<int64_t>(Hq) * D) return W4A4_ERR_SHAPE;
  if (t.workspace_bytes < w4a4_kv_attend_workspace_bytes(t.n_seqs, Hq, Hk, D)) return W4A4_ERR_SHAPE;
  if (!ptr_aligned16(t.q) || !ptr_aligned4(t.lens) || !ptr_aligned16(t.out) || !ptr_aligned4(t.lse) ||
      !ptr_aligned16(t.workspace) || t.q_stride % 8)
    return W4A4_ERR_ALIGN;
  if (out_in_q(t.q, t.q_stride, t.n_seqs, static_cast<int64_t>(Hq) * D, t.out)) return W4A4_ERR_ARG;
  a.pages = {t.pages, t.n_seqs, t.max_pages};
  a.q = t.q;
  a.q_stride = t.q_stride;
  a.q_heads = Hq;
  a.lens = t.lens;
  a.group = Hq / Hk;
  a.chunks = (a.group + kChunk - 1) / kChunk;
  a.chunk = (a.group + a.chunks - 1) / a.chunks;
  const int64_t room = static_cast<int64_t>(t.max_pages) * a.cache.page_size;
  // Neighbouring cache heads in a team, except where rows are long and there is little to do
  // for each warp (as far as the host knows): then shares of single heads, whose parts a
  // block joins by itself, win.  us with teams and without, 8 heads of 128: 1 sequence of 1024
  // tokens (in L2) 7.8 and 7.1, 23 of up to 4001 38.4 and 37.6; 64 of 2048 83.9 and 87.5, 16 of 16384
  // 158.2 and 160.5.  Of 64 (16 heads, 64 of 2048, by token): 87.7 and 94.5.
  const int64_t warps = 3 * kAttendWarps * device_sm_count();
  if (D == 64 || (room / 16) * Hk * a.chunks >= 32 * warps / t.n_seqs)
    a.team = Hk % 4 == 0 ? 4 : Hk % 2 == 0 ? 2 : 1;
  else
    a.team = 1;
  {  // the line of pieces is counted in 32 bits
    const int64_t pieces = (room + 15) / 16;
    const int64_t items = static_cast<int64_t>(Hk / a.team) * a.chunks;
    if (items * pieces >= (int64_t(1) << 31) / t.n_seqs) return W4A4_ERR_SHAPE;
  }
  {  // nothing that is written lies in what is read, nor in another output
    const size_t rows = static_cast<size_t>(t.n_seqs) * Hq;
    const struct {
      const void *at;
      size_t bytes;
    } written[3] = {{t.out, 2 * rows * D}, {t.workspace, part_bytes(a.group, D)}, {t.lse, t.lse ? 4 * rows : 0}},
      read[2] = {{t.pages, 4 * static_cast<size_t>(t.n_seqs) * t.max_pages}, {t.lens, 4 * static_cast<size_t>(t.n_seqs)}};
    for (int i = 0; i < 3; ++i) {
      if (!written[i].bytes) continue;
      for (int j = 0; j < i; ++j)
        if (overlap_bytes(written[i].at, written[i].bytes, written[j].at, written[j].bytes)) return W4A4_ERR_ARG;
      for (const auto &r : read)
        if (r.bytes && overlap_bytes(written[i].at, written[i].bytes, r.at, r.bytes)) return W4A4_ERR_ARG;
      if (i > 0 && overlap(t.q, t.n_seqs, static_cast<int64_t>(Hq) * D, t.q_stride,
                           static_cast<const uint16_t *>(written[i].at), (written[i].bytes + 1) / 2))
        return W4A4_ERR_ARG;
    }
  }
  int shift = 0;  // page_size <= 2^shift
  while ((int64_t(1) << shift) < a.cache.page_size) ++shift;
  a.div_shift = 31 + shift;
  a.div_mul = static_cast<uint32_t>((uint64_t(1) << a.div_shift) / a.cache.page_size + 1);
  a.scale_log2 = t.scale * kLog2e;
  a.window = t.window;
  a.out = t.out;
  a.lse = t.lse;
  a.part = static_cast<float *>(t.workspace);
  const bool fp16 = (cache->flags & W4A4_FLAG_FP16) != 0, wide = a.chunk > 8;
  if (D == 64) {
    if (fp16) return wide ? launch_attend<Fp16, 64, 2>(a, stream) : launch_attend<Fp16, 64, 1>(a, stream);
    return wide ? launch_attend<Bf16, 64, 2>(a, stream) : launch_attend<Bf16, 64, 1>(a, stream);
  }
  if (fp16) return wide ? launch_attend<Fp16, 128, 2>(a, stream) : launch_attend<Fp16, 128, 1>(a, stream);
  return wide ? launch_attend<Bf16, 128, 2>(a, stream) : launch_attend<Bf16, 128, 1>(a, stream);
}

}  // extern "C"
