// group.cu -- 4-bit weights with one step per group of inputs, and their
// product with a few tokens (include/decode.h, w4a4_group_*).
#include <cuda_runtime.h>

#include <cstdint>

#include "ctxcache.h"
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

// Bytes of the record of a tile and block: 1024 of codes, then for r = 0..7 the
// steps of rows r and r + 8, group by group.
__host__ __device__ constexpr int record_bytes(int group) { return 1024 + 32 * (kBlockK / group); }

// ------------------------------------------------- quantize, pack, dequantize
//
// One pass over the weights, bound by HBM (2 bytes in, half a byte and the steps
// out, or back).  A warp takes one tile and block, 16 rows by 128 inputs, in the
// packed order itself: lane 4 r + c holds, of rows r and r + 8, the inputs 32 j +
// 8 c .. + 7 for j = 0..3, so that its codes are the 16 bytes it stores (a whole
// warp's 512 in a row), a group's maximum needs two exchanges between four
// lanes, and all eight 16-byte loads are in flight at once.  (One thread per 8
// inputs, with the rows' order on both sides: 20000 x 8192 there and back took 411
// us; now 65 and 64, 99 % of a copy's rate.  Packing, whose loads are 4 bytes, all asked for before the
// first store: 47.4 us at 32768 x 8192, 90 %.)

constexpr int kPackWarps = 8;

struct Unit {
  int64_t at;  // tile * blocks + block
  int row, k;  // of this lane: rows row and row + 8, inputs k + 32 j
};

__device__ __forceinline__ bool unit_of_warp(const GroupShape &s, Unit &u) {
  const int lane = threadIdx.x & 31;
  u.at = static_cast<int64_t>(blockIdx.x) * kPackWarps + (threadIdx.x >> 5);
  if (u.at >= static_cast<int64_t>(s.tiles) * s.blocks) return false;
  const int t = static_cast<int>(u.at / s.blocks), b = static_cast<int>(u.at % s.blocks);
  u.row = t * kTileRows + (lane >> 2);
  u.k = b * kBlockK + 8 * (lane & 3);
  return true;
}

// round-half-even(x / step) for |x| <= max, two's complement in the low 4 bits of
// o.  x and step have at most 11 significant bits, so a quotient that is not half
// an integer is at least 2^-13 away from one: x * inv (off by less than 2^-19)
// rounded to multiples of 2^-16, which the sum with 1.5 * 2^7 does, is exact at the
// halves and on the right side elsewhere; the sum with 1.5 * 2^23 then rounds to an
// integer.
__device__ __forceinline__ void quantize_pair(float x0, float x1, unsigned long long inv, uint32_t &o0, uint32_t &o1) {
  const unsigned long long t = fma2(f2(x0, x1), inv, f2(192.0f, 192.0f));
  float a, b;
  f2_split(t, a, b);
  o0 = __float_as_uint(a + 12582720.0f);
  o1 = __float_as_uint(b + 12582720.0f);
}

__device__ __forceinline__ float rcp_approx(float x) {  // within 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __noinline__ int slow_code(float x, float step) {
  return step > 0.0f ? static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, step)), -8.0f), 7.0f)) : 0;
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(32 * kPackWarps)
    group_quantize_kernel(const uint16_t *W, GroupShape s, uint8_t *data) {
  constexpr int kPer = kBlockK / GROUP, kWords = 4 / kPer;  // groups of a block, words j of a group
  griddep_wait();
  griddep_launch_dependents();
  Unit u;
  if (!unit_of_warp(s, u)) return;
  const int lane = threadIdx.x & 31;
  uint4 v[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[h][j] = make_uint4(0u, 0u, 0u, 0u);  // padding: zero codes and steps
      if (u.row + 8 * h < s.N && u.k + 32 * j < s.K)
        v[h][j] = __ldcs(
            reinterpret_cast<const uint4 *>(W + static_cast<int64_t>(u.row + 8 * h) * s.K + u.k + 32 * j));
    }
  uint32_t steps[kPer];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word[4];
#pragma unroll
    for (int g = 0; g < kPer; ++g) {
      uint32_t top = 0;  // of the magnitudes, in pairs
#pragma unroll
      for (int j = g * kWords; j < (g + 1) * kWords; ++j) {
        top = T::max2(top, T::max2(v[h][j].x & 0x7FFF7FFFu, v[h][j].y & 0x7FFF7FFFu));
        top = T::max2(top, T::max2(v[h][j].z & 0x7FFF7FFFu, v[h][j].w & 0x7FFF7FFFu));
      }
      top = T::max2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = T::max2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m = fmaxf(T::lo(top), T::hi(top));
      // m / 7: a product is as good, for m has at most 11 bits and no such quotient lies
      // within 2^-14 of the middle between two 16-bit values
      const uint16_t step16 = T::round(m * (1.0f / 7.0f));
      const float step = T::to_f32(step16);
      steps[g] = h == 0 ? step16 : steps[g] | (static_cast<uint32_t>(step16) << 16);
      const float inv = rcp_approx(step);
      // a step so small that its own rounding, or its reciprocal's range, matters
      const bool plain = step >= 0x1p-100f && m * inv < 7.4f;
#pragma unroll
      for (int j = g * kWords; j < (g + 1) * kWords; ++j) {
        const uint32_t x[4] = {v[h][j].x, v[h][j].y, v[h][j].z, v[h][j].w};
        uint32_t w = 0;
#pragma unroll
        for (int p = 3; p >= 0; --p) {
          uint32_t a, b;
          if (plain) {
            quantize_pair(T::lo(x[p]), T::hi(x[p]), f2(inv, inv), a, b);
          } else {
            a = static_cast<uint32_t>(slow_code(T::lo(x[p]), step));
            b = static_cast<uint32_t>(slow_code(T::hi(x[p]), step));
          }
          w = (w << 4) | (__byte_perm(a, b, 0x5410) & 0x000F000Fu);
        }
        word[j] = w;
      }
    }
    *reinterpret_cast<uint4 *>(data + u.at * record_bytes(GROUP) + 512 * h + 16 * lane) =
        make_uint4(word[0], word[1], word[2], word[3]);
  }
  if ((lane & 3) == 0) {
    uint32_t *to = reinterpret_cast<uint32_t *>(data + u.at * record_bytes(GROUP) + 1024) + (lane >> 2) * kPer;
#pragma unroll
    for (int g = 0; g < kPer; ++g) to[g] = steps[g];
  }
}

__global__ void __launch_bounds__(32 * kPackWarps)
    group_pack_kernel(const uint8_t *codes, const uint16_t *scales, GroupShape s, uint8_t *data) {
  griddep_wait();
  griddep_launch_dependents();
  Unit u;
  if (!unit_of_warp(s, u)) return;
  const int lane = threadIdx.x & 31, per = kBlockK / s.group;
  uint8_t *record = data + u.at * record_bytes(s.group);
  const int g = (u.k / kBlockK) * per + (lane & 3), groups = s.K / s.group;  // this lane's group, where it has one
  uint32_t v[2][4];
  uint16_t step[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = u.row + 8 * h;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[h][j] = 0;
      if (n < s.N && u.k + 32 * j < s.K)
        v[h][j] = *reinterpret_cast<const uint32_t *>(codes + static_cast<int64_t>(n) * (s.K / 2) + (u.k + 32 * j) / 2);
    }
    if ((lane & 3) < per && n < s.N && g < groups) step[h] = scales[static_cast<int64_t>(n) * groups + g];
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // nibbles 0, 2, 4, 6 meet in bytes 0 and 2 of one word, 1, 3, 5, 7 in those of another
      const uint32_t even = v[h][j] & 0x0F0F0F0Fu, odd = (v[h][j] >> 4) & 0x0F0F0F0Fu;
      word[j] = __byte_perm(even | (even >> 4), odd | (odd >> 4), 0x6420);
    }
    *reinterpret_cast<uint4 *>(record + 512 * h + 16 * lane) = make_uint4(word[0], word[1], word[2], word[3]);
    if ((lane & 3) < per)
      reinterpret_cast<uint16_t *>(record + 1024)[((lane >> 2) * per + (lane & 3)) * 2 + h] = step[h];
  }
}

template <typename T, int GROUP>
__global__ void __launch_bounds__(32 * kPackWarps)
    group_dequantize_kernel(const uint8_t *data, GroupShape s, uint16_t *W) {
  constexpr int kPer = kBlockK / GROUP, kWords = 4 / kPer;
  griddep_wait();
  griddep_launch_dependents();
  Unit u;
  if (!unit_of_warp(s, u)) return;
  const int lane = threadIdx.x & 31;
  const uint8_t *record = data + u.at * record_bytes(GROUP);
  uint32_t steps[kPer];
#pragma unroll
  for (int g = 0; g < kPer; ++g) steps[g] = reinterpret_cast<const uint32_t *>(record + 1024)[(lane >> 2) * kPer + g];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(record + 512 * h + 16 * lane));
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t step = __byte_perm(steps[j / kWords], 0u, h ? 0x3232 : 0x1010);  // twice
      uint32_t c[4];
      T::codes(word[j], c);
      // an exact code times a step, rounded once
      if (u.row + 8 * h < s.N && u.k + 32 * j < s.K)
        __stcs(reinterpret_cast<uint4 *>(W + static_cast<int64_t>(u.row + 8 * h) * s.K + u.k + 32 * j),
               make_uint4(T::mul2(c[0], step), T::mul2(c[1], step), T::mul2(c[2], step), T::mul2(c[3], step)));
    }
  }
}

// -------------------------------------------------------------------- gemv
//
// Y[m, n] = sum_g s[n, g] sum_{k in g} c[n, k] x[m, k] + b[n] for at most 16
// tokens m.  Every code is read once and used M times: bound by the weights'
// traffic, N K / 2 bytes and the steps.  What the SMs have to do meanwhile is turn
// 8 codes per 4 bytes into operands, so products run as m16n8k16 on the tensor
// cores (A = 16 rows of weights, B = 8 tokens; a 128-row tcgen05 tile with one to
// 16 columns would read its operands from shared memory, to which every widened
// weight would have to be written first).
//
//  * The packed order is that of the operand: the 16 bytes that a lane copies
//    are its codes of one row of A for 8 products, no exchange between lanes.
//    In a word, elements 2 p and 2 p + 1 are nibbles p and p + 4, so one masked
//    xor gives a pair of 16-bit values 2^7 + u (bf16) or 2^10 + u, u = c + 8, and a
//    subtraction the exact codes.
//  * A group's products are summed in fp32 by the tensor core, multiplied by the
//    step and added to the fp32 total: the codes stay exact and no weight is rounded.
//  * One block of 16 warps (8, for large shapes and more than 8 tokens) per SM takes an equal
//    share of the 16-row tiles, up to RT at a time, and keeps their sums in registers.  The line (block of 128 inputs, tile)
//    is cut evenly between the warps: a warp reads a block's tokens once and uses them for
//    all the tiles, while codes and steps stream through its own ring of
//    asynchronous copies.  At the end the warps' sums meet in shared memory, where the rings
//    were.  (Tiles in pairs with the inputs split over the warps, so that every pair read
//    all tokens again, took 34 us for 8 tokens at 32768 x 8192, half of it waiting for
//    tokens that L1 could not hold.)
//  * Before it waits for the kernel in front, a block asks for its first weights
//    to be brought into L2: those do not depend on that kernel, and where they do
//    (a quantization right before) L2 is where the new values appear.  (One call after the
//    other, 8 tokens: 5.5 us instead of 5.6 at 2048 x 8192, 7.3 instead of 7.5 at 8192 x
//    4096; the smallest lose 0.1.)
//
// 32768 x 8192, groups of 128, no bias: 1 token 29.2 us, 8 29.6 (4.7 TB/s, 72 % of a copy), 16 41.5.
// At 8 tokens (30.7 with a bias) no single thing is full: issue slots 64 %, the integer and
// logic pipe 60 %, the tensor pipe 26 %.  Widening the codes is 5 us of it (26.2 with codes used as
// they are), the products 2 more (24.2 without).  16 tokens take as many instructions (20.8
// million warp instructions, 20.7 with 8), but from half the warps, two to a scheduler, at 46 %
// of the issue slots: a warp waits for its own results (1.3 cycles an issue for dependences, 0.6
// for the tensor pipe, 38 % busy, 0.4 for tokens) and there is too little else to issue.

// Warps of a block: 16 tiles of two sets of columns need twice the registers, and their sums
// would not fit into shared memory 16 times.  16 warps have 128 registers a thread, which does not
// hold everything: per thread, 8 tiles of two sets spill 140 to 236 bytes, 4 tiles of two sets up to 40, 16
// tiles of one set 12 to 52, 8 of one set up to 12 in groups of 32; 16 tiles of two sets, with 8 warps, up to 16.
constexpr int gemv_warps(int RT, int NT) { return RT * NT > 16 ? 8 : 16; }
// Tiles that a warp takes in one go: two, whose products do not depend on one another and
// which share the waiting and counting, unless there is only one.
constexpr int gemv_pair(int RT) { return RT > 1 ? 2 : 1; }
// The warps' rings hold 64 records together.  (96 and 128: 30.8 us instead of 31.0 for 8 tokens
// at 32768 x 8192, 11.0 and 11.9 instead of 10.1 for one at 16384 x 4096: what is asked for at the start
// has to arrive before the first product.)
constexpr int kRingRecords = 64;
constexpr int gemv_stages(int RT, int NT) { return kRingRecords / gemv_warps(RT, NT) / gemv_pair(RT); }

struct GemvArgs {
  const uint16_t *X;
  int M;
  const uint8_t *data;
  GroupShape s;
  const uint16_t *bias;
  uint16_t *Y;
  bool gelu;
  int sets;  // sets of tiles, a multiple of the number of blocks; set i: tiles i * tiles / sets ..
};

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// GROUP inputs per step, at most RT tiles of 16 rows at a time, NT times 8 tokens.
template <typename T, int GROUP, int RT, int NT>
__global__ void __launch_bounds__(32 * gemv_warps(RT, NT), 1) group_gemv_kernel(GemvArgs a) {
  constexpr int kPer = kBlockK / GROUP;             // groups of a block of inputs
  constexpr int kScaleRow = 4 * kPer;               // bytes of the steps of rows r and r + 8
  constexpr int kRecord = record_bytes(GROUP), kPair = gemv_pair(RT), kStage = kPair * kRecord;
  constexpr int kStages = gemv_stages(RT, NT), kGemvWarps = gemv_warps(RT, NT);
  constexpr int kCols = 8 * NT, kTileSums = 16 * kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const GroupShape &s = a.s;
  const uint32_t ring = smem_u32(smem) + warp * kStages * kStage;
  const int64_t tile_bytes = static_cast<int64_t>(s.blocks) * kRecord;
  // Tokens r and r + 8 as the B operand; columns behind the last token repeat it
  // (their sums are not used).
  const uint16_t *x_row[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) x_row[n] = a.X + static_cast<int64_t>(min(8 * n + r, a.M - 1)) * s.K + 8 * c;
  auto load_x = [&](uint4 (&x)[NT][4], int kb) {
    const int k = kb * kBlockK;
    if (k + kBlockK <= s.K) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = *reinterpret_cast<const uint4 *>(x_row[n] + k + 32 * j);
    } else {  // the padding's codes are 0, but what stands behind a token may not be finite
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[n][j] = k + 32 * j < s.K ? *reinterpret_cast<const uint4 *>(x_row[n] + k + 32 * j)
                                     : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  for (int set = blockIdx.x; set < a.sets; set += gridDim.x) {
    const int tile0 = static_cast<int>(static_cast<int64_t>(set) * s.tiles / a.sets);
    const int tiles = static_cast<int>(static_cast<int64_t>(set + 1) * s.tiles / a.sets) - tile0;
    // this warp's part of the line, in units of kPair tiles
    const int units = (tiles + kPair - 1) / kPair;
    const int begin = static_cast<int>(static_cast<int64_t>(warp) * s.blocks * units / kGemvWarps);
    const int end = static_cast<int>(static_cast<int64_t>(warp + 1) * s.blocks * units / kGemvWarps);
    int kb = begin / units, u0 = begin - kb * units, left = end - begin;
    // the copies' place in it: units until the next block of inputs, and in all; an odd last
    // tile is its own second
    const int64_t to_next = kRecord - (units - 1) * kPair * tile_bytes;
    int copy_u = units - u0, copies = left;
    uint32_t copy_dst = ring + 16 * lane;
    const uint32_t last = ring + (kStages - 1) * kStage;
    const uint8_t *from = a.data + (tile0 + kPair * u0) * tile_bytes + static_cast<int64_t>(kb) * kRecord + 16 * lane;
    auto second = [&]() { return copy_u == 1 && tiles % 2 ? from : from + tile_bytes; };
    auto advance = [&]() {
      from += --copy_u ? kPair * tile_bytes : to_next;
      if (copy_u == 0) copy_u = units;
    };
    if (set == blockIdx.x) {
      const uint8_t *const from0 = from;
      for (int i = 0; i < min(left, kStages - 1); ++i) {
        if (128 * lane < kRecord) {  // 128 bytes a lane
          prefetch_l2(from + 112 * lane);
          if (kPair == 2) prefetch_l2(second() + 112 * lane);
        }
        advance();
      }
      from = from0, copy_u = units - u0;
      griddep_wait();
      griddep_launch_dependents();
    }
    auto fill = [&]() {
      if (--copies >= 0) {
        copy16(copy_dst, from);
        copy16(copy_dst + 512, from + 512);
        if (lane < 2 * kPer) copy16(copy_dst + 1024, from + 1024);
        if (kPair == 2) {
          const uint8_t *f = second();
          copy16(copy_dst + kRecord, f);
          copy16(copy_dst + kRecord + 512, f + 512);
          if (lane < 2 * kPer) copy16(copy_dst + kRecord + 1024, f + 1024);
        }
        copy_dst = copy_dst >= last ? ring + 16 * lane : copy_dst + kStage;
        advance();
      }
      copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) fill();

    float total[RT][NT][4];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) total[t][n][e] = 0.0f;
    uint4 x[NT][4];
    uint32_t stage = ring + 16 * lane;
    const int steps_at = 1024 + r * kScaleRow - 16 * lane;
    while (left > 0) {
      const int u1 = min(units, u0 + left);  // units u0 .. u1 - 1 of block kb
      load_x(x, kb);
#pragma unroll
      for (int u = 0; u < RT / kPair; ++u) {
        if (u < u0 || u >= u1) continue;
        copy_wait<kStages - 2>();
        __syncwarp();
        fill();
        uint4 w[kPair][2];
#pragma unroll
        for (int t = 0; t < kPair; ++t) {
          w[t][0] = lds16(stage + t * kRecord);
          w[t][1] = lds16(stage + t * kRecord + 512);
        }
        float part[kPair][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int t = 0; t < kPair; ++t) {
            uint32_t p[4], q[4];
            T::codes(j == 0 ? w[t][0].x : j == 1 ? w[t][0].y : j == 2 ? w[t][0].z : w[t][0].w, p);
            T::codes(j == 0 ? w[t][1].x : j == 1 ? w[t][1].y : j == 2 ? w[t][1].z : w[t][1].w, q);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (j % (GROUP / 32) == 0)
                T::mma0(part[t][n], p[0], q[0], p[1], q[1], x[n][j].x, x[n][j].y);
              else
                T::mma(part[t][n], p[0], q[0], p[1], q[1], x[n][j].x, x[n][j].y);
              T::mma(part[t][n], p[2], q[2], p[3], q[3], x[n][j].z, x[n][j].w);
            }
          }
          if ((j + 1) % (GROUP / 32) == 0) {
#pragma unroll
            for (int t = 0; t < kPair; ++t) {
              const uint32_t steps = lds4(stage + t * kRecord + steps_at + 4 * (j / (GROUP / 32)));
              const float s0 = T::lo(steps), s1 = T::hi(steps);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float(&sum)[4] = total[kPair * u + t][n];
                sum[0] = fmaf(s0, part[t][n][0], sum[0]);
                sum[1] = fmaf(s0, part[t][n][1], sum[1]);
                sum[2] = fmaf(s1, part[t][n][2], sum[2]);
                sum[3] = fmaf(s1, part[t][n][3], sum[3]);
              }
            }
          }
        }
        stage = stage >= last ? ring + 16 * lane : stage + kStage;
      }
      left -= u1 - u0;
      u0 = 0;
      ++kb;
    }
    copy_wait<0>();
    __syncthreads();  // the rings are free: [warp][tile][row][token]
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int t = 0; t < RT; ++t)
      if (t < tiles)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2 *>(&sums[(warp * tiles + t) * kTileSums + (r + 8 * h) * kCols + 8 * n + 2 * c]) =
                make_float2(total[t][n][2 * h], total[t][n][2 * h + 1]);
    __syncthreads();
    for (int i = tid; i < tiles * kTileSums; i += 32 * kGemvWarps) {
      const int m = i % kCols, n = tile0 * kTileRows + i / kCols;
      if (m >= a.M || n >= s.N) continue;
      float y = 0.0f;
#pragma unroll
      for (int w = 0; w < kGemvWarps; ++w) y += sums[w * tiles * kTileSums + i];
      if (a.bias) y += T::to_f32(a.bias[n]);
      uint16_t v = T::round(y);
      if (a.gelu) v = static_cast<uint16_t>(gelu_pair_bf16(v) & 0xFFFFu);
      a.Y[m * static_cast<int64_t>(s.N) + n] = v;
    }
    __syncthreads();  // before the rings are filled again
  }
}

constexpr uint32_t kGroupFlags = W4A4_FLAG_FP16;

bool group_ok(int32_t group) { return group == 32 || group == 64 || group == 128; }
bool group_shape_ok(int32_t N, int32_t K, int32_t group) {
  return N >= 1 && N <= (1 << 24) && K >= group && K % group == 0 && K <= (1 << 20);
}

GroupShape shape_of(int32_t N, int32_t K, int32_t group) {
  return {N, K, group, (N - 1) / kTileRows + 1, (K + kBlockK - 1) / kBlockK};
}

size_t weight_bytes(const w4a4_group_weights_t *w) { return 2 * static_cast<size_t>(w->N) * w->K; }
size_t packed_bytes(const w4a4_group_weights_t *w) { return w4a4_group_weights_bytes(w->N, w->K, w->group); }

w4a4_status check_group(const w4a4_group_weights_t *w) {
  if (!w) return W4A4_ERR_ARG;
  if (!group_ok(w->group) || (w->flags & ~kGroupFlags)) return W4A4_ERR_UNSUPPORTED;
  if (!group_shape_ok(w->N, w->K, w->group)) return W4A4_ERR_SHAPE;
  if (!w->data) return W4A4_ERR_ARG;
  if (!ptr_aligned16(w->data)) return W4A4_ERR_ALIGN;
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

// a warp per tile and block
int64_t pack_grid(const GroupShape &s) {
  return (static_cast<int64_t>(s.tiles) * s.blocks + kPackWarps - 1) / kPackWarps;
}

template <typename T>
w4a4_status launch_quantize(const uint16_t *W, const w4a4_group_weights_t *w, void *stream) {
  const GroupShape s = shape_of(w->N, w->K, w->group);
  auto kern = w->group == 32   ? group_quantize_kernel<T, 32>
              : w->group == 64 ? group_quantize_kernel<T, 64>
                               : group_quantize_kernel<T, 128>;
  return launch_status(launch(kern, pack_grid(s), 32 * kPackWarps, 0, stream, W, s, w->data));
}

template <typename T>
w4a4_status launch_dequantize(const w4a4_group_weights_t *w, uint16_t *W, void *stream) {
  const GroupShape s = shape_of(w->N, w->K, w->group);
  auto kern = w->group == 32   ? group_dequantize_kernel<T, 32>
              : w->group == 64 ? group_dequantize_kernel<T, 64>
                               : group_dequantize_kernel<T, 128>;
  return launch_status(launch(kern, pack_grid(s), 32 * kPackWarps, 0, stream, w->data, s, W));
}

template <typename T, int GROUP, int RT, int NT>
w4a4_status launch_gemv_t(GemvArgs a, void *stream) {
  constexpr int kGemvWarps = gemv_warps(RT, NT), kRing = kRingRecords * record_bytes(GROUP);
  constexpr int kSums = kGemvWarps * RT * 16 * 8 * NT * 4, kSmem = kRing > kSums ? kRing : kSums;
  static ContextCache<int> ready;  // per context: attribute set
  int done = 0;
  if (ready.get(&done, [](int *v) {
        *v = 1;
        return cudaFuncSetAttribute(group_gemv_kernel<T, GROUP, RT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmem);
      }) != cudaSuccess)
    return W4A4_ERR_CUDA;
  const int sms = device_sm_count(), grid = a.s.tiles < sms ? a.s.tiles : sms;
  a.sets = ((a.s.tiles - 1) / (grid * RT) + 1) * grid;
  return launch_status(launch(group_gemv_kernel<T, GROUP, RT, NT>, grid, 32 * kGemvWarps, kSmem, stream, a));
}

template <typename T, int GROUP>
w4a4_status launch_gemv(const GemvArgs &a, void *stream) {
  // As many tiles at a time as a block has, in steps: what is not used costs instructions, and with two
  // sets of columns spilled registers; a single tile is taken alone, with 4 stages of its ring
  // instead of 2 pairs (us at N x K on 148 SMs, 8 or 16 tokens):
  //   1 tile: alone 5.6 and 6.4, as 4 with three empty 6.7 and 8.1 (2048 x 8192)
  //   2 to 4: up to 8 tokens 8 at a time are as good as 4 (7.2 both, 8192 x 4096); 16 tokens, 4 at a time 9.3, 8 10.7
  //   5 to 8: 8 at a time 11.0 and 16.5, 16 11.6 and 17.4 (16384 x 4096)
  //   more:   16 at a time 31.1 and 45.6, 16 tokens with 8 50.3, with 4 52.1 (32768 x 8192)
  const int tiles = (a.s.tiles - 1) / device_sm_count() + 1;
  if (a.M <= 8) {
    if (tiles == 1) return launch_gemv_t<T, GROUP, 1, 1>(a, stream);
    return tiles <= 8 ? launch_gemv_t<T, GROUP, 8, 1>(a, stream) : launch_gemv_t<T, GROUP, 16, 1>(a, stream);
  }
  if (tiles == 1) return launch_gemv_t<T, GROUP, 1, 2>(a, stream);
  if (tiles <= 4) return launch_gemv_t<T, GROUP, 4, 2>(a, stream);
  return tiles <= 8 ? launch_gemv_t<T, GROUP, 8, 2>(a, stream) : launch_gemv_t<T, GROUP, 16, 2>(a, stream);
}

}  // namespace
}  // namespace w4a4

extern "C" {

size_t w4a4_group_weights_bytes(int32_t N, int32_t K, int32_t group) {
  using namespace w4a4;
  if (!group_ok(group) || !group_shape_ok(N, K, group)) return 0;
  const GroupShape s = shape_of(N, K, group);
  return static_cast<size_t>(s.tiles) * s.blocks * record_bytes(group);
}

w4a4_status w4a4_group_bind(void *base, size_t bytes, int32_t N, int32_t K, int32_t group, uint32_t flags,
                            w4a4_group_weights_t *out) {
  using namespace w4a4;
  if (!base || !out) return W4A4_ERR_ARG;
  if (!group_ok(group) || (flags & ~kGroupFlags)) return W4A4_ERR_UNSUPPORTED;
  if (!ptr_aligned16(base)) return W4A4_ERR_ALIGN;
  if (!group_shape_ok(N, K, group)) return W4A4_ERR_SHAPE;
  if (bytes < w4a4_group_weights_bytes(N, K, group)) return W4A4_ERR_SHAPE;
  out->N = N;
  out->K = K;
  out->group = group;
  out->flags = flags;
  out->data = static_cast<uint8_t *>(base);
  return W4A4_OK;
}

w4a4_status w4a4_group_quantize(const uint16_t *W, const w4a4_group_weights_t *w, void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!W) return W4A4_ERR_ARG;
  if (!ptr_aligned16(W)) return W4A4_ERR_ALIGN;
  if (overlap_bytes(W, weight_bytes(w), w->data, packed_bytes(w))) return W4A4_ERR_ARG;
  return (w->flags & W4A4_FLAG_FP16) ? launch_quantize<Fp16>(W, w, stream) : launch_quantize<Bf16>(W, w, stream);
}

w4a4_status w4a4_group_pack(const uint8_t *codes, const uint16_t *scales, const w4a4_group_weights_t *w,
                            void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!codes || !scales) return W4A4_ERR_ARG;
  if (!ptr_aligned16(codes) || !ptr_aligned16(scales)) return W4A4_ERR_ALIGN;
  if (overlap_bytes(codes, weight_bytes(w) / 4, w->data, packed_bytes(w)) ||
      overlap_bytes(scales, weight_bytes(w) / w->group, w->data, packed_bytes(w)))
    return W4A4_ERR_ARG;
  const GroupShape s = shape_of(w->N, w->K, w->group);
  return launch_status(
      launch(group_pack_kernel, pack_grid(s), 32 * kPackWarps, 0, stream, codes, scales, s, w->data));
}

w4a4_status w4a4_group_dequantize(const w4a4_group_weights_t *w, uint16_t *W, void *stream) {
  using namespace w4a4;
  const w4a4_status st = check_group(w);
  if (st != W4A4_OK) return st;
  if (!W) return W4A4_ERR_ARG;
  if (!ptr_aligned16(W)) return W4A4_ERR_ALIGN;
  if (overlap_bytes(W, weight_bytes(w), w->data, packed_bytes(w))) return W4A4_ERR_ARG;
  return (w->flags & W4A4_FLAG_FP16) ? launch_dequantize<Fp16>(w, W, stream) : launch_dequantize<Bf16>(w, W, stream);
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
  const size_t y_bytes = 2 * static_cast<size_t>(M) * w->N;
  if (overlap_bytes(X, 2 * static_cast<size_t>(M) * w->K, Y, y_bytes) || overlap_bytes(w->data, packed_bytes(w), Y, y_bytes) ||
      (bias && overlap_bytes(bias, 2 * static_cast<size_t>(w->N), Y, y_bytes)))
    return W4A4_ERR_ARG;
  const GemvArgs a{X, static_cast<int>(M), w->data, shape_of(w->N, w->K, w->group), bias, Y, gelu, 0};
  switch (w->group) {
    case 32: return fp16 ? launch_gemv<Fp16, 32>(a, stream) : launch_gemv<Bf16, 32>(a, stream);
    case 64: return fp16 ? launch_gemv<Fp16, 64>(a, stream) : launch_gemv<Bf16, 64>(a, stream);
    default: return fp16 ? launch_gemv<Fp16, 128>(a, stream) : launch_gemv<Bf16, 128>(a, stream);
  }
}

}  // extern "C"
