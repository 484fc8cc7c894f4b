// Products with 4-bit expert weights, for serving: rows grouped by expert, a few rows each.
//   y[r,n] = act( sum_k x[r,k] s[e,k/G,n] (c[e,n,k] - 8) + b[e,n] ),   c in 0..15, s bf16, G = 32, 64 or 128
// ("MoE Training: Mixture of Experts" page, Quick Start: the expert's Linear layers, with the weights held in
// 4 bits and a scale for each group of G inputs of an output column.)
//
// Bound: reading the weights from HBM (half a byte each), as decode with bf16 weights is by four times the bytes.
// Mathematics: a sum over up to 64 inputs of a group,  d[n,r] = sum_k (c - 8) x[r,k],  runs on mma.sync m16n8k16 with
// the weights as the 16-row operand (c - 8 is exact in bf16) and eight rows of x as the 8-column one, and joins the
// fp32 accumulator as  acc += s d:  no weight is rounded, and tensor-core sums (which cut) are short.  fp32 rows are
// split exactly into three bf16 parts (8 bits of the significand each), three products a step.
// The codes' differences are taken as (c - 8) / 1024: 128 of them at 8 / 1024 are one x at most, so no sum of a group
// overflows where x is finite, and the result is multiplied back once (both exact; fp32 rows below 2^-110 lose what their
// third part has below 2^-133, the least of a bf16).
// Unpacking sets the pace next to the bytes: a turn of the word and one logic instruction make 16 + c of two codes, a
// subtraction c - 8 (all / 1024).  (Taking 24 sum x from the result instead, by one more product with a constant operand for both
// tiles, measured no faster: the tensor pipe's clocks cost what the subtractions do.)
// mma.sync rather than tcgen05: at up to 16 rows the product is a small part of what the tensor pipe could do in the
// time that the weights take, and its register operand is what unpacking produces.
//
// Layout (moe_q4_pack): 16 columns (a tile) x 128 inputs (a step) are 1024 bytes of codes in the order of the mma's
// register operand; a block holds two tiles of a step and their scales, and the blocks of a pair of tiles follow each
// other along K.
// Split: a piece of work is two tiles of an expert's block of up to 16 rows, over all of K.  The pieces are shared over
// one CTA per SM, and its 16 warps work alone: each streams its piece's blocks through a ring of its own (16-byte
// asynchronous copies, 9 KB in flight a warp, each lane the codes that it will read itself) and reads x through L1,
// once for its two tiles.  The steps of a CTA's pieces laid end to end are shared evenly over its warps (two rounds of
// whole pieces cost the layer of many experts 1.6 times as much); where a piece is cut, the warp that has its beginning
// adds the others' sums from shared memory, in order.  Nothing crosses a CTA: with K split over CTAs, joining parts
// through global memory took 4 to 5 us each of a call that streams for 10; with stages and x shared by a CTA's warps,
// the waits for one another and a fragment of x for every tile took as long as the bytes; and bulk copies of 1 KB are
// too slow: an SM issues one in about 64 clocks.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "activation.cuh"
#include "moe_internal.cuh"
#include "segments.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int kWarps = 16;     // of a CTA
constexpr int kRows = 16;      // rows of a piece (two mma column groups)
constexpr int kStepK = 128;    // inputs of a step
constexpr int kStages = 5;     // of a warp's ring, each a block
constexpr size_t kQ4WsBytes = 256;  // the error word

// two tiles' codes, then their scales: for each group, 8 words of the scales of columns g and g + 8
__host__ __device__ constexpr int block_bytes(int group) { return 2 * (1024 + (kStepK / group) * 32); }

struct Q4Shape {  // the packed layout of one expert
  int pairs, steps, blk;
  __host__ __device__ Q4Shape(int K, int N, int group)
      : pairs((N + 31) / 32), steps((K + kStepK - 1) / kStepK), blk(block_bytes(group)) {}
  __host__ __device__ size_t expert_bytes() const { return (size_t)pairs * steps * blk; }
  __host__ __device__ size_t at(int pair, int step) const { return ((size_t)pair * steps + step) * blk; }
};

struct Q4Args {
  const int32_t* offsets;
  const uint8_t* x;
  const uint8_t* w;
  const void* bias;
  void* y;
  int32_t* status;
  long long rows_cap, ldx, ldy;
  int E, K, N, act, bf16_out;
  int steps, pairs;  // of one expert's packed weights
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b + c
__device__ __forceinline__ void mma16816_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// The eight codes of a word (four in each half) as bf16 pairs of (c - 8) / 1024: 0x3c80 | c << 3 is (16 + c) / 1024 in bf16,
// and taking 24 / 1024 away is exact.  One three-input logic instruction a pair, its two constants in registers.
constexpr float kCodeUnit = 1.f / 1024, kCodeUnits = 1024.f;
struct Unpack {
  uint32_t mask, magic;
  __nv_bfloat162 off;
  __device__ __forceinline__ Unpack() {
    asm volatile("mov.b32 %0, 0x00780078;\nmov.b32 %1, 0x3c803c80;\n" : "=r"(mask), "=r"(magic));
    off = __halves2bfloat162(__float2bfloat16_rn(24.f * kCodeUnit), __float2bfloat16_rn(24.f * kCodeUnit));
  }
  __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&a)[4]) const {
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      uint32_t v;
      asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(v) : "r"(__funnelshift_r(w, w, 4 * f)), "r"(mask), "r"(magic));  // (w & mask) | magic
      const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), off);
      a[f] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};

// A lane's inputs of 64: for each block of 32 and group of 8 rows, 8 inputs of row g of the group.  Past the end of K
// (k32 blocks are left in the step) the weights are zero; the inputs there have to be too, since 0 x infinity is not.
template <bool F32X, int RB>
struct XUnit {
  uint4 v[2][RB][F32X ? 2 : 1];
  // p[rb]: the lane's place in its row at the step's first input
  __device__ __forceinline__ void load(const uint8_t* const (&p)[2], int unit, int k32) {
    if (k32 >= 4) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int h = 0; h < (F32X ? 2 : 1); ++h)
            v[b][rb][h] = __ldg(reinterpret_cast<const uint4*>(p[rb] + (2 * unit + b) * (F32X ? 128 : 64) + h * 16));
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
          for (int h = 0; h < (F32X ? 2 : 1); ++h) {
            v[b][rb][h] = make_uint4(0u, 0u, 0u, 0u);
            if (2 * unit + b < k32)
              v[b][rb][h] = __ldg(reinterpret_cast<const uint4*>(p[rb] + (2 * unit + b) * (F32X ? 128 : 64) + h * 16));
          }
    }
  }
};

__device__ __forceinline__ void scale_add(float (&acc)[4], uint32_t scales, const float (&d)[4]) {
  const float s0 = __uint_as_float(scales << 16), s1 = __uint_as_float(scales & 0xffff0000u);
  acc[0] = fmaf(s0, d[0], acc[0]);
  acc[1] = fmaf(s0, d[1], acc[1]);
  acc[2] = fmaf(s1, d[2], acc[2]);
  acc[3] = fmaf(s1, d[3], acc[3]);
}

// acc += 64 inputs (unit U of a step) of two tiles: GP groups a step, RB groups of 8 rows.  wl: the lane's codes, sl: its
// scales.  With two row groups the blocks of a group of 64 or 128 share a chain of products (fewer additions); with one
// the shorter chains are faster (62 against 65 us over 8 experts of 4096 x 14336 with 8 rows each).
template <int GP, int RB, int U>
__device__ __forceinline__ void q4_unit(float (&acc)[2][2][4], uint32_t wl, uint32_t sl, const XUnit<false, RB>& x,
                                        const Unpack& unpack) {
  constexpr int BG = GP == 4 || RB == 1 ? 1 : 2;
  const float zero[4] = {0.f, 0.f, 0.f, 0.f};
  uint4 w[2];
  uint32_t sc[2][GP == 4 ? 2 : 1];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    w[m] = lds128(wl + m * 1024 + U * 512);
#pragma unroll
    for (int i = 0; i < (GP == 4 ? 2 : 1); ++i) sc[m][i] = lds32(sl + (m * GP + (GP == 4 ? 2 * U + i : (GP == 2 ? U : 0))) * 32);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float d[2 / BG][RB][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t a0[4], a1[4];
      unpack(b ? w[m].z : w[m].x, a0);
      unpack(b ? w[m].w : w[m].y, a1);
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        if (b % BG == 0) mma16816_from(d[b / BG][rb], a0, x.v[b][rb][0].x, x.v[b][rb][0].y, zero);
        else mma16816(d[b / BG][rb], a0, x.v[b][rb][0].x, x.v[b][rb][0].y);
        mma16816(d[b / BG][rb], a1, x.v[b][rb][0].z, x.v[b][rb][0].w);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 / BG; ++i)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) scale_add(acc[m][rb], sc[m][GP == 4 ? i : 0], d[i][rb]);
  }
}

// x = h + m + l exactly, each with 8 bits of the significand (cut, so that h never rounds up to infinity; an
// infinity is kept whole in h, a NaN reaches all parts)
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = __float_as_uint(x) & 0xffff0000u;
  const float r = fabsf(x) == INFINITY ? 0.f : x - __uint_as_float(h);
  m = __float_as_uint(r) & 0xffff0000u;
  l = __float_as_uint(r - __uint_as_float(m));
}

template <int GP, int RB, int U>
__device__ __forceinline__ void q4_unit(float (&acc)[2][2][4], uint32_t wl, uint32_t sl, const XUnit<true, RB>& x,
                                        const Unpack& unpack) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t a[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      unpack(lds32(wl + m * 1024 + U * 512 + b * 8), a[m][0]);
      unpack(lds32(wl + m * 1024 + U * 512 + b * 8 + 4), a[m][1]);
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const uint4 v0 = x.v[b][rb][0], v1 = x.v[b][rb][1];
      const uint32_t f[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      uint32_t p[3][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo[3], hi[3];
        split3(__uint_as_float(f[2 * j]), lo[0], lo[1], lo[2]);
        split3(__uint_as_float(f[2 * j + 1]), hi[0], hi[1], hi[2]);
#pragma unroll
        for (int q = 0; q < 3; ++q) p[q][j] = __byte_perm(lo[q], hi[q], 0x7632);
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 2; q >= 0; --q) {  // the smallest part of x first
          mma16816(d, a[m][0], p[q][0], p[q][1]);
          mma16816(d, a[m][1], p[q][2], p[q][3]);
        }
        scale_add(acc[m][rb], lds32(sl + (m * GP + (2 * U + b) * GP / 4) * 32), d);
      }
    }
  }
}

// a / b for a >= 0, b > 0.  Below 2^20 by a reciprocal: (a + 1/2) / b is at least 1 / (2 b) from a whole number, and the
// quotient's error below a 2^-21 / b.  The divisions at the start are latency that every call pays.
__device__ __forceinline__ int idiv(int a, int b) {
  if (a < (1 << 20)) return (int)__fdividef((float)a + 0.5f, (float)b);
  return a / b;
}

struct Q4Piece {
  int e, pair, row0, rows;
};
// Piece i: the pairs of tiles of a block of rows follow each other, then the blocks of an expert, then the experts.
__device__ __forceinline__ Q4Piece find_piece(int i, const int* offs, const int* prefix, int E, int pairs) {
  Q4Piece p;
  const int block = idiv(i, pairs);
  p.e = find_segment(prefix, E, block);
  p.pair = i - block * pairs;
  p.row0 = offs[p.e] + (block - prefix[p.e]) * kRows;
  p.rows = min(kRows, offs[p.e + 1] - p.row0);
  return p;
}

constexpr int kStageBytes = block_bytes(32);
constexpr int kPartOff = kWarps * kStages * kStageBytes;  // 2 KB a warp: its sums of a piece that another began
constexpr int kOffsOff = kPartOff + kWarps * 2048;
constexpr int kSmemBytes = 128 + kOffsOff + 2 * 260 * 4;
static_assert(kSmemBytes <= 232448 && kStageBytes % 128 == 0, "shared-memory plan");

// A warp starts the copies of a block: each lane the codes that it reads itself, the first lanes the scales.
template <int GP>
__device__ __forceinline__ void fill(uint32_t stage, const uint8_t* block, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) copy16(stage + i * 512 + lane * 16, block + i * 512 + lane * 16);
  if (lane < 4 * GP) copy16(stage + 2048 + lane * 16, block + 2048 + lane * 16);
}

// A warp's stream of blocks: its steps [s, end) of the CTA's pieces, from the first on
template <int GP>
struct Q4Stream {
  static constexpr int kBlk = block_bytes(kStepK / GP);
  const uint8_t* block;  // of step s
  int s, end, left;      // left: steps until the blocks go on elsewhere (another expert, or its next rows)
  uint32_t ring, stage, fresh;
  __device__ __forceinline__ void seek(const Q4Args& a, const Q4Piece& p, int k) {
    block = a.w + (((size_t)p.e * a.pairs + p.pair) * a.steps + k) * kBlk;
    left = (a.pairs - p.pair) * a.steps - k;
  }
  __device__ __forceinline__ void issue(const Q4Args& a, int p0, const int* offs, const int* prefix, uint32_t to, int lane) {
    if (s < end) {
      if (left == 0) {
        const int i = idiv(s, a.steps);  // s is a piece's first step
        seek(a, find_piece(p0 + i, offs, prefix, a.E, a.pairs), 0);
      }
      fill<GP>(to, block, lane);
      block += kBlk;
      --left;
      ++s;
    }
    copies_commit();
  }
};

// acc += steps [k, k1) of a piece, the next ones of the stream.
template <int GP, bool F32X, int RB>
__device__ __forceinline__ void q4_run(const Q4Args& a, const Q4Piece& p, int k, int k1, int p0, const int* offs, const int* prefix,
                                       Q4Stream<GP>& stream, int lane, const Unpack& unpack, float (&acc)[2][2][4]) {
  constexpr int ES = F32X ? 4 : 2;
  const uint8_t* xp[2] = {nullptr, nullptr};
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = min(rb * 8 + (lane >> 2), p.rows - 1);  // a row that is not there: another's inputs, its sums are not used
    xp[rb] = a.x + ((size_t)p.row0 + r) * a.ldx * ES + ((size_t)k * kStepK + (lane & 3) * 8) * ES;
  }
  XUnit<F32X, RB> x0, x1;
  int k32 = (a.K - k * kStepK) >> 5;
  x0.load(xp, 0, k32);
  for (; k < k1; ++k) {
    stream.issue(a, p0, offs, prefix, stream.fresh, lane);  // into the stage that the step before has read
    copies_wait<kStages - 1>();
    __syncwarp();  // the scales have come by way of other lanes
    const uint32_t wl = stream.stage + lane * 16, sl = stream.stage + 2048 + (lane >> 2) * 4;
    x1.load(xp, 1, k32);
    q4_unit<GP, RB, 0>(acc, wl, sl, x0, unpack);
    if (k + 1 < k1) {
      k32 -= 4;
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) xp[rb] += kStepK * ES;
      x0.load(xp, 0, k32);
    }
    q4_unit<GP, RB, 1>(acc, wl, sl, x1, unpack);
    stream.fresh = stream.stage;
    stream.stage = stream.stage == stream.ring + (kStages - 1) * kStageBytes ? stream.ring : stream.stage + kStageBytes;
    __syncwarp();  // every lane has read the stage
  }
}

struct Q4Sums {
  float v[2][2][4];  // tile, group of 8 rows
};
// The results of a piece: bias, activation, one rounding.  A lane holds columns g and g + 8 of each tile and rows 2t and
// 2t + 1 of each group.
template <int ACT, bool F32X, typename O>
__device__ __forceinline__ void store_piece(const Q4Args& a, const Q4Piece& p, const Q4Sums& sums, int lane) {
  const int t = lane & 3;
  float b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = p.pair * 32 + (lane >> 2) + 8 * i;
    b[i] = 0.f;
    if (a.bias != nullptr && n < a.N)
      b[i] = F32X ? static_cast<const float*>(a.bias)[(size_t)p.e * a.N + n]
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[(size_t)p.e * a.N + n]);
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = (r >> 1) * 8 + 2 * t + (r & 1);
    if (row >= p.rows) continue;
    O* y = static_cast<O*>(a.y) + ((size_t)p.row0 + row) * a.ldy;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = p.pair * 32 + (lane >> 2) + 8 * i;
      const float v = activate<ACT, sizeof(O) == 2>(fmaf(sums.v[i >> 1][r >> 1][(i & 1) * 2 + (r & 1)], kCodeUnits, b[i]));
      if (n < a.N) y[n] = (O)v;
    }
  }
}
template <bool F32X>
__device__ __noinline__ void finish_piece(const Q4Args& a, const Q4Piece p, const Q4Sums sums, int lane) {
  if (!F32X && a.bf16_out) {
    if (a.act == MOE_ACT_GELU) store_piece<MOE_ACT_GELU, F32X, __nv_bfloat16>(a, p, sums, lane);
    else if (a.act == MOE_ACT_SILU) store_piece<MOE_ACT_SILU, F32X, __nv_bfloat16>(a, p, sums, lane);
    else store_piece<MOE_ACT_NONE, F32X, __nv_bfloat16>(a, p, sums, lane);
  } else {
    if (a.act == MOE_ACT_GELU) store_piece<MOE_ACT_GELU, F32X, float>(a, p, sums, lane);
    else if (a.act == MOE_ACT_SILU) store_piece<MOE_ACT_SILU, F32X, float>(a, p, sums, lane);
    else store_piece<MOE_ACT_NONE, F32X, float>(a, p, sums, lane);
  }
}

template <int GP, bool F32X>
__global__ void __launch_bounds__(32 * kWarps, 1) q4_matmul_kernel(const __grid_constant__ Q4Args a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  const uint32_t sbase = smem_u32(smem);
  int* offs = reinterpret_cast<int*>(smem + kOffsOff);
  int* prefix = offs + 260;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kBlk = block_bytes(kStepK / GP);

  if (warp == 0) load_segments(a.offsets, a.E, a.rows_cap, kRows, 1, offs, prefix, a.status, blockIdx.x == 0);
  __syncthreads();

  // this CTA's pieces [p0, p0 + n), and this warp's steps [s0, s1) of them
  const int total = prefix[a.E] * a.pairs;
  const int base = idiv(total, gridDim.x), extra = total - base * gridDim.x;
  const int p0 = blockIdx.x * base + min((int)blockIdx.x, extra), n = base + ((int)blockIdx.x < extra);
  const int all = n * a.steps;
  auto first_step = [&](int w) { return (all >> 4) * w + ((all & 15) * w >> 4); };
  const int s0 = first_step(warp), s1 = first_step(warp + 1);
  static_assert(kWarps == 16, "first_step");

  Q4Stream<GP> stream;
  stream.s = s0;
  stream.end = s1;
  stream.ring = stream.stage = sbase + warp * (kStages * kStageBytes);
  stream.fresh = stream.ring + (kStages - 1) * kStageBytes;
  Q4Piece p{};
  int i = idiv(s0, a.steps), k = s0 - i * a.steps;
  if (s0 < s1) {
    p = find_piece(p0 + i, offs, prefix, a.E, a.pairs);
    stream.seek(a, p, k);
  }
#pragma unroll 1
  for (int s = 0; s < kStages - 1; ++s) stream.issue(a, p0, offs, prefix, stream.ring + s * kStageBytes, lane);
  float4* parts = reinterpret_cast<float4*>(smem + kPartOff);
  const Unpack unpack;
  Q4Sums sums;
  int open = 0;  // > 0: the sums are the beginning of piece p, which ends at this step of the CTA's
  for (int s = s0; s < s1;) {
    const int k1 = min(a.steps, k + s1 - s);
#pragma unroll
    for (int q = 0; q < 16; ++q) sums.v[q >> 3][q >> 2 & 1][q & 3] = 0.f;
    if (p.rows <= 8) q4_run<GP, F32X, 1>(a, p, k, k1, p0, offs, prefix, stream, lane, unpack, sums.v);
    else q4_run<GP, F32X, 2>(a, p, k, k1, p0, offs, prefix, stream, lane, unpack, sums.v);
    s += k1 - k;
    if (k > 0) {  // the end (or middle) of a piece that began with another warp
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < 2 || p.rows > 8)
          parts[(warp * 4 + q) * 32 + lane] = make_float4(sums.v[q & 1][q >> 1][0], sums.v[q & 1][q >> 1][1], sums.v[q & 1][q >> 1][2],
                                                          sums.v[q & 1][q >> 1][3]);
    } else if (k1 < a.steps) {
      open = (i + 1) * a.steps;
    } else {
      finish_piece<F32X>(a, p, sums, lane);
    }
    if (s < s1) {
      ++i;
      k = 0;
      p = find_piece(p0 + i, offs, prefix, a.E, a.pairs);
    }
  }
  __syncthreads();
  if (open > 0) {
    for (int w = warp + 1; w < kWarps && first_step(w) < open; ++w) {
      if (first_step(w) == first_step(w + 1)) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (q >= 2 && p.rows <= 8) continue;
        const float4 v = parts[(w * 4 + q) * 32 + lane];
        sums.v[q & 1][q >> 1][0] += v.x;
        sums.v[q & 1][q >> 1][1] += v.y;
        sums.v[q & 1][q >> 1][2] += v.z;
        sums.v[q & 1][q >> 1][3] += v.w;
      }
    }
    finish_piece<F32X>(a, p, sums, lane);
  }
}

// ---------------------------------------------------------------- laying the weights out --------
// One thread a lane's 16 bytes of a tile's 64 inputs: word 2h + i holds inputs 32h + 8t + 4i + {0..3} of columns
// g and g + 8, its 16-bit halves the even and the odd ones, each with (g, first), (g + 8, first), (g, second),
// (g + 8, second), the word turned left by 3: code j sits at bits 3 + 4 j of its half, where a turn right by 4 j and a
// mask leave it in the mantissa of 16 + c.  Columns and inputs past the edge are code 8 (zero) with scale zero.
__global__ void __launch_bounds__(256) q4_pack_kernel(int E, int K, int N, int group, const uint8_t* __restrict__ q,
                                                      const uint16_t* __restrict__ s, uint8_t* __restrict__ packed) {
  const Q4Shape sh(K, N, group);
  const int tiles = 2 * sh.pairs;
  const long long units = (long long)E * tiles * sh.steps * 2;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= units) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = (int)(i & 1);
  const long long b = i >> 1;
  const int step = (int)(b % sh.steps);
  const int tile = (int)((b / sh.steps) % tiles), e = (int)(b / sh.steps / tiles);
  uint8_t* dst = packed + (size_t)e * sh.expert_bytes() + sh.at(tile >> 1, step);
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = step * kStepK + u * 64 + h * 32 + t * 8;
    uint32_t v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = tile * 16 + g + 8 * j;
      v[j] = n < N && k < K ? *reinterpret_cast<const uint32_t*>(q + ((size_t)e * N + n) * (K / 2) + k / 2) : 0x88888888u;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t r = 0;
#pragma unroll
      for (int o = 0; o < 2; ++o)  // even inputs to the low half, odd ones to the high half
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int j = 0; j < 2; ++j) r |= ((v[j] >> (16 * p + 8 * f + 4 * o)) & 15u) << (16 * o + 8 * f + 4 * j);
      w[2 * h + p] = r << 3 | r >> 29;
    }
  }
  *reinterpret_cast<uint4*>(dst + (tile & 1) * 1024 + u * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  const int gp = kStepK / group;
  if (u == 0 && lane < gp * 8) {
    const int grp = lane >> 3, kg = step * gp + grp, groups = K / group;
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = tile * 16 + (lane & 7) + 8 * j;
      if (n < N && kg < groups) v |= (uint32_t)s[((size_t)e * groups + kg) * N + n] << (16 * j);
    }
    *reinterpret_cast<uint32_t*>(dst + 2048 + (tile & 1) * gp * 32 + lane * 4) = v;
  }
}

// The value of one weight in the packed layout
__device__ __forceinline__ float q4_value(const uint8_t* expert, const Q4Shape& sh, int group, int k, int n) {
  const int r = k % kStepK, m = (n >> 4) & 1;
  const uint8_t* blk = expert + sh.at(n >> 5, k / kStepK);
  const int lane = (n & 7) * 4 + ((r & 31) >> 3);
  const int word = ((r & 63) >> 5) * 2 + ((r & 7) >> 2), field = ((r & 3) >> 1) * 2 + ((n >> 3) & 1);
  const uint32_t turned = *reinterpret_cast<const uint32_t*>(blk + m * 1024 + (r >> 6) * 512 + lane * 16 + word * 4);
  const uint32_t w = turned >> 3 | turned << 29;
  const int code = (int)((w >> (16 * (r & 1) + 4 * field)) & 15u);
  const uint32_t sc = *reinterpret_cast<const uint32_t*>(blk + 2048 + (m * (kStepK / group) + r / group) * 32 + (n & 7) * 4);
  return (float)(code - 8) * __uint_as_float((n & 8) ? sc & 0xffff0000u : sc << 16);  // 4 by 8 bits: exact
}

template <typename T>
__global__ void __launch_bounds__(256) q4_dequantize_kernel(int E, int K, int N, int group, const uint8_t* __restrict__ packed,
                                                            T* __restrict__ W) {
  const Q4Shape sh(K, N, group);
  const long long total = (long long)E * K * N;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const int n = (int)(i % N);
    const long long ek = i / N;
    const int k = (int)(ek % K);
    W[i] = (T)q4_value(packed + (size_t)(ek / K) * sh.expert_bytes(), sh, group, k, n);
  }
}

// Codes and scale of one group of one column a thread (columns across a warp: reads are coalesced).  The scale is
// bf16(max |w| / 7), c = 8 + round_half_even(w / s) within 0..15; a group of zeros (or one whose scale rounds to
// zero) is all 8, and a group that holds an infinity or NaN gets a NaN scale: it reads back as NaN throughout.
template <typename T>
__global__ void __launch_bounds__(256) q4_quantize_kernel(int E, int K, int N, int group, const T* __restrict__ W,
                                                          uint8_t* __restrict__ q, uint16_t* __restrict__ s) {
  const int groups = K / group;
  const long long total = (long long)E * groups * N;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const int n = (int)(i % N);
    const long long eg = i / N;
    const int kg = (int)(eg % groups), e = (int)(eg / groups);
    const T* w = W + ((size_t)e * K + (size_t)kg * group) * N + n;
    float m = 0.f;
    bool finite = true;
    for (int k = 0; k < group; ++k) {
      const float v = fabsf((float)w[(size_t)k * N]);
      finite = finite && v < INFINITY;
      m = fmaxf(m, v);
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(finite ? m / 7.f : __uint_as_float(0x7fffffffu));
    const float sc = __bfloat162float(sb);
    const bool flat = !finite || sc == 0.f;
    uint8_t* dst = q + ((size_t)e * N + n) * (K / 2) + (size_t)kg * (group / 2);
    for (int k = 0; k < group; k += 8) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = flat ? 0.f : fminf(fmaxf(rintf((float)w[(size_t)(k + j) * N] / sc), -8.f), 7.f);
        v |= (uint32_t)((int)r + 8) << (4 * j);
      }
      *reinterpret_cast<uint32_t*>(dst + k / 2) = v;
    }
    s[i] = __bfloat16_as_ushort(sb);
  }
}

bool misaligned(const void* p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

// Sizes that every call of this file takes
moe_status_t check_q4(int64_t E, int64_t K, int64_t N, int group) {
  if (E < 1 || E > kMaxExperts || K < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (K % group != 0 || K > (1 << 24) || N > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  const Q4Shape q((int)K, (int)N, group);
  if ((long long)q.pairs * q.steps >= 1LL << 31) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Pieces of a call at most: its rows in blocks of 16, one ragged block an expert
long long most_pieces(const moe_q4_t& m) {
  return (m.rows_cap / kRows + (m.rows_cap < m.E ? m.rows_cap : m.E)) * (((long long)m.N + 31) / 32);
}

unsigned copy_grid(long long threads) {
  const long long blocks = (threads + 255) / 256;
  return (unsigned)(blocks < 1 << 20 ? blocks : 1 << 20);
}

template <int GP, bool F32X>
cudaError_t launch_q4(const Q4Args& a, int grid, cudaStream_t st) {
  const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(q4_matmul_kernel<GP, F32X>), kSmemBytes);
  if (err != cudaSuccess) return err;
  q4_matmul_kernel<GP, F32X><<<grid, 32 * kWarps, kSmemBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

moe_status_t check_q4_matmul(const moe_q4_t* m) {
  if (m == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_status_t st = check_q4(m->E, m->K, m->N, m->group);
  if (st == MOE_ERR_INVALID_ARG || m->rows_cap < 0) return MOE_ERR_INVALID_ARG;
  if (m->dtype != MOE_DTYPE_F32 && m->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (m->out_dtype != MOE_DTYPE_F32 && m->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (m->activation != MOE_ACT_GELU && m->activation != MOE_ACT_SILU && m->activation != MOE_ACT_NONE)
    return MOE_ERR_INVALID_ARG;
  const long long ldx = m->ldx == 0 ? m->K : m->ldx, ldy = m->ldy == 0 ? m->N : m->ldy;
  if (ldx < m->K || ldy < m->N) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (m->dtype == MOE_DTYPE_F32 && m->out_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (ldx % (m->dtype == MOE_DTYPE_BF16 ? 8 : 4) != 0 || m->rows_cap >= (1LL << 31) - 1024) return MOE_ERR_UNSUPPORTED;
  if (ldx >= (1LL << 31) || ldy >= (1LL << 31) || most_pieces(*m) >= 1LL << 31) return MOE_ERR_UNSUPPORTED;
  // a CTA counts its steps in 32 bits (the kernel runs on 148 SMs)
  if ((most_pieces(*m) / 128 + 1) * ((m->K + kStepK - 1) / kStepK) >= 1LL << 31) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// m and the pointers have been checked
cudaError_t launch_q4_matmul(const moe_q4_t& m, const int32_t* offsets, const void* x, const void* packed, const void* bias,
                             void* y, int32_t* status, cudaStream_t st) {
  Q4Args a{};
  a.offsets = offsets;
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(packed);
  a.bias = bias;
  a.y = y;
  a.status = status;
  a.rows_cap = m.rows_cap;
  a.ldx = m.ldx == 0 ? m.K : m.ldx;
  a.ldy = m.ldy == 0 ? m.N : m.ldy;
  a.E = m.E;
  a.K = m.K;
  a.N = m.N;
  a.act = m.activation;
  a.bf16_out = m.out_dtype == MOE_DTYPE_BF16;
  const Q4Shape q(m.K, m.N, m.group);
  a.steps = q.steps;
  a.pairs = q.pairs;
  const long long pieces = most_pieces(m);
  const int grid = pieces < sm_count() ? (int)pieces : sm_count();
  const bool f32 = m.dtype == MOE_DTYPE_F32;
  if (m.group == 32) return f32 ? launch_q4<4, true>(a, grid, st) : launch_q4<4, false>(a, grid, st);
  if (m.group == 64) return f32 ? launch_q4<2, true>(a, grid, st) : launch_q4<2, false>(a, grid, st);
  return f32 ? launch_q4<1, true>(a, grid, st) : launch_q4<1, false>(a, grid, st);
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_q4_packed_size(int32_t E, int32_t K, int32_t N, int32_t group) {
  if (check_q4(E, K, N, group) != MOE_OK) return 0;
  return (size_t)E * Q4Shape(K, N, group).expert_bytes();
}

size_t moe_q4_workspace_size(void) { return kQ4WsBytes; }

moe_status_t moe_q4_pack(int32_t E, int32_t K, int32_t N, int32_t group, const void* codes, const void* scales, void* packed,
                         cudaStream_t stream) {
  NvtxRange nvtx_range("moe_q4_pack");
  launch_count() = 0;
  const moe_status_t st = check_q4(E, K, N, group);
  if (st != MOE_OK) return st;
  if (codes == nullptr || scales == nullptr || packed == nullptr || misaligned(codes, 16) || misaligned(scales, 2) ||
      misaligned(packed, 16))
    return MOE_ERR_INVALID_ARG;
  const Q4Shape q(K, N, group);
  const long long blocks = ((long long)E * q.pairs * q.steps * 4 + 7) / 8;
  if (blocks >= 1LL << 31) return MOE_ERR_UNSUPPORTED;
  q4_pack_kernel<<<(unsigned)blocks, 256, 0, stream>>>(E, K, N, group, static_cast<const uint8_t*>(codes),
                                                       static_cast<const uint16_t*>(scales), static_cast<uint8_t*>(packed));
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  ++launch_count();
  return MOE_OK;
}

moe_status_t moe_q4_quantize(int32_t E, int32_t K, int32_t N, int32_t group, moe_dtype_t dtype, const void* W, void* codes,
                             void* scales, cudaStream_t stream) {
  NvtxRange nvtx_range("moe_q4_quantize");
  launch_count() = 0;
  const moe_status_t st = check_q4(E, K, N, group);
  if (st == MOE_ERR_INVALID_ARG || (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (W == nullptr || codes == nullptr || scales == nullptr || misaligned(W, dtype == MOE_DTYPE_BF16 ? 2 : 4) ||
      misaligned(codes, 16) || misaligned(scales, 2))
    return MOE_ERR_INVALID_ARG;
  const unsigned grid = copy_grid((long long)E * (K / group) * N);
  if (dtype == MOE_DTYPE_BF16)
    q4_quantize_kernel<<<grid, 256, 0, stream>>>(E, K, N, group, static_cast<const __nv_bfloat16*>(W),
                                                 static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales));
  else
    q4_quantize_kernel<<<grid, 256, 0, stream>>>(E, K, N, group, static_cast<const float*>(W), static_cast<uint8_t*>(codes),
                                                 static_cast<uint16_t*>(scales));
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  ++launch_count();
  return MOE_OK;
}

moe_status_t moe_q4_dequantize(int32_t E, int32_t K, int32_t N, int32_t group, const void* packed, moe_dtype_t dtype, void* W,
                               cudaStream_t stream) {
  NvtxRange nvtx_range("moe_q4_dequantize");
  launch_count() = 0;
  const moe_status_t st = check_q4(E, K, N, group);
  if (st == MOE_ERR_INVALID_ARG || (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)) return MOE_ERR_INVALID_ARG;
  if (st != MOE_OK) return st;
  if (packed == nullptr || W == nullptr || misaligned(packed, 16) || misaligned(W, dtype == MOE_DTYPE_BF16 ? 2 : 4))
    return MOE_ERR_INVALID_ARG;
  const unsigned grid = copy_grid((long long)E * K * N);
  if (dtype == MOE_DTYPE_BF16)
    q4_dequantize_kernel<<<grid, 256, 0, stream>>>(E, K, N, group, static_cast<const uint8_t*>(packed), static_cast<__nv_bfloat16*>(W));
  else
    q4_dequantize_kernel<<<grid, 256, 0, stream>>>(E, K, N, group, static_cast<const uint8_t*>(packed), static_cast<float*>(W));
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  ++launch_count();
  return MOE_OK;
}

moe_status_t moe_q4_matmul(const moe_q4_t* m, const int32_t* offsets, const void* x, const void* packed, const void* bias,
                           void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
  NvtxRange nvtx_range("moe_q4_matmul");
  launch_count() = 0;
  const moe_status_t st = check_q4_matmul(m);
  if (st != MOE_OK) return st;
  if (ws == nullptr || misaligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kQ4WsBytes) return MOE_ERR_WORKSPACE;
  if (m->rows_cap == 0) return MOE_OK;
  const uintptr_t es = m->dtype == MOE_DTYPE_BF16 ? 2 : 4, os = m->out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (offsets == nullptr || x == nullptr || packed == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  if (misaligned(offsets, 4) || misaligned(x, 16) || misaligned(packed, 16) || misaligned(bias, es) || misaligned(y, os))
    return MOE_ERR_INVALID_ARG;
  if (y == x || y == packed || y == bias) return MOE_ERR_INVALID_ARG;  // other pieces still read what one has overwritten
  if (launch_q4_matmul(*m, offsets, x, packed, bias, y, static_cast<int32_t*>(ws), stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++launch_count();
  return MOE_OK;
}

}  // extern "C"
