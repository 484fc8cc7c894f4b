// Products with 4-bit expert weights, for serving: rows grouped by expert, a few rows each.
//   y[r,n] = act( sum_k x[r,k] s[e,k/G,n] (c[e,n,k] - 8) + b[e,n] ),   c in 0..15, s bf16, G = 32, 64 or 128
// ("MoE Training: Mixture of Experts" page, Quick Start: the expert's Linear layers, with the weights held in
// 4 bits and a scale for each group of G inputs of an output column.)
//
// Bound: reading the weights from HBM (half a byte each), as decode with bf16 weights is by four times the bytes.
// Mathematics: a group's sum  d[n,r] = sum_{k in group} (c - 8) x[r,k]  runs on mma.sync m16n8k16 with the weights
// as the 16-row operand (c - 8 is exact in bf16) and eight rows of x as the 8-column one, and joins the fp32
// accumulator as  acc += s d:  no weight is rounded, and tensor-core sums (which cut) are at most 64 terms long.
// fp32 rows are split exactly into three bf16 parts (8 bits of the significand each), three products a step.
// mma.sync rather than tcgen05: at up to 32 rows the product is 1 / 8 of what the tensor pipe could do in the time
// that the weights take, and its register operand is what unpacking produces; tcgen05 wants them in shared memory.
//
// Layout (moe_q4_pack): 16 columns x 128 inputs make a block of 1024 bytes of codes in the order of the
// mma's register operand, then the block's scales; the blocks of up to 16 column tiles at one 128-input step lie
// together, so a CTA's step is one contiguous run of up to 18 KB that one bulk copy brings.
// Split: work is (256-column strip of an expert, up to 32 rows of it) x steps of 128 inputs; the steps of all of it
// laid end to end are shared evenly over one CTA per SM.  A CTA that holds part of a strip's steps leaves its
// fp32 sums in the workspace, and the last one to finish adds them in CTA order (the same bits every run).
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

constexpr int kWarps = 16;              // consumer warps: one 16-column tile each
constexpr int kRows = 32;               // rows of a work item (four mma column groups)
constexpr int kStepK = 128;             // inputs of a pipeline step
constexpr int kThreadsQ4 = 32 * (kWarps + 1);
constexpr int kXPitch = kStepK * 2 + 64;  // bytes between staged bf16 rows: reads of 8 rows x 16 bytes miss no bank twice
constexpr int kMaxCtas = 160;
constexpr size_t kCounterOff = 256, kPartialOff = 4096;
constexpr size_t kPartialBytes = (size_t)kWarps * (kRows / 8) * 32 * 16;  // fp32 sums of a 256 x 32 strip
constexpr size_t kQ4WsBytes = kPartialOff + (size_t)kMaxCtas * 2 * kPartialBytes;

__host__ __device__ constexpr int block_bytes(int group) { return 1024 + (kStepK / group) * 32; }

struct Q4Shape {  // the packed layout of one expert
  int tiles, steps, blk;
  __host__ __device__ Q4Shape(int K, int N, int group)
      : tiles((N + 15) / 16), steps((K + kStepK - 1) / kStepK), blk(block_bytes(group)) {}
  __host__ __device__ size_t expert_bytes() const { return (size_t)tiles * steps * blk; }
  __host__ __device__ int strip_tiles(int strip) const { return tiles - strip * kWarps < kWarps ? tiles - strip * kWarps : kWarps; }
  // first block of a strip's step
  __host__ __device__ size_t at(int strip, int step) const {
    return ((size_t)strip * kWarps * steps + (size_t)step * strip_tiles(strip)) * blk;
  }
};

struct Q4Args {
  const int32_t* offsets;
  const uint8_t* x;
  const uint8_t* w;
  const void* bias;
  void* y;
  int32_t* status;
  unsigned* counters;
  float4* partials;
  long long rows_cap, ldx, ldy;
  int E, K, N, act, bf16_out;
  long long wait_limit;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
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
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// all consumer threads meet; true when every one of them says so
__device__ __forceinline__ bool consumers_all(bool ok) {
  int r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbarrier.red.and.pred q, 1, %2, p;\nselp.b32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)ok), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The eight codes of a word (four in each half) as bf16 pairs: 0x4300 | c is 128 + c in bf16 (step 1 there), and
// taking 136 away is exact.
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&a)[4]) {
  const __nv_bfloat162 bias = __halves2bfloat162(__float2bfloat16_rn(136.f), __float2bfloat16_rn(136.f));
#pragma unroll
  for (int f = 0; f < 4; ++f) {
    const uint32_t v = ((w >> (4 * f)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 h = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), bias);
    a[f] = *reinterpret_cast<const uint32_t*>(&h);
  }
}

// One step of a warp's tile: GP groups a step, P bf16 planes of x, RB groups of 8 rows, k32 blocks of 32 inputs.
template <int GP, int P, int RB>
__device__ __forceinline__ void q4_step(float (&acc)[kRows / 8][4], uint32_t wblk, uint32_t xs, int k32, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t xrow = xs + (uint32_t)(g * kXPitch + t * 16);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    if (2 * u >= k32) break;
    const uint4 wv = lds128(wblk + u * 512 + lane * 16);
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
    float d[RB][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (2 * u + h >= k32) break;
      uint32_t a0[4], a1[4];
      unpack_codes(ww[2 * h], a0);
      unpack_codes(ww[2 * h + 1], a1);
      if (GP == 4 || h == 0) {
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) d[rb][0] = d[rb][1] = d[rb][2] = d[rb][3] = 0.f;
      }
#pragma unroll
      for (int p = P - 1; p >= 0; --p)  // the smallest part of x first
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const uint4 xv = lds128(xrow + (uint32_t)(p * kRows * kXPitch + rb * 8 * kXPitch + (2 * u + h) * 64));
          mma16816(d[rb], a0, xv.x, xv.y);
          mma16816(d[rb], a1, xv.z, xv.w);
        }
      if (GP == 4 || h == 1 || 2 * u + 1 == k32) {  // the group's end, or half of a 128-input one
        const int grp = GP == 4 ? 2 * u + h : (GP == 2 ? u : 0);
        const uint32_t sc = lds32(wblk + 1024 + grp * 32 + g * 4);
        const float s0 = __uint_as_float(sc << 16), s1 = __uint_as_float(sc & 0xffff0000u);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          acc[rb][0] = fmaf(s0, d[rb][0], acc[rb][0]);
          acc[rb][1] = fmaf(s0, d[rb][1], acc[rb][1]);
          acc[rb][2] = fmaf(s1, d[rb][2], acc[rb][2]);
          acc[rb][3] = fmaf(s1, d[rb][3], acc[rb][3]);
        }
      }
    }
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

template <bool F32X>
struct Q4Cfg {
  static constexpr int kXBytes = F32X ? kRows * kStepK * 4 : kRows * kXPitch;
  static constexpr int kWBytes = kWarps * block_bytes(32);
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kStages = F32X ? 4 : 6;
  static constexpr int kPlaneOff = kStages * kStageBytes;
  static constexpr int kPlaneBytes = F32X ? 2 * 3 * kRows * kXPitch : 0;  // double-buffered
  static constexpr int kBarOff = kPlaneOff + kPlaneBytes;
  static constexpr int kMiscOff = kBarOff + 2 * kStages * 8;
  static constexpr int kOffsOff = kMiscOff + 16;
  static constexpr int kSmemBytes = 128 + kOffsOff + 2 * 260 * 4;
  static_assert(kSmemBytes <= 232448 && kStageBytes % 128 == 0 && kBarOff % 16 == 0, "shared-memory plan");
};

// The work of all CTAs laid end to end: items of `steps` steps, item i of expert e, strip, row block.
struct Q4Item {
  int e, strip, row0, rows;
};
__device__ __forceinline__ Q4Item find_item(long long i, const int* offs, const int* prefix, int E, int strips) {
  Q4Item it;
  it.e = find_segment(prefix, E, (int)(i / strips));
  const int blocks = prefix[it.e + 1] - prefix[it.e];
  const long long local = i - (long long)prefix[it.e] * strips;
  it.strip = (int)(local / blocks);
  const int rb = (int)(local % blocks);  // row blocks of one strip follow each other: its weights come from L2 then
  it.row0 = offs[it.e] + rb * kRows;
  it.rows = min(kRows, offs[it.e + 1] - it.row0);
  return it;
}

template <int GP, bool F32X>
__global__ void __launch_bounds__(kThreadsQ4, 1) q4_matmul_kernel(Q4Args a) {
  using C = Q4Cfg<F32X>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~(uintptr_t)127);
  const uint32_t sbase = smem_u32(smem);
  auto full_bar = [&](int s) { return sbase + C::kBarOff + 8u * s; };
  auto empty_bar = [&](int s) { return sbase + C::kBarOff + 8u * (C::kStages + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff);
  volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  int* offs = reinterpret_cast<int*>(smem + C::kOffsOff);
  int* prefix = offs + 260;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), kWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    fence_async_smem();
  }
  if (warp == 0) load_segments(a.offsets, a.E, a.rows_cap, kRows, 1, offs, prefix, a.status, blockIdx.x == 0);
  __syncthreads();

  const Q4Shape q(a.K, a.N, kStepK / GP);
  const int strips = (q.tiles + kWarps - 1) / kWarps;
  const long long total = (long long)prefix[a.E] * strips * q.steps;
  const long long ctas = min((long long)gridDim.x, total);  // every CTA up to here has a step at least
  const int c = blockIdx.x;
  const long long u0 = c < ctas ? total * c / ctas : 0, u1 = c < ctas ? total * (c + 1) / ctas : 0;

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer ---------------------
    int stage = 0;
    uint32_t phase = 0;
    int armed[C::kStages];
#pragma unroll
    for (int s = 0; s < C::kStages; ++s) armed[s] = -1;
    bool ok = true;
    constexpr int ES = F32X ? 4 : 2;
    for (long long u = u0; u < u1 && ok;) {
      const long long item = u / q.steps;
      const int k_first = (int)(u - item * q.steps);
      const int k_last = (int)min((long long)q.steps, k_first + (u1 - u));
      const Q4Item it = find_item(item, offs, prefix, a.E, strips);
      const int nt = q.strip_tiles(it.strip);
      const uint8_t* w = a.w + (size_t)it.e * q.expert_bytes();
      const uint8_t* xrow = a.x + ((size_t)it.row0 + lane) * a.ldx * ES;
      for (int k = k_first; k < k_last; ++k) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(stage), phase ^ 1u, a.wait_limit, abort_flag, a.status,
                                               kDevTimeoutProducer))) {
          ok = false;
          break;
        }
        const uint32_t dst = sbase + stage * C::kStageBytes;
        const uint32_t wbytes = (uint32_t)(nt * q.blk), xbytes = (uint32_t)(min(kStepK, a.K - k * kStepK) * ES);
        if (lane == 0) {
          mbar_arrive_expect_tx(full_bar(stage), wbytes + (uint32_t)it.rows * xbytes);
          bulk_load(dst, w + q.at(it.strip, k), wbytes, full_bar(stage));
        }
        __syncwarp();
        if (lane < it.rows)
          bulk_load(dst + C::kWBytes + lane * (F32X ? kStepK * 4 : kXPitch), xrow + (size_t)k * kStepK * ES, xbytes,
                    full_bar(stage));
#pragma unroll
        for (int s = 0; s < C::kStages; ++s)
          if (s == stage) armed[s] = (int)phase;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      u += k_last - k_first;
    }
    if (!ok || *abort_flag) {
      // every armed stage's copies must land before the CTA exits
#pragma unroll
      for (int s = 0; s < C::kStages; ++s)
        if (armed[s] >= 0) {
          volatile int dummy = 0;
          mbar_wait(full_bar(s), (uint32_t)armed[s], a.wait_limit, &dummy, a.status, kDevTimeoutDrain);
        }
    }
    return;
  }

  // -------------------------------------------------------------- consumers --------------------
  const int g = lane >> 2, t = lane & 3;
  int stage = 0, plane = 0;
  uint32_t phase = 0;
  bool ok = true;  // after a wait that ran out the loops go on without work, so that the barriers below still match
  for (long long u = u0; u < u1;) {
    const long long item = u / q.steps;
    const int k_first = (int)(u - item * q.steps);
    const int k_last = (int)min((long long)q.steps, k_first + (u1 - u));
    const Q4Item it = find_item(item, offs, prefix, a.E, strips);
    const int nt = q.strip_tiles(it.strip);
    const bool mine = warp < nt;
    const int nrb = (it.rows + 7) / 8;
    float acc[kRows / 8][4] = {};
    for (int k = k_first; k < k_last; ++k) {
      if (ok) ok = mbar_wait(full_bar(stage), phase, a.wait_limit, abort_flag, a.status, kDevTimeoutMma);
      ok = __all_sync(0xffffffffu, ok);
      const uint32_t st = sbase + stage * C::kStageBytes;
      const int kk = min(kStepK, a.K - k * kStepK);
      uint32_t xs = st + C::kWBytes;
      if constexpr (F32X) {
        // eight inputs of one row a thread: raw fp32 into three planes of bf16
        const uint32_t raw = xs;
        xs = sbase + C::kPlaneOff + plane * (3 * kRows * kXPitch);
        const int row = threadIdx.x >> 4, seg = threadIdx.x & 15;
        if (ok && row < it.rows && seg * 8 < kk) {
          const uint4 v0 = lds128(raw + row * (kStepK * 4) + seg * 32), v1 = lds128(raw + row * (kStepK * 4) + seg * 32 + 16);
          const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
          uint32_t p[3][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t lo[3], hi[3];
            split3(__uint_as_float(v[2 * j]), lo[0], lo[1], lo[2]);
            split3(__uint_as_float(v[2 * j + 1]), hi[0], hi[1], hi[2]);
#pragma unroll
            for (int i = 0; i < 3; ++i) p[i][j] = __byte_perm(lo[i], hi[i], 0x7632);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i)
            sts128(xs + i * kRows * kXPitch + row * kXPitch + seg * 16, p[i][0], p[i][1], p[i][2], p[i][3]);
        }
        plane ^= 1;  // the other planes are free: every warp has passed the barrier behind their last use
        ok = consumers_all(ok);
      }
      if (ok && mine) {
        const uint32_t wblk = st + warp * q.blk;
        constexpr int P = F32X ? 3 : 1;
        if (nrb == 1) q4_step<GP, P, 1>(acc, wblk, xs, kk / 32, lane);
        else if (nrb == 2) q4_step<GP, P, 2>(acc, wblk, xs, kk / 32, lane);
        else q4_step<GP, P, 4>(acc, wblk, xs, kk / 32, lane);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(stage));
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    u += k_last - k_first;

    bool write = ok;
    if (k_last - k_first < q.steps) {
      // part of the item's sum: leave it, and let the last of its CTAs add all parts
      const long long f = item * q.steps;
      const int c0 = (int)(((f + 1) * ctas - 1) / total), c1 = (int)(((f + q.steps) * ctas - 1) / total);
      auto slot = [&](int cta) {  // a CTA's first item may have begun before it, its last one end after it
        return a.partials + ((size_t)cta * 2 + (cta > c0 ? 0 : 1)) * (kPartialBytes / 16) + (size_t)warp * (kRows / 8) * 32 + lane;
      };
      if (mine) {
        float4* dst = slot(c);
#pragma unroll
        for (int rb = 0; rb < kRows / 8; ++rb)
          if (rb < nrb) __stcg(dst + rb * 32, make_float4(acc[rb][0], acc[rb][1], acc[rb][2], acc[rb][3]));
      }
      __threadfence();
      write = consumers_all(ok);
      if (threadIdx.x == 0) {
        int last = 0;
        if (write) {
          last = atomicAdd(a.counters + c0, 1u) == (unsigned)(c1 - c0);
          if (last) a.counters[c0] = 0;  // for the next call
        }
        *last_flag = last;
        __threadfence();
      }
      consumers_all(true);
      write = *last_flag != 0;
      if (write && mine) {
#pragma unroll
        for (int rb = 0; rb < kRows / 8; ++rb) acc[rb][0] = acc[rb][1] = acc[rb][2] = acc[rb][3] = 0.f;
        for (int o = c0; o <= c1; o += 4) {
          float4 v[4][kRows / 8];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int rb = 0; rb < kRows / 8; ++rb)
              v[j][rb] = o + j <= c1 && rb < nrb ? __ldcg(slot(o + j) + rb * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int rb = 0; rb < kRows / 8; ++rb) {
              acc[rb][0] += v[j][rb].x;
              acc[rb][1] += v[j][rb].y;
              acc[rb][2] += v[j][rb].z;
              acc[rb][3] += v[j][rb].w;
            }
        }
      }
    }
    if (write && mine) {
      // lane: columns n and n + 8, rows 2t and 2t + 1 of each group of 8
      const int n0 = it.strip * (16 * kWarps) + warp * 16 + g;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + (j >> 1) * 8;
        if (n >= a.N) continue;
        float b = 0.f;
        if (a.bias != nullptr)
          b = F32X ? static_cast<const float*>(a.bias)[(size_t)it.e * a.N + n]
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[(size_t)it.e * a.N + n]);
#pragma unroll
        for (int rb = 0; rb < kRows / 8; ++rb) {
          const int r = rb * 8 + 2 * t + (j & 1);
          if (r >= it.rows) continue;
          float v = acc[rb][j] + b;
          const size_t at = ((size_t)it.row0 + r) * a.ldy + n;
          if (a.bf16_out) {
            if (a.act == MOE_ACT_GELU) v = activate<MOE_ACT_GELU, true>(v);
            else if (a.act == MOE_ACT_SILU) v = activate<MOE_ACT_SILU, true>(v);
            static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
          } else {
            if (a.act == MOE_ACT_GELU) v = activate<MOE_ACT_GELU, false>(v);
            else if (a.act == MOE_ACT_SILU) v = activate<MOE_ACT_SILU, false>(v);
            static_cast<float*>(a.y)[at] = v;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- laying the weights out --------
// One thread a lane's 16 bytes of a tile's 64 inputs: word 2h + i holds inputs 32h + 8t + 4i + {0..3} of columns
// g and g + 8, its 16-bit halves the even and the odd ones, each with (g, first), (g + 8, first), (g, second),
// (g + 8, second).  Columns and inputs past the edge are code 8 (zero) with scale zero.
__global__ void __launch_bounds__(256) q4_pack_kernel(int E, int K, int N, int group, const uint8_t* __restrict__ q,
                                                      const uint16_t* __restrict__ s, uint8_t* __restrict__ packed) {
  const Q4Shape sh(K, N, group);
  const long long units = (long long)E * sh.tiles * sh.steps * 2;
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (i >= units) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int u = (int)(i & 1);
  const long long b = i >> 1;
  const int step = (int)(b % sh.steps);
  const int tile = (int)((b / sh.steps) % sh.tiles), e = (int)(b / sh.steps / sh.tiles);
  const int strip = tile / kWarps;
  uint8_t* dst = packed + (size_t)e * sh.expert_bytes() + sh.at(strip, step) + (size_t)(tile - strip * kWarps) * sh.blk;
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
      w[2 * h + p] = r;
    }
  }
  *reinterpret_cast<uint4*>(dst + u * 512 + lane * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  const int gp = kStepK / group;
  if (u == 0 && lane < gp * 8) {
    const int grp = lane >> 3, kg = step * gp + grp, groups = K / group;
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = tile * 16 + (lane & 7) + 8 * j;
      if (n < N && kg < groups) v |= (uint32_t)s[((size_t)e * groups + kg) * N + n] << (16 * j);
    }
    *reinterpret_cast<uint32_t*>(dst + 1024 + lane * 4) = v;
  }
}

// The value of one weight in the packed layout
__device__ __forceinline__ float q4_value(const uint8_t* expert, const Q4Shape& sh, int group, int k, int n) {
  const int tile = n >> 4, strip = tile / kWarps, step = k / kStepK, r = k % kStepK;
  const uint8_t* blk = expert + sh.at(strip, step) + (size_t)(tile - strip * kWarps) * sh.blk;
  const int lane = (n & 7) * 4 + ((r & 31) >> 3);
  const int word = ((r & 63) >> 5) * 2 + ((r & 7) >> 2), field = ((r & 3) >> 1) * 2 + ((n >> 3) & 1);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + (r >> 6) * 512 + lane * 16 + word * 4);
  const int code = (int)((w >> (16 * (r & 1) + 4 * field)) & 15u);
  const uint32_t sc = *reinterpret_cast<const uint32_t*>(blk + 1024 + (r / group) * 32 + (n & 7) * 4);
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
  return MOE_OK;
}

unsigned copy_grid(long long threads) {
  const long long blocks = (threads + 255) / 256;
  return (unsigned)(blocks < 1 << 20 ? blocks : 1 << 20);
}

template <int GP, bool F32X>
cudaError_t launch_q4(const Q4Args& a, int grid, cudaStream_t st) {
  const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(q4_matmul_kernel<GP, F32X>), Q4Cfg<F32X>::kSmemBytes);
  if (err != cudaSuccess) return err;
  q4_matmul_kernel<GP, F32X><<<grid, kThreadsQ4, Q4Cfg<F32X>::kSmemBytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

moe_status_t check_q4_matmul(const moe_q4_t* m, const void* ws, size_t ws_bytes) {
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
  if (ldx >= (1LL << 31) || ldy >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (ws == nullptr || misaligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < kQ4WsBytes) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// m, ws and the pointers have been checked; status may be another workspace's error word
cudaError_t launch_q4_matmul(const moe_q4_t& m, const int32_t* offsets, const void* x, const void* packed, const void* bias,
                             void* y, void* ws, int32_t* status, cudaStream_t st) {
  Q4Args a{};
  a.offsets = offsets;
  a.x = static_cast<const uint8_t*>(x);
  a.w = static_cast<const uint8_t*>(packed);
  a.bias = bias;
  a.y = y;
  a.status = status;
  a.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + kCounterOff);
  a.partials = reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + kPartialOff);
  a.rows_cap = m.rows_cap;
  a.ldx = m.ldx == 0 ? m.K : m.ldx;
  a.ldy = m.ldy == 0 ? m.N : m.ldy;
  a.E = m.E;
  a.K = m.K;
  a.N = m.N;
  a.act = m.activation;
  a.bf16_out = m.out_dtype == MOE_DTYPE_BF16;
  a.wait_limit = wait_limit();
  const Q4Shape q(m.K, m.N, m.group);
  const long long most = (m.rows_cap / kRows + (m.rows_cap < m.E ? m.rows_cap : m.E)) * ((q.tiles + kWarps - 1) / kWarps) * q.steps;
  int grid = sm_count();
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (grid > most) grid = (int)most;
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
  const long long blocks = ((long long)E * q.tiles * q.steps * 2 + 7) / 8;
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
  const moe_status_t st = check_q4_matmul(m, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (m->rows_cap == 0) return MOE_OK;
  const uintptr_t es = m->dtype == MOE_DTYPE_BF16 ? 2 : 4, os = m->out_dtype == MOE_DTYPE_BF16 ? 2 : 4;
  if (offsets == nullptr || x == nullptr || packed == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  if (misaligned(offsets, 4) || misaligned(x, 16) || misaligned(packed, 16) || misaligned(bias, es) || misaligned(y, os))
    return MOE_ERR_INVALID_ARG;
  if (launch_q4_matmul(*m, offsets, x, packed, bias, y, ws, static_cast<int32_t*>(ws), stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  ++launch_count();
  return MOE_OK;
}

}  // extern "C"
