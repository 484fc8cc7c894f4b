// Matrix products grouped by expert over ragged row segments, as entry points of their own:
//   moe_grouped_matmul   y[r,n] = sum_k x[r,k] W[e,k,n] + b[e,n]      (or W[e,n,k])
//   moe_grouped_wgrad    dW[e,k,n] = sum_{r in e} x[r,k] dy[r,n],  db[e,n] = sum_{r in e} dy[r,n]
// ("MoE Training: Mixture of Experts" page, Quick Start: the expert's two Linear layers, and the chain
// rule through them.)  bf16 runs on the tcgen05 kernels of grouped_gemm_sm100.cu; this file holds the
// argument checks, the fp32 products on CUDA cores and the bias gradient.
#include <cuda_bf16.h>
#include <stdint.h>

#include "moe_internal.cuh"
#include "segments.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------- fp32 products ----------------
// One 64 x 128 output tile per block, 128 threads of 8 x 8 outputs, contraction in steps of 16 through a
// double-buffered pair of shared tiles [k][m], [k][n].  Bound: the FMA pipes.  A thread reads 8 + 8 words
// of shared memory per k (6 wavefronts a warp, 24 of the 64 cycles its 32 packed FMAs take on four
// sub-partitions) and issues them as fma.rn.f32x2, two products an instruction, which leaves issue slots
// for the loads.  64-row tiles rather than 128: ragged segments of a few dozen rows waste less of them.
// Where that gives too few tiles, 64 x 64 ones, and up to 8 groups of threads that share a tile's steps and add their
// sums at the end: a warp or two a sub-partition leave the latency of every step open (1003 rows of 516 x 780 for 16
// experts: 100 us with one group of 128 threads a tile, see launch_f32 for the rest).  Where even those leave SMs idle
// and the contraction is long, a cluster's blocks share it and add their sums through distributed shared memory, each a
// share of them, in the blocks' order (f32_parts).
constexpr int FM = 64, FK = 16;
constexpr int FA = FM + 4;  // padded rows: 16-byte reads stay aligned

enum { MODE_NN = 0, MODE_NT = 1, MODE_TN = 2 };

struct F32Args {
  const int32_t* offsets;
  int E;
  long long rows_cap;
  const float* A;  // NN, NT: x rows; TN: x rows
  const float* B;  // NN: W[E,K,N]; NT: W[E,N,K]; TN: dy rows
  long long lda, ldb;
  const float* bias;
  float* D;
  long long ldd;
  int M, N, K;  // TN: M x N per expert, contraction over its rows; else N columns, contraction K
  int parts;    // blocks of a cluster (along z) that share a tile's contraction: 1, 2, 4 or 8
  int32_t* status;
};

__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

__device__ __forceinline__ void fma2(unsigned long long& d, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ void add2(unsigned long long& d, unsigned long long a) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(a));
}
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}

// this thread's four sums of the same shared-memory words in every block of the cluster, added in the blocks' order
__device__ __forceinline__ ulonglong2 cluster_sum(const ulonglong2* own, int parts) {
  ulonglong2 sum = make_ulonglong2(0ull, 0ull);
  for (int b = 0; b < parts; ++b) {
    const uint32_t at = sm100::peer_addr((uint32_t)__cvta_generic_to_shared(own), (uint32_t)b);
    ulonglong2 v;
    asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];\n" : "=l"(v.x), "=l"(v.y) : "r"(at) : "memory");
    add2(sum.x, v.x);
    add2(sum.y, v.y);
  }
  return sum;
}

constexpr int f32_group_floats(int fn) { return 2 * FK * (FA + fn + 4); }
constexpr int f32_smem(int fn, int groups) {
  const int steps = groups * f32_group_floats(fn) * 4, sums = (groups - (groups < 8)) * FM * fn * 4;  // 8: its own too
  return (steps > sums ? steps : sums);
}

// Blocks an SM holds at least (0: as the registers fall out).  Two of 4 groups, in 128 registers a thread, although a few
// words then spill (1003 rows of 516 x 780 for 16 experts 60 -> 49 us).  Four of 2 groups would spill too and lose by it
// (2500 rows of 712 x 1000 for 126 experts 262 and 271 us).
constexpr int f32_blocks(int groups) { return groups == 4 ? 2 : 0; }

template <int MODE, int FN, int KG>
__global__ void __launch_bounds__(FN * KG, f32_blocks(KG)) matmul_f32_kernel(F32Args a) {
  constexpr int FT = FN, FB = FN + 4;  // threads of a group: 8 x 8 outputs each
  constexpr int kGroup = f32_group_floats(FN);
  __shared__ int offs[kMaxExperts + 1], prefix[kMaxExperts + 1];
  extern __shared__ __align__(16) float tiles[];
  const int tid = threadIdx.x % FT, group = threadIdx.x / FT;
  float(*As)[FK][FA] = reinterpret_cast<float(*)[FK][FA]>(tiles + group * kGroup);
  float(*Bs)[FK][FB] = reinterpret_cast<float(*)[FK][FB]>(tiles + group * kGroup + 2 * FK * FA);
  auto group_sync = [&]() {
    if constexpr (KG == 1) __syncthreads();
    else asm volatile("barrier.sync %0, %1;\n" ::"r"(1 + group), "n"(FT) : "memory");
  };
  if (threadIdx.x < 32)
    load_segments(a.offsets, a.E, a.rows_cap, FM, 1, offs, MODE == MODE_TN ? nullptr : prefix, a.status,
                  blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
  __syncthreads();
  const int parts = KG == 8 ? a.parts : 1;
  int e, m0, mrows, K;  // mrows: valid output rows of the tile
  long long arow0;      // first A row of the tile (NN, NT), first contraction row (TN)
  if constexpr (MODE == MODE_TN) {
    e = blockIdx.z / parts;
    m0 = blockIdx.x * FM;
    mrows = min(FM, a.M - m0);
    arow0 = offs[e];
    K = offs[e + 1] - offs[e];
  } else {
    if ((int)blockIdx.x >= prefix[a.E]) return;
    e = find_segment(prefix, a.E, blockIdx.x);
    const int ml = ((int)blockIdx.x - prefix[e]) * FM;
    m0 = 0;
    arow0 = (long long)offs[e] + ml;
    mrows = min(FM, offs[e + 1] - offs[e] - ml);
    K = a.K;
  }
  const int n0 = blockIdx.y * FN, ncols = min(FN, a.N - n0);
  const float* A = a.A + arow0 * a.lda + m0;
  const float* B = MODE == MODE_NN   ? a.B + (size_t)e * a.K * a.N + n0
                   : MODE == MODE_NT ? a.B + (size_t)e * a.K * a.N + (size_t)n0 * a.K
                                     : a.B + arow0 * a.ldb + n0;
  const long long ldb = MODE == MODE_NN ? a.N : (MODE == MODE_NT ? a.K : a.ldb);
  if (KG == 8 && parts > 1) {  // this block's share of the contraction
    const int share = (K + parts * FK - 1) / (parts * FK) * FK, k0 = (int)(blockIdx.z % parts) * share;
    A += MODE == MODE_TN ? k0 * a.lda : k0;
    B += MODE == MODE_NT ? k0 : k0 * ldb;
    K = min(share, K - k0);  // 0 or less: nothing left
  }

  // this thread's 16-byte pieces of the next k step (K, M, N are multiples of 4, so a piece
  // is wholly inside or wholly outside)
  constexpr int PA = FM * FK / 4 / FT, PB = FN * FK / 4 / FT;
  float4 ra[PA], rb[PB];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < PA; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_TN) {  // 16 rows of 64 columns
        const int kk = i >> 4, c = (i & 15) * 4;
        ra[j] = k0 + kk < K && c < mrows ? __ldg(reinterpret_cast<const float4*>(A + (long long)(k0 + kk) * a.lda + c))
                                         : zero4();
      } else {  // 64 rows of 16 columns
        const int r = i >> 2, kk = (i & 3) * 4;
        ra[j] = r < mrows && k0 + kk < K ? __ldg(reinterpret_cast<const float4*>(A + (long long)r * a.lda + k0 + kk))
                                         : zero4();
      }
    }
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_NT) {
        const int r = i >> 2, kk = (i & 3) * 4;
        rb[j] = r < ncols && k0 + kk < K ? __ldg(reinterpret_cast<const float4*>(B + (long long)r * ldb + k0 + kk))
                                         : zero4();
      } else {
        const int kk = i / (FN / 4), c = (i % (FN / 4)) * 4;
        rb[j] = k0 + kk < K && c < ncols ? __ldg(reinterpret_cast<const float4*>(B + (long long)(k0 + kk) * ldb + c))
                                         : zero4();
      }
    }
  };
  auto put = [&](int s) {
#pragma unroll
    for (int j = 0; j < PA; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_TN) {
        *reinterpret_cast<float4*>(&As[s][i >> 4][(i & 15) * 4]) = ra[j];
      } else {
        const int r = i >> 2, kk = (i & 3) * 4;
        As[s][kk][r] = ra[j].x;
        As[s][kk + 1][r] = ra[j].y;
        As[s][kk + 2][r] = ra[j].z;
        As[s][kk + 3][r] = ra[j].w;
      }
    }
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_NT) {
        const int r = i >> 2, kk = (i & 3) * 4;
        Bs[s][kk][r] = rb[j].x;
        Bs[s][kk + 1][r] = rb[j].y;
        Bs[s][kk + 2][r] = rb[j].z;
        Bs[s][kk + 3][r] = rb[j].w;
      } else {
        *reinterpret_cast<float4*>(&Bs[s][i / (FN / 4)][(i % (FN / 4)) * 4]) = rb[j];
      }
    }
  };

  const int tx = tid % (FN / 8), ty = tid / (FN / 8);  // columns 4 tx .. and FN / 2 + 4 tx .., rows 8 ty ..
  unsigned long long acc[8][4] = {};
  int s = 0;
  const int first = group * FK;  // a group takes every KG-th step
  if (first < K) {
    fetch(first);
    put(0);
  }
  group_sync();
  for (int k0 = first; k0 < K; k0 += KG * FK) {
    const bool more = k0 + KG * FK < K;
    if (more) fetch(k0 + KG * FK);
#pragma unroll
    for (int kk = 0; kk < FK; ++kk) {
      const float4 a0 = *reinterpret_cast<const float4*>(&As[s][kk][ty * 8]);
      const float4 a1 = *reinterpret_cast<const float4*>(&As[s][kk][ty * 8 + 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&Bs[s][kk][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&Bs[s][kk][FN / 2 + tx * 4]);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned long long aa = pack2(av[i], av[i]);
        fma2(acc[i][0], aa, b0.x);
        fma2(acc[i][1], aa, b0.y);
        fma2(acc[i][2], aa, b1.x);
        fma2(acc[i][3], aa, b1.y);
      }
    }
    if (more) put(s ^ 1);
    group_sync();
    s ^= 1;
  }
  if constexpr (KG > 1) {
    // the groups' sums, in order
    ulonglong2* sums = reinterpret_cast<ulonglong2*>(tiles);
    __syncthreads();  // the tiles have been read
    if (group > 0) {
#pragma unroll
      for (int q = 0; q < 16; ++q) sums[((group - 1) * 16 + q) * FT + tid] = make_ulonglong2(acc[q >> 1][2 * (q & 1)], acc[q >> 1][2 * (q & 1) + 1]);
    }
    __syncthreads();
    if (group == 0) {
      for (int o = 0; o < KG - 1; ++o)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const ulonglong2 v = sums[(o * 16 + q) * FT + tid];
          add2(acc[q >> 1][2 * (q & 1)], v.x);
          add2(acc[q >> 1][2 * (q & 1) + 1], v.y);
        }
    }
  }

  float* D = MODE == MODE_TN ? a.D + (size_t)e * a.M * a.N + (size_t)m0 * a.N + n0 : a.D + arow0 * a.ldd + n0;
  const long long ldd = MODE == MODE_TN ? a.N : a.ldd;
  if constexpr (KG == 8) {
    if (parts > 1) {
      // the blocks' sums, 16 bytes a thread: block p finishes pieces 16 p / parts .. of every thread's 16
      ulonglong2* mine = reinterpret_cast<ulonglong2*>(tiles + (KG - 1) * FM * FN);
      if (group == 0) {
#pragma unroll
        for (int q = 0; q < 16; ++q) mine[q * FT + tid] = make_ulonglong2(acc[q >> 1][2 * (q & 1)], acc[q >> 1][2 * (q & 1) + 1]);
      }
      sm100::cluster_sync_all();
      const int part = blockIdx.z % parts;
      const int q = part * (16 / parts) + group, c = (q & 1) * (FN / 2) + tx * 4, r = ty * 8 + (q >> 1);
      if (group < 16 / parts && c < ncols && r < mrows) {
        const ulonglong2 sum = cluster_sum(mine + q * FT + tid, parts);
        const float4 b = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + (size_t)e * a.N + n0 + c)) : zero4();
        float4 v;
        unpack2(sum.x, v.x, v.y);
        unpack2(sum.y, v.z, v.w);
        v.x += b.x;
        v.y += b.y;
        v.z += b.z;
        v.w += b.w;
        *reinterpret_cast<float4*>(D + (long long)r * ldd + c) = v;
      }
      __syncwarp();
      sm100::cluster_sync_all();  // no block leaves while another may still read its sums
      return;
    }
  }
  if (group > 0) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = h * (FN / 2) + tx * 4;
    if (c >= ncols) continue;
    const float4 b = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + (size_t)e * a.N + n0 + c)) : zero4();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = ty * 8 + i;
      if (r >= mrows) break;
      float4 v;
      unpack2(acc[i][2 * h], v.x, v.y);
      unpack2(acc[i][2 * h + 1], v.z, v.w);
      v.x += b.x;
      v.y += b.y;
      v.z += b.z;
      v.w += b.w;
      *reinterpret_cast<float4*>(D + (long long)r * ldd + c) = v;
    }
  }
}

// ---------------------------------------------------------------- fp32 products of a few rows ----
// Up to 8 rows of an expert a block, where a 64-row tile would multiply mostly zeros.  Bound: reading W.  16 warps; x in
// shared memory, 1024 inputs at a time.  W[E,K,N]: a lane has 4 columns (128 a block) and a warp every 16th run of 4
// inputs, the warps' sums join in shared memory.  W[E,N,K]: a warp has 4 columns (64 a block), its lanes share the
// inputs, 128 a step, and join by shuffles.  Both in a fixed order.  A cluster's blocks share a long K where there are few
// (f32_parts).
constexpr int kFewRows = 8, kFewWarps = 16, kFewK = 1024, kFewAvg = 16;
constexpr int few_cols(int mode) { return mode == MODE_NN ? 128 : 4 * kFewWarps; }
constexpr int few_smem(int mode) {
  const int x = kFewRows * kFewK * 4, sums = mode == MODE_NN ? kFewWarps * kFewRows * 128 * 4 : 0;
  return x > sums ? x : sums;
}

template <int MODE>
__global__ void __launch_bounds__(32 * kFewWarps) matmul_f32_few_kernel(F32Args a) {
  __shared__ int offs[kMaxExperts + 1], prefix[kMaxExperts + 1];
  extern __shared__ __align__(16) float few[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0)
    load_segments(a.offsets, a.E, a.rows_cap, kFewRows, 1, offs, prefix, a.status, blockIdx.x == 0 && blockIdx.y == 0);
  __syncthreads();
  if ((int)blockIdx.x >= prefix[a.E]) return;
  const int e = find_segment(prefix, a.E, blockIdx.x);
  const int row0 = offs[e] + ((int)blockIdx.x - prefix[e]) * kFewRows, rows = min(kFewRows, offs[e + 1] - row0);
  const float* x = a.A + (long long)row0 * a.lda;
  const float* W = a.B + (size_t)e * a.K * a.N;
  const int n0 = blockIdx.y * few_cols(MODE) + (MODE == MODE_NN ? 4 * lane : 4 * warp);  // this lane's (warp's) 4 columns
  const int parts = a.parts, part = blockIdx.z;
  const int share = (a.K + 128 * parts - 1) / (128 * parts) * 128, kfirst = part * share, kend = min(a.K, kfirst + share);
  float acc[kFewRows][4] = {};
  for (int k0 = kfirst; k0 < kend; k0 += kFewK) {
    const int kn = min(kFewK, kend - k0);
    if (k0 > kfirst) __syncthreads();
    for (int i = threadIdx.x; i < kFewRows * kFewK / 4; i += 32 * kFewWarps) {
      const int r = i / (kFewK / 4), k = 4 * (i % (kFewK / 4));
      reinterpret_cast<float4*>(few)[i] =
          r < rows && k < kn ? __ldg(reinterpret_cast<const float4*>(x + (long long)r * a.lda + k0 + k)) : zero4();
    }
    __syncthreads();
    if (MODE == MODE_NN) {
      if (n0 >= a.N) continue;
#pragma unroll 2
      for (int k = 4 * warp; k < kn; k += 4 * kFewWarps) {
        float4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(reinterpret_cast<const float4*>(W + (size_t)(k0 + k + j) * a.N + n0));
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(few + r * kFewK + k);
          const float xv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[r][0] = fmaf(xv[j], w[j].x, acc[r][0]);
            acc[r][1] = fmaf(xv[j], w[j].y, acc[r][1]);
            acc[r][2] = fmaf(xv[j], w[j].z, acc[r][2]);
            acc[r][3] = fmaf(xv[j], w[j].w, acc[r][3]);
          }
        }
      }
    } else {
#pragma unroll 2
      for (int k = 4 * lane; k < kn; k += 128) {
        float4 w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          w[c] = n0 + c < a.N ? __ldg(reinterpret_cast<const float4*>(W + (size_t)(n0 + c) * a.K + k0 + k)) : zero4();
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(few + r * kFewK + k);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            acc[r][c] = fmaf(v.x, w[c].x, fmaf(v.y, w[c].y, fmaf(v.z, w[c].z, fmaf(v.w, w[c].w, acc[r][c]))));
        }
      }
    }
  }
  if (MODE == MODE_NN) {
    __syncthreads();  // x has been read
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
      reinterpret_cast<float4*>(few)[(warp * kFewRows + r) * 32 + lane] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    __syncthreads();
    for (int i = threadIdx.x; i < kFewRows * 128; i += 32 * kFewWarps) {
      const int r = i >> 7, n = blockIdx.y * 128 + (i & 127);
      if (r >= rows || n >= a.N) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += few[w * kFewRows * 128 + i];
      if (parts > 1) {
        few[i] = v;  // nobody else reads these words
        continue;
      }
      if (a.bias) v += __ldg(a.bias + (size_t)e * a.N + n);
      a.D[(long long)(row0 + r) * a.ldd + n] = v;
    }
  } else {
    // 32 sums over 32 lanes: each step halves the sums a lane keeps, until lane 4 r + c has row r, column c
    float v[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) v[q] = acc[q >> 2][q & 3];
#pragma unroll
    for (int h = 16; h > 0; h >>= 1) {
      const bool up = lane & h;
#pragma unroll
      for (int q = 0; q < h; ++q) {
        const float give = up ? v[q] : v[q + h], keep = up ? v[q + h] : v[q];
        v[q] = keep + __shfl_xor_sync(0xffffffffu, give, h);
      }
    }
    const int r = lane >> 2, n = n0 + (lane & 3);
    if (parts > 1) {
      __syncthreads();  // x has been read
      few[r * few_cols(MODE) + 4 * warp + (lane & 3)] = v[0];
    } else if (r < rows && n < a.N)
      a.D[(long long)(row0 + r) * a.ldd + n] = v[0] + (a.bias ? __ldg(a.bias + (size_t)e * a.N + n) : 0.f);
  }
  if (parts > 1) {
    // the blocks' sums, 4 columns a thread, each block its share of them
    constexpr int pieces = kFewRows * few_cols(MODE) / 4;
    __syncwarp();
    sm100::cluster_sync_all();
    const int i = part * (pieces / parts) + threadIdx.x, r = i / (few_cols(MODE) / 4), c = i % (few_cols(MODE) / 4) * 4;
    const int n = blockIdx.y * few_cols(MODE) + c;
    if ((int)threadIdx.x < pieces / parts && r < rows && n < a.N) {
      const ulonglong2 sum = cluster_sum(reinterpret_cast<const ulonglong2*>(few) + i, parts);
      float4 v, b = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + (size_t)e * a.N + n)) : zero4();
      unpack2(sum.x, v.x, v.y);
      unpack2(sum.y, v.z, v.w);
      *reinterpret_cast<float4*>(a.D + (long long)(row0 + r) * a.ldd + n) = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
    }
    __syncwarp();
    sm100::cluster_sync_all();  // no block leaves while another may still read its sums
  }
}

// ---------------------------------------------------------------- bias gradient ----------------
// db[e,n] = sum of dy[r,n] over the expert's rows.  Bound: reading dy, or the latency of a long segment's rows.  A block
// of 32 warps takes one (expert, 32 x V columns) strip, each warp every 32nd row with 8 of them in flight; the warps'
// sums join in shared memory in a fixed order, so there are no atomics and the bits do not change from run to run.
// Where there are fewer strips than SMs, a cluster of 8 blocks shares a strip's rows and joins its sums through
// distributed shared memory, since one SM reads about 95 GB/s (8000 rows of 520 columns: 44 us in 3 blocks, 8 in
// 24).  Otherwise its barriers cost more than they save (64 experts of 1 to 1900 rows: 22 us, 14 without).
constexpr int kDbWarps = 32;

template <typename T, int S>
__global__ void __cluster_dims__(1, 1, S) __launch_bounds__(32 * kDbWarps)
    rows_sum_kernel(const int32_t* __restrict__ offsets, int E, long long rows_cap, const T* __restrict__ dy,
                    long long ldy, int N, float* __restrict__ db) {
  constexpr int V = 16 / sizeof(T);
  __shared__ int offs[kMaxExperts + 1];
  __shared__ float part[kDbWarps][32 * V];
  __shared__ float sum[32 * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  if (warp == 0) load_segments(offsets, E, rows_cap, 1, 1, offs, nullptr, nullptr, false);
  __syncthreads();
  const int r1 = offs[e + 1], n = (blockIdx.x * 32 + lane) * V;
  float acc[V] = {};
  if (n < N) {
    constexpr int U = 8;  // rows in flight
    constexpr int step = kDbWarps * S;
    for (long long r = (long long)offs[e] + blockIdx.z * kDbWarps + warp; r < r1; r += step * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = r + u * step < r1 ? __ldg(reinterpret_cast<const uint4*>(dy + (r + u * step) * ldy + n))
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            acc[2 * j] += __uint_as_float(w[j] << 16);
            acc[2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
          }
        } else {
          acc[0] += __uint_as_float(v[u].x);
          acc[1] += __uint_as_float(v[u].y);
          acc[2] += __uint_as_float(v[u].z);
          acc[3] += __uint_as_float(v[u].w);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) part[warp][j * 32 + lane] = acc[j];
  __syncthreads();
  const int c = threadIdx.x;
  const int col = (blockIdx.x * 32 + (c & 31)) * V + (c >> 5);
  float s = 0.f;
  if (c < 32 * V) {
#pragma unroll
    for (int w = 0; w < kDbWarps; ++w) s += part[w][c];
  }
  if constexpr (S > 1) {
    if (c < 32 * V) sum[c] = s;
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    if (blockIdx.z == 0 && c < 32 * V) {
      for (int b = 1; b < S; ++b) {
        float v;
        asm volatile("{\n.reg .u32 ra;\nmapa.shared::cluster.u32 ra, %1, %2;\nld.shared::cluster.f32 %0, [ra];\n}\n"
                     : "=f"(v)
                     : "r"((uint32_t)__cvta_generic_to_shared(&sum[c])), "r"(b)
                     : "memory");
        s += v;
      }
    }
    // no block leaves while block 0 may still read its sums
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  }
  if (blockIdx.z == 0 && c < 32 * V && col < N) db[(size_t)e * N + col] = s;
}

// kernel on clusters of a.parts blocks along z
template <typename Kernel>
cudaError_t launch_parts(Kernel* kernel, const F32Args& a, dim3 grid, int threads, int smem, cudaStream_t st) {
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = cluster.val.clusterDim.y = 1;
  cluster.val.clusterDim.z = (unsigned)a.parts;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(grid.x, grid.y, grid.z * (unsigned)a.parts);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = st;
  config.attrs = &cluster;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, a);
}

// How many blocks share a contraction of k: 1, 2, 4 or 8, as long as they all find an SM at once and a share keeps
// `least` of it.  One expert of 7000 x 640: 40 rows 186 -> 29 us in 8 parts; 8192 x 64, 10 rows 82 -> 13; 64 rows of
// 8000 x 2000 224 -> 112 in 4; 60 rows of 1200 x 300 37 -> 14.  With more blocks than SMs, clusters of 8 fill only about
// 128 of them and take longer than whole tiles: 200 rows of 4000 x 2000 169 and 111 us.
int f32_parts(long long blocks, long long k, int least) {
  int parts = 1;
  while (parts < 8 && 2 * parts * blocks <= sm_count() && k >= 2LL * parts * least) parts *= 2;
  return parts;
}

template <int MODE, int FN, int KG>
cudaError_t launch_f32_groups(const F32Args& a, dim3 grid, cudaStream_t st) {
  const int smem = f32_smem(FN, KG);
  const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(matmul_f32_kernel<MODE, FN, KG>), smem);
  if (err != cudaSuccess) return err;
  grid.y = (unsigned)((a.N + FN - 1) / FN);
  return launch_parts(matmul_f32_kernel<MODE, FN, KG>, a, grid, FN * KG, smem, st);
}
// rows: about how many row tiles of the grid have work.  64 x 128 tiles where they fill the GPU twice over; else 64 x 64
// ones, with 8 groups where there is at most one tile an SM, 4 up to four of them (2000 rows of 2048 x 1024 for 4 experts,
// 528 tiles: 224 us, 260 with 2 groups; 2400 of 1024 x 600 for 60, 670 tiles: 144 and 140), else 2.
// k: how long the contraction is, about.
template <int MODE>
cudaError_t launch_f32(F32Args a, dim3 grid, long long rows, long long k, cudaStream_t st) {
  const long long sms = sm_count();
  if (rows * ((a.N + 127) / 128) >= 6 * sms) return launch_f32_groups<MODE, 128, 1>(a, grid, st);
  const long long tiles = rows * ((a.N + 63) / 64);
  if (tiles <= sms) {
    a.parts = f32_parts(tiles, k, 256);
    return launch_f32_groups<MODE, 64, 8>(a, grid, st);
  }
  if (tiles <= 4 * sms) return launch_f32_groups<MODE, 64, 4>(a, grid, st);
  return launch_f32_groups<MODE, 64, 2>(a, grid, st);
}

cudaError_t launch_matmul_f32(const GroupedArgs& g, cudaStream_t st) {
  F32Args a{};
  a.parts = 1;
  a.offsets = g.offsets;
  a.E = g.E;
  a.rows_cap = g.rows_cap;
  a.A = static_cast<const float*>(g.x);
  a.B = static_cast<const float*>(g.W);
  a.lda = g.ldx;
  a.bias = static_cast<const float*>(g.bias);
  a.D = static_cast<float*>(g.y);
  a.ldd = g.ldy;
  a.N = g.N;
  a.K = g.K;
  a.status = g.status;
  const long long touched = g.rows_cap < g.E ? g.rows_cap : g.E;  // upper bound on the row tiles: a ragged one each
  // Few rows an expert: 4 experts of 5 rows in all, 652 x 7956, 48 -> 11 us; a 64-row tile would stay nearly empty.  These
  // blocks against the tiles at 15 rows an expert: 16 experts of 2048 x 1408 100 and 200 us, 60 of them 361 and 465,
  // 126 of 712 x 1000 229 and 261 (318 and 270 with W transposed); at 30 rows: 162 and 201, 615 and 468, 396 and 225.
  if (g.rows_cap <= kFewAvg * touched) {
    const int cols = g.transpose_w ? few_cols(MODE_NT) : few_cols(MODE_NN);
    const dim3 few_grid((unsigned)(g.rows_cap / kFewRows + touched), (unsigned)((g.N + cols - 1) / cols));
    a.parts = f32_parts((long long)few_grid.x * few_grid.y, g.K, 512);
    auto kernel = g.transpose_w ? matmul_f32_few_kernel<MODE_NT> : matmul_f32_few_kernel<MODE_NN>;
    const int smem = g.transpose_w ? few_smem(MODE_NT) : few_smem(MODE_NN);
    const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
    if (err != cudaSuccess) return err;
    return launch_parts(kernel, a, few_grid, 32 * kFewWarps, smem, st);
  }
  const dim3 grid((unsigned)(g.rows_cap / FM + touched));
  const long long rows = g.rows_cap / FM + (touched + 1) / 2;  // half of the ragged ones
  return g.transpose_w ? launch_f32<MODE_NT>(a, grid, rows, g.K, st) : launch_f32<MODE_NN>(a, grid, rows, g.K, st);
}

cudaError_t launch_wgrad_f32(const GroupedArgs& g, const float* dy, float* dW, cudaStream_t st) {
  F32Args a{};
  a.parts = 1;
  a.offsets = g.offsets;
  a.E = g.E;
  a.rows_cap = g.rows_cap;
  a.A = static_cast<const float*>(g.x);
  a.B = dy;
  a.lda = g.ldx;
  a.ldb = g.ldy;
  a.D = dW;
  a.M = g.K;
  a.N = g.N;
  a.status = g.status;
  const dim3 grid((unsigned)((g.K + FM - 1) / FM), 1, (unsigned)g.E);
  // tiles of experts with few rows end at once: with fewer rows than a step for every expert one group is enough
  const long long rows = g.rows_cap < (long long)FK * g.E ? 1LL << 31 : (long long)grid.x * grid.z;
  return launch_f32<MODE_TN>(a, grid, rows, g.rows_cap / g.E, st);
}

template <typename T>
cudaError_t launch_rows_sum(const GroupedArgs& g, const void* dy, float* db, cudaStream_t st) {
  constexpr int cols = 32 * 16 / (int)sizeof(T);
  const dim3 grid((unsigned)((g.N + cols - 1) / cols), (unsigned)g.E);
  const T* d = static_cast<const T*>(dy);
  if ((long long)grid.x * grid.y < sm_count() && g.rows_cap >= 32LL * kDbWarps)
    rows_sum_kernel<T, 8><<<dim3(grid.x, grid.y, 8), 32 * kDbWarps, 0, st>>>(g.offsets, g.E, g.rows_cap, d, g.ldy, g.N, db);
  else
    rows_sum_kernel<T, 1><<<grid, 32 * kDbWarps, 0, st>>>(g.offsets, g.E, g.rows_cap, d, g.ldy, g.N, db);
  return cudaGetLastError();
}

bool misaligned(const void* p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

}  // namespace

moe_status_t check_matmul(const moe_matmul_t* m, bool wgrad, GroupedArgs* g) {
  if (m == nullptr) return MOE_ERR_INVALID_ARG;
  if (m->E < 1 || m->E > kMaxExperts || m->rows_cap < 0 || m->K < 1 || m->N < 1) return MOE_ERR_INVALID_ARG;
  if (m->dtype != MOE_DTYPE_F32 && m->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (!wgrad && m->out_dtype != MOE_DTYPE_F32 && m->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  const long long ldx = m->ldx == 0 ? m->K : m->ldx, ldy = m->ldy == 0 ? m->N : m->ldy;
  if (ldx < m->K || ldy < m->N) return MOE_ERR_INVALID_ARG;
  const bool bf16 = m->dtype == MOE_DTYPE_BF16;
  if (!wgrad && !bf16 && m->out_dtype != MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  const int step = bf16 ? 8 : 4;
  if (m->K % step != 0 || m->N % step != 0 || ldx % step != 0 || ldy % step != 0) return MOE_ERR_UNSUPPORTED;
  if (m->rows_cap >= (1LL << 31) - 1024) return MOE_ERR_UNSUPPORTED;  // row numbers past the last tile stay 32-bit
  if (m->K > 1 << 30) return MOE_ERR_UNSUPPORTED;                     // as do steps past the last input
  // tile counters and grid sizes are 32-bit; a row pitch must fit a TMA stride (below 2^40 bytes)
  const long long mt = wgrad ? ((long long)m->K + 63) / 64 * m->E : m->rows_cap / 64 + m->E;
  const long long nt = ((long long)m->N + 63) / 64;
  if (mt >= (1LL << 31) / nt || nt > 65535 || ldx >= (1LL << 36) || ldy >= (1LL << 36)) return MOE_ERR_UNSUPPORTED;
  g->E = m->E;
  g->rows_cap = m->rows_cap;
  g->K = m->K;
  g->N = m->N;
  g->ldx = ldx;
  g->ldy = ldy;
  g->transpose_w = m->transpose_w != 0;
  g->bf16_out = m->out_dtype == MOE_DTYPE_BF16;
  return MOE_OK;
}

}  // namespace moe

extern "C" {

moe_status_t moe_grouped_matmul(const moe_matmul_t* m, const int32_t* offsets, const void* x, const void* W,
                                const void* bias, void* y, int32_t* status, cudaStream_t stream) {
  moe::NvtxRange nvtx_range("moe_grouped_matmul");
  int& launches = moe::launch_count();
  launches = 0;
  moe::GroupedArgs g{};
  const moe_status_t st = moe::check_matmul(m, false, &g);
  if (st != MOE_OK) return st;
  if (moe::misaligned(status, 4)) return MOE_ERR_INVALID_ARG;
  if (m->rows_cap == 0) return MOE_OK;
  if (offsets == nullptr || x == nullptr || W == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  if (moe::misaligned(offsets, 4) || moe::misaligned(x, 16) || moe::misaligned(W, 16) || moe::misaligned(y, 16) ||
      moe::misaligned(bias, 16))
    return MOE_ERR_INVALID_ARG;
  if (y == x || y == W || y == bias) return MOE_ERR_INVALID_ARG;  // other tiles still read what one has overwritten
  g.offsets = offsets;
  g.x = x;
  g.W = W;
  g.bias = bias;
  g.y = y;
  g.status = status;
  const cudaError_t err = m->dtype == MOE_DTYPE_BF16 ? moe::launch_grouped_matmul_sm100(g, stream)
                                                     : moe::launch_matmul_f32(g, stream);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  ++launches;
  return MOE_OK;
}

moe_status_t moe_debug_matmul_form(const moe_matmul_t* m, int32_t* form) {
  moe::GroupedArgs g{};
  const moe_status_t st = moe::check_matmul(m, false, &g);
  if (st != MOE_OK) return st;
  if (form == nullptr) return MOE_ERR_INVALID_ARG;
  if (m->dtype != MOE_DTYPE_BF16 || m->rows_cap == 0) return MOE_ERR_UNSUPPORTED;
  const moe::RowsForm f = moe::rows_form(g);
  form[0] = f.pair;
  form[1] = f.bn;
  form[2] = f.box_rows;
  form[3] = f.splits;
  return MOE_OK;
}

moe_status_t moe_grouped_wgrad(const moe_matmul_t* m, const int32_t* offsets, const void* x, const void* dy, float* dW,
                               float* db, int32_t* status, cudaStream_t stream) {
  moe::NvtxRange nvtx_range("moe_grouped_wgrad");
  int& launches = moe::launch_count();
  launches = 0;
  moe::GroupedArgs g{};
  const moe_status_t st = moe::check_matmul(m, true, &g);
  if (st != MOE_OK) return st;
  if (dW == nullptr || moe::misaligned(dW, 16) || moe::misaligned(db, 16) || moe::misaligned(status, 4))
    return MOE_ERR_INVALID_ARG;
  if (m->rows_cap == 0) {
    if (cudaMemsetAsync(dW, 0, (size_t)m->E * m->K * m->N * sizeof(float), stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (db != nullptr && cudaMemsetAsync(db, 0, (size_t)m->E * m->N * sizeof(float), stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (offsets == nullptr || x == nullptr || dy == nullptr) return MOE_ERR_INVALID_ARG;
  if (moe::misaligned(offsets, 4) || moe::misaligned(x, 16) || moe::misaligned(dy, 16)) return MOE_ERR_INVALID_ARG;
  if (dW == x || dW == dy || db == x || db == dy || db == dW) return MOE_ERR_INVALID_ARG;
  g.offsets = offsets;
  g.x = x;
  g.status = status;
  const bool bf16 = m->dtype == MOE_DTYPE_BF16;
  cudaError_t err = bf16 ? moe::launch_grouped_wgrad_sm100(g, dy, dW, stream)
                         : moe::launch_wgrad_f32(g, static_cast<const float*>(dy), dW, stream);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  ++launches;
  if (db == nullptr) return MOE_OK;
  err = bf16 ? moe::launch_rows_sum<__nv_bfloat16>(g, dy, db, stream) : moe::launch_rows_sum<float>(g, dy, db, stream);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  ++launches;
  return MOE_OK;
}

}  // extern "C"
