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

namespace moe {
namespace {

// ---------------------------------------------------------------- fp32 products ----------------
// One 64 x 128 output tile per block, 128 threads of 8 x 8 outputs, contraction in steps of 16 through a
// double-buffered pair of shared tiles [k][m], [k][n].  Bound: the FMA pipes.  A thread reads 8 + 8 words
// of shared memory per k (6 wavefronts a warp, 24 of the 64 cycles its 32 packed FMAs take on four
// sub-partitions) and issues them as fma.rn.f32x2, two products an instruction, which leaves issue slots
// for the loads.  64-row tiles rather than 128: ragged segments of a few dozen rows waste less of them.
constexpr int FM = 64, FN = 128, FK = 16, FT = 128;
constexpr int FA = FM + 4, FB = FN + 4;  // padded rows: 16-byte reads stay aligned

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
  int32_t* status;
};

__device__ __forceinline__ float4 zero4() { return make_float4(0.f, 0.f, 0.f, 0.f); }

__device__ __forceinline__ void fma2(unsigned long long& d, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}

template <int MODE>
__global__ void __launch_bounds__(FT) matmul_f32_kernel(F32Args a) {
  __shared__ int offs[kMaxExperts + 1], prefix[kMaxExperts + 1];
  __shared__ __align__(16) float As[2][FK][FA];
  __shared__ __align__(16) float Bs[2][FK][FB];
  const int tid = threadIdx.x;
  if (tid < 32)
    load_segments(a.offsets, a.E, a.rows_cap, FM, 1, offs, MODE == MODE_TN ? nullptr : prefix, a.status,
                  blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0);
  __syncthreads();
  int e, m0, mrows, K;  // mrows: valid output rows of the tile
  long long arow0;      // first A row of the tile (NN, NT), first contraction row (TN)
  if constexpr (MODE == MODE_TN) {
    e = blockIdx.z;
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

  // this thread's 16-byte pieces of the next k step: 2 of A, 4 of B (K, M, N are multiples of 4, so a piece
  // is wholly inside or wholly outside)
  float4 ra[2], rb[4];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
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
    for (int j = 0; j < 4; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_NT) {
        const int r = i >> 2, kk = (i & 3) * 4;
        rb[j] = r < ncols && k0 + kk < K ? __ldg(reinterpret_cast<const float4*>(B + (long long)r * ldb + k0 + kk))
                                         : zero4();
      } else {
        const int kk = i >> 5, c = (i & 31) * 4;
        rb[j] = k0 + kk < K && c < ncols ? __ldg(reinterpret_cast<const float4*>(B + (long long)(k0 + kk) * ldb + c))
                                         : zero4();
      }
    }
  };
  auto put = [&](int s) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
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
    for (int j = 0; j < 4; ++j) {
      const int i = tid + j * FT;
      if constexpr (MODE == MODE_NT) {
        const int r = i >> 2, kk = (i & 3) * 4;
        Bs[s][kk][r] = rb[j].x;
        Bs[s][kk + 1][r] = rb[j].y;
        Bs[s][kk + 2][r] = rb[j].z;
        Bs[s][kk + 3][r] = rb[j].w;
      } else {
        *reinterpret_cast<float4*>(&Bs[s][i >> 5][(i & 31) * 4]) = rb[j];
      }
    }
  };

  const int tx = tid & 15, ty = tid >> 4;  // columns 4 tx .. and 64 + 4 tx .., rows 8 ty ..
  unsigned long long acc[8][4] = {};
  int s = 0;
  if (K > 0) {
    fetch(0);
    put(0);
  }
  __syncthreads();
  for (int k0 = 0; k0 < K; k0 += FK) {
    const bool more = k0 + FK < K;
    if (more) fetch(k0 + FK);
#pragma unroll
    for (int kk = 0; kk < FK; ++kk) {
      const float4 a0 = *reinterpret_cast<const float4*>(&As[s][kk][ty * 8]);
      const float4 a1 = *reinterpret_cast<const float4*>(&As[s][kk][ty * 8 + 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&Bs[s][kk][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&Bs[s][kk][64 + tx * 4]);
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
    __syncthreads();
    s ^= 1;
  }

  float* D = MODE == MODE_TN ? a.D + (size_t)e * a.M * a.N + (size_t)m0 * a.N + n0 : a.D + arow0 * a.ldd + n0;
  const long long ldd = MODE == MODE_TN ? a.N : a.ldd;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = h * 64 + tx * 4;
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

// ---------------------------------------------------------------- bias gradient ----------------
// db[e,n] = sum of dy[r,n] over the expert's rows.  Bound: reading dy, or the latency of a long segment's rows.  A block
// of 32 warps takes one (expert, 32 x V columns) strip, each warp every 32nd row with 8 of them in flight; the warps'
// sums join in shared memory in a fixed order, so there are no atomics and the bits do not change from run to run.  (A
// cluster of 8 blocks of 8 warps that joined through distributed shared memory took 22 us for 64 experts of 1 to 1900
// rows of 520 columns, most of it in the cluster's barriers.)
constexpr int kDbWarps = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kDbWarps)
    rows_sum_kernel(const int32_t* __restrict__ offsets, int E, long long rows_cap, const T* __restrict__ dy,
                    long long ldy, int N, float* __restrict__ db) {
  constexpr int V = 16 / sizeof(T);
  __shared__ int offs[kMaxExperts + 1];
  __shared__ float part[kDbWarps][32 * V];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = blockIdx.y;
  if (warp == 0) load_segments(offsets, E, rows_cap, 1, 1, offs, nullptr, nullptr, false);
  __syncthreads();
  const int r1 = offs[e + 1], n = (blockIdx.x * 32 + lane) * V;
  float acc[V] = {};
  if (n < N) {
    constexpr int U = 8;  // rows in flight
    for (long long r = (long long)offs[e] + warp; r < r1; r += kDbWarps * U) {
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = r + u * kDbWarps < r1 ? __ldg(reinterpret_cast<const uint4*>(dy + (r + u * kDbWarps) * ldy + n))
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
  for (int c = threadIdx.x; c < 32 * V; c += 32 * kDbWarps) {
    const int col = (blockIdx.x * 32 + (c & 31)) * V + (c >> 5);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kDbWarps; ++w) s += part[w][c];
    if (col < N) db[(size_t)e * N + col] = s;
  }
}

cudaError_t launch_matmul_f32(const GroupedArgs& g, cudaStream_t st) {
  F32Args a{};
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
  const dim3 grid((unsigned)(g.rows_cap / FM + touched), (unsigned)((g.N + FN - 1) / FN));
  if (g.transpose_w) matmul_f32_kernel<MODE_NT><<<grid, FT, 0, st>>>(a);
  else matmul_f32_kernel<MODE_NN><<<grid, FT, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_wgrad_f32(const GroupedArgs& g, const float* dy, float* dW, cudaStream_t st) {
  F32Args a{};
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
  const dim3 grid((unsigned)((g.K + FM - 1) / FM), (unsigned)((g.N + FN - 1) / FN), (unsigned)g.E);
  matmul_f32_kernel<MODE_TN><<<grid, FT, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows_sum(const GroupedArgs& g, const void* dy, float* db, cudaStream_t st) {
  constexpr int cols = 32 * 16 / (int)sizeof(T);
  const dim3 grid((unsigned)((g.N + cols - 1) / cols), (unsigned)g.E);
  rows_sum_kernel<T><<<grid, 32 * kDbWarps, 0, st>>>(g.offsets, g.E, g.rows_cap, static_cast<const T*>(dy), g.ldy, g.N, db);
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
