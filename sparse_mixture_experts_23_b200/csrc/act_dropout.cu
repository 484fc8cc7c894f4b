// The expert's hidden step in training: activation, optional gate, dropout.
//   forward   y = m act(u) g / (1 - p)
//   backward  dg = m dy act(u) / (1 - p),  du = m dy g act'(u) / (1 - p)
// ("MoE Training: Mixture of Experts" page, Quick Start: the activation between the expert's two Linear
// layers.)  g is 1 without a gate.  The mask m is never stored: element (row r, column c) keeps its value
// when word c % 4 of Philox4x32-10 (J. Salmon et al., Parallel random numbers: as easy as 1, 2, 3, SC 2011)
// at counter (c / 4, r, offset, offset >> 32) under key (seed, seed >> 32) is at least p 2^32, and the
// backward pass computes the same words again.  A dropped element is 0 whatever its inputs hold.
//
// Bound: issue slots next to HBM (4099 x 14336 gated bf16 forward and backward: 705 MB, 107 us at the copy rate; 940
// MB and 143 us as the two calls that both read u and gate).  A vector of 16 bytes (8 bf16 or 4 fp32 columns: whole
// Philox blocks) of one row per thread and step, the next row's vectors loaded before this one's arithmetic, 24 warps an
// SM that walk down the rows.  Ten Philox rounds are 20 wide multiplies and 20 three-input xors for four elements; the
// round keys, the same for all elements, stay in registers.
// Measured 163 us replayed from a graph, 5.8 TB/s, and 175 to 179 as two calls a step (298 us with two rows a thread and
// short-lived blocks; 174 us replayed with 32 warps an SM, whose 64 registers a thread do not hold the keys).  24 and 36
// instructions an element forward and backward, ALU pipe at 49%.  The block fits widths of 2048 bf16 columns: 1408 of
// them leave 31% of its threads idle.
// All arithmetic is fp32; each output is rounded once.
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "activation.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

struct ActArgs {
  const void* dy;
  const void* u;
  const void* gate;  // or null
  void* y;           // forward: y; backward: du
  void* dgate;
  const int32_t* rows;  // device count, or null
  const unsigned long long* rng;
  long long rows_cap, ld_in, ld_y, ld_grad;
  int F;
  unsigned thr;  // an element is kept when its word is at least this: 0 keeps all
  int drop, drop_all;  // some are dropped (words are needed), all are
  float scale;
};

struct PhiloxKeys {
  uint32_t k0[10], k1[10];
  __device__ __forceinline__ PhiloxKeys(uint32_t a, uint32_t b) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      k0[i] = a + i * 0x9E3779B9u;
      k1[i] = b + i * 0xBB67AE85u;
    }
  }
};
__device__ __forceinline__ void philox4x32_10(uint32_t (&c)[4], const PhiloxKeys& key) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c[0], p1 = (uint64_t)0xCD9E8D57u * c[2];
    c[0] = (uint32_t)(p1 >> 32) ^ c[1] ^ key.k0[i];
    c[1] = (uint32_t)p1;
    c[2] = (uint32_t)(p0 >> 32) ^ c[3] ^ key.k1[i];
    c[3] = (uint32_t)p0;
  }
}

// V columns of one row as they lie in memory: with VEC one 16-byte access, otherwise element by element up to n columns
// (rows or widths that 16 bytes do not divide)
template <typename T, bool VEC>
struct Cols {
  static constexpr int V = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (VEC) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          const uint32_t lo = 2 * j < n ? reinterpret_cast<const uint16_t*>(p)[2 * j] : 0u;
          const uint32_t hi = 2 * j + 1 < n ? reinterpret_cast<const uint16_t*>(p)[2 * j + 1] : 0u;
          w[j] = lo | hi << 16;
        } else {
          w[j] = j < n ? __float_as_uint(p[j]) : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 2) return j & 1 ? __uint_as_float(w[j >> 1] & 0xffff0000u) : __uint_as_float(w[j >> 1] << 16);
    else return __uint_as_float(w[j]);
  }
};
template <typename T, int V, bool VEC>
__device__ __forceinline__ void store_cols(T* p, int n, const float (&v)[V]) {
  if constexpr (VEC) {
    uint32_t a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        a[j] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        a[j] = __float_as_uint(v[j]);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(a[0], a[1], a[2], a[3]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) p[j] = (T)v[j];
  }
}

constexpr int kActThreads = 256, kActBlocks = 3;  // a block, blocks an SM

template <typename T, int ACT, bool BWD, bool GATE, bool VEC>
__global__ void __launch_bounds__(kActThreads, kActBlocks) act_dropout_kernel(ActArgs a) {
  constexpr int V = 16 / sizeof(T);
  constexpr bool FAST = sizeof(T) == 2;
  const int col = (blockIdx.x * blockDim.x + threadIdx.x) * V;
  if (col >= a.F) return;
  const int n = a.F - col;
  long long rows = a.rows_cap;
  if (a.rows != nullptr) {
    const int r = *a.rows;
    rows = r < 0 ? 0 : (r < rows ? r : rows);
  }
  const long long step = (long long)gridDim.y * blockDim.y;
  long long r = (long long)blockIdx.y * blockDim.y + threadIdx.y;
  if (r >= rows) return;
  uint32_t off[2] = {}, seed[2] = {};
  if (a.drop) {
    const unsigned long long s = a.rng[0], o = a.rng[1];
    seed[0] = (uint32_t)s;
    seed[1] = (uint32_t)(s >> 32);
    off[0] = (uint32_t)o;
    off[1] = (uint32_t)(o >> 32);
  }
  const PhiloxKeys key(seed[0], seed[1]);
  const T* up = static_cast<const T*>(a.u) + r * a.ld_in + col;
  const T* gp = static_cast<const T*>(a.gate) + r * a.ld_in + col;
  const T* dp = static_cast<const T*>(a.dy) + r * a.ld_y + col;
  T* yp = static_cast<T*>(a.y) + r * (BWD ? a.ld_grad : a.ld_y) + col;
  T* dgp = static_cast<T*>(a.dgate) + r * a.ld_grad + col;
  const long long in_step = step * a.ld_in, y_step = step * a.ld_y, out_step = step * (BWD ? a.ld_grad : a.ld_y);
  Cols<T, VEC> u, g, d;
  u.load(up, n);
  if constexpr (GATE) g.load(gp, n);
  if constexpr (BWD) d.load(dp, n);
  if (a.drop_all) {  // 0 whatever the inputs hold
    const float zero[V] = {};
    for (; r < rows; r += step) {
      store_cols<T, V, VEC>(yp, n, zero);
      yp += out_step;
      if constexpr (BWD && GATE) {
        store_cols<T, V, VEC>(dgp, n, zero);
        dgp += out_step;
      }
    }
    return;
  }
  for (; r < rows; r += step) {
    Cols<T, VEC> un = u, gn = g, dn = d;
    if (r + step < rows) {  // another row: nothing that this thread or one before it still writes
      up += in_step;
      un.load(up, n);
      if constexpr (GATE) {
        gp += in_step;
        gn.load(gp, n);
      }
      if constexpr (BWD) {
        dp += y_step;
        dn.load(dp, n);
      }
    }
    float y[V], dg[V];
#pragma unroll
    for (int b = 0; b < V / 4; ++b) {
      uint32_t c[4] = {(uint32_t)(col / 4 + b), (uint32_t)r, off[0], off[1]};
      if (a.drop) philox4x32_10(c, key);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * b + i;
        const bool keep = c[i] >= a.thr;
        if constexpr (BWD) {
          float da;
          const float act = activate_grad<ACT, FAST>(u.get(j), da);
          const float dm = a.scale * d.get(j);
          y[j] = keep ? (GATE ? dm * g.get(j) * da : dm * da) : 0.f;
          if constexpr (GATE) dg[j] = keep ? dm * act : 0.f;
        } else {
          const float v = a.scale * activate<ACT, FAST>(u.get(j));
          y[j] = keep ? (GATE ? v * g.get(j) : v) : 0.f;
        }
      }
    }
    store_cols<T, V, VEC>(yp, n, y);
    yp += out_step;
    if constexpr (BWD && GATE) {
      store_cols<T, V, VEC>(dgp, n, dg);
      dgp += out_step;
    }
    u = un;
    g = gn;
    d = dn;
  }
}

template <typename T, int ACT, bool BWD, bool GATE, bool VEC>
cudaError_t launch_act(const ActArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const int vecs = (a.F + V - 1) / V;
  int bx = 32;  // threads across a row: a power of two up to the block, so narrow rows share one
  while (bx < kActThreads && bx < vecs) bx *= 2;
  const int by = kActThreads / bx;
  const long long gx = (vecs + bx - 1) / bx;
  // as many blocks as run at once: each thread then takes several rows, whose loads overlap
  long long gy = (long long)kActBlocks * sm_count() / gx;
  if (gy < 1) gy = 1;
  const long long most = (a.rows_cap + by - 1) / by;
  if (gy > most) gy = most;
  act_dropout_kernel<T, ACT, BWD, GATE, VEC><<<dim3((unsigned)gx, (unsigned)gy), dim3(bx, by), 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int ACT, bool BWD>
cudaError_t launch_by_form(const ActArgs& a, bool vec, cudaStream_t st) {
  if (a.gate != nullptr) return vec ? launch_act<T, ACT, BWD, true, true>(a, st) : launch_act<T, ACT, BWD, true, false>(a, st);
  return vec ? launch_act<T, ACT, BWD, false, true>(a, st) : launch_act<T, ACT, BWD, false, false>(a, st);
}

template <bool BWD>
cudaError_t launch_by_type(const ActArgs& a, int dtype, int act, bool vec, cudaStream_t st) {
  if (dtype == MOE_DTYPE_BF16) {
    if (act == MOE_ACT_GELU) return launch_by_form<__nv_bfloat16, MOE_ACT_GELU, BWD>(a, vec, st);
    if (act == MOE_ACT_SILU) return launch_by_form<__nv_bfloat16, MOE_ACT_SILU, BWD>(a, vec, st);
    return launch_by_form<__nv_bfloat16, MOE_ACT_NONE, BWD>(a, vec, st);
  }
  if (act == MOE_ACT_GELU) return launch_by_form<float, MOE_ACT_GELU, BWD>(a, vec, st);
  if (act == MOE_ACT_SILU) return launch_by_form<float, MOE_ACT_SILU, BWD>(a, vec, st);
  return launch_by_form<float, MOE_ACT_NONE, BWD>(a, vec, st);
}

moe_status_t run_act(const moe_act_t* m, const void* dy, const void* u, const void* gate, void* y, void* dgate, bool bwd,
                     cudaStream_t st) {
  int& launches = launch_count();
  launches = 0;
  if (m == nullptr || m->rows_cap < 0 || m->F < 1) return MOE_ERR_INVALID_ARG;
  if (m->dtype != MOE_DTYPE_F32 && m->dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (m->activation != MOE_ACT_GELU && m->activation != MOE_ACT_SILU && m->activation != MOE_ACT_NONE)
    return MOE_ERR_INVALID_ARG;
  if (!(m->p >= 0.0 && m->p <= 1.0) || (m->p > 0.0 && m->rng == nullptr)) return MOE_ERR_INVALID_ARG;
  ActArgs a{};
  a.ld_in = m->ld_in == 0 ? m->F : m->ld_in;
  a.ld_y = m->ld_y == 0 ? m->F : m->ld_y;
  a.ld_grad = m->ld_grad == 0 ? m->F : m->ld_grad;
  if (a.ld_in < m->F || a.ld_y < m->F || a.ld_grad < m->F) return MOE_ERR_INVALID_ARG;
  const uintptr_t es = m->dtype == MOE_DTYPE_BF16 ? 2 : 4;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(gate) |
                         reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(dgate);
  if (bits % es != 0 || reinterpret_cast<uintptr_t>(m->rng) % 8 != 0 || reinterpret_cast<uintptr_t>(m->rows) % 4 != 0)
    return MOE_ERR_INVALID_ARG;
  if (m->rows_cap >= (1LL << 32) || m->F > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (m->rows_cap == 0) return MOE_OK;
  if (u == nullptr || y == nullptr || (bwd && (dy == nullptr || (gate != nullptr) != (dgate != nullptr))))
    return MOE_ERR_INVALID_ARG;
  if (m->rows_cap > 1) {
    // a result in place of an input lies as the input does (else rows that are still to be read would be overwritten)
    for (const void* out : {static_cast<const void*>(y), static_cast<const void*>(dgate)}) {
      const long long ld = bwd ? a.ld_grad : a.ld_y;
      if (out != nullptr && (((out == u || out == gate) && ld != a.ld_in) || (out == dy && ld != a.ld_y))) return MOE_ERR_INVALID_ARG;
    }
  }
  if (dgate != nullptr && dgate == y) return MOE_ERR_INVALID_ARG;
  a.dy = dy;
  a.u = u;
  a.gate = gate;
  a.y = y;
  a.dgate = dgate;
  a.rows = m->rows;
  a.rng = reinterpret_cast<const unsigned long long*>(m->rng);
  a.rows_cap = m->rows_cap;
  a.F = m->F;
  const double t = floor(m->p * 4294967296.0);
  a.drop_all = t >= 4294967296.0;
  a.thr = a.drop_all ? 0u : (unsigned)t;
  a.drop = !a.drop_all && a.thr > 0u;
  a.scale = a.drop_all ? 0.f : (float)(1.0 / (1.0 - m->p));
  const int v = 16 / (int)es;
  const bool vec = bits % 16 == 0 && m->F % v == 0 && a.ld_in % v == 0 && a.ld_y % v == 0 && a.ld_grad % v == 0;
  const cudaError_t err = bwd ? launch_by_type<true>(a, m->dtype, m->activation, vec, st)
                              : launch_by_type<false>(a, m->dtype, m->activation, vec, st);
  if (err != cudaSuccess) return MOE_ERR_CUDA;
  ++launches;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status_t moe_act_dropout(const moe_act_t* m, const void* u, const void* gate, void* y, cudaStream_t stream) {
  moe::NvtxRange nvtx_range("moe_act_dropout");
  return moe::run_act(m, nullptr, u, gate, y, nullptr, false, stream);
}

moe_status_t moe_act_dropout_backward(const moe_act_t* m, const void* dy, const void* u, const void* gate, void* du,
                                      void* dgate, cudaStream_t stream) {
  moe::NvtxRange nvtx_range("moe_act_dropout_backward");
  return moe::run_act(m, dy, u, gate, du, dgate, true, stream);
}

}  // extern "C"
