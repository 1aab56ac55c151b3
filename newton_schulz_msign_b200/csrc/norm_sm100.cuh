// norm_sm100.cuh - root-mean-square norm of rows, with the residual's
// addition in front, int8 output behind, and its gradients.
//
//   z = x + r  (rounded to the io type where r is given: the stored sum)
//   y_j = z_j w_j / sqrt(mean_j z_j^2 + eps)
//   int8: scale = max_j |y_j| / 127, q_j = rint(y_j / scale)
//   dz_j = rstd (dy_j w_j - n_j mean_j(dy_j w_j n_j)) + ds_j,  n = z rstd
//   dw_j = sum over rows of dy_j n_j
//
// All of it is HBM-bound: each row is read once and written once.  A row
// stays in the registers of the threads that own it (kNormVpt 16-byte pieces
// each at most), so the statistic, the output and the int8 maximum come from
// one pass over memory.  Sums and statistics are fp32; y is formed in fp32
// and rounded once (int8: the fp32 y is quantised, never a rounded one).
//
// Measured (B200, copy rate 6.54 TB/s): 8192 x 4096 bf16 with a residual 41.7
// us (268 MB, 41.0 at the copy rate), to int8 39.8 (235 MB, 35.9; by now
// bound by instructions), one row 2.3, gradients 49 (268 MB).
//
// Rows off 16-byte boundaries move by 16 bytes about them where all matrices
// of a call lie alike, else by elements; rows longer than 1024 threads hold
// take the *_loop kernels, which read the row again for each pass (it is still
// in L1 or L2 then).  norm_plan.h chooses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "gemm_sm100.cuh"
#include "norm_plan.h"
#include "ptx_sm100.cuh"

namespace msb {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// `bytes` (a multiple of 16, both addresses too) from global to this CTA's
// shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <typename T>
struct Elem {};
template <>
struct Elem<float> {
  static constexpr int vec = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int vec = 8;
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Elem<__half> {
  static constexpr int vec = 8;
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Two fp32 values at a time: the gradients' kernel is bound by instructions
// as soon as its loads are asynchronous.
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pair2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 unpair2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The same value, as something that the compiler knows nothing of: it then
// unpacks a piece again instead of holding the unpacked values in registers.
__device__ __forceinline__ void opaque(uint4& u) {
  asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
}

template <typename T>
__device__ __forceinline__ void unpack2(const uint4& u, f32x2 (&v)[Elem<T>::vec / 2]) {
  float f[Elem<T>::vec];
  Elem<T>::unpack(u, f);
#pragma unroll
  for (int j = 0; j < Elem<T>::vec / 2; ++j) v[j] = pair2(f[2 * j], f[2 * j + 1]);
}

struct NormArgs {
  const void *x, *r, *w;  // r, w: may be null
  void *y, *s;            // y: io type, or int8 (scale set); s: the sum, may be null
  float* scale;           // int8 output: one a row
  long long xs, rs, ys, ss;  // row strides in elements
  long long rows;
  int cols;
  int w_f32;  // the weight is fp32 (else the io type)
  float eps;
};

struct NormBwdArgs {
  const void *dy, *z, *w, *ds;  // w, ds: may be null
  void* dz;
  float* part;  // [gridDim.x][cols] partial sums of dw, or null
  float* rstd;  // loop form: [rows]
  long long dys, zs, dss, dzs;
  long long rows;
  int cols;
  int w_f32;
  float eps;
  int* err;  // device error word, and the limit of a wait
  unsigned long long timeout_ns;
};

// Sums of a and b over the threads of a row: one warp (blockDim.x = 32) or
// the whole block.  `red` holds 2 x 32 float2; `par` alternates between rows
// so that one barrier a row is enough (a warp writes a buffer again only
// after the barrier of the row in between).
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* red, int par) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  const int nw = blockDim.x >> 5;
  if (nw > 1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    red += par * 32;
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    const float2 f = lane < nw ? red[lane] : make_float2(0.0f, 0.0f);
    a = f.x, b = f.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
  }
  return make_float2(a, b);
}

// Whether fp32 holds the mean of squares with all its digits.  Where it does
// not (magnitudes past 1e15, or eps 0 and magnitudes below 1e-15), the row is
// summed again times norm_rescale().
__device__ __forceinline__ bool mean_holds(float ms) { return ms > 1e-30f && ms < 1e30f; }
__device__ __forceinline__ float norm_rescale(float ms) {
  return ms < 1.0f ? 7.922816251426434e28f : 1.262177448353619e-29f;  // 2^96, 2^-96
}

// max(|v|, m) that keeps a NaN of either.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// Largest magnitude of a row (not negative, or NaN: as whole numbers the bits
// order like the values, with infinity and then NaN on top).
__device__ __forceinline__ float row_max(float v, uint32_t* red) {
  uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu);
  const int nw = blockDim.x >> 5;
  if (nw > 1) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xFFFFFFFFu, lane < nw ? red[lane] : 0u);
  }
  return __uint_as_float(m);
}

// The scale of an int8 row and the factors that take y to q: q = rint((y
// pre) f).  pre is 1 but for rows so small that 127 / max overflows.  A row
// of zeros has scale 0 and q = 0; one that holds an infinity or a NaN has
// that as its scale and q = 0 (f = 0 says so), so that what it stands for is
// NaN throughout.
__device__ __forceinline__ float q8_factor(float amax, float* scale, float* pre) {
  *scale = __fdiv_rn(amax, 127.0f);
  *pre = amax < 1e-30f ? 1.8446744073709552e19f : 1.0f;
  if (!(amax > 0.0f) || __float_as_uint(amax) >= 0x7F800000u) return 0.0f;
  return __fdiv_rn(127.0f, amax * *pre);
}

// Four values to int8, packed.  Adding 1.5 2^23 rounds the sum to a whole
// number (ties to even) and leaves it in the low mantissa bits: one fused
// multiply-add a value instead of a conversion, a clamp and a mask (|y f| is
// at most 127 and two roundings, which cannot reach 127.5).
__device__ __forceinline__ uint32_t q8_pack(float a, float b, float c, float d, float f) {
  constexpr float kRound = 12582912.0f;
  const uint32_t x = __float_as_uint(fmaf(a, f, kRound)), y = __float_as_uint(fmaf(b, f, kRound));
  const uint32_t z = __float_as_uint(fmaf(c, f, kRound)), w = __float_as_uint(fmaf(d, f, kRound));
  return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
}

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int c, float (&v)[Elem<T>::vec]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < Elem<T>::vec; ++i) v[i] = 1.0f;
  } else if (sizeof(T) == 4 || !w_f32) {
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const T*>(w) + c), v);
  } else {
#pragma unroll
    for (int i = 0; i < Elem<T>::vec / 4; ++i) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + 4 * i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  }
}

// Rows off 16-byte boundaries, by 16 bytes all the same: where every matrix of
// the call has the same phase (the index of a row's first element past a
// boundary, modulo the elements of 16 bytes), piece k of a row with phase ph
// starts at column k vec - ph, and only its first and its last piece are not
// whole (8192 rows with a residual, bf16: 1002 columns 17 us, by pairs 23;
// 2001 33, one by one 61; 8191 137 and 224).  The 16-bit form of four pieces a
// thread still spills 8 to 16 bytes at its 64 registers.
template <typename T>
__device__ __forceinline__ int row_phase(const void* p, long long at) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) / sizeof(T) + static_cast<unsigned long long>(at)) %
                          Elem<T>::vec);
}

template <typename T>
__device__ __forceinline__ bool whole(int c, int cols) {
  return c >= 0 && c + Elem<T>::vec <= cols;
}

// The piece at column c of a row, zeros outside the row.
template <typename T, bool SHIFT>
__device__ __forceinline__ uint4 load_piece(const T* row, int c, int cols) {
  if (SHIFT ? whole<T>(c, cols) : c < cols) return *reinterpret_cast<const uint4*>(row + c);
  uint4 u = make_uint4(0, 0, 0, 0);
  if (SHIFT && c < cols) {
    float v[Elem<T>::vec];
#pragma unroll
    for (int j = 0; j < Elem<T>::vec; ++j)
      v[j] = c + j >= 0 && c + j < cols ? Elem<T>::get(row[c + j]) : 0.0f;
    u = Elem<T>::pack(v);
  }
  return u;
}

template <typename T, bool SHIFT>
__device__ __forceinline__ void store_piece(T* row, int c, int cols, const uint4& u) {
  if (SHIFT ? whole<T>(c, cols) : c < cols) {
    *reinterpret_cast<uint4*>(row + c) = u;
  } else if (SHIFT && c < cols) {
    float v[Elem<T>::vec];
    Elem<T>::unpack(u, v);
#pragma unroll
    for (int j = 0; j < Elem<T>::vec; ++j)
      if (c + j >= 0 && c + j < cols) row[c + j] = Elem<T>::put(v[j]);
  }
}

// Elements of a piece outside the row become zeros (what was read there
// belongs to the row's neighbours).
template <typename T>
__device__ __forceinline__ void keep_row(uint4& u, int c, int cols) {
  float v[Elem<T>::vec];
  Elem<T>::unpack(u, v);
#pragma unroll
  for (int j = 0; j < Elem<T>::vec; ++j)
    if (c + j < 0 || c + j >= cols) v[j] = 0.0f;
  u = Elem<T>::pack(v);
}

template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int w_f32, int c) {
  if (w == nullptr) return 1.0f;
  return w_f32 ? static_cast<const float*>(w)[c] : Elem<T>::get(static_cast<const T*>(w)[c]);
}

// (One by one off the boundaries: cut out of the two 16-byte pieces about them
// 8192 x 2001 takes as long, 8192 x 301 12 us instead of 10.6.)
template <typename T, bool SHIFT>
__device__ __forceinline__ void load_weights(const void* w, int w_f32, int c, int cols, float (&v)[Elem<T>::vec]) {
  if (!SHIFT) {
    load_weight<T>(w, w_f32, c, v);
  } else {
#pragma unroll
    for (int j = 0; j < Elem<T>::vec; ++j) v[j] = c + j >= 0 && c + j < cols ? weight_at<T>(w, w_f32, c + j) : 0.0f;
  }
}

// One row per blockDim.x threads (32: a warp a row, blockDim.y rows a block;
// more: one row a block).  Piece i of thread t starts at column
// (i blockDim.x + t) vec.
template <typename T, int VPT, bool Q8, bool SHIFT>
__global__ void __launch_bounds__(kNormMaxThreads) rms_norm_kernel(const NormArgs a) {
  constexpr int V = Elem<T>::vec;
  __shared__ float2 red[64];
  __shared__ uint32_t redm[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;  // (blocks of several rows have no barrier)
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const int ph = SHIFT ? row_phase<T>(a.x, row * a.xs) : 0;
  uint4 raw[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V - ph;
    raw[i] = load_piece<T, SHIFT>(x, c, a.cols);
  }
  if (a.r != nullptr) {
    const T* r = static_cast<const T*>(a.r) + row * a.rs;
    T* s = static_cast<T*>(a.s) + row * a.ss;
    uint4 rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      rr[i] = load_piece<T, SHIFT>(r, c, a.cols);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      float xv[V], rv[V];
      Elem<T>::unpack(raw[i], xv);
      Elem<T>::unpack(rr[i], rv);
#pragma unroll
      for (int j = 0; j < V; ++j) xv[j] += rv[j];
      raw[i] = Elem<T>::pack(xv);  // the stored sum: what the norm and its gradient see
      if (a.s != nullptr) store_piece<T, SHIFT>(s, c, a.cols, raw[i]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float v[V];
    Elem<T>::unpack(raw[i], v);
#pragma unroll
    for (int j = 0; j < V; ++j) ss = fmaf(v[j], v[j], ss);
  }
  ss = row_sum2(ss, 0.0f, red, 0).x;
  float rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps);
  if (!mean_holds(ss / static_cast<float>(a.cols) + a.eps)) {  // (the same for the whole row)
    const float p = norm_rescale(ss / static_cast<float>(a.cols) + a.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float v[V];
      Elem<T>::unpack(raw[i], v);
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[j] * p, v[j] * p, ss);
    }
    ss = row_sum2(ss, 0.0f, red, 1).x;
    rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps * p * p) * p;
  }
  if (!Q8) {
    T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      if (c < a.cols) {
        float v[V], w[V];
        Elem<T>::unpack(raw[i], v);
        load_weights<T, SHIFT>(a.w, a.w_f32, c, a.cols, w);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = v[j] * rstd * w[j];
        store_piece<T, SHIFT>(y, c, a.cols, Elem<T>::pack(v));
      }
    }
  } else {
    int8_t* y = static_cast<int8_t*>(a.y) + row * a.ys;
    float v[VPT][V];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      Elem<T>::unpack(raw[i], v[i]);
      if (c < a.cols) {
        float w[V];
        load_weights<T, SHIFT>(a.w, a.w_f32, c, a.cols, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] = v[i][j] * rstd * w[j];
          m = max_abs(m, v[i][j]);
        }
      }
    }
    float scale, pre;
    const float f = q8_factor(row_max(m, redm), &scale, &pre);
    if (threadIdx.x == 0) a.scale[row] = scale;
    if (pre != 1.0f) {  // (the same for the whole row)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] *= pre;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      if (c < a.cols) {
        uint32_t p[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
          p[j] = f == 0.0f ? 0u : q8_pack(v[i][4 * j], v[i][4 * j + 1], v[i][4 * j + 2], v[i][4 * j + 3], f);
        if (SHIFT && !whole<T>(c, a.cols)) {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c + j >= 0 && c + j < a.cols) y[c + j] = static_cast<int8_t>(p[j / 4] >> (8 * (j % 4)) & 0xFFu);
        } else if (V == 8)
          *reinterpret_cast<uint2*>(y + c) = make_uint2(p[0], p[V / 4 - 1]);
        else
          *reinterpret_cast<uint32_t*>(y + c) = p[0];
      }
    }
  }
}

// P consecutive elements (1 or 2), as floats.  Two move as one access, which
// their address has to allow.
template <typename T, int P>
__device__ __forceinline__ void load_p(const T* p, float (&v)[P]) {
  if (P == 1) {
    v[0] = Elem<T>::get(p[0]);
  } else if (sizeof(T) == 4) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x, v[P - 1] = f.y;
  } else {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    const uint16_t h[2] = {static_cast<uint16_t>(u), static_cast<uint16_t>(u >> 16)};
    v[0] = Elem<T>::get(*reinterpret_cast<const T*>(&h[0]));
    v[P - 1] = Elem<T>::get(*reinterpret_cast<const T*>(&h[1]));
  }
}

template <typename T, int P>
__device__ __forceinline__ void store_p(T* p, const float (&v)[P]) {
  if (P == 1) {
    p[0] = Elem<T>::put(v[0]);
  } else if (sizeof(T) == 4) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[P - 1]);
  } else {
    const T h[2] = {Elem<T>::put(v[0]), Elem<T>::put(v[P - 1])};
    uint16_t u[2];
    memcpy(u, h, 4);
    *reinterpret_cast<uint32_t*>(p) = u[0] | static_cast<uint32_t>(u[1]) << 16;
  }
}

template <typename T, int P>
__device__ __forceinline__ void weight_p(const void* w, int w_f32, int c, float (&v)[P]) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = 1.0f;
  } else if (w_f32) {
    load_p<float, P>(static_cast<const float*>(w) + c, v);
  } else {
    load_p<T, P>(static_cast<const T*>(w) + c, v);
  }
}

// Rows without 16-byte alignment whose phases differ or that are short, up to
// 8 accesses a thread: like the kernel above with P elements for a piece (piece i of thread t starts at column (i
// blockDim.x + t) P, so that a warp's accesses lie side by side).
template <typename T, int P, bool Q8>
__global__ void __launch_bounds__(kNormMaxThreads) rms_norm_elem_kernel(const NormArgs a) {
  constexpr int E = kNormElems;
  __shared__ float2 red[64];
  __shared__ uint32_t redm[32];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;  // (blocks of several rows have no barrier)
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  float v[E][P];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * P;
#pragma unroll
    for (int j = 0; j < P; ++j) v[i][j] = 0.0f;
    if (c < a.cols) load_p<T, P>(x + c, v[i]);
  }
  if (a.r != nullptr) {
    const T* r = static_cast<const T*>(a.r) + row * a.rs;
    float rv[E][P];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * P;
#pragma unroll
      for (int j = 0; j < P; ++j) rv[i][j] = 0.0f;
      if (c < a.cols) load_p<T, P>(r + c, rv[i]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * P;
#pragma unroll
      for (int j = 0; j < P; ++j) v[i][j] = Elem<T>::get(Elem<T>::put(v[i][j] + rv[i][j]));
      if (c < a.cols && a.s != nullptr) store_p<T, P>(static_cast<T*>(a.s) + row * a.ss + c, v[i]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i)
#pragma unroll
    for (int j = 0; j < P; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  ss = row_sum2(ss, 0.0f, red, 0).x;
  float rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps);
  if (!mean_holds(ss / static_cast<float>(a.cols) + a.eps)) {
    const float p = norm_rescale(ss / static_cast<float>(a.cols) + a.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) ss = fmaf(v[i][j] * p, v[i][j] * p, ss);
    ss = row_sum2(ss, 0.0f, red, 1).x;
    rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps * p * p) * p;
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * P;
    if (c < a.cols) {
      float w[P];
      weight_p<T, P>(a.w, a.w_f32, c, w);
#pragma unroll
      for (int j = 0; j < P; ++j) v[i][j] = v[i][j] * rstd * w[j];
      if (Q8) {
#pragma unroll
        for (int j = 0; j < P; ++j) m = max_abs(m, v[i][j]);
      } else {
        store_p<T, P>(static_cast<T*>(a.y) + row * a.ys + c, v[i]);
      }
    }
  }
  if (Q8) {
    float scale, pre;
    const float f = q8_factor(row_max(m, redm), &scale, &pre);
    if (threadIdx.x == 0) a.scale[row] = scale;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * P;
      if (c < a.cols) {
        const uint32_t q = f == 0.0f ? 0u : q8_pack(v[i][0] * pre, v[i][P - 1] * pre, 0.0f, 0.0f, f);
        int8_t* y = static_cast<int8_t*>(a.y) + row * a.ys + c;
        if (P == 1)
          *y = static_cast<int8_t>(q & 0xFFu);
        else
          *reinterpret_cast<uint16_t*>(y) = static_cast<uint16_t>(q);
      }
    }
  }
}

// The loop forms' sums: a thread adds at most this many terms one after another,
// then adds that sum to its total, so that the error does not grow with rows of
// millions of columns (one sum all along was off by 1.8e-3 at 2^30 columns).
constexpr int kLoopRun = 1024;

// f(c) for this thread's columns, 256 threads a row; behind every kLoopRun of
// them join().  (The one run of an ordinary row stands apart: inside the outer
// loop the gradients of 777 x 9001 bf16, phases apart, take 61 us instead of 53.)
template <typename F, typename J>
__device__ __forceinline__ void loop_columns(int cols, F f, J join) {
  if (cols <= 256 * kLoopRun) {
#pragma unroll 4
    for (int c = threadIdx.x; c < cols; c += 256) f(c);
    join();
    return;
  }
  for (int c0 = 0; c0 < cols; c0 += 256 * kLoopRun) {
    const int c1 = min(cols, c0 + 256 * kLoopRun);
    for (int c = c0 + threadIdx.x; c < c1; c += 256) f(c);
    join();
  }
}

// Rows longer than that: one row a block of 256 threads.  A thread reads
// back only what it wrote itself, so the sum may replace x or r in place.
template <typename T, bool Q8>
__global__ void __launch_bounds__(256) rms_norm_loop_kernel(const NormArgs a) {
  __shared__ float2 red[64];
  __shared__ uint32_t redm[32];
  pdl_wait();
  pdl_trigger();
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const T* r = a.r == nullptr ? nullptr : static_cast<const T*>(a.r) + row * a.rs;
  T* s = a.s == nullptr ? nullptr : static_cast<T*>(a.s) + row * a.ss;
  // the row's element c as the norm sees it
  const auto z_at = [&](int c) {
    float z = Elem<T>::get(x[c]);
    if (r != nullptr) z = Elem<T>::get(Elem<T>::put(z + Elem<T>::get(r[c])));
    return z;
  };
  float ss = 0.0f, run = 0.0f;
  const auto join = [&] { ss += run, run = 0.0f; };
  loop_columns(a.cols, [&](int c) {
    const float z = z_at(c);
    if (s != nullptr) s[c] = Elem<T>::put(z);
    run = fmaf(z, z, run);
  }, join);
  if (s != nullptr) x = s, r = nullptr;
  ss = row_sum2(ss, 0.0f, red, 0).x;
  float rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps);
  if (!mean_holds(ss / static_cast<float>(a.cols) + a.eps)) {
    const float p = norm_rescale(ss / static_cast<float>(a.cols) + a.eps);
    ss = 0.0f;
    loop_columns(a.cols, [&](int c) { run = fmaf(z_at(c) * p, z_at(c) * p, run); }, join);
    ss = row_sum2(ss, 0.0f, red, 1).x;
    rstd = __frsqrt_rn(ss / static_cast<float>(a.cols) + a.eps * p * p) * p;
  }
  if (!Q8) {
    T* y = static_cast<T*>(a.y) + row * a.ys;
    for (int c = threadIdx.x; c < a.cols; c += 256)
      y[c] = Elem<T>::put(z_at(c) * rstd * weight_at<T>(a.w, a.w_f32, c));
  } else {
    int8_t* y = static_cast<int8_t*>(a.y) + row * a.ys;
    float m = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += 256)
      m = max_abs(m, z_at(c) * rstd * weight_at<T>(a.w, a.w_f32, c));
    float scale, pre;
    const float f = q8_factor(row_max(m, redm), &scale, &pre);
    if (threadIdx.x == 0) a.scale[row] = scale;
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float v = z_at(c) * rstd * weight_at<T>(a.w, a.w_f32, c) * pre;
      y[c] = f == 0.0f ? int8_t(0) : static_cast<int8_t>(q8_pack(v, 0.0f, 0.0f, 0.0f, f) & 0xFFu);
    }
  }
}

// ---------------------------------------------------------------- gradients

// Sums of (z p)^2 and dy w z p over a row, by one warp.  A call of its own:
// inlined, the rare case's registers made the common one spill (8192 x 4096
// with ds 62 us, 56 so; without ds 56 and 49).
template <typename T>
__device__ __noinline__ float2 warp_sums(const T* z, const T* dy, const void* w, int w_f32, int cols, float p) {
  float ss = 0.0f, dot = 0.0f;
  for (int c = threadIdx.x & 31; c < cols; c += 32) {
    const float zp = Elem<T>::get(z[c]) * p;
    ss = fmaf(zp, zp, ss);
    dot = fmaf(Elem<T>::get(dy[c]) * weight_at<T>(w, w_f32, c), zp, dot);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  }
  return make_float2(ss, dot);
}

// Persistent: a block takes blockDim.y rows at a time, blockDim.x threads
// each (whole warps; piece i of thread t starts at column (i blockDim.x + t)
// vec), block b the row groups b, b + gridDim.x, ...  The rows' dy, z and ds
// come through a ring of `stages` slots of shared memory filled by bulk
// copies, so that the loads in flight depend neither on registers nor on the
// barrier that joins a row's sums.  A slot is filled again after the barrier
// of the group behind it: every thread has passed its last read of the slot
// by then.  Each thread keeps its columns' share of dw in registers to the
// end: one partial row of dw a block, joined in a fixed order by
// dw_reduce_kernel (no atomics: the result does not depend on the order of
// blocks).
//
// NORM_FULL: every thread has a column and a row in every turn.  NORM_SHIFT:
// rows off 16-byte boundaries, all matrices in the same phase (row_phase); a
// thread's rows have one phase, so that its columns stay the same (16384 x 1001
// bf16 with ds 44 us; by elements, dy and z read again for dw, 97).  Its 16-bit
// form of two pieces a thread spills 48 bytes at 80 registers; the others, and
// all of the two kinds above, none.
//
// What bounds it: 8192 x 4096 bf16 with ds 49 us, 41 of them HBM's; 3 are
// dw_reduce_kernel, 1 the last turn of rows, the rest the first copies'
// latency.  Before, it was instructions (31 a warp and 32 values, 56 us;
// 27 now): threads that may be idle as branches, unpacked values held over
// the barrier and spilled.  A running pointer to dz's row costs registers
// (53), four blocks an SM spill (59), a warp a row leaves the instruction
// caches (68).
enum { NORM_ROWS, NORM_FULL, NORM_SHIFT };

template <typename T, int VPT, int KIND>
__global__ void __launch_bounds__(norm_bwd_threads(VPT), VPT <= 2 ? 3 : 1)
    rms_norm_bwd_kernel(const NormBwdArgs a, int stages) {
  constexpr int V = Elem<T>::vec, H = V / 2;
  constexpr bool FULL = KIND == NORM_FULL, SHIFT = KIND == NORM_SHIFT;
  // The second pass unpacks z and dy again, from registers, or where a thread
  // holds four pieces from shared memory (8192 x 8192 bf16 92 us from
  // registers, 89 so; at two pieces no difference).
  constexpr bool kReread = VPT >= 4;
  extern __shared__ __align__(128) uint8_t ring[];  // [stages][z, dy, ds][blockDim.y][cols]
  __shared__ __align__(16) float2 red[2][16];
  __shared__ uint64_t full[kNormRing];
  const int lane = threadIdx.x & 31;
  const int ny = blockDim.y, nwarp = blockDim.x >> 5;       // rows of a group, warps of a row
  const int warp = threadIdx.y * nwarp + (threadIdx.x >> 5);
  const int red0 = threadIdx.y * ((nwarp + 1) & ~1);        // where this row's warps leave their sums, in pairs
  const uint32_t row_bytes = norm_row_bytes<uint32_t>(a.cols, sizeof(T), SHIFT);
  const int arrays = a.ds != nullptr ? 3 : 2;
  const uint32_t slot = static_cast<uint32_t>(arrays * ny) * row_bytes;
  const long long step = static_cast<long long>(gridDim.x) * ny;
  // the group of rows from `row0` on into slot st, by the first warp: a copy a lane
  const auto fill = [&](long long row0, int st) {
    const int n = static_cast<int>(min(static_cast<long long>(ny), a.rows - row0));
    if constexpr (SHIFT) {  // (24 copies at most)
      const int arr = lane / n, y = lane - arr * n;
      const bool mine = lane < arrays * n;
      const long long row = row0 + y;
      const T* src = static_cast<const T*>(arr == 0 ? a.z : arr == 1 ? a.dy : a.ds) +
                     row * (arr == 0 ? a.zs : arr == 1 ? a.dys : a.dss);
      uint8_t* dst = ring + st * slot + (arr * ny + y) * row_bytes;
      uint32_t off = 0, bytes = 0;
      if (mine) {
        // whole 16-byte units, the neighbours' elements in the first and the
        // last one too; but nothing before the matrix or behind it: what that
        // cuts off comes element by element
        const int ph = row_phase<T>(src, 0);
        const int past = (ph + a.cols) % V;
        int c0 = -ph, c1 = past == 0 ? a.cols : a.cols - past + V;
        T* d = reinterpret_cast<T*>(dst) + ph;
        if (row == 0 && ph != 0) {
          c0 += V;
          for (int c = 0; c < c0; ++c) d[c] = src[c];
          fence_proxy_async_smem();  // (a later row's copy writes there)
        }
        if (row == a.rows - 1 && past != 0) {
          c1 -= V;
          for (int c = c1; c < a.cols; ++c) d[c] = src[c];
        }
        src += c0;
        off = static_cast<uint32_t>(c0 + ph) * sizeof(T);
        bytes = static_cast<uint32_t>(c1 - c0) * sizeof(T);
      }
      const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
      __syncwarp();  // the lanes' elements come before the arrive that publishes them (the sum orders no memory)
      if (lane == 0) mbar_arrive_expect_tx(&full[st], total);
      __syncwarp();
      if (mine) bulk_load(dst + off, src, bytes, &full[st]);
      return;
    }
    if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(arrays * n) * row_bytes);
    __syncwarp();
    for (int i = lane; i < arrays * n; i += 32) {
      const int arr = i / n, y = i - arr * n;
      const void* src = arr == 0   ? static_cast<const T*>(a.z) + (row0 + y) * a.zs
                        : arr == 1 ? static_cast<const T*>(a.dy) + (row0 + y) * a.dys
                                   : static_cast<const T*>(a.ds) + (row0 + y) * a.dss;
      bulk_load(ring + st * slot + (arr * ny + y) * row_bytes, src, row_bytes, &full[st]);
    }
  };
  if (threadIdx.x == 0 && threadIdx.y == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  if (warp == 0) reinterpret_cast<float2*>(red)[lane] = make_float2(0.0f, 0.0f);  // (an odd row's last one stays so)
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  long long row0 = static_cast<long long>(blockIdx.x) * ny;
  if (warp == 0)
    for (int i = 0; i < stages; ++i)
      if (row0 + i * step < a.rows) fill(row0 + i * step, i);
  // (the same in every turn: `step` is a multiple of the phases' period)
  const int ph = SHIFT ? row_phase<T>(a.z, (row0 + threadIdx.y) * a.zs) : 0;
  f32x2 dw[VPT][H], w[VPT][H];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V - ph;
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 0.0f;
    if (c < a.cols) load_weights<T, SHIFT>(a.w, a.w_f32, c, a.cols, f);
#pragma unroll
    for (int j = 0; j < H; ++j) dw[i][j] = 0, w[i][j] = pair2(f[2 * j], f[2 * j + 1]);
  }
  const float inv = 1.0f / static_cast<float>(a.cols);
  int st = 0, last = -1;
  uint32_t phase = 0;
  bool ok = true;
  for (int par = 0; row0 < a.rows; row0 += step, par ^= 1) {
    const long long row = row0 + threadIdx.y;
    const bool mine = row < a.rows;
    ok = ok && wait_bounded(&full[st], phase, nullptr, a.err, a.timeout_ns);
    const uint8_t* src = ring + st * slot + threadIdx.y * row_bytes;
    uint4 rz[kReread ? 1 : VPT], ry[kReread ? 1 : VPT];
    f32x2 ss2 = 0, dot2 = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      if (FULL || (mine && c < a.cols)) {
        f32x2 zv[H], gv[H];
        uint4 uz = *reinterpret_cast<const uint4*>(src + (c + ph) * sizeof(T));
        uint4 uy = *reinterpret_cast<const uint4*>(src + ny * row_bytes + (c + ph) * sizeof(T));
        if (SHIFT && !whole<T>(c, a.cols)) keep_row<T>(uz, c, a.cols), keep_row<T>(uy, c, a.cols);
        if (!kReread) rz[i] = uz, ry[i] = uy;
        unpack2<T>(uz, zv);
        unpack2<T>(uy, gv);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          ss2 = fma2(zv[j], zv[j], ss2);
          dot2 = fma2(mul2(gv[j], w[i][j]), zv[j], dot2);
        }
      }
    }
    float ss = unpair2(ss2).x + unpair2(ss2).y, dot = unpair2(dot2).x + unpair2(dot2).y;
    // the lower half of the warp joins ss, the upper half dot
    float v = (lane < 16 ? ss : dot) + __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? dot : ss, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((lane & 15) == 0) reinterpret_cast<float*>(&red[par][red0 + (threadIdx.x >> 5)])[lane >> 4] = v;
    __syncthreads();
    // (past the barrier: the slot of the group before is free)
    if (warp == 0 && last >= 0 && row0 + (stages - 1) * step < a.rows) fill(row0 + (stages - 1) * step, last);
    {  // every thread adds the row's warps up, always in the same order
      // (loads that do not wait for one another: 8192 x 2560 36 us, a loop 68)
      const ulonglong2* r = reinterpret_cast<const ulonglong2*>(&red[par][red0]);
      constexpr int Q = norm_bwd_threads(VPT) / 64;
      f32x2 q[Q];
      if (nwarp == 2 * Q) {
#pragma unroll
        for (int i = 0; i < Q; ++i) q[i] = add2(r[i].x, r[i].y);
      } else {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          q[i] = 0;
          if (2 * i < nwarp) q[i] = add2(r[i].x, r[i].y);
        }
      }
#pragma unroll
      for (int o = Q / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) q[i] = add2(q[2 * i], q[2 * i + 1]);
      const f32x2 t = q[0];
      ss = unpair2(t).x, dot = unpair2(t).y;
    }
    float rstd = rsqrtf(fmaf(ss, inv, a.eps));
    float m = -dot * rstd * inv;  // minus the mean of dy w n
    if ((FULL || mine) && !mean_holds(fmaf(ss, inv, a.eps))) {
      // (the same for the whole row) each warp sums the row by itself: no
      // barrier that the block's other rows would have to meet
      const float p = norm_rescale(fmaf(ss, inv, a.eps));
      const float2 t = warp_sums<T>(reinterpret_cast<const T*>(src) + ph,
                                    reinterpret_cast<const T*>(src + ny * row_bytes) + ph,
                                    a.w, a.w_f32, a.cols, p);
      const float r = rsqrtf(fmaf(t.x, inv, a.eps * p * p));
      m = -t.y * r * inv;
      rstd = r * p;
    }
    const f32x2 rstd2 = pair2(rstd, rstd), m2 = pair2(m, m);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      if (FULL || (mine && c < a.cols)) {
        f32x2 zv[H], gv[H], sv[H];
        uint4 uz, uy;
        if (kReread) {
          uz = *reinterpret_cast<const uint4*>(src + (c + ph) * sizeof(T));
          uy = *reinterpret_cast<const uint4*>(src + ny * row_bytes + (c + ph) * sizeof(T));
          if (SHIFT && !whole<T>(c, a.cols)) keep_row<T>(uz, c, a.cols), keep_row<T>(uy, c, a.cols);
        } else {
          uz = rz[i], uy = ry[i];
          opaque(uz), opaque(uy);
        }
        unpack2<T>(uz, zv);
        unpack2<T>(uy, gv);
        if (arrays == 3) {
          unpack2<T>(*reinterpret_cast<const uint4*>(src + 2 * ny * row_bytes + (c + ph) * sizeof(T)), sv);
        } else {
#pragma unroll
          for (int j = 0; j < H; ++j) sv[j] = 0;
        }
        float o[V];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const f32x2 n = mul2(zv[j], rstd2);
          dw[i][j] = fma2(gv[j], n, dw[i][j]);
          const float2 d = unpair2(fma2(rstd2, fma2(n, m2, mul2(gv[j], w[i][j])), sv[j]));
          o[2 * j] = d.x, o[2 * j + 1] = d.y;
        }
        T* dz = static_cast<T*>(a.dz) + row * a.dzs;
        if (SHIFT)
          store_piece<T, SHIFT>(dz, c, a.cols, Elem<T>::pack(o));
        else
          *reinterpret_cast<uint4*>(dz + c) = Elem<T>::pack(o);
      }
    }
    last = st;
    if (++st == stages) {
      st = 0;
      phase ^= 1u;
    }
  }
  if (!ok && warp == 0 && lane == 0) {
    // a wait ran out: no copy may still be landing when the block ends
    const long long groups = (a.rows - static_cast<long long>(blockIdx.x) * ny + step - 1) / step;
    for (int i = 0; i < stages && i < groups; ++i)
      wait_bounded(&full[i], static_cast<uint32_t>((groups - 1 - i) / stages) & 1u, nullptr, a.err, a.timeout_ns);
  }
  if (a.part == nullptr) return;
  float* out = a.part + static_cast<long long>(blockIdx.x) * a.cols;
  const auto leave = [&](float* to, int c, const f32x2(&v)[H]) {
#pragma unroll
    for (int j = 0; j < H; j += 2) {
      const float2 lo = unpair2(v[j]), hi = unpair2(v[j + 1]);
      const float f[4] = {lo.x, lo.y, hi.x, hi.y};
      if constexpr (SHIFT) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + 2 * j + k >= 0 && c + 2 * j + k < a.cols) to[c + 2 * j + k] = f[k];
      } else {
        *reinterpret_cast<float4*>(to + c + 2 * j) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  };
  if (ny == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * V - ph;
      if (c < a.cols) leave(out, c, dw[i]);
    }
    return;
  }
  // the group's rows first join their shares in the ring, which is free now
  float* sdw = reinterpret_cast<float*>(ring);  // [blockDim.y][cols]
  __syncthreads();
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V - ph;
    if (c < a.cols) leave(sdw + threadIdx.y * a.cols, c, dw[i]);
  }
  __syncthreads();
  for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < a.cols; c += blockDim.x * ny) {
    float v = 0.0f;
    for (int y = 0; y < ny; ++y) v += sdw[y * a.cols + c];
    out[c] = v;
  }
}

// Rows without 16-byte alignment whose phases differ or that are short, P
// elements an access, up to 8 a thread: dz
// and the row statistic in one pass, a row a block (or a warp a row).
template <typename T, int P>
__global__ void __launch_bounds__(kNormBwdElemThreads) rms_norm_bwd_elem_kernel(const NormBwdArgs a) {
  constexpr int E = kNormElems;
  __shared__ float2 red[64];
  const long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;  // (blocks of several rows have no barrier)
  const T* z = static_cast<const T*>(a.z) + row * a.zs;
  const T* dy = static_cast<const T*>(a.dy) + row * a.dys;
  const T* ds = a.ds == nullptr ? nullptr : static_cast<const T*>(a.ds) + row * a.dss;
  float zv[E][P], gw[E][P], d[E][P];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * P;
#pragma unroll
    for (int j = 0; j < P; ++j) zv[i][j] = gw[i][j] = d[i][j] = 0.0f;
    if (c < a.cols) {
      load_p<T, P>(z + c, zv[i]);
      load_p<T, P>(dy + c, gw[i]);
      if (ds != nullptr) load_p<T, P>(ds + c, d[i]);  // (now, so that one latency covers all three)
    }
  }
  float ss = 0.0f, dot = 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * P;
    if (c < a.cols) {
      float w[P];
      weight_p<T, P>(a.w, a.w_f32, c, w);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        gw[i][j] *= w[j];
        ss = fmaf(zv[i][j], zv[i][j], ss);
        dot = fmaf(gw[i][j], zv[i][j], dot);
      }
    }
  }
  float2 t = row_sum2(ss, dot, red, 0);
  const float ms = t.x / static_cast<float>(a.cols) + a.eps;
  float rstd = __frsqrt_rn(ms);
  float m = t.y * rstd / static_cast<float>(a.cols);
  if (!mean_holds(ms)) {
    const float p = norm_rescale(ms);
    ss = dot = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        ss = fmaf(zv[i][j] * p, zv[i][j] * p, ss);
        dot = fmaf(gw[i][j], zv[i][j] * p, dot);
      }
    t = row_sum2(ss, dot, red, 1);
    const float r = __frsqrt_rn(t.x / static_cast<float>(a.cols) + a.eps * p * p);
    m = t.y * r / static_cast<float>(a.cols);
    rstd = r * p;
  }
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * P;
    if (c < a.cols) {
#pragma unroll
      for (int j = 0; j < P; ++j) d[i][j] = fmaf(rstd, fmaf(-zv[i][j] * rstd, m, gw[i][j]), d[i][j]);
      store_p<T, P>(static_cast<T*>(a.dz) + row * a.dzs + c, d[i]);
    }
  }
}

// Any width and alignment, one row a block at a time.  With dynamic shared
// memory for a row of dw (`sums`) the block takes every gridDim.x-th row and
// leaves a partial row of dw like the kernel above (each thread adds to its
// own columns only); else it leaves the row statistic for
// rms_norm_dw_kernel.
template <typename T>
__global__ void __launch_bounds__(256) rms_norm_bwd_loop_kernel(const NormBwdArgs a, int sums) {
  extern __shared__ float sdw[];  // [cols] with sums
  __shared__ float2 red[64];
  pdl_wait();
  pdl_trigger();
  if (sums)
    for (int c = threadIdx.x; c < a.cols; c += 256) sdw[c] = 0.0f;
  int par = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, par ^= 1) {
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    const T* dy = static_cast<const T*>(a.dy) + row * a.dys;
    float ss = 0.0f, dot = 0.0f, run = 0.0f, drun = 0.0f;
    const auto join = [&] { ss += run, dot += drun, run = drun = 0.0f; };
    loop_columns(a.cols, [&](int c) {
      const float zv = Elem<T>::get(z[c]);
      run = fmaf(zv, zv, run);
      drun = fmaf(Elem<T>::get(dy[c]) * weight_at<T>(a.w, a.w_f32, c), zv, drun);
    }, join);
    const float2 t = row_sum2(ss, dot, red, par);
    const float ms = t.x / static_cast<float>(a.cols) + a.eps;
    float rstd = __frsqrt_rn(ms);
    float m = t.y * rstd / static_cast<float>(a.cols);
    if (!mean_holds(ms)) {
      const float p = norm_rescale(ms);
      ss = dot = 0.0f;
      loop_columns(a.cols, [&](int c) {
        const float zp = Elem<T>::get(z[c]) * p;
        run = fmaf(zp, zp, run);
        drun = fmaf(Elem<T>::get(dy[c]) * weight_at<T>(a.w, a.w_f32, c), zp, drun);
      }, join);
      __syncthreads();  // every thread has read the first sums
      const float2 t2 = row_sum2(ss, dot, red, par);
      const float r = __frsqrt_rn(t2.x / static_cast<float>(a.cols) + a.eps * p * p);
      m = t2.y * r / static_cast<float>(a.cols);
      rstd = r * p;
    }
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
    T* dz = static_cast<T*>(a.dz) + row * a.dzs;
    const T* ds = a.ds == nullptr ? nullptr : static_cast<const T*>(a.ds) + row * a.dss;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      const float n = Elem<T>::get(z[c]) * rstd;
      const float gv = Elem<T>::get(dy[c]);
      const float d = rstd * fmaf(-n, m, gv * weight_at<T>(a.w, a.w_f32, c));
      dz[c] = Elem<T>::put(ds != nullptr ? d + Elem<T>::get(ds[c]) : d);
      if (sums) sdw[c] = fmaf(gv, n, sdw[c]);
    }
  }
  if (sums)
    for (int c = threadIdx.x; c < a.cols; c += 256) a.part[static_cast<long long>(blockIdx.x) * a.cols + c] = sdw[c];
}

// Partial sums of dw over the rows of one chunk (blockIdx.y): a thread owns P
// columns.  Reads what the rows' kernel left in rstd.
template <typename T, int P>
__global__ void __launch_bounds__(128) rms_norm_dw_kernel(const NormBwdArgs a, int chunk) {
  pdl_wait();
  pdl_trigger();
  const long long c = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) * P;
  if (c >= a.cols) return;
  const long long r0 = static_cast<long long>(blockIdx.y) * chunk;
  const long long r1 = min(r0 + chunk, a.rows);
  float v[P];
#pragma unroll
  for (int j = 0; j < P; ++j) v[j] = 0.0f;
#pragma unroll 8
  for (long long r = r0; r < r1; ++r) {
    float g[P], z[P];
    load_p<T, P>(static_cast<const T*>(a.dy) + r * a.dys + c, g);
    load_p<T, P>(static_cast<const T*>(a.z) + r * a.zs + c, z);
    const float rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = fmaf(g[j], z[j] * rstd, v[j]);
  }
#pragma unroll
  for (int j = 0; j < P; ++j) a.part[static_cast<long long>(blockIdx.y) * a.cols + c + j] = v[j];
}

// dw[c] = sum of part[0..parts)[c], in a fixed order: 8 threads of P columns a
// block, 32 threads a column take every 32nd partial, joined in shared memory.
template <int P>
struct DwPiece {
  using type = float;
};
template <>
struct DwPiece<4> {
  using type = float4;
};

template <int P>
__global__ void __launch_bounds__(256) dw_reduce_kernel(const float* part, int parts, int cols, void* dw, int dt) {
  constexpr int kCols = 8 * P;
  __shared__ float sh[32][kCols + 1];
  pdl_wait();
  pdl_trigger();
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int c = blockIdx.x * kCols + tx * P;
  float v[P];
#pragma unroll
  for (int j = 0; j < P; ++j) v[j] = 0.0f;
  if (c < cols) {
    // sixteen loads at a time: the partials are few, and their latency is the
    // kernel's time (rows past the last one are read as that one, so that no
    // load waits for a branch)
    for (int p0 = ty; p0 < parts; p0 += 32 * 16) {
      typename DwPiece<P>::type t[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        t[i] = *reinterpret_cast<const typename DwPiece<P>::type*>(
            part + static_cast<long long>(min(p0 + 32 * i, parts - 1)) * cols + c);
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j)
          if (p0 + 32 * i < parts) v[j] += reinterpret_cast<const float*>(&t[i])[j];
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j) sh[ty][tx * P + j] = v[j];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < P; ++j) {
    float r = sh[lane][warp * P + j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    const int oc = blockIdx.x * kCols + warp * P + j;
    if (lane == 0 && oc < cols) store_elem(static_cast<char*>(dw) + static_cast<long long>(oc) * dtype_size(dt), dt, r);
  }
}

}  // namespace msb
