// host_sm100.cuh - what the host code of the library's translation units
// shares: the per-device state, launch records, workspace carving and the
// description of a matrix that a tensor map is made of.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "gemm_sm100.cuh"
#include "msign_b200.h"

namespace msb {

constexpr unsigned long long kWaitLimitNs = 4000000000ull;  // 4 s per wait

// ---------------------------------------------------------------- device state

struct DeviceState {
  bool ready = false;
  int sms = 0;
  int max_pairs = 0;  // CTA pairs of the GEMM kernel that fit on the GPU at once
  int ingest_blocks = 0;  // ingest_kernel blocks resident at once on the whole GPU
  int* err = nullptr;
};

// The current device's state, set up on first use (msign_b200.cu).
msign_status device_state(DeviceState** out);
extern PFN_cuTensorMapEncodeTiled_v12000 g_encode;

// Launch records (see msign_profile_enable): every launch is bracketed by
// prof_begin and prof_end on its stream.
void prof_begin(cudaStream_t s);
void prof_end(int kind, cudaStream_t s, double flops, double bytes);

// ---------------------------------------------------------------- helpers

inline int64_t round_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int to_dt(msign_dtype d) { return d == MSIGN_BF16 ? DT_BF16 : d == MSIGN_FP16 ? DT_FP16 : DT_FP32; }

inline bool valid_dtype(msign_dtype d) { return d == MSIGN_BF16 || d == MSIGN_FP16 || d == MSIGN_FP32; }

// Workspace carving: the same routine sizes and slices the workspace.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    off = (off + 1023) & ~size_t(1023);
    void* p = base ? base + off : nullptr;
    off += bytes;
    return p;
  }
};

// A dense batched matrix: rows x cols, leading dimension ld, batch stride bs
// (both in elements).
struct Mat {
  const void* ptr;
  int dt;
  int64_t rows, cols, ld, bs;
};

inline bool tma_ok(const Mat& m) {
  const int es = dtype_size(m.dt);
  return (reinterpret_cast<uintptr_t>(m.ptr) % 16) == 0 && (m.ld * es) % 16 == 0 && (m.bs * es) % 16 == 0;
}

inline msign_status launch_ok() { return cudaGetLastError() == cudaSuccess ? MSIGN_OK : MSIGN_ERR_CUDA; }

}  // namespace msb
