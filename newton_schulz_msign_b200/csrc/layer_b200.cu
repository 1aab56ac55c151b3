// layer_b200.cu - C ABI of the layer operators around the Muon step
// (declared in include/msign_b200.h): RMS norm with its int8 output and its
// gradients, the gated feed-forward block with its gradients, and the int8
// product with scales.  Argument checks, workspace layout, tensor maps and
// launches; the kernels are in norm_sm100.cuh and dense_sm100.cuh.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "dense_sm100.cuh"
#include "host_sm100.cuh"
#include "msign_b200.h"
#include "norm_sm100.cuh"

namespace msb {

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
// int8 products: |a b| <= 2^14, so K < 2^17 keeps every int32 sum exact
constexpr int64_t kMaxI8K = (int64_t(1) << 17) - 1;

// Launch with the programmatic-dependent attribute (every kernel here waits
// for its predecessor before it touches memory) and, where cluster > 0, that
// cluster width.
template <typename... KArgs, typename... Args>
msign_status launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, int kind, double flops,
                    double bytes, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 0) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = at;
  prof_begin(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  prof_end(kind, stream, flops, bytes);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return MSIGN_ERR_CUDA;
  }
  return MSIGN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) % 16) == 0; }

// A row stride argument: 0 means rows back to back.
int64_t stride_of(int64_t stride, int64_t cols) { return stride > 0 ? stride : cols; }
bool valid_stride(int64_t stride, int64_t cols) { return stride == 0 || stride >= cols; }

// Rows that 16-byte accesses reach: an aligned base, and a stride of whole
// 16-byte pieces where there is more than one row.
bool rows_aligned(const void* p, int64_t stride, int64_t rows, int es) {
  return aligned16(p) && (rows <= 1 || (stride * es) % 16 == 0);
}

// Whether an output is one of the other buffers of its call (the same
// address: the overlap that a slip makes; nullptr matches nothing).
bool is_one_of(const void* p, std::initializer_list<const void*> others) {
  if (p == nullptr) return false;
  for (const void* o : others)
    if (o == p) return true;
  return false;
}

// Whether every address is a multiple of its element's size, which each access
// needs (es bytes; nullptr is).
bool on_elements(std::initializer_list<const void*> ps, int es) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % es != 0) return false;
  return true;
}

// Whether a product's 256 x 128 tiles can be counted in an int (the kernels'
// tile numbers): looked at before anything is enqueued.
bool countable(int64_t rows, int64_t cols) { return ceil_div(rows, 256) * ceil_div(cols, 128) <= INT32_MAX / 4; }

// ---------------------------------------------------------------- RMS norm

struct NormMatrix {
  const void* p;
  int64_t stride;
  int es;
};

NormReach norm_reach(std::initializer_list<NormMatrix> ms, const void* weight, bool w_f32, int es, int64_t rows,
                     int64_t cols) {
  const int v = 16 / es;
  // whether accesses of n elements reach every row of every matrix
  const auto reach = [&](int n) {
    // (a weight of fp32 is read 16 bytes at a time too)
    const int ws = std::min(16, n * (w_f32 ? 4 : es));
    if (cols % n != 0 || reinterpret_cast<uintptr_t>(weight) % ws != 0) return false;
    for (const NormMatrix& m : ms)
      if (m.p != nullptr &&
          (reinterpret_cast<uintptr_t>(m.p) % (n * m.es) != 0 || (rows > 1 && m.stride % n != 0)))
        return false;
    return true;
  };
  const NormMatrix& first = *ms.begin();
  bool shift = cols >= 32 * v;
  for (const NormMatrix& m : ms) {
    if (m.p == nullptr) continue;
    const auto at = reinterpret_cast<uintptr_t>(m.p), to = reinterpret_cast<uintptr_t>(first.p);
    shift = shift && at % m.es == 0 && at / m.es % v == to / first.es % v &&
            (rows <= 1 || m.stride % v == first.stride % v);
  }
  const bool vec = reach(v);
  return {vec, !vec && shift, reach(2) ? 2 : 1};
}

template <typename T, bool Q8>
msign_status norm_run(const NormArgs& a, const NormReach& by, double bytes, cudaStream_t stream) {
  const NormPlan p = norm_plan(a.cols, sizeof(T), by);
  auto* k = rms_norm_loop_kernel<T, Q8>;
  if (p.form == NormForm::kElems) {
    k = by.pair == 2 ? rms_norm_elem_kernel<T, 2, Q8> : rms_norm_elem_kernel<T, 1, Q8>;
  } else if (p.form == NormForm::kPieces) {
    // (rows that are shifted have more than 32 pieces)
    k = by.shift ? (p.vpt == 2 ? rms_norm_kernel<T, 2, Q8, true> : rms_norm_kernel<T, 4, Q8, true>)
                 : (p.vpt == 1   ? rms_norm_kernel<T, 1, Q8, false>
                    : p.vpt == 2 ? rms_norm_kernel<T, 2, Q8, false>
                                 : rms_norm_kernel<T, 4, Q8, false>);
  }
  return launch(k, dim3(static_cast<unsigned>(ceil_div(a.rows, p.y))), dim3(p.x, p.y), 0, 0, 3, 0.0, bytes, stream, a);
}

msign_status norm_call(const void* x, const void* residual, const void* weight, void* y, void* sum_out, float* scale,
                       msign_dtype io_dtype, msign_dtype w_dtype, int64_t rows, int64_t cols, int64_t x_stride,
                       int64_t r_stride, int64_t y_stride, int64_t s_stride, float eps, msign_stream_t stream) {
  const bool q8 = scale != nullptr;
  if (!valid_dtype(io_dtype) || !valid_dtype(w_dtype)) return MSIGN_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return MSIGN_ERR_INVALID_ARG;
  if (!valid_stride(x_stride, cols) || !valid_stride(r_stride, cols) || !valid_stride(y_stride, cols) ||
      !valid_stride(s_stride, cols))
    return MSIGN_ERR_INVALID_ARG;
  if (residual == nullptr && sum_out != nullptr) return MSIGN_ERR_INVALID_ARG;
  if (rows > 0 && cols > 0 &&
      (is_one_of(y, {sum_out, weight}) || is_one_of(sum_out, {weight}) || (q8 && is_one_of(y, {x, residual})) ||
       is_one_of(scale, {x, residual, weight, y, sum_out})))
    return MSIGN_ERR_INVALID_ARG;
  if (weight != nullptr && w_dtype != io_dtype && w_dtype != MSIGN_FP32) return MSIGN_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return MSIGN_OK;
  if (x == nullptr || y == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (rows > kMaxDim || cols > kMaxDim) return MSIGN_ERR_UNSUPPORTED;
  if (!on_elements({x, residual, sum_out}, dtype_size(to_dt(io_dtype))) ||
      !on_elements({y}, q8 ? 1 : dtype_size(to_dt(io_dtype))) || !on_elements({weight}, dtype_size(to_dt(w_dtype))) ||
      !on_elements({scale}, 4))
    return MSIGN_ERR_INVALID_ARG;
  // an output over an input: row over row, or one row's block would write what another still reads
  const auto apart = [&](const void* o, int64_t o_stride, const void* in, int64_t in_stride) {
    return rows > 1 && o == in && o != nullptr && stride_of(o_stride, cols) != stride_of(in_stride, cols);
  };
  if (apart(y, y_stride, x, x_stride) || apart(y, y_stride, residual, r_stride) ||
      apart(sum_out, s_stride, x, x_stride) || apart(sum_out, s_stride, residual, r_stride))
    return MSIGN_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  msign_status st = device_state(&dev);
  if (st != MSIGN_OK) return st;
  NormArgs a = {};
  a.x = x, a.r = residual, a.w = weight, a.y = y, a.s = sum_out, a.scale = scale;
  a.xs = stride_of(x_stride, cols), a.rs = stride_of(r_stride, cols);
  a.ys = stride_of(y_stride, cols), a.ss = stride_of(s_stride, cols);
  a.rows = rows, a.cols = static_cast<int>(cols), a.eps = eps;
  a.w_f32 = w_dtype == MSIGN_FP32;
  const int dt = to_dt(io_dtype), es = dtype_size(dt);
  const NormReach by = norm_reach({{x, a.xs, es}, {residual, a.rs, es}, {sum_out, a.ss, es}, {y, a.ys, q8 ? 1 : es}},
                                  weight, a.w_f32, es, rows, cols);
  const double e = static_cast<double>(rows) * cols;
  const double bytes = e * es * (1 + (residual != nullptr) + (sum_out != nullptr)) + e * (q8 ? 1 : es);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == DT_BF16)
    return q8 ? norm_run<__nv_bfloat16, true>(a, by, bytes, s) : norm_run<__nv_bfloat16, false>(a, by, bytes, s);
  if (dt == DT_FP16) return q8 ? norm_run<__half, true>(a, by, bytes, s) : norm_run<__half, false>(a, by, bytes, s);
  return q8 ? norm_run<float, true>(a, by, bytes, s) : norm_run<float, false>(a, by, bytes, s);
}

template <typename T, int KIND>
auto* norm_bwd_kernel(int vpt) {
  if constexpr (KIND != NORM_SHIFT)  // (rows that are shifted have more than 32 pieces)
    if (vpt == 1) return rms_norm_bwd_kernel<T, 1, KIND>;
  return vpt == 2 ? rms_norm_bwd_kernel<T, 2, KIND> : rms_norm_bwd_kernel<T, 4, KIND>;
}

template <typename T>
msign_status norm_bwd_run(NormBwdArgs a, void* dw, int dw_dt, const NormReach& by, char* ws, double bytes,
                          cudaStream_t stream) {
  Carver cv(ws);
  float* part = static_cast<float*>(cv.take(sizeof(float) * std::min<int64_t>(a.rows, kDwParts) * a.cols));
  float* rstd = static_cast<float*>(cv.take(sizeof(float) * a.rows));
  a.part = dw != nullptr ? part : nullptr;
  const NormBwdPlan plan = norm_bwd_plan(a.rows, a.cols, sizeof(T), by, a.ds != nullptr, dw != nullptr);
  const NormPlan& p = plan.p;
  const dim3 block(p.x, p.y);
  int64_t parts = plan.parts;
  const int pair = by.pair;
  msign_status st;
  if (p.form == NormForm::kPieces) {
    auto* k = by.shift    ? norm_bwd_kernel<T, NORM_SHIFT>(p.vpt)
              : plan.full ? norm_bwd_kernel<T, NORM_FULL>(p.vpt)
                          : norm_bwd_kernel<T, NORM_ROWS>(p.vpt);
    st = launch(k, dim3(static_cast<unsigned>(parts)), block, static_cast<size_t>(plan.stages) * plan.slot, 0, 3, 0.0,
                bytes, stream, a, plan.stages);
    if (st != MSIGN_OK) return st;
  } else if (p.form == NormForm::kLoopSums) {
    st = launch(rms_norm_bwd_loop_kernel<T>, dim3(static_cast<unsigned>(parts)), block, sizeof(float) * a.cols, 0, 3,
                0.0, bytes, stream, a, 1);
    if (st != MSIGN_OK) return st;
  } else {
    a.rstd = dw != nullptr ? rstd : nullptr;
    if (p.form == NormForm::kElems)
      st = launch(pair == 2 ? rms_norm_bwd_elem_kernel<T, 2> : rms_norm_bwd_elem_kernel<T, 1>,
                  dim3(static_cast<unsigned>(ceil_div(a.rows, p.y))), block, 0, 0, 3, 0.0, bytes, stream, a);
    else
      st = launch(rms_norm_bwd_loop_kernel<T>, dim3(static_cast<unsigned>(a.rows)), block, 0, 0, 3, 0.0, bytes, stream,
                  a, 0);
    if (st != MSIGN_OK || dw == nullptr) return st;
    const int chunk = static_cast<int>(ceil_div(a.rows, std::min<int64_t>(a.rows, kDwLoopParts)));
    parts = ceil_div(a.rows, chunk);
    st = launch(pair == 2 ? rms_norm_dw_kernel<T, 2> : rms_norm_dw_kernel<T, 1>,
                dim3(static_cast<unsigned>(ceil_div(a.cols, 128 * pair)), static_cast<unsigned>(parts)), dim3(128), 0, 0,
                3, 0.0, 0.0, stream, a, chunk);
    if (st != MSIGN_OK) return st;
  }
  if (dw == nullptr) return MSIGN_OK;
  const int quad = a.cols % 4 == 0 ? 4 : 1;
  return launch(quad == 4 ? dw_reduce_kernel<4> : dw_reduce_kernel<1>,
                dim3(static_cast<unsigned>(ceil_div(a.cols, 8 * quad))), dim3(256), 0, 0, 3, 0.0,
                4.0 * parts * a.cols, stream, static_cast<const float*>(part), static_cast<int>(parts), a.cols, dw,
                dw_dt);
}

// ---------------------------------------------------------------- products

CUtensorMapDataType tma_type(int dt, bool i8) {
  if (i8) return CU_TENSOR_MAP_DATA_TYPE_UINT8;
  return dt == DT_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
         : dt == DT_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
}

// Tensor map of rows x cols elements (es bytes each, row stride ld), `z` of
// them zs elements apart, in the 128-byte swizzle.  Elements of a box beyond
// the extents read as 0 and are not written.
bool map_rows(CUtensorMap* tm, const void* p, CUtensorMapDataType type, int es, int64_t rows, int64_t cols, int64_t ld,
              int box_cols, int box_rows, int64_t z = 1, int64_t zs = 0, bool out = false) {
  const int64_t row_bytes = rows > 1 || z > 1 ? ld * es : round_up(cols * es, 16);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(z)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes),
                           static_cast<cuuint64_t>(z > 1 ? zs * es : row_bytes * rows)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return g_encode(tm, type, 3, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B,
                  out ? CU_TENSOR_MAP_L2_PROMOTION_NONE : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// From row to row, in elements, of an operand that this file lays out: a
// multiple of 128 bytes, so that a box's row of 128 bytes is one line of the L2
// (at 16-byte multiples int8 4096 x 4096 x 4098 takes 75 us instead of 60, 2048
// x 4096 x 11016 103 instead of 85, the gradients of 513 x 1000 x 2730 32
// instead of 30.5); of 16 bytes where that would add more than a quarter.
int64_t pitch_of(int64_t cols, int es) { return round_up(cols, (cols * es >= 512 ? 128 : 16) / es); }

// An operand's rows as a tensor map takes them: where they lie, or copied
// into the workspace.
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
  int es;
  bool direct() const { return rows_aligned(p, ld, rows, es); }
  int64_t padded_ld() const { return pitch_of(cols, es); }
  size_t padded_bytes() const { return static_cast<size_t>(rows) * padded_ld() * es; }
};

void carve_operand(Carver& cv, const Operand& o, void** copy) { *copy = o.direct() ? nullptr : cv.take(o.padded_bytes()); }

// Copies the operands that have a place for it (copies[i] not null), all in
// one launch, and points them there.
msign_status place_operands(std::initializer_list<Operand*> ops, std::initializer_list<void*> copies,
                            cudaStream_t stream) {
  PadArgs a = {};
  int n = 0;
  int64_t most = 0;
  double bytes = 0.0;
  auto copy = copies.begin();
  for (Operand* o : ops) {
    void* to = *copy++;
    if (to == nullptr) continue;
    a.in[n] = static_cast<const uint8_t*>(o->p), a.out[n] = static_cast<uint8_t*>(to);
    a.ld[n] = o->ld * o->es, a.ld_out[n] = o->padded_ld() * o->es, a.rows[n] = o->rows, a.bytes[n] = o->cols * o->es;
    most = std::max(most, o->rows * ceil_div(a.bytes[n], 16));
    bytes += 2.0 * o->rows * o->cols * o->es;
    o->p = to;
    o->ld = o->padded_ld();
    ++n;
  }
  if (n == 0) return MSIGN_OK;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(most, 256), 16 * kPlanSms)), static_cast<unsigned>(n));
  return launch(pad_rows_kernel, grid, dim3(256), 0, 0, 2, 0.0, bytes, stream, a);
}

// Instruction descriptor: D type (fp32 or int32), A and B types, which of
// them is read MN-major, N and M of the MMA.
uint32_t make_idesc(int dt, bool i8, bool a_mn, bool b_mn, int n, int m) {
  const uint32_t fmt = i8 ? 1u : (dt == DT_BF16 ? 1u : 0u);  // signed int8; bf16 or fp16
  return ((i8 ? 2u : 1u) << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

template <typename K>
msign_status smem_limit(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess
             ? MSIGN_OK
             : MSIGN_ERR_CUDA;
}

template <typename T>
msign_status norm_bwd_limits() {
  for (int vpt : {1, 2, 4})
    for (auto* k : {norm_bwd_kernel<T, NORM_ROWS>(vpt), norm_bwd_kernel<T, NORM_FULL>(vpt), norm_bwd_kernel<T, NORM_SHIFT>(vpt)})
      if (const msign_status st = smem_limit(k, kNormRingMax); st != MSIGN_OK) return st;
  return MSIGN_OK;
}

std::mutex g_layer_mu;
bool g_layer_ready[64] = {};

// The device's state, with the kernels' shared memory limits raised.
msign_status layer_state(DeviceState** out) {
  msign_status st = device_state(out);
  if (st != MSIGN_OK) return st;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MSIGN_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_layer_mu);
  if (g_layer_ready[dev]) return MSIGN_OK;
  for (msign_status s :
       {smem_limit(dense_pair_kernel<PAIR_GATED>, kPairSmemBytes), smem_limit(dense_pair_kernel<PAIR_I8>, kPairSmemBytes),
        smem_limit(dense_pair_kernel<PAIR_DX>, kPairSmemBytes), smem_limit(dense_pair_kernel<PAIR_DW>, kPairSmemBytes),
        smem_limit(dense_stream_kernel<PAIR_GATED>, kSmemMax), smem_limit(dense_stream_kernel<PAIR_I8>, kSmemMax),
        smem_limit(dense_stream_kernel<PAIR_DX>, kSmemMax), smem_limit(dense_stream_kernel<PAIR_DW>, kSmemMax),
        norm_bwd_limits<__nv_bfloat16>(), norm_bwd_limits<__half>(), norm_bwd_limits<float>()})
    if (s != MSIGN_OK) return s;
  g_layer_ready[dev] = true;
  return MSIGN_OK;
}

// Outputs o of the pair kernel, M x N each.
bool pair_outputs(PairParams* p, int n, void* const* out, const int64_t* ld, int odt) {
  const int es = dtype_size(odt);
  p->odt = odt;
  p->tma_out = 1;
  for (int o = 0; o < n; ++o) {
    p->out[o] = out[o];
    p->ldo[o] = ld[o];
    if (out[o] != nullptr && !rows_aligned(out[o], ld[o], p->M, es)) p->tma_out = 0;
  }
  if (p->tma_out)
    for (int o = 0; o < n; ++o)
      if (out[o] != nullptr &&
          !map_rows(&p->tmO[o], out[o], tma_type(odt, false), es, p->M, p->N, ld[o], 128 / es, 32, 1, 0, true))
        return false;
  return true;
}

template <int MODE>
msign_status pair_launch(PairParams* p, int64_t nz, double flops, double bytes, DeviceState* dev, cudaStream_t stream) {
  const int cols = MODE == PAIR_GATED ? 128 : kBN;
  p->tiles_m = static_cast<int>(ceil_div(p->M, kBM));
  p->tiles_n = static_cast<int>(ceil_div(p->N, cols));
  const int64_t total = int64_t(p->tiles_m) * p->tiles_n * nz;
  if (total > INT32_MAX / 2) return MSIGN_ERR_UNSUPPORTED;
  p->total = static_cast<int>(total);
  // Tile rows walked together: as many as hold their A rows in about a
  // quarter of the L2, so that B is read from HBM once a band (sustained,
  // int8 8192 x 14336 x 4096: 8 rows 357 us, 16 343; gated block 4096 x 4096 x
  // 14336: 734 and 720); at least 8, whose tiles share K slices in time.
  const double panel = 256.0 * p->nk * p->segs * kRowBytes;
  p->band = std::min(p->tiles_m, std::max(8, std::min(32, static_cast<int>(36e6 / panel))));
  p->err = dev->err;
  p->timeout_ns = kWaitLimitNs;
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(total, dev->max_pairs));
  // (the cluster width is compiled into the kernel)
  return launch(dense_pair_kernel<MODE>, dim3(grid), dim3(kThreads), kPairSmemBytes, 0, 0, flops, bytes, stream, *p);
}

// Whether a product of `rows` x `cols` outputs (`z` of them) goes to the
// stream kernel: few rows, or too few 256-row tiles to keep the CTA pairs
// busy.  Measured, stream and pair in us: int8 64 x 14336 x 4096 16.5 and 18.8,
// 128 x 14336 x 4096 20.0 and 19.6, 256 x 14336 x 4096 (56 tiles) 26 and 18,
// 256 x 4096 x 14336 (16 tiles) 21.4 and 39; gated 128 x 4096 x 14336 48 and
// 56, 256 x 4096 x 14336 81 and 57, 256 x 4096 x 4096 (32 tiles) 22 and 28.
template <int MODE>
bool stream_takes(int64_t rows, int64_t cols, int64_t z) {
  return rows <= 128 || ceil_div(rows, kBM) * ceil_div(cols, MODE == PAIR_GATED ? 128 : kBN) * z < 48;
}

// Tile of a stream launch: the N operand's width (output rows a tile), the K
// splits (the cluster's width) and the shared memory of a CTA.  The least of
// an estimate in microseconds: the loads (each stage's 128 + bn rows of 128
// bytes) at 120 KB/us on the busiest SM and 100 on the average one, 0.02 a row
// of the tile for the join and the store, 1 and a quarter a rank for a join
// between ranks, and 3 for every further generation of CTAs.  Measured against
// single choices for all: tiles of at most 128 rows lose 22% on the 400 x 1000
// x 2736 gated block (18.7 against 14.5 us), tiles of 256 rows 25% on 256 x
// 4096 x 4096 int8 (15 against 11.8), two CTAs an SM for every narrow tile 12%
// on 64 x 14336 x 4096 int8 (18.3 against 16.3), one wherever they fit 20% on
// 16 x 4096 x 4096 int8 (5.4 against 4.5), and clusters counted as if they
// filled all SMs 38% on dx of 1000 x 768 x 2048 (23.1 against 16.8).
struct StreamPlan {
  int bn, splits, budget;
};

// CTAs that run at once as clusters of 1, 2, 4 and 8, one and two an SM (what
// the occupancy query answers on a B200: clusters do not span the GPCs, and
// some SMs of each are left over).
constexpr int kClusterCtas[2][4] = {{148, 148, 132, 120}, {296, 296, 284, 264}};

template <int MODE>
StreamPlan stream_plan(int64_t rows, int64_t cols, int64_t z, int64_t steps) {
  const int64_t unit = MODE == PAIR_DW ? 64 : 16;
  const int64_t tiles = ceil_div(cols, MODE == PAIR_GATED ? 64 : 128) * z;
  StreamPlan best = {};
  double least = 0.0;
  int64_t tried = 0;
  for (int64_t wide : {256, 192, 160, 128, 96, 64}) {
    const int64_t bn = round_up(ceil_div(rows, ceil_div(rows, wide)), unit);  // equal tiles
    if (bn == tried) continue;
    tried = bn;
    for (int splits = 1, log2 = 0; splits <= 8 && (splits == 1 || steps >= 2 * splits); splits *= 2, ++log2) {
      const int64_t ctas = tiles * ceil_div(rows, bn) * splits;
      const double kb = ceil_div(steps, splits) * (128 + bn) * 128 / 1e3;  // loads of a CTA
      // CTAs an SM, by shared memory: narrow tiles two, unless one a SM are
      // all of them and busy for long.  (Two of a long-lived cluster may share
      // an SM while others are idle; short ones gain by overlapping the next
      // launch.)
      const bool fit = ctas <= kClusterCtas[0][log2], brief = kb < 320;
      const int64_t per_sm = bn <= 128 && (!fit || brief) ? 2 : 1;
      const int64_t gens = ceil_div(ctas, kClusterCtas[per_sm - 1][log2]);
      const double busiest = static_cast<double>(
          per_sm == 1 ? gens : std::max<int64_t>(fit || brief ? 1 : 2, ceil_div(ctas, kPlanSms)));
      const double mean = per_sm == 1 ? static_cast<double>(gens) : std::max(1.0, static_cast<double>(ctas) / kPlanSms);
      const double us = std::max(kb * busiest / 120, kb * mean / 100) + 0.02 * bn +
                        (splits > 1 ? 1.0 + 0.25 * splits : 0.0) +
                        3.0 * (gens - 1);
      if (best.bn == 0 || us < least) {
        least = us;
        best = {static_cast<int>(bn), splits, per_sm == 2 ? 113 * 1024 : 220 * 1024};
      }
    }
  }
  return best;
}

template <int MODE>
msign_status stream_launch(StreamParams* p, const StreamPlan& plan, int64_t z, double flops, double bytes,
                           DeviceState* dev, cudaStream_t stream) {
  const int64_t tiles = ceil_div(p->N, MODE == PAIR_GATED ? 64 : 128), rows = ceil_div(p->tokens, plan.bn);
  if (tiles > INT32_MAX / 16 || rows > 65535) return MSIGN_ERR_UNSUPPORTED;
  p->bn = plan.bn;
  p->splits = plan.splits;
  // A CTA's share of an SM's TMEM (512 columns) never exceeds its share of the
  // shared memory: allocations then fit wherever the CTAs do, and no CTA waits
  // for one that waits, in its cluster, for another.
  p->tmem_cols = 32;
  while (p->tmem_cols < p->bn) p->tmem_cols *= 2;
  // what a rank holds of the sums
  const int join = p->splits * static_cast<int>(ceil_div(std::min(p->bn, p->tokens), p->splits)) * 512;
  p->push = p->splits > 1 && join <= 32 * 1024;
  const int fixed = 2048 + (p->push ? join : 0);  // alignment, barriers, the pushed sums
  p->stages = std::min(kStreamMaxStages, (plan.budget - fixed) / stream_stage_bytes(p->bn));
  // pulled sums lie where the stages were
  while (!p->push && p->stages * stream_stage_bytes(p->bn) < p->bn * 512) ++p->stages;
  p->join_off = stream_join_off(p->bn, p->stages);
  const int smem = p->stages * stream_stage_bytes(p->bn) + fixed;
  if (smem > kSmemMax || int64_t(smem) * 512 < int64_t(kSmemMax) * p->tmem_cols) return MSIGN_ERR_UNSUPPORTED;
  p->err = dev->err;
  p->timeout_ns = kWaitLimitNs;
  return launch(dense_stream_kernel<MODE>,
                dim3(static_cast<unsigned>(tiles * p->splits), static_cast<unsigned>(rows), static_cast<unsigned>(z)),
                dim3(kStreamThreads), smem, p->splits, 0, flops, bytes, stream, *p);
}

// Output pointers and row strides of a stream launch.
void stream_outputs(StreamParams* p, int n, void* const* out, const int64_t* ld, int odt) {
  const int es = dtype_size(odt);
  p->odt = odt;
  p->vec_out = 1;
  for (int o = 0; o < n; ++o) {
    p->out[o] = out[o], p->ldo[o] = ld[o];
    if (out[o] != nullptr && (reinterpret_cast<uintptr_t>(out[o]) % (4 * es) != 0 || (p->tokens > 1 && ld[o] % 4 != 0)))
      p->vec_out = 0;
  }
}

msign_status zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int es, cudaStream_t stream) {
  if (p == nullptr || rows == 0 || cols == 0) return MSIGN_OK;
  return cudaMemset2DAsync(p, static_cast<size_t>(ld) * es, 0, static_cast<size_t>(cols) * es,
                           static_cast<size_t>(rows), stream) == cudaSuccess
             ? MSIGN_OK
             : MSIGN_ERR_CUDA;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && (reinterpret_cast<uintptr_t>(ws) % 256) == 0);
}

size_t carved(const Carver& cv) { return cv.off == 0 ? 0 : cv.off + 1024; }

char* carve_base(void* ws) { return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 1023) & ~uintptr_t(1023)); }

// ---------------------------------------------------------------- gated feed-forward

struct FfnShape {
  int64_t t, d, h;
};

struct FfnCopies {
  void *x, *wg, *wu, *dgu;
};

void carve_ffn(Carver& cv, const FfnShape& s, const Operand& x, const Operand& wg, const Operand& wu, bool backward,
               FfnCopies* c) {
  carve_operand(cv, x, &c->x);
  carve_operand(cv, wg, &c->wg);
  carve_operand(cv, wu, &c->wu);
  c->dgu = backward ? cv.take(size_t(4) * s.t * pitch_of(s.h, 2)) : nullptr;
}

// Checks that the forward and the backward call share.
msign_status ffn_check(msign_dtype dtype, int act, const FfnShape& s, int64_t x_stride, int64_t w_stride) {
  if (!valid_dtype(dtype) || act < 0 || act > 2 || s.t < 0 || s.d < 0 || s.h < 0) return MSIGN_ERR_INVALID_ARG;
  if (!valid_stride(x_stride, s.d) || !valid_stride(w_stride, s.d)) return MSIGN_ERR_INVALID_ARG;
  if (dtype == MSIGN_FP32) return MSIGN_ERR_UNSUPPORTED;
  if (s.t > kMaxDim || s.d > kMaxDim || s.h > kMaxDim || !countable(s.t, s.h) || !countable(s.t, s.d) ||
      !countable(s.h, s.d))
    return MSIGN_ERR_UNSUPPORTED;
  return MSIGN_OK;
}

template <typename T>
msign_status dact_run(const void* dh, int64_t ldh, const void* gate, const void* up, int64_t ldp_in, void* dgu,
                      const FfnShape& s, int act, cudaStream_t stream) {
  const int64_t ldp = pitch_of(s.h, 2);
  // whether accesses of n elements reach every row
  const auto reach = [&](int n) {
    const auto in = [&](const void* p, int64_t ld) {
      return reinterpret_cast<uintptr_t>(p) % (2 * n) == 0 && (s.t <= 1 || ld % n == 0);
    };
    return s.h % n == 0 && in(dh, ldh) && in(gate, ldp_in) && in(up, ldp_in);
  };
  // about 16 blocks an SM, each a few rows
  const int64_t gx = ceil_div(ldp, 512);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>(
                                                 ceil_div(s.t, 4), std::max<int64_t>(1, 16 * kPlanSms / gx))));
  auto* k = reach(8) ? gated_dact_kernel<T, 8> : reach(2) ? gated_dact_kernel<T, 2> : gated_dact_kernel<T, 1>;
  return launch(k, grid, dim3(64, 4), 0, 0, 3, 0.0, 10.0 * s.t * s.h, stream, static_cast<const T*>(dh), ldh,
                static_cast<const T*>(gate), static_cast<const T*>(up), ldp_in, static_cast<T*>(dgu), ldp, s.t,
                static_cast<int>(s.h), act);
}

}  // namespace

}  // namespace msb

using namespace msb;

extern "C" {

// ---------------------------------------------------------------- RMS norm

msign_status rms_norm(const void* x, const void* residual, const void* weight, void* y, void* sum_out,
                      msign_dtype io_dtype, msign_dtype w_dtype, int64_t rows, int64_t cols, int64_t x_stride,
                      int64_t r_stride, int64_t y_stride, int64_t s_stride, float eps, msign_stream_t stream) {
  return norm_call(x, residual, weight, y, sum_out, nullptr, io_dtype, w_dtype, rows, cols, x_stride, r_stride,
                   y_stride, s_stride, eps, stream);
}

msign_status rms_norm_q8(const void* x, const void* residual, const void* weight, int8_t* q, float* scale,
                         void* sum_out, msign_dtype io_dtype, msign_dtype w_dtype, int64_t rows, int64_t cols,
                         int64_t x_stride, int64_t r_stride, int64_t q_stride, int64_t s_stride, float eps,
                         msign_stream_t stream) {
  if (rows > 0 && scale == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (rows > 0 && cols == 0) {
    if (rows > kMaxDim) return MSIGN_ERR_UNSUPPORTED;
    return cudaMemsetAsync(scale, 0, sizeof(float) * static_cast<size_t>(rows), reinterpret_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? MSIGN_OK
               : MSIGN_ERR_CUDA;
  }
  return norm_call(x, residual, weight, q, sum_out, scale, io_dtype, w_dtype, rows, cols, x_stride, r_stride, q_stride,
                   s_stride, eps, stream);
}

size_t rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  Carver cv(nullptr);
  cv.take(sizeof(float) * std::min<int64_t>(rows, kDwParts) * cols);
  cv.take(sizeof(float) * rows);
  return cv.off + 1024;
}

msign_status rms_norm_backward(const void* dy, const void* sum, const void* weight, const void* dsum, void* dx,
                               void* dw, msign_dtype io_dtype, msign_dtype w_dtype, int64_t rows, int64_t cols,
                               int64_t dy_stride, int64_t sum_stride, int64_t dsum_stride, int64_t dx_stride, float eps,
                               void* workspace, size_t workspace_bytes, msign_stream_t stream) {
  if (!valid_dtype(io_dtype) || !valid_dtype(w_dtype)) return MSIGN_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return MSIGN_ERR_INVALID_ARG;
  if (!valid_stride(dy_stride, cols) || !valid_stride(sum_stride, cols) || !valid_stride(dsum_stride, cols) ||
      !valid_stride(dx_stride, cols))
    return MSIGN_ERR_INVALID_ARG;
  if ((weight != nullptr || dw != nullptr) && w_dtype != io_dtype && w_dtype != MSIGN_FP32)
    return MSIGN_ERR_UNSUPPORTED;
  if (cols == 0) return MSIGN_OK;
  if (rows > kMaxDim || cols > kMaxDim) return MSIGN_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int dt = to_dt(io_dtype), es = dtype_size(dt);
  const int wdt = to_dt(w_dtype);
  if (rows == 0) return zero_rows(dw, cols, 1, cols, dtype_size(wdt), s);  // a sum over no rows
  if (dy == nullptr || sum == nullptr || dx == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (!on_elements({dy, sum, dsum, dx}, es) || !on_elements({weight, dw}, dtype_size(wdt))) return MSIGN_ERR_INVALID_ARG;
  if (is_one_of(dx, {dy, sum, weight, dsum, dw}) || is_one_of(dw, {dy, sum, weight, dsum})) return MSIGN_ERR_INVALID_ARG;
  if (dw != nullptr && !workspace_ok(workspace, workspace_bytes, rms_norm_backward_workspace_size(rows, cols)))
    return MSIGN_ERR_WORKSPACE;
  if (dw != nullptr && is_one_of(workspace, {dy, sum, weight, dsum, dx, dw})) return MSIGN_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  msign_status st = layer_state(&dev);
  if (st != MSIGN_OK) return st;
  NormBwdArgs a = {};
  a.dy = dy, a.z = sum, a.w = weight, a.ds = dsum, a.dz = dx;
  a.dys = stride_of(dy_stride, cols), a.zs = stride_of(sum_stride, cols);
  a.dss = stride_of(dsum_stride, cols), a.dzs = stride_of(dx_stride, cols);
  a.rows = rows, a.cols = static_cast<int>(cols), a.w_f32 = w_dtype == MSIGN_FP32, a.eps = eps;
  a.err = dev->err, a.timeout_ns = kWaitLimitNs;
  const NormReach by = norm_reach({{sum, a.zs, es}, {dy, a.dys, es}, {dsum, a.dss, es}, {dx, a.dzs, es}}, weight,
                                  a.w_f32, es, rows, cols);
  const double bytes = static_cast<double>(rows) * cols * es * (3 + (dsum != nullptr));
  char* ws = dw != nullptr ? carve_base(workspace) : nullptr;
  if (dt == DT_BF16) return norm_bwd_run<__nv_bfloat16>(a, dw, wdt, by, ws, bytes, s);
  if (dt == DT_FP16) return norm_bwd_run<__half>(a, dw, wdt, by, ws, bytes, s);
  return norm_bwd_run<float>(a, dw, wdt, by, ws, bytes, s);
}

// ---------------------------------------------------------------- int8 product

size_t i8_matmul_workspace_size(int64_t m, int64_t n, int64_t k, const int8_t* a, int64_t a_stride, const int8_t* b,
                                int64_t b_stride) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  Carver cv(nullptr);
  void* c;
  carve_operand(cv, Operand{a, m, k, stride_of(a_stride, k), 1}, &c);
  carve_operand(cv, Operand{b, n, k, stride_of(b_stride, k), 1}, &c);
  return carved(cv);
}

msign_status i8_matmul(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, void* out,
                       msign_dtype out_dtype, int64_t m, int64_t n, int64_t k, int64_t a_stride, int64_t b_stride,
                       int64_t out_stride, void* workspace, size_t workspace_bytes, msign_stream_t stream_) {
  if (!valid_dtype(out_dtype) || m < 0 || n < 0 || k < 0) return MSIGN_ERR_INVALID_ARG;
  if (!valid_stride(a_stride, k) || !valid_stride(b_stride, k) || !valid_stride(out_stride, n))
    return MSIGN_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return MSIGN_OK;
  if (out == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (m > kMaxDim || n > kMaxDim || k > kMaxI8K || !countable(m, n)) return MSIGN_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int odt = to_dt(out_dtype), oes = dtype_size(odt);
  const int64_t ldo = stride_of(out_stride, n);
  if (k == 0) return zero_rows(out, ldo, m, n, oes, stream);
  if (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (!on_elements({a_scale, b_scale}, 4) || !on_elements({out}, oes)) return MSIGN_ERR_INVALID_ARG;
  const size_t need = i8_matmul_workspace_size(m, n, k, a, a_stride, b, b_stride);
  if (!workspace_ok(workspace, workspace_bytes, need)) return MSIGN_ERR_WORKSPACE;
  if (is_one_of(out, {a, b, a_scale, b_scale}) || (need > 0 && is_one_of(workspace, {a, b, a_scale, b_scale, out})))
    return MSIGN_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  msign_status st = layer_state(&dev);
  if (st != MSIGN_OK) return st;
  Operand oa{a, m, k, stride_of(a_stride, k), 1}, ob{b, n, k, stride_of(b_stride, k), 1};
  {
    Carver cv(carve_base(workspace));
    void *ca, *cb;
    carve_operand(cv, oa, &ca);
    carve_operand(cv, ob, &cb);
    if ((st = place_operands({&oa, &ob}, {ca, cb}, stream)) != MSIGN_OK) return st;
  }
  const double flops = 2.0 * m * n * k;
  const double bytes = static_cast<double>(m) * k + static_cast<double>(n) * k + static_cast<double>(oes) * m * n;
  const CUtensorMapDataType type = tma_type(0, true);
  if (stream_takes<PAIR_I8>(m, n, 1)) {
    StreamParams p;
    std::memset(&p, 0, sizeof(p));
    p.tokens = static_cast<int>(m), p.N = static_cast<int>(n), p.nk = static_cast<int>(ceil_div(k, 128)), p.segs = 1;
    const StreamPlan plan = stream_plan<PAIR_I8>(m, n, 1, p.nk);
    if (!map_rows(&p.tmW[0], ob.p, type, 1, n, k, ob.ld, 128, 128) ||
        !map_rows(&p.tmX, oa.p, type, 1, m, k, oa.ld, 128, plan.bn))
      return MSIGN_ERR_CUDA;
    stream_outputs(&p, 1, &out, &ldo, odt);
    p.sx = a_scale, p.sw = b_scale;
    p.idesc = make_idesc(0, true, false, false, plan.bn, 128);
    return stream_launch<PAIR_I8>(&p, plan, 1, flops, bytes, dev, stream);
  }
  PairParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = static_cast<int>(m), p.N = static_cast<int>(n), p.nk = static_cast<int>(ceil_div(k, 128)), p.segs = 1;
  if (!map_rows(&p.tmA, oa.p, type, 1, m, k, oa.ld, 128, 128) ||
      !map_rows(&p.tmB[0], ob.p, type, 1, n, k, ob.ld, 128, 128))
    return MSIGN_ERR_CUDA;
  p.tmB[1] = p.tmB[0];
  void* outs[1] = {out};
  if (!pair_outputs(&p, 1, outs, &ldo, odt)) return MSIGN_ERR_CUDA;
  p.sa = a_scale, p.sb = b_scale;
  p.idesc = make_idesc(0, true, false, false, kBN, kBM);
  return pair_launch<PAIR_I8>(&p, 1, flops, bytes, dev, stream);
}

// ---------------------------------------------------------------- gated feed-forward

size_t gated_ffn_workspace_size(int64_t tokens, int64_t d, int64_t h, const void* x, int64_t x_stride,
                                const void* w_gate, const void* w_up, int64_t w_stride) {
  if (tokens <= 0 || d <= 0 || h <= 0) return 0;
  const int64_t ldw = stride_of(w_stride, d);
  Carver cv(nullptr);
  FfnCopies c;
  carve_ffn(cv, {tokens, d, h}, Operand{x, tokens, d, stride_of(x_stride, d), 2}, Operand{w_gate, h, d, ldw, 2},
            Operand{w_up, h, d, ldw, 2}, false, &c);
  return carved(cv);
}

msign_status gated_ffn(const void* x, const void* w_gate, const void* w_up, void* out, void* gate_out, void* up_out,
                       msign_dtype dtype, msign_activation activation, int64_t tokens, int64_t d, int64_t h,
                       int64_t x_stride, int64_t w_stride, int64_t out_stride, int64_t pre_stride, void* workspace,
                       size_t workspace_bytes, msign_stream_t stream_) {
  const FfnShape s{tokens, d, h};
  const int act = static_cast<int>(activation);
  msign_status st = ffn_check(dtype, act, s, x_stride, w_stride);
  if (st != MSIGN_OK) return st;
  if (!valid_stride(out_stride, h) || !valid_stride(pre_stride, h)) return MSIGN_ERR_INVALID_ARG;
  if ((gate_out == nullptr) != (up_out == nullptr)) return MSIGN_ERR_INVALID_ARG;
  if (tokens == 0 || h == 0) return MSIGN_OK;
  if (out == nullptr) return MSIGN_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int64_t ldh = stride_of(out_stride, h), ldp = stride_of(pre_stride, h), ldw = stride_of(w_stride, d);
  void* outs[3] = {out, gate_out, up_out};
  const int64_t lds[3] = {ldh, ldp, ldp};
  if (d == 0) {  // both projections are empty sums: gate = up = 0, h = act(0) 0
    for (int o = 0; o < 3; ++o)
      if ((st = zero_rows(outs[o], lds[o], tokens, h, 2, stream)) != MSIGN_OK) return st;
    return MSIGN_OK;
  }
  if (x == nullptr || w_gate == nullptr || w_up == nullptr) return MSIGN_ERR_INVALID_ARG;
  if (!on_elements({x, w_gate, w_up, out, gate_out, up_out}, 2)) return MSIGN_ERR_INVALID_ARG;
  if (is_one_of(out, {x, w_gate, w_up, gate_out, up_out}) || is_one_of(gate_out, {x, w_gate, w_up, up_out}) ||
      is_one_of(up_out, {x, w_gate, w_up}))
    return MSIGN_ERR_INVALID_ARG;
  const size_t need = gated_ffn_workspace_size(tokens, d, h, x, x_stride, w_gate, w_up, w_stride);
  if (!workspace_ok(workspace, workspace_bytes, need)) return MSIGN_ERR_WORKSPACE;
  if (need > 0 && is_one_of(workspace, {x, w_gate, w_up, out, gate_out, up_out})) return MSIGN_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  if ((st = layer_state(&dev)) != MSIGN_OK) return st;
  Operand ox{x, tokens, d, stride_of(x_stride, d), 2}, og{w_gate, h, d, ldw, 2}, ou{w_up, h, d, ldw, 2};
  {
    Carver cv(carve_base(workspace));
    FfnCopies c;
    carve_ffn(cv, s, ox, og, ou, false, &c);
    if ((st = place_operands({&ox, &og, &ou}, {c.x, c.wg, c.wu}, stream)) != MSIGN_OK) return st;
  }
  const int dt = to_dt(dtype);
  const CUtensorMapDataType type = tma_type(dt, false);
  const double flops = 4.0 * tokens * d * h;
  const double bytes = 2.0 * (static_cast<double>(tokens) * d + 2.0 * h * d + (gate_out ? 3.0 : 1.0) * tokens * h);
  if (stream_takes<PAIR_GATED>(tokens, h, 1)) {
    StreamParams p;
    std::memset(&p, 0, sizeof(p));
    p.tokens = static_cast<int>(tokens), p.N = static_cast<int>(h), p.nk = static_cast<int>(ceil_div(d, 64)), p.segs = 1;
    const StreamPlan plan = stream_plan<PAIR_GATED>(tokens, h, 1, p.nk);
    if (!map_rows(&p.tmW[0], og.p, type, 2, h, d, og.ld, 64, 64) ||
        !map_rows(&p.tmW[1], ou.p, type, 2, h, d, ou.ld, 64, 64) ||
        !map_rows(&p.tmX, ox.p, type, 2, tokens, d, ox.ld, 64, plan.bn))
      return MSIGN_ERR_CUDA;
    stream_outputs(&p, 3, outs, lds, dt);
    p.act = act;
    p.idesc = make_idesc(dt, false, false, false, plan.bn, 128);
    return stream_launch<PAIR_GATED>(&p, plan, 1, flops, bytes, dev, stream);
  }
  PairParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = static_cast<int>(tokens), p.N = static_cast<int>(h), p.nk = static_cast<int>(ceil_div(d, 64)), p.segs = 1;
  if (!map_rows(&p.tmA, ox.p, type, 2, tokens, d, ox.ld, 64, 128) ||
      !map_rows(&p.tmB[0], og.p, type, 2, h, d, og.ld, 64, 128) ||
      !map_rows(&p.tmB[1], ou.p, type, 2, h, d, ou.ld, 64, 128) || !pair_outputs(&p, 3, outs, lds, dt))
    return MSIGN_ERR_CUDA;
  p.act = act;
  p.idesc = make_idesc(dt, false, false, false, kBN, kBM);
  return pair_launch<PAIR_GATED>(&p, 1, flops, bytes, dev, stream);
}

size_t gated_ffn_backward_workspace_size(int64_t tokens, int64_t d, int64_t h, const void* x, int64_t x_stride,
                                         const void* w_gate, const void* w_up, int64_t w_stride) {
  if (tokens <= 0 || d <= 0 || h <= 0) return 0;
  const int64_t ldw = stride_of(w_stride, d);
  Carver cv(nullptr);
  FfnCopies c;
  carve_ffn(cv, {tokens, d, h}, Operand{x, tokens, d, stride_of(x_stride, d), 2}, Operand{w_gate, h, d, ldw, 2},
            Operand{w_up, h, d, ldw, 2}, true, &c);
  return carved(cv);
}

msign_status gated_ffn_backward(const void* dh, const void* x, const void* w_gate, const void* w_up, const void* gate,
                                const void* up, void* dx, void* dw_gate, void* dw_up, msign_dtype dtype,
                                msign_dtype grad_dtype, msign_activation activation, int64_t tokens, int64_t d,
                                int64_t h, int64_t dh_stride, int64_t x_stride, int64_t w_stride, int64_t pre_stride,
                                int64_t dx_stride, int64_t dw_stride, void* workspace, size_t workspace_bytes,
                                msign_stream_t stream_) {
  const FfnShape s{tokens, d, h};
  const int act = static_cast<int>(activation);
  msign_status st = ffn_check(dtype, act, s, x_stride, w_stride);
  if (st != MSIGN_OK) return st;
  if (!valid_dtype(grad_dtype) || !valid_stride(dh_stride, h) || !valid_stride(pre_stride, h) ||
      !valid_stride(dx_stride, d) || !valid_stride(dw_stride, d))
    return MSIGN_ERR_INVALID_ARG;
  if (grad_dtype != dtype && grad_dtype != MSIGN_FP32) return MSIGN_ERR_UNSUPPORTED;
  if ((dw_gate == nullptr) != (dw_up == nullptr) || (dx == nullptr && dw_gate == nullptr))
    return MSIGN_ERR_INVALID_ARG;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int dt = to_dt(dtype), gdt = to_dt(grad_dtype);
  const int64_t ldw = stride_of(w_stride, d), ldx = stride_of(x_stride, d), ldh = stride_of(dh_stride, h);
  const int64_t lddx = stride_of(dx_stride, d), lddw = stride_of(dw_stride, d), ldpre = stride_of(pre_stride, h);
  if (d == 0) return MSIGN_OK;
  if (tokens == 0 || h == 0) {  // empty sums
    if ((st = zero_rows(dx, lddx, tokens, d, 2, stream)) != MSIGN_OK) return st;
    if ((st = zero_rows(dw_gate, lddw, h, d, dtype_size(gdt), stream)) != MSIGN_OK) return st;
    return zero_rows(dw_up, lddw, h, d, dtype_size(gdt), stream);
  }
  if (dh == nullptr || x == nullptr || w_gate == nullptr || w_up == nullptr || gate == nullptr || up == nullptr)
    return MSIGN_ERR_INVALID_ARG;
  if (!on_elements({dh, x, w_gate, w_up, gate, up, dx}, 2) || !on_elements({dw_gate, dw_up}, dtype_size(gdt)))
    return MSIGN_ERR_INVALID_ARG;
  if (is_one_of(dx, {dh, x, w_gate, w_up, gate, up, dw_gate, dw_up}) ||
      is_one_of(dw_gate, {dh, x, w_gate, w_up, gate, up, dw_up}) || is_one_of(dw_up, {dh, x, w_gate, w_up, gate, up}))
    return MSIGN_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes,
                    gated_ffn_backward_workspace_size(tokens, d, h, x, x_stride, w_gate, w_up, w_stride)))
    return MSIGN_ERR_WORKSPACE;
  if (is_one_of(workspace, {dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up})) return MSIGN_ERR_INVALID_ARG;
  DeviceState* dev = nullptr;
  if ((st = layer_state(&dev)) != MSIGN_OK) return st;
  Operand ox{x, tokens, d, ldx, 2}, og{w_gate, h, d, ldw, 2}, ou{w_up, h, d, ldw, 2};
  Carver cv(carve_base(workspace));
  FfnCopies c;
  carve_ffn(cv, s, ox, og, ou, true, &c);
  // (x feeds the weights' gradients only, the weights feed dx only)
  st = place_operands({&ox, &og, &ou}, {dw_gate != nullptr ? c.x : nullptr, dx != nullptr ? c.wg : nullptr,
                                        dx != nullptr ? c.wu : nullptr}, stream);
  if (st != MSIGN_OK) return st;
  st = dt == DT_BF16 ? dact_run<__nv_bfloat16>(dh, ldh, gate, up, ldpre, c.dgu, s, act, stream)
                     : dact_run<__half>(dh, ldh, gate, up, ldpre, c.dgu, s, act, stream);
  if (st != MSIGN_OK) return st;
  const CUtensorMapDataType type = tma_type(dt, false);
  const int64_t hp = pitch_of(h, 2);
  const double flops = 4.0 * tokens * d * h;
  if (dx != nullptr) {
    const double bytes = 2.0 * (2.0 * tokens * h + 2.0 * h * d + static_cast<double>(tokens) * d);
    const int nk = static_cast<int>(ceil_div(h, 64));
    if (stream_takes<PAIR_DX>(tokens, d, 1)) {
      StreamParams p;
      std::memset(&p, 0, sizeof(p));
      p.tokens = static_cast<int>(tokens), p.N = static_cast<int>(d), p.nk = nk, p.segs = 2;
      const StreamPlan plan = stream_plan<PAIR_DX>(tokens, d, 1, 2 * static_cast<int64_t>(nk));
      if (!map_rows(&p.tmW[0], og.p, type, 2, h, d, og.ld, 64, 64) ||
          !map_rows(&p.tmW[1], ou.p, type, 2, h, d, ou.ld, 64, 64) ||
          !map_rows(&p.tmX, c.dgu, type, 2, tokens, h, hp, 64, plan.bn, 2, tokens * hp))
        return MSIGN_ERR_CUDA;
      stream_outputs(&p, 1, &dx, &lddx, dt);
      p.idesc = make_idesc(dt, false, true, false, plan.bn, 128);
      st = stream_launch<PAIR_DX>(&p, plan, 1, flops, bytes, dev, stream);
    } else {
      PairParams p;
      std::memset(&p, 0, sizeof(p));
      p.M = static_cast<int>(tokens), p.N = static_cast<int>(d), p.nk = nk, p.segs = 2;
      if (!map_rows(&p.tmA, c.dgu, type, 2, tokens, h, hp, 64, 128, 2, tokens * hp) ||
          !map_rows(&p.tmB[0], og.p, type, 2, h, d, og.ld, 64, 64) ||
          !map_rows(&p.tmB[1], ou.p, type, 2, h, d, ou.ld, 64, 64) || !pair_outputs(&p, 1, &dx, &lddx, dt))
        return MSIGN_ERR_CUDA;
      p.idesc = make_idesc(dt, false, false, true, kBN, kBM);
      st = pair_launch<PAIR_DX>(&p, 1, flops, bytes, dev, stream);
    }
    if (st != MSIGN_OK) return st;
  }
  if (dw_gate != nullptr) {
    const double bytes = 2.0 * (2.0 * tokens * h + static_cast<double>(tokens) * d) + 2.0 * dtype_size(gdt) * h * d;
    const int nk = static_cast<int>(ceil_div(tokens, 64));
    void* outs[2] = {dw_gate, dw_up};
    const int64_t lds[2] = {lddw, lddw};
    if (ceil_div(h, kBM) * ceil_div(d, kBN) * 2 < 48 && nk >= 32) {
      StreamParams p;
      std::memset(&p, 0, sizeof(p));
      p.tokens = static_cast<int>(h), p.N = static_cast<int>(d), p.nk = nk, p.segs = 1;
      const StreamPlan plan = stream_plan<PAIR_DW>(h, d, 2, nk);
      if (!map_rows(&p.tmW[0], ox.p, type, 2, tokens, d, ox.ld, 64, 64) ||
          !map_rows(&p.tmX, c.dgu, type, 2, tokens, h, hp, 64, 64, 2, tokens * hp))
        return MSIGN_ERR_CUDA;
      stream_outputs(&p, 2, outs, lds, gdt);
      p.idesc = make_idesc(dt, false, true, true, plan.bn, 128);
      st = stream_launch<PAIR_DW>(&p, plan, 2, flops, bytes, dev, stream);
    } else {
      PairParams p;
      std::memset(&p, 0, sizeof(p));
      p.M = static_cast<int>(h), p.N = static_cast<int>(d), p.nk = nk, p.segs = 1;
      if (!map_rows(&p.tmA, c.dgu, type, 2, tokens, h, hp, 64, 64, 2, tokens * hp) ||
          !map_rows(&p.tmB[0], ox.p, type, 2, tokens, d, ox.ld, 64, 64) || !pair_outputs(&p, 2, outs, lds, gdt))
        return MSIGN_ERR_CUDA;
      p.tmB[1] = p.tmB[0];
      p.idesc = make_idesc(dt, false, true, true, kBN, kBM);
      st = pair_launch<PAIR_DW>(&p, 2, flops, bytes, dev, stream);
    }
    if (st != MSIGN_OK) return st;
  }
  return MSIGN_OK;
}

}  // extern "C"
