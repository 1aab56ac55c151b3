// norm_plan.h - how the RMS norms' launches are laid out: which form takes
// rows of a width and how many threads, rows and ring slots a block has.
// Whole numbers only and no CUDA, so that a host program can ask for the plan
// of any width; 64 bits throughout, since a row may have 2^30 columns (4 GB).
#pragma once

#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define MSB_HOST_DEVICE __host__ __device__
#else
#define MSB_HOST_DEVICE
#endif

namespace msb {

constexpr int kPlanSms = 148;  // launch plans must not depend on the device: workspace sizes are host-only queries

constexpr int kNormMaxThreads = 1024;
constexpr int kNormVpt = 4;     // 16-byte pieces of a row that one thread holds at most
constexpr int kNormElems = 8;   // accesses of a thread in the *_elem kernels
constexpr int kNormBwdVpt = 4;  // pieces of a row that a thread of the gradients' kernel holds at most
// Largest block of the gradients' kernel, by the pieces of a row that a thread
// holds.
MSB_HOST_DEVICE constexpr int norm_bwd_threads(int vpt) { return vpt <= 2 ? 256 : 512; }
constexpr int kNormBwdElemThreads = 512;
constexpr int kNormRing = 8;  // ring slots of the gradients' kernel at most

// Partial rows of dw that the gradients leave at most: four blocks an SM.
constexpr int64_t kDwParts = 4 * kPlanSms;
constexpr int64_t kDwLoopParts = 128;  // row chunks of the loop form for rows whose sums shared memory does not hold
constexpr int64_t kLoopSums = 12000;   // columns whose sums it does (48 KB without a raised limit)
constexpr int kSmemMax = 232448;       // shared memory of a block
constexpr int kNormRingMax = kSmemMax - 2048;  // (the gradients' kernel has some static shared memory too)

// A row in 16-byte pieces, in bytes: with `shift` as it lies about its 16-byte
// boundaries.  On the host I is 64 bits wide (2^30 columns do not fit 32); a
// kernel that holds a row in pieces has one of a few KB.
template <typename I>
MSB_HOST_DEVICE inline I norm_row_bytes(I cols, I es, bool shift) {
  return shift ? (cols * es + I(31) - es) / I(16) * I(16) : cols * es;
}

// How the norms' kernels reach the rows: by 16 bytes; by 16 bytes about the
// boundaries that the rows are off (NORM_SHIFT's condition: one phase, and rows
// of at least 32 pieces: gradients of 8192 x 151 bf16 13 us either way, 301 21
// and 19, 1002 46 and 29); by `pair` elements.
struct NormReach {
  bool vec, shift;
  int pair;
};

enum class NormForm {
  kPieces,    // 16-byte pieces in registers (gradients: through the ring)
  kElems,     // elements in registers
  kLoop,      // any width, read again for each pass
  kLoopSums,  // gradients: the loop form with the sums of dw in shared memory
};

struct NormPlan {
  NormForm form = NormForm::kLoop;
  int vpt = 0;         // pieces a thread
  int x = 256, y = 1;  // threads of a row, rows of a block
};

inline int norm_threads(int64_t pieces, int vpt) { return static_cast<int>(((pieces + vpt - 1) / vpt + 31) / 32 * 32); }

// Threads of the *_elem kernels: a warp a row where that holds it, four rows a
// block; else a block a row.
inline NormPlan norm_elems(int64_t cols, int pair) {
  NormPlan p;
  p.form = NormForm::kElems;
  p.x = norm_threads(cols, pair * kNormElems);
  p.y = p.x == 32 ? 4 : 1;
  return p;
}

// Rows of `cols` elements of `es` bytes.  Up to 128 pieces a warp takes a row
// (no block barrier) and a block four, beyond that a block takes one.
inline NormPlan norm_plan(int64_t cols, int es, const NormReach& by) {
  const int64_t pieces = norm_row_bytes<int64_t>(cols, es, by.shift) / 16;
  if ((by.vec || by.shift) && pieces <= int64_t(kNormMaxThreads) * kNormVpt) {
    NormPlan p;
    p.form = NormForm::kPieces;
    if (pieces <= 32 * kNormVpt) {
      p.vpt = pieces <= 32 ? 1 : pieces <= 64 ? 2 : 4;
      p.x = 32, p.y = 4;
    } else {
      p.vpt = pieces <= 2 * kNormMaxThreads ? 2 : kNormVpt;
      p.x = norm_threads(pieces, p.vpt);
    }
    return p;
  }
  // Measured, the row in registers against the loop form, 8192 rows with a
  // residual: two elements an access, bf16, 1002 columns 23 and 31 us, 4098 93
  // and 109; fp32 4586 107 and 124; one element, bf16, 101 columns 6.7 and
  // 14.1, 2001 63 and 65, 4099 135 and 116.
  if (cols <= int64_t(by.pair) * kNormElems * kNormMaxThreads && (by.pair == 2 || es == 4 || cols <= 2048))
    return norm_elems(cols, by.pair);
  return {};
}

struct NormBwdPlan {
  NormPlan p;
  bool full = false;  // kPieces: no thread is ever idle
  int slot = 0;       // kPieces: bytes of a ring slot
  int stages = 0;     // kPieces: ring slots
  int64_t parts = 0;  // partial rows of dw
};

inline NormBwdPlan norm_bwd_plan(int64_t rows, int64_t cols, int es, const NormReach& by, bool ds, bool dw) {
  NormBwdPlan b;
  const int64_t pieces = norm_row_bytes<int64_t>(cols, es, by.shift) / 16;
  if ((by.vec || by.shift) && pieces <= norm_bwd_threads(kNormBwdVpt) * kNormBwdVpt) {
    // one or two pieces a thread as far as 256 threads a row hold it, then four
    // (up to 512 threads: 2048 x 16001 bf16 74 us, eight pieces 81; 4096 x 4700
    // fp32 51 and 66; 8192 x 10240 bf16 129 and 123), the block filled up with
    // rows, and the ring as deep as the SM's blocks leave room for
    int vpt = pieces <= 32 ? 1 : 2;
    if (pieces > vpt * norm_bwd_threads(vpt)) vpt = kNormBwdVpt;
    const int x = norm_threads(pieces, vpt), y = std::max(1, 256 / x);
    b.p.form = NormForm::kPieces, b.p.vpt = vpt, b.p.x = x, b.p.y = y;
    b.full = by.vec && pieces == int64_t(x) * vpt && rows % y == 0;
    // by the kernel's registers (80 a thread; with four pieces 128, fp32 with idle threads 112)
    int per_sm = std::min(4, (vpt <= 2 ? 768 : es == 4 && !b.full ? 576 : 512) / (x * y));
    b.slot = (ds ? 3 : 2) * y * static_cast<int>(pieces * 16);
    // (an SM has 228 KB; each block 1 KB of its own and what the kernel declares)
    const auto depth = [&] { return std::min(kNormRing, std::min(kNormRingMax, 228 * 1024 / per_sm - 1536) / b.slot); };
    b.stages = depth();
    while (b.stages < 2) --per_sm, b.stages = depth();
    b.parts = std::min<int64_t>({(rows + y - 1) / y, int64_t(kPlanSms) * per_sm, kDwParts});  // what the workspace holds
    // a thread's rows have one phase: the rows from turn to turn are a multiple of a piece's elements apart
    const int64_t period = std::max(1, 16 / es / y);
    if (by.shift && b.parts * y < rows) b.parts = b.parts / period * period;
    return b;
  }
  // few rows: one launch less (777 x 1001 fp32, phases apart: 20 us a call
  // with the host's part, 17 so; 16384 x 1001 129 us, and 93 with the sums of
  // dw apart)
  if (dw && cols <= kLoopSums && rows <= 2 * kDwParts) {
    b.p.form = NormForm::kLoopSums;
    b.parts = std::min<int64_t>(rows, kDwParts);
    return b;
  }
  // the row in registers (8192 x 1002 bf16 46 us, by the loop 76; 4098 175
  // and 249)
  if (cols <= int64_t(by.pair) * kNormElems * kNormBwdElemThreads) b.p = norm_elems(cols, by.pair);
  return b;  // (the sums of dw by a launch of their own)
}

}  // namespace msb
