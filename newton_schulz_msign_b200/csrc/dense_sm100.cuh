// dense_sm100.cuh - tcgen05 products of a transformer layer: the gated
// feed-forward block, its gradients, and the int8 product with scales.
//
// Two kernels:
//
//   dense_pair_kernel    many rows.  Persistent CTA pairs, one 256 x 256
//                        accumulator tile a pair (tcgen05.mma.cta_group::2),
//                        two tiles in TMEM so that one is stored while the
//                        next is formed, a ring of TMA-fed operand stages.
//   dense_stream_kernel  few rows (a decoding step), and whatever has too
//                        few 256 x 256 tiles to fill the GPU.  The weights
//                        are the M operand and stream through once; the
//                        tokens are the N operand, as narrow as they are.  A
//                        cluster of CTAs splits K and joins its parts
//                        through distributed shared memory.
//
// A stage holds 128 bytes of K for every operand row whatever the type (64
// 16-bit elements or 128 int8), so the 16-bit and the int8 forms share the
// geometry: four MMAs of 32 bytes of K a stage.
//
// Measured (B200): the pair kernel forms the gated block at 4096 tokens x 4096
// x 14336 in 604 us with gate and up kept (1.59 PFLOP/s; 730 sustained under
// the power cap), int8 8192 x 14336 x 4096 in 291 us (3.3 POP/s; 346
// sustained); both keep the tensor pipe over 80% busy.  The stream kernel
// takes 39.6 us for 4 tokens through the same block (235 MB of weights, 5.9
// TB/s) and 12.9 for one token through an int8 14336 x 4096 (59 MB).
//
// No load uses cluster multicast: each CTA fetches its own operands.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gemm_sm100.cuh"
#include "norm_sm100.cuh"
#include "ptx_sm100.cuh"

namespace msb {

// int8 x int8 -> int32, K = 32 a MMA; pair and single-CTA forms, issued by
// one elected lane of a converged warp.
__device__ __forceinline__ void umma_i8_pair_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void umma_i8_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void umma_f16_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

__device__ __forceinline__ void umma_commit_w(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)));
}

__device__ __forceinline__ void tma_load_3d_w(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)));
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ---------------------------------------------------------------- activations

enum : int { ACT_SILU = 0, ACT_GELU = 1, ACT_GELU_TANH = 2 };

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 2^x and 1 / x to a few steps of fp32, subnormal results flushed to 0.
__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// g sigmoid(v) = (g / 4) / (1/4 + 2^(-v log2 e - 2)).  The quarters keep the
// divisor's reciprocal a normal number for as long as exp(-v) is finite (1 +
// exp(-v) reaches 2^128, and the reciprocal of anything past 2^126 flushes:
// silu from -87.3 to -88.7 is still 1e-36); past that the product is 0, as it
// should be.  A power of two that flushes is nothing beside the 1/4.
__device__ __forceinline__ float g_sigmoid(float g, float v) {
  return 0.25f * g * rcp_ftz(0.25f + ex2_ftz(fmaf(v, -1.4426950408889634f, -2.0f)));
}

template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if (ACT == ACT_SILU) return g_sigmoid(g, g);
  if (ACT == ACT_GELU) return g * (0.5f * erfcf(-0.70710678118654752f * g));  // (1 + erf would lose the tail's digits)
  // (1 + tanh z) / 2 = sigmoid(2 z)
  return g_sigmoid(g, 2.0f * kGeluC * fmaf(kGeluA * g * g, g, g));
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ float2 act_grad(float g) {
  if (ACT == ACT_SILU) {
    const float p = g_sigmoid(1.0f, g);
    return make_float2(g * p, p * fmaf(g, 1.0f - p, 1.0f));
  }
  if (ACT == ACT_GELU) {
    const float c = 0.5f * erfcf(-0.70710678118654752f * g);
    return make_float2(g * c, fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), c));
  }
  // past |g| = 30 p is 0 or 1 to the last bit: the clamp only keeps the cube finite (and keeps a NaN)
  const float c = fabsf(g) > 30.0f ? copysignf(30.0f, g) : g;
  const float p = g_sigmoid(1.0f, 2.0f * kGeluC * fmaf(kGeluA * c * c, c, c));
  return make_float2(g * p, fmaf(2.0f * p * (1.0f - p), kGeluC * fmaf(3.0f * kGeluA * c * c, c, c), p));
}

// u_i <- act(g_i) u_i.  The choice stands outside the loops: inside, every
// unrolled element carried all three activations, and the gated epilogue
// spent its time on fetching code (10100 cycles a tile against 4000).
template <int ACT, int N>
__device__ __forceinline__ void gate_mul_as(const float (&g)[N], float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) u[i] *= act_of<ACT>(g[i]);
}

template <int N>
__device__ __forceinline__ void gate_mul(const float (&g)[N], float (&u)[N], int act) {
  if (act == ACT_SILU)
    gate_mul_as<ACT_SILU>(g, u);
  else if (act == ACT_GELU)
    gate_mul_as<ACT_GELU>(g, u);
  else
    gate_mul_as<ACT_GELU_TANH>(g, u);
}

// From d = dh, g and u: g <- dh u act'(g), d <- dh act(g).
template <int ACT, int N>
__device__ __forceinline__ void gate_grad_as(float (&d)[N], float (&g)[N], const float (&u)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 a = act_grad<ACT>(g[i]);
    g[i] = d[i] * u[i] * a.y;
    d[i] = d[i] * a.x;
  }
}

template <int N>
__device__ __forceinline__ void gate_grad(float (&d)[N], float (&g)[N], const float (&u)[N], int act) {
  if (act == ACT_SILU)
    gate_grad_as<ACT_SILU>(d, g, u);
  else if (act == ACT_GELU)
    gate_grad_as<ACT_GELU>(d, g, u);
  else
    gate_grad_as<ACT_GELU_TANH>(d, g, u);
}

// ---------------------------------------------------------------- many rows

// What a launch forms (the layout notes are the pair kernel's):
//   PAIR_GATED  h = act(x Wg^T) (x Wu^T): the 256 accumulator columns of a
//               tile are 128 hidden units' gate columns, then the same
//               units' up columns.  In cta_group::2 each CTA stages half of
//               the B rows: the leader stages Wg's, the peer Wu's.
//   PAIR_I8     (a b^T) sa sb
//   PAIR_DX     dg Wg + du Wu: one K loop over both segments; B is read
//               MN-major (the weights as they lie)
//   PAIR_DW     dg^T x and du^T x (z = 0, 1): both operands MN-major
enum : int { PAIR_GATED = 0, PAIR_I8 = 1, PAIR_DX = 2, PAIR_DW = 3 };

constexpr int kPairBoxBytes = 32 * 128;  // an epilogue warp's staging box: 32 rows of 128 bytes

struct PairParams {
  CUtensorMap tmA;     // K-major: (k, row, seg) box 128 bytes x 128; MN-major: (row, k, z) box 64 x 64
  CUtensorMap tmB[2];  // K-major: (k, col) box 128 bytes x 128; MN-major: (col, k) box 64 x 64
  CUtensorMap tmO[3];  // outputs (col, row), box 128 bytes x 32
  void* out[3];        // PAIR_GATED: h, gate, up (the last two may be null); PAIR_DW: dWg, dWu
  long long ldo[3];    // in elements
  const float *sa, *sb;
  int M, N;            // output rows and columns (PAIR_GATED: hidden units)
  int nk, segs;        // K stages a segment, segments
  int tiles_m, tiles_n, total;
  int band;            // tile rows walked together (see pair_tile)
  int odt;             // output type
  int tma_out;         // outputs leave by bulk tensor stores (else lane stores)
  int act;
  uint32_t idesc;
  int* err;
  unsigned long long timeout_ns;
};

struct PairTile {
  int z, tm, tn;
};

// Tiles in bands of `band` tile rows, column by column inside a band: the
// tiles that the pairs work on at once share `band` row blocks of A and a
// few column blocks of B, which stay in L2.
__device__ __forceinline__ PairTile pair_tile(const PairParams& p, int t) {
  const int per = p.tiles_m * p.tiles_n;
  const int z = t / per;
  int r = t - z * per;
  const int g0 = r / (p.band * p.tiles_n) * p.band;
  r -= g0 * p.tiles_n;
  const int gh = min(p.band, p.tiles_m - g0);
  return {z, g0 + r % gh, r / gh};
}

// One staged box of a warp: 32 rows x 128 bytes, 16-byte piece i of row r at
// piece i ^ (r & 7) (the tensor map's 128-byte swizzle; conflict-free when
// each lane writes a piece of its own row).
__device__ __forceinline__ void box_put16(uint8_t* box, int lane, int j, const float (&v)[32], int dt) {
  uint32_t h[16];
  pack16(v, dt, h);
  uint8_t* rowp = box + lane * 128;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(rowp + 16 * ((4 * j + i) ^ (lane & 7))) =
        make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
}

__device__ __forceinline__ void box_put32(uint8_t* box, int lane, const float (&v)[32]) {
  uint8_t* rowp = box + lane * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<float4*>(rowp + 16 * (i ^ (lane & 7))) =
        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// One row of a staged box to global memory, lane l the four bytes at 4 l of
// its 128: 32-bit values, or pairs of 16-bit ones.  A row of 16-bit values
// that starts in the middle of a word goes out shifted by one value.
__device__ __forceinline__ void box_row_out(const uint8_t* box, int r, char* dst, int es, int cols, int lane) {
  const auto word = [&](int l) {
    return *reinterpret_cast<const uint32_t*>(box + r * 128 + 16 * ((l >> 2) ^ (r & 7)) + 4 * (l & 3));
  };
  const uint32_t v = word(lane);
  if (es == 4) {
    if (lane < cols) *reinterpret_cast<uint32_t*>(dst + 4 * lane) = v;
    return;
  }
  if ((reinterpret_cast<uintptr_t>(dst) & 2) == 0) {
    if (2 * lane + 1 < cols)
      *reinterpret_cast<uint32_t*>(dst + 4 * lane) = v;
    else if (2 * lane < cols)
      *reinterpret_cast<uint16_t*>(dst + 4 * lane) = static_cast<uint16_t>(v);
    return;
  }
  const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, v, 1);
  if (lane == 0) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(v);
  if (2 * lane + 2 < cols)
    *reinterpret_cast<uint32_t*>(dst + 4 * lane + 2) = (v >> 16) | (next << 16);
  else if (2 * lane + 1 < cols)
    *reinterpret_cast<uint16_t*>(dst + 4 * lane + 2) = static_cast<uint16_t>(v >> 16);
}

// Sends a staged box to output o at (row0, col0), clipped to M x N.
__device__ __forceinline__ void box_send(const PairParams& p, int o, uint8_t* box, int lane, int row0, int col0) {
  if (p.tma_out) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(&p.tmO[o], box, col0, row0, 0);
      bulk_commit_group();
    }
    return;
  }
  __syncwarp();
  const int es = dtype_size(p.odt);
  const int rows = min(32, p.M - row0), cols = min(128 / es, p.N - col0);
  const long long step = p.ldo[o] * es;
  char* dst = static_cast<char*>(p.out[o]) + row0 * step + static_cast<long long>(col0) * es;
  int r = 0;
  for (; r + 4 <= rows; r += 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) box_row_out(box, r + i, dst + (r + i) * step, es, cols, lane);
  for (; r < rows; ++r) box_row_out(box, r, dst + r * step, es, cols, lane);
}

// The warp's staging box may be written again: its last bulk store has read
// it.  (Two boxes in turn, at the price of a stage: no gain, 1% lost.)
__device__ __forceinline__ void box_free(const PairParams& p, int lane) {
  if (p.tma_out && lane == 0) bulk_wait_read_all();
  __syncwarp();
}

__device__ __forceinline__ void tmem_block(uint32_t taddr, float (&v)[32]) {
  uint32_t raw[32];
  tmem_ld_32x32b_x32(taddr, raw);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(raw[i]);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_pair_kernel(const __grid_constant__ PairParams p) {
  constexpr bool kI8 = MODE == PAIR_I8;
  constexpr bool kAmn = MODE == PAIR_DW;
  constexpr bool kBmn = MODE == PAIR_DX || MODE == PAIR_DW;
  constexpr int kBke = kI8 ? 128 : 64;                    // K elements a stage
  constexpr int kCols = MODE == PAIR_GATED ? 128 : kBN;   // output columns a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kATileBytes;
  uint8_t* sOut = sB + kStages * kBTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOut + kEpiWarps * kPairBoxBytes);
  uint64_t* full = bars;                 // leader: both CTAs' loads of a stage landed
  uint64_t* empty = bars + kStages;      // both: the MMAs reading a stage finished
  uint64_t* tfull = bars + 2 * kStages;  // both: accumulator ready
  uint64_t* tempty = tfull + 2;          // leader: both epilogues drained an accumulator
  uint64_t* drain = tempty + 2;          // leader: every issued MMA finished
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + kNumBarriers);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1;
  const int num_pairs = gridDim.x >> 1;
  const uint64_t limit = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB[0]);
    tma_prefetch_desc(&p.tmB[1]);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers are initialised before either signals the other's
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();
  pdl_trigger();

  const int steps = p.nk * p.segs;
  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs, warp-converged)
    int stage = 0;
    uint32_t phase = 0, used = 0, last_phase = 0;
    bool ok = true;
    const void* tmA = &p.tmA;
    for (int t = pair; ok && t < p.total; t += num_pairs) {
      const PairTile tc = pair_tile(p, t);
      const int arow = tc.tm * kBM + static_cast<int>(rank) * kHalfM;
      const int bcol = MODE == PAIR_GATED ? tc.tn * kCols : tc.tn * kBN + static_cast<int>(rank) * kHalfN;
      int seg = 0, kb = 0;
      for (int step = 0; step < steps; ++step) {
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(&empty[stage], phase ^ 1u, s_abort, p.err, limit))) {
          ok = false;
          break;
        }
        if (leader) mbar_arrive_expect_tx_w(&full[stage], 2u * kStageBytes);
        const uint32_t fbar = mapa_shared(smem_u32(&full[stage]), 0);
        uint8_t* a_dst = sA + stage * kATileBytes;
        uint8_t* b_dst = sB + stage * kBTileBytes;
        const int k0 = kb * kBke;
        const void* tmB = &p.tmB[MODE == PAIR_GATED ? rank : (MODE == PAIR_DX ? seg : 0)];
        if (kAmn) {
          tma_load_3d_pair_w(a_dst, tmA, fbar, arow, k0, tc.z);
          tma_load_3d_pair_w(a_dst + 8192, tmA, fbar, arow + 64, k0, tc.z);
        } else {
          tma_load_3d_pair_w(a_dst, tmA, fbar, k0, arow, seg);
        }
        if (kBmn) {
          tma_load_3d_pair_w(b_dst, tmB, fbar, bcol, k0, 0);
          tma_load_3d_pair_w(b_dst + 8192, tmB, fbar, bcol + 64, k0, 0);
        } else {
          tma_load_3d_pair_w(b_dst, tmB, fbar, k0, bcol, 0);
        }
        used |= 1u << stage;
        last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++kb == p.nk) {
          kb = 0;
          ++seg;
        }
      }
    }
    // never leave with copies still landing (see gemm_sm100.cuh)
    if (leader && lane == 0)
      for (int s = 0; s < kStages; ++s)
        if ((used >> s) & 1u) wait_bounded(&full[s], (last_phase >> s) & 1u, nullptr, p.err, limit);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader, warp-converged)
    if (leader) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      const uint32_t idesc = p.idesc;
      const uint64_t dA = kAmn ? smem_desc_sw128(smem_u32(sA), 8192, 1024) : smem_desc_sw128(smem_u32(sA), 16, 1024);
      const uint64_t dB = kBmn ? smem_desc_sw128(smem_u32(sB), 8192, 1024) : smem_desc_sw128(smem_u32(sB), 16, 1024);
      constexpr uint32_t ka = kAmn ? 2048 >> 4 : 32 >> 4, kb = kBmn ? 2048 >> 4 : 32 >> 4;
      for (int t = pair; t < p.total; t += num_pairs) {
        if (!__all_sync(0xFFFFFFFFu, wait_bounded(&tempty[buf], bphase ^ 1u, s_abort, p.err, limit))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kBN);
        for (int step = 0; step < steps; ++step) {
          if (!__all_sync(0xFFFFFFFFu, wait_bounded(&full[stage], phase, s_abort, p.err, limit))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = dA + static_cast<uint64_t>((stage * kATileBytes) >> 4);
          const uint64_t db = dB + static_cast<uint64_t>((stage * kBTileBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = (step | kk) != 0 ? 1u : 0u;
            if (kI8)
              umma_i8_pair_w(d_tmem, da + kk * ka, db + kk * kb, idesc, acc);
            else
              umma_f16_pair_w(d_tmem, da + kk * ka, db + kk * kb, idesc, acc);
          }
          umma_commit_pair_mc_w(&empty[stage], 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc_w(&tfull[buf], 0x3);
        buf ^= 1;
        if (buf == 0) bphase ^= 1u;
      }
      umma_commit_pair_mc_w(drain, 0x1);  // every MMA issued so far finishes before TMEM is released
      if (lane == 0) wait_bounded(drain, 0, nullptr, p.err, limit);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int q = warp & 3;       // TMEM lane quarter
    const int ew = warp - 2;
    const int half = ew >> 2;     // which half of the tile's columns
    uint8_t* box = sOut + ew * kPairBoxBytes;
    const uint32_t tempty_leader0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const uint32_t tempty_leader1 = mapa_shared(smem_u32(&tempty[1]), 0);
    int buf = 0;
    uint32_t bphase = 0;
    for (int t = pair; t < p.total; t += num_pairs) {
      const PairTile tc = pair_tile(p, t);
      const int row0 = tc.tm * kBM + static_cast<int>(rank) * kHalfM + q * 32;
      const int col0 = tc.tn * kCols + half * (kCols / 2);
      // int8: this lane's row scale, and its columns' scales of the warp's four blocks
      float sa = 0.0f, sb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (kI8) {
        if (row0 + lane < p.M) sa = p.sa[row0 + lane];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col0 + 32 * j + lane < p.N) sb[j] = p.sb[col0 + 32 * j + lane];
      }
      int ok = 1;
      if (lane == 0) ok = wait_bounded(&tfull[buf], bphase, s_abort, p.err, limit) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                            static_cast<uint32_t>(buf * kBN + half * (kCols / 2));
      if (row0 < p.M && col0 < p.N) {
        if (MODE == PAIR_GATED) {
          // 64 hidden units: the gate's and the up projection's columns lie
          // 128 apart in this lane's accumulator row
          box_free(p, lane);
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {
            float g[32], u[32];
            tmem_block(acc0 + j * 32, g);
            tmem_block(acc0 + 128 + j * 32, u);
            gate_mul(g, u, p.act);
            box_put16(box, lane, j, u, p.odt);
          }
          box_send(p, 0, box, lane, row0, col0);
#pragma unroll 1
          for (int o = 1; o < 3 && p.out[1] != nullptr; ++o) {
            box_free(p, lane);
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              float v[32];
              tmem_block(acc0 + (o - 1) * 128 + j * 32, v);
              box_put16(box, lane, j, v, p.odt);
            }
            box_send(p, o, box, lane, row0, col0);
          }
        } else {
          const int per = p.odt == DT_FP32 ? 1 : 2;  // 32-column blocks a box
#pragma unroll 1
          for (int j = 0; j < 4 && col0 + 32 * j < p.N; j += per) {
            box_free(p, lane);
#pragma unroll 1
            for (int i2 = 0; i2 < per; ++i2) {
              float v[32];
              tmem_block(acc0 + (j + i2) * 32, v);
              if (kI8) {
                // the int32 sum is exact; one rounding to fp32, one for each scale
                const int b = j + i2;
                const float s = b == 0 ? sb[0] : b == 1 ? sb[1] : b == 2 ? sb[2] : sb[3];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = static_cast<float>(__float_as_int(v[i])) * sa * __shfl_sync(0xFFFFFFFFu, s, i);
              }
              if (p.odt == DT_FP32)
                box_put32(box, lane, v);
              else
                box_put16(box, lane, i2, v, p.odt);
            }
            box_send(p, MODE == PAIR_DW ? tc.z : 0, box, lane, row0, col0 + 32 * j);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(buf ? tempty_leader1 : tempty_leader0);
      buf ^= 1;
      if (buf == 0) bphase ^= 1u;
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  __syncthreads();
  cluster_sync_all();  // no CTA of the pair leaves while the other may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

constexpr int kPairSmemBytes =
    1024 + kStages * kStageBytes + kEpiWarps * kPairBoxBytes + kNumBarriers * 8 + 16;
static_assert(kPairSmemBytes <= 232448, "shared memory of a block");

// ---------------------------------------------------------------- few rows

// out^T = W x^T: 128 output columns a CTA are the M operand (PAIR_GATED: 64
// hidden units' gate rows, then the same units' up rows), bn output rows
// ("tokens") the N operand, so that a single token costs an MMA of N = 16.
//   PAIR_GATED, PAIR_I8  both operands K-major, as they lie
//   PAIR_DX              M operand Wg, then Wu, MN-major; N operand dg, du
//   PAIR_DW              M operand x, N operand dg or du (blockIdx.z), both
//                        MN-major; the "tokens" are the hidden units
// gridDim.x = splits * column tiles, a cluster being the splits of one tile;
// gridDim.y = row tiles.
struct StreamParams {
  CUtensorMap tmW[2];  // K-major: (k, col), box 128 bytes x 128 (gated: x 64, of Wg and Wu); MN-major: (col, k), box 64 x 64
  CUtensorMap tmX;     // K-major: (k, row, seg), box 128 bytes x bn; MN-major: (row, k, z), box 64 x 64
  void* out[3];        // PAIR_GATED: h, gate, up (the last two may be null); PAIR_DW: dWg, dWu
  long long ldo[3];
  const float *sx, *sw;  // int8: a scale an output row and column
  int tokens, N;         // rows and columns of the output
  int nk, segs;          // K stages a segment, segments
  int splits, bn, stages, tmem_cols;
  int push, join_off;    // the splits' sums are pushed, into memory of their own behind the barriers (else pulled)
  int odt, vec_out;      // vec_out: four output columns can be stored at once
  int act;
  uint32_t idesc;
  int* err;
  unsigned long long timeout_ns;
};

constexpr int kStreamThreads = 192;  // producer, MMA issuer, four epilogue warps
constexpr int kStreamMaxStages = 8;
constexpr int kStreamATile = 128 * kRowBytes;
__host__ __device__ inline int stream_stage_bytes(int bn) { return kStreamATile + bn * kRowBytes; }
// Behind the stages: the barriers, then (from the next 1024 bytes on) the join's own memory where it has some.
__host__ __device__ inline int stream_join_off(int bn, int stages) { return stages * stream_stage_bytes(bn) + 1024; }
static_assert((2 * kStreamMaxStages + 1) * 8 + 16 <= 1024, "the barriers fit");

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void st_dsmem(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void store4(void* base, long long at, int dt, bool vec, int n, const float (&v)[4]) {
  char* p = static_cast<char*>(base) + at * dtype_size(dt);
  if (vec && n >= 4) {
    if (dt == DT_FP32) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (dt == DT_BF16) {
          __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<uint32_t*>(&h);
        } else {
          __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
    return;
  }
  for (int i = 0; i < 4 && i < n; ++i) store_elem(p + i * dtype_size(dt), dt, v[i]);
}

template <int MODE>
__global__ void __launch_bounds__(kStreamThreads, 2) dense_stream_kernel(const __grid_constant__ StreamParams p) {
  constexpr bool I8 = MODE == PAIR_I8;
  constexpr bool GATED = MODE == PAIR_GATED;
  constexpr bool kAmn = MODE == PAIR_DX || MODE == PAIR_DW;
  constexpr bool kBmn = MODE == PAIR_DW;
  constexpr int kBke = I8 ? 128 : 64;
  constexpr int kUnits = GATED ? 64 : 128;  // output columns a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = stream_stage_bytes(p.bn);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.stages * stage_bytes);
  uint64_t* empty = full + kStreamMaxStages;
  uint64_t* done = empty + kStreamMaxStages;  // every MMA of the tile finished
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = static_cast<int>(cluster_ctarank());
  const int unit0 = static_cast<int>(blockIdx.x) / p.splits * kUnits;
  const int tok0 = static_cast<int>(blockIdx.y) * p.bn;
  const int z = MODE == PAIR_DW ? static_cast<int>(blockIdx.z) : 0;
  const uint64_t limit = p.timeout_ns;
  // this CTA's K stages
  const int steps = p.nk * p.segs;
  const int kbeg = static_cast<int>(static_cast<long long>(steps) * split / p.splits);
  const int kend = static_cast<int>(static_cast<long long>(steps) * (split + 1) / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, p.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    tma_prefetch_desc(&p.tmW[0]);
    if (GATED || MODE == PAIR_DX) tma_prefetch_desc(&p.tmW[1]);
    tma_prefetch_desc(&p.tmX);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.push) cluster_arrive();
  const uint32_t tmem_base = *s_tmem;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0, used = 0, last_phase = 0;
    for (int step = kbeg; step < kend; ++step) {
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(&empty[stage], phase ^ 1u, s_abort, p.err, limit))) break;
      uint8_t* dst = smem + stage * stage_bytes;
      uint8_t* dstx = dst + kStreamATile;
      mbar_arrive_expect_tx_w(&full[stage], static_cast<uint32_t>(stage_bytes));
      const int seg = MODE == PAIR_DX && step >= p.nk ? 1 : 0;
      const int k0 = (step - seg * p.nk) * kBke;
      if (kAmn) {
        tma_load_3d_w(dst, &p.tmW[seg], &full[stage], unit0, k0, 0);
        tma_load_3d_w(dst + kStreamATile / 2, &p.tmW[seg], &full[stage], unit0 + 64, k0, 0);
      } else {
        tma_load_3d_w(dst, &p.tmW[0], &full[stage], k0, unit0, 0);
        if (GATED) tma_load_3d_w(dst + kStreamATile / 2, &p.tmW[1], &full[stage], k0, unit0, 0);
      }
      if (kBmn) {
        for (int c = 0; c < p.bn; c += 64) tma_load_3d_w(dstx + c * kRowBytes, &p.tmX, &full[stage], tok0 + c, k0, z);
      } else {
        tma_load_3d_w(dstx, &p.tmX, &full[stage], k0, tok0, seg);
      }
      used |= 1u << stage;
      last_phase = (last_phase & ~(1u << stage)) | (phase << stage);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // no copy is still landing when the stages are used again below
    if (lane == 0)
      for (int s = 0; s < p.stages; ++s)
        if ((used >> s) & 1u) wait_bounded(&full[s], (last_phase >> s) & 1u, nullptr, p.err, limit);
  } else if (warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    const uint32_t s0 = smem_u32(smem), x0 = s0 + kStreamATile;
    const uint64_t dA = kAmn ? smem_desc_sw128(s0, 8192, 1024) : smem_desc_sw128(s0, 16, 1024);
    const uint64_t dB = kBmn ? smem_desc_sw128(x0, 8192, 1024) : smem_desc_sw128(x0, 16, 1024);
    constexpr uint32_t ka = kAmn ? 2048 >> 4 : 32 >> 4, kb = kBmn ? 2048 >> 4 : 32 >> 4;
    for (int step = kbeg; step < kend; ++step) {
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(&full[stage], phase, s_abort, p.err, limit))) break;
      tc_fence_after();
      const uint64_t at = static_cast<uint64_t>((stage * stage_bytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const uint32_t acc = (step > kbeg || kk > 0) ? 1u : 0u;
        if (I8)
          umma_i8_w(tmem_base, dA + at + kk * ka, dB + at + kk * kb, p.idesc, acc);
        else
          umma_f16_w(tmem_base, dA + at + kk * ka, dB + at + kk * kb, p.idesc, acc);
      }
      umma_commit_w(&empty[stage]);
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_w(done);
    if (lane == 0) wait_bounded(done, 0, nullptr, p.err, limit);
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();  // the MMAs are done and no copy is in flight
  // Join the splits: each rank of the cluster owns `chunk` of the tile's
  // rows.  Few rows (push): every rank writes its sums of a row to the owner
  // through distributed shared memory, which waits for nothing.  More (pull):
  // each rank keeps its sums where its stages were, and the owner reads them
  // 16 bytes at a time -- single remote words cost more than the round trip
  // from about 32 rows on (77 x 4096 x 14336 int8: 17.7 us pushed, 15.7
  // pulled; 1 x 4096 x 4096: 4.9 and 5.5).
  const int toks = min(p.bn, p.tokens - tok0);
  const int chunk = (toks + p.splits - 1) / p.splits;
  const bool push = p.push != 0;
  float* part = reinterpret_cast<float*>(smem + (push ? p.join_off : 0));  // push: [rank][chunk][128]; pull: [row][128]
  if (push) cluster_wait();  // every rank has started
  if (warp >= 2) {
    tc_fence_after();
    const int q = warp & 3;
    const uint32_t acc0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const int col = q * 32 + lane;
    const uint32_t mine = smem_u32(part + split * chunk * 128 + col);
    int owner = 0, local = 0;  // of the row being written
    for (int c = 0; c < toks; c += 16) {
      uint32_t raw[16];
      tmem_ld_32x32b_x16(acc0 + c, raw);
      tmem_wait_ld();
      if (!push) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * 128 + col] = __uint_as_float(raw[i]);  // int8: the int32 bits
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i < toks) st_dsmem(mapa_shared(mine, owner) + static_cast<uint32_t>(local) * 512u, raw[i]);
          if (++local == chunk) local = 0, ++owner;
        }
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  if (p.splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // Sum the ranks' parts in their order (int8: whole numbers) and store: four
  // consecutive columns of one row a thread, a row's columns side by side.
  constexpr int kQuads = kUnits / 4;
  const int items = max(0, min(chunk, toks - split * chunk)) * kQuads;
  for (int i = threadIdx.x; i < items; i += kStreamThreads) {
    const int local = i / kQuads, c = (i - local * kQuads) * 4;
    if (unit0 + c >= p.N) continue;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int iv[4] = {0, 0, 0, 0};
    const auto add = [&](const float4& f, const float4& g) {
      if (I8) {
        iv[0] += __float_as_int(f.x), iv[1] += __float_as_int(f.y);
        iv[2] += __float_as_int(f.z), iv[3] += __float_as_int(f.w);
      } else {
        v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
      }
      if (GATED) u[0] += g.x, u[1] += g.y, u[2] += g.z, u[3] += g.w;
    };
    if (push || p.splits == 1) {
      const float4* at = reinterpret_cast<const float4*>(part) + local * 32 + (c >> 2);
      for (int s = 0; s < p.splits; ++s, at += chunk * 32) add(at[0], GATED ? at[16] : at[0]);
    } else {
      const uint32_t at = smem_u32(part + (split * chunk + local) * 128 + c);
      // two or more ranks, a power of two: four loads on their way at a time
      for (int s = 0; s < p.splits; s += 4) {
        float4 f[4], g[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t from = mapa_shared(at, min(s + r, p.splits - 1));
          f[r] = ld_dsmem_f4(from);
          if (GATED) g[r] = ld_dsmem_f4(from + 256);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (s + r < p.splits) add(f[r], GATED ? g[r] : f[r]);
      }
    }
    const int n = p.N - (unit0 + c);
    const long long tk = tok0 + split * chunk + local;
    if (I8) {
      const float sx = p.sx[tk];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = j < n ? static_cast<float>(iv[j]) * sx * p.sw[unit0 + c + j] : 0.0f;
    }
    if (GATED) {
      float h[4] = {u[0], u[1], u[2], u[3]};
      gate_mul(v, h, p.act);
      store4(p.out[0], tk * p.ldo[0] + unit0 + c, p.odt, p.vec_out, n, h);
      if (p.out[1] != nullptr) {
        store4(p.out[1], tk * p.ldo[1] + unit0 + c, p.odt, p.vec_out, n, v);
        store4(p.out[2], tk * p.ldo[2] + unit0 + c, p.odt, p.vec_out, n, u);
      }
    } else {
      store4(p.out[z], tk * p.ldo[z] + unit0 + c, p.odt, p.vec_out, n, v);
    }
  }
  __syncwarp();
  if (!push && p.splits > 1) cluster_sync_all();  // no CTA leaves while another may read its part
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// ---------------------------------------------------------------- around the products

// Rows copied as whole 16-byte pieces, the rest of the last one zero:
// what a tensor map needs where the caller's rows do not start on 16-byte
// boundaries.  One launch for up to three matrices (blockIdx.y).  Sizes in
// bytes.  HBM-bound: a piece is cut out of the two aligned ones about it, except
// where one of them reaches out of the matrix (4096 x 14335 int8 20 us, by
// single elements 38; two of 14336 x 4095 bf16 84 and 98).  One piece a thread
// and turn at full occupancy; four of them at once 24 and 102.
struct PadArgs {
  const uint8_t* in[3];
  uint8_t* out[3];
  long long ld[3], ld_out[3], rows[3], bytes[3];  // from row to row; rows; bytes of one
};

// The 16 bytes at p of which the first n are the row's (the others become
// zeros), in a matrix from `first` to `end`.
__device__ __forceinline__ uint4 cut_piece(const uint8_t* p, int n, const uint8_t* first, const uint8_t* end) {
  const int by = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
  const uint8_t* at = p - by;
  const bool two = by + n > 16;
  uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (at >= first && at + (two ? 32 : 16) <= end) {
    const uint4 lo = *reinterpret_cast<const uint4*>(at);
    w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w;
    if (two) {
      const uint4 hi = *reinterpret_cast<const uint4*>(at + 16);
      w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    }
    if (by & 8) {
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (by & 4) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (by & 3));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;  // of word i
    w[i] = left >= 4 ? w[i] : left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) pad_rows_kernel(const __grid_constant__ PadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int m = blockIdx.y;
  const uint8_t* in = a.in[m];
  const long long ld = a.ld[m], ld_out = a.ld_out[m], rows = a.rows[m], bytes = a.bytes[m], per = (bytes + 15) / 16;
  const uint8_t* end = in + (rows - 1) * ld + bytes;
  // piece j of row r, and from turn to turn (the grid's threads and a row's
  // pieces are counted in 32 bits)
  const uint32_t first = blockIdx.x * 256u + threadIdx.x, step = 256u * gridDim.x, p32 = static_cast<uint32_t>(per);
  long long r = first / p32, j = first % p32;
  const uint32_t step_r = step / p32, step_j = step % p32;
  while (r < rows) {
    *reinterpret_cast<uint4*>(a.out[m] + r * ld_out + j * 16) =
        cut_piece(in + r * ld + j * 16, static_cast<int>(min(bytes - j * 16, 16ll)), in, end);
    r += step_r, j += step_j;
    if (j >= per) j -= per, ++r;
  }
}

// P elements of a 16-bit type (8, 2 or 1) as one access.
template <typename T, int P>
__device__ __forceinline__ void load_n(const T* p, float* v) {
  if constexpr (P == 8)
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<float(*)[8]>(v));
  else
    load_p<T, P>(p, *reinterpret_cast<float(*)[P]>(v));
}

template <typename T, int P>
__device__ __forceinline__ void store_n(T* p, const float* v) {
  if constexpr (P == 8)
    *reinterpret_cast<uint4*>(p) = Elem<T>::pack(*reinterpret_cast<const float(*)[8]>(v));
  else
    store_p<T, P>(p, *reinterpret_cast<const float(*)[P]>(v));
}

// dg = dh u act'(g) and du = dh act(g), one after the other in `out` with
// rows of ldp elements (a multiple of 8).  HBM-bound; both are rounded to the
// io type here, as the operands of the products that follow: a 16-bit MMA
// takes no more, and splitting each into two operands would double the
// products.  It costs dx and the weights' gradients a factor of sqrt 2 in error
// (8192 x 4096 x 14336 bf16 2.3e-3 against 1.7e-3 for unrounded ones), and in
// fp16 the range: past 65504 infinity, below 6e-5 fewer digits, below 3e-8 zero.
//
// 64 threads of a block take 512 columns, eight each, loaded by accesses of P
// elements (what the rows' alignment allows: 8, 2 or 1); the block's four rows
// of threads take every (4 gridDim.y)-th row.  Pairs are spread so that a
// warp's accesses lie side by side, P = 2: 4096 x 2730 by pairs 7 us less than
// one by one.  Single elements stay eight in a row, for the sake of a 16-byte
// store (spread, 4096 x 2731 6 us more).
template <typename T, int P>
__global__ void __launch_bounds__(256) gated_dact_kernel(const T* dh, long long ldh, const T* gate, const T* up,
                                                         long long ldg, T* out, long long ldp, long long rows,
                                                         int cols, int act) {
  constexpr int E = 8 / P;
  constexpr int S = P == 2 ? 2 : 8;  // elements a store
  pdl_wait();
  pdl_trigger();
  const long long c0 = static_cast<long long>(blockIdx.x) * 512 + threadIdx.x * S;
  if (c0 >= ldp) return;
  const int left = static_cast<int>(min(cols - c0, 512ll));  // columns from the thread's first one on
  constexpr int kNext = P == 2 ? 64 * 2 : P;                 // from access to access
  const long long zs = rows * ldp;
  for (long long r = static_cast<long long>(blockIdx.y) * 4 + threadIdx.y; r < rows; r += 4ll * gridDim.y) {
    const T *pd = dh + r * ldh + c0, *pg = gate + r * ldg + c0, *pu = up + r * ldg + c0;
    float d[8], g[8], u[8];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const bool in = i * kNext < left;  // (the padding: zeros)
      if constexpr (P == 1) {
        d[i] = in ? Elem<T>::get(pd[i]) : 0.0f;
        g[i] = in ? Elem<T>::get(pg[i]) : 0.0f;
        u[i] = in ? Elem<T>::get(pu[i]) : 0.0f;
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) d[i * P + j] = g[i * P + j] = u[i * P + j] = 0.0f;
        if (in) {
          load_n<T, P>(pd + i * kNext, d + i * P);
          load_n<T, P>(pg + i * kNext, g + i * P);
          load_n<T, P>(pu + i * kNext, u + i * P);
        }
      }
    }
    gate_grad(d, g, u, act);
#pragma unroll
    for (int i = 0; i < 8 / S; ++i) {
      if (c0 + i * kNext < ldp) {
        store_n<T, S>(out + r * ldp + c0 + i * kNext, g + i * S);
        store_n<T, S>(out + zs + r * ldp + c0 + i * kNext, d + i * S);
      }
    }
  }
}

}  // namespace msb
