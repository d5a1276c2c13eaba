// linear.cu -- matrix product with bias, activation and residual in its
// epilogue, and its gradient, in bf16 on the tcgen05 tensor cores:
//   y  = act(z) + residual,  z = x . W^T + b         x [M, K], W [N, K]
//   dz = g * act'(z),  dx = dz . W,  dW = dz^T . x,  db = sum over rows of dz
// A draft head's residual block and its LM head are this product; sums are
// held in fp32 (tensor memory) and each result is rounded once.
//
// Three products, one kernel: the operands of D[r, c] = sum_k A[r, k] B[c, k]
// are read where they lie, the summed dimension contiguous (x and W of the
// forward product, dz of dx) or strided (W of dx, dz and x of dW); TMA brings
// either into 128-byte swizzled tiles and the matrix descriptor tells the
// tensor core which way they run, so nothing is transposed in memory.
//   gemm_kernel      CTA pairs (cta_group::2), 256 x 256 / 128 / 64 tiles,
//                    persistent.  Tensor-bound, in runs too short for the power
//                    cap: 4096 x 8192 x 4096 without an epilogue 140.5 us = 1.96
//                    PFLOP/s (cuBLAS 136 to 142 us in the same processes; after a
//                    second of load 165, cuBLAS 150 to 160); the gradient of 4096^3
//                    without an activation 147 us.
//   few_rows_kernel  few rows or tiles: the weight is the MMA's 128-row operand
//                    and a cluster splits the summed dimension, joined through
//                    distributed shared memory.  Bound by the weight's stream and
//                    the join: 96 x 8192 x 4096 16.5 us, weight from HBM.
//   dot_kernel       at most four rows, on CUDA cores.  HBM- and latency-bound:
//                    1 x 4096 x 4096 7.0 us in a graph, 1 x 152064 x 2048 85.5 us = 7.3 TB/s.
//   dz_kernel        dz and db, 81 % of the copy rate.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "pipe.cuh"

namespace cg = cooperative_groups;

namespace sga {
namespace {

// ------------------------------------------------------------- activations

// z / (1 + e^-u) with the hardware's 2^x and 1/x (2 ulp each; e^-u past the
// range of fp32 gives 0, as it should).
__device__ __forceinline__ float sigmoid_times(float z, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r;
}

// The normal distribution's cdf at z, and e = e^(-z^2 / 2).  With a = |z|,
//   cdf(-a) = e t P(t),  t = 1 / (1 + 0.282 a),
// P the polynomial of degree 8 nearest to e^(a^2 / 2) erfc(a / sqrt 2) / (2 t) over
// 0 < t <= 1 (a weighted least-squares fit, relative error below 1.4e-7).  The left
// tail keeps its relative accuracy: (1 + erf(z / sqrt 2)) / 2 cancels there (off by 4 %
// at z = -5, 0 from -5.5).  4096 x 8192 x 4096 and its dz 163 and 47 us; with erfcf
// 186 and 95.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float a = fabsf(z);
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * -0.7213475204444817f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.282f, a, 1.0f)));
  float p = fmaf(0.025004314f, t, -0.09206650f);
  p = fmaf(p, t, 0.08681425f);
  p = fmaf(p, t, -0.003813729f);
  p = fmaf(p, t, 0.07129859f);
  p = fmaf(p, t, 0.08408976f);
  p = fmaf(p, t, 0.10367318f);
  p = fmaf(p, t, 0.11249836f);
  p = fmaf(p, t, 0.11250174f);
  const float tail = e * (t * p);
  return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case SGA_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case SGA_ACT_SILU: return sigmoid_times(z, z);
    case SGA_ACT_GELU: {
      float e;
      return z * normal_cdf(z, e);
    }
    case SGA_ACT_GELU_TANH:  // z (1 + tanh u) / 2 = z / (1 + e^-2u)
      return sigmoid_times(z, 2.0f * kGeluA * fmaf(kGeluB * z * z, z, z));
    default: return z;
  }
}

__device__ __forceinline__ float activate_grad(float z, int act) {
  switch (act) {
    case SGA_ACT_SILU: {
      const float q = sigmoid_times(1.0f, z);
      return q * fmaf(z, 1.0f - q, 1.0f);
    }
    case SGA_ACT_GELU: {
      float e;
      const float cdf = normal_cdf(z, e);
      return fmaf(z * 0.3989422804014327f, e, cdf);
    }
    case SGA_ACT_GELU_TANH: {
      // beyond +-16 the derivative is 0 or 1 (and z^3 stays finite below)
      z = z < -16.0f ? -16.0f : (z > 16.0f ? 16.0f : z);
      const float z2 = z * z;
      const float q = sigmoid_times(1.0f, z * fmaf(2.0f * kGeluA * kGeluB, z2, 2.0f * kGeluA));
      const float du = fmaf(6.0f * kGeluA * kGeluB, z2, 2.0f * kGeluA);
      return fmaf(z * q * (1.0f - q), du, q);
    }
    default: return 1.0f;
  }
}

__device__ __forceinline__ float ld_bf16(const __nv_bfloat16 *p) {
  return __uint_as_float(
      static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(p)) << 16);
}

__device__ __forceinline__ float ld_bias(const void *bias, int f32, int64_t c) {
  if (bias == nullptr) return 0.0f;
  return f32 ? static_cast<const float *>(bias)[c]
             : ld_bf16(static_cast<const __nv_bfloat16 *>(bias) + c);
}

// What happens to an accumulator: out[r, c] = act(acc + bias[c]) + res[r, c],
// pre[r, c] = acc + bias[c] (each of bias, res, pre nullable).
struct Epilogue {
  __nv_bfloat16 *out, *pre;
  const __nv_bfloat16 *res;
  const void *bias;
  int64_t ldo, ldp, ldr;
  int bias_f32, act;
  int aligned;  // gemm_kernel: rows of out, pre and res start on 16-byte boundaries
};

// ------------------------------------------------------------- descriptors

// Shared-memory descriptor of an operand tile with the 128-byte swizzle.
// Summed dimension contiguous: rows of 128 bytes, 8-row groups 1024 B apart.
// Summed dimension strided: rows of 64 elements of the other dimension, one
// row per summed index, 8-row groups 1024 B apart (stride offset) and the next
// 64 elements of the other dimension one 64-row box (8192 B) on (leading
// offset).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool strided) {
  return smem_desc_sw128(addr) + (strided ? static_cast<uint64_t>((8192 >> 4) - 1) << 16 : 0);
}

// Instruction descriptor (bf16 x bf16 -> fp32) with the operands' directions.
__device__ __forceinline__ uint32_t operand_idesc(uint32_t m, uint32_t n, bool a_strided,
                                                  bool b_strided) {
  return instr_desc<false>(m, n) | (a_strided ? 1u << 15 : 0u) | (b_strided ? 1u << 16 : 0u);
}

// 16-byte descriptor units between the 16-deep K steps of a 64-deep block.
__device__ __forceinline__ uint32_t k_step(bool strided) { return strided ? 2048 >> 4 : 32 >> 4; }

__device__ __forceinline__ void mma_pair_rt(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_one_rt(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------------------
// gemm_kernel: warp 0 TMA producer, warp 1 MMA issuer (leader CTA of the
// pair), warps 2..9 epilogue; the roles and barriers are those of the LM-head
// kernel of lmhead.cu.  A launch runs one or two products (dx and dW of one
// gradient): their tiles form one list, so the second fills the SMs that the
// first one's last wave leaves idle.
// ---------------------------------------------------------------------------
constexpr int kMaxProducts = 2;

constexpr int kBand = 8;  // row tiles of a band (see tile_at)

struct Product {
  int rows, cols, num_kb;       // D's size; 64-deep blocks of the summed dimension
  int tiles_r, tiles_c;         // 256 x kBN tiles
  uint32_t inv_band, inv_last;  // reciprocals of a band's tiles, of the last band's height
  int a_strided, b_strided;
  Epilogue ep;
};

// Pair i of CTAs takes tiles i, i + pairs, ... of product 0 and a contiguous
// run of product 1's: `lead` pairs (those with one tile more of product 0)
// take runs of run[0], the others of run[1], so that all end together although
// the two products' tiles differ in length.
struct Products {
  int tiles[kMaxProducts];  // (0: no such product)
  int lead, run[2];
  Product p[kMaxProducts];
};

// A pair's tiles in order, without divisions on the way.
struct PairTiles {
  int t0, step, own0;   // product 0: t0, t0 + step, ... (own0 of them)
  int first1, own1;     // product 1: first1, first1 + 1, ...

  __device__ __forceinline__ PairTiles(const Products &prods, int pair, int num_pairs) {
    const bool lead = pair < prods.lead;
    t0 = pair;
    step = num_pairs;
    own0 = prods.tiles[0] / num_pairs + (lead ? 1 : 0);
    first1 = lead ? pair * prods.run[0]
                  : prods.lead * prods.run[0] + (pair - prods.lead) * prods.run[1];
    own1 = max(0, min(prods.run[lead ? 0 : 1], prods.tiles[1] - first1));
  }

  // The i-th: product and tile number; false past the last.
  __device__ __forceinline__ bool at(int i, int &pi, int &t) const {
    pi = i < own0 ? 0 : 1;
    t = pi == 0 ? t0 + i * step : first1 + i - own0;
    return i < own0 + own1;
  }
};

struct Maps {
  CUtensorMap a[kMaxProducts], b[kMaxProducts];
};

constexpr int kGemmThreads = 320;        // producer, MMA, eight epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kTileA = 128 * ROW_BYTES;  // 16 KB: this CTA's 128 rows of A
template <int kBN>
constexpr int tile_b = kBN / 2 * ROW_BYTES;  // this CTA's half of B
template <int kBN>
constexpr int gemm_stage = kTileA + tile_b<kBN>;
constexpr int kBox = 32 * ROW_BYTES;         // 32 rows x 64 columns of results
constexpr int kEpiBytes = kEpiWarps * kBox;  // one box per epilogue warp
template <int kBN>
constexpr int gemm_stages = (227 * 1024 - 2560 - kEpiBytes) / gemm_stage<kBN>;
template <int kBN>
constexpr int gemm_smem = 1024 + gemm_stages<kBN> * gemm_stage<kBN> + kEpiBytes + 1536;

template <int kBN>
struct SharedGemm {
  uint64_t full[gemm_stages<kBN>];
  uint64_t empty[gemm_stages<kBN>];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) float bias[kBN];  // the tile's
};
static_assert(sizeof(SharedGemm<256>) <= 1536 && sizeof(SharedGemm<64>) <= 1536, "shared block");

// t / d from the reciprocal m = 2^32 / d (rounded down): the estimate is short
// by at most one.
__device__ __forceinline__ int quotient(int t, int d, uint32_t m) {
  const int q = static_cast<int>(__umulhi(static_cast<uint32_t>(t), m));
  return t - q * d >= d ? q + 1 : q;
}

// Tile t of a product: bands of kBand row tiles, row tiles fastest, so that the
// pairs at work share a few A and B panels through L2.
__device__ __forceinline__ void tile_at(const Product &p, int t, int &tr, int &tc) {
  const int band = quotient(t, kBand * p.tiles_c, p.inv_band);
  const int in = t - band * kBand * p.tiles_c;
  const int height = min(kBand, p.tiles_r - band * kBand);
  tc = height == kBand ? in / kBand : quotient(in, height, p.inv_last);
  tr = band * kBand + in - tc * height;
}

// A warp's box of results in shared memory: 32 rows of 64 bf16, 16-byte piece j
// of row r at piece j ^ (r & 7), so that a lane per row (from the accumulators)
// and eight lanes per row (to global memory) access it without bank conflicts.
// (TMA stores from the box were slower: their reads of it hold up the next box
// by 350 to 750 cycles, the eight 16-byte stores a lane by about 250.)
__device__ __forceinline__ uint4 *box_piece(uint8_t *box, int r, int j) {
  return reinterpret_cast<uint4 *>(box + r * ROW_BYTES + ((j ^ (r & 7)) << 4));
}

__device__ __forceinline__ unsigned short *box_elem(uint8_t *box, int r, int c) {
  return reinterpret_cast<unsigned short *>(box_piece(box, r, c >> 3)) + (c & 7);
}

// Box <-> global memory, whole boxes: eight lanes per row.  Rows on 16-byte
// boundaries (kAligned) as they are; else, with the row `off` bytes past a
// boundary, its aligned 16-byte pieces go as such, put together from two pieces
// of the box, and the eight columns at its ends one by one.  (Two-byte accesses
// throughout: 3660 x 14645 x 144 took 81 us.)  Boxes at the right edge: two
// columns a lane.
template <bool kAligned>
__device__ __forceinline__ void box_store_rows(uint8_t *box, __nv_bfloat16 *p, int64_t ld, int rows,
                                               int cols, int lane) {
  if (cols >= 64) {
    const int j = lane & 7;
    if constexpr (kAligned) {
      uint4 *q = reinterpret_cast<uint4 *>(p + (lane >> 3) * ld) + j;
#pragma unroll
      for (int r = lane >> 3; r < 32; r += 4) {
        const uint4 w = *box_piece(box, r, j);
        if (r < rows) *q = w;
        q += ld / 2;  // four rows on
      }
    } else {
#pragma unroll 2
      for (int r = lane >> 3; r < 32; r += 4) {
        unsigned short *q = reinterpret_cast<unsigned short *>(p + r * ld);
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 15);
        const uint4 w =
            bytes_of(*box_piece(box, r, max(j - 1, 0)), *box_piece(box, r, j), 16 - off);
        const int e = 2 * j < 16 - off ? j : 56 + j;
        const unsigned short edge = *box_elem(box, r, e);
        if (r < rows && (j > 0 || off == 0))
          *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(q) - off + 16 * j) = w;
        if (r < rows && off != 0) q[e] = edge;
      }
    }
    return;
  }
  const int c = 2 * lane;
  unsigned short *q = reinterpret_cast<unsigned short *>(p) + c;
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(box_elem(box, r, c));
    if (c < cols) q[0] = static_cast<unsigned short>(w);
    if (c + 1 < cols) q[1] = static_cast<unsigned short>(w >> 16);
    q += ld;
  }
}

template <bool kAligned>
__device__ __forceinline__ void box_load_rows(uint8_t *box, const __nv_bfloat16 *p, int64_t ld,
                                              int rows, int cols, int lane) {
  if (cols >= 64) {
    const int j = lane & 7;
    if (kAligned) {
      uint4 w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        w[u] = *(reinterpret_cast<const uint4 *>(p + min((lane >> 3) + 4 * u, rows - 1) * ld) + j);
#pragma unroll
      for (int u = 0; u < 8; ++u) *box_piece(box, (lane >> 3) + 4 * u, j) = w[u];
      return;
    }
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int r0 = lane >> 3; r0 < 32; r0 += 4 * kBatch) {
      uint4 w[kBatch];
      unsigned short edge[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const unsigned short *q = reinterpret_cast<const unsigned short *>(
            p + min(r0 + 4 * u, rows - 1) * ld);
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(q) & 15);
        // (piece 0 of an unaligned row starts before it: piece 1 is read again)
        const int at = j > 0 || off == 0 ? j : 1;
        w[u] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(q) - off + 16 * at);
        edge[u] = q[2 * j < 16 - off ? j : 56 + j];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int r = r0 + 4 * u;
        const int off = static_cast<int>(
            reinterpret_cast<uintptr_t>(p + min(r, rows - 1) * ld) & 15);
        uint4 next;
        next.x = __shfl_down_sync(0xffffffffu, w[u].x, 1);
        next.y = __shfl_down_sync(0xffffffffu, w[u].y, 1);
        next.z = __shfl_down_sync(0xffffffffu, w[u].z, 1);
        next.w = __shfl_down_sync(0xffffffffu, w[u].w, 1);
        *box_piece(box, r, j) = bytes_of(w[u], next, off);
        __syncwarp();
        if (off != 0) *box_elem(box, r, 2 * j < 16 - off ? j : 56 + j) = edge[u];
      }
    }
    return;
  }
  const int c = 2 * lane;
  const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
  // (loads at clamped addresses, not behind branches: eight rows in flight)
  const int lo = c < cols ? c : cols - 1, hi = c + 1 < cols ? c + 1 : cols - 1;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    unsigned short a[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = min(r0 + i, rows - 1);
      a[i] = q[r * ld + lo];
      b[i] = q[r * ld + hi];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<uint32_t *>(box_elem(box, r0 + i, c)) =
          a[i] | (static_cast<uint32_t>(b[i]) << 16);
  }
}

// Eight accumulators (columns 8 j .. + 7 of the box) -> box: plus bias, through
// the activation, plus what the box holds there when `add` (the residual).
template <int kAct>
__device__ __forceinline__ void box_fill_piece(uint8_t *box, const uint32_t *r, const float *bias,
                                               int j, bool add, int lane) {
  uint4 *q = box_piece(box, lane, j);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    float4 b = {0.0f, 0.0f, 0.0f, 0.0f};
    if (bias != nullptr) b = *reinterpret_cast<const float4 *>(bias + j * 8 + i);
    y[i] = activate(__uint_as_float(r[i]) + b.x, kAct);
    y[i + 1] = activate(__uint_as_float(r[i + 1]) + b.y, kAct);
    y[i + 2] = activate(__uint_as_float(r[i + 2]) + b.z, kAct);
    y[i + 3] = activate(__uint_as_float(r[i + 3]) + b.w, kAct);
  }
  if (add) {
    const uint4 w = *q;
    y[0] += bf16_lo(w.x);
    y[1] += bf16_hi(w.x);
    y[2] += bf16_lo(w.y);
    y[3] += bf16_hi(w.y);
    y[4] += bf16_lo(w.z);
    y[5] += bf16_hi(w.z);
    y[6] += bf16_lo(w.w);
    y[7] += bf16_hi(w.w);
  }
  *q = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
}

// Columns taddr .. + 63 of this warp's 32 TMEM lanes (a lane per row) -> box.
// `done` runs once the accumulators are in registers.  All 64 columns are
// asked for at once: a tcgen05.ld and its wait take some 300 cycles.
template <int kAct, typename Done>
__device__ __forceinline__ void box_fill_act(uint8_t *box, uint32_t taddr, const float *bias,
                                             bool add, int lane, Done done) {
  uint32_t r[2][32];
  tmem_ld32(taddr, r[0]);
  tmem_ld32(taddr + 32, r[1]);
  tmem_ld_wait();
  done();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    box_fill_piece<kAct>(box, r[j / 4] + j % 4 * 8, bias, j, add, lane);
}

template <typename Done>
__device__ __forceinline__ void box_fill(uint8_t *box, uint32_t taddr, const float *bias, int act,
                                         bool add, int lane, Done done) {
  switch (act) {
    case SGA_ACT_RELU: return box_fill_act<SGA_ACT_RELU>(box, taddr, bias, add, lane, done);
    case SGA_ACT_SILU: return box_fill_act<SGA_ACT_SILU>(box, taddr, bias, add, lane, done);
    case SGA_ACT_GELU: return box_fill_act<SGA_ACT_GELU>(box, taddr, bias, add, lane, done);
    case SGA_ACT_GELU_TANH:
      return box_fill_act<SGA_ACT_GELU_TANH>(box, taddr, bias, add, lane, done);
    default: return box_fill_act<SGA_ACT_NONE>(box, taddr, bias, add, lane, done);
  }
}

template <int kBN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Products prods,
                uint32_t *err) {
  constexpr int kStages = gemm_stages<kBN>;
  constexpr int kStageB = gemm_stage<kBN>;
  constexpr int kCols = 2 * kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *boxes = base + kStages * kStageB;
  SharedGemm<kBN> *sh =
      reinterpret_cast<SharedGemm<kBN> *>(base + kStages * kStageB + kEpiBytes);
  const volatile int *abort_flag = &sh->abort;
  const int warp = uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = uniform(cluster_rank());
  const bool leader = rank == 0;
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int num_pairs = static_cast<int>(gridDim.x >> 1);
  const PairTiles tiles(prods, pair, num_pairs);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);
      mbar_init(smem_u32(&sh->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&sh->tmem_full[b]), 1);
      // this CTA's epilogue warps, and in the leader the follower's word
      mbar_init(smem_u32(&sh->tmem_empty[b]), kEpiWarps + (leader ? 1 : 0));
    }
    mbar_init(smem_u32(&sh->drain), 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh->tmem_base)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem_base = uniform(sh->tmem_base);
  pdl_wait();

  int prod_stage = 0;
  uint32_t prod_phase = 0;
  long long issued = 0;

  if (warp == 0) {
    // -------------------------------------------------- producer (both CTAs)
    int pi, t;
    for (int n = 0; tiles.at(n, pi, t) && !aborted(abort_flag); ++n) {
      const Product &p = prods.p[pi];
      int tr, tc;
      tile_at(p, t, tr, tc);
      const int row = tr * 256 + static_cast<int>(rank) * 128;
      const int col = tc * kBN + static_cast<int>(rank) * (kBN / 2);
      // held in registers: inside the loop the asm statements would make the
      // compiler read the table again for every K block
      const int num_kb = p.num_kb;
      const bool a_strided = p.a_strided != 0, b_strided = p.b_strided != 0;
      const CUtensorMap *map_a = &maps.a[pi], *map_b = &maps.b[pi];
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!warp_wait(smem_u32(&sh->empty[prod_stage]), prod_phase ^ 1, abort_flag)) {
          if (lane == 0) raise_abort(&sh->abort, err);
          break;
        }
        const uint32_t full = map_to_rank(smem_u32(&sh->full[prod_stage]), 0);
        if (elect_one()) {
          if (leader) mbar_expect_tx(smem_u32(&sh->full[prod_stage]), 2 * kStageB);
          const uint32_t a = smem_u32(base + prod_stage * kStageB);
          if (a_strided) {
            tma_load_2d_pair(a, map_a, row, kb * 64, full);
            tma_load_2d_pair(a + 8192, map_a, row + 64, kb * 64, full);
          } else {
            tma_load_2d_pair(a, map_a, kb * 64, row, full);
          }
          if (b_strided) {
#pragma unroll
            for (int i = 0; i < kBN / 128; ++i)
              tma_load_2d_pair(a + kTileA + i * 8192, map_b, col + i * 64, kb * 64, full);
          } else {
            tma_load_2d_pair(a + kTileA, map_b, kb * 64, col, full);
          }
        }
        __syncwarp();
        ++issued;
        if (++prod_stage == kStages) {
          prod_stage = 0;
          prod_phase ^= 1;
        }
      }
    }
  } else if (warp == 1 && leader) {
    // --------------------------------------------------- MMA issuer (leader)
    int stage = 0, acc = 0, pi, t;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    for (int n = 0;
         tiles.at(n, pi, t) && ok && !aborted(abort_flag); ++n) {
      const Product &p = prods.p[pi];
      const int num_kb = p.num_kb;
      const bool a_strided = p.a_strided != 0, b_strided = p.b_strided != 0;
      const uint32_t idesc = operand_idesc(256, kBN, a_strided, b_strided);
      const uint32_t step_a = k_step(a_strided), step_b = k_step(b_strided);
      if (!warp_wait(smem_u32(&sh->tmem_empty[acc]), acc_phase ^ 1, abort_flag)) {
        if (lane == 0) raise_abort(&sh->abort, err);
        break;
      }
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * kBN;
      for (int kb = 0; kb < num_kb; ++kb) {
        if (!warp_wait(smem_u32(&sh->full[stage]), phase, abort_flag)) {
          if (lane == 0) raise_abort(&sh->abort, err);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(base + stage * kStageB);
        const uint64_t a_desc = operand_desc(a, a_strided);
        const uint64_t b_desc = operand_desc(a + kTileA, b_strided);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_pair_rt(d_tmem, a_desc + step_a * kk, b_desc + step_b * kk, idesc, (kb | kk) != 0);
          mma_commit_pair(smem_u32(&sh->empty[stage]));
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit_pair(smem_u32(&sh->tmem_full[acc]));
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else if (warp == 1) {
    // ----------------------------------------------------- word to the leader
    // The follower's epilogue warps release an accumulator on a barrier of
    // their own; this otherwise idle warp passes that on.  (An arrival at the
    // peer waits for the writes before it: 1400 cycles of an epilogue warp.)
    int acc = 0, pi, t;
    uint32_t acc_phase = 0;
    const uint32_t at_leader[2] = {map_to_rank(smem_u32(&sh->tmem_empty[0]), 0),
                                   map_to_rank(smem_u32(&sh->tmem_empty[1]), 0)};
    for (int n = 0; tiles.at(n, pi, t); ++n) {
      if (!warp_wait(smem_u32(&sh->tmem_empty[acc]), acc_phase, abort_flag)) {
        if (lane == 0) raise_abort(&sh->abort, err);
        break;
      }
      tc_fence_after();
      tc_fence_before();
      if (lane == 0) mbar_arrive_remote(at_leader[acc]);
      __syncwarp();
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else if (warp >= 2) {
    // -------------------------------------------------- epilogue (both CTAs)
    // Warps 2..5 and 6..9 each cover the four TMEM lane quarters and take the
    // tile's 64-column pieces alternately.
    const int quarter = warp & 3;
    const int half = warp >= 6;
    uint8_t *box = boxes + (warp - 2) * kBox;
    int acc = 0, pi, t;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int n = 0; ok && tiles.at(n, pi, t); ++n) {
      const Product &p = prods.p[pi];
      int tr, tc;
      tile_at(p, t, tr, tc);
      const Epilogue ep = p.ep;
      const int cols = p.cols;
      const int row0 = tr * 256 + static_cast<int>(rank) * 128 + quarter * 32;
      const int rows = min(32, p.rows - row0);
      if (ep.bias != nullptr) {
        // the tile's bias, once every warp is done with the last tile's
        asm volatile("bar.sync 1, 256;" ::: "memory");
        for (int c = threadIdx.x - 64; c < kBN; c += 32 * kEpiWarps)
          sh->bias[c] = tc * kBN + c < cols
                            ? ld_bias(ep.bias, ep.bias_f32, static_cast<int64_t>(tc) * kBN + c)
                            : 0.0f;
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      auto load = [&](const __nv_bfloat16 *q, int64_t ld, int col0) {
        if (ep.aligned)
          box_load_rows<true>(box, q + row0 * ld + col0, ld, rows, cols - col0, lane);
        else
          box_load_rows<false>(box, q + row0 * ld + col0, ld, rows, cols - col0, lane);
        __syncwarp();
      };
      auto store = [&](__nv_bfloat16 *q, int64_t ld, int col0) {
        __syncwarp();
        if (ep.aligned)
          box_store_rows<true>(box, q + row0 * ld + col0, ld, rows, cols - col0, lane);
        else
          box_store_rows<false>(box, q + row0 * ld + col0, ld, rows, cols - col0, lane);
        __syncwarp();
      };
      const int first = tc * kBN + half * 64;
      // the first piece's residual, ahead of the accumulators
      const bool early = rows > 0 && half * 64 < kBN && first < cols && ep.res != nullptr &&
                         ep.pre == nullptr;
      if (early) load(ep.res, ep.ldr, first);
      ok = warp_wait(smem_u32(&sh->tmem_full[acc]), acc_phase, abort_flag);
      if (!ok && lane == 0) raise_abort(&sh->abort, err);
      if (ok) {
        tc_fence_after();
        const uint32_t tlane =
            tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kBN;
        // the accumulators have been read: the MMA may overwrite them
        bool released = false;
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->tmem_empty[acc]));
          released = true;
        };
#pragma unroll 1
        for (int q = half * 64; q < kBN; q += 128) {
          const int col0 = tc * kBN + q;
          if (rows <= 0 || col0 >= cols) break;
          const bool last = q + 128 >= kBN || col0 + 128 >= cols;
          const float *bias = ep.bias != nullptr ? sh->bias + q : nullptr;
          if (ep.pre != nullptr) {
            box_fill_act<SGA_ACT_NONE>(box, tlane + q, bias, false, lane, [] {});
            store(ep.pre, ep.ldp, col0);
          }
          if (ep.res != nullptr && !(early && q < 128)) load(ep.res, ep.ldr, col0);
          box_fill(box, tlane + q, bias, ep.act, ep.res != nullptr, lane, [&] {
            if (last) release();
          });
          store(ep.out, ep.ldo, col0);
        }
        if (!released) release();
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
      // (an epilogue warp that gives up keeps to the barriers of the others)
      if (!ok) {
        for (int u = n + 1; tiles.at(u, pi, t); ++u) {
          if (prods.p[pi].ep.bias == nullptr) continue;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
      }
    }
  }

  pdl_launch_dependents();
  __syncthreads();
  if (*abort_flag) {
    const int zero = 0;
    if (warp == 0 && lane == 0) {
      if (leader) {
        // the leader's full barriers count the copies of both CTAs
        const long long outstanding = issued < kStages ? issued : kStages;
        for (long long i = 1; i <= outstanding; ++i) {
          int s = prod_stage - static_cast<int>(i);
          uint32_t ph = prod_phase;
          if (s < 0) {
            s += kStages;
            ph ^= 1;
          }
          mbar_wait(smem_u32(&sh->full[s]), ph, &zero);
        }
      } else if (issued > 0) {
        // the follower's copies complete on the leader's barriers, which it
        // cannot wait on: give them a bounded 1 ms to land
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
    if (warp == 1 && leader && elect_one()) {  // the lane that issued the MMAs
      mma_commit_pair(smem_u32(&sh->drain));
      mbar_wait(smem_u32(&sh->drain), 0, &zero);
    }
  }
  // the peer may still read this CTA's shared memory or write its TMEM
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kCols)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// few_rows_kernel: out[m, r] = act(sum_k A[r, k] x[m, k] + bias[r]) + res[m, r]
// with A the weight (128 rows r per CTA, its TMEM lanes) and up to kN rows of x
// the MMA's columns (kN <= 128; more rows: blocks of 128).  For M <= 128 the
// weight is read once and sets the pace; for more rows this form pays where the
// product has too few 256-row tiles to fill the SMs.
// A cluster of `splits` CTAs shares a tile: each sums its range of K blocks
// (maybe none), stores its fp32 partial tile in its own shared memory, and
// finishes 128 / splits of the rows from every CTA's part, in rank order (a
// fixed order: results do not vary from run to run).
// ---------------------------------------------------------------------------
template <int kN>
constexpr int few_stage = kTileA + kN * ROW_BYTES;
// Ring stages with two CTAs per SM, and where one per SM holds all of them
// and they turn the smaller ring three times (96 x 4096 x 4096 12.7 -> 11.9 us, 24 x
// 1024 x 8192 9.1 -> 8.8; at two and a half turns, 333 x 1531 x 2056 11.6 -> 12.0).
template <int kN>
constexpr int few_stages = (110 * 1024) / few_stage<kN>;
template <int kN>
constexpr int few_most_stages = (220 * 1024) / few_stage<kN>;
template <int kN>
constexpr int few_cols = kN < 32 ? 32 : kN;  // TMEM columns (a power of two, at least 32)

template <int kN>
struct SharedFew {
  uint64_t full[few_most_stages<kN>];
  uint64_t empty[few_most_stages<kN>];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
};

template <int kN>
constexpr int few_smem(int stages) {
  return 1024 + stages * few_stage<kN> + static_cast<int>(sizeof(SharedFew<kN>));
}
static_assert(few_stages<128> * few_stage<128> >= 128 * 128 * 4, "a partial tile fits the ring");
static_assert(2 * (few_smem<16>(few_stages<16>) + 1024) <= 228 * 1024 &&
                  few_smem<16>(few_most_stages<16>) <= 227 * 1024,
              "ring sizes");

// n <= 4 consecutive bf16, as one access where they are four and aligned.
__device__ __forceinline__ void load_four(const __nv_bfloat16 *p, int n, float (&x)[4]) {
  if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    x[0] = bf16_lo(w.x);
    x[1] = bf16_hi(w.x);
    x[2] = bf16_lo(w.y);
    x[3] = bf16_hi(w.y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ld_bf16(p + (i < n ? i : n - 1));
  }
}

__device__ __forceinline__ void store_four(__nv_bfloat16 *p, int n, const float (&x)[4]) {
  if (n == 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(x[i]);
  }
}

// A CTA's share of the tile's rows, for every m: a thread takes rows r .. r + 3 of
// two m at a time and asks for all of their parts at once (one after the other,
// the reads of the peers' memory took 500 cycles each; four m at a time: no gain).
__device__ __forceinline__ void join_parts(const float *part, int M, int first_m, int row0, int rows,
                                           int num_kb, int log_splits, int r,
                                           const float (&bias)[4], const Epilogue &ep) {
  const int at_once = THREADS / 32 << log_splits;
  const int64_t col = row0 + r;
  const int n = min(4, rows - row0 - r);
  if (n > 0) {
    uint32_t src[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      src[i] = i < 1 << log_splits && num_kb * i >> log_splits != num_kb * (i + 1) >> log_splits
                   ? map_to_rank(smem_u32(part) + r * 4, i)
                   : 0u;  // (a CTA without K blocks has no part)
    for (int m0 = static_cast<int>(threadIdx.x) >> (5 - log_splits); m0 < M; m0 += 2 * at_once) {
      float4 v[2][8];
      float res[2][4] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int m = min(m0 + u * at_once, M - 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[u][i] = {0.0f, 0.0f, 0.0f, 0.0f};
          if (src[i] != 0 && (u == 0 || M > u * at_once))
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v[u][i].x), "=f"(v[u][i].y), "=f"(v[u][i].z), "=f"(v[u][i].w)
                         : "r"(src[i] + m * 512));
        }
        if (ep.res != nullptr)
          load_four(ep.res + (first_m + m) * ep.ldr + col, n, res[u]);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t m = first_m + m0 + u * at_once;
        if (m0 + u * at_once >= M) break;
        float z[4] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          z[0] += v[u][i].x;
          z[1] += v[u][i].y;
          z[2] += v[u][i].z;
          z[3] += v[u][i].w;
        }
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += bias[i];
        if (ep.pre != nullptr) store_four(ep.pre + m * ep.ldp + col, n, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = activate(z[i], ep.act) + res[u][i];
        store_four(ep.out + m * ep.ldo + col, n, y);
      }
    }
  }
}

template <int kN>
__global__ void __launch_bounds__(THREADS, 2)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmap_w,
                    const __grid_constant__ CUtensorMap tmap_x, int all_m, int rows, int num_kb,
                    int blocks, int stages, int log_splits, int box, int strided, const Epilogue ep,
                    uint32_t *err) {
  constexpr int kStageB = few_stage<kN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  SharedFew<kN> *sh = reinterpret_cast<SharedFew<kN> *>(base + stages * kStageB);
  const volatile int *abort_flag = &sh->abort;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = 1 << log_splits;
  const int unit = static_cast<int>(blockIdx.x) >> log_splits;
  const int split = static_cast<int>(blockIdx.x) & (splits - 1);
  const int tile = unit / blocks;
  const int first_m = (unit - tile * blocks) * kN;  // this CTA's rows of x
  const int M = min(kN, all_m - first_m);
  const int kb0 = num_kb * split >> log_splits;  // (num_kb <= 2^18)
  const int kb1 = num_kb * (split + 1) >> log_splits;
  const int row0 = tile * 128;

  if (threadIdx.x == 64) {
    // Warm L2 with the first ring of the weight while the previous kernel
    // drains: a prefetch only fills L2, which stays coherent with any later
    // write, so it may precede the dependency wait.
    for (int kb = kb0; kb < kb1 && kb < kb0 + stages; ++kb) {
      if (strided) {
        tma_prefetch_2d(&tmap_w, row0, kb * 64);
        tma_prefetch_2d(&tmap_w, row0 + 64, kb * 64);
      } else {
        tma_prefetch_2d(&tmap_w, kb * 64, row0);
      }
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);
      mbar_init(smem_u32(&sh->empty[s]), 1);
    }
    mbar_init(smem_u32(&sh->done), 1);
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh->tmem_base)),
                 "r"(few_cols<kN>)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = sh->tmem_base;
  pdl_wait();

  // The rows r .. r + 3 of the tile that this thread finishes; their bias is asked
  // for now, and L2 for the residual.
  const int quads = 32 >> log_splits;
  const int r = (split * quads + (static_cast<int>(threadIdx.x) & (quads - 1))) * 4;
  float bias[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    bias[i] = row0 + r + i < rows ? ld_bias(ep.bias, ep.bias_f32, row0 + r + i) : 0.0f;
  if (ep.res != nullptr && static_cast<int>(threadIdx.x) < M && row0 + split * quads * 4 < rows)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(ep.res + (first_m + threadIdx.x) * ep.ldr + row0 +
                                                  split * quads * 4));

  int prod_stage = 0;
  uint32_t prod_phase = 0;
  int issued = 0;
  bool good = true;
  float *part = reinterpret_cast<float *>(base);  // [kN][128], once the ring has been read
  if (warp == 0 && lane == 0) {
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(smem_u32(&sh->empty[prod_stage]), prod_phase ^ 1, abort_flag)) {
        raise_abort(&sh->abort, err);
        break;
      }
      const uint32_t full = smem_u32(&sh->full[prod_stage]);
      const uint32_t a = smem_u32(base + prod_stage * kStageB);
      mbar_expect_tx(full, kTileA + box * ROW_BYTES);
      if (strided) {
        tma_load_2d(a, &tmap_w, row0, kb * 64, full);
        tma_load_2d(a + 8192, &tmap_w, row0 + 64, kb * 64, full);
      } else {
        tma_load_2d(a, &tmap_w, kb * 64, row0, full);
      }
      tma_load_2d(a + kTileA, &tmap_x, kb * 64, first_m, full);
      ++issued;
      if (++prod_stage == stages) {
        prod_stage = 0;
        prod_phase ^= 1;
      }
    }
  } else if (warp == 1 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0;
    const uint32_t idesc = operand_idesc(128, box, strided, false);
    const uint32_t step_a = k_step(strided);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(smem_u32(&sh->full[stage]), phase, abort_flag)) {
        raise_abort(&sh->abort, err);
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t a = smem_u32(base + stage * kStageB);
      const uint64_t a_desc = operand_desc(a, strided);
      const uint64_t b_desc = smem_desc_sw128(a + kTileA);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_one_rt(tmem_base, a_desc + step_a * kk, b_desc + 2 * kk, idesc,
                   (kb != kb0) || kk != 0);
      mma_commit(smem_u32(&sh->empty[stage]));
      if (++stage == stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (ok && kb1 > kb0) mma_commit(smem_u32(&sh->done));
  } else if (warp >= 2 && kb1 > kb0) {
    good = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh->done), 0, abort_flag));
    if (!good && lane == 0) raise_abort(&sh->abort, err);
    if (good) {
      tc_fence_after();
      const int quarter = warp & 3;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int m0 = 0; m0 < M; m0 += 16) {
        uint32_t r[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + m0));
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          part[(m0 + i) * 128 + quarter * 32 + lane] = __uint_as_float(r[i]);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (*abort_flag) {
    // let this CTA's own copies and MMAs land before its memory is released
    const int zero = 0;
    if (warp == 0 && lane == 0) {
      const int outstanding = issued < stages ? issued : stages;
      for (int i = 1; i <= outstanding; ++i) {
        int s = prod_stage - i;
        uint32_t ph = prod_phase;
        if (s < 0) {
          s += stages;
          ph ^= 1;
        }
        mbar_wait(smem_u32(&sh->full[s]), ph, &zero);
      }
    }
    if (warp == 1 && lane == 0) {
      mma_commit(smem_u32(&sh->done));
      mbar_wait(smem_u32(&sh->done), 0, &zero);
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  pdl_launch_dependents();
  join_parts(part, M, first_m, row0, rows, num_kb, log_splits, r, bias, ep);
  cluster.sync();  // partial tiles stay alive until every CTA has read them
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(few_cols<kN>)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// dot_kernel, M <= 4 (single tokens): CUDA cores, since the weight's stream is
// all there is and the tensor-core kernels' barriers, tensor memory and joins
// are latency.  A CTA takes kDotRows weight rows; its threads share their
// columns, so that every 16-byte load of a pass over up to 4096 columns is in
// flight at once and nothing is staged.  x comes from L2.
// ---------------------------------------------------------------------------
constexpr int kDotRows = 8;
constexpr int kDotMaxM = 4;

template <int kM, int kThreads>
__global__ void __launch_bounds__(kThreads)
    dot_kernel(const __nv_bfloat16 *__restrict__ x, int64_t ldx, const __nv_bfloat16 *__restrict__ w,
               int64_t ldw, int M, int N, int K, const Epilogue ep) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kSteps = kM > 2 ? 1 : 2;  // 16-byte loads of a row per thread and pass
  __shared__ float parts[kWarps][kDotRows * kM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * kDotRows;
  const int nvec = K / 8;
  pdl_wait();
  uint64_t acc[kDotRows][kM] = {};  // sums over even and odd columns
  for (int v0 = threadIdx.x; v0 < nvec; v0 += kSteps * kThreads) {
    uint4 a[kSteps][kDotRows], b[kSteps][kM];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int v = v0 + s * kThreads;
      const bool in = v < nvec;
#pragma unroll
      for (int r = 0; r < kDotRows; ++r)  // (rows past the last read it again)
        a[s][r] = in ? ld_stream_v4(w + min(row0 + r, N - 1) * ldw + v * 8)
                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int m = 0; m < kM; ++m)
        b[s][m] = in ? __ldg(reinterpret_cast<const uint4 *>(x + min(m, M - 1) * ldx) + v)
                     : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint64_t xf[kM][4];
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const uint32_t xb[4] = {b[s][m].x, b[s][m].y, b[s][m].z, b[s][m].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) xf[m][i] = pack_f32(bf16_lo(xb[i]), bf16_hi(xb[i]));
      }
#pragma unroll
      for (int r = 0; r < kDotRows; ++r) {
        const uint32_t wb[4] = {a[s][r].x, a[s][r].y, a[s][r].z, a[s][r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t wf = pack_f32(bf16_lo(wb[i]), bf16_hi(wb[i]));
#pragma unroll
          for (int m = 0; m < kM; ++m) acc[r][m] = fma2(wf, xf[m][i], acc[r][m]);
        }
      }
    }
  }
  pdl_launch_dependents();
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    // eight sums over the warp's lanes in nine exchanges: each of the first
    // three halves the sums a lane holds
    float t[kDotRows];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) {
      float lo, hi;
      unpack_f32(acc[r][m], lo, hi);
      t[r] = lo + hi;
    }
#pragma unroll
    for (int n = kDotRows / 2, bit = 16; n > 0; n /= 2, bit /= 2) {
      const bool upper = (lane & bit) != 0;
#pragma unroll
      for (int r = 0; r < n; ++r) {
        const float send = upper ? t[r] : t[n + r];
        t[r] = (upper ? t[n + r] : t[r]) + __shfl_xor_sync(0xffffffffu, send, bit);
      }
    }
    t[0] += __shfl_xor_sync(0xffffffffu, t[0], 2);
    t[0] += __shfl_xor_sync(0xffffffffu, t[0], 1);
    if ((lane & 3) == 0) parts[warp][(lane >> 2) * kM + m] = t[0];
  }
  __syncthreads();
  const int e = threadIdx.x;
  if (e >= kDotRows * kM) return;
  const int m = e / kDotRows, r = e % kDotRows;  // rows fastest: neighbouring results
  const int64_t col = row0 + r;
  if (m >= M || col >= N) return;
  float z = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) z += parts[i][r * kM + m];
  z += ld_bias(ep.bias, ep.bias_f32, col);
  if (ep.pre != nullptr) ep.pre[m * ep.ldp + col] = __float2bfloat16_rn(z);
  float y = activate(z, ep.act);
  if (ep.res != nullptr) y += ld_bf16(ep.res + m * ep.ldr + col);
  ep.out[m * ep.ldo + col] = __float2bfloat16_rn(y);
}

// ---------------------------------------------------------------------------
// dz = g * act'(z) in bf16 (dz nullable) and db = the column sums of dz in
// fp32, before the rounding (db nullable).  dz is rounded because the tensor cores
// take 16 bits from both operands: the products' error in the 2-norm is 0.0023, of
// which the rounding of the results alone is 0.0017; a second product of what the
// rounding leaves out would take the tensor time twice.  g and z are read once and dz
// written once: 8192 x 8192 73 us, 5.5 TB/s of a copy's 6.8, with four rows in flight a
// thread and 44 % of the warps.  A cluster covers a strip of columns, its CTAs
// contiguous ranges of rows; their column sums meet in the first CTA through
// distributed shared memory, in a fixed order, so db needs no second launch.
// A strip has 64 columns, or 32 or 16 where that leaves SMs idle; a thread takes
// eight columns of a row.  Rows of g and z that do not start on 16-byte
// boundaries (kAligned false) are put together from the aligned pieces that hold
// them (with two-byte loads the gradient of 3899 x 3205 x 536 took 109 us, so
// 71); a strip's columns at a row's ends, where such pieces would leave the row,
// go one by one.  4096 x 4096, tanh gelu: 19 us.
// ---------------------------------------------------------------------------
constexpr int kDzThreads = 256;
constexpr int kDzMaxSplits = 8;

// (A product of its own, not contracted into the column sum: db is the same
// whether dz is asked for or not.  relu chooses: what it cut off has no gradient,
// though g be infinite or NaN there; a NaN z stays one.)
template <int kAct>
__device__ __forceinline__ float dz_term(float g, float z) {
  if (kAct == SGA_ACT_NONE) return g;
  if (kAct == SGA_ACT_RELU) return z > 0.0f ? g : (z != z ? z : 0.0f);
  return __fmul_rn(g, activate_grad(z, kAct));
}

// Eight bf16 at p, and with kAligned false what surrounds them (see above).
template <bool kAligned>
struct Eight {
  uint4 a, b;
  int off;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    if (kAligned) {
      a = ld_stream_v4(p);
    } else {
      off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
      const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(p) - off);
      a = __ldg(q);
      b = __ldg(q + (off != 0 ? 1 : 0));
    }
  }
  __device__ __forceinline__ uint4 get() const { return kAligned ? a : bytes_of(a, b, off); }
};

template <int kAct, bool kAligned>
__global__ void __launch_bounds__(kDzThreads)
    dz_kernel(const __nv_bfloat16 *__restrict__ g, int64_t ldg,
              const __nv_bfloat16 *__restrict__ z, int64_t ldz, int M, int N, int cols, int splits,
              __nv_bfloat16 *__restrict__ dz, int64_t lddz, void *__restrict__ db, int f32) {
  constexpr int kBatch = kAligned ? 4 : 2;  // rows in flight per thread
  __shared__ float sums[kDzThreads * 8];  // [rows at once][cols]
  __shared__ float total[64];
  const int tid = threadIdx.x;
  const int lanes = cols / 8;  // threads per row: 8, 4 or 2
  const int rows_at_once = kDzThreads / lanes;
  const int split = static_cast<int>(blockIdx.x) % splits;
  const int strip = static_cast<int>(blockIdx.x) / splits;
  const int m0 = static_cast<int>(static_cast<int64_t>(M) * split / splits);
  const int m1 = static_cast<int>(static_cast<int64_t>(M) * (split + 1) / splits);
  const int r0 = tid / lanes;
  const int c0 = tid % lanes * 8;
  const int64_t col = static_cast<int64_t>(strip) * cols + c0;
  pdl_wait();
  float s[8] = {};
  if (kAligned ? col + 8 <= N : col >= 8 && col + 16 <= N) {
    for (int m = m0 + r0; m < m1; m += kBatch * rows_at_once) {
      Eight<kAligned> vg[kBatch], vz[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        // (a row past the end reads the last one again)
        const int64_t r = min(m + u * rows_at_once, m1 - 1);
        vg[u].load(g + r * ldg + col);
        if (kAct != SGA_ACT_NONE) vz[u].load(z + r * ldz + col);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int64_t r = m + u * rows_at_once;
        if (r >= m1) continue;
        const uint4 qg = vg[u].get();
        uint4 qz = qg;
        if (kAct != SGA_ACT_NONE) qz = vz[u].get();
        const uint32_t wg[4] = {qg.x, qg.y, qg.z, qg.w};
        const uint32_t wz[4] = {qz.x, qz.y, qz.z, qz.w};
        uint32_t wo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float d0 = dz_term<kAct>(bf16_lo(wg[i]), bf16_lo(wz[i]));
          const float d1 = dz_term<kAct>(bf16_hi(wg[i]), bf16_hi(wz[i]));
          s[2 * i] += d0;
          s[2 * i + 1] += d1;
          wo[i] = pack2(d0, d1);
        }
        if (dz != nullptr)
          *reinterpret_cast<uint4 *>(dz + r * lddz + col) = make_uint4(wo[0], wo[1], wo[2], wo[3]);
      }
    }
  } else if (col < N) {
    const int n = static_cast<int>(min(static_cast<int64_t>(8), N - col));
    for (int m = m0 + r0; m < m1; m += rows_at_once) {
      const __nv_bfloat16 *pg = g + m * ldg + col;
      const __nv_bfloat16 *pz = kAct != SGA_ACT_NONE ? z + m * ldz + col : pg;
      float vg[8], vz[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // (columns past the end read the last one again)
        vg[i] = ld_bf16(pg + min(i, n - 1));
        vz[i] = ld_bf16(pz + min(i, n - 1));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = dz_term<kAct>(vg[i], vz[i]);
        if (i < n) {
          s[i] += d;
          if (dz != nullptr) dz[m * lddz + col + i] = __float2bfloat16_rn(d);
        }
      }
    }
  }
  pdl_launch_dependents();
  if (db == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[r0 * cols + c0 + i] = s[i];
  __syncthreads();
  if (tid < cols) {
    float t = 0.0f;
#pragma unroll 8
    for (int r = 0; r < min(rows_at_once, m1 - m0); ++r) t += sums[r * cols + tid];
    total[tid] = t;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  if (split == 0 && tid < cols && strip * cols + tid < N) {
    float t = 0.0f;
    for (int i = 0; i < splits; ++i) t += cluster.map_shared_rank(total, i)[tid];
    const int c = strip * cols + tid;
    if (f32)
      static_cast<float *>(db)[c] = t;
    else
      static_cast<__nv_bfloat16 *>(db)[c] = __float2bfloat16_rn(t);
  }
  cluster.sync();  // the totals stay alive until they have been read
}

// ------------------------------------------------------------------ host

// Tensor map over a row-major bf16 [rows, cols] matrix with row stride ld;
// box = box_rows x 64 columns (one 128-byte swizzled row), zero fill outside.
bool make_map_ld(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld,
                 int box_rows) {
  auto encode = get_encode_fn();
  if (encode == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * 2)};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides,
                box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// One operand of a product: `other` (rows of D, or columns) x `summed`.
struct Operand {
  const void *ptr;
  int64_t ld;
  bool strided;  // the summed dimension is the strided one
};

struct Mat {  // D[rows, cols] = sum over `summed` of A B
  Operand a, b;
  int64_t rows, cols, summed;
  Epilogue ep;
};

bool operand_map(CUtensorMap *map, const Operand &o, int64_t other, int64_t summed, int box) {
  return o.strided ? make_map_ld(map, o.ptr, summed, other, o.ld, 64)
                   : make_map_ld(map, o.ptr, other, summed, o.ld, box);
}

// Length of a tile in K blocks: its own, at least what its epilogue takes, and
// the turn of the pipeline between tiles.
int64_t tile_cost(int num_kb) { return (num_kb > 12 ? num_kb : 12) + 2; }

uint32_t reciprocal(int d) {  // for quotient(); 2^32 / 1 does not fit, and is short by one too
  return static_cast<uint32_t>(d == 1 ? 0xffffffffu : (uint64_t(1) << 32) / d);
}

bool aligned_rows(const void *p, int64_t ld) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) | (2 * ld)) % 16 == 0;
}

template <int kBN>
cudaError_t launch_gemm(const Mat *mats, int n, int num_sms, uint32_t *err, cudaStream_t stream) {
  Maps maps = {};
  Products prods = {};
  for (int i = 0; i < n; ++i) {
    const Mat &m = mats[i];
    Product &p = prods.p[i];
    p.rows = static_cast<int>(m.rows);
    p.cols = static_cast<int>(m.cols);
    p.num_kb = static_cast<int>((m.summed + 63) / 64);
    p.tiles_r = static_cast<int>((m.rows + 255) / 256);
    p.tiles_c = static_cast<int>((m.cols + kBN - 1) / kBN);
    p.inv_band = reciprocal(kBand * p.tiles_c);
    p.inv_last = reciprocal(p.tiles_r % kBand != 0 ? p.tiles_r % kBand : kBand);
    p.a_strided = m.a.strided;
    p.b_strided = m.b.strided;
    p.ep = m.ep;
    prods.tiles[i] = p.tiles_r * p.tiles_c;
    if (!operand_map(&maps.a[i], m.a, m.rows, m.summed, 128) ||
        !operand_map(&maps.b[i], m.b, m.cols, m.summed, kBN / 2))
      return cudaErrorNotSupported;
    p.ep.aligned = aligned_rows(m.ep.out, m.ep.ldo) && aligned_rows(m.ep.pre, m.ep.ldp) &&
                   aligned_rows(m.ep.res, m.ep.ldr);
  }
  auto kern = gemm_kernel<kBN>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), gemm_smem<kBN>,
                                      kBN == 256 ? 0 : (kBN == 128 ? 1 : 2));
  if (e != cudaSuccess) return e;
  const int all = prods.tiles[0] + prods.tiles[1];
  const int pairs = num_sms / 2 < all ? num_sms / 2 : all;
  prods.lead = prods.tiles[0] % pairs;
  if (n > 1) {
    // the shortest end time for which the runs of product 1 fit: the lead pairs
    // take about what levels all, the others what is left
    const int64_t c0 = tile_cost(prods.p[0].num_kb), c1 = tile_cost(prods.p[1].num_kb);
    const int64_t q = prods.tiles[0] / pairs;
    const int64_t level = (prods.tiles[0] * c0 + prods.tiles[1] * c1) / pairs;
    const int64_t guess = (level - (q + 1) * c0) / c1;
    int64_t best = -1;
    for (int64_t a = guess > 1 ? guess - 1 : 0; a <= (guess > 0 ? guess : 0) + 2; ++a) {
      const int64_t rest = prods.tiles[1] - a * prods.lead;
      const int64_t b = rest <= 0 ? 0 : (rest + pairs - prods.lead - 1) / (pairs - prods.lead);
      const int64_t end_lead = prods.lead > 0 ? (q + 1) * c0 + a * c1 : 0;
      const int64_t end_rest = q * c0 + b * c1;
      const int64_t end = end_lead > end_rest ? end_lead : end_rest;
      if (best < 0 || end < best) {
        best = end;
        prods.run[0] = static_cast<int>(a);
        prods.run[1] = static_cast<int>(b);
      }
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = gemm_smem<kBN>;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, maps, prods, err);
}

// Columns of a tile: the widest that does not leave SMs idle.  A K block of a
// 256-column tile takes 280 ns, of a 128-column one 215 ns and of a 64-column
// one 200 ns (the copies and issues that a block needs whatever its width);
// the time of a width is the waves of pairs times the length of a tile.
struct Width {
  int index;
  int64_t ns;
};

Width pick_width(const Mat *mats, int n, int num_sms) {
  constexpr int widths[3] = {256, 128, 64};
  constexpr int64_t kb_ns[3] = {280, 215, 200};
  const int64_t pairs = num_sms / 2;
  bool strided = false;
  for (int i = 0; i < n; ++i) strided = strided || mats[i].b.strided;
  Width best = {0, 0};
  for (int w = 0; w < (strided ? 2 : 3); ++w) {
    int64_t work = 0, longest = 0;
    for (int i = 0; i < n; ++i) {
      const int64_t tiles =
          (mats[i].rows + 255) / 256 * ((mats[i].cols + widths[w] - 1) / widths[w]);
      const int64_t tile = tile_cost(static_cast<int>((mats[i].summed + 63) / 64)) * kb_ns[w];
      // one product alone: whole waves; two fill each other's last wave
      work += n == 1 ? (tiles + pairs - 1) / pairs * pairs * tile : tiles * tile;
      if (tile > longest) longest = tile;
    }
    const int64_t ns = work / pairs > longest ? work / pairs : longest;
    if (w == 0 || ns < best.ns) best = {w, ns};
  }
  return best;
}

cudaError_t launch_products(const Mat *mats, int n, int num_sms, uint32_t *err,
                            cudaStream_t stream) {
  switch (pick_width(mats, n, num_sms).index) {
    case 0: return launch_gemm<256>(mats, n, num_sms, err, stream);
    case 1: return launch_gemm<128>(mats, n, num_sms, err, stream);
    default: return launch_gemm<64>(mats, n, num_sms, err, stream);
  }
}

// Clusters of `splits` few_rows CTAs that run at once, at `per_sm` CTAs per SM: a
// cluster lies in one GPC, whose SMs are not all a multiple of it (152 SMs hold 36
// clusters of 4 or 15 of 8).
int64_t resident_clusters(int splits, int per_sm, int num_sms) {
  const int64_t ctas = static_cast<int64_t>(per_sm) * num_sms;
  if (splits < 4) return ctas / splits;
  return per_sm == 1 ? (splits == 4 ? ctas * 19 / 80 : ctas / 10)
                     : (splits == 4 ? ctas * 39 / 160 : ctas * 19 / 160);
}

// CTAs per tile of few_rows_kernel: while all of them are resident (two per SM;
// 128 x 4736 x 8192, 37 clusters of 8: 26.1 us, 36 of them 18.8; 96 x 9728 x 8192,
// 76 of 4: 44.5, 74 of them 30.3).  A CTA's share of K blocks may be one or none; it
// still takes its share of the results.  Eight only for a long sum, or the least rows
// (M x N x K, 4 / 8 CTAs: 64 x 4096 x 4096 11.8 / 12.6 us, 64 x 1024 x 8192 14.8 /
// 11.0, 16 x 2560 x 4096 9.1 / 8.0, 48 x 2560 x 8192 13.7 / 12.8), and with many rows
// only while there is one CTA per SM (128 x 2560 x 8192 16.3 / 18.1, 128 x 4096 x 8192
// 17.7 / 19.9, 16 x 4096 x 8192 14.9 / 13.4).
int few_splits(int64_t units, int num_kb, int64_t m, int num_sms) {
  const bool eight = m <= 16 ? num_kb >= 32 : num_kb >= 80 && (m <= 48 || units * 8 <= num_sms);
  const int most = eight ? 8 : 4;
  int splits = 1;
  while (splits < most && units <= resident_clusters(2 * splits, 2, num_sms) && num_kb >= splits)
    splits *= 2;
  return splits;
}

template <int kN>
cudaError_t launch_few_rows(const Mat &m, int num_sms, uint32_t *err, cudaStream_t stream) {
  // m: D^T, rows = weight rows, cols = M
  CUtensorMap map_w, map_x;
  // rows of x that a K block brings: no more than there are, in steps of the MMA
  const int box = m.cols < kN ? static_cast<int>((m.cols + 15) / 16 * 16) : kN;
  if (!operand_map(&map_w, m.a, m.rows, m.summed, 128) ||
      !operand_map(&map_x, m.b, m.cols, m.summed, box))
    return cudaErrorNotSupported;
  const int num_kb = static_cast<int>((m.summed + 63) / 64);
  const int blocks = static_cast<int>((m.cols + kN - 1) / kN);
  const int64_t units = (m.rows + 127) / 128 * blocks;
  const int splits = few_splits(units, num_kb, m.cols, num_sms);
  int log_splits = 0;
  while (1 << log_splits < splits) ++log_splits;
  const bool wide = units <= resident_clusters(splits, 1, num_sms) && num_kb >= 3 * few_stages<kN> * splits;
  const int stages = wide ? few_most_stages<kN> : few_stages<kN>;
  auto kern = few_rows_kernel<kN>;
  const cudaError_t e =
      set_smem_once(reinterpret_cast<const void *>(kern), few_smem<kN>(few_most_stages<kN>),
                    kN == 16 ? 3 : (kN == 32 ? 4 : (kN == 64 ? 5 : 6)));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = few_smem<kN>(stages);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, static_cast<int>(m.cols),
                            static_cast<int>(m.rows), num_kb, blocks, stages, log_splits, box,
                            static_cast<int>(m.a.strided), m.ep, err);
}

// Estimated time of a product as few_rows_kernel, over what gemm_kernel takes
// besides its K blocks: 330 ns a K block for each CTA of an SM (its copies), and
// 0.5 to 3 us, growing with the rows, to join the parts.
int64_t few_rows_ns(const Mat &m, int num_sms) {
  const int num_kb = static_cast<int>((m.summed + 63) / 64);
  const int64_t units = (m.cols + 127) / 128 * ((m.rows + 127) / 128);
  const int splits = few_splits(units, num_kb, m.rows, num_sms);
  const int64_t ctas = units * splits > num_sms ? units * splits : num_sms;
  const int64_t rows = m.rows < 128 ? m.rows : 128;
  return ctas * ((num_kb + splits - 1) / splits) * 330 / num_sms + 500 + rows * 20;
}

// Whether a product runs as few_rows_kernel: where its tiles, split over K, end
// sooner than the pairs' (measured, few rows / pairs: 96 x 4096 x 4096 11.0 /
// 16.6 us, 512 x 1024 x 8192 15.8 / 27.9, 96 x 512 x 512 6.5 / 5.4, 512 x 4096 x
// 1024 14.0 / 8.4).
bool few_rows_form(const Mat &m, int num_sms) {
  return !m.a.strided && m.rows <= 2048 &&
         few_rows_ns(m, num_sms) < pick_width(&m, 1, num_sms).ns;
}

// As few_rows_kernel: the weight becomes the row operand.
cudaError_t launch_few(const Mat &m, int num_sms, uint32_t *err, cudaStream_t stream) {
  const Mat t = {m.b, m.a, m.cols, m.rows, m.summed, m.ep};
  if (m.rows <= 16) return launch_few_rows<16>(t, num_sms, err, stream);
  if (m.rows <= 32) return launch_few_rows<32>(t, num_sms, err, stream);
  if (m.rows <= 64) return launch_few_rows<64>(t, num_sms, err, stream);
  return launch_few_rows<128>(t, num_sms, err, stream);
}

template <int kThreads>
cudaError_t launch_dot_threads(const Mat &m, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((m.cols + kDotRows - 1) / kDotRows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = m.rows == 1 ? dot_kernel<1, kThreads>
                          : (m.rows == 2 ? dot_kernel<2, kThreads> : dot_kernel<4, kThreads>);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const __nv_bfloat16 *>(m.a.ptr), m.a.ld,
                            static_cast<const __nv_bfloat16 *>(m.b.ptr), m.b.ld,
                            static_cast<int>(m.rows), static_cast<int>(m.cols),
                            static_cast<int>(m.summed), m.ep);
}

// Threads of a dot_kernel CTA: a quarter of a row's 16-byte vectors, 32 to 128
// (more idle in short rows, fewer wait longer in long ones), twice that where
// the CTAs are few.  Measured, 32 / 64 / 128 / 256 threads: 1 x 4096 x 4096 10.2
// / 7.9 / 7.0 / 8.3 us, 1 x 1024 x 8192 15.8 / 9.4 / 6.4 / 5.6, 1 x 16384 x 512
// 4.8 / 5.9 / 8.0 / 12.5, 1 x 152064 x 2048 85 / 85 / 87 / 130.
cudaError_t launch_dot(const Mat &m, cudaStream_t stream, int num_sms) {
  int threads = 32;
  while (threads < 128 && threads * 4 < m.summed / 8) threads *= 2;
  if ((m.cols + kDotRows - 1) / kDotRows < 2 * num_sms) threads *= 2;
  switch (threads) {
    case 32: return launch_dot_threads<32>(m, stream);
    case 64: return launch_dot_threads<64>(m, stream);
    case 128: return launch_dot_threads<128>(m, stream);
    default: return launch_dot_threads<256>(m, stream);
  }
}

// Whether a product of at most four rows runs as dot_kernel.  With more than one
// row its reads of x from L2 weigh on a large weight of long rows (few_rows_kernel
// / dot_kernel: 4 x 8192 x 8192 24.4 / 30.6 us, 4 x 2048 x 2048 6.5 / 4.6, 4 x
// 152064 x 2048 149 / 118).
bool dot_form(const Mat &m) {
  return m.rows == 1 || (m.rows <= kDotMaxM &&
                         (m.summed <= 2048 || m.cols * m.summed <= (int64_t(1) << 23)));
}

int64_t dz_ld(int64_t N) { return (N + 7) / 8 * 8; }

template <int kAct>
cudaError_t launch_dz(const __nv_bfloat16 *g, int64_t ldg, const __nv_bfloat16 *z, int64_t ldz,
                      int64_t M, int64_t N, __nv_bfloat16 *dz, void *db, bool f32, int num_sms,
                      cudaStream_t stream) {
  uintptr_t bits = reinterpret_cast<uintptr_t>(g) | (2 * ldg);
  if (kAct != SGA_ACT_NONE) bits |= reinterpret_cast<uintptr_t>(z) | (2 * ldz);
  const bool aligned = bits % 16 == 0;
  int splits = 1;  // 32 rows or more per CTA
  while (splits < kDzMaxSplits && M >= 64 * splits) splits *= 2;
  int cols = 64;
  while (cols > 16 && M > 256 && (N + cols - 1) / cols * splits < 3 * num_sms) cols /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((N + cols - 1) / cols * splits));
  cfg.blockDim = dim3(kDzThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto kern = aligned ? dz_kernel<kAct, true> : dz_kernel<kAct, false>;
  return cudaLaunchKernelEx(&cfg, kern, g, ldg, z, ldz, static_cast<int>(M), static_cast<int>(N),
                            cols, splits, dz, dz_ld(N), db, static_cast<int>(f32));
}

}  // namespace

cudaError_t launch_linear(const void *x, int64_t M, int64_t K, int64_t ldx, const void *weight,
                          int64_t N, int64_t ldw, const void *bias, int bias_dtype, int act,
                          const void *residual, int64_t ldr, void *preact, int64_t ldp, void *out,
                          int64_t ldo, int num_sms, uint32_t *err, cudaStream_t stream) {
  Mat m = {};
  m.a = {x, ldx, false};
  m.b = {weight, ldw, false};
  m.rows = M;
  m.cols = N;
  m.summed = K;
  m.ep = {static_cast<__nv_bfloat16 *>(out), static_cast<__nv_bfloat16 *>(preact),
          static_cast<const __nv_bfloat16 *>(residual), bias, ldo, ldp, ldr,
          bias_dtype == SGA_F32, act};
  if (dot_form(m)) return launch_dot(m, stream, num_sms);
  return few_rows_form(m, num_sms) ? launch_few(m, num_sms, err, stream)
                                   : launch_products(&m, 1, num_sms, err, stream);
}

size_t linear_grad_workspace_bytes(int64_t M, int64_t N) {
  return static_cast<size_t>((M * dz_ld(N) * 2 + 15) / 16 * 16);
}

cudaError_t launch_linear_grad(const void *grad_out, int64_t M, int64_t N, int64_t ldg,
                               const void *preact, int64_t ldp, int act, const void *x, int64_t K,
                               int64_t ldx, const void *weight, int64_t ldw, void *grad_x,
                               int64_t ldgx, void *grad_weight, int64_t ldgw, void *grad_bias,
                               int bias_dtype, void *workspace, int num_sms, uint32_t *err,
                               cudaStream_t stream) {
  // dz lies where g lies when there is nothing to multiply and TMA can read it
  const bool direct =
      act == SGA_ACT_NONE && ldg % 8 == 0 && reinterpret_cast<uintptr_t>(grad_out) % 16 == 0;
  const bool products = grad_x != nullptr || grad_weight != nullptr;
  auto *dz = static_cast<__nv_bfloat16 *>(workspace);
  cudaError_t e;
  if ((products && !direct) || grad_bias != nullptr) {
    decltype(&launch_dz<SGA_ACT_NONE>) const launch[] = {
        launch_dz<SGA_ACT_NONE>, launch_dz<SGA_ACT_RELU>, launch_dz<SGA_ACT_SILU>,
        launch_dz<SGA_ACT_GELU>, launch_dz<SGA_ACT_GELU_TANH>};
    e = launch[act](static_cast<const __nv_bfloat16 *>(grad_out), ldg,
                    static_cast<const __nv_bfloat16 *>(preact), ldp, M, N,
                    products && !direct ? dz : nullptr, grad_bias, bias_dtype == SGA_F32, num_sms,
                    stream);
    if (e != cudaSuccess) return e;
  }
  const Operand d = direct ? Operand{grad_out, ldg, false} : Operand{dz, dz_ld(N), false};
  Mat dx = {}, dw = {};
  dx.a = d;
  dx.b = {weight, ldw, true};
  dx.rows = M;
  dx.cols = K;
  dx.summed = N;
  dx.ep.out = static_cast<__nv_bfloat16 *>(grad_x);
  dx.ep.ldo = ldgx;
  dw.a = {d.ptr, d.ld, true};
  dw.b = {x, ldx, true};
  dw.rows = N;
  dw.cols = K;
  dw.summed = M;
  dw.ep.out = static_cast<__nv_bfloat16 *>(grad_weight);
  dw.ep.ldo = ldgw;
  const Mat both[2] = {dx, dw};
  // grad_x and grad_weight share a launch unless grad_x as few_rows_kernel, a
  // launch of its own (5 us more), ends sooner.  (Decided as if both were asked
  // for: the forms add up in different orders.)
  const bool few =
      M <= 2048 && few_rows_ns(dx, num_sms) + pick_width(&dw, 1, num_sms).ns + 5000 <
                       pick_width(both, 2, num_sms).ns;
  if (grad_x != nullptr && few) {
    e = launch_few(dx, num_sms, err, stream);
    if (e != cudaSuccess) return e;
  }
  const bool with_x = grad_x != nullptr && !few;
  if (with_x && grad_weight != nullptr) return launch_products(both, 2, num_sms, err, stream);
  if (with_x) return launch_products(&dx, 1, num_sms, err, stream);
  return grad_weight != nullptr ? launch_products(&dw, 1, num_sms, err, stream) : cudaSuccess;
}

}  // namespace sga
