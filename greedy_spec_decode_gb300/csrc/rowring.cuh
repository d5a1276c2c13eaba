// rowring.cuh -- rows of logits held in the shared memory of a cluster, shared by
// probs.cu and distill.cu: what a row is split into, the ring that a copy warp
// fills, the running sum of exponentials, and the exchange of a row's pieces.
//
// Both kernels read a row twice, for its sum and then to write something of each
// of its logits.  A cluster of CTAs (one for short rows) shares a row, and each
// keeps its piece in a ring of stages until it has been written: the logits come
// from HBM once.  Summing and writing are done by warps of their own, so that one
// row is summed while another is written and a third is loaded (in turns by the
// same warps, two CTAs per SM: probabilities of 2048 x 202048 bf16 460 us instead of
// 382, loss and gradient of 4096 x 152064 bf16 651 instead of 391).  A piece with more
// stages than the ring keeps its last ones; the others are loaded a second time (in
// which order, and who frees a slot: ringorder.h).
#pragma once

#include <mutex>
#include <type_traits>

#include "pipe.cuh"
#include "ringorder.h"
#include "scan.cuh"

namespace sga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kVecPerThread = 4;  // 16-byte vectors of a stage per thread
constexpr int kMaxCluster = 8;
template <int kT>
constexpr int kStageVec = kT * kVecPerThread;
constexpr int kMaxSlots = 13;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float nan_f32() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bytes kS .. kS + 15 (kS even, below 16) of two 16-byte pieces that follow each other.
template <int kS>
__device__ __forceinline__ uint4 shifted(const uint4 a, const uint4 b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  constexpr int i = kS / 4;
  if constexpr (kS % 4 == 0) return make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  return make_uint4(__funnelshift_r(w[i], w[i + 1], 16), __funnelshift_r(w[i + 1], w[i + 2], 16),
                    __funnelshift_r(w[i + 2], w[i + 3], 16),
                    __funnelshift_r(w[i + 3], w[i + 4], 16));
}

// f with the shift that an output's alignment needs, in steps of kStep bytes below 16,
// as a constant (loss and gradient of 333 x 50257 fp32 ids into rows of another
// alignment: 36 us with the shift as a variable, 32 so, 29 at the same alignment).
template <int kStep, int kS = kStep, class F>
__device__ __forceinline__ void with_shift(int s, F &&f) {
  if constexpr (kS < 16) {
    if (s == kS)
      f(std::integral_constant<int, kS>{});
    else
      with_shift<kStep, kS + kStep>(s, f);
  }
}

template <int kT>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kT) : "memory");
}

// ------------------------------------------------------------------ pieces

// A CTA's piece of a row: columns [c0, c1), of which [b0, b1) are whole 16-byte
// vectors (loaded in stages) and at most seven at either end of the row are not.
struct Piece {
  const char *p;
  int c0, b0, b1, c1, stages;
};

template <bool kBf16, int kT>
__device__ __forceinline__ Piece piece_of(const char *p, int valid, int chunk, int chunks) {
  constexpr int kElt = kBf16 ? 2 : 4, kVec = 16 / kElt;
  Piece q;
  q.p = p;
  int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / kElt);
  if (head > valid) head = valid;
  const uint32_t nvec = static_cast<uint32_t>((valid - head) / kVec);  // <= 2^22, chunks <= 2^9
  const int v0 = static_cast<int>(nvec * chunk / chunks);
  const int v1 = static_cast<int>(nvec * (chunk + 1) / chunks);
  q.b0 = head + v0 * kVec;
  q.b1 = head + v1 * kVec;
  q.c0 = chunk == 0 ? 0 : q.b0;
  q.c1 = chunk == chunks - 1 ? valid : q.b1;
  q.stages = (v1 - v0 + kStageVec<kT> - 1) / kStageVec<kT>;
  return q;
}

// Column of the single element that a thread takes at one end (0: before b0, 1:
// from b1) of its piece, or -1.
__device__ __forceinline__ int end_column(const Piece &q, int side, int tid) {
  const int j = (side == 0 ? q.c0 : q.b1) + tid;
  return j < (side == 0 ? q.b0 : q.c1) ? j : -1;
}

// What a CTA goes over: every step-th row from `first`, its chunk of each (the CTAs of
// a cluster share rows), or every step-th piece of all rows' `chunks` pieces.
template <bool kPieces>
struct Walk {
  int64_t first, step;
  uint32_t n;
  int chunks, chunk;
  __device__ __forceinline__ int64_t row(uint32_t it) const {
    const int64_t i = first + it * step;
    return kPieces ? static_cast<uint32_t>(i) / static_cast<uint32_t>(chunks) : i;
  }
  __device__ __forceinline__ int chunk_of(uint32_t it) const {
    return kPieces ? static_cast<int>(static_cast<uint32_t>(first + it * step) %
                                     static_cast<uint32_t>(chunks))
                  : chunk;
  }
};

template <bool kPieces>
__device__ __forceinline__ Walk<kPieces> walk_of(int64_t rows, int chunks) {
  Walk<kPieces> w;
  const int64_t all = kPieces ? rows * chunks : rows;  // (pieces: at most 2^30)
  w.first = kPieces ? blockIdx.x : blockIdx.x / chunks;
  w.step = kPieces ? gridDim.x : gridDim.x / chunks;
  w.n = static_cast<uint32_t>(w.first < all ? (all - w.first + w.step - 1) / w.step : 0);
  w.chunks = chunks;
  w.chunk = kPieces ? 0 : static_cast<int>(blockIdx.x % chunks);
  return w;
}

// -------------------------------------------------------------------- ring

struct Ring {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int abort;
};

// A sum warp has seen a load of a kept row (and read it): its part in freeing the slot.
__device__ __forceinline__ void sum_frees(Ring &ring, const Place &at, int load, int stages,
                                          int slots, int lane) {
  __syncwarp();
  if (lane < sum_arrivals(load, stages, slots)) mbar_arrive(smem_u32(&ring.empty[at.slot]));
}

// bulk_load of what is read once: first to leave L2.  (Rows that are not kept: loss of
// 4096 x 152064 bf16 ids 174.7 -> 173.1 us, the gradient alone of 4096 x 32000 88.5 -> 84, of
// 2048 x 200064 263 -> 255; of rows that are, it makes loss and gradient of 4096 x 152064
// 13 us slower.)
__device__ __forceinline__ void bulk_load_once(uint32_t dst, const void *src, uint32_t bytes,
                                               uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// The copy warp: the stages of `num_its` pieces into the ring.  load(it, q) says which is
// the it-th, and how often its stages are loaded in all (those past the last one are the
// first again).  What is loaded once is first to leave L2.
template <bool kBf16, int kT, class F>
__device__ __forceinline__ void copy_rows(Ring &ring, uint4 *buf, int slots, bool kept,
                                          uint32_t num_its, F &&load, int lane, uint32_t *err) {
  constexpr int kElt = kBf16 ? 2 : 4, kVec = 16 / kElt;
  const volatile int *abort_flag = &ring.abort;
  Place at = {0, 0};
  int filled = 0;
  bool ok = true;
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  for (uint32_t it = 0; it < num_its && ok; ++it) {
    Piece q;
    const int loads = load(it, q);
    for (int j = 0; j < loads; ++j) {
      if (filled < slots) {
        ++filled;
      } else if (!warp_wait(smem_u32(&ring.empty[at.slot]), at.phase ^ 1, abort_flag)) {
        if (lane == 0) raise_abort(&ring.abort, err);
        ok = false;
        break;
      }
      if (elect_one()) {
        const int c = q.b0 + (j < q.stages ? j : j - q.stages) * kStageVec<kT> * kVec;
        const uint32_t bytes = static_cast<uint32_t>(min(kStageVec<kT> * kVec, q.b1 - c)) * kElt;
        mbar_expect_tx(smem_u32(&ring.full[at.slot]), bytes);
        const uint32_t dst = smem_u32(buf + at.slot * kStageVec<kT>);
        const char *src = q.p + static_cast<int64_t>(c) * kElt;
        if (kept || loads > q.stages)
          bulk_load(dst, src, bytes, smem_u32(&ring.full[at.slot]));
        else
          bulk_load_once(dst, src, bytes, smem_u32(&ring.full[at.slot]), policy);
      }
      __syncwarp();
      step(at, slots);
    }
  }
  // every copy has landed before the CTA ends
  const int zero = 0;
  for (int i = 0; i < filled; ++i) {
    if (at.slot == 0) {
      at.slot = slots;
      at.phase ^= 1;
    }
    --at.slot;
    pipe_wait(smem_u32(&ring.full[at.slot]), at.phase, &zero);
  }
}

// --------------------------------------------------- sum of exponentials

// A thread's running sum of 2^((x - m) scale), in two halves; m is one of its
// logits, moved up when a logit passes `limit` (2^12 above it; -inf: there is
// none yet, m = 0).  The difference is taken before it is scaled, so neither
// offset nor scale of the logits costs accuracy or range.
struct RunSum {
  float m, limit;
  uint64_t s;
};

__device__ __forceinline__ float sum_total(const RunSum &a) {
  float lo, hi;
  unpack_f32(a.s, lo, hi);
  return lo + hi;
}

// Before logits whose maximum is `most` join.
__device__ __forceinline__ void sum_rebase(RunSum &a, float most, float scale, float room) {
  if (!(most > a.limit)) return;
  const float s = sum_total(a);
  a.s = pack_f32(s == 0.0f ? 0.0f : s * ex2((a.m - most) * scale), 0.0f);
  a.m = most;
  a.limit = most + room;
}

__device__ __forceinline__ void sum_add(RunSum &a, float lo, float hi, float scale) {
  const uint64_t t = mul2(add2(pack_f32(lo, hi), pack_f32(-a.m, -a.m)), pack_f32(scale, scale));
  float t0, t1;
  unpack_f32(t, t0, t1);
  a.s = add2(a.s, pack_f32(ex2(t0), ex2(t1)));
}

template <bool kBf16>
__device__ __forceinline__ void sum_vector(RunSum &a, const uint4 q, float scale) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum_add(a, bf16_lo(w[i]), bf16_hi(w[i]), scale);
  } else {
    sum_add(a, __uint_as_float(w[0]), __uint_as_float(w[1]), scale);
    sum_add(a, __uint_as_float(w[2]), __uint_as_float(w[3]), scale);
  }
}

// The larger of each pair of logits of two vectors (NaN wins).
template <bool kBf16>
__device__ __forceinline__ uint4 vec_larger(const uint4 a, const uint4 b) {
  auto larger = [](uint32_t x, uint32_t y) {
    return kBf16 ? max_nan_bf16x2(x, y)
                 : __float_as_uint(max_nan(__uint_as_float(x), __uint_as_float(y)));
  };
  return make_uint4(larger(a.x, b.x), larger(a.y, b.y), larger(a.z, b.z), larger(a.w, b.w));
}

// A sum and its reference; one without terms has m = -inf, s = 0.  A NaN in
// either row stays in the sum.
struct Sum {
  float m, s;
};

__device__ __forceinline__ Sum sum_result(const RunSum &a) {
  return {a.limit == neg_inf() ? neg_inf() : a.m, sum_total(a)};
}

__device__ __forceinline__ float sum_at(const Sum &a, float m, float scale) {
  return a.s == 0.0f ? 0.0f : a.s * ex2((a.m - m) * scale);
}

__device__ __forceinline__ Sum sum_merge(const Sum &a, const Sum &b, float scale) {
  const float m = fmaxf(a.m, b.m);
  return {m, sum_at(a, m, scale) + sum_at(b, m, scale)};
}

// Over groups of kN lanes of a warp.
template <int kN = 32>
__device__ __forceinline__ Sum sum_warp(Sum a, float scale) {
  float m = a.m;
#pragma unroll
  for (int off = kN / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float s = sum_at(a, m, scale);
#pragma unroll
  for (int off = kN / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return {m, s};
}

// ---------------------------------------------------------------- exchange

// What the CTAs of a cluster tell each other about their it-th row, 16 bytes each,
// by turns in kN buffers.
template <int kN>
struct Exchange {
  uint64_t bar[kN];
  alignas(16) uint4 part[kN][kMaxCluster];
};

template <int kN>
__device__ __forceinline__ void exchange_init(Exchange<kN> &ex, int chunks) {
  for (int i = 0; i < kN; ++i) {
    mbar_init(smem_u32(&ex.bar[i]), 1);
    mbar_expect_tx(smem_u32(&ex.bar[i]), static_cast<uint32_t>(chunks) * 16);
  }
}

__device__ __forceinline__ void st_async(uint32_t addr, const uint4 v, uint32_t bar, int rank) {
  uint32_t a, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(bar), "r"(rank));
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(a),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(b)
      : "memory");
}

// One warp tells every CTA (its own too).
template <int kN>
__device__ __forceinline__ void exchange_tell(Exchange<kN> &ex, uint32_t it, const uint4 mine,
                                              int chunk, int chunks, int lane) {
  if (lane < chunks)
    st_async(smem_u32(&ex.part[it % kN][chunk]), mine, smem_u32(&ex.bar[it % kN]), lane);
  __syncwarp();
}

template <int kN>
__device__ __forceinline__ bool exchange_wait(Exchange<kN> &ex, uint32_t it,
                                              const volatile int *abort_flag) {
  return warp_wait(smem_u32(&ex.bar[it % kN]), (it / kN) & 1, abort_flag);
}

// The buffer's next use; by one warp that has waited for this one.
template <int kN>
__device__ __forceinline__ void exchange_rearm(Exchange<kN> &ex, uint32_t it, int chunks, int lane) {
  if (lane == 0) mbar_expect_tx(smem_u32(&ex.bar[it % kN]), static_cast<uint32_t>(chunks) * 16);
}

// The sum of the parts, whose first two words are a Sum (in every lane; the same in
// every CTA).
template <int kN>
__device__ __forceinline__ Sum exchange_sum(const Exchange<kN> &ex, uint32_t it, int chunks,
                                            int lane, float scale) {
  Sum s = {neg_inf(), 0.0f};
  const int c = lane % kMaxCluster;
  if (c < chunks) {
    const uint4 q = ex.part[it % kN][c];
    s = {__uint_as_float(q.x), __uint_as_float(q.y)};
  }
  return sum_warp<kMaxCluster>(s, scale);
}

// The end of a kernel: no CTA ends while another may write to it.  After a wait that
// gave up, what was told may still be on its way (some us).
__device__ __forceinline__ void leave(const Ring &ring, int chunks) {
  __syncwarp();
  if (chunks > 1)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  if (*static_cast<const volatile int *>(&ring.abort) != 0) {
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000) {
    }
  }
}

// ------------------------------------------------------------------- host

// A kernel of this kind and how it is launched.
struct RowKernel {
  const void *kern;
  int threads, smem;  // dynamic shared memory
  int slot;           // of this file's kernels, 0 .. 13
};

constexpr int kWidths[6] = {8, 6, 4, 3, 2, 1};  // CTAs that may share a row

// Clusters of each width that run at once (a cluster lies in one GPC, whose SMs are
// not all a multiple of it: of 152 SMs 8 x 15, 6 x 23, 4 x 36, 3 x 46, 2 x 76, or with
// two CTAs per SM 36, 46, 74, 97, 152).  A grid with more would leave its last clusters
// a second round.  Asked once per device.
inline cudaError_t resident_clusters(const RowKernel &k, int64_t (&out)[6]) {
  struct Entry {
    uintptr_t ctx;
    int n[6];
  };
  static std::mutex mu;
  static Entry cache[14][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const uintptr_t ctx = current_context_key();
  std::lock_guard<std::mutex> lock(mu);
  Entry &c = cache[k.slot][dev];
  if (ctx == 0 || c.ctx != ctx) {
    e = cudaFuncSetAttribute(k.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 6; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(kWidths[i]));
      cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
      cfg.dynamicSmemBytes = k.smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = kWidths[i];
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&c.n[i], k.kern, &cfg);
      if (e != cudaSuccess) return e;
    }
    c.ctx = current_context_key();
  }
  for (int i = 0; i < 6; ++i) out[i] = c.n[i] > 0 ? c.n[i] : 1;
  return cudaSuccess;
}

// The launch of rows, `chunks` CTAs each, as a persistent grid.
inline void row_launch(const RowKernel &k, int64_t rows, int chunks, const int64_t (&resident)[6],
                       cudaStream_t stream, cudaLaunchAttribute (&attr)[2],
                       cudaLaunchConfig_t &cfg) {
  int64_t n = rows;
  for (int i = 0; i < 6; ++i)
    if (kWidths[i] == chunks && resident[i] < n) n = resident[i];
  cfg.gridDim = dim3(static_cast<unsigned>(n * chunks));
  cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = chunks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Many rows of up to 48 KB: small CTAs, several per SM, a row each.  4096 rows of 1000 /
// 8000 / 16000 / 24000 bf16 ids, small and wide, graphs of 20 calls: probabilities 13.5 / 34 /
// 69 / 105 us and 44 / 51 / 66 / 99; loss and gradient 23 / 37 / 57 / 79 and 69 / 67 / 83 / 93;
// loss 18.9 / 21.7 / 29.7 / 38.7 and 23.3 / 24.4 / 31.2 / 37.7; gradient alone 19.4 / 27.4 / 46.8 /
// 67 and 21.9 / 28.6 / 45.7 / 65.  (One border for all four: between 32 and 48 KB the wide CTAs
// are up to 6 % faster but for loss and gradient together.)
inline bool small_rows(int64_t rows, int64_t bytes, int num_sms) {
  return bytes <= (48 << 10) && rows > 2 * num_sms;
}

// CTAs that share a row: the width with the least rounds of rows x time of a piece, in
// bytes, 16 KB standing for what a row costs besides (pieces of 4 KB or more).  With
// rows kept in a ring of `ring` bytes per CTA a piece leaves some of it for the next
// row's loads, unless there is one round, and clusters of 4 or 8 cost more than their
// share of the SMs says.  Graphs of 20 calls, 1 / 2 / 3 / 4 CTAs: probabilities of 2048 rows of
// 202048 bf16 ids 452 / 393 / 382 / 390 us, of 96 of 200064 28.7 / 29.9 / 28.3 / 22.4, of 333 of
// 50257 fp32 ids 32.3 / 26.0 / 27.4 / 28.5; loss and gradient of 4096 of 152064 bf16 ids 415 / 391 /
// - / 420, of 333 of 50257 fp32 33.7 / 29.3 / - / 33.8.  Without a ring (0) a row is split only
// if all run at once (loss of 333 rows of 50257 fp32 ids 14.0 / 14.9 / - / 15.9).
inline int pick_chunks(int64_t rows, int64_t bytes, int64_t ring, const int64_t (&resident)[6]) {
  int best = kMaxCluster;
  int64_t least = INT64_MAX;
  for (int i = 0; i < 6; ++i) {
    const int c = kWidths[i];
    const int64_t rounds = (rows + resident[i] - 1) / resident[i], piece = bytes / c;
    if (c > 1 && (piece < 4096 || (ring == 0 && rounds > 1))) continue;
    int64_t cost = rounds * (piece + 16384);
    if (c % 4 == 0 && rounds > 1) cost += cost / 16;
    if (ring > 0 && 10 * piece > 7 * ring) cost += cost / 12;
    if (ring > 0 && (rounds > 1 ? 10 * piece > 9 * ring : 4 * piece > 5 * ring)) cost *= 4;
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

}  // namespace
}  // namespace sga
