// logprobs.cu -- log probabilities of given tokens over (shards of) a
// vocabulary, with the entropy and the best alternatives of each row, and
// their gradient with respect to the logits.
//
// With x the row's logits, lse = log sum_j e^x_j and p_j = e^(x_j - lse):
//   logprob = x_token - lse,  entropy = lse - sum_j p_j x_j,
//   alternatives: the top_k ids in the argmax order, each with x - lse.
// One pass over the row keeps, relative to a reference r near the maximum,
//   sum = sum_j 2^(x_j log2e - r)  and  wsum = sum_j (x_j log2e - r) 2^(...),
// so that lse = ln2 (r + log2 sum) and entropy = ln2 (log2 sum - wsum / sum);
// two such triples merge by rescaling one to the other's reference, which is
// how threads and warps are joined.  Once a row's maximum is known its pieces
// are restated relative to that maximum (sga_logprob_part), which is how CTAs
// and vocab shards are joined.
#include <cooperative_groups.h>

#include "pipe.cuh"
#include "scan.cuh"

namespace cg = cooperative_groups;

namespace sga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Logits below kLow count as kLow in the fast pass (their terms are zero
// there); a row whose maximum lies outside +-kFastMax takes the exact pass.
constexpr float kLow = -8.507059e37f;  // -2^126
constexpr float kUnset = -1e6f;
constexpr float kFastMax = 5e5f;
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// A row's running statistics relative to the base-2 reference r.
struct Lse {
  float r, s, w;
};

// The same sums relative to r >= a.r (or with a empty, s == 0):
// sum (t + d) 2^(t + d) = 2^d (w + d s); what vanishes contributes 0.
__device__ __forceinline__ void lse_restate(Lse &a, float r) {
  const float d = a.r - r;
  const float f = a.s == 0.0f ? 0.0f : ex2(d);
  a.w = f == 0.0f ? 0.0f : f * fmaf(d, a.s, a.w);
  a.s = f * a.s;
  a.r = r;
}

// ---------------------------------------------------------------- forward
// HBM-bound, with little issue to spare: 4096 x 202048 bf16 231 us without
// alternatives (7.2 TB/s), 265 with 5, 308 with 20; 2048 x 202048 fp32 229, 239,
// 345; one row of 152064 3.8 us without and 7.7 with 20, latency.  The 2^x of every
// logit and the packed fp32 sums take 65 % of the issue slots, which is why the
// reference is only moved when it has to be and candidates are tested a vector at a
// time.
//
// A row is read once through a shared-memory ring (cp.async.bulk by a copy
// warp; the row's unaligned ends element by element), three stages of 16 KB in
// each of three CTAs per SM.  CTAs are persistent and the copy warp runs on into
// the next row while a row is being finished.  Few rows: a cluster of `chunks`
// CTAs shares a row and its first CTA joins the pieces through distributed shared
// memory (one launch, no workspace).
//
// Alternatives.  A sorted list kept while streaming costs a serial insertion
// for every element that enters it (measured: 4096 x 202048 bf16, 5
// alternatives 809 us against 278 without).  Instead a threshold is taken
// from what the ring holds at first (24576 bf16 ids): the top_k-th largest of
// the maxima of 64 groups of threads, which at least top_k elements reach.
// Vectors that reach it go to a candidate buffer (some tens to hundreds of
// 25000), from which the top_k are selected at the end by counting, on 64-bit
// keys that order (value, id) pairs.  -inf is never a candidate: where fewer than
// top_k elements are above it, the lowest masked ids fill the list.  If the
// buffer overflows the piece is read again: for what lies above the threshold,
// the lowest ids that equal it filling up (rows with very many equal values),
// and if that overflows too with per-warp sorted lists (rows that keep rising).
constexpr int kGroups = 64;
constexpr int kVecPerThread = 4;  // 16-byte vectors of a ring stage per thread
constexpr int kRing = 3;
constexpr int kMaxChunks = 8;
constexpr int kMaxWarps = 8;

struct RowOut {
  // final results (nullable each), or with part set the shard's statistics
  float *logprob, *entropy, *lse, *top_logprobs;
  int32_t *top_ids;
  sga_logprob_part *part;
  sga_stat *top;
};

using Key = unsigned long long;

// Unsigned order of the values of the argmax order (NaN above +inf, +0 == -0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 becomes +0
  if (is_nan(v)) return 0xffffffffu;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float order_value(uint32_t o) {
  if (o == 0xffffffffu) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// Key of a (value, id) pair: the argmax order, larger is better; 0 is no pair.
__device__ __forceinline__ Key pair_key(float v, int32_t id) {
  return (static_cast<Key>(order_key(v)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}
__device__ __forceinline__ float key_value(Key k) {
  return k == 0 ? neg_inf() : order_value(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int32_t key_id(Key k) {
  return k == 0 ? kNoId : static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(k));
}

// Sums of a piece relative to its maximum (sga_logprob_part).
struct Stats {
  float max, s, w;
};

template <int kT>
struct PieceShared {
  static constexpr int kVecs = 2 * kT;  // candidate vectors
  static constexpr int kKeys = 4 * kT;  // candidate elements
  uint64_t full[kRing], empty[kRing];
  int abort, num_vecs, num_keys;
  uint32_t threshold;
  float sum, wsum;
  Stats piece[kMaxChunks];  // the row's pieces, in its first CTA
  Lse warp_lse[kMaxWarps];
  float warp_max[kMaxWarps];
  alignas(16) uint32_t group[kGroups];
  alignas(16) uint4 vec[kVecs];
  int32_t vec_id[kVecs];
  alignas(16) Key key[kKeys];
  alignas(16) Key list[kMaxWarps * SGA_MAX_TOP];     // lists of warps
  alignas(16) Key pieces[kMaxChunks * SGA_MAX_TOP];  // lists of the row's pieces, in its first CTA
  Key best[SGA_MAX_TOP];
};
template <int kT>
constexpr int ring_bytes = kRing * kT * kVecPerThread * 16;

// A warp's best keys so far: lane i holds the i-th.
__device__ __forceinline__ void top_offer(Key &t, Key x, int lane, int k) {
  Key kth = __shfl_sync(0xffffffffu, t, k - 1);
  unsigned m = __ballot_sync(0xffffffffu, x > kth);
  while (m != 0) {
    const int src = __ffs(m) - 1;
    m &= m - 1;
    const Key v = __shfl_sync(0xffffffffu, x, src);
    if (v <= kth) continue;
    const int pos = __popc(__ballot_sync(0xffffffffu, t > v));
    const Key up = __shfl_up_sync(0xffffffffu, t, 1);
    if (lane > pos)
      t = up;
    else if (lane == pos)
      t = v;
    kth = __shfl_sync(0xffffffffu, t, k - 1);
  }
}

// The number of keys[0 .. n) above `mine`; n is rounded up to even, the entry
// past an odd end has to be 0.
__device__ __forceinline__ int keys_above(const Key *keys, int n, Key mine) {
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2 *>(keys + j);
    rank += o.x > mine;
    rank += o.y > mine;
  }
  return rank;
}

// The reported log probability of a logit.
__device__ __forceinline__ float to_logprob(float x, float lse) {
  return x == neg_inf() ? (is_nan(lse) ? lse : x) : x - lse;
}

// lse and entropy from the sums relative to the row's maximum.
__device__ __forceinline__ void finish_row(float max, float s, float w, float &lse,
                                           float &entropy) {
  if (max == neg_inf()) {
    lse = max;  // nothing above -inf: no distribution
    entropy = 0.0f;
  } else if (is_nan(max) || max == __int_as_float(0x7f800000)) {
    lse = entropy = __int_as_float(0x7fc00000);
  } else {
    const float l = logf(s);
    lse = max + l;
    entropy = max_nan(fmaf(-kLn2, w / s, l), 0.0f);  // (rounding can leave it just below)
  }
}

// A thread's running statistics: two interleaved pairs of sums relative to r.
struct ThreadSums {
  float r;
  float limit;  // a logit above it moves the reference (kUnset: there is none yet)
  uint64_t s, w;
};

// Two more logits (none below kLow).
__device__ __forceinline__ void sums_add(ThreadSums &a, float lo, float hi) {
  const uint64_t t = fma2(pack_f32(lo, hi), pack_f32(kLog2e, kLog2e), pack_f32(-a.r, -a.r));
  float t0, t1;
  unpack_f32(t, t0, t1);
  const uint64_t e = pack_f32(ex2(t0), ex2(t1));
  a.s = add2(a.s, e);
  a.w = fma2(e, t, a.w);
}

__device__ __forceinline__ Lse sums_total(const ThreadSums &a) {
  float s0, s1, w0, w1;
  unpack_f32(a.s, s0, s1);
  unpack_f32(a.w, w0, w1);
  return {a.r, s0 + s1, w0 + w1};
}

// Move the reference up to m where the sums would grow too large (rarely: it
// only has to stay within 2^12 of the maximum).
__device__ __forceinline__ void sums_rebase(ThreadSums &a, float m) {
  if (!(m > a.limit)) return;
  // (rounded by itself: were it contracted into the difference below, the sums so far
  // would be restated to the unrounded reference, up to 2^0.03 off at 5e5)
  const float r = __fmul_rn(m, kLog2e);
  if (a.limit > kUnset) {
    const Lse b = sums_total(a);
    const float d = a.r - r, f = ex2(d);
    a.w = pack_f32(f == 0.0f ? 0.0f : f * fmaf(d, b.s, b.w), 0.0f);
    a.s = pack_f32(f * b.s, 0.0f);
  }
  a.r = r;
  a.limit = m + 8.0f;
}

// The logits of a 16-byte vector.
template <bool kBf16>
__device__ __forceinline__ void vec_elems(const uint4 q, float (&x)[kBf16 ? 8 : 4]) {
  const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kBf16) {
      x[2 * i] = bf16_lo(wd[i]);
      x[2 * i + 1] = bf16_hi(wd[i]);
    } else {
      x[i] = __uint_as_float(wd[i]);
    }
  }
}

constexpr uint32_t kLowBf16x2 = 0xfe80fe80u;  // -2^126, twice

template <bool kBf16>
__device__ __forceinline__ void sums_vector(ThreadSums &a, const uint4 q) {
  if constexpr (kBf16) {
    const uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = max_nan_bf16x2(wd[i], kLowBf16x2);
      sums_add(a, bf16_lo(w), bf16_hi(w));
    }
  } else {
    sums_add(a, max_nan(__uint_as_float(q.x), kLow), max_nan(__uint_as_float(q.y), kLow));
    sums_add(a, max_nan(__uint_as_float(q.z), kLow), max_nan(__uint_as_float(q.w), kLow));
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

// A candidate: reaches the threshold and is not masked.
__device__ __forceinline__ bool reaches(float x, float threshold) {
  return !(x < threshold) && x != neg_inf();
}

// Whether a vector holds a logit that reaches `lo` (or a NaN), on the way to
// which its maximum joins the thread's.  lo: two copies for bf16.
template <bool kBf16>
__device__ __forceinline__ bool vec_reaches(const uint4 q, uint32_t &mx, uint32_t lo) {
  if constexpr (kBf16) {
    const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(q.x, q.y), max_nan_bf16x2(q.z, q.w));
    mx = max_nan_bf16x2(mx, m);
    uint32_t hit;
    asm("{\n\t.reg .pred p, q;\n\t"
        "setp.geu.bf16x2 p|q, %1, %2;\n\t"
        "or.pred p, p, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(hit)
        : "r"(m), "r"(lo));
    return hit != 0;
  } else {
    const float m = vec_max<false>(q);
    mx = __float_as_uint(max_nan(__uint_as_float(mx), m));
    return !(m < __uint_as_float(lo));
  }
}

// The larger of the reference limit and the candidates' threshold may be
// ignored by vec_reaches; what it compares with is the smaller.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack_lo(float limit, float threshold) {
  const float lo = threshold < limit ? threshold : limit;  // threshold is exact in the logits' type
  if (!kBf16) return __float_as_uint(lo);
  const uint32_t b = __float_as_uint(lo) >> 16;
  return b | (b << 16);
}

// Element i of an array of vectors in shared memory.
template <bool kBf16>
__device__ __forceinline__ float load_shared_elem(const uint4 *v, int i) {
  if (kBf16)
    return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(v)[i])
                           << 16);
  return reinterpret_cast<const float *>(v)[i];
}

template <int kT>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kT) : "memory");
}

template <int kT>
__device__ __forceinline__ void push_key(PieceShared<kT> &sh, float x, int32_t id) {
  const int at = atomicAdd(&sh.num_keys, 1);
  if (at < sh.kKeys) sh.key[at] = pair_key(x, id);
}

// The top_k of the n <= kKeys candidates into best (sorted), by counting.  Many
// candidates are first cut by a threshold, as the row was: the top_k-th largest
// of the maxima of 64 groups.
template <int kT>
__device__ __forceinline__ void select_top(PieceShared<kT> &sh, int n, int k, int tid) {
  const Key *from = sh.key;
  if (n > kGroups) {
    if (tid < kGroups) {
      Key m = 0;
      for (int i = tid; i < n; i += kGroups) m = max(m, sh.key[i]);
      sh.list[tid] = m;
    }
    if (tid == 0) sh.num_vecs = 0;
    consumers_sync<kT>();
    if (tid < kGroups) {
      const Key mine = sh.list[tid];
      if (keys_above(sh.list, kGroups, mine) == k - 1) sh.best[0] = mine;
    }
    consumers_sync<kT>();
    const Key threshold = sh.best[0];
    Key *kept = reinterpret_cast<Key *>(sh.vec);  // (the candidate vectors have been read)
    for (int i = tid; i < n; i += kT) {
      const Key mine = sh.key[i];
      if (mine >= threshold) kept[atomicAdd(&sh.num_vecs, 1)] = mine;
    }
    consumers_sync<kT>();
    n = sh.num_vecs;
    if (tid == 0 && (n & 1)) kept[n] = 0;
    from = kept;
  } else if (tid == 0 && (n & 1)) {
    sh.key[n] = 0;
  }
  consumers_sync<kT>();
  for (int i = tid; i < n; i += kT) {
    const Key mine = from[i];
    const int rank = keys_above(from, n, mine);
    if (rank < k) sh.best[rank] = mine;
  }
}

// The best k of the n pieces' sorted lists into best.  At least k entries reach
// the largest of the lists' last entries, and the smallest of their (k / n)-th: what
// does not reach the larger of the two is left out of the counting where there is
// much.  best[] and num_keys are 0 on entry.
template <int kT>
__device__ __forceinline__ void join_lists(PieceShared<kT> &sh, int n, int k, int tid) {
  int m = n * k;  // (even: n is)
  const Key *from = sh.pieces;
  if (m > 64) {
    Key threshold = 0, least = ~Key(0);
    const int share = (k + n - 1) / n - 1;
    for (int l = 0; l < n; ++l) {
      threshold = max(threshold, sh.pieces[l * k + k - 1]);
      least = min(least, sh.pieces[l * k + share]);
    }
    threshold = max(threshold, least);
    for (int c = tid; c < m; c += kT) {
      const Key mine = sh.pieces[c];
      if (mine != 0 && mine >= threshold) sh.key[atomicAdd(&sh.num_keys, 1)] = mine;
    }
    consumers_sync<kT>();
    m = sh.num_keys;
    if (tid == 0 && (m & 1)) sh.key[m] = 0;
    consumers_sync<kT>();
    from = sh.key;
  }
  for (int c = tid; c < m; c += kT) {
    const Key mine = from[c];
    const int rank = keys_above(from, m, mine);
    if (mine != 0 && rank < k) sh.best[rank] = mine;
  }
}

template <bool kBf16, int kT>
__global__ void __launch_bounds__(kT + 32, kT == 256 ? 3 : 10)
    logprobs_kernel(const char *__restrict__ logits, int64_t ld_bytes, int64_t num_rows, int valid,
                    int32_t id0, const int32_t *__restrict__ tokens, int k, int chunks, RowOut out,
                    uint32_t *err) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  constexpr int kStageVec = kT * kVecPerThread;
  constexpr int kWarps = kT / 32;
  constexpr int kPerGroup = kT / kGroups;
  constexpr uint32_t kMasked = kBf16 ? 0xff80ff80u : 0xff800000u;  // -inf
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ PieceShared<kT> sh;
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const int64_t row0 = blockIdx.x / chunks, row_step = gridDim.x / chunks;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const volatile int *abort_flag = &sh.abort;

  // This CTA's piece of a row: columns [c0, c1), of which [b0, b1) are whole
  // 16-byte vectors.
  struct Piece {
    const char *p;
    int c0, b0, b1, c1, stages;
  };
  auto piece_of = [&](int64_t row) {
    Piece q;
    q.p = logits + row * ld_bytes;
    int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(q.p) & 15u)) & 15u) / kElt);
    if (head > valid) head = valid;
    const int nvec = (valid - head) / kVec;
    // (nvec < 2^22, chunks <= 8)
    const int v0 = chunks == 1 ? 0 : static_cast<int>(static_cast<uint32_t>(nvec * chunk) / chunks);
    const int v1 = chunks == 1 ? nvec
                               : static_cast<int>(static_cast<uint32_t>(nvec * (chunk + 1)) / chunks);
    q.b0 = head + v0 * kVec;
    q.b1 = head + v1 * kVec;
    q.c0 = chunk == 0 ? 0 : q.b0;
    q.c1 = chunk == chunks - 1 ? valid : q.b1;
    q.stages = (v1 - v0 + kStageVec - 1) / kStageVec;
    return q;
  };

  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), kWarps);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cg::cluster_group cluster = cg::this_cluster();
  // Two cluster barriers: every CTA has begun (its memory may be written; nothing
  // else is handed over), every piece has reached the row's first CTA.
  if (chunks > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_wait();

  if (warp == kWarps) {
    // ------------------------------------------------------------- copy warp
    int g = 0;  // stages issued
    bool ok = true;
    for (int64_t row = row0; row < num_rows && ok; row += row_step) {
      const Piece q = piece_of(row);
      for (int j = 0; j < q.stages; ++j, ++g) {
        const int slot = g % kRing;
        if (g >= kRing && !warp_wait(smem_u32(&sh.empty[slot]), (g / kRing - 1) & 1, abort_flag)) {
          if (lane == 0) raise_abort(&sh.abort, err);
          ok = false;
          break;
        }
        if (elect_one()) {
          const int at = q.b0 + j * kStageVec * kVec;
          const uint32_t bytes = static_cast<uint32_t>(min(kStageVec * kVec, q.b1 - at)) * kElt;
          mbar_expect_tx(smem_u32(&sh.full[slot]), bytes);
          bulk_load(smem_u32(ring + slot * kStageVec), q.p + static_cast<int64_t>(at) * kElt,
                    bytes, smem_u32(&sh.full[slot]));
        }
        __syncwarp();
      }
    }
    // every copy has landed before the CTA ends
    const int zero = 0;
    for (int j = max(0, g - kRing); j < g; ++j)
      pipe_wait(smem_u32(&sh.full[j % kRing]), (j / kRing) & 1, &zero);
    pdl_launch_dependents();
    if (chunks > 1) {  // (the barriers count every thread that has not ended)
      __syncwarp();
      cluster.barrier_wait();
      cluster.barrier_arrive();
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  int g = 0;  // stages consumed
  int32_t tok_next = tid == 0 && tokens != nullptr && row0 < num_rows ? tokens[row0] : -1;
  bool ok = true;
  for (int64_t row = row0; row < num_rows; row += row_step) {
    const Piece pc = piece_of(row);
    const char *p = pc.p;
    if (tid == 0) {
      sh.num_vecs = sh.num_keys = 0;
      sh.threshold = 0xffffffffu;
    }
    const int32_t tok = tok_next;
    consumers_sync<kT>();

    ThreadSums a = {0.0f, kUnset, 0u, 0u};
    float threshold = __int_as_float(0x7f800000);
    if (k > 0) {
      threshold = neg_inf();
      const int held = min(kRing, pc.stages);
      if (held > 0) {
        float m = neg_inf();
        for (int j = 0; j < held; ++j) {
          const int slot = (g + j) % kRing;
          ok = ok && warp_wait(smem_u32(&sh.full[slot]), ((g + j) / kRing) & 1, abort_flag);
          const int n = min(kStageVec, (pc.b1 - pc.b0) / kVec - j * kStageVec);
          for (int i = tid; i < n; i += kT) m = max_nan(m, vec_max<kBf16>(ring[slot * kStageVec + i]));
        }
        sums_rebase(a, m);  // a reference to begin with
#pragma unroll
        for (int off = kPerGroup / 2; off > 0; off >>= 1)
          m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (tid % kPerGroup == 0) sh.group[tid / kPerGroup] = order_key(m);
        consumers_sync<kT>();
        if (tid < kGroups) {
          const uint32_t me = sh.group[tid];
          int above = 0;
#pragma unroll 4
          for (int i = 0; i < kGroups; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(sh.group + i);
            above += (o.x > me) + (o.y > me) + (o.z > me) + (o.w > me);
          }
          // the k-th largest: the smallest with fewer than k above it
          if (above < k) atomicMin(&sh.threshold, me);
        }
        consumers_sync<kT>();
        threshold = order_value(sh.threshold);
      }
    }

    float xt = neg_inf();  // the token's logit (thread 0; asked for here, used at the row's end)
    if (tid == 0) {
      if (tokens != nullptr && row + row_step < num_rows) tok_next = tokens[row + row_step];
      const int64_t at = static_cast<int64_t>(tok) - id0;
      if (tok >= 0 && at >= 0 && at < valid) xt = load_elem<kBf16>(p, static_cast<int>(at));
    }
    uint32_t mxb = kMasked;
    uint32_t lo = pack_lo<kBf16>(a.limit, threshold);
    for (int j = 0; j < pc.stages; ++j, ++g) {
      const int slot = g % kRing;
      ok = ok && warp_wait(smem_u32(&sh.full[slot]), (g / kRing) & 1, abort_flag);
      if (!ok) continue;  // (every warp keeps to the rows' barriers)
      const int at = pc.b0 + j * kStageVec * kVec;
      const int n = min(kStageVec, (pc.b1 - at) / kVec);
      const uint4 *st = ring + slot * kStageVec;
      // All of the thread's vectors at once, with one test for all: with a test and a
      // branch for each their latencies follow one another (4096 x 202048 242 us, so
      // 231; vectors past a piece's end count as masked).
      uint4 q[kVecPerThread];
#pragma unroll
      for (int u = 0; u < kVecPerThread; ++u) {
        const int i = u * kT + tid;
        q[u] = i < n ? st[i] : make_uint4(kMasked, kMasked, kMasked, kMasked);
      }
      uint4 most = q[0];
#pragma unroll
      for (int u = 1; u < kVecPerThread; ++u) most = vec_larger<kBf16>(most, q[u]);
      if (vec_reaches<kBf16>(most, mxb, lo)) {
        const float m = vec_max<kBf16>(most);
        sums_rebase(a, m);
        lo = pack_lo<kBf16>(a.limit, threshold);
        if (k > 0 && !(m < threshold)) {
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) {
            const float vm = vec_max<kBf16>(q[u]);
            if (vm < threshold || vm == neg_inf()) continue;
            const int c = atomicAdd(&sh.num_vecs, 1);
            if (c < sh.kVecs) {
              sh.vec[c] = q[u];
              sh.vec_id[c] = id0 + at + (u * kT + tid) * kVec;
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kVecPerThread; ++u) sums_vector<kBf16>(a, q[u]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.empty[slot]));
    }
    if (!ok && lane == 0) raise_abort(&sh.abort, err);
    float mx = kBf16 ? max_nan(bf16_lo(mxb), bf16_hi(mxb)) : __uint_as_float(mxb);
    // the unaligned ends: at most one element per thread on either side
    for (int side = 0; side < 2; ++side) {
      const int j = (side == 0 ? pc.c0 : pc.b1) + tid;
      if (j < (side == 0 ? pc.b0 : pc.c1)) {
        const float x = load_elem<kBf16>(p, j);
        mx = max_nan(mx, x);
        sums_rebase(a, x);
        sums_add(a, max_nan(x, kLow), kLow);
        if (k > 0 && reaches(x, threshold)) push_key(sh, x, id0 + j);
      }
    }
    {
      // the warp's sums, relative to its largest reference
      Lse t = sums_total(a);
      mx = order_value(__reduce_max_sync(0xffffffffu, order_key(mx)));
      const float r = order_value(
          __reduce_max_sync(0xffffffffu, order_key(t.s == 0.0f ? neg_inf() : t.r)));
      lse_restate(t, r);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        t.s += __shfl_xor_sync(0xffffffffu, t.s, off);
        t.w += __shfl_xor_sync(0xffffffffu, t.w, off);
      }
      if (lane == 0) {
        sh.warp_max[warp] = mx;
        sh.warp_lse[warp] = t;
      }
    }
    consumers_sync<kT>();  // every candidate vector is in the buffer

    // ---- the piece's alternatives into best[]
    if (k > 0) {
      const int nv = min(sh.num_vecs, sh.kVecs);
      for (int i = tid; i < nv * kVec; i += kT) {
        const int e = i % kVec;
        const float x = load_shared_elem<kBf16>(sh.vec, i);
        if (reaches(x, threshold)) push_key(sh, x, sh.vec_id[i / kVec] + e);
      }
      if (tid < k) sh.best[tid] = 0;
      consumers_sync<kT>();
      const int n = sh.num_keys;
      if (sh.num_vecs <= sh.kVecs && n <= sh.kKeys) {
        select_top(sh, n, k, tid);
        if (n < k && warp == 0) {
          // masked elements fill the list, lowest ids first
          int have = n;
          for (int base = pc.c0; base < pc.c1 && have < k; base += 32) {
            const int j = base + lane;
            const bool masked = j < pc.c1 && load_elem<kBf16>(p, j) == neg_inf();
            const unsigned m = __ballot_sync(0xffffffffu, masked);
            const int at = have + __popc(m & ((1u << lane) - 1));
            if (masked && at < k) sh.best[at] = pair_key(neg_inf(), id0 + j);
            have += __popc(m);
          }
        }
      } else {
        // Too many reach the threshold.  Usually they equal it (a mask of the
        // type's lowest value, constant rows): take those above it, and of
        // the equal ones the lowest ids.
        consumers_sync<kT>();
        if (tid == 0) sh.num_keys = 0;
        consumers_sync<kT>();
        auto above = [&](float x, int j) {
          if (!(x <= threshold)) push_key(sh, x, id0 + j);
        };
        const uint4 *body = reinterpret_cast<const uint4 *>(p + static_cast<int64_t>(pc.b0) * kElt);
        const int nvec = (pc.b1 - pc.b0) / kVec;
        constexpr int kBatch = 4;
        for (int v = tid; v < nvec; v += kBatch * kT) {
          uint4 q[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if (v + u * kT < nvec) q[u] = ld_stream_v4(body + v + u * kT);
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            if (v + u * kT >= nvec || vec_max<kBf16>(q[u]) <= threshold) continue;
            float x[kVec];
            vec_elems<kBf16>(q[u], x);
#pragma unroll
            for (int e = 0; e < kVec; ++e) above(x[e], pc.b0 + (v + u * kT) * kVec + e);
          }
        }
        for (int side = 0; side < 2; ++side) {
          const int j = (side == 0 ? pc.c0 : pc.b1) + tid;
          if (j < (side == 0 ? pc.b0 : pc.c1)) above(load_elem<kBf16>(p, j), j);
        }
        consumers_sync<kT>();
        int n = sh.num_keys;
        for (int base = pc.c0; base < pc.c1 && n < k; base += kT) {
          consumers_sync<kT>();  // everyone has read the count
          const int j = base + tid;
          const float x = j < pc.c1 ? load_elem<kBf16>(p, j) : __int_as_float(0x7fc00000);
          if (x == threshold) push_key(sh, x, id0 + j);
          consumers_sync<kT>();
          n = sh.num_keys;
        }
        if (n <= sh.kKeys) {
          select_top(sh, n, k, tid);
        } else {
          // rows that keep rising: a sorted list per warp
          Key top = 0;
          for (int base = pc.c0 + warp * 32; base < pc.c1; base += kT) {
            const int j = base + lane;
            top_offer(top, j < pc.c1 ? pair_key(load_elem<kBf16>(p, j), id0 + j) : 0, lane, k);
          }
          if (lane < k) sh.list[warp * k + lane] = top;
          consumers_sync<kT>();
          for (int c = tid; c < kWarps * k; c += kT) {
            const Key mine = sh.list[c];
            const int rank = keys_above(sh.list, kWarps * k, mine);
            if (mine != 0 && rank < k) sh.best[rank] = mine;
          }
        }
      }
    }
    // ---- the piece's sums, restated relative to its maximum
    float max = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) max = max_nan(max, sh.warp_max[w]);
    // An extreme finite maximum: sums relative to the maximum itself, in
    // differences from it, over the piece once more.
    const bool exact = (max > kFastMax && max < __int_as_float(0x7f800000)) ||
                       (max < -kFastMax && max > neg_inf());
    if (exact) {
      float es = 0.0f, ew = 0.0f;
      for (int j = pc.c0 + tid; j < pc.c1; j += kT) {
        const float t = max_nan((load_elem<kBf16>(p, j) - max) * kLog2e, -1e30f);
        const float e = ex2(t);
        es += e;
        ew = fmaf(e, t, ew);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        es += __shfl_xor_sync(0xffffffffu, es, off);
        ew += __shfl_xor_sync(0xffffffffu, ew, off);
      }
      consumers_sync<kT>();  // the others have read the sums of the first pass
      if (lane == 0) sh.warp_lse[warp] = {0.0f, es, ew};
    }
    // (best[] and, after an exact pass, the sums)
    consumers_sync<kT>();
    float s = 0.0f, w = 0.0f;
    if (warp == 0) {
      Lse t = {0.0f, 0.0f, 0.0f};
      if (lane < kWarps) t = sh.warp_lse[lane];
      // (the difference to the maximum in one rounding)
      const float d = exact ? 0.0f : fmaf(-max, kLog2e, t.r);
      const float f = t.s == 0.0f ? 0.0f : ex2(d);
      s = f * t.s;
      w = f == 0.0f ? 0.0f : f * fmaf(d, t.s, t.w);
#pragma unroll
      for (int off = kMaxWarps / 2; off > 0; off >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, off);
        w += __shfl_xor_sync(0xffffffffu, w, off);
      }
      if (lane == 0 && chunks == 1) {
        sh.sum = s;
        sh.wsum = w;
      }
    }
    if (chunks > 1) {
      // every piece to the row's first CTA
      cluster.barrier_wait();
      if (tid < k) cluster.map_shared_rank(sh.pieces, 0)[chunk * k + tid] = sh.best[tid];
      if (tid == 0) cluster.map_shared_rank(sh.piece, 0)[chunk] = {max, s, w};
      __syncwarp();
      cluster.barrier_arrive();
      if (chunk > 0) return;  // (such a launch has a row per cluster)
      if (tid < k) sh.best[tid] = 0;
      if (tid == 0) sh.num_keys = 0;
      cluster.barrier_wait();
      for (int c = 0; c < chunks; ++c) max = max_nan(max, sh.piece[c].max);
      if (warp == 0) {
        s = w = 0.0f;
        if (lane < chunks) {
          const Stats q = sh.piece[lane];
          const float d = (q.max - max) * kLog2e;  // <= 0
          const float f = q.max == neg_inf() ? 0.0f : ex2(d);
          s = f * q.s;
          w = f == 0.0f ? 0.0f : f * fmaf(d, q.s, q.w);
        }
#pragma unroll
        for (int off = kMaxChunks / 2; off > 0; off >>= 1) {
          s += __shfl_xor_sync(0xffffffffu, s, off);
          w += __shfl_xor_sync(0xffffffffu, w, off);
        }
        if (lane == 0) {
          sh.sum = s;
          sh.wsum = w;
        }
      }
      if (k > 0) join_lists(sh, chunks, k, tid);
    }
    consumers_sync<kT>();
    float lse, entropy;
    finish_row(max, sh.sum, sh.wsum, lse, entropy);
    if (tid == 0) {
      s = sh.sum;
      w = sh.wsum;
      if (out.part != nullptr) {
        out.part[row] = {max, s, w, xt};
      } else {
        if (out.logprob != nullptr) out.logprob[row] = tok < 0 ? 0.0f : to_logprob(xt, lse);
        if (out.entropy != nullptr) out.entropy[row] = entropy;
        if (out.lse != nullptr) out.lse[row] = lse;
      }
    }
    if (tid < k) {
      const float v = key_value(sh.best[tid]);
      const int32_t id = key_id(sh.best[tid]);
      if (out.part != nullptr) {
        out.top[row * k + tid] = {v, id};
      } else {
        if (out.top_ids != nullptr) out.top_ids[row * k + tid] = id == kNoId ? -1 : id;
        if (out.top_logprobs != nullptr) out.top_logprobs[row * k + tid] = to_logprob(v, lse);
      }
    }
    consumers_sync<kT>();  // what this row kept in shared memory has been read
  }
}

// ------------------------------------------------------------------ reduce
// One warp per row: lanes share the row's n parts and its n sorted lists of k
// entries.  At least k entries reach the largest of the lists' last entries, and
// the smallest of their (k / n)-th; what reaches the larger of the two (some 2 k
// entries) goes to shared memory and finds its place by counting.  Latency-bound:
// 96 rows of 4 lists of 5 3.2 us, of 8 lists of 20 5.6 us (searching the other
// lists in global memory for each entry's place took 4.2 and 31.7).
constexpr int kReduceWarps = 4;
constexpr int kReduceKeys = 256;  // a row's entries that reach the threshold

__device__ __forceinline__ Key stat_key(const sga_stat &q) {
  return q.id == kNoId ? 0 : pair_key(q.v, q.id);
}

// Of the m <= kReduceKeys keys, k of which reach lo, leaves at least k and at most
// 32 in keys[] and returns how many: the threshold is raised by bisection (counting
// 200 keys against each other instead took 10 us).
__device__ __forceinline__ int raise_threshold(Key *keys, int m, int k, Key lo, int lane) {
  constexpr int kMine = kReduceKeys / 32;
  Key mine[kMine];
  uint32_t most = 0;
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
    const int c = r * 32 + lane;
    mine[r] = c < m ? keys[c] : 0;
    most = max(most, static_cast<uint32_t>(mine[r] >> 32));
  }
  const int held = m;
  Key hi = (static_cast<Key>(__reduce_max_sync(0xffffffffu, most)) << 32) | 0xffffffffu;
  while (m > 32 && lo < hi) {
    const Key mid = hi - (hi - lo) / 2;
    int n = 0;
#pragma unroll
    for (int r = 0; r < kMine; ++r)
      if (r * 32 < held) n += __popc(__ballot_sync(0xffffffffu, mine[r] >= mid));
    if (n >= k) {
      lo = mid;
      m = n;
    } else {
      hi = mid - 1;
    }
  }
  __syncwarp();  // every lane has read its keys
  m = 0;
#pragma unroll
  for (int r = 0; r < kMine; ++r) {
    const bool take = mine[r] >= lo && mine[r] != 0;
    const unsigned votes = __ballot_sync(0xffffffffu, take);
    const int at = m + __popc(votes & ((1u << lane) - 1));
    if (take && at < 32) keys[at] = mine[r];
    m += __popc(votes);
  }
  return min(m, 32);
}

__global__ void __launch_bounds__(32 * kReduceWarps)
    logprob_reduce_kernel(const sga_logprob_part *__restrict__ parts,
                          const sga_stat *__restrict__ tops, int n, int64_t rows, int k,
                          const int32_t *__restrict__ tokens, RowOut out) {
  __shared__ alignas(16) Key held[kReduceWarps][kReduceKeys + 2];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kReduceWarps + warp;
  if (row >= rows) return;
  const int32_t tok = tokens != nullptr ? tokens[row] : -1;
  float max = neg_inf(), xt = neg_inf();
  for (int i = lane; i < n; i += 32) {
    const sga_logprob_part q = parts[i * rows + row];
    max = max_nan(max, q.max);
    xt = max_nan(xt, q.token);
  }
  // (reads every entry, so that the second pass finds them in L1)
  Key threshold = 0, least = ~Key(0);
  const int share = (k + n - 1) / n - 1;
#pragma unroll 4
  for (int c = lane; c < n * k; c += 32) {
    const int own = c / k, idx = c - own * k;
    const Key q = stat_key(tops[(own * rows + row) * k + idx]);
    if (idx == k - 1 && q > threshold) threshold = q;
    if (idx == share && q < least) least = q;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    max = max_nan(max, __shfl_xor_sync(0xffffffffu, max, off));
    xt = max_nan(xt, __shfl_xor_sync(0xffffffffu, xt, off));
    const Key o = __shfl_xor_sync(0xffffffffu, threshold, off);
    threshold = o > threshold ? o : threshold;
    const Key l = __shfl_xor_sync(0xffffffffu, least, off);
    least = l < least ? l : least;
  }
  if (least > threshold) threshold = least;
  float s = 0.0f, w = 0.0f;
  for (int i = lane; i < n; i += 32) {
    const sga_logprob_part q = parts[i * rows + row];
    const float d = (q.max - max) * kLog2e;  // <= 0; -inf for a shard with nothing
    const float f = q.max == neg_inf() ? 0.0f : ex2(d);
    if (f != 0.0f) {
      s = fmaf(f, q.sum, s);
      w = fmaf(f, fmaf(d, q.sum, q.wsum), w);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    w += __shfl_xor_sync(0xffffffffu, w, off);
  }
  float lse, entropy;
  finish_row(max, s, w, lse, entropy);
  if (lane == 0) {
    if (out.logprob != nullptr) out.logprob[row] = tok < 0 ? 0.0f : to_logprob(xt, lse);
    if (out.entropy != nullptr) out.entropy[row] = entropy;
    if (out.lse != nullptr) out.lse[row] = lse;
  }
  auto put = [&](int rank, Key q) {
    if (out.top_ids != nullptr) out.top_ids[row * k + rank] = q == 0 ? -1 : key_id(q);
    if (out.top_logprobs != nullptr)
      out.top_logprobs[row * k + rank] = to_logprob(key_value(q), lse);
  };
  int m = 0;
#pragma unroll 4
  for (int base = 0; base < n * k; base += 32) {
    const int c = base + lane;
    Key q = 0;
    if (c < n * k) {
      const int own = c / k;
      q = stat_key(tops[(own * rows + row) * k + (c - own * k)]);
    }
    const bool take = q != 0 && q >= threshold;
    const unsigned votes = __ballot_sync(0xffffffffu, take);
    const int at = m + __popc(votes & ((1u << lane) - 1));
    if (take && at < kReduceKeys) held[warp][at] = q;
    m += __popc(votes);
  }
  if (m <= kReduceKeys) {
    __syncwarp();
    if (m > 32) m = raise_threshold(held[warp], m, k, threshold, lane);
    if (lane == 0) held[warp][m] = 0;
    __syncwarp();
    if (lane < m) {
      const Key mine = held[warp][lane];
      const int rank = keys_above(held[warp], m, mine);
      if (rank < k) put(rank, mine);
    }
  } else {
    // (more lists than that: a sorted list in the warp's registers)
    Key top = 0;
    for (int base = 0; base < n * k; base += 32) {
      const int c = base + lane, own = c / k;
      top_offer(top, c < n * k ? stat_key(tops[(own * rows + row) * k + (c - own * k)]) : 0, lane,
                k);
    }
    m = __popc(__ballot_sync(0xffffffffu, lane < k && top != 0));
    if (lane < m) put(lane, top);
  }
  if (lane >= m && lane < k) put(lane, 0);
}

// ---------------------------------------------------------------- gradient
constexpr int kThreads = 256;
constexpr int kGradPiece = 65536;  // bytes of a row per CTA

// dx_j = p_j (A + B (log p_j + H)) plus, at the token and at the alternatives,
// their upstream gradients; A = -(sum of those), B = -(gradient of the
// entropy).  One pass, each logit read and each gradient written once; the few
// ids with an extra term are computed from the logits read before the pass and
// written after it, each as one sum rounded once.  HBM-bound: 4096 x 152064 bf16
// 363 us = 6.86 TB/s read and written, the copy rate, with four 16-byte loads in
// flight per thread (one: 502 us); issue slots 58 % busy.  A CTA per 64 KB of a
// row: nothing is shared along a row but three scalars, so pieces need no join.
struct GradIn {
  const int32_t *tokens;
  const float *lse, *entropy, *g_logprob, *g_entropy, *g_top;
  const int32_t *top_ids;
};

__device__ __forceinline__ float grad_term(float x, float lse, float a, float bh, float b) {
  const float lp = max_nan(x - lse, -256.0f);  // p is 0 from there on: times a finite factor
  return ex2(lp * kLog2e) * fmaf(b, lp, fmaf(b, bh, a));
}

// kShift: some rows of the logits and of the gradient lie at different 16-byte
// offsets (apart from the other case, whose registers it would double).
template <bool kBf16, bool kShift>
__global__ void __launch_bounds__(kThreads)
    logprobs_grad_kernel(const char *logits, int64_t ld_bytes, int valid, int width, int32_t id0,
                         GradIn in, int k, int chunks, char *grad, int64_t ldg_bytes) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  __shared__ int32_t ids[SGA_MAX_TOP + 1];
  __shared__ float gs[SGA_MAX_TOP + 1];
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const int64_t row = blockIdx.x / chunks;
  const int tid = threadIdx.x;
  const char *x = logits + row * ld_bytes;
  char *g = grad + row * ldg_bytes;
  pdl_wait();

  const float lse = in.lse[row];
  const float bh = in.entropy != nullptr ? in.entropy[row] : 0.0f;
  const float b = in.g_entropy != nullptr ? -in.g_entropy[row] : 0.0f;
  const bool live = lse != neg_inf();
  // the ids with an upstream gradient of their own: the token, the alternatives
  if (tid <= k) {
    const int32_t id = tid == 0 ? (in.tokens != nullptr ? in.tokens[row] : -1)
                                : in.top_ids[row * k + tid - 1];
    ids[tid] = id;
    gs[tid] = id < 0 ? 0.0f
                     : (tid == 0 ? (in.g_logprob != nullptr ? in.g_logprob[row] : 0.0f)
                                 : in.g_top[row * k + tid - 1]);
  }
  __syncthreads();
  float a = 0.0f;
  for (int i = 0; i <= k; ++i) a -= gs[i];
  // this CTA's columns: whole 16-byte groups of the output row
  int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(g) & 15u)) & 15u) / kElt);
  if (head > width) head = width;
  const int nvec = (width - head) / kVec;
  const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * chunk / chunks);
  const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (chunk + 1) / chunks);
  const int c0 = chunk == 0 ? 0 : head + v0 * kVec;
  const int c1 = chunk == chunks - 1 ? width : head + v1 * kVec;
  float fix = 0.0f;
  int fix_col = -1;
  if (tid <= k && ids[tid] >= 0) {
    const int64_t col = static_cast<int64_t>(ids[tid]) - id0;
    if (col >= c0 && col < c1 && col < valid) {
      bool first = true;
      for (int i = 0; i < tid; ++i) first = first && ids[i] != ids[tid];
      if (first) {
        fix_col = static_cast<int>(col);
        fix = grad_term(read_elem<kBf16>(x, fix_col), lse, a, bh, b);
        for (int i = tid; i <= k; ++i)
          if (ids[i] == ids[tid]) fix += gs[i];
      }
    }
  }
  __syncthreads();  // every special logit is read before the pass may overwrite it

  auto one = [&](int j) {
    float v = 0.0f;
    if (live && j < valid) v = grad_term(read_elem<kBf16>(x, j), lse, a, bh, b);
    store_elem<kBf16>(g, j, v);
  };
  if (chunk == 0 && tid < head) one(tid);
  // whole vectors of the output without padding ids.  Where the logits' row
  // lies at another 16-byte offset, a vector is put together from the two
  // aligned ones that hold it; the row's first and last vectors are left to
  // the single columns, so that no load leaves the row.
  const int offset = kShift ? static_cast<int>((reinterpret_cast<uintptr_t>(x) -
                                                reinterpret_cast<uintptr_t>(g)) & 15u)
                            : 0;
  const int full = valid > head ? (valid - head) / kVec : 0;
  const int vs = offset != 0 && v0 == 0 ? min(1, v1) : v0;
  const int ve = max(vs, min(v1, offset != 0 ? full - 1 : full));
  const char *xv = x + head * kElt - offset;  // 16-byte aligned
  char *gv = g + head * kElt;
  constexpr int kBatch = 4;  // loads in flight per thread
  for (int v = vs + tid; v < ve; v += kBatch * kThreads) {
    uint4 q[kBatch], q1[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (v + u * kThreads >= ve) continue;
      const uint4 *src = reinterpret_cast<const uint4 *>(xv) + v + u * kThreads;
      if (!kShift || offset == 0) {
        q[u] = __ldcs(src);
      } else {
        q[u] = src[0];
        q1[u] = src[1];
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (v + u * kThreads >= ve) continue;
      const uint4 xq = kShift && offset != 0 ? bytes_of(q[u], q1[u], offset) : q[u];
      uint32_t wd[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!live) {
          wd[i] = 0u;
        } else if (kBf16) {
          wd[i] = pack2(grad_term(bf16_lo(wd[i]), lse, a, bh, b),
                        grad_term(bf16_hi(wd[i]), lse, a, bh, b));
        } else {
          wd[i] = __float_as_uint(grad_term(__uint_as_float(wd[i]), lse, a, bh, b));
        }
      }
      __stcs(reinterpret_cast<uint4 *>(gv) + v + u * kThreads,
             make_uint4(wd[0], wd[1], wd[2], wd[3]));
    }
  }
  if (vs > v0)
    for (int j = head + v0 * kVec + tid; j < head + vs * kVec; j += kThreads) one(j);
  for (int j = head + ve * kVec + tid; j < c1; j += kThreads) one(j);
  pdl_launch_dependents();
  __syncthreads();
  if (fix_col >= 0 && live) store_elem<kBf16>(g, fix_col, fix);
}

// Pieces per row: a row is split (in powers of two) while the grid stays
// within the resident CTAs and a piece keeps a ring stage.  Whole rows go to
// persistent CTAs.
int pick_row_chunks(int64_t rows, int64_t nvec, int num_sms) {
  int chunks = 1;
  while (chunks < kMaxChunks && rows * chunks * 2 <= num_sms * 3 && nvec / (2 * chunks) >= 1024)
    chunks *= 2;
  return chunks;
}

template <bool kBf16, int kT>
cudaError_t launch_rows(const void *logits, int64_t rows, int64_t ld, int64_t shard_start,
                        int64_t valid, const int32_t *tokens, int top_k, int chunks, int num_sms,
                        const RowOut &out, uint32_t *err, cudaStream_t stream) {
  auto kern = logprobs_kernel<kBf16, kT>;
  const int64_t resident = static_cast<int64_t>(num_sms) * (kT == 256 ? 3 : 10);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(chunks > 1 || rows < resident ? rows * chunks
                                                                         : resident));
  cfg.blockDim = dim3(kT + 32);
  cfg.dynamicSmemBytes = ring_bytes<kT>;
  cfg.stream = stream;
  if (kT == 256) {
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kern), ring_bytes<kT>,
                                        kBf16 ? 0 : 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = chunks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits),
                            ld * (kBf16 ? 2 : 4), rows, static_cast<int>(valid),
                            static_cast<int32_t>(shard_start), tokens, top_k, chunks, out, err);
}

}  // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int64_t rows, int64_t ld,
                            int64_t shard_start, int64_t valid, const int32_t *tokens, int top_k,
                            float *logprob, float *entropy, float *lse, int32_t *top_ids,
                            float *top_logprobs, sga_logprob_part *part, sga_stat *top,
                            int num_sms, uint32_t *err, cudaStream_t stream) {
  const RowOut out = {logprob, entropy, lse, top_logprobs, top_ids, part, top};
  const int64_t nvec = valid * (dtype == SGA_BF16 ? 2 : 4) / 16;
  const int chunks = pick_row_chunks(rows, nvec, num_sms);
  // Many short rows: small CTAs, ten per SM (bf16, 5 alternatives, wide / small:
  // 1000 rows of 6000 ids 14.2 / 8.7 us, 4000 of 20000 66 / 54; 300 of 6000 5.6 /
  // 6.0, 4096 of 32000 75 / 77), while their shorter ring leaves few candidates: with
  // many alternatives some rows would overflow the buffer (20: 4096 of 24000 73 / 106,
  // 600 of 20000 15 / 31).
  constexpr int64_t held = ring_bytes<64> / 16;  // vectors that give the threshold
  const bool small = chunks == 1 && rows > 3 * num_sms && nvec <= 4 * held &&
                     nvec * (top_k > 0 ? top_k : 1) <= 48 * held;
  if (dtype == SGA_BF16)
    return small ? launch_rows<true, 64>(logits, rows, ld, shard_start, valid, tokens, top_k,
                                         chunks, num_sms, out, err, stream)
                 : launch_rows<true, 256>(logits, rows, ld, shard_start, valid, tokens, top_k,
                                          chunks, num_sms, out, err, stream);
  return small ? launch_rows<false, 64>(logits, rows, ld, shard_start, valid, tokens, top_k,
                                        chunks, num_sms, out, err, stream)
               : launch_rows<false, 256>(logits, rows, ld, shard_start, valid, tokens, top_k,
                                         chunks, num_sms, out, err, stream);
}

cudaError_t launch_logprob_reduce(const sga_logprob_part *parts, const sga_stat *tops,
                                  int num_shards, int64_t rows, int top_k, const int32_t *tokens,
                                  float *logprob, float *entropy, float *lse, int32_t *top_ids,
                                  float *top_logprobs, cudaStream_t stream) {
  const RowOut out = {logprob, entropy, lse, top_logprobs, top_ids, nullptr, nullptr};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kReduceWarps - 1) / kReduceWarps));
  cfg.blockDim = dim3(32 * kReduceWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprob_reduce_kernel, parts, tops, num_shards, rows, top_k,
                            tokens, out);
}

cudaError_t launch_logprobs_grad(const void *logits, int dtype, int64_t rows, int64_t ld,
                                 int64_t shard_start, int64_t width, int64_t valid,
                                 const int32_t *tokens, const float *lse, const float *entropy,
                                 const float *g_logprob, const float *g_entropy, int top_k,
                                 const int32_t *top_ids, const float *g_top, void *grad,
                                 int64_t ldg, cudaStream_t stream) {
  const int elt = dtype == SGA_BF16 ? 2 : 4;
  int64_t chunks = (width * elt + kGradPiece - 1) / kGradPiece;
  if (rows * chunks > (int64_t(1) << 30)) chunks = (int64_t(1) << 30) / rows;
  const GradIn in = {tokens, lse, entropy, g_logprob, g_entropy, g_top, top_ids};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * chunks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool shift = ((reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(grad)) |
                      ((ld - ldg) * elt)) % 16 != 0;
  auto kern = dtype == SGA_BF16
                  ? (shift ? logprobs_grad_kernel<true, true> : logprobs_grad_kernel<true, false>)
                  : (shift ? logprobs_grad_kernel<false, true> : logprobs_grad_kernel<false, false>);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * elt,
                            static_cast<int>(valid), static_cast<int>(width),
                            static_cast<int32_t>(shard_start), in, top_k,
                            static_cast<int>(chunks), static_cast<char *>(grad), ldg * elt);
}

}  // namespace sga
