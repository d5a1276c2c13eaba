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
#include <cuda_bf16.h>

#include "common.cuh"
#include "scan.cuh"

namespace cg = cooperative_groups;

namespace sga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Logits below kLow count as kLow in the fast pass (their terms are zero
// there); a row whose maximum lies outside +-kFastMax takes the exact pass.
constexpr float kLow = -1e38f;
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

// a += b.  An empty side (s == 0) leaves the other's reference; otherwise the
// larger reference stays and the other side is scaled down to it.
__device__ __forceinline__ void lse_merge(Lse &a, const Lse &b) {
  if (b.s == 0.0f) return;
  if (a.s == 0.0f) {
    a = b;
    return;
  }
  const float r = max_nan(a.r, b.r);
  const float da = a.r - r, db = b.r - r;  // <= 0, one of them 0
  const float fa = ex2(da), fb = ex2(db);
  // sum (t + d) 2^(t + d) = 2^d (w + d s); a vanished side contributes 0
  const float wa = fa == 0.0f ? 0.0f : fa * fmaf(da, a.s, a.w);
  const float wb = fb == 0.0f ? 0.0f : fb * fmaf(db, b.s, b.w);
  a.s = fa * a.s + fb * b.s;
  a.w = wa + wb;
  a.r = r;
}

// ------------------------------------------------------------ alternatives
// A warp's best entries so far, in the argmax order: lane i holds the i-th.
struct WarpTop {
  float v;
  int32_t id;
  float kth_v;     // entry k - 1: what a new element has to beat
  int32_t kth_id;
};

__device__ __forceinline__ void top_insert(WarpTop &t, float v, int32_t id, int lane, int k) {
  const unsigned before = __ballot_sync(0xffffffffu, pair_beats(t.v, t.id, v, id));
  const int pos = __popc(before);  // the list is sorted: the entries that stay ahead are a prefix
  const float up_v = __shfl_up_sync(0xffffffffu, t.v, 1);
  const int32_t up_id = __shfl_up_sync(0xffffffffu, t.id, 1);
  if (lane > pos) {
    t.v = up_v;
    t.id = up_id;
  } else if (lane == pos) {
    t.v = v;
    t.id = id;
  }
  t.kth_v = __shfl_sync(0xffffffffu, t.v, k - 1);
  t.kth_id = __shfl_sync(0xffffffffu, t.id, k - 1);
}

// Offer one element per lane (id kNoId: none) to the warp's list.
__device__ __forceinline__ void top_offer(WarpTop &t, float x, int32_t id, int lane, int k) {
  unsigned m = __ballot_sync(0xffffffffu, pair_beats(x, id, t.kth_v, t.kth_id));
  while (m != 0) {
    const int src = __ffs(m) - 1;
    m &= m - 1;
    const float v = __shfl_sync(0xffffffffu, x, src);
    const int32_t i = __shfl_sync(0xffffffffu, id, src);
    if (pair_beats(v, i, t.kth_v, t.kth_id)) top_insert(t, v, i, lane, k);
  }
}

// ---------------------------------------------------------------- forward
// One cluster of `chunks` CTAs per row; each CTA reads a contiguous piece of
// the row and the first CTA joins the pieces through distributed shared
// memory, so that a row needs one launch and no workspace.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kMaxChunks = 8;

struct RowOut {
  // final results (nullable each), or with part set the shard's statistics
  float *logprob, *entropy, *lse, *top_logprobs;
  int32_t *top_ids;
  sga_logprob_part *part;
  sga_stat *top;
};

// What one CTA knows of its piece.
struct PieceShared {
  Lse lse;
  float max;
  float cand_v[kWarps * SGA_MAX_TOP];  // the warps' sorted lists, then the CTA's
  int32_t cand_id[kWarps * SGA_MAX_TOP];
  float best_v[SGA_MAX_TOP];
  int32_t best_id[SGA_MAX_TOP];
  Lse warp_lse[kWarps];
  float warp_max[kWarps];
};

// Element-wise absorption of one logit (row heads and tails).
__device__ __forceinline__ void lse_absorb(Lse &a, float x) {
  const float c = max_nan(x, kLow);
  if (c > kUnset && (a.s == 0.0f || c * kLog2e > a.r + 12.0f)) {
    const float r = c * kLog2e;
    if (a.s != 0.0f) {
      const float d = a.r - r, f = ex2(d);
      a.w = f == 0.0f ? 0.0f : f * fmaf(d, a.s, a.w);
      a.s *= f;
    }
    a.r = r;
  }
  const float t = fmaf(c, kLog2e, -a.r);
  const float e = ex2(t);
  a.s += e;
  a.w = fmaf(e, t, a.w);
}

// The position of entry (v, id) of list `own` among n sorted lists of k
// entries each: its index in its own list plus the entries of the others that
// come before it (a binary search per list).  Empty entries (kNoId) compare
// equal and go by list.
__device__ __forceinline__ int rank_in_lists(const float *vs, const int32_t *ids, int n, int k,
                                             int own, int idx) {
  const float v = vs[own * k + idx];
  const int32_t id = ids[own * k + idx];
  int rank = idx;
  for (int l = 0; l < n; ++l) {
    if (l == own) continue;
    int lo = 0, hi = k;  // entries [0, lo) of list l come before (v, id)
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      const float ov = vs[l * k + mid];
      const int32_t oi = ids[l * k + mid];
      const bool before = oi == id ? l < own : pair_beats(ov, oi, v, id);
      if (before)
        lo = mid + 1;
      else
        hi = mid;
    }
    rank += lo;
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
    entropy = fmaf(-kLn2, w / s, l);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
    logprobs_kernel(const char *__restrict__ logits, int64_t ld_bytes, int valid, int32_t id0,
                    const int32_t *__restrict__ tokens, int k, int chunks, RowOut out) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  __shared__ PieceShared sh;
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const int64_t row = blockIdx.x / chunks;
  const char *p = logits + row * ld_bytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / kElt);
  if (head > valid) head = valid;
  const int nvec = (valid - head) / kVec;
  const int tail = valid - head - nvec * kVec;
  const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * chunk / chunks);
  const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (chunk + 1) / chunks);
  const uint4 *vp = reinterpret_cast<const uint4 *>(p + head * kElt);
  pdl_wait();

  Lse a = {0.0f, 0.0f, 0.0f};
  float mx = neg_inf();
  WarpTop top = {neg_inf(), kNoId, neg_inf(), kNoId};

  // head (first piece) and tail (last piece): one element per thread
  {
    const bool h = chunk == 0 && tid < head;
    const bool t = chunk == chunks - 1 && tid >= 32 && tid - 32 < tail;
    if (warp < 2) {
      const int j = h ? tid : head + nvec * kVec + tid - 32;
      const float x = h || t ? load_elem<kBf16>(p, j) : neg_inf();
      if (h || t) {
        lse_absorb(a, x);
        mx = x;
      }
      if (k > 0) top_offer(top, x, h || t ? id0 + j : kNoId, lane, k);
    }
  }

  for (int base = v0 + warp * 32; base < v1; base += kThreads * kUnroll) {
    uint4 q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = base + u * kThreads + lane;
      q[u] = v < v1 ? ld_stream_v4(vp + v)
                    : (kBf16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                             : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const float vm = vec_max<kBf16>(q[u]);
      mx = max_nan(mx, vm);
      const uint32_t wd[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      float x[kVec];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kBf16) {
          x[2 * i] = bf16_lo(wd[i]);
          x[2 * i + 1] = bf16_hi(wd[i]);
        } else {
          x[i] = __uint_as_float(wd[i]);
        }
      }
      if (vm > kUnset && (a.s == 0.0f || vm * kLog2e > a.r + 12.0f)) {
        const float r = vm * kLog2e;
        if (a.s != 0.0f) {
          const float d = a.r - r, f = ex2(d);
          a.w = f == 0.0f ? 0.0f : f * fmaf(d, a.s, a.w);
          a.s *= f;
        }
        a.r = r;
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float t = fmaf(max_nan(x[i], kLow), kLog2e, -a.r);
        const float e = ex2(t);
        a.s += e;
        a.w = fmaf(e, t, a.w);
      }
      if (k > 0 && __any_sync(0xffffffffu, !(vm < top.kth_v))) {
        const int v = base + u * kThreads + lane;
        const int32_t id = id0 + head + v * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          top_offer(top, x[i], v < v1 ? id + i : kNoId, lane, k);
      }
    }
  }

  // ---- the CTA's pieces
  auto block_max = [&](float m) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh.warp_max[warp] = m;
  };
  auto block_lse = [&](Lse b) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const Lse o = {__shfl_xor_sync(0xffffffffu, b.r, off), __shfl_xor_sync(0xffffffffu, b.s, off),
                     __shfl_xor_sync(0xffffffffu, b.w, off)};
      lse_merge(b, o);
    }
    if (lane == 0) sh.warp_lse[warp] = b;
  };
  block_max(mx);
  block_lse(a);
  if (lane < k) {
    sh.cand_v[warp * k + lane] = top.v;
    sh.cand_id[warp * k + lane] = top.id;
  }
  __syncthreads();
  for (int c = tid; c < kWarps * k; c += kThreads) {
    const int rank = rank_in_lists(sh.cand_v, sh.cand_id, kWarps, k, c / k, c % k);
    if (rank < k) {
      sh.best_v[rank] = sh.cand_v[c];
      sh.best_id[rank] = sh.cand_id[c];
    }
  }
  if (tid == 0) {
    float m = sh.warp_max[0];
    Lse t = sh.warp_lse[0];
    for (int w = 1; w < kWarps; ++w) {
      m = max_nan(m, sh.warp_max[w]);
      lse_merge(t, sh.warp_lse[w]);
    }
    sh.max = m;
    sh.lse = t;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();

  // ---- the row: every CTA joins the maxima (the exact pass needs it)
  float row_max = sh.max;
  for (int c = 0; c < chunks; ++c) row_max = max_nan(row_max, *cluster.map_shared_rank(&sh.max, c));
  // An extreme finite maximum: sums relative to the maximum itself, in
  // differences from it, over the piece once more.
  const bool exact = (row_max > kFastMax && row_max < __int_as_float(0x7f800000)) ||
                     (row_max < -kFastMax && row_max > neg_inf());
  if (exact) {
    float es = 0.0f, ew = 0.0f;
    auto term = [&](float x) {
      const float t = max_nan((x - row_max) * kLog2e, -1e30f);
      const float e = ex2(t);
      es += e;
      ew = fmaf(e, t, ew);
    };
    if (chunk == 0 && tid < head) term(load_elem<kBf16>(p, tid));
    for (int j = head + v0 * kVec + tid; j < head + v1 * kVec; j += kThreads)
      term(load_elem<kBf16>(p, j));
    if (chunk == chunks - 1 && tid < tail) term(load_elem<kBf16>(p, head + nvec * kVec + tid));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      es += __shfl_xor_sync(0xffffffffu, es, off);
      ew += __shfl_xor_sync(0xffffffffu, ew, off);
    }
    if (lane == 0) sh.warp_lse[warp] = {0.0f, es, ew};
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) {
        es += sh.warp_lse[w].s;
        ew += sh.warp_lse[w].w;
      }
      sh.lse = {0.0f, es, ew};
    }
  } else if (tid == 0) {
    // restate the piece relative to the row's maximum
    const Lse t = sh.lse;
    const float d = fmaf(-row_max, kLog2e, t.r);
    const float f = t.s == 0.0f ? 0.0f : ex2(d);
    sh.lse = {0.0f, f * t.s, f == 0.0f ? 0.0f : f * fmaf(d, t.s, t.w)};
  }
  cluster.sync();
  pdl_launch_dependents();

  if (chunk == 0) {
    // gather the pieces' lists (the warps' lists are no longer needed)
    for (int c = tid; c < chunks * k; c += kThreads) {
      sh.cand_v[c] = *cluster.map_shared_rank(&sh.best_v[c % k], c / k);
      sh.cand_id[c] = *cluster.map_shared_rank(&sh.best_id[c % k], c / k);
    }
    float s = sh.lse.s, w = sh.lse.w;
    for (int c = 1; c < chunks; ++c) {
      const Lse o = *cluster.map_shared_rank(&sh.lse, c);
      s += o.s;
      w += o.w;
    }
    __syncthreads();
    const int32_t tok = tokens != nullptr ? tokens[row] : -1;
    const int64_t at = static_cast<int64_t>(tok) - id0;
    const float xt = tok >= 0 && at >= 0 && at < valid ? load_elem<kBf16>(p, static_cast<int>(at))
                                                       : neg_inf();
    float lse, entropy;
    finish_row(row_max, s, w, lse, entropy);
    if (tid == 0) {
      if (out.part != nullptr) {
        out.part[row] = {row_max, s, w, xt};
      } else {
        if (out.logprob != nullptr) out.logprob[row] = tok < 0 ? 0.0f : to_logprob(xt, lse);
        if (out.entropy != nullptr) out.entropy[row] = entropy;
        if (out.lse != nullptr) out.lse[row] = lse;
      }
    }
    for (int c = tid; c < chunks * k; c += kThreads) {
      const int rank = rank_in_lists(sh.cand_v, sh.cand_id, chunks, k, c / k, c % k);
      if (rank >= k) continue;
      const float v = sh.cand_v[c];
      const int32_t id = sh.cand_id[c];
      if (out.part != nullptr) {
        out.top[row * k + rank] = {v, id};
      } else {
        if (out.top_ids != nullptr) out.top_ids[row * k + rank] = id == kNoId ? -1 : id;
        if (out.top_logprobs != nullptr) out.top_logprobs[row * k + rank] = to_logprob(v, lse);
      }
    }
  }
  cluster.sync();  // the pieces' shared memory stays alive until it has been read
}

// ------------------------------------------------------------------ reduce
// One warp per row: lanes share the row's parts, then its n sorted lists of k
// entries (each entry finds its own place by binary searches in the others).
__global__ void logprob_reduce_kernel(const sga_logprob_part *__restrict__ parts,
                                      const sga_stat *__restrict__ tops, int n, int64_t rows,
                                      int k, const int32_t *__restrict__ tokens, RowOut out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  float max = neg_inf(), xt = neg_inf();
  for (int i = lane; i < n; i += 32) {
    const sga_logprob_part q = parts[i * rows + row];
    max = max_nan(max, q.max);
    xt = max_nan(xt, q.token);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    max = max_nan(max, __shfl_xor_sync(0xffffffffu, max, off));
    xt = max_nan(xt, __shfl_xor_sync(0xffffffffu, xt, off));
  }
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
    const int32_t tok = tokens != nullptr ? tokens[row] : -1;
    if (out.logprob != nullptr) out.logprob[row] = tok < 0 ? 0.0f : to_logprob(xt, lse);
    if (out.entropy != nullptr) out.entropy[row] = entropy;
    if (out.lse != nullptr) out.lse[row] = lse;
  }
  for (int c = lane; c < n * k; c += 32) {
    const int own = c / k, idx = c % k;
    const sga_stat q = tops[(own * rows + row) * k + idx];
    int rank = idx;
    for (int l = 0; l < n && rank < k; ++l) {
      if (l == own) continue;
      const sga_stat *list = tops + (l * rows + row) * k;
      int lo = 0, hi = k;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const sga_stat o = list[mid];
        const bool before = o.id == q.id ? l < own : pair_beats(o.v, o.id, q.v, q.id);
        if (before)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank < k) {
      if (out.top_ids != nullptr) out.top_ids[row * k + rank] = q.id == kNoId ? -1 : q.id;
      if (out.top_logprobs != nullptr) out.top_logprobs[row * k + rank] = to_logprob(q.v, lse);
    }
  }
}

// ---------------------------------------------------------------- gradient
// dx_j = p_j (A + B (log p_j + H)) plus, at the token and at the alternatives,
// their upstream gradients; A = -(sum of those), B = -(gradient of the
// entropy).  One pass, each logit read and each gradient written once; the few
// ids with an extra term are computed from the logits read before the pass and
// written after it, each as one sum rounded once.
struct GradIn {
  const int32_t *tokens;
  const float *lse, *entropy, *g_logprob, *g_entropy, *g_top;
  const int32_t *top_ids;
};

__device__ __forceinline__ float grad_term(float x, float lse, float a, float bh, float b) {
  const float lp = max_nan(x - lse, -1e30f);  // a masked logit: p = 0 times a finite factor
  return ex2(lp * kLog2e) * fmaf(b, lp, fmaf(b, bh, a));
}

template <bool kBf16>
__device__ __forceinline__ void store_elem(char *p, int j, float v) {
  if (kBf16)
    reinterpret_cast<__nv_bfloat16 *>(p)[j] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float *>(p)[j] = v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ float read_elem(const char *p, int j) {  // the buffer may be the output
  if (kBf16)
    return __uint_as_float(static_cast<uint32_t>(
                               reinterpret_cast<const volatile unsigned short *>(p)[j])
                           << 16);
  return reinterpret_cast<const volatile float *>(p)[j];
}

template <bool kBf16>
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
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15u) == 0;
  if (!same) {
    for (int j = c0 + tid; j < c1; j += kThreads) one(j);
  } else {
    if (chunk == 0 && tid < head) one(tid);
    const int full = valid > head ? (valid - head) / kVec : 0;  // vectors without padding ids
    const int ve = v1 < full ? v1 : full;
    const char *xv = x + head * kElt;
    char *gv = g + head * kElt;
    for (int v = v0 + tid; v < ve; v += kThreads) {
      uint4 q = __ldcs(reinterpret_cast<const uint4 *>(xv) + v);
      uint32_t wd[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!live) {
          wd[i] = 0u;
        } else if (kBf16) {
          wd[i] = pack_bf16(grad_term(bf16_lo(wd[i]), lse, a, bh, b),
                            grad_term(bf16_hi(wd[i]), lse, a, bh, b));
        } else {
          wd[i] = __float_as_uint(grad_term(__uint_as_float(wd[i]), lse, a, bh, b));
        }
      }
      __stcs(reinterpret_cast<uint4 *>(gv) + v, make_uint4(wd[0], wd[1], wd[2], wd[3]));
    }
    for (int j = head + (ve > v0 ? ve : v0) * kVec + tid; j < c1; j += kThreads) one(j);
  }
  pdl_launch_dependents();
  __syncthreads();
  if (fix_col >= 0 && live) store_elem<kBf16>(g, fix_col, fix);
}

// Pieces per row: a row is split (in powers of two) while the grid stays
// within the resident CTAs and a piece keeps a few vectors per thread.
int pick_row_chunks(int64_t rows, int64_t width, int elt, int num_sms, int most) {
  const int64_t nvec = width * elt / 16;
  int chunks = 1;
  while (chunks < most && rows * chunks * 2 <= num_sms * 4 && nvec / (2 * chunks) >= kThreads)
    chunks *= 2;
  return chunks;
}

}  // namespace

cudaError_t launch_logprobs(const void *logits, int dtype, int64_t rows, int64_t ld,
                            int64_t shard_start, int64_t valid, const int32_t *tokens, int top_k,
                            float *logprob, float *entropy, float *lse, int32_t *top_ids,
                            float *top_logprobs, sga_logprob_part *part, sga_stat *top,
                            int num_sms, cudaStream_t stream) {
  const int elt = dtype == SGA_BF16 ? 2 : 4;
  const int chunks = pick_row_chunks(rows, valid, elt, num_sms, kMaxChunks);
  const RowOut out = {logprob, entropy, lse, top_logprobs, top_ids, part, top};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * chunks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = chunks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto kern = dtype == SGA_BF16 ? logprobs_kernel<true> : logprobs_kernel<false>;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * elt,
                            static_cast<int>(valid), static_cast<int32_t>(shard_start), tokens,
                            top_k, chunks, out);
}

cudaError_t launch_logprob_reduce(const sga_logprob_part *parts, const sga_stat *tops,
                                  int num_shards, int64_t rows, int top_k, const int32_t *tokens,
                                  float *logprob, float *entropy, float *lse, int32_t *top_ids,
                                  float *top_logprobs, cudaStream_t stream) {
  const RowOut out = {logprob, entropy, lse, top_logprobs, top_ids, nullptr, nullptr};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 3) / 4));
  cfg.blockDim = dim3(128);
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
                                 int64_t ldg, int num_sms, cudaStream_t stream) {
  const int elt = dtype == SGA_BF16 ? 2 : 4;
  int64_t chunks = (width * elt + 32767) / 32768;  // 32 KB of a row per CTA
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
  auto kern = dtype == SGA_BF16 ? logprobs_grad_kernel<true> : logprobs_grad_kernel<false>;
  (void)num_sms;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * elt,
                            static_cast<int>(valid), static_cast<int>(width),
                            static_cast<int32_t>(shard_start), in, top_k,
                            static_cast<int>(chunks), static_cast<char *>(grad), ldg * elt);
}

}  // namespace sga
