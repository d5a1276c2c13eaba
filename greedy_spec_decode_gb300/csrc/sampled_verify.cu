// sampled_verify.cu -- verification of drafted tokens by rejection sampling.
//
// With p the target's and q the draft's probabilities of a row, draft t is
// accepted with probability min(1, p_t / q_t) (u q_t < p_t for a uniform u); at
// the first rejection a token is drawn from max(p - q, 0), after the last draft
// from p of the bonus row.  What is emitted then has the target's distribution.
//
// Drawing inverts the cumulative sum in ascending id order.  A sum in fp32
// depends on its order, and near the end of a vocabulary neighbouring sums
// differ by less than its rounding, so weights are counted in whole units of
// 2^-38: 64-bit sums of up to 2^24 weights of at most 1 are exact (at most 2^62), and
// any split of the row draws the same id.  How fine a draw is goes by the uniform's 24
// bits, not by the units.
#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace sga {
namespace {

using Units = unsigned long long;

constexpr int kBatch = 16;          // loads in flight per thread and row
constexpr int kStep = 32 * kBatch;  // ids that a warp takes at once
constexpr int kMaxSegments = 256;   // sums kept of a CTA's ids
constexpr int kMaxCtas = 8;         // CTAs per request
constexpr int kThreads = 256;

// A weight in units of 2^-38 (a NaN counts as 0).
__device__ __forceinline__ Units units(float w) {
  return __float2ull_rn(fminf(fmaxf(w, 0.0f), 1.0f) * 274877906944.0f);
}

__device__ __forceinline__ Units warp_sum(Units v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The sums up to and with each lane.
__device__ __forceinline__ Units warp_prefix(Units v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Units o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

struct VerifyArgs {
  const float *target, *draft;
  int64_t rows, ldt, ldd;
  int vocab, num_reqs, max_k;
  const int32_t *cu, *tokens;
  const uint8_t *in_prefill;
  const float *accept_u, *sample_u;
  int32_t *sampled, *num_sampled, *num_rejected, *last;
};

// A running sum of weights w = max(x - y, 0) in units, for one thread: w 2^38 is
// split into hi 2^23 + lo, hi = rint(w 2^15) and lo the rounded rest (in -2^22 ..
// 2^22), both read off the mantissa of a sum with 1.5 2^23.  The integers carry that
// constant's bits once per weight; fewer than 2^9 weights (lo could add up to 2^31), then
// unit_total.  (A conversion to 64 bits per weight takes 4 x the time of these eight
// operations.)
struct UnitSum {
  uint32_t hi, lo;
};
constexpr float kMagic = 12582912.0f;       // 1.5 2^23
constexpr uint32_t kMagicBits = 0x4b400000u;
static_assert(kBatch < 512, "weights per UnitSum");

__device__ __forceinline__ void unit_add(UnitSum &a, float x, float y) {
  float w;  // rounded once, clamped to [0, 1], a NaN becomes 0
  asm("sub.rn.sat.f32 %0, %1, %2;" : "=f"(w) : "f"(x), "f"(y));
  const float t = __fmaf_rn(w, 32768.0f, kMagic);
  const float rest = __fmaf_rn(w, 32768.0f, -__fsub_rn(t, kMagic));
  a.hi += __float_as_uint(t);
  a.lo += __float_as_uint(__fmaf_rn(rest, 8388608.0f, kMagic));
}

__device__ __forceinline__ Units unit_total(const UnitSum &a, uint32_t weights) {
  const uint32_t hi = a.hi - weights * kMagicBits;
  const int32_t lo = static_cast<int32_t>(a.lo - weights * kMagicBits);
  return (static_cast<Units>(hi) << 23) + static_cast<Units>(static_cast<int64_t>(lo));
}

// The sum of the weights of ids [j0, j1), for one warp.  kRow: q is a row of draft
// probabilities; otherwise the one id `hot` (or none) has all of them.  kVec: rows
// and j0 are 16-byte aligned.
template <bool kRow, bool kVec>
__device__ __forceinline__ Units warp_units(const float *p, const float *q, int32_t hot, int j0,
                                            int j1, int lane) {
  Units sum = 0;
  int j = j0;
  for (; j + kStep <= j1; j += kStep) {
    float x[kBatch], y[kBatch];
    if (kVec) {
#pragma unroll
      for (int u = 0; u < kBatch; u += 4) {
        const int at = j + u * 32 + lane * 4;
        *reinterpret_cast<float4 *>(x + u) = __ldcs(reinterpret_cast<const float4 *>(p + at));
        if (kRow)
          *reinterpret_cast<float4 *>(y + u) = __ldcs(reinterpret_cast<const float4 *>(q + at));
      }
    } else {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        x[u] = __ldcs(p + j + u * 32 + lane);
        if (kRow) y[u] = __ldcs(q + j + u * 32 + lane);
      }
    }
    UnitSum a = {0u, 0u};
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int at = kVec ? j + (u & ~3) * 32 + lane * 4 + (u & 3) : j + u * 32 + lane;
      if (!kRow) y[u] = at == hot ? 1.0f : 0.0f;
      unit_add(a, x[u], y[u]);
    }
    sum += unit_total(a, kBatch);
  }
  if (j < j1) {
    UnitSum a = {0u, 0u};
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int at = j + u * 32 + lane;
      const float x = at < j1 ? __ldcs(p + at) : 0.0f;
      unit_add(a, x, kRow ? (at < j1 ? __ldcs(q + at) : 0.0f) : (at == hot ? 1.0f : 0.0f));
    }
    sum += unit_total(a, kBatch);
  }
  return warp_sum(sum);
}

// A cluster of CTAs per request, each with a run of the row's ids.  Bound by HBM
// where requests are many (512 of 152064 ids, half of them with a rejection: 467 MB
// in 70 us = 6.7 TB/s; with 8 loads of a row in flight per thread instead of 16 76),
// by the chain of dependent steps where they are few: offsets, drafts, their
// probabilities, the row's sum (segment sums stay in shared memory), the totals'
// exchange, the segment of the drawn id once more (from L2).
__global__ void __launch_bounds__(kThreads, 4)
    sampled_verify_kernel(VerifyArgs in, int ctas, uint32_t *err) {
  constexpr int kWarps = kThreads / 32;
  __shared__ Units seg[kMaxSegments];
  __shared__ Units totals[2][kMaxCtas];  // of the request's CTAs, by pass
  __shared__ Units warp_sums[kWarps];
  __shared__ int s_accepted, s_segment;
  __shared__ int32_t s_draft[32], s_token;
  __shared__ Units s_below;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x % ctas);
  const int64_t req = blockIdx.x / ctas;
  // (every CTA of the cluster has begun: its memory may be written)
  if (ctas > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  pdl_wait();
  // (not after the offsets: a dependent load is 1 us)
  const uint8_t prefill = in.in_prefill != nullptr ? in.in_prefill[req] : 0;
  const float u = in.sample_u[req];
  const int64_t c = in.cu[req];
  const int64_t k = in.cu[req + 1] - c;
  int32_t *sampled = in.sampled + req * (in.max_k + 1);
  const bool bad = k < 0 || k > in.max_k || c < 0 || c + k > in.rows - in.num_reqs;
  if (bad || prefill != 0) {
    if (rank == 0) {
      if (tid <= in.max_k) sampled[tid] = -1;
      if (tid == 0) {
        in.num_sampled[req] = 0;
        in.num_rejected[req] = 0;
        in.last[req] = -1;
        if (bad) atomicOr(err, SGA_DEVERR_K_RANGE);
      }
    }
    if (ctas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
    return;
  }
  // the first draft that is not accepted (every CTA finds it by itself)
  if (warp == 0) {
    bool fails = false;
    if (lane < k) {
      const int32_t t = in.tokens[c + lane];
      const float accept = in.accept_u[c + lane];
      s_draft[lane] = t;
      fails = true;
      if (t >= 0 && t < in.vocab) {
        const float p = in.target[(c + req + lane) * in.ldt + t];
        const float q = in.draft != nullptr ? in.draft[(c + lane) * in.ldd + t] : 1.0f;
        fails = !(__fmul_rn(accept, q) < p);
      }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, fails);
    if (lane == 0) s_accepted = votes != 0 ? __ffs(votes) - 1 : static_cast<int>(k);
  }
  __syncthreads();
  const int a = s_accepted;
  const float *p = in.target + (c + req + a) * in.ldt;
  const float *q = nullptr;  // the draft's row, where there is one
  int32_t hot = -1;          // or the id that has all of its probability
  if (a < k) {
    const int32_t t = s_draft[a];
    if (t >= 0 && t < in.vocab) {
      if (in.draft != nullptr)
        q = in.draft + (c + a) * in.ldd;
      else
        hot = t;
    }
  }
  // this CTA's ids, in segments of whole steps
  const int share = ((in.vocab + ctas - 1) / ctas + 3) & ~3;
  const int c0 = min(in.vocab, rank * share), c1 = min(in.vocab, c0 + share);
  int len = kStep;
  while (static_cast<int64_t>(len) * kMaxSegments < share) len *= 2;
  const int segments = (c1 - c0 + len - 1) / len;
  const bool vec = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;

  Units total = 0, own = 0, before = 0;  // the row's, this CTA's, those of the CTAs before it
  bool found = false;
  for (int pass = 0;; ++pass) {
    for (int s = warp; s < segments; s += kWarps) {
      const int j0 = c0 + s * len, j1 = min(c1, j0 + len);
      const Units sum =
          vec ? (q != nullptr ? warp_units<true, true>(p, q, hot, j0, j1, lane)
                              : warp_units<false, true>(p, q, hot, j0, j1, lane))
              : (q != nullptr ? warp_units<true, false>(p, q, hot, j0, j1, lane)
                              : warp_units<false, false>(p, q, hot, j0, j1, lane));
      if (lane == 0) seg[s] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      Units sum = 0;
      for (int s = lane; s < segments; s += 32) sum += seg[s];
      sum = warp_sum(sum);
      if (ctas == 1) {
        if (lane == 0) totals[pass][0] = sum;
      } else {
        if (pass == 0) asm volatile("barrier.cluster.wait;" ::: "memory");
        if (lane < ctas) *cg::this_cluster().map_shared_rank(&totals[pass][rank], lane) = sum;
        __syncwarp();
      }
    } else if (ctas > 1 && pass == 0) {
      asm volatile("barrier.cluster.wait;" ::: "memory");
    }
    if (ctas > 1)
      asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    else
      __syncthreads();
    total = before = 0;
    own = totals[pass][rank];
    for (int i = 0; i < ctas; ++i) {
      if (i < rank) before += totals[pass][i];
      total += totals[pass][i];
    }
    found = total != 0;
    if (found || (q == nullptr && hot < 0)) break;
    q = nullptr;  // p nowhere above q: from p itself
    hot = -1;
  }
  pdl_launch_dependents();
  Units edge = 0;
  if (found) {
    edge = u > 0.0f ? __double2ull_rd(__dmul_rn(u, __ull2double_rn(total))) : 0;
    if (edge > total - 1) edge = total - 1;
  }
  // the CTA whose ids hold the edge goes on alone
  if (found ? edge < before || edge - before >= own : rank != 0) return;
  if (tid == 0) s_token = -1;
  if (found) {
    edge -= before;
    if (warp == 0) {  // its segment
      constexpr int kPer = kMaxSegments / 32;
      Units part = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) part += lane * kPer + i < segments ? seg[lane * kPer + i] : 0;
      const Units upto = warp_prefix(part, lane);
      Units below = upto - part;
      if (below <= edge && edge < upto) {
        int s = lane * kPer;
        while (below + seg[s] <= edge) below += seg[s++];
        s_segment = s;
        s_below = below;
      }
    }
    __syncthreads();
    edge -= s_below;
    // the segment again, a run of ids per thread
    const int j0 = c0 + s_segment * len, n = min(len, c1 - j0);
    const int run = (n + kThreads - 1) / kThreads;
    const int b0 = j0 + min(n, tid * run), b1 = j0 + min(n, (tid + 1) * run);
    auto weight = [&](int j) {
      return units(__fsub_rn(__ldg(p + j), q != nullptr ? __ldg(q + j) : (j == hot ? 1.0f : 0.0f)));
    };
    Units part = 0;
    for (int j = b0; j < b1; ++j) part += weight(j);
    const Units upto = warp_prefix(part, lane);
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    Units sum = upto - part;
    for (int w = 0; w < warp; ++w) sum += warp_sums[w];
    if (sum <= edge && edge < sum + part) {
      int j = b0;
      while ((sum += weight(j)) <= edge) ++j;
      s_token = j;
    }
  }
  __syncthreads();
  if (tid <= in.max_k)
    sampled[tid] = tid < a ? s_draft[tid] : (tid == a ? s_token : -1);
  if (tid == 0) {
    in.num_sampled[req] = a + 1;
    in.num_rejected[req] = static_cast<int32_t>(k) - a;
    in.last[req] = s_token;
  }
}

// CTAs per request, four per SM: as many as let all requests run at once, with at least
// 4096 ids each.  (The three counts are what runs at once of this kernel on 152 SMs, at 64
// registers and 256 threads: they have to be looked at again when those change.  Requests of
// 152064 ids: 76 x 6 13.7 us, x 8, of which 74 run at once, 17.5; 100 x 4 15.0, x 6 17.8;
// 154 x 2 28.6, x 4 33.6; 512 x 1 69, x 2 74.  24 of 200064 x 8 9.2, x 6 10.3; CTAs of 512
// threads x 8 9.4.)
int pick_ctas(int num_reqs, int64_t vocab, int num_sms) {
  constexpr int kWidths[3] = {8, 6, 4};
  constexpr int kClusters[3] = {74, 97, 148};  // at once, of 608 CTAs (GPCs hold whole clusters)
  for (int i = 0; i < 3; ++i)
    if (vocab >= 4096 * kWidths[i] && num_reqs <= kClusters[i] * num_sms / 152) return kWidths[i];
  return num_reqs <= 2ll * num_sms && vocab >= 8192 ? 2 : 1;
}

}  // namespace

cudaError_t launch_sampled_verify(const float *target, int64_t rows, int64_t ldt,
                                  const float *draft, int64_t ldd, int64_t vocab, int num_reqs,
                                  const int32_t *cu_num_draft, const int32_t *draft_tokens,
                                  const uint8_t *in_prefill, const float *accept_u,
                                  const float *sample_u, int max_k, int32_t *out_sampled,
                                  int32_t *out_num_sampled, int32_t *out_num_rejected,
                                  int32_t *out_last, int num_sms, uint32_t *err,
                                  cudaStream_t stream) {
  const VerifyArgs in = {target,     draft,       rows,     ldt,
                         ldd,        static_cast<int>(vocab), num_reqs, max_k,
                         cu_num_draft, draft_tokens, in_prefill, accept_u,
                         sample_u,   out_sampled, out_num_sampled, out_num_rejected,
                         out_last};
  const int ctas = pick_ctas(num_reqs, vocab, num_sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_reqs * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sampled_verify_kernel, in, ctas, err);
}

}  // namespace sga
