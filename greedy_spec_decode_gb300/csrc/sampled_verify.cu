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
// 2^-38: 64-bit sums of up to 2^24 weights of at most 1 are exact (< 2^62), and
// any split of the row draws the same id.  An id of probability 1e-9 still has
// 275 units.
#include "common.cuh"

namespace sga {
namespace {

using Units = unsigned long long;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegments = 64;  // sums kept of a row

// A weight in units of 2^-38 (a NaN counts as 0).
__device__ __forceinline__ Units units(float w) {
  return __float2ull_rn(fminf(fmaxf(w, 0.0f), 1.0f) * 274877906944.0f);
}

__device__ __forceinline__ Units warp_sum(Units v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
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

__global__ void __launch_bounds__(kThreads) sampled_verify_kernel(VerifyArgs in, uint32_t *err) {
  __shared__ Units seg[kSegments];
  __shared__ Units sums[kWarps];
  __shared__ int s_accepted;
  __shared__ int32_t s_token;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t req = blockIdx.x;
  const int64_t c = in.cu[req];
  const int64_t k = in.cu[req + 1] - c;
  int32_t *sampled = in.sampled + req * (in.max_k + 1);
  const bool bad = k < 0 || k > in.max_k || c < 0 || c + k > in.rows - in.num_reqs;
  if (bad || (in.in_prefill != nullptr && in.in_prefill[req] != 0)) {
    if (tid <= in.max_k) sampled[tid] = -1;
    if (tid == 0) {
      in.num_sampled[req] = 0;
      in.num_rejected[req] = 0;
      in.last[req] = -1;
      if (bad) atomicOr(err, SGA_DEVERR_K_RANGE);
    }
    return;
  }
  // the first draft that is not accepted
  if (warp == 0) {
    bool fails = false;
    if (lane < k) {
      const int32_t t = in.tokens[c + lane];
      fails = true;
      if (t >= 0 && t < in.vocab) {
        const float p = in.target[(c + req + lane) * in.ldt + t];
        const float q = in.draft != nullptr ? in.draft[(c + lane) * in.ldd + t] : 1.0f;
        fails = !(__fmul_rn(in.accept_u[c + lane], q) < p);
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
    const int32_t t = in.tokens[c + a];
    if (t >= 0 && t < in.vocab) {
      if (in.draft != nullptr)
        q = in.draft + (c + a) * in.ldd;
      else
        hot = t;
    }
  }
  auto weight = [&](int j) {
    const float w = p[j];
    return units(q != nullptr ? __fsub_rn(w, q[j]) : (j == hot ? __fsub_rn(w, 1.0f) : w));
  };
  const int len = (in.vocab + kSegments - 1) / kSegments;
  Units total = 0;
  while (true) {
    for (int s = warp; s < kSegments; s += kWarps) {
      const int64_t j1 = min(static_cast<int64_t>(in.vocab), static_cast<int64_t>(s + 1) * len);
      Units sum = 0;
      for (int64_t j = static_cast<int64_t>(s) * len + lane; j < j1; j += 32)
        sum += weight(static_cast<int>(j));
      sum = warp_sum(sum);
      if (lane == 0) seg[s] = sum;
    }
    __syncthreads();
    total = 0;
    for (int s = 0; s < kSegments; ++s) total += seg[s];
    if (total != 0 || (q == nullptr && hot < 0)) break;
    q = nullptr;  // p nowhere above q: from p itself
    hot = -1;
    __syncthreads();
  }
  if (tid == 0) s_token = -1;
  if (total != 0) {
    const float u = in.sample_u[req];
    Units edge = u > 0.0f ? __double2ull_rd(__dmul_rn(u, __ull2double_rn(total))) : 0;
    if (edge > total - 1) edge = total - 1;
    int s = 0;
    Units below = 0;
    while (below + seg[s] <= edge) below += seg[s++];
    // the segment again, a run of ids per thread
    const int j0 = s * len, n = min(len, in.vocab - j0), run = (n + kThreads - 1) / kThreads;
    const int b0 = j0 + min(n, tid * run), b1 = j0 + min(n, (tid + 1) * run);
    Units own = 0;
    for (int j = b0; j < b1; ++j) own += weight(j);
    Units upto = own;  // with the lanes before
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const Units o = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += o;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    Units sum = below + upto - own;
    for (int w = 0; w < warp; ++w) sum += sums[w];
    if (sum <= edge && edge < sum + own) {
      int j = b0;
      while ((sum += weight(j)) <= edge) ++j;
      s_token = j;
    }
  }
  __syncthreads();
  if (tid <= in.max_k)
    sampled[tid] = tid < a ? in.tokens[c + tid] : (tid == a ? s_token : -1);
  if (tid == 0) {
    in.num_sampled[req] = a + 1;
    in.num_rejected[req] = static_cast<int32_t>(k) - a;
    in.last[req] = s_token;
  }
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
  (void)num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_reqs));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sampled_verify_kernel, in, err);
}

}  // namespace sga
