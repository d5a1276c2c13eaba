// distill.cu -- divergence of a draft model's rows from a teacher's top logits,
// and its gradient with respect to the draft's logits.
//
// With y = x / T, s_j = e^(y_j - lse), the teacher's list (id_i, p_i) and p_r the
// teacher's probability off the list:
//   loss   = sum_i p_i (log p_i - log s_id_i) + p_r (log p_r - (lse_rest - lse)),
//   grad_j = g / T (P s_j - sum over id_i = j of p_i - [j off the list] p_r
//            e^(y_j - lse_rest)),   P = sum_i p_i + p_r.
// Off the list both terms are multiples of e^(y_j - lse_rest), the factor being
// P e^(lse_rest - lse) - p_r.  The k entries are written after the row's pass.
// lse_rest is summed without the listed ids: as a difference of sums it would
// lose what a draft that agrees with its teacher leaves off the list.  The
// teacher's few numbers are kept in 64 bits, p_r being 1 less a sum near 1.
#include "scan.cuh"

namespace sga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512;
constexpr int kTile = 8192;  // ids whose list membership is held as bits

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float nan_f32() { return __int_as_float(0x7fc00000); }

__device__ float block_sum(float v, float *part) {
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kThreads / 32; ++w) v += part[w];
  return v;
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
    distill_kernel(const char *logits, int64_t ld_bytes, int valid, int width, DistillArgs in,
                   char *grad, int64_t ldg_bytes) {
  __shared__ float part[32];
  __shared__ int32_t ids[SGA_MAX_TEACHER];
  __shared__ double prob[SGA_MAX_TEACHER], logp[SGA_MAX_TEACHER];
  __shared__ float xs[SGA_MAX_TEACHER];
  __shared__ uint32_t bits[kTile / 32];
  __shared__ double s_rest_p, s_sum_p;
  __shared__ int s_entries;
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const int k = in.k;
  const char *x = logits + row * ld_bytes;
  const double inv_t = 1.0 / static_cast<double>(in.temperature);
  // the teacher's list
  if (tid < k) {
    int32_t id = in.ids[row * k + tid];
    if (id < 0 || id >= valid) id = -1;
    ids[tid] = id;
    logp[tid] = in.logits[row * k + tid] * inv_t;
    xs[tid] = id >= 0 ? read_elem<kBf16>(x, id) : neg_inf();
  }
  __syncthreads();
  if (tid == 0) {
    int entries = 0;
    double norm = 0.0, most = -INFINITY, sum = 0.0;
    for (int i = 0; i < k; ++i)
      if (ids[i] >= 0) {
        ++entries;
        most = !(logp[i] <= most) ? logp[i] : most;  // (a NaN stays)
      }
    if (in.lse != nullptr) {
      norm = in.lse[row];
    } else if (most == -INFINITY) {
      entries = 0;
    } else {
      for (int i = 0; i < k; ++i)
        if (ids[i] >= 0) sum += exp(logp[i] - most);
      norm = most + log(sum);
    }
    sum = 0.0;
    for (int i = 0; i < k; ++i) {
      logp[i] -= norm;
      prob[i] = ids[i] >= 0 && entries > 0 ? exp(logp[i]) : 0.0;
      sum += prob[i];
    }
    s_entries = entries;
    s_sum_p = sum;
    s_rest_p = in.lse != nullptr && entries > 0 ? (sum > 1.0 ? 0.0 : 1.0 - sum) : 0.0;
  }
  __syncthreads();
  const float scale = static_cast<float>(kLog2e * inv_t);
  float lse, lse_rest;
  if (in.in_lse != nullptr) {
    lse = in.in_lse[row];
    lse_rest = in.in_lse_rest != nullptr ? in.in_lse_rest[row] : neg_inf();
  } else {
    float m = neg_inf();
    for (int j = tid; j < valid; j += kThreads) m = max_nan(m, read_elem<kBf16>(x, j));
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) part[warp] = m;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) m = max_nan(m, part[w]);
    // the maximum off the list, and the sums
    float mr = neg_inf(), sum = 0.0f, rest = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int j0 = 0; j0 < valid; j0 += kTile) {
        __syncthreads();
        for (int i = tid; i < kTile / 32; i += kThreads) bits[i] = 0;
        __syncthreads();
        if (tid < k && ids[tid] >= j0 && ids[tid] < j0 + kTile)
          atomicOr(&bits[(ids[tid] - j0) / 32], 1u << ((ids[tid] - j0) & 31));
        __syncthreads();
        for (int j = j0 + tid; j < min(valid, j0 + kTile); j += kThreads) {
          const float v = read_elem<kBf16>(x, j);
          const bool listed = (bits[(j - j0) / 32] >> ((j - j0) & 31)) & 1;
          if (pass == 0) {
            if (!listed) mr = max_nan(mr, v);
          } else {
            if (m != neg_inf()) sum += exp2f((v - m) * scale);
            if (!listed && mr != neg_inf()) rest += exp2f((v - mr) * scale);
          }
        }
      }
      if (pass == 0) {
        for (int off = 16; off > 0; off >>= 1)
          mr = max_nan(mr, __shfl_xor_sync(0xffffffffu, mr, off));
        __syncthreads();
        if (lane == 0) part[warp] = mr;
        __syncthreads();
        for (int w = 0; w < kThreads / 32; ++w) mr = max_nan(mr, part[w]);
      }
    }
    sum = block_sum(sum, part);
    rest = block_sum(rest, part);
    const bool bad = is_nan(sum);  // a NaN or +inf in the row
    lse = m == neg_inf() ? m : static_cast<float>(m * inv_t + log(static_cast<double>(sum)));
    lse_rest = mr == neg_inf() ? mr : static_cast<float>(mr * inv_t + log(static_cast<double>(rest)));
    if (bad) lse = lse_rest = nan_f32();
    if (tid == 0) {
      const double rp = lse_rest == neg_inf() ? 0.0 : s_rest_p;
      const double l = bad ? nan("") : m * inv_t + log(static_cast<double>(sum));
      double loss = 0.0;
      for (int i = 0; i < k; ++i)
        if (!(prob[i] <= 0.0))
          loss += prob[i] * (logp[i] - (xs[i] == neg_inf() ? -INFINITY : xs[i] * inv_t - l));
      if (!(rp <= 0.0)) {
        const double lr = mr * inv_t + log(static_cast<double>(rest));
        loss += rp * (log(rp) - (lr - l));
      }
      if (s_entries == 0) loss = 0.0;
      else if (bad) loss = nan("");
      if (in.out_loss != nullptr) in.out_loss[row] = static_cast<float>(loss);
      if (in.out_lse != nullptr) in.out_lse[row] = lse;
      if (in.out_lse_rest != nullptr) in.out_lse_rest[row] = lse_rest;
    }
  }
  if (grad == nullptr) return;
  char *g = grad + row * ldg_bytes;
  __syncthreads();
  const float up = (in.grad_loss != nullptr ? in.grad_loss[row] : 1.0f) * static_cast<float>(inv_t);
  const double rp = lse_rest == neg_inf() ? 0.0 : s_rest_p;
  const double total = s_sum_p + rp;
  const bool live = s_entries > 0 && lse != neg_inf();
  // off the list relative to lse_rest: s_r <= 1 times e^(y_j - lse_rest), where s_j itself may
  // vanish (a rest that is masked by a low value)
  const bool by_rest = rp > 0.0;
  const float base = by_rest ? lse_rest : lse;
  const float off_list =
      up * static_cast<float>(
               by_rest ? total * exp(static_cast<double>(lse_rest) - static_cast<double>(lse)) - rp
                       : total);
  const float on_list = static_cast<float>(total);
  auto e_of = [&](float v, float l) { return exp2f((v * static_cast<float>(inv_t) - l) * kLog2e); };
  for (int j = tid; j < width; j += kThreads)
    store_elem<kBf16>(g, j, live && j < valid ? off_list * e_of(read_elem<kBf16>(x, j), base) : 0.0f);
  __syncthreads();
  if (live && tid < k && ids[tid] >= 0) {
    bool first = true;
    double p = 0.0;
    for (int i = 0; i < k; ++i)
      if (ids[i] == ids[tid]) {
        p += prob[i];
        first = first && i >= tid;
      }
    if (first)
      store_elem<kBf16>(g, ids[tid], up * (on_list * e_of(xs[tid], lse) - static_cast<float>(p)));
  }
}

}  // namespace

cudaError_t launch_distill(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                           int64_t valid, const DistillArgs &args, int64_t ldg, int num_sms,
                           uint32_t *err, cudaStream_t stream) {
  (void)num_sms;
  (void)err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool bf16 = dtype == SGA_BF16;
  const int elt = bf16 ? 2 : 4;
  return cudaLaunchKernelEx(&cfg, bf16 ? distill_kernel<true> : distill_kernel<false>,
                            static_cast<const char *>(logits), ld * elt, static_cast<int>(valid),
                            static_cast<int>(width), args, static_cast<char *>(args.grad),
                            ldg * elt);
}

}  // namespace sga
