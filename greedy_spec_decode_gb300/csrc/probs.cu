// probs.cu -- probabilities of logits rows at a temperature.
//
// p_j = 2^((x_j - max) log2e / T) / sum_i 2^(...): the difference to the row's
// maximum is formed first, so that the largest term is exactly 1 at any
// temperature and offset.  A greedy row (T = 0) is 1 at its argmax.
#include "scan.cuh"

namespace sga {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThreads = 512;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
    probs_kernel(const char *logits, int64_t ld_bytes, int valid, int width,
                 const float *temperature, float *probs, int64_t ldp) {
  __shared__ float part[32];
  __shared__ int32_t part_id[32];
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x;
  const char *x = logits + row * ld_bytes;
  float *out = probs + row * ldp;
  const float t = temperature != nullptr ? temperature[row] : 1.0f;
  float m = neg_inf();
  int32_t id = kNoId;
  for (int j = tid; j < valid; j += kThreads) {
    const float v = read_elem<kBf16>(x, j);
    if (id == kNoId || scan_better(v, m)) {
      m = v;
      id = j;
    }
  }
  warp_argmax(m, id);
  if (lane == 0) {
    part[warp] = m;
    part_id[warp] = id;
  }
  __syncthreads();
  m = neg_inf();
  id = kNoId;
  for (int w = 0; w < kThreads / 32; ++w)
    if (pair_beats(part[w], part_id[w], m, id)) {
      m = part[w];
      id = part_id[w];
    }
  __syncthreads();
  const bool greedy = t == 0.0f;
  const float scale = t > 0.0f ? fminf(kLog2e / t, 3e38f) : __int_as_float(0x7fc00000);
  auto term = [&](int j) { return exp2f((read_elem<kBf16>(x, j) - m) * scale); };
  float s = 0.0f;
  if (!greedy && m != neg_inf()) {
    for (int j = tid; j < valid; j += kThreads) s += term(j);
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) part[warp] = s;
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  }
  for (int j = tid; j < width; j += kThreads) {
    float p = 0.0f;
    if (j < valid) {
      if (greedy)
        p = j == id ? 1.0f : 0.0f;
      else if (m != neg_inf() || t != t || t < 0.0f)
        p = term(j) / s;
    }
    out[j] = p;
  }
}

}  // namespace

cudaError_t launch_probs(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                         int64_t valid, const float *temperature, float *probs, int64_t ldp,
                         int num_sms, uint32_t *err, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, bf16 ? probs_kernel<true> : probs_kernel<false>,
                            static_cast<const char *>(logits), ld * (bf16 ? 2 : 4),
                            static_cast<int>(valid), static_cast<int>(width), temperature, probs,
                            ldp);
}

}  // namespace sga
