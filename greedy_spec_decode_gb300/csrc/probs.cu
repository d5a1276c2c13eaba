// probs.cu -- probabilities of logits rows at a temperature.
//
// p_j = 2^((x_j - m) log2e / T) / sum_i 2^(...), m a logit within 2^12 (in terms)
// of the row's maximum, by which the exponents are exact differences at any
// offset and temperature.  A greedy row (T = 0) is 1 at its argmax.
#include "rowring.cuh"

namespace sga {
namespace {

// Stages of the ring: the most that fits two CTAs per SM (16 KB), or eight (4 KB).
template <int kT>
constexpr int kSlots = kT == 256 ? 7 : 6;
template <int kT>
constexpr int kRingBytes = kSlots<kT> * kStageVec<kT> * 16;

template <int kT>
struct ProbsShared {
  Ring ring;
  Exchange<2> ex;
  Sum warp_sum[kT / 32];
  int32_t warp_id[kT / 32];
};

// Unit of the output: 16 bytes, four probabilities.
template <bool kBf16>
__device__ __forceinline__ void load4(const uint4 *stage, int unit, float (&x)[4]) {
  if constexpr (kBf16) {
    const uint2 q = reinterpret_cast<const uint2 *>(stage)[unit];
    x[0] = bf16_lo(q.x);
    x[1] = bf16_hi(q.x);
    x[2] = bf16_lo(q.y);
    x[3] = bf16_hi(q.y);
  } else {
    const uint4 q = stage[unit];
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
}

template <bool kBf16, int kT>
__global__ void __launch_bounds__(kT + 32, kPerSm<kT>)
    probs_kernel(const char *logits, int64_t ld_bytes, int64_t num_rows, int valid, int width,
                 const float *temperature, float *probs, int64_t ldp, int chunks, uint32_t *err) {
  constexpr int slots = kSlots<kT>;
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  constexpr int kWarps = kT / 32;
  constexpr uint32_t kMasked = kBf16 ? 0xff80ff80u : 0xff800000u;  // -inf
  extern __shared__ __align__(128) uint4 buf[];
  __shared__ ProbsShared<kT> sh;
  const auto walk = walk_of<false>(num_rows, chunks);
  const int chunk = walk.chunk;
  const int64_t row0 = walk.first, row_step = walk.step;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const volatile int *abort_flag = &sh.ring.abort;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&sh.ring.full[i]), 1);
      mbar_init(smem_u32(&sh.ring.empty[i]), kWarps);
    }
    sh.ring.abort = 0;
    exchange_init(sh.ex, chunks);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (chunks > 1) {  // every CTA's barriers are ready
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
  pdl_wait();

  if (warp == kWarps) {
    copy_rows<kBf16, kT>(sh.ring, buf, slots, true, logits, ld_bytes, walk, valid, lane, err);
    pdl_launch_dependents();
  } else {
    Place at = {0, 0};
    bool ok = true;
    int64_t it = 0;
    float t_next = temperature != nullptr && row0 < num_rows ? temperature[row0] : 1.0f;
    for (int64_t row = row0; row < num_rows; row += row_step, ++it) {
      const Piece pc = piece_of<kBf16, kT>(logits + row * ld_bytes, valid, chunk, chunks);
      const float t = t_next;
      if (temperature != nullptr && row + row_step < num_rows) t_next = temperature[row + row_step];
      const bool greedy = t == 0.0f;
      const float scale = t > 0.0f ? fminf(kLog2e / t, 3e38f) : nan_f32();
      const float room = 12.0f / scale;
      RunSum a = {0.0f, neg_inf(), 0u};
      float best = neg_inf();
      int32_t best_id = kNoId;
      // the single elements at the row's ends
      float end_x[2] = {neg_inf(), neg_inf()};
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, tid);
        if (j >= 0) end_x[side] = read_elem<kBf16>(pc.p, j);
      }
      // ---- the row's sum (a greedy row's argmax)
      Place r = at;
      const int kept = max(0, pc.stages - slots);  // the first stage that stays
      for (int j = 0; j < pc.stages; ++j) {
        ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        const uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
        uint4 q[kVecPerThread];
#pragma unroll
        for (int u = 0; u < kVecPerThread; ++u) {
          const int i = u * kT + tid;
          q[u] = i < n ? st[i] : make_uint4(kMasked, kMasked, kMasked, kMasked);
        }
        if (greedy) {
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u)
            if (u * kT + tid < n && (best_id == kNoId || scan_better(vec_max<kBf16>(q[u]), best))) {
              const int32_t id = c + (u * kT + tid) * kVec;
              if (best_id == kNoId) best_id = id;  // (a first id, if nothing is above -inf)
              scan_vec<kBf16>(q[u], id, best, best_id);
            }
        } else {
          uint4 most = q[0];
#pragma unroll
          for (int u = 1; u < kVecPerThread; ++u) most = vec_larger<kBf16>(most, q[u]);
          sum_rebase(a, vec_max<kBf16>(most), scale, room);
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) sum_vector<kBf16>(a, q[u], scale);
        }
        if (j < kept) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
        }
        step(r, slots);
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, tid);
        if (j < 0) continue;
        if (greedy) {
          if (best_id == kNoId || pair_beats(end_x[side], j, best, best_id)) {
            best = end_x[side];
            best_id = j;
          }
        } else {
          sum_rebase(a, end_x[side], scale, room);
          sum_add(a, end_x[side], neg_inf(), scale);
        }
      }
      // ---- joined over the warps and the cluster
      Sum total = {best, 0.0f};
      if (greedy)
        warp_argmax(total.m, best_id);
      else
        total = sum_warp(sum_result(a), scale);
      if (lane == 0) {
        sh.warp_sum[warp] = total;
        sh.warp_id[warp] = best_id;
      }
      consumers_sync<kT>();
      if (warp == 0) {
        total = lane < kWarps ? sh.warp_sum[lane] : Sum{neg_inf(), 0.0f};
        best_id = lane < kWarps ? sh.warp_id[lane] : kNoId;
        if (greedy)
          warp_argmax(total.m, best_id);
        else
          total = sum_warp(total, scale);
      }
      if (warp == 0 && ok)
        exchange_tell(sh.ex, static_cast<uint32_t>(it),
                      make_uint4(__float_as_uint(total.m), __float_as_uint(total.s),
                                 static_cast<uint32_t>(best_id), 0u),
                      chunk, chunks, lane);
      ok = ok && exchange_wait(sh.ex, static_cast<uint32_t>(it), abort_flag);
      if (ok && warp == 0) exchange_rearm(sh.ex, static_cast<uint32_t>(it), chunks, lane);
      total = {neg_inf(), 0.0f};
      best_id = kNoId;
      for (int c = 0; c < chunks; ++c) {
        const uint4 q = sh.ex.part[it & 1][c];
        const Sum o = {__uint_as_float(q.x), __uint_as_float(q.y)};
        if (!greedy) {
          total = sum_merge(total, o, scale);
        } else if (pair_beats(o.m, static_cast<int32_t>(q.z), total.m, best_id)) {
          total.m = o.m;
          best_id = static_cast<int32_t>(q.z);
        }
      }
      // a row without terms is 0 (its sum is 0; a NaN stays)
      const float m = total.m == neg_inf() ? 0.0f : total.m;
      const float inv = total.s == 0.0f ? 0.0f : 1.0f / total.s;

      // ---- the probabilities
      float *out = probs + row * ldp;
      auto value = [&](float x) { return ex2((x - m) * scale) * inv; };
      const bool aligned = (reinterpret_cast<uintptr_t>(out + pc.b0) & 15u) == 0;
      r = later(at, kept, slots);
      for (int i = 0; i < pc.stages; ++i) {
        const bool again = i >= pc.stages - kept;  // loaded a second time
        const int j = again ? i - (pc.stages - kept) : kept + i;
        if (again) ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        const uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT> * kVec, pc.b1 - c);
        float *o = out + c;
        if (aligned) {
          const int hot = best_id - c;
#pragma unroll
          for (int u = 0; u < kVecPerThread * kVec / 4; ++u) {
            const int unit = u * kT + tid;
            if (unit * 4 >= n) continue;
            float4 p;
            if (greedy) {
              const int e = hot - unit * 4;
              p = make_float4(e == 0 ? 1.0f : 0.0f, e == 1 ? 1.0f : 0.0f, e == 2 ? 1.0f : 0.0f,
                              e == 3 ? 1.0f : 0.0f);
            } else {
              float x[4];
              load4<kBf16>(st, unit, x);
              p = make_float4(value(x[0]), value(x[1]), value(x[2]), value(x[3]));
            }
            reinterpret_cast<float4 *>(o)[unit] = p;
          }
        } else {
          for (int e = tid; e < n; e += kT)
            o[e] = greedy ? (c + e == best_id ? 1.0f : 0.0f)
                          : value(read_elem<kBf16>(reinterpret_cast<const char *>(st), e));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
        step(r, slots);
      }
      if (!ok) {  // (every warp keeps to the rows' barriers)
        if (lane == 0) raise_abort(&sh.ring.abort, err);
        continue;
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, tid);
        if (j >= 0) out[j] = greedy ? (j == best_id ? 1.0f : 0.0f) : value(end_x[side]);
      }
      if (chunk == chunks - 1)
        for (int j = valid + tid; j < width; j += kT) out[j] = 0.0f;
      at = later(at, num_loads(pc.stages, slots, true), slots);
    }
  }
  leave(sh.ring, chunks);
}

template <bool kBf16, int kT>
cudaError_t launch_rows(const void *logits, int64_t rows, int64_t ld, int64_t width, int64_t valid,
                        const float *temperature, float *probs, int64_t ldp, uint32_t *err,
                        cudaStream_t stream) {
  auto kern = probs_kernel<kBf16, kT>;
  const RowKernel k = {reinterpret_cast<const void *>(kern), kT + 32, kRingBytes<kT>,
                       (kBf16 ? 0 : 1) + (kT == 256 ? 0 : 2)};
  int64_t resident[6];
  const cudaError_t e = resident_clusters(k, resident);
  if (e != cudaSuccess) return e;
  const int chunks =
      kT == 256 ? pick_chunks(rows, valid * (kBf16 ? 2 : 4), kRingBytes<kT>, 0.625, resident) : 1;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  row_launch(k, rows, chunks, resident, stream, attr, cfg);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits),
                            ld * (kBf16 ? 2 : 4), rows, static_cast<int>(valid),
                            static_cast<int>(width), temperature, probs, ldp, chunks, err);
}

}  // namespace

cudaError_t launch_probs(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                         int64_t valid, const float *temperature, float *probs, int64_t ldp,
                         int num_sms, uint32_t *err, cudaStream_t stream) {
  const bool small = small_rows(rows, valid * (dtype == SGA_BF16 ? 2 : 4), num_sms);
  auto launch = dtype == SGA_BF16 ? (small ? launch_rows<true, 64> : launch_rows<true, 256>)
                                  : (small ? launch_rows<false, 64> : launch_rows<false, 256>);
  return launch(logits, rows, ld, width, valid, temperature, probs, ldp, err, stream);
}

}  // namespace sga
