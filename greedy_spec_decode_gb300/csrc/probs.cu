// probs.cu -- probabilities of logits rows at a temperature.
//
// p_j = 2^((x_j - m) log2e / T) / sum_i 2^(...), m a logit within 2^12 (in terms)
// of the row's maximum, by which the exponents are exact differences at any
// offset and temperature.  A greedy row (T = 0) is 1 at its argmax.
#include "rowring.cuh"

namespace sga {
namespace {

// Long rows (kT 256) and short ones (64): CTAs per SM and stages of the ring (16 or
// 4 KB), the most that fits.
template <int kT>
struct Form {
  static constexpr int kPerSm = kT == 256 ? 1 : 6;
  static constexpr int kSlots = kT == 256 ? 13 : 8;
  static constexpr int kRingBytes = kSlots * kStageVec<kT> * 16;
  static constexpr int kThreads = 2 * kT + 32;
};

constexpr uint32_t kHeld = 4;  // rows between a sum and its output

template <int kT>
struct ProbsShared {
  Ring ring;
  uint64_t stored[kHeld];  // a row's probabilities are written
  Exchange<2 * kHeld> ex;
  Sum warp_sum[2][kT / 32];
  int32_t warp_id[2][kT / 32];
};

// Logits 4 unit + kShift .. 4 unit + kShift + 3 of a stage.
template <bool kBf16, int kShift>
__device__ __forceinline__ void load4(const uint4 *stage, int unit, float (&x)[4]) {
  if constexpr (kBf16) {
    const uint2 *p = reinterpret_cast<const uint2 *>(stage);
    uint2 q = p[unit];
    if constexpr (kShift != 0) {
      const uint2 r = p[unit + 1];
      const uint4 v = shifted<2 * kShift>(make_uint4(q.x, q.y, r.x, r.y), make_uint4(0, 0, 0, 0));
      q = make_uint2(v.x, v.y);
    }
    x[0] = bf16_lo(q.x);
    x[1] = bf16_hi(q.x);
    x[2] = bf16_lo(q.y);
    x[3] = bf16_hi(q.y);
  } else {
    uint4 q = stage[unit];
    if constexpr (kShift != 0) q = shifted<4 * kShift>(q, stage[unit + 1]);
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
}

// Three kinds of warps: the copy warp fills the ring, the sum warps add up a row's
// piece (a greedy row: find its argmax), the output warps write the probabilities of
// what the ring has kept, up to kHeld rows behind.
template <bool kBf16, int kT>
__global__ void __launch_bounds__(Form<kT>::kThreads, Form<kT>::kPerSm)
    probs_kernel(const char *logits, int64_t ld_bytes, int64_t num_rows, int valid, int width,
                 const float *temperature, float *probs, int64_t ldp, int chunks, uint32_t *err) {
  constexpr int slots = Form<kT>::kSlots;
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  constexpr int kWarps = kT / 32;
  constexpr uint32_t kMasked = kBf16 ? 0xff80ff80u : 0xff800000u;  // -inf
  extern __shared__ __align__(128) uint4 buf[];
  __shared__ ProbsShared<kT> sh;
  const auto walk = walk_of<false>(num_rows, chunks);
  const uint32_t num_its = walk.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const volatile int *abort_flag = &sh.ring.abort;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&sh.ring.full[i]), 1);
      mbar_init(smem_u32(&sh.ring.empty[i]), ring_arrivals(kWarps));
    }
    for (uint32_t i = 0; i < kHeld; ++i) mbar_init(smem_u32(&sh.stored[i]), kWarps);
    sh.ring.abort = 0;
    exchange_init(sh.ex, chunks);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (chunks > 1)  // every CTA's barriers are ready
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  pdl_wait();

  auto piece = [&](uint32_t it) {
    return piece_of<kBf16, kT>(logits + walk.row(it) * ld_bytes, valid, walk.chunk, chunks);
  };
  auto temp = [&](uint32_t it) {
    return temperature != nullptr && it < num_its ? temperature[walk.row(it)] : 1.0f;
  };
  auto scale_of = [](float t) { return t > 0.0f ? fminf(kLog2e / t, 3e38f) : nan_f32(); };
  bool ok = true;
  float t_next = temp(0);
  if (warp < kWarps) {
    // ------------------------------------------------------------- sum warps
    Place at = {0, 0};
    for (uint32_t it = 0; it < num_its; ++it) {
      const Piece pc = piece(it);
      const float t = t_next;
      t_next = temp(it + 1);
      const bool greedy = t == 0.0f;
      const float scale = scale_of(t), room = 12.0f / scale;
      RunSum a = {0.0f, neg_inf(), 0u};
      float best = neg_inf();
      int best_stage = -1;
      int32_t best_id = kNoId;
      // the single elements at the row's ends
      float end_x[2] = {neg_inf(), neg_inf()};
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, tid);
        if (j >= 0) end_x[side] = read_elem<kBf16>(pc.p, j);
      }
      Place r = at;
      const int kept = max(0, pc.stages - slots);  // the first stage that stays
      for (int j = 0; j < pc.stages; ++j) {
        ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        const uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
        uint4 q[kVecPerThread];
        if (n == kStageVec<kT>) {
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) q[u] = st[u * kT + tid];
        } else {
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) {
            const int i = u * kT + tid;
            q[u] = i < n ? st[i] : make_uint4(kMasked, kMasked, kMasked, kMasked);
          }
        }
        uint4 most = q[0];
#pragma unroll
        for (int u = 1; u < kVecPerThread; ++u) most = vec_larger<kBf16>(most, q[u]);
        if (greedy) {
          const float v = vec_max<kBf16>(most);
          if (scan_better(v, best)) {
            best = v;
            best_stage = j;
          }
        } else {
          sum_rebase(a, vec_max<kBf16>(most), scale, room);
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) sum_vector<kBf16>(a, q[u], scale);
        }
        sum_frees(sh.ring, r, j, pc.stages, slots, lane);
        step(r, slots);
      }
      if (greedy && ok) {
        // where the warp's best logit is (a first id, if nothing is above -inf)
        float top = best;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
          top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (best_stage < 0) {
          if (tid < (pc.b1 - pc.b0) / kVec) best_id = pc.b0 + tid * kVec;
        } else if (best == top || is_nan(best)) {
          const int c = pc.b0 + best_stage * kStageVec<kT> * kVec;
          const uint4 *st = best_stage >= kept
                                ? buf + later(at, best_stage, slots).slot * kStageVec<kT>
                                : reinterpret_cast<const uint4 *>(pc.p + static_cast<int64_t>(c) * kElt);
          best = neg_inf();
          for (int u = 0; u < kVecPerThread; ++u) {
            const int i = u * kT + tid;
            if (i < (pc.b1 - c) / kVec) scan_vec<kBf16>(st[i], c + i * kVec, best, best_id);
          }
        }
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
      // ---- joined over the warps, and told
      Sum total = {best, 0.0f};
      auto join = [&] {
        if (greedy)
          warp_argmax(total.m, best_id);
        else
          total = sum_warp(total, scale);
      };
      if (!greedy) total = sum_result(a);
      join();
      if (lane == 0) {
        sh.warp_sum[it & 1][warp] = total;
        sh.warp_id[it & 1][warp] = best_id;
      }
      consumers_sync<kT>();  // (every warp keeps to the rows' barriers)
      if (warp == static_cast<int>(it % kWarps)) {
        total = lane < kWarps ? sh.warp_sum[it & 1][lane] : Sum{neg_inf(), 0.0f};
        best_id = lane < kWarps ? sh.warp_id[it & 1][lane] : kNoId;
        join();
        if (it >= kHeld)  // the buffer's last row has been read everywhere
          ok = ok && warp_wait(smem_u32(&sh.stored[it % kHeld]), (it / kHeld - 1) & 1, abort_flag);
        if (ok)
          exchange_tell(sh.ex, it,
                        make_uint4(__float_as_uint(total.m), __float_as_uint(total.s),
                                   static_cast<uint32_t>(best_id), 0u),
                        walk.chunk, chunks, lane);
      }
      // (every use of a slot is waited for, the second loads' too: see ring_arrivals)
      for (int j = 0; j < kept && ok; ++j, step(r, slots)) {
        ok = warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (ok) sum_frees(sh.ring, r, pc.stages + j, pc.stages, slots, lane);
      }
      if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
      at = later(at, num_loads(pc.stages, slots, true), slots);
    }
  } else if (warp < 2 * kWarps) {
    // ---------------------------------------------------------- output warps
    Place at = {0, 0};
    const int otid = tid - kT;
    for (uint32_t it = 0; it < num_its; ++it) {
      const Piece pc = piece(it);
      const float t = t_next;
      t_next = temp(it + 1);
      const bool greedy = t == 0.0f;
      const float scale = scale_of(t);
      float end_x[2] = {neg_inf(), neg_inf()};
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, otid);
        if (j >= 0) end_x[side] = read_elem<kBf16>(pc.p, j);
      }
      ok = exchange_wait(sh.ex, it, abort_flag);
      if (!ok) break;
      Sum total = {neg_inf(), 0.0f};
      int32_t best_id = kNoId;
      if (greedy) {
        for (int c = 0; c < chunks; ++c) {
          const uint4 q = sh.ex.part[it % (2 * kHeld)][c];
          const float v = __uint_as_float(q.x);
          if (pair_beats(v, static_cast<int32_t>(q.z), total.m, best_id)) {
            total.m = v;
            best_id = static_cast<int32_t>(q.z);
          }
        }
      } else {
        total = exchange_sum(sh.ex, it, chunks, lane, scale);
      }
      if (warp == kWarps) exchange_rearm(sh.ex, it, chunks, lane);
      // a row without terms is 0 (its sum is 0; a NaN stays)
      const float m = total.m == neg_inf() ? 0.0f : total.m;
      const float inv = total.s == 0.0f ? 0.0f : 1.0f / total.s;
      float *out = probs + walk.row(it) * ldp;
      auto value = [&](float x) { return ex2((x - m) * scale) * inv; };
      const uint64_t m2 = pack_f32(-m, -m), s2 = pack_f32(scale, scale), i2 = pack_f32(inv, inv);
      auto values = [&](const float (&x)[4]) {
        float4 p;
        unpack_f32(mul2(add2(pack_f32(x[0], x[1]), m2), s2), p.x, p.y);
        unpack_f32(mul2(add2(pack_f32(x[2], x[3]), m2), s2), p.z, p.w);
        unpack_f32(mul2(pack_f32(ex2(p.x), ex2(p.y)), i2), p.x, p.y);
        unpack_f32(mul2(pack_f32(ex2(p.z), ex2(p.w)), i2), p.z, p.w);
        return p;
      };
      const int kept = max(0, pc.stages - slots);
      Place r = later(at, kept, slots);
      for (int i = 0; i < pc.stages; ++i) {
        const bool again = i >= pc.stages - kept;  // loaded a second time
        const int j = again ? i - (pc.stages - kept) : kept + i;
        ok = warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        const uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT> * kVec, pc.b1 - c);
        float *o = out + c;
        // elements of the stage before the output's first whole vector
        const int skip = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(o) & 15u)) & 15u) / 4);
        const int units = (n - skip) / 4;
        float4 *ov = reinterpret_cast<float4 *>(o + skip);
        if (greedy) {
          const int hot = best_id - c - skip;
          for (int u = otid; u < units; u += kT) {
            const int e = hot - u * 4;
            __stcs(ov + u, make_float4(e == 0 ? 1.0f : 0.0f, e == 1 ? 1.0f : 0.0f,
                                       e == 2 ? 1.0f : 0.0f, e == 3 ? 1.0f : 0.0f));
          }
        } else if (skip == 0 && n == kStageVec<kT> * kVec) {
          constexpr int kUnits = kVecPerThread * kVec / 4;
#pragma unroll
          for (int h = 0; h < kUnits; h += 4) {
            float x[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u) load4<kBf16, 0>(st, (h + u) * kT + otid, x[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) __stcs(ov + (h + u) * kT + otid, values(x[u]));
          }
        } else if (skip == 0) {
          for (int u = otid; u < units; u += kT) {
            float x[4];
            load4<kBf16, 0>(st, u, x);
            __stcs(ov + u, values(x));
          }
        } else {
          with_shift<4>(skip * 4, [&](auto by) {
            constexpr int kUnits = kVecPerThread * kVec / 4;
            for (int h = 0; h < kUnits; h += 4) {
              float x[4][4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                load4<kBf16, decltype(by)::value / 4>(
                    st, min((h + u) * kT + otid, max(0, units - 1)), x[u]);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float4 p = values(x[u]);
                if ((h + u) * kT + otid < units) __stcs(ov + (h + u) * kT + otid, p);
              }
            }
          });
        }
        // both ends (at most six), a warp after the other
        if (otid / 32 == j % kWarps && lane < n - units * 4) {
          const int e = lane < skip ? lane : units * 4 + lane;
          o[e] = greedy ? (c + e == best_id ? 1.0f : 0.0f)
                        : value(read_elem<kBf16>(reinterpret_cast<const char *>(st), e));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
        step(r, slots);
      }
      if (!ok) break;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, otid);
        if (j >= 0) out[j] = greedy ? (j == best_id ? 1.0f : 0.0f) : value(end_x[side]);
      }
      if (walk.chunk == chunks - 1)
        for (int j = valid + otid; j < width; j += kT) out[j] = 0.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.stored[it % kHeld]));
      at = later(at, num_loads(pc.stages, slots, true), slots);
    }
    if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
  } else {
    auto load = [&](uint32_t it, Piece &q) {
      q = piece(it);
      return num_loads(q.stages, slots, true);
    };
    copy_rows<kBf16, kT>(sh.ring, buf, slots, true, num_its, load, lane, err);
    pdl_launch_dependents();
  }
  leave(sh.ring, chunks);
}

template <bool kBf16, int kT>
cudaError_t launch_rows(const void *logits, int64_t rows, int64_t ld, int64_t width, int64_t valid,
                        const float *temperature, float *probs, int64_t ldp, uint32_t *err,
                        cudaStream_t stream) {
  auto kern = probs_kernel<kBf16, kT>;
  const RowKernel k = {reinterpret_cast<const void *>(kern), Form<kT>::kThreads, Form<kT>::kRingBytes,
                       (kBf16 ? 0 : 1) + (kT == 256 ? 0 : 2)};
  int64_t resident[6];
  const cudaError_t e = resident_clusters(k, resident);
  if (e != cudaSuccess) return e;
  const int chunks =
      kT == 256 ? pick_chunks(rows, valid * (kBf16 ? 2 : 4), Form<kT>::kRingBytes, resident) : 1;
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
