// distill.cu -- divergence of a draft model's rows from a teacher's top logits,
// and its gradient with respect to the draft's logits.
//
// With y = x / T, s_j = e^(y_j - lse), the teacher's list (id_i, p_i) and p_r the
// teacher's probability off the list:
//   loss   = sum_i p_i (log p_i - log s_id_i) + p_r (log p_r - (lse_rest - lse)),
//   grad_j = g / T (P s_j - sum over id_i = j of p_i - [j off the list] p_r
//            e^(y_j - lse_rest)),   P = sum_i p_i + p_r.
// Off the list both terms are multiples of e^(y_j - lse_rest), the factor being
// P e^(lse_rest - lse) - p_r: one exponential per id.  The list's few ids are
// written after the row's pass.
//
// lse_rest is summed without the listed ids: as a difference of sums it would
// lose what a draft that agrees with its teacher leaves off the list.  The
// teacher's few numbers are kept in 64 bits, p_r being 1 less a sum near 1.
#include <type_traits>

#include "rowring.cuh"

namespace sga {
namespace {

// ------------------------------------------------------------- the teacher

// A row's list, and what follows from it.
struct List {
  int32_t id[SGA_MAX_TEACHER];  // -1: no entry
  float z[SGA_MAX_TEACHER];
  float x[SGA_MAX_TEACHER];     // the row's logits there
  double p[SGA_MAX_TEACHER];    // probabilities; at an id's first entry those of all its entries
  uint8_t first[SGA_MAX_TEACHER];  // no earlier entry has the id
  Sum listed;                   // sum of exponentials of the listed ids
  double sum_p, rest_p;         // probability on and off the list
  double part;                  // sum of p_i (log p_i - y_i)
  float total, on_list, rest;   // sum_p + rest_p, sum_p, rest_p
  int any;                      // the row has a teacher
};

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One warp works out a row's list; l.id (entries only), l.z and l.x are given.
__device__ __forceinline__ void teacher_row(List &l, int k, const float *teacher_lse, int64_t row,
                                            double inv_t, float scale, int lane) {
  // the normaliser, and which entries are the first of their id
  double norm = 0.0, most = -INFINITY;
  bool some = false, again = false;
#pragma unroll 1
  for (int i = lane; i < k; i += 32) {
    const int32_t id = l.id[i];
    bool first = id >= 0;
    if (id >= 0) {
      some = true;
      const double z = l.z[i] * inv_t;
      if (!(z <= most)) most = z;  // (a NaN goes on into the sums)
#pragma unroll 4
      for (int j = 0; j < i; ++j) first = first && l.id[j] != id;
      again = again || !first;
    }
    l.first[i] = first;
  }
  bool any = __any_sync(0xffffffffu, some);
  again = __any_sync(0xffffffffu, again);
  if (teacher_lse != nullptr) {
    norm = teacher_lse[row];
  } else {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double o = __shfl_xor_sync(0xffffffffu, most, off);
      if (!(o <= most)) most = o;
    }
    any = any && most != -INFINITY;
    double sum = 0.0;
#pragma unroll 1
    for (int i = lane; i < k; i += 32)
      if (l.id[i] >= 0) sum += exp(l.z[i] * inv_t - most);
    norm = most + log(warp_sum_f64(sum));
  }
  // probabilities, the list's part of the loss, and its sum of exponentials
  double sum_p = 0.0, part = 0.0;
  Sum listed = {neg_inf(), 0.0f};
#pragma unroll 1
  for (int i = lane; i < k; i += 32) {
    double p = 0.0;
    if (l.id[i] >= 0 && any) {
      const double logp = l.z[i] * inv_t - norm;
      p = exp(logp);
      sum_p += p;
      if (!(p <= 0.0)) part += p * (logp - l.x[i] * inv_t);
    }
    l.p[i] = p;
    const float x = l.first[i] ? l.x[i] : neg_inf();
    if (x != neg_inf()) listed = sum_merge(listed, {is_nan(x) ? neg_inf() : x, x - x + 1.0f}, scale);
  }
  __syncwarp();
  sum_p = warp_sum_f64(sum_p);
  part = warp_sum_f64(part);
  listed = sum_warp(listed, scale);
  if (again) {  // (entries are visited in the same order by every CTA of a row)
#pragma unroll 1
    for (int i = lane; i < k; i += 32)
      if (l.first[i])
        for (int j = i + 1; j < k; ++j)
          if (l.id[j] == l.id[i]) l.p[i] += l.p[j];
  }
  const double rest = teacher_lse != nullptr && any ? (sum_p > 1.0 ? 0.0 : 1.0 - sum_p) : 0.0;
  if (lane == 0) {
    l.listed = listed;
    l.sum_p = sum_p;
    l.rest_p = rest;
    l.part = part;
    l.total = static_cast<float>(sum_p + rest);
    l.on_list = static_cast<float>(sum_p);
    l.rest = static_cast<float>(rest);
    l.any = any;
  }
  __syncwarp();
}

// ------------------------------------------------------------ loss (and gradient)

constexpr int kPerLane = SGA_MAX_TEACHER / 32;  // entries of a list per lane

// Stages of the ring: the most that fits two CTAs per SM (16 KB), or eight (4 KB).
template <int kT>
constexpr int kSlots = kT == 256 ? 6 : 5;
template <int kT>
constexpr int kRingBytes = kSlots<kT> * kStageVec<kT> * 16;

template <int kT>
struct DistillShared {
  Ring ring;
  uint64_t ready[2], stored[2];  // a row's list is there; its gradient is written
  Exchange<1> ex;
  Sum warp_sum[kT / 32];
  Sum total[2], rest[2];  // the row's sums, for the list warp
  List list[2];
};

// Gradient of 16 bytes of logits off the list: coef 2^((x - m) scale).
template <bool kBf16>
__device__ __forceinline__ uint4 grad_vec(const uint4 q, float m, float scale, float coef) {
  const uint64_t m2 = pack_f32(-m, -m), s2 = pack_f32(scale, scale), c2 = pack_f32(coef, coef);
  auto pair = [&](float &lo, float &hi) {
    unpack_f32(mul2(add2(pack_f32(lo, hi), m2), s2), lo, hi);
    unpack_f32(mul2(pack_f32(ex2(lo), ex2(hi)), c2), lo, hi);
  };
  uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (kBf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = bf16_lo(w[i]), hi = bf16_hi(w[i]);
      pair(lo, hi);
      w[i] = pack2(lo, hi);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float lo = __uint_as_float(w[i]), hi = __uint_as_float(w[i + 1]);
      pair(lo, hi);
      w[i] = __float_as_uint(lo);
      w[i + 1] = __float_as_uint(hi);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row's piece is read once and kept (rowring.cuh) for the gradient.  Before a warp
// sums its part of a stage it takes the listed logits out (-inf in their place), so
// that the sum is the rest's and no other logit is compared with an id.  A list warp
// works out the teacher's numbers a row ahead, reading the listed logits by itself,
// and writes the loss and the listed ids' gradients a row behind.
template <bool kBf16, int kT, bool kGrad>
__global__ void __launch_bounds__(kT + 64, kPerSm<kT>)
    distill_kernel(const char *logits, int64_t ld_bytes, int64_t num_rows, int valid, int width,
                   DistillArgs in, int64_t ldg_bytes, int chunks, uint32_t *err) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  constexpr int kWarps = kT / 32;
  constexpr int slots = kSlots<kT>;
  constexpr uint32_t kMasked = kBf16 ? 0xff80ff80u : 0xff800000u;  // -inf
  extern __shared__ __align__(128) uint4 buf[];
  __shared__ DistillShared<kT> sh;
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const int64_t row0 = blockIdx.x / chunks, row_step = gridDim.x / chunks;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const volatile int *abort_flag = &sh.ring.abort;
  const double inv_t = 1.0 / static_cast<double>(in.temperature);
  const float scale = static_cast<float>(1.4426950408889634 * inv_t);
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&sh.ring.full[i]), 1);
      mbar_init(smem_u32(&sh.ring.empty[i]), kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.ready[i]), 1);
      mbar_init(smem_u32(&sh.stored[i]), kWarps);
    }
    sh.ring.abort = 0;
    exchange_init(sh.ex, chunks);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (chunks > 1)  // every CTA's barriers are ready
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  pdl_wait();

  if (warp == kWarps) {
    copy_rows<kBf16, kT>(sh.ring, buf, slots, kGrad, logits, ld_bytes, row0, row_step, num_rows,
                         valid, chunk, chunks, lane, err);
    pdl_launch_dependents();
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------- list warp
    auto finish = [&](int64_t row, int64_t it) {
      const int par = static_cast<int>(it & 1);
      if (!warp_wait(smem_u32(&sh.stored[par]), static_cast<uint32_t>(it >> 1) & 1, abort_flag))
        return false;
      const List &l = sh.list[par];
      const Sum total = sh.total[par], rest = sh.rest[par];
      const bool bad = is_nan(total.s);
      const double rest_p = rest.s == 0.0f ? 0.0 : l.rest_p;
      if (chunk == 0 &&
          (in.out_loss != nullptr || in.out_lse != nullptr || in.out_lse_rest != nullptr)) {
        // lane 0: lse, lane 1: lse_rest, lane 2: log p_r
        const double lg =
            log(lane == 0 ? static_cast<double>(total.s)
                          : (lane == 1 ? static_cast<double>(rest.s) : rest_p));
        const Sum own = lane == 0 ? total : rest;
        const double v = bad ? nan("") : (own.s == 0.0f ? -INFINITY : own.m * inv_t + lg);
        const double lse = __shfl_sync(0xffffffffu, v, 0);
        const double lse_rest = __shfl_sync(0xffffffffu, v, 1);
        const double log_rest = __shfl_sync(0xffffffffu, lg, 2);
        if (lane == 1 && in.out_lse_rest != nullptr)
          in.out_lse_rest[row] = static_cast<float>(v);
        if (lane == 0) {
          if (in.out_lse != nullptr) in.out_lse[row] = static_cast<float>(v);
          double loss = l.part;
          if (lse != -INFINITY) loss += l.sum_p * lse;  // (else it is +inf or 0)
          if (!(rest_p <= 0.0)) loss += rest_p * (log_rest - (lse_rest - lse));
          if (!l.any) loss = 0.0;
          if (in.out_loss != nullptr) in.out_loss[row] = static_cast<float>(loss);
        }
      }
      if (kGrad && l.any && total.s != 0.0f) {
        const Piece pc = piece_of<kBf16, kT>(logits + row * ld_bytes, valid, chunk, chunks);
        char *g = static_cast<char *>(in.grad) + row * ldg_bytes;
        const float up = (in.grad_loss != nullptr ? in.grad_loss[row] : 1.0f) *
                         static_cast<float>(inv_t);
        const float of = (rest.s == 0.0f ? l.on_list : l.total) / total.s;
        for (int i = lane; i < in.k; i += 32) {
          const int32_t id = l.id[i];
          if (!l.first[i] || id < pc.c0 || id >= pc.c1) continue;
          const float s = of * ex2((l.x[i] - total.m) * scale);
          store_elem<kBf16>(g, id, up * (s - static_cast<float>(l.p[i])));
        }
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    int64_t it = 0;
    int32_t id[kPerLane];
    float z[kPerLane];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        const int i = r * 32 + lane;
        id[r] = i < in.k ? in.ids[row * in.k + i] : -1;
        z[r] = i < in.k ? in.logits[row * in.k + i] : 0.0f;
      }
    };
    if (row0 < num_rows) fetch(row0);
    for (int64_t row = row0; row < num_rows && ok; row += row_step, ++it) {
      List &l = sh.list[it & 1];
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        const int i = r * 32 + lane;
        if (i >= in.k) continue;
        const bool entry = id[r] >= 0 && id[r] < valid;
        l.id[i] = entry ? id[r] : -1;
        l.z[i] = z[r];
        l.x[i] = entry ? read_elem<kBf16>(logits + row * ld_bytes, id[r]) : neg_inf();
      }
      if (row + row_step < num_rows) fetch(row + row_step);
      __syncwarp();
      teacher_row(l, in.k, in.lse, row, inv_t, scale, lane);
      if (lane == 0) mbar_arrive(smem_u32(&sh.ready[it & 1]));
      if (it > 0) ok = finish(row - row_step, it - 1);
    }
    if (ok && it > 0) ok = finish(row0 + (it - 1) * row_step, it - 1);
    if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
  } else {
    // ------------------------------------------------------------- consumers
    const float room = 12.0f / scale;
    Place at = {0, 0};
    bool ok = true;
    int64_t it = 0;
    int32_t next_id[kPerLane];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        next_id[r] = -1;
        if (r * 32 + lane < in.k) next_id[r] = in.ids[row * in.k + r * 32 + lane];
      }
    };
    if (row0 < num_rows) fetch(row0);
    for (int64_t row = row0; row < num_rows; row += row_step, ++it) {
      const int par = static_cast<int>(it & 1);
      const Piece pc = piece_of<kBf16, kT>(logits + row * ld_bytes, valid, chunk, chunks);
      int32_t id[kPerLane];
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) id[r] = next_id[r];
      if (row + row_step < num_rows) fetch(row + row_step);
      float up = static_cast<float>(inv_t);
      if (kGrad && in.grad_loss != nullptr) up *= in.grad_loss[row];
      // the single elements at the piece's ends (warp 0), without listed ones
      float end_x[2] = {neg_inf(), neg_inf()};
      if (warp == 0 && (pc.c0 < pc.b0 || pc.b1 < pc.c1)) {
        uint32_t mask = 0;
#pragma unroll
        for (int r = 0; r < kPerLane; ++r) {
          if (id[r] >= pc.c0 && id[r] < pc.b0) mask |= 1u << (id[r] - pc.c0);
          if (id[r] >= pc.b1 && id[r] < pc.c1) mask |= 256u << (id[r] - pc.b1);
        }
        mask = __reduce_or_sync(0xffffffffu, mask);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int j = end_column(pc, side, tid);
          if (j >= 0 && !((mask >> (side * 8 + tid)) & 1)) end_x[side] = read_elem<kBf16>(pc.p, j);
        }
      }
      // ---- the sum off the list
      RunSum a = {0.0f, neg_inf(), 0u};
      Place r = at;
      const int kept = kGrad ? max(0, pc.stages - slots) : pc.stages;  // the first that stays
      for (int j = 0; j < pc.stages; ++j) {
        ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
        // listed logits among this warp's vectors
        bool mine[kPerLane], here = false;
#pragma unroll
        for (int s = 0; s < kPerLane; ++s) {
          mine[s] = false;
          if (s * 32 >= in.k) continue;
          const uint32_t e = static_cast<uint32_t>(id[s] - c);
          mine[s] = e < static_cast<uint32_t>(n * kVec) &&
                    static_cast<int>(e / (32 * kVec)) % kWarps == warp;
          here = here || mine[s];
        }
        if (__any_sync(0xffffffffu, here)) {
#pragma unroll
          for (int s = 0; s < kPerLane; ++s)
            if (mine[s]) store_elem<kBf16>(reinterpret_cast<char *>(st), id[s] - c, neg_inf());
          // (the slot's next copy is ordered behind these writes)
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        uint4 q[kVecPerThread];
#pragma unroll
        for (int u = 0; u < kVecPerThread; ++u) {
          const int i = u * kT + tid;
          q[u] = i < n ? st[i] : make_uint4(kMasked, kMasked, kMasked, kMasked);
        }
        uint4 most = q[0];
#pragma unroll
        for (int u = 1; u < kVecPerThread; ++u) most = vec_larger<kBf16>(most, q[u]);
        sum_rebase(a, vec_max<kBf16>(most), scale, room);
#pragma unroll
        for (int u = 0; u < kVecPerThread; ++u) sum_vector<kBf16>(a, q[u], scale);
        if (j < kept) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
        }
        step(r, slots);
      }
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        sum_rebase(a, end_x[side], scale, room);
        sum_add(a, end_x[side], neg_inf(), scale);
      }
      // ---- joined over the warps and the cluster
      Sum rest = sum_warp(sum_result(a), scale);
      if (lane == 0) sh.warp_sum[warp] = rest;
      consumers_sync<kT>();
      if (warp == 0)
        rest = sum_warp(lane < kWarps ? sh.warp_sum[lane] : Sum{neg_inf(), 0.0f}, scale);
      // (the list warp has read its logits before any CTA of the row may write over them)
      ok = ok && warp_wait(smem_u32(&sh.ready[par]), static_cast<uint32_t>(it >> 1) & 1, abort_flag);
      const uint4 part[1] = {make_uint4(__float_as_uint(rest.m), __float_as_uint(rest.s), 0u, 0u)};
      ok = exchange<kT>(sh.ex, part, it, chunk, chunks, tid, ok, abort_flag);
      if (!ok) {  // (every warp keeps to the rows' barriers)
        if (lane == 0) raise_abort(&sh.ring.abort, err);
        continue;
      }
      rest = {neg_inf(), 0.0f};
      for (int c = 0; c < chunks; ++c) {
        const uint4 q = sh.ex.part[par][c][0];
        rest = sum_merge(rest, {__uint_as_float(q.x), __uint_as_float(q.y)}, scale);
      }
      const List &l = sh.list[par];
      const Sum total = sum_merge(l.listed, rest, scale);
      if (tid == 0) {
        sh.total[par] = total;
        sh.rest[par] = rest;
      }
      if (kGrad) {
        // ---- the gradient off the list
        const bool bad = is_nan(total.s);
        const bool live = l.any && total.s != 0.0f;
        const float m = rest.m == neg_inf() ? 0.0f : rest.m;
        float coef = nan_f32();
        if (!bad) {
          const float share = sum_at(rest, total.m, scale) / total.s;  // s_r
          coef = rest.s == 0.0f ? 0.0f : up * fmaf(l.total, share, -l.rest) / rest.s;
        }
        char *g = static_cast<char *>(in.grad) + row * ldg_bytes;
        auto value = [&](float x) { return live ? coef * ex2((x - m) * scale) : 0.0f; };
        r = later(at, kept, slots);
        for (int i = 0; i < pc.stages; ++i) {
          const bool again = i >= pc.stages - kept;  // loaded a second time
          const int j = again ? i - (pc.stages - kept) : kept + i;
          if (again) ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
          if (!ok) break;
          const uint4 *st = buf + r.slot * kStageVec<kT>;
          const int c = pc.b0 + j * kStageVec<kT> * kVec;
          const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
          char *o = g + static_cast<int64_t>(c) * kElt;
          // bytes of the stage before the output's first whole vector
          const int skip = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(o) & 15u)) & 15u);
          uint4 *ov = reinterpret_cast<uint4 *>(o + skip);
          if (skip == 0) {
#pragma unroll
            for (int u = 0; u < kVecPerThread; ++u) {
              const int v = u * kT + tid;
              if (v < n)
                __stcs(ov + v, live ? grad_vec<kBf16>(st[v], m, scale, coef) : make_uint4(0, 0, 0, 0));
            }
          } else {
            for (int v = tid; v < n - 1; v += kT)
              __stcs(ov + v, live ? grad_vec<kBf16>(bytes_of(st[v], st[v + 1], skip), m, scale, coef)
                                  : make_uint4(0, 0, 0, 0));
            // the vector's worth of elements at both ends
            if (tid < kVec) {
              const int e = tid * kElt < skip ? tid : (n - 1) * kVec + tid;
              store_elem<kBf16>(o, e, value(read_elem<kBf16>(reinterpret_cast<const char *>(st), e)));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
          step(r, slots);
        }
        if (!ok) {
          if (lane == 0) raise_abort(&sh.ring.abort, err);
          continue;
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int j = end_column(pc, side, tid);
          if (j >= 0) store_elem<kBf16>(g, j, value(end_x[side]));
        }
        if (chunk == chunks - 1)
          for (int j = valid + tid; j < width; j += kT) store_elem<kBf16>(g, j, 0.0f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.stored[par]));
      at = later(at, num_loads(pc.stages, slots, kGrad), slots);
    }
  }
  if (chunks > 1) {  // no CTA ends while another may write to it
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
}

template <bool kBf16, int kT, bool kGrad>
cudaError_t launch_rows(const void *logits, int64_t rows, int64_t ld, int64_t width, int64_t valid,
                        const DistillArgs &in, int64_t ldg, int chunks, int num_sms, uint32_t *err,
                        cudaStream_t stream) {
  constexpr int kElt = kBf16 ? 2 : 4;
  auto kern = distill_kernel<kBf16, kT, kGrad>;
  const cudaError_t e =
      set_smem_once(reinterpret_cast<const void *>(kern), kRingBytes<kT>,
                    (kBf16 ? 0 : 1) + (kT == 256 ? 0 : 2) + (kGrad ? 0 : 4));
  if (e != cudaSuccess) return e;
  const int64_t resident = resident_clusters(chunks, kPerSm<kT>, num_sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows < resident ? rows : resident) * chunks));
  cfg.blockDim = dim3(kT + 64);
  cfg.dynamicSmemBytes = kRingBytes<kT>;
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
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * kElt, rows,
                            static_cast<int>(valid), static_cast<int>(width), in, ldg * kElt,
                            chunks, err);
}

// ---------------------------------------------------------- gradient alone

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // loads in flight per thread

// One pass from the saved sums, a CTA per piece of a row (nothing but the teacher's
// few numbers is shared along it).  The first loads are under way while one warp
// works those out.  kShift: some rows of the logits and of the gradient lie at
// different 16-byte offsets.
template <bool kBf16, bool kShift>
__global__ void __launch_bounds__(kThreads)
    distill_grad_kernel(const char *logits, int64_t ld_bytes, int valid, int width, DistillArgs in,
                        int chunks, int64_t ldg_bytes) {
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  __shared__ List l;
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const int64_t row = blockIdx.x / chunks;
  const int tid = threadIdx.x;
  const char *x = logits + row * ld_bytes;
  char *g = static_cast<char *>(in.grad) + row * ldg_bytes;
  pdl_wait();
  // this CTA's columns: whole 16-byte groups of the output row
  int head = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(g) & 15u)) & 15u) / kElt);
  if (head > width) head = width;
  const int nvec = (width - head) / kVec;
  const int v0 = static_cast<int>(static_cast<int64_t>(nvec) * chunk / chunks);
  const int v1 = static_cast<int>(static_cast<int64_t>(nvec) * (chunk + 1) / chunks);
  const int c0 = chunk == 0 ? 0 : head + v0 * kVec;
  const int c1 = chunk == chunks - 1 ? width : head + v1 * kVec;
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
  uint4 q[kBatch], q1[kBatch];
  auto load = [&](int v) {
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
  };
  load(vs + tid);

  const double inv_t = 1.0 / static_cast<double>(in.temperature);
  const float scale = static_cast<float>(1.4426950408889634 * inv_t);
  const float lse = in.in_lse[row];
  const float lse_rest = in.in_lse_rest != nullptr ? in.in_lse_rest[row] : neg_inf();
  const float up =
      (in.grad_loss != nullptr ? in.grad_loss[row] : 1.0f) * static_cast<float>(inv_t);
  if (tid < 32) {
    for (int i = tid; i < in.k; i += 32) {
      const int32_t id = in.ids[row * in.k + i];
      const bool entry = id >= 0 && id < valid;
      l.id[i] = entry ? id : -1;
      l.z[i] = in.logits[row * in.k + i];
      // (read before the pass may write over it)
      l.x[i] = entry && id >= c0 && id < c1 ? read_elem<kBf16>(x, id) : neg_inf();
    }
    __syncwarp();
    teacher_row(l, in.k, in.lse, row, inv_t, scale, tid);
  }
  __syncthreads();
  const bool live = l.any && lse != neg_inf();
  // off the list relative to lse_rest: s_r <= 1 times e^(y_j - lse_rest), where s_j itself may
  // vanish (a rest that is masked by a low value)
  const bool by_rest = l.rest > 0.0f && lse_rest != neg_inf();
  const float total = by_rest ? l.total : l.on_list;
  const float base = -(by_rest ? lse_rest : lse) * kLog2e;
  const float coef =
      up * (by_rest ? fmaf(total, ex2((lse_rest - lse) * kLog2e), -l.rest) : total);
  auto value = [&](float v) { return coef * ex2(fmaf(v, scale, base)); };
  auto one = [&](int j) {
    store_elem<kBf16>(g, j, live && j < valid ? value(read_elem<kBf16>(x, j)) : 0.0f);
  };
  if (chunk == 0 && tid < head) one(tid);
  for (int v = vs + tid; v < ve; v += kBatch * kThreads) {
    if (v != vs + tid) load(v);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (v + u * kThreads >= ve) continue;
      const uint4 xq = kShift && offset != 0 ? bytes_of(q[u], q1[u], offset) : q[u];
      uint32_t w[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!live)
          w[i] = 0u;
        else if (kBf16)
          w[i] = pack2(value(bf16_lo(w[i])), value(bf16_hi(w[i])));
        else
          w[i] = __float_as_uint(value(__uint_as_float(w[i])));
      }
      __stcs(reinterpret_cast<uint4 *>(gv) + v + u * kThreads, make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  if (vs > v0)
    for (int j = head + v0 * kVec + tid; j < head + vs * kVec; j += kThreads) one(j);
  for (int j = head + ve * kVec + tid; j < c1; j += kThreads) one(j);
  pdl_launch_dependents();
  __syncthreads();
  if (live && tid < in.k && l.first[tid] && l.id[tid] >= c0 && l.id[tid] < c1) {
    const float s = total * ex2(fmaf(l.x[tid], scale, -lse * kLog2e));
    store_elem<kBf16>(g, l.id[tid], up * (s - static_cast<float>(l.p[tid])));
  }
}

cudaError_t launch_grad(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                        int64_t valid, const DistillArgs &in, int64_t ldg, int num_sms,
                        cudaStream_t stream) {
  const int elt = dtype == SGA_BF16 ? 2 : 4;
  // pieces of 64 KB, or down to 16 KB where the SMs would not have eight each
  const int64_t bytes = width * elt;
  int64_t piece = 65536;
  while (piece > 16384 && rows * ((bytes + piece - 1) / piece) < 8 * num_sms) piece /= 2;
  int64_t chunks = (bytes + piece - 1) / piece;
  if (rows * chunks > (int64_t(1) << 30)) chunks = (int64_t(1) << 30) / rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * chunks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool shift =
      ((reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(in.grad)) |
       ((ld - ldg) * elt)) % 16 != 0;
  auto kern = dtype == SGA_BF16
                  ? (shift ? distill_grad_kernel<true, true> : distill_grad_kernel<true, false>)
                  : (shift ? distill_grad_kernel<false, true> : distill_grad_kernel<false, false>);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * elt,
                            static_cast<int>(valid), static_cast<int>(width), in,
                            static_cast<int>(chunks), ldg * elt);
}

}  // namespace

cudaError_t launch_distill(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                           int64_t valid, const DistillArgs &args, int64_t ldg, int num_sms,
                           uint32_t *err, cudaStream_t stream) {
  if (args.in_lse != nullptr)
    return launch_grad(logits, dtype, rows, ld, width, valid, args, ldg, num_sms, stream);
  const int64_t bytes = valid * (dtype == SGA_BF16 ? 2 : 4);
  const bool kept = args.grad != nullptr;
  const bool small = small_rows(rows, bytes, num_sms);
  const int chunks = small ? 1 : pick_chunks(rows, bytes, kept ? kRingBytes<256> : 0, num_sms);
  auto launch = [&](auto bf16, auto grad) {
    constexpr bool kBf16 = decltype(bf16)::value, kGrad = decltype(grad)::value;
    return (small ? launch_rows<kBf16, 64, kGrad> : launch_rows<kBf16, 256, kGrad>)(
        logits, rows, ld, width, valid, args, ldg, chunks, num_sms, err, stream);
  };
  if (dtype == SGA_BF16)
    return kept ? launch(std::true_type{}, std::true_type{})
                : launch(std::true_type{}, std::false_type{});
  return kept ? launch(std::false_type{}, std::true_type{})
              : launch(std::false_type{}, std::false_type{});
}

}  // namespace sga
