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
#include "rowring.cuh"

namespace sga {
namespace {

// The call's arguments, and what follows from the temperature (a 64-bit division per
// thread would take some us of every CTA).
struct Args : DistillArgs {
  double inv_t;          // 1 / T
  float inv_t32, scale;  // 1 / T, log2(e) / T
};

// ------------------------------------------------------------- the teacher

// A row's list, and what follows from it.
struct alignas(16) List {
  int32_t id[SGA_MAX_TEACHER];  // -1: no entry
  float x[SGA_MAX_TEACHER];     // the row's logits there
  float p[SGA_MAX_TEACHER];     // at an id's first entry: the probability of all its entries
  uint8_t first[SGA_MAX_TEACHER];  // no earlier entry has the id
  Sum listed;                   // sum of exponentials of the listed ids
  double sum_p, rest_p;         // probability on and off the list
  double part;                  // sum of p_i (log p_i - y_i)
  float total, on_list, rest;   // sum_p + rest_p, sum_p, rest_p
  int any;                      // the row has a teacher
  float m, coef, of;            // (kBackward) off the list the gradient is coef 2^((x - m) scale)
  int anew;                     // (kBackward) the row's sums are taken anew
};

// The largest log-sum-exp that a gradient is worked out from: 2^-15 of the gradient is
// lost by its rounding to fp32.  Larger ones hold less of the sum (a rest masked by -1e9
// nothing), and one below T = 1 may be infinite though no logit is.
constexpr float kMostLse = 512.0f;

// Whether the gradient needs more of a row's sums than its saved lse and lse_rest hold.
__device__ __forceinline__ bool sums_lost(float lse, float lse_rest, const Args &in) {
  auto lost = [&](float v) {
    return fabsf(v) > kMostLse && !(v == neg_inf() && in.temperature >= 1.0f);
  };
  return lost(lse) || (in.lse != nullptr && lost(lse_rest));
}

// Sums of a and b over a warp: a's in lanes 0-15, b's in 16-31 (64-bit additions are
// 1/64 of the 32-bit rate here, so the two share theirs).
__device__ __forceinline__ void warp_sums_f64(double &a, double &b, int lane) {
  const bool low = lane < 16;
  double v = (low ? a : b) + __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

// log of a positive normal number: that of its mantissa in [0.7, 1.4] in 32 bits (off
// by 2^-25 of it), the exponent's part in 64.
__device__ __forceinline__ double log_of(float v) {
  const int e = (__float_as_int(v) - 0x3f3504f3) >> 23;
  return fma(static_cast<double>(e), 0.69314718055994530942,
             static_cast<double>(logf(__int_as_float(__float_as_int(v) - (e << 23)))));
}

constexpr int kPerLane = SGA_MAX_TEACHER / 32;

// A lane's entries of a list: r * 32 + lane.
struct Entries {
  int32_t id[kPerLane];  // -1: no entry
  float z[kPerLane], x[kPerLane];
};

// Loads a row's entries.
__device__ __forceinline__ void entries_load(Entries &e, const Args &in, int64_t row, int valid,
                                             int lane) {
#pragma unroll
  for (int r = 0; r < kPerLane; ++r) {
    const int i = r * 32 + lane;
    e.id[r] = i < in.k ? in.ids[row * in.k + i] : -1;
    e.z[r] = i < in.k ? in.logits[row * in.k + i] : 0.0f;
    if (e.id[r] < 0 || e.id[r] >= valid) e.id[r] = -1;
  }
}

// The row's logits there, if they are in columns [c0, c1).
template <bool kBf16>
__device__ __forceinline__ void entries_look(Entries &e, const char *x, int c0, int c1) {
#pragma unroll
  for (int r = 0; r < kPerLane; ++r)
    e.x[r] = e.id[r] >= 0 && e.id[r] >= c0 && e.id[r] < c1 ? read_elem<kBf16>(x, e.id[r]) : neg_inf();
}

// One warp works out a row's list from its entries, in kN rounds of 32 (their
// exponentials side by side: one takes 1100 cycles, mostly of latency).  The logits are
// needed last: their loads, which hang on those of the ids, run under the rest.
template <int kN>
__device__ __forceinline__ void teacher_rounds(List &l, const Entries &e, int k, float lse,
                                               bool with_lse, double inv_t, float scale,
                                               int lane) {
#pragma unroll
  for (int r = 0; r < kN; ++r) l.id[r * 32 + lane] = e.id[r];
  __syncwarp();
  // which entries are the first of their id
  bool first[kN], some = false, again = false;
  const int4 *ids = reinterpret_cast<const int4 *>(l.id);
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    const int i = r * 32 + lane;
    first[r] = e.id[r] >= 0;
    some = some || first[r];
#pragma unroll 4
    for (int j = 0; j < min(k, r * 32 + 32); j += 4) {
      const int4 o = ids[j >> 2];
      if ((o.x == e.id[r] && j < i) || (o.y == e.id[r] && j + 1 < i) ||
          (o.z == e.id[r] && j + 2 < i) || (o.w == e.id[r] && j + 3 < i))
        first[r] = false;
    }
    again = again || (e.id[r] >= 0 && !first[r]);
    l.first[i] = first[r];
  }
  bool any = __any_sync(0xffffffffu, some);
  again = __any_sync(0xffffffffu, again);
  // terms relative to the teacher's log-sum-exp, or to the list's largest
  double base = lse;
  if (!with_lse) {
    float most = neg_inf();
#pragma unroll
    for (int r = 0; r < kN; ++r)
      if (e.id[r] >= 0) most = max_nan(most, e.z[r]);  // (a NaN goes on into the sums)
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off));
    any = any && most != neg_inf();
    base = most * inv_t;
  }
  double t[kN], p[kN], sum = 0.0, part = 0.0;  // sum of p, of p (t - y)
#pragma unroll
  for (int r = 0; r < kN; ++r) t[r] = e.z[r] * inv_t - base;
#pragma unroll
  for (int r = 0; r < kN; ++r) p[r] = exp(t[r]);
  Sum listed = {neg_inf(), 0.0f};  // the list's sum of exponentials
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    if (e.id[r] < 0 || !any) p[r] = 0.0;
    sum += p[r];
    if (!(p[r] <= 0.0)) part += p[r] * (t[r] - e.x[r] * inv_t);
    l.x[r * 32 + lane] = e.x[r];
    const float x = first[r] ? e.x[r] : neg_inf();
    if (x != neg_inf()) listed = sum_merge(listed, {is_nan(x) ? neg_inf() : x, x - x + 1.0f}, scale);
  }
  warp_sums_f64(sum, part, lane);
  listed = sum_warp(listed, scale);
  float norm = 1.0f;
  if (!with_lse && any) {  // p_i = p / sum, log p_i = t - log sum
    const float s = static_cast<float>(sum);
    double inv = 1.0f / s;
    inv *= 2.0 - sum * inv;
    part = part * inv - (log_of(s) + (sum - s) * inv);
    norm = static_cast<float>(inv);
    sum = is_nan(s) ? sum : 1.0;
  }
#pragma unroll
  for (int r = 0; r < kN; ++r) l.p[r * 32 + lane] = static_cast<float>(p[r]) * norm;
  __syncwarp();
  if (again) {
#pragma unroll 1
    for (int i = lane; i < k; i += 32)
      if (l.first[i]) {
        float q = l.p[i];
        for (int j = i + 1; j < k; ++j)
          if (l.id[j] == l.id[i]) q += l.p[j];
        l.p[i] = q;
      }
  }
  const double rest = with_lse && any ? (sum > 1.0 ? 0.0 : 1.0 - sum) : 0.0;
  if (lane == 0) {
    l.listed = listed;
    l.sum_p = sum;
    l.rest_p = rest;
    l.part = part;
    l.total = static_cast<float>(sum + rest);
    l.on_list = static_cast<float>(sum);
    l.rest = static_cast<float>(rest);
    l.any = any;
  }
  __syncwarp();
}

__device__ __forceinline__ void teacher_row(List &l, const Entries &e, int k, float lse,
                                            bool with_lse, double inv_t, float scale, int lane) {
  if (k <= 32)
    teacher_rounds<1>(l, e, k, lse, with_lse, inv_t, scale, lane);
  else if (k <= 64)
    teacher_rounds<2>(l, e, k, lse, with_lse, inv_t, scale, lane);
  else
    teacher_rounds<kPerLane>(l, e, k, lse, with_lse, inv_t, scale, lane);
}

// ------------------------------------------------------------ loss (and gradient)

// The loss; the loss and its gradient; the gradient from the saved sums.
enum Mode { kLoss, kBoth, kBackward };

// Long rows (kT 256) and short ones (64): CTAs per SM, stages of the ring (16 or
// 4 KB; the most that fits), and list warps.  The loss alone keeps nothing, so more
// CTAs serve it better than longer rings (3 CTAs, 3 stages, 3 lists: 4096 x 152064 bf16
// 173 us, 4096 x 32000 45; 2, 5, 4: 182 and 48), and the gradient alone is like it
// (700 x 50257 fp32 47.1 us, 47.8).  Short rows, loss and gradient: 5, 7, 2 4096 x 8000 bf16
// with 64 entries 55 us, 4, 9, 2 72; 6, 6, 1 71.  The loss and the gradient alone, six CTAs and
// five: 4096 x 1000 / 8000 / 16000 18.9 / 21.7 / 29.7 us and 18.6 / 21.5 / 30.4 (at six the loss
// spills 92 bytes of registers), 19.4 / 27.4 / 46.8 and 19.8 / 28.8 / 47.4.  Between them (128,
// of 8 KB): 4096 x 32000 3, 7, 3 92 us (256: 100), 2, 12, 3 92, 2, 11, 4 95; 4096 x 24000 73.5
// (64: 79).
template <int kT, Mode kMode>
struct Form {
  static constexpr bool kSum = kMode != kBackward, kGrad = kMode != kLoss;
  static constexpr bool kKeeps = kMode == kBoth;
  static constexpr int kPerSm = kT == 256 ? (kKeeps ? 1 : 3) : kT == 128 ? 3 : (kKeeps ? 5 : 6);
  static constexpr int kSlots = kT == 256 ? (kKeeps ? 12 : 3) : kT == 128 ? 7 : (kKeeps ? 7 : 5);
  static constexpr int kLists = kT == 256 ? (kKeeps ? 4 : 3) : kT == 128 ? 3 : 2;
  static constexpr int kRingBytes = kSlots * kStageVec<kT> * 16;
  static constexpr int kThreads = (kMode == kBoth ? 2 : 1) * kT + 32 + 32 * kLists;
};

// kLists list warps work on rows in turn, each one ahead.
template <int kT, int kLists>
struct DistillShared {
  static constexpr int kHeld = 2 * kLists;  // lists held
  Ring ring;
  uint64_t ready[kHeld], stored[kHeld];  // a row's list is there; its gradient is written
  Exchange<2 * kHeld> ex;
  uint64_t joined;  // (kBackward) the parts of a row's sum are there
  Sum warp_sum[2][kT / 32];
  List list[kHeld];
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

// Four kinds of warps: the copy warp fills the ring; the sum warps add up a row's
// piece, taking the listed logits out of it first (-inf in their place: the sum is
// the rest's, and no other logit is compared with an id); the gradient warps write
// out what the ring has kept, a row or two behind; list warps work out the teacher's
// numbers a row ahead, reading the listed logits by themselves, and write the loss
// and the listed ids' gradients a row behind.  kBackward has no sum warps: a row's
// pieces have nothing in common but the teacher's numbers, and are rows of their own.
// Where the saved sums hold too little (sums_lost), the CTA of one of a row's pieces takes
// the whole row: its gradient warps sum it, as the sum warps do, and go over it again.
template <bool kBf16, int kT, Mode kMode>
__global__ void __launch_bounds__(Form<kT, kMode>::kThreads, Form<kT, kMode>::kPerSm)
    distill_kernel(const char *logits, int64_t ld_bytes, int64_t num_rows, int valid, int width,
                   Args in, int64_t ldg_bytes, int chunks, uint32_t *err) {
  using F = Form<kT, kMode>;
  using Shared = DistillShared<kT, F::kLists>;
  constexpr bool kGrad = F::kGrad;
  constexpr int kElt = kBf16 ? 2 : 4;
  constexpr int kVec = 16 / kElt;
  constexpr int kWarps = kT / 32;
  constexpr int kSumWarps = F::kSum ? kWarps : 0, kGradWarps = kGrad ? kWarps : 0;
  constexpr int slots = F::kSlots;
  constexpr uint32_t kHeld = Shared::kHeld;
  constexpr uint32_t kMasked = kBf16 ? 0xff80ff80u : 0xff800000u;  // -inf
  extern __shared__ __align__(128) uint4 buf[];
  __shared__ Shared sh;
  const auto walk = walk_of<kMode == kBackward>(num_rows, chunks);
  const uint32_t num_its = walk.n;
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const volatile int *abort_flag = &sh.ring.abort;
  const double inv_t = in.inv_t;
  const float scale = in.scale;
  if (tid == 0) {
    for (int i = 0; i < slots; ++i) {
      mbar_init(smem_u32(&sh.ring.full[i]), 1);
      mbar_init(smem_u32(&sh.ring.empty[i]), F::kKeeps ? ring_arrivals(kWarps) : kWarps);
    }
    for (uint32_t i = 0; i < kHeld; ++i) {
      mbar_init(smem_u32(&sh.ready[i]), 1);
      mbar_init(smem_u32(&sh.stored[i]), kWarps);
    }
    mbar_init(smem_u32(&sh.joined), kWarps);
    sh.ring.abort = 0;
    exchange_init(sh.ex, chunks);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (F::kSum && chunks > 1)  // every CTA's barriers are ready
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  pdl_wait();

  auto piece = [&](uint32_t it) {
    return piece_of<kBf16, kT>(logits + walk.row(it) * ld_bytes, valid, walk.chunk_of(it), chunks);
  };
  // the same where the row's sums are taken anew: all of it for one of its pieces (not the
  // first one of every row, which some of the CTAs have all of: gradient of 2048 x 200064
  // bf16 728 us where all rows are such ones, 368 so)
  auto has_row = [&](uint32_t it) {
    const uint32_t row = static_cast<uint32_t>(walk.row(it)), n = static_cast<uint32_t>(chunks);
    return walk.chunk_of(it) == static_cast<int>((row + row * n / gridDim.x) % n);
  };
  auto whole_piece = [&](uint32_t it) {
    Piece q = piece_of<kBf16, kT>(logits + walk.row(it) * ld_bytes, valid, 0, 1);
    if (!has_row(it)) q.c0 = q.b0 = q.b1 = q.c1 = q.stages = 0;
    return q;
  };
  // waits for the it-th row's list, or its stored gradient
  auto wait_held = [&](uint64_t (&bar)[kHeld], uint32_t it) {
    return warp_wait(smem_u32(&bar[it % kHeld]), (it / kHeld) & 1, abort_flag);
  };
  bool ok = true;
  // One warp's sum of a piece's logits off the list, from the stages at r on: the warp is
  // the by-th, the thread the at-th of those that share the piece.
  auto piece_sum = [&](const Piece &pc, const int32_t (&id)[kPerLane], Place &r, int at, int by) {
    // the single elements at the piece's ends (warp 0), without listed ones
    float end_x[2] = {neg_inf(), neg_inf()};
    if (by == 0 && (pc.c0 < pc.b0 || pc.b1 < pc.c1)) {
      uint32_t mask = 0;
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        if (id[r] >= pc.c0 && id[r] < pc.b0) mask |= 1u << (id[r] - pc.c0);
        if (id[r] >= pc.b1 && id[r] < pc.c1) mask |= 256u << (id[r] - pc.b1);
      }
      mask = __reduce_or_sync(0xffffffffu, mask);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, at);
        if (j >= 0 && !((mask >> (side * 8 + at)) & 1)) end_x[side] = read_elem<kBf16>(pc.p, j);
      }
    }
    // the stages (mod 32) with listed logits among this warp's vectors
    auto owns = [&](int c) {
      return c >= pc.b0 && c < pc.b1 &&
             static_cast<int>(static_cast<uint32_t>(c - pc.b0) / (32 * kVec)) % kWarps == by;
    };
    uint32_t listed = 0;
#pragma unroll
    for (int s = 0; s < kPerLane; ++s)
      if (owns(id[s])) listed |= 1u << ((id[s] - pc.b0) / (kStageVec<kT> * kVec) % 32);
    listed = __reduce_or_sync(0xffffffffu, listed);
    const float room = 12.0f / scale;
    RunSum a = {0.0f, neg_inf(), 0u};
    for (int j = 0; j < pc.stages; ++j) {
      ok = ok && warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
      if (!ok) break;
      uint4 *st = buf + r.slot * kStageVec<kT>;
      const int c = pc.b0 + j * kStageVec<kT> * kVec;
      const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
      if ((listed >> (j % 32)) & 1) {
#pragma unroll
        for (int s = 0; s < kPerLane; ++s)
          if (owns(id[s]) && id[s] >= c && id[s] < c + n * kVec)
            store_elem<kBf16>(reinterpret_cast<char *>(st), id[s] - c, neg_inf());
        // (the slot's next copy is ordered behind these writes)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      uint4 q[kVecPerThread];
      if (n == kStageVec<kT>) {
#pragma unroll
        for (int u = 0; u < kVecPerThread; ++u) q[u] = st[u * kT + at];
      } else {
#pragma unroll
        for (int u = 0; u < kVecPerThread; ++u) {
          const int i = u * kT + at;
          q[u] = i < n ? st[i] : make_uint4(kMasked, kMasked, kMasked, kMasked);
        }
      }
      uint4 most = q[0];
#pragma unroll
      for (int u = 1; u < kVecPerThread; ++u) most = vec_larger<kBf16>(most, q[u]);
      sum_rebase(a, vec_max<kBf16>(most), scale, room);
#pragma unroll
      for (int u = 0; u < kVecPerThread; ++u) sum_vector<kBf16>(a, q[u], scale);
      if (kMode == kBoth) {
        sum_frees(sh.ring, r, j, pc.stages, slots, lane);
      } else {
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
    return sum_warp(sum_result(a), scale);
  };
  if (warp < kSumWarps) {
    // ------------------------------------------------------------- sum warps
    Place at = {0, 0};
    int32_t next_id[kPerLane];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) {
        next_id[r] = -1;
        if (r * 32 + lane < in.k) next_id[r] = in.ids[row * in.k + r * 32 + lane];
      }
    };
    if (num_its > 0) fetch(walk.row(0));
    for (uint32_t it = 0; it < num_its; ++it) {
      const Piece pc = piece(it);
      int32_t id[kPerLane];
#pragma unroll
      for (int r = 0; r < kPerLane; ++r) id[r] = next_id[r];
      if (it + 1 < num_its) fetch(walk.row(it + 1));
      Place r = at;
      Sum rest = piece_sum(pc, id, r, tid, warp);
      if (lane == 0) sh.warp_sum[it & 1][warp] = rest;
      consumers_sync<kT>();  // (every warp keeps to the rows' barriers)
      if (warp == static_cast<int>(it % kWarps)) {
        rest = sum_warp(lane < kWarps ? sh.warp_sum[it & 1][lane] : Sum{neg_inf(), 0.0f}, scale);
        // (the list warp has read its logits before any CTA of the row may write over
        // them, and the row kHeld before this one is done with)
        ok = ok && wait_held(sh.ready, it);
        if (ok)
          exchange_tell(sh.ex, it, make_uint4(__float_as_uint(rest.m), __float_as_uint(rest.s), 0u, 0u),
                        walk.chunk, chunks, lane);
      }
      // (every use of a slot is waited for, the second loads' too: see ring_arrivals)
      for (int j = slots; kMode == kBoth && j < pc.stages && ok; ++j, step(r, slots)) {
        ok = warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (ok) sum_frees(sh.ring, r, pc.stages + j - slots, pc.stages, slots, lane);
      }
      if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
      at = later(at, num_loads(pc.stages, slots, kMode == kBoth), slots);
    }
  } else if (warp < kSumWarps + kGradWarps) {
    // -------------------------------------------------------- gradient warps
    Place at = {0, 0};
    const int gtid = tid - kSumWarps * 32;
    const bool with_up = kMode == kBoth && in.grad_loss != nullptr;
    uint32_t sums = 0;  // rows whose sums were taken anew
    float next_up = with_up && num_its > 0 ? in.grad_loss[walk.row(0)] : 1.0f;
    for (uint32_t it = 0; it < num_its; ++it) {
      const int64_t row = walk.row(it);
      Piece pc = piece(it);
      float up = next_up * in.inv_t32;
      if (with_up && it + 1 < num_its) next_up = in.grad_loss[walk.row(it + 1)];
      float end_x[2] = {neg_inf(), neg_inf()};
      auto ends = [&] {
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int j = end_column(pc, side, gtid);
          if (j >= 0) end_x[side] = read_elem<kBf16>(pc.p, j);
        }
      };
      ends();
      ok = (kMode != kBoth || exchange_wait(sh.ex, it, abort_flag)) && wait_held(sh.ready, it);
      if (!ok) break;
      List &l = sh.list[it % kHeld];
      bool live = l.any;
      float m = l.m, coef = l.coef;
      Sum total = {neg_inf(), 0.0f};
      auto by_sums = [&](const Sum &rest) {
        total = sum_merge(l.listed, rest, scale);
        live = live && total.s != 0.0f;
        m = rest.m == neg_inf() ? 0.0f : rest.m;
        coef = nan_f32();
        if (!is_nan(total.s)) {
          const float share = sum_at(rest, total.m, scale) / total.s;  // s_r
          coef = rest.s == 0.0f ? 0.0f : up * fmaf(l.total, share, -l.rest) / rest.s;
        }
      };
      const bool anew = kMode == kBackward && l.anew;
      if constexpr (kMode == kBoth) by_sums(exchange_sum(sh.ex, it, chunks, lane, scale));
      if (kMode == kBackward && anew) {
        pc = whole_piece(it);
        ends();
        if (pc.c1 > 0) {
          int32_t id[kPerLane];
#pragma unroll
          for (int s = 0; s < kPerLane; ++s)
            id[s] = s * 32 + lane < in.k ? l.id[s * 32 + lane] : -1;
          up = coef;
          Sum rest = piece_sum(pc, id, at, gtid, warp);
          if (lane == 0) sh.warp_sum[sums & 1][warp] = rest;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.joined));
          ok = ok && warp_wait(smem_u32(&sh.joined), sums & 1, abort_flag);
          if (!ok) break;
          rest = lane < kWarps ? sh.warp_sum[sums & 1][lane] : Sum{neg_inf(), 0.0f};
          rest = sum_warp(rest, scale);
          ++sums;
          by_sums(rest);
          if (gtid == 0) {  // (all warps have read what was there)
            l.m = total.m;
            l.of = (rest.s == 0.0f ? l.on_list : l.total) / total.s;
            l.any = live;
          }
        }
      }
      char *g = static_cast<char *>(in.grad) + row * ldg_bytes;
      auto value = [&](float x) { return live ? coef * ex2((x - m) * scale) : 0.0f; };
      const int kept = kMode == kBoth ? max(0, pc.stages - slots) : 0;
      Place r = later(at, kept, slots);
      for (int i = 0; i < pc.stages; ++i) {
        // (stages that stayed are there since the row's sum; waiting again costs nothing)
        const bool again = i >= pc.stages - kept;  // loaded a second time
        const int j = again ? i - (pc.stages - kept) : kept + i;
        ok = warp_wait(smem_u32(&sh.ring.full[r.slot]), r.phase, abort_flag);
        if (!ok) break;
        const uint4 *st = buf + r.slot * kStageVec<kT>;
        const int c = pc.b0 + j * kStageVec<kT> * kVec;
        const int n = min(kStageVec<kT>, (pc.b1 - c) / kVec);
        char *o = g + static_cast<int64_t>(c) * kElt;
        // bytes of the stage before the output's first whole vector
        const int skip = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(o) & 15u)) & 15u);
        uint4 *ov = reinterpret_cast<uint4 *>(o + skip);
        if (skip == 0 && live && n == kStageVec<kT>) {
          uint4 q[kVecPerThread];
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u) q[u] = st[u * kT + gtid];
#pragma unroll
          for (int u = 0; u < kVecPerThread; ++u)
            __stcs(ov + u * kT + gtid, grad_vec<kBf16>(q[u], m, scale, coef));
        } else if (skip == 0) {
          for (int v = gtid; v < n; v += kT)
            __stcs(ov + v, live ? grad_vec<kBf16>(st[v], m, scale, coef) : make_uint4(0, 0, 0, 0));
        } else {
          with_shift<kElt>(skip, [&](auto by) {
            uint4 q[kVecPerThread];
#pragma unroll
            for (int u = 0; u < kVecPerThread; ++u) {
              const int v = min(u * kT + gtid, max(0, n - 2));
              q[u] = shifted<decltype(by)::value>(st[v], st[v + 1]);
            }
#pragma unroll
            for (int u = 0; u < kVecPerThread; ++u) {
              const uint4 d = live ? grad_vec<kBf16>(q[u], m, scale, coef) : make_uint4(0, 0, 0, 0);
              if (u * kT + gtid < n - 1) __stcs(ov + u * kT + gtid, d);
            }
          });
          // the vector's worth of elements at both ends, a warp after the other
          if (gtid / 32 == j % kWarps && lane < kVec) {
            const int e = lane * kElt < skip ? lane : (n - 1) * kVec + lane;
            store_elem<kBf16>(o, e, value(read_elem<kBf16>(reinterpret_cast<const char *>(st), e)));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.ring.empty[r.slot]));
        step(r, slots);
      }
      if (!ok) break;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const int j = end_column(pc, side, gtid);
        if (j >= 0) store_elem<kBf16>(g, j, value(end_x[side]));
      }
      if (anew ? has_row(it) : walk.chunk_of(it) == chunks - 1)
        for (int j = valid + gtid; j < width; j += kT) store_elem<kBf16>(g, j, 0.0f);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.stored[it % kHeld]));
      at = later(at, num_loads(pc.stages, slots, kMode == kBoth), slots);
    }
    if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
  } else if (warp == kSumWarps + kGradWarps) {
    // (kBackward) the saved sums, a row ahead: do they hold enough?
    float next_own = 0.0f, next_rest = 0.0f;
    auto fetch = [&](uint32_t it) {
      if (kMode != kBackward || it >= num_its) return;
      next_own = in.in_lse[walk.row(it)];
      if (in.lse != nullptr) next_rest = in.in_lse_rest[walk.row(it)];
    };
    fetch(0);
    auto load = [&](uint32_t it, Piece &q) {
      const bool anew = kMode == kBackward && sums_lost(next_own, next_rest, in);
      fetch(it + 1);
      q = anew ? whole_piece(it) : piece(it);
      return anew ? 2 * q.stages : num_loads(q.stages, slots, kMode == kBoth);
    };
    copy_rows<kBf16, kT>(sh.ring, buf, slots, kMode == kBoth, num_its, load, lane, err);
    pdl_launch_dependents();
  } else {
    // ------------------------------------------------------------ list warps
    auto fix = [&](uint32_t it, float up, float m, float of) {
      const List &l = sh.list[it % kHeld];
      const Piece pc = kMode == kBackward && l.anew ? whole_piece(it) : piece(it);
      char *g = static_cast<char *>(in.grad) + walk.row(it) * ldg_bytes;
      for (int i = lane; i < in.k; i += 32) {
        const int32_t id = l.id[i];
        if (!l.first[i] || id < pc.c0 || id >= pc.c1) continue;
        store_elem<kBf16>(g, id, up * (of * ex2((l.x[i] - m) * scale) - l.p[i]));
      }
    };
    const uint32_t first = static_cast<uint32_t>(warp - kSumWarps - kGradWarps - 1);
    Entries next;
    float next_lse = 0.0f, next_own = 0.0f, next_rest = neg_inf(), next_up = 1.0f;
    auto fetch = [&](uint32_t it) {
      const int64_t row = walk.row(it);
      int c0 = 0, c1 = valid;
      if (kMode == kBackward) {
        next_own = in.in_lse[row];
        if (in.in_lse_rest != nullptr) next_rest = in.in_lse_rest[row];
        if (in.grad_loss != nullptr) next_up = in.grad_loss[row];
      }
      if (in.lse != nullptr) next_lse = in.lse[row];
      entries_load(next, in, row, valid, lane);
      if (kMode == kBackward) {  // (other pieces may be written already)
        const Piece pc = sums_lost(next_own, next_rest, in) ? whole_piece(it) : piece(it);
        c0 = pc.c0;
        c1 = pc.c1;
      }
      entries_look<kBf16>(next, logits + row * ld_bytes, c0, c1);
    };
    if (first < num_its) fetch(first);
    for (uint32_t it = first; ok && it < num_its + F::kLists; it += F::kLists) {
      if (it < num_its) {
        List &l = sh.list[it % kHeld];
        teacher_row(l, next, in.k, next_lse, in.lse != nullptr, inv_t, scale, lane);
        if (kMode == kBackward && lane == 0) {
          // relative to lse_rest, where there is a rest: s_r <= 1 times e^(y_j - lse_rest), where
          // s_j itself may vanish (a rest that is masked by a low value).  m is rounded; what the
          // exponents lose by that is in the factors.
          const bool by_rest = l.rest > 0.0f && next_rest != neg_inf();
          const float total = by_rest ? l.total : l.on_list, base = by_rest ? next_rest : next_own;
          auto lost = [&](float lse) {
            return 1.0f - static_cast<float>(lse - (lse * in.temperature) * inv_t);
          };
          l.m = base * in.temperature;
          l.coef = next_up * in.inv_t32 * lost(base) *
                   (by_rest ? fmaf(total, ex2((next_rest - next_own) * kLog2e), -l.rest) : total);
          l.of = total * lost(next_own);
          l.anew = sums_lost(next_own, next_rest, in);
          if (l.anew)
            l.coef = next_up * in.inv_t32;
          else if (next_own == neg_inf())
            l.any = 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.ready[it % kHeld]));
        if (it + F::kLists < num_its) fetch(it + F::kLists);
      }
      if (it < F::kLists || it - F::kLists >= num_its) continue;
      // the row before it
      const uint32_t last = it - F::kLists;
      const int64_t row = walk.row(last);
      const List &l = sh.list[last % kHeld];
      float up = in.inv_t32;
      if (kGrad && in.grad_loss != nullptr) up *= in.grad_loss[row];
      if (kMode == kBackward) {
        const float lse = in.in_lse[row];
        ok = wait_held(sh.stored, last);
        if (ok && l.any) fix(last, up, l.anew ? l.m : lse * in.temperature, l.of);
        __syncwarp();
        continue;
      }
      ok = exchange_wait(sh.ex, last, abort_flag);
      if (!ok) continue;
      exchange_rearm(sh.ex, last, chunks, lane);
      const Sum rest = exchange_sum(sh.ex, last, chunks, lane, scale);
      const Sum total = sum_merge(l.listed, rest, scale);
      if (walk.chunk == 0 &&
          (in.out_loss != nullptr || in.out_lse != nullptr || in.out_lse_rest != nullptr)) {
        // lane 0: lse, lane 1: lse_rest, lane 2: log p_r
        const double rest_p = rest.s == 0.0f ? 0.0 : l.rest_p;
        const float of = lane == 0 ? total.s : (lane == 1 ? rest.s : static_cast<float>(rest_p));
        const Sum own = lane == 0 ? total : rest;
        const double lg = log_of(of);
        const double v = is_nan(total.s) ? nan("") : (own.s == 0.0f ? -INFINITY
                                                                    : own.m * inv_t + lg);
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
      if (kGrad) {
        ok = wait_held(sh.stored, last);
        if (ok && l.any && total.s != 0.0f)
          fix(last, up, total.m, (rest.s == 0.0f ? l.on_list : l.total) / total.s);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) raise_abort(&sh.ring.abort, err);
  }
  leave(sh.ring, F::kSum ? chunks : 1);
}

// Pieces of a row in the gradient from saved sums: few rows are split over all CTAs, in
// pieces of 8 KB or more; many into pieces of at most 128 KB (2048 of 200064 bf16 ids: 50
// KB 257 us, 100 to 400 KB 255-256; 700 of 50257 fp32 ids: 200 KB 47.2 us, 100 KB 47.1, 50
// KB 46.3).  From more than half as many rows as CTAs (456 of 256 threads) up to as many, rows
// stay whole: 333 of 50257 fp32 ids 26.2 us, in two pieces 24.0, in four 23.8; 240 19.7, 19.5,
// 18.5; 450 31.2, 30.7, 31.0.
int backward_pieces(int64_t rows, int64_t bytes, int64_t ctas) {
  int64_t n = rows < ctas ? ctas / rows : (bytes + 131071) / 131072;
  if (n > bytes / 8192) n = bytes / 8192;
  if (n > 512) n = 512;  // (what piece_of multiplies stays below 2^32)
  if (rows * n > (int64_t(1) << 30)) n = (int64_t(1) << 30) / rows;
  return n < 1 ? 1 : static_cast<int>(n);
}

template <bool kBf16, int kT, Mode kMode>
cudaError_t launch_rows(const void *logits, int64_t rows, int64_t ld, int64_t width, int64_t valid,
                        const Args &in, int64_t ldg, uint32_t *err, cudaStream_t stream) {
  using F = Form<kT, kMode>;
  constexpr int kElt = kBf16 ? 2 : 4;
  auto kern = distill_kernel<kBf16, kT, kMode>;
  const RowKernel k = {reinterpret_cast<const void *>(kern), F::kThreads, F::kRingBytes,
                       (kBf16 ? 0 : 1) + 2 * (kT == 128 ? 6 : (kT == 256 ? 0 : 1) + 2 * kMode)};
  int64_t resident[6];
  const cudaError_t e = resident_clusters(k, resident);
  if (e != cudaSuccess) return e;
  int chunks = 1, width_of = 1;
  int64_t walks = rows;
  if (kMode == kBackward) {
    chunks = backward_pieces(rows, valid * kElt, resident[5]);
    walks = rows * chunks;
  } else if (kT == 256) {
    width_of = chunks =
        pick_chunks(rows, valid * kElt, kMode == kBoth ? F::kRingBytes : 0, resident);
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  row_launch(k, walks, width_of, resident, stream, attr, cfg);
  return cudaLaunchKernelEx(&cfg, kern, static_cast<const char *>(logits), ld * kElt, rows,
                            static_cast<int>(valid), static_cast<int>(width), in, ldg * kElt,
                            chunks, err);
}

}  // namespace

cudaError_t launch_distill(const void *logits, int dtype, int64_t rows, int64_t ld, int64_t width,
                           int64_t valid, const DistillArgs &in, int64_t ldg, int num_sms,
                           uint32_t *err, cudaStream_t stream) {
  const double inv_t = 1.0 / static_cast<double>(in.temperature);
  const Args args = {in, inv_t, static_cast<float>(inv_t),
                     static_cast<float>(1.4426950408889634 * inv_t)};
  const int64_t bytes = valid * (dtype == SGA_BF16 ? 2 : 4);
  const bool small = small_rows(rows, bytes, num_sms);
  // (many rows of 36 to 72 KB: see Form)
  const bool middle = bytes > (36 << 10) && bytes <= (72 << 10) && rows > 3 * num_sms;
  auto launch = [&](auto bf16, auto mode) {
    constexpr bool kBf16 = decltype(bf16)::value;
    constexpr Mode kMode = static_cast<Mode>(decltype(mode)::value);
    if (kMode == kBoth && middle)
      return launch_rows<kBf16, 128, kBoth>(logits, rows, ld, width, valid, args, ldg, err, stream);
    return (small ? launch_rows<kBf16, 64, kMode> : launch_rows<kBf16, 256, kMode>)(
        logits, rows, ld, width, valid, args, ldg, err, stream);
  };
  auto by_mode = [&](auto bf16) {
    if (in.in_lse != nullptr) return launch(bf16, std::integral_constant<int, kBackward>{});
    return in.grad != nullptr ? launch(bf16, std::integral_constant<int, kBoth>{})
                              : launch(bf16, std::integral_constant<int, kLoss>{});
  };
  return dtype == SGA_BF16 ? by_mode(std::true_type{}) : by_mode(std::false_type{});
}

}  // namespace sga
