// k_split12_moe.cu -- a mixture-of-experts layer for a few tokens, from the
// router's logits on, the experts' weights in two Split12 containers
// (wc12_moe, include/wc_split12.h):
//   S_t = the k largest logits of token t (ties: the lower expert)
//   p   = softmax of the logits over S_t, or over all experts
//   out[t] = sum over e in S_t of p_e D_e (silu(G_e x_t) * U_e x_t)
//
// The bytes of the chosen experts' weights bound it, so both kernels stream
// them through registers (wc12_few.cuh), 8 of the tokens that chose an expert
// at a time (an item; more than 8 are rare, and read the weights again, from
// L2):
//   * k12_moe_up: the CTAs go through (item, 16 rows of F) one after another,
//     as many as run at once, so that the routing is found once and the
//     copies in flight run on from one to the next.  A warp takes a part of H
//     for the 16 rows of G_e and the same of U_e, and p_e silu(g) u is
//     written as the sum of two bf16 numbers (16 bits: rounding it to 8 would
//     cost the output as much again as its own rounding to bf16);
//   * k12_moe_down: a cluster takes rows of the output and walks through D_e
//     of every item as through one long row, whose parts its warps take.  The
//     weighted sum over experts is part of the product's sum: no atomics, one
//     rounding, one write.
// Both find the experts from the logits themselves, a warp a token (a few
// hundred logits), instead of waiting for a third kernel; the second starts
// while the first one ends (programmatic dependent launch) and by then has
// its routing, exceptions and first weights.
#include <cstdint>

#include "wc12_few.cuh"

namespace wc12l {
int device_sms();
}

namespace wc12m {

using namespace wc12f;

constexpr uint32_t kMaxTokens = 32;  // of a launch
constexpr uint32_t kMaxTop = 16;
constexpr uint32_t kMaxExperts = 512;

struct Params {
  const uint8_t *gate_up, *down;
  uint64_t gate_up_bytes, down_bytes;
  const uint16_t *x;    // [T, H]
  const float *logits;  // [T, E]
  uint16_t *hs;         // two planes of [T k, F]
  void *out;            // [T, H]
  uint32_t T, E, H, F, k;
  uint32_t renormalize, wide;
  int32_t *status;
};

constexpr uint32_t kMaxPairs = kMaxTokens * kMaxTop;

// The tokens' experts, and the items: an expert and up to 8 (token, expert)
// pairs that chose it, experts ascending.
struct Route {
  int16_t id[kMaxTokens][kMaxTop];  // expert, -1: none
  float p[kMaxTokens][kMaxTop];
  uint16_t pair[kMaxPairs];         // token * k + j, by expert
  uint16_t item_e[kMaxPairs], item_first[kMaxPairs];
  uint8_t item_n[kMaxPairs];
  uint32_t items;
};
// while it is found (in shared memory that the ring takes later)
struct RouteScratch {
  uint32_t key[kWarps][kMaxExperts];
  uint32_t who[kMaxExperts];    // the tokens that chose each expert, a bit each
  uint16_t first[kMaxExperts];  // their first place in pair[]
};

// ascending in the logits' order; -0 like +0, NaN above all
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // order_key(-inf)

__device__ void route(Route &r, RouteScratch &w, const Params &p) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (uint32_t e = tid; e < p.E; e += kThreads) w.who[e] = 0;
  __syncthreads();
  for (uint32_t m = warp; m < p.T; m += kWarps) {
    const float *l = p.logits + uint64_t(m) * p.E;
    uint32_t *key = w.key[warp];
    // each lane looks at its own experts only: no barrier needed
    for (uint32_t e = lane; e < p.E; e += 32) key[e] = order_key(l[e]);
    uint32_t taken = 0;  // of the lane's experts
    float top = 0.0f, sum = 0.0f, ex = 0.0f;
    for (uint32_t j = 0; j < p.k; j++) {
      uint32_t best = 0, at = 0xFFFFFFFFu;
      for (uint32_t i = 0, e = lane; e < p.E; i++, e += 32)
        if (!((taken >> i) & 1u) && key[e] > best) {
          best = key[e];
          at = e;
        }
      const uint32_t high = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(0xffffffffu, best == high ? at : 0xFFFFFFFFu);
      const bool none = high <= kMinusInf;  // only -inf is left
      if (!none) {
        if ((e & 31u) == lane) taken |= 1u << (e >> 5);
        const float v = l[e];
        if (j == 0) top = v;
        const float q = expf(v - top);
        if (lane == j) ex = q;
        sum += q;
        if (lane == 0) atomicOr(&w.who[e], 1u << m);
      }
      if (lane == 0) r.id[m][j] = none ? int16_t(-1) : int16_t(e);
    }
    if (!p.renormalize) {
      sum = 0.0f;
      for (uint32_t e = lane; e < p.E; e += 32) sum += expf(l[e] - top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (lane < p.k) r.p[m][lane] = ex / sum;
  }
  __syncthreads();
  // the experts' places in pair[], and their items
  if (warp == 0) {
    uint32_t pairs = 0, items = 0;
    for (uint32_t e0 = 0; e0 < p.E; e0 += 32) {
      const uint32_t e = e0 + lane, n = e < p.E ? __popc(w.who[e]) : 0u, blocks = (n + 7) / 8;
      uint32_t a = n, b = blocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= uint32_t(o)) {
          a += x;
          b += y;
        }
      }
      const uint32_t first = pairs + a - n;
      if (e < p.E) w.first[e] = uint16_t(first);
      for (uint32_t i = 0; i < blocks; i++) {
        const uint32_t at = items + b - blocks + i;
        r.item_e[at] = uint16_t(e);
        r.item_first[at] = uint16_t(first + 8 * i);
        r.item_n[at] = uint8_t(n - 8 * i < 8 ? n - 8 * i : 8);
      }
      pairs += __shfl_sync(0xffffffffu, a, 31);
      items += __shfl_sync(0xffffffffu, b, 31);
    }
    if (lane == 0) r.items = items;
  }
  __syncthreads();
  // by token within an expert, so that every CTA has the same items
  for (uint32_t i = tid; i < p.T * p.k; i += kThreads) {
    const int32_t e = r.id[i / p.k][i % p.k];
    if (e >= 0) r.pair[w.first[e] + __popc(w.who[e] & ((1u << i / p.k) - 1u))] = uint16_t(i);
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
struct Up {
  using R = Ring<2, 1, 1>;
  static constexpr uint32_t kDepth = 3;
  static constexpr uint32_t kSums = 8 * kRedTok;  // floats a warp and matrix
  static constexpr uint32_t kRoute = kWarps * kDepth * R::kBytes;
  static constexpr uint32_t kLists = (kRoute + uint32_t(sizeof(Route)) + 15) / 16 * 16;
  static constexpr uint32_t kRed = kLists + kWarps * kListCap * 4;
  static constexpr uint32_t kSmem = kRed + kWarps * 2 * kSums * 4;
};
static_assert(sizeof(RouteScratch) <= Up::kRoute, "scratch");

__global__ void __launch_bounds__(kThreads) k12_moe_up(const __grid_constant__ Params p) {
  launch_dependents();
  extern __shared__ __align__(16) uint8_t dyn[];
  Route &route_s = *reinterpret_cast<Route *>(dyn + Up::kRoute);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  View v;
  open_planes(v, p.gate_up, uint64_t(p.E) * 2 * p.F * p.H);
  const bool ok = open_header(v, p.gate_up, p.gate_up_bytes);
  route(route_s, *reinterpret_cast<RouteScratch *>(dyn), p);
  if (!ok) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    return;
  }
  const uint32_t K = p.H, units = K / kUnit, u0 = units * warp / kWarps, u1 = units * (warp + 1) / kWarps;
  const uint32_t groups = p.F / kRows, jobs = route_s.items * groups;
  // rows of job j: 16 of G_e, and the same of U_e
  auto row_of = [&](uint32_t job, uint32_t which) {
    const uint32_t item = job / groups;
    return (uint64_t(route_s.item_e[item]) * 2 + which) * p.F + (job - item * groups) * kRows;
  };
  // copies run ahead of the products, over the ends of jobs
  uint32_t load_job = blockIdx.x, load_u = u0;
  const uint8_t *pi[2], *pl[2];
  const uint16_t *px = p.x;
  uint32_t live = 0;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * Up::kDepth * Up::R::kBytes;
  auto load = [&](uint32_t slot) {
    if (load_job < jobs && u0 < u1) {
      if (load_u == u0) {
#pragma unroll
        for (uint32_t w = 0; w < 2; w++) {
          const uint64_t at = (row_of(load_job, w) + g) * K + u0 * kUnit;
          pi[w] = v.idx + at / 2 + 8 * t;
          pl[w] = v.lo + at + 16 * t;
        }
        const uint32_t item = load_job / groups;
        live = g < route_s.item_n[item];
        const uint32_t m = live ? route_s.pair[route_s.item_first[item] + g] / p.k : 0u;
        px = p.x + uint64_t(m) * K + u0 * kUnit + 16 * t;
      }
      Up::R::load(ring + slot * Up::R::kBytes, lane, pi, pl, K, &px, live, 1, 0);
#pragma unroll
      for (uint32_t w = 0; w < 2; w++) {
        pi[w] += kUnit / 2;
        pl[w] += kUnit;
      }
      px += kUnit;
      if (++load_u == u1) {
        load_u = u0;
        load_job += gridDim.x;
      }
    }
    copies_commit();
  };
#pragma unroll
  for (uint32_t i = 0; i < Up::kDepth; i++) load(i);
  // the exceptions of a job are in flight during the one before, their
  // offsets during the one before that
  Window now[2], next[2];
  auto offsets = [&](Window *w, uint32_t job) {
    if (v.ne > 0 && job < jobs)
      for (uint32_t i = 0; i < 2; i++) window_offsets(w[i], v.exc_off, row_of(job, i), K, lane);
  };
  auto entries = [&](Window *w, uint32_t job) {
    if (v.ne > 0 && job < jobs)
      for (uint32_t i = 0; i < 2; i++) window_entries(w[i], v, lane);
  };
  offsets(now, blockIdx.x);
  offsets(next, blockIdx.x + gridDim.x);
  entries(now, blockIdx.x);
  Exceptions x;
  x.list = reinterpret_cast<uint32_t *>(dyn + Up::kLists) + warp * kListCap;
  float *red = reinterpret_cast<float *>(dyn + Up::kRed);
  const uint64_t plane = uint64_t(p.T) * p.k * p.F;
  uint32_t slot = 0;
  for (uint32_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    exceptions_reset(x);
    if (v.ne > 0) {
      for (uint32_t i = 0; i < 2; i++) window_keep(x, now[i], v, row_of(job, i), K, i, u0, u1, lane, p.status);
      exceptions_ready(x, lane);
    }
    now[0] = next[0];
    now[1] = next[1];
    entries(now, job + gridDim.x);
    offsets(next, job + 2 * gridDim.x);
    const uint64_t row_g[2] = {row_of(job, 0) + g, row_of(job, 1) + g};
    float tot[2][1][4] = {};
    for (uint32_t u = u0; u < u1; u++) {
      copies_wait<Up::kDepth - 1>();
      unit_product<2, 1, 1>(tot, ring + slot * Up::R::kBytes, v.book, v, 1, x, u, row_g, K, lane);
      load(slot);
      slot = slot + 1 == Up::kDepth ? 0 : slot + 1;
    }
    put_sums<1>(red + 2 * warp * Up::kSums, tot[0], lane);
    put_sums<1>(red + (2 * warp + 1) * Up::kSums, tot[1], lane);
    __syncthreads();
    const uint32_t item = job / groups, row = tid % kRows, c = tid / kRows;  // 16 x 8 threads
    if (c < route_s.item_n[item]) {
      float gate = 0.0f, up = 0.0f;
#pragma unroll
      for (uint32_t w = 0; w < kWarps; w++) {
        gate += red[2 * w * Up::kSums + c * kRedTok + row];
        up += red[(2 * w + 1) * Up::kSums + c * kRedTok + row];
      }
      const uint32_t pair = route_s.pair[route_s.item_first[item] + c];
      const float h = gate / (1.0f + expf(-gate)) * up * route_s.p[pair / p.k][pair % p.k];
      // two bf16 numbers, each rounded to nearest: off by at most 2^-18
      uint16_t *dst = p.hs + uint64_t(pair) * p.F + (job - item * groups) * kRows + row;
      const uint32_t hi = bf16_bits(h);
      dst[0] = uint16_t(hi);
      dst[plane] = uint16_t((hi & 0x7F80u) == 0x7F80u ? 0u : bf16_bits(h - __uint_as_float(hi << 16)));
    }
    __syncthreads();  // red is read until here
  }
  copies_wait<0>();
}

// ---------------------------------------------------------------------------
// A warp has the part `part` of 2^sbits of its cluster rank's units, for one
// of the CTA's 4 >> sbits groups of 16 rows.
struct Down {
  using R = Ring<1, 1, 2>;
  static constexpr uint32_t kDepth = 3;
  static constexpr uint32_t kRoute = kWarps * kDepth * R::kBytes;
  static constexpr uint32_t kLists = (kRoute + uint32_t(sizeof(Route)) + 15) / 16 * 16;
  static constexpr uint32_t kAcc = kLists + kWarps * kListCap * 4;
  static __host__ __device__ uint32_t smem(uint32_t T) { return kAcc + kWarps * T * kRedTok * 4; }
};
static_assert(sizeof(RouteScratch) <= Down::kRoute, "scratch");

__global__ void __launch_bounds__(kThreads) k12_moe_down(const __grid_constant__ Params p, uint32_t csize,
                                                        uint32_t sbits) {
  extern __shared__ __align__(16) uint8_t dyn[];
  Route &route_s = *reinterpret_cast<Route *>(dyn + Down::kRoute);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = blockIdx.x % csize, rows = kRows * kWarps >> sbits, n0 = blockIdx.x / csize * rows;
  const uint32_t part = (rank << sbits) + (warp & ((1u << sbits) - 1)), parts = csize << sbits;
  const uint32_t row0 = n0 + kRows * (warp >> sbits);
  View v;
  open_planes(v, p.down, uint64_t(p.E) * p.H * p.F);
  const bool ok = open_header(v, p.down, p.down_bytes);
  route(route_s, *reinterpret_cast<RouteScratch *>(dyn), p);
  float *acc = reinterpret_cast<float *>(dyn + Down::kAcc) + warp * p.T * kRedTok;  // [token][row]
  for (uint32_t i = lane; i < p.T * kRedTok; i += 32) acc[i] = 0.0f;
  if (ok) {
    // the items' units one after another; this warp's: [q0, q1)
    const uint32_t K = p.F, units = K / kUnit, all = route_s.items * units;
    const uint32_t q0 = uint32_t(uint64_t(all) * part / parts), q1 = uint32_t(uint64_t(all) * (part + 1) / parts);
    const uint64_t plane = uint64_t(p.T) * p.k * p.F;
    auto row_of = [&](uint32_t item) { return uint64_t(route_s.item_e[item]) * p.H + row0; };
    uint32_t load_q = q0, load_item = q0 / units, load_u = q0 - load_item * units;
    const uint8_t *pi = nullptr, *pl = nullptr;
    const uint16_t *px = p.hs;
    uint32_t live = 0;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * Down::kDepth * Down::R::kBytes;
    // the weights of the first units are on their way before hs is waited
    // for, its values follow
    auto load = [&](uint32_t slot, bool weights, bool values) {
      if (load_q < q1) {
        if (load_q == q0 || load_u == 0) {
          const uint64_t at = (row_of(load_item) + g) * K + load_u * kUnit;
          pi = v.idx + at / 2 + 8 * t;
          pl = v.lo + at + 16 * t;
          live = g < route_s.item_n[load_item];
          const uint32_t pair = live ? route_s.pair[route_s.item_first[load_item] + g] : 0u;
          px = p.hs + uint64_t(pair) * K + load_u * kUnit + 16 * t;
        }
        const uint32_t to = ring + slot * Down::R::kBytes;
        if (weights) Down::R::load_weights(to, lane, &pi, &pl, K);
        if (values) Down::R::load_values(to, lane, &px, live, 1, plane);
        pi += kUnit / 2;
        pl += kUnit;
        px += kUnit;
        load_q++;
        if (++load_u == units) {
          load_u = 0;
          load_item++;
        }
      }
    };
    uint32_t item = load_item, u = load_u;
#pragma unroll
    for (uint32_t i = 0; i < Down::kDepth; i++) load(i, true, false);
    const uint32_t last = q0 < q1 ? (q1 - 1) / units : 0u;
    Window now, next;
    auto offsets = [&](Window &w, uint32_t i) {
      if (v.ne > 0 && i <= last) window_offsets(w, v.exc_off, row_of(i), K, lane);
    };
    auto entries = [&](Window &w, uint32_t i) {
      if (v.ne > 0 && i <= last) window_entries(w, v, lane);
    };
    if (q0 < q1) {
      offsets(now, item);
      offsets(next, item + 1);
      entries(now, item);
    }
    wait_prerequisites();  // hs
    load_q = q0;
    load_item = item;
    load_u = u;
#pragma unroll
    for (uint32_t i = 0; i < Down::kDepth; i++) {
      load(i, false, true);
      copies_commit();
    }
    Exceptions x;
    x.list = reinterpret_cast<uint32_t *>(dyn + Down::kLists) + warp * kListCap;
    uint32_t slot = 0;
    for (uint32_t q = q0; q < q1; item++, u = 0) {
      const uint32_t end = q1 - q < units - u ? u + (q1 - q) : units;
      exceptions_reset(x);
      if (v.ne > 0) {
        window_keep(x, now, v, row_of(item), K, 0, u, end, lane, p.status);
        exceptions_ready(x, lane);
      }
      now = next;
      entries(now, item + 1);
      offsets(next, item + 2);
      const uint64_t row_g = row_of(item) + g;
      float tot[1][1][4] = {};
      for (; u < end; u++, q++) {
        copies_wait<Down::kDepth - 1>();
        unit_product<1, 1, 2>(tot, ring + slot * Down::R::kBytes, v.book, v, 1, x, u, &row_g, K, lane);
        load(slot, true, true);
        copies_commit();
        slot = slot + 1 == Down::kDepth ? 0 : slot + 1;
      }
      // columns to tokens; a token that did not choose the expert gets
      // nothing (not even zero times an infinite weight)
      const uint32_t n = route_s.item_n[item], first = route_s.item_first[item];
#pragma unroll
      for (uint32_t i = 0; i < 2; i++)
        if (2 * t + i < n) {
          float *to = acc + route_s.pair[first + 2 * t + i] / p.k * kRedTok + g;
          to[0] += tot[0][0][i];
          to[8] += tot[0][0][2 + i];
        }
    }
    copies_wait<0>();
  } else {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    wait_prerequisites();
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  if (ok) {
    const float *sums = reinterpret_cast<const float *>(dyn + Down::kAcc);
    for (uint32_t o = tid + rank * kThreads; o < p.T * rows; o += kThreads * csize) {
      const uint32_t row = o % rows, m = o / rows;
      const float *from = sums + ((row / kRows << sbits) * p.T + m) * kRedTok + row % kRows;
      float sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++)
        for (uint32_t i = 0; i < 1u << sbits; i++) {
          const float *f = from + i * p.T * kRedTok;
          sum += csize > 1 ? cluster_load(f, c) : *f;
        }
      const uint64_t at = uint64_t(m) * p.H + n0 + row;
      if (p.wide) static_cast<float *>(p.out)[at] = sum;
      else static_cast<uint16_t *>(p.out)[at] = uint16_t(bf16_bits(sum));
    }
  }
  if (csize > 1) cluster_sync();  // the others' sums are read until here
}

}  // namespace wc12m

extern "C" uint64_t wc12_moe_work_bytes(uint32_t T, uint32_t k, uint32_t F) {
  const uint64_t t = T < wc12m::kMaxTokens ? T : wc12m::kMaxTokens;
  return t * k * F * 4;
}

extern "C" int32_t wc12_moe(const void *d_gate_up, uint64_t gate_up_bytes, const void *d_down, uint64_t down_bytes,
                            uint32_t E, uint32_t H, uint32_t F, const void *d_x, const float *d_logits, uint32_t T,
                            uint32_t k, int32_t renormalize, void *d_out, int32_t out_dtype, void *d_work,
                            uint64_t work_bytes, int32_t *d_status, void *stream) {
  using namespace wc12m;
  auto aligned = [](const void *q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; };
  if (d_gate_up == nullptr || d_down == nullptr || d_status == nullptr) return WC_ERR_INVALID_ARG;
  if (!aligned(d_gate_up, 16) || !aligned(d_down, 16) || !aligned(d_status, 4)) return WC_ERR_INVALID_ARG;
  if (E == 0 || E > kMaxExperts || k == 0 || k > kMaxTop || k > E) return WC_ERR_INVALID_ARG;
  if (H == 0 || F == 0 || H % 64 != 0 || F % 64 != 0 || H > kMaxK || F > kMaxK) return WC_ERR_INVALID_ARG;
  if (out_dtype != WC_BF16 && out_dtype != WC_FP32) return WC_ERR_INVALID_ARG;
  if (gate_up_bytes < 96 || down_bytes < 96) return WC_ERR_INVALID_ARG;
  const uint64_t n_up = uint64_t(E) * 2 * F * H, n_down = uint64_t(E) * H * F;
  if (gate_up_bytes < wc12::lay(n_up, 0).off_lo + n_up || down_bytes < wc12::lay(n_down, 0).off_lo + n_down)
    return WC_ERR_INVALID_ARG;
  if (T == 0) return WC_OK;
  if (d_x == nullptr || d_logits == nullptr || d_out == nullptr || d_work == nullptr) return WC_ERR_INVALID_ARG;
  if (!aligned(d_x, 16) || !aligned(d_logits, 4) || !aligned(d_out, 4) || !aligned(d_work, 16)) return WC_ERR_INVALID_ARG;
  if (work_bytes < wc12_moe_work_bytes(T, k, F)) return WC_ERR_CAPACITY;
  const int sms = wc12l::device_sms();
  if (sms <= 0) return WC_ERR_CUDA;
  Params p;
  p.gate_up = static_cast<const uint8_t *>(d_gate_up);
  p.gate_up_bytes = gate_up_bytes;
  p.down = static_cast<const uint8_t *>(d_down);
  p.down_bytes = down_bytes;
  p.hs = static_cast<uint16_t *>(d_work);
  p.E = E;
  p.H = H;
  p.F = F;
  p.k = k;
  p.renormalize = renormalize != 0;
  p.wide = out_dtype == WC_FP32;
  p.status = d_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int up_per_sm = 0;
  if (cudaFuncSetAttribute(k12_moe_up, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Up::kSmem)) != cudaSuccess ||
      cudaFuncSetAttribute(k12_moe_down, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Down::smem(kMaxTokens))) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&up_per_sm, k12_moe_up, kThreads, Up::kSmem) != cudaSuccess || up_per_sm < 1)
    return WC_ERR_CUDA;
  for (uint32_t m = 0; m < T; m += kMaxTokens) {
    p.T = T - m < kMaxTokens ? T - m : kMaxTokens;
    p.x = static_cast<const uint16_t *>(d_x) + uint64_t(m) * H;
    p.logits = d_logits + uint64_t(m) * E;
    p.out = static_cast<uint8_t *>(d_out) + uint64_t(m) * H * (p.wide ? 4 : 2);
    // up: as many CTAs as run at once
    const uint32_t pairs = p.T * k, jobs = pairs * (F / kRows), slots = uint32_t(sms * up_per_sm);
    // down: CTAs that split the items (and, with few rows, warps that do),
    // until about 4 CTAs an SM have work
    uint32_t csize = 1, sbits = 0;
    const uint32_t some = (pairs < E ? pairs : E) * (F / kUnit);  // units of a row, about
    while (csize < 8 && H / 64 * csize * 2 <= 4u * uint32_t(sms) && some >= 2 * csize * Down::kDepth) csize *= 2;
    while (sbits < 2 && ((H / 64 * csize) << (sbits + 1)) <= 4u * uint32_t(sms) &&
           some >= (2 * csize << sbits) * Down::kDepth)
      sbits++;
    if (launch(k12_moe_up, dim3(jobs < slots ? jobs : slots), 1, Up::kSmem, s, false, p) != cudaSuccess) return WC_ERR_CUDA;
    if (launch(k12_moe_down, dim3((H / 64 * csize) << sbits), csize, Down::smem(p.T), s, true, p, csize, sbits) != cudaSuccess)
      return WC_ERR_CUDA;
  }
  return WC_OK;
}
