// k_split12_moe.cu -- a mixture-of-experts layer for a few tokens, from the
// router's logits on, the experts' weights in two Split12 containers
// (wc12_moe, include/wc_split12.h):
//   S_t = the k largest logits of token t (ties: the lower expert)
//   p   = softmax of the logits over S_t, or over all experts
//   out[t] = sum over e in S_t of p_e D_e (silu(G_e x_t) * U_e x_t)
//
// The bytes of the chosen experts' weights bound it, so both kernels stream
// them through a ring (wc12_few.cuh), 8 of the tokens that chose an expert at
// a time (an item; more than 8 are rare, and read the weights again, from
// L2):
//   * k12_moe_up: a job is 64 rows of G_e and the same of U_e for one item.
//     With many jobs as many CTAs as run at once go through them, so that the
//     routing is found once and the ring runs on from one to the next; with
//     few, the CTAs of a cluster split H.  p_e silu(g) u is written as the sum
//     of two bf16 numbers (16 bits: rounding it to 8 would cost the output as
//     much again as its own rounding to bf16);
//   * k12_moe_down: a cluster takes 64 rows of the output and walks through
//     D_e of every item as through one long row, whose parts its CTAs take.
//     The weighted sum over experts is part of the product's sum: no atomics,
//     one rounding, one write.
// Times of graph replays: 1 token, 8 of 64 experts of 2048 x 768: 29 us (57 MB);
// 5 tokens, 2 of 8, 4096 x 1792: 55 (200 MB); 16 tokens, 4 of 32, 1024 x 1408: 63
// (180 MB); 32 tokens, 8 of 128, 2048 x 768: 206 (790 MB, 3.8 TB/s).  In the last
// the up product alone takes 110 us for 524 MB of weights, 4.8 TB/s; from DRAM
// come 609 MB, some of it twice.
//
// k12_moe_route finds the experts first, a warp a token.  The up product starts
// when that is done; the down product starts beside the up product (programmatic
// dependent launch) and has its route, exceptions and first weights by the time
// that hs is there.  The up product is no dependent launch itself: the down
// product reads the route before it waits for the up product, and a kernel sees
// before that wait only what was finished before the up product began.
#include <cmath>
#include <cstdint>

#include "wc12_few.cuh"

namespace wc12m {

using namespace wc12f;

constexpr uint32_t kMaxTokens = 32;  // of a launch
constexpr uint32_t kMaxTop = 16;
constexpr uint32_t kMaxExperts = 512;

constexpr uint32_t kMaxPairs = kMaxTokens * kMaxTop;

// How many stages' exceptions go into the lanes' queues at once, 64 values of a
// lane in each: about 4 of the 16 that a queue holds, by the container's own
// share of them, so that a warp hardly ever has to look its values up (see
// stage_product_slow).  With one filling for a whole row that began at 16,384
// values of H with an exception in 2,500 (8 tokens, 2 experts, 16384 x 8192: 2433
// us, 399 so; 32768 x 4096: 4914 and 547), and in one of 4096 with one in 200
// (5 tokens, 2 of 8, 4096 x 896: 246 us, 82 so; one in 100: 458 and 145).  The
// rows that the shallow ring is for are not cut, though they come to looking up
// at one in 200 (16 tokens, 4 of 32, 1024 x 1408: 298 us for 54): the loop over
// their parts made its kernel spill registers, at every share of exceptions (63.5
// -> 67.7 us on that shape's listed case).
constexpr uint32_t kFill = 128;
__device__ __forceinline__ uint32_t fill_stages(const View &v) {
  const float room = float(v.n) / (16.0f * float(v.ne));  // an infinity without exceptions
  return room < 2.0f ? 2u : room < float(kFill) ? uint32_t(room) : kFill;
}

// The (token, expert) pairs by expert, and the items: an expert and up to 8 of
// its pairs; experts ascending.
struct Route {
  float weight[kMaxPairs];   // of each pair
  uint16_t pair[kMaxPairs];  // token * k + j, by expert
  uint16_t item_e[kMaxPairs], item_first[kMaxPairs];
  uint8_t item_n[kMaxPairs];
  uint32_t items;
};
struct Params {
  const uint8_t *gate_up, *down;
  uint64_t gate_up_bytes, down_bytes;
  const uint16_t *x;    // [T, H]
  const float *logits;  // [T, E]
  Route *route;
  uint16_t *hs;         // two planes of [T k, F]
  void *out;            // [T, H]
  uint32_t T, E, H, F, k;
  uint32_t renormalize, wide;
  int32_t *status;
};

// ascending in the logits' order; -0 like +0, NaN above all
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // order_key(-inf)
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// Finds the experts: one CTA, a warp a token, whose lanes hold kPer logits
// each.  Latency bounds it (two reductions a choice): 4 us for one token and 8
// choices.  In the up product's CTAs, each for itself, it took 9,000 cycles for
// one token and 54,000 for 32.
template <int kPer>
__global__ void __launch_bounds__(32 * kMaxTokens) k12_moe_route(const __grid_constant__ Params p) {
  __shared__ uint32_t who[kMaxExperts];    // the tokens that chose each expert, a bit each
  __shared__ uint16_t place[kMaxExperts];  // their first place in pair[]
  Route &r = *p.route;
  const uint32_t tid = threadIdx.x, lane = tid & 31, m = tid >> 5;
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    const uint32_t e = lane + 32 * i;
    key[i] = e < p.E ? order_key(p.logits[uint64_t(m) * p.E + e]) : 0u;
  }
  for (uint32_t e = tid; e < p.E; e += blockDim.x) who[e] = 0;
  __syncthreads();
  uint32_t mine = 0, mine_e = 0, top = 0;  // lane j: the j-th largest key and its expert
  {
    uint32_t left[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) left[i] = key[i];
    for (uint32_t j = 0; j < p.k; j++) {
      uint32_t best = 0, at = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < kPer; i++)
        if (left[i] > best) {
          best = left[i];
          at = lane + 32 * i;
        }
      const uint32_t high = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(0xffffffffu, best == high ? at : 0xFFFFFFFFu);
      if (high <= kMinusInf) break;  // only -inf is left
#pragma unroll
      for (int i = 0; i < kPer; i++)
        if (e == lane + 32 * i) left[i] = 0;
      if (lane == j) {
        mine = high;
        mine_e = e;
      }
      if (j == 0) top = high;
    }
  }
  const float largest = key_value(top);
  const float ex = mine != 0 ? expf(key_value(mine) - largest) : 0.0f;
  float sum = ex;
  if (!p.renormalize) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; i++)
      if (lane + 32 * i < p.E) sum += expf(key_value(key[i]) - largest);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < p.k && mine != 0) atomicOr(&who[mine_e], 1u << m);
  __syncthreads();
  // the experts' places in pair[], and their items
  if (m == 0) {
    uint32_t pairs = 0, items = 0;
    for (uint32_t e0 = 0; e0 < p.E; e0 += 32) {
      const uint32_t e = e0 + lane, n = e < p.E ? __popc(who[e]) : 0u, blocks = (n + 7) / 8;
      if (__all_sync(0xffffffffu, n == 0)) continue;
      uint32_t both = n | (blocks << 16);  // both at most 512
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, both, o);
        if (lane >= uint32_t(o)) both += u;
      }
      const uint32_t first = pairs + (both & 0xFFFFu) - n, at = items + (both >> 16) - blocks;
      if (n > 0) place[e] = uint16_t(first);
      for (uint32_t i = 0; i < blocks; i++) {
        r.item_e[at + i] = uint16_t(e);
        r.item_first[at + i] = uint16_t(first + 8 * i);
        r.item_n[at + i] = uint8_t(n - 8 * i < 8 ? n - 8 * i : 8);
      }
      both = __shfl_sync(0xffffffffu, both, 31);
      pairs += both & 0xFFFFu;
      items += both >> 16;
    }
    if (lane == 0) r.items = items;
  }
  __syncthreads();
  // by token within an expert
  if (lane < p.k && mine != 0) {
    const uint32_t at = place[mine_e] + __popc(who[mine_e] & ((1u << m) - 1u));
    r.pair[at] = uint16_t(m * p.k + lane);
    r.weight[at] = ex / sum;
  }
}

// The route, as the two products have it: from the workspace into shared
// memory (every thread; a barrier has to follow).  As much as there can be of
// it is copied, not as much as there is, which would have to be read first.
__device__ __forceinline__ void take_route(Route &r, const Route *from, uint32_t most) {
  const uint32_t tid = threadIdx.x;
  for (uint32_t i = tid; i < most; i += kThreads) {
    const float weight = from->weight[i];
    const uint16_t pair = from->pair[i], e = from->item_e[i], first = from->item_first[i];
    const uint8_t n = from->item_n[i];
    r.weight[i] = weight;
    r.pair[i] = pair;
    r.item_e[i] = e;
    r.item_first[i] = first;
    r.item_n[i] = n;
  }
  if (tid == 0) r.items = from->items;
}

// ---------------------------------------------------------------------------
constexpr uint32_t align128(uint32_t v) { return (v + 127) / 128 * 128; }

// kDepth: stages of the ring
template <uint32_t kDepth>
struct Up {
  static constexpr uint32_t kStage = align128(2 * kSubBytes + 8 * kXRow);
  static constexpr uint32_t kOwn = own_words(16);  // words of a warp: its queues, then its sums of G_e and U_e
  static constexpr uint32_t kRoute = kDepth * kStage;
  static constexpr uint32_t kQueues = align128(kRoute + uint32_t(sizeof(Route)));
  static constexpr uint32_t kBars = kQueues + kWarps * kOwn * 4;
  static constexpr uint32_t kSmem = kBars + sizeof(Bars);
};

// p_e silu(gate) up as two bf16 numbers, each rounded to nearest: off by at
// most 2^-18 of it.  A finite one that would round to infinity keeps its upper
// half, and the rest is the second; an infinite one has no second.
__device__ __forceinline__ void put_gated(uint16_t *dst, uint64_t plane, float gate, float up, float weight) {
  const float h = gate / (1.0f + expf(-gate)) * up * weight;
  uint32_t hi = bf16_bits(h);
  if ((hi & 0x7F80u) == 0x7F80u && fabsf(h) < INFINITY) hi = __float_as_uint(h) >> 16;
  dst[0] = uint16_t(hi);
  dst[plane] = uint16_t((hi & 0x7F80u) == 0x7F80u ? 0u : bf16_bits(h - __uint_as_float(hi << 16)));
}

// A stage's two subtiles: 64 rows of G_e and of U_e, the same values of H.
template <uint32_t kDepth>
__global__ void __launch_bounds__(kThreads, kDepth == 3 ? 4 : 3) k12_moe_up(const __grid_constant__ Params p,
                                                          const __grid_constant__ Planes planes, uint32_t csize) {
  extern __shared__ __align__(128) uint8_t dyn[];
  Route &r = *reinterpret_cast<Route *>(dyn + Up<kDepth>::kRoute);
  Bars &bars = *reinterpret_cast<Bars *>(dyn + Up<kDepth>::kBars);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x % csize, first = blockIdx.x / csize, clusters = gridDim.x / csize;
  View v;
  open_planes(v, p.gate_up, uint64_t(p.E) * 2 * p.F * p.H);
  const bool ok = open_header(v, p.gate_up, p.gate_up_bytes);  // the same for every thread
  launch_dependents();  // the down product's CTAs
  if (tid == 0) bars_init(bars);
  take_route(r, p.route, p.T * p.k);
  __syncthreads();
  if (!ok) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    return;
  }
  const uint32_t K = p.H, units = K / kUnit, u0 = units * rank / csize, u1 = units * (rank + 1) / csize;
  const uint32_t tiles = p.F / kSubRows, jobs = r.items * tiles, ring = smem_u32(dyn);
  Turn<kDepth> turn;
  if (warp == kWarps) {
    uint32_t s = 0;
    bool alive = true;
    for (uint32_t job = first; alive && job < jobs; job += clusters) {
      const uint32_t item = job / tiles, n = r.item_n[item];
      const uint32_t row = uint32_t(r.item_e[item]) * 2 * p.F + (job - item * tiles) * kSubRows;
      const uint16_t *px = p.x;
      if (lane < n) px += uint64_t(r.pair[r.item_first[item] + lane] / p.k) * K;
      for (uint32_t u = u0; u < u1; u++, s++, turn.next()) {
        if ((s >= kDepth && !bar_wait(bars, &bars.empty[turn.slot], turn.parity ^ 1, true, p.status)) ||
            (s == 1 && !bar_wait(bars, &bars.asked, 0, true, p.status))) {
          alive = false;
          break;
        }
        uint64_t *full = &bars.full[turn.slot];
        const uint32_t slot = ring + turn.slot * Up<kDepth>::kStage;
        if (lane == 0) {
          bar_expect(full, 2 * kSubBytes + n * 2 * kUnit);
          load_subtile(slot, planes, u * kUnit, row, full);
          load_subtile(slot + kSubBytes, planes, u * kUnit, row + p.F, full);
        }
        __syncwarp();
        if (lane < n) load_row(slot + 2 * kSubBytes + lane * kXRow, px + u * kUnit, 2 * kUnit, full);
      }
    }
    finish_copies(bars, turn, s, p.status);
    if (csize > 1 && first < jobs) {  // with the others' barriers
      cluster_sync();
      cluster_sync();
    }
    return;
  }
  auto row_of = [&](uint32_t job, uint32_t which) {
    const uint32_t item = job / tiles;
    return (uint64_t(r.item_e[item]) * 2 + which) * p.F + (job - item * tiles) * kSubRows + kRows * warp;
  };
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
  offsets(now, first);
  offsets(next, first + clusters);
  entries(now, first);
  __syncwarp();
  if (lane == 0) bar_arrive(&bars.asked);
  Exceptions x;
  x.q = reinterpret_cast<Queues *>(dyn + Up<kDepth>::kQueues + warp * Up<kDepth>::kOwn * 4);
  float *sums = reinterpret_cast<float *>(dyn + Up<kDepth>::kQueues);
  const uint64_t plane = uint64_t(p.T) * p.k * p.F;
  const XAt xat = x_rows(lane);
  const uint32_t g = lane >> 2, t = lane & 3;
  bool alive = true;
  const uint32_t fill = fill_stages(v);
  constexpr bool kParts = kDepth > 3;
  for (uint32_t job = first; job < jobs; job += clusters) {
    float gate[1][4] = {}, up[1][4] = {};
    uint32_t u = u0;
    do {
      const uint32_t end = kParts && u1 - u > fill ? u + fill : u1;
      exceptions_reset(x, lane);
      if (v.ne > 0) {
#pragma unroll 1
        for (uint32_t i = 0; i < 2; i++) window_keep(x, i ? now[1] : now[0], v, row_of(job, i), K, u, end, 2, i, lane, p.status);
        exceptions_ready(x, u, end, lane);
      }
      if (end == u1) {
        now[0] = next[0];
        now[1] = next[1];
        entries(now, job + clusters);
        offsets(next, job + 2 * clusters);
      }
      for (; alive && u < end; u++, turn.next()) {
        const uint32_t most = exceptions_most(x, 2 * u);
        alive = bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status);
        if (!alive) break;
        const uint32_t slot = ring + turn.slot * Up<kDepth>::kStage, xs = slot + 2 * kSubBytes;
        const StageAt at{slot, warp, xs, xs, 0, false, 2 * u, u, u, row_of(job, 0), row_of(job, 1)};
        stage<1, 1, true, false>(gate, up, at, xat, v, x, most, K, lane, p.status);
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.empty[turn.slot]);
      }
    } while (kParts && alive && u < u1);
    const uint32_t item = job / tiles, n = r.item_n[item], from = r.item_first[item], f0 = (job - item * tiles) * kSubRows;
    if (csize == 1) {  // a lane has both sums of its rows and columns
#pragma unroll
      for (uint32_t i = 0; i < 4; i++) {
        const uint32_t c = 2 * t + (i & 1), row = f0 + kRows * warp + g + 8 * (i >> 1);
        if (c < n) {
          const uint32_t pair = r.pair[from + c];
          put_gated(p.hs + uint64_t(pair) * p.F + row, plane, gate[0][i], up[0][i], r.weight[from + c]);
        }
      }
      continue;
    }
    __syncwarp();
    put_sums<1>(sums + warp * Up<kDepth>::kOwn, gate, lane);
    put_sums<1>(sums + warp * Up<kDepth>::kOwn + 8 * kRedTok, up, lane);
    cluster_sync();
    for (uint32_t o = tid + rank * kConsumers; o < n * kSubRows; o += kConsumers * csize) {
      const uint32_t row = o % kSubRows, c = o / kSubRows;
      const float *at = sums + row / kRows * Up<kDepth>::kOwn + c * kRedTok + row % kRows;
      float a = 0.0f, b = 0.0f;
      for (uint32_t i = 0; i < csize; i++) {
        a += cluster_load(at, i);
        b += cluster_load(at + 8 * kRedTok, i);
      }
      const uint32_t pair = r.pair[from + c];
      put_gated(p.hs + uint64_t(pair) * p.F + f0 + row, plane, a, b, r.weight[from + c]);
    }
    cluster_sync();  // the others' sums are read until here
  }
}

// ---------------------------------------------------------------------------
// A stage's two subtiles are successive ranges of F.
struct Down {
  static constexpr uint32_t kDepth = 3;
  static constexpr uint32_t kStage = align128(2 * kSubBytes + 16 * kXRow);
  static constexpr uint32_t kRoute = kDepth * kStage;
  static constexpr uint32_t kQueues = align128(kRoute + uint32_t(sizeof(Route)));
  static constexpr uint32_t kBars = kQueues + kWarps * uint32_t(sizeof(Queues));
  static constexpr uint32_t kAcc = align128(kBars + uint32_t(sizeof(Bars)));
  static __host__ __device__ uint32_t smem(uint32_t T) { return kAcc + kWarps * T * kRedTok * 4; }
};

__global__ void __launch_bounds__(kThreads, 3) k12_moe_down(const __grid_constant__ Params p,
                                                            const __grid_constant__ Planes planes, uint32_t csize) {
  constexpr uint32_t kDepth = Down::kDepth;
  extern __shared__ __align__(128) uint8_t dyn[];
  Route &r = *reinterpret_cast<Route *>(dyn + Down::kRoute);
  Bars &bars = *reinterpret_cast<Bars *>(dyn + Down::kBars);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x % csize, n0 = blockIdx.x / csize * kSubRows;
  View v;
  open_planes(v, p.down, uint64_t(p.E) * p.H * p.F);
  const bool ok = open_header(v, p.down, p.down_bytes);  // the same for every thread
  if (tid == 0) bars_init(bars);
  float *acc = reinterpret_cast<float *>(dyn + Down::kAcc) + warp * p.T * kRedTok;  // [token][row]
  if (warp < kWarps)
    for (uint32_t i = lane; i < p.T * kRedTok; i += 32) acc[i] = 0.0f;
  take_route(r, p.route, p.T * p.k);  // finished before the up product, beside which this one runs, began
  __syncthreads();
  // the items' stages one after another; this CTA's: [q0, q1)
  const uint32_t K = p.F, units = K / kUnit, per = (units + 1) / 2, all = r.items * per, ring = smem_u32(dyn);
  const uint32_t q0 = ok ? uint32_t(uint64_t(all) * rank / csize) : 0u, q1 = ok ? uint32_t(uint64_t(all) * (rank + 1) / csize) : 0u;
  const uint32_t first = q0 / per, st0 = q0 - first * per;  // item, stage of it
  if (!ok && blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
  Turn<kDepth> turn;
  if (warp == kWarps) {
    const uint64_t plane = uint64_t(p.T) * p.k * p.F;
    struct At {
      uint32_t item, st;
    } at{first, st0};
    auto step = [&](At &a) {
      if (++a.st == per) {
        a.st = 0;
        a.item++;
      }
    };
    auto subs_of = [&](uint32_t st) { return 2 * st + 1 < units ? 2u : 1u; };
    auto weights = [&](const Turn<kDepth> &turn, const At &a) {
      uint64_t *full = &bars.full[turn.slot];
      const uint32_t slot = ring + turn.slot * Down::kStage, subs = subs_of(a.st);
      const uint32_t row = uint32_t(r.item_e[a.item]) * p.H + n0;
      if (lane == 0) {
        bar_expect(full, subs * (kSubBytes + r.item_n[a.item] * 4 * kUnit));
        for (uint32_t i = 0; i < subs; i++) load_subtile(slot + i * kSubBytes, planes, (2 * a.st + i) * kUnit, row, full);
      }
      __syncwarp();
    };
    auto values = [&](const Turn<kDepth> &turn, const At &a) {  // lanes 0-7: the first plane, 8-15: the second
      const uint32_t i = lane & 7;
      if (lane < 16 && i < r.item_n[a.item])
        load_row(ring + turn.slot * Down::kStage + 2 * kSubBytes + lane * kXRow,
                 p.hs + (lane >> 3) * plane + uint64_t(r.pair[r.item_first[a.item] + i]) * K + 2 * a.st * kUnit,
                 subs_of(a.st) * 2 * kUnit, &bars.full[turn.slot]);
    };
    // the weights of the first stages are on their way before hs is waited
    // for, its values follow
    uint32_t s = 0;
    for (; q0 + s < q1 && s < kDepth; s++, turn.next()) {
      weights(turn, at);
      step(at);
    }
    wait_prerequisites();
    asm volatile("fence.proxy.async.global;" ::: "memory");
    Turn<kDepth> turn2;
    At at2{first, st0};
    for (uint32_t i = 0; i < s; i++, turn2.next()) {
      values(turn2, at2);
      step(at2);
    }
    for (; q0 + s < q1; s++, turn.next()) {
      if (!bar_wait(bars, &bars.empty[turn.slot], turn.parity ^ 1, true, p.status)) break;
      weights(turn, at);
      values(turn, at);
      step(at);
    }
    finish_copies(bars, turn, s, p.status);
  } else if (q0 < q1) {
    const uint32_t row0 = n0 + kRows * warp, last = (q1 - 1) / per;
    auto row_of = [&](uint32_t item) { return uint64_t(r.item_e[item]) * p.H + row0; };
    Window now, next;
    auto offsets = [&](Window &w, uint32_t i) {
      if (v.ne > 0 && i <= last) window_offsets(w, v.exc_off, row_of(i), K, lane);
    };
    auto entries = [&](Window &w, uint32_t i) {
      if (v.ne > 0 && i <= last) window_entries(w, v, lane);
    };
    offsets(now, first);
    offsets(next, first + 1);
    entries(now, first);
    Exceptions x;
    x.q = reinterpret_cast<Queues *>(dyn + Down::kQueues + warp * sizeof(Queues));
    const XAt xat = x_rows(lane);
    const bool wild = book_wild(v.book);
    const uint32_t fill = fill_stages(v);
    uint32_t st = st0;
    bool alive = true;
    for (uint32_t q = q0, item = first; alive && q < q1;) {
      const uint32_t last_st = q1 - q < per - st ? st + (q1 - q) : per, end = last_st - st > fill ? st + fill : last_st;
      exceptions_reset(x, lane);
      if (v.ne > 0) {
        const bool some = window_keep(x, now, v, row_of(item), K, 2 * st, 2 * end, 1, 0, lane, p.status);
        exceptions_ready(x, 2 * st, 2 * end, lane);
        x.short_of = x.short_of || __any_sync(0xffffffffu, some);
      }
      x.short_of = x.short_of || wild;
      if (end == last_st) {
        now = next;
        entries(now, item + 1);
        offsets(next, item + 2);
      }
      float tot0[1][4] = {}, tot1[1][4] = {};
      for (; st < end; st++, q++, turn.next()) {
        const uint32_t most = exceptions_most(x, 2 * st);
        alive = bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status);
        if (!alive) break;
        const uint32_t slot = ring + turn.slot * Down::kStage, xs = slot + 2 * kSubBytes, u = 2 * st;
        const StageAt at{slot, warp, xs, xs + 2 * kUnit, 8 * kXRow, u + 1 == units, u, u, u + 1, row_of(item), row_of(item)};
        stage<1, 2, false, false>(tot0, tot1, at, xat, v, x, most, K, lane, p.status);
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.empty[turn.slot]);
      }
      // columns to tokens; a token that did not choose the expert gets
      // nothing (not even zero times an infinite weight)
      const uint32_t n = r.item_n[item], from = r.item_first[item], g = lane >> 2, t = lane & 3;
#pragma unroll
      for (uint32_t i = 0; i < 2; i++)
        if (2 * t + i < n) {
          float *to = acc + r.pair[from + 2 * t + i] / p.k * kRedTok + g;
          to[0] += tot0[0][i] + tot1[0][i];
          to[8] += tot0[0][2 + i] + tot1[0][2 + i];
        }
      if (st == per) {
        item++;
        st = 0;
      }
    }
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  wait_prerequisites();
  if (ok) {
    const float *sums = reinterpret_cast<const float *>(dyn + Down::kAcc);
    for (uint32_t o = tid + rank * kThreads; o < p.T * kSubRows; o += kThreads * csize) {
      const uint32_t row = o % kSubRows, m = o / kSubRows;
      const float *from = sums + (row / kRows * p.T + m) * kRedTok + row % kRows;
      float sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += csize > 1 ? cluster_load(from, c) : *from;
      const uint64_t at = uint64_t(m) * p.H + n0 + row;
      if (p.wide) static_cast<float *>(p.out)[at] = sum;
      else static_cast<uint16_t *>(p.out)[at] = uint16_t(bf16_bits(sum));
    }
  }
  if (csize > 1) cluster_sync();  // the others' sums are read until here
}

// the CTAs of the up product that run at once on the device, the kernels set
// up
template <uint32_t kDepth>
int up_slots() {
  static DeviceSetup setup;
  return setup.get([] {
    int per_sm = 0;
    if (!share_sm(k12_moe_route<1>) || !share_sm(k12_moe_route<2>) || !share_sm(k12_moe_route<4>) || !share_sm(k12_moe_route<8>) ||
        !share_sm(k12_moe_route<16>) ||
        cudaFuncSetAttribute(k12_moe_up<kDepth>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Up<kDepth>::kSmem)) != cudaSuccess ||
        cudaFuncSetAttribute(k12_moe_down, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Down::smem(kMaxTokens))) != cudaSuccess ||
        cudaFuncSetAttribute(k12_moe_down, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k12_moe_up<kDepth>, kThreads, Up<kDepth>::kSmem) != cudaSuccess)
      return 0;
    return per_sm * wc12l::device_sms();
  });
}

}  // namespace wc12m

extern "C" uint64_t wc12_moe_work_bytes(uint32_t T, uint32_t k, uint32_t F) {
  const uint64_t t = T < wc12m::kMaxTokens ? T : wc12m::kMaxTokens;
  return wc12m::align128(sizeof(wc12m::Route)) + t * k * F * 4;
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
  // rows of H that are long enough fill a deeper ring of fewer CTAs (32 tokens,
  // 128 experts, H 2048: 200 us with 4 stages, 216 with 3, both before the up
  // product became an ordinary launch); of shorter ones more CTAs run, whose
  // ends overlap (16 tokens, H 1024: 64 us against 76)
  const bool deep = H >= 2048;
  const int slots = deep ? up_slots<4>() : up_slots<3>(), sms = slots > 0 ? wc12l::device_sms() : 0;
  if (sms <= 0) return cuda_failed();
  Params p;
  p.gate_up = static_cast<const uint8_t *>(d_gate_up);
  p.gate_up_bytes = gate_up_bytes;
  p.down = static_cast<const uint8_t *>(d_down);
  p.down_bytes = down_bytes;
  p.route = static_cast<Route *>(d_work);
  p.hs = reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(d_work) + align128(sizeof(Route)));
  p.E = E;
  p.H = H;
  p.F = F;
  p.k = k;
  p.renormalize = renormalize != 0;
  p.wide = out_dtype == WC_FP32;
  p.status = d_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Planes up, down;
  if (!make_planes(up, d_gate_up, uint64_t(E) * 2 * F, H) || !make_planes(down, d_down, uint64_t(E) * H, F)) return WC_ERR_CUDA;
  for (uint32_t m = 0; m < T; m += kMaxTokens) {
    p.T = T - m < kMaxTokens ? T - m : kMaxTokens;
    p.x = static_cast<const uint16_t *>(d_x) + uint64_t(m) * H;
    p.logits = d_logits + uint64_t(m) * E;
    p.out = static_cast<uint8_t *>(d_out) + uint64_t(m) * H * (p.wide ? 4 : 2);
    // up: clusters that split H until about 4 CTAs an SM have work; with
    // more jobs than that, as many CTAs as run at once
    const uint32_t pairs = p.T * k, jobs = pairs * (F / kSubRows);
    uint32_t cu = 1;
    while (cu < 8 && jobs * cu * 2 <= 4u * uint32_t(sms) && H / kUnit >= 8 * cu) cu *= 2;
    // down: CTAs that split the items, the same
    const uint32_t some = (pairs < E ? pairs : E) * (F / kUnit);  // units of a row, about
    uint32_t cd = 1;
    while (cd < 8 && H / kSubRows * (cd + 1) <= 3u * uint32_t(sms) && some >= 6 * (cd + 1)) cd++;
    // (clusters of 9 to 15 find no room beside one another: 32 tokens, 128
    // experts 203 -> 213 us)
    if (cd == 8 && H / kSubRows * 16 <= 3u * uint32_t(sms) && some >= 96) cd = 16;
    const uint32_t per = (E + 31) / 32;  // logits of a lane
    auto route = per <= 1 ? k12_moe_route<1> : per <= 2 ? k12_moe_route<2> : per <= 4 ? k12_moe_route<4> : per <= 8 ? k12_moe_route<8> : k12_moe_route<16>;
    if (launch(route, dim3(1), 32 * p.T, 1, 0, s, false, p) != cudaSuccess ||
        launch(deep ? k12_moe_up<4> : k12_moe_up<3>, dim3(cu > 1 ? jobs * cu : jobs < uint32_t(slots) ? jobs : uint32_t(slots)), kThreads, cu, deep ? Up<4>::kSmem : Up<3>::kSmem, s, false, p, up, cu) !=
            cudaSuccess ||
        launch(k12_moe_down, dim3(H / kSubRows * cd), kThreads, cd, Down::smem(p.T), s, true, p, down, cd) != cudaSuccess)
      return cuda_failed();
  }
  return WC_OK;
}
