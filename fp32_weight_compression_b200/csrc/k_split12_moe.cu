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
// k12_moe_route finds the experts first, a warp a token.  Each kernel starts
// while the one before it ends (programmatic dependent launch); the down
// product's has its route, exceptions and first weights by the time that the
// up product is done.
#include <cstdint>

#include "wc12_few.cuh"

namespace wc12m {

using namespace wc12f;

constexpr uint32_t kMaxTokens = 32;  // of a launch
constexpr uint32_t kMaxTop = 16;
constexpr uint32_t kMaxExperts = 512;

constexpr uint32_t kMaxPairs = kMaxTokens * kMaxTop;

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
  uint32_t *tickets;    // [kMaxTickets] of the up product, then of the down product; zeroed with the route
  float *parts;         // two segments' sums of each CTA, of one product, then of the other
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
// each.
template <int kPer>
__global__ void __launch_bounds__(32 * kMaxTokens) k12_moe_route(const __grid_constant__ Params p) {
  launch_dependents();
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
  for (uint32_t i = tid; i < 2 * kMaxTickets; i += blockDim.x) p.tickets[i] = 0;
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

struct Up {
  static constexpr uint32_t kStage = align128(2 * kSubBytes + 8 * kXRow);
  static constexpr uint32_t kRoute = kDepth * kStage;
  static constexpr uint32_t kQueues = align128(kRoute + uint32_t(sizeof(Route)));
  static constexpr uint32_t kBars = kQueues + kWarps * uint32_t(sizeof(Queues));
  static constexpr uint32_t kSmem = kBars + sizeof(Bars);
  static constexpr uint32_t kPart = 8 * kConsumers;  // floats of a segment's sums, 8 a lane
};

// p_e silu(gate) up as two bf16 numbers, each rounded to nearest: off by at
// most 2^-18 of it
__device__ __forceinline__ void put_gated(uint16_t *dst, uint64_t plane, float gate, float up, float weight) {
  const float h = gate / (1.0f + expf(-gate)) * up * weight;
  const uint32_t hi = bf16_bits(h);
  dst[0] = uint16_t(hi);
  dst[plane] = uint16_t((hi & 0x7F80u) == 0x7F80u ? 0u : bf16_bits(h - __uint_as_float(hi << 16)));
}

// A block (a job) is 64 rows of G_e and the same of U_e for one item, a
// stage's two subtiles those rows with the same values of H.
__global__ void __launch_bounds__(kThreads, 3) k12_moe_up(const __grid_constant__ Params p, const __grid_constant__ Planes planes) {
  extern __shared__ __align__(128) uint8_t dyn[];
  Route &r = *reinterpret_cast<Route *>(dyn + Up::kRoute);
  Bars &bars = *reinterpret_cast<Bars *>(dyn + Up::kBars);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  View v;
  open_planes(v, p.gate_up, uint64_t(p.E) * 2 * p.F * p.H);
  const bool ok = open_header(v, p.gate_up, p.gate_up_bytes);  // the same for every thread
  if (tid == 0) bars_init(bars);
  wait_prerequisites();  // the route
  launch_dependents();   // the down product's CTAs, which read the route too
  take_route(r, p.route, p.T * p.k);
  __syncthreads();
  if (!ok) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    return;
  }
  const uint32_t K = p.H, per = K / kUnit, tiles = p.F / kSubRows, ring = smem_u32(dyn);
  const Deal deal(r.items * tiles, per);
  if (blockIdx.x >= deal.ctas) return;
  const uint64_t q0 = deal.begin(blockIdx.x), q1 = deal.begin(blockIdx.x + 1);
  const uint32_t first = uint32_t(q0 / per), last = uint32_t((q1 - 1) / per), u_first = uint32_t(q0 - uint64_t(first) * per);
  Turn turn;
  if (warp == kWarps) {
    uint32_t n = 0;
    bool alive = true;
    for (uint32_t job = first, u = u_first; alive && job <= last; job++, u = 0) {
      const uint32_t item = job / tiles, columns = r.item_n[item];
      const uint32_t row = uint32_t(r.item_e[item]) * 2 * p.F + (job - item * tiles) * kSubRows;
      const uint16_t *px = p.x;
      if (lane < columns) px += uint64_t(r.pair[r.item_first[item] + lane] / p.k) * K;
      for (; u < per && n < uint32_t(q1 - q0); u++, n++, turn.next()) {
        if (n >= kDepth && !bar_wait(bars, &bars.empty[turn.slot], turn.parity ^ 1, true, p.status)) {
          alive = false;
          break;
        }
        uint64_t *full = &bars.full[turn.slot];
        const uint32_t slot = ring + turn.slot * Up::kStage;
        if (lane == 0) {
          bar_expect(full, 2 * kSubBytes + columns * 2 * kUnit);
          load_subtile(slot, planes, u * kUnit, row, full);
          load_subtile(slot + kSubBytes, planes, u * kUnit, row + p.F, full);
        }
        __syncwarp();
        if (lane < columns) load_row(slot + 2 * kSubBytes + lane * kXRow, px + u * kUnit, 2 * kUnit, full);
      }
    }
    finish_copies(bars, turn, n, p.status);  // no copy is in flight when the CTA ends
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
    if (v.ne > 0 && job <= last)
      for (uint32_t i = 0; i < 2; i++) window_offsets(w[i], v.exc_off, row_of(job, i), K, lane);
  };
  auto entries = [&](Window *w, uint32_t job) {
    if (v.ne > 0 && job <= last)
      for (uint32_t i = 0; i < 2; i++) window_entries(w[i], v, lane);
  };
  offsets(now, first);
  offsets(next, first + 1);
  entries(now, first);
  Exceptions x;
  x.q = reinterpret_cast<Queues *>(dyn + Up::kQueues + warp * sizeof(Queues));
  const uint64_t plane = uint64_t(p.T) * p.k * p.F;
  const XAt xat = x_rows(lane);
  const uint32_t g = lane >> 2, t = lane & 3;
  bool alive = true;
  uint64_t q = q0;
  for (uint32_t job = first, u = u_first; q < q1; job++, u = 0) {
    const uint32_t begin = u, end = q1 - q < per - u ? u + uint32_t(q1 - q) : per;
    exceptions_reset(x, lane);
    if (v.ne > 0) {
#pragma unroll 1
      for (uint32_t i = 0; i < 2; i++) window_keep(x, i ? now[1] : now[0], v, row_of(job, i), K, u, end, 2, i, lane, p.status);
      exceptions_ready(x, lane);
    }
    now[0] = next[0];
    now[1] = next[1];
    entries(now, job + 1);
    offsets(next, job + 2);
    const uint64_t row0 = row_of(job, 0), row1 = row_of(job, 1);
    float gate[1][4] = {}, up[1][4] = {};
    for (; u < end; u++, q++, turn.next()) {
      const uint32_t most = exceptions_most(x, 2 * u);
      alive = alive && bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status);
      if (!alive) {  // on to the end, with the others' barriers
        q += end - u;
        break;
      }
      const uint32_t slot = ring + turn.slot * Up::kStage, xs = slot + 2 * kSubBytes;
      const StageAt at{slot, warp, xs, xs, 0, false, 2 * u, u, u, row0, row1};
      stage<1, 1, true>(gate, up, at, xat, v, x, most, K, lane);
      __syncwarp();
      if (lane == 0) bar_arrive(&bars.empty[turn.slot]);
    }
    if (begin > 0 || end < per) {
      const uint32_t c0 = deal.cta_of(uint64_t(job) * per), c1 = deal.cta_of(uint64_t(job + 1) * per - 1);
      // a CTA's first segment's sums, then its last one's
      auto part_of = [&](uint32_t cta) {
        const uint32_t which = uint32_t(deal.begin(cta) / per) == job ? 0u : 1u;
        return reinterpret_cast<float4 *>(p.parts + (2 * uint64_t(cta) + which) * Up::kPart) + tid;
      };
      __stcg(part_of(blockIdx.x), make_float4(gate[0][0], gate[0][1], gate[0][2], gate[0][3]));
      __stcg(part_of(blockIdx.x) + kConsumers, make_float4(up[0][0], up[0][1], up[0][2], up[0][3]));
      if (!last_ticket(p.tickets, c0, c1 - c0 + 1, &bars.last)) continue;
#pragma unroll
      for (int i = 0; i < 4; i++) gate[0][i] = up[0][i] = 0.0f;
#pragma unroll 4
      for (uint32_t c = c0; c <= c1; c++) {
        const float4 a = __ldcg(part_of(c)), b = __ldcg(part_of(c) + kConsumers);
        gate[0][0] += a.x;
        gate[0][1] += a.y;
        gate[0][2] += a.z;
        gate[0][3] += a.w;
        up[0][0] += b.x;
        up[0][1] += b.y;
        up[0][2] += b.z;
        up[0][3] += b.w;
      }
    }
    const uint32_t item = job / tiles, n = r.item_n[item], from = r.item_first[item], f0 = (job - item * tiles) * kSubRows;
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {  // a lane has both sums of its rows and columns
      const uint32_t c = 2 * t + (i & 1), row = f0 + kRows * warp + g + 8 * (i >> 1);
      if (c < n)
        put_gated(p.hs + uint64_t(r.pair[from + c]) * p.F + row, plane, gate[0][i], up[0][i], r.weight[from + c]);
    }
  }
}

// ---------------------------------------------------------------------------
// A block is 64 rows of the output, its stages those of D_e's rows for every
// item, one item after another; a stage's two subtiles are successive ranges
// of F.
struct Down {
  static constexpr uint32_t kStage = align128(2 * kSubBytes + 16 * kXRow);
  static constexpr uint32_t kRoute = kDepth * kStage;
  static constexpr uint32_t kQueues = align128(kRoute + uint32_t(sizeof(Route)));
  static constexpr uint32_t kBars = kQueues + kWarps * uint32_t(sizeof(Queues));
  static constexpr uint32_t kAcc = align128(kBars + uint32_t(sizeof(Bars)));
  static constexpr uint32_t kPart = kSubRows;  // floats of a segment's sums and token
  static __host__ __device__ uint32_t smem(uint32_t T) { return kAcc + kWarps * T * kRedTok * 4; }
};

__global__ void __launch_bounds__(kThreads, 2) k12_moe_down(const __grid_constant__ Params p, const __grid_constant__ Planes planes) {
  extern __shared__ __align__(128) uint8_t dyn[];
  Route &r = *reinterpret_cast<Route *>(dyn + Down::kRoute);
  Bars &bars = *reinterpret_cast<Bars *>(dyn + Down::kBars);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  View v;
  open_planes(v, p.down, uint64_t(p.E) * p.H * p.F);
  const bool ok = open_header(v, p.down, p.down_bytes);  // the same for every thread
  if (tid == 0) bars_init(bars);
  take_route(r, p.route, p.T * p.k);  // the up product's CTAs had it before this one could start
  __syncthreads();
  const uint32_t K = p.F, units = K / kUnit, per = (units + 1) / 2;  // stages of an item
  const uint32_t all = r.items * per, blocks = p.H / kSubRows, ring = smem_u32(dyn);
  if (all == 0) {  // no token has an expert
    wait_prerequisites();
    for (uint64_t i = uint64_t(blockIdx.x) * kThreads + tid; i < uint64_t(p.T) * p.H; i += uint64_t(gridDim.x) * kThreads) {
      if (p.wide) static_cast<float *>(p.out)[i] = 0.0f;
      else static_cast<uint16_t *>(p.out)[i] = 0;
    }
    return;
  }
  const Deal deal(blocks, all);
  if (!ok || blockIdx.x >= deal.ctas) {
    if (!ok && blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    wait_prerequisites();
    return;
  }
  const uint64_t q0 = deal.begin(blockIdx.x), q1 = deal.begin(blockIdx.x + 1);
  // where a stage of the deal is: the block, the item, the item's stage
  struct At {
    uint32_t block, item, st;
  };
  auto at_of = [&](uint64_t q) {
    const uint32_t block = uint32_t(q / all), in = uint32_t(q - uint64_t(block) * all);
    return At{block, in / per, in - in / per * per};
  };
  auto step = [&](At &a) {
    if (++a.st == per) {
      a.st = 0;
      if (++a.item == r.items) {
        a.item = 0;
        a.block++;
      }
    }
  };
  Turn turn;
  if (warp == kWarps) {
    const uint64_t plane = uint64_t(p.T) * p.k * p.F;
    auto subs_of = [&](uint32_t st) { return 2 * st + 1 < units ? 2u : 1u; };
    auto weights = [&](const Turn &turn, const At &a) {
      uint64_t *full = &bars.full[turn.slot];
      const uint32_t slot = ring + turn.slot * Down::kStage, subs = subs_of(a.st);
      const uint32_t row = uint32_t(r.item_e[a.item]) * p.H + a.block * kSubRows;
      if (lane == 0) {
        bar_expect(full, subs * (kSubBytes + r.item_n[a.item] * 4 * kUnit));
        for (uint32_t i = 0; i < subs; i++) load_subtile(slot + i * kSubBytes, planes, (2 * a.st + i) * kUnit, row, full);
      }
      __syncwarp();
    };
    auto values = [&](const Turn &turn, const At &a) {  // lanes 0-7: the first plane, 8-15: the second
      const uint32_t i = lane & 7;
      if (lane < 16 && i < r.item_n[a.item])
        load_row(ring + turn.slot * Down::kStage + 2 * kSubBytes + lane * kXRow,
                 p.hs + (lane >> 3) * plane + uint64_t(r.pair[r.item_first[a.item] + i]) * K + 2 * a.st * kUnit,
                 subs_of(a.st) * 2 * kUnit, &bars.full[turn.slot]);
    };
    // the weights of the first stages are on their way before hs is waited
    // for, its values follow
    uint32_t n = 0;
    At at = at_of(q0);
    for (; q0 + n < q1 && n < kDepth; n++, turn.next()) {
      weights(turn, at);
      step(at);
    }
    wait_prerequisites();
    asm volatile("fence.proxy.async.global;" ::: "memory");
    Turn turn2;
    At at2 = at_of(q0);
    for (uint32_t i = 0; i < n; i++, turn2.next()) {
      values(turn2, at2);
      step(at2);
    }
    for (; q0 + n < q1; n++, turn.next()) {
      if (!bar_wait(bars, &bars.empty[turn.slot], turn.parity ^ 1, true, p.status)) break;
      weights(turn, at);
      values(turn, at);
      step(at);
    }
    finish_copies(bars, turn, n, p.status);
    return;
  }
  float *acc = reinterpret_cast<float *>(dyn + Down::kAcc) + warp * p.T * kRedTok;  // [token][row]
  const uint32_t g = lane >> 2, t = lane & 3;
  auto row_of = [&](const At &a) { return uint64_t(r.item_e[a.item]) * p.H + a.block * kSubRows + kRows * warp; };
  // the windows go from item to item, and on to the next block's first
  const At end_at = at_of(q1 - 1);
  auto after = [&](At a) {
    a.st = per - 1;
    step(a);
    return a;
  };
  auto has = [&](const At &a) { return v.ne > 0 && (a.block < end_at.block || (a.block == end_at.block && a.item <= end_at.item)); };
  At at = at_of(q0);
  Window now, next;
  if (has(at)) window_offsets(now, v.exc_off, row_of(at), K, lane);
  if (has(after(at))) window_offsets(next, v.exc_off, row_of(after(at)), K, lane);
  if (has(at)) window_entries(now, v, lane);
  Exceptions x;
  x.q = reinterpret_cast<Queues *>(dyn + Down::kQueues + warp * sizeof(Queues));
  const XAt xat = x_rows(lane);
  bool alive = true;
  uint64_t q = q0;
  while (q < q1) {
    const uint32_t block = at.block, begin = uint32_t(q - uint64_t(block) * all);
    const uint64_t block_end = q1 < uint64_t(block + 1) * all ? q1 : uint64_t(block + 1) * all;
    for (uint32_t i = lane; i < p.T * kRedTok; i += 32) acc[i] = 0.0f;
    __syncwarp();
    while (q < block_end) {  // an item
      const uint32_t item = at.item;
      const uint64_t left = block_end - q;
      uint32_t st = at.st;
      const uint32_t end = left < per - st ? st + uint32_t(left) : per;
      const uint64_t row0 = row_of(at);
      exceptions_reset(x, lane);
      if (v.ne > 0) {
        window_keep(x, now, v, row0, K, 2 * st, 2 * end, 1, 0, lane, p.status);
        exceptions_ready(x, lane);
      }
      now = next;
      const At at1 = after(at), at2 = after(at1);
      if (has(at1)) window_entries(now, v, lane);
      if (has(at2)) window_offsets(next, v.exc_off, row_of(at2), K, lane);
      float tot0[1][4] = {}, tot1[1][4] = {};
      for (; st < end; st++, q++, turn.next()) {
        const uint32_t most = exceptions_most(x, 2 * st);
        alive = alive && bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status);
        if (!alive) {  // on to the end, with the others' barriers
          q += end - st;
          break;
        }
        const uint32_t slot = ring + turn.slot * Down::kStage, xs = slot + 2 * kSubBytes, u = 2 * st;
        const StageAt sa{slot, warp, xs, xs + 2 * kUnit, 8 * kXRow, u + 1 == units, u, u, u + 1, row0, row0};
        stage<1, 2, false>(tot0, tot1, sa, xat, v, x, most, K, lane);
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.empty[turn.slot]);
      }
      // columns to tokens; a token that did not choose the expert gets
      // nothing (not even zero times an infinite weight)
      const uint32_t n = r.item_n[item], from = r.item_first[item];
#pragma unroll
      for (uint32_t i = 0; i < 2; i++)
        if (2 * t + i < n) {
          float *to = acc + r.pair[from + 2 * t + i] / p.k * kRedTok + g;
          to[0] += tot0[0][i] + tot1[0][i];
          to[8] += tot0[0][2 + i] + tot1[0][2 + i];
        }
      at = at1;
    }
    __syncwarp();
    const bool whole = begin == 0 && block_end == uint64_t(block + 1) * all;
    const uint32_t c0 = deal.cta_of(uint64_t(block) * all), c1 = deal.cta_of(uint64_t(block + 1) * all - 1);
    // a CTA's first segment's sums, then its last one's, a warp's [token][row]
    auto part_of = [&](uint32_t cta) {
      const uint32_t which = uint32_t(deal.begin(cta) / all) == block ? 0u : 1u;
      return p.parts + (2 * uint64_t(cta) + which) * Down::kPart * p.T + warp * kRows * p.T;
    };
    if (!whole) {
      float *mine = part_of(blockIdx.x);
      for (uint32_t i = lane; i < p.T * kRows; i += 32) __stcg(mine + i, acc[i / kRows * kRedTok + i % kRows]);
      wait_prerequisites();  // the tickets are zero since before this kernel could start
      if (!last_ticket(p.tickets + kMaxTickets, c0, c1 - c0 + 1, &bars.last)) continue;
    }
    for (uint32_t i = lane; i < p.T * kRows; i += 32) {
      float sum = 0.0f;
      if (whole) {
        sum = acc[i / kRows * kRedTok + i % kRows];
      } else {
#pragma unroll 4
        for (uint32_t c = c0; c <= c1; c++) sum += __ldcg(part_of(c) + i);
      }
      const uint64_t to = uint64_t(i / kRows) * p.H + block * kSubRows + kRows * warp + i % kRows;
      if (p.wide) static_cast<float *>(p.out)[to] = sum;
      else static_cast<uint16_t *>(p.out)[to] = uint16_t(bf16_bits(sum));
    }
    __syncwarp();  // acc is read until here
  }
}

// the device's SMs, the kernels set up
int moe_sms() {
  static DeviceSetup setup;
  return setup.get([] {
    return cudaFuncSetAttribute(k12_moe_up, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Up::kSmem)) == cudaSuccess &&
                   cudaFuncSetAttribute(k12_moe_down, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Down::smem(kMaxTokens))) ==
                       cudaSuccess
               ? wc12l::device_sms() : 0;
  });
}

// The workspace of a slice of at most kMaxTokens tokens.
struct Work {
  uint64_t tickets, parts, hs, total;
};
Work work_of(uint32_t T, uint32_t k, uint32_t F) {
  const uint64_t t = T < kMaxTokens ? T : kMaxTokens;
  Work w;
  w.tickets = align128(sizeof(Route));
  w.parts = w.tickets + 2 * kMaxTickets * 4;
  const uint64_t up = Up::kPart, down = Down::kPart * t;  // the down product's come after the up product's are read
  w.hs = w.parts + 2ull * kMaxTickets * 4 * (up > down ? up : down);
  w.total = w.hs + t * k * F * 4;
  return w;
}

}  // namespace wc12m

extern "C" uint64_t wc12_moe_work_bytes(uint32_t T, uint32_t k, uint32_t F) { return wc12m::work_of(T, k, F).total; }

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
  const int sms = moe_sms();
  if (sms <= 0) return WC_ERR_CUDA;
  Params p;
  p.gate_up = static_cast<const uint8_t *>(d_gate_up);
  p.gate_up_bytes = gate_up_bytes;
  p.down = static_cast<const uint8_t *>(d_down);
  p.down_bytes = down_bytes;
  const Work w = work_of(T, k, F);
  uint8_t *work = static_cast<uint8_t *>(d_work);
  p.route = reinterpret_cast<Route *>(work);
  p.tickets = reinterpret_cast<uint32_t *>(work + w.tickets);
  p.parts = reinterpret_cast<float *>(work + w.parts);
  p.hs = reinterpret_cast<uint16_t *>(work + w.hs);
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
    // CTAs that run at once: three an SM of the up product, two of the down
    // product (what its stages leave room for)
    const uint32_t most_up = 3u * uint32_t(sms) < kMaxTickets ? 3u * uint32_t(sms) : kMaxTickets;
    const uint32_t most_down = 2u * uint32_t(sms) < kMaxTickets ? 2u * uint32_t(sms) : kMaxTickets;
    const uint32_t per = (E + 31) / 32;  // logits of a lane
    auto route = per <= 1 ? k12_moe_route<1> : per <= 2 ? k12_moe_route<2> : per <= 4 ? k12_moe_route<4> : per <= 8 ? k12_moe_route<8> : k12_moe_route<16>;
    if (launch(route, dim3(1), 32 * p.T, 1, 0, s, false, p) != cudaSuccess ||
        launch(k12_moe_up, dim3(most_up), kThreads, 1, Up::kSmem, s, true, p, up) != cudaSuccess ||
        launch(k12_moe_down, dim3(most_down), kThreads, 1, Down::smem(p.T), s, true, p, down) != cudaSuccess)
      return WC_ERR_CUDA;
  }
  return WC_OK;
}
