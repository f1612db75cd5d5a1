// k_split12_moe.cu -- a mixture-of-experts layer for a few tokens, from the
// router's logits on, the experts' weights in two Split12 containers
// (wc12_moe, include/wc_split12.h):
//   S_t = the k largest logits of token t (ties: the lower expert)
//   p   = softmax of the logits over S_t, or over all experts
//   out[t] = sum over e in S_t of p_e D_e (silu(G_e x_t) * U_e x_t)
//
// The bytes of the chosen experts' weights bound it, so both kernels stream
// them through registers (wc12_few.cuh):
//   * k12_moe_up: a CTA takes 16 rows of G_e and the same of U_e for one
//     chosen expert e (4 warps each, splitting H) and the tokens that chose
//     it, and writes p_e silu(g) u, held as the sum of two bf16 numbers
//     (16 bits: rounding it to 8 would cost the output as much again as its
//     own rounding to bf16);
//   * k12_moe_down: a CTA takes 16 rows of the output and walks through D_e
//     of every chosen expert as through one long row, so that the weighted
//     sum over experts is part of the product's sum: no atomics, one
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
constexpr uint32_t kMaxK = 16;
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

struct Route {
  int16_t id[kMaxTokens][kMaxK];  // expert, -1: none
  float p[kMaxTokens][kMaxK];
  uint32_t bits[kMaxExperts / 32];  // chosen experts
  uint16_t act[kMaxExperts];        // the same, ascending
  uint32_t count;
};

// ascending in the logits' order; -0 like +0, NaN above all
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t b = v == 0.0f ? 0u : __float_as_uint(v);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;  // order_key(-inf)

// keys: kMaxExperts words a warp
__device__ void route(Route &r, uint32_t (*keys)[kMaxExperts], const Params &p) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kMaxExperts / 32) r.bits[tid] = 0;
  __syncthreads();
  for (uint32_t m = warp; m < p.T; m += kWarps) {
    const float *l = p.logits + uint64_t(m) * p.E;
    uint32_t *key = keys[warp];
    for (uint32_t e = lane; e < p.E; e += 32) key[e] = order_key(l[e]);
    // each lane looks at its own experts only: no barrier needed
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
      if (!none && (e & 31u) == lane) taken |= 1u << (e >> 5);
      if (!none) {
        const float v = l[e];
        if (j == 0) top = v;
        const float w = expf(v - top);
        if (lane == j) ex = w;
        sum += w;
        if (lane == 0) atomicOr(&r.bits[e >> 5], 1u << (e & 31u));
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
  // the chosen experts in order
  if (warp == 0) {
    const uint32_t b = lane < kMaxExperts / 32 ? r.bits[lane] : 0u;
    uint32_t incl = __popc(b);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= uint32_t(o)) incl += u;
    }
    uint32_t at = incl - __popc(b);
    for (uint32_t rest = b; rest; rest &= rest - 1) r.act[at++] = uint16_t(32 * lane + __ffs(rest) - 1);
    if (lane == 31) r.count = incl;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
struct UpSmem {
  Lists lists;
  Route route;
  float part[2 * kMaxTokens * kRows];  // the CTA's g and u, [token][row]
  uint32_t columns;
  uint16_t pair[kMaxTokens];  // of each column: token * k + j
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) k12_moe_up(const __grid_constant__ Params p, uint32_t csize) {
  launch_dependents();
  __shared__ UpSmem s;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = blockIdx.x % csize, f0 = blockIdx.x / csize * kRows;
  const uint32_t K = p.H, stages = (K + kStage - 1) / kStage, step = 4 * csize;
  route(s.route, s.lists.raw, p);
  if (blockIdx.y >= s.route.count) return;  // the whole cluster
  const uint32_t e = s.route.act[blockIdx.y];
  View v;
  open_planes(v, p.gate_up, uint64_t(p.E) * 2 * p.F * K);
  // warps 0-3: G_e, 4-7: U_e
  auto row_of = [&](uint32_t which) { return (uint64_t(e) * 2 + which) * p.F + f0; };
  const uint64_t row_g = row_of(warp >> 2) + g;
  const uint8_t *pi = v.idx + (row_g * K) / 2 + 8 * t, *pl = v.lo + row_g * K + 16 * t;
  const uint32_t gw = rank * 4 + (warp & 3);
  const uint32_t its = gw < stages ? (stages - gw + step - 1) / step : 0u;
  auto k_of = [&](uint32_t it) { return (gw + it * step) * kStage; };
  Frag f[2];
#pragma unroll
  for (uint32_t i = 0; i < 2; i++)
    if (i < its) load_frag(f[i], pi + k_of(i) / 2, pl + k_of(i), K, k_of(i) + 64 < K);
  if (!open_header(v, p.gate_up, p.gate_up_bytes)) {
    if (tid == 0) report(p.status, WC_ERR_CORRUPT);
    return;
  }
  // the tokens that chose e, in order: the columns
  if (warp == 0) {
    uint32_t j = 0xFFu;
    if (lane < p.T)
      for (uint32_t i = 0; i < p.k; i++)
        if (s.route.id[lane][i] == int16_t(e)) j = i;
    const uint32_t in = __ballot_sync(0xffffffffu, j != 0xFFu);
    if (j != 0xFFu) s.pair[__popc(in & ((1u << lane) - 1u))] = uint16_t(lane * p.k + j);
    if (lane == 0) s.columns = __popc(in);
  }
  gather(s.lists, v, K, 2, row_of,
         [&](uint32_t which, uint32_t stage, uint32_t &w, uint32_t &it) {
           const uint32_t o = stage % step;
           w = 4 * which + o % 4;
           it = stage / step;
           return o / 4 == rank;
         },
         p.status);
  const Exceptions x = exceptions_of(s.lists, warp, lane, (stages + step - 1) / step);
  const uint32_t columns = s.columns;
  const uint16_t *px[NT];
  uint32_t live = 0, tiles = 0;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const uint32_t c = 8 * nt + g;
    tiles |= 8u * nt < columns ? 1u << nt : 0u;
    live |= c < columns ? 1u << nt : 0u;
    px[nt] = p.x + uint64_t(c < columns ? s.pair[c] / p.k : 0u) * K + 16 * t;
  }
  float tot[NT][4] = {};
  for (uint32_t it0 = 0; it0 < its; it0 += 2) {
#pragma unroll
    for (uint32_t i = 0; i < 2; i++) {
      const uint32_t it = it0 + i;
      if (it >= its) break;
      const uint32_t k0 = k_of(it);
      const uint16_t *q[NT];
#pragma unroll
      for (int nt = 0; nt < NT; nt++) q[nt] = px[nt] + k0;
      const bool second = k0 + 64 < K;
      if (x.walk) stage_product<NT, 1, false, true>(tot, f[i], v, q, live, tiles, 0, second, x, it, row_g, K, k0, lane);
      else stage_product<NT, 1, false, false>(tot, f[i], v, q, live, tiles, 0, second, x, it, row_g, K, k0, lane);
      if (it + 2 < its) {
        const uint32_t k2 = k_of(it + 2);
        load_frag(f[i], pi + k2 / 2, pl + k2, K, k2 + 64 < K);
      }
    }
  }
  __syncthreads();  // the lists are read until here
  put_sums<NT>(s.lists.sums(warp, NT), tot, lane);
  __syncthreads();
  constexpr uint32_t kOut = 8 * NT * kRows;
  for (uint32_t o = tid; o < 2 * kOut; o += kThreads) {
    const uint32_t which = o / kOut, c = o % kOut / kRows, row = o % kRows;
    float sum = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < 4; w++) sum += s.lists.sums(4 * which + w, NT)[c * kRedTok + row];
    s.part[o] = sum;
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  const uint64_t plane = uint64_t(p.T) * p.k * p.F;
  for (uint32_t o = tid + rank * kThreads; o < kOut; o += kThreads * csize) {
    const uint32_t row = o % kRows, c = o / kRows;
    if (c >= columns) continue;
    float gate = s.part[o], up = s.part[kOut + o];
    if (csize > 1) {
      gate = up = 0.0f;
      for (uint32_t i = 0; i < csize; i++) {
        gate += cluster_load(&s.part[o], i);
        up += cluster_load(&s.part[kOut + o], i);
      }
    }
    const uint32_t pair = s.pair[c];
    const float h = gate / (1.0f + expf(-gate)) * up * s.route.p[pair / p.k][pair % p.k];
    // two bf16 numbers, each rounded to nearest: off by at most 2^-18
    uint16_t *dst = p.hs + uint64_t(pair) * p.F + f0 + row;
    const uint32_t hi = bf16_bits(h);
    dst[0] = uint16_t(hi);
    const float rest = h - __uint_as_float(hi << 16);
    dst[plane] = uint16_t((hi & 0x7F80u) == 0x7F80u ? 0u : bf16_bits(rest));
  }
  if (csize > 1) cluster_sync();  // the others' sums are read until here
}

// ---------------------------------------------------------------------------
struct DownSmem {
  Lists lists;
  Route route;
  float part[kMaxTokens * kRows];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) k12_moe_down(const __grid_constant__ Params p, uint32_t csize) {
  __shared__ DownSmem s;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = blockIdx.x % csize, n0 = blockIdx.x / csize * kRows;
  const uint32_t K = p.F, stages = (K + kStage - 1) / kStage, step = kWarps * csize;
  route(s.route, s.lists.raw, p);
  const uint32_t count = s.route.count, all = count * stages;
  View v;
  open_planes(v, p.down, uint64_t(p.E) * p.H * K);
  // the chosen experts' stages one after another; stage it of this warp is
  // stage gw + it * step of them
  const uint32_t gw = rank * kWarps + warp;
  const uint32_t its = gw < all ? (all - gw + step - 1) / step : 0u;
  auto row_of = [&](uint32_t a) { return uint64_t(s.route.act[a]) * p.H + n0; };
  auto load = [&](Frag &f, uint32_t it) {
    const uint32_t q = gw + it * step, a = q / stages, k0 = (q - a * stages) * kStage;
    const uint64_t at = (row_of(a) + g) * K + k0;
    load_frag(f, v.idx + at / 2 + 8 * t, v.lo + at + 16 * t, K, k0 + 64 < K);
  };
  Frag f[2];
#pragma unroll
  for (uint32_t i = 0; i < 2; i++)
    if (i < its) load(f[i], i);
  if (!open_header(v, p.down, p.down_bytes)) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    wait_prerequisites();
    return;
  }
  gather(s.lists, v, K, count, row_of,
         [&](uint32_t a, uint32_t stage, uint32_t &w, uint32_t &it) {
           const uint32_t q = a * stages + stage, o = q % step;
           w = o % kWarps;
           it = q / step;
           return o / kWarps == rank;
         },
         p.status);
  const Exceptions x = exceptions_of(s.lists, warp, lane, its > 0 ? its : 1);
  wait_prerequisites();  // hs
  const uint64_t plane = uint64_t(p.T) * p.k * p.F;
  float tot[NT][4] = {};
  for (uint32_t it0 = 0; it0 < its; it0 += 2) {
#pragma unroll
    for (uint32_t i = 0; i < 2; i++) {
      const uint32_t it = it0 + i;
      if (it >= its) break;
      const uint32_t q = gw + it * step, a = q / stages, k0 = (q - a * stages) * kStage;
      const int16_t e = int16_t(s.route.act[a]);
      const uint16_t *px[NT];
      uint32_t live = 0, tiles = 0;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        const uint32_t m = 8 * nt + g;
        px[nt] = p.hs;
        bool in = false;
        if (m < p.T)
          for (uint32_t j = 0; j < p.k; j++)
            if (s.route.id[m][j] == e) {
              in = true;
              px[nt] = p.hs + uint64_t(m * p.k + j) * K + k0 + 16 * t;
            }
        live |= in ? 1u << nt : 0u;
        if (NT > 1) tiles |= __any_sync(0xffffffffu, in) ? 1u << nt : 0u;
      }
      const bool second = k0 + 64 < K;
      const uint64_t row_g = row_of(a) + g;
      if (x.walk) stage_product<NT, 2, true, true>(tot, f[i], v, px, live, tiles, plane, second, x, it, row_g, K, k0, lane);
      else stage_product<NT, 2, true, false>(tot, f[i], v, px, live, tiles, plane, second, x, it, row_g, K, k0, lane);
      if (it + 2 < its) load(f[i], it + 2);
    }
  }
  __syncthreads();  // the lists are read until here
  put_sums<NT>(s.lists.sums(warp, NT), tot, lane);
  __syncthreads();
  constexpr uint32_t kOut = 8 * NT * kRows;
  for (uint32_t o = tid; o < kOut; o += kThreads) {
    const uint32_t row = o % kRows, m = o / kRows;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) sum += s.lists.sums(w, NT)[m * kRedTok + row];
    s.part[o] = sum;
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  for (uint32_t o = tid + rank * kThreads; o < kOut; o += kThreads * csize) {
    const uint32_t row = o % kRows, m = o / kRows;
    if (m >= p.T) continue;
    float sum = s.part[o];
    if (csize > 1) {
      sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += cluster_load(&s.part[o], c);
    }
    const uint64_t at = uint64_t(m) * p.H + n0 + row;
    if (p.wide) static_cast<float *>(p.out)[at] = sum;
    else static_cast<uint16_t *>(p.out)[at] = uint16_t(bf16_bits(sum));
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
  if (E == 0 || E > kMaxExperts || k == 0 || k > kMaxK || k > E) return WC_ERR_INVALID_ARG;
  if (H == 0 || F == 0 || H % 64 != 0 || F % 64 != 0 || H > (1u << 20) || F > (1u << 20)) return WC_ERR_INVALID_ARG;
  if (out_dtype != WC_BF16 && out_dtype != WC_FP32) return WC_ERR_INVALID_ARG;
  if (gate_up_bytes < 96 || down_bytes < 96) return WC_ERR_INVALID_ARG;
  const uint64_t n_up = uint64_t(E) * 2 * F * H, n_down = uint64_t(E) * H * F;
  if (gate_up_bytes < wc12::lay(n_up, 0).off_lo + n_up || down_bytes < wc12::lay(n_down, 0).off_lo + n_down)
    return WC_ERR_INVALID_ARG;
  // a warp meets at most 2^13 stages of the down product
  const uint32_t t0 = T < kMaxTokens ? T : kMaxTokens;
  const uint32_t most = t0 * k < E ? t0 * k : E;
  if (uint64_t(most) * ((F + kStage - 1) / kStage) > (uint64_t(kWarps) << kItBits)) return WC_ERR_INVALID_ARG;
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
  for (uint32_t m = 0; m < T; m += kMaxTokens) {
    p.T = T - m < kMaxTokens ? T - m : kMaxTokens;
    p.x = static_cast<const uint16_t *>(d_x) + uint64_t(m) * H;
    p.logits = d_logits + uint64_t(m) * E;
    p.out = static_cast<uint8_t *>(d_out) + uint64_t(m) * H * (p.wide ? 4 : 2);
    const uint32_t chosen = p.T * k < E ? p.T * k : E;  // experts, at most
    // CTAs that split a row: until every SM has two, while each warp has
    // a stage
    uint32_t cu = 1, cd = 1;
    while (cu < 8 && F / kRows * chosen * cu < 2u * uint32_t(sms) && (H + kStage - 1) / kStage >= 2 * cu * 4) cu *= 2;
    while (cd < 8 && H / kRows * cd < 2u * uint32_t(sms) && chosen * ((F + kStage - 1) / kStage) >= 2 * cd * kWarps) cd *= 2;
    auto up = p.T <= 8 ? k12_moe_up<1> : p.T <= 16 ? k12_moe_up<2> : k12_moe_up<4>;
    auto down = p.T <= 8 ? k12_moe_down<1> : p.T <= 16 ? k12_moe_down<2> : k12_moe_down<4>;
    if (launch(up, dim3(F / kRows * cu, chosen), cu, s, false, p, cu) != cudaSuccess) return WC_ERR_CUDA;
    if (launch(down, dim3(H / kRows * cd), cd, s, true, p, cd) != cudaSuccess) return WC_ERR_CUDA;
  }
  return WC_OK;
}
