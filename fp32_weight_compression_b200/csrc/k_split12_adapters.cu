// k_split12_adapters.cu -- the Split12 linear layer with low-rank adapters of
// many requests (wc12_linear_adapters, include/wc_split12.h):
//   y[m] = x[m] W^T + s_a (x[m] A_a^T) B_a^T,   a = adapter[m], none if -1,
// W (N x K bf16) held as a Split12 container, A (L x r x K) and B (L x N x r)
// bf16, s and y fp32.
//
// t[m] = s_a x[m] A_a^T is a few kilobytes, kept in fp32 in the caller's
// workspace (rounding it to bf16 would cost the output 2^-9 of the adapter's
// share).  Two ways on from there:
//   * few tokens (kFewTokens): one kernel streams W through registers
//     (wc12_few.cuh), waits for t only when its sums are done, and adds t B^T
//     to them.  The kernel that makes t runs beside it (programmatic dependent
//     launch).  Graph replays: 4096 x 4096, 1 token: 10.3 us (25 MB, from L2);
//     4096 x 14336, 7 tokens: 25.3 (90 MB); 14336 x 4096, 16 tokens: 32.5 (99 MB),
//     where the tensor-memory kernel takes 36.5 for the shared product alone;
//   * more: Y starts as the adapters' part, from a tensor-core product of t
//     (as the sum of three bf16 numbers) and B, and the tensor-memory kernel
//     of k_split12_linear.cu, which starts beside that and needs Y at its end
//     only, adds the shared product to it.  Graph replays: 4096 x 4096, 203
//     tokens, rank 64: 36.5 us (41 one after another); 14336 x 4096, 2048 tokens:
//     503 to 514, of which the shared product's eight slices take 475: each brings
//     all tokens to each block of rows again, and twice as many a slice took
//     twice as long.
#include <cstdint>

#include "wc12_few.cuh"
#include "wc12_plan.cuh"
#include "wc12_ranks.cuh"

namespace wc12l {
int32_t linear(const void *d_w, uint64_t w_bytes, const void *d_plan, uint64_t plan_bytes, uint32_t N, uint32_t K,
               const void *d_x, uint32_t M, float *d_y, bool add, int32_t *d_status, void *stream);
int32_t check_linear(const void *d_w, uint64_t w_bytes, const void *d_plan, uint64_t plan_bytes, uint32_t N, uint32_t K,
                     const void *d_x, uint32_t M, const float *d_y, const int32_t *d_status);
}  // namespace wc12l

namespace wc12a {

using namespace wc12f;

constexpr uint32_t kFewTokens = 16;
constexpr uint32_t kMaxRank = 256;
// of the two small products with A and B
constexpr int kSideWarps = 4, kSideThreads = 32 * kSideWarps;
constexpr uint32_t kDepth = 3;  // stages of the ring, for four CTAs an SM

struct Params {
  const uint8_t *w;
  uint64_t w_bytes;
  const uint16_t *x;       // [M, K]
  const int32_t *adapter;  // [M]
  const uint16_t *a, *b;   // [L, r, K], [L, N, r]
  const float *scale;      // [L]
  float *t;                // [M, r], or three planes of bf16
  float *y;                // [M, N]
  uint32_t M, N, K, r, L;
  int32_t *status;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a value as the sum of three bf16 numbers, exact to 2^-24 and better of its
// size (each takes 8 bits off; truncated, so that the rest is exact in fp32);
// what is not finite in the first alone, since infinity less infinity is none
__device__ __forceinline__ void split3(float v, uint32_t &h0, uint32_t &h1, uint32_t &h2) {
  if ((__float_as_uint(v) & 0x7F800000u) == 0x7F800000u) {
    h0 = v != v ? 0x7FC00000u : __float_as_uint(v);  // a NaN whose upper half could read as infinity
    h1 = h2 = 0u;
    return;
  }
  h0 = __float_as_uint(v) & 0xFFFF0000u;
  const float r1 = v - __uint_as_float(h0);
  h1 = __float_as_uint(r1) & 0xFFFF0000u;
  h2 = __float_as_uint(r1 - __uint_as_float(h1)) & 0xFFFF0000u;
}

// loads that stay where they are written: all of a batch before its first use
__device__ __forceinline__ uint4 load16(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint16_t *p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// ---------------------------------------------------------------------------
// one adapter's part: the tokens `same` of the 8 kTiles from m0 on
template <int kTiles>
__device__ __forceinline__ void shrink_one(const Params &p, uint32_t csize, uint32_t rank, uint32_t m0, uint32_t j0, int32_t mine,
                                           uint32_t same, float (*red)[8 * kTiles * kRedTok], float *part) {
  constexpr int kTokens = 8 * kTiles, kBatch = kTiles == 1 ? 4 : 2;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  // ranks and tokens that do not exist are read as the last ones: their sums
  // are dropped, and the loads need no condition
  const uint32_t ra = j0 + g < p.r ? j0 + g : p.r - 1, rb = j0 + g + 8 < p.r ? j0 + g + 8 : p.r - 1;
  const uint16_t *pa = p.a + (uint64_t(mine) * p.r + ra) * p.K + 16 * t, *pb = p.a + (uint64_t(mine) * p.r + rb) * p.K + 16 * t;
  const uint16_t *px[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; i++) {
    const uint32_t m = m0 + 8 * i + g;
    px[i] = p.x + uint64_t(m < p.M ? m : p.M - 1) * p.K + 16 * t;
  }
  float tot[kTiles][4] = {};
  const uint32_t step = 64 * kSideWarps * csize;
  for (uint32_t k0 = 64 * (rank * kSideWarps + warp); k0 < p.K; k0 += kBatch * step) {
    uint4 a0[kBatch][2], a1[kBatch][2], xv[kBatch][kTiles][2];
#pragma unroll
    for (int b = 0; b < kBatch; b++) {
      const uint32_t k = k0 + b * step < p.K ? k0 + b * step : k0;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        a0[b][h] = load16(pa + k + 8 * h);
        a1[b][h] = load16(pb + k + 8 * h);
#pragma unroll
        for (int i = 0; i < kTiles; i++) xv[b][i][h] = load16(px[i] + k + 8 * h);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; b++) {
      if (k0 + b * step >= p.K) break;
#pragma unroll
      for (int i = 0; i < kTiles; i++) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const uint32_t u0[4] = {a0[b][h].x, a1[b][h].x, a0[b][h].y, a1[b][h].y}, u1[4] = {a0[b][h].z, a1[b][h].z, a0[b][h].w, a1[b][h].w};
          mma(d, u0, xv[b][i][h].x, xv[b][i][h].y);
          mma(d, u1, xv[b][i][h].z, xv[b][i][h].w);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) tot[i][j] += d[j];
      }
    }
  }
  put_sums<kTiles>(red[warp], tot, lane);
  __syncthreads();
  for (uint32_t o = tid; o < kTokens * 16; o += kSideThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kSideWarps; w++) sum += red[w][(o >> 4) * kRedTok + (o & 15)];
    part[o] = sum;
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  for (uint32_t o = tid + rank * kSideThreads; o < kTokens * 16; o += kSideThreads * csize) {
    const uint32_t j = o & 15, m = o >> 4;
    if (!((same >> m) & 1u) || j0 + j >= p.r) continue;
    float sum = part[o];
    if (csize > 1) {
      sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += cluster_load(&part[o], c);
    }
    sum *= p.scale[mine];
    const uint64_t at = uint64_t(m0 + m) * p.r + j0 + j;
    if (kTiles == 1) {
      p.t[at] = sum;
    } else {
      uint32_t h0, h1, h2;
      split3(sum, h0, h1, h2);
      uint16_t *q = reinterpret_cast<uint16_t *>(p.t) + at;
      const uint64_t plane = uint64_t(p.M) * p.r;
      q[0] = uint16_t(h0 >> 16);
      q[plane] = uint16_t(h1 >> 16);
      q[2 * plane] = uint16_t(h2 >> 16);
    }
  }
  if (csize > 1) cluster_sync(); else __syncthreads();  // the sums are read until here
}

// t[m][j] = s_a sum_k x[m][k] A_a[j][k].  A cluster takes 8 kTiles tokens (x),
// 16 ranks (y) and, of the adapters that its tokens have, the z-th and every
// gridDim.z-th one after it.  The warps of its CTAs split K, 64 values at a
// time (16 a lane, as in wc12_few.cuh, A's rows in the place of the
// weights'), kBatch of them in flight.  With 8 tokens t is written in fp32, with 32 (which the
// tensor-core product of t and B follows) as three planes of bf16.
template <int kTiles>
__global__ void __launch_bounds__(kSideThreads) k12_adapter_shrink(const __grid_constant__ Params p, uint32_t csize) {
  constexpr int kTokens = 8 * kTiles;
  launch_dependents();
  __shared__ float red[kSideWarps][kTokens * kRedTok];
  __shared__ float part[kTokens * 16];
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = blockIdx.x % csize, m0 = kTokens * (blockIdx.x / csize), j0 = 16 * blockIdx.y, z = blockIdx.z;
  int32_t ad = -1;
  if (lane < kTokens && m0 + lane < p.M) ad = p.adapter[m0 + lane];
  if (ad < -1 || ad >= int32_t(p.L)) {
    report(p.status, WC_ERR_INVALID_ARG);
    ad = -1;
  }
  // tokens that are the first with their adapter
  const uint32_t with_it = __match_any_sync(0xffffffffu, ad);  // every lane, before any condition
  uint32_t rest = __ballot_sync(0xffffffffu, ad >= 0 && uint32_t(__ffs(with_it) - 1) == lane);
  for (uint32_t i = 0; rest; rest &= rest - 1, i++) {
    if (i % gridDim.z != z) continue;
    const int32_t mine = __shfl_sync(0xffffffffu, ad, __ffs(rest) - 1);
    shrink_one<kTiles>(p, csize, rank, m0, j0, mine, __ballot_sync(0xffffffffu, ad == mine), red, part);
  }
}

// ---------------------------------------------------------------------------
// Few tokens: a CTA takes 64 weight rows and all tokens, the CTAs of a
// cluster split K.  A stage's two subtiles are successive ranges of K.
template <int NT>
struct Few {
  static constexpr uint32_t kXBox = NT * 1024;  // 8 NT tokens' values of a unit
  static constexpr uint32_t kStage = 2 * kSubBytes + 2 * kXBox;
  static constexpr uint32_t kOwn = own_words(8 * NT);  // words of a warp: its queues, then its sums
  static constexpr uint32_t kQueues = kDepth * kStage;
  static constexpr uint32_t kBars = kQueues + kWarps * kOwn * 4;
  static constexpr uint32_t kSmem = 1024 + kBars + sizeof(Bars);  // 1024: the boxes' swizzle counts from there
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 4) k12_few_adapters(const __grid_constant__ Params p,
                                                                const __grid_constant__ Planes planes,
                                                                const __grid_constant__ CUtensorMap tm_x, uint32_t csize) {
  using F = Few<NT>;
  extern __shared__ __align__(128) uint8_t raw[];
  uint8_t *dyn = raw + (1024 - smem_u32(raw) % 1024) % 1024;  // the same place in every CTA of the cluster
  Bars &bars = *reinterpret_cast<Bars *>(dyn + F::kBars);
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = blockIdx.x % csize, n0 = blockIdx.x / csize * kSubRows;
  const uint32_t K = p.K, units = K / kUnit, u0 = units * rank / csize, u1 = units * (rank + 1) / csize;
  const uint32_t ring = smem_u32(dyn);
  View v;
  open_planes(v, p.w, uint64_t(p.N) * K);
  if (tid == 0) bars_init(bars);
  __syncthreads();
  bool ok;
  float *red = reinterpret_cast<float *>(dyn + F::kQueues);
  if (warp == kWarps) {
    Turn<kDepth> turn;
    auto load = [&](uint32_t u) {
      if (lane == 0) {
        uint64_t *full = &bars.full[turn.slot];
        const uint32_t slot = ring + turn.slot * F::kStage, subs = u + 1 < u1 ? 2 : 1;
        bar_expect(full, subs * (kSubBytes + F::kXBox));
        for (uint32_t i = 0; i < subs; i++) {
          load_subtile(slot + i * kSubBytes, planes, (u + i) * kUnit, n0, full);
          load_box(slot + 2 * kSubBytes + i * F::kXBox, &tm_x, (u + i) * kUnit, 0, full);
        }
      }
      __syncwarp();
    };
    uint32_t u = u0;
    load(u);
    u += 2;
    turn.next();
    if (bar_wait(bars, &bars.asked, 0, false, p.status))
      for (uint32_t i = 1; i < kDepth && u < u1; i++, u += 2, turn.next()) load(u);
    ok = open_header(v, p.w, p.w_bytes);  // the same for every thread
    // B's rows for the tokens' adapters, on their way to L2 for the end
    if (lane < p.M) {
      const int32_t ad = p.adapter[lane];
      if (ad >= 0 && ad < int32_t(p.L)) prefetch_l2(p.b + (uint64_t(ad) * p.N + n0) * p.r, kSubRows * p.r * 2);
    }
    for (; ok && u < u1; u += 2, turn.next()) {
      if (!bar_wait(bars, &bars.empty[turn.slot], turn.parity ^ 1, true, p.status)) break;
      load(u);
    }
    // no copy is in flight when the CTA ends
    finish_copies(bars, turn, (u - u0) / 2, p.status);
  } else {
    const uint32_t row0 = n0 + kRows * warp;
    Window win;
    window_offsets(win, v.exc_off, row0, K, lane);
    Exceptions x;
    x.q = reinterpret_cast<Queues *>(dyn + F::kQueues + warp * F::kOwn * 4);
    exceptions_reset(x, lane);
    ok = open_header(v, p.w, p.w_bytes);
    float tot0[NT][4] = {}, tot1[NT][4] = {};
    if (ok && v.ne > 0) window_entries(win, v, lane);
    __syncwarp();
    if (lane == 0) bar_arrive(&bars.asked);
    if (ok) {
      if (v.ne > 0) {
        window_keep(x, win, v, row0, K, u0, u1, 1, 0, lane, p.status);
        exceptions_ready(x, u0, u1, lane);
      }
      const XAt xat = x_boxes(lane);
      Turn<kDepth> turn;
      for (uint32_t u = u0; u < u1; u += 2, turn.next()) {
        const uint32_t most = exceptions_most(x, u);
        if (!bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status)) break;
        const uint32_t slot = ring + turn.slot * F::kStage, xs = slot + 2 * kSubBytes;
        const StageAt at{slot, warp, xs, xs + F::kXBox, 1024, u + 1 == u1, u, u, u + 1, row0, row0};
        stage<NT, 1, false, true>(tot0, tot1, at, xat, v, x, most, K, lane, p.status);
        __syncwarp();
        if (lane == 0) bar_arrive(&bars.empty[turn.slot]);
      }
    } else if (blockIdx.x == 0 && tid == 0) {
      report(p.status, WC_ERR_CORRUPT);
    }
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) tot0[i][j] += tot1[i][j];
    __syncwarp();
    put_sums<NT>(red + warp * F::kOwn, tot0, lane);
  }
  // a thread has one row of every so many tokens; their adapters, and the
  // first 16 ranks' values of B, are read before the others are waited for
  constexpr uint32_t kOut = 8 * NT * kSubRows / kConsumers;
  const uint32_t row = tid % kSubRows, m0 = tid / kSubRows + kConsumers / kSubRows * rank, per = kConsumers / kSubRows * csize;
  int32_t ad[kOut];
  uint4 b0[kOut], b1[kOut];
  const bool puts = ok && warp < kWarps;
#pragma unroll
  for (uint32_t i = 0; i < kOut; i++) {
    const uint32_t m = m0 + i * per;
    ad[i] = puts && m < p.M ? p.adapter[m] : -1;
    if (ad[i] >= int32_t(p.L)) ad[i] = -1;
  }
  auto b_of = [&](uint32_t i) { return reinterpret_cast<const uint4 *>(p.b + (uint64_t(ad[i]) * p.N + n0 + row) * p.r); };
#pragma unroll
  for (uint32_t i = 0; i < kOut; i++) {
    b0[i] = b1[i] = make_uint4(0u, 0u, 0u, 0u);
    if (ad[i] >= 0) {
      b0[i] = b_of(i)[0];
      if (p.r > 8) b1[i] = b_of(i)[1];
    }
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  wait_prerequisites();  // t
  if (puts) {
#pragma unroll
    for (uint32_t i = 0; i < kOut; i++) {
      const uint32_t m = m0 + i * per;
      if (m >= p.M) break;
      const float *from = red + row / kRows * F::kOwn + m * kRedTok + row % kRows;
      float sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += csize > 1 ? cluster_load(from, c) : *from;
      if (ad[i] >= 0) {
        const float4 *pt = reinterpret_cast<const float4 *>(p.t + uint64_t(m) * p.r);
        float add = 0.0f;
        auto take = [&](uint4 b, uint32_t j) {
          const float4 t0 = pt[2 * j], t1 = pt[2 * j + 1];
          add += t0.x * bf16_lo(b.x) + t0.y * bf16_hi(b.x) + t0.z * bf16_lo(b.y) + t0.w * bf16_hi(b.y);
          add += t1.x * bf16_lo(b.z) + t1.y * bf16_hi(b.z) + t1.z * bf16_lo(b.w) + t1.w * bf16_hi(b.w);
        };
        take(b0[i], 0);
        if (p.r > 8) take(b1[i], 1);
        for (uint32_t j = 2; j < p.r / 8; j++) take(b_of(i)[j], j);
        sum += add;
      }
      p.y[uint64_t(m) * p.N + n0 + row] = sum;
    }
  }
  if (csize > 1) cluster_sync();  // the others' sums are read until here
}

template <int NT>
int32_t launch_few(const Params &p, int sms, cudaStream_t s) {
  using F = Few<NT>;
  Planes planes;
  CUtensorMap tm_x;
  if (!make_planes(planes, p.w, p.N, p.K) ||
      !wc12l::make_map(&tm_x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.x, p.K, p.M, uint64_t(p.K) * 2, kUnit, 8 * NT,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B))
    return WC_ERR_CUDA;
  // CTAs that split K: as many as run at once (4 an SM), while each fills
  // its ring
  const uint32_t blocks = p.N / kSubRows, units = p.K / kUnit;
  uint32_t csize = 1;
  while (csize < 8 && blocks * csize * 2 <= 4u * uint32_t(sms) && units >= 4 * csize * kDepth) csize *= 2;
  return launch(k12_few_adapters<NT>, dim3(blocks * csize), kThreads, csize, F::kSmem, s, true, p, planes, tm_x, csize) ==
                 cudaSuccess
             ? WC_OK : cuda_failed();
}

// ---------------------------------------------------------------------------
// More tokens: Y = the adapters' part (zero for a token without one).  A warp
// takes 16 rows of N and 32 tokens; t enters as three bf16 numbers.
__global__ void __launch_bounds__(kSideThreads, 6) k12_adapter_expand(const __grid_constant__ Params p) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  launch_dependents();  // the shared product, which adds to Y at its end only
  const uint32_t n0 = (blockIdx.y * kSideWarps + warp) * kRows, m0 = 32 * blockIdx.x;
  int32_t ad = m0 + lane < p.M ? p.adapter[m0 + lane] : -1;
  if (ad < 0 || ad >= int32_t(p.L)) ad = -1;
  const uint64_t plane = uint64_t(p.M) * p.r;
  const uint16_t *pt[4];  // tokens that do not exist are read as the last one, and dropped
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t m = m0 + 8 * i + g;
    pt[i] = reinterpret_cast<const uint16_t *>(p.t) + uint64_t(m < p.M ? m : p.M - 1) * p.r;
  }
  // a token's part goes to Y as its adapter's turn comes: another adapter's
  // infinite values never meet it
  auto put = [&](const float (*c)[4], uint32_t tokens) {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t m = 8 * i + 2 * t + (j & 1);
        if ((tokens >> m) & 1u) p.y[uint64_t(m0 + m) * p.N + n0 + g + 8 * (j >> 1)] = c[i][j];
      }
  };
  wait_prerequisites();
  uint32_t rest = __ballot_sync(0xffffffffu, ad >= 0);
  const uint32_t exist = __ballot_sync(0xffffffffu, m0 + lane < p.M);
  if (exist & ~rest) {
    const float zero[4][4] = {};
    put(zero, exist & ~rest);
  }
  while (rest) {
    const int32_t cur = __shfl_sync(0xffffffffu, ad, __ffs(rest) - 1);
    const uint32_t same = __ballot_sync(0xffffffffu, ad == cur);
    rest &= ~same;
    const uint16_t *pb = p.b + (uint64_t(cur) * p.N + n0 + g) * p.r;
    float c[4][4] = {};
#pragma unroll 1
    for (uint32_t j = 0; j < p.r; j += 16) {
      const bool in = has_ranks(j, t, p.r);
      const uint32_t k = ranks_from(j, t, p.r);
      uint2 b0 = load8(pb + k), b1 = load8(pb + uint64_t(8) * p.r + k), v[4][3];
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int part = 0; part < 3; part++) v[i][part] = load8(pt[i] + k + part * plane);
      if (!in) {  // ranks past the last, in the last step of a rank that is no multiple of 16
        b0 = b1 = make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
          for (int part = 0; part < 3; part++) v[i][part] = make_uint2(0u, 0u);
      }
      // an infinite B times t's first part is infinite; times a lower one, a
      // zero or of the other sign, it would make that NaN
      const uint32_t a[4] = {b0.x, b1.x, b0.y, b1.y}, low[4] = {finite2(b0.x), finite2(b1.x), finite2(b0.y), finite2(b1.y)};
#pragma unroll
      for (int part = 2; part >= 0; part--)
#pragma unroll
        for (int i = 0; i < 4; i++) mma(c[i], part ? low : a, v[i][part].x, v[i][part].y);
    }
    put(c, same);
  }
}

// the device's SMs, the kernels set up
int device_sms() {
  static DeviceSetup setup;
  return setup.get([] {
    return cudaFuncSetAttribute(k12_few_adapters<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Few<1>::kSmem)) == cudaSuccess &&
                   share_sm(k12_adapter_shrink<1>) && share_sm(k12_adapter_shrink<4>) && share_sm(k12_adapter_expand) &&
                   cudaFuncSetAttribute(k12_few_adapters<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Few<2>::kSmem)) ==
                       cudaSuccess
               ? wc12l::device_sms() : 0;
  });
}

}  // namespace wc12a

extern "C" uint64_t wc12_linear_adapters_work_bytes(uint32_t M, uint32_t r) {
  return uint64_t(M) * r * (M <= wc12a::kFewTokens ? 4 : 6);
}

extern "C" int32_t wc12_linear_adapters(const void *d_w, uint64_t w_bytes, const void *d_plan, uint64_t plan_bytes,
                                        uint32_t N, uint32_t K, const void *d_x, uint32_t M, const int32_t *d_adapter,
                                        const void *d_a, const void *d_b, const float *d_scale, uint32_t L, uint32_t r,
                                        float *d_y, void *d_work, uint64_t work_bytes, int32_t *d_status,
                                        void *stream) {
  using namespace wc12a;
  auto aligned = [](const void *q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; };
  const int32_t rc = wc12l::check_linear(d_w, w_bytes, d_plan, plan_bytes, N, K, d_x, M, d_y, d_status);
  if (rc != WC_OK) return rc;
  if (d_adapter == nullptr || d_a == nullptr || d_b == nullptr || d_scale == nullptr || d_work == nullptr)
    return WC_ERR_INVALID_ARG;
  if (!aligned(d_adapter, 4) || !aligned(d_a, 16) || !aligned(d_b, 16) || !aligned(d_scale, 4) || !aligned(d_work, 16))
    return WC_ERR_INVALID_ARG;
  if (L == 0 || L > 0x7FFFFFFFu || r == 0 || r % 8 != 0 || r > kMaxRank || K > kMaxK || N / (kRows * kSideWarps) > 65535 || M > 0x7FFFFFFFu)
    return WC_ERR_INVALID_ARG;
  if (work_bytes < wc12_linear_adapters_work_bytes(M, r)) return WC_ERR_CAPACITY;
  const int sms = device_sms();
  if (sms <= 0) return cuda_failed();
  Params p;
  p.w = static_cast<const uint8_t *>(d_w);
  p.w_bytes = w_bytes;
  p.x = static_cast<const uint16_t *>(d_x);
  p.adapter = d_adapter;
  p.a = static_cast<const uint16_t *>(d_a);
  p.b = static_cast<const uint16_t *>(d_b);
  p.scale = d_scale;
  p.t = static_cast<float *>(d_work);
  p.y = d_y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.r = r;
  p.L = L;
  p.status = d_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  {
    const uint32_t tokens = M <= kFewTokens ? 8 : 32, tiles = (M + tokens - 1) / tokens, ranks = (r + 15) / 16;
    // the tokens' adapters side by side, and CTAs that split K, until each
    // SM has some CTAs (while a warp has two pieces)
    uint32_t z = 1, csize = 1;
    while (z < tokens && z < M && tiles * ranks * z < 2u * uint32_t(sms)) z *= 2;
    while (csize < 8 && tiles * ranks * csize < 2u * uint32_t(sms) && K / 64 >= 4 * csize * kSideWarps) csize *= 2;
    if (launch(M <= kFewTokens ? k12_adapter_shrink<1> : k12_adapter_shrink<4>, dim3(tiles * csize, ranks, z), kSideThreads, csize, 0, s,
               false, p, csize) != cudaSuccess)
      return cuda_failed();
  }
  if (M <= kFewTokens) return M <= 8 ? launch_few<1>(p, sms, s) : launch_few<2>(p, sms, s);
  if (launch(k12_adapter_expand, dim3((M + 31) / 32, N / (kRows * kSideWarps)), kSideThreads, 1, 0, s, true, p) != cudaSuccess)
    return cuda_failed();
  return wc12l::linear(d_w, w_bytes, d_plan, plan_bytes, N, K, d_x, M, d_y, true, d_status, stream);
}
