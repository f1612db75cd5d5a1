// k_split12_adapters.cu -- the Split12 linear layer with low-rank adapters of
// many requests (wc12_linear_adapters, include/wc_split12.h):
//   y[m] = x[m] W^T + s_a (x[m] A_a^T) B_a^T,   a = adapter[m], none if -1,
// W (N x K bf16) held as a Split12 container, A (L x r x K) and B (L x N x r)
// bf16, s and y fp32.
//
// t[m] = s_a x[m] A_a^T is a few kilobytes, kept in fp32 in the caller's
// workspace (rounding it to bf16 would cost the output 2^-9 of the adapter's
// share).  Two ways on from there:
//   * few tokens (kFewTokens): the shared product is bound by W's bytes; one
//     kernel streams W through registers (wc12_few.cuh), waits for t only
//     when its sums are done, and adds t B^T to them.  The kernel that makes
//     t runs beside it (programmatic dependent launch).
//   * more: Y starts as the adapters' part, from a tensor-core product of t
//     (as the sum of three bf16 numbers) and B, and the tensor-memory kernel
//     of k_split12_linear.cu adds the shared product to it.
#include <cstdint>

#include "wc12_few.cuh"
#include "wc12_plan.cuh"

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

struct Params {
  const uint8_t *w;
  uint64_t w_bytes;
  const uint16_t *x;       // [M, K]
  const int32_t *adapter;  // [M]
  const uint16_t *a, *b;   // [L, r, K], [L, N, r]
  const float *scale;      // [L]
  float *t;                // [M, r]
  float *y;                // [M, N]
  uint32_t M, N, K, r, L;
  int32_t *status;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a value as the sum of three bf16 numbers, exact to 2^-24 and better of its
// size (each takes 8 bits off; truncated, so that the rest is exact in fp32)
__device__ __forceinline__ void split3(float v, uint32_t &h0, uint32_t &h1, uint32_t &h2) {
  h0 = __float_as_uint(v) & 0xFFFF0000u;
  const float r1 = v - __uint_as_float(h0);
  h1 = __float_as_uint(r1) & 0xFFFF0000u;
  h2 = __float_as_uint(r1 - __uint_as_float(h1)) & 0xFFFF0000u;
}

// ---------------------------------------------------------------------------
// t[m][j] = s_a sum_k x[m][k] A_a[j][k].  A cluster takes 8 tokens (x), 16
// ranks (y) and one adapter: that of token z of the 8, if it is the first
// with it.  The warps of its CTAs split K, 64 values at a time (16 a lane, as
// in wc12_few.cuh, A's rows in the place of the weights').
__global__ void __launch_bounds__(kSideThreads) k12_adapter_shrink(const __grid_constant__ Params p, uint32_t csize) {
  launch_dependents();
  __shared__ float red[kSideWarps][8 * kRedTok];
  __shared__ float part[128];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = blockIdx.x % csize, m0 = 8 * (blockIdx.x / csize), j0 = 16 * blockIdx.y, z = blockIdx.z;
  int32_t ad = -1;
  if (lane < 8 && m0 + lane < p.M) ad = p.adapter[m0 + lane];
  if (ad < -1 || ad >= int32_t(p.L)) {
    report(p.status, WC_ERR_INVALID_ARG);
    ad = -1;
  }
  const int32_t mine = __shfl_sync(0xffffffffu, ad, z);
  const uint32_t same = __ballot_sync(0xffffffffu, lane < 8 && ad == mine);
  if (mine < 0 || (same & ((1u << z) - 1u)) != 0) return;  // the whole cluster
  const bool live = (same >> g) & 1u;
  const uint16_t *px = p.x + uint64_t(m0 + g) * p.K + 16 * t;
  const bool r0 = j0 + g < p.r, r1 = j0 + g + 8 < p.r;
  const uint16_t *pa = p.a + (uint64_t(mine) * p.r + j0 + g) * p.K + 16 * t;
  float tot[1][4] = {};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
  for (uint32_t k = 64 * (rank * kSideWarps + warp); k < p.K; k += 64 * kSideWarps * csize) {
    uint4 a0[2] = {zero, zero}, a1[2] = {zero, zero}, xv[2] = {zero, zero};
    if (r0) {
      a0[0] = *reinterpret_cast<const uint4 *>(pa + k);
      a0[1] = *reinterpret_cast<const uint4 *>(pa + k + 8);
    }
    if (r1) {
      a1[0] = *reinterpret_cast<const uint4 *>(pa + uint64_t(8) * p.K + k);
      a1[1] = *reinterpret_cast<const uint4 *>(pa + uint64_t(8) * p.K + k + 8);
    }
    if (live) {
      xv[0] = *reinterpret_cast<const uint4 *>(px + k);
      xv[1] = *reinterpret_cast<const uint4 *>(px + k + 8);
    }
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t u0[4] = {a0[h].x, a1[h].x, a0[h].y, a1[h].y}, u1[4] = {a0[h].z, a1[h].z, a0[h].w, a1[h].w};
      mma(d, u0, xv[h].x, xv[h].y);
      mma(d, u1, xv[h].z, xv[h].w);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) tot[0][i] += d[i];
  }
  put_sums<1>(red[warp], tot, lane);
  __syncthreads();
  const uint32_t j = tid & 15, m = tid >> 4;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kSideWarps; w++) sum += red[w][m * kRedTok + j];
  if (csize > 1) {
    part[tid] = sum;
    cluster_sync();
    if (rank == 0) {
      sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += cluster_load(&part[tid], c);
    }
    cluster_sync();  // the others' sums are read until here
  }
  if (rank == 0 && ((same >> m) & 1u) && j0 + j < p.r) p.t[uint64_t(m0 + m) * p.r + j0 + j] = p.scale[mine] * sum;
}

// ---------------------------------------------------------------------------
// Few tokens: a CTA takes 64 weight rows and all tokens, the CTAs of a
// cluster split K.  A stage's two subtiles are successive ranges of K.
template <int NT>
struct Few {
  static constexpr uint32_t kXBox = NT * 1024;  // 8 NT tokens' values of a unit
  static constexpr uint32_t kStage = 2 * kSubBytes + 2 * kXBox;
  static constexpr uint32_t kOwn = own_words(8 * NT);  // words of a warp: its list, then its sums
  static constexpr uint32_t kLists = kDepth * kStage;
  static constexpr uint32_t kBars = kLists + kWarps * kOwn * 4;
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
  float *red = reinterpret_cast<float *>(dyn + F::kLists);
  if (warp == kWarps) {
    Turn turn;
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
    for (uint32_t i = 0; i < kDepth && u < u1; i++, u += 2, turn.next()) load(u);
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
    x.list = reinterpret_cast<uint32_t *>(dyn + F::kLists) + warp * F::kOwn;
    exceptions_reset(x);
    ok = open_header(v, p.w, p.w_bytes);
    float tot0[NT][4] = {}, tot1[NT][4] = {};
    if (ok) {
      if (v.ne > 0) {
        window_entries(win, v, lane);
        window_keep(x, win, v, row0, K, u0, u1, 1, 0, lane, p.status);
        exceptions_ready(x, lane);
      }
      const XAt xat = x_boxes(lane);
      Turn turn;
      for (uint32_t u = u0; u < u1; u += 2, turn.next()) {
        Handed h;
        const uint32_t most = exceptions_hand(x, h, u, lane);
        if (!bar_wait(bars, &bars.full[turn.slot], turn.parity, true, p.status)) break;
        const uint32_t slot = ring + turn.slot * F::kStage, xs = slot + 2 * kSubBytes;
        const StageAt at{slot, warp, xs, xs + F::kXBox, 1024, u + 1 == u1, u, u, u + 1, row0, row0};
        if (most == 1) stage_product<NT, 1, false, false>(tot0, tot1, at, xat, v.book, h, lane);
        else if (most == 2) stage_product<NT, 1, false, true>(tot0, tot1, at, xat, v.book, h, lane);
        else stage_product_slow<NT, 1, false>(tot0, tot1, at, xat, v, x, K, lane);
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

// the device's SMs, the kernels set up
int device_sms() {
  static DeviceSetup setup;
  return setup.get([] {
    return cudaFuncSetAttribute(k12_few_adapters<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Few<1>::kSmem)) == cudaSuccess &&
                   cudaFuncSetAttribute(k12_few_adapters<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Few<2>::kSmem)) ==
                       cudaSuccess
               ? wc12l::device_sms() : 0;
  });
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
             ? WC_OK : WC_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// More tokens: Y = the adapters' part (zero for a token without one).  A warp
// takes 16 rows of N and 32 tokens; t enters as three bf16 numbers.
__global__ void __launch_bounds__(kSideThreads) k12_adapter_expand(const __grid_constant__ Params p) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t n0 = (blockIdx.y * kSideWarps + warp) * kRows, m0 = 32 * blockIdx.x;
  int32_t ad = -1;
  if (m0 + lane < p.M) ad = p.adapter[m0 + lane];
  if (ad < 0 || ad >= int32_t(p.L)) ad = -1;
  float d[4][4] = {};
  wait_prerequisites();
  uint32_t rest = __ballot_sync(0xffffffffu, ad >= 0);
  while (rest) {
    const int32_t cur = __shfl_sync(0xffffffffu, ad, __ffs(rest) - 1);
    const uint32_t same = __ballot_sync(0xffffffffu, ad == cur);
    rest &= ~same;
    const uint16_t *pb = p.b + (uint64_t(cur) * p.N + n0 + g) * p.r + 4 * t;
    float c[4][4] = {};
    for (uint32_t j = 0; j < p.r; j += 16) {
      uint2 b0 = make_uint2(0u, 0u), b1 = b0;
      const bool in = j + 4 * t < p.r;
      if (in) {
        b0 = *reinterpret_cast<const uint2 *>(pb + j);
        b1 = *reinterpret_cast<const uint2 *>(pb + uint64_t(8) * p.r + j);
      }
      const uint32_t a[4] = {b0.x, b1.x, b0.y, b1.y};
#pragma unroll
      for (int nt = 0; nt < 4; nt++) {
        if (((same >> (8 * nt)) & 0xFFu) == 0) continue;
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in && ((same >> (8 * nt + g)) & 1u))
          q = *reinterpret_cast<const float4 *>(p.t + uint64_t(m0 + 8 * nt + g) * p.r + j + 4 * t);
        uint32_t h[4][3];
        split3(q.x, h[0][0], h[0][1], h[0][2]);
        split3(q.y, h[1][0], h[1][1], h[1][2]);
        split3(q.z, h[2][0], h[2][1], h[2][2]);
        split3(q.w, h[3][0], h[3][1], h[3][2]);
#pragma unroll
        for (int part = 2; part >= 0; part--)
          mma(c[nt], a, (h[0][part] >> 16) | h[1][part], (h[2][part] >> 16) | h[3][part]);
      }
    }
    // to this adapter's tokens only: another's zeros times an infinite value
    // of B would be NaN
#pragma unroll
    for (int nt = 0; nt < 4; nt++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        if ((same >> (8 * nt + 2 * t + (i & 1))) & 1u) d[nt][i] = c[nt][i];
  }
#pragma unroll
  for (int nt = 0; nt < 4; nt++)
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t m = m0 + 8 * nt + 2 * t + (i & 1), row = n0 + g + 8 * (i >> 1);
      if (m < p.M) p.y[uint64_t(m) * p.N + row] = d[nt][i];
    }
}

}  // namespace wc12a

extern "C" uint64_t wc12_linear_adapters_work_bytes(uint32_t M, uint32_t r) { return uint64_t(M) * r * 4; }

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
  if (sms <= 0) return WC_ERR_CUDA;
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
    const uint32_t tiles = (M + 7) / 8, ranks = (r + 15) / 16, z = M < 8 ? M : 8;
    uint32_t csize = 1;  // CTAs that split K: until each SM has two, while a warp has two pieces
    while (csize < 8 && tiles * ranks * csize < 2u * uint32_t(sms) && K / 64 >= 4 * csize * kSideWarps) csize *= 2;
    if (launch(k12_adapter_shrink, dim3(tiles * csize, ranks, z), kSideThreads, csize, 0, s, false, p, csize) != cudaSuccess)
      return WC_ERR_CUDA;
  }
  if (M <= kFewTokens) return M <= 8 ? launch_few<1>(p, sms, s) : launch_few<2>(p, sms, s);
  if (launch(k12_adapter_expand, dim3((M + 31) / 32, N / (kRows * kSideWarps)), kSideThreads, 1, 0, s, true, p) != cudaSuccess)
    return WC_ERR_CUDA;
  return wc12l::linear(d_w, w_bytes, d_plan, plan_bytes, N, K, d_x, M, d_y, true, d_status, stream);
}
