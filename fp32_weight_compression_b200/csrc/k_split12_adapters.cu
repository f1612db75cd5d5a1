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
int device_sms();
}  // namespace wc12l

namespace wc12a {

using namespace wc12f;

constexpr uint32_t kFewTokens = 16;
constexpr uint32_t kMaxRank = 256;

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
// t[m][j] = s_a sum_k x[m][k] A_a[j][k].  A CTA takes 8 tokens (blockIdx.x),
// 16 ranks (y) and one adapter: that of token z of the 8, if it is the first
// with it.  Its 8 warps split K, 64 values at a time (16 a lane, as in
// wc12_few.cuh, A's rows in the place of the weights').
__global__ void __launch_bounds__(kThreads) k12_adapter_shrink(const __grid_constant__ Params p) {
  launch_dependents();
  __shared__ float red[kWarps][8 * kRedTok];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t m0 = 8 * blockIdx.x, j0 = 16 * blockIdx.y, z = blockIdx.z;
  int32_t ad = -1;
  if (lane < 8 && m0 + lane < p.M) ad = p.adapter[m0 + lane];
  if (ad < -1 || ad >= int32_t(p.L)) {
    report(p.status, WC_ERR_INVALID_ARG);
    ad = -1;
  }
  const int32_t mine = __shfl_sync(0xffffffffu, ad, z);
  const uint32_t same = __ballot_sync(0xffffffffu, lane < 8 && ad == mine);
  if (mine < 0 || (same & ((1u << z) - 1u)) != 0) return;
  const bool live = (same >> g) & 1u;
  const uint16_t *px = p.x + uint64_t(m0 + g) * p.K + 16 * t;
  const bool r0 = j0 + g < p.r, r1 = j0 + g + 8 < p.r;
  const uint16_t *pa = p.a + (uint64_t(mine) * p.r + j0 + g) * p.K + 16 * t;
  float tot[1][4] = {};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
  for (uint32_t k = 64 * warp; k < p.K; k += 64 * kWarps) {
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
  if (tid < 128) {
    const uint32_t j = tid & 15, m = tid >> 4;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) sum += red[w][m * kRedTok + j];
    if (((same >> m) & 1u) && j0 + j < p.r) p.t[uint64_t(m0 + m) * p.r + j0 + j] = p.scale[mine] * sum;
  }
}

// ---------------------------------------------------------------------------
// Few tokens: 16 weight rows a cluster (its CTAs split K), all tokens.
struct FewSmem {
  Lists lists;
  float part[kFewTokens * kRows];  // the CTA's sums, [token][row]
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2) k12_few_adapters(const __grid_constant__ Params p, uint32_t csize) {
  __shared__ FewSmem s;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t rank = blockIdx.x % csize, n0 = blockIdx.x / csize * kRows;
  const uint32_t K = p.K, stages = (K + kStage - 1) / kStage, step = kWarps * csize;
  View v;
  open_planes(v, p.w, uint64_t(p.N) * K);
  // stage it of this warp is stage gw + it * step of the row
  const uint32_t gw = rank * kWarps + warp;
  const uint8_t *pi = v.idx + (uint64_t(n0 + g) * K) / 2 + 8 * t, *pl = v.lo + uint64_t(n0 + g) * K + 16 * t;
  const uint32_t its = gw < stages ? (stages - gw + step - 1) / step : 0u;
  auto k_of = [&](uint32_t it) { return (gw + it * step) * kStage; };
  Frag f[2];
#pragma unroll
  for (uint32_t i = 0; i < 2; i++)
    if (i < its) load_frag(f[i], pi + k_of(i) / 2, pl + k_of(i), K, k_of(i) + 64 < K);
  const bool ok = open_header(v, p.w, p.w_bytes);  // the same in every CTA
  if (!ok) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    wait_prerequisites();
    return;
  }
  gather(s.lists, v, K, 1, [&](uint32_t) { return uint64_t(n0); },
         [&](uint32_t, uint32_t stage, uint32_t &w, uint32_t &it) {
           const uint32_t o = stage % step;
           w = o % kWarps;
           it = stage / step;
           return o / kWarps == rank;
         },
         p.status);
  const Exceptions x = exceptions_of(s.lists, warp, lane, (stages + step - 1) / step);
  const uint16_t *px[NT];
  uint32_t live = 0;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const uint32_t m = 8 * nt + g;
    live |= m < p.M ? 1u << nt : 0u;
    px[nt] = p.x + uint64_t(m) * K + 16 * t;
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
      if (x.walk) stage_product<NT, 1, false, true>(tot, f[i], v, q, live, ~0u, 0, second, x, it, n0 + g, K, k0, lane);
      else stage_product<NT, 1, false, false>(tot, f[i], v, q, live, ~0u, 0, second, x, it, n0 + g, K, k0, lane);
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
  for (uint32_t o = tid; o < kOut; o += kThreads) {
    const uint32_t row = o % kRows, m = o / kRows;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) sum += s.lists.sums(w, NT)[m * kRedTok + row];
    s.part[o] = sum;
  }
  if (csize > 1) cluster_sync(); else __syncthreads();
  wait_prerequisites();  // t
  for (uint32_t o = tid + rank * kThreads; o < kOut; o += kThreads * csize) {
    const uint32_t row = o % kRows, m = o / kRows;
    if (m >= p.M) continue;
    float sum = s.part[o];
    if (csize > 1) {
      sum = 0.0f;
      for (uint32_t c = 0; c < csize; c++) sum += cluster_load(&s.part[o], c);
    }
    const int32_t ad = p.adapter[m];
    if (ad >= 0 && ad < int32_t(p.L)) {
      const uint4 *pb = reinterpret_cast<const uint4 *>(p.b + (uint64_t(ad) * p.N + n0 + row) * p.r);
      const float4 *pt = reinterpret_cast<const float4 *>(p.t + uint64_t(m) * p.r);
      float add = 0.0f;
      for (uint32_t j = 0; j < p.r / 8; j++) {
        const uint4 b = pb[j];
        const float4 t0 = pt[2 * j], t1 = pt[2 * j + 1];
        add += t0.x * bf16_lo(b.x) + t0.y * bf16_hi(b.x) + t0.z * bf16_lo(b.y) + t0.w * bf16_hi(b.y);
        add += t1.x * bf16_lo(b.z) + t1.y * bf16_hi(b.z) + t1.z * bf16_lo(b.w) + t1.w * bf16_hi(b.w);
      }
      sum += add;
    }
    p.y[uint64_t(m) * p.N + n0 + row] = sum;
  }
  if (csize > 1) cluster_sync();  // the others' sums are read until here
}

// ---------------------------------------------------------------------------
// More tokens: Y = the adapters' part (zero for a token without one).  A warp
// takes 16 rows of N and 32 tokens; t enters as three bf16 numbers.
__global__ void __launch_bounds__(kThreads) k12_adapter_expand(const __grid_constant__ Params p) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t n0 = (blockIdx.y * kWarps + warp) * kRows, m0 = 32 * blockIdx.x;
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
  if (L == 0 || L > 0x7FFFFFFFu || r == 0 || r % 8 != 0 || r > kMaxRank || K > (1u << 20) || N / 128 > 65535 || M > 0x7FFFFFFFu)
    return WC_ERR_INVALID_ARG;
  if (work_bytes < wc12_linear_adapters_work_bytes(M, r)) return WC_ERR_CAPACITY;
  const int sms = wc12l::device_sms();
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
  k12_adapter_shrink<<<dim3((M + 7) / 8, (r + 15) / 16, M < 8 ? M : 8), kThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return WC_ERR_CUDA;
  if (M <= kFewTokens) {
    // CTAs that split K: until every SM has two, while each warp has a stage
    const uint32_t groups = N / kRows, stages = (K + kStage - 1) / kStage;
    uint32_t csize = 1;
    while (csize < 8 && groups * csize < 2u * uint32_t(sms) && stages >= 2 * csize * kWarps) csize *= 2;
    auto kernel = M <= 8 ? k12_few_adapters<1> : k12_few_adapters<2>;
    if (launch(kernel, dim3(groups * csize), csize, s, true, p, csize) != cudaSuccess) return WC_ERR_CUDA;
    return WC_OK;
  }
  if (launch(k12_adapter_expand, dim3((M + 31) / 32, N / (kRows * kWarps)), 1, s, true, p) != cudaSuccess)
    return WC_ERR_CUDA;
  return wc12l::linear(d_w, w_bytes, d_plan, plan_bytes, N, K, d_x, M, d_y, true, d_status, stream);
}
