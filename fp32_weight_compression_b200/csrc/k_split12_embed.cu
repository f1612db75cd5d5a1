// k_split12_embed.cu -- embedding lookup out of a table held as a Split12
// container (wc12_embed, include/wc_split12.h): out[t] = scale * table[ids[t]],
// the rows asked for read at 12 bits a value, the rest of the table never.
//
// A CTA expands one row: a thread takes 8 values at a time (4 index bytes, 8
// low bytes, 16 or 32 bytes out).  The row's exceptions are a short run in
// the list of each 65,536-value chunk that it touches (usually one); the CTA
// looks through the list, or first narrows it down when it is long, and
// writes the exceptions' values over the row after a barrier.
#include <cstdint>

#include "wc12_few.cuh"

namespace wc12e {

using namespace wc12f;

constexpr uint32_t kMaxThreads = 256;

struct Params {
  const uint8_t *w;
  uint64_t w_bytes;
  const void *ids;
  void *out;
  uint64_t V;
  uint32_t K;
  float scale;
  int32_t *status;
};

// two bf16 values (a word) times scale
template <bool kWide>
__device__ __forceinline__ void store8(void *row, uint32_t col, const uint32_t *w, float scale) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(w[i] << 16) * scale;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * scale;
  }
  if (kWide) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(row) + col);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint4 o = make_uint4(w[0], w[1], w[2], w[3]);  // scale 1: the bits themselves
    if (scale != 1.0f)
      o = make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row) + col) = o;
  }
}

template <class Id, bool kWide>
__global__ void __launch_bounds__(kMaxThreads) k12_embed(const __grid_constant__ Params p) {
  const uint32_t tid = threadIdx.x, K = p.K, nthr = blockDim.x;
  const Id id = static_cast<const Id *>(p.ids)[blockIdx.x];
  View v;
  open_planes(v, p.w, p.V * K);
  if (!open_header(v, p.w, p.w_bytes)) {
    if (blockIdx.x == 0 && tid == 0) report(p.status, WC_ERR_CORRUPT);
    return;
  }
  void *row = kWide ? static_cast<void *>(static_cast<float *>(p.out) + uint64_t(blockIdx.x) * K)
                    : static_cast<void *>(static_cast<uint16_t *>(p.out) + uint64_t(blockIdx.x) * K);
  if (id < 0 || uint64_t(id) >= p.V) {
    if (tid == 0) report(p.status, WC_ERR_INVALID_ARG);
    const uint32_t zero[4] = {0u, 0u, 0u, 0u};
    for (uint32_t c = 8 * tid; c < K; c += 8 * nthr) store8<kWide>(row, c, zero, 1.0f);
    return;
  }
  const uint64_t f0 = uint64_t(id) * K, f1 = f0 + K;
  const uint8_t *idx = v.idx + f0 / 2, *lo = v.lo + f0;
#pragma unroll 2
  for (uint32_t c = 8 * tid; c < K; c += 8 * nthr) {
    const uint32_t q = *reinterpret_cast<const uint32_t *>(idx + c / 2);
    const uint2 l = *reinterpret_cast<const uint2 *>(lo + c);
    uint32_t hi[2];
    high8<false>(hi, q, v.book, 0);
    const uint2 e0 = join4(l.x, hi[0]), e1 = join4(l.y, hi[1]);
    const uint32_t w[4] = {e0.x, e0.y, e1.x, e1.y};
    store8<kWide>(row, c, w, p.scale);
  }
  if (v.ne == 0) return;
  __syncthreads();
  for (uint64_t ch = f0 / kChunk; ch * kChunk < f1; ch++) {
    uint64_t e0 = v.exc_off[ch], e1 = v.exc_off[ch + 1];
    if (e0 > e1 || e1 > v.ne) {
      if (tid == 0) report(p.status, WC_ERR_CORRUPT);
      continue;
    }
    // positions of the chunk that belong to the row: [b, e)
    const uint32_t b = f0 > ch * kChunk ? uint32_t(f0 - ch * kChunk) : 0u;
    const uint64_t left = f1 - ch * kChunk;
    const uint32_t e = left < kChunk ? uint32_t(left) : uint32_t(kChunk);
    // a long list: drop what lies before the row, a block-wide probe at a
    // time (positions ascend)
    while (e1 - e0 > 4ull * nthr) {
      const uint64_t step = (e1 - e0 + nthr - 1) / nthr;
      const uint64_t at = e0 + step * (tid + 1) - 1;  // the last of this thread's part
      const uint32_t before = __syncthreads_count(at < e1 && v.exc_pos[at] < b);
      if (before == 0) break;
      e0 += step * before;
    }
    for (uint64_t i = e0 + tid; i < e1; i += nthr) {
      const uint32_t pos = v.exc_pos[i];
      if (pos >= e) {
        // past the row: nothing further on in a valid container
        const uint64_t len = v.n - ch * kChunk < kChunk ? v.n - ch * kChunk : kChunk;
        if (pos >= len) report(p.status, WC_ERR_CORRUPT);
        break;
      }
      if (pos < b) continue;
      const uint32_t c = uint32_t(ch * kChunk + pos - f0);
      const uint32_t bits = (uint32_t(v.exc_val[i]) << 8) | lo[c];
      const float f = __uint_as_float(bits << 16) * p.scale;
      if (kWide) static_cast<float *>(row)[c] = f;
      else static_cast<uint16_t *>(row)[c] = uint16_t(p.scale == 1.0f ? bits : bf16_bits(f));
    }
  }
}

}  // namespace wc12e

extern "C" int32_t wc12_embed(const void *d_w, uint64_t w_bytes, uint64_t V, uint32_t K, const void *d_ids,
                              uint32_t id_bytes, uint64_t T, float scale, void *d_out, int32_t out_dtype,
                              int32_t *d_status, void *stream) {
  auto aligned = [](const void *q, uintptr_t a) { return (reinterpret_cast<uintptr_t>(q) & (a - 1)) == 0; };
  if (d_w == nullptr || d_status == nullptr || !aligned(d_w, 16) || !aligned(d_status, 4)) return WC_ERR_INVALID_ARG;
  if (V == 0 || K == 0 || K % 8 != 0 || V > wc12::kMaxN / K || w_bytes < 96) return WC_ERR_INVALID_ARG;
  if ((id_bytes != 4 && id_bytes != 8) || (out_dtype != WC_BF16 && out_dtype != WC_FP32)) return WC_ERR_INVALID_ARG;
  const uint64_t n = V * K;
  const wc12::Lay L = wc12::lay(n, 0);
  if (w_bytes < L.off_lo + n) return WC_ERR_INVALID_ARG;
  if (T > 0x7FFFFFFFu) return WC_ERR_INVALID_ARG;
  if (T == 0) return WC_OK;
  if (d_ids == nullptr || d_out == nullptr || !aligned(d_ids, id_bytes) || !aligned(d_out, 16)) return WC_ERR_INVALID_ARG;
  wc12e::Params p;
  p.w = static_cast<const uint8_t *>(d_w);
  p.w_bytes = w_bytes;
  p.ids = d_ids;
  p.out = d_out;
  p.V = V;
  p.K = K;
  p.scale = scale;
  p.status = d_status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t thr = (K / 8 + 31) / 32 * 32;
  if (thr > wc12e::kMaxThreads) thr = wc12e::kMaxThreads;
  const bool wide = out_dtype == WC_FP32;
  if (id_bytes == 8) {
    if (wide) wc12e::k12_embed<int64_t, true><<<unsigned(T), thr, 0, s>>>(p);
    else wc12e::k12_embed<int64_t, false><<<unsigned(T), thr, 0, s>>>(p);
  } else {
    if (wide) wc12e::k12_embed<int32_t, true><<<unsigned(T), thr, 0, s>>>(p);
    else wc12e::k12_embed<int32_t, false><<<unsigned(T), thr, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? WC_OK : WC_ERR_CUDA;
}
