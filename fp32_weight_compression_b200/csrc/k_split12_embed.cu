// k_split12_embed.cu -- embedding lookup out of a table held as a Split12
// container (wc12_embed, include/wc_split12.h): out[t] = scale * table[ids[t]],
// the rows asked for read at 12 bits a value, the rest of the table never.
//
// A CTA expands one row: a thread takes pieces of 8 values (4 index bytes, 8
// low bytes, 16 or 32 bytes out), four of them at once, so that a row is on
// its way as a whole.  The row's exceptions are a short run in the list of
// each 65,536-value chunk that it touches (usually one): their offsets are
// read beside the row's bytes, the list's entries before the row is written,
// and the exceptions' values go over it after a barrier.  A long list is
// narrowed down first.  Times of graph replays: latency bounds few rows (id,
// row, write: three round trips; 2.3 us for 1 or 61 rows of 1024, of which the
// launch is most), issue and memory many: 8192 rows of 4096, 118 MB, in 23 us,
// 5.1 TB/s, with 76 % of the issue slots taken (36 us
// with one piece of a row in flight and the exceptions read after it; 34 with
// two pieces; six CTAs an SM, 25.5 without the bound on registers).
#include <cstdint>

#include "wc12_few.cuh"

namespace wc12e {

using namespace wc12f;

constexpr uint32_t kMaxThreads = 256;
constexpr uint32_t kBatch = 4;  // pieces of 8 values of a thread at once
// A row's columns are counted with 32 bits, up to one round of the CTA's pieces
// (8 kBatch kMaxThreads values) past its end.
constexpr uint32_t kMaxColumns = 1u << 31;

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
__global__ void __launch_bounds__(kMaxThreads, 6) k12_embed(const __grid_constant__ Params p) {
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
  // the first chunk's list: its offsets now, this thread's entry once they
  // have come
  uint64_t ch = f0 / kChunk, e0 = v.exc_off[ch], e1 = v.exc_off[ch + 1];
  uint32_t pos = 0, high = 0;
  auto entry = [&] {
    if (v.ne > 0 && e0 + tid < e1 && e1 <= v.ne) {
      pos = v.exc_pos[e0 + tid];
      high = v.exc_val[e0 + tid];
    }
  };
  if (8 * tid >= K) entry();  // no piece of the row
  for (uint32_t c0 = 8 * tid; c0 < K; c0 += 8 * kBatch * nthr) {
    uint32_t q[kBatch];
    uint2 l[kBatch];
#pragma unroll
    for (uint32_t i = 0; i < kBatch; i++) {
      const uint32_t c = c0 + 8 * i * nthr < K ? c0 + 8 * i * nthr : c0;
      q[i] = *reinterpret_cast<const uint32_t *>(idx + c / 2);
      l[i] = *reinterpret_cast<const uint2 *>(lo + c);
    }
    if (c0 == 8 * tid) entry();
#pragma unroll
    for (uint32_t i = 0; i < kBatch; i++) {
      const uint32_t c = c0 + 8 * i * nthr;
      if (c >= K) break;
      uint32_t hi[2];
      if (v.runs) high8<true>(hi, q[i], v.book, v.base4);
      else high8<false>(hi, q[i], v.book, v.base4);
      const uint2 a = join4(l[i].x, hi[0]), b = join4(l[i].y, hi[1]);
      const uint32_t w[4] = {a.x, a.y, b.x, b.y};
      store8<kWide>(row, c, w, p.scale);
    }
  }
  if (v.ne == 0) return;
  __syncthreads();
  const uint64_t ch0 = ch;
  for (; ch * kChunk < f1; ch++) {
    if (ch > ch0) {
      e0 = e1;
      e1 = v.exc_off[ch + 1];
    }
    if (e0 > e1 || e1 > v.ne) {
      if (tid == 0) report(p.status, WC_ERR_CORRUPT);
      continue;
    }
    // positions of the chunk that belong to the row: [b, e)
    const uint32_t b = f0 > ch * kChunk ? uint32_t(f0 - ch * kChunk) : 0u;
    const uint64_t left = f1 - ch * kChunk;
    const uint32_t e = left < kChunk ? uint32_t(left) : uint32_t(kChunk);
    const uint64_t len = v.n - ch * kChunk < kChunk ? v.n - ch * kChunk : kChunk;
    uint64_t from = e0;
    // a long list: drop what lies before the row, a block-wide probe at a
    // time (positions ascend)
    while (e1 - from > 4ull * nthr) {
      const uint64_t step = (e1 - from + nthr - 1) / nthr;
      const uint64_t at = from + step * (tid + 1) - 1;  // the last of this thread's part
      const uint32_t before = __syncthreads_count(at < e1 && v.exc_pos[at] < b);
      if (before == 0) break;
      from += step * before;
    }
    for (uint64_t i = from + tid; i < e1; i += nthr) {
      const bool early = ch == ch0 && i == e0 + tid;  // read beside the row
      const uint32_t at = early ? pos : v.exc_pos[i];
      if (at >= e) {
        // past the row: nothing further on in a valid container
        if (at >= len) report(p.status, WC_ERR_CORRUPT);
        break;
      }
      if (at < b) continue;
      const uint32_t c = uint32_t(ch * kChunk + at - f0);
      const uint32_t bits = ((early ? high : v.exc_val[i]) << 8) | lo[c];
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
  if (V == 0 || K == 0 || K % 8 != 0 || K > wc12e::kMaxColumns || V > wc12::kMaxN / K || w_bytes < 96) return WC_ERR_INVALID_ARG;
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
  uint32_t thr = (K / (8 * wc12e::kBatch) + 31) / 32 * 32;
  if (T <= 256) thr = (K / 8 + 31) / 32 * 32;  // few rows: a piece a thread
  if (thr < 32) thr = 32;
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
