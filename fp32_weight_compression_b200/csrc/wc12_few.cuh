// wc12_few.cuh -- products of Split12 weights with a few tokens, shared by the
// linear layer with adapters (k_split12_adapters.cu) and the mixture-of-
// experts layer (k_split12_moe.cu).
//
// A few tokens make the product memory-bound: each weight crosses HBM once
// (12 bits) and meets 8 to 32 tokens.  So the weights go from global memory
// to registers, are expanded there straight into the A fragments of
// mma.sync.m16n8k16 (16 weight rows x 16 values of K) and never touch shared
// memory: the tensor-memory path of k_split12_linear.cu writes every expanded
// tile to shared memory and back, which costs more than the product itself
// at these sizes.
//
// Fragment layout.  Lane 4 g + t of a warp holds rows g and g + 8 of the 16-
// row group.  The order of K inside a product is free as long as both
// operands agree, so lane t takes 16 consecutive values of K at a time: 8
// bytes of indices and 16 low bytes a row, one 8-byte and one 16-byte load,
// and the same 16 values of its token (column g) as 32 bytes.  Four products
// (steps) use them up, 4 values of a lane's row each.  A stage is 128 values
// of K: two such pieces (c = 0, 1; values 64 c + 16 t ..).
//
// Exceptions.  Their high bytes replace the codebook's in the fragments,
// before the product, so that an output has the exact weights and nothing
// else in its sum.  The CTA gathers the exceptions of its rows from the
// container's per-chunk lists while its first weights are in flight, one
// list a warp, sorted by the iteration in which the warp meets them.  A warp
// with more exceptions than its list holds looks each lane's values up in
// the container's sorted lists instead (slow, and right for any container).
#pragma once

#include <cstdint>

#include "wc.h"
#include "wc_split12.cuh"

namespace wc12f {

using wc12::kChunk;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kRows = 16;    // weight rows of a CTA's group
constexpr uint32_t kStage = 128;  // values of K of a stage
constexpr uint32_t kListCap = 512;
constexpr uint32_t kBins = 128;
constexpr uint32_t kItBits = 13;  // iterations of a warp: at most 8192
constexpr uint32_t kRedTok = 20;  // floats a token's 16 partial sums take (padded: no bank conflicts)

__device__ __forceinline__ void report(int32_t *status, int32_t code) { atomicCAS(status, 0, code); }

// a value rounded to nearest bf16 (its bits), or two of them as a word
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// programmatic dependent launch: let the next kernel of the stream start its
// prologue; wait for the one before (all of it, its writes visible)
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float at `p`'s place in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), b;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(b) : "memory");
  return v;
}

// A container opened for a rows x K matrix.
struct View {
  const uint8_t *idx, *lo;  // planes
  const uint64_t *exc_off;
  const uint16_t *exc_pos;
  const uint8_t *exc_val;
  uint64_t n, ne;
  uint4 book;
};

// The planes' places depend on the number of values only.
__device__ __forceinline__ void open_planes(View &v, const uint8_t *w, uint64_t n) {
  const wc12::Lay L = wc12::lay(n, 0);
  v.n = n;
  v.idx = w + L.off_idx;
  v.lo = w + L.off_lo;
}
// Checks the header (what wc12_linear checks) and sets the rest.
__device__ __forceinline__ bool open_header(View &v, const uint8_t *w, uint64_t w_bytes) {
  const uint32_t *h32 = reinterpret_cast<const uint32_t *>(w);
  const uint64_t *h64 = reinterpret_cast<const uint64_t *>(w);
  const uint4 q0 = *reinterpret_cast<const uint4 *>(h32);       // magic, version/dtype/K, n
  const uint4 q1 = *reinterpret_cast<const uint4 *>(h32 + 4);   // chunk, nc, ne
  const ulonglong2 q2 = *reinterpret_cast<const ulonglong2 *>(h64 + 4), q3 = *reinterpret_cast<const ulonglong2 *>(h64 + 6);
  v.book = *reinterpret_cast<const uint4 *>(w + wc12::kBookOff);
  v.ne = uint64_t(q1.z) | (uint64_t(q1.w) << 32);
  const uint32_t kk = q0.y >> 24;
  const uint64_t n = uint64_t(q0.z) | (uint64_t(q0.w) << 32);
  if (q0.x != wc12::kMagic || (q0.y & 0xFFFFFFu) != (1u | (1u << 16)) || kk < 1 || kk > 16 || n != v.n || v.ne > n ||
      q1.x != uint32_t(kChunk))
    return false;
  const wc12::Lay L = wc12::lay(n, v.ne);
  v.exc_off = reinterpret_cast<const uint64_t *>(w + wc12::kExcOffOff);
  v.exc_pos = reinterpret_cast<const uint16_t *>(w + L.off_exc);
  v.exc_val = w + L.off_excval;
  return q1.y == uint32_t(L.nc) && q2.x == L.off_idx && q2.y == L.off_lo && q3.x == L.off_exc && q3.y == L.total &&
         L.total <= w_bytes;
}

// ---------------------------------------------------------------------------
// Fragments: a lane's pieces of one stage, [row g or g + 8][c].
struct Frag {
  uint2 i[2][2];
  uint4 l[2][2];
};

__device__ __forceinline__ uint2 load_idx(const uint8_t *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_lo(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// pi, pl: this lane's place in row g of the stage's first piece; K: the row
// length; second: whether the stage has its second piece
__device__ __forceinline__ void load_frag(Frag &f, const uint8_t *pi, const uint8_t *pl, uint32_t K, bool second) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    f.i[h][0] = load_idx(pi + h * (uint64_t(K) * 4));
    f.l[h][0] = load_lo(pl + h * (uint64_t(K) * 8));
  }
  if (second) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      f.i[h][1] = load_idx(pi + h * (uint64_t(K) * 4) + 32);
      f.l[h][1] = load_lo(pl + h * (uint64_t(K) * 8) + 64);
    }
  }
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(s));
  return d;
}

// wc12::expand4 with the selectors of 8 nibbles split beforehand: sel is the
// entry within its half (3 bits), up 1 for entries 8..15, in the low 16 bits
__device__ __forceinline__ uint2 expand4(uint32_t sel, uint32_t up, uint4 book, uint32_t lo4) {
  const uint32_t r0 = prmt(book.x, book.y, sel);
  const uint32_t r1 = prmt(book.z, book.w, sel);
  const uint32_t m = prmt(0x0000FF00u, 0u, up);
  const uint32_t hi4 = (r0 & ~m) | (r1 & m);
  return make_uint2(prmt(lo4, hi4, 0x5140), prmt(lo4, hi4, 0x7362));
}

__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// Exceptions.  An entry: high byte (bits 0-7), row of the group (8-11),
// column of the stage (12-18), iteration of the warp (19-31).
__device__ __forceinline__ uint32_t pack_exc(uint32_t it, uint32_t col, uint32_t row, uint32_t high) {
  return high | (row << 8) | (col << 12) | (it << 19);
}
__device__ __forceinline__ uint32_t exc_step(uint32_t e) {  // the product (0..7) that uses it
  return ((e >> 16) & 4u) | ((e >> 14) & 3u);
}
// puts the entry's high byte into the A words of its step, in its lane
__device__ __forceinline__ void patch(uint32_t *a, uint32_t e, uint32_t lane) {
  const uint32_t owner = ((e >> 8) & 7u) * 4 + ((e >> 16) & 3u);
  if (lane != owner) return;
  const uint32_t word = ((e >> 11) & 1u) | ((e >> 12) & 2u);  // row half, then the pair of the step
  const uint32_t sel = (e >> 12) & 1u ? 0x4210u : 0x3240u;     // the pair's second or first value
#pragma unroll
  for (uint32_t i = 0; i < 4; i++)
    if (word == i) a[i] = prmt(a[i], e, sel);
}

// Shared memory of the gather.
struct Lists {
  uint64_t e0[kThreads];          // a batch of (region, chunk) items: first exception
  uint32_t pre[kThreads + 1];     // exceptions before the item
  uint32_t wsum[kWarps];
  uint32_t cnt[kWarps];           // exceptions of each warp (may pass kListCap)
  uint32_t raw[kWarps][kListCap];
  uint32_t list[kWarps][kListCap];
  uint32_t start[kWarps][kBins + 1];

  // A warp's sums at the end, [token][row], over the lists (which no warp
  // reads any more: a barrier before the first use): 32 tokens of 8 warps.
  __device__ __forceinline__ float *sums(uint32_t warp, int tiles) {
    return reinterpret_cast<float *>(&raw[0][0]) + warp * (8 * kRedTok) * tiles;
  }
};
static_assert(sizeof(Lists::raw) + sizeof(Lists::list) >= sizeof(float) * kWarps * 32 * kRedTok, "sums");

// Gathers the exceptions of `regions` groups of 16 rows (the first at row
// row0(r)) of a rows x K matrix into the warps' lists; own(r, stage, warp,
// it) says which warp of this CTA meets that stage and when (false: none).
// Every thread calls it.
template <class Row0, class Own>
__device__ void gather(Lists &s, const View &v, uint32_t K, uint32_t regions, Row0 row0, Own own, int32_t *status) {
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < kWarps) s.cnt[tid] = 0;
  const uint64_t span = uint64_t(kRows) * K;
  const uint32_t per = uint32_t((span - 1) / kChunk) + 2;  // chunks that 16 rows can touch
  const uint32_t items = v.ne == 0 ? 0u : regions * per;
  for (uint32_t first = 0; first < items; first += kThreads) {
    // an item a thread: its chunk's exceptions
    uint32_t count = 0;
    uint64_t e0 = 0;
    if (first + tid < items) {
      const uint32_t r = (first + tid) / per;
      const uint64_t f0 = row0(r) * K, c = f0 / kChunk + (first + tid) % per;
      if (c * kChunk < f0 + span) {
        e0 = v.exc_off[c];
        const uint64_t e1 = v.exc_off[c + 1];
        if (e0 > e1 || e1 > v.ne || e1 - e0 > kChunk) report(status, WC_ERR_CORRUPT);
        else count = uint32_t(e1 - e0);
      }
    }
    uint32_t incl = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= uint32_t(o)) incl += u;
    }
    if (lane == 31) s.wsum[warp] = incl;
    __syncthreads();  // also: the batch before is done with e0 and pre
    uint32_t base = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) base += uint32_t(w) < warp ? s.wsum[w] : 0u;
    s.e0[tid] = e0;
    s.pre[tid + 1] = base + incl;
    if (tid == 0) s.pre[0] = 0;
    __syncthreads();
    const uint32_t total = s.pre[kThreads];
    for (uint32_t i = tid; i < total; i += kThreads) {
      uint32_t lo = 0, hi = kThreads - 1;  // the last item with pre <= i
      while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) >> 1;
        if (s.pre[mid] <= i) lo = mid; else hi = mid - 1;
      }
      const uint32_t item = first + lo, r = item / per;
      const uint64_t e = s.e0[lo] + (i - s.pre[lo]);
      const uint64_t f0 = row0(r) * K, c = f0 / kChunk + item % per;
      const uint64_t len = v.n - c * kChunk < kChunk ? v.n - c * kChunk : kChunk;
      const uint32_t pos = v.exc_pos[e];
      if (pos >= len) {
        report(status, WC_ERR_CORRUPT);
        continue;
      }
      const uint64_t f = c * kChunk + pos;
      if (f < f0 || f - f0 >= span) continue;
      const uint32_t lf = uint32_t(f - f0), row = lf / K, col = lf - row * K;  // 16 K < 2^32
      uint32_t w, it;
      if (!own(r, col / kStage, w, it)) continue;
      const uint32_t slot = atomicAdd(&s.cnt[w], 1u);
      if (slot < kListCap) s.raw[w][slot] = pack_exc(it, col % kStage, row, v.exc_val[e]);
    }
    __syncthreads();
  }
  __syncthreads();
}

// Sorts the warp's list by iteration (bins of 2^shift iterations, its of them
// in all).  Returns the number of exceptions, or ~0 if they passed the list.
__device__ __forceinline__ uint32_t sort_list(Lists &s, uint32_t warp, uint32_t lane, uint32_t its, uint32_t &shift) {
  const uint32_t cnt = s.cnt[warp];
  shift = 0;
  while (((its - 1) >> shift) >= kBins) shift++;
  if (cnt == 0) return 0;
  if (cnt > kListCap) return ~0u;
  uint32_t *start = s.start[warp];
  for (uint32_t i = lane; i <= kBins; i += 32) start[i] = 0;
  __syncwarp();
  for (uint32_t i = lane; i < cnt; i += 32) atomicAdd(&start[s.raw[warp][i] >> (19 + shift)], 1u);
  __syncwarp();
  uint32_t run = 0;
  for (uint32_t b0 = 0; b0 < kBins; b0 += 32) {  // counts -> ends
    uint32_t incl = start[b0 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= uint32_t(o)) incl += u;
    }
    __syncwarp();
    start[b0 + lane] = run + incl;
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) start[kBins] = cnt;
  __syncwarp();
  // place from each bin's end backwards: the ends become the starts
  for (uint32_t i = lane; i < cnt; i += 32) {
    const uint32_t e = s.raw[warp][i];
    s.list[warp][atomicSub(&start[e >> (19 + shift)], 1u) - 1] = e;
  }
  __syncwarp();
  return cnt;
}

// A warp's exceptions: its sorted list, or (walk) the container's.
struct Exceptions {
  const uint32_t *list, *start;
  uint32_t cnt, shift;
  bool walk;
};
__device__ __forceinline__ Exceptions exceptions_of(Lists &s, uint32_t warp, uint32_t lane, uint32_t its) {
  Exceptions x;
  x.list = s.list[warp];
  x.start = s.start[warp];
  x.cnt = sort_list(s, warp, lane, its, x.shift);
  x.walk = x.cnt == ~0u;
  return x;
}

// The high bytes of a lane's 16 values at flat position f (a multiple of 16)
// that are exceptions, from the container's lists: a mask and the first
// one's place.
__device__ __forceinline__ uint32_t walk_mask(const View &v, uint64_t f, uint64_t &first) {
  const uint64_t c = f / kChunk;
  const uint32_t pos = uint32_t(f % kChunk);
  uint64_t lo = v.exc_off[c], hi = v.exc_off[c + 1];
  if (lo > hi || hi > v.ne) hi = lo = 0;
  const uint64_t end = hi;
  while (lo < hi) {
    const uint64_t mid = (lo + hi) >> 1;
    if (v.exc_pos[mid] < pos) lo = mid + 1; else hi = mid;
  }
  first = lo;
  uint32_t m = 0;
  for (uint64_t e = lo; e < end && e < lo + 16; e++) {
    const uint32_t p = v.exc_pos[e];
    if (p < pos || p >= pos + 16) break;
    m |= 1u << (p - pos);
  }
  return m;
}

// The exceptions that one stage of a warp meets, as its steps need them.
struct StageExc {
  uint32_t e;      // this lane's entry of the list's page
  uint32_t hit;    // lanes whose entries are of this stage
  uint32_t steps;  // steps that have one (bit 8: more than a page holds)
  uint32_t b0, b1;
};
__device__ __forceinline__ StageExc stage_exceptions(const Exceptions &x, uint32_t it, uint32_t lane) {
  StageExc q;
  q.hit = q.steps = q.e = 0;
  q.b0 = q.b1 = 0;
  if (x.cnt == 0) return q;
  q.b0 = x.start[it >> x.shift];
  q.b1 = x.start[(it >> x.shift) + 1];
  if (q.b0 == q.b1) return q;
  const bool in = q.b0 + lane < q.b1;
  q.e = in ? x.list[q.b0 + lane] : 0u;
  const bool mine = in && (q.e >> 19) == it;
  q.hit = __ballot_sync(0xffffffffu, mine);
  q.steps = __reduce_or_sync(0xffffffffu, mine ? 1u << exc_step(q.e) : 0u);
  if (q.b1 - q.b0 > 32) q.steps = 0x1FFu;
  return q;
}

// One stage: the fragments' 16 rows x 128 (or 64) values times 8 NT tokens.
// px: this lane's place in its tokens' rows (column g of each group of 8
// tokens), at the stage's first piece; live: bit nt set where that token
// exists, tiles where the group of 8 has any.  kMask: a token that does not
// exist here is not given the stage's sums (its zeros times an infinite
// weight would be NaN); without it such tokens' sums are the caller's to
// drop.  kParts planes of the tokens' values, `plane` values apart, are
// summed (a value held as the sum of kParts bf16 numbers).  The products of
// a stage are added up in the tensor cores, stages in fp32 registers: the
// tensor cores cut off what their accumulator cannot hold, so that long
// sums there drift toward zero.
template <int NT, int kParts, bool kMask, bool kWalk>
__device__ __forceinline__ void stage_product(float tot[NT][4], const Frag &f, const View &v, const uint16_t *const *px,
                                              uint32_t live, uint32_t tiles, uint64_t plane, bool second, const Exceptions &x,
                                              uint32_t it, uint64_t row_g, uint32_t K, uint32_t k0, uint32_t lane) {
  float d[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.0f;
  StageExc q{};
  if (!kWalk) q = stage_exceptions(x, it, lane);
#pragma unroll
  for (int c = 0; c < 2; c++) {
    if (c == 1 && !second) break;
    uint4 xv[NT][kParts];
    uint32_t wm[2] = {0u, 0u};
    uint64_t we[2] = {0u, 0u};
    if (kWalk) {
      const uint64_t f0 = row_g * K + k0 + 64 * c + 16 * (lane & 3u);
      wm[0] = walk_mask(v, f0, we[0]);
      wm[1] = walk_mask(v, f0 + uint64_t(K) * 8, we[1]);
    }
#pragma unroll
    for (int s = 0; s < 4; s++) {
      if ((s & 1) == 0) {  // 8 values of each token, for two steps
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
          for (int part = 0; part < kParts; part++) {
            xv[nt][part] = make_uint4(0u, 0u, 0u, 0u);
            if ((live >> nt) & 1u)
              xv[nt][part] = *reinterpret_cast<const uint4 *>(px[nt] + part * plane + 64 * c + 4 * s);
          }
      }
      uint32_t a[4];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const uint32_t qw = s < 2 ? f.i[h][c].x : f.i[h][c].y;
        const uint32_t sel = (qw & 0x77777777u) >> (16 * (s & 1)), up = ((qw >> 3) & 0x11111111u) >> (16 * (s & 1));
        const uint32_t lw = s == 0 ? f.l[h][c].x : s == 1 ? f.l[h][c].y : s == 2 ? f.l[h][c].z : f.l[h][c].w;
        const uint2 e = expand4(sel, up, v.book, lw);
        a[h] = e.x;
        a[h + 2] = e.y;
      }
      if (kWalk) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            if ((wm[h] >> (4 * s + i)) & 1u) {
              const uint32_t high = v.exc_val[we[h] + __popc(wm[h] & ((1u << (4 * s + i)) - 1u))];
              a[h + 2 * (i >> 1)] = prmt(a[h + 2 * (i >> 1)], high, i & 1 ? 0x4210u : 0x3240u);
            }
      } else if ((q.steps >> (4 * c + s)) & 1u) {
        if (q.steps & 0x100u) {
          for (uint32_t i = q.b0; i < q.b1; i++) {
            const uint32_t e = x.list[i];
            if ((e >> 19) == it && exc_step(e) == uint32_t(4 * c + s)) patch(a, e, lane);
          }
        } else {
          for (uint32_t rest = q.hit; rest; rest &= rest - 1) {
            const uint32_t e = __shfl_sync(0xffffffffu, q.e, __ffs(rest) - 1);
            if (exc_step(e) == uint32_t(4 * c + s)) patch(a, e, lane);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        if (NT > 1 && !((tiles >> nt) & 1u)) continue;
#pragma unroll
        for (int part = 0; part < kParts; part++) {
          const uint4 xq = xv[nt][part];
          mma(d[nt], a, s & 1 ? xq.z : xq.x, s & 1 ? xq.w : xq.y);
        }
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    // d[nt][i] is of column 2 t + (i & 1), whose token lane 8 t + 4 (i & 1)
    // knows
    const uint32_t in = kMask ? __ballot_sync(0xffffffffu, (live >> nt) & 1u) >> (8 * (lane & 3u)) : 0u;
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (!kMask || ((in >> (4 * (i & 1))) & 1u)) tot[nt][i] += d[nt][i];
  }
}

// A warp's sums into its part of the reduction buffer, [token][row].
template <int NT>
__device__ __forceinline__ void put_sums(float *red, const float tot[NT][4], uint32_t lane) {
  const uint32_t g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    float *p = red + (8 * nt + 2 * t) * kRedTok + g;
    p[0] = tot[nt][0];
    p[kRedTok] = tot[nt][1];
    p[8] = tot[nt][2];
    p[kRedTok + 8] = tot[nt][3];
  }
}

// Launches a kernel of kThreads threads in clusters of `cluster` CTAs along
// x; dependent: it may start while the kernel before it in the stream runs
// (it waits with wait_prerequisites).
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, uint32_t cluster, cudaStream_t s, bool dependent, Args... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(kThreads);
  c.stream = s;
  cudaLaunchAttribute at[2];
  uint32_t n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    n++;
  }
  if (dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    n++;
  }
  c.attrs = at;
  c.numAttrs = n;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace wc12f
