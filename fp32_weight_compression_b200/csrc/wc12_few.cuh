// wc12_few.cuh -- products of Split12 weights with a few tokens, shared by the
// linear layer with adapters (k_split12_adapters.cu) and the mixture-of-
// experts layer (k_split12_moe.cu).
//
// A few tokens make the product memory-bound: each weight crosses HBM once
// (12 bits) and meets 8 or 16 tokens.  So the weights are expanded in
// registers straight into the A fragments of mma.sync.m16n8k16 (16 weight
// rows x 16 values of K): the tensor-memory path of k_split12_linear.cu writes
// every expanded tile to shared memory and back, which costs more than the
// product itself at these sizes.
//
// Fragment layout.  Lane 4 g + t of a warp holds rows g and g + 8 of a group
// of 16 rows.  The order of K inside a product is free as long as both
// operands agree, so lane t takes 16 consecutive values of K of a unit of 64:
// 8 bytes of indices and 16 low bytes a row, and the same 16 values of its
// token (column g) as 32 bytes.  Four products (steps) use them up, 4 values
// of a lane's row each.
//
// Loads.  A stage is two subtiles of 64 rows x 64 values of K, 16 rows of
// each the work of a warp: two successive ranges of K, or two matrices' rows
// with the same values of K.  One warp brings the subtiles' planes with TMA
// and the tokens' values into a ring of kDepth stages, four warps expand and
// multiply.  No barrier of the CTA in the loop: a "full" and an "empty"
// mbarrier a stage.  The planes' boxes are stored as rows of 32 and 64 bytes,
// so that the lanes that read together read 128 bytes in a row.
//
// What bounds it: the expansion's instructions (see high8) and, in short rows,
// what comes before the first stage and after the last (header, exceptions,
// joining the parts of K: 4 to 6 us), not the memory.  14336 x 4096, 16
// tokens, adapters of rank 16 (98.6 MB), replayed from a graph: 32.5 us, 3.0
// TB/s, where the boxes alone stream in 17, and the kernel without products and
// exceptions takes 23.  Ways that were left: loads into registers (57 us: the
// tokens' values came from L2 at the moment of use); copies by cp.async, a
// lane its own pieces (56: twice the product's instructions); eight warps a
// CTA with a subtile each (64: half the independent products a lane has,
// tests for exceptions between them); equal parts of the stages for
// every CTA, joined through the workspace (40: the join costs 3 to 5 us, a
// cluster's 1.5).
//
// Every wait is bounded and gives up once another thread has; the kernel then
// reports WC_ERR_TIMEOUT, waits for its copies in flight and ends.
//
// Exceptions.  Their high bytes replace the codebook's in the fragments,
// before the product, so that an output has the exact weights and nothing
// else in its sum.  A warp takes the exceptions of its 16 rows from the
// container's per-chunk lists, 64 entries a load, while its first weights are
// in flight (or the ones of the rows before), and gives those of its part of
// K to the lanes that will hold their values, each of which has a short
// queue.  The products take a lane's next entry in passing, without a branch.
// More than a queue holds: the queues are filled again on the way, or for a part
// of the row at a time, or each lane's values are looked up in the container's
// sorted lists (see stage_product_slow).
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda.h>

#include "wc.h"
#include "wc_split12.cuh"

namespace wc {
// Identity of the CUDA context current on this thread, 0 if none
// (csrc/wc_noalloc.cu).
unsigned long long current_context_id();
}  // namespace wc

namespace wc12l {
// k_split12_linear.cu: a 2-D tensor map; the device's SMs (0 on failure)
bool make_map(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t rows,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle sw,
              CUtensorMapL2promotion l2);
int device_sms();
}  // namespace wc12l

namespace wc12f {

using wc12::kChunk;

constexpr int kWarps = 4;                   // that multiply
constexpr int kConsumers = 32 * kWarps;
constexpr int kThreads = kConsumers + 32;   // and one that loads
constexpr uint32_t kRows = 16;       // weight rows of a group
constexpr uint32_t kSubRows = 64;    // of a subtile
constexpr uint32_t kUnit = 64;       // values of K of a subtile
constexpr uint32_t kMaxK = 1 << 16;  // a group's rows touch at most 17 chunks
constexpr uint32_t kQueue = 16;      // exceptions a lane keeps
constexpr uint32_t kRedTok = 18;     // floats a token's 16 sums take (padded: few bank conflicts)
constexpr uint32_t kMaxDepth = 4;    // stages of the ring, at most
constexpr uint32_t kSpinLimit = 1u << 24;

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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float at `p`'s place in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), b;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(b));
  return v;
}

// A container opened for a rows x K matrix.
struct View {
  const uint8_t *w;
  const uint8_t *idx, *lo;  // planes
  const uint64_t *exc_off;
  const uint16_t *exc_pos;
  const uint8_t *exc_val;
  uint64_t n, ne;
  uint4 book;
  // the codebook is base .. base + 7 and the same with the sign bit, as it is
  // for weights spread alike to both sides of zero: base in each byte
  bool runs;
  uint32_t base4;
};

// The planes' places, and the start of the exceptions' lists, depend on the
// number of values only.
__device__ __forceinline__ void open_planes(View &v, const uint8_t *w, uint64_t n) {
  const wc12::Lay L = wc12::lay(n, 0);
  v.w = w;
  v.n = n;
  v.exc_off = reinterpret_cast<const uint64_t *>(w + wc12::kExcOffOff);
  v.exc_pos = reinterpret_cast<const uint16_t *>(w + L.off_exc);
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
  v.exc_val = w + L.off_excval;
  v.base4 = (v.book.x & 0xFFu) * 0x01010101u;
  v.runs = kk == 16 && (v.book.x & 0x80u) == 0 && (v.book.w >> 31) != 0 && v.book.x == v.base4 + 0x03020100u &&
           v.book.y == v.base4 + 0x07060504u && v.book.z == (v.book.x | 0x80808080u) && v.book.w == (v.book.y | 0x80808080u);
  return q1.y == uint32_t(L.nc) && q2.x == L.off_idx && q2.y == L.off_lo && q3.x == L.off_exc && q3.y == L.total &&
         L.total <= w_bytes;
}

// Whether a high byte of infinities and NaN (and of values from 2^127 on) is in
// the codebook.
__device__ __forceinline__ bool book_wild(uint4 book) {
  auto in = [](uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); };
  return (in(book.x) | in(book.y) | in(book.z) | in(book.w)) != 0;
}
// two bf16 values, those that are not finite as zeros
__device__ __forceinline__ uint32_t finite2(uint32_t w) { return w & ~__vcmpeq2(w & 0x7F807F80u, 0x7F807F80u); }

// ---------------------------------------------------------------------------
// The exceptions' lists of a container whose header was found to be right,
// again: code that runs rarely gets its few values from there, and the
// products keep none of them in registers.
__device__ __forceinline__ void open_lists(View &v, const uint8_t *w, uint64_t n) {
  open_planes(v, w, n);
  v.ne = *reinterpret_cast<const uint64_t *>(w + 24);
  v.exc_val = w + wc12::lay(n, v.ne).off_excval;
}

// ---------------------------------------------------------------------------
// The ring.
constexpr uint32_t kIdxBytes = kSubRows * kUnit / 2, kLoBytes = kSubRows * kUnit;
constexpr uint32_t kSubBytes = kIdxBytes + kLoBytes;
// The tokens' values of a stage, from 2 kSubBytes on, as the lanes read them:
// from the start of the stage's values to this lane's token's (the first of
// each 8), its first and second 8 of the 16 values of a unit.  Copied a row
// at a time: kXRow bytes a token (so that 8 lanes read from all banks), the
// second unit's values behind the first's.  By TMA: a box of 8 kTiles rows of
// 128 bytes a unit, 128-byte swizzle.
struct XAt {
  uint32_t first, second;
};
constexpr uint32_t kXRow = 272;
__device__ __forceinline__ XAt x_rows(uint32_t lane) {
  const uint32_t at = (lane >> 2) * kXRow + 32 * (lane & 3);
  return {at, at + 16};
}
__device__ __forceinline__ XAt x_boxes(uint32_t lane) {
  const uint32_t g = lane >> 2, t = lane & 3;
  return {128 * g + (((2 * t) ^ g) << 4), 128 * g + (((2 * t + 1) ^ g) << 4)};
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint4 shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 shared8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// A warp's own part of shared memory: its lanes' queues, then its sums.
struct Queues {
  uint32_t count[32];
  uint32_t until, end;  // refilled queues: the unit that they go up to, the last one's end
  uint16_t entry[kQueue][32];
  uint8_t high[kQueue][32];
};
constexpr uint32_t own_words(uint32_t tokens) {
  return tokens * kRedTok * 4 > sizeof(Queues) ? tokens * kRedTok : uint32_t(sizeof(Queues)) / 4;
}

__device__ __forceinline__ uint32_t shared4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t shared2(uint32_t a) {
  uint32_t v;
  asm volatile("{\n\t.reg .b16 h;\n\tld.shared.b16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}" : "=r"(v) : "r"(a));
  return v;
}

struct Bars {
  uint64_t full[kMaxDepth], empty[kMaxDepth];
  // The multiplying warps have asked for their first exceptions: the loading
  // warp fills the ring beyond its first stage after that, since those few
  // bytes would otherwise wait behind 20 MB of other CTAs' stages, and the
  // products for them (14336 x 4096, 16 tokens: 34.1 -> 32.7 us; 32 tokens
  // through 128 experts 202 -> 200).
  uint64_t asked;
  int failed;
};
// by one thread, before a barrier of the CTA
__device__ __forceinline__ void bars_init(Bars &b) {
  for (uint32_t i = 0; i < kMaxDepth; i++) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&b.full[i])) : "memory");
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&b.empty[i])), "n"(kWarps) : "memory");
  }
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&b.asked)), "n"(kWarps) : "memory");
  b.failed = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
// A place in the ring: stage s is in slot s % kDepth, its turn s / kDepth.
template <uint32_t kDepth>
struct Turn {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kDepth) {
      slot = 0;
      parity ^= 1;
    }
  }
};
// whether the phase of the given parity came to its end, for the whole warp
__device__ __forceinline__ bool bar_wait(Bars &b, uint64_t *bar, uint32_t parity, bool heed_failure, int32_t *status) {
  const uint32_t a = smem_u32(bar);
  auto look = [&] {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, r != 0);
  };
  if (look()) return true;
  for (uint32_t i = 0; i < kSpinLimit; i++) {
    if (look()) return true;
    if (heed_failure && __any_sync(0xffffffffu, *static_cast<volatile int *>(&b.failed) != 0)) return false;
  }
  report(status, WC_ERR_TIMEOUT);
  *static_cast<volatile int *>(&b.failed) = 1;
  return false;
}
// the loading warp, before it ends: no copy may be in flight then.  turn: the
// place after the last of `count` stages
template <uint32_t kDepth>
__device__ __forceinline__ void finish_copies(Bars &b, Turn<kDepth> turn, uint32_t count, int32_t *status) {
  // back to the first of the last kDepth stages (or of all)
  const uint32_t n = count < kDepth ? count : kDepth;
  for (uint32_t i = 0; i < n; i++) {
    if (turn.slot == 0) {
      turn.slot = kDepth;
      turn.parity ^= 1;
    }
    turn.slot--;
  }
  for (uint32_t i = 0; i < n; i++, turn.next()) bar_wait(b, &b.full[turn.slot], turn.parity, false, status);
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// a box of 64 rows of a plane, from byte x of row y on, into this CTA
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, uint32_t x, uint32_t y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void load_row(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *src, uint32_t bytes) {  // a multiple of 16
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// A container's planes as TMA sees them.
struct Planes {
  CUtensorMap idx, lo;
};
__device__ __forceinline__ void load_subtile(uint32_t dst, const Planes &m, uint32_t k, uint32_t row, uint64_t *bar) {
  load_box(dst, &m.idx, k / 2, row, bar);
  load_box(dst + kIdxBytes, &m.lo, k, row, bar);
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(s));
  return d;
}

// The high bytes of 8 values, hi[0] the first 4's, from their 8 nibbles.  The
// expansion is what bounds the products: byte permutes, shifts and logic
// issue every other cycle, 64 a cycle and SM, against 29 values a cycle and SM
// that come from memory.  By the codebook in registers (kRuns false) 8 values
// take 13 of them and 4 to join the low bytes; where the codebook is two runs
// the nibble's low bits and sign are put together instead: 7 and 4 (the
// shift to the left and the sums go to the multiply-add pipe).
template <bool kRuns>
__device__ __forceinline__ void high8(uint32_t *hi, uint32_t q, uint4 book, uint32_t base4) {
  if (kRuns) {
    const uint32_t even = ((q & 0x07070707u) + base4) | ((q << 4) & 0x80808080u);
    const uint32_t odd = (((q >> 4) & 0x07070707u) + base4) | (q & 0x80808080u);
    hi[0] = prmt(even, odd, 0x5140);
    hi[1] = prmt(even, odd, 0x7362);
  } else {
    const uint32_t sel = q & 0x77777777u, up = (q >> 3) & 0x11111111u;  // the entry within its half; which half
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint32_t si = sel >> (16 * i), m = prmt(0x0000FF00u, 0u, up >> (16 * i));
      hi[i] = (prmt(book.x, book.y, si) & ~m) | (prmt(book.z, book.w, si) & m);
    }
  }
}
__device__ __forceinline__ uint2 join4(uint32_t lo4, uint32_t hi4) {
  return make_uint2(prmt(lo4, hi4, 0x5140), prmt(lo4, hi4, 0x7362));
}
__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same with nothing to add to
__device__ __forceinline__ void mma_first(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// ---------------------------------------------------------------------------
// Exceptions.  A lane's entry: which subtile, as the warp meets them (bits
// 5-15), which of the lane's 8 sets of 4 values there (2 step + row half;
// bits 2-4), which value of the set (0-1).
constexpr uint32_t kNever = 0x7FFFFFFFu;  // the set of no entry
constexpr uint32_t kTooMany = 0x40000000u;
// the byte `high` (in bits 16-23) into place `entry` & 3 of four
__device__ __forceinline__ uint32_t put_high(uint32_t hi4, uint32_t entry) {
  const uint32_t i = 4 * (entry & 3u);
  return prmt(hi4, entry, (0x3210u & ~(0xFu << i)) | (6u << i));
}

// The container's exceptions around a group of 16 rows, in flight: lane j
// has the offset of the j-th chunk that the rows touch (`chunks` of them,
// and the end), then two entries of the first 64.
struct Window {
  uint64_t off;
  uint32_t pos, val;
};
__device__ __forceinline__ uint32_t window_chunks(uint64_t row0, uint32_t K) {
  return uint32_t((row0 * K + uint64_t(kRows) * K - 1) / kChunk - row0 * K / kChunk) + 1;
}
__device__ __forceinline__ void window_offsets(Window &w, const uint64_t *exc_off, uint64_t row0, uint32_t K,
                                               uint32_t lane) {
  const uint32_t chunks = window_chunks(row0, K);
  w.off = exc_off[row0 * K / kChunk + (lane < chunks ? lane : chunks)];
}
__device__ __forceinline__ void window_pairs(const View &v, uint64_t e, uint64_t e1, uint32_t &pos, uint32_t &val) {
  // two entries from an even place on; the lists are padded to 16 bytes
  pos = val = 0;
  if (e < e1) {
    pos = *reinterpret_cast<const uint32_t *>(v.exc_pos + e);
    val = *reinterpret_cast<const uint16_t *>(v.exc_val + e);
  }
}
// offsets have come: the first 64 entries
__device__ __forceinline__ void window_entries(Window &w, const View &v, uint32_t lane) {
  const uint64_t e0 = __shfl_sync(0xffffffffu, w.off, 0), e1 = __shfl_sync(0xffffffffu, w.off, 31);
  window_pairs(v, (e0 & ~uint64_t(1)) + 2 * lane, e1 <= v.ne ? e1 : 0, w.pos, w.val);
}

// A lane's exceptions, ascending: the next kOut of its queue are out, each as
// its set (entry >> 2, kNever for none) and the entry with its high byte in
// bits 16-23.  more: the n-entry queue of some lane of the warp has others, from
// i on.  short_of (the same for the warp): the queues are too short for the
// exceptions of all units, which are looked up, or the queues are filled again
// on the way.  The experts' down product, whose values come in two parts, also
// sets it where weights may be infinite: see stage_product_slow.
constexpr int kOut = 4;
struct Exceptions {
  Queues *q;
  uint32_t n, i;
  uint32_t set[kOut], entry[kOut];
  bool more, short_of;
};
// Entries have come: keeps those of the group's units [u0, u1), as of
// subtile mul * unit + plus.  Returns whether a value among this lane's entries
// may not be finite.
__device__ __forceinline__ bool window_keep(Exceptions &x, const Window &w, const View &v, uint64_t row0, uint32_t K,
                                            uint32_t u0, uint32_t u1, uint32_t mul, uint32_t plus, uint32_t lane, int32_t *status) {
  const uint64_t e0 = __shfl_sync(0xffffffffu, w.off, 0), e1 = __shfl_sync(0xffffffffu, w.off, 31);
  const uint64_t before = __shfl_up_sync(0xffffffffu, w.off, 1);
  if (__any_sync(0xffffffffu, (lane > 0 && w.off < before) || w.off > v.ne)) {
    if (lane == 0) report(status, WC_ERR_CORRUPT);
    return false;
  }
  if (e1 - e0 > 1u << 14) {  // too many to go through them
    x.q->count[lane] = kTooMany;
    return false;
  }
  bool wild = false;
  const uint64_t f0 = row0 * K, c0 = f0 / kChunk;
  const uint32_t chunks = window_chunks(row0, K), count = uint32_t(e1 - e0), skew = uint32_t(e0 & 1);
  const uint32_t rel = uint32_t(w.off - e0);                              // the lane's chunk's first entry
  const uint32_t begin = uint32_t(f0 - c0 * kChunk), span = kRows * K;    // of the rows, from the first chunk on
  const uint64_t left = v.n - c0 * kChunk;                                // values from the first chunk on
  const float inv = 1.0f / float(K);
  uint32_t pos = w.pos, val = w.val, pos2 = 0, val2 = 0;
  for (uint32_t base = 0; base < count + skew; base += 64, pos = pos2, val = val2) {  // entry base - skew + 2 lane + i
    if (base + 64 < count + skew) window_pairs(v, e0 - skew + base + 64 + 2 * lane, e1, pos2, val2);
#pragma unroll
    for (uint32_t i = 0; i < 2; i++) {
      const uint32_t e = base + 2 * lane + i - skew;  // wraps for the one before the first
      uint32_t c = 0;
      for (uint32_t j = 1; j < chunks; j++) c += e >= __shfl_sync(0xffffffffu, rel, j) ? 1u : 0u;
      const uint32_t f = c * uint32_t(kChunk) + ((pos >> (16 * i)) & 0xFFFFu);
      bool in = e < count;
      if (in && f >= left) report(status, WC_ERR_CORRUPT);
      in = in && f >= begin && f - begin < span;
      const uint32_t lf = in ? f - begin : 0u;
      // lf / K: (lf + 1/2) / K is at least 2^-17 away from a whole number, and
      // off by less than 2^-19
      const uint32_t row = uint32_t((float(lf) + 0.5f) * inv), col = lf - row * K, u = col / kUnit;
      in = in && u >= u0 && u < u1;
      if (in) {
        const uint32_t owner = (row & 7u) * 4 + ((col >> 4) & 3u), at = atomicAdd(&x.q->count[owner], 1u);
        if (at < kQueue) {
          x.q->entry[at][owner] = uint16_t((mul * u + plus) << 5 | ((col >> 2) & 3u) << 3 | (row >> 3) << 2 | (col & 3u));
          x.q->high[at][owner] = uint8_t(val >> (8 * i));
        }
        wild = wild || ((val >> (8 * i)) & 0x7Fu) == 0x7Fu;
      }
    }
  }
  return wild;
}
// the queue's next entry
__device__ __forceinline__ void exceptions_pull(Exceptions &x, uint32_t &set, uint32_t &entry, uint32_t lane) {
  set = kNever;
  entry = 0;
  if (x.i < x.n) {
    const uint32_t e = x.q->entry[x.i][lane];
    set = e >> 2;
    entry = e | uint32_t(x.q->high[x.i][lane]) << 16;
    x.i++;
  }
}
__device__ __forceinline__ void exceptions_reset(Exceptions &x, uint32_t lane) {
  __syncwarp();
  x.q->count[lane] = 0;
  x.n = x.i = 0;
#pragma unroll
  for (int i = 0; i < kOut; i++) {
    x.set[i] = kNever;
    x.entry[i] = 0;
  }
  x.more = x.short_of = false;
  __syncwarp();
}
// a queue's n entries ascending
__device__ __forceinline__ void queue_sort(Queues *q, uint32_t n, uint32_t lane) {
#pragma unroll 1
  for (uint32_t i = 1; i < n; i++) {  // a few at most: by insertion
    const uint16_t entry = q->entry[i][lane];
    const uint8_t high = q->high[i][lane];
    uint32_t j = i;
#pragma unroll 1
    for (; j > 0 && q->entry[j - 1][lane] > entry; j--) {
      q->entry[j][lane] = q->entry[j - 1][lane];
      q->high[j][lane] = q->high[j - 1][lane];
    }
    q->entry[j][lane] = entry;
    q->high[j][lane] = high;
  }
}
// all windows' entries of units [u0, u1) are in the queues
__device__ __forceinline__ void exceptions_ready(Exceptions &x, uint32_t u0, uint32_t u1, uint32_t lane) {
  __syncwarp();
  x.n = x.q->count[lane];
  x.short_of = __any_sync(0xffffffffu, x.n > kQueue);
  if (x.short_of) {
    x.n = 0;
    x.q->until = u0;  // the same by all lanes
    x.q->end = u1;
  }
  queue_sort(x.q, x.n, lane);
#pragma unroll
  for (int i = 0; i < kOut; i++) exceptions_pull(x, x.set[i], x.entry[i], lane);
  x.more = __any_sync(0xffffffffu, x.i < x.n);
}
// Fills the queues with the exceptions of the units from u on, of the group of
// 16 rows from row0 on: to the last unit, or of as many (an even number) as
// the queues hold.  until: the unit that they go up to; its highest bit: not
// even two units' fit, so that these have to be looked up.
static __device__ __noinline__ void queues_refill(Queues *q, const uint8_t *w12, uint64_t n, uint64_t row0, uint32_t K, uint32_t u,
                                                  int32_t *status) {
  const uint32_t lane = threadIdx.x & 31;
  View v;
  open_lists(v, w12, n);
  Exceptions x;
  x.q = q;
  uint32_t span = q->end - u, mine, dense = 0;
  for (;;) {
    __syncwarp();
    q->count[lane] = 0;
    __syncwarp();
    Window w;
    window_offsets(w, v.exc_off, row0, K, lane);
    window_entries(w, v, lane);
    window_keep(x, w, v, row0, K, u, u + span, 1, 0, lane, status);
    __syncwarp();
    mine = q->count[lane];
    const uint32_t most = __reduce_max_sync(0xffffffffu, mine);
    if (most <= kQueue) break;
    if (span <= 2 || most >= kTooMany) {
      mine = 0;
      dense = 1u << 31;
      break;
    }
    // as many as should fit, fewer than now
    const uint32_t fewer = span * (kQueue - 4) / most & ~1u, least = (span - 1) & ~1u;
    span = fewer < 2 ? 2 : fewer < least ? fewer : least;
  }
  q->count[lane] = mine;
  queue_sort(q, mine, lane);
  q->until = (u + span) | dense;
  __syncwarp();
}
// How many entries a lane has at most in the stage whose first subtile is
// key: 0, 1, 2, or 3 for more (or where the queues are too short)
__device__ __forceinline__ uint32_t exceptions_most(const Exceptions &x, uint32_t key) {
  if (x.short_of) return 3;
  if (!__any_sync(0xffffffffu, x.set[0] - 8 * key < 16)) return 0;
  if (!__any_sync(0xffffffffu, x.set[1] - 8 * key < 16)) return 1;
  return __any_sync(0xffffffffu, x.set[2] - 8 * key < 16) ? 3 : 2;
}
// the stage is done: its entries go, the next ones move up
__device__ __forceinline__ void exceptions_pass(Exceptions &x, uint32_t key, uint32_t most, uint32_t lane) {
  for (uint32_t j = 0; j < most; j++) {
    const bool gone = x.set[0] - 8 * key < 16;
#pragma unroll
    for (int i = 0; i + 1 < kOut; i++) {
      x.set[i] = gone ? x.set[i + 1] : x.set[i];
      x.entry[i] = gone ? x.entry[i + 1] : x.entry[i];
    }
    if (gone) x.set[kOut - 1] = kNever;
    if (x.more && x.set[kOut - 1] == kNever) exceptions_pull(x, x.set[kOut - 1], x.entry[kOut - 1], lane);
    if (most == 3 && __any_sync(0xffffffffu, x.set[0] - 8 * key < 16)) j = 0;
  }
}
// The container's exceptions among 4 values, the first at flat position f,
// onto their high bytes.
__device__ __forceinline__ uint32_t exceptions_walk(uint32_t hi4, const uint8_t *w12, uint64_t n, uint64_t f) {
  View v;
  open_lists(v, w12, n);
  const uint64_t c = f / kChunk;
  const uint32_t pos = uint32_t(f % kChunk);
  uint64_t lo = v.exc_off[c], hi = v.exc_off[c + 1];
  if (lo > hi || hi > v.ne) hi = lo = 0;
  const uint64_t end = hi;
  while (lo < hi) {
    const uint64_t mid = (lo + hi) >> 1;
    if (v.exc_pos[mid] < pos) lo = mid + 1; else hi = mid;
  }
  for (uint64_t e = lo; e < end && e < lo + 4; e++) {
    const uint32_t p = v.exc_pos[e];
    if (p < pos || p >= pos + 4) break;
    const uint32_t i = 4 * (p - pos);
    hi4 = prmt(hi4, v.exc_val[e], (0x3210u & ~(0xFu << i)) | (4u << i));
  }
  return hi4;
}
// A lane's 16 values of two rows of a subtile, as stored.
struct Piece {
  uint2 idx[2];
  uint4 lo[2];
};
// sub: the subtile's start, group: which 16 rows
__device__ __forceinline__ void read_piece(Piece &f, uint32_t sub, uint32_t group, uint32_t lane) {
  const uint32_t g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    f.idx[h] = shared8(sub + (group * kRows + g + 8 * h) * 32 + 8 * t);
    f.lo[h] = shared16(sub + kIdxBytes + (group * kRows + g + 8 * h) * 64 + 16 * t);
  }
}
template <int kTiles, int kParts>
__device__ __forceinline__ void read_values(uint4 xv[kTiles][kParts], uint32_t at, uint32_t tile_bytes) {
#pragma unroll
  for (int i = 0; i < kTiles; i++)
#pragma unroll
    for (int part = 0; part < kParts; part++) xv[i][part] = shared16(at + (part * kTiles + i) * tile_bytes);
}
// What a warp needs to know of a stage.
struct StageAt {
  uint32_t slot, group;   // the stage's start; which 16 rows of the subtiles
  uint32_t xs, xs2;       // the tokens' values for either subtile
  uint32_t tile_bytes;    // from 8 tokens to the next 8, then to the next part
  bool only;              // the first subtile only
  uint32_t key;           // the first subtile's
  uint32_t unit0, unit1;  // which units of their rows the subtiles are,
  uint64_t row0, row1;    // and the group's first row (for the container's lists)
};

// A warp's 16 rows of both subtiles of a stage times 8 kTiles tokens, added to
// tot0 and tot1; kShare: both take the values at xs.  A token's value is held
// as the sum of kParts bf16 numbers.  The four products of a subtile are
// added up in the tensor cores, subtiles in fp32 registers: the tensor cores
// cut off what their accumulator cannot hold, so that long sums there drift
// toward zero.  Columns without a token hold sums that the caller drops.
// kMost: exceptions that a lane may have (two in one stage in a hundred, where
// the containers have one in 2,500 values; four warps share a stage, so that
// code which is slow one time in a hundred is felt).
template <int kTiles, int kParts, bool kShare, bool kRuns, int kMost>
__device__ __forceinline__ void stage_product(float tot0[kTiles][4], float tot1[kTiles][4], const StageAt &at, XAt xat, const View &v,
                                              const Exceptions &x, uint32_t lane) {
  const uint32_t set1 = x.set[0] - 8 * at.key, set2 = x.set[1] - 8 * at.key, i1 = 4 * (x.entry[0] & 3u);
  const uint32_t sel1 = (0x3210u & ~(0xFu << i1)) | (6u << i1);
  Piece f[2];
  read_piece(f[0], at.slot, at.group, lane);
  read_piece(f[1], at.slot + kSubBytes, at.group, lane);
  float d[2][kTiles][4];
  uint4 xv[2][kTiles][kParts];
#pragma unroll
  for (int w = 0; w < 2; w++) {  // 8 values of a row: two steps
    read_values<kTiles, kParts>(xv[0], at.xs + (w ? xat.second : xat.first), at.tile_bytes);
    if (!kShare) read_values<kTiles, kParts>(xv[1], at.xs2 + (w ? xat.second : xat.first), at.tile_bytes);
#pragma unroll
    for (int sub = 0; sub < 2; sub++) {
      uint32_t a[2][4];
#pragma unroll
      for (int r = 0; r < 2; r++) {
        uint32_t hi[2];
        high8<kRuns>(hi, w ? f[sub].idx[r].y : f[sub].idx[r].x, v.book, v.base4);
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const uint32_t set = 8 * sub + 2 * (2 * w + i) + r;
          if (kMost > 0 && set1 == set) hi[i] = prmt(hi[i], x.entry[0], sel1);
          if (kMost > 1 && set2 == set) hi[i] = put_high(hi[i], x.entry[1]);
          const uint2 e = join4(w ? i ? f[sub].lo[r].w : f[sub].lo[r].z : i ? f[sub].lo[r].y : f[sub].lo[r].x, hi[i]);
          a[i][r] = e.x;
          a[i][r + 2] = e.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int tile = 0; tile < kTiles; tile++)
#pragma unroll
          for (int part = 0; part < kParts; part++) {
            const uint4 q = xv[kShare ? 0 : sub][tile][part];
            if (w == 0 && i == 0 && part == 0) mma_first(d[sub][tile], a[i], q.x, q.y);
            else mma(d[sub][tile], a[i], i ? q.z : q.x, i ? q.w : q.y);
          }
    }
  }
#pragma unroll
  for (int i = 0; i < kTiles; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      tot0[i][j] += d[0][i][j];
      if (!at.only) tot1[i][j] += d[1][i][j];
    }
}

// The same for a stage with more exceptions than two a lane, a step at a time.
// Where the queues are too short for all units, each value is looked up in the
// container's lists: a warp that does so takes 200 us for rows of 4096 values,
// however few of its lanes need it.  With kRefill the queues are filled again
// here instead, from the lists, for as many units as they hold (14336 x 4096,
// 8 tokens, an exception in 200 values: 227 -> 67 us, one in 100: 412 -> 99).
// The experts' kernels do without: the compiler keeps more of their loops'
// values elsewhere with it (5 tokens, large experts 53.4 -> 56.3 us, 16 tokens
// 63 -> 68).  They fill the queues for a part of a row at a time instead, outside
// the loop over the part's stages.
// Weights that are not finite meet a value's first part only: times a second
// part, which is zero or of the other sign as often as not, an infinite one
// would turn the sum into NaN.
template <int kTiles, int kParts, bool kShare, bool kRefill>
__device__ __forceinline__ void stage_product_slow(float tot0[kTiles][4], float tot1[kTiles][4], const StageAt &at, XAt xat,
                                                   const View &v, Exceptions &x, uint32_t K, uint32_t lane, int32_t *status) {
  const uint32_t g = lane >> 2, t = lane & 3;
  bool dense = !kRefill && x.short_of;
  if (kRefill && x.short_of) {
    if (at.unit0 >= (x.q->until & 0x7FFFFFFFu)) {
      queues_refill(x.q, v.w, v.n, at.row0, K, at.unit0, status);
      x.n = x.q->count[lane];
      x.i = 0;
#pragma unroll
      for (int i = 0; i < kOut; i++) exceptions_pull(x, x.set[i], x.entry[i], lane);
      x.more = __any_sync(0xffffffffu, x.i < x.n);
    }
    dense = x.q->until >> 31;
  }
#pragma unroll 1
  for (uint32_t step = 0; step < (at.only ? 4 : 8); step++) {
    const uint32_t sub = step >> 2, s = step & 3, from = at.slot + sub * kSubBytes;
    uint32_t a[4], low[4];
#pragma unroll
    for (uint32_t r = 0; r < 2; r++) {
      const uint32_t row = at.group * kRows + g + 8 * r;
      const uint32_t q = shared2(from + row * 32 + 8 * t + 2 * s), lw = shared4(from + kIdxBytes + row * 64 + 16 * t + 4 * s);
      uint32_t hi[2];
      high8<false>(hi, q, v.book, 0);
      uint32_t hi4 = hi[0];
      if (dense) {
        const uint64_t at_row = (sub ? at.row1 : at.row0) + g + 8 * r;
        hi4 = exceptions_walk(hi4, v.w, v.n, at_row * K + kUnit * (sub ? at.unit1 : at.unit0) + 16 * t + 4 * s);
      } else {
        const uint32_t set = 8 * (at.key + sub) + 2 * s + r;
#pragma unroll
        for (int i = 0; i < kOut; i++)
          if (x.set[i] == set) hi4 = put_high(hi4, x.entry[i]);
        for (uint32_t i = x.i; i < x.n && (x.q->entry[i][lane] >> 2) <= set; i++)
          if ((x.q->entry[i][lane] >> 2) == set)
            hi4 = put_high(hi4, x.q->entry[i][lane] | uint32_t(x.q->high[i][lane]) << 16);
      }
      const uint2 e = join4(lw, hi4);
      a[r] = e.x;
      a[r + 2] = e.y;
    }
#pragma unroll
    for (int i = 0; i < kTiles; i++) {
      float d[4] = {};
#pragma unroll
      for (int part = 0; part < kParts; part++) {
        if (part == 1) {
#pragma unroll
          for (int j = 0; j < 4; j++) low[j] = finite2(a[j]);
        }
        const uint2 q = shared8((!kShare && sub ? at.xs2 : at.xs) + (s & 2 ? xat.second : xat.first) + 8 * (s & 1) +
                                (part * kTiles + i) * at.tile_bytes);
        mma(d, part ? low : a, q.x, q.y);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        tot0[i][j] += sub ? 0.0f : d[j];
        tot1[i][j] += sub ? d[j] : 0.0f;
      }
    }
  }
}

// The one of these that the stage needs.
template <int kTiles, int kParts, bool kShare, bool kRefill>
__device__ __forceinline__ void stage(float tot0[kTiles][4], float tot1[kTiles][4], const StageAt &at, XAt xat, const View &v,
                                      Exceptions &x, uint32_t most, uint32_t K, uint32_t lane, int32_t *status) {
  if (most == 3) {
    stage_product_slow<kTiles, kParts, kShare, kRefill>(tot0, tot1, at, xat, v, x, K, lane, status);
  } else if (v.runs) {
    if (most == 0) stage_product<kTiles, kParts, kShare, true, 0>(tot0, tot1, at, xat, v, x, lane);
    else if (most == 1) stage_product<kTiles, kParts, kShare, true, 1>(tot0, tot1, at, xat, v, x, lane);
    else stage_product<kTiles, kParts, kShare, true, 2>(tot0, tot1, at, xat, v, x, lane);
  } else {
    if (most < 2) stage_product<kTiles, kParts, kShare, false, 1>(tot0, tot1, at, xat, v, x, lane);
    else stage_product<kTiles, kParts, kShare, false, 2>(tot0, tot1, at, xat, v, x, lane);
  }
  if (most > 0) exceptions_pass(x, at.key, most, lane);
}

// A warp's sums of a group, [token][row] with kRedTok floats a token.
template <int kTiles>
__device__ __forceinline__ void put_sums(float *red, const float tot[kTiles][4], uint32_t lane) {
  const uint32_t g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < kTiles; i++) {
    float *p = red + (8 * i + 2 * t) * kRedTok + g;
    p[0] = tot[i][0];
    p[kRedTok] = tot[i][1];
    p[8] = tot[i][2];
    p[kRedTok + 8] = tot[i][3];
  }
}

// The tensor maps of a rows x K container's planes: boxes of 64 rows x 64
// values (the planes' 256-byte L2 promotion is what lets such narrow boxes
// stream at the memory's rate).
inline bool make_planes(Planes &m, const void *w, uint64_t rows, uint32_t K) {
  const wc12::Lay L = wc12::lay(rows * K, 0);
  const uint8_t *p = static_cast<const uint8_t *>(w);
  return wc12l::make_map(&m.idx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p + L.off_idx, K / 2, rows, K / 2, kUnit / 2, kSubRows,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) &&
         wc12l::make_map(&m.lo, CU_TENSOR_MAP_DATA_TYPE_UINT8, p + L.off_lo, K, rows, K, kUnit, kSubRows,
                         CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// What a device's set-up gave (0: failed), once per device, and again in a
// context created afresh (the kernels' attributes must be set again then).
class DeviceSetup {
 public:
  template <class F>
  int get(F setup) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu_);
    const unsigned long long ctx = wc::current_context_id();
    if (value_[dev] == 0 || ctx == 0 || ctx_[dev] != ctx) {
      value_[dev] = setup();
      ctx_[dev] = wc::current_context_id();  // the set-up made the device's context current
    }
    return value_[dev];
  }

 private:
  std::mutex mu_;
  int value_[64] = {};
  unsigned long long ctx_[64] = {};
};

// Lets the next kernel's CTAs onto the SMs where this one's run: an SM keeps
// one division of its memory into L1 and shared memory while it has any CTA,
// so that a kernel which needs little shared memory would shut out one that
// needs most of it (4 to 10 us late for half of its CTAs).
template <class Kernel>
bool share_sm(Kernel kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) == cudaSuccess;
}

// Launches a kernel in clusters of `cluster` CTAs along x; dependent: it may start while the kernel before it in the stream runs
// (it waits with wait_prerequisites).
template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, uint32_t block, uint32_t cluster, uint32_t smem, cudaStream_t s, bool dependent, Args... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
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

// What a call returns after a CUDA error, which it has reported then: the next
// call's check of its own launches must not find it again.
inline int32_t cuda_failed() {
  cudaGetLastError();
  return WC_ERR_CUDA;
}

}  // namespace wc12f
