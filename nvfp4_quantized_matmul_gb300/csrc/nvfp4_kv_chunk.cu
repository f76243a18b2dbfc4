// Attention over the 8-bit paged key/value cache for chunks of many tokens
// (nvfp4_kv_attention): both products on tcgen05, accumulators in TMEM.
//
// The formulas are those of nvfp4_kv_attention.cu. A CTA takes NQ blocks of
// 128 query rows (token, head of the group) of one key/value head and walks
// the visible tiles of 128 keys:
//   S = Q K^T   kind::f8f6f4: a query row, scaled by a power of two, is the
//               sum of an E4M3 term and one (bf16) or two (f16) E5M2 terms,
//               each one product with the key codes as they lie in the
//               cache, whose pages are the swizzled operand; no key is
//               converted. The sum is exact for queries down to 2^-13 of the
//               row's largest, and within 2^-21 (bf16) or 2^-24 (f16) of it
//               below that: further terms in E4M3 would share the first
//               one's smallest step of 2^-9 and end at 2^-17
//   P = 2^(t - m + 7) in f16, written over S: products with f32's 10-bit form
//               would take twice the time. A key lighter than 2^-21 of the
//               heaviest has fewer than 11 bits, none below 2^-32: that is
//               what it is off by at most, 2^-15 in all of 2^17 such keys
//   O += P V    kind::f16: P from TMEM, values converted to f16 (exactly)
// Bound by the tensor cores where a chunk is long: 2048 tokens at 14000 keys
// (32 / 16 heads of 128, bf16) take 353 us, 1427 TFLOP/s, 75% of the measured
// bf16 rate; a prompt of 8192 (32 / 4 heads) 419 us, 69%; six prompts of 100
// to 2500 tokens with 256 channels, f16, 196 us, 38% (three query terms, and
// queries and results of a block of rows last as long as four tiles). Times
// here are those of captured graphs.
//
// Roles: a warpgroup per 128 rows for the softmax (a thread is a row, so
// maxima and sums need no exchange), four warps that convert values, one that
// copies (with 256 channels two), one that issues the products. With 256
// channels there is one block of rows, whose softmax both warpgroups do, half
// of the keys and channels each: the two threads of a row exchange the tile's
// maximum. TMEM has room for one buffer of scores beside the weights and sums
// of both blocks of rows: a warpgroup takes its scores into registers as soon
// as it has passed on its weights, so the buffer is free again for the other
// block's scores, and the products of tile k + 1 are done while the softmax of
// tile k is under way.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 (the
// weights stay below f16's largest value until then), which after the first
// tiles is rare. The list of (rows, tile) pairs of all sequences and heads is
// cut into equal contiguous runs, one a CTA, in which a block of rows counts
// kItemCost tiles more than it has (its queries and results); rows cut by a
// run's end are joined by whichever of their CTAs arrives last, in a fixed
// order.
#include <atomic>

#include "nvfp4_kv.cuh"
#include "nvfp4_pipe.cuh"

namespace nvfp4 {
namespace {

using namespace kv;
using namespace pipe;

__device__ int g_chunk_error = 0;  // first error code recorded by a bounded wait

constexpr int kKeys = 128;       // keys of a tile
constexpr int kPanel = 64;       // tokens of a panel of converted values: rows of 128 bytes
constexpr float kPUp = 7.0f;     // the weights are held times 2^7
constexpr float kSlack = 8.0f;   // growth of a maximum that is left to the weights
// Beyond this a tile's scores are subtracted from one another before the values' exponents are added to them (as the
// streaming kernel always does): the sum of both, and of what the weights are held up by, would be rounded by more than the
// weights are to f16. Up to it the three go into the exponential's multiply-add, which takes no instruction more.
constexpr float kFar = 4096.0f;
constexpr int kThreads = 512;    // two softmax warpgroups, the converters, copies and products
// Units (see Walk) of a run at least, for blocks of rows of so many units: shorter runs use more SMs, but the last CTA of
// a block joins a result of each, which takes it about half as long as a tile. The sum is least at sqrt(units / 2).
// 40 tokens at 600 keys, 16 / 8 heads: 20 us with 2, 31 with 8, 22 so; 8 tokens at 14000, 32 / 4 heads: 63, 39 and 42 us.
__device__ __forceinline__ int min_run(int units) { return max((int)sqrtf(0.5f * (float)units), 2); }
// Cost of a block of rows, in tiles: its queries and results. A prompt of 8192 tokens takes 444, 414, 415 and 421 us with 3,
// 4, 5 and 6; 6 prompts with 256 channels 190, 189, 188 and 195.
constexpr int kItemCost = 5;
constexpr int kMeta = 4;         // tiles whose scales are kept

struct ChunkArgs {
  KvCache c;
  KvBatch b;
  KvAttention a;
  Waits waits;
  int few;         // sequences of up to so many rows are the other kernel's
  float* ws;       // partial results, two a CTA
  unsigned* done;  // [CTAs] arrivals at the rows that start in a CTA and go on after it; zero between calls
};

template <int D, int TERMS>
struct Shape {
  static constexpr int NQ = D == 256 ? 1 : 2;              // blocks of 128 rows
  static constexpr int kRows = 128 * NQ;
  static constexpr int W = D < 128 ? D : 128;              // bytes of an operand row
  static constexpr int kPanels = D / W;
  static constexpr int kQTerm = 128 * D;
  static constexpr int kQ = NQ * TERMS * kQTerm;
  static constexpr int kK = kKeys * D;
  static constexpr int kKStages = D == 256 && TERMS == 3 ? 1 : 2;
  static constexpr int kRaw = kPanel * D;                  // codes of a panel of values
  static constexpr int kVal = kPanel * D * 2;              // the panel in f16
  static constexpr int kSlots = D == 256 ? 2 : 4;          // panels of each
  static constexpr int kSmem = kQ + kKStages * kK + kSlots * (kRaw + kVal);
  static constexpr uint32_t kPCol = 128, kOCol = 256;      // TMEM: scores from column 0, weights, sums
  static constexpr int64_t kPart = (int64_t)kRows * (D + 3);  // floats of a partial result: sums, maxima, denominators, exponents
};

// A wait of a whole warp, bounded by its number of tries. Each lasts up to 3.75 us (measured: the hardware suspends the
// warp meanwhile), so the limit is about the call's in time. Looking at a clock every 256 tries takes more code, and the
// roles' loops have to share the instruction cache: a prompt of 8192 tokens then takes 463 us, with the count 412.
constexpr uint32_t kNsATry = 3750;
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Tries that a wait is given, and the CTA's flag that one has run out.
struct Limit {
  int* abort_flag;
  uint32_t tries;
  __device__ __forceinline__ void give_up(int code) const {
    if (atomicExch(abort_flag, 1) == 0) atomicCAS(&g_chunk_error, 0, code);
  }
};
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Limit& limit, int code, uint32_t bar2 = 0, uint32_t parity2 = 0) {
  for (uint32_t n = 0; !__all_sync(0xFFFFFFFFu, try_bar(bar, parity) & (bar2 == 0 || try_bar(bar2, parity2))); ++n)
    if (n > limit.tries) {
      limit.give_up(code);
      return false;
    }
  return true;
}

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// K-major operand whose rows of W bytes are swizzled over W bytes: groups of
// eight rows lie 8 W bytes apart.
template <int W>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  constexpr uint64_t mode = W == 128 ? 2 : 4;
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(8 * W >> 4) << 32) | ((uint64_t)1 << 46) | (mode << 61);
}
// f32 accumulator, M = 128, both operands K-major; E4M3 and f16 are format 0 of their kinds, E5M2 is format 1 (of A, bit 7).
constexpr uint32_t kE5m2Queries = 1u << 7;
__host__ __device__ constexpr uint32_t instruction(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

#define NVFP4_OUT8(i) "=f"(r[i]), "=f"(r[i + 1]), "=f"(r[i + 2]), "=f"(r[i + 3]), "=f"(r[i + 4]), "=f"(r[i + 5]), "=f"(r[i + 6]), "=f"(r[i + 7])
#define NVFP4_IN8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of this warp's 32 TMEM lanes
__device__ __forceinline__ void tmem_load(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : NVFP4_OUT8(0), NVFP4_OUT8(8), NVFP4_OUT8(16), NVFP4_OUT8(24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_store(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::NVFP4_IN8(0),
      NVFP4_IN8(8), NVFP4_IN8(16), NVFP4_IN8(24), "r"(addr)
      : "memory");
}
#undef NVFP4_OUT8
#undef NVFP4_IN8
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// 32 bytes, a whole sector where they are aligned.
__device__ __forceinline__ void store32(void* p, const uint32_t (&y)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
                 "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t e4m3x2_of(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}

__device__ __forceinline__ uint32_t e5m2x2_of(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
// An E5M2 code is the upper byte of the f16 it stands for.
__device__ __forceinline__ __half2 half2_of_e5m2x2(uint32_t codes) { return as_half2(__byte_perm(codes, 0, 0x1404)); }

// Two f32 operations an instruction, and the maximum of three.
__device__ __forceinline__ float2 fma2(const float2& a, const float2& b, const float2& c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(const float2& a, const float2& b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---------------------------------------------------------------- the list of tiles

// Rows qt * ROWS .. of one (sequence, head) and the tiles that they see.
struct Item {
  Seq sq;
  int b, head, qt, qts;  // qts: row blocks of the sequence, 0 if it is not this kernel's
  int t0, t1;
};

template <int ROWS>
__device__ __forceinline__ int row_blocks(const ChunkArgs& g, const Seq& sq) {
  const int rows = sq.n * (int)g.a.group;
  return rows > g.few ? (rows + ROWS - 1) / ROWS : 0;
}
template <int ROWS>
__device__ __forceinline__ void tiles_of(const ChunkArgs& g, const Seq& sq, int qt, int* t0, int* t1) {
  const int rows = sq.n * (int)g.a.group, start = sq.length - sq.n;
  const int first = start + qt * ROWS / (int)g.a.group, last = start + (min((qt + 1) * ROWS, rows) - 1) / (int)g.a.group;
  const int64_t from = g.a.window > 0 ? (int64_t)first - g.a.window + 1 : 0;
  *t0 = from > 0 ? (int)(from / kKeys) : 0;
  // rows without keys still have to be written: one tile, all masked
  *t1 = max(last < 0 ? 0 : last / kKeys + 1, *t0 + 1);
}

// The list's units are tiles, and kItemCost before each block of rows' first
// tile that stand for its own work.
template <int ROWS>
struct Walk {
  Item it;
  int t;           // next tile
  long long left;  // units of the run from t on; none left: the end
  __device__ __forceinline__ void next_item(const ChunkArgs& g) {
    if (++it.qt == it.qts) {
      it.qt = 0;
      if (++it.head == (int)g.c.kv_heads) {
        it.head = 0;
        while (++it.b < (int)g.b.seqs) {
          it.sq = sequence(g.b, it.b);
          it.qts = row_blocks<ROWS>(g, it.sq);
          if (it.qts > 0) break;
        }
      }
    }
    if (it.b < (int)g.b.seqs) tiles_of<ROWS>(g, it.sq, it.qt, &it.t0, &it.t1);
    t = it.t0;
    left -= kItemCost;
  }
  // one past the last tile of the piece that begins at t
  __device__ __forceinline__ int piece_end() const { return (int)min((long long)it.t1, t + left); }
  __device__ __forceinline__ void advance(const ChunkArgs& g, int to) {
    left -= to - t;
    t = to;
    if (t == it.t1 && left > 0) next_item(g);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) kv_chunk_kernel(const ChunkArgs g) {
  constexpr int TERMS = sizeof(T) == 2 && __is_same(T, __half) ? 3 : 2;
  using S = Shape<D, TERMS>;
  constexpr int ROWS = S::kRows, NQ = S::NQ;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bars[35];
  __shared__ float4 s_scale[kMeta][8];  // of a tile's blocks: key scale, value exponent, 2^-value exponent, tokens (integer)
  __shared__ int s_tokens[kMeta];                                 // of a tile
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last, s_failed;
  __shared__ int s_arrived[2];  // of the partial results: 0 not there yet, 1 counted, 2 counted as the last one
  // threads that share a row: the largest magnitude of its queries, and what each half has found
  // (its exponent)
  __shared__ uint8_t s_most[NQ == 1 ? ROWS : 1];
  __shared__ __align__(16) float s_half[NQ == 1 ? 2 : 1][2][128];
  long long* const s_total = reinterpret_cast<long long*>(&s_half[0][0][0]);  // of the warps, before the roles part
  __shared__ Walk<ROWS> s_walk;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int seqs = (int)g.b.seqs, group = (int)g.a.group;
  uint8_t* const smem = smem_raw;
  const uint32_t base = smem_addr(smem);
  const uint32_t q_at = base, k_at = q_at + S::kQ, val_at = k_at + S::kKStages * S::kK, raw_at = val_at + S::kSlots * S::kVal;
  const uint32_t bars = smem_addr(s_bars);
  // barriers
  auto k_full = [&](int s) { return bars + 8 * s; };
  auto k_empty = [&](int s) { return bars + 8 * (2 + s); };
  auto raw_full = [&](int s) { return bars + 8 * (4 + s); };
  auto raw_empty = [&](int s) { return bars + 8 * (8 + s); };
  auto val_full = [&](int s) { return bars + 8 * (12 + s); };
  auto val_empty = [&](int s) { return bars + 8 * (16 + s); };
  auto meta_full = [&](int s) { return bars + 8 * (20 + s); };
  auto q_full = [&](int q) { return bars + 8 * (24 + q); };
  auto s_full = [&](int q) { return bars + 8 * (26 + q); };
  auto s_free = [&](int q) { return bars + 8 * (28 + q); };  // block q has taken its scores
  auto p_full = [&](int q) { return bars + 8 * (30 + q); };
  auto o_full = [&](int q) { return bars + 8 * (32 + q); };  // and its weights are used
  const uint32_t joined = bars + 8 * 34;  // the softmax warps, around a join
  auto pair_bar = [&](int s) { return bars + 8 * (25 + 2 * s); };  // one block: the two warps that share rows (in place of the second block's)

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(k_full(s), 1 + g.waits.stalls());
      mbar_init(k_empty(s), 1);
      mbar_init(q_full(s), NQ == 1 && s == 1 ? 2 : 8 / NQ);
      mbar_init(s_full(s), NQ == 1 && s == 1 ? 2 : 1);
      mbar_init(s_free(s), NQ == 1 && s == 1 ? 2 : 8 / NQ);
      mbar_init(p_full(s), NQ == 1 && s == 1 ? 2 : 8 / NQ);
      mbar_init(o_full(s), 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), 4);
      mbar_init(val_full(s), 4);
      mbar_init(val_empty(s), 1);
      mbar_init(meta_full(s), 1);
    }
    mbar_init(joined, 8);
    s_abort = s_failed = s_arrived[0] = s_arrived[1] = 0;
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- the list's length and this CTA's run. A thread owns `per` sequences;
  // its warp adds up the tiles of each one's row blocks together.
  const int per = (seqs + kThreads - 1) / kThreads;
  auto tiles_a_head = [&](int b) -> long long {  // of sequence b of each lane, all lanes together
    Seq sq{0, 0, 0};
    if (b < seqs) sq = sequence(g.b, b);
    const int qts = b < seqs ? row_blocks<ROWS>(g, sq) : 0;
    long long sum = 0;
    for (uint32_t m = __ballot_sync(0xFFFFFFFFu, qts > 0); m; m &= m - 1) {
      const int o = __ffs(m) - 1;
      Seq x;
      x.first = 0;
      x.n = __shfl_sync(0xFFFFFFFFu, sq.n, o);
      x.length = __shfl_sync(0xFFFFFFFFu, sq.length, o);
      const int n = __shfl_sync(0xFFFFFFFFu, qts, o);
      long long part = 0;
      for (int qt = lane; qt < n; qt += 32) {
        int t0, t1;
        tiles_of<ROWS>(g, x, qt, &t0, &t1);
        part += t1 - t0 + kItemCost;
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
      if (lane == o) sum = part;
    }
    return sum;
  };
  long long mine = 0;
  for (int j = 0; j < per; ++j) mine += tiles_a_head(tid * per + j < seqs ? tid * per + j : seqs) * g.c.kv_heads;
  long long upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xFFFFFFFFu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) s_total[warp] = upto;
  // units that a block of rows has at most: those of the longest sequence, or of a window
  int longest = 0;
  for (int b = lane; b < seqs; b += 32) {
    const Seq sq = sequence(g.b, b);
    if (row_blocks<ROWS>(g, sq) > 0) longest = max(longest, sq.length);
  }
  longest = __reduce_max_sync(0xFFFFFFFFu, longest) / kKeys;
  if (g.a.window > 0) longest = (int)min((int64_t)longest, g.a.window / kKeys + 2);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  long long before = upto - mine, total = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) {
    if (w < warp) before += s_total[w];
    total += s_total[w];
  }
  const int runs = (int)max(min((long long)gridDim.x, total / min_run(longest + kItemCost)), 1ll);
  const long long each = total / runs, more = total - each * runs;
  auto run_start = [&](int w) { return w >= runs ? total : w * each + min((long long)w, more); };
  const long long at0 = run_start((int)blockIdx.x), at1 = run_start((int)blockIdx.x + 1);
  const uint32_t owner = __ballot_sync(0xFFFFFFFFu, at0 < at1 && at0 >= before && at0 < before + mine);
  if (owner) {  // this warp's lane that counted the run's first tile looks for it, all lanes helping
    const int o = __ffs(owner) - 1;
    long long rem = at0 - __shfl_sync(0xFFFFFFFFu, before, o);
    int b = 0;
    long long head_tiles = 1;
    for (int j = 0; j < per; ++j) {
      const long long n = tiles_a_head(tid * per + j < seqs ? tid * per + j : seqs);
      const long long no = __shfl_sync(0xFFFFFFFFu, n, o);
      b = __shfl_sync(0xFFFFFFFFu, tid * per + j, o);
      head_tiles = no;
      if (rem < no * g.c.kv_heads) break;
      rem -= no * g.c.kv_heads;
    }
    Walk<ROWS> w;
    w.it.b = b;
    w.it.sq = sequence(g.b, b);
    w.it.qts = row_blocks<ROWS>(g, w.it.sq);
    w.it.head = (int)(rem / head_tiles);
    rem -= w.it.head * head_tiles;
    for (int q0 = 0;; q0 += 32) {
      int t0 = 0, t1 = 0;
      if (q0 + lane < w.it.qts) tiles_of<ROWS>(g, w.it.sq, q0 + lane, &t0, &t1);
      const int units = q0 + lane < w.it.qts ? t1 - t0 + kItemCost : 0;
      int sum = units;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += x;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, sum > rem);
      if (past || q0 + 32 >= w.it.qts) {
        const int i = past ? __ffs(past) - 1 : 0;
        w.it.qt = q0 + i;
        w.it.t0 = __shfl_sync(0xFFFFFFFFu, t0, i);
        w.it.t1 = __shfl_sync(0xFFFFFFFFu, t1, i);
        rem -= __shfl_sync(0xFFFFFFFFu, sum - units, i);
        break;
      }
      rem -= __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    // inside the units before the first tile: the rest of them goes by
    const int into = (int)rem - kItemCost;
    w.t = w.it.t0 + max(into, 0);
    w.left = at1 - at0 + min(into, 0);
    if (lane == 0) s_walk = w;
  }
  __syncthreads();
  const Limit limit{&s_abort, g.waits.limit_ns / kNsATry};

  if (at0 < at1) {
    Walk<ROWS> w = s_walk;
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
      // ------------------------------------------------ softmax: thread = row of block q, or with a single block half
      // of a row's keys and channels (a warpgroup alone takes 4000 cycles a tile, the products 2600; 247 -> 208 us)
      constexpr bool kHalves = NQ == 1;
      constexpr int kOwn = kHalves ? kKeys / 2 : kKeys, kOwnCh = kHalves ? D / 2 : D;  // keys and channels of a thread
      const int q = kHalves ? 0 : warp >> 2, half = kHalves ? warp >> 2 : 0, r = tid & 127;
      if (w.left > 0) {
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 TMEM lanes
        const uint32_t p_at = lanes + S::kPCol + q * 64 + half * 32, o_at = lanes + S::kOCol + q * D;
        struct Row {
          bool is;
          int pos, low;
          uint32_t most;  // bits of its largest magnitude
          float fq;       // scale of its scores, with the logarithm's base and the queries' power of two
          T* out;
        };
        auto up_exponent = [](uint32_t bits) { return min(7 - ((int)(bits >> 23) - 127), 126); };
        // this thread's row of the piece; the warp's queries as terms in swizzled rows
        auto queries = [&](Row& row) {
          const Item& it = w.it;
          const int index = it.qt * ROWS + q * 128 + r, i = index / group;
          row.is = i < it.sq.n;
          row.pos = row.is ? it.sq.length - it.sq.n + i : 0x3FFFFFFF;  // beyond any token
          row.low = row.is && g.a.window > 0 ? (int)max((int64_t)row.pos - g.a.window + 1, (int64_t)0) : 0;
          const int64_t token = it.sq.first + (row.is ? i : 0), col = (int64_t)(it.head * group + index % group) * D;
          row.out = static_cast<T*>(g.a.out) + token * g.a.out_stride + col;
          const T* src = row.is ? static_cast<const T*>(g.a.q) + token * g.a.q_stride + col : nullptr;
          // The warp reads its rows together, kLanes lanes a row (a lane has eight channels), kBatch loads in flight.
          constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 8;
          const int part = lane % kLanes, c8 = part * 8, panel = c8 / S::W, chunk = c8 % S::W / 16;
          uint32_t own = 0;  // largest magnitude of this lane's own row
          const int i_from = kHalves ? half * (kLanes / 2) : 0, i_to = kHalves ? i_from + kLanes / 2 : kLanes;
#pragma unroll 1
          for (int i0 = i_from; i0 < i_to; i0 += kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const T* p = reinterpret_cast<const T*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src), (i0 + i) * kAtOnce + lane / kLanes));
              x[i] = p ? __ldg(reinterpret_cast<const uint4*>(p) + part) : make_uint4(0, 0, 0, 0);
            }
            // largest magnitudes of the batch's rows side by side: a lane's, then over the lanes of a row
            uint32_t most[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const uint32_t m2 = __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu), __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
              most[i] = max(m2 & 0xFFFFu, m2 >> 16);  // the bits of non-negative floats order as they do
            }
            if (kLanes == 32) {
#pragma unroll
              for (int i = 0; i < kBatch; ++i) most[i] = __reduce_max_sync(0xFFFFFFFFu, most[i]);
            } else {
#pragma unroll
              for (int d = 1; d < kLanes; d <<= 1)
#pragma unroll
                for (int i = 0; i < kBatch; ++i) most[i] = max(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], d));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
              const uint32_t bits = __float_as_uint(unpack2<T>(most[i]).x);
              if (kHalves) {
                if (part == 0) s_most[(warp & 3) * 32 + (i0 + i) * kAtOnce + lane / kLanes] = (uint8_t)(bits >> 23);
              } else {
                const uint32_t of_own = __shfl_sync(0xFFFFFFFFu, bits, lane % kAtOnce * kLanes);
                if (lane / kAtOnce == i0 + i) own = of_own;
              }
              // largest magnitude into [2^7, 2^8); a row with a value that is not finite becomes no number
              // (the scale's sign goes to the queries, so that scores only ever grow with the products)
              const float up = bits < 0x7F800000u ? copysignf(exp2i(up_exponent(bits)), g.a.scale) : __int_as_float(0x7FC00000);
              // in f16 from here on: its 11 bits hold the scaled values, and what the terms leave of them, down to 2^-24
              __half2 v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = unpack2<T>(xs[j]);
                v[j] = __floats2half2_rn(f.x * up, f.y * up);
              }
              const int rr = (warp & 3) * 32 + (i0 + i) * kAtOnce + lane / kLanes, turn = S::W == 128 ? rr & 7 : (rr >> 1) & 3;
              uint32_t dst = q_at + q * TERMS * S::kQTerm + panel * (128 * S::W) + rr * S::W + ((chunk ^ turn) << 4) + 8 * (part & 1);
#pragma unroll
              for (int n = 0; n < TERMS; ++n) {
                uint32_t code[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t c0 = n == 0 ? e4m3x2_of(v[2 * j]) : e5m2x2_of(v[2 * j]);
                  const uint32_t c1 = n == 0 ? e4m3x2_of(v[2 * j + 1]) : e5m2x2_of(v[2 * j + 1]);
                  code[j] = c0 | (c1 << 16);
                  if (n < TERMS - 1) {
                    v[2 * j] = __hsub2(v[2 * j], n == 0 ? as_half2(e4m3x2_to_f16x2(c0)) : half2_of_e5m2x2(c0));
                    v[2 * j + 1] = __hsub2(v[2 * j + 1], n == 0 ? as_half2(e4m3x2_to_f16x2(c1)) : half2_of_e5m2x2(c1));
                  }
                }
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(code[0]), "r"(code[1]) : "memory");
                dst += S::kQTerm;
              }
            }
          }
          // the next block's rows, mostly of the same head, on their way to the second-level cache
          const int next = (index + ROWS) / group;
          if (next < it.sq.n) {
            const char* p = reinterpret_cast<const char*>(static_cast<const T*>(g.a.q) + (it.sq.first + next) * g.a.q_stride +
                                                          (int64_t)(it.head * group + (index + ROWS) % group) * D);
#pragma unroll
            for (int c = half * kOwnCh; c < (half + 1) * kOwnCh; c += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 2 * c));
          }
          row.most = own;
          proxy_fence();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full(q));
        };
        int k = 0;  // tiles so far
        uint32_t meets = 0;
        bool ok = true;
        auto meet = [&]() {  // all softmax warps; bounded, unlike a named barrier
          __syncwarp();
          if (lane == 0) mbar_arrive(joined);
          ok = wait_warp(joined, meets++ & 1, limit, 63);
          return ok;
        };
        uint32_t pairs = 0;
        auto other_half = [&](float mine, float& other) {
          float* const at = &s_half[kHalves ? pairs & 1 : 0][half][r];
          *at = mine;
          __syncwarp();
          if (lane == 0) mbar_arrive(pair_bar(warp & 3));
          ok = wait_warp(pair_bar(warp & 3), pairs++ & 1, limit, 56);
          other = at[half ? -128 : 128];
          return ok;
        };
        // A piece's results are written after the next one's queries (its products with the old ones are done by then),
        // so that the next scores are under way meanwhile.
        struct Result {
          bool is, begins;         // begins: the piece has the rows' first tile
          int to_end, tiles;       // tiles of the rows after the piece, and of all
          long long at;            // place of the piece's end in the list
          T* out;
        } old;
        // score and value exponent that the row's weights refer to (their sum, in m alone, up to kFar), denominator
        float m = -INFINITY, me = 0.f, l = 0.f;
        uint32_t piece_ph = 1;
        bool finished = false;
        for (bool first = true;; first = false) {
          const bool more_pieces = w.left > 0;
          piece_ph ^= 1;
          Row row;
          if (more_pieces) queries(row);
          if (!first) {
            if (!wait_warp(o_full(q), (k - 1) & 1, limit, 54)) {
              ok = false;
              break;
            }
            tc_after();
            if (kHalves) {
              float l2;
              if (!other_half(l, l2)) break;
              l = half ? l2 + l : l + l2;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool whole = old.begins && old.to_end == 0;
            // rows that go on after this run's end: second partial result; that began before it: first
            float* part = g.ws + ((int64_t)blockIdx.x * 2 + (old.begins ? 1 : 0)) * S::kPart;
            const int pr = q * 128 + r;
#pragma unroll 1
            for (int c = half * kOwnCh; c < (half + 1) * kOwnCh; c += 32) {
              float o[32];
              tmem_load(o_at + c, o);
              tmem_load_wait();
              if (whole) {
                if (old.is) {
#pragma unroll
                  for (int j = 0; j < 32; j += 16) {
                    uint32_t y[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) y[u] = pack2<T>(o[j + 2 * u] * inv, o[j + 2 * u + 1] * inv);
                    store32(old.out + c + j, y);
                  }
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4)  // four channels of all rows lie together
                  *reinterpret_cast<float4*>(part + (int64_t)((c + j) / 4 * ROWS + pr) * 4) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
              }
            }
            tc_before();
            if (!whole) {
              if (half == 0) {
                part[(int64_t)ROWS * D + pr] = m;
                part[(int64_t)ROWS * D + ROWS + pr] = l;
                part[(int64_t)ROWS * D + 2 * ROWS + pr] = me;
              }
              // places of the rows' tiles in the list, and the CTAs that hold some of them
              const long long to = old.at + old.to_end, from = to - old.tiles;
              const long long longer = more * (each + 1);
              auto cta_of = [&](long long at) { return (int)(at < longer ? at / (each + 1) : more + (at - longer) / each); };
              const int c0 = cta_of(from), n = cta_of(to - 1) - c0 + 1;
              __threadfence();
              if (!meet()) break;
              if (tid == 0) {
                s_last = atomicAdd(g.done + c0, 1u) == (unsigned)(n - 1);
                s_arrived[old.begins] = s_last ? 2 : 1;
              }
              if (!meet()) break;
              if (s_last) {
                __threadfence();
                auto part_of = [&](int j) { return g.ws + ((int64_t)(c0 + j) * 2 + (j == 0 ? 1 : 0)) * S::kPart; };
                float top = -INFINITY, te = 0.f, sum = 0.f;
                auto max_of = [&](int j) { return __ldcg(part_of(j) + (int64_t)ROWS * D + pr); };
                auto exp_of = [&](int j) { return __ldcg(part_of(j) + (int64_t)ROWS * D + 2 * ROWS + pr); };
                for (int j = 0; j < n; ++j) {
                  const float s = max_of(j), e = exp_of(j);
                  if ((s - top) + (e - te) > 0.f) top = s, te = e;
                }
                const float ref = top == -INFINITY ? 0.f : top;
                auto weight = [&](int j) { return ex2((max_of(j) - ref) + (exp_of(j) - te)); };
                for (int j = 0; j < n; ++j) sum = fmaf(weight(j), __ldcg(part_of(j) + (int64_t)ROWS * D + ROWS + pr), sum);
                const float inv_all = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
                for (int c = half * kOwnCh; c < (half + 1) * kOwnCh; c += 32) {
                  float4 acc[8];
#pragma unroll
                  for (int u = 0; u < 8; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                  for (int j = 0; j < n; ++j) {
                    const float* p = part_of(j);
                    const float f = weight(j);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                      const float4 v = __ldcg(reinterpret_cast<const float4*>(p + (int64_t)((c / 4 + u) * ROWS + pr) * 4));
                      acc[u].x = fmaf(f, v.x, acc[u].x), acc[u].y = fmaf(f, v.y, acc[u].y);
                      acc[u].z = fmaf(f, v.z, acc[u].z), acc[u].w = fmaf(f, v.w, acc[u].w);
                    }
                  }
                  if (old.is) {
#pragma unroll
                    for (int u = 0; u < 8; u += 2)
                      *reinterpret_cast<uint4*>(old.out + c + 4 * u) =
                          make_uint4(pack2<T>(acc[u].x * inv_all, acc[u].y * inv_all), pack2<T>(acc[u].z * inv_all, acc[u].w * inv_all),
                                     pack2<T>(acc[u + 1].x * inv_all, acc[u + 1].y * inv_all), pack2<T>(acc[u + 1].z * inv_all, acc[u + 1].w * inv_all));
                  }
                }
                if (tid == 0) g.done[c0] = 0;
              }
              if (!meet()) break;
            }
          }
          if (!more_pieces) {
            finished = true;
            break;
          }
          if (kHalves) {
            if (!wait_warp(q_full(q), piece_ph, limit, 52)) break;
            row.most = (uint32_t)s_most[r] << 23;
          }
          // Never zero, not even times a block's scale (2^-48 at least): a masked key's minus infinity has to stay one. A
          // factor that is raised to 2^-98 gives scores below 2^-25 with any keys (products below 2^25 times 2^48).
          row.fq = fmaxf(score_factor(fabsf(g.a.scale), up_exponent(row.most)), exp2i(-98));
          const int t_begin = w.t, t_end = w.piece_end();
          m = -INFINITY;
          me = 0.f;
          l = 0.f;
          for (int t = t_begin; t < t_end; ++t, ++k) {
            const int ms = k % kMeta;
            if (!wait_warp(meta_full(ms), (k / kMeta) & 1, limit, 51, s_full(q), k & 1)) {
              ok = false;
              break;
            }
            tc_after();
            float x[kOwn];
#pragma unroll
            for (int c = 0; c < kOwn; c += 32) tmem_load(lanes + half * kOwn + c, x + c);
            tmem_load_wait();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(q));
            const int tok0 = t * kKeys + half * kOwn, blk0 = half * (kOwn / kBlock);
            bool part = !(tok0 + kOwn - 1 <= row.pos && tok0 >= row.low);
            part |= s_tokens[ms] != kKeys;
            if (__any_sync(0xFFFFFFFFu, part)) {
#pragma unroll
              for (int j = 0; j < kOwn / kBlock; ++j) {
                const int n = min(__float_as_int(s_scale[ms][blk0 + j].w), row.pos - (tok0 + 16 * j) + 1), from = row.low - (tok0 + 16 * j);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  if (c >= n || c < from) x[16 * j + c] = -INFINITY;
              }
            }
            // scores are f x, and with them a key weighs f x + e, f and e those of a block
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < kOwn / kBlock; ++j) {
              const float* y = x + 16 * j;
              float a = max3(y[0], y[1], y[2]), b = max3(y[3], y[4], y[5]);
              a = max3(a, y[6], y[7]), b = max3(b, y[8], y[9]);
              a = max3(a, y[10], y[11]), b = max3(b, y[12], y[13]);
              a = max3(a, y[14], y[15]);
              const float4 sc = s_scale[ms][blk0 + j];
              top = fmaxf(top, fmaf(fmaxf(a, b), row.fq * sc.x, sc.y));
            }
            if (kHalves) {
              float top2;
              if (!other_half(top, top2)) break;
              top = fmaxf(top, top2);
            }
            // a larger maximum is taken over only where the weights would grow too large
            float keep = 1.f;
            const float held = m + me;
            const bool more = top > held + kSlack || m == -INFINITY;
            const float mn = more ? top : m;
            const bool far = __any_sync(0xFFFFFFFFu, fabsf(mn) > kFar && mn != -INFINITY);
            if (far) {  // x becomes the difference to the heaviest key's score
              float bs = -INFINITY, be = 0.f;
#pragma unroll
              for (int j = 0; j < kOwn / kBlock; ++j) {
                const float4 sc = s_scale[ms][blk0 + j];
                const float f = row.fq * sc.x;
                float most = -INFINITY;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  x[16 * j + c] *= f;
                  most = fmaxf(most, x[16 * j + c]);
                }
                if ((most - bs) + (sc.y - be) > 0.f) bs = most, be = sc.y;
              }
              if (kHalves) {  // both threads of a row choose alike, the larger score where two keys weigh the same
                float s2, e2;
                if (!other_half(bs, s2) || !other_half(be, e2)) break;
                const float over = (s2 - bs) + (e2 - be);
                if (over > 0.f || (over == 0.f && s2 > bs)) bs = s2, be = e2;
              }
              if ((bs - m) + (be - me) > kSlack) {
                keep = m == -INFINITY ? 0.f : ex2((m - bs) + (me - be));
                m = bs;
                me = be;
              }
              const float from = m == -INFINITY ? 0.f : m;
#pragma unroll
              for (int c = 0; c < kOwn; ++c) x[c] -= from;
            } else if (more) {
              keep = m == -INFINITY ? 0.f : ex2((m - top) + me);
              m = top;
              me = 0.f;
            }
            auto used = [&]() {  // the weights of the tile before, and with them its sums
              if (t > t_begin) ok = wait_warp(o_full(q), (k - 1) & 1, limit, 53);
              tc_after();
              return ok;
            };
            const bool grew = t > t_begin && __any_sync(0xFFFFFFFFu, keep != 1.f);
            if (grew) {
              if (!used()) break;
              l *= keep;
#pragma unroll 1
              for (int c = half * kOwnCh; c < (half + 1) * kOwnCh; c += 32) {
                float o[32];
                uint32_t y[32];
                tmem_load(o_at + c, o);
                tmem_load_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(o[j] * keep);
                tmem_store(o_at + c, y);
              }
            }
            const float ref = (far || m == -INFINITY ? 0.f : m) + (me - kPUp);
            uint32_t p[kOwn / 2];
#pragma unroll
            for (int j = 0; j < kOwn / kBlock; ++j) {
              const float4 sc = s_scale[ms][blk0 + j];
              const float fj = far ? 1.f : row.fq * sc.x, ej = sc.y - ref;
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                float2 y = fma2(make_float2(x[16 * j + c], x[16 * j + c + 1]), make_float2(fj, fj), make_float2(ej, ej));
                y = make_float2(ex2(y.x), ex2(y.y));
                sum = add2(sum, y);
                p[8 * j + c / 2] = pack2<__half>(y.x, y.y);
              }
              l = fmaf(sum.x + sum.y, sc.z, l);
            }
            // the weights of the tile before have to be used up only now
            if (!grew && !used()) break;
#pragma unroll
            for (int c = 0; c < kOwn / 2; c += 32) tmem_store(p_at + c, p + c);
            tmem_store_wait();
            tc_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(q));
          }
          if (!ok) break;
          old = Result{row.is, t_begin == w.it.t0, w.it.t1 - t_end, w.it.t1 - w.it.t0, at1 - (w.left - (t_end - t_begin)), row.out};
          w.advance(g, t_end);
        }
        // A wait gave up: the run's rows come out as no numbers, and what other CTAs count on still arrives, so that the
        // counts are zero again after the call. (All softmax warps get here, since every wait ends.)
        auto all_here = []() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        if (!finished) s_failed = 1;
        all_here();
        if (s_failed) {
          for (Walk<ROWS> v = s_walk; v.left > 0;) {
            const int end = v.piece_end();
            const bool begins = v.t == v.it.t0;
            bool lost = begins && end == v.it.t1;
            if (!lost) {
              const long long to = at1 - (v.left - (end - v.t)) + (v.it.t1 - end), from = to - (v.it.t1 - v.it.t0), longer = more * (each + 1);
              auto cta_of = [&](long long at) { return (int)(at < longer ? at / (each + 1) : more + (at - longer) / each); };
              const int c0 = cta_of(from), n = cta_of(to - 1) - c0 + 1;
              if (s_arrived[begins] == 0) {
                float* const part = g.ws + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * S::kPart;
                for (int j = tid; j < ROWS; j += 256) part[(int64_t)ROWS * D + ROWS + j] = __int_as_float(0x7FC00000);
                __threadfence();
                all_here();
                if (tid == 0) s_arrived[begins] = atomicAdd(g.done + c0, 1u) == (unsigned)(n - 1) ? 2 : 1;
                all_here();
              }
              lost = s_arrived[begins] == 2;
              if (lost && tid == 0) g.done[c0] = 0;
            }
            if (lost) {
              for (int j = tid; j < ROWS * D / 2; j += 256) {
                const int index = v.it.qt * ROWS + j / (D / 2), i = index / group;
                if (i >= v.it.sq.n) break;
                T* const y = static_cast<T*>(g.a.out) + (int64_t)(v.it.sq.first + i) * g.a.out_stride + (int64_t)(v.it.head * group + index % group) * D;
                reinterpret_cast<uint32_t*>(y)[j % (D / 2)] = 0x7FFF7FFFu;  // two numbers that are none, in f16 and in bf16
              }
            }
            v.advance(g, end);
          }
        }
      }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
      // Warps on one scheduler share its issue slots: the warp that issues the products has only softmax warps beside it.
      constexpr int kKeyCopier = 12, kIssuer = 13, kValueCopier = 15;
      // With few stages of keys their copy must not wait for the values' buffers, nor for the scales that go with it: a
      // warp each (256 channels: 199 us, 208 with one warp). With 128 channels one more warp that polls costs more than
      // that gives (a prompt of 8192 tokens: 435 us, 425 with one warp).
      constexpr bool kTwoCopiers = NQ == 1;
      const int conv = warp == 8 ? 0 : warp == 10 ? 1 : warp == 11 ? 2 : warp == 14 ? 3 : -1;
      if (conv >= 0) {
      // ------------------------------------------------ values: codes -> f16, rows of 64 tokens a channel
      const int c0 = conv * 32 + lane;
      // p: panels so far, two a tile
      for (int p = 0; w.left > 0; ++p, w.advance(g, w.t + ((p & 1) ^ 1))) {
        const int s = p % S::kSlots;
        const uint32_t ph = (p / S::kSlots) & 1;
        if (!wait_warp(raw_full(s), ph, limit, 55, val_empty(s), ph ^ 1)) break;
        if (kTwoCopiers && (p & 1) == 0 && !wait_warp(meta_full((p >> 1) % kMeta), ((p >> 1) / kMeta) & 1, limit, 59)) break;
        const uint32_t src = raw_at + s * S::kRaw, dst = val_at + s * S::kVal;
        const float4* of_blocks = &s_scale[(p >> 1) % kMeta][4 * (p & 1)];
        const int4 valid = make_int4(__float_as_int(of_blocks[0].w), __float_as_int(of_blocks[1].w), __float_as_int(of_blocks[2].w), __float_as_int(of_blocks[3].w));
        if (valid.x + valid.y + valid.z + valid.w < kPanel) {
          // bytes beyond the last token may hold no numbers: cleared first
#pragma unroll 1
          for (int idx = c0; idx < D * 4; idx += 128) {
            const int blk = idx / D, n = blk == 0 ? valid.x : blk == 1 ? valid.y : blk == 2 ? valid.z : valid.w;
            const uint32_t at = src + idx * 16;
            const uint4 v = lds128(at);
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int k = min(max(n - 4 * u, 0), 4);
              x[u] &= k == 4 ? ~0u : (1u << (8 * k)) - 1u;
            }
            sts128(at, make_uint4(x[0], x[1], x[2], x[3]));
          }
        }
        // a thread's items: channel d = c0 % D (+ 128) of every block (of every other one with 64 channels)
        const int d0 = c0 % D;
        const uint32_t from = src + c0 * 16, to = dst + d0 * 128;
        const uint32_t turn = (d0 & 7) << 4;
#pragma unroll
        for (int j = 0; j < D * 4 / 128; ++j) {
          // D = 64: blocks 2 j and 2 j + 1 side by side; 256: channels d0 and d0 + 128 in turn
          const uint32_t chunk = D == 64 ? (uint32_t)(2 * j + c0 / D) << 5 : D == 128 ? (uint32_t)j << 5 : (uint32_t)(j / 2) << 5;
          const uint4 v = lds128(from + j * 2048);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int u = 0; u < 2; ++u)
            sts128(to + (D == 256 ? (j & 1) * 16384 : 0) + ((chunk + 16 * u) ^ turn),
                   make_uint4(e4m3x2_to_f16x2(x[2 * u]), e4m3x2_to_f16x2(x[2 * u] >> 16), e4m3x2_to_f16x2(x[2 * u + 1]),
                              e4m3x2_to_f16x2(x[2 * u + 1] >> 16)));
        }
        proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(s));
          mbar_arrive(val_full(s));
        }
      }
      } else if (warp == kKeyCopier || (kTwoCopiers && warp == kValueCopier)) {
        // ------------------------------------------------ copies: lane j (0..7) is block j of a tile
        const bool keys = warp == kKeyCopier, values = kTwoCopiers != keys;
        struct Ref {
          int head, len, tok, page, inner;
          bool there;
        };
        auto look_up = [&](Ref& x) {  // the next tile; none: `there` is false
          x.page = -1;
          x.tok = 0;
          x.len = 0;
          x.there = w.left > 0;
          if (!x.there) return;
          const int blk = w.t * (kKeys / kBlock) + (lane & 7), col = blk / (int)g.c.blocks;
          x.head = w.it.head;
          x.len = w.it.sq.length;
          x.tok = blk * kBlock;
          x.inner = blk - col * (int)g.c.blocks;
          if (x.tok < x.len) x.page = __ldg(g.b.page_table + (int64_t)w.it.b * g.b.table_stride + col);
          w.advance(g, w.t + 1);
        };
        struct Scales {
          int64_t at;
          int ek, ev, valid;
          bool there;
        };
        auto fetch = [&](const Ref& x, Scales& y) {
          const bool ok = x.page >= 0 && x.page < g.c.pages;
          y.at = ok ? ((int64_t)x.page * g.c.kv_heads + x.head) * g.c.blocks + x.inner : 0;
          y.valid = ok ? min(x.len - x.tok, kBlock) : 0;
          y.there = x.there;
          y.ek = ok ? (int)__ldg(g.c.k_exp + y.at) - 127 : 0;
          y.ev = ok ? (int)__ldg(g.c.v_exp + y.at) - 127 : 0;
        };
        Ref r1;  // pages of the next tile but one, scales of the next one
        Scales s0;
        look_up(r1);
        fetch(r1, s0);
        look_up(r1);
        int issued_k = 0, issued_v = 0;
        for (int k = 0; s0.there; ++k) {
          const int ms = k % kMeta;
          Scales s1;
          if (!kTwoCopiers) {
            fetch(r1, s1);
            look_up(r1);
          }
          const bool has = lane < 8 && s0.valid > 0;
          const uint32_t there = __ballot_sync(0xFFFFFFFFu, has);
          auto publish = [&]() {
            if (lane < 8) s_scale[ms][lane] = make_float4(exp2i(s0.ek), (float)s0.ev, exp2i(-s0.ev), __int_as_float(s0.valid));
            const int tokens = __reduce_add_sync(0xFFFFFFFFu, lane < 8 ? s0.valid : 0);
            if (lane == 0) s_tokens[ms] = tokens;
            __syncwarp();
            if (lane == 0) mbar_arrive(meta_full(ms));
          };
          bool ok = true;
          // (little between a buffer's release and its copy: this code comes from a cold instruction cache)
          if (keys) {
            const int ks = k % S::kKStages;
            ok = wait_warp(k_empty(ks), ((k / S::kKStages) & 1) ^ 1, limit, 57);
            if (!ok) break;
            if (!kTwoCopiers) publish();
            if (lane == 0) mbar_arrive_tx(k_full(ks), __popc(there) * kBlock * D);
            __syncwarp();
            if (has) {
#pragma unroll
              for (int p = 0; p < S::kPanels; ++p)
                bulk_load(k_at + ks * S::kK + p * (kKeys * S::W) + lane * (kBlock * S::W), g.c.k + s0.at * (kBlock * D) + p * (kBlock * S::W),
                          kBlock * S::W, k_full(ks));
            }
            ++issued_k;
            if (kTwoCopiers) publish();
          }
          if (values) {
            for (int h = 0; h < 2; ++h) {
              const int p = 2 * k + h, s = p % S::kSlots;
              ok = wait_warp(raw_empty(s), ((p / S::kSlots) & 1) ^ 1, limit, 58);
              if (!ok) break;
              if (lane == 0) mbar_arrive_tx(raw_full(s), __popc(there >> (4 * h) & 0xFu) * kBlock * D);
              __syncwarp();
              if (has && (lane >> 2) == h) bulk_load(raw_at + s * S::kRaw + (lane & 3) * (kBlock * D), g.c.v + s0.at * (kBlock * D), kBlock * D, raw_full(s));
              ++issued_v;
            }
            if (!ok) break;
          }
          if (kTwoCopiers) {
            fetch(r1, s1);
            look_up(r1);
          }
          s0 = s1;
        }
        if (s_abort) {  // let the copies in flight land before the CTA ends
          for (int i = max(issued_k - S::kKStages, 0); i < issued_k; ++i) wait_bar_quiet(k_full(i % S::kKStages), (i / S::kKStages) & 1, g.waits.limit_ns);
          for (int i = max(issued_v - S::kSlots, 0); i < issued_v; ++i) wait_bar_quiet(raw_full(i % S::kSlots), (i / S::kSlots) & 1, g.waits.limit_ns);
        }
      } else if (warp == kIssuer) {
        // ------------------------------------------------ products: the whole warp walks the list, one lane issues; an
        // operand's descriptor is that of its buffer plus an offset in 16-byte units
        const bool issues = elect();
        const uint64_t q_op = operand<S::W>(q_at), k_op = operand<S::W>(k_at), v_op = operand<128>(val_at);
        // Issuing products lasts as long as doing them but for the couple that are queued, so between two groups of
        // them the tensor cores soon idle (two warps that issue in turn are slower still): what stands between groups
        // is kept short, and the waits of a group are polled together.
        auto wait = [&](int code, auto... polls) {  // every lane polls for itself; the one that issues has seen the phases
          bool ok = true;
          for (uint32_t left = limit.tries; ok && !(polls() & ...); --left)
            if (left == 0) {
              limit.give_up(code);
              ok = false;
            }
          // No lane goes on before all have seen the phases: they turn every tile, and a lane that fell two turns behind
          // the one that issues would wait for a phase that is over.
          ok = __all_sync(0xFFFFFFFFu, ok);
          tc_after();
          return ok;
        };
        uint32_t ph = 0;            // phase of what turns once a tile, of the tile whose sums come next
        uint32_t ks = 0, kph = 0;   // stage and phase of the next scores' keys
        uint32_t vs = 0, vph = 0;   // slot and phase of the next sums' values
        auto keys = [&]() { return try_bar(k_full(ks), kph); };
        // with one tile's slots a panel is used as soon as it is there, and its slot is free again after its products
        constexpr bool kByPanel = S::kSlots == 2;
        auto values = [&]() { return try_bar(val_full(vs), vph) & (kByPanel || try_bar(val_full(vs + 1), vph)); };
        auto scores = [&](int q) {
          constexpr uint32_t idesc = instruction(kKeys);
          const uint64_t kt = k_op + ks * (S::kK / 16), qt = q_op + (uint32_t)q * (TERMS * S::kQTerm / 16);
          if (issues) {
#pragma unroll
            for (int n = TERMS - 1; n >= 0; --n)
#pragma unroll
              for (int p = 0; p < S::kPanels; ++p)
#pragma unroll
                for (int s = 0; s < S::W / 32; ++s)
                  mma_f8(tmem, qt + (n * S::kQTerm + p * (128 * S::W) + 32 * s) / 16, kt + (p * (kKeys * S::W) + 32 * s) / 16,
                         n > 0 ? idesc | kE5m2Queries : idesc, n < TERMS - 1 || p > 0 || s > 0);
            tc_commit(s_full(q));
            if (q == NQ - 1) tc_commit(k_empty(ks));
          }
          if (q == NQ - 1) {
            ks = ks + 1 == S::kKStages ? 0 : ks + 1;
            kph ^= ks == 0;
          }
        };
        auto sums = [&](int q, bool add) {
          constexpr uint32_t idesc = instruction(D);
          const uint64_t v = v_op + vs * (S::kVal / 16);
          const uint32_t p = tmem + S::kPCol + q * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (kByPanel && h == 1 && !wait(66, [&]() { return try_bar(val_full(vs + 1), vph); })) return false;
            if (issues) {
#pragma unroll
              for (int s = 4 * h; s < 4 * h + 4; ++s)
                mma_f16(tmem + S::kOCol + q * D, p + 8 * s, v + h * (S::kVal / 16) + 2 * (s % 4), idesc, add || s > 0);
              if (h == 1) tc_commit(o_full(q));
              if (q == NQ - 1 && kByPanel) tc_commit(val_empty(vs + h));
            }
          }
          if (q == NQ - 1 && !kByPanel && issues) {
            tc_commit(val_empty(vs));
            tc_commit(val_empty(vs + 1));
          }
          if (q == NQ - 1) {
            vs = vs + 2 == S::kSlots ? 0 : vs + 2;
            vph ^= vs == 0;
          }
          return true;
        };
        bool ok = true, any = false;  // any: scores have been issued before
        for (uint32_t piece_ph = 0; w.left > 0 && ok; piece_ph ^= 1) {
          const int begin = w.t, end = w.piece_end();
          // a tile's scores of block q: the ones before have been taken, of the other block or of this one with a single block
          auto first = [&](int q) {
            return wait(60, [&]() { return try_bar(q_full(q), piece_ph); },
                        [&]() { return q > 0 ? try_bar(s_free(0), ph) : !any || try_bar(s_free(NQ - 1), ph ^ 1); },
                        [&]() { return q > 0 || keys(); });
          };
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            ok = ok && first(q);
            if (!ok) break;
            scores(q);
            any = true;
          }
#pragma unroll 1
          for (int t = begin; t < end && ok; ++t, ph ^= 1) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              if (t + 1 < end) {
                if (q == 0)
                  ok = wait(64, [&]() { return try_bar(s_free(NQ - 1), ph); }, keys);
                else
                  ok = wait(64, [&]() { return try_bar(s_free(0), ph ^ 1); });
                if (!ok) break;
                scores(q);
              }
              auto passed = [&]() { return try_bar(p_full(q), ph); };
              ok = q == 0 ? wait(61, passed, values) : wait(61, passed);
              if (!ok) break;
              ok = sums(q, t > begin);
              if (!ok) break;
            }
          }
          w.advance(g, end);
        }
        if (!ok) {  // products in flight still read shared memory and TMEM
          const uint64_t t0 = gtimer();
          while (gtimer() - t0 < 1000000ull) {
          }
        }
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 15) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

constexpr int kDevices = 64;

template <typename T, int D>
cudaError_t launch_shape(ChunkArgs g, cudaStream_t st) {
  constexpr int TERMS = __is_same(T, __half) ? 3 : 2;
  using S = Shape<D, TERMS>;
  auto kern = kv_chunk_kernel<T, D>;
  int dev = 0, sms = 0;
  static std::atomic<int> ready[kDevices];  // SMs of a device on which the kernel's shared memory is allowed
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices) sms = ready[dev].load(std::memory_order_acquire);
  if (sms == 0) {
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, kern)) != cudaSuccess) return e;
    // the warpgroups' shares (2 x 192 + 2 x 64) have to come out of what the block is launched with
    if (at.numRegs < 128) return cudaErrorInvalidConfiguration;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (sms > kKvMaxCtas) sms = kKvMaxCtas;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem)) != cudaSuccess) return e;
    if (dev < kDevices) ready[dev].store(sms, std::memory_order_release);
  }
  if ((e = kv_workspace(dev, st, (size_t)sms * 2 * S::kPart * sizeof(float), &g.done, &g.ws)) != cudaSuccess) return e;
  kern<<<sms, kThreads, S::kSmem, st>>>(g);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const ChunkArgs& g, cudaStream_t st) {
  switch (g.c.head_dim) {
    case 64: return launch_shape<T, 64>(g, st);
    case 128: return launch_shape<T, 128>(g, st);
    default: return launch_shape<T, 256>(g, st);
  }
}

}  // namespace

cudaError_t launch_kv_chunk(const KvCache& c, const KvBatch& b, const KvAttention& a, int few, int dtype, cudaStream_t st) {
  const ChunkArgs g{c, b, a, waits(), few, nullptr, nullptr};
  return dtype == kBF16 ? launch_t<__nv_bfloat16>(g, st) : launch_t<__half>(g, st);
}

int read_kv_chunk_error() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_chunk_error, sizeof(int)) != cudaSuccess) return -1;
  if (v) {
    const int zero = 0;
    cudaMemcpyToSymbol(g_chunk_error, &zero, sizeof(int));
  }
  return v;
}

}  // namespace nvfp4
