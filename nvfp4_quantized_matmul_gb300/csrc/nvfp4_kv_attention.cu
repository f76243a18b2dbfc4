// Attention over the 8-bit paged key/value cache for single tokens and short
// runs of tokens (nvfp4_kv_attention): a persistent kernel that streams the
// cache once.
//
// With block exponents eK, eV and codes k, v of a visible key j, in f32:
//   s_j = scale * log2(e) * 2^eK * (q . k_j)
//   m = the key whose s_m + eV_m is largest,  p_j = 2^((s_j - s_m) + (eV_j - eV_m))
//   out = sum_j p_j v_j / sum_j p_j 2^-eV
// The value scale costs an addition in the exponent and a multiplication per
// block in the sum instead of one per code. Scores are subtracted from scores
// before the exponents are added: where scores are so large that their
// spacing exceeds the exponents (or the constant that the weights are held
// up by), a sum of the two would be rounded to another weight, one that f16
// may not hold.
//
// Bound by the cache's bytes: an SM receives about 23 bytes a cycle at the
// measured copy rate. One token of 64 sequences (1 to 8191 keys, 32 / 16
// heads of 128) takes 195 us, 5.8 TB/s, 86% of a copy's rate; one token over
// 131072 keys (32 / 4 heads) 38 us, of which 20 are the bytes; one token over
// 500 keys 10.1 us. Times here are those of captured graphs; a call from the
// Python binding takes 14 us at least, its host side.
//
// The work is the list of 64-token tiles of every (sequence, row tile,
// key/value head), from lengths read on the device, in equal contiguous
// shares a CTA, which its warps divide in runs. Each warp has its own tile in
// shared memory, filled by bulk copies (the cache's layout needs no
// rearranging; the next tile's keys are on their way as soon as the scores are
// done, its values after the sums), and its own softmax state, so that the
// main loop has no barrier. What a run begins or ends in the middle of a head
// is joined in the CTA, then between CTAs by whichever arrives last, always
// in the same order.
//
// q . k runs on the f8 tensor instructions with the codes as they lie: a
// query row is scaled by a power of two and split into E4M3 terms (two for
// bf16, three for f16; each further term scaled up by 16), which costs a
// fourth of the f16 instructions and no conversion of keys. The terms' sum is
// exact for queries down to 2^-13 of the row's largest and within 2^-21
// (bf16) or 2^-25 (f16) of it below that, where the first term ends at E4M3's
// smallest step. Up to eight rows, the first two terms are the upper and lower
// half of one 16-row operand. The weights p are rounded to f16 (scaled by
// 2^14, so that a key counts until it is 2^38 lighter than the heaviest) and
// multiply values converted to f16, which is exact: half the tensor time of a
// product in f32's 10-bit form, and a key lighter than 2^-28 of the heaviest,
// whose weight has fewer than 11 bits, is off by 2^-39 of that at most. The
// values are the 16-row operand (sixteen channels) and up to eight rows of
// weights the other, so that no half of it is wasted on few rows.
//
// Fragments: lane (g, t) = (lane / 4, lane % 4). Score column c of step j
// (j = 0..7) is token 16 (c / 2) + 2 j + c % 2 of the tile, so that lane
// (g, t) ends up with row g's scores of the 16 tokens of block t: one scale
// pair a lane, and its weights are already the second product's operand,
// whose value operand is then one 16-byte load (a channel's 16 tokens).
#include <atomic>

#include "nvfp4_kv.cuh"
#include "nvfp4_pipe.cuh"

namespace nvfp4 {
namespace {

using namespace kv;
using namespace pipe;

__device__ int g_kv_error = 0;  // first error code recorded by a bounded wait

constexpr int kTile = 64;      // tokens a tile
// Tiles a CTA takes at least: 40 sequences of up to 300 keys, 24 / 2 heads, take 11.2 us with 1 to 4, 12.8 with 8 and 18.6
// with 16; one of 3000 keys, 32 / 8 heads, 13.3, 14.1 and 17.7.
constexpr int kMinShare = 4;
// Heads of up to so many tiles stay in one CTA: half of them more or less in a share is worth less time than joining
// between CTAs. 32 sequences of 5 tokens and 16 heads, 16 tiles each: 48.5 us, 57.0 without; 300 short sequences: 23.6
// and 27.7; 64 long ones, where it moves no end worth mentioning, the same. One token of 16 heads of 128, with and without:
//                 400 keys     1024         1536         1600 (25 tiles: no head is kept whole)
//   1 sequence    10.1, 14.2   14.4, 13.4   16.8, 13.5   13.6
//   4             10.2, 15.6   14.4, 16.6   17.0, 16.1   18.4
//   10            12.9, 17.0   21.0, 24.2   26.1, 28.1   28.7
//   20            15.8, 21.7   28.1, 31.2   36.2, 37.4   37.7
// so it costs up to a quarter where a few long heads are all there is, and gains elsewhere.
constexpr int kWholeHead = 24;
constexpr float kPUp = 14.0f;  // the weights are held times 2^14
// A sequence of more query rows (new tokens x heads of a group) goes to the
// tensor-core kernel of nvfp4_kv_chunk.cu. This one's time grows with every 16
// rows, that one's not up to 128. Here and there, 16 sequences:
//    64 channels, group 12:  72 rows 30 us, 32 us     132 rows  41 us, 32 us
//   128 channels, group 2:   32 rows 127 us, 136 us    48 rows 177 us, 134 us
//   256 channels, group 2:    8 rows 67 us, 77 us      16 rows  90 us, 72 us
// 32 sequences, 128 channels, group 8: 32 rows 86 us, 105 us, 40 rows 124 us,
// 107 us. (A single sequence is the exception: 14000 keys, group 8, 64 rows
// take 46 us here and 53 there.)
constexpr int few_rows(int64_t head_dim) { return head_dim == 64 ? 96 : head_dim == 128 ? 32 : 8; }

struct AttnArgs {
  KvCache c;
  KvBatch b;
  KvAttention a;
  Waits waits;
  int few;         // sequences of more rows are the other kernel's
  float* ws;       // partial results: 2 a CTA, then 1 a warp
  unsigned* done;  // [CTAs] arrivals at the head that starts in a CTA and goes on after it; zero between calls
};

// Operand registers of the query terms: two terms and eight rows share one
// 16-row operand.
template <typename T> constexpr int terms() { return 2; }
template <> constexpr int terms<__half>() { return 3; }

// ROWS: query rows a tile holds (8 or 16). A warp has one tile's keys and one
// tile's values in shared memory; as many warps as that and the registers
// allow keep the copies in flight: with 128 channels and 8 rows 9, 10, 11 and
// 12 warps take 202, 202, 197 and 204 us (64 sequences), with 16 rows 8 and 9
// take 49 and 71 (the ninth makes registers spill), with 64 channels and 16
// rows 8, 10, 12 and 16 take 25.3, 24.6, 23.8 and 30.3 (300 sequences).
template <typename T, int D, int ROWS>
struct Shape {
  static constexpr int kOps = ROWS == 8 ? terms<T>() - 1 : terms<T>();
  static constexpr int kSteps = D / 32;                  // f8 tensor steps of q . k
  static constexpr int kKBytes = kTile * D;              // keys of a tile
  static constexpr int kVBlock = kBlock * D + 32;        // a value block, padded against bank conflicts
  static constexpr int kStage = kKBytes + 4 * kVBlock;
  static constexpr int kQBytes = kOps * kSteps * 512;
  static constexpr int kFit = 225950 / (kStage + kQBytes);  // of 232448 bytes, the rest for what joins the pieces
  static constexpr int kMost = D == 64 ? (ROWS == 8 ? 16 : 12) : D == 128 ? (ROWS == 8 ? 11 : 8) : 6;
  static constexpr int kWarps = kFit < kMost ? kFit : kMost;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kSmem = kWarps * (kStage + kQBytes);
  static constexpr int kPart = ROWS * D + 3 * ROWS;      // floats of a partial result: sums, maxima, denominators, maxima's exponents
};

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void mma_f8(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Whether key a (score, value exponent) weighs more than key b; false where there is no a.
__device__ __forceinline__ bool heavier(float sa, float ea, float sb, float eb) { return (sa - sb) + (ea - eb) > 0.f; }
// The heavier of the lane's key and that of lane ^ d; both lanes choose alike, the larger score where they weigh the same.
__device__ __forceinline__ void heavier_of(float& s, float& e, int d) {
  const float s2 = __shfl_xor_sync(0xFFFFFFFFu, s, d), e2 = __shfl_xor_sync(0xFFFFFFFFu, e, d), more = (s2 - s) + (e2 - e);
  if (more > 0.f || (more == 0.f && s2 > s)) s = s2, e = e2;
}

// A sequence's share of the list: row tiles x heads x tiles.
struct Work {
  Seq sq;
  int t0, nt, rts;  // first tile, tiles, row tiles
};
template <int ROWS>
__device__ __forceinline__ Work work_of(const AttnArgs& g, int b) {
  Work w;
  w.sq = sequence(g.b, b);
  const int start = w.sq.length - w.sq.n;
  const int64_t from = g.a.window > 0 ? (int64_t)start - g.a.window + 1 : 0;
  w.t0 = from > 0 ? (int)(from / kTile) : 0;
  // a sequence without keys still has rows to write: one tile, all masked
  w.nt = max((w.sq.length + kTile - 1) / kTile - w.t0, 1);
  const int rows = w.sq.n * (int)g.a.group;
  w.rts = rows > g.few ? 0 : (rows + ROWS - 1) / ROWS;
  return w;
}

template <int ROWS>
struct Cursor {
  int b, rt, head, tile;
  Work w;
  __device__ __forceinline__ void next(const AttnArgs& g) {
    if (++tile < w.nt) return;
    tile = 0;
    if (++head < (int)g.c.kv_heads) return;
    head = 0;
    if (++rt < w.rts) return;
    rt = 0;
    while (++b < (int)g.b.seqs) {
      w = work_of<ROWS>(g, b);
      if (w.rts > 0) break;
    }
  }
};

// A piece of a (sequence, row tile, head) that a warp could not finish.
struct Piece {
  const float* at;       // partial result (shared or global memory); null: no piece
  long long from, to;    // the whole head's place in the list of tiles
  int rt, head, first, n;  // first, n: the sequence's new tokens
};

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(Shape<T, D, ROWS>::kThreads, 1) kv_stream_kernel(const AttnArgs g) {
  using S = Shape<T, D, ROWS>;
  constexpr int kOps = S::kOps, kOut = D / 16, H = ROWS / 8;
  constexpr int kAhead = 8;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t s_bar[S::kWarps * 2 + 1];  // of a warp's keys and values; of a join
  __shared__ long long s_scan[S::kWarps], s_before[S::kThreads];
  __shared__ int s_tiles[S::kThreads];
  __shared__ int s_abort[S::kWarps], s_last[2];
  // what the joins need again after the main loop, whose registers are short: the share, and the runs' beginnings
  __shared__ long long s_share[4], s_run[S::kWarps];
  __shared__ Piece s_piece[2 * S::kWarps];
  __shared__ uint32_t s_mates[2 * S::kWarps];      // the pieces of a piece's head, itself included
  __shared__ int s_heads[2 * S::kWarps], s_nheads;  // first piece of each head that has some
  __shared__ __align__(16) float s_max[2 * S::kWarps][ROWS], s_sum[2 * S::kWarps][ROWS], s_weight[2 * S::kWarps][ROWS],
      s_top[2 * S::kWarps][ROWS], s_inv[2 * S::kWarps][ROWS], s_max_e[2 * S::kWarps][ROWS], s_top_e[2 * S::kWarps][ROWS];
  // of the pieces: maxima, denominators (a head's first piece: the head's), weights in their head; of heads, at the first
  // piece: maxima, reciprocals of the denominators; value exponents of both maxima

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, t = lane & 3;
  const int seqs = (int)g.b.seqs, group = (int)g.a.group;

  if (lane == 0) {  // a warp's barriers are its own
    mbar_init(smem_addr(&s_bar[2 * warp]), 1 + (warp == 0 ? g.waits.stalls() : 0));
    mbar_init(smem_addr(&s_bar[2 * warp + 1]), 1);
    s_abort[warp] = 0;
    s_piece[2 * warp].at = s_piece[2 * warp + 1].at = nullptr;
  }
  const uint32_t bar_join = smem_addr(&s_bar[2 * S::kWarps]);
  if (tid == 0) mbar_init(bar_join, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncwarp();

  // ---- the list's length, and where each warp's run begins. Up to 32 sequences every warp looks at them by itself, a
  // lane each, without a barrier.
  const bool by_lane = seqs <= 32;
  const int per = by_lane ? 1 : (seqs + S::kThreads - 1) / S::kThreads;
  auto units = [&](const Work& w) { return (long long)w.rts * w.nt * g.c.kv_heads; };
  Work work{};  // by lane: of the lane's sequence
  long long mine = 0;
  if (by_lane) {
    if (lane < seqs) {
      work = work_of<ROWS>(g, lane);
      mine = units(work);
    }
  } else {
    for (int b = tid * per; b < min(tid * per + per, seqs); ++b) {
      const Work w = work_of<ROWS>(g, b);
      mine += units(w);
      s_tiles[tid] = w.nt;  // of a head, where a thread has one sequence
    }
  }
  auto scan = [&](long long x) {
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += o;
    }
    return x;
  };
  const long long upto = scan(mine);
  long long total = 0;
  if (by_lane) {
    total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  } else {
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long before = upto - mine;
#pragma unroll 1
    for (int w = 0; w < S::kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    s_before[tid] = before;
    __syncthreads();
  }
  if (total == 0) return;
  // Equal shares for the CTAs, the first `more` of them one tile longer; a few tiles each at least.
  const unsigned ctas = (unsigned)min((long long)gridDim.x, (total + kMinShare - 1) / kMinShare);
  long long each, more;
  if (total <= 0xFFFFFFFFll) {  // a 64-bit division takes several times as long
    each = (unsigned)total / ctas;
    more = (unsigned)total - (unsigned)each * ctas;
  } else {
    each = total / ctas;
    more = total - each * ctas;
  }
  // The sequence that holds a place in the list, and where its tiles begin there.
  auto locate = [&](long long at, long long* begins) {
    if (by_lane) {
      const int b = __ffs(__ballot_sync(0xFFFFFFFFu, upto > at)) - 1;
      *begins = __shfl_sync(0xFFFFFFFFu, upto - mine, b);
      return b;
    }
    // the thread that counted it, then among its sequences
    const int w = __popc(__ballot_sync(0xFFFFFFFFu, lane < S::kWarps && s_before[lane * 32] <= at)) - 1;
    const int th = w * 32 + __popc(__ballot_sync(0xFFFFFFFFu, s_before[w * 32 + lane] <= at)) - 1;
    long long from = s_before[th];
    int b = th * per;
    for (const int end = min(b + per, seqs); per > 1; b += 32) {
      const long long n = b + lane < end ? units(work_of<ROWS>(g, b + lane)) : 0, all = scan(n);
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, from + all > at);
      if (past) {
        const int i = __ffs(past) - 1;
        from += __shfl_sync(0xFFFFFFFFu, all - n, i);
        b += i;
        break;
      }
      from += __shfl_sync(0xFFFFFFFFu, all, 31);
    }
    *begins = from;
    return b;
  };
  auto mod = [](long long a, int b) { return a <= 0xFFFFFFFFll ? (int)((unsigned)a % (unsigned)b) : (int)(a % b); };
  // This CTA's share, then this warp's run in it. A share's end inside a head of few tiles moves to the nearer end of the
  // head, which then needs no joining between CTAs (and every CTA finds the same ends).
  long long cta_lo = 0, cta_hi = 0;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const unsigned c = blockIdx.x + e;
    long long at = c >= ctas ? total : c * each + min((long long)c, more), begins;
    if (at < total) {
      const int b = locate(at, &begins);
      const int nt = by_lane ? __shfl_sync(0xFFFFFFFFu, work.nt, b) : per == 1 ? s_tiles[b] : work_of<ROWS>(g, b).nt;
      if (nt <= kWholeHead) {
        const int tile = mod(at - begins, nt);
        at += 2 * tile < nt ? -tile : nt - tile;
      }
    }
    cta_lo = cta_hi;
    cta_hi = at;
  }
  if (cta_lo >= cta_hi) return;
  int count;
  Cursor<ROWS> out;  // the tile in work
  {
    const long long len = cta_hi - cta_lo, run = len / S::kWarps, longer = len - run * S::kWarps;
    const long long at = cta_lo + warp * run + min((long long)warp, longer);
    count = (int)run + (warp < longer ? 1 : 0);
    if (lane == 0) s_run[warp] = at;
    if (tid == 0) s_share[0] = cta_lo, s_share[1] = cta_hi, s_share[2] = each, s_share[3] = more;
    if (count > 0) {
      long long begins;
      out.b = locate(at, &begins);
      if (by_lane) {
        out.w.sq.first = __shfl_sync(0xFFFFFFFFu, work.sq.first, out.b);
        out.w.sq.n = __shfl_sync(0xFFFFFFFFu, work.sq.n, out.b);
        out.w.sq.length = __shfl_sync(0xFFFFFFFFu, work.sq.length, out.b);
        out.w.t0 = __shfl_sync(0xFFFFFFFFu, work.t0, out.b);
        out.w.nt = __shfl_sync(0xFFFFFFFFu, work.nt, out.b);
        out.w.rts = __shfl_sync(0xFFFFFFFFu, work.rts, out.b);
      } else {
        out.w = work_of<ROWS>(g, out.b);
      }
      const long long rem = at - begins;
      const int seg = rem <= 0xFFFFFFFFll ? (int)((unsigned)rem / (unsigned)out.w.nt) : (int)(rem / out.w.nt);
      out.tile = (int)(rem - (long long)seg * out.w.nt);
      out.rt = (unsigned)seg / (unsigned)g.c.kv_heads;
      out.head = seg - out.rt * (int)g.c.kv_heads;
    }
  }

  uint8_t* const stage = smem + warp * S::kStage;
  const uint32_t kt = smem_addr(stage), vt = kt + S::kKBytes;
  const uint32_t qfrag = smem_addr(smem + S::kWarps * S::kStage) + (uint32_t)warp * S::kQBytes;
  const uint32_t bar_k = smem_addr(&s_bar[2 * warp]), bar_v = bar_k + 8;
  volatile int* abort_flag = &s_abort[warp];

  // partial results: a CTA's two, then one a warp
  auto warp_part = [&](int w) { return g.ws + ((int64_t)gridDim.x * 2 + (int64_t)blockIdx.x * S::kWarps + w) * S::kPart; };
  if (count > 0) {
    Cursor<ROWS> in = out;  // next tile to copy
    int32_t page = -1;  // of block t of the next tile to copy
    int inner = 0;      // and its place in the page
    auto find_page = [&]() {
      const int blk = (in.w.t0 + in.tile) * (kTile / kBlock) + t, col = blk / (int)g.c.blocks;
      inner = blk - col * (int)g.c.blocks;
      page = blk * kBlock < in.w.sq.length ? __ldg(g.b.page_table + (int64_t)in.b * g.b.table_stride + col) : -1;
    };
    int64_t at = 0;           // block t of the tile last copied
    int ek = 0, ev = 0;       // its exponents
    uint32_t there = 0;       // blocks of the tile that hold tokens
    auto copy_keys = [&]() {
      const bool ok = page >= 0 && page < g.c.pages;
      at = ((int64_t)(ok ? page : 0) * g.c.kv_heads + in.head) * g.c.blocks + inner;
      ek = ok ? (int)__ldg(g.c.k_exp + at) - 127 : 0;
      ev = ok ? (int)__ldg(g.c.v_exp + at) - 127 : 0;
      there = __ballot_sync(0xFFFFFFFFu, ok) & 0xFu;
      if (lane == 0) mbar_arrive_tx(bar_k, __popc(there) * kBlock * D);
      __syncwarp();
      if (lane < 4 && ok) bulk_load(kt + t * (kBlock * D), g.c.k + at * (kBlock * D), kBlock * D, bar_k);
    };
    auto copy_values = [&]() {
      if (lane == 0) mbar_arrive_tx(bar_v, __popc(there) * kBlock * D);
      __syncwarp();
      if (lane < 4 && (there >> t & 1)) bulk_load(vt + t * S::kVBlock, g.c.v + at * (kBlock * D), kBlock * D, bar_v);
    };
    find_page();
    copy_keys();
    copy_values();
    if (count > 1) {
      in.next(g);
      find_page();
    }

    // accumulators of rows 8 h + 2 t, + 1 and channels 16 i + g, + 8: [channel][row]
    float o[kOut][H][4];
    // of row 8 h + g: score and value exponent of the heaviest key so far, this lane's share of the denominator, scale of
    // the scores, position, first key
    float m[H], me[H], l[H], fq[H];
    int pos[H], low[H], pos_min = 0, low_max = 0;

    // the rows of a (row tile, head): their positions, and the queries as operands
    auto begin = [&]() {
      const Seq& sq = out.w.sq;
      const int start = sq.length - sq.n;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int row = out.rt * ROWS + gr + 8 * h, i = row / group;
        const bool ok = i < sq.n;
        pos[h] = ok ? start + i : 0x3FFFFFFF;  // no row: beyond any token, so that it needs no mask
        low[h] = ok && g.a.window > 0 ? (int)max((int64_t)pos[h] - g.a.window + 1, (int64_t)0) : 0;
        m[h] = -INFINITY;
        me[h] = 0.f;
        l[h] = 0.f;
        const T* q = static_cast<const T*>(g.a.q) + (int64_t)(sq.first + (ok ? i : 0)) * g.a.q_stride + (int64_t)(out.head * group + row % group) * D;
        // a panel's chunks 2 t and 2 t + 1 of 16 channels are this lane's (64 channels: chunk t)
        uint4 w[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const int d0 = D == 64 ? 16 * t + 8 * c : (c >> 2) * 128 + 32 * t + 8 * (c & 3);
          w[c] = ok ? __ldg(reinterpret_cast<const uint4*>(q + d0)) : make_uint4(0, 0, 0, 0);
        }
        uint32_t bits = 0;  // the bits of non-negative floats order as they do, infinities and no numbers above all
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<T>(ws[j]);
            bits = max(bits, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
          }
        }
        bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 1));
        bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, 2));
        // largest magnitude into [2^7, 2^8); a row with a value that is not finite becomes no number
        const int up_e = min(7 - ((int)(bits >> 23) - 127), 126);
        const float up = bits < 0x7F800000u ? exp2i(up_e) : __int_as_float(0x7FC00000);
        fq[h] = score_factor(g.a.scale, up_e);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // step c
            const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            float r[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = unpack2<T>(ws[j]);
              r[2 * j] = f.x * up;
              r[2 * j + 1] = f.y * up;
            }
#pragma unroll
            for (int n = 0; n < terms<T>(); ++n) {
              // operand and half of it: eight rows hold terms 0 and 1 in operand 0, term 2 below zeros in operand 1
              const int op = ROWS == 8 ? n / 2 : n, half = ROWS == 8 ? (n > 0 ? 1 : 0) : h;
              const uint32_t at = qfrag + ((uint32_t)(c * kOps + op) * 32 + lane) * 16 + 4 * half;
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float* x = r + 4 * k;
                const uint32_t cd = e4m3x4(x[0], x[1], x[2], x[3]);
                sts32(at + 8 * k, cd);
                if (ROWS == 8 && n == 2) sts32(at + 8 * k - 4, 0);
                const float2 lo = unpack2<__half>(e4m3x2_to_f16x2(cd & 0xFFFFu)), hi = unpack2<__half>(e4m3x2_to_f16x2(cd >> 16));
                x[0] = (x[0] - lo.x) * 16.f;
                x[1] = (x[1] - lo.y) * 16.f;
                x[2] = (x[2] - hi.x) * 16.f;
                x[3] = (x[3] - hi.y) * 16.f;
              }
            }
          }
      }
      __syncwarp();
      // for the test whether a tile needs a mask (a row before the sequence's first token sees none of its keys)
      int lo_pos = pos[0], hi_low = low[0];
#pragma unroll
      for (int h = 1; h < H; ++h) lo_pos = min(lo_pos, pos[h]), hi_low = max(hi_low, low[h]);
      pos_min = __reduce_min_sync(0xFFFFFFFFu, lo_pos);
      low_max = __reduce_max_sync(0xFFFFFFFFu, hi_low);
#pragma unroll
      for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.f;
    };

    float sc[8][4];
    auto scores = [&]() {
#pragma unroll
      for (int j = 0; j < 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
      // keys of column g of step j: block g / 2, row 2 j + g % 2
      constexpr int W = D < 128 ? D : 128;
      const uint32_t krow = kt + (gr >> 1) * (kBlock * D) + (gr & 1) * W;
      // the smallest term first; each larger one counts 16 times as much
#pragma unroll 1
      for (int n = kOps - 1; n >= 0; --n) {
        if (n < kOps - 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[j][c] *= 0.0625f;
        }
        // panels of 128 channels (or the 64 there are); a chunk of 16 channels is two steps
        constexpr int kChunks = D == 64 ? 1 : 2;
#pragma unroll 1
        for (int pn = 0; pn < D / 64 / kChunks; ++pn)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const uint32_t qa = qfrag + ((uint32_t)(2 * (pn * kChunks + c) * kOps + n) * 32 + lane) * 16;
            const uint4 a0 = lds128(qa), a1 = lds128(qa + kOps * 512);
            // kAhead columns at a time: a product does not wait for the one before it
#pragma unroll
            for (int j0 = 0; j0 < 8; j0 += kAhead) {
              uint4 kk[kAhead];
#pragma unroll
              for (int j = 0; j < kAhead; ++j) {
                const int ch = D == 64 ? t ^ ((j0 + j) & 3) : (2 * t + c) ^ ((2 * (j0 + j) + (gr & 1)) & 7);
                kk[j] = lds128(krow + pn * (kBlock * 128) + 2 * (j0 + j) * W + ch * 16);
              }
#pragma unroll
              for (int j = 0; j < kAhead; ++j) mma_f8(sc[j0 + j], a0, kk[j].x, kk[j].y);
#pragma unroll
              for (int j = 0; j < kAhead; ++j) mma_f8(sc[j0 + j], a1, kk[j].z, kk[j].w);
            }
          }
      }
    };

    uint32_t p[H][8];  // weights: token pair j of block t, row 8 h + g
    auto weights = [&](int tok0, int k_e, int v_e, uint32_t blocks, bool clean) {
      const float fk = exp2i(k_e), fe = (float)v_e, fl = exp2i(-v_e);
      float keep[H], base[H], up[H];
      bool grew = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float f = fq[h] * fk;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // eight rows: rows 8..15 of the product are the second term
            float& v = sc[j][2 * h + i];
            v = (ROWS == 8 ? fmaf(sc[j][2 + i], 0.0625f, v) : v) * f;
          }
        if (!clean) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int tok = tok0 + kBlock * t + 2 * j + i;
              if (!(tok <= pos[h] && tok >= low[h] && (blocks >> t & 1))) sc[j][2 * h + i] = -INFINITY;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(sc[j][2 * h], sc[j][2 * h + 1]));
        float te = fe;
        heavier_of(top, te, 1);
        heavier_of(top, te, 2);
        const bool more = heavier(top, te, m[h], me[h]);
        const float mn = more ? top : m[h], en = more ? te : me[h];
        base[h] = mn == -INFINITY ? 0.f : mn;
        keep[h] = ex2((m[h] - base[h]) + (me[h] - en));
        grew |= more;
        m[h] = mn;
        me[h] = en;
        up[h] = fe - en + kPUp;
      }
      if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          l[h] *= keep[h];
          const float k0 = __shfl_sync(0xFFFFFFFFu, keep[h], 8 * t), k1 = __shfl_sync(0xFFFFFFFFu, keep[h], 8 * t + 4);
#pragma unroll
          for (int i = 0; i < kOut; ++i) o[i][h][0] *= k0, o[i][h][1] *= k1, o[i][h][2] *= k0, o[i][h][3] *= k1;
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = ex2((sc[j][2 * h] - base[h]) + up[h]), y = ex2((sc[j][2 * h + 1] - base[h]) + up[h]);
          sum += x + y;
          p[h][j] = pack2<__half>(x, y);
        }
        l[h] = fmaf(sum, fl, l[h]);
      }
    };

    // values: a channel's 16 tokens of block t
    const uint32_t vrow = vt + t * S::kVBlock + gr * 16;
    auto clear_tail = [&](int tok0, uint32_t blocks) {
      // bytes beyond the last token may hold no numbers, which no weight of zero would hide
      const int n = blocks >> t & 1 ? min(max(out.w.sq.length - tok0 - kBlock * t, 0), kBlock) : 0;
      uint32_t vm[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = min(max(n - 4 * j, 0), 4);
        vm[j] = k == 4 ? ~0u : (1u << (8 * k)) - 1u;
      }
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = lds128(vrow + i * 128);
        sts128(vrow + i * 128, make_uint4(v.x & vm[0], v.y & vm[1], v.z & vm[2], v.w & vm[3]));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the copy that overwrites them
      __syncwarp();
    };
    auto sums = [&]() {
#pragma unroll
      for (int i0 = 0; i0 < kOut; i0 += 2) {  // two at a time, so that a product does not wait for the one before it
        uint4 va[2], vb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) va[i] = lds128(vrow + (i0 + i) * 256), vb[i] = lds128(vrow + (i0 + i) * 256 + 128);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x[4] = {va[i].x, va[i].y, va[i].z, va[i].w}, y[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w};
            const uint32_t a0 = e4m3x2_to_f16x2(x[j] & 0xFFFFu), a2 = e4m3x2_to_f16x2(x[j] >> 16);
            const uint32_t a1 = e4m3x2_to_f16x2(y[j] & 0xFFFFu), a3 = e4m3x2_to_f16x2(y[j] >> 16);
#pragma unroll
            for (int h = 0; h < H; ++h) mma_f16(o[i0 + i][h], a0, a1, a2, a3, p[h][2 * j], p[h][2 * j + 1]);
          }
      }
    };

    // a row's denominator, over the four lanes that share it
    auto row_sum = [&](int h) {
      float x = l[h];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
    };
    // lanes g and g ^ 1 exchange, so that each has two neighbouring channels of row 8 h + 2 t + g % 2
    const int odd = gr & 1, own_row = 2 * t + odd;
    auto pair = [&](int i, int h, int half) {
      const float x = o[i][h][2 * half], y = o[i][h][2 * half + 1], mine = odd ? y : x;
      const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? x : y, 4);
      return odd ? make_float2(other, mine) : make_float2(mine, other);
    };
    auto store_part = [&](float* dst, int piece) {  // sums [channel][row]
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float sum = row_sum(h);
        if (t == 0) s_max[piece][gr + 8 * h] = m[h], s_max_e[piece][gr + 8 * h] = me[h], s_sum[piece][gr + 8 * h] = sum;
        float* p = dst + gr * ROWS + 8 * h + 2 * t;
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
          *reinterpret_cast<float2*>(p + 16 * i * ROWS) = make_float2(o[i][h][0], o[i][h][1]);
          *reinterpret_cast<float2*>(p + (16 * i + 8) * ROWS) = make_float2(o[i][h][2], o[i][h][3]);
        }
      }
    };
    auto store_out = [&]() {
      const Seq& sq = out.w.sq;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int row = out.rt * ROWS + own_row + 8 * h, i0 = row / group;
        const float sum = __shfl_sync(0xFFFFFFFFu, row_sum(h), own_row * 4);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        T* y = static_cast<T*>(g.a.out) + (int64_t)(sq.first + i0) * g.a.out_stride + (int64_t)(out.head * group + row % group) * D;
#pragma unroll
        for (int i = 0; i < kOut; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const float2 v = pair(i, h, half);
            if (i0 < sq.n) *reinterpret_cast<uint32_t*>(y + 16 * i + 8 * half + gr - odd) = pack2<T>(v.x * inv, v.y * inv);
          }
      }
    };

    bool fresh = true;           // the tile in work is the first one here of its head
    bool whole = out.tile == 0;  // this run holds the head from its first tile on
    int it = 0;
    for (; it < count; ++it) {
      if (fresh) begin();
      fresh = false;
      const int tok0 = (out.w.t0 + out.tile) * kTile, k_e = ek, v_e = ev;
      const uint32_t blocks = there;
      const bool clean = blocks == 0xFu && tok0 + kTile - 1 <= pos_min && tok0 >= low_max;
      bool ok = wait_bar_warp(bar_k, it & 1, abort_flag, 41, &g_kv_error, g.waits.limit_ns);
      if (ok) {
        scores();
        __syncwarp();
        if (it + 1 < count) copy_keys();
        weights(tok0, k_e, v_e, blocks, clean);
        ok = wait_bar_warp(bar_v, it & 1, abort_flag, 42, &g_kv_error, g.waits.limit_ns);
        if (!ok && it + 1 < count) wait_bar_quiet(bar_k, (it + 1) & 1, g.waits.limit_ns);
      } else {
        wait_bar_quiet(bar_k, it & 1, g.waits.limit_ns);
        wait_bar_quiet(bar_v, it & 1, g.waits.limit_ns);
      }
      if (!ok) break;  // the copies in flight have landed or been given up on
      if (!clean) clear_tail(tok0, blocks);
      sums();
      __syncwarp();
      if (it + 1 < count) copy_values();
      const bool end = out.tile + 1 == out.w.nt;
      if (it + 1 == count || end) {
        const long long from = s_run[warp] + it - out.tile, to = from + out.w.nt;
        if (end && whole) {
          store_out();
        } else {
          // a head that ends here began in an earlier run: aside until all warps are done; one
          // that goes on takes the tile's place, whose copies have all been used
          float* dst = end ? warp_part(warp) : reinterpret_cast<float*>(stage);
          const int piece = 2 * warp + (end ? 0 : 1);
          store_part(dst, piece);
          if (lane == 0) s_piece[piece] = Piece{dst, from, to, out.rt, out.head, out.w.sq.first, out.w.sq.n};
        }
        fresh = whole = true;
      }
      if (it + 1 < count) out.next(g);
      if (it + 2 < count) {
        in.next(g);
        find_page();
      }
    }
    // A wait gave up: the rest of the run comes out as no numbers, and its pieces are there for the joins, so that the
    // counts are zero again after the call.
    const float none = __int_as_float(0x7FC00000);
    if (it < count && lane == 0) s_abort[warp] = 0;  // (a join's wait has a limit of its own)
    while (it < count) {
      const bool end = out.tile + 1 == out.w.nt;
      if (end && whole) {
        for (int j = lane; j < ROWS * D; j += 32) {
          const int row = out.rt * ROWS + j / D, i = row / group;
          if (i < out.w.sq.n)
            static_cast<T*>(g.a.out)[(int64_t)(out.w.sq.first + i) * g.a.out_stride + (int64_t)(out.head * group + row % group) * D + j % D] = from_f32<T>(none);
        }
      } else if (end || it + 1 == count) {
        const int piece = 2 * warp + (end ? 0 : 1);
        const long long from = s_run[warp] + it - out.tile;
        if (lane < ROWS) s_max[piece][lane] = s_max_e[piece][lane] = 0.f, s_sum[piece][lane] = none;
        if (lane == 0)
          s_piece[piece] = Piece{end ? warp_part(warp) : reinterpret_cast<float*>(stage), from, from + out.w.nt, out.rt, out.head, out.w.sq.first, out.w.sq.n};
      }
      if (end) whole = true;
      if (++it < count) out.next(g);
    }
  }
  __syncthreads();

  // ---- pieces of one head are neighbours in the list: join them here, and
  // where a head reaches into other CTAs, by the last of its CTAs to arrive.
  // (This code runs once and from a cold instruction cache: it is short rather than unrolled.)
  const bool is_piece = lane < 2 * S::kWarps && s_piece[lane].at != nullptr;
  const uint32_t pieces = __ballot_sync(0xFFFFFFFFu, is_piece);
  const long long lo = s_share[0], hi = s_share[1];
  if (!pieces) return;
  if (warp == 0) {
    int n = 0;
    for (uint32_t left = pieces; left; ++n) {
      const int i = __ffs(left) - 1;
      const uint32_t mates = __ballot_sync(0xFFFFFFFFu, is_piece && s_piece[lane].from == s_piece[i].from);
      if (mates >> lane & 1) s_mates[lane] = mates;
      if (lane == 0) s_heads[n] = i;
      left &= ~mates;
    }
    if (lane == 0) s_nheads = n;
  }
  __syncthreads();
  for (int idx = tid; idx < 2 * S::kWarps * ROWS; idx += S::kThreads) {  // weights of the pieces' rows
    const int i = idx / ROWS, r = idx % ROWS;
    if (!(pieces >> i & 1)) continue;
    float top = -INFINITY, te = 0.f;
    for (uint32_t k = s_mates[i]; k; k &= k - 1) {
      const float s = s_max[__ffs(k) - 1][r], e = s_max_e[__ffs(k) - 1][r];
      if (heavier(s, e, top, te)) top = s, te = e;
    }
    const float base = top == -INFINITY ? 0.f : top;
    auto weight = [&](int j) { return ex2((s_max[j][r] - base) + (s_max_e[j][r] - te)); };
    s_weight[i][r] = weight(i);
    if (__ffs(s_mates[i]) - 1 != i) continue;
    float sum = 0.f;
    for (uint32_t k = s_mates[i]; k; k &= k - 1) sum = fmaf(weight(__ffs(k) - 1), s_sum[__ffs(k) - 1][r], sum);
    s_top[i][r] = top;
    s_top_e[i][r] = te;
    s_sum[i][r] = sum;
    s_inv[i][r] = sum == 0.f ? 0.f : 1.f / sum;
  }
  __syncthreads();

  constexpr int kItems = ROWS * D / 4;  // channel d = idx % D of rows 4 (idx / D) ..: a warp's are of the same rows
  auto add = [](float4& x, const float4& f, const float4& v) {
    x.x = fmaf(f.x, v.x, x.x), x.y = fmaf(f.y, v.y, x.y), x.z = fmaf(f.z, v.z, x.z), x.w = fmaf(f.w, v.w, x.w);
  };
  // channel d of rows r .., four to each of `x` and of their reciprocal denominators
  auto finish = [&](const Piece& pc, int r, int d, const auto& x, const float* inv) {
    const int row = pc.rt * ROWS + r;
    int i = row / group, h = row - i * group;  // token, head of the group
    T* const y = static_cast<T*>(g.a.out) + (int64_t)pc.first * g.a.out_stride + (int64_t)pc.head * group * D + d;
#pragma unroll
    for (int n = 0; n < (int)(sizeof(x) / sizeof(float4)); ++n) {
      const float4 f = *reinterpret_cast<const float4*>(inv + r + 4 * n);
      const float y4[4] = {x[n].x * f.x, x[n].y * f.y, x[n].z * f.z, x[n].w * f.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i < pc.n) y[(int64_t)i * g.a.out_stride + (int64_t)h * D] = from_f32<T>(y4[u]);
        if (++h == group) h = 0, ++i;
      }
    }
  };
  auto cta_of = [&](long long at) {  // the CTA whose share holds place `at` of a head that reaches into several
    const long long each = s_share[2], more = s_share[3];
    const long long longer = more * (each + 1);
    const long long off = at < longer ? at : at - longer, len = at < longer ? each + 1 : each;
    return (int)(((off | len) <= 0xFFFFFFFFll ? (long long)((unsigned)off / (unsigned)len) : off / len) + (at < longer ? 0 : more));
  };
  const int heads = s_nheads;
#pragma unroll 1
  for (int idx = tid; idx < heads * kItems / 2; idx += S::kThreads) {  // eight rows at a time
    const int i0 = s_heads[idx / (kItems / 2)], d = idx % D, r = idx % (kItems / 2) / D * 8;
    const Piece& pc = s_piece[i0];
    float4 x[2] = {};
#pragma unroll 1
    for (uint32_t k = s_mates[i0]; k;) {  // four pieces at a time, whose loads do not wait for one another
      float4 v[4][2];
      int of[4];
#pragma unroll
      for (int u = 0; u < 4; ++u, k &= k - 1) {
        const int i = of[u] = __ffs(k) - 1;
        if (i < 0) continue;
        // a warp's second piece lies in its tile's place, the first in global memory
        const float* at = i & 1 ? reinterpret_cast<const float*>(smem + (i >> 1) * S::kStage) : warp_part(i >> 1);
        v[u][0] = *reinterpret_cast<const float4*>(at + d * ROWS + r);
        v[u][1] = *reinterpret_cast<const float4*>(at + d * ROWS + r + 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (of[u] < 0) continue;
        add(x[0], *reinterpret_cast<const float4*>(&s_weight[of[u]][r]), v[u][0]);
        add(x[1], *reinterpret_cast<const float4*>(&s_weight[of[u]][r + 4]), v[u][1]);
      }
    }
    if (pc.from >= lo && pc.to <= hi) {
      finish(pc, r, d, x, s_inv[i0]);
    } else {
      float* const part = g.ws + ((int64_t)blockIdx.x * 2 + (pc.from >= lo ? 1 : 0)) * S::kPart;
      *reinterpret_cast<float4*>(part + d * ROWS + r) = x[0];
      *reinterpret_cast<float4*>(part + d * ROWS + r + 4) = x[1];
      if (d < 8) {
        part[ROWS * D + r + d] = s_top[i0][r + d];
        part[ROWS * D + ROWS + r + d] = s_sum[i0][r + d];
        part[ROWS * D + 2 * ROWS + r + d] = s_top_e[i0][r + d];
      }
    }
  }
  // heads that reach into other CTAs: one that began before this share, one that goes on after it
  const int head_lo = s_heads[0], head_hi = s_heads[heads - 1];
  const bool reaches_lo = s_piece[head_lo].from < lo, reaches_hi = s_piece[head_hi].from >= lo && s_piece[head_hi].to > hi;
  if (!reaches_lo && !reaches_hi) return;
  __threadfence();
  proxy_fence();
  __syncthreads();
  if (tid < 2 && (tid ? reaches_hi : reaches_lo)) {
    const Piece& pc = s_piece[tid ? head_hi : head_lo];
    const int c0 = cta_of(pc.from), n = cta_of(pc.to - 1) - c0 + 1;
    s_last[tid] = atomicAdd(g.done + c0, 1u) == (unsigned)(n - 1);
  }
  __syncthreads();
  int joins = 0;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    if (!(e ? reaches_hi : reaches_lo) || !s_last[e]) continue;
    const Piece& pc = s_piece[e ? head_hi : head_lo];
    const int c0 = cta_of(pc.from), n = cta_of(pc.to - 1) - c0 + 1;
    __threadfence();
    // the first CTA's result is its second one, the others' their first
    auto part_of = [&](int i) { return g.ws + (int64_t)((c0 + i) * 2 + (i == 0 ? 1 : 0)) * S::kPart; };
    // Weights of the results in shared memory, and after them as many results' sums at a time as there is room for:
    // loads in a loop would each wait for the one before.
    constexpr int kBytes = ROWS * D * 4, kPer = (kItems + S::kThreads - 1) / S::kThreads;
    const int at = (3 * n * ROWS * 4 + 127) / 128 * 128, room = (S::kSmem - at) / kBytes;
    float* const weight = reinterpret_cast<float*>(smem);
    float4 x[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    bool ok = true;
    for (int j0 = 0; j0 < n && ok; j0 += room, ++joins) {
      const int m = min(room, n - j0);
      __syncthreads();
      if (warp == 0) {
        proxy_fence();
        if (lane == 0) mbar_arrive_tx(bar_join, m * kBytes);
        __syncwarp();
        for (int i = lane; i < m; i += 32) bulk_load(smem_addr(smem) + at + i * kBytes, part_of(j0 + i), kBytes, bar_join);
      }
      if (j0 == 0) {
        for (int i = tid; i < n * ROWS; i += S::kThreads) {
          const float* p = part_of(i / ROWS) + ROWS * D + i % ROWS;
          weight[i] = __ldcg(p);
          weight[n * ROWS + i] = __ldcg(p + ROWS);
          weight[2 * n * ROWS + i] = __ldcg(p + 2 * ROWS);
        }
        __syncthreads();
        for (int r = warp; r < ROWS; r += S::kWarps) {
          float top = -INFINITY, te = 0.f, sum = 0.f;
          for (int i = lane; i < n; i += 32) {
            const float s = weight[i * ROWS + r], e = weight[(2 * n + i) * ROWS + r];
            if (heavier(s, e, top, te)) top = s, te = e;
          }
#pragma unroll 1
          for (int o = 16; o; o >>= 1) heavier_of(top, te, o);
          const float base = top == -INFINITY ? 0.f : top;
          for (int i = lane; i < n; i += 32) {
            const float f = ex2((weight[i * ROWS + r] - base) + (weight[(2 * n + i) * ROWS + r] - te));
            weight[i * ROWS + r] = f;
            sum = fmaf(f, weight[(n + i) * ROWS + r], sum);
          }
#pragma unroll 1
          for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
          if (lane == 0) s_inv[0][r] = sum == 0.f ? 0.f : 1.f / sum;
        }
        __syncthreads();
      }
      ok = wait_bar_warp(bar_join, joins & 1, abort_flag, 43, &g_kv_error, g.waits.limit_ns);
      if (!ok) wait_bar_quiet(bar_join, joins & 1, g.waits.limit_ns);
      ok = __syncthreads_and(ok);
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int idx = tid + u * S::kThreads, d = idx % D, r = idx / D * 4;
        if (idx >= kItems || !ok) break;
#pragma unroll 4
        for (int i = 0; i < m; ++i)
          add(x[u], *reinterpret_cast<const float4*>(&weight[(j0 + i) * ROWS + r]),
              *reinterpret_cast<const float4*>(smem + at + i * kBytes + (d * ROWS + r) * 4));
      }
    }
    const float lost = ok ? 0.f : __int_as_float(0x7FC00000);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int idx = tid + u * S::kThreads, d = idx % D, r = idx / D * 4;
      const float4 xs[1] = {make_float4(x[u].x + lost, x[u].y + lost, x[u].z + lost, x[u].w + lost)};
      if (idx < kItems) finish(pc, r, d, xs, s_inv[0]);
    }
    if (tid == 0) g.done[c0] = 0;
    __syncthreads();
  }
}

constexpr int kDevices = 64;

template <typename T, int D, int ROWS>
cudaError_t launch_shape(AttnArgs g, cudaStream_t st) {
  using S = Shape<T, D, ROWS>;
  constexpr int smem = S::kSmem;
  static_assert(S::kStage >= S::kPart * 4, "a partial result takes a tile's place");
  static_assert(S::kSmem >= 3 * kKvMaxCtas * ROWS * 4 + ROWS * D * 4, "a join has room for the weights and one result");
  auto kern = kv_stream_kernel<T, D, ROWS>;
  int dev = 0, sms = 0;
  static std::atomic<int> ready[kDevices];  // SMs of a device on which the kernel's shared memory is allowed
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices) sms = ready[dev].load(std::memory_order_acquire);
  if (sms == 0) {
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (sms > kKvMaxCtas) sms = kKvMaxCtas;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    if (dev < kDevices) ready[dev].store(sms, std::memory_order_release);
  }
  if ((e = kv_workspace(dev, st, (size_t)sms * (2 + S::kWarps) * S::kPart * sizeof(float), &g.done, &g.ws)) != cudaSuccess) return e;
  kern<<<sms, S::kThreads, smem, st>>>(g);
  return cudaGetLastError();
}

// Sixteen rows a tile only where there may be more than eight: one token of 64 sequences takes 193 us with eight and 266
// with sixteen, whose second half would be empty; of one sequence of 131072 keys 38 and 58.
template <typename T>
cudaError_t launch_t(const AttnArgs& g, cudaStream_t st) {
  const bool few = (g.a.max_q * g.a.group < g.few ? g.a.max_q * g.a.group : g.few) <= 8;
  switch (g.c.head_dim) {
    case 64: return few ? launch_shape<T, 64, 8>(g, st) : launch_shape<T, 64, 16>(g, st);
    case 128: return few ? launch_shape<T, 128, 8>(g, st) : launch_shape<T, 128, 16>(g, st);
    default: return launch_shape<T, 256, 8>(g, st);  // few_rows(256) is 8
  }
}

}  // namespace

cudaError_t launch_kv_attention(const KvCache& c, const KvBatch& b, const KvAttention& a, int dtype, cudaStream_t st) {
  // one sequence has all the tokens; of several, max_q bounds each
  const int64_t most = b.seqs == 1 || a.max_q > b.tokens ? b.tokens : a.max_q;
  const int few = few_rows(c.head_dim);
  const bool chunks = most * a.group > few;
  if (chunks) {
    // sequences that all have as many tokens as there may be: nothing is left for the other kernel, whose launch and look at
    // the lengths take 3 us (2 sequences of 4 tokens, 48 / 4 heads: 23 us with both, 20 with one)
    const bool all = b.tokens == b.seqs * most;
    const cudaError_t e = launch_kv_chunk(c, b, a, all ? 0 : few, dtype, st);
    if (e != cudaSuccess || all) return e;
  }
  AttnArgs g{c, b, a, waits(), chunks ? few : 0x7FFFFFFF, nullptr, nullptr};
  g.a.max_q = most;  // (the caller's may be any number; times the group it would overflow)
  return dtype == kBF16 ? launch_t<__nv_bfloat16>(g, st) : launch_t<__half>(g, st);
}

int read_kv_error() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(int)) != cudaSuccess) return -1;
  const int chunk = read_kv_chunk_error();
  if (chunk < 0) return -1;
  if (!v) v = chunk;
  if (v) {
    const int zero = 0;
    cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(int));
  }
  return v;
}

}  // namespace nvfp4
