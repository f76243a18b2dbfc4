// Appending to the 8-bit paged key/value cache, with the position rotation of
// queries and keys applied on the way (nvfp4_kv_append).
//
// A CTA takes one touched block of 16 tokens of one key/value head: its keys,
// its values and the queries of the heads that share it, so the rotation's
// cosines are fetched once for all of them and the block's scales need no
// exchange between CTAs. Per block:
//   k' = rotation of k by the token's position, in f32;
//   e  = max(exponent of the new tokens' largest |k'|, the old exponent when
//        the block already holds older tokens);
//   older codes *= 2^(e_old - e), new codes = e4m3(k' * 2^-e), the rest 0;
// and the same for v, unrotated. Everything is read once and written once.
//
// Bound by bytes: 16384 tokens of 32 query and 16 key/value heads of 128
// bf16 channels move 478 MB in 95 us, 5.0 TB/s, 74% of a plain copy's rate
// (a CTA's load latency, with 28 warps an SM to cover it, takes the rest). A
// single token takes 3.3 us, most of them the launch. Times here are those of
// captured graphs; a call from the Python binding takes 20 us at least, its
// host side.
#include "nvfp4_kv.cuh"

namespace nvfp4 {
namespace {

using namespace kv;

struct AppendArgs {
  KvCache c;
  KvBatch b;
  KvAppend a;
};

// The two 8-channel pieces that thread i of a row takes: channels A..A+7 and
// B..B+7, and whether they are a rotated pair (pair index 8 i .. 8 i + 7).
// "half": channel d turns with d + rotary / 2; "interleaved": 2 j with 2 j + 1
// (the pieces are then 16 consecutive channels).
struct Pieces {
  int A, B;
  bool turned;
};
__device__ __forceinline__ Pieces pieces(int i, int rotary, int interleaved) {
  Pieces p;
  p.turned = 16 * i < rotary;
  if (!p.turned || interleaved) {
    p.A = 16 * i;
    p.B = 16 * i + 8;
  } else {
    p.A = 8 * i;
    p.B = rotary / 2 + 8 * i;
  }
  return p;
}

struct Turn {
  float c[8], s[8];
};
// Row pos of the cosine and sine tables, pairs 8 i .. 8 i + 7; NaN outside the
// table, which marks whatever is turned by it.
__device__ __forceinline__ void load_turn(Turn& t, const KvAppend& a, int pos, int i) {
  if (pos < a.positions) {
    const int64_t o = (int64_t)pos * (a.rotary / 2) + 8 * i;
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(a.cos + o)), c1 = __ldg(reinterpret_cast<const float4*>(a.cos + o) + 1);
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(a.sin + o)), s1 = __ldg(reinterpret_cast<const float4*>(a.sin + o) + 1);
    t.c[0] = c0.x, t.c[1] = c0.y, t.c[2] = c0.z, t.c[3] = c0.w, t.c[4] = c1.x, t.c[5] = c1.y, t.c[6] = c1.z, t.c[7] = c1.w;
    t.s[0] = s0.x, t.s[1] = s0.y, t.s[2] = s0.z, t.s[3] = s0.w, t.s[4] = s1.x, t.s[5] = s1.y, t.s[6] = s1.z, t.s[7] = s1.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) t.c[j] = t.s[j] = __int_as_float(0x7FC00000);
  }
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack2<T>(u[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
}

// The products and the sum are rounded one by one (no fused multiply-add), so
// that any plain f32 evaluation of the formula gives the same bits, and with
// them the same codes.
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  const float b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
  y = b;
}
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const Turn& t, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      turn_pair(a[2 * j], a[2 * j + 1], t.c[j], t.s[j]);
      turn_pair(b[2 * j], b[2 * j + 1], t.c[4 + j], t.s[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], t.c[j], t.s[j]);
  }
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// Threads of an SM that the registers are kept for: all the loads of a block go out at once and the kernel waits for them
// most of the time. 512, 640, 768, 896 and 1024 threads (the last leave 64 registers, too few): 16384 tokens
// take 113, 99, 104, 95 and 114 us, 7 chunks of 33 to 1500 tokens with 256 channels 20.8, 20.7, 18.4, 18.4 and 21.2 us.
constexpr int kThreadsAnSm = 896;

// D threads. Item blockIdx.x is a touched block of some sequence: sequence b
// starts at item q_offsets[b] / 16 + 2 b (n tokens touch at most n / 16 + 2
// blocks, so the ranges never overlap; items past a sequence's last block
// have nothing to do). Without q_offsets every sequence touches one block.
template <typename T, int D>
__global__ void __launch_bounds__(D, kThreadsAnSm / D) kv_append_kernel(const AppendArgs g) {
  const KvCache& c = g.c;
  const KvAppend& a = g.a;
  const int tid = threadIdx.x, head = blockIdx.y, lane = tid & 31, warp = tid >> 5;
  __shared__ float s_amax[2][D / 32];
  __shared__ uint32_t s_bad[D / 32];

  int b = blockIdx.x, nth = 0;
  Seq sq;
  if (g.b.q_offsets) {
    // every warp looks for the item's sequence by itself: the last one that starts at the item or before
    b = -1;
    for (int64_t j0 = 0; j0 < g.b.seqs; j0 += 32) {
      const int64_t j = j0 + lane;
      Seq x{0, 0, 0};
      bool before = false;
      if (j < g.b.seqs) {
        x = sequence(g.b, (int)j);
        before = (int64_t)(g.b.q_offsets[j] / kBlock) + 2 * j <= (int64_t)blockIdx.x;
      }
      const int k = __popc(__ballot_sync(0xFFFFFFFFu, before));
      if (k > 0) {
        b = (int)j0 + k - 1;
        sq.first = __shfl_sync(0xFFFFFFFFu, x.first, k - 1);
        sq.n = __shfl_sync(0xFFFFFFFFu, x.n, k - 1);
        sq.length = __shfl_sync(0xFFFFFFFFu, x.length, k - 1);
      }
      if (k < 32) break;
    }
    if (b < 0) return;
    nth = (int)blockIdx.x - (sq.first / kBlock + 2 * b);
  } else {
    sq = sequence(g.b, b);
  }
  const int start = sq.length - sq.n;  // position of the first new token
  const int blk = (start < 0 ? 0 : start / kBlock) + nth;
  // tokens without a place (more new tokens than the length says) are skipped
  const int lo = start > blk * kBlock ? start - blk * kBlock : 0;       // first new token's slot in the block
  const int hi = min(sq.length - blk * kBlock, kBlock);                   // one past the last one's
  if (nth < 0 || hi <= lo || sq.n == 0) return;
  const int page = blk / (int)c.blocks, inner = blk % (int)c.blocks;
  const int32_t pg = g.b.page_table[(int64_t)b * g.b.table_stride + page];
  const bool there = pg >= 0 && (int64_t)pg < c.pages;
  const int64_t at = ((int64_t)(there ? pg : 0) * c.kv_heads + head) * c.blocks + inner;
  uint8_t* kb = c.k + at * (kBlock * D);
  uint8_t* vb = c.v + at * (kBlock * D);
  const bool older = lo > 0;
  const int ek_old = older && there ? (int)c.k_exp[at] - 127 : kExpMin, ev_old = older && there ? (int)c.v_exp[at] - 127 : kExpMin;
  // token of slot r: row first + blk * 16 + r - start of the call's tensors
  const int64_t row0 = (int64_t)sq.first + (int64_t)blk * kBlock - start;

  // keys: thread (r, i) holds two 8-channel pieces of token r
  const int r = tid / (D / 16), i = tid % (D / 16);
  const Pieces pc = pieces(i, a.rotary, a.interleaved);
  const bool fresh = r >= lo && r < hi;
  const bool turned = pc.turned;
  uint4 kwa = make_uint4(0, 0, 0, 0), kwb = kwa;
  Turn t;
  uint2 oa = make_uint2(0, 0), ob = make_uint2(0, 0);
  if (fresh) {
    const T* kr = static_cast<const T*>(a.k) + (row0 + r) * a.k_stride + (int64_t)head * D;
    kwa = *reinterpret_cast<const uint4*>(kr + pc.A);
    kwb = *reinterpret_cast<const uint4*>(kr + pc.B);
    if (turned) load_turn(t, a, blk * kBlock + r, i);
  } else if (r < lo && there) {
    oa = *reinterpret_cast<const uint2*>(kb + k_place<D>(r, pc.A));
    ob = *reinterpret_cast<const uint2*>(kb + k_place<D>(r, pc.B));
  }
  // values: lanes 2 j and 2 j + 1 hold channels 2 ch and 2 ch + 1, tokens 0..7 and 8..15
  const int ch = tid >> 1, half = tid & 1;
  uint32_t vw[8];
  const T* vr = static_cast<const T*>(a.v) + (int64_t)head * D + 2 * ch;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int tok = 8 * half + j;
    vw[j] = tok >= lo && tok < hi ? *reinterpret_cast<const uint32_t*>(vr + (row0 + tok) * a.v_stride) : 0u;
  }
  uint4 vold = make_uint4(0, 0, 0, 0);
  if (older && there) vold = *reinterpret_cast<const uint4*>(vb + tid * 16);

  // queries: thread (r, i) takes token lo + r % rows and every step-th head from r / rows on, so that a single token's
  // heads are spread over the threads; the first head's loads go out before anything is waited for
  const int rows = hi - lo, group = (int)a.group, step = kBlock / rows;
  const int qr = lo + r % rows, h0 = r / rows;
  const bool asks = a.q && h0 < step;
  const T* qrow = static_cast<const T*>(a.q) + (row0 + qr) * a.q_stride + (int64_t)head * group * D;
  uint4 qwa = make_uint4(0, 0, 0, 0), qwb = qwa;
  auto fetch = [&](int h) {
    if (asks && h < group) {
      qwa = *reinterpret_cast<const uint4*>(qrow + (int64_t)h * D + pc.A);
      qwb = *reinterpret_cast<const uint4*>(qrow + (int64_t)h * D + pc.B);
    }
  };
  fetch(h0);

  float ka[8], kc[8];
  unpack8<T>(kwa, ka);
  unpack8<T>(kwb, kc);
  if (fresh && turned) rotate(ka, kc, t, a.interleaved);
  float km = 0.f, vm = 0.f;
  uint32_t bad = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (finite(ka[j])) km = fmaxf(km, fabsf(ka[j])); else bad |= 1u << r;
    if (finite(kc[j])) km = fmaxf(km, fabsf(kc[j])); else bad |= 1u << r;
    const float2 f = unpack2<T>(vw[j]);
    if (finite(f.x)) vm = fmaxf(vm, fabsf(f.x)); else bad |= 1u << (8 * half + j);
    if (finite(f.y)) vm = fmaxf(vm, fabsf(f.y)); else bad |= 1u << (8 * half + j);
  }
  // non-negative floats order as their bits
  km = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(km)));
  vm = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vm)));
  bad = __reduce_or_sync(0xFFFFFFFFu, bad);
  if (lane == 0) s_amax[0][warp] = km, s_amax[1][warp] = vm, s_bad[warp] = bad;
  __syncthreads();
  km = vm = 0.f;
  bad = 0;
#pragma unroll
  for (int w = 0; w < D / 32; ++w) km = fmaxf(km, s_amax[0][w]), vm = fmaxf(vm, s_amax[1][w]), bad |= s_bad[w];
  const int ek = max(scale_exponent(km), ek_old), ev = max(scale_exponent(vm), ev_old);

  if (there) {
    const float ks = exp2i(-ek), vs = exp2i(-ev);
    uint8_t *pa = kb + k_place<D>(r, pc.A), *pb = kb + k_place<D>(r, pc.B);
    if (r >= lo) {  // new tokens; zeros beyond them
      uint2 na, nb;
      if (bad >> r & 1) {
        na = nb = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      } else {
        na = make_uint2(e4m3x4(ka[0] * ks, ka[1] * ks, ka[2] * ks, ka[3] * ks), e4m3x4(ka[4] * ks, ka[5] * ks, ka[6] * ks, ka[7] * ks));
        nb = make_uint2(e4m3x4(kc[0] * ks, kc[1] * ks, kc[2] * ks, kc[3] * ks), e4m3x4(kc[4] * ks, kc[5] * ks, kc[6] * ks, kc[7] * ks));
      }
      *reinterpret_cast<uint2*>(pa) = na;
      *reinterpret_cast<uint2*>(pb) = nb;
    } else if (ek > ek_old) {
      const float up = exp2i(ek_old - ek);
      *reinterpret_cast<uint2*>(pa) = make_uint2(rescale4(oa.x, up), rescale4(oa.y, up));
      *reinterpret_cast<uint2*>(pb) = make_uint2(rescale4(ob.x, up), rescale4(ob.y, up));
    }
    uint32_t v0[2] = {0, 0}, v1[2] = {0, 0};  // channels 2 ch and 2 ch + 1, this lane's eight tokens
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 f0 = unpack2<T>(vw[j]), f1 = unpack2<T>(vw[j + 1]);
      if (bad >> (8 * half + j) & 1) f0 = make_float2(0.f, 0.f);
      if (bad >> (8 * half + j + 1) & 1) f1 = make_float2(0.f, 0.f);
      v0[j / 4] |= e4m3x2(f0.x * vs, f1.x * vs) << (8 * (j & 2));
      v1[j / 4] |= e4m3x2(f0.y * vs, f1.y * vs) << (8 * (j & 2));
    }
    // the even lane takes all tokens of channel 2 ch, the odd one of 2 ch + 1
    const uint32_t x0 = __shfl_xor_sync(0xFFFFFFFFu, half ? v0[0] : v1[0], 1);
    const uint32_t x1 = __shfl_xor_sync(0xFFFFFFFFu, half ? v0[1] : v1[1], 1);
    uint32_t w[4] = {half ? x0 : v0[0], half ? x1 : v0[1], half ? v1[0] : x0, half ? v1[1] : x1};
    if (older) {
      const uint32_t old[4] = {vold.x, vold.y, vold.z, vold.w};
      const float up = exp2i(ev_old - ev);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int keep = min(max(lo - 4 * j, 0), 4);  // older tokens in this word
        const uint32_t m = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
        w[j] = (w[j] & ~m) | ((ev > ev_old ? rescale4(old[j], up) : old[j]) & m);
      }
    }
    *reinterpret_cast<uint4*>(vb + tid * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (tid == 0) c.k_exp[at] = (uint8_t)(ek + 127), c.v_exp[at] = (uint8_t)(ev + 127);
  }

  if (!asks) return;
  if (turned && (rows < kBlock)) load_turn(t, a, blk * kBlock + qr, i);  // else the thread's own key's
  T* orow = static_cast<T*>(a.q_out) + (row0 + qr) * a.q_out_stride + (int64_t)head * group * D;
  for (int h = h0; h < group; h += step) {
    float x[8], y[8];
    unpack8<T>(qwa, x);
    unpack8<T>(qwb, y);
    fetch(h + step);
    if (turned) rotate(x, y, t, a.interleaved);
    store8(orow + (int64_t)h * D + pc.A, x);
    store8(orow + (int64_t)h * D + pc.B, y);
  }
}

template <typename T>
cudaError_t launch_t(const AppendArgs& g, cudaStream_t st) {
  const int64_t items = g.b.q_offsets ? g.b.tokens / kBlock + 2 * g.b.seqs : g.b.seqs;
  const dim3 grid((unsigned)items, (unsigned)g.c.kv_heads);
  if (g.c.head_dim == 64)
    kv_append_kernel<T, 64><<<grid, 64, 0, st>>>(g);
  else if (g.c.head_dim == 128)
    kv_append_kernel<T, 128><<<grid, 128, 0, st>>>(g);
  else
    kv_append_kernel<T, 256><<<grid, 256, 0, st>>>(g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvCache& c, const KvBatch& b, const KvAppend& a, int dtype, cudaStream_t st) {
  const AppendArgs g{c, b, a};
  return dtype == kBF16 ? launch_t<__nv_bfloat16>(g, st) : launch_t<__half>(g, st);
}

}  // namespace nvfp4
