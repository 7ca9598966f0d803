// The 4-bit KV cache's bookkeeping and storage: block tables and slot maps from request
// lengths, the append that quantizes new keys and values into the paged cache, and the read
// that gives stored values back. The quantizer's readings are those of wq_quantize_rtn_g128
// ("DL S067 - Quantization", sections 1-2): one S', Z per group along the head dimension.
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/wq.h"
#include "common.cuh"
#include "kv4.h"

namespace wq {
namespace {

// ------------------------------------------------------------------ tables and slot maps

constexpr int kTabThreads = 512;

// Inclusive scan of (a, b) over the block; totals in ta, tb.
__device__ __forceinline__ void block_scan2(int64_t& a, int64_t& b, int64_t& ta, int64_t& tb,
                                            int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    part[warp][0] = a;
    part[warp][1] = b;
  }
  __syncthreads();
  int64_t sa = 0, sb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) {
      sa += part[w][0];
      sb += part[w][1];
    }
    ta += part[w][0];
    tb += part[w][1];
  }
  a += sa;
  b += sb;
  __syncthreads();
}

// Every CTA scans the lengths of all requests (two integers each, from L2) and then serves its
// own range of slots and of newly taken blocks, so one launch does without a scan across CTAs.
// Bound by the latency of that chain of loads and barriers, not by bytes.
__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(Kv4TablesArgs a) {
  __shared__ int64_t part[kTabThreads / 32][2];
  __shared__ int s_tok[kTabThreads + 1], s_blk[kTabThreads + 1], s_ctx[kTabThreads];
  const int bs = 1 << a.block_log2;
  const int per = (a.n_slots + gridDim.x - 1) / gridDim.x;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * per;
  const int64_t hi = lo + per < a.n_slots ? lo + per : a.n_slots;
  int64_t tok0 = 0, blk0 = 0;  // totals of the requests before this round's
  bool bad = false;
  for (int r0 = 0; r0 < a.requests; r0 += kTabThreads) {
    const int n = a.requests - r0 < kTabThreads ? a.requests - r0 : kTabThreads;
    const int t = threadIdx.x;
    int ctx = 0, add = 0;
    if (t < n) {
      ctx = a.ctx_lens[r0 + t];
      add = a.new_lens[r0 + t];
      if (ctx < 0 || add < 0 || ctx > 0x7fffffff - bs - add) {  // no such request: it holds nothing
        bad = true;
        ctx = add = 0;
      }
    }
    const int kv = ctx + add;
    const int held = (ctx + bs - 1) >> a.block_log2, need = (kv + bs - 1) >> a.block_log2;
    int64_t tok = add, blk = need - held, tt, tb;
    block_scan2(tok, blk, tt, tb, part);
    // positions are relative to this round's start: they stay below 2^31 where they are used
    s_tok[t + 1] = static_cast<int>(tok < 0x7fffffff ? tok : 0x7fffffff);
    s_blk[t + 1] = static_cast<int>(blk < 0x7fffffff ? blk : 0x7fffffff);
    s_ctx[t] = ctx;
    if (t == 0) s_tok[0] = s_blk[0] = 0;
    if (blockIdx.x == 0 && t < n) {
      const int64_t e = tok0 + tok;
      a.q_starts[r0 + t + 1] = static_cast<int>(e < 0x7fffffff ? e : 0x7fffffff);
      a.kv_lens[r0 + t] = kv;
      if (r0 + t == 0) a.q_starts[0] = 0;
      if (need > a.width) bad = true;
    }
    __syncthreads();
    // index of the last request of this round whose first entry is <= v
    auto find = [&](const int* s, int v) {
      int l = 0, h = n;  // s[l] <= v < s[h]
      while (h - l > 1) {
        const int m = (l + h) >> 1;
        if (s[m] <= v) l = m; else h = m;
      }
      return l;
    };
    // newly taken blocks, spread over the whole grid, as far as there are free ones (wild lengths
    // would ask for 2^36 of them)
    const int64_t there = a.n_free - blk0 < tb ? a.n_free - blk0 : tb;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kTabThreads + t; i < there;
         i += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      const int k = find(s_blk, static_cast<int>(i));
      const int place = ((s_ctx[k] + bs - 1) >> a.block_log2) + static_cast<int>(i) - s_blk[k];
      if (place < a.width)
        a.tables[(r0 + k) * a.ld_tables + place] = a.free_blocks[blk0 + i];
      else
        bad = true;
    }
    // this CTA's slots
    const int64_t s0 = lo > tok0 ? lo : tok0, s1 = hi < tok0 + tt ? hi : tok0 + tt;
    for (int64_t i = s0 + t; i < s1; i += kTabThreads) {
      const int rel = static_cast<int>(i - tok0);
      const int k = find(s_tok, rel);
      const int pos = s_ctx[k] + rel - s_tok[k];
      const int place = pos >> a.block_log2;
      const int held_k = (s_ctx[k] + bs - 1) >> a.block_log2;
      int b = -1;
      if (place < a.width) {
        if (place < held_k) {
          b = a.tables[(r0 + k) * a.ld_tables + place];
        } else {
          const int64_t f = blk0 + s_blk[k] + (place - held_k);
          if (f < a.n_free) b = a.free_blocks[f];
        }
      }
      const bool ok = b >= 0 && b <= (0x7fffffff >> a.block_log2) - 1;
      if (!ok) bad = true;
      a.slots[i] = ok ? (b << a.block_log2) + (pos & (bs - 1)) : -1;
    }
    tok0 += tt;
    blk0 += tb;
    __syncthreads();
  }
  if (tok0 > a.n_slots || blk0 > a.n_free) bad = true;
  for (int64_t i = (lo > tok0 ? lo : tok0) + threadIdx.x; i < hi; i += kTabThreads) a.slots[i] = -1;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (a.requests == 0) a.q_starts[0] = 0;
    a.taken[0] = static_cast<int>(blk0 < a.n_free ? blk0 : a.n_free);
  }
  if (bad) set_status(a.status, kStRange);
}

// ------------------------------------------------------------------------ append and read

// Two 16-bit floats of a word -> floats.
template <bool kBf16>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if (kBf16) return make_float2(bf16_lo(w), bf16_hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Codes of 8 weights v of a finite group (|v / S'| < 32 then), as round-half-even of the exact
// quotient plus Z, clipped to [0, 15], without a test per weight. With w = M_w 2^a and
// S' = M_s 2^b (M_w < 2^11 for bf16 and binary16, M_s < 2^11, both odd) the quotient is either a
// half-integer or more than 2^-12 away from every half-integer: for a >= b - 1 the difference
// has the denominator 2 M_s; for d = b - a > 1 a quotient near k + 1/2 means
// M_w ~ (2k + 1) M_s 2^(d-1), so the denominator M_s 2^d is at most 2^12. The product with
// RN(1/S') is within 2^-19 of it, and one FMA onto the 2^-13 grid (floats in [1024, 2048)) puts
// a half-integer on itself and leaves the others on their side. Adding 1.5 2^23 - 1536 + Ze, Ze
// the zero-point rounded up to even, rounds to an integer with ties to even k; the low byte is
// code + (Z & 1). The clipping is left out where the caller knows that no code leaves [0, 15].
template <bool kClip>
__device__ __forceinline__ uint32_t encode8_snap(const float2 (&v)[4], float inv_s, int z) {
  const float z1 = static_cast<float>(z & 1);
  const float lo = 12582912.0f + z1, hi = lo + 15.0f;
  const float2 inv2 = make_float2(inv_s, inv_s), g2 = make_float2(1536.0f, 1536.0f);
  const float cz = 12581376.0f + (static_cast<float>(z) + z1);
  const float2 c2 = make_float2(cz, cz);
  uint32_t t[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __fadd2_rn(__ffma2_rn(v[j], inv2, g2), c2);
    t[2 * j] = __float_as_uint(kClip ? fminf(fmaxf(x.x, lo), hi) : x.x);
    t[2 * j + 1] = __float_as_uint(kClip ? fminf(fmaxf(x.y, lo), hi) : x.y);
  }
  const uint32_t ev = __byte_perm(__byte_perm(t[0], t[2], 0x0040), __byte_perm(t[4], t[6], 0x0040), 0x5410);
  const uint32_t od = __byte_perm(__byte_perm(t[1], t[3], 0x0040), __byte_perm(t[5], t[7], 0x0040), 0x5410);
  return ev + (od << 4) - (z & 1u) * 0x11111111u;
}

// The code of a weight before it is clipped, by the same steps.
__device__ __forceinline__ float code_level(float v, float inv_s, int z) {
  const int odd = z & 1;
  const float t = __fadd_rn(__fmaf_rn(v, inv_s, 1536.0f), 12581376.0f + static_cast<float>(z + odd));
  return t - (12582912.0f + static_cast<float>(odd));
}

// How lanes share the rows of one kind (K or V) so that the stored order needs no exchange, or
// one, between lanes: a lane's words (of 8 dimensions) are those that stand side by side in the
// cache. K: lane c of 4 has the words 4 u + c, D/8 bytes at c D/8. V: lane h + 2 k of D/32 has the
// words 2 (4 k + u) + h; a transpose of its 4 x 4 bytes gives for each byte column g = 4 h + b the
// rows 4 k .. 4 k + 3. (One word a lane with its bytes moved by shuffles, four words stored apart:
// 293 instructions for 256 elements of an append, 163 of a read, which bounded both.)
template <int D, int G, bool kV>
struct Share {
  static constexpr int kLanes = kV ? D / 32 : 4;      // lanes of a row
  static constexpr int kWords = D / 8 / kLanes;       // words of a lane
  static constexpr int kRows = 32 / kLanes;           // rows of a warp
  // groups of a lane, and the lanes that a group lies in, which hold the same groups
  static constexpr int kGroups = kV ? (G >= 64 ? 1 : 2) : D / G;
  static constexpr int kShared = kV ? (G == 128 ? 4 : 2) : 4;
  static_assert(kWords % kGroups == 0 && kGroups <= kShared, "");
  __device__ static int dim(int l, int u) {           // first dimension of lane l's word u
    return kV ? 8 * (2 * (4 * (l >> 1) + u) + (l & 1)) : 8 * (4 * u + l);
  }
  __device__ static int first_group(int l) { return kV && G < 128 ? (l >> 1) * kGroups : 0; }
};

// 4 x 4 bytes: word i's byte b becomes word b's byte i. Its own inverse.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[0], w[1], 0x7362);
  const uint32_t c = __byte_perm(w[2], w[3], 0x5140), d = __byte_perm(w[2], w[3], 0x7362);
  w[0] = __byte_perm(a, c, 0x5410);
  w[1] = __byte_perm(a, c, 0x7632);
  w[2] = __byte_perm(b, d, 0x5410);
  w[3] = __byte_perm(b, d, 0x7632);
}

// A V row of 128: lane l and lane l ^ 2 hold the halves of the same byte columns 4 h + b in word
// b; after join_halves lane l holds columns 4 h + 2 k and 4 h + 2 k + 1 whole, in two words each.
__device__ __forceinline__ void join_halves(uint32_t (&w)[4], int l) {
  const bool k = l & 2;
  const uint32_t a = __shfl_xor_sync(0xffffffffu, k ? w[0] : w[2], 2);
  const uint32_t b = __shfl_xor_sync(0xffffffffu, k ? w[1] : w[3], 2);
  const uint32_t w1 = w[1];
  w[0] = k ? a : w[0];
  w[1] = k ? w[2] : a;
  w[2] = k ? b : w1;
  w[3] = k ? w[3] : b;
}
__device__ __forceinline__ void split_halves(uint32_t (&w)[4], int l) {
  const bool k = l & 2;
  const uint32_t a = __shfl_xor_sync(0xffffffffu, k ? w[0] : w[1], 2);
  const uint32_t b = __shfl_xor_sync(0xffffffffu, k ? w[2] : w[3], 2);
  const uint32_t w1 = w[1];
  w[0] = k ? a : w[0];
  w[1] = k ? b : w[2];
  w[2] = k ? w1 : a;
  w[3] = k ? w[3] : b;
}

// Byte offset within a stored row of lane l's bytes.
template <int D, bool kV>
__device__ __forceinline__ int lane_place(int l, int t) {
  if (!kV) return l * (D / 8);
  if (D == 64) return 16 * l;
  return (32 * (l & 1) + 8 * (l & 2)) ^ (t & 2 ? 32 : 0);
}

// Rows (token, head) in the order of the input, stepped through without divisions.
struct Rows {
  int64_t tok, step_tok;
  int head, step_head, heads;
  __device__ Rows(int kv_heads, int64_t first, int64_t step) : heads(kv_heads) {
    tok = first / heads;
    head = static_cast<int>(first - tok * heads);
    step_tok = step / heads;
    step_head = static_cast<int>(step - step_tok * heads);
  }
  __device__ void next() {
    tok += step_tok;
    head += step_head;
    if (head >= heads) {
      head -= heads;
      ++tok;
    }
  }
};

// Packed 16-bit minimum and maximum; a NaN propagates.
template <bool kBf16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kBf16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  if (kBf16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The group's range is reduced in 16 bits, in the lane first, then over the lanes that share it.
// S', Z and the codes are decided exactly, as in quantize.cu; the lanes that share groups decide
// one each and hand the results round.
// Codes are clipped only in warps with a group whose end codes leave [0, 15], as there (rare: a
// tie at both ends, or a subnormal S').
// Bytes: 2 an element in, D/2 + 4 D/g a row out: 16384 tokens of 8 heads of 128 in 20.9 us, 4.1
// TB/s; 69 % of the issue slots, so bound by instructions as much as by memory (50 us with a word a lane; 22.9 with every code clipped, 25 if two rows a lane share the
// decisions too).
template <int D, int G, bool kBf16, bool kV>
__device__ __forceinline__ void append_rows(const Kv4AppendArgs& a) {
  using S = Share<D, G, kV>;
  const Kv4Cache c = a.cache;
  const int lane = threadIdx.x & 31, l = lane % S::kLanes;
  const int share = l % S::kShared, share0 = lane - share;
  constexpr int kPer = S::kWords / S::kGroups;  // words of a group
  const int64_t limit = c.num_blocks << c.block_log2;
  const int64_t chunk_bytes = c.chunk_bytes();
  const int codes = c.block * (D / 2);
  const uint16_t* base = kV ? a.V : a.K;
  const int64_t s_tok = kV ? a.v_tok : a.k_tok, s_head = kV ? a.v_head : a.k_head;
  bool range = false, nonfinite = false;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  Rows p(c.kv_heads, warp * S::kRows + lane / S::kLanes, warps * S::kRows);
  while (__any_sync(0xffffffffu, p.tok < a.tokens)) {
    const bool in = p.tok < a.tokens;
    const int head = p.head;
    const uint16_t* row = base + (in ? p.tok * s_tok + p.head * s_head : 0) + S::dim(l, 0);
    uint4 x[S::kWords];
#pragma unroll
    for (int u = 0; u < S::kWords; ++u)
      x[u] = in ? ld_stream_u4(row + (S::dim(0, u) - S::dim(0, 0))) : make_uint4(0, 0, 0, 0);
    const int slot = in ? __ldg(a.slots + p.tok) : -1;
    p.next();
    uint32_t mn = 0, mx = 0;  // the range of this lane's group
#pragma unroll
    for (int g = 0; g < S::kGroups; ++g) {
      uint32_t lo = x[g * kPer].x, hi = lo;
#pragma unroll
      for (int u = g * kPer; u < (g + 1) * kPer; ++u) {
        lo = min2<kBf16>(min2<kBf16>(lo, x[u].x), min2<kBf16>(min2<kBf16>(x[u].y, x[u].z), x[u].w));
        hi = max2<kBf16>(max2<kBf16>(hi, x[u].x), max2<kBf16>(max2<kBf16>(x[u].y, x[u].z), x[u].w));
      }
#pragma unroll
      for (int o = 1; o < S::kShared; o <<= 1) {
        lo = min2<kBf16>(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max2<kBf16>(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      const bool own = share % S::kGroups == g;
      mn = own ? lo : mn;
      mx = own ? hi : mx;
    }
    const float2 l2 = widen<kBf16>(mn), h2 = widen<kBf16>(mx);
    const float least = fmin_nan(0.0f, fmin_nan(l2.x, l2.y));
    const float most = fmax_nan(0.0f, fmax_nan(h2.x, h2.y));
    const AsymScale sz = asym_scale_zero(least, most);
    const uint32_t mine = sz.bad ? 0x80003C00u : sz.sbits | static_cast<uint32_t>(sz.z) << 16;
    // codes grow with the weights: none is clipped unless those of the ends are
    const int zero = static_cast<int>(sz.z);
    const bool clip = __any_sync(0xffffffffu,
                                 !sz.bad && (code_level(least, sz.inv_s, zero) < 0.0f ||
                                             code_level(most, sz.inv_s, zero) > 15.0f));
    uint32_t word[S::kWords], got = mine;
    float inv_s = sz.inv_s;
    auto encode = [&](auto clipped) {
#pragma unroll
      for (int u = 0; u < S::kWords; ++u) {
        if (S::kGroups > 1 && u % kPer == 0) {
          got = __shfl_sync(0xffffffffu, mine, share0 + u / kPer);
          inv_s = __shfl_sync(0xffffffffu, sz.inv_s, share0 + u / kPer);
        }
        const float2 f[4] = {widen<kBf16>(x[u].x), widen<kBf16>(x[u].y), widen<kBf16>(x[u].z),
                             widen<kBf16>(x[u].w)};
        word[u] = got >> 31 ? 0u
                            : encode8_snap<decltype(clipped)::value>(f, inv_s, (got >> 16) & 15);
      }
    };
    if (clip) encode(std::true_type());
    else encode(std::false_type());
    if constexpr (kV) {
      transpose4(word);
      if (D == 128) join_halves(word, l);
    }
    if (slot >= limit) range = true;
    if (slot < 0 || slot >= limit) continue;
    const int t = slot & (c.block - 1);
    uint8_t* chunk = c.data +
        (static_cast<int64_t>(slot >> c.block_log2) * c.kv_heads + head) * chunk_bytes;
    uint8_t* dst = chunk + (kV ? codes : 0) + t * (D / 2) + lane_place<D, kV>(l, t);
    if constexpr (S::kWords == 4)
      *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
    if (share < S::kGroups) {
      reinterpret_cast<uint32_t*>(chunk + 2 * codes)[((kV ? c.block : 0) + t) * (D / G) +
                                                     S::first_group(l) + share] =
          (mine & 0xFFFFu) | f32_to_f16_bits(static_cast<float>((mine >> 16) & 15)) << 16;
      if (sz.bad) nonfinite = true;
    }
  }
  if (range) set_status(a.status, kStRange);
  if (nonfinite) set_status(a.status, kStNonFinite);
}

// CTAs of 4 warps; at most 16 of a kind for each SM, then each goes on to further rows (65536
// tokens of 8 heads of 128, append with every code clipped and fp32 read: 74 and 106 us; with 8:
// 78 and 128; with 4: 81 and 112).
constexpr int kRowThreads = 128, kRowCtas = 16;

// blockIdx.y: 0 the keys, 1 the values.
template <int D, int G, bool kBf16>
__global__ void __launch_bounds__(kRowThreads) append_kernel(Kv4AppendArgs a) {
  if (blockIdx.y == 0) append_rows<D, G, kBf16, false>(a);
  else append_rows<D, G, kBf16, true>(a);
}

// The inverse, with the lanes and words of the append: values S'(q - Z), exact in fp32, or
// rounded once to 16 bits; slot < 0 gives zeros. The slots of the next rows are loaded ahead.
// Bound by HBM: 16384 tokens of 8 heads of 128 to fp32 in 29 us, 5.3 TB/s (39 us with a word a
// lane; 51 us where each lane stores its own 32 bytes in two halves), to 16 bits in 17 us.
template <int D, int G, int kOut, bool kV>  // kOut: WQ_F32, WQ_BF16, WQ_F16
__device__ __forceinline__ void read_rows(const Kv4ReadArgs& a) {
  using S = Share<D, G, kV>;
  const Kv4Cache c = a.cache;
  const int lane = threadIdx.x & 31, l = lane % S::kLanes;
  const int64_t limit = c.num_blocks << c.block_log2;
  const int64_t chunk_bytes = c.chunk_bytes();
  const int codes = c.block * (D / 2);
  bool range = false;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  Rows p(c.kv_heads, warp * S::kRows + lane / S::kLanes, warps * S::kRows);
  int next = p.tok < a.tokens ? __ldg(a.slots + p.tok) : -1;
  while (__any_sync(0xffffffffu, p.tok < a.tokens)) {
    const bool in = p.tok < a.tokens;
    const int64_t row = p.tok * c.kv_heads + p.head;
    const int head = p.head;
    int slot = next;
    p.next();
    next = p.tok < a.tokens ? __ldg(a.slots + p.tok) : -1;
    if (slot >= limit) {
      range = true;
      slot = -1;
    }
    uint32_t word[S::kWords], sz[S::kGroups];
#pragma unroll
    for (int u = 0; u < S::kWords; ++u) word[u] = 0;
#pragma unroll
    for (int g = 0; g < S::kGroups; ++g) sz[g] = 0;
    if (slot >= 0) {
      const int t = slot & (c.block - 1);
      const uint8_t* chunk =
          c.data + (static_cast<int64_t>(slot >> c.block_log2) * c.kv_heads + head) * chunk_bytes;
      const uint8_t* src = chunk + (kV ? codes : 0) + t * (D / 2) + lane_place<D, kV>(l, t);
      if constexpr (S::kWords == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
        word[0] = v.x, word[1] = v.y, word[2] = v.z, word[3] = v.w;
      } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
        word[0] = v.x, word[1] = v.y;
      }
#pragma unroll
      for (int g = 0; g < S::kGroups; ++g)
        sz[g] = __ldg(reinterpret_cast<const uint32_t*>(chunk + 2 * codes) +
                      ((kV ? c.block : 0) + t) * (D / G) + S::first_group(l) + g);
    }
    if constexpr (kV) {
      if (D == 128) split_halves(word, l);
      transpose4(word);
    }
#pragma unroll
    for (int u = 0; u < S::kWords; ++u) {
      const uint32_t g = sz[u / (S::kWords / S::kGroups)];
      const float s = f16_bits_to_f32(g & 0xFFFFu);
      // q - Z as (2^23 + q) - (2^23 + Z), exact
      const float z = -(8388608.0f + f16_bits_to_f32(g >> 16));
      const uint32_t ev = word[u] & 0x0F0F0F0Fu, od = (word[u] >> 4) & 0x0F0F0F0Fu;
      auto value2 = [&](uint32_t e, uint32_t o, int j) {  // of bytes j of e and o
        const float2 q = make_float2(__uint_as_float(__byte_perm(e, 0x4B000000u, 0x7650 + j)),
                                     __uint_as_float(__byte_perm(o, 0x4B000000u, 0x7650 + j)));
        return __fmul2_rn(__fadd2_rn(q, make_float2(z, z)), make_float2(s, s));
      };
      if (kOut == WQ_F32) {
        // two neighbours (of one group) write 32 bytes of one's word, then of the other's
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t n = __shfl_sync(0xffffffffu, word[u], (lane & ~1) + i) >> (16 * (l & 1));
          const float2 v0 = value2(n & 0x0F0Fu, (n >> 4) & 0x0F0Fu, 0);
          const float2 v1 = value2(n & 0x0F0Fu, (n >> 4) & 0x0F0Fu, 1);
          if (in)
            *reinterpret_cast<float4*>(static_cast<float*>(kV ? a.V : a.K) + row * D +
                                       S::dim((l & ~1) + i, u) + 4 * (l & 1)) =
                make_float4(v0.x, v0.y, v1.x, v1.y);
        }
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = value2(ev, od, j);
          if (kOut == WQ_BF16) {
            o[j] = pack_bf16x2(v.x, v.y);
          } else {
            const __half2 h = __floats2half2_rn(v.x, v.y);
            o[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
        if (in)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kV ? a.V : a.K) + row * D +
                                    S::dim(l, u)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  if (range) set_status(a.status, kStRange);
}

template <int D, int G, int kOut>
__global__ void __launch_bounds__(kRowThreads) read_kernel(Kv4ReadArgs a) {
  if (blockIdx.y == 0) read_rows<D, G, kOut, false>(a);
  else read_rows<D, G, kOut, true>(a);
}

int grid_for(int64_t items, int per_cta, int cap) {
  const int64_t n = (items + per_cta - 1) / per_cta;
  return static_cast<int>(n < 1 ? 1 : n < cap ? n : cap);
}

}  // namespace

cudaError_t launch_kv4_block_tables(const Kv4TablesArgs& a, int sms, cudaStream_t st) {
  block_tables_kernel<<<grid_for(a.n_slots, kTabThreads, sms), kTabThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// CTAs of each kind for tokens x heads rows, 8 (of V, D = 64: 16) a warp.
static dim3 row_grid(int64_t tokens, const Kv4Cache& c, int sms) {
  return dim3(grid_for(tokens * c.kv_heads, 8 * (kRowThreads / 32), sms * kRowCtas), 2);
}

template <int D, int G>
static void read_any(const Kv4ReadArgs& a, dim3 grid, cudaStream_t st) {
  if (a.out_dtype == WQ_F32)
    read_kernel<D, G, WQ_F32><<<grid, kRowThreads, 0, st>>>(a);
  else if (a.out_dtype == WQ_BF16)
    read_kernel<D, G, WQ_BF16><<<grid, kRowThreads, 0, st>>>(a);
  else
    read_kernel<D, G, WQ_F16><<<grid, kRowThreads, 0, st>>>(a);
}

template <int D, int G>
static void append_any(const Kv4AppendArgs& a, dim3 grid, cudaStream_t st) {
  if (a.bf16) append_kernel<D, G, true><<<grid, kRowThreads, 0, st>>>(a);
  else append_kernel<D, G, false><<<grid, kRowThreads, 0, st>>>(a);
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sms, cudaStream_t st) {
  const Kv4Cache& c = a.cache;
  const dim3 grid = row_grid(a.tokens, c, sms);
  if (c.dim == 64) {
    if (c.group == 32) append_any<64, 32>(a, grid, st);
    else append_any<64, 64>(a, grid, st);
  } else {
    if (c.group == 32) append_any<128, 32>(a, grid, st);
    else if (c.group == 64) append_any<128, 64>(a, grid, st);
    else append_any<128, 128>(a, grid, st);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int sms, cudaStream_t st) {
  const Kv4Cache& c = a.cache;
  const dim3 grid = row_grid(a.tokens, c, sms);
  if (c.dim == 64) {
    if (c.group == 32) read_any<64, 32>(a, grid, st);
    else read_any<64, 64>(a, grid, st);
  } else {
    if (c.group == 32) read_any<128, 32>(a, grid, st);
    else if (c.group == 64) read_any<128, 64>(a, grid, st);
    else read_any<128, 128>(a, grid, st);
  }
  return cudaGetLastError();
}

}  // namespace wq
