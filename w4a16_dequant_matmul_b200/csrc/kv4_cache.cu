// The 4-bit KV cache's bookkeeping and storage: block tables and slot maps from request
// lengths, the append that quantizes new keys and values into the paged cache, and the read
// that gives stored values back. The quantizer's readings are those of wq_quantize_rtn_g128
// ("DL S067 - Quantization", sections 1-2): one S', Z per group along the head dimension.
#include <cuda_fp16.h>

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
    // newly taken blocks, spread over the whole grid
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kTabThreads + t; i < tb;
         i += static_cast<int64_t>(gridDim.x) * kTabThreads) {
      const int k = find(s_blk, static_cast<int>(i));
      const int place = ((s_ctx[k] + bs - 1) >> a.block_log2) + static_cast<int>(i) - s_blk[k];
      const int64_t f = blk0 + i;
      if (place < a.width && f < a.n_free)
        a.tables[(r0 + k) * a.ld_tables + place] = a.free_blocks[f];
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
// code + (Z & 1).
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
    t[2 * j] = __float_as_uint(fminf(fmaxf(x.x, lo), hi));
    t[2 * j + 1] = __float_as_uint(fminf(fmaxf(x.y, lo), hi));
  }
  const uint32_t ev = __byte_perm(__byte_perm(t[0], t[2], 0x0040), __byte_perm(t[4], t[6], 0x0040), 0x5410);
  const uint32_t od = __byte_perm(__byte_perm(t[1], t[3], 0x0040), __byte_perm(t[5], t[7], 0x0040), 0x5410);
  return ev + (od << 4) - (z & 1u) * 0x11111111u;
}

// 4 x 4 bytes over the four lanes whose numbers differ in bits 1 and 2 only: lane j of them
// (those two bits) gives up its bytes for byte j of each. Its own inverse.
__device__ __forceinline__ uint32_t transpose_bytes(uint32_t w, int lane) {
  uint32_t t = __shfl_xor_sync(0xffffffffu, w, 2);
  w = __byte_perm(w, t, lane & 2 ? 0x3715 : 0x6240);
  t = __shfl_xor_sync(0xffffffffu, w, 4);
  return __byte_perm(w, t, lane & 4 ? 0x3276 : 0x5410);
}

// Byte offset within its row of the 32-bit word that lane w of a row's D/8 holds: of K, word w
// of the dimensions' order (4 j + c is stored at c (D/32) + j); of V, after transpose_bytes,
// byte column g = 4 (w & 1) + (w >> 1 & 3), rows 4 (w >> 3) .. + 3 (bytes 8 i + g of the
// dimensions' order are stored at g (D/16) + i).
template <int D>
__device__ __forceinline__ int word_place(bool is_v, int w, int t) {
  if (!is_v) return 4 * ((w & 3) * (D / 32) + (w >> 2));
  const int at = (4 * (w & 1) + ((w >> 1) & 3)) * (D / 16) + 4 * (w >> 3);
  return D == 128 && (t & 2) ? at ^ 32 : at;
}

// The (token, head) pairs that a warp's lanes work on: 128 / D of them at a time, the D/8 lanes
// of a K row and of its V row side by side. Pairs are stepped through without divisions.
template <int D>
struct Pairs {
  static constexpr int kLanes = D / 8, kPerWarp = 16 / kLanes;
  int64_t tok, step_tok;
  int head, step_head, heads;
  __device__ Pairs(int kv_heads, int lane) : heads(kv_heads) {
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) +
                           (threadIdx.x >> 5)) * kPerWarp + lane / (2 * kLanes);
    const int64_t step = warps * kPerWarp;
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

// One lane holds 8 consecutive dimensions of a row (one 16-byte load, one 32-bit word of codes);
// the group's range is reduced among its group/8 lanes by shuffles, in 16 bits. S', Z and the
// codes are decided exactly, as in quantize.cu. A warp takes kRounds rounds of pairs at a time and
// each lane decides S' and Z of one of their groups (the exact decision is half of a round's
// instructions: 58 us for 16384 tokens of 8 heads of 128 with every lane deciding its own).
// V's words are formed by a byte transpose among four lanes, so that every store is a word.
// Bytes: 2 an element in, D/2 + 4 D/g a row out.
template <int D, bool kBf16, int kRounds>
__global__ void __launch_bounds__(256, 4) append_kernel(Kv4AppendArgs a) {
  using P = Pairs<D>;
  const Kv4Cache c = a.cache;
  const int lane = threadIdx.x & 31;
  const int glanes = c.group >> 3, groups = c.groups();
  const int nseg = 32 / glanes;  // groups of a round
  const bool is_v = (lane / P::kLanes) & 1;
  const int w = lane % P::kLanes;
  const int64_t limit = c.num_blocks << c.block_log2;
  const int64_t chunk_bytes = c.chunk_bytes();
  const int64_t codes = static_cast<int64_t>(c.block) * (D / 2);
  const uint16_t* base = (is_v ? a.V : a.K) + 8 * w;
  const int64_t s_tok = is_v ? a.v_tok : a.k_tok, s_head = is_v ? a.v_head : a.k_head;
  bool range = false, nonfinite = false;
  P p(c.kv_heads, lane);
  while (__any_sync(0xffffffffu, p.tok < a.tokens)) {
    uint4 x[kRounds];
    int slot[kRounds], head[kRounds];
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      x[u] = make_uint4(0, 0, 0, 0);
      slot[u] = -1;
      head[u] = p.head;
      if (p.tok < a.tokens) {
        x[u] = ld_stream_u4(base + p.tok * s_tok + p.head * s_head);
        slot[u] = __ldg(a.slots + p.tok);
      }
      p.next();
    }
    // the range of each round's groups; then this lane's group of all rounds
    float mn = 0.0f, mx = 0.0f;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      uint32_t lo = min2<kBf16>(min2<kBf16>(x[u].x, x[u].y), min2<kBf16>(x[u].z, x[u].w));
      uint32_t hi = max2<kBf16>(max2<kBf16>(x[u].x, x[u].y), max2<kBf16>(x[u].z, x[u].w));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        if (o < glanes) {
          lo = min2<kBf16>(lo, __shfl_xor_sync(0xffffffffu, lo, o));
          hi = max2<kBf16>(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
      }
      const int from = (lane % nseg) * glanes;
      lo = __shfl_sync(0xffffffffu, lo, from);
      hi = __shfl_sync(0xffffffffu, hi, from);
      if (lane / nseg == u) {
        const float2 l2 = widen<kBf16>(lo), h2 = widen<kBf16>(hi);
        mn = fmin_nan(0.0f, fmin_nan(l2.x, l2.y));
        mx = fmax_nan(0.0f, fmax_nan(h2.x, h2.y));
      }
    }
    const AsymScale sz = asym_scale_zero(mn, mx);
    const uint32_t mine = sz.bad ? 0x80003C00u : sz.sbits | static_cast<uint32_t>(sz.z) << 16;
#pragma unroll
    for (int u = 0; u < kRounds; ++u) {
      const int from = u * nseg + lane / glanes;
      const uint32_t got = __shfl_sync(0xffffffffu, mine, from);
      const float inv_s = __shfl_sync(0xffffffffu, sz.inv_s, from);
      const bool bad = got >> 31;
      const int z = (got >> 16) & 15;
      const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = widen<kBf16>(xs[i]);
      uint32_t word = bad ? 0u : encode8_snap(v, inv_s, z);
      const uint32_t turned = transpose_bytes(word, lane);
      if (slot[u] >= limit) range = true;
      if (slot[u] < 0 || slot[u] >= limit) continue;
      if (is_v) word = turned;
      const int t = slot[u] & (c.block - 1);
      uint8_t* chunk = c.data + (static_cast<int64_t>(slot[u] >> c.block_log2) * c.kv_heads +
                                 head[u]) * chunk_bytes;
      *reinterpret_cast<uint32_t*>(chunk + (is_v ? codes : 0) + t * (D / 2) +
                                   word_place<D>(is_v, w, t)) = word;
      if (w % glanes == 0) {
        uint32_t* szp = reinterpret_cast<uint32_t*>(chunk + 2 * codes) +
                        (is_v ? c.block * groups : 0) + t * groups + w / glanes;
        *szp = (got & 0xFFFFu) | f32_to_f16_bits(static_cast<float>(z)) << 16;
        if (bad) nonfinite = true;
      }
    }
  }
  if (range) set_status(a.status, kStRange);
  if (nonfinite) set_status(a.status, kStNonFinite);
}

// The inverse: one lane gives 8 consecutive values S'(q - Z) of a row (exact in fp32, or
// rounded once to 16 bits); slot < 0 gives zeros. Bound by HBM: the values written.
template <int D, int kOut>  // kOut: WQ_F32, WQ_BF16, WQ_F16
__global__ void __launch_bounds__(256) read_kernel(Kv4ReadArgs a) {
  using P = Pairs<D>;
  const Kv4Cache c = a.cache;
  const int lane = threadIdx.x & 31;
  const bool is_v = (lane / P::kLanes) & 1;
  const int w = lane % P::kLanes;
  const int64_t limit = c.num_blocks << c.block_log2;
  const int64_t chunk_bytes = c.chunk_bytes();
  const int64_t codes = static_cast<int64_t>(c.block) * (D / 2);
  const int groups = c.groups(), my_group = 8 * w / c.group;
  bool range = false;
  // two pairs ahead the slot, one ahead what is stored there
  P p(c.kv_heads, lane), q1 = p, q2 = p;
  int slot_next = -1;
  uint32_t word_next = 0, sz_next = 0;
  auto load_slot = [&]() { slot_next = q2.tok < a.tokens ? __ldg(a.slots + q2.tok) : -1; };
  auto load_row = [&]() {
    int slot = slot_next;
    word_next = sz_next = 0;
    if (slot >= limit) {
      range = true;
      slot = -1;
    }
    if (slot >= 0) {
      const int t = slot & (c.block - 1);
      const uint8_t* chunk =
          c.data + (static_cast<int64_t>(slot >> c.block_log2) * c.kv_heads + q1.head) * chunk_bytes;
      word_next = __ldg(reinterpret_cast<const uint32_t*>(
          chunk + (is_v ? codes : 0) + t * (D / 2) + word_place<D>(is_v, w, t)));
      sz_next = __ldg(reinterpret_cast<const uint32_t*>(chunk + 2 * codes) +
                      (is_v ? c.block * groups : 0) + t * groups + my_group);
    }
  };
  load_slot();
  load_row();
  q2.next();
  load_slot();
  for (; __any_sync(0xffffffffu, p.tok < a.tokens); p.next()) {
    const bool in = p.tok < a.tokens;
    uint32_t word = word_next;
    const uint32_t sz = sz_next;
    q1.next();
    load_row();
    q2.next();
    load_slot();
    const uint32_t turned = transpose_bytes(word, lane);
    if (!in) continue;
    if (is_v) word = turned;
    const float s = f16_bits_to_f32(sz & 0xFFFFu), z = f16_bits_to_f32(sz >> 16);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s * (static_cast<float>((word >> (4 * j)) & 15u) - z);
    const int64_t at = (p.tok * c.kv_heads + p.head) * D + 8 * w;
    if (kOut == WQ_F32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(is_v ? a.V : a.K) + at);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kOut == WQ_BF16) {
          o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
        } else {
          const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.V : a.K) + at) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (range) set_status(a.status, kStRange);
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

// A warp works on 128 / D pairs at a time.
static int pair_grid(int64_t tokens, const Kv4Cache& c, int sms) {
  return grid_for(tokens * c.kv_heads, 8 * (128 / c.dim), sms * 8);
}

template <int D>
static void read_any(const Kv4ReadArgs& a, int grid, cudaStream_t st) {
  if (a.out_dtype == WQ_F32)
    read_kernel<D, WQ_F32><<<grid, 256, 0, st>>>(a);
  else if (a.out_dtype == WQ_BF16)
    read_kernel<D, WQ_BF16><<<grid, 256, 0, st>>>(a);
  else
    read_kernel<D, WQ_F16><<<grid, 256, 0, st>>>(a);
}

// Four rounds a warp where there are that many for all warps of the device (16384 tokens of 8
// heads: 85 us with their read, 94 with one round), else one, for more warps at work (4099
// tokens of 6 heads of 64: 19 us, 23 with four).
template <int D, bool kBf16>
static void append_any(const Kv4AppendArgs& a, int sms, cudaStream_t st) {
  const int64_t per_round = static_cast<int64_t>(sms) * 4 * 8 * (128 / D);
  const int grid = pair_grid(a.tokens, a.cache, sms);
  if (a.tokens * a.cache.kv_heads >= 4 * per_round)
    append_kernel<D, kBf16, 4><<<grid, 256, 0, st>>>(a);
  else
    append_kernel<D, kBf16, 1><<<grid, 256, 0, st>>>(a);
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sms, cudaStream_t st) {
  if (a.cache.dim == 128) {
    if (a.bf16) append_any<128, true>(a, sms, st);
    else append_any<128, false>(a, sms, st);
  } else {
    if (a.bf16) append_any<64, true>(a, sms, st);
    else append_any<64, false>(a, sms, st);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int sms, cudaStream_t st) {
  const int grid = pair_grid(a.tokens, a.cache, sms);
  if (a.cache.dim == 128) read_any<128>(a, grid, st);
  else read_any<64>(a, grid, st);
  return cudaGetLastError();
}

}  // namespace wq
