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

// One thread holds 8 consecutive dimensions of a row (one 16-byte load, one 32-bit word of
// codes); the D/8 threads of a row are neighbours, the group's range is reduced among its
// group/8 of them by shuffles. S', Z and the codes are decided exactly, as in quantize.cu.
// Bound by HBM: 2 B an element in, D/2 + 4 D/g bytes a row out. K words are stored whole, V
// bytes one by one (the V order spreads a row's neighbouring bytes over the lanes' shares);
// both stay within the row, whose sectors L2 puts together.
template <bool kBf16>
__global__ void __launch_bounds__(256) append_kernel(Kv4AppendArgs a) {
  const Kv4Cache c = a.cache;
  const int lanes = c.dim >> 3, glanes = c.group >> 3;
  const int rows_per_cta = 256 / lanes;
  const int sub = threadIdx.x / lanes, w = threadIdx.x - sub * lanes;
  const int64_t rows = a.tokens * c.kv_heads * 2;  // K and V rows of a (token, head) side by side
  const int64_t limit = c.num_blocks << c.block_log2;
  bool range = false, nonfinite = false;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * rows_per_cta + sub;
       r - sub < rows;  // the same trip count for a whole warp: the shuffles need every lane
       r += static_cast<int64_t>(gridDim.x) * rows_per_cta) {
    const bool in = r < rows;
    const bool is_v = r & 1;
    const int64_t th = r >> 1;
    const int64_t tok = th / c.kv_heads;
    const int head = static_cast<int>(th - tok * c.kv_heads);
    int slot = in ? a.slots[tok] : -1;
    if (slot >= limit) {
      range = true;
      slot = -1;
    }
    const bool live = slot >= 0;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) {
      const uint16_t* src = is_v ? a.V + tok * a.v_tok + head * a.v_head
                                 : a.K + tok * a.k_tok + head * a.k_head;
      x = ld_stream_u4(src + 8 * w);
    }
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
    float v[8];
    float mn = 0.0f, mx = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = widen<kBf16>(xs[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
      mn = fmin_nan(mn, fmin_nan(f.x, f.y));
      mx = fmax_nan(mx, fmax_nan(f.x, f.y));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const float omn = __shfl_xor_sync(0xffffffffu, mn, o);
      const float omx = __shfl_xor_sync(0xffffffffu, mx, o);
      if (o < glanes) {
        mn = fmin_nan(mn, omn);
        mx = fmax_nan(mx, omx);
      }
    }
    if (!live) continue;
    const AsymScale sz = asym_scale_zero(mn, mx);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = sz.bad ? 0.0f : rne_quotient(v[i], sz.s, sz.inv_s) + sz.z;
      q = fminf(fmaxf(q, 0.0f), 15.0f);
      word |= static_cast<uint32_t>(__float2int_rz(q)) << (4 * i);
    }
    const int half = c.dim >> 1;
    const int t = slot & (c.block - 1);
    uint8_t* chunk = c.data + (static_cast<int64_t>(slot >> c.block_log2) * c.kv_heads + head) *
                                  c.chunk_bytes();
    uint8_t* row = chunk + (is_v ? c.block * half : 0) + t * half;
    if (!is_v) {
      const int at = (w & 3) * (c.dim >> 5) + (w >> 2);
      *reinterpret_cast<uint32_t*>(row + 4 * at) = word;
    } else {
      const int flip = (c.dim == 128 && (t & 2)) ? 32 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 4 * w + i;  // byte of the natural order
        row[((n & 7) * (c.dim >> 4) + (n >> 3)) ^ flip] = static_cast<uint8_t>(word >> (8 * i));
      }
    }
    if (w % glanes == 0) {
      const int g = w / glanes, groups = c.groups();
      uint32_t* szp = reinterpret_cast<uint32_t*>(chunk + 2 * c.block * half) +
                      (is_v ? c.block * groups : 0) + t * groups + g;
      *szp = sz.sbits | f32_to_f16_bits(sz.z) << 16;
      if (sz.bad) nonfinite = true;
    }
  }
  if (range) set_status(a.status, kStRange);
  if (nonfinite) set_status(a.status, kStNonFinite);
}

// The inverse: one thread gives 8 consecutive values S'(q - Z) of a row (exact in fp32, or
// rounded once to 16 bits); slot < 0 gives zeros. Bound by HBM: the values written.
template <int kOut>  // WQ_F32, WQ_BF16, WQ_F16
__global__ void __launch_bounds__(256) read_kernel(Kv4ReadArgs a) {
  const Kv4Cache c = a.cache;
  const int lanes = c.dim >> 3;
  const int64_t limit = c.num_blocks << c.block_log2;
  const int64_t total = a.tokens * c.kv_heads * 2 * lanes;
  bool range = false;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / lanes;
    const int w = static_cast<int>(i - r * lanes);
    const int64_t rows = a.tokens * c.kv_heads;
    const bool is_v = r >= rows;
    const int64_t th = is_v ? r - rows : r;
    const int64_t tok = th / c.kv_heads;
    const int head = static_cast<int>(th - tok * c.kv_heads);
    int slot = a.slots[tok];
    if (slot >= limit) {
      range = true;
      slot = -1;
    }
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0) {
      const int half = c.dim >> 1, t = slot & (c.block - 1);
      const uint8_t* chunk =
          c.data + (static_cast<int64_t>(slot >> c.block_log2) * c.kv_heads + head) *
                       c.chunk_bytes();
      const uint8_t* row = chunk + (is_v ? c.block * half : 0) + t * half;
      uint32_t word = 0;
      if (!is_v) {
        word = *reinterpret_cast<const uint32_t*>(row + 4 * ((w & 3) * (c.dim >> 5) + (w >> 2)));
      } else {
        const int flip = (c.dim == 128 && (t & 2)) ? 32 : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = 4 * w + j;
          word |= static_cast<uint32_t>(row[((n & 7) * (c.dim >> 4) + (n >> 3)) ^ flip]) << (8 * j);
        }
      }
      const int groups = c.groups();
      const uint32_t sz = *(reinterpret_cast<const uint32_t*>(chunk + 2 * c.block * half) +
                            (is_v ? c.block * groups : 0) + t * groups + 8 * w / c.group);
      const float s = f16_bits_to_f32(sz & 0xFFFFu), z = f16_bits_to_f32(sz >> 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = s * (static_cast<float>((word >> (4 * j)) & 15u) - z);
    }
    const int64_t at = th * c.dim + 8 * w;
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

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, int sms, cudaStream_t st) {
  const int grid = grid_for(a.tokens * a.cache.kv_heads * 2, 256 / (a.cache.dim >> 3), sms * 8);
  if (a.bf16)
    append_kernel<true><<<grid, 256, 0, st>>>(a);
  else
    append_kernel<false><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs& a, int sms, cudaStream_t st) {
  const int grid = grid_for(a.tokens * a.cache.kv_heads * 2 * (a.cache.dim >> 3), 256, sms * 8);
  if (a.out_dtype == WQ_F32)
    read_kernel<WQ_F32><<<grid, 256, 0, st>>>(a);
  else if (a.out_dtype == WQ_BF16)
    read_kernel<WQ_BF16><<<grid, 256, 0, st>>>(a);
  else
    read_kernel<WQ_F16><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace wq
