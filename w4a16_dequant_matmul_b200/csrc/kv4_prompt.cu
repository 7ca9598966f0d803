// Attention over the 4-bit KV cache for prompts: requests with many query rows (a row is one
// token and query head of a KV head's group). Same mathematics as kv4_decode.cu, on tcgen05.
//
// A CTA (one per SM) takes 256 rows of one (request, KV head), as two tiles of 128, against
// tiles of 128 keys:
//     S_i = Q_i C_k^T        tcgen05.mma, both operands in shared memory, S_i in TMEM
//     p   = 2^(S_i ks + lv - m + 7),  l += p / S_v
//     O_i += P_i C_v         P_i (binary16) from TMEM, O_i in TMEM
// C_k, C_v are the codes less their Z, exact in 16 bits: a key's scale meets its score in fp32
// (ks = S_k scale log2(e)), a value's joins the exponent (lv = log2 S_v), so that no operand
// is rounded but p. A key outside the request has lv = -inf. One thread owns a row: it reads
// its 128 scores from TMEM, and m moves (which rescales O_i in TMEM) only when a score passes
// it by 2^8; the scores are read again then.
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (and Q's load, the output); 8-11 expand: codes
// straight from global memory, one tile ahead in registers, into the two-deep rings of K
// (rows = keys) and V^T (rows = dimensions, built from octets of keys) in the 128-byte
// swizzle; 12 issues the MMAs (13-15 are idle and give their registers to the softmax). K and Q hold each eight dimensions in the order 0 4 1 5 2 6 3 7,
// in which a word's codes come apart by shifts.
//
// S_i and P_i share TMEM: S_i of the next keys is issued behind the product that reads P_i.
// When the softmax of tile i wakes for S_i, that product has completed too (the same commit),
// so it may touch O_i.
#include <atomic>

#include "common.cuh"
#include "kv4.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace wq {
namespace {

constexpr int kM = 128;       // rows of a Q tile
constexpr int kN = 128;       // keys of a tile
constexpr int kRowsCta = 2 * kM;
constexpr int kThreads = 512;
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr float kLift = 7.0f, kHeadroom = 8.0f;

// Registers of a thread after the split: the launch gives every warpgroup 128, and the four
// shares add up to the same.
constexpr int kRegsSoftmax = 184, kRegsExpand = 96, kRegsIssue = 48;
static_assert(2 * kRegsSoftmax + kRegsExpand + kRegsIssue == 4 * 128, "register split");
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

struct Ctl {
  uint64_t q_full[2];
  uint64_t k_full[2], k_empty[2];
  uint64_t v_full[2], v_empty[2];
  uint64_t vec_full[4];
  uint64_t s_full[2], p_full[2];
  uint64_t o_full;
  int64_t scan[16];
  int b, tile, head;  // this CTA's unit; b < 0: none
  uint32_t tmem_base;
  volatile int abort;
};

template <int D>
struct Cfg {
  static constexpr int kQBytes = kM * D * 2;   // one Q tile
  static constexpr int kKBytes = kN * D * 2;   // one K tile, one V^T tile
  static constexpr int kVecFloats = 3 * kN;    // ks, lv, 1 / S_v
  static constexpr int kSmem = 1024 + 2 * kQBytes + 4 * kKBytes + 4 * kVecFloats * 4 +
                               static_cast<int>(sizeof(Ctl));
};

__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                          unsigned* status) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait_spin_bounded(bar, parity, kLimitNs) && !ctl->abort);
  if (!ok && (threadIdx.x & 31) == 0) {
    set_status(status, kStTimeout);
    ctl->abort = 1;
  }
  return ok;
}
__device__ __forceinline__ bool wait_lane(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                          unsigned* status) {
  if (mbar_wait_spin_bounded(bar, parity, kLimitNs) && !ctl->abort) return true;
  set_status(status, kStTimeout);
  ctl->abort = 1;
  return false;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  return kBf16 ? pack_bf16x2(lo, hi) : half2_bits(lo, hi);
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Eight codes of a word less Z as 16-bit floats, pairs (i, i + 4). zz: Z + 128 (bf16) or
// Z + 1024 (fp16) twice; zh: -(Z + 64) twice (fp16).
template <bool kBf16>
__device__ __forceinline__ uint4 expand_k(uint32_t w, uint32_t zz, uint32_t zh) {
  uint4 o;
  if (kBf16) {
    o.x = bsub2(and_or(w, 0x000F000Fu, 0x43004300u), zz);
    o.y = bsub2(and_or(w >> 4, 0x000F000Fu, 0x43004300u), zz);
    o.z = bsub2(and_or(w >> 8, 0x000F000Fu, 0x43004300u), zz);
    o.w = bsub2(and_or(w >> 12, 0x000F000Fu, 0x43004300u), zz);
  } else {
    const uint32_t v = w >> 8;
    o.x = hsub2(and_or(w, 0x000F000Fu, 0x64006400u), zz);
    o.y = hfma2(and_or(w, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);
    o.z = hsub2(and_or(v, 0x000F000Fu, 0x64006400u), zz);
    o.w = hfma2(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);
  }
  return o;
}

struct Unit {
  int q0, rows, kv, row0;  // request's first row of Q, its rows and keys, the CTA's first row
  int shift;               // keys before the first query: row i sees keys up to shift + i / ratio
  int t0, nt;              // first tile of 128 keys, number of tiles
};

__device__ __forceinline__ void request_rows(const Kv4AttnArgs& a, int b, int& q0, int& qn) {
  int lo = a.q_starts[b], hi = a.q_starts[b + 1];
  lo = lo < 0 ? 0 : lo < a.tokens ? lo : a.tokens;
  hi = hi < lo ? lo : hi < a.tokens ? hi : a.tokens;
  q0 = lo;
  qn = hi - lo;
}
__device__ __forceinline__ int request_tiles(const Kv4AttnArgs& a, int b) {
  int q0, qn;
  request_rows(a, b, q0, qn);
  const int64_t rows = static_cast<int64_t>(qn) * a.ratio;
  return rows > a.most_rows ? static_cast<int>((rows + kRowsCta - 1) / kRowsCta) : 0;
}

// One row's 128 scores: p = 2^(s + lv + up) as binary16 pairs, their sum over S_v, and the
// largest exponent. kMask: only keys low < pos <= lim count.
template <bool kMask>
__device__ __forceinline__ float row_pass(uint32_t t_s, uint32_t vs, float up, int pos0, int lim,
                                          int low, uint32_t (&p)[kN / 64][32], float2& sum) {
  const float2 up2 = make_float2(up, up);
  float mx = -INFINITY;
  sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < kN / 32; ++c) {
    uint32_t v[32];
    tmem_ld32(t_s + 32 * c, v);
    tmem_wait_ld();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float4 ks = lds_f4(vs + (32 * c + 4 * q) * 4);
      const float4 lv = lds_f4(vs + (kN + 32 * c + 4 * q) * 4);
      const float4 is = lds_f4(vs + (2 * kN + 32 * c + 4 * q) * 4);
      float2 s0 = __ffma2_rn(make_float2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])),
                             make_float2(ks.x, ks.y), __fadd2_rn(make_float2(lv.x, lv.y), up2));
      float2 s1 = __ffma2_rn(make_float2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])),
                             make_float2(ks.z, ks.w), __fadd2_rn(make_float2(lv.z, lv.w), up2));
      if (kMask) {
        const int pos = pos0 + 32 * c + 4 * q;
        if (pos > lim || pos <= low) s0.x = -INFINITY;
        if (pos + 1 > lim || pos + 1 <= low) s0.y = -INFINITY;
        if (pos + 2 > lim || pos + 2 <= low) s1.x = -INFINITY;
        if (pos + 3 > lim || pos + 3 <= low) s1.y = -INFINITY;
      }
      mx = fmaxf(fmaxf(mx, fmaxf(s0.x, s0.y)), fmaxf(s1.x, s1.y));
      const float2 p0 = make_float2(ex2(s0.x), ex2(s0.y));
      const float2 p1 = make_float2(ex2(s1.x), ex2(s1.y));
      sum = __ffma2_rn(p0, make_float2(is.x, is.y), sum);
      sum = __ffma2_rn(p1, make_float2(is.z, is.w), sum);
      p[c >> 1][16 * (c & 1) + 2 * q] = half2_bits(p0.x, p0.y);
      p[c >> 1][16 * (c & 1) + 2 * q + 1] = half2_bits(p1.x, p1.y);
    }
  }
  return mx;
}

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1) kv4_prompt_kernel(const Kv4AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                      // [2][atom][128 rows][128 B]
  uint8_t* sK = sQ + 2 * C::kQBytes;       // [2][atom][128 keys][128 B]
  uint8_t* sV = sK + 2 * C::kKBytes;       // [2][2 atoms of 64 keys][D rows][128 B]
  float* vec = reinterpret_cast<float*>(sV + 2 * C::kKBytes);  // [4][ks, lv, isv][128]
  Ctl* ctl = reinterpret_cast<Ctl*>(vec + 4 * C::kVecFloats);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // --- which unit: the CTA's index in the line of all requests' (row tile, KV head) pairs
  {
    const int per = (a.requests + kThreads - 1) / kThreads;
    const int64_t r0 = static_cast<int64_t>(threadIdx.x) * per;
    int64_t mine = 0;
    for (int64_t b = r0; b < r0 + per && b < a.requests; ++b)
      mine += static_cast<int64_t>(request_tiles(a, static_cast<int>(b))) * a.cache.kv_heads;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) ctl->scan[warp] = incl;
    if (threadIdx.x == 0) ctl->b = -1;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 16; ++w)
      if (w < warp) incl += ctl->scan[w];
    const int64_t want = blockIdx.x;
    if (want >= incl - mine && want < incl) {
      int64_t off = want - (incl - mine);
      int b = static_cast<int>(r0);
      int n;
      while (true) {
        n = request_tiles(a, b);
        if (off < static_cast<int64_t>(n) * a.cache.kv_heads) break;
        off -= static_cast<int64_t>(n) * a.cache.kv_heads;
        ++b;
      }
      ctl->b = b;
      // the last tiles first: under a causal mask they have the most keys
      ctl->tile = n - 1 - static_cast<int>(off / a.cache.kv_heads);
      ctl->head = static_cast<int>(off % a.cache.kv_heads);
    }
    if (threadIdx.x == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&ctl->q_full[i], 4);
        mbar_init(&ctl->k_full[i], 4);
        mbar_init(&ctl->k_empty[i], 1);
        mbar_init(&ctl->v_full[i], 4);
        mbar_init(&ctl->v_empty[i], 1);
        mbar_init(&ctl->s_full[i], 1);
        mbar_init(&ctl->p_full[i], 4);
      }
      for (int i = 0; i < 4; ++i) mbar_init(&ctl->vec_full[i], 4);
      mbar_init(&ctl->o_full, 1);
      ctl->abort = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  if (ctl->b < 0) return;
  if (warp == 12) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

  const int b = ctl->b, head = ctl->head;
  Unit u;
  {
    int qn;
    request_rows(a, b, u.q0, qn);
    u.kv = a.kv_lens[b] < 0 ? 0 : a.kv_lens[b];
    u.rows = qn * a.ratio;
    u.row0 = ctl->tile * kRowsCta;
    u.shift = u.kv - qn;
    const int last_row = u.row0 + kRowsCta < u.rows ? u.row0 + kRowsCta - 1 : u.rows - 1;
    // keys [first, end) are seen by some row
    int64_t end = a.causal ? static_cast<int64_t>(u.shift) + last_row / a.ratio + 1 : u.kv;
    const int64_t reach = static_cast<int64_t>(a.width) << a.cache.block_log2;
    if (end > reach) {
      end = reach;
      if (threadIdx.x == 0) set_status(a.status, kStRange);
    }
    int64_t first = 0;
    if (a.window > 0)
      first = (a.causal ? static_cast<int64_t>(u.shift) + u.row0 / a.ratio : u.kv - 1) - a.window + 1;
    if (first < 0) first = 0;
    u.t0 = static_cast<int>(first / kN);
    const int64_t last_tile = (end + kN - 1) / kN;
    u.nt = last_tile > u.t0 ? static_cast<int>(last_tile - u.t0) : 1;
  }

  if (warp < 8) {
    reg_inc<kRegsSoftmax>();
    // --------------------------------------------------------------- softmax, one row a thread
    const int i = warp >> 2;
    const int r = threadIdx.x & 127;
    const int row = u.row0 + i * kM + r;
    const bool live = row < u.rows;
    const int tok = row / a.ratio, h = head * a.ratio + row - tok * a.ratio;
    {
      const uint16_t* src = a.Q + static_cast<int64_t>(u.q0 + tok) * a.q_tok +
                            static_cast<int64_t>(h) * a.q_head;
      const uint32_t dst = smem_u32(sQ + i * C::kQBytes) + r * 128;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (live) x = ld_nc_u4(src + 8 * c);
        const uint4 y = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                   __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
        sts128(dst + (c >> 3) * (kM * 128) + (((c & 7) ^ (r & 7)) << 4), y);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->q_full[i]);
    }
    // the last key that this row sees, and what all rows of the tile see
    const int lim = !live ? -1 : a.causal ? u.shift + tok : u.kv - 1;
    const int tile_first = u.row0 + i * kM;
    int tile_last = tile_first + kM - 1;
    if (tile_last >= u.rows) tile_last = u.rows - 1;
    const int safe_end = (a.causal ? u.shift + tile_first / a.ratio : u.kv - 1) + 1;
    const int safe_begin =
        a.window > 0 ? (a.causal ? u.shift + tile_last / a.ratio : u.kv - 1) - a.window + 1 : 0;
    const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t t_s = t_row + i * kN;
    const uint32_t t_o = t_row + 2 * kN + i * 128;
    const uint32_t vec_s = smem_u32(vec);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < u.nt; ++j) {
      if (!wait_warp(&ctl->s_full[i], j & 1, ctl, a.status) ||
          !wait_warp(&ctl->vec_full[j & 3], (j >> 2) & 1, ctl, a.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t vs = vec_s + (j & 3) * C::kVecFloats * 4;
      const int pos0 = (u.t0 + j) * kN;
      const bool safe = pos0 + kN <= safe_end && pos0 >= safe_begin;
      uint32_t p[kN / 64][32];
      float2 sum;
      // two passes settle any scores that fp32 can tell apart; the bound ends it for others
      for (int pass = 0; pass < 3; ++pass) {
        const float ref = m == -INFINITY ? 0.0f : m;
        float mx = safe ? row_pass<false>(t_s, vs, kLift - ref, 0, 0, 0, p, sum)
                        : row_pass<true>(t_s, vs, kLift - ref, pos0, lim,
                                         a.window > 0 ? lim - a.window : -1, p, sum);
        // mx is relative to m: above kLift + kHeadroom m has to move (from -inf: always)
        const bool over = m == -INFINITY ? mx > -INFINITY : mx > kLift + kHeadroom;
        if (!__any_sync(0xffffffffu, over)) break;
        const float to = fmaxf(m, ref + (mx - kLift));
        const float f = to == -INFINITY || m == to ? 1.0f : ex2(m - to);
        m = to;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(t_o + 32 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
            tmem_st32(t_o + 32 * c, v);
          }
        }
      }
      l += sum.x + sum.y;
#pragma unroll
      for (int c = 0; c < kN / 64; ++c) tmem_st32(t_s + 32 * c, p[c]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[i]);
    }
    // --- the rows' results
    if (ok && wait_warp(&ctl->o_full, 0, ctl, a.status)) {
      tc_fence_after();
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      uint16_t* dst = a.out + static_cast<int64_t>(u.q0 + tok) * a.o_tok +
                      static_cast<int64_t>(h) * a.o_head;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(t_o + 32 * c, v);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = narrow2<kBf16>(__uint_as_float(v[8 * q + 2 * e]) * inv,
                                    __uint_as_float(v[8 * q + 2 * e + 1]) * inv);
            *reinterpret_cast<uint4*>(dst + 32 * c + 8 * q) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && a.lse)
        a.lse[static_cast<int64_t>(u.q0 + tok) * a.heads + h] =
            l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
    }
  } else if (warp < 12) {
    reg_dec<kRegsExpand>();
    // ------------------------------------------------------------------------ expand
    const Kv4Cache& kc = a.cache;
    const int e = threadIdx.x - 256;  // 0..127: the key of K that this thread expands
    // V: an octet of keys, and the column group g whose bytes hold dimensions 16 i + 2 g, + 1;
    // eight lanes that store together differ in row mod 8 or octet, so on banks
    constexpr int VB = D / 16;  // bytes of a column group
    const int vg = (lane & 3) | ((lane >> 1) & 4) | 0;  // lane bits 0, 1, 3
    const int vo = 4 * (warp - 8) + (((lane >> 2) & 1) | ((lane >> 3) & 2));  // lane bits 2, 4
    const int64_t codes = static_cast<int64_t>(kc.block) * (D / 2);
    const int32_t* table = a.tables + b * a.ld_tables;
    const int bmask = kc.block - 1;
    // chunk of the block that holds a key, or nullptr where there is none
    auto chunk_of = [&](int64_t pos) -> const uint8_t* {
      if (pos >= u.kv) return nullptr;
      const int64_t place = pos >> kc.block_log2;
      const int blk = place < a.width ? table[place] : -1;
      if (blk < 0 || blk >= kc.num_blocks) {
        set_status(a.status, kStRange);
        return nullptr;
      }
      return kc.data + (static_cast<int64_t>(blk) * kc.kv_heads + head) * kc.chunk_bytes();
    };
    uint4 kw[D / 32];
    uint32_t ksz, ksv;  // scale words of the thread's key, of K and V
    bool k_there;
    uint32_t vw[8][VB / 4];
    uint32_t vsz[8];
    auto load_k = [&](int j) {
      const int64_t pos = static_cast<int64_t>(u.t0 + j) * kN + e;
      const uint8_t* ch = chunk_of(pos);
      k_there = ch != nullptr;
      ksz = ksv = 0;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) kw[c] = make_uint4(0, 0, 0, 0);
      if (ch) {
        const int t = static_cast<int>(pos) & bmask;
        // word c (D/32) + j of the row is word 4 j + c of its dimensions
        const uint4* src = reinterpret_cast<const uint4*>(ch + t * (D / 2));
#pragma unroll
        for (int c = 0; c < D / 32; ++c) kw[c] = ld_nc_u4(src + c);
        const uint32_t* sz = reinterpret_cast<const uint32_t*>(ch + 2 * codes);
        ksz = __ldg(sz + t);
        ksv = __ldg(sz + kc.block + t);
      }
    };
    auto load_v = [&](int j) {
      const int64_t pos = static_cast<int64_t>(u.t0 + j) * kN + 8 * vo;
      const uint8_t* ch = chunk_of(pos);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        vsz[k] = 0;
#pragma unroll
        for (int q = 0; q < VB / 4; ++q) vw[k][q] = 0;
      }
      if (ch) {
        const int t = static_cast<int>(pos) & bmask;
        const uint32_t* sz = reinterpret_cast<const uint32_t*>(ch + 2 * codes) + kc.block;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (pos + k < u.kv) {
            const int flip = (D == 128 && (k & 2)) ? 32 : 0;
            const uint8_t* src = ch + codes + (t + k) * (D / 2) + ((VB * vg) ^ flip);
            if (VB == 8) {
              const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
              vw[k][0] = x.x;
              vw[k][VB / 4 - 1] = x.y;
            } else {
              vw[k][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
            vsz[k] = __ldg(sz + t + k);
          }
        }
      }
    };
    load_k(0);
    load_v(0);
    const uint32_t sK0 = smem_u32(sK), sV0 = smem_u32(sV), vec0 = smem_u32(vec);
    for (int j = 0; j < u.nt; ++j) {
      const int buf = j & 1;
      if (j >= 2 && !wait_warp(&ctl->k_empty[buf], ((j >> 1) - 1) & 1, ctl, a.status)) break;
      {
        const uint32_t z = ksz >> 16;
        const uint32_t z2 = z | z << 16;
        // Z as a binary16 integer: to Z + 128 in bf16, Z + 1024 and -(Z + 64) in binary16
        uint32_t zz, zh = 0;
        if (kBf16) {
          const float zf = f16_bits_to_f32(z) + 128.0f;
          zz = pack_bf16x2(zf, zf);
        } else {
          zz = hfma2(z2, 0x3C003C00u, 0x64006400u);
          zh = hfma2(z2, 0xBC00BC00u, 0xD400D400u);
        }
        const uint32_t dst = sK0 + buf * C::kKBytes + e * 128;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          // chunk n of the row: natural word n = 4 j + c, stored word c (D/32) + j
          const int at = (n & 3) * (D / 32) + (n >> 2);
          const uint4 q4 = kw[at >> 2];
          const uint32_t w = (at & 3) == 0 ? q4.x : (at & 3) == 1 ? q4.y : (at & 3) == 2 ? q4.z : q4.w;
          sts128(dst + (n >> 3) * (kN * 128) + (((n & 7) ^ (e & 7)) << 4), expand_k<kBf16>(w, zz, zh));
        }
        const float sv = fmaxf(f16_bits_to_f32(ksv & 0xFFFFu), 5.9604644775390625e-8f);
        const uint32_t vs = vec0 + (j & 3) * C::kVecFloats * 4 + e * 4;
        sts_f32(vs, k_there ? f16_bits_to_f32(ksz & 0xFFFFu) * a.scale_log2 : 0.0f);
        sts_f32(vs + kN * 4, k_there ? lg2(sv) : -INFINITY);
        sts_f32(vs + 2 * kN * 4, k_there ? __fdividef(1.0f, sv) : 0.0f);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->k_full[buf]);
          mbar_arrive(&ctl->vec_full[j & 3]);
        }
      }
      if (j + 1 < u.nt) load_k(j + 1);
      if (j >= 2 && !wait_warp(&ctl->v_empty[buf], ((j >> 1) - 1) & 1, ctl, a.status)) break;
      {
        uint32_t zz[4], zh[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t z2 = __byte_perm(vsz[2 * k], vsz[2 * k + 1], 0x7632);
          zz[k] = hfma2(z2, 0x3C003C00u, 0x64006400u);
          zh[k] = hfma2(z2, 0xBC00BC00u, 0xD400D400u);
        }
        const uint32_t dst = sV0 + buf * C::kKBytes + (vo >> 3) * (D * 128);
#pragma unroll
        for (int n = 0; n < VB; ++n) {  // byte n: dimensions 16 n + 2 vg (low nibble), + 1
          uint32_t lo[4], hi[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t y = __byte_perm(vw[2 * k][n >> 2], vw[2 * k + 1][n >> 2],
                                           static_cast<uint32_t>(n & 3) |
                                               (static_cast<uint32_t>(4 + (n & 3)) << 8));
            lo[k] = hsub2(and_or(y, 0x000F000Fu, 0x64006400u), zz[k]);
            hi[k] = hfma2(and_or(y, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh[k]);
          }
          const int d0 = 16 * n + 2 * vg;
          sts128(dst + d0 * 128 + (((vo & 7) ^ (d0 & 7)) << 4), make_uint4(lo[0], lo[1], lo[2], lo[3]));
          sts128(dst + (d0 + 1) * 128 + (((vo & 7) ^ ((d0 + 1) & 7)) << 4),
                 make_uint4(hi[0], hi[1], hi[2], hi[3]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->v_full[buf]);
      }
      if (j + 1 < u.nt) load_v(j + 1);
    }
  } else {
    reg_dec<kRegsIssue>();
    if (warp == 12 && lane == 0) {
    // ---------------------------------------------------------------------- MMA issuer
    constexpr uint32_t kFmt = kBf16 ? (1u << 7) | (1u << 10) : 0u;
    constexpr uint32_t kIdescS = (1u << 4) | kFmt | ((kN >> 3) << 17) | ((kM >> 4) << 24);
    constexpr uint32_t kIdescO = (1u << 4) | ((D >> 3) << 17) | ((kM >> 4) << 24);
    auto scores = [&](int i, int buf) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = (k >> 2) * (128 * 128) + (k & 3) * 32;
        tc_mma(tmem + i * kN, sw128_desc(sQ + i * C::kQBytes + at),
               sw128_desc(sK + buf * C::kKBytes + at), kIdescS, k != 0);
      }
      tc_commit(&ctl->s_full[i]);
    };
    bool ok = wait_lane(&ctl->q_full[0], 0, ctl, a.status) &&
              wait_lane(&ctl->q_full[1], 0, ctl, a.status) &&
              wait_lane(&ctl->k_full[0], 0, ctl, a.status);
    if (ok) {
      tc_fence_after();
      scores(0, 0);
      scores(1, 0);
      tc_commit(&ctl->k_empty[0]);
    }
    for (int j = 0; j < u.nt && ok; ++j) {
      const int buf = j & 1;
      const bool more = j + 1 < u.nt;
      ok = wait_lane(&ctl->v_full[buf], (j >> 1) & 1, ctl, a.status);
      for (int i = 0; i < 2 && ok; ++i) {
        ok = wait_lane(&ctl->p_full[i], j & 1, ctl, a.status);
        if (ok && more && i == 0) ok = wait_lane(&ctl->k_full[buf ^ 1], ((j + 1) >> 1) & 1, ctl, a.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          tc_mma_tmem_a(tmem + 2 * kN + i * 128, tmem + i * kN + 8 * k,
                        sw128_desc(sV + buf * C::kKBytes + (k >> 2) * (D * 128) + (k & 3) * 32),
                        kIdescO, (j | k) != 0);
        if (more) scores(i, buf ^ 1);
      }
      if (!ok) break;
      tc_commit(&ctl->v_empty[buf]);
      if (more) tc_commit(&ctl->k_empty[buf ^ 1]);
    }
    // all issued MMAs have completed once this arrives
    tc_commit(&ctl->o_full);
    if (!mbar_wait_bounded(&ctl->o_full, 0, kLimitNs)) set_status(a.status, kStTimeout);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool kBf16>
cudaError_t launch_t(const Kv4AttnArgs& a, int64_t units, cudaStream_t st) {
  auto kern = kv4_prompt_kernel<D, kBf16>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr[dev & 63].load(std::memory_order_acquire)) {
    e = set_smem_attrs(kern, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    attr[dev & 63].store(true, std::memory_order_release);
  }
  kern<<<static_cast<unsigned>(units), kThreads, Cfg<D>::kSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool kv4_prompt_ok(const Kv4AttnArgs& a) { return a.cache.groups() == 1; }

cudaError_t launch_kv4_prompt(const Kv4AttnArgs& a, cudaStream_t st) {
  // an upper bound of the units: the lengths are on the device, CTAs without a unit return
  const int64_t units = (static_cast<int64_t>(a.tokens) * a.ratio / kRowsCta + a.requests) *
                        a.cache.kv_heads;
  if (a.cache.dim == 128)
    return a.bf16 ? launch_t<128, true>(a, units, st) : launch_t<128, false>(a, units, st);
  return a.bf16 ? launch_t<64, true>(a, units, st) : launch_t<64, false>(a, units, st);
}

}  // namespace wq
