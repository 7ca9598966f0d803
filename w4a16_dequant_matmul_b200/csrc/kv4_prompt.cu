// Attention over the 4-bit KV cache for prompts: requests with many query rows (a row is one
// token and query head of a KV head's group). Same mathematics as kv4_decode.cu, on tcgen05.
//
// A CTA (one per SM) takes 256 rows of one (request, KV head), as two tiles of 128, against
// tiles of 128 keys:
//     S_i = Q_i K^T          tcgen05.mma, both operands in shared memory, S_i in TMEM
//     p   = 2^(S_i ks + E - m + 6),  l += p 2^-E
//     O_i += P_i (V 2^-E)    P_i (binary16) from TMEM, O_i in TMEM
// Where a key's row has one scale, K is its codes less Z, exact in 16 bits, and the scale meets
// the score in fp32 (ks = S_k scale log2(e)). With several, K is S_k (q - Z) as a sum of two
// 16-bit numbers (15 bits in all, so the sum is exact) and the product runs twice; ks is then
// one number for bf16. binary16 has no room for every S_k (q - Z): there each key has a power of
// two of its own that brings its largest S_k into [2^11, 2^12), and ks is the key's again. (A
// fixed 2^-4 had made S_k below 2^-10 binary16 subnormals: 0.3 % off at 2e-5, 0 at 2^-21.)
// For bf16 results V 2^-E is S_v 2^-E (q - Z) rounded once to binary16 (half a step is 2^-11,
// an eighth of out's); for fp16 results that would show, so V stays exact: with one scale the
// codes less Z, S_v 2^-E meeting p, with several a sum of two numbers as for K.
// E joins the exponent of p, so m is the row's own largest S_i ks + E and values of any magnitude
// keep their bits. Where the largest S_v of the tile's keys lie within 2^6 of each other (as
// nearly everywhere) E is one number for the tile; else every key has its own, from shared
// memory: a key that a row does not see, were its S_v ever so large, takes no bits from the
// others. (One E for all tiles so far, as it was, made the values of a row subnormal where a
// later key's were 2^18 as large.)
// One thread owns a row: it reads its 128 scores from TMEM, and m moves (which rescales O_i in
// TMEM) only when a score passes it by 2^8; the scores are read again then. Of the constants of
// a key only ks comes from shared memory for every score: three of them (scale, logarithm
// and reciprocal of S_v) cost 10 % more.
//
// Measured: 1024 new tokens behind 15360 cached ones, 64 query and 8 KV heads of 128: 604 us,
// 881 TFLOP/s; 2.4 us for a step of 128 keys, whose products take 1.1 us of the tensor core at
// 1.8 GHz and whose powers as long of the exponential unit. A row tile's softmax and its products
// take turns, and the two tiles overlap each other's only in part: that latency chain is what
// bounds the loop, not one unit. Dropped, each slower: score products of half a tile with two in
// flight (they read the query tile from shared memory twice as often, 740 us), polling waits,
// more registers for the softmax. (All forms spill, 20 to 150 bytes a thread, for the most part
// around the softmax loop and in the expansion of several scales.)
//
// Warps: 0-3 and 4-7 softmax of tile 0 and 1 (and Q's load, the output); 8-11 expand the codes
// into the two-deep rings of K (rows = keys) and V^T (rows = dimensions, built from octets of
// keys) in the 128-byte swizzle; 12 issues the MMAs; 13 copies the codes and scales of a tile
// into shared memory (in registers, loaded a tile ahead, they were spilled and waited for:
// 3000 of a step's 5700 cycles). K and Q hold each eight dimensions in the order
// 0 4 1 5 2 6 3 7, in which a word's codes come apart by shifts.
//
// Where the units are fewer than the SMs, as with a short chunk behind a long context, each is
// split over its keys among several CTAs, which leave (O, m, l) in the workspace for a second
// kernel to join in order.
//
// S_i and P_i share TMEM: S_i of the next keys is issued behind the product that reads P_i.
// When the softmax of tile i wakes for S_i, that product has completed too (the same commit),
// so it may touch O_i.
#include <atomic>

#include "common.cuh"
#include "kv4.h"
#include "kv4_math.cuh"
#include "mma_frag.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace wq {
namespace {

constexpr int kM = 128;       // rows of a Q tile
constexpr int kN = 128;       // keys of a tile
constexpr int kRowsCta = 2 * kM;
constexpr int kThreads = 512;
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr float kLift = 6.0f, kHeadroom = 8.0f;  // p <= 2^14
constexpr int kEach = 1 << 20;  // in place of a tile's E: every key has its own
// Exponents of S_v within a tile of one E differ by this at most. The chunk below takes 602 us with
// one E a tile and 1483 with E a key throughout, so the rule should hold for what models have
// (tokens whose values are 30 times smaller among others); each step doubles what a
// probability that is a binary16 subnormal may bring into a row's result, 2^-24 of 15 S at 6.
constexpr int kApart = 6;

// Registers of a thread after the split: the launch gives every warpgroup 128, and the four
// shares add up to the same.
constexpr int kRegsSoftmax = 176, kRegsExpand = 96, kRegsIssue = 64;
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
  uint64_t rk_full, rk_empty, rv_full, rv_empty;  // the raw tiles
  uint64_t s_full[2], p_full[2];
  uint64_t o_full;
  int64_t scan[16];
  uint32_t there[4][4];  // which keys of a tile exist, by the ring of vec
  int exponent[4];       // E of a tile, or kEach, by the same ring

  int b, tile, head;  // this CTA's unit; b < 0: none
  uint32_t tmem_base;
  volatile int abort;
};

template <int D, int G, bool kBf16>
struct Cfg {
  static constexpr bool kSplitK = G > 1;            // K = hi + lo
  static constexpr bool kKeyScale = !kSplitK || !kBf16;  // ks is the key's own
  static constexpr bool kSplitV = G > 1 && !kBf16;  // V = hi + lo
  static constexpr bool kScaleP = G == 1 && !kBf16; // S_v 2^-E meets p
  static constexpr int kKBufs = kSplitK ? 1 : 2;
  static constexpr int kVBufs = kSplitV ? 1 : 2;
  static constexpr int kQBytes = kM * D * 2;  // one Q tile
  static constexpr int kTBytes = kN * D * 2;  // one K tile, one V^T tile; hi and lo are two
  static constexpr int kTop = kScaleP ? 0 : 4;  // exponent of the largest S_v 2^-E
  static constexpr int kSvAt = kKeyScale ? kN : 0, kEAt = kSvAt + (kScaleP ? kN : 0);
  static constexpr int kVecFloats = kEAt + kN;  // ks, S_v 2^-E, E
  static constexpr int kRawK = kN * (D / 2 + 8 * G);  // K codes, K and V scale words of a tile
  static constexpr int kRawV = kN * (D / 2 + 4 * G);  // V codes, V scale words
  static constexpr int kSmem = 1024 + 2 * kQBytes + 4 * kTBytes + kRawK + kRawV +
                               4 * kVecFloats * 4 + static_cast<int>(sizeof(Ctl));
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// Waits suspend the warp: one that polls takes issue slots from the softmax warps beside it
// (a step of 128 keys took 3.2 us with polling expand warps).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                          unsigned* status) {
  const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kLimitNs) && !ctl->abort);
  if (!ok && (threadIdx.x & 31) == 0) {
    set_status(status, kStTimeout);
    ctl->abort = 1;
  }
  return ok;
}

__device__ __forceinline__ uint32_t bsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
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

// The exponent of a positive binary16 number (of its smallest for 0), and a power of two.
__device__ __forceinline__ int half_exponent(uint32_t bits) {
  return static_cast<int>(__float_as_uint(f16_bits_to_f32(max(bits, 1u))) >> 23) - 127;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((127 + e) << 23); }

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
  int first;               // first key that some row sees
  int t0, nt;              // first tile of 128 keys, number of tiles
};

// Workspace of split units: a descriptor per unit, then per CTA kRowsCta rows of D sums, m and l.
struct JoinDesc {
  int32_t parts;  // CTAs with a part; 0: no such unit, 1: already done
  int32_t q0, rows, row0, head;
  int32_t pad[3];
};
__host__ __device__ constexpr int64_t part_floats(int dim) {
  return static_cast<int64_t>(kRowsCta) * (dim + 2);
}
constexpr int kLeastTiles = 4;  // tiles of a part, against the fixed cost of a CTA

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

// One row's 128 scores: p = 2^(s ks + up) as binary16 pairs (times the key's value scale where
// C::kScaleP), their sum, and the largest exponent. ks from shared memory where C::kKeyScale,
// else `k1`. kMask: only keys low < pos <= lim count that `there` has.
template <class C, bool kMask>
__device__ __forceinline__ float row_pass(uint32_t t_s, uint32_t vs, float k1, float up, int pos0,
                                          int lim, int low, const uint32_t* there,
                                          uint32_t (&p)[kN / 64][32], float2& sum) {
  const float2 up2 = make_float2(up, up), k2 = make_float2(k1, k1);
  float mx = -INFINITY;
  sum = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int c = 0; c < kN / 32; ++c) {
    uint32_t v[32];
    tmem_ld32(t_s + 32 * c, v);
    tmem_wait_ld();
    uint32_t bits = 0;
    if (kMask) bits = there[c];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float2 ka = k2, kb = k2;
      if (C::kKeyScale) {
        const float4 ks = lds_f4(vs + (32 * c + 4 * q) * 4);
        ka = make_float2(ks.x, ks.y);
        kb = make_float2(ks.z, ks.w);
      }
      float2 s0 = __ffma2_rn(make_float2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])),
                             ka, up2);
      float2 s1 = __ffma2_rn(make_float2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])),
                             kb, up2);
      if (kMask) {
        const int pos = pos0 + 32 * c + 4 * q;
        if (pos > lim || pos <= low || !((bits >> (4 * q)) & 1u)) s0.x = -INFINITY;
        if (pos + 1 > lim || pos + 1 <= low || !((bits >> (4 * q + 1)) & 1u)) s0.y = -INFINITY;
        if (pos + 2 > lim || pos + 2 <= low || !((bits >> (4 * q + 2)) & 1u)) s1.x = -INFINITY;
        if (pos + 3 > lim || pos + 3 <= low || !((bits >> (4 * q + 3)) & 1u)) s1.y = -INFINITY;
      }
      mx = fmaxf(fmaxf(mx, fmaxf(s0.x, s0.y)), fmaxf(s1.x, s1.y));
      float2 p0 = make_float2(ex2(s0.x), ex2(s0.y));
      float2 p1 = make_float2(ex2(s1.x), ex2(s1.y));
      sum = __fadd2_rn(p0, sum);
      sum = __fadd2_rn(p1, sum);
      if (C::kScaleP) {
        const float4 sv = lds_f4(vs + (C::kSvAt + 32 * c + 4 * q) * 4);
        p0 = __fmul2_rn(p0, make_float2(sv.x, sv.y));
        p1 = __fmul2_rn(p1, make_float2(sv.z, sv.w));
      }
      p[c >> 1][16 * (c & 1) + 2 * q] = half2_bits(p0.x, p0.y);
      p[c >> 1][16 * (c & 1) + 2 * q + 1] = half2_bits(p1.x, p1.y);
    }
  }
  return mx;
}

// The same where every key has its own E, without `p`: 32 scores at a time. The largest exponent
// s ks + E first; then, m being settled, p = 2^(s ks + E + up) to TMEM in place of the scores (of
// keys that have been read) and the sum of p 2^-E.
template <class C, class F>
__device__ __forceinline__ void own_exponents(uint32_t t_s, uint32_t vs, float k1, int c, F use) {
  uint32_t v[32];
  tmem_ld32(t_s + 32 * c, v);
  tmem_wait_ld();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float4 ks = make_float4(k1, k1, k1, k1);
    if (C::kKeyScale) ks = lds_f4(vs + (32 * c + 4 * q) * 4);
    const float4 e = lds_f4(vs + (C::kEAt + 32 * c + 4 * q) * 4);
    use(4 * q, fmaf(__uint_as_float(v[4 * q]), ks.x, e.x), e.x);
    use(4 * q + 1, fmaf(__uint_as_float(v[4 * q + 1]), ks.y, e.y), e.y);
    use(4 * q + 2, fmaf(__uint_as_float(v[4 * q + 2]), ks.z, e.z), e.z);
    use(4 * q + 3, fmaf(__uint_as_float(v[4 * q + 3]), ks.w, e.w), e.w);
  }
}
template <class C>
__device__ __forceinline__ float own_max(uint32_t t_s, uint32_t vs, float k1, int pos0, int lim,
                                         int low, const uint32_t* there) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < kN / 32; ++c) {
    const uint32_t bits = there[c];
    own_exponents<C>(t_s, vs, k1, c, [&](int i, float x, float) {
      const int pos = pos0 + 32 * c + i;
      if (pos <= lim && pos > low && ((bits >> i) & 1u)) mx = fmaxf(mx, x);
    });
  }
  return mx;
}
template <class C>
__device__ __forceinline__ float own_store(uint32_t t_s, uint32_t vs, float k1, float up, int pos0,
                                           int lim, int low, const uint32_t* there) {
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < kN / 32; ++c) {
    const uint32_t bits = there[c];
    float h[32];
    own_exponents<C>(t_s, vs, k1, c, [&](int i, float x, float e) {
      const int pos = pos0 + 32 * c + i;
      const float p = pos <= lim && pos > low && ((bits >> i) & 1u) ? ex2(x + up) : 0.0f;
      sum = fmaf(p, ex2(-e), sum);
      h[i] = p;
      if (C::kScaleP) h[i] *= __uint_as_float(lds32(vs + (C::kSvAt + 32 * c + i) * 4));
    });
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = half2_bits(h[2 * i], h[2 * i + 1]);
    tmem_st16(t_s + 16 * c, w);
    tmem_wait_st();
  }
  return sum;
}

// kJoin: units may be split. (A kernel of its own: with the choice at run time the loop of the
// unsplit one was compiled 8 % slower.)
template <int D, int G, bool kBf16, bool kJoin>
__global__ void __launch_bounds__(kThreads, 1)
kv4_prompt_kernel(const Kv4AttnArgs a, int splits_arg) {
  const int splits = kJoin ? splits_arg : 1;
  using C = Cfg<D, G, kBf16>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;                      // [2][atom][128 rows][128 B]
  uint8_t* sK = sQ + 2 * C::kQBytes;       // [2: buffer, or hi and lo][atom][128 keys][128 B]
  uint8_t* sV = sK + 2 * C::kTBytes;       // [2: as for K][2 atoms of 64 keys][D rows][128 B]
  uint8_t* rawK = sV + 2 * C::kTBytes;     // [128 rows of K codes][K scale words][V's]
  uint8_t* rawV = rawK + C::kRawK;         // [128 rows of V codes][V scale words]
  float* vec = reinterpret_cast<float*>(rawV + C::kRawV);  // [4][ks, S_v 2^-E, E][128]
  Ctl* ctl = reinterpret_cast<Ctl*>(vec + 4 * C::kVecFloats);
  // (broadcast, so that the compiler knows the roles' branches, and the operands of the MMAs,
  // to be the same for a whole warp)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // --- which unit: the CTA's index in the line of all requests' (row tile, KV head) pairs
  {
    const int per = (a.requests + kThreads - 1) / kThreads;
    const int64_t r0 = static_cast<int64_t>(threadIdx.x) * per;
    int64_t mine = 0;
    for (int64_t b = r0; b < r0 + per && b < a.requests; ++b) {
      mine += static_cast<int64_t>(request_tiles(a, static_cast<int>(b))) * a.cache.kv_heads;
      if (blockIdx.x == 0 && !kv4_starts_ok(a, b)) set_status(a.status, kStRange);
    }
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
    const int64_t want = blockIdx.x / splits;
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
      mbar_init(&ctl->rk_full, 1);
      mbar_init(&ctl->rk_empty, 4);
      mbar_init(&ctl->rv_full, 1);
      mbar_init(&ctl->rv_empty, 4);
      mbar_init(&ctl->o_full, 1);
      ctl->abort = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  if (kJoin) pdl_launch_dependents();
  const int split = kJoin ? blockIdx.x % splits : 0;
  JoinDesc* desc = static_cast<JoinDesc*>(a.workspace) + blockIdx.x / splits;
  if (ctl->b < 0) {
    if (kJoin && split == 0 && threadIdx.x == 0) desc->parts = 0;
    return;
  }

  const int b = ctl->b, head = ctl->head;
  Unit u;
  int parts = 1;
  {
    int qn;
    request_rows(a, b, u.q0, qn);
    const int kv = a.kv_lens[b];
    u.kv = kv < 0 ? 0 : kv < kKv4MaxKeys ? kv : kKv4MaxKeys;
    if (u.kv == kKv4MaxKeys && threadIdx.x == 0) set_status(a.status, kStRange);
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
    u.first = static_cast<int>(first);
    u.t0 = u.first / kN;
    const int64_t last_tile = (end + kN - 1) / kN;
    u.nt = last_tile > u.t0 ? static_cast<int>(last_tile - u.t0) : 1;
    if (kJoin) {  // this CTA's share of the unit's tiles
      parts = (u.nt + kLeastTiles - 1) / kLeastTiles;
      if (parts > splits) parts = splits;
      if (split == 0 && threadIdx.x == 0) *desc = {parts, u.q0, u.rows, u.row0, head, {0, 0, 0}};
      if (split >= parts) return;
      const int from = static_cast<int>(static_cast<int64_t>(u.nt) * split / parts);
      u.nt = static_cast<int>(static_cast<int64_t>(u.nt) * (split + 1) / parts) - from;
      u.t0 += from;
    }
  }
  if (warp == 12) {
    tmem_alloc(&ctl->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;

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
    auto rescale = [&](float f) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(t_o + 32 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
        tmem_st32(t_o + 32 * c, v);
      }
      // it may run again in this step, and a load is not ordered behind a store in flight
      tmem_wait_st();
    };
    for (int j = 0; j < u.nt; ++j) {
      if (!wait_warp(&ctl->s_full[i], j & 1, ctl, a.status) ||
          !wait_warp(&ctl->vec_full[j & 3], (j >> 2) & 1, ctl, a.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t vs = vec_s + (j & 3) * C::kVecFloats * 4;
      const uint32_t* there = ctl->there[j & 3];
      const int pos0 = (u.t0 + j) * kN;
      const bool safe = pos0 + kN <= safe_end && pos0 >= safe_begin &&
                        (there[0] & there[1] & there[2] & there[3]) == 0xFFFFFFFFu;
      const int e = ctl->exponent[j & 3];
      const int low = a.window > 0 ? lim - a.window : -1;
      // m moves to a row's largest exponent
      auto move = [&](float to) {
        const float f = to == -INFINITY || m == to ? 1.0f : ex2(m - to);
        m = to;
        l *= f;
        if (j > 0) rescale(f);
      };
      if (e != kEach) {
        const float lift = kLift + static_cast<float>(e);
        uint32_t p[kN / 64][32];
        float2 sum;
        // two passes settle any scores that fp32 can tell apart; the bound ends it for others
        for (int pass = 0; pass < 3; ++pass) {
          const float ref = m == -INFINITY ? 0.0f : m;
          const float mx =
              safe ? row_pass<C, false>(t_s, vs, a.scale_log2, lift - ref, 0, 0, 0, there, p, sum)
                   : row_pass<C, true>(t_s, vs, a.scale_log2, lift - ref, pos0, lim, low, there, p,
                                       sum);
          // mx is relative to m: above kLift + kHeadroom m has to move (from -inf: always)
          const bool over = m == -INFINITY ? mx > -INFINITY : mx > kLift + kHeadroom;
          if (!__any_sync(0xffffffffu, over)) break;
          move(fmaxf(m, ref + (mx - kLift)));
        }
        l += (sum.x + sum.y) * pow2(-e);
#pragma unroll
        for (int c = 0; c < kN / 64; ++c) tmem_st32(t_s + 32 * c, p[c]);
      } else {
        const float mx = own_max<C>(t_s, vs, a.scale_log2, pos0, lim, low, there);
        if (__any_sync(0xffffffffu, mx > m + kHeadroom)) move(fmaxf(m, mx));
        l += own_store<C>(t_s, vs, a.scale_log2, kLift - (m == -INFINITY ? 0.0f : m), pos0, lim, low,
                          there);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->p_full[i]);
    }
    // --- the rows' results
    if (ok && wait_warp(&ctl->o_full, 0, ctl, a.status)) {
      tc_fence_after();
      if (kJoin && parts > 1) {
        float* dst = reinterpret_cast<float*>(static_cast<JoinDesc*>(a.workspace) +
                                              gridDim.x / splits) +
                     blockIdx.x * part_floats(D);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(t_o + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(dst + (i * kM + r) * D + 32 * c + q) =
                make_float4(__uint_as_float(v[q]), __uint_as_float(v[q + 1]),
                            __uint_as_float(v[q + 2]), __uint_as_float(v[q + 3]));
        }
        dst[kRowsCta * D + i * kM + r] = m;
        dst[kRowsCta * (D + 1) + i * kM + r] = l;
      } else {
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
    }
  } else if (warp < 12) {
    reg_dec<kRegsExpand>();
    // ------------------------------------------------------------------------ expand
    const int e = threadIdx.x - 256;  // 0..127: the key of K that this thread expands
    // V: an octet of keys, and the column group vg whose bytes hold dimensions 16 n + 2 vg, + 1;
    // eight lanes that store together differ in row mod 8 or octet, so on banks
    constexpr int VB = D / 16;  // bytes of a column group
    const int vg = (lane & 3) | ((lane >> 1) & 4);                              // lane bits 0, 1, 3
    const int vo = 4 * (warp - 8) + (((lane >> 2) & 1) | ((lane >> 3) & 2));    // lane bits 2, 4
    const uint32_t rk = smem_u32(rawK), rv = smem_u32(rawV);
    const uint32_t rk_sz = rk + kN * (D / 2), rk_szv = rk_sz + kN * 4 * G, rv_sz = rv + kN * (D / 2);
    const uint32_t sK0 = smem_u32(sK), sV0 = smem_u32(sV), vec0 = smem_u32(vec);
    for (int j = 0; j < u.nt; ++j) {
      const int kb = C::kKBufs == 2 ? j & 1 : 0, vb = C::kVBufs == 2 ? j & 1 : 0;
      if (!wait_warp(&ctl->rk_full, j & 1, ctl, a.status)) break;
      if (j >= C::kKBufs &&
          !wait_warp(&ctl->k_empty[kb], (j / C::kKBufs - 1) & 1, ctl, a.status))
        break;
      // what lies where no key is may be anything: its scales and zero-points count as 0
      const uint32_t* there = ctl->there[j & 3];
      const bool k_there = (there[warp - 8] >> lane) & 1u;
      // E of the tile, before anything that uses it: S_v 2^-E is below 2 where it meets p
      // (p <= 2^14), below 2^5 where it meets the codes
      int exponent;
      {
        const uint32_t four = there[lane >> 3] >> (4 * (lane & 7));
        uint32_t top[4] = {0, 0, 0, 0};  // binary16 patterns >= 0 compare as integers
#pragma unroll
        for (int i = 0; i < G; ++i) {  // G words of each of the lane's four keys
          const uint4 x = lds128(rk_szv + 16 * (G * lane + i));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            top[(4 * i + q) / G] = max(top[(4 * i + q) / G], w[q] & 0xFFFFu);
        }
        uint32_t most = 0, least = 0x7C00u;
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if ((four >> q) & 1u) {
            most = max(most, top[q]);
            least = min(least, top[q]);
          }
        most = __reduce_max_sync(0xffffffffu, most);  // alike in the four warps
        least = __reduce_min_sync(0xffffffffu, least);
        exponent = half_exponent(most) - C::kTop;
        if (half_exponent(most) - half_exponent(least) > kApart) exponent = kEach;
        if (e == 0) ctl->exponent[j & 3] = exponent;
      }
      const float down = exponent == kEach ? 0.0f : pow2(-exponent);
      {
        uint32_t words[G], zz[G], zh[G], sh[G], sl[G];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          words[i] = k_there ? lds32(rk_sz + 4 * (G * e + i)) : 0u;
          top = max(top, words[i] & 0xFFFFu);
        }
        // binary16 parts: the key's exponent, S_k 2^-ek (q - Z) < 2^16
        const int ek = C::kSplitK && !kBf16 ? half_exponent(top) - 11 : 0;
        const float ks = C::kSplitK ? pow2(ek) : f16_bits_to_f32(top);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const uint32_t z = words[i] >> 16, z2 = z | z << 16;
          const float s = f16_bits_to_f32(words[i] & 0xFFFFu);
          // Z as a binary16 integer: to Z + 128 in bf16, Z + 1024 and -(Z + 64) in binary16
          if (kBf16) {
            const float zf = f16_bits_to_f32(z) + 128.0f;
            zz[i] = pack_bf16x2(zf, zf);
            sh[i] = pack_bf16x2(s, s);  // S = sh + sl, 8 bits and the other 3
            const float rest = s - bf16_lo(sh[i]);
            sl[i] = pack_bf16x2(rest, rest);
          } else {
            zz[i] = hfma2(z2, 0x3C003C00u, 0x64006400u);
            zh[i] = hfma2(z2, 0xBC00BC00u, 0xD400D400u);
            sh[i] = half2_bits(s * pow2(-ek), s * pow2(-ek));
          }
        }
        const uint32_t dst = sK0 + kb * C::kTBytes + e * 128;
#pragma unroll 1  // (the roles' code shares the instruction cache: 643 us unrolled, 614 so)
        for (int c = 0; c < 4; ++c) {
          // stored words cc (D/32) + q of the row are words 4 q + cc of its dimensions; lanes
          // begin with different cc, so that the rows (D/2 bytes apart) do not meet on banks
          const int cc = (c + (e >> 1)) & 3;
          uint32_t w[D / 32];
          if (D == 128) {
            const uint4 x = lds128(rk + e * (D / 2) + 16 * cc);
            w[0] = x.x, w[1] = x.y, w[D / 32 - 2] = x.z, w[D / 32 - 1] = x.w;
          } else {
            const uint2 x = lds64(rk + e * (D / 2) + 8 * cc);
            w[0] = x.x, w[1] = x.y;
          }
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            const int n = 4 * q + cc;  // chunk: dimensions 8 n .. 8 n + 7
            constexpr int kPer = D / 32 / G > 0 ? D / 32 / G : 1;
            const int gi = q / kPer;
            const uint4 x = expand_k<kBf16>(w[q], zz[gi], zh[gi]);
            const uint32_t at = dst + (n >> 3) * (kN * 128) + (((n & 7) ^ (e & 7)) << 4);
            if (!C::kSplitK) {
              sts128(at, x);
            } else {
              const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (kBf16) {
                  hi[k] = bfma2(xs[k], sh[gi], 0x80008000u);
                  lo[k] = bfma2(xs[k], sl[gi], bfma2(xs[k], sh[gi], hi[k] ^ 0x80008000u));
                } else {
                  hi[k] = hfma2(xs[k], sh[gi], 0x80008000u);
                  lo[k] = hfma2(xs[k], sh[gi], hi[k] ^ 0x80008000u);
                }
              }
              sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
              sts128(at + C::kTBytes, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            }
          }
        }
        const uint32_t vs = vec0 + (j & 3) * C::kVecFloats * 4 + e * 4;
        if (C::kKeyScale) sts_f32(vs, ks * a.scale_log2);
        if (C::kScaleP || exponent == kEach) {
          uint32_t sv = 0;
#pragma unroll
          for (int i = 0; i < G; ++i)
            if (k_there) sv = max(sv, lds32(rk_szv + 4 * (G * e + i)) & 0xFFFFu);
          const int own = exponent == kEach ? half_exponent(sv) - C::kTop : exponent;
          if (C::kScaleP) sts_f32(vs + C::kSvAt * 4, f16_bits_to_f32(sv) * pow2(-own));
          if (exponent == kEach) sts_f32(vs + C::kEAt * 4, static_cast<float>(own));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->k_full[kb]);
          mbar_arrive(&ctl->vec_full[j & 3]);
          mbar_arrive(&ctl->rk_empty);
        }
      }
      if (!wait_warp(&ctl->rv_full, j & 1, ctl, a.status)) break;
      if (j >= C::kVBufs &&
          !wait_warp(&ctl->v_empty[vb], (j / C::kVBufs - 1) & 1, ctl, a.status))
        break;
      {
        uint32_t vw[8][VB / 4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int flip = (D == 128 && (k & 2)) ? 32 : 0;
          const uint32_t at = rv + (8 * vo + k) * (D / 2) + ((VB * vg) ^ flip);
          if (VB == 8) {
            const uint2 x = lds64(at);
            vw[k][0] = x.x;
            vw[k][VB / 4 - 1] = x.y;
          } else {
            vw[k][0] = lds32(at);
          }
        }
        const uint32_t eight = there[vo >> 2] >> (8 * (vo & 3));
        uint32_t zz[G][4], zh[G][4], sv[G][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w0[G], w1[G], top0 = 0, top1 = 0;
#pragma unroll
          for (int i = 0; i < G; ++i) {
            w0[i] = lds32(rv_sz + 4 * (G * (8 * vo + 2 * k) + i));
            w1[i] = lds32(rv_sz + 4 * (G * (8 * vo + 2 * k + 1) + i));
            if (!((eight >> (2 * k)) & 1u)) w0[i] = 0;
            if (!((eight >> (2 * k + 1)) & 1u)) w1[i] = 0;
            top0 = max(top0, w0[i] & 0xFFFFu);
            top1 = max(top1, w1[i] & 0xFFFFu);
          }
          float d0 = down, d1 = down;
          if (!C::kScaleP && exponent == kEach) {
            d0 = pow2(C::kTop - half_exponent(top0));
            d1 = pow2(C::kTop - half_exponent(top1));
          }
#pragma unroll
          for (int i = 0; i < G; ++i) {
            const uint32_t z2 = __byte_perm(w0[i], w1[i], 0x7632);
            zz[i][k] = hfma2(z2, 0x3C003C00u, 0x64006400u);
            zh[i][k] = hfma2(z2, 0xBC00BC00u, 0xD400D400u);
            if (!C::kScaleP)
              sv[i][k] = half2_bits(f16_bits_to_f32(w0[i] & 0xFFFFu) * d0,
                                    f16_bits_to_f32(w1[i] & 0xFFFFu) * d1);
          }
        }
        const uint32_t dst = sV0 + vb * C::kTBytes + (vo >> 3) * (D * 128);
#pragma unroll
        for (int n = 0; n < VB; ++n) {  // byte n: dimensions 16 n + 2 vg (low nibble), + 1
          const int gi = n * G / VB;
          const int d0 = 16 * n + 2 * vg;
          uint32_t x[2][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t y = __byte_perm(vw[2 * k][n >> 2], vw[2 * k + 1][n >> 2],
                                           static_cast<uint32_t>(n & 3) |
                                               (static_cast<uint32_t>(4 + (n & 3)) << 8));
            x[0][k] = hsub2(and_or(y, 0x000F000Fu, 0x64006400u), zz[gi][k]);
            x[1][k] = hfma2(and_or(y, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh[gi][k]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = dst + (d0 + h) * 128 + (((vo & 7) ^ ((d0 + h) & 7)) << 4);
            uint32_t hi[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              hi[k] = C::kScaleP ? x[h][k] : hfma2(x[h][k], sv[gi][k], 0x80008000u);
            sts128(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            if (C::kSplitV) {
#pragma unroll
              for (int k = 0; k < 4; ++k) hi[k] = hfma2(x[h][k], sv[gi][k], hi[k] ^ 0x80008000u);
              sts128(at + C::kTBytes, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->v_full[vb]);
          mbar_arrive(&ctl->rv_empty);
        }
      }
    }
  } else {
    reg_dec<kRegsIssue>();
    if (warp == 12) {
      // -------------------------------------------------------------------- MMA issuer
      constexpr uint32_t kFmt = kBf16 ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t kIdescS = (1u << 4) | kFmt | ((kN >> 3) << 17) | ((kM >> 4) << 24);
      constexpr uint32_t kIdescO = (1u << 4) | ((D >> 3) << 17) | ((kM >> 4) << 24);
      const bool leader = elect_one();
      const uint32_t q_lo = sw128_desc_lo(sQ), k_lo = sw128_desc_lo(sK), v_lo = sw128_desc_lo(sV);
      auto scores = [&](int i, int buf) {
        const uint32_t qd = q_lo + i * (C::kQBytes >> 4), kd = k_lo + buf * (C::kTBytes >> 4);
#pragma unroll
        for (int part = 0; part < (C::kSplitK ? 2 : 1); ++part)
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = ((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
            tc_mma_lo(tmem + i * kN, qd + at, kd + part * (C::kTBytes >> 4) + at, kIdescS,
                      (part | k) != 0);
          }
        tc_commit(&ctl->s_full[i]);
      };
      bool ok = wait_warp(&ctl->q_full[0], 0, ctl, a.status) &&
                wait_warp(&ctl->q_full[1], 0, ctl, a.status) &&
                wait_warp(&ctl->k_full[0], 0, ctl, a.status);
      if (ok) {
        tc_fence_after();
        if (leader) {
          scores(0, 0);
          scores(1, 0);
          tc_commit(&ctl->k_empty[0]);
        }
      }
      for (int j = 0; j < u.nt && ok; ++j) {
        const int vb = C::kVBufs == 2 ? j & 1 : 0;
        const int kb = C::kKBufs == 2 ? (j + 1) & 1 : 0;  // of the next keys
        const bool more = j + 1 < u.nt;
        const uint32_t vd = v_lo + vb * (C::kTBytes >> 4);
        ok = wait_warp(&ctl->v_full[vb], (j / C::kVBufs) & 1, ctl, a.status);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ok = ok && wait_warp(&ctl->p_full[i], j & 1, ctl, a.status);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int part = 0; part < (C::kSplitV ? 2 : 1); ++part)
#pragma unroll
              for (int k = 0; k < kN / 16; ++k)
                tc_mma_tmem_a_lo(tmem + 2 * kN + i * 128, tmem + i * kN + 8 * k,
                                 vd + ((part * C::kTBytes + (k >> 2) * (D * 128) + (k & 3) * 32) >> 4),
                                 kIdescO, (part | k) != 0 ? 1u : j != 0);
          }
          if (more) {
            if (i == 0) {
              ok = wait_warp(&ctl->k_full[kb], ((j + 1) / C::kKBufs) & 1, ctl, a.status);
              if (!ok) break;
              tc_fence_after();
            }
            if (leader) scores(i, kb);
          }
        }
        if (!ok) break;
        if (leader) {
          tc_commit(&ctl->v_empty[vb]);
          if (more) tc_commit(&ctl->k_empty[kb]);
        }
      }
      // all issued MMAs have completed once this arrives
      if (leader) tc_commit(&ctl->o_full);
      if (!mbar_wait_bounded(&ctl->o_full, 0, kLimitNs)) set_status(a.status, kStTimeout);
    } else if (warp == 13) {
      // ---------------------------------------------------------------------- producer
      // Bulk copies of a tile's pieces (of blocks, or of 128 keys of longer ones): lane p takes
      // piece p, for K as soon as the expand warps have read the last tile's, then for V.
      const Kv4Cache& kc = a.cache;
      const int plog = kc.block_log2 < 7 ? kc.block_log2 : 7;
      const int piece = 1 << plog, pieces = kN >> plog;
      const int64_t codes = static_cast<int64_t>(kc.block) * (D / 2);
      const int32_t* table = a.tables + b * a.ld_tables;
      auto pos_of = [&](int j) { return (u.t0 + j) * kN + lane * piece; };  // <= 2^30 + a tile
      // pieces that some row sees a key of: below `high`, above `low` (blocks that end before the
      // first key seen may be gone: their entries are not read)
      const int high = lane < pieces ? u.kv : 0, low = u.first - piece;
      auto needed = [&](int pos) { return pos < high && pos > low; };
      auto block_of = [&](int j) -> int {  // -1 too where the table does not reach
        const int place = pos_of(j) >> kc.block_log2;
        return needed(pos_of(j)) && place < a.width ? __ldg(table + place) : -1;
      };
      int next = block_of(0), j = 0;
      bool ok = true;
      for (; j < u.nt; ++j) {
        const int blk = next;
        if (j + 1 < u.nt) next = block_of(j + 1);
        const bool good = blk >= 0 && blk < kc.num_blocks;
        const int pos = pos_of(j);
        if (!good && needed(pos)) set_status(a.status, kStRange);
        const uint32_t copied = __ballot_sync(0xffffffffu, good), n = __popc(copied);
        // the keys that exist, 32 a word: lanes 0 .. 3 (made ahead of the wait: behind it, key by
        // key, they held up the copies, 649 us for the chunk above)
        const int key = 32 * (lane & 3), left = u.kv - (u.t0 + j) * kN - key;
        uint32_t bits = ((copied >> (key >> plog)) & 1u ? 0xFFFFu : 0u) |
                        ((copied >> ((key + 16) >> plog)) & 1u ? 0xFFFF0000u : 0u);
        bits &= left >= 32 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << left) - 1u;
        const int at = pos & (kc.block - 1);
        const uint8_t* src =
            kc.data + (static_cast<int64_t>(good ? blk : 0) * kc.kv_heads + head) * kc.chunk_bytes();
        const uint8_t* szk = src + 2 * codes + at * 4 * G;
        const uint8_t* szv = szk + kc.block * 4 * G;
        if (j > 0 && !wait_warp(&ctl->rk_empty, (j - 1) & 1, ctl, a.status)) {
          ok = false;
          break;
        }
        if (lane < 4) ctl->there[j & 3][lane] = bits;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&ctl->rk_full, n * piece * (D / 2 + 8 * G));
        __syncwarp();
        if (good) {
          bulk_g2s(rawK + lane * piece * (D / 2), src + at * (D / 2), piece * (D / 2), &ctl->rk_full);
          bulk_g2s(rawK + kN * (D / 2) + lane * piece * 4 * G, szk, piece * 4 * G, &ctl->rk_full);
          bulk_g2s(rawK + kN * (D / 2 + 4 * G) + lane * piece * 4 * G, szv, piece * 4 * G,
                   &ctl->rk_full);
        }
        if (j > 0 && !wait_warp(&ctl->rv_empty, (j - 1) & 1, ctl, a.status)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&ctl->rv_full, n * piece * (D / 2 + 4 * G));
        __syncwarp();
        if (good) {
          bulk_g2s(rawV + lane * piece * (D / 2), src + codes + at * (D / 2), piece * (D / 2),
                   &ctl->rv_full);
          bulk_g2s(rawV + kN * (D / 2) + lane * piece * 4 * G, szv, piece * 4 * G, &ctl->rv_full);
        }
      }
      // never leave with copies in flight: the last tile that each buffer was asked for
      const int last_k = ok ? u.nt - 1 : j, last_v = ok ? u.nt - 1 : j - 1;
      if (!mbar_wait_bounded(&ctl->rk_full, last_k & 1, kLimitNs) ||
          (last_v >= 0 && !mbar_wait_bounded(&ctl->rv_full, last_v & 1, kLimitNs)))
        set_status(a.status, kStTimeout);
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

// Rows of a split unit: out = sum_i O_i 2^(m_i - m) / l over its parts i, one warp a row.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) kv4_join_kernel(const Kv4AttnArgs a, int units, int splits) {
  pdl_wait();
  const JoinDesc d = static_cast<const JoinDesc*>(a.workspace)[blockIdx.x];
  const int lane = threadIdx.x & 31, row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int rr = d.row0 + row;
  if (d.parts <= 1 || rr >= d.rows) return;
  constexpr int V = D / 32;
  const float* base = reinterpret_cast<const float*>(
                          static_cast<const JoinDesc*>(a.workspace) + units) +
                      static_cast<int64_t>(blockIdx.x) * splits * part_floats(D);
  float m = -INFINITY;
  for (int i = lane; i < d.parts; i += 32)
    m = fmaxf(m, base[i * part_floats(D) + kRowsCta * D + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f, o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < d.parts; ++i) {
    const float* p = base + i * part_floats(D);
    const float x = p[kRowsCta * D + row];
    const float f = x == -INFINITY ? 1.0f : ex2(x - m);  // O and l are 0 there, or NaN
    l += f * p[kRowsCta * (D + 1) + row];
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      const float2 v = *reinterpret_cast<const float2*>(p + row * D + V * lane + k);
      o[k] += f * v.x;
      o[k + 1] += f * v.y;
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int tok = rr / a.ratio, h = d.head * a.ratio + rr - tok * a.ratio;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(d.q0 + tok) * a.o_tok +
                                              static_cast<int64_t>(h) * a.o_head);
#pragma unroll
  for (int k = 0; k < V; k += 2) dst[(V * lane + k) >> 1] = narrow2<kBf16>(o[k] * inv, o[k + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(d.q0 + tok) * a.heads + h] =
        l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
}

template <int D, int G, bool kBf16, bool kJoin>
cudaError_t launch_t(const Kv4AttnArgs& a, int64_t units, int splits, cudaStream_t st) {
  using C = Cfg<D, G, kBf16>;
  auto kern = kv4_prompt_kernel<D, G, kBf16, kJoin>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr[dev & 63].load(std::memory_order_acquire)) {
    e = set_smem_attrs(kern, C::kSmem);
    if (e != cudaSuccess) return e;
    attr[dev & 63].store(true, std::memory_order_release);
  }
  kern<<<static_cast<unsigned>(units * splits), kThreads, C::kSmem, st>>>(a, splits);
  e = cudaGetLastError();
  if (e != cudaSuccess || !kJoin) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units), kRowsCta / 8, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, kBf16>, a, static_cast<int>(units), splits);
}

template <int D, int G>
cudaError_t launch_g(const Kv4AttnArgs& a, int64_t units, int splits, cudaStream_t st) {
  if (splits > 1)
    return a.bf16 ? launch_t<D, G, true, true>(a, units, splits, st)
                  : launch_t<D, G, false, true>(a, units, splits, st);
  return a.bf16 ? launch_t<D, G, true, false>(a, units, 1, st)
                : launch_t<D, G, false, false>(a, units, 1, st);
}

}  // namespace

size_t kv4_prompt_workspace_bytes(int sms) {
  return static_cast<size_t>(sms) * (sizeof(JoinDesc) + part_floats(128) * sizeof(float));
}

int64_t kv4_prompt_units(int64_t tokens, int64_t ratio, int64_t requests, int64_t kv_heads) {
  return (tokens * ratio / kRowsCta + requests) * kv_heads;
}

cudaError_t launch_kv4_prompt(const Kv4AttnArgs& a, int sms, cudaStream_t st) {
  const int64_t units = kv4_prompt_units(a.tokens, a.ratio, a.requests, a.cache.kv_heads);
  // (units splits <= sms, for which the workspace is made)
  const int splits = units < sms ? static_cast<int>(sms / units) : 1;
  const int groups = a.cache.groups();
  if (a.cache.dim == 128) {
    if (groups == 1) return launch_g<128, 1>(a, units, splits, st);
    return groups == 2 ? launch_g<128, 2>(a, units, splits, st)
                       : launch_g<128, 4>(a, units, splits, st);
  }
  return groups == 1 ? launch_g<64, 1>(a, units, splits, st)
                     : launch_g<64, 2>(a, units, splits, st);
}

}  // namespace wq
