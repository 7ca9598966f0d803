// Attention over the 4-bit KV cache for few query rows (decode, drafted tokens), and for any
// call that the prompt kernel does not take. A row is one (token, query head) of a KV head's
// group of `ratio` query heads.
//
// Arithmetic. With c = q_code - Z the score of a row x and a token t is
//     s = scale log2(e) sum_g S_k[t,g] (x_g . c_g),
// computed per group as S_k (16 sum x (1 + q/16) - (16 + Z) sum x): the codes stand in the top
// mantissa bits of a 16-bit 1.0 (exact), the products are exact and summed in fp32 by
// mma.sync m16n8k16 with 16 tokens as its rows and 8 query rows as its columns. The softmax is
// taken in one pass with a running reference m. The value's scale joins the exponent:
//     p = 2^(s + log2 S_v - m + 7),   l += p / S_v,   O += p (q_code - Z)
// so p needs no range beyond its own and is rounded once to binary16 (half a step, 2^-11); the
// codes less Z are exact there, and O = sum p c / l. m moves only when a score passes it by
// 2^8 (p <= 2^15 then); everything else is fp32. With several groups a row, S_v is the
// largest of the token's and the others enter p as their ratio to it.
//
// Work split. The tiles of 128 tokens of all (request, KV head, row tile) units form one line,
// cut into equal shares, one per CTA, whatever the lengths are: a ragged batch and one long
// request balance alike, and the host needs no lengths. Each unit also has two empty places on
// the line before its tiles, which is about what its beginning and end cost a CTA: without them,
// CTAs with the short requests of a batch came in last (64 requests of up to 8192 keys: 108 us
// with no, 99 / 98 / 100 with 1 / 2 / 3 places; 48 short ones of up to 3001: 62, 47 / 43 / 41).
// A share that covers a unit only in part leaves (O, m, l) in the workspace, and a second kernel
// (programmatic dependent launch) sums a unit's parts in CTA order, so results do not depend on
// timing.
//
// Data path. A producer warp streams each tile's blocks by bulk copies (one per block of a
// head) through an mbarrier ring; four warps take 32 tokens of every tile each (two MMA blocks
// side by side: with one, a warp waited out the latency of every step), with their own softmax
// state, joined at the end of a unit. A lane turns the scale words of one of the warp's 32
// tokens into the constants of the formulas above (every lane doing that for its own MMA rows,
// four times over, was a tenth of all instructions; the producer doing it for all was late).
//
// Measured: one token over 131072 keys, 64 query and 8 KV heads of 128: 50 us, 2.9 TB/s (45 % of
// a copy), 40 of it with no arithmetic at all: about 13 us are the launch, the search for the
// share, the first copies and the joining kernel, and the copies alone run at 5.3 TB/s. A batch
// of 64 such requests of up to 8192 keys in blocks of 16: 86 us, 3.3 TB/s. With the arithmetic
// the ALU pipe is half busy (shifts, masks and byte permutes: 16 for 16 codes of K, 12 for 16 of
// V) and 12 warps an SM do not hide all latencies.
#include <atomic>

#include "common.cuh"
#include "kv4.h"
#include "kv4_math.cuh"
#include "mma_frag.cuh"
#include "ptx.cuh"

namespace wq {
namespace {

// named_barrier, and whether any of its threads brought `flag`: one answer for all of them.
__device__ __forceinline__ bool named_barrier_or(int id, int threads, bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(flag ? 1u : 0u)
      : "memory");
  return any != 0;
}

constexpr int kTile = 128;  // tokens per tile
constexpr int kTileLog2 = 7;
constexpr int kUnitCost = 2;  // places of a unit on the line before its first tile
constexpr int kWarps = 4;   // consumer warps, 32 tokens of the tile each
constexpr int kThreads = 32 * (kWarps + 1);
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr float kHeadroom = 8.0f;  // m moves when a score passes it by this
constexpr float kLift = 7.0f;      // p is taken times 2^kLift

template <int D, int G, int NT>
struct Cfg {
  static constexpr int kStageBytes = kTile * (D + 8 * G);
  // Constants of a token: k1[G], k2[G], lv, 1 / S_v, S_v,g / S_v (G > 1), padded to 16 bytes;
  // and a word of Z for its values (below).
  static constexpr int kRec = G == 1 ? 4 : G == 2 ? 8 : 16;
  static constexpr int kConstBytes = kTile * 4 * (kRec + G);  // 32 tokens of each warp
  static constexpr int kRows = 8 * NT;
  // by registers and shared memory
  static constexpr int kCtasPerSm = NT == 1 && (G == 1 || D == 64) ? 3 : 2;
  static constexpr int kStages = D == 64 ? 4 : G == 1 && NT == 1 ? 3 : 4;
  static constexpr int kMergeFloats = 2 * kRows * (D + 1);  // two warps' O rows, padded
};

// What one request asks of this kernel.
struct Req {
  int q0, qn, kv;     // first row of Q, rows, keys
  int row_tiles, t0, nt;  // row tiles, first tile of keys, tiles
  int first;              // first key that some row sees
  __device__ int64_t places(int kv_heads) const {
    return static_cast<int64_t>(kv_heads) * row_tiles * (nt + kUnitCost);
  }
};

struct Ctl {
  uint64_t full[8];   // a tile's bytes have landed
  uint64_t empty[8];  // the consumers have read them
  uint32_t pieces[8];  // bit i: piece i of the stage's tile is there
  int32_t left[8];     // keys from the tile's first on
  int64_t scan[kWarps + 1];
  int64_t total;
  int64_t off0;  // tiles of request b0 before this CTA's share
  int b0;
  Req r0;        // that request
  volatile int abort;
  float ml[kWarps][2][32];
};

template <int D, int G, int NT>
constexpr int smem_bytes() {
  using C = Cfg<D, G, NT>;
  return C::kStages * C::kStageBytes + C::kConstBytes + C::kMergeFloats * 4 +
         static_cast<int>(sizeof(Ctl));
}

template <int kRows>
__device__ __forceinline__ Req request(const Kv4AttnArgs& a, int b) {
  Req r;
  int lo = a.q_starts[b], hi = a.q_starts[b + 1];
  lo = lo < 0 ? 0 : lo < a.tokens ? lo : a.tokens;
  hi = hi < lo ? lo : hi < a.tokens ? hi : a.tokens;
  const int kv = a.kv_lens[b];
  r.q0 = lo;
  r.qn = hi - lo;
  r.kv = kv < 0 ? 0 : kv < kKv4MaxKeys ? kv : kKv4MaxKeys;
  const int64_t rows = static_cast<int64_t>(r.qn) * a.ratio;
  r.row_tiles = rows > a.most_rows ? 0 : static_cast<int>((rows + kRows - 1) / kRows);
  int first = 0;
  if (a.window > 0) {
    const int64_t f = static_cast<int64_t>(r.kv) - (a.causal ? r.qn - 1 : 0) - a.window;
    first = f > 0 ? static_cast<int>(f) : 0;
  }
  r.first = first;
  r.t0 = first / kTile;
  // tiles that hold keys and that the table reaches (keys beyond it are left out)
  const int64_t reach = static_cast<int64_t>(a.width) << a.cache.block_log2;
  const int last = r.kv < reach ? r.kv : static_cast<int>(reach);
  const int end = last > 0 ? (last - 1) / kTile + 1 : 0;
  r.nt = end > r.t0 ? end - r.t0 : 1;          // an empty request still has its rows written
  return r;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// (1 + q/16) pairs of a word's codes as bf16 or fp16: out[i] = (code i, code i + 4).
template <bool kBf16>
__device__ __forceinline__ void unpack_hi(uint32_t w, uint32_t (&out)[4]) {
  if (kBf16) {
    unpack_bf16_hi(w, 0x00780078u, 0x3F803F80u, out);
  } else {
    out[0] = and_or(w << 6, 0x03C003C0u, 0x3C003C00u);
    out[1] = and_or(w << 2, 0x03C003C0u, 0x3C003C00u);
    out[2] = and_or(w >> 2, 0x03C003C0u, 0x3C003C00u);
    out[3] = and_or(w >> 6, 0x03C003C0u, 0x3C003C00u);
  }
}
template <bool kBf16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if (kBf16) mma_bf16_16816(d, a, b0, b1);
  else mma_f16_16816(d, a, b0, b1);
}
template <bool kBf16>
__device__ __forceinline__ float sum2(uint32_t w) {
  if (kBf16) return bf16_lo(w) + bf16_hi(w);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return f.x + f.y;
}
template <bool kBf16>
__device__ __forceinline__ uint16_t narrow(float v) {
  if (kBf16) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&h);
  }
  return static_cast<uint16_t>(f32_to_f16_bits(v));
}

// Workspace: per CTA a descriptor of the unit whose parts begin with it, then per CTA two
// parts (0: the share's first unit where it begins inside it, 1: its last) of kRows rows of
// D sums, m and l.
struct Desc {
  int32_t first_row;  // row of the unit's request where the row tile begins, -1: none
  int q0, rows, head;  // request's first row of Q, its rows (tokens x ratio), KV head
  int last_cta;
  int pad[3];  // 32 bytes: the parts behind the descriptors are 16-byte aligned
};
constexpr int kMaxRows = 16;
__host__ __device__ constexpr int part_floats(int dim) { return kMaxRows * (dim + 2); }

// First place of share i of `live` equal ones (a 32-bit division where that suffices: the 64-bit
// one is a subroutine).
__device__ __forceinline__ int64_t share_begin(int64_t total, int live, int i) {
  if (total < (1 << 21))  // live <= 2^11
    return static_cast<uint32_t>(total) * static_cast<uint32_t>(i) / static_cast<uint32_t>(live);
  return total * i / live;
}

template <int D, int G, int NT, bool kBf16>
__global__ void __launch_bounds__(kThreads, Cfg<D, G, NT>::kCtasPerSm)
kv4_decode_kernel(const Kv4AttnArgs a) {
  using C = Cfg<D, G, NT>;
  constexpr int kRows = C::kRows;
  constexpr int kStages = C::kStages;
  constexpr int KW = D / 32;  // K words of a lane's share of a row; one 32-dim step each
  constexpr int VT = D / 16;  // 16-dim tiles of V: one byte of a lane's share each
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* consts = smem + kStages * C::kStageBytes;
  float* merge = reinterpret_cast<float*>(consts + C::kConstBytes);
  Ctl* ctl = reinterpret_cast<Ctl*>(merge + C::kMergeFloats);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], kWarps);
    }
    ctl->abort = 0;
    fence_barrier_init();
  }

  // --- this CTA's share of the line of tiles
  int64_t begin, end;
  int live;
  {
    const int per = (a.requests + kThreads - 1) / kThreads;
    const int64_t r0 = static_cast<int64_t>(threadIdx.x) * per;
    int64_t mine = 0;
    for (int64_t b = r0; b < r0 + per && b < a.requests; ++b) {
      const Req r = request<kRows>(a, static_cast<int>(b));
      mine += r.places(a.cache.kv_heads);
      if (blockIdx.x == 0 && !kv4_starts_ok(a, b)) set_status(a.status, kStRange);
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) ctl->scan[warp] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps + 1; ++w) {
      if (w < warp) before += ctl->scan[w];
      total += ctl->scan[w];
    }
    incl += before;
    live = total < gridDim.x ? static_cast<int>(total) : gridDim.x;
    begin = end = 0;
    if (static_cast<int>(blockIdx.x) < live) {
      begin = share_begin(total, live, blockIdx.x);
      end = share_begin(total, live, blockIdx.x + 1);
    }
    if (threadIdx.x == 0) ctl->total = total;
    if (begin < end && begin >= incl - mine && begin < incl) {  // one thread's requests hold it
      int64_t off = begin - (incl - mine);
      int b = static_cast<int>(r0);
      Req r;
      while (true) {
        r = request<kRows>(a, b);
        const int64_t w = r.places(a.cache.kv_heads);
        if (off < w) break;
        off -= w;
        ++b;
      }
      ctl->b0 = b;
      ctl->off0 = off;
      ctl->r0 = r;
    }
    __syncthreads();
  }
  const int64_t total = ctl->total;
  Desc* descs = static_cast<Desc*>(a.workspace);
  float* parts = reinterpret_cast<float*>(descs + gridDim.x);
  if (threadIdx.x == 0) descs[blockIdx.x].first_row = -1;
  if (begin == end) return;

  const Kv4Cache& kc = a.cache;
  const int piece_log2 = kc.block_log2 < kTileLog2 ? kc.block_log2 : kTileLog2;
  const int piece = 1 << piece_log2;  // tokens of one copied piece
  const int npieces = kTile >> piece_log2;
  const int piece_bytes = piece * (D + 8 * G);

  // Position in the line: request, KV head, row tile, tile. The divisions are made once.
  int b = ctl->b0;
  Req r = ctl->r0;
  int h, rt, t;
  int64_t left = end - begin;  // places from the tile's on
  int64_t line = begin;        // the unit's first place
  {
    const int64_t off = ctl->off0;
    const int each = r.nt + kUnitCost;
    const int unit = off >> 32 ? static_cast<int>(off / each)  // < KV heads x row tiles
                               : static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(each));
    const int place = static_cast<int>(off - static_cast<int64_t>(unit) * each);
    h = unit / r.row_tiles;
    rt = unit - h * r.row_tiles;
    t = place - kUnitCost;
    line -= place;
    if (t < 0) {
      left += t;
      t = 0;
    }
  }
  if (left <= 0) return;  // no tile in the share
  // to the next unit; false if no tile of it is in the share
  auto next_unit = [&]() -> bool {
    line += r.nt + kUnitCost;
    left -= kUnitCost;
    if (left <= 0) return false;
    t = 0;
    if (++rt < r.row_tiles) return true;
    rt = 0;
    if (++h < kc.kv_heads) return true;
    h = 0;
    do {
      r = request<kRows>(a, ++b);
    } while (r.row_tiles == 0);
    return true;
  };

  if (warp == kWarps) {
    // ------------------------------------------------------------------ producer warp
    uint32_t s = 0, phase = 0;  // ring position, and the parity of its fill
    uint32_t it = 0;
    int table_of = -1, first = 0, cached = -1;  // 32 pieces' blocks, read ahead by the lanes
    const int64_t chunk = kc.chunk_bytes();
    const int64_t codes = static_cast<int64_t>(kc.block) * (D / 2);
    const int64_t reach = static_cast<int64_t>(a.width) << kc.block_log2;
    bool ok = true;
    while (true) {
      const int tile = r.t0 + t;
      const int p0 = tile << (kTileLog2 - piece_log2);  // first piece of the tile
      if (table_of != b || p0 < first || p0 + npieces > first + 32) {
        if (table_of != b && (r.kv > reach || r.kv == kKv4MaxKeys)) set_status(a.status, kStRange);
        table_of = b;
        first = p0;
        const int64_t pos = static_cast<int64_t>(p0 + lane) << piece_log2;
        const int64_t place = pos >> kc.block_log2;
        cached = -1;
        // (blocks that end before the first key seen may be gone: their entries are not read)
        if (pos < r.kv && pos + piece > r.first && place < a.width) {
          cached = a.tables[b * a.ld_tables + place];
          if (cached < 0 || cached >= kc.num_blocks) {
            cached = -1;
            set_status(a.status, kStRange);
          }
        }
      }
      const int blk = __shfl_sync(0xffffffffu, cached, (p0 - first + lane) & 31);
      const bool mine = lane < npieces && blk >= 0;
      const uint32_t there = __ballot_sync(0xffffffffu, mine);
      const uint8_t* src = kc.data + (static_cast<int64_t>(blk) * kc.kv_heads + h) * chunk;
      if (it >= kStages) {
        ok = mbar_wait_bounded(&ctl->empty[s], phase ^ 1u, kLimitNs);
        ok = __all_sync(0xffffffffu, ok && !ctl->abort);
        if (!ok) break;
      }
      if (lane == 0) {
        ctl->pieces[s] = there;
        const int64_t n = static_cast<int64_t>(r.kv) - static_cast<int64_t>(tile) * kTile;
        ctl->left[s] = n < 0 ? 0 : n < kTile ? static_cast<int>(n) : kTile;
        mbar_arrive_expect_tx(&ctl->full[s], __popc(there) * piece_bytes);
      }
      __syncwarp();
      if (mine) {
        uint8_t* dst = smem + s * C::kStageBytes + lane * piece_bytes;
        if (kc.block <= kTile) {
          bulk_g2s(dst, src, piece_bytes, &ctl->full[s]);
        } else {  // part of a longer block: its four arrays
          const int at = (tile * kTile) & (kc.block - 1);
          bulk_g2s(dst, src + at * (D / 2), kTile * (D / 2), &ctl->full[s]);
          bulk_g2s(dst + kTile * (D / 2), src + codes + at * (D / 2), kTile * (D / 2),
                   &ctl->full[s]);
          bulk_g2s(dst + kTile * D, src + 2 * codes + at * 4 * G, kTile * 4 * G, &ctl->full[s]);
          bulk_g2s(dst + kTile * (D + 4 * G), src + 2 * codes + (kc.block + at) * 4 * G,
                   kTile * 4 * G, &ctl->full[s]);
        }
      }
      ++it;
      if (++s == kStages) {
        s = 0;
        phase ^= 1u;
      }
      if (--left == 0) break;
      if (++t == r.nt && !next_unit()) break;
    }
    if (!ok && lane == 0) {
      set_status(a.status, kStTimeout);
      ctl->abort = 1;
    }
    // never leave with copies in flight
    if (lane == 0)
      for (uint32_t q = 0; q < kStages && q < it; ++q)
        if (!mbar_wait_bounded(&ctl->full[q], ((it - 1 - q) / kStages) & 1u, kLimitNs))
          set_status(a.status, kStTimeout);
    return;
  }

  // ---------------------------------------------------------------------- consumer warps
  const int g = lane >> 2, c = lane & 3;
  // token (of the warp's 16) that stands in MMA row / k slot rho: chosen so that the rows a
  // warp loads at once, of K (16 bytes a lane) and of V (8), fall on different banks
  auto token_of = [](int rho) { return (rho & 8) + ((rho & 1) ? 4 + (((rho & 7) >> 1) ^ 3) : ((rho & 7) >> 1)); };
  const int tk0 = token_of(g);                        // K rows g (and + 8)
  const int tv0 = token_of(2 * c), tv1 = token_of(2 * c + 1);  // V slots (and + 8)
  const uint32_t stage0 = smem_u32(smem);
  const uint32_t ct = smem_u32(consts) + warp * 32 * 4 * (C::kRec + G);  // the warp's constants
  // the warp's two blocks of 16 tokens within a stage: their rows of K and of V
  uint32_t off_k[2], off_v[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int tok = 32 * warp + 16 * w;
    off_k[w] = (tok >> piece_log2) * piece_bytes + (tok & (piece - 1)) * (D / 2);
    off_v[w] = off_k[w] + piece * (D / 2);
  }
  const int flip0 = (D == 128 && (tv0 & 2)) ? 32 : 0, flip1 = (D == 128 && (tv1 & 2)) ? 32 : 0;

  uint32_t s = 0, phase = 0;
  bool ok = true;
  while (true) {
    {
      // ------------------------------------------------ one unit (or this CTA's part of it)
      const int rows = r.qn * a.ratio;
      const int row0 = rt * kRows;
      const int u_begin = t;
      const int u_end = left < r.nt - t ? t + static_cast<int>(left) : r.nt;

      // Q fragments (B operand), row = 8 n + g, dims 32 j + 8 c .. + 7 per word j
      uint32_t qf[NT][KW][4];
      float xs[NT][G][2];  // sums over each group's dims of rows 2c, 2c + 1
      int lim[NT][2];      // last key seen by rows 2c, 2c + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = row0 + 8 * n + g;
        float sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i) sum[i] = 0.0f;
        const int tok = row / a.ratio;
        const uint16_t* src = a.Q + static_cast<int64_t>(r.q0 + tok) * a.q_tok +
                              static_cast<int64_t>(h * a.ratio + row - tok * a.ratio) * a.q_head;
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < rows) x = ld_nc_u4(src + 32 * j + 8 * c);
          qf[n][j][0] = __byte_perm(x.x, x.z, 0x5410);
          qf[n][j][1] = __byte_perm(x.x, x.z, 0x7632);
          qf[n][j][2] = __byte_perm(x.y, x.w, 0x5410);
          qf[n][j][3] = __byte_perm(x.y, x.w, 0x7632);
          sum[j * G / KW] += sum2<kBf16>(x.x) + sum2<kBf16>(x.y) + sum2<kBf16>(x.z) + sum2<kBf16>(x.w);
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
          xs[n][i][0] = __shfl_sync(0xffffffffu, sum[i], 8 * c);
          xs[n][i][1] = __shfl_sync(0xffffffffu, sum[i], 8 * c + 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rr = row0 + 8 * n + 2 * c + e;
          lim[n][e] = rr >= rows ? -1
                      : a.causal ? r.kv - r.qn + rr / a.ratio : r.kv - 1;
        }
      }
      // keys that every row of the tile sees (warp-uniform): no masks below `safe_end`
      const int last_row = row0 + kRows < rows ? row0 + kRows - 1 : rows - 1;
      const int safe_end = (a.causal ? r.kv - r.qn + row0 / a.ratio : r.kv - 1) + 1;
      const int safe_begin =
          a.window > 0 ? (a.causal ? r.kv - r.qn + last_row / a.ratio : r.kv - 1) - a.window + 1
                       : 0;

      float o[NT][VT][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[n][e] = -INFINITY;
          l[n][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][i][e] = 0.0f;
      }

      for (int tl = u_begin; tl < u_end; ++tl) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&ctl->full[s], phase, kLimitNs))) {
          set_status(a.status, kStTimeout);
          ctl->abort = 1;
          ok = false;
          break;
        }
        const uint32_t st = stage0 + s * C::kStageBytes;
        const int pos0 = (r.t0 + tl) * kTile + 32 * warp;  // first of the warp's 32 tokens
        // (tokens of them that do not exist have lv = -inf, and codes of some kind)
        const int keys = ctl->left[s] - 32 * warp;
        if (keys > 0) {
          // -- constants of token `lane` of the warp's 32
          {
            const int tok = 32 * warp + lane;
            const int pc = tok >> piece_log2;
            const bool in = lane < keys && ((ctl->pieces[s] >> pc) & 1u);
            const uint32_t sz = st + pc * piece_bytes + piece * D + (tok & (piece - 1)) * 4 * G;
            float k[C::kRec];
#pragma unroll
            for (int i = 0; i < C::kRec; ++i) k[i] = 0.0f;
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < G; ++i) {
              const uint32_t ks = in ? lds32(sz + 4 * i) : 0u;
              const uint32_t vz = in ? lds32(sz + (piece * G + i) * 4) : 0u;
              const float sk = f16_bits_to_f32(ks & 0xFFFFu) * a.scale_log2;
              k[i] = 16.0f * sk;
              k[G + i] = sk * (16.0f + f16_bits_to_f32(ks >> 16));
              const float sv = f16_bits_to_f32(vz & 0xFFFFu);
              if (G > 1) k[G > 1 ? 2 * G + 2 + i : 0] = sv;
              top = fmaxf(top, sv);
              // 1024 + Z (low) and -(64 + Z) as binary16: what the two nibbles of a byte are
              // expanded with
              const uint32_t z = vz >> 16;
              sts32(ct + (32 * C::kRec + lane * G + i) * 4,
                    (hfma2(z, 0x3C003C00u, 0x64006400u) & 0xFFFFu) |
                        hfma2(z, 0xBC00BC00u, 0xD400D400u) << 16);
            }
            top = fmaxf(top, 5.9604644775390625e-8f);  // a cache of zeros: S = 0 counts as its value 0
            k[2 * G] = in ? lg2(top) : -INFINITY;
            k[2 * G + 1] = __fdividef(1.0f, top);
            if (G > 1) {
#pragma unroll
              for (int i = 0; i < G; ++i) k[G > 1 ? 2 * G + 2 + i : 0] *= k[2 * G + 1];
            }
#pragma unroll
            for (int q = 0; q < C::kRec; q += 4)
              sts128(ct + (lane * C::kRec + q) * 4,
                     make_uint4(__float_as_uint(k[q]), __float_as_uint(k[q + 1]),
                                __float_as_uint(k[q + 2]), __float_as_uint(k[q + 3])));
          }
          // -- scores: two blocks of 16 tokens x 8 NT rows
          float d[2][NT][G][4];
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < G; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[w][n][i][e] = 0.0f;
          uint32_t kw[2][2][4];
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t at = st + off_k[w] + (tk0 + 8 * e) * (D / 2) + c * (D / 8);
              if (KW == 4) {
                const uint4 x = lds128(at);
                kw[w][e][0] = x.x, kw[w][e][1] = x.y, kw[w][e][2] = x.z, kw[w][e][3] = x.w;
              } else {
                const uint2 x = lds64(at);
                kw[w][e][0] = x.x, kw[w][e][1] = x.y;
              }
            }
#pragma unroll
          for (int j = 0; j < KW; ++j) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t u0[4], u1[4];
              unpack_hi<kBf16>(kw[w][0][j], u0);
              unpack_hi<kBf16>(kw[w][1][j], u1);
              const uint32_t fa[4] = {u0[0], u1[0], u0[1], u1[1]};
              const uint32_t fb[4] = {u0[2], u1[2], u0[3], u1[3]};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16<kBf16>(d[w][n][j * G / KW], fa, qf[n][j][0], qf[n][j][1]);
                mma16<kBf16>(d[w][n][j * G / KW], fb, qf[n][j][2], qf[n][j][3]);
              }
            }
          }
          __syncwarp();  // the constants are written
          // s = k1 D - k2 X + lv, in place of the block's D of group 0
          float isv[2][2], ratio[2][2][G];
          bool over = false;
          const bool safe = pos0 + 32 <= safe_end && pos0 >= safe_begin;
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float k[C::kRec];
              const int tok = 16 * w + tk0 + 8 * e;
#pragma unroll
              for (int q = 0; q < C::kRec; q += 4) {
                const uint4 x = lds128(ct + (tok * C::kRec + q) * 4);
                k[q] = __uint_as_float(x.x);
                k[q + 1] = __uint_as_float(x.y);
                k[q + 2] = __uint_as_float(x.z);
                k[q + 3] = __uint_as_float(x.w);
              }
              isv[w][e] = k[2 * G + 1];
#pragma unroll
              for (int i = 0; i < G; ++i) ratio[w][e][i] = G > 1 ? k[G > 1 ? 2 * G + 2 + i : 0] : 1.0f;
              const int pos = pos0 + tok;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  float v = k[2 * G];
#pragma unroll
                  for (int i = 0; i < G; ++i)
                    v += k[i] * d[w][n][i][2 * e + x] - k[G + i] * xs[n][i][x];
                  if (!safe && (pos > lim[n][x] || (a.window > 0 && pos <= lim[n][x] - a.window)))
                    v = -INFINITY;
                  d[w][n][0][2 * e + x] = v;
                  over |= v > m[n][x] + kHeadroom;
                }
            }
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float x = fmaxf(fmaxf(d[0][n][0][e], d[0][n][0][e + 2]),
                                fmaxf(d[1][n][0][e], d[1][n][0][e + 2]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                x = fmaxf(x, m[n][e]);
                const float f = x == -INFINITY ? 1.0f : ex2(m[n][e] - x);
                m[n][e] = x;
                l[n][e] *= f;
#pragma unroll
                for (int i = 0; i < VT; ++i) {
                  o[n][i][e] *= f;
                  o[n][i][e + 2] *= f;
                }
              }
            }
          }
          // -- probabilities: binary16 pairs, transposed into the B operand of the V product
          uint32_t pb[2][NT][G][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float r0 = kLift - (m[n][0] == -INFINITY ? 0.0f : m[n][0]);
            const float r1 = kLift - (m[n][1] == -INFINITY ? 0.0f : m[n][1]);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p0 = ex2(d[w][n][0][2 * e] + r0), p1 = ex2(d[w][n][0][2 * e + 1] + r1);
                l[n][0] += p0 * isv[w][e];
                l[n][1] += p1 * isv[w][e];
#pragma unroll
                for (int i = 0; i < G; ++i)
                  pb[w][n][i][e] = movmatrix_trans(
                      half2_bits(p0 * ratio[w][e][i], p1 * ratio[w][e][i]));
              }
          }
          // -- O^T += V^T P^T: A rows are dims 16 i + 2 g (and + 1), k slots the tokens
          uint32_t wv[2][4][2];  // the values' codes, of the tokens of the lane's k slots
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tv = ((e & 1) ? tv1 : tv0) + 8 * (e >> 1);
              const uint32_t at = st + off_v[w] + tv * (D / 2) +
                                  ((g * (D / 16)) ^ ((e & 1) ? flip1 : flip0));
              if (VT == 8) {
                const uint2 x = lds64(at);
                wv[w][e][0] = x.x;
                wv[w][e][1] = x.y;
              } else {
                wv[w][e][0] = lds32(at);
              }
            }
          uint32_t zlo[2][G][2], zhi[2][G][2];  // 1024 + Z and -(64 + Z) of the slot pairs
          const uint32_t zt = ct + 32 * 4 * C::kRec;
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int tok = 16 * w + 8 * q;
                const uint32_t za = lds32(zt + ((tok + tv0) * G + i) * 4);
                const uint32_t zb = lds32(zt + ((tok + tv1) * G + i) * 4);
                zlo[w][i][q] = __byte_perm(za, zb, 0x5410);
                zhi[w][i][q] = __byte_perm(za, zb, 0x7632);
              }
#pragma unroll
          for (int i = 0; i < VT; ++i) {
            const int gi = i * G / VT;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t fa[4];
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                // byte i of the first token in the low half, of the second in the high half
                const uint32_t y = __byte_perm(wv[w][2 * q][i >> 2], wv[w][2 * q + 1][i >> 2],
                                               static_cast<uint32_t>(i & 3) |
                                                   (static_cast<uint32_t>(4 + (i & 3)) << 8));
                fa[2 * q] = hsub2(and_or(y, 0x000F000Fu, 0x64006400u), zlo[w][gi][q]);
                fa[2 * q + 1] =
                    hfma2(and_or(y, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zhi[w][gi][q]);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16_16816(o[n][i], fa, pb[w][n][gi][0], pb[w][n][gi][1]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->empty[s]);
        if (++s == kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      // a timeout in any warp ends the work of all four (the barriers below need them all, so
      // they have to decide alike)
      if (named_barrier_or(1, 32 * kWarps, !ok)) {
        ok = false;
        break;
      }

      // ---------------------------------------------------- join the four warps' states
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
          if (g == 0) {
            ctl->ml[warp][0][8 * n + 2 * c + e] = m[n][e];
            ctl->ml[warp][1][8 * n + 2 * c + e] = l[n][e];
          }
        }
      }
      named_barrier(1, 32 * kWarps);
      float mt[NT][2], lt[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * c + e;
          float x = -INFINITY;
#pragma unroll
          for (int q = 0; q < kWarps; ++q) x = fmaxf(x, ctl->ml[q][0][row]);
          float sum = 0.0f;
#pragma unroll
          for (int q = 0; q < kWarps; ++q) {
            const float mq = ctl->ml[q][0][row], lq = ctl->ml[q][1][row];
            sum += mq == -INFINITY ? lq : lq * ex2(mq - x);  // lq is 0 there, or NaN
          }
          mt[n][e] = x;
          lt[n][e] = sum;
          const float f = m[n][e] == -INFINITY ? 1.0f : ex2(m[n][e] - x);
#pragma unroll
          for (int i = 0; i < VT; ++i) {
            o[n][i][e] *= f;
            o[n][i][e + 2] *= f;
          }
        }
      }
      // warps 2, 3 hand their sums to 0, 1, then 1 to 0: a fixed order
      auto put = [&](float* to) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < VT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[(8 * n + 2 * c + (e & 1)) * (D + 1) + 16 * i + 2 * g + (e >> 1)] = o[n][i][e];
      };
      auto add = [&](const float* from) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < VT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[n][i][e] += from[(8 * n + 2 * c + (e & 1)) * (D + 1) + 16 * i + 2 * g + (e >> 1)];
      };
      if (warp >= 2) put(merge + (warp - 2) * kRows * (D + 1));
      named_barrier(1, 32 * kWarps);
      if (warp < 2) add(merge + warp * kRows * (D + 1));
      named_barrier(1, 32 * kWarps);
      if (warp == 1) put(merge);
      named_barrier(1, 32 * kWarps);
      if (warp == 0) {
        add(merge);
        const bool whole = u_begin == 0 && u_end == r.nt;
        if (whole) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = row0 + 8 * n + 2 * c + e;
              if (row >= rows) continue;
              const int tok = row / a.ratio, head = h * a.ratio + row - tok * a.ratio;
              // no key seen: l = 0 (a NaN stays one)
              const float inv = lt[n][e] == 0.0f ? 0.0f : 1.0f / lt[n][e];
              uint16_t* dst = a.out + static_cast<int64_t>(r.q0 + tok) * a.o_tok +
                              static_cast<int64_t>(head) * a.o_head;
#pragma unroll
              for (int i = 0; i < VT; ++i) {
                const uint32_t lo = narrow<kBf16>(o[n][i][e] * inv);
                const uint32_t hi = narrow<kBf16>(o[n][i][e + 2] * inv);
                *reinterpret_cast<uint32_t*>(dst + 16 * i + 2 * g) = lo | hi << 16;
              }
              if (a.lse && g == 0)
                a.lse[static_cast<int64_t>(r.q0 + tok) * a.heads + head] =
                    lt[n][e] == 0.0f ? -INFINITY
                                     : (mt[n][e] - kLift + log2f(lt[n][e])) * 0.6931471805599453f;
            }
          }
        } else {
          const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u_begin == 0 ? 1 : 0);
          float* dst = parts + slot * part_floats(D);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = 8 * n + 2 * c + e;
#pragma unroll
              for (int i = 0; i < VT; ++i)
                *reinterpret_cast<float2*>(dst + row * D + 16 * i + 2 * g) =
                    make_float2(o[n][i][e], o[n][i][e + 2]);
              if (g == 0) {
                dst[kMaxRows * D + row] = mt[n][e];
                dst[kMaxRows * (D + 1) + row] = lt[n][e];
              }
            }
          }
          if (u_begin == 0 && lane == 0) {  // the unit's first part: tell who holds the others
            Desc d;
            d.first_row = row0;
            d.q0 = r.q0;
            d.rows = rows;
            d.head = h;
            // the CTA whose share holds the unit's last tile
            d.last_cta =
                static_cast<int>(((line + kUnitCost + r.nt) * live + total - 1) / total) - 1;
            descs[blockIdx.x] = d;
          }
        }
      }
      named_barrier(1, 32 * kWarps);
      left -= u_end - u_begin;
      if (left == 0 || !next_unit()) break;
    }
  }
}

// A unit that several CTAs share: out = sum_i O_i 2^(m_i - m) / l over its parts i, one CTA for
// four of its rows. kSplit warps of a row take every kSplit-th part, in a fixed order, so that a row of
// a few hundred parts (one long request) is a few rounds of loads; 16 bytes (8 for 64
// dimensions) a lane and part.
constexpr int kJoinRows = 4;
template <int D, bool kBf16>
__global__ void __launch_bounds__(512)
kv4_combine_kernel(const Kv4AttnArgs a, int ctas) {
  constexpr int V = D / 32;  // dimensions of a lane
  constexpr int kRows = kJoinRows, kSplit = 16 / kRows;
  __shared__ float acc[kRows][kSplit][D];
  __shared__ float sum[kRows][kSplit];
  pdl_wait();
  const Desc* descs = static_cast<const Desc*>(a.workspace);
  const Desc d = descs[blockIdx.x];
  if (d.first_row < 0 || d.first_row + kRows * static_cast<int>(blockIdx.y) >= d.rows) return;
  const float* parts = reinterpret_cast<const float*>(descs + ctas);
  const int n = d.last_cta - static_cast<int>(blockIdx.x) + 1;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) / kRows;
  const int local = (threadIdx.x >> 5) % kRows, row = kRows * blockIdx.y + local;
  auto part = [&](int i) {  // the first CTA's last unit, the others' first
    return parts + (2 * static_cast<int64_t>(blockIdx.x + i) + (i == 0 ? 1 : 0)) * part_floats(D);
  };
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, part(i)[kMaxRows * D + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f, o[V];
#pragma unroll
  for (int k = 0; k < V; ++k) o[k] = 0.0f;
#pragma unroll 8
  for (int i = warp; i < n; i += kSplit) {
    const float* p = part(i);
    const float x = p[kMaxRows * D + row];
    const float f = x == -INFINITY ? 1.0f : ex2(x - m);  // O and l are 0 there, or NaN
    l += f * p[kMaxRows * (D + 1) + row];
    float v[V];
    if (V == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + row * D + 4 * lane);
      v[0] = q.x, v[1] = q.y, v[V - 2] = q.z, v[V - 1] = q.w;
    } else {
      const float2 q = *reinterpret_cast<const float2*>(p + row * D + 2 * lane);
      v[0] = q.x, v[1] = q.y;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] += f * v[k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) acc[local][warp][V * lane + k] = o[k];
  if (lane == 0) sum[local][warp] = l;
  __syncthreads();
  const int rr = d.first_row + row;
  if (warp > 0 || rr >= d.rows) return;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kSplit; ++w) l += sum[local][w];
  const int tok = rr / a.ratio, head = d.head * a.ratio + rr - tok * a.ratio;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + static_cast<int64_t>(d.q0 + tok) * a.o_tok +
                                              static_cast<int64_t>(head) * a.o_head);
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int w = 0; w < kSplit; ++w) {
      x += acc[local][w][V * lane + k];
      y += acc[local][w][V * lane + k + 1];
    }
    dst[(V * lane + k) >> 1] = narrow<kBf16>(x * inv) | static_cast<uint32_t>(narrow<kBf16>(y * inv)) << 16;
  }
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(d.q0 + tok) * a.heads + head] =
        l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
}

constexpr int kMaxCtasPerSm = 4;

template <int D, int G, int NT, bool kBf16>
cudaError_t launch_t(const Kv4AttnArgs& a, int sms, cudaStream_t st) {
  using C = Cfg<D, G, NT>;
  static_assert(C::kCtasPerSm <= kMaxCtasPerSm && C::kRows <= kMaxRows, "workspace");
  constexpr int smem = smem_bytes<D, G, NT>();
  static_assert(C::kCtasPerSm * (smem + 1024) <= 228 * 1024, "shared memory of an SM");
  auto kern = kv4_decode_kernel<D, G, NT, kBf16>;
  static std::atomic<bool> attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!attr[dev & 63].load(std::memory_order_acquire)) {
    e = set_smem_attrs(kern, smem);
    if (e != cudaSuccess) return e;
    attr[dev & 63].store(true, std::memory_order_release);
  }
  const int grid = sms * C::kCtasPerSm;
  kern<<<grid, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, C::kRows / kJoinRows, 1);
  cfg.blockDim = dim3(512, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, kBf16>, a, grid);
}

template <int D, int G>
cudaError_t launch_g(const Kv4AttnArgs& a, bool wide, int sms, cudaStream_t st) {
  if (a.bf16)
    return wide ? launch_t<D, G, 2, true>(a, sms, st) : launch_t<D, G, 1, true>(a, sms, st);
  return wide ? launch_t<D, G, 2, false>(a, sms, st) : launch_t<D, G, 1, false>(a, sms, st);
}

}  // namespace

size_t kv4_decode_workspace_bytes(int sms) {
  const size_t ctas = static_cast<size_t>(sms) * kMaxCtasPerSm;
  return ctas * sizeof(Desc) + 2 * ctas * part_floats(128) * sizeof(float);
}

// Row tiles of 8, or of 16 where a request may have more rows than 8: one pass over the keys
// for all of them then.
cudaError_t launch_kv4_decode(const Kv4AttnArgs& a, int max_q, int sms, cudaStream_t st) {
  const bool wide = static_cast<int64_t>(max_q) * a.ratio > 8;
  const int groups = a.cache.groups();
  if (a.cache.dim == 128) {
    if (groups == 1) return launch_g<128, 1>(a, wide, sms, st);
    if (groups == 2) return launch_g<128, 2>(a, wide, sms, st);
    return launch_g<128, 4>(a, wide, sms, st);
  }
  return groups == 1 ? launch_g<64, 1>(a, wide, sms, st) : launch_g<64, 2>(a, wide, sms, st);
}

}  // namespace wq
