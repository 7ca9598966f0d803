// C ABI of the 4-bit KV cache operators (declared in include/wq.h): argument validation and
// launches.
#include <cmath>

#include "../../include/wq.h"
#include "kernels.h"
#include "kv4.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffffLL;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool count_ok(int64_t v) { return v >= 0 && v <= kIntMax; }
wq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA; }

int block_log2(int32_t block) {
  for (int i = 4; i <= 8; ++i)
    if (block == 1 << i) return i;
  return -1;
}

// The cache's description without its memory.
wq_status check_shape(const wq_kv4_cache* c) {
  if (!c) return WQ_ERR_NULL;
  if (c->num_blocks < 0 || c->kv_heads <= 0 || c->kv_heads > 65535) return WQ_ERR_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return WQ_ERR_UNSUPPORTED;
  if (c->group != 32 && c->group != 64 && c->group != 128) return WQ_ERR_UNSUPPORTED;
  if (c->group > c->head_dim) return WQ_ERR_SHAPE;
  const int l = block_log2(c->block_size);
  if (l < 0) return WQ_ERR_UNSUPPORTED;
  if (c->num_blocks > (kIntMax >> l)) return WQ_ERR_SHAPE;  // slots are 32-bit integers
  return WQ_OK;
}

wq_status check_cache(const wq_kv4_cache* c, wq::Kv4Cache* k) {
  const wq_status s = check_shape(c);
  if (s != WQ_OK) return s;
  if (c->num_blocks > 0 && !c->data) return WQ_ERR_NULL;
  if (!aligned(c->data, 16)) return WQ_ERR_ALIGN;
  *k = {static_cast<uint8_t*>(c->data), c->num_blocks, c->kv_heads, c->head_dim, c->group,
        c->block_size, block_log2(c->block_size)};
  return WQ_OK;
}

// The prompt and the decode kernels of a call use it one after the other.
size_t workspace_bytes(int sms) {
  const size_t d = wq::kv4_decode_workspace_bytes(sms), p = wq::kv4_prompt_workspace_bytes(sms);
  return d > p ? d : p;
}

}  // namespace

extern "C" {

size_t wq_kv4_cache_bytes(const wq_kv4_cache* c) {
  if (check_shape(c) != WQ_OK) return 0;
  return static_cast<size_t>(c->num_blocks) * c->kv_heads * c->block_size *
         (c->head_dim + 8 * (c->head_dim / c->group));
}

wq_status wq_kv4_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t B,
                              const int32_t* free_blocks, int64_t n_free, int32_t block_size,
                              int32_t* tables, int64_t width, int64_t ld_tables, int32_t* slots,
                              int64_t n_slots, int32_t* q_starts, int32_t* kv_lens,
                              int32_t* taken, void* stream) {
  if (B < 0 || n_free < 0 || width < 0 || n_slots < 0) return WQ_ERR_SHAPE;
  const int l = block_log2(block_size);
  if (l < 0) return WQ_ERR_UNSUPPORTED;
  if (!count_ok(B) || !count_ok(n_free) || !count_ok(width) || !count_ok(n_slots) ||
      ld_tables < width)
    return WQ_ERR_SHAPE;
  if (!q_starts || !taken || (B > 0 && (!ctx_lens || !new_lens || !kv_lens)) ||
      (n_free > 0 && !free_blocks) || (B > 0 && width > 0 && !tables) || (n_slots > 0 && !slots))
    return WQ_ERR_NULL;
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) ||
      !aligned(tables, 4) || !aligned(slots, 4) || !aligned(q_starts, 4) ||
      !aligned(kv_lens, 4) || !aligned(taken, 4))
    return WQ_ERR_ALIGN;
  int sms = 0;
  unsigned* status = nullptr;
  if (!wq::current_device(&sms, &status)) return WQ_ERR_NODEVICE;
  if (!wq::pointers_on_current_device(
          {ctx_lens, new_lens, free_blocks, tables, slots, q_starts, kv_lens, taken}))
    return WQ_ERR_DEVICE;
  const wq::Kv4TablesArgs a{ctx_lens, new_lens, static_cast<int>(B), free_blocks,
                            static_cast<int>(n_free), l, tables, static_cast<int>(width),
                            ld_tables, slots, static_cast<int>(n_slots), q_starts, kv_lens,
                            taken, status};
  return from_cuda(wq::launch_kv4_block_tables(a, sms, static_cast<cudaStream_t>(stream)));
}

wq_status wq_kv4_append(const uint16_t* K, const uint16_t* V, wq_dtype dtype, int64_t T,
                        int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                        int64_t v_head_stride, const int32_t* slots, const wq_kv4_cache* cache,
                        void* stream) {
  if (T < 0) return WQ_ERR_SHAPE;
  if (dtype != WQ_BF16 && dtype != WQ_F16) return WQ_ERR_DTYPE;
  wq::Kv4Cache c;
  const wq_status s = check_cache(cache, &c);
  if (s != WQ_OK) return s;
  if (T == 0) return WQ_OK;
  if (!K || !V || !slots) return WQ_ERR_NULL;
  if (!count_ok(T)) return WQ_ERR_SHAPE;
  if (k_token_stride < 0 || k_head_stride < 0 || v_token_stride < 0 || v_head_stride < 0)
    return WQ_ERR_SHAPE;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 4) || k_token_stride % 8 != 0 ||
      k_head_stride % 8 != 0 || v_token_stride % 8 != 0 || v_head_stride % 8 != 0)
    return WQ_ERR_ALIGN;
  int sms = 0;
  unsigned* status = nullptr;
  if (!wq::current_device(&sms, &status)) return WQ_ERR_NODEVICE;
  if (!wq::pointers_on_current_device({K, V, slots, c.data})) return WQ_ERR_DEVICE;
  const wq::Kv4AppendArgs a{K, V, dtype == WQ_BF16, T, k_token_stride, k_head_stride,
                            v_token_stride, v_head_stride, slots, c, status};
  return from_cuda(wq::launch_kv4_append(a, sms, static_cast<cudaStream_t>(stream)));
}

wq_status wq_kv4_read(const wq_kv4_cache* cache, const int32_t* slots, int64_t T, void* K,
                      void* V, wq_dtype out_dtype, void* stream) {
  if (T < 0) return WQ_ERR_SHAPE;
  if (out_dtype != WQ_F32 && out_dtype != WQ_BF16 && out_dtype != WQ_F16) return WQ_ERR_DTYPE;
  wq::Kv4Cache c;
  const wq_status s = check_cache(cache, &c);
  if (s != WQ_OK) return s;
  if (T == 0) return WQ_OK;
  if (!slots || !K || !V) return WQ_ERR_NULL;
  if (!count_ok(T)) return WQ_ERR_SHAPE;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 4)) return WQ_ERR_ALIGN;
  int sms = 0;
  unsigned* status = nullptr;
  if (!wq::current_device(&sms, &status)) return WQ_ERR_NODEVICE;
  if (!wq::pointers_on_current_device({slots, K, V, c.data})) return WQ_ERR_DEVICE;
  const wq::Kv4ReadArgs a{c, slots, T, K, V, static_cast<int>(out_dtype), status};
  return from_cuda(wq::launch_kv4_read(a, sms, static_cast<cudaStream_t>(stream)));
}

size_t wq_kv4_attention_workspace_bytes(void) {
  int sms = 0;
  unsigned* status = nullptr;
  if (!wq::current_device(&sms, &status)) sms = 148;
  return workspace_bytes(sms);
}

wq_status wq_kv4_attention(const wq_kv4_attention_args* p, void* stream) {
  if (!p) return WQ_ERR_NULL;
  if (p->T < 0 || p->B < 0 || p->heads <= 0 || p->max_q < 0 || p->window < 0 ||
      p->window > (1 << 30) || p->width < 0)
    return WQ_ERR_SHAPE;
  if (p->dtype != WQ_BF16 && p->dtype != WQ_F16) return WQ_ERR_DTYPE;
  wq::Kv4Cache c;
  const wq_status s = check_cache(&p->cache, &c);
  if (s != WQ_OK) return s;
  if (p->heads % c.kv_heads != 0 || !std::isfinite(p->scale)) return WQ_ERR_SHAPE;
  if (p->T == 0 || p->B == 0) return WQ_OK;
  if (!p->Q || !p->q_starts || !p->kv_lens || !p->out || !p->workspace ||
      (p->width > 0 && !p->tables))
    return WQ_ERR_NULL;
  if (p->q_token_stride < 0 || p->q_head_stride < 0 || p->o_token_stride < 0 ||
      p->o_head_stride < 0 || p->ld_tables < p->width)
    return WQ_ERR_SHAPE;
  // rows of a request are counted in 32 bits
  if (p->B > 65536 || p->T > kIntMax / p->heads || !count_ok(p->width)) return WQ_ERR_SHAPE;
  const int32_t ratio = p->heads / c.kv_heads;
  const bool prompts = static_cast<int64_t>(p->max_q) * ratio > wq::kKv4DecodeRows;
  if (prompts && wq::kv4_prompt_units(p->T, ratio, p->B, c.kv_heads) > kIntMax) return WQ_ERR_SHAPE;
  if (p->Q == p->out) return WQ_ERR_UNSUPPORTED;  // CTAs that share a row read it at their own times
  if (!aligned(p->Q, 16) || !aligned(p->out, 16) || !aligned(p->lse, 4) ||
      !aligned(p->q_starts, 4) || !aligned(p->kv_lens, 4) || !aligned(p->tables, 4) ||
      !aligned(p->workspace, 16) || p->q_token_stride % 8 != 0 || p->q_head_stride % 8 != 0 ||
      p->o_token_stride % 8 != 0 || p->o_head_stride % 8 != 0)
    return WQ_ERR_ALIGN;
  int sms = 0;
  unsigned* status = nullptr;
  if (!wq::current_device(&sms, &status)) return WQ_ERR_NODEVICE;
  if (p->workspace_bytes < workspace_bytes(sms)) return WQ_ERR_SHAPE;
  if (!wq::pointers_on_current_device({p->Q, p->q_starts, p->kv_lens, p->tables, p->out, p->lse,
                                       p->workspace, c.data}))
    return WQ_ERR_DEVICE;
  wq::Kv4AttnArgs a;
  a.Q = p->Q;
  a.bf16 = p->dtype == WQ_BF16;
  a.tokens = static_cast<int>(p->T);
  a.heads = p->heads;
  a.ratio = ratio;
  a.q_tok = p->q_token_stride;
  a.q_head = p->q_head_stride;
  a.o_tok = p->o_token_stride;
  a.o_head = p->o_head_stride;
  a.cache = c;
  a.tables = p->tables;
  a.width = static_cast<int>(p->width);
  a.ld_tables = p->ld_tables;
  a.q_starts = p->q_starts;
  a.kv_lens = p->kv_lens;
  a.requests = static_cast<int>(p->B);
  a.scale_log2 = static_cast<float>(static_cast<double>(p->scale) * 1.4426950408889634);
  a.causal = p->causal != 0;
  a.window = p->window;
  a.out = p->out;
  a.lse = p->lse;
  a.workspace = p->workspace;
  a.status = status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Where some request may have more rows than the decode kernel takes in one pass, the prompt
  // kernel gets those requests and the decode kernel the others; which are which is read on
  // the device. A single request needs no such split.
  a.most_rows = static_cast<int>(kIntMax);
  if (prompts) {
    a.most_rows = a.requests == 1 ? 0 : wq::kKv4DecodeRows;
    const wq_status e = from_cuda(wq::launch_kv4_prompt(a, sms, st));
    if (e != WQ_OK || a.requests == 1) return e;
  }
  return from_cuda(wq::launch_kv4_decode(a, p->max_q, sms, st));
}

}  // extern "C"
