// fa_cache_api.cu -- the C entry points of the serving operators
// (include/fa_cache.h): argument validation and parameter blocks.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_params.h"
#include "fa_device.h"

namespace fa {
namespace {

constexpr long long kIntMax = 0x7fffffffLL;

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
long long align256(long long bytes) { return (bytes + 255) / 256 * 256; }

int invalid(const char* what) {
  set_error("%s", what);
  return FA_ERR_INVALID_ARGUMENT;
}

// Byte strides that 16-byte accesses and tensor maps take; a dimension of
// extent 1 is never stepped.
bool stride_ok(long long bytes, long long extent, long long least) {
  return extent <= 1 || (bytes >= least && bytes % 16 == 0 && bytes < (1LL << 40));
}

int check_cache(const fa_cache& c) {
  if (!c.k || !c.v || !c.k_scale || !c.v_scale) return invalid("the cache's k, v, k_scale and v_scale must be non-NULL");
  if (c.P <= 0 || c.H_kv <= 0) return invalid("the cache's P and H_kv must be > 0");
  if (c.kind != FA_CACHE_E4M3 && c.kind != FA_CACHE_INT8) {
    set_error("cache kind %d is not FA_CACHE_E4M3 (0) or FA_CACHE_INT8 (1)", c.kind);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) {
    set_error("page = %d tokens is not supported (16, 32, 64 or 128)", c.page);
    return FA_ERR_UNSUPPORTED;
  }
  if (c.D != 64 && c.D != 128 && c.D != 256) {
    set_error("head dim D = %d is not supported (64, 128 or 256)", c.D);
    return FA_ERR_UNSUPPORTED;
  }
  if (c.H_kv > 32767) {
    set_error("H_kv (%d) must be at most 32767", c.H_kv);
    return FA_ERR_UNSUPPORTED;
  }
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)) {
    set_error("the cache's k and v must be 16-byte aligned, its scales 4-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  const struct {
    const long long* s;
    const char* name;
  } views[2] = {{c.k_strides, "k"}, {c.v_strides, "v"}};
  for (const auto& w : views)
    if (!stride_ok(w.s[0], c.P, c.D) || !stride_ok(w.s[1], c.H_kv, c.D) || !stride_ok(w.s[2], c.page, c.D)) {
      set_error("the cache's %s strides {%lld, %lld, %lld} must be multiples of 16 bytes, at least D", w.name, w.s[0],
                w.s[1], w.s[2]);
      return FA_ERR_MISALIGNED;
    }
  return FA_OK;
}

int check_table(const int* table, long long stride, const int* lens, int B, int M, int page) {
  if (!table || !lens) return invalid("table and lens must be non-NULL");
  if (B <= 0 || M <= 0) {
    set_error("B (%d) and M (%d) must be > 0", B, M);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (stride < M && B > 1) {
    set_error("the table's row stride (%lld) is smaller than M (%d)", stride, M);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (B > 65535 || (long long)M * page > kIntMax - 65536) {
    set_error("B (%d) must be at most 65535 and M * page below 2^31 - 65537", B);
    return FA_ERR_UNSUPPORTED;
  }
  if (!aligned(table, 4) || !aligned(lens, 4)) {
    set_error("table and lens must be 4-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

CacheView view_of(const fa_cache& c, const int* table, long long stride, int M, unsigned int* status) {
  CacheView v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  for (int i = 0; i < 3; ++i) v.ks[i] = c.k_strides[i], v.vs[i] = c.v_strides[i];
  v.P = c.P;
  v.H = c.H_kv;
  v.page = c.page;
  v.page_log2 = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
  v.D = c.D;
  v.table = table;
  v.table_stride = stride;
  v.M = M;
  v.status = status;
  return v;
}

int check_rows(const long long* s, long long B, long long H, long long n, int D, int esz, const char* name) {
  if (!stride_ok(s[0] * esz, B, 16) || !stride_ok(s[1] * esz, H, 16) || !stride_ok(s[2] * esz, n, (long long)D * esz)) {
    set_error("%s strides {%lld, %lld, %lld} (elements) must be positive multiples of 16 bytes, rows at least D apart",
              name, s[0], s[1], s[2]);
    return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

int check_workspace(const void* ws, long long bytes, long long need, const char* fn) {
  if (need > 0 && !ws) {
    set_error("workspace is NULL: this call needs %lld bytes (%s)", need, fn);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (ws && !aligned(ws, 256)) {
    set_error("workspace must be 256-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  if (bytes < need) {
    set_error("workspace of %lld bytes is smaller than the %lld this call needs (%s)", bytes, need, fn);
    return FA_ERR_INVALID_ARGUMENT;
  }
  return FA_OK;
}

int check_append(const fa_cache_append_args* a) {
  if (!a) return invalid("args is NULL");
  int rc = check_cache(a->cache);
  if (rc == FA_OK) rc = check_table(a->table, a->table_stride, a->lens, a->B, a->M, a->cache.page);
  if (rc != FA_OK) return rc;
  if (!a->k || !a->v) return invalid("k and v must be non-NULL");
  if (a->n <= 0) {
    set_error("n (%d) must be > 0", a->n);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (a->dtype != FA_DTYPE_F32 && a->dtype != FA_DTYPE_BF16 && a->dtype != FA_DTYPE_F16) {
    set_error("dtype %d is not FA_DTYPE_F32 (0), FA_DTYPE_BF16 (1) or FA_DTYPE_F16 (2)", a->dtype);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if ((a->weights || a->positions) && a->W <= 0) return invalid("W must be > 0 with weights or positions");
  if (!aligned(a->k, 16) || !aligned(a->v, 16)) {
    set_error("k and v must be 16-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  if (!aligned(a->weights, 4) || !aligned(a->positions, 4) || !aligned(a->n_new, 4) || !aligned(a->seen, 4)) {
    set_error("weights, positions, n_new and seen must be 4-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  const int esz = a->dtype == FA_DTYPE_F32 ? 4 : 2;
  rc = check_rows(a->k_strides, a->B, a->cache.H_kv, a->n, a->cache.D, esz, "k");
  return rc != FA_OK ? rc : check_rows(a->v_strides, a->B, a->cache.H_kv, a->n, a->cache.D, esz, "v");
}

int check_attn(const fa_cache_attn_args* a) {
  if (!a) return invalid("args is NULL");
  int rc = check_cache(a->cache);
  if (rc == FA_OK) rc = check_table(a->table, a->table_stride, a->lens, a->B, a->M, a->cache.page);
  if (rc != FA_OK) return rc;
  if (!a->q || !a->o || !a->lse) return invalid("q, o and lse must be non-NULL");
  if (a->n <= 0 || a->H_q <= 0) {
    set_error("n (%d) and H_q (%d) must be > 0", a->n, a->H_q);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (a->H_q % a->cache.H_kv != 0) {
    set_error("H_q (%d) must be divisible by H_kv (%d)", a->H_q, a->cache.H_kv);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (a->dtype != FA_DTYPE_BF16 && a->dtype != FA_DTYPE_F16) {
    set_error("dtype %d is not FA_DTYPE_BF16 (1) or FA_DTYPE_F16 (2)", a->dtype);
    return a->dtype == FA_DTYPE_F32 ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID_ARGUMENT;
  }
  if (!std::isfinite(a->scale)) return invalid("scale must be finite");
  if (a->window < 0) {
    set_error("window (%d) must be >= 0 (0 = no sliding window)", a->window);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (!std::isfinite(a->softcap) || a->softcap < 0.0f) return invalid("softcap must be finite and >= 0 (0 = off)");
  if (a->weights && a->W <= 0) return invalid("W must be > 0 with weights");
  if ((long long)a->n > kIntMax / ((long long)a->B * a->H_q)) {
    set_error("B * H_q * n exceeds 2^31 - 1");
    return FA_ERR_UNSUPPORTED;
  }
  if (a->H_q > 65535) {
    set_error("H_q (%d) must be at most 65535", a->H_q);
    return FA_ERR_UNSUPPORTED;
  }
  if (!aligned(a->q, 16) || !aligned(a->o, 16)) {
    set_error("q and o must be 16-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  if (!aligned(a->lse, 4) || !aligned(a->weights, 4) || !aligned(a->n_q, 4)) {
    set_error("lse, weights and n_q must be 4-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  rc = check_rows(a->q_strides, a->B, a->H_q, a->n, a->cache.D, 2, "q");
  return rc != FA_OK ? rc : check_rows(a->o_strides, a->B, a->H_q, a->n, a->cache.D, 2, "o");
}

CacheAttnParams attn_params(const fa_cache_attn_args* a, unsigned int* status, long long timeout) {
  CacheAttnParams p;
  p.c = view_of(a->cache, a->table, a->table_stride, a->M, status);
  p.q = a->q;
  p.o = a->o;
  p.lse = a->lse;
  p.weights = a->weights;
  for (int i = 0; i < 3; ++i) p.qs[i] = a->q_strides[i], p.os[i] = a->o_strides[i];
  p.lens = a->lens;
  p.n_q = a->n_q;
  p.B = a->B;
  p.Hq = a->H_q;
  p.group = a->H_q / a->cache.H_kv;
  p.n = a->n;
  p.W = a->W;
  p.causal = a->causal ? 1 : 0;
  p.window = a->window;
  p.scale_log2 = (float)((double)a->scale * 1.4426950408889634);
  p.cap_in = a->softcap > 0.0f ? a->scale / a->softcap : 0.0f;
  p.cap_out = (float)((double)a->softcap * 1.4426950408889634);
  p.timeout_cycles = timeout;
  p.ws = static_cast<uint8_t*>(a->workspace);
  return p;
}

long long attn_workspace(const CacheAttnParams& p, int num_sms) {
  return p.c.D == 64    ? cache_attn_workspace_d64(p, num_sms)
         : p.c.D == 128 ? cache_attn_workspace_d128(p, num_sms)
                        : cache_attn_workspace_d256(p, num_sms);
}

int check_evict(const fa_cache_evict_args* a) {
  if (!a) return invalid("args is NULL");
  int rc = check_cache(a->cache);
  if (rc == FA_OK) rc = check_table(a->table, a->table_stride, a->lens, a->B, a->M, a->cache.page);
  if (rc != FA_OK) return rc;
  if (!a->weights || !a->lens_out) return invalid("weights and lens_out must be non-NULL");
  if (a->W <= 0) return invalid("W must be > 0");
  if (a->keep <= 0 || a->recent < 0 || a->recent > a->keep) {
    set_error("keep (%d) must be > 0 and recent (%d) lie in [0, keep]", a->keep, a->recent);
    return FA_ERR_INVALID_ARGUMENT;
  }
  if (!a->into && !a->positions) return invalid("eviction in place needs positions: slots lose their order");
  if (a->into) {
    if (a->M_into <= 0 || (long long)a->M_into * a->cache.page < a->keep) {
      set_error("into holds %d blocks of %d tokens, fewer than keep = %d", a->M_into, a->cache.page, a->keep);
      return FA_ERR_INVALID_ARGUMENT;
    }
    if (a->into_stride < a->M_into && a->B > 1) return invalid("into's row stride is smaller than M_into");
    if ((a->weights_out || a->positions_out) && a->W_out < a->keep) return invalid("W_out must be at least keep");
  }
  // Past the table there is nothing to keep, and the workspace grows with keep.
  if ((long long)a->B * a->cache.H_kv > kIntMax / a->keep) {
    set_error("B * H_kv * keep exceeds 2^31 - 1");
    return FA_ERR_UNSUPPORTED;
  }
  if (!aligned(a->weights, 4) || !aligned(a->positions, 4) || !aligned(a->into, 4) || !aligned(a->weights_out, 4) ||
      !aligned(a->positions_out, 4) || !aligned(a->lens_out, 4)) {
    set_error("weights, positions, into, weights_out, positions_out and lens_out must be 4-byte aligned");
    return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

// Slots that eviction names per head (src, mover), and counts.
long long evict_slots(const fa_cache_evict_args* a) { return (long long)a->B * a->cache.H_kv * a->keep; }
long long evict_workspace(const fa_cache_evict_args* a) {
  const long long heads = (long long)a->B * a->cache.H_kv;
  return 2 * align256(evict_slots(a) * 4) + align256(heads * 4);
}

}  // namespace
}  // namespace fa

extern "C" {

int fa_cache_append(const fa_cache_append_args* a) {
  using namespace fa;
  clear_error();
  int rc = check_append(a);
  if (rc != FA_OK) return rc;
  DeviceInfo dev;
  rc = current_device(&dev);
  if (rc != FA_OK) return rc;
  AppendParams p;
  p.c = view_of(a->cache, a->table, a->table_stride, a->M, dev.status);
  p.k = a->k;
  p.v = a->v;
  for (int i = 0; i < 3; ++i) p.ks[i] = a->k_strides[i], p.vs[i] = a->v_strides[i];
  p.lens = a->lens;
  p.n_new = a->n_new;
  p.seen = a->seen;
  p.weights = a->weights;
  p.positions = a->positions;
  p.B = a->B;
  p.n = a->n;
  p.W = a->W;
  // n tokens that start at any slot touch at most this many blocks.
  p.spans = (int)(((long long)a->n + a->cache.page - 2) / a->cache.page + 1);
  return launch_cache_append(p, a->cache.kind, a->dtype, {static_cast<cudaStream_t>(a->stream), dev.num_sms, dev.dev, dev.max_ctas});
}

int fa_cache_attn(const fa_cache_attn_args* a) {
  using namespace fa;
  clear_error();
  int rc = check_attn(a);
  if (rc != FA_OK) return rc;
  DeviceInfo dev;
  rc = current_device(&dev);
  if (rc != FA_OK) return rc;
  const CacheAttnParams p = attn_params(a, dev.status, dev.timeout_cycles);
  rc = check_workspace(a->workspace, a->workspace_bytes, attn_workspace(p, dev.num_sms),
                       "fa_cache_attn_workspace_bytes");
  if (rc != FA_OK) return rc;
  const LaunchCtx ctx = {static_cast<cudaStream_t>(a->stream), dev.num_sms, dev.dev, dev.max_ctas};
  const bool f16 = a->dtype == FA_DTYPE_F16;
  return p.c.D == 64    ? launch_cache_attn_d64(p, a->cache.kind, f16, ctx)
         : p.c.D == 128 ? launch_cache_attn_d128(p, a->cache.kind, f16, ctx)
                        : launch_cache_attn_d256(p, a->cache.kind, f16, ctx);
}

long long fa_cache_attn_workspace_bytes(const fa_cache_attn_args* a) {
  using namespace fa;
  clear_error();
  if (check_attn(a) != FA_OK) return -1;
  DeviceInfo dev;
  if (current_device(&dev) != FA_OK) return -1;
  return attn_workspace(attn_params(a, dev.status, dev.timeout_cycles), dev.num_sms);
}

int fa_cache_evict(const fa_cache_evict_args* a) {
  using namespace fa;
  clear_error();
  int rc = check_evict(a);
  if (rc == FA_OK)
    rc = check_workspace(a->workspace, a->workspace_bytes, evict_workspace(a), "fa_cache_evict_workspace_bytes");
  if (rc != FA_OK) return rc;
  DeviceInfo dev;
  rc = current_device(&dev);
  if (rc != FA_OK) return rc;
  EvictParams p;
  p.c = view_of(a->cache, a->table, a->table_stride, a->M, dev.status);
  p.lens = a->lens;
  p.weights = a->weights;
  p.positions = a->positions;
  p.into = a->into;
  p.into_stride = a->into_stride;
  p.weights_out = a->weights_out;
  p.positions_out = a->positions_out;
  p.lens_out = a->lens_out;
  p.B = a->B;
  p.W = a->W;
  p.M_into = a->M_into;
  p.W_out = a->W_out;
  p.keep = a->keep;
  p.recent = a->recent;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  const long long slots = align256(evict_slots(a) * 4);
  p.src = reinterpret_cast<int*>(ws);
  p.mover = reinterpret_cast<int*>(ws + slots);
  p.count = reinterpret_cast<int*>(ws + 2 * slots);
  return launch_cache_evict(p, a->cache.kind, {static_cast<cudaStream_t>(a->stream), dev.num_sms, dev.dev, dev.max_ctas});
}

long long fa_cache_evict_workspace_bytes(const fa_cache_evict_args* a) {
  using namespace fa;
  clear_error();
  return check_evict(a) == FA_OK ? evict_workspace(a) : -1;
}

}  // extern "C"
