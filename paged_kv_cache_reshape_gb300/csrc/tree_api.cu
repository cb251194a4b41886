// Host side of the tree operators: validation, the handle and the launches.
// As in api.cu nothing here reads a device length.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <memory>
#include <new>
#include <string>

#include "../../include/pa.h"
#include "step.h"
#include "tree.h"

struct pa_tree_handle_s {
  pa_config cfg;
  int device = 0, num_sms = 0;
  int max_draft = 0, words = 0, max_kv = 0;
  float scale = 0.f;
  bool bf16 = false;
  int tile_tokens = 1, part_rows = 0, n_ranges = 1, rep = 1;
  void* ws = nullptr;
  int* err = nullptr;
  pa::TreeCounters* counters = nullptr;
  pa::Cut* cuts = nullptr;
  int* groups = nullptr;
  float2* part_ml = nullptr;
  float4* part_o = nullptr;
  std::string msg = "no error";
};

namespace {

constexpr double kPi = 3.14159265358979323846;

pa_status tree_fail(pa_tree_handle h, pa_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  if (h) h->msg = buf;
  return pa::host_fail(st, "%s", buf);
}

pa_status tree_cuda_fail(pa_tree_handle h, cudaError_t e, const char* what) {
  return tree_fail(h, PA_CUDA_ERROR, "%s: %s", what, cudaGetErrorString(e));
}

struct OnDevice {  // the handle's device for the duration of a call
  int prev = -1;
  explicit OnDevice(int dev) {
    if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) cudaSetDevice(dev);
    else prev = -1;
  }
  ~OnDevice() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A tensor of T rows: `width` bytes every `stride` bytes.
struct Rows {
  const void* p;
  long long T, stride, width;
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + (T > 0 ? (uintptr_t)((T - 1) * stride + width) : 0); }
};

// Whether two row tensors may share a byte (slices of one row layout with
// disjoint columns do not).
bool overlap(const Rows& a, const Rows& b) {
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  if (a.stride != b.stride) return true;
  const Rows& x = a.lo() <= b.lo() ? a : b;
  const Rows& y = a.lo() <= b.lo() ? b : a;
  const long long d = (long long)((y.lo() - x.lo()) % (uintptr_t)a.stride);
  return !(x.width <= d && d + y.width <= a.stride);
}

// What a call writes must be apart from what it reads besides its rows.
struct Named {
  Rows rows;
  const char* name;
};
Named plain(const void* p, long long bytes, const char* name) { return {{p, 1, bytes, bytes}, name}; }

template <int W, int R>
pa_status check_apart(pa_tree_handle h, const Named (&writes)[W], const Named (&reads)[R]) {
  for (const Named& w : writes)
    for (const Named& r : reads)
      if (w.rows.p && r.rows.p && overlap(w.rows, r.rows))
        return tree_fail(h, PA_INVALID_ARGUMENT, "%s must not overlap %s", w.name, r.name);
  return PA_OK;
}

bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride && a.width == b.width; }

pa_status check_rotary(pa_tree_handle h, const pa_rotary_config* rc) {
  if (!rc) return tree_fail(h, PA_INVALID_ARGUMENT, "rotary config: NULL");
  if (rc->head_size <= 0 || rc->head_size % 8 || rc->head_size > 512)
    return tree_fail(h, PA_INVALID_ARGUMENT, "head_size must be a multiple of 8 in [8, 512] (got %d)", rc->head_size);
  const int R = rc->rotary_dim ? rc->rotary_dim : rc->head_size;
  if (R <= 0 || R % 16 || R > rc->head_size)
    return tree_fail(h, PA_INVALID_ARGUMENT, "rotary_dim must be a multiple of 16 in [16, head_size] (got %d)", R);
  if (rc->rotary_offset < 0 || rc->rotary_offset % 8 || rc->rotary_offset + R > rc->head_size)
    return tree_fail(h, PA_INVALID_ARGUMENT,
                     "rotary_offset must be a multiple of 8 with rotary_offset + rotary_dim <= head_size (got %d)",
                     rc->rotary_offset);
  if ((rc->interleaved | 1) != 1)
    return tree_fail(h, PA_INVALID_ARGUMENT, "interleaved must be 0 or 1 (got %d)", rc->interleaved);
  if ((rc->conjugate | 1) != 1)
    return tree_fail(h, PA_INVALID_ARGUMENT, "conjugate must be 0 or 1 (got %d)", rc->conjugate);
  if (rc->dtype < PA_ROTARY_FP16 || rc->dtype > PA_ROTARY_FP32)
    return tree_fail(h, PA_INVALID_ARGUMENT, "dtype must be PA_ROTARY_FP16, BF16 or FP32 (got %d)", rc->dtype);
  if (!std::isfinite(rc->attention_factor))
    return tree_fail(h, PA_INVALID_ARGUMENT, "attention_factor must be finite (got %g)", rc->attention_factor);
  return PA_OK;
}

// One tensor of a rotation; *stride is set to the dense one when 0, or when
// there is one row only.
pa_status check_rows(pa_tree_handle h, const char* name, const void* p, int T, int heads, int D, int64_t* stride) {
  if (*stride == 0 || T == 1) *stride = (int64_t)heads * D;
  if (!p) return tree_fail(h, PA_INVALID_ARGUMENT, "%s must not be NULL", name);
  if (!aligned(p, 16)) return tree_fail(h, PA_INVALID_ARGUMENT, "%s must be 16-byte aligned", name);
  if (*stride < (int64_t)heads * D || *stride % 8 || *stride > (INT64_C(1) << 40))
    return tree_fail(h, PA_INVALID_ARGUMENT, "%s's row stride must be a multiple of 8, at least heads * head_size (got %lld)",
                     name, (long long)*stride);
  return PA_OK;
}

void fill_rotary(pa::RotaryParams* p, const pa_rotary_config* rc, const uint64_t* steps, const int32_t* positions,
                 int T) {
  p->steps = reinterpret_cast<const unsigned long long*>(steps);
  p->positions = positions;
  p->T = T;
  p->D = rc->head_size;
  p->R = rc->rotary_dim ? rc->rotary_dim : rc->head_size;
  p->off = rc->rotary_offset;
  p->factor = rc->attention_factor;
  p->sin_sign = rc->conjugate ? -1.f : 1.f;
}

// Ranges that the line of work is cut into: with Hk chunks each they should
// fill the SMs evenly, and few ranges leave few partial results: the fewest
// that keep 94 % of the SMs busy, else the best of up to four rounds.
int pick_ranges(int sms, int Hk) {
  int best = 1;
  double best_share = 0.0;
  for (int n = std::max(1, sms / Hk); n <= std::max(1, 4 * sms / Hk); ++n) {
    const int chunks = n * Hk, rounds = (chunks + sms - 1) / sms;
    const double share = (double)chunks / (rounds * sms);
    if (share > best_share + 1e-9) {
      best = n;
      best_share = share;
    }
    if (share >= 0.94) break;
  }
  return best;
}

// Arguments every paged call of a step has.
pa_status check_paged(pa_tree_handle h, const void* key_cache, const void* value_cache, const int32_t* block_table,
                      const int32_t* cum, const int32_t* past, int batch, int token_count) {
  const pa_config& c = h->cfg;
  if (batch < 1 || batch > c.max_batch)
    return tree_fail(h, PA_INVALID_ARGUMENT, "batch must be in [1, max_batch=%d] (got %d)", c.max_batch, batch);
  if (token_count < 0 || token_count > c.max_tokens)
    return tree_fail(h, PA_INVALID_ARGUMENT, "token_count must be in [0, max_tokens=%d] (got %d)", c.max_tokens,
                     token_count);
  struct { const void* p; const char* name; size_t align; } args[] = {
      {key_cache, "key_cache", 16}, {value_cache, "value_cache", 16}, {block_table, "block_table", 4},
      {cum, "cumulative_sequence_lengths", 4}, {past, "past_sequence_lengths", 4}};
  for (auto& a : args) {
    if (!a.p) return tree_fail(h, PA_INVALID_ARGUMENT, "%s must not be NULL", a.name);
    if (!aligned(a.p, a.align))
      return tree_fail(h, PA_INVALID_ARGUMENT, "%s must be %zu-byte aligned", a.name, a.align);
  }
  if (key_cache == value_cache)
    return tree_fail(h, PA_INVALID_ARGUMENT, "key_cache and value_cache must be distinct buffers");
  return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_rotary_steps(const pa_rotary_scaling* sc, int rotary_dim, uint64_t* steps, float* attention_factor) {
  if (!sc) return pa::host_fail(PA_INVALID_ARGUMENT, "scaling must not be NULL");
  if (!steps) return pa::host_fail(PA_INVALID_ARGUMENT, "steps must not be NULL");
  if (rotary_dim <= 0 || rotary_dim % 2 || rotary_dim > 512)
    return pa::host_fail(PA_INVALID_ARGUMENT, "rotary_dim must be even and in [2, 512] (got %d)", rotary_dim);
  if (sc->type < PA_ROTARY_SCALE_NONE || sc->type > PA_ROTARY_SCALE_BY_WAVELENGTH)
    return pa::host_fail(PA_INVALID_ARGUMENT, "type must be one of PA_ROTARY_SCALE_* (got %d)", sc->type);
  if (!(sc->base > 1.0) || !std::isfinite(sc->base))
    return pa::host_fail(PA_INVALID_ARGUMENT, "base must be finite and > 1 (got %g)", sc->base);
  const double s = sc->type == PA_ROTARY_SCALE_NONE ? 1.0 : sc->factor;
  if (!(s >= 1.0) || !std::isfinite(s))
    return pa::host_fail(PA_INVALID_ARGUMENT, "factor must be finite and >= 1 (got %g)", s);
  const bool ramped = sc->type >= PA_ROTARY_SCALE_BY_PARTS;
  const double L = sc->original_positions;
  if (ramped && (!(L > 0.0) || !std::isfinite(L)))
    return pa::host_fail(PA_INVALID_ARGUMENT, "original_positions must be finite and > 0 (got %g)", L);
  if (ramped && !(sc->low > 0.0 && sc->high > sc->low && std::isfinite(sc->high)))
    return pa::host_fail(PA_INVALID_ARGUMENT, "low and high must be finite with 0 < low < high (got %g, %g)", sc->low,
                         sc->high);
  const double R = rotary_dim;
  double base = sc->base, lo = 0.0, hi = 1.0;
  if (sc->type == PA_ROTARY_SCALE_BASE && rotary_dim > 2) base *= std::pow(s, R / (R - 2.0));
  if (sc->type == PA_ROTARY_SCALE_BY_PARTS) {
    auto at = [&](double turns) { return R * std::log(L / (2.0 * kPi * turns)) / (2.0 * std::log(base)); };
    lo = std::max(std::floor(at(sc->high)), 0.0);
    hi = std::min(std::ceil(at(sc->low)), R - 1.0);
    if (hi - lo < 0.001) hi = lo + 0.001;  // a step instead of a ramp
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (sc->type == PA_ROTARY_SCALE_LINEAR) f /= s;
    if (sc->type == PA_ROTARY_SCALE_BY_PARTS) {
      const double r = std::min(std::max((i - lo) / (hi - lo), 0.0), 1.0);
      f = f / s * r + f * (1.0 - r);
    }
    if (sc->type == PA_ROTARY_SCALE_BY_WAVELENGTH) {
      const double k = std::min(std::max((L * f / (2.0 * kPi) - sc->low) / (sc->high - sc->low), 0.0), 1.0);
      f = f / s * (1.0 - k) + f * k;
    }
    // f <= 1 radian, so the step is below 2^63
    steps[i] = (uint64_t)std::llround(std::ldexp(f / (2.0 * kPi), 64));
  }
  if (attention_factor)
    *attention_factor = sc->type == PA_ROTARY_SCALE_BY_PARTS ? (float)(0.1 * std::log(s) + 1.0) : 1.f;
  return PA_OK;
}

void pa_rotary_config_init(pa_rotary_config* rc) {
  if (!rc) return;
  memset(rc, 0, sizeof(*rc));
  rc->attention_factor = 1.f;
}

pa_status pa_rotary(const pa_rotary_config* rc, const uint64_t* steps, const int32_t* positions, int token_count,
                    int num_heads, const void* query, int64_t query_stride, void* query_out,
                    int64_t query_out_stride, int kv_num_heads, const void* key, int64_t key_stride, void* key_out,
                    int64_t key_out_stride, void* stream) {
  pa_status st = check_rotary(nullptr, rc);
  if (st != PA_OK) return st;
  if (token_count < 0) return pa::host_fail(PA_INVALID_ARGUMENT, "token_count must be >= 0 (got %d)", token_count);
  if (num_heads < 0 || kv_num_heads < 0 || num_heads > pa::kRotaryMaxHeads || kv_num_heads > pa::kRotaryMaxHeads)
    return pa::host_fail(PA_INVALID_ARGUMENT, "num_heads and kv_num_heads must be in [0, 4096] (got %d, %d)",
                         num_heads, kv_num_heads);
  if (token_count == 0 || num_heads + kv_num_heads == 0) return PA_OK;
  if (!steps || !aligned(steps, 8))
    return pa::host_fail(PA_INVALID_ARGUMENT, "steps must be an 8-byte aligned device pointer");
  if (!positions || !aligned(positions, 4))
    return pa::host_fail(PA_INVALID_ARGUMENT, "positions must be a 4-byte aligned device pointer");
  const int D = rc->head_size;
  const long long e = rc->dtype == PA_ROTARY_FP32 ? 4 : 2;
  struct { const char* in; const char* out; int heads; const void* src; int64_t ss; void* dst; int64_t ds; } t[2] = {
      {"query", "query_out", num_heads, query, query_stride, query_out, query_out_stride},
      {"key", "key_out", kv_num_heads, key, key_stride, key_out, key_out_stride}};
  Rows in[2] = {}, out[2] = {};
  for (int i = 0; i < 2; ++i) {
    if (t[i].heads == 0) continue;
    if ((st = check_rows(nullptr, t[i].in, t[i].src, token_count, t[i].heads, D, &t[i].ss)) != PA_OK) return st;
    if ((st = check_rows(nullptr, t[i].out, t[i].dst, token_count, t[i].heads, D, &t[i].ds)) != PA_OK) return st;
    in[i] = Rows{t[i].src, token_count, t[i].ss * e, (long long)t[i].heads * D * e};
    out[i] = Rows{t[i].dst, token_count, t[i].ds * e, (long long)t[i].heads * D * e};
    if (!same(in[i], out[i]) && overlap(in[i], out[i]))
      return pa::host_fail(PA_INVALID_ARGUMENT, "%s overlaps %s without being it", t[i].out, t[i].in);
  }
  if (num_heads && kv_num_heads && (overlap(out[0], out[1]) || overlap(out[0], in[1]) || overlap(out[1], in[0])))
    return pa::host_fail(PA_INVALID_ARGUMENT, "query_out and key_out must not overlap each other or the other input");
  const Named writes[] = {{out[0], "query_out"}, {out[1], "key_out"}};
  const Named reads[] = {plain(positions, 4LL * token_count, "positions"),
                         plain(steps, 8LL * ((rc->rotary_dim ? rc->rotary_dim : D) / 2), "steps")};
  if ((st = check_apart(nullptr, writes, reads)) != PA_OK) return st;
  pa::RotaryParams p{};
  fill_rotary(&p, rc, steps, positions, token_count);
  p.q = {t[0].src, t[0].dst, t[0].ss, t[0].ds, t[0].heads};
  p.k = {t[1].src, t[1].dst, t[1].ss, t[1].ds, t[1].heads};
  cudaError_t ce = pa::launch_rotary(p, rc->dtype, rc->interleaved, static_cast<cudaStream_t>(stream));
  if (ce != cudaSuccess) return tree_cuda_fail(nullptr, ce, "rotary launch");
  return PA_OK;
}

pa_status pa_tree_create(const pa_config* cfg, int max_draft_tokens, pa_tree_handle* out) {
  if (!out) return pa::host_fail(PA_INVALID_ARGUMENT, "out must not be NULL");
  *out = nullptr;
  if (!cfg) return pa::host_fail(PA_INVALID_ARGUMENT, "config: NULL");
  pa_config c = *cfg;
  c.do_rotary = 0;  // the layer's own rotary is not used here
  c.rotary_offset = 0;
  char msg[512];
  pa_status st = pa_validate_config(&c, msg, sizeof(msg));
  if (st != PA_OK) return pa::host_fail(st, "%s", msg);
  if (max_draft_tokens < 1 || max_draft_tokens > pa::kTreeMaxDraft)
    return pa::host_fail(PA_INVALID_ARGUMENT, "max_draft_tokens must be in [1, %d] (got %d)", pa::kTreeMaxDraft,
                         max_draft_tokens);
  if (c.kv_cache_layout != PA_LAYOUT_SEPARATE)
    return pa::host_fail(PA_NOT_SUPPORTED, "trees are built for separate K and V caches (kv_cache_layout SEPARATE)");
  if (c.cache_dtype != PA_CACHE_FP16 && c.cache_dtype != PA_CACHE_BF16)
    return pa::host_fail(PA_NOT_SUPPORTED, "trees are built for a cache_dtype of fp16 or bfloat16");
  if (c.num_heads > pa::kRotaryMaxHeads)
    return pa::host_fail(PA_NOT_SUPPORTED, "trees are built for num_heads <= %d (got %d)", pa::kRotaryMaxHeads, c.num_heads);
  if (c.packed_qkv || c.qk_norm)
    return pa::host_fail(PA_NOT_SUPPORTED, "trees take neither packed_qkv nor qk_norm");
  pa_tree_handle h = new (std::nothrow) pa_tree_handle_s();
  if (!h) return pa::host_fail(PA_CUDA_ERROR, "pa_tree_create: out of host memory");
  h->cfg = *cfg;
  h->max_draft = max_draft_tokens;
  h->words = (max_draft_tokens + 31) / 32;
  h->scale = c.scale > 0.f ? c.scale : 1.f / std::sqrt((float)c.head_size);
  h->bf16 = c.cache_dtype == PA_CACHE_BF16;
  const int kv_cap = c.max_blocks_per_seq * c.block_size;
  h->max_kv = c.max_kv_len_bound > 0 ? std::min(c.max_kv_len_bound, kv_cap) : kv_cap;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
  if (e != cudaSuccess) {
    delete h;
    return tree_cuda_fail(nullptr, e, "pa_tree_create");
  }
  // Workspace: error word, counters, the cut units, the starts of the groups
  // of sequences (per CTA) and two partial results per chunk (256-byte
  // aligned pieces).
  const int G = c.num_heads / c.kv_num_heads;
  // Replicas of the rows where few rows would leave most softmax warps idle.
  // At head_size 128 the K/V stream covers one warp's softmax, and there is
  // no shared memory left to join replicas in.
  const int rows = max_draft_tokens * G;
  h->rep = c.head_size == 64 ? (rows <= 32 ? 4 : rows <= 64 ? 2 : 1) : 1;
  h->tile_tokens = pa::kPrefillRows / h->rep / G;
  if (e == cudaSuccess)
    e = c.head_size == 64    ? pa::tree_configure<64>(h->bf16, h->rep)
        : c.head_size == 128 ? pa::tree_configure<128>(h->bf16, h->rep)
                             : pa::tree_configure<256>(h->bf16, h->rep);
  // rows of a unit: two row tiles at most, one at head_size 256
  h->part_rows = max_draft_tokens <= h->tile_tokens ? (max_draft_tokens * G + 31) / 32 * 32
                 : c.head_size == 256               ? pa::kPrefillRows
                                                    : 2 * pa::kPrefillRows;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  h->n_ranges = pick_ranges(h->num_sms, c.kv_num_heads);
  const size_t chunks = (size_t)h->n_ranges * c.kv_num_heads, D = c.head_size;
  const size_t o_cnt = 256, o_cut = 512, o_grp = o_cut + up(sizeof(pa::Cut) * chunks);
  const size_t o_ml = o_grp + up(sizeof(int) * h->num_sms * ((c.max_batch + 31) / 32));
  const size_t o_po = o_ml + up(sizeof(float2) * 2 * chunks * h->part_rows);
  const size_t ws_bytes = o_po + sizeof(float) * 2 * chunks * h->part_rows * D;
  if (e == cudaSuccess) e = cudaMalloc(&h->ws, ws_bytes);
  if (e == cudaSuccess) e = cudaMemset(h->ws, 0, o_cut);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    if (h->ws) cudaFree(h->ws);
    delete h;
    return tree_cuda_fail(nullptr, e, "pa_tree_create");
  }
  uint8_t* w = static_cast<uint8_t*>(h->ws);
  h->err = reinterpret_cast<int*>(w);
  h->counters = reinterpret_cast<pa::TreeCounters*>(w + o_cnt);
  h->cuts = reinterpret_cast<pa::Cut*>(w + o_cut);
  h->groups = reinterpret_cast<int*>(w + o_grp);
  h->part_ml = reinterpret_cast<float2*>(w + o_ml);
  h->part_o = reinterpret_cast<float4*>(w + o_po);
  *out = h;
  return PA_OK;
}

pa_status pa_tree_destroy(pa_tree_handle h) {
  if (!h) return PA_OK;
  OnDevice g(h->device);
  if (h->ws) cudaFree(h->ws);
  delete h;
  return PA_OK;
}

const char* pa_tree_last_error_message(pa_tree_handle h) { return h ? h->msg.c_str() : pa_last_error_message(nullptr); }

pa_status pa_tree_check_device_error(pa_tree_handle h, int* code) {
  if (!h || !code) return tree_fail(h, PA_INVALID_ARGUMENT, "bad arguments");
  OnDevice g(h->device);
  cudaError_t e = cudaDeviceSynchronize();
  int v[2] = {0, 0};
  if (e == cudaSuccess) e = cudaMemcpy(v, h->err, sizeof(v), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, sizeof(v));
  if (e != cudaSuccess) return tree_cuda_fail(h, e, "pa_tree_check_device_error");
  *code = v[0];
  if (v[0] && v[1])
    return tree_fail(h, PA_DEVICE_DATA_ERROR, "device data error bits 0x%x; a wait gave up at site 0x%x", v[0], v[1]);
  if (v[0]) return tree_fail(h, PA_DEVICE_DATA_ERROR, "device data error bits 0x%x", v[0]);
  return PA_OK;
}

pa_status pa_tree_write(pa_tree_handle h, const pa_rotary_config* rc, const uint64_t* steps, const int32_t* positions,
                        const void* query, int64_t query_stride, const void* key, int64_t key_stride,
                        const void* value, int64_t value_stride, void* query_out, void* key_cache, void* value_cache,
                        const int32_t* block_table, const int32_t* cum, const int32_t* past, int batch,
                        int token_count, void* stream) {
  if (!h) return pa::host_fail(PA_INVALID_ARGUMENT, "handle must not be NULL");
  const pa_config& c = h->cfg;
  pa_status st = check_rotary(h, rc);
  if (st != PA_OK) return st;
  if (rc->head_size != c.head_size || rc->dtype != (h->bf16 ? PA_ROTARY_BF16 : PA_ROTARY_FP16))
    return tree_fail(h, PA_INVALID_ARGUMENT, "the rotary config's head_size and dtype must be the handle's");
  if ((st = check_paged(h, key_cache, value_cache, block_table, cum, past, batch, token_count)) != PA_OK) return st;
  if (token_count == 0) return PA_OK;
  if (!steps || !aligned(steps, 8)) return tree_fail(h, PA_INVALID_ARGUMENT, "steps must be an 8-byte aligned device pointer");
  if (!positions || !aligned(positions, 4))
    return tree_fail(h, PA_INVALID_ARGUMENT, "positions must be a 4-byte aligned device pointer");
  const int H = c.num_heads, Hk = c.kv_num_heads, D = c.head_size;
  int64_t out_stride = 0;
  if ((st = check_rows(h, "query", query, token_count, H, D, &query_stride)) != PA_OK ||
      (st = check_rows(h, "key", key, token_count, Hk, D, &key_stride)) != PA_OK ||
      (st = check_rows(h, "value", value, token_count, Hk, D, &value_stride)) != PA_OK ||
      (st = check_rows(h, "query_out", query_out, token_count, H, D, &out_stride)) != PA_OK)
    return st;
  const Rows qi{query, token_count, query_stride * 2, (long long)H * D * 2};
  const Rows qo{query_out, token_count, out_stride * 2, (long long)H * D * 2};
  const Rows ki{key, token_count, key_stride * 2, (long long)Hk * D * 2};
  const Rows vi{value, token_count, value_stride * 2, (long long)Hk * D * 2};
  const long long pool = (long long)c.num_blocks * c.block_size * Hk * D * 2;
  const Rows kc{key_cache, 1, pool, pool}, vc{value_cache, 1, pool, pool};
  if ((!same(qi, qo) && overlap(qi, qo)) || overlap(qo, ki) || overlap(qo, vi))
    return tree_fail(h, PA_INVALID_ARGUMENT, "query_out must be query or overlap no input");
  for (const Rows* r : {&qi, &qo, &ki, &vi})
    if (overlap(*r, kc) || overlap(*r, vc))
      return tree_fail(h, PA_INVALID_ARGUMENT, "the pools must not overlap query, key, value or query_out");
  if (overlap(kc, vc)) return tree_fail(h, PA_INVALID_ARGUMENT, "key_cache and value_cache must not overlap");
  const Named writes[] = {{qo, "query_out"}, {kc, "key_cache"}, {vc, "value_cache"}};
  const Named reads[] = {plain(positions, 4LL * token_count, "positions"),
                         plain(steps, 8LL * ((rc->rotary_dim ? rc->rotary_dim : D) / 2), "steps"),
                         plain(block_table, 4LL * batch * c.max_blocks_per_seq, "block_table"),
                         plain(cum, 4LL * (batch + 1), "cumulative_sequence_lengths"),
                         plain(past, 4LL * batch, "past_sequence_lengths")};
  if ((st = check_apart(h, writes, reads)) != PA_OK) return st;
  OnDevice g(h->device);
  pa::RotaryParams p{};
  fill_rotary(&p, rc, steps, positions, token_count);
  p.q = {query, query_out, query_stride, out_stride, H};
  p.k = {key, nullptr, key_stride, 0, Hk};
  p.v = {value, nullptr, value_stride, 0, Hk};
  p.key_cache = key_cache;
  p.value_cache = value_cache;
  p.block_table = block_table;
  p.cum = cum;
  p.past = past;
  p.batch = batch;
  p.bs = c.block_size;
  p.NB = c.num_blocks;
  p.MB = c.max_blocks_per_seq;
  p.err = h->err;
  cudaError_t e = pa::launch_rotary(p, rc->dtype, rc->interleaved, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return tree_cuda_fail(h, e, "tree write launch");
  return PA_OK;
}

pa_status pa_tree_attention(pa_tree_handle h, const void* query, const void* key_cache, const void* value_cache,
                            const int32_t* block_table, const int32_t* cum, const int32_t* past, int batch,
                            int token_count, const pa_tree_inputs* inputs, void* output, void* stream) {
  if (!h) return pa::host_fail(PA_INVALID_ARGUMENT, "handle must not be NULL");
  const pa_config& c = h->cfg;
  pa_status st = check_paged(h, key_cache, value_cache, block_table, cum, past, batch, token_count);
  if (st != PA_OK) return st;
  if (token_count == 0) return PA_OK;
  static const pa_tree_inputs kNone = {};
  const pa_tree_inputs* x = inputs ? inputs : &kNone;
  if (!query || !aligned(query, 16)) return tree_fail(h, PA_INVALID_ARGUMENT, "query must be a 16-byte aligned device pointer");
  if (!output || !aligned(output, 16))
    return tree_fail(h, PA_INVALID_ARGUMENT, "output must be a 16-byte aligned device pointer");
  if (!aligned(x->positions, 4) || !aligned(x->tree_mask, 4) || !aligned(x->distance_slopes, 4))
    return tree_fail(h, PA_INVALID_ARGUMENT, "positions, tree_mask and distance_slopes must be 4-byte aligned");
  if (!aligned(x->head_sink, 2)) return tree_fail(h, PA_INVALID_ARGUMENT, "head_sink must be 2-byte aligned");
  const int H = c.num_heads, Hk = c.kv_num_heads, D = c.head_size;
  const long long row = (long long)H * D * 2, pool = (long long)c.num_blocks * c.block_size * Hk * D * 2;
  const Rows q{query, token_count, row, row}, o{output, token_count, row, row};
  const Rows kc{key_cache, 1, pool, pool}, vc{value_cache, 1, pool, pool};
  if (overlap(o, q) || overlap(o, kc) || overlap(o, vc))
    return tree_fail(h, PA_INVALID_ARGUMENT, "output must not overlap query or the pools");
  const Named writes[] = {{o, "output"}};
  const Named reads[] = {plain(x->positions, 4LL * token_count, "positions"),
                         plain(x->tree_mask, 4LL * token_count * h->words, "tree_mask"),
                         plain(x->distance_slopes, 4LL * H, "distance_slopes"),
                         plain(x->head_sink, 2LL * H, "head_sink"),
                         plain(block_table, 4LL * batch * c.max_blocks_per_seq, "block_table"),
                         plain(cum, 4LL * (batch + 1), "cumulative_sequence_lengths"),
                         plain(past, 4LL * batch, "past_sequence_lengths")};
  if ((st = check_apart(h, writes, reads)) != PA_OK) return st;
  OnDevice g(h->device);
  pa::TreeParams p{};
  p.value_cache = static_cast<const __half*>(value_cache);
  p.block_table = block_table;
  p.cum = cum;
  p.past = past;
  p.positions = x->positions;
  p.mask = x->tree_mask;
  p.slopes = x->distance_slopes;
  p.head_sink = static_cast<const __half*>(x->head_sink);
  p.out = static_cast<__half*>(output);
  p.batch = batch;
  p.T = token_count;
  p.H = H;
  p.Hk = Hk;
  p.G = H / Hk;
  p.D = D;
  p.bs = c.block_size;
  p.log_bs = 0;
  while ((1 << p.log_bs) < c.block_size) ++p.log_bs;
  p.NB = c.num_blocks;
  p.MB = c.max_blocks_per_seq;
  p.max_draft = h->max_draft;
  p.words = h->words;
  p.max_kv = h->max_kv;
  p.window = c.local_window_size;
  p.scale = h->scale;
  p.softcap = c.softcap;
  p.tile_tokens = h->tile_tokens;
  p.unit_tokens = D == 256 ? h->tile_tokens : 2 * h->tile_tokens;
  p.inv_unit = (1 << 20) / p.unit_tokens + 1;
  const int page_rows = std::min(c.block_size, D == 256 ? 64 : 128);  // of a key tile
  p.log_page_rows = 0;
  while ((1 << p.log_page_rows) < page_rows) ++p.log_page_rows;
  p.oob_row = c.num_blocks * c.block_size;
  p.n_ranges = h->n_ranges;
  p.rep = h->rep;
  p.q_tiles = D != 256 && h->max_draft > h->tile_tokens ? 2 : 1;
  p.counters = h->counters;
  p.groups = h->groups;
  p.n_groups = (batch + 31) / 32;
  p.cuts = h->cuts;
  p.part_ml = h->part_ml;
  p.part_o = h->part_o;
  p.part_rows = h->part_rows;
  p.err = h->err;
  p.err_site = h->err + 1;
  CUtensorMap tq, tk, tv;
  if (!pa::encode_rows_map(&tq, query, D, H, token_count, p.G, p.tile_tokens) ||
      !pa::encode_groups_map(&tk, key_cache, D, Hk, (long long)c.num_blocks * c.block_size, page_rows) ||
      !pa::encode_groups_map(&tv, value_cache, D, Hk, (long long)c.num_blocks * c.block_size, page_rows))
    return tree_fail(h, PA_CUDA_ERROR, "cuTensorMapEncodeTiled failed");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = D == 64    ? pa::launch_tree<64>(tq, tk, tv, p, h->bf16, h->num_sms, s)
                  : D == 128 ? pa::launch_tree<128>(tq, tk, tv, p, h->bf16, h->num_sms, s)
                             : pa::launch_tree<256>(tq, tk, tv, p, h->bf16, h->num_sms, s);
  if (e != cudaSuccess) return tree_cuda_fail(h, e, "tree attention launch");
  return PA_OK;
}

pa_status pa_tree_commit(pa_tree_handle h, void* const* key_caches, void* const* value_caches, int num_layers,
                         const int32_t* block_table, const int32_t* past, const int32_t* accepted,
                         const int32_t* accepted_count, int max_accepted, int batch, int32_t* new_past,
                         void* stream) {
  if (!h) return pa::host_fail(PA_INVALID_ARGUMENT, "handle must not be NULL");
  const pa_config& c = h->cfg;
  if (num_layers < 1 || num_layers > 65536)
    return tree_fail(h, PA_INVALID_ARGUMENT, "num_layers must be in [1, 65536] (got %d)", num_layers);
  if (!key_caches || !value_caches)
    return tree_fail(h, PA_INVALID_ARGUMENT, "key_caches and value_caches must not be NULL");
  if (batch < 1 || batch > c.max_batch)
    return tree_fail(h, PA_INVALID_ARGUMENT, "batch must be in [1, max_batch=%d] (got %d)", c.max_batch, batch);
  if (max_accepted < 1 || max_accepted > h->max_draft)
    return tree_fail(h, PA_INVALID_ARGUMENT, "max_accepted must be in [1, max_draft_tokens=%d] (got %d)", h->max_draft,
                     max_accepted);
  struct { const void* p; const char* name; } args[] = {{block_table, "block_table"},
                                                        {past, "past_sequence_lengths"},
                                                        {accepted, "accepted"},
                                                        {accepted_count, "accepted_count"}};
  for (auto& a : args)
    if (!a.p || !aligned(a.p, 4))
      return tree_fail(h, PA_INVALID_ARGUMENT, "%s must be a 4-byte aligned device pointer", a.name);
  if (!aligned(new_past, 4)) return tree_fail(h, PA_INVALID_ARGUMENT, "new_past must be 4-byte aligned");
  const Named writes[] = {plain(new_past, 4LL * batch, "new_past")};
  const Named reads[] = {plain(past, 4LL * batch, "past_sequence_lengths"),
                         plain(accepted_count, 4LL * batch, "accepted_count"),
                         plain(accepted, 4LL * batch * max_accepted, "accepted"),
                         plain(block_table, 4LL * batch * c.max_blocks_per_seq, "block_table")};
  pa_status st = check_apart(h, writes, reads);
  if (st != PA_OK) return st;
  // Pools: present, aligned and apart from one another.
  const uintptr_t bytes = (uintptr_t)c.num_blocks * c.block_size * c.kv_num_heads * c.head_size * 2;
  std::unique_ptr<uintptr_t[]> store(new (std::nothrow) uintptr_t[2 * (size_t)num_layers]);
  if (!store) return tree_fail(h, PA_CUDA_ERROR, "pa_tree_commit: out of host memory");
  uintptr_t *at = store.get(), *end = at;
  for (int l = 0; l < num_layers; ++l) {
    for (void* q : {key_caches[l], value_caches[l]}) {
      if (!q || !aligned(q, 16))
        return tree_fail(h, PA_INVALID_ARGUMENT, "layer %d: key_cache and value_cache must be 16-byte aligned device pointers", l);
      if (new_past && overlap(writes[0].rows, Rows{q, 1, (long long)bytes, (long long)bytes}))
        return tree_fail(h, PA_INVALID_ARGUMENT, "new_past must not overlap the pools");
      *end++ = reinterpret_cast<uintptr_t>(q);
    }
  }
  if (!std::is_sorted(at, end)) std::sort(at, end);
  for (uintptr_t* q = at + 1; q < end; ++q)
    if (q[0] - q[-1] < bytes) return tree_fail(h, PA_INVALID_ARGUMENT, "two of the pools overlap");
  OnDevice g(h->device);
  pa::CommitParams p{};
  p.row_vecs = c.kv_num_heads * c.head_size / 8;
  p.block_table = block_table;
  p.past = past;
  p.accepted = accepted;
  p.count = accepted_count;
  p.max_accepted = max_accepted;
  p.max_draft = h->max_draft;
  p.batch = batch;
  p.bs = c.block_size;
  p.NB = c.num_blocks;
  p.MB = c.max_blocks_per_seq;
  p.err = h->err;
  for (int l0 = 0; l0 < num_layers; l0 += pa::kCommitLayers) {
    const int n = std::min(pa::kCommitLayers, num_layers - l0);
    for (int l = 0; l < n; ++l) {
      p.pools[2 * l] = key_caches[l0 + l];
      p.pools[2 * l + 1] = value_caches[l0 + l];
    }
    p.n_pools = 2 * n;
    p.new_past = l0 == 0 ? new_past : nullptr;
    cudaError_t e = pa::launch_commit(p, h->num_sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return tree_cuda_fail(h, e, "commit launch");
  }
  return PA_OK;
}

}  // extern "C"
