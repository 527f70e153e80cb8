// extern "C" entry points of the latent-attention calls: validation, plan, workspace.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "kernels.h"
#include "latent.h"

using namespace v4a;

int v4a::sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
    return v;
  return 152;
}

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool positive(float x) { return x > 0.f && std::isfinite(x); }
inline bool known_type(int32_t t) { return t == V4A_FP32 || t == V4A_BF16; }
inline size_t elem_size(int32_t t) { return t == V4A_BF16 ? 2 : 4; }

int check_rope(const v4a_rope_cfg* r) {
  if (!r) return V4A_ERR_ARG;
  if (r->layout != V4A_ROPE_INTERLEAVED && r->layout != V4A_ROPE_HALF) return V4A_ERR_UNSUPPORTED;
  if (r->scaling < V4A_ROPE_SCALE_NONE || r->scaling > V4A_ROPE_SCALE_YARN) return V4A_ERR_UNSUPPORTED;
  if (r->dim < 2 || r->dim % 2 != 0 || r->dim > 2 * kRotMaxPairs) return V4A_ERR_UNSUPPORTED;
  if (r->reserved != 0 || !positive(r->base) || !positive(r->amplitude)) return V4A_ERR_ARG;
  if (r->scaling != V4A_ROPE_SCALE_NONE && !positive(r->factor)) return V4A_ERR_ARG;
  if (r->scaling >= V4A_ROPE_SCALE_BY_PARTS &&
      (!positive(r->orig_max_pos) || !positive(r->low) || !positive(r->high) || !(r->low < r->high)))
    return V4A_ERR_ARG;
  if (r->scaling == V4A_ROPE_SCALE_YARN && !(r->base > 1.f)) return V4A_ERR_ARG;
  return V4A_OK;
}

RotTab make_rot(const v4a_rope_cfg* r) {
  RotTab t{};
  t.dim = r->dim;
  t.layout = r->layout;
  t.amp = r->amplitude;
  const double two_pi = 6.283185307179586476925286766559;
  const double d = r->dim, base = r->base, f = r->factor, orig = r->orig_max_pos;
  double a = 0, b = 1;
  if (r->scaling == V4A_ROPE_SCALE_YARN) {
    auto pair = [&](double turns) { return d * std::log(orig / (turns * two_pi)) / (2 * std::log(base)); };
    a = std::fmax(std::floor(pair(r->high)), 0.0);
    b = std::fmin(std::ceil(pair(r->low)), d - 1);
    b = a + std::fmax(b - a, 1e-3);
  }
  // theta_i = base^(-2i/d): a power for every eighth pair, products in between
  double step[8] = {1};
  for (int k = 1; k < 8; ++k) step[k] = std::pow(base, -2.0 * k / d);
  double theta0 = 1;
  for (int i = 0; i < r->dim / 2; ++i) {
    if (i % 8 == 0) theta0 = std::pow(base, -2.0 * i / d);
    double theta = theta0 * step[i % 8];
    double keep = 1;
    if (r->scaling == V4A_ROPE_SCALE_LINEAR) keep = 0;
    if (r->scaling == V4A_ROPE_SCALE_BY_PARTS)
      keep = (orig * theta / two_pi - r->low) / ((double)r->high - r->low);
    if (r->scaling == V4A_ROPE_SCALE_YARN) keep = 1 - (i - a) / (b - a);
    keep = std::fmin(std::fmax(keep, 0.0), 1.0);
    if (r->scaling != V4A_ROPE_SCALE_NONE) theta *= keep + (1 - keep) / f;
    double phi = theta / two_pi;
    phi -= std::floor(phi);                      // whole turns a position change nothing
    double psi = 4096.0 * phi;
    psi -= std::floor(psi);
    t.phi_hi[i] = (float)phi;
    t.phi_lo[i] = (float)(phi - (double)t.phi_hi[i]);
    t.psi_hi[i] = (float)psi;
    t.psi_lo[i] = (float)(psi - (double)t.psi_hi[i]);
  }
  return t;
}

int check_latent(const v4a_latent_cfg* c) {
  if (!c) return V4A_ERR_ARG;
  if (!known_type(c->dtype)) return V4A_ERR_UNSUPPORTED;
  const int rc = check_rope(&c->rope);
  if (rc) return rc;
  if (c->reserved != 0 || c->n_heads <= 0 || c->n_heads > 1024) return V4A_ERR_ARG;
  if (c->latent_dim < 8 || c->latent_dim % 8 || c->latent_dim > 1024) return V4A_ERR_UNSUPPORTED;
  if (c->rope.dim % 8 || c->rope.dim > 128) return V4A_ERR_UNSUPPORTED;
  if (c->nope_dim < 0 || c->nope_dim % 8 || c->nope_dim > 256) return V4A_ERR_UNSUPPORTED;
  if (c->v_dim < 8 || c->v_dim % 8 || c->v_dim > 256) return V4A_ERR_UNSUPPORTED;
  if (!(c->rms_eps >= 0.f) || !std::isfinite(c->rms_eps) || !positive(c->softmax_scale)) return V4A_ERR_ARG;
  return V4A_OK;
}

int check_latent_cache(const v4a_latent_cfg* c, const v4a_cache* cache) {
  const int rc = check_cache(cache, kBlock, c->latent_dim + c->rope.dim, false);
  if (rc) return rc;
  // tensor maps count pool rows in 31 bits
  return cache->n_pages * kBlock > INT32_MAX ? V4A_ERR_UNSUPPORTED : V4A_OK;
}

int check_batch(int32_t n_seq, int32_t n, const int32_t* cu, const int64_t* start) {
  if (n_seq < 0 || n < 0) return V4A_ERR_ARG;
  if (n_seq > V4A_MAX_SEQ) return V4A_ERR_UNSUPPORTED;
  if (n == 0 || n_seq == 0) return V4A_OK;
  return cu && start ? V4A_OK : V4A_ERR_ARG;
}

bool on_tensor_cores(const v4a_latent_cfg* c) {
  return c->dtype == V4A_BF16 && c->latent_dim == 512 && c->rope.dim == 64;
}

// The device counts the steps of a call in 31 bits, sums of two of them included.
constexpr int64_t kMostSteps = (int64_t)1 << 30;

// The plan of an absorbed call. False when there are too many steps.
bool make_plan(const v4a_latent_cfg* c, int32_t n_seq, int32_t n_tokens, int64_t max_pos, LatentPlan* pl) {
  const bool tc = on_tensor_cores(c);
  pl->tc = tc;
  pl->NR = tc ? 64 : 16;
  pl->TK = tc ? 128 : 32;
  const int64_t rows = (int64_t)n_tokens * c->n_heads;
  const int64_t units = (rows + pl->NR - 1) / pl->NR + n_seq;   // at most, over the sequences
  const int64_t tiles = max_pos / pl->TK + 1;
  if (rows > INT32_MAX / 2) return false;
  // sharing key tiles pays where an average sequence has several units (the device decides)
  pl->max_U = 1;
  while (tc && pl->max_U < 4 && rows / n_seq >= 2 * pl->max_U * pl->NR) pl->max_U *= 2;
  const int64_t most = tc ? sm_count() / 4 * 4 : 2 * sm_count();  // CTAs at once
  // Units are split along the keys where that fills the GPU (fewer than four a CTA) or evens
  // out sequences of different lengths (few new tokens each). Prompts, whose units' key counts
  // rise from one to the next, go as whole units, neighbours to neighbouring CTAs, unless single
  // units are long beside a CTA's part of all: only the device sees that (latent_split).
  const bool few = units < 4 * most || n_tokens < 4 * (int64_t)n_seq;
  pl->split = tiles == 1 ? kSplitNone : few ? kSplitAll : kSplitOnDevice;
  if (units * tiles >= kMostSteps) {
    if (pl->split == kSplitAll) return false;
    pl->split = kSplitNone;
  }
  const int64_t want = (pl->split == kSplitAll ? units * tiles : units) + 3;
  pl->split_ctas = (int32_t)(want < most ? want / 4 * 4 : most);
  pl->ctas = tc || pl->split == kSplitAll ? pl->split_ctas : (int32_t)(want < 65536 ? want / 4 * 4 : 65536);
  return true;
}

size_t part_bytes(const v4a_latent_cfg* c, const LatentPlan& pl, size_t* ml_at, size_t* job_at) {
  const size_t slots = (size_t)pl.split_ctas * 2;
  *ml_at = align_up(slots * pl.NR * c->latent_dim * sizeof(float), 256);
  *job_at = *ml_at + align_up(slots * pl.NR * 2 * sizeof(float), 256);
  return pl.split != kSplitNone ? *job_at + align_up(slots * 2 * sizeof(int32_t), 256) : 0;
}

// Steps that starting an item counts for when the line is cut into equal parts. Its copies, first
// logits and output take about two; counting more evens out the pairs that get many short items.
// us on the device with 0, 2, 4 and 6: 8,192-token prompt, 64 heads 1159, 975, 861, 880; 4,096
// tokens, 32 heads 211, 169, 162, 160; five ragged chunks, 16 heads 337, 307, 288, 279; four, 32
// heads 213, 161, 156, 154; four, 8 heads 123, 96, 83, 85.
constexpr int kExpandedSetup = 4;

// The plan of an expanded call (p->tc, pairs, split) and its workspace. False when there are
// too many steps.
bool plan_expanded(const v4a_latent_cfg* c, int32_t n_seq, int32_t n_q, int32_t n_k, LatentExpandedParams* p,
                   size_t* ml_at, size_t* job_at, size_t* bytes) {
  p->tc = c->dtype == V4A_BF16 && c->nope_dim == 128 && c->rope.dim == 64 && c->v_dim == 128;
  p->pairs = p->split = 0;
  *ml_at = *job_at = *bytes = 0;
  if (!p->tc) return true;
  const int64_t items = ((int64_t)n_q / 512 + n_seq) * c->n_heads;                     // at most
  const int64_t tiles = (int64_t)n_k / 128 + 1 + kExpandedSetup;
  if (items * tiles >= kMostSteps) return false;
  const int64_t pairs = sm_count() / 2;
  p->pairs = (int32_t)(items * tiles < pairs ? items * tiles : pairs);
  p->split = n_k > 128;
  p->setup = p->split ? kExpandedSetup : 0;
  if (p->split) {
    const size_t rows = (size_t)p->pairs * 2 * 512;
    *ml_at = rows * 128 * sizeof(float);
    *job_at = *ml_at + rows * 2 * sizeof(float);
    *bytes = *job_at + align_up((size_t)p->pairs * 8 * sizeof(int32_t), 256);
  }
  return true;
}

}  // namespace

extern "C" {

int v4a_rope(const v4a_rope_cfg* rope, int32_t dtype, int32_t n_tokens, int32_t n_heads, const int64_t* pos,
             const void* x, int64_t x_token_stride, int64_t x_head_stride, void* y, int64_t y_token_stride,
             int64_t y_head_stride, int32_t inverse, int32_t* dev_err, v4a_stream_t stream) {
  const int rc = check_rope(rope);
  if (rc) return rc;
  if (!known_type(dtype)) return V4A_ERR_UNSUPPORTED;
  if (n_tokens < 0 || n_heads < 0) return V4A_ERR_ARG;
  if (n_tokens == 0 || n_heads == 0) return V4A_OK;
  if (!pos || !x || !y || !aligned(x, elem_size(dtype)) || !aligned(y, elem_size(dtype))) return V4A_ERR_ARG;
  if (x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0) return V4A_ERR_ARG;
  // y's rows are apart from one another
  if (n_heads > 1 && y_head_stride < rope->dim) return V4A_ERR_ARG;
  if (n_tokens > 1 && y_token_stride < rope->dim) return V4A_ERR_ARG;
  if (x == y && ((n_tokens > 1 && x_token_stride != y_token_stride) ||
                 (n_heads > 1 && x_head_stride != y_head_stride)))
    return V4A_ERR_ARG;
  RopeParams p{};
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.inverse = inverse != 0;
  p.pos = pos;
  p.x = x;
  p.y = y;
  p.x_ts = x_token_stride;
  p.x_hs = x_head_stride;
  p.y_ts = y_token_stride;
  p.y_hs = y_head_stride;
  p.err = dev_err;
  p.rot = make_rot(rope);
  return launch_rope(p, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int v4a_latent_insert(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens, const int32_t* cu_tokens,
                      const int64_t* start_pos, const void* c, int64_t c_stride, const void* k_pe,
                      int64_t k_stride, const float* gamma, const v4a_cache* cache, int32_t* dev_err,
                      v4a_stream_t stream) {
  int rc = check_latent(cfg);
  if (rc) return rc;
  if ((rc = check_batch(n_seq, n_tokens, cu_tokens, start_pos))) return rc;
  if (n_seq == 0 || n_tokens == 0) return V4A_OK;
  if ((rc = check_latent_cache(cfg, cache))) return rc;
  const int64_t unit = 16 / (int64_t)elem_size(cfg->dtype);
  if (!c || !k_pe || !aligned(c, 16) || !aligned(k_pe, 16) || !aligned(gamma, 16)) return V4A_ERR_ARG;
  if (c_stride < 0 || k_stride < 0 || c_stride % unit || k_stride % unit) return V4A_ERR_ARG;
  LatentInsertParams p{};
  p.n_seq = n_seq;
  p.n_tokens = n_tokens;
  p.C = cfg->latent_dim;
  p.cu = cu_tokens;
  p.start = start_pos;
  p.c = c;
  p.k_pe = k_pe;
  p.c_stride = c_stride;
  p.k_stride = k_stride;
  p.gamma = gamma;
  p.eps = cfg->rms_eps;
  p.cache = view_of(cache);
  p.err = dev_err;
  p.rot = make_rot(&cfg->rope);
  return launch_latent_insert(p, cfg->dtype, reinterpret_cast<cudaStream_t>(stream));
}

int v4a_latent_gather(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_rows, const int32_t* cu_rows,
                      const int64_t* start_pos, const v4a_cache* cache, void* out, int32_t* dev_err,
                      v4a_stream_t stream) {
  int rc = check_latent(cfg);
  if (rc) return rc;
  if ((rc = check_batch(n_seq, n_rows, cu_rows, start_pos))) return rc;
  if (n_seq == 0 || n_rows == 0) return V4A_OK;
  if ((rc = check_latent_cache(cfg, cache))) return rc;
  if (!out || !aligned(out, 16)) return V4A_ERR_ARG;
  LatentGatherParams p{};
  p.n_seq = n_seq;
  p.n_rows = n_rows;
  p.row_bytes = (int32_t)((cfg->latent_dim + cfg->rope.dim) * elem_size(cfg->dtype));
  p.cu = cu_rows;
  p.start = start_pos;
  p.cache = view_of(cache);
  p.out = out;
  p.err = dev_err;
  return launch_latent_gather(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t v4a_latent_attn_workspace_size(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens,
                                      int64_t max_pos) {
  LatentPlan pl;
  size_t ml_at, job_at;
  if (check_latent(cfg) || n_seq < 0 || n_seq > V4A_MAX_SEQ || n_tokens < 0 || max_pos < 0 ||
      max_pos >= V4A_MAX_POS || n_tokens == 0 || n_seq == 0)
    return 0;
  return make_plan(cfg, n_seq, n_tokens, max_pos, &pl) ? part_bytes(cfg, pl, &ml_at, &job_at) : 0;
}

int v4a_latent_attn(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_tokens, const int32_t* cu_tokens,
                    const int64_t* start_pos, int64_t max_pos, const void* q, const v4a_cache* cache, void* out,
                    void* workspace, size_t workspace_bytes, int32_t* dev_err, v4a_stream_t stream) {
  int rc = check_latent(cfg);
  if (rc) return rc;
  if ((rc = check_batch(n_seq, n_tokens, cu_tokens, start_pos))) return rc;
  if (max_pos < 0 || max_pos >= V4A_MAX_POS) return V4A_ERR_ARG;
  if (n_seq == 0 || n_tokens == 0) return V4A_OK;
  if ((rc = check_latent_cache(cfg, cache))) return rc;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16)) return V4A_ERR_ARG;
  LatentAttnParams p{};
  if (!make_plan(cfg, n_seq, n_tokens, max_pos, &p.plan)) return V4A_ERR_UNSUPPORTED;
  size_t ml_at = 0, job_at = 0;
  const size_t need = part_bytes(cfg, p.plan, &ml_at, &job_at);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return V4A_ERR_ARG;
  p.n_seq = n_seq;
  p.n_tokens = n_tokens;
  p.H = cfg->n_heads;
  p.C = cfg->latent_dim;
  p.R = cfg->rope.dim;
  p.scale = cfg->softmax_scale;
  p.max_pos = max_pos;
  const int64_t reach = (int64_t)cache->max_blocks * kBlock;
  p.end = max_pos + 1 < reach ? max_pos + 1 : reach;
  p.cu = cu_tokens;
  p.start = start_pos;
  p.q = q;
  p.out = out;
  p.cache = view_of(cache);
  p.part_o = reinterpret_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + ml_at);
  p.part_job = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) + job_at);
  p.err = dev_err;
  return launch_latent_attn(p, cfg->dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t v4a_latent_attn_expanded_workspace_size(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_q, int32_t n_k) {
  LatentExpandedParams p{};
  size_t ml_at, job_at, bytes;
  if (check_latent(cfg) || n_seq <= 0 || n_seq > V4A_MAX_SEQ || n_q <= 0 || n_k < 0) return 0;
  return plan_expanded(cfg, n_seq, n_q, n_k, &p, &ml_at, &job_at, &bytes) ? bytes : 0;
}

int v4a_latent_attn_expanded(const v4a_latent_cfg* cfg, int32_t n_seq, int32_t n_q, const int32_t* cu_q,
                             int32_t n_k, const int32_t* cu_k, const void* q, const void* k,
                             int64_t k_token_stride, int64_t k_head_stride, const void* k_pe, int64_t k_pe_stride,
                             const void* v, int64_t v_token_stride, int64_t v_head_stride, int32_t causal,
                             void* out, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                             v4a_stream_t stream) {
  int rc = check_latent(cfg);
  if (rc) return rc;
  if (cfg->nope_dim < 8) return V4A_ERR_UNSUPPORTED;
  if (n_seq < 0 || n_q < 0 || n_k < 0) return V4A_ERR_ARG;
  if (n_seq > V4A_MAX_SEQ) return V4A_ERR_UNSUPPORTED;
  if (n_seq == 0 || n_q == 0) return V4A_OK;
  if (!cu_q || !cu_k || !q || !out || !aligned(q, 16) || !aligned(out, 16)) return V4A_ERR_ARG;
  const int64_t unit = 16 / (int64_t)elem_size(cfg->dtype);
  if (n_k > 0) {
    if (!k || !k_pe || !v || !aligned(k, 16) || !aligned(k_pe, 16) || !aligned(v, 16)) return V4A_ERR_ARG;
    const int64_t strides[5] = {k_token_stride, k_head_stride, k_pe_stride, v_token_stride, v_head_stride};
    for (int64_t s : strides)
      if (s <= 0 || s % unit || s > ((int64_t)1 << 36)) return V4A_ERR_ARG;
  }
  LatentExpandedParams p{};
  size_t ml_at, job_at, need;
  if (!plan_expanded(cfg, n_seq, n_q, n_k, &p, &ml_at, &job_at, &need)) return V4A_ERR_UNSUPPORTED;
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return V4A_ERR_ARG;
  p.part_o = reinterpret_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + ml_at);
  p.part_job = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) + job_at);
  p.n_seq = n_seq;
  p.n_q = n_q;
  p.n_k = n_k;
  p.H = cfg->n_heads;
  p.DN = cfg->nope_dim;
  p.DR = cfg->rope.dim;
  p.DV = cfg->v_dim;
  p.causal = causal != 0;
  p.scale = cfg->softmax_scale;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.q = q;
  p.k = k;
  p.k_pe = k_pe;
  p.v = v;
  p.out = out;
  p.k_ts = k_token_stride;
  p.k_hs = k_head_stride;
  p.pe_ts = k_pe_stride;
  p.v_ts = v_token_stride;
  p.v_hs = v_head_stride;
  p.err = dev_err;
  return launch_latent_expanded(p, cfg->dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
