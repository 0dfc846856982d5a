// Host runtime of the operators around a bank of experts and of gradient
// clipping: argument validation (all-or-nothing, before anything is enqueued),
// workspace sizes, launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "clip.hpp"
#include "experts.hpp"
#include "linear_host.hpp"

using namespace mr;

namespace {

constexpr int64_t kMaxTotal = (int64_t(1) << 31) - 1;  // choices, sorted rows

// A small contiguous array of 4-byte values.
mr_status check_array(const char* name, const void* p) {
  if (!p) return fail(MR_ERR_NULL, "%s is NULL", name);
  if (!aligned(p, 4)) return fail(MR_ERR_PARAM, "%s is not aligned to its type", name);
  return MR_OK;
}

mr_status check_choices(int64_t tokens, int64_t k, int64_t most) {
  MR_TRY(check_size("tokens", tokens, 0, kMaxRows));
  MR_TRY(check_size("k", k, 1, most));
  return check_size("tokens x k", tokens * k, 0, kMaxTotal);
}

}  // namespace

extern "C" {

// --------------------------------------------------------------- routing
mr_status route_tokens(const mr_route_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("experts", p->experts, 1, kMaxRouteExperts));
  MR_TRY(check_choices(p->tokens, p->k, p->experts < kMaxRouted ? p->experts : kMaxRouted));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if (p->normalize != 0 && p->normalize != 1) return fail(MR_ERR_PARAM, "normalize %d", p->normalize);
  if (p->tokens == 0) return MR_OK;
  const size_t es = size_of(p->dtype);
  MR_TRY(check_matrix("logits", p->logits, p->experts, p->ldl, es));
  MR_TRY(check_array("chosen", p->chosen));
  MR_TRY(check_array("weights", p->weights));
  MR_TRY(check_array("log_sum", p->log_sum));
  const int64_t c = p->tokens * p->k;
  Aliases al;
  al.in("logits", p->logits, p->tokens, p->experts, p->ldl, es);
  al.out("chosen", p->chosen, 1, c, c, 4);
  al.out("weights", p->weights, 1, c, c, 4);
  al.out("log_sum", p->log_sum, 1, p->tokens, p->tokens, 4);
  MR_TRY(al.set.check());
  RouteArgs a;
  memset(&a, 0, sizeof a);
  a.logits = p->logits, a.ldl = p->ldl;
  a.experts = p->chosen, a.weights = p->weights, a.log_sum = p->log_sum;
  a.tokens = p->tokens, a.n = (int32_t)p->experts, a.k = (int32_t)p->k, a.normalize = p->normalize;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrRoute, true, s, [&] { return launch_route(a, p->dtype, s); }, "routing launch");
}

mr_status route_tokens_backward(const mr_route_grad_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("experts", p->experts, 1, kMaxRouteExperts));
  MR_TRY(check_choices(p->tokens, p->k, p->experts < kMaxRouted ? p->experts : kMaxRouted));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if (p->normalize != 0 && p->normalize != 1) return fail(MR_ERR_PARAM, "normalize %d", p->normalize);
  if (p->tokens == 0) return MR_OK;
  const size_t es = size_of(p->dtype);
  if (!p->normalize) MR_TRY(check_matrix("logits", p->logits, p->experts, p->ldl, es));
  MR_TRY(check_array("chosen", p->chosen));
  MR_TRY(check_array("weights", p->weights));
  MR_TRY(check_array("dweights", p->dweights));
  MR_TRY(check_matrix("dlogits", p->dlogits, p->experts, p->ldd, es));
  const int64_t c = p->tokens * p->k;
  Aliases al;
  if (!p->normalize) al.in("logits", p->logits, p->tokens, p->experts, p->ldl, es);
  al.in("chosen", p->chosen, 1, c, c, 4);
  al.in("weights", p->weights, 1, c, c, 4);
  al.in("dweights", p->dweights, 1, c, c, 4);
  al.out("dlogits", p->dlogits, p->tokens, p->experts, p->ldd, es);
  MR_TRY(al.set.check());
  RouteGradArgs a;
  memset(&a, 0, sizeof a);
  a.logits = p->logits, a.ldl = p->ldl;
  a.experts = p->chosen, a.weights = p->weights, a.dweights = p->dweights;
  a.dlogits = p->dlogits, a.ldd = p->ldd;
  a.tokens = p->tokens, a.n = (int32_t)p->experts, a.k = (int32_t)p->k, a.normalize = p->normalize;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrRouteGrad, true, s, [&] { return launch_route_grad(a, p->dtype, s); }, "routing gradient launch");
}

// ----------------------------------------------------------------- order
size_t order_by_expert_workspace(const mr_order_problem* p) {
  if (!p || p->tokens < 1 || p->tokens > kMaxRows || p->k < 1 || p->k > kMaxChoices || p->tokens * p->k > kMaxTotal ||
      p->experts < 1 || p->experts > kMaxExperts)
    return 0;
  int32_t chunk, blocks, waves;
  order_plan(p->tokens * p->k, p->experts, &chunk, &blocks, &waves);
  return blocks > 1 ? align256((size_t)blocks * (size_t)(p->experts + 1) * sizeof(int32_t)) : 0;
}

mr_status order_by_expert(const mr_order_problem* p, void* ws, size_t ws_bytes, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("experts", p->experts, 1, kMaxExperts));
  MR_TRY(check_choices(p->tokens, p->k, kMaxChoices));
  if (p->index_bits != 32 && p->index_bits != 64) return fail(MR_ERR_PARAM, "index_bits %d: 32 or 64", p->index_bits);
  MR_TRY(check_array("offsets", p->offsets));
  const size_t is = (size_t)p->index_bits / 8;
  if (p->tokens > 0) {
    MR_TRY(check_matrix("chosen", p->chosen, p->k, p->ldc, is));
    MR_TRY(check_array("place", p->place));
  }
  const int64_t c = p->tokens * p->k;
  Aliases al;
  al.in("chosen", p->chosen, p->tokens, p->k, p->ldc, is);
  al.out("offsets", p->offsets, 1, p->experts + 1, p->experts + 1, 4);
  if (c) al.out("place", p->place, 1, c, c, 4);
  const size_t need = order_by_expert_workspace(p);
  MR_TRY(check_workspace(ws, ws_bytes, need));
  if (need) al.out("workspace", ws, 1, (int64_t)need, (int64_t)need, 1);
  MR_TRY(al.set.check());
  OrderArgs a;
  memset(&a, 0, sizeof a);
  a.experts = p->chosen, a.lde = p->ldc, a.wide = p->index_bits == 64;
  a.k = (int32_t)p->k, a.n = (int32_t)p->experts, a.total = (int32_t)c;
  order_plan(c, p->experts, &a.chunk, &a.blocks, &a.waves);
  a.offsets = p->offsets, a.place = p->place;
  a.counts = static_cast<int32_t*>(need ? ws : nullptr);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrOrder, true, s, [&] { return launch_order(a, s); }, "expert order launch");
}

// ------------------------------------------------------------------ rows
mr_status dispatch_rows(const mr_dispatch_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("experts", p->experts, 1, kMaxExperts));
  MR_TRY(check_size("width", p->width, 1, kMaxCols));
  MR_TRY(check_choices(p->tokens, p->k, kMaxChoices));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if ((p->Z != nullptr) != (p->dots != nullptr)) return fail(MR_ERR_NULL, "Z and dots: both or none");
  if (p->weights && !p->Z) return fail(MR_ERR_UNSUPPORTED, "weights without Z and dots");
  if (p->tokens == 0) return MR_OK;
  const size_t es = size_of(p->dtype);
  const int64_t c = p->tokens * p->k, w = p->width;
  MR_TRY(check_matrix("X", p->X, w, p->ldx, es));
  MR_TRY(check_matrix("Y", p->Y, w, p->ldy, es));
  MR_TRY(check_array("place", p->place));
  MR_TRY(check_array("offsets", p->offsets));
  if (p->weights) MR_TRY(check_array("weights", p->weights));
  if (p->Z) {
    MR_TRY(check_matrix("Z", p->Z, w, p->ldz, es));
    MR_TRY(check_array("dots", p->dots));
  }
  Aliases al;
  al.in("X", p->X, p->tokens, w, p->ldx, es);
  al.in("place", p->place, 1, c, c, 4);
  al.in("offsets", p->offsets, 1, p->experts + 1, p->experts + 1, 4);
  al.in("weights", p->weights, 1, c, c, 4);
  al.in("Z", p->Z, c, w, p->ldz, es);
  al.out("Y", p->Y, c, w, p->ldy, es);
  al.out("dots", p->dots, 1, c, c, 4);
  MR_TRY(al.set.check());
  RowsArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->X, a.ldx = p->ldx;
  a.rows = p->Z, a.ldr = p->ldz;
  a.out = p->Y, a.ldo = p->ldy;
  a.place = p->place, a.offsets = p->offsets, a.weights = p->weights, a.dots = p->dots;
  a.tokens = p->tokens, a.width = (int32_t)w, a.k = (int32_t)p->k, a.experts = (int32_t)p->experts;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrDispatch, true, s, [&] { return launch_dispatch(a, p->dtype, s); }, "dispatch launch");
}

mr_status combine_rows(const mr_combine_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("experts", p->experts, 1, kMaxExperts));
  MR_TRY(check_size("width", p->width, 1, kMaxCols));
  MR_TRY(check_choices(p->tokens, p->k, kMaxChoices));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if (p->tokens == 0) return MR_OK;
  const size_t es = size_of(p->dtype);
  const int64_t c = p->tokens * p->k, w = p->width;
  MR_TRY(check_matrix("Y", p->Y, w, p->ldy, es));
  MR_TRY(check_matrix("OUT", p->OUT, w, p->ldo, es));
  MR_TRY(check_array("place", p->place));
  MR_TRY(check_array("offsets", p->offsets));
  if (p->weights) MR_TRY(check_array("weights", p->weights));
  if (p->residual) MR_TRY(check_matrix("residual", p->residual, w, p->ldres, es));
  Aliases al;
  al.in("Y", p->Y, c, w, p->ldy, es);
  al.in("place", p->place, 1, c, c, 4);
  al.in("offsets", p->offsets, 1, p->experts + 1, p->experts + 1, 4);
  al.in("weights", p->weights, 1, c, c, 4);
  al.in("residual", p->residual, p->tokens, w, p->ldres, es);
  al.out("OUT", p->OUT, p->tokens, w, p->ldo, es);
  MR_TRY(al.set.check());
  RowsArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->residual, a.ldx = p->ldres;
  a.rows = p->Y, a.ldr = p->ldy;
  a.out = p->OUT, a.ldo = p->ldo;
  a.place = p->place, a.offsets = p->offsets, a.weights = p->weights;
  a.tokens = p->tokens, a.width = (int32_t)w, a.k = (int32_t)p->k, a.experts = (int32_t)p->experts;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrCombine, true, s, [&] { return launch_combine(a, p->dtype, s); }, "combine launch");
}

}  // extern "C"

// -------------------------------------------------------------- clipping
namespace {

constexpr int64_t kMaxValues = int64_t(1) << 40;  // of a gradient
constexpr int64_t kClipUnits = 2048;              // of 8 values: a workgroup's least share

bool clip_flat(const mr_clip_problem& p) { return p.m <= 1 || (p.ldg == p.n && (!p.OUT || p.ldo == p.n)); }

// Units of eight values, or what is left of a row.
int64_t clip_units(const mr_clip_problem& p) {
  return clip_flat(p) ? (p.m * p.n + 7) / 8 : p.m * ((p.n + 7) / 8);
}

// Units of 8 values for each workgroup of a call: all workgroups are resident at
// once (8 on each of 256 CUs, and one more for each gradient), and a few
// thousand partial sums are added up.
int64_t clip_per_block(const mr_clip_problem* p, int32_t count) {
  int64_t all = 0;
  for (int i = 0; i < count; ++i) all += clip_units(p[i]);
  const int64_t per = (all / 2048 + 1023) / 1024 * 1024;
  return per < kClipUnits ? kClipUnits : per;
}
int64_t clip_blocks(const mr_clip_problem& p, int64_t per) {
  const int64_t b = (clip_units(p) + per - 1) / per;
  return b < 1 ? 1 : b;  // an empty gradient has a sum too
}
bool clip_shape(const mr_clip_problem& p) {
  return p.m >= 0 && p.n >= 0 && p.m <= kMaxValues && p.n <= kMaxValues && (p.n == 0 || p.m <= kMaxValues / p.n);
}

// More partial sums than this are added up by a launch of their own, fewer by every workgroup of the scaling.
constexpr int64_t kClipSums = 4096;

// The call's launches of one kind of gradients, from its `slot`th workgroup on.
template <typename Jobs, typename Launch>
mr_status clip_batches(const mr_clip_problem* p, int32_t count, ClipBatch<Jobs>& b, int64_t& slot, Launch&& launch) {
  b.njobs = b.blocks = 0;
  b.slot = (int32_t)slot;
  auto flush = [&]() -> mr_status {
    if (b.njobs == 0) return MR_OK;
    MR_TRY(launch(b));
    slot += b.blocks;
    b.njobs = b.blocks = 0;
    b.slot = (int32_t)slot;
    return MR_OK;
  };
  for (int i = 0; i < count; ++i) {
    const mr_clip_problem& q = p[i];
    if (clip_flat(q) == Jobs::kRows) continue;
    const int j = b.njobs++;
    b.job.g[j] = q.G;
    b.job.out[j] = q.OUT ? q.OUT : q.G;
    b.job.type[j] = (uint8_t)(q.dtype | (q.OUT ? q.out_dtype : q.dtype) << 4);
    b.job.problem[j] = i;
    b.job.begin[j] = b.blocks;
    if constexpr (Jobs::kRows) {
      b.job.cols[j] = q.n, b.job.rows[j] = q.m;
      b.job.ldg[j] = q.ldg, b.job.ldo[j] = q.OUT ? q.ldo : q.ldg;
    } else {
      b.job.cols[j] = q.m * q.n;
    }
    b.blocks += (int32_t)clip_blocks(q, b.per);
    if (b.njobs == Jobs::kJobs) MR_TRY(flush());
  }
  return flush();
}

}  // namespace

extern "C" {

size_t clip_gradients_batched_workspace(const mr_clip_problem* p, int32_t count) {
  if (!p || count <= 0) return 0;
  for (int i = 0; i < count; ++i)
    if (!clip_shape(p[i])) return 0;
  const int64_t per = clip_per_block(p, count);
  int64_t slots = 0;
  for (int i = 0; i < count; ++i) slots += clip_blocks(p[i], per);
  return align256((size_t)(slots + 1) * sizeof(double));
}

mr_status clip_gradients_batched(const mr_clip_problem* p, int32_t count, double max_norm, double* norms_dev, void* ws,
                                 size_t ws_bytes, void* hip_stream) {
  if (count < 0) return fail(MR_ERR_PARAM, "count %d < 0", count);
  if (count > 0 && !p) return fail(MR_ERR_NULL, "problems is NULL");
  if (!(max_norm >= 0.0)) return fail(MR_ERR_PARAM, "max_norm %g must be >= 0", max_norm);
  if (!norms_dev) return fail(MR_ERR_NULL, "norms is NULL");
  if (!aligned(norms_dev, 8)) return fail(MR_ERR_PARAM, "norms is not aligned to its type");
  AliasSet al;
  for (int i = 0; i < count; ++i) {
    const mr_clip_problem& q = p[i];
    if (!clip_shape(q)) return fail(MR_ERR_SHAPE, "problem %d: m=%lld n=%lld", i, (long long)q.m, (long long)q.n);
    if (!is_float(q.dtype)) return fail(MR_ERR_PARAM, "problem %d: dtype %d", i, q.dtype);
    if (q.m == 0 || q.n == 0) continue;
    const size_t es = size_of(q.dtype);
    if (!q.G) return fail(MR_ERR_NULL, "problem %d: G is NULL", i);
    if (q.m > 1 && (q.ldg < q.n || q.ldg > kMaxValues / q.m))
      return fail(MR_ERR_STRIDE, "problem %d: leading dimension %lld", i, (long long)q.ldg);
    if (!aligned(q.G, es)) return fail(MR_ERR_PARAM, "problem %d: G is not aligned to its type", i);
    const Range g = range_of(q.G, q.m, q.n, q.m > 1 ? q.ldg : q.n, es);
    if (!q.OUT) {
      al.out(g, i, "G");
      continue;
    }
    if (q.out_dtype != q.dtype && q.out_dtype != MR_F32)
      return fail(MR_ERR_PARAM, "problem %d: output dtype %d: dtype or MR_F32", i, q.out_dtype);
    const size_t os = size_of(q.out_dtype);
    if (q.m > 1 && (q.ldo < q.n || q.ldo > kMaxValues / q.m))
      return fail(MR_ERR_STRIDE, "problem %d: output leading dimension %lld", i, (long long)q.ldo);
    if (!aligned(q.OUT, os)) return fail(MR_ERR_PARAM, "problem %d: OUT is not aligned to its type", i);
    al.in(g, i, "G");
    al.out(range_of(q.OUT, q.m, q.n, q.m > 1 ? q.ldo : q.n, os), i, "OUT");
  }
  al.out(range_of(norms_dev, 1, count + 1, count + 1, 8), count, "norms");
  const size_t need = clip_gradients_batched_workspace(p, count);
  MR_TRY(check_workspace(ws, ws_bytes, need));
  if (need) al.out(range_of(ws, 1, (int64_t)need, (int64_t)need, 1), count, "workspace");
  MR_TRY(al.check());
  const int64_t per = count > 0 ? clip_per_block(p, count) : 0;
  int64_t slots = 0;
  for (int i = 0; i < count; ++i) slots += clip_blocks(p[i], per);
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  double* partial = static_cast<double*>(ws);
  const bool fold = slots > kClipSums;
  auto over = [&](auto&& launch) -> mr_status {
    int64_t slot = 0;
    ClipBatch<ClipFlat> f;
    ClipBatch<ClipRows> r;
    memset(&f, 0, sizeof f);
    memset(&r, 0, sizeof r);
    f.partial = r.partial = partial;
    f.sums = r.sums = fold ? partial + slots : partial;
    f.nsums = r.nsums = fold ? 1 : (int32_t)slots;
    f.norms = r.norms = norms_dev;
    f.max_norm = r.max_norm = max_norm;
    f.per = r.per = per;
    MR_TRY(clip_batches(p, count, f, slot, launch));
    return clip_batches(p, count, r, slot, launch);
  };
  MR_TRY(over([&](const auto& b) {
    return traced(kTrClipNorm, true, s, [&] { return launch_clip_squares(b, s); }, "clip squares launch");
  }));
  if (fold || count == 0)
    MR_TRY(traced(kTrClipNorm, true, s,
                  [&] { return launch_clip_fold(partial, (int)slots, count ? partial + slots : norms_dev, s); },
                  "clip fold launch"));
  return over([&](const auto& b) {
    return traced(kTrClipScale, true, s, [&] { return launch_clip_scale(b, s); }, "clip scale launch");
  });
}

}  // extern "C"
