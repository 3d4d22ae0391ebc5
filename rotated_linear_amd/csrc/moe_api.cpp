// Host side of the mixture-of-experts calls (include/paro_block.h): argument checks, workspace and launches. Every
// error path returns before anything is enqueued on the stream.
#include "host_checks.h"
#include "moe_internal.h"

using namespace paro;

namespace {

bool good_sizes(int M, int E, int top_k, bool routed) {
  return M >= 0 && M <= PARO_MOE_MAX_M && E >= 1 && E <= PARO_MOE_MAX_E && top_k >= 1 && top_k <= PARO_MOE_MAX_K &&
         (!routed || top_k <= E);
}

// A workspace's sections, each at a multiple of 256 bytes.
struct Layout {
  size_t logits, x, a, a_rotated, part, units, unit, slot, power, total;
};
Layout layout(int M, int D, int F, int E, int top_k) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  const size_t pairs = size_t(M) * top_k;
  l.logits = take(size_t(M) * E * 8);
  l.x = take(size_t(M) * D * 4);
  l.a = take(pairs * F * 4);  // two float16 parts, or float32 where a transform follows
  l.a_rotated = take(pairs * F * 4);
  const int splits = moe_down_plan(M, D, F, E, top_k).splits;
  l.part = take(splits > 1 ? size_t(splits) * M * D * 4 : 0);
  l.units = take(4);
  l.unit = take(size_t(moe_units_max(M, E, top_k)) * sizeof(MoeUnit));
  l.slot = take(pairs * sizeof(MoeSlot));
  l.power = take(size_t(M) * 4);
  l.total = at;
  return l;
}

struct Router {
  const void* router;
  int dtype, scoring, renormalize;
};

paro_status check_router(const Router& r) {
  if (r.dtype != PARO_F16 && r.dtype != PARO_F32) return PARO_EINVAL;
  if (r.scoring != PARO_MOE_SOFTMAX && r.scoring != PARO_MOE_SIGMOID) return PARO_EINVAL;
  return PARO_OK;
}

size_t router_bytes(const Router& r, int D, int E) { return size_t(E) * D * (r.dtype == PARO_F32 ? 4 : 2); }

// r: the layer's router, or nullptr where ids and weights are given.
paro_status experts(int M, int D, int F, int E, int top_k, const void* x, const Router* r, int32_t* ids, float* weights,
                    const paro_rotation* rot_x, const paro_rotation* rot_a, const paro_w4_experts* gate_up,
                    const paro_w4_experts* down, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream) {
  if (!good_sizes(M, E, top_k, r != nullptr) || (ydtype != PARO_F16 && ydtype != PARO_F32)) return PARO_EINVAL;
  if (r)
    if (paro_status e = check_router(*r)) return e;
  if (!good_D(D) || !good_D(F)) return PARO_ESHAPE;
  DevRot rx, ra;
  Span dx, da;
  if (paro_status e = check_rot(rot_x, D, &rx, &dx)) return e;
  if (paro_status e = check_rot(rot_a, F, &ra, &da)) return e;
  if (M == 0) return PARO_OK;
  if (!gate_up || !down) return PARO_EINVAL;
  for (const void* p : {x, static_cast<const void*>(ids), static_cast<const void*>(weights), static_cast<const void*>(y),
                        static_cast<const void*>(gate_up->qweight), gate_up->scales, gate_up->zeros,
                        static_cast<const void*>(down->qweight), down->scales, down->zeros})
    if (!good_ptr(p)) return PARO_EINVAL;
  if (r && !good_ptr(r->router)) return PARO_EINVAL;
  const Layout l = layout(M, D, F, E, top_k);
  if (!ws || ws_bytes < l.total) return PARO_EWORKSPACE;
  if (!aligned16(ws)) return PARO_EINVAL;
  const size_t gu = size_t(E) * 2 * F * D, dn = size_t(E) * F * D, pairs = size_t(M) * top_k * 4;
  const Span out_y{y, size_t(M) * D * (ydtype == PARO_F32 ? 4 : 2)}, out_ws{ws, l.total};
  const Span ins[] = {{x, size_t(M) * D * 2}, dx, da, {gate_up->qweight, gu / 2}, {gate_up->scales, gu / PARO_GROUP * 2},
                      {gate_up->zeros, gu / PARO_GROUP * 2}, {down->qweight, dn / 2}, {down->scales, dn / PARO_GROUP * 2},
                      {down->zeros, dn / PARO_GROUP * 2}, {r ? r->router : nullptr, r ? router_bytes(*r, D, E) : 0},
                      {r ? nullptr : ids, pairs}, {r ? nullptr : weights, pairs}};
  const Span outs[] = {out_y, out_ws, {r ? ids : nullptr, pairs}, {r ? weights : nullptr, pairs}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;

  char* const base = static_cast<char*>(ws);
  MoeCall c{};
  c.M = M;
  c.D = D;
  c.F = F;
  c.E = E;
  c.top_k = top_k;
  c.x = static_cast<const uint16_t*>(x);
  c.gu_qw = gate_up->qweight;
  c.gu_sc = static_cast<const uint16_t*>(gate_up->scales);
  c.gu_zr = static_cast<const uint16_t*>(gate_up->zeros);
  c.dn_qw = down->qweight;
  c.dn_sc = static_cast<const uint16_t*>(down->scales);
  c.dn_zr = static_cast<const uint16_t*>(down->zeros);
  c.a = base + l.a;
  c.a_down = reinterpret_cast<const uint16_t*>(c.a);
  c.a_fragments = rot_a == nullptr;
  c.part = reinterpret_cast<float*>(base + l.part);
  c.t = MoeTables{reinterpret_cast<int*>(base + l.units), reinterpret_cast<MoeUnit*>(base + l.unit), reinterpret_cast<MoeSlot*>(base + l.slot)};
  int* const power = reinterpret_cast<int*>(base + l.power);
  c.power = power;
  c.y = y;
  c.ydtype = ydtype;
  const hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (r) {
    const MoeRoute route{M, D, E, top_k, c.x, r->router, r->dtype == PARO_F32, r->scoring == PARO_MOE_SIGMOID, r->renormalize != 0,
                         reinterpret_cast<double*>(base + l.logits), ids, weights, power};
    e = launch_moe_logits(route, st);
    if (e == hipSuccess) e = launch_moe_select(route, &c.t, st);
  } else {
    e = launch_moe_group(M, D, E, top_k, c.x, ids, weights, c.t, power, st);
  }
  if (e == hipSuccess && rot_x) {
    uint16_t* const xr = reinterpret_cast<uint16_t*>(base + l.x);
    e = launch_rotate_parts(rx, M, c.x, xr, RowPower{power, 1, 0, 1}, st);
    c.x = xr;
    c.x_parts = true;
  }
  if (e == hipSuccess) e = launch_moe_gate_up(c, st);
  if (e == hipSuccess && rot_a) {
    // (every row there may be: those of pairs without an expert hold what they held, and no product reads them)
    uint16_t* const ar = reinterpret_cast<uint16_t*>(base + l.a_rotated);
    e = launch_rotate_f32_parts(ra, M * top_k, static_cast<const float*>(c.a), ar, RowPower{power, top_k, kLiftA, 2}, st);
    c.a_down = ar;
  }
  if (e == hipSuccess) e = launch_moe_down(c, st);
  return from_hip(e);
}

}  // namespace

extern "C" {

size_t paro_moe_route_workspace_bytes(int M, int E) {
  return M > 0 && good_sizes(M, E, 1, true) ? align256(size_t(M) * E * 8) : 0;
}

paro_status paro_moe_route(int M, int D, int E, int top_k, const void* x, const void* router, int router_dtype, int scoring,
                           int renormalize, int32_t* ids, float* weights, void* ws, size_t ws_bytes, void* stream) {
  const Router r{router, router_dtype, scoring, renormalize};
  if (!good_sizes(M, E, top_k, true)) return PARO_EINVAL;
  if (paro_status e = check_router(r)) return e;
  if (!good_D(D)) return PARO_ESHAPE;
  if (M == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(router) || !good_ptr(ids) || !good_ptr(weights)) return PARO_EINVAL;
  const size_t need = paro_moe_route_workspace_bytes(M, E), pairs = size_t(M) * top_k * 4;
  if (!ws || ws_bytes < need) return PARO_EWORKSPACE;
  if (!aligned16(ws)) return PARO_EINVAL;
  const Span outs[] = {{ids, pairs}, {weights, pairs}, {ws, need}};
  const Span ins[] = {{x, size_t(M) * D * 2}, {router, router_bytes(r, D, E)}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  const MoeRoute route{M, D, E, top_k, static_cast<const uint16_t*>(x), router, router_dtype == PARO_F32, scoring == PARO_MOE_SIGMOID,
                       renormalize != 0, static_cast<double*>(ws), ids, weights, nullptr};
  const hipStream_t st = as_stream(stream);
  hipError_t e = launch_moe_logits(route, st);
  if (e == hipSuccess) e = launch_moe_select(route, nullptr, st);
  return from_hip(e);
}

size_t paro_moe_workspace_bytes(int M, int D, int F, int E, int top_k) {
  return M > 0 && good_sizes(M, E, top_k, false) && good_D(D) && good_D(F) ? layout(M, D, F, E, top_k).total : 0;
}

paro_status paro_moe_w4a16(int M, int D, int F, int E, int top_k, const void* x, const int32_t* ids, const float* weights,
                           const paro_rotation* rot_x, const paro_rotation* rot_a, const paro_w4_experts* gate_up,
                           const paro_w4_experts* down, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream) {
  return experts(M, D, F, E, top_k, x, nullptr, const_cast<int32_t*>(ids), const_cast<float*>(weights), rot_x, rot_a, gate_up, down, y,
                 ydtype, ws, ws_bytes, stream);
}

paro_status paro_moe_layer_w4a16(int M, int D, int F, int E, int top_k, const void* x, const void* router, int router_dtype,
                                 int scoring, int renormalize, const paro_rotation* rot_x, const paro_rotation* rot_a,
                                 const paro_w4_experts* gate_up, const paro_w4_experts* down, void* y, int ydtype, int32_t* ids,
                                 float* weights, void* ws, size_t ws_bytes, void* stream) {
  const Router r{router, router_dtype, scoring, renormalize};
  return experts(M, D, F, E, top_k, x, &r, ids, weights, rot_x, rot_a, gate_up, down, y, ydtype, ws, ws_bytes, stream);
}

void paro_internal_moe_gate_up_plan(int M, int D, int F, int E, int top_k, int parts, int* waves, int* groups, int* once) {
  const MoeGateUpPlan p = moe_gate_up_plan(M, D, F, E, top_k, parts);
  *waves = p.waves;
  *groups = p.groups;
  *once = p.once;
}

void paro_internal_moe_down_plan(int M, int D, int F, int E, int top_k, int* tiles, int* splits) {
  const MoeDownPlan p = moe_down_plan(M, D, F, E, top_k);
  *tiles = p.tiles;
  *splits = p.splits;
}

void paro_internal_moe_down_kernel(int M, int D, int F, int E, int top_k, int* tiles, int* few, int* once) {
  const MoeDownPlan p = moe_down_plan(M, D, F, E, top_k);
  *tiles = p.tiles;
  *few = p.few;
  *once = p.once;
}

}  // extern "C"
