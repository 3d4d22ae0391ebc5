// The experts' products of a mixture-of-experts layer for a few tokens, on INT4 weights: gate and up with their
// activation, then down with the sum over a token's experts.
#include <algorithm>

#include "moe_internal.h"
#include "w4_device.h"

namespace paro {
namespace {

constexpr int kMaxM = PARO_MOE_MAX_M;
constexpr int kFrags = kMaxM / 16;  // 16-row fragments of an expert's tokens

__device__ inline _Float16 as_half(uint16_t v) { return __builtin_bit_cast(_Float16, v); }

// 16 weight rows times 128 channels: a lane's 16 bytes (row lane & 15, channels 32 (lane >> 4) on) with the row's scale and
// zero, against the fragments of 16 rows in a: acc[f][row of a][row of w] += products.
__device__ inline void group_product(const uint4& w, uint16_t scale, uint16_t zero, const h8 (&a)[kFrags][4], int frags, f4 (&acc)[kFrags]) {
  const _Float16 z = as_half(zero);
  const _Float16 zl = -(static_cast<_Float16>(1024.0f) + z), zh = -(static_cast<_Float16>(64.0f) + z);
  const h2 zlo = {zl, zl}, zhi = {zh, zh};
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
  h8 b[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = dequant_word(wv[k], zlo, zhi, 0x000F000Fu, 0x00F000F0u, 0x64006400u);
  const float s = static_cast<float>(as_half(scale));
#pragma unroll
  for (int f = 0; f < kFrags; ++f)
    if (f < frags) {  // uniform
      f4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) g = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[f][k], b[k], g, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][i] = __builtin_fmaf(s, g[i], acc[f][i]);
    }
}

// A lane's part of a row's 128 channels, from its first one on.
__device__ inline void load_rows(const uint16_t* p, h8 (&a)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) a[k] = decode_order(*reinterpret_cast<const h8*>(p + k * 8));
}

// A workgroup has 16 gate and 16 up rows of one expert; its waves take the groups of channels in turn.
__global__ __launch_bounds__(256) void gate_up_kernel(const MoeCall c) {
  __shared__ f4 red[4][2][kFrags][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nl = lane & 15, h = lane >> 4;
  if (int(blockIdx.y) >= *c.t.active_count) return;
  const MoeActive ex = c.t.active[blockIdx.y];
  const int G = c.D / PARO_GROUP, frags = (ex.count + 15) / 16;
  const uint16_t* xp[kFrags];
#pragma unroll
  for (int f = 0; f < kFrags; ++f) xp[f] = c.x + size_t(c.t.slot_token[ex.first + min(f * 16 + nl, ex.count - 1)]) * c.D + h * 32;
  const size_t row = size_t(ex.expert) * 2 * c.F + blockIdx.x * 16 + nl;  // this lane's gate row; its up row is F further on
  const uint8_t* const wp = c.gu_qw + qw_row_offset<size_t>(row, c.D) + h * 16;
  const size_t up = size_t(c.F) * (c.D / 2), ups = size_t(c.F) * G;
  f4 acc[2][kFrags] = {};
  for (int g = wave; g < G; g += 4) {
    h8 a[kFrags][4];
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
      if (f < frags) load_rows(xp[f] + g * PARO_GROUP, a[f]);
    const size_t si = row * G + g;
    group_product(*reinterpret_cast<const uint4*>(wp + size_t(g) * 1024), c.gu_sc[si], c.gu_zr[si], a, frags, acc[0]);
    group_product(*reinterpret_cast<const uint4*>(wp + up + size_t(g) * 1024), c.gu_sc[si + ups], c.gu_zr[si + ups], a, frags, acc[1]);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
      if (f < frags) red[wave][j][f][lane] = acc[j][f];
  __syncthreads();
  for (int o = tid; o < ex.count * 16; o += 256) {
    const int m = o >> 4, n = o & 15, f = m >> 4, l = ((m & 15) >> 2) * 16 + n, i = m & 3;
    float gate = 0, upv = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      gate += red[w][0][f][l][i];
      upv += red[w][1][f][l][i];
    }
    const float v = gate / (1.0f + expf(-gate)) * upv;
    c.a[size_t(ex.first + m) * c.F + blockIdx.x * 16 + n] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  }
}

// A workgroup has 16 columns of y. Its waves share out the (expert, group) pairs, in order, each with sums of its own
// for every token.
__global__ __launch_bounds__(512) void down_kernel(const MoeCall c) {
  __shared__ float sums[8][kMaxM][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nl = lane & 15, h = lane >> 4;
  for (int i = lane; i < kMaxM * 16; i += 64) sums[wave][i / 16][i % 16] = 0;
  const int G = c.F / PARO_GROUP, total = *c.t.active_count * G;
  const int begin = int(size_t(total) * wave / 8), end = int(size_t(total) * (wave + 1) / 8);
  int at = begin / G, g = begin % G;
  for (int item = begin; item < end; ++at, g = 0) {
    const MoeActive ex = c.t.active[at];
    const int stop = min(G, g + end - item), frags = (ex.count + 15) / 16;
    const uint16_t* ap[kFrags];
#pragma unroll
    for (int f = 0; f < kFrags; ++f) ap[f] = c.a_down + size_t(ex.first + min(f * 16 + nl, ex.count - 1)) * c.F + h * 32;
    const size_t row = size_t(ex.expert) * c.D + blockIdx.x * 16 + nl;
    const uint8_t* const wp = c.dn_qw + qw_row_offset<size_t>(row, c.F) + h * 16;
    f4 acc[kFrags] = {};
    item += stop - g;
    for (; g < stop; ++g) {
      h8 a[kFrags][4];
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        if (f < frags) load_rows(ap[f] + g * PARO_GROUP, a[f]);
      group_product(*reinterpret_cast<const uint4*>(wp + size_t(g) * 1024), c.dn_sc[row * G + g], c.dn_zr[row * G + g], a, frags, acc);
    }
#pragma unroll
    for (int f = 0; f < kFrags; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = f * 16 + 4 * h + i;
        if (r < ex.count) {
          // (an expert has a token once: no two lanes meet)
          float& s = sums[wave][c.t.slot_token[ex.first + r]][nl];
          s = __builtin_fmaf(c.t.slot_weight[ex.first + r], acc[f][i], s);
        }
      }
  }
  __syncthreads();
  for (int o = tid; o < c.M * 16; o += 512) {
    const int m = o >> 4, n = o & 15;
    float v = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[w][m][n];
    const size_t i = size_t(m) * c.D + blockIdx.x * 16 + n;
    if (c.ydtype == PARO_F32)
      static_cast<float*>(c.y)[i] = v;
    else
      static_cast<_Float16*>(c.y)[i] = static_cast<_Float16>(v);
  }
}

}  // namespace

hipError_t launch_moe_gate_up(const MoeCall& c, hipStream_t st) {
  const dim3 grid(unsigned(c.F / 16), unsigned(std::min(c.E, c.M * c.top_k)));
  hipLaunchKernelGGL(gate_up_kernel, grid, dim3(256), 0, st, c);
  return hipGetLastError();
}

hipError_t launch_moe_down(const MoeCall& c, hipStream_t st) {
  hipLaunchKernelGGL(down_kernel, dim3(unsigned(c.D / 16)), dim3(512), 0, st, c);
  return hipGetLastError();
}

}  // namespace paro
