// The row quantiser behind the activation-side transform: K stages of disjoint-pair Givens rotations
// and the division by the channel scales in float32 (rotation_core.h), then 8-bit codes, in one
// kernel. The rotated row never leaves the chip and is not rounded to 16 bits in between.
//
// Built like the 16-bit transform (rotate.hip): a workgroup holds R rows in
// LDS as float32, interleaved by channel, streams the stages' records through a register ring, and
// walks blocks of R rows with the next block's rows on their way meanwhile. After the last stage the
// rows are read twice: once for each row's largest magnitude, once for its codes. The second read
// costs LDS the half of one stage and saves the registers that would hold the row in between.
// Measured (graph replays, cold rows), K = 8: 4096 x 4096 37.5 us (the 16-bit transform alone 35.0), 4096 x
// 1536 16.1 (19.1), 2048 x 8960 46.8 (45.6), 64 x 4096 6.2 (6.4), 1000 x 14336 39.6 (39.4), 16 x 1536 4.2 (4.3).
//
// What bounds it: the stages, 16 of the 19 passes over the row in LDS. No unit is full (4096 x 4096: LDS
// active 39 % of a CU's cycles and stalled by bank conflicts 10 %, VALU 43 %, HBM 10.6 us of 37.5), and the
// barriers are not it either (a timing copy of the 16-bit transform without them 34.6 us against 37.0). A
// copy of its stages with half the LDS traffic ran a four-row stage in 1300 cycles instead of 2000: carrying
// one channel of each pair in a register from stage to stage is what is left to build.
#include <algorithm>

#include "q8_device.h"
#include "rotation_core.h"

namespace paro {
namespace {

constexpr int kCUs = 256;

struct RotQ8Args {
  const uint16_t* x;
  const PairRec* rec;
  const float* inv_s;
  int8_t* q;
  float* scales;
  int M, K, D;
};

// The thread index, opaque at the point of use: addresses formed from it are not hoisted out of the
// block loop and kept live (or spilled) across the stages.
__device__ inline int fresh_tid() {
  int t = int(threadIdx.x);
  asm volatile("" : "+v"(t));
  return t;
}

__device__ inline float from_lane(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

template <int CTRL, int ROWS>
__device__ inline uint32_t dpp_max(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false)));
}
// The wave's maximum, in lane 63.
__device__ inline uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xF>(v);
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);
  return dpp_max<0x143, 0xC>(v);
}

template <int DT, int NT, int R, int PPT, int PD, bool EXACT>
__global__ __launch_bounds__(NT) void rotate_q8_kernel(const RotQ8Args a) {
  extern __shared__ __attribute__((aligned(16))) float lds[];  // [D][R], then the waves' maxima [NT / 64][R]
  const int D = a.D, K = a.K, M = a.M, P = D / 2;
  const int tid = threadIdx.x;
  using V = typename RowVec<R>::T;
  V* const rows = reinterpret_cast<V*>(lds);
  uint32_t* const tops = reinterpret_cast<uint32_t*>(lds + size_t(D) * R);
  const int nblk = (M + R - 1) / R;

  uint32_t hv[PPT][R];  // a block's rows on their way: two adjacent channels per lane and row
  auto load_rows = [&](int b) {
    const int tl = fresh_tid();
    uintptr_t xb = reinterpret_cast<uintptr_t>(a.x);
    asm volatile("" : "+s"(xb));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const gptr<const uint32_t> xr = (gptr<const uint32_t>)(xb + size_t(min(b * R + r, M - 1)) * D * sizeof(uint16_t));
#pragma unroll
      for (int u = 0; u < PPT; ++u) hv[u][r] = xr[min(tl + u * NT, P - 1)];
    }
  };
  auto fill = [&]() {
    const int tl = fresh_tid();
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      const int cp = tl + u * NT;  // channels 2 cp (low half) and 2 cp + 1
      if (cp < P) {
        float f0[R], f1[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          f0[r] = from_bits16<DT>(hv[u][r] & 0xFFFFu);
          f1[r] = from_bits16<DT>(hv[u][r] >> 16);
        }
        // lanes with bit 32/R set write their odd channel first: every aligned run of 16 (R = 4), 32
        // or 64 lanes then hits distinct bank slots in each of the two writes
        const bool sw = (tl & (32 / R)) != 0;
        const V v0 = make_vec<R>(f0), v1 = make_vec<R>(f1);
        rows[2 * cp + (sw ? 1 : 0)] = sw ? v1 : v0;
        rows[2 * cp + (sw ? 0 : 1)] = sw ? v0 : v1;
      }
    }
  };
  // the rotated row over the channel scales, channels 2j and 2j + 1 of all R rows (read in the order
  // that keeps each run of 32/R lanes on distinct bank slots, as above)
  auto scaled_pair = [&](int j, float sa, float sb, float (&va)[R], float (&vb)[R]) {
    const bool sw = (j & (32 / R)) != 0;
    const V w1 = rows[2 * j + (sw ? 1 : 0)], w2 = rows[2 * j + (sw ? 0 : 1)];
    const V wa = sw ? w2 : w1, wb = sw ? w1 : w2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      va[r] = vec_at<R>(wa, r) * sa;
      vb[r] = vec_at<R>(wb, r) * sb;
    }
  };

  int blk = blockIdx.x;
  load_rows(blk);
  StageRing<NT, PPT, PD, EXACT> ring;
  if (K > 0) ring_prime(ring, K, P, tid, a.rec);
  fill();
  __syncthreads();
  for (;;) {
    const int next = blk + int(gridDim.x);
    const bool more = next < nblk;  // uniform
    if (more) load_rows(next);
    if (K > 0) ring_run<R>(ring, lds, K, P, tid, a.rec);  // ends with a barrier

    const int to = fresh_tid();
    uintptr_t isb = reinterpret_cast<uintptr_t>(a.inv_s);
    asm volatile("" : "+s"(isb));
    using f32x2 = float __attribute__((ext_vector_type(2)));
    const gptr<const f32x2> isp = (gptr<const f32x2>)isb;
    // 1/s of the pairs: kept from one read of the rows to the next, or (the widest 4-row blocks, whose
    // registers are full) loaded for each
    constexpr bool kHoldS = !(R == 4 && PPT > 4);
    f32x2 held[kHoldS ? PPT : 1];
    if constexpr (kHoldS) {
#pragma unroll
      for (int u = 0; u < PPT; ++u) held[u] = isp[min(to + u * NT, P - 1)];
    }
    uint32_t top[R];
#pragma unroll
    for (int r = 0; r < R; ++r) top[r] = 0;
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      const int j = min(to + u * NT, P - 1);
      f32x2 is;
      if constexpr (kHoldS)
        is = held[u];
      else
        is = isp[j];
      float va[R], vb[R];
      scaled_pair(j, is.x, is.y, va, vb);
#pragma unroll
      for (int r = 0; r < R; ++r) top[r] = max(top[r], max(abs_order(va[r]), abs_order(vb[r])));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      top[r] = wave_max(top[r]);
      if ((to & 63) == 63) tops[(to >> 6) * R + r] = top[r];
    }
    __syncthreads();
    // Lane l works out row l % R's scale and step (their divisions once, not R times), which then are
    // the same in every lane: in scalar registers, of which there are plenty.
    RowQuant rq[R];
    {
      uint32_t t = 0;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) t = max(t, tops[w * R + (to & (R - 1))]);
      const RowQuant mine = row_quant(t);
#pragma unroll
      for (int r = 0; r < R; ++r)
        rq[r] = RowQuant{from_lane(mine.scale, r), from_lane(mine.step, r), from_lane(mine.low, r),
                         uint32_t(__builtin_amdgcn_readlane(int(t), r)) >= kAbsInf};
    }
    uint32_t ov[PPT][(R + 1) / 2];  // two codes a row, two rows a word
#pragma unroll
    for (int u = 0; u < PPT; ++u) {
      const int j = min(to + u * NT, P - 1);
      f32x2 is;
      if constexpr (kHoldS)
        is = held[u];
      else
        is = isp[j];
      float va[R], vb[R];
      scaled_pair(j, is.x, is.y, va, vb);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint32_t w = __builtin_amdgcn_perm(code_bits(vb[r], rq[r]), code_bits(va[r], rq[r]), 0x0c0c0400u);
        if (rq[r].bad) w = 0;
        if (r & 1)
          ov[u][r / 2] |= w << 16;
        else
          ov[u][r / 2] = w;
      }
    }
    __syncthreads();  // every read of this block's rows is done
    if (more) {
      if (K > 0) ring_prime(ring, K, P, tid, a.rec);
      fill();
    }
    {
      const int ts = fresh_tid();
      uintptr_t qb = reinterpret_cast<uintptr_t>(a.q);
      asm volatile("" : "+s"(qb));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (blk * R + r < M) {
          const gptr<uint16_t> qrow = (gptr<uint16_t>)(qb + size_t(blk * R + r) * D);
#pragma unroll
          for (int u = 0; u < PPT; ++u)
            if (ts + u * NT < P) qrow[ts + u * NT] = uint16_t(r & 1 ? ov[u][r / 2] >> 16 : ov[u][r / 2]);
          if (ts == 0) a.scales[blk * R + r] = rq[r].scale;
        }
      }
    }
    if (!more) break;
    __syncthreads();  // the next block's rows are in LDS
    blk = next;
  }
}

template <int DT, int NT, int R, int PPT, int PD, bool EXACT>
hipError_t launch(const RotQ8Args& a, hipStream_t st) {
  static_assert((R == 4 ? 9216 : PARO_MAX_D) * R * sizeof(float) + NT / 64 * R * sizeof(uint32_t) <= 160 * 1024, "one CU's LDS");
  const size_t lds = size_t(a.D) * R * sizeof(float) + NT / 64 * R * sizeof(uint32_t);
  const void* fn = reinterpret_cast<const void*>(&rotate_q8_kernel<DT, NT, R, PPT, PD, EXACT>);
  if (lds > 64 * 1024)
    if (hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, int(lds))) return e;
  // persistent workgroups, as many as the CUs hold at once
  int per_cu = 0;
  if (hipError_t e = hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, fn, NT, lds)) return e;
  const long blocks = (long(a.M) + R - 1) / R;
  const unsigned grid = unsigned(std::min<long>(blocks, long(std::max(per_cu, 1)) * kCUs));
  hipLaunchKernelGGL((rotate_q8_kernel<DT, NT, R, PPT, PD, EXACT>), dim3(grid), dim3(NT), lds, st, a);
  return hipGetLastError();
}

template <int DT, int NT, int R, int PPT, int PD>
hipError_t launch_exact(const RotQ8Args& a, hipStream_t st) {
  return a.D / 2 == PPT * NT ? launch<DT, NT, R, PPT, PD, true>(a, st) : launch<DT, NT, R, PPT, PD, false>(a, st);
}

// Threads, pairs per thread and stages of records in flight by row width: the smallest set that wastes few
// slots, since a stage takes as long as its fullest thread (K = 8: 4096 x 1536 20.4 us with 512 x 2 slots for
// its 768 pairs, 16.5 with 384 x 2; 2048 x 7168 41.5 with 512 x 7, 38.1 with 896 x 4). Two stages ahead, not
// four (4096 x 2048 23.1 -> 19.9 us); one where two would take the registers of the widest blocks (1000 x
// 14336 40.4 us, 55 with two). One and two rows have the registers for more threads with fewer pairs (256 x
// 4096 7.3 -> 7.0 us); four rows have not (4096 x 4096 39.9 -> 43.0).
template <int DT, int R>
hipError_t launch_ppt(const RotQ8Args& a, hipStream_t st) {
  const int P = a.D / 2;
  constexpr bool few = R < 4;
  if (P <= 256) return launch_exact<DT, 256, R, 1, 2>(a, st);
  if (P <= 384) return launch_exact<DT, 384, R, 1, 2>(a, st);
  if (P <= 512) return launch_exact<DT, few ? 512 : 256, R, few ? 1 : 2, 2>(a, st);
  if (P <= 384 * 2) return launch_exact<DT, 384, R, 2, 2>(a, st);
  if (P <= 512 * 2) return launch_exact<DT, 512, R, 2, 2>(a, st);
  if (P <= 512 * 3) return launch_exact<DT, 512, R, 3, 2>(a, st);
  if (P <= 1024 * 2) return launch_exact<DT, few ? 1024 : 512, R, few ? 2 : 4, 2>(a, st);
  if (P <= 1024 * 3) return launch_exact<DT, 1024, R, 3, 2>(a, st);
  if (P <= 896 * 4) return launch_exact<DT, 896, R, 4, 2>(a, st);
  if (P <= 1024 * 4) return launch_exact<DT, 1024, R, 4, few ? 2 : 1>(a, st);
  if (P <= 896 * 5) return launch_exact<DT, 896, R, 5, few ? 2 : 1>(a, st);
  if constexpr (!few) {
    return launch_exact<DT, 1024, R, 5, 1>(a, st);  // 4-row blocks go to 9216 channels
  } else {
    if (P <= 1024 * 5) return launch_exact<DT, 1024, R, 5, 2>(a, st);
    if (P <= 1024 * 6) return launch_exact<DT, 1024, R, 6, (R == 1 ? 2 : 1)>(a, st);
    if (P <= 1024 * 7) return launch_exact<DT, 1024, R, 7, 1>(a, st);
    return launch_exact<DT, 1024, R, 8, 1>(a, st);
  }
}

template <int DT>
hipError_t launch_rows(const RotQ8Args& a, hipStream_t st) {
  // rows per block: as few as give every CU one block; two rows of any width fit in LDS, four up to 9216 channels
  if (a.M <= kCUs) return launch_ppt<DT, 1>(a, st);
  if (a.M <= 2 * kCUs || a.D > 9216) return launch_ppt<DT, 2>(a, st);
  return launch_ppt<DT, 4>(a, st);
}

}  // namespace

hipError_t launch_rotate_q8(const DevRot& R, int M, int dtype, const void* x, int8_t* q, float* scales,
                            hipStream_t st) {
  const RotQ8Args a{static_cast<const uint16_t*>(x), R.rec, R.inv_s, q, scales, M, R.K, R.D};
  return dtype == PARO_F16 ? launch_rows<PARO_F16>(a, st) : launch_rows<PARO_BF16>(a, st);
}

}  // namespace paro
