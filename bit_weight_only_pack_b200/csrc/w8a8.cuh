// W8A8: INT8 weights with one FP32 scale per output channel times INT8
// activations with one FP32 scale per token, dense or routed to experts:
//   Y[m][n] = sx[m] sw[n] sum_k xq[m][k] wq[n][k]
// The sum is exact in int32 (at most 2^14 per product, K <= 65536), so the
// result does not depend on tiling or order; the two scales are applied in
// FP32 and the product is rounded once to the output type.
//
//  * Activations: quantize_int8_rows_kernel, one scale per row.
//  * Product: w8a8_gemm_kernel on tcgen05.mma.kind::i8 (s8 x s8 -> s32), with
//    the operands swapped (Y^T = W X^T): the channels are the MMA's M (TMEM
//    lanes) and the tokens its N, so a few tokens cost a narrow MMA instead of
//    a padded one and the weights, the large operand of a decode step, are
//    streamed once whatever the batch.
#pragma once

#include "common.cuh"
#include "tma.cuh"
#include "gemm_tc.cuh"
#include "stream_k.cuh"
#include "w4a8.cuh"

namespace lbq {

// ---------------------------------------------------------------------------- activations

// One block per row of X, the row in registers (VPT chunks of 8 per thread):
// s = amax / 127 in IEEE FP32 and xq = clamp(rint(x / s), -127, 127), 0 where
// s = 0. The maximum is taken over the bit patterns of |x| as integers, which
// order like the values with infinity and NaN above every finite one, so a row
// with a NaN or infinity gets that scale and codes 0: its products are NaN
// instead of passing for finite. The quotient is the one of
// quantize_int8_kernel: the product with RN(1/s) wherever it is at least 2^-14
// away from a half-integer, the IEEE quotient elsewhere; same codes as the
// division everywhere.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(1024) quantize_int8_rows_kernel(const uint16_t* __restrict__ X, int K,
                                                                  int8_t* __restrict__ xq, float* __restrict__ sx) {
  __shared__ uint32_t warp_max[32];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int tid = threadIdx.x, chunks = K >> 3;
  const size_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(X + row * (size_t)K);
  uint4 v[VPT];
  uint32_t m2 = 0u;  // running maxima of the two halves' magnitude bits
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * blockDim.x;
    v[i] = c < chunks ? ld_nc_v4(xr + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    m2 = __vmaxu2(m2, v[i].x & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, v[i].y & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, v[i].z & 0x7FFF7FFFu);
    m2 = __vmaxu2(m2, v[i].w & 0x7FFF7FFFu);
  }
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (blockDim.x > 32) {
    if ((tid & 31) == 0) warp_max[tid >> 5] = m;
    __syncthreads();
    const uint32_t w = (tid & 31) < (int)(blockDim.x >> 5) ? warp_max[tid & 31] : 0u;
    m = __reduce_max_sync(0xFFFFFFFFu, w);
  }
  const float s = __fdiv_rn(x2f<BF16>((uint16_t)m), 127.0f);
  const float inv = __fdiv_rn(1.0f, s);
  const bool use_inv = inv <= 3.4028234663852886e38f;
  const bool zero = !(s > 0.0f && s <= 3.4028234663852886e38f);  // all-zero rows; rows with inf or NaN
  auto code = [&](uint32_t bits) -> uint32_t {
    const float x = x2f<BF16>((uint16_t)bits);
    const float t = __fmul_rn(x, inv);
    float r = rintf(t);
    if (!use_inv || 0.5f - fabsf(t - r) < 6.103515625e-05f) r = rintf(__fdiv_rn(x, s));
    r = fminf(fmaxf(r, -127.0f), 127.0f);
    return zero ? 0u : (uint32_t)(int)r & 0xFFu;
  };
  uint2* out = reinterpret_cast<uint2*>(xq + row * (size_t)K);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * blockDim.x;
    if (c < chunks) {
      const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t o[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        o[h] = code(u[2 * h] & 0xFFFFu) | (code(u[2 * h] >> 16) << 8) | (code(u[2 * h + 1] & 0xFFFFu) << 16) |
               (code(u[2 * h + 1] >> 16) << 24);
      out[c] = make_uint2(o[0], o[1]);
    }
  }
  if (tid == 0) sx[row] = s;
}

// ---------------------------------------------------------------------------- weights (offline)

// FP32 weight [K][N] -> codes [N][K] and a scale per channel, by the same rule.
// Block = 32 channels x 8 k rows; pass 1 the channels' maxima, pass 2 the codes,
// turned through a 32 x 32 tile so that both sides are read and written in rows.
__global__ void __launch_bounds__(256) quantize_int8_weight_kernel(const float* __restrict__ W, int K, int N,
                                                                   int8_t* __restrict__ wq, float* __restrict__ sw) {
  __shared__ float red[8][32];
  __shared__ int8_t tile[32][33];
  const int cx = threadIdx.x & 31, ky = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + cx;
  float amax = 0.0f;
  bool nan = false;
  if (n < N)
    for (int k = ky; k < K; k += 8) {
      const float a = fabsf(W[(size_t)k * N + n]);
      nan |= a != a;
      amax = fmaxf(amax, a);
    }
  red[ky][cx] = nan ? __int_as_float(0x7FC00000) : amax;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = red[i][cx];
    s = (a != a || s != s) ? __int_as_float(0x7FC00000) : fmaxf(s, a);
  }
  s = __fdiv_rn(s, 127.0f);
  const bool ok = s > 0.0f && s <= 3.4028234663852886e38f;
  if (ky == 0 && n < N) sw[n] = s;
  for (int k0 = 0; k0 < K; k0 += 32) {
    __syncthreads();
    for (int i = ky; i < 32; i += 8) {
      const int k = k0 + i;
      float r = 0.0f;
      if (n < N && k < K && ok) r = fminf(fmaxf(rintf(__fdiv_rn(W[(size_t)k * N + n], s)), -127.0f), 127.0f);
      tile[i][cx] = (int8_t)(int)r;
    }
    __syncthreads();
    for (int i = ky; i < 32; i += 8) {
      const int nn = blockIdx.x * 32 + i, k = k0 + cx;
      if (nn < N && k < K) wq[(size_t)nn * K + k] = tile[cx][i];
    }
  }
}

// ---------------------------------------------------------------------------- product

constexpr int kW8BK = 128;        // k per ring stage: one 128-byte swizzle span, four MMAs of K = 32
constexpr int kW8MaxHt = 128;     // channels per tile (MMA M, TMEM lanes)
constexpr int kW8MaxBn = 256;     // tokens per tile (MMA N)
constexpr int kW8MaxStages = 16;
constexpr int kW8Threads = 192;   // TMA producer, MMA issuer, four epilogue warps
constexpr int kW8MaxExperts = 2048;
constexpr int kW8MaxK = 65536;        // 2^16 products of at most 2^14: the sum stays in int32
constexpr int kW8SmemBudget = 226 * 1024;  // dynamic; the static barriers take the rest of 227 KB

struct W8a8Args {
  void* Y;                  // [M][N]
  const float* sx;          // [M]
  const float* sw;          // [E][N]
  const int32_t* offsets;   // [E + 1] first row of each expert's run, or null (dense)
  int M, N, E;
  int ht, n_tiles;          // channels per tile, tiles along N
  int bn, m_tiles;          // tokens per tile; tiles along M (dense)
  int bx;                   // token rows per TMA box (bn is a multiple)
  int k_blocks, stages, a_bytes, stage_bytes;
  int acc_stride, tmem_cols;
  int y_bf16;
};

// Instruction descriptor of kind::i8: D = S32 (2), A = B = S8 (1), both
// K-major, M = 128, N = n.
__host__ __device__ constexpr uint32_t umma_idesc_i8(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\t"
               "setp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
}

// One output tile: channels n0 .. n0 + nh - 1 (of expert e), rows m0 .. m0 + mh - 1.
struct W8Tile {
  int n0, nh, m0, mh, e;
};

// Tile `t` of the call. Dense: bands of token tiles (stream_k.cuh). Routed:
// start[e] = token tiles of the experts before e (shared memory), channels
// inner, so an expert's tiles are neighbours.
__device__ __forceinline__ W8Tile w8_tile(const W8a8Args& a, const int* start, int t) {
  W8Tile w;
  int nt, mt;
  if (a.offsets == nullptr) {
    sk_tile_coords(t, a.n_tiles, a.m_tiles, nt, mt);
    w.e = 0;
    w.m0 = mt * a.bn;
    w.mh = min(a.bn, a.M - w.m0);
  } else {
    mt = t / a.n_tiles;
    nt = t - mt * a.n_tiles;
    int lo = 0, hi = a.E;  // the last e with start[e] <= mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= mt) lo = mid;
      else hi = mid;
    }
    w.e = lo;
    const int first = min(max(__ldg(a.offsets + lo), 0), a.M), end = min(max(__ldg(a.offsets + lo + 1), 0), a.M);
    w.m0 = first + (mt - start[lo]) * a.bn;
    w.mh = min(a.bn, end - w.m0);
  }
  w.n0 = nt * a.ht;
  w.nh = min(a.ht, a.N - w.n0);
  return w;
}

// start[0 .. E] of the routed form, by the whole block (contiguous ranges of
// experts per thread, a warp scan, then the warps' totals).
__device__ __forceinline__ void w8_expert_tiles(const W8a8Args& a, int* start) {
  __shared__ int warp_sum[kW8Threads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.E + kW8Threads - 1) / kW8Threads, e0 = min(a.E, tid * per), e1 = min(a.E, e0 + per);
  auto tiles_of = [&](int e) {
    const int first = min(max(__ldg(a.offsets + e), 0), a.M), end = min(max(__ldg(a.offsets + e + 1), 0), a.M);
    return end > first ? (end - first + a.bn - 1) / a.bn : 0;
  };
  int mine = 0;
  for (int e = e0; e < e1; ++e) mine += tiles_of(e);
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int o = incl - mine;
  for (int w = 0; w < warp; ++w) o += warp_sum[w];
  for (int e = e0; e < e1; ++e) {
    start[e] = o;
    o += tiles_of(e);
  }
  if (tid == kW8Threads - 1) start[a.E] = o;
  __syncthreads();
}

// Warp 0: TMA producer (per k-block the tile's weight rows and token rows, both
// 128-byte swizzled); warp 1: TMEM owner and MMA issuer; warps 2..5: epilogue,
// one TMEM lane quarter each (lane = channel), into Y with 64-byte row segments
// per warp. Two accumulators alternate, so the MMAs of a tile run while the last
// one is written. Persistent: one block per SM takes every gridDim.x-th tile and
// the ring runs on across tiles.
//
// A tile of fewer than 128 channels loads only its own rows; the MMA's other
// rows read whatever follows in shared memory (integers, so no NaN can arise)
// and their lanes are not stored. The ring ends with that much slack.
__global__ void __launch_bounds__(kW8Threads, 1)
    w8a8_gemm_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                     const W8a8Args a) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kW8MaxStages], empty_bar[kW8MaxStages], d_full[2], d_empty[2];
  __shared__ uint32_t tmem_base_sh;
  uint8_t* ring = dsmem + ((1024u - (smem_u32(dsmem) & 1023u)) & 1023u);
  int* start = reinterpret_cast<int*>(ring + (size_t)a.stages * a.stage_bytes + kW8MaxHt * kW8BK);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  w8_griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 4);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&tmem_base_sh)), "r"((uint32_t)a.tmem_cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tw);
    tma_prefetch_desc(&tx);
  }
  if (a.offsets != nullptr) {
    w8_griddep_wait();  // the offsets come from a kernel before
    w8_expert_tiles(a, start);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int total = (a.offsets == nullptr ? a.m_tiles : start[a.E]) * a.n_tiles;

  if (warp == 0) {
    if (lane == 0) {
      // the weights of the first stages are requested before the kernel that
      // writes the activations has ended
      int pre = 0;
      for (int tile = blockIdx.x; tile < total && pre < a.stages; tile += gridDim.x) {
        const W8Tile w = w8_tile(a, start, tile);
        const int boxes = (w.mh + a.bx - 1) / a.bx;
        for (int kb = 0; kb < a.k_blocks && pre < a.stages; ++kb, ++pre) {
          mbar_arrive_expect_tx(&full_bar[pre], (uint32_t)((a.ht + boxes * a.bx) * kW8BK));
          tma_load_2d(ring + (size_t)pre * a.stage_bytes, &tw, kb * kW8BK, w.e * a.N + w.n0, &full_bar[pre]);
        }
      }
      w8_griddep_wait();
      int it = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const W8Tile w = w8_tile(a, start, tile);
        const int boxes = (w.mh + a.bx - 1) / a.bx;
        for (int kb = 0; kb < a.k_blocks; ++kb, ++it) {
          const int s = it % a.stages;
          uint8_t* st = ring + (size_t)s * a.stage_bytes;
          if (it >= pre) {
            if (!mbar_wait_sleep(&empty_bar[s], ((it / a.stages) & 1) ^ 1)) { ok = false; break; }
            mbar_arrive_expect_tx(&full_bar[s], (uint32_t)((a.ht + boxes * a.bx) * kW8BK));
            tma_load_2d(st, &tw, kb * kW8BK, w.e * a.N + w.n0, &full_bar[s]);
          }
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(st + a.a_bytes + b * a.bx * kW8BK, &tx, kb * kW8BK, w.m0 + b * a.bx, &full_bar[s]);
        }
      }
      // every copy this block issued lands before it may exit
      for (int v = max(0, it - a.stages); v < it; ++v)
        if (!mbar_wait_sleep(&full_bar[v % a.stages], (v / a.stages) & 1)) break;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int it = 0, t_iter = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x, ++t_iter) {
        const W8Tile w = w8_tile(a, start, tile);
        const uint32_t idesc = umma_idesc_i8((w.mh + 15) & ~15);
        const int ai = t_iter & 1;
        const uint32_t d = tmem + (uint32_t)(ai * a.acc_stride);
        if (t_iter >= 2 && !mbar_wait_sleep(&d_empty[ai], ((t_iter >> 1) & 1) ^ 1)) break;
        tc_fence_after();
        for (int kb = 0; kb < a.k_blocks; ++kb, ++it) {
          const int s = it % a.stages;
          if (!mbar_wait_sleep(&full_bar[s], (it / a.stages) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t st = smem_u32(ring + (size_t)s * a.stage_bytes);
          const uint64_t da = umma_desc_sw128(st), db = umma_desc_sw128(st + (uint32_t)a.a_bytes);
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk)
            umma_i8(d, da + kk * 2, db + kk * 2, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&empty_bar[s]);
        }
        if (ok) umma_commit(&d_full[ai]);
      }
    }
  } else {
    w8_griddep_wait();  // sx is read (and Y written) after the kernels before
    const int q = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
    int t_iter = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x, ++t_iter) {
      const W8Tile w = w8_tile(a, start, tile);
      const int ai = t_iter & 1;
      const int r = 32 * q + lane;  // channel within the tile
      const bool row_ok = r < w.nh;
      const float sw = row_ok ? __ldg(a.sw + (size_t)w.e * a.N + w.n0 + r) : 0.0f;
      if (!mbar_wait_sleep(&d_full[ai], (t_iter >> 1) & 1)) break;
      tc_fence_after();
      for (int j = 0; j < w.mh; j += 32) {
        const float sxl = j + lane < w.mh ? __ldg(a.sx + w.m0 + j + lane) : 0.0f;
        uint32_t v[32];
        tmem_ld32(lane_base + (uint32_t)(ai * a.acc_stride + j), v);
        if (j + 32 >= w.mh) {  // the accumulator is in registers: the MMAs may fill it again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[ai]);
        }
        uint16_t* y = static_cast<uint16_t*>(a.Y) + (size_t)(w.m0 + j) * a.N + w.n0 + r;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float f = ((float)(int)v[i] * sw) * __shfl_sync(0xFFFFFFFFu, sxl, i);
          const uint16_t h =
              a.y_bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
          if (row_ok && j + i < w.mh) y[(size_t)i * a.N] = h;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 :: "r"(tmem), "r"((uint32_t)a.tmem_cols) : "memory");
  }
}

}  // namespace lbq
