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
//
// What a kernel before may write is read after griddepcontrol.wait and by coherent
// loads (ld_v4, ld_once_v4, or plain ones from pointers without __restrict__): the
// non-coherent path may return what lay there before, and the compiler may move a
// __ldg, or a load it takes for one, up across the wait. Only weights are read
// through the non-coherent path.
#pragma once

#include "common.cuh"
#include "tma.cuh"
#include "gemm_tc.cuh"
#include "stream_k.cuh"
#include "w4a8.cuh"

namespace lbq {

// ---------------------------------------------------------------------------- activations

// A row's scale from the largest magnitude's bits: s = amax / 127 in IEEE FP32.
// The maximum is taken over the bit patterns of |x| as integers, which order
// like the values with infinity and NaN above every finite one, so a row with a
// NaN or infinity gets that scale and codes 0: its products are NaN instead of
// passing for finite.
struct W8Scale {
  float s, inv;
  bool zero;   // codes are 0: an all-zero row, or one with an infinity or NaN
  bool exact;  // 1 / s overflows: every quotient by division
  __device__ __forceinline__ explicit W8Scale(float amax) {
    s = __fdiv_rn(amax, 127.0f);
    inv = __fdiv_rn(1.0f, s);
    zero = !(s > 0.0f && s <= 3.4028234663852886e38f);
    exact = !(inv <= 3.4028234663852886e38f);
  }
};

// Larger magnitude bits of either half of each word of v.
__device__ __forceinline__ uint32_t w8_max_bits(uint32_t m2, const uint4& v) {
  m2 = __vmaxu2(m2, v.x & 0x7FFF7FFFu);
  m2 = __vmaxu2(m2, v.y & 0x7FFF7FFFu);
  m2 = __vmaxu2(m2, v.z & 0x7FFF7FFFu);
  return __vmaxu2(m2, v.w & 0x7FFF7FFFu);
}

// Codes of 8 values: xq = rint(x / s), ties to even. As in quantize_int8_kernel
// the product t = RN(x RN(1/s)) decides wherever it is at least 2^-14 from a
// half-integer; one value closer than that in the eight (about one chunk in a
// thousand) sends the chunk to the IEEE quotients. |t| < 127.5 because |x| <=
// amax, so no clamp is needed. Adding 1.5 2^23 rounds t to an integer whose
// two's complement is the low byte of the sum.
template <bool BF16>
__device__ __forceinline__ uint2 w8_codes(const uint4& v, const W8Scale& q) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t b[8];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = __fmul_rn(x2f<BF16>((uint16_t)(u[i >> 1] >> (16 * (i & 1)))), q.inv);
    const float r = __fadd_rn(t, 12582912.0f);
    far = fmaxf(far, fabsf(__fadd_rn(t, -__fadd_rn(r, -12582912.0f))));
    b[i] = __float_as_uint(r);
  }
  if (q.exact || far > 0.5f - 6.103515625e-05f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = (uint32_t)(int)rintf(__fdiv_rn(x2f<BF16>((uint16_t)(u[i >> 1] >> (16 * (i & 1)))), q.s));
  }
  if (q.zero) return make_uint2(0u, 0u);
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// One warp per row, the row in registers (VPT chunks of 8 per lane): for many
// rows, where the rows of an SM's warps together are the bytes in flight and no
// block-wide exchange stops them (32768 rows of 2048: 38 us, 5.3 TB/s; 54 with a
// block per row).
template <bool BF16, int VPT>
__global__ void __launch_bounds__(256) quantize_int8_rows_warp_kernel(const uint16_t* X, int M, int K,
                                                                      int8_t* xq,
                                                                      float* sx) {
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int lane = threadIdx.x & 31, chunks = K >> 3;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= M) return;  // whole warps leave
  const uint4* xr = reinterpret_cast<const uint4*>(X + row * (size_t)K);
  uint4 v[VPT];
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * 32;
    v[i] = c < chunks ? ld_once_v4(xr + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) m2 = w8_max_bits(m2, v[i]);
  const W8Scale q(x2f<BF16>((uint16_t)__reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16))));
  uint2* out = reinterpret_cast<uint2*>(xq + row * (size_t)K);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = lane + i * 32;
    if (c < chunks) out[c] = w8_codes<BF16>(v[i], q);
  }
  if (lane == 0) sx[row] = q.s;
}

// One block per row of X, the row in registers (VPT chunks of 8 per thread): for
// few rows, whose latency counts (one of 4096 values: 1.9 us), and for long ones
// (8192 rows of 4096: 22 us, 4.5 TB/s; 30 with a warp per row, whose 16 chunks a
// lane cost half of the occupancy).
template <bool BF16, int VPT>
__global__ void __launch_bounds__(1024) quantize_int8_rows_kernel(const uint16_t* X, int K,
                                                                  int8_t* xq, float* sx) {
  __shared__ uint32_t warp_max[32];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int tid = threadIdx.x, chunks = K >> 3;
  const size_t row = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(X + row * (size_t)K);
  uint4 v[VPT];
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * blockDim.x;
    v[i] = c < chunks ? ld_v4(xr + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) m2 = w8_max_bits(m2, v[i]);
  uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
  if (blockDim.x > 32) {
    if ((tid & 31) == 0) warp_max[tid >> 5] = m;
    __syncthreads();
    const uint32_t w = (tid & 31) < (int)(blockDim.x >> 5) ? warp_max[tid & 31] : 0u;
    m = __reduce_max_sync(0xFFFFFFFFu, w);
  }
  const W8Scale q(x2f<BF16>((uint16_t)m));
  uint2* out = reinterpret_cast<uint2*>(xq + row * (size_t)K);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * blockDim.x;
    if (c < chunks) out[c] = w8_codes<BF16>(v[i], q);
  }
  if (tid == 0) sx[row] = q.s;
}

// ---------------------------------------------------------------------------- weights (offline)

// FP32 weight [K][N] -> codes [N][K] and a scale per channel, by the same rule.
// Block = 32 channels x 8 k rows; pass 1 the channels' maxima, pass 2 the codes,
// turned through a 32 x 32 tile so that both sides are read and written in rows. Run
// once per weight, so built for being simple: W is read twice, by N / 32 blocks (K = N
// = 4096 264 us, 4096 x 14336 444, 8192 x 28672 979, 0.3-1.2 TB/s of W and codes).
__global__ void __launch_bounds__(256) quantize_int8_weight_kernel(const float* W, int K, int N,
                                                                   int8_t* wq, float* sw) {
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

// ---------------------------------------------------------------------------- product, a few tokens

constexpr int kW8GvWarps = 8;
constexpr int kW8GvRows = 2;    // channels per warp at a time
constexpr int kW8GvUnroll = 4;  // 16-byte chunks per lane and channel at a time
constexpr int kW8GvMaxM = 4;
constexpr int kW8GvFusedM = 2;    // the most tokens of the quantising form
constexpr int kW8GvAhead = 2;     // steps that it prefetches into L2
constexpr int kW8GvFusedVpt = 8;  // X chunks of 8 per thread that the quantising form keeps in registers

struct W8GemvArgs {
  const void* X;     // QUANT: [M][K] FP16 / BF16; else int8 codes [M][K]
  const float* sx;   // [M] (codes only)
  const int8_t* wq;  // [N][K]
  const float* sw;   // [N]
  void* Y;           // [M][N]
  int M, K, N;
  int pairs;         // groups of kW8GvRows channels
  int y_bf16;
};

// Batch 1..MB on the CUDA cores: HBM-bound on the weights, 4 dp4a per 16 weight
// bytes and token. A warp takes two channels at a time, lanes take 16-byte chunks of
// their rows, and the next eight chunks per lane are requested before the last
// eight are multiplied; the tokens' codes lie in shared memory and serve both
// channels. Lane sums are integers, so one redux per channel and token joins them.
// The first weights are requested before anything else: the block then waits for
// the kernel before (which may write X), and, with QUANT, quantises the tokens
// itself (every block the same: reading a few KB from L2 costs less than a kernel
// in front). There the early request brings the weights of two steps into L2 only,
// and the loads follow those of X: X behind 64 KB of an SM's weights comes 1 us later
// (K = N = 4096 5.7 us instead of 4.6; one step ahead 4.9). With the quantiser, one
// token: 4.6-5.7 us at K = N = 4096 (9.4 on the tensor cores), 10.5-12.0 at N = 14336
// (4.9-5.6 TB/s), 34.6 at 8192 x 28672 (6.8 TB/s); four: 7.5 (9.6), 15 (15). More tokens
// are dp4a-bound and slower than the tensor cores: see w8_gemv_ok.
template <int MB, bool QUANT, bool BF16>
__global__ void __launch_bounds__(kW8GvWarps * 32, 2) w8a8_gemv_kernel(const W8GemvArgs a) {
  static_assert(!QUANT || MB <= kW8GvFusedM, "no call quantises more tokens in the block");
  extern __shared__ __align__(16) uint8_t xs[];  // [MB][K] codes
  __shared__ uint32_t max_sh[MB][kW8GvWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = a.K >> 4;
  const int steps = (chunks + 32 * kW8GvUnroll - 1) / (32 * kW8GvUnroll);  // per pair
  w8_griddep_launch_dependents();

  int pair = blockIdx.x * kW8GvWarps + warp, step = 0;  // the next loads
  const int stride = gridDim.x * kW8GvWarps;
  uint4 w[kW8GvRows][kW8GvUnroll];
  auto request = [&] {
#pragma unroll
    for (int r = 0; r < kW8GvRows; ++r) {
      const int n = min(pair * kW8GvRows + r, a.N - 1);
      const int8_t* row = a.wq + (size_t)n * a.K;
#pragma unroll
      for (int u = 0; u < kW8GvUnroll; ++u) {
        const int c = (step * kW8GvUnroll + u) * 32 + lane;
        w[r][u] = c < chunks ? ld_stream_v4(row + (size_t)c * 16) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  };
  const bool any = pair < a.pairs;
  if constexpr (!QUANT) {
    if (any) request();
  } else {
    int p = pair, t = step;
#pragma unroll 1
    for (int i = 0; i < kW8GvAhead && p < a.pairs; ++i) {
#pragma unroll
      for (int r = 0; r < kW8GvRows; ++r) {
        const int8_t* row = a.wq + (size_t)min(p * kW8GvRows + r, a.N - 1) * a.K;
#pragma unroll
        for (int u = 0; u < kW8GvUnroll; ++u) {
          const int c = (t * kW8GvUnroll + u) * 32 + lane;
          if (c < chunks) asm volatile("prefetch.global.L2 [%0];" :: "l"(row + (size_t)c * 16));
        }
      }
      if (++t == steps) {
        t = 0;
        p += stride;
      }
    }
  }

  float sx[MB];
  w8_griddep_wait();
  if constexpr (QUANT) {
    const int xchunks = a.K >> 3;
    constexpr int kVpt = kW8GvFusedVpt / MB;
    uint4 v[MB][kVpt];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.X) + (size_t)m * a.K);
#pragma unroll
      for (int i = 0; i < kVpt; ++i) {
        const int c = tid + i * (kW8GvWarps * 32);
        v[m][i] = m < a.M && c < xchunks ? ld_v4(xr + c) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (any) request();
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      uint32_t m2 = 0u;
#pragma unroll
      for (int i = 0; i < kVpt; ++i) m2 = w8_max_bits(m2, v[m][i]);
      const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
      if (lane == 0) max_sh[m][warp] = t;
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      uint32_t t = 0u;
#pragma unroll
      for (int i = 0; i < kW8GvWarps; ++i) t = max(t, max_sh[m][i]);
      const W8Scale q(x2f<BF16>((uint16_t)t));
      sx[m] = q.s;
#pragma unroll
      for (int i = 0; i < kVpt; ++i) {
        const int c = tid + i * (kW8GvWarps * 32);
        if (c < xchunks) *reinterpret_cast<uint2*>(xs + (size_t)m * a.K + (size_t)c * 8) = w8_codes<BF16>(v[m][i], q);
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      sx[m] = m < a.M ? a.sx[m] : 0.0f;
      const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const int8_t*>(a.X) + (size_t)m * a.K);
      for (int c = tid; c < chunks; c += kW8GvWarps * 32)
        reinterpret_cast<uint4*>(xs + (size_t)m * a.K)[c] = m < a.M ? ld_v4(xr + c) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  if (!any) return;

  int acc[kW8GvRows][MB];
  for (;;) {
    const int p = pair, s = step;  // what `w` holds
    if (s == 0) {
#pragma unroll
      for (int r = 0; r < kW8GvRows; ++r)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[r][m] = 0;
    }
    if (++step == steps) {
      step = 0;
      pair += stride;
    }
    uint4 cur[kW8GvRows][kW8GvUnroll];
#pragma unroll
    for (int r = 0; r < kW8GvRows; ++r)
#pragma unroll
      for (int u = 0; u < kW8GvUnroll; ++u) cur[r][u] = w[r][u];
    const bool more = pair < a.pairs;
    if (more) request();
#pragma unroll
    for (int u = 0; u < kW8GvUnroll; ++u) {
      const int c = min((s * kW8GvUnroll + u) * 32 + lane, chunks - 1);  // past the row: weights 0
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const uint4 x = *reinterpret_cast<const uint4*>(xs + (size_t)m * a.K + (size_t)c * 16);
#pragma unroll
        for (int r = 0; r < kW8GvRows; ++r) {
          acc[r][m] = __dp4a((int)cur[r][u].x, (int)x.x, acc[r][m]);
          acc[r][m] = __dp4a((int)cur[r][u].y, (int)x.y, acc[r][m]);
          acc[r][m] = __dp4a((int)cur[r][u].z, (int)x.z, acc[r][m]);
          acc[r][m] = __dp4a((int)cur[r][u].w, (int)x.w, acc[r][m]);
        }
      }
    }
    if (s == steps - 1) {
#pragma unroll
      for (int r = 0; r < kW8GvRows; ++r) {
        const int n = p * kW8GvRows + r;
        const float sw = n < a.N ? a.sw[n] : 0.0f;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          const int sum = __reduce_add_sync(0xFFFFFFFFu, acc[r][m]);
          if (lane == r * MB + m && n < a.N && m < a.M)
            store_out(a.Y, (size_t)m * a.N + n, ((float)sum * sw) * sx[m], a.y_bf16);
        }
      }
    }
    if (!more) break;
  }
}

// ---------------------------------------------------------------------------- product

constexpr int kW8BK = 128;        // k per block: one 128-byte swizzle span, four MMAs of K = 32
constexpr int kW8MaxHt = 128;     // channels per block and tile (TMEM lanes)
constexpr int kW8MaxBn = 256;     // tokens per tile (MMA N)
constexpr int kW8MaxStages = 16;
constexpr int kW8EpWarps = 8;     // two per TMEM lane quarter
constexpr int kW8Threads = (2 + kW8EpWarps) * 32;  // TMA producer, MMA issuer, epilogue
constexpr int kW8MaxSplits = 8;   // blocks that share one tile's K (one cluster)
constexpr int kW8MaxSplitBn = 128;  // ... of at most so many tokens: their sums lie beside the ring
static_assert(kW8MaxStages <= 16 && kW8MaxSplits <= 8, "one lane initialises each barrier and flag");
constexpr int kW8MaxExperts = 2048;
constexpr int kW8MaxK = 65536;        // 2^16 products of at most 2^14: the sum stays in int32
constexpr int kW8MaxRows = 0x7FFFFFFF - 1024;  // of either operand
constexpr int kW8SmemBudget = 222 * 1024;  // dynamic; barriers and the epilogue's scales take the rest of 227 KB

// Division of 0 <= a < 2^31 by a fixed b >= 1 through 2^32 / b (one correction
// suffices: the product is less than 1 too large). A division by a run-time value
// costs 100 clocks and more, and every role of a block needs two per tile.
struct W8Div {
  uint32_t b, m;
  static W8Div by(uint32_t d) { return W8Div{d, d > 1 ? (uint32_t)((1ull << 32) / d) + 1u : 0u}; }
  __device__ __forceinline__ int div(int a) const {
    if (b == 1) return a;
    uint32_t q = __umulhi((uint32_t)a, m);
    if (q * b > (uint32_t)a) --q;
    return (int)q;
  }
};

struct W8a8Args {
  void* Y;                  // [M][N]
  const float* sx;          // [M]
  const float* sw;          // [E][N]
  const int32_t* offsets;   // [E + 1] first row of each expert's run, or null (dense)
  int M, N, E;
  int ht, n_tiles;          // channels per block, tiles along N (CG ht channels each)
  W8Div by_n, by_band, by_last;  // n_tiles; tiles of a band of kSkBand token tiles; token tiles of the last band
  int n_unit, n_each, n_more;  // dense, CG = 1: a tile has n_unit n_each channels, the first n_more one unit more
  int bn, m_tiles;          // tokens per tile; tiles along M (dense)
  int k_stages, splits;     // ring stages of a tile's K; blocks that share them (CG = 1)
  int sub;                  // whole 128-k blocks per ring stage
  int k_whole, k_tail;      // K / 128; 1 if K % 128: one more stage, of the rest
  int stages, a_sub, b_off, stage_bytes;  // bytes: a weight block, offset of the token blocks, a stage
  int acc_stride, tmem_cols;
  int y_bf16;
  int hold;                 // test hook: the token rows are never copied, so every wait runs out
};

constexpr int kW8XMaps = 5;

// Tensor maps. Whole blocks: dimensions (128 bytes of k, row, k-block), so one
// copy fetches `sub` blocks, each a 128-byte swizzled tile (one copy per operand
// and stage: issuing a copy costs its warp some 150 clocks). Rest of K:
// dimensions (k, row), zeros past K. x[i] has boxes of x_rows(i) token rows:
// dense, only the tile's (i = 0); routed, 16 << i, so that a short run of rows
// is not fetched as a full tile.
struct W8Maps {
  CUtensorMap w, x[kW8XMaps], w_tail, x_tail[kW8XMaps];
};

// Instruction descriptor of kind::i8: D = S32 (2), A = B = S8 (1), both
// K-major, M = m, N = n.
__host__ __device__ constexpr uint32_t umma_idesc_i8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
  else
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc) : "memory");
}

// Arrive on `bar` (in both blocks of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void w8_commit(uint64_t* bar) {
  if constexpr (CG == 1)
    umma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

template <int CG>
__device__ __forceinline__ void w8_tmem_alloc(uint32_t* dst, uint32_t cols) {
  if constexpr (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(dst)), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}

template <int CG>
__device__ __forceinline__ void w8_tmem_dealloc(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(cols) : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(cols) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; writes before it are visible after it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this block's shared-memory location `addr` in block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Relaxed: what has to precede it are tensor-memory loads, and tcgen05.wait::ld has
// waited for those; a release would also wait for the output stores under way.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(addr) : "memory");
}
// mbar_wait_sleep that also orders what other blocks of the cluster did before their arrivals.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity) {
  for (uint32_t i = 0; i < kSleepPolls; ++i) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(kSleepHintNs) : "memory");
    if (ok) return true;
  }
  atomicOr(&g_device_error, kDevErrTimeout);
  return false;
}

// Tiled TMA loads into this block's shared memory; bytes counted on the barrier
// at shared::cluster address `bar` (for a pair: the first block's).
template <int CG>
__device__ __forceinline__ void w8_load_blocks(uint32_t dst, const CUtensorMap* m, int row, int kb, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(row), "r"(kb), "r"(bar) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(row), "r"(kb), "r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void w8_load_tail(uint32_t dst, const CUtensorMap* m, int row, int k, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(k), "r"(row), "r"(bar) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
                 "[%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(k), "r"(row), "r"(bar) : "memory");
}

// One output tile: channels n0 .. n0 + nh - 1 (this block's; of expert e), rows m0 .. m0 + mh - 1.
struct W8Tile {
  int n0, nh, m0, mh, e;
};

// Tile `t` of the call. Dense: bands of token tiles (stream_k.cuh); with CG = 1
// the channels are shared out evenly, tiles of at most ht (a tile's copy may take
// in a few rows of the next, which that one reads at the same time anyway).
// Routed: start[e] = token tiles of the experts before e and first[e] = the first
// row of e (shared memory), channels inner, so an expert's tiles are neighbours.
template <int CG>
__device__ __forceinline__ W8Tile w8_tile(const W8a8Args& a, const int* start, const int* first, int t, int rank) {
  W8Tile w;
  int nt = t, mt = 0;
  if (a.offsets == nullptr) {
    if (a.m_tiles > 1) {  // sk_tile_coords
      const int band = a.by_band.div(t), at = t - band * (int)a.by_band.b;
      const int wide = min(kSkBand, a.m_tiles - band * kSkBand);
      nt = wide == kSkBand ? at / kSkBand : a.by_last.div(at);
      mt = band * kSkBand + at - nt * wide;
    }
    w.e = 0;
    w.m0 = mt * a.bn;
    w.mh = min(a.bn, a.M - w.m0);
    if (CG == 1) {
      w.n0 = a.n_unit * (nt * a.n_each + min(nt, a.n_more));
      w.nh = min(a.N - w.n0, a.n_unit * (a.n_each + (nt < a.n_more ? 1 : 0)));
      return w;
    }
  } else {
    mt = a.by_n.div(t);
    nt = t - mt * a.n_tiles;
    int lo = 0, hi = a.E;  // the last e with start[e] <= mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= mt) lo = mid;
      else hi = mid;
    }
    w.e = lo;
    w.m0 = first[lo] + (mt - start[lo]) * a.bn;
    w.mh = min(a.bn, first[lo + 1] - w.m0);
  }
  w.n0 = (CG * nt + (CG == 2 ? rank : 0)) * a.ht;
  w.nh = max(0, min(a.ht, a.N - w.n0));
  return w;
}

// MMA N of a tile of mh rows: 16 columns a step, 32 for a pair.
template <int CG>
__device__ __forceinline__ int w8_mma_n(int mh) { return (mh + 16 * CG - 1) / (16 * CG) * (16 * CG); }

// The map of a tile's token rows (its index) and that map's rows per box.
template <int CG>
__device__ __forceinline__ int w8_x_map(const W8a8Args& a, int mh) {
  if (a.offsets == nullptr) return 0;
  const int rows = w8_mma_n<CG>(mh) / CG;  // a multiple of 16
  return rows <= 16 ? 0 : 32 - __clz((rows - 1) >> 4);
}
template <int CG>
__device__ __forceinline__ int w8_x_rows(const W8a8Args& a, int map) {
  return a.offsets == nullptr ? a.bn / CG : 16 << map;
}

// Inclusive scan over the block's threads (warp shuffles, then the warps' totals).
template <typename Op>
__device__ __forceinline__ int w8_block_scan(int v, Op op) {
  __shared__ int warp_total[kW8Threads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v = op(u, v);
  }
  __syncthreads();  // the last scan's totals have been read
  if (lane == 31) warp_total[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v = op(warp_total[w], v);
  return v;
}

// start[0 .. E] and first[0 .. E] of the routed form, by the whole block, each
// thread a contiguous range of experts. Offsets are clamped to the rows and taken
// as not decreasing (a smaller one counts as the largest before it), so runs never
// overlap and the tiles stay below M / bn + E whatever the array holds.
__device__ __forceinline__ void w8_expert_tiles(const W8a8Args& a, int* start, int* first) {
  const int per = (a.E + kW8Threads) / kW8Threads;  // of the E + 1 entries
  const int e0 = min(a.E + 1, (int)threadIdx.x * per), e1 = min(a.E + 1, e0 + per);
  int top = 0;
  for (int e = e0; e < e1; ++e) {
    top = max(top, min(a.offsets[e], a.M));
    first[e] = top;
  }
  const int highest = w8_block_scan(top, [](int x, int y) { return max(x, y); });
  int before = __shfl_up_sync(0xFFFFFFFFu, highest, 1);
  __shared__ int warp_top[kW8Threads / 32];
  if ((threadIdx.x & 31) == 31) warp_top[threadIdx.x >> 5] = highest;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) before = threadIdx.x ? warp_top[(threadIdx.x >> 5) - 1] : 0;
  for (int e = e0; e < e1; ++e) first[e] = max(first[e], before);
  __syncthreads();
  auto tiles_of = [&](int e) { return e < a.E ? (first[e + 1] - first[e] + a.bn - 1) / a.bn : 0; };
  int mine = 0;
  for (int e = e0; e < e1; ++e) mine += tiles_of(e);
  int o = w8_block_scan(mine, [](int x, int y) { return x + y; }) - mine;
  for (int e = e0; e < e1; ++e) {
    start[e] = o;
    o += tiles_of(e);
  }
  __syncthreads();
}

template <bool BF16>
__device__ __forceinline__ uint16_t w8_round(float f) {
  return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f)) : __half_as_ushort(__float2half_rn(f));
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool w8_elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Position in the ring, without a division per step.
struct W8Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
};

template <bool BF16>
__device__ __forceinline__ uint32_t w8_round2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// C accumulator columns (tokens; the first n count) of the warp's 32 channels
// into Y, y at the first token's row and the warp's first channel. PAIR (N even):
// lanes 2i and 2i + 1 exchange halves, so that a lane holds two channels of one
// token and a store writes 64 contiguous bytes of two tokens' rows; else one
// token's per store.
template <int C, bool BF16, bool PAIR>
__device__ __forceinline__ void w8_store(const uint32_t (&v)[C], float sw, const float* sxs, uint16_t* y, int N, int n,
                                         bool row_ok) {
  const int lane = threadIdx.x & 31;
  uint32_t h[C / 2];  // tokens 2i (low half), 2i + 1
#pragma unroll
  for (int i = 0; i < C; i += 4) {
    const float4 s4 = *reinterpret_cast<const float4*>(sxs + i);
    h[i / 2] = w8_round2<BF16>(((float)(int)v[i] * sw) * s4.x, ((float)(int)v[i + 1] * sw) * s4.y);
    h[i / 2 + 1] = w8_round2<BF16>(((float)(int)v[i + 2] * sw) * s4.z, ((float)(int)v[i + 3] * sw) * s4.w);
  }
  if constexpr (PAIR) {
    const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) h[i] = __byte_perm(h[i], __shfl_xor_sync(0xFFFFFFFFu, h[i], 1), sel);
    if (!row_ok) return;
    const int odd = lane & 1;  // this lane's token of each pair
    uint32_t* p = reinterpret_cast<uint32_t*>(y + (size_t)odd * N + (lane & ~1));
    if (n >= C) {
#pragma unroll
      for (int i = 0; i < C / 2; ++i) p[(size_t)i * N] = h[i];
    } else {
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        if (2 * i + odd < n) p[(size_t)i * N] = h[i];
    }
  } else {
    if (!row_ok) return;
    y += lane;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      if (2 * i < n) y[(size_t)(2 * i) * N] = (uint16_t)h[i];
      if (2 * i + 1 < n) y[(size_t)(2 * i + 1) * N] = (uint16_t)(h[i] >> 16);
    }
  }
}

// Accumulator columns of the warp's lanes; one statement with its wait, so that no
// use of a value can be placed before it.
__device__ __forceinline__ void w8_tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
               "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                 "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                 "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                 "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr) : "memory");
}
__device__ __forceinline__ void w8_tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
               "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                 "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                 "=r"(r[15])
               : "r"(taddr) : "memory");
}

// One warp's share of a finished accumulator: columns in chunks of C, every
// second (from chunk `half`). `taddr` is the accumulator at the warp's lanes, `y`
// the tile's first row at the warp's first channel, sx its first token's scale,
// sx_first that of column C half + lane. The barrier at `empty` is told as soon
// as the last chunk is in registers.
template <int C>
__device__ __forceinline__ void w8_epilogue(uint32_t taddr, int half, int mh, float sw, const float* sx, float sx_first,
                                            float* sxs, uint16_t* y, int N, int y_bf16, bool row_ok, uint32_t empty) {
  const int lane = threadIdx.x & 31;
  float sxl = sx_first;
  for (int j = C * half; j < mh; j += 2 * C) {
    __syncwarp();  // the last scales have been read
    if (lane < C) sxs[lane] = sxl;
    const int next = j + 2 * C + lane;
    sxl = lane < C && next < mh ? sx[next] : 0.0f;
    __syncwarp();
    uint32_t v[C];
    w8_tmem_ld(taddr + (uint32_t)j, v);
    if (j + 2 * C >= mh) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty);
    }
    uint16_t* yj = y + (size_t)j * N;
    if ((N & 1) == 0) {
      if (y_bf16) w8_store<C, true, true>(v, sw, sxs, yj, N, mh - j, row_ok);
      else w8_store<C, false, true>(v, sw, sxs, yj, N, mh - j, row_ok);
    } else {
      if (y_bf16) w8_store<C, true, false>(v, sw, sxs, yj, N, mh - j, row_ok);
      else w8_store<C, false, false>(v, sw, sxs, yj, N, mh - j, row_ok);
    }
  }
  if (C * half >= mh) {  // nothing for this warp
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(empty);
  }
}

// Warp 0: TMA producer (per ring stage one copy of the tile's weight rows and one
// of its token rows, `sub` blocks of 128 k each, 128-byte swizzled); warp 1: TMEM
// owner and MMA issuer; warps 2..9: epilogue, two for each TMEM lane quarter (lane =
// channel), 16 or 32 tokens at a time in turn. Two accumulators alternate, so the
// MMAs of a tile run while the last one is written. Persistent: block (or pair) u of
// U takes the tiles u, u + U, ..., and the ring runs on across them.
//
// Warps 0 and 1 run their loops converged and elect a lane for each issue: with
// warp-uniform control flow the descriptors stay in uniform registers. A loop of
// wait, four MMAs and commit measured 340 clocks so (128 x 16 tile; 512, the full
// rate, at 128 x 256) against 690 with one lane branching off for the whole loop.
//
// CG = 1: a tile of fewer than 128 channels loads only its own rows; the MMA's
// other rows read whatever follows in shared memory (integers, so no NaN can
// arise) and their lanes are not stored. The ring ends with that much slack.
// With splits > 1 the blocks of a cluster share the K of one tile: each sends its
// int32 sums to the shared memory of the block that finishes the token (token
// number modulo splits), which adds them up (integers: in any order the same).
//
// CG = 2: two blocks of a cluster share one MMA of 256 channels: each loads its
// own 128 weight rows and half of the token rows, so the token operand crosses
// shared memory once per pair. The first block issues the MMAs; copies of both
// are counted on its barrier, and its commits arrive in both blocks.
//
// Measured (K = 4096, N = 14336 unless stated): 16 tokens 13.8 us, 64 14.3, 512
// 29.4 (2.05 P operations/s), 2048 79-83 (2.9-3.05), 8192 295-310 (3.1-3.26, 92-96% of
// twice the measured BF16 rate; CG = 1 takes 348); 16 tokens at 8192 x 28672 41.5 us
// (5.7 TB/s); routed, 32768 rows over 256 experts of 2048 x 1024, 113-118 us (5.7-5.9
// TB/s).
template <int CG>
__global__ void __launch_bounds__(kW8Threads, 1)
    w8a8_gemm_kernel(const __grid_constant__ W8Maps maps, const W8a8Args a) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kW8MaxStages], empty_bar[kW8MaxStages], d_full[2], d_empty[2];
  __shared__ __align__(16) float sx_sh[kW8EpWarps][32];  // an epilogue warp's token scales
  __shared__ uint32_t tmem_base_sh;
  __shared__ int split_ok[kW8MaxSplits];  // the block's sums have been sent
  uint8_t* ring = dsmem + ((1024u - (smem_u32(dsmem) & 1023u)) & 1023u);
  uint8_t* behind = ring + (size_t)a.stages * a.stage_bytes + kW8MaxHt * kW8BK;
  int* start = reinterpret_cast<int*>(behind);  // routed: see w8_expert_tiles
  int* first = start + a.E + 1;
  int* sums = reinterpret_cast<int*>(behind);   // splits: [token / splits][source block][128 channels]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool split = CG == 1 && a.splits > 1;
  const int rank = (CG == 2 || split) ? (int)cluster_rank() : 0;
  const int share = CG == 2 ? 2 : a.splits;  // blocks per tile
  const uint32_t ring_u = smem_u32(ring), full_u = smem_u32(full_bar);
  const uint32_t full_c = CG == 2 ? cluster_addr(full_u, 0) : full_u;  // the barriers that count the bytes
  const int unit = blockIdx.x / share, units = gridDim.x / share;
  // this block's stages of each of its tiles
  const int ks0 = split ? a.k_stages * rank / a.splits : 0;
  const int ks1 = split ? a.k_stages * (rank + 1) / a.splits : a.k_stages;
  // weights of k-stage ks of tile w into ring stage `slot`, and the announcement of all the stage's bytes
  const int tail_stage = a.k_tail ? a.k_stages - 1 : -1;
  auto load_w = [&](const W8Tile& w, int xrows, int ks, int slot) {
    const uint32_t st = ring_u + (uint32_t)(slot * a.stage_bytes), bar = full_c + 8u * slot;
    const bool tail = ks == tail_stage;
    if (w8_elect()) {
      if (CG == 1 || rank == 0)
        mbar_arrive_expect_tx(&full_bar[slot], (uint32_t)(CG * (tail ? 1 : a.sub) * (a.ht + xrows) * kW8BK));
      if (!tail) w8_load_blocks<CG>(st, &maps.w, w.e * a.N + w.n0, ks * a.sub, bar);
      else w8_load_tail<CG>(st, &maps.w_tail, w.e * a.N + w.n0, a.k_whole * kW8BK, bar);
    }
  };
  // the weights of the first stages, requested before the kernel that writes the
  // activations has ended (and, where nothing else is needed for it, before the
  // rest of the block is set up); returns their number
  auto load_first = [&](int total) {
    int pre = 0;
    for (int tile = unit; tile < total && pre < a.stages; tile += units) {
      const W8Tile w = w8_tile<CG>(a, start, first, tile, rank);
      const int xrows = w8_x_rows<CG>(a, w8_x_map<CG>(a, w.mh));
      for (int ks = ks0; ks < ks1 && pre < a.stages; ++ks, ++pre) load_w(w, xrows, ks, pre);
    }
    return pre;
  };
  const bool early = CG == 1 && a.offsets == nullptr;
  int pre = 0;
  w8_griddep_launch_dependents();
  if (warp == 0) {
    // a lane per barrier (one lane for all of them takes 1000 clocks)
    if (lane < a.stages) {
      mbar_init(&full_bar[lane], 1);
      mbar_init(&empty_bar[lane], 1);
    } else if (lane >= kW8MaxStages && lane < kW8MaxStages + 2) {
      mbar_init(&d_full[lane - kW8MaxStages], 1);
      mbar_init(&d_empty[lane - kW8MaxStages], kW8EpWarps * CG);
    } else if (lane >= 24) {
      split_ok[lane - 24] = 0;
    }
    fence_barrier_init();
    __syncwarp();
    if (early) pre = load_first(a.m_tiles * a.n_tiles);
  }
  if (warp == 1) w8_tmem_alloc<CG>(&tmem_base_sh, (uint32_t)a.tmem_cols);
  if (split) cluster_arrive();  // this block runs and its flags are cleared
  if (a.offsets != nullptr) {
    w8_griddep_wait();  // the offsets come from a kernel before
    w8_expert_tiles(a, start, first);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the other block's barriers are ready
  if (split) cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const int total = (a.offsets == nullptr ? a.m_tiles : start[a.E]) * a.n_tiles;

  if (warp == 0) {
    auto load_x = [&](int map, int row, int ks, int slot) {
      const uint32_t st = ring_u + (uint32_t)(slot * a.stage_bytes + a.b_off), bar = full_c + 8u * slot;
      if (w8_elect() && !a.hold) {
        if (ks != tail_stage) w8_load_blocks<CG>(st, &maps.x[map], row, ks * a.sub, bar);
        else w8_load_tail<CG>(st, &maps.x_tail[map], row, a.k_whole * kW8BK, bar);
      }
    };
    if (!early) pre = load_first(total);
    w8_griddep_wait();
    W8Ring r;
    int it = 0;
    bool ok = true;
    for (int tile = unit; tile < total && ok; tile += units) {
      const W8Tile w = w8_tile<CG>(a, start, first, tile, rank);
      const int map = w8_x_map<CG>(a, w.mh), xrows = w8_x_rows<CG>(a, map);
      const int x0 = w.m0 + (CG == 2 ? rank * (w8_mma_n<2>(w.mh) / 2) : 0);  // a pair: half of the MMA's N each
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        if (it >= pre) {
          ok = mbar_wait_sleep(&empty_bar[r.s], r.phase ^ 1);
          if (!ok) break;
          load_w(w, xrows, ks, r.s);
        }
        load_x(map, x0, ks, r.s);
        r.next(a.stages);
      }
    }
    // before the block may exit, its last copies have landed and the commits
    // on its barriers have arrived (after a timed-out wait: the copies, which
    // had that wait's time as well)
    for (int i = 0; i < a.stages; ++i) {
      if (!mbar_wait_sleep(&empty_bar[r.s], r.phase ^ 1)) {
        if (CG == 1) mbar_wait_sleep(&full_bar[r.s], r.phase ^ 1);
        break;
      }
      r.next(a.stages);
    }
  } else if (warp == 1) {
    if (CG == 1 || rank == 0) {
      W8Ring r;
      int t_iter = 0;
      bool ok = true;
      for (int tile = unit; tile < total && ok; tile += units, ++t_iter) {
        const W8Tile w = w8_tile<CG>(a, start, first, tile, rank);
        const uint32_t idesc = umma_idesc_i8(128 * CG, w8_mma_n<CG>(w.mh));
        const int ai = t_iter & 1;
        const uint32_t d = tmem + (uint32_t)(ai * a.acc_stride);
        if (t_iter >= 2) {
          ok = mbar_wait_cluster(&d_empty[ai], ((t_iter >> 1) & 1) ^ 1);
          if (!ok) break;
        }
        tc_fence_after();
        // 16-byte units between a stage's blocks
        const uint64_t a_step = (uint64_t)((uint32_t)a.a_sub >> 4);
        const uint64_t b_step = (uint64_t)((uint32_t)(w8_x_rows<CG>(a, w8_x_map<CG>(a, w.mh)) * kW8BK) >> 4);
        for (int ks = ks0; ks < ks1; ++ks) {
          ok = mbar_wait_sleep(&full_bar[r.s], r.phase);
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = ring_u + (uint32_t)(r.s * a.stage_bytes);
          // blocks of this stage (past K they are zeros: not multiplied)
          const int nb = a.k_tail && ks == a.k_stages - 1 ? 1 : min(a.sub, a.k_whole - ks * a.sub);
          if (w8_elect()) {
            uint64_t da = umma_desc_sw128(st), db = umma_desc_sw128(st + (uint32_t)a.b_off);
            for (int u = 0; u < nb; ++u) {
#pragma unroll
              for (uint32_t kk = 0; kk < 4; ++kk)
                umma_i8<CG>(d, da + kk * 2, db + kk * 2, idesc, (ks > ks0 || u > 0 || kk > 0) ? 1u : 0u);
              da += a_step;
              db += b_step;
            }
            w8_commit<CG>(&empty_bar[r.s]);
          }
          r.next(a.stages);
        }
        if (ok && w8_elect()) w8_commit<CG>(&d_full[ai]);
      }
    }
  } else {
    w8_griddep_wait();  // sx is read (and Y written) after the kernels before
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t d_empty_c = CG == 2 ? cluster_addr(smem_u32(d_empty), 0) : smem_u32(d_empty);
    float* sxs = sx_sh[warp - 2];
    const int r = 32 * q + lane;  // channel within the block's part of the tile
    // what a tile needs from global memory, requested a tile ahead
    struct Ahead {
      W8Tile w;
      float sw, sx;
    } cur{}, nxt{};
    auto request = [&](int tile) {
      Ahead t{};
      t.w = w8_tile<CG>(a, start, first, tile, rank);
      if (r < t.w.nh) t.sw = a.sw[(size_t)t.w.e * a.N + t.w.n0 + r];
      const int c = (t.w.mh > 32 ? 32 : 16), j = c * half + lane;
      if (lane < c && j < t.w.mh) t.sx = a.sx[t.w.m0 + j];
      return t;
    };
    if (unit < total) nxt = request(unit);
    int t_iter = 0;
    for (int tile = unit; tile < total; tile += units, ++t_iter) {
      cur = nxt;
      if (tile + units < total) nxt = request(tile + units);
      const W8Tile& w = cur.w;
      const int ai = t_iter & 1;
      if (!mbar_wait_sleep(&d_full[ai], (t_iter >> 1) & 1)) break;
      tc_fence_after();
      if (split) {
        const uint32_t dst = smem_u32(sums) + 4u * (uint32_t)(rank * kW8MaxHt + r);
        for (int c = half; 32 * c < w.mh; c += 2) {
          uint32_t v[32];
          w8_tmem_ld(lane_base + (uint32_t)(ai * a.acc_stride + 32 * c), v);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int t = 32 * c + i;
            if (t < w.mh)
              st_cluster(cluster_addr(dst + (uint32_t)((t & -a.splits) * kW8MaxHt * 4), (uint32_t)(t & (a.splits - 1))),
                         (int)v[i]);  // splits: a power of two
          }
        }
        if (warp == 2 && lane < a.splits) st_cluster(cluster_addr(smem_u32(&split_ok[rank]), (uint32_t)lane), 1);
        break;
      }
      const uint32_t taddr = lane_base + (uint32_t)(ai * a.acc_stride), empty = d_empty_c + 8u * ai;
      uint16_t* y = static_cast<uint16_t*>(a.Y) + (size_t)w.m0 * a.N + w.n0 + 32 * q;
      if (w.mh > 32)
        w8_epilogue<32>(taddr, half, w.mh, cur.sw, a.sx + w.m0, cur.sx, sxs, y, a.N, a.y_bf16, r < w.nh, empty);
      else
        w8_epilogue<16>(taddr, half, w.mh, cur.sw, a.sx + w.m0, cur.sx, sxs, y, a.N, a.y_bf16, r < w.nh, empty);
    }
  }
  __syncwarp();

  if (split) {
    // lane = four channels; warp = every eighth of this block's tokens rank, rank + splits, ...
    const bool mine = warp >= 2 && unit < total;
    W8Tile w{};
    const int c0 = lane << 2;
    float sw[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sxl = 0.0f;
    if (mine) {
      w = w8_tile<CG>(a, start, first, unit, rank);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c0 + i < w.nh) sw[i] = a.sw[(size_t)w.e * a.N + w.n0 + c0 + i];
      const int t = rank + a.splits * (warp - 2 + kW8EpWarps * lane);
      if (t < w.mh) sxl = a.sx[w.m0 + t];
    }
    cluster_sync();  // every block's sums have arrived
    if (mine) {
      bool ok = true;
      for (int c = 0; c < a.splits; ++c) ok = ok && *const_cast<volatile int*>(&split_ok[c]) != 0;
      const int left = w.nh - c0;
      for (int i = 0; rank + a.splits * (warp - 2 + kW8EpWarps * i) < w.mh; ++i) {
        const int k = warp - 2 + kW8EpWarps * i, t = rank + a.splits * k;
        const float sx = __shfl_sync(0xFFFFFFFFu, sxl, i);
        int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int c = 0; c < kW8MaxSplits; ++c)
          if (c < a.splits) {
            const int4 v = *reinterpret_cast<const int4*>(sums + (size_t)(k * a.splits + c) * kW8MaxHt + c0);
            sum.x += v.x;
            sum.y += v.y;
            sum.z += v.z;
            sum.w += v.w;
          }
        if (!ok || left <= 0) continue;
        const float f[4] = {((float)sum.x * sw[0]) * sx, ((float)sum.y * sw[1]) * sx, ((float)sum.z * sw[2]) * sx,
                            ((float)sum.w * sw[3]) * sx};
        uint16_t* y = static_cast<uint16_t*>(a.Y) + (size_t)(w.m0 + t) * a.N + w.n0 + c0;
        if (a.n_unit == 4) {  // rows and tiles in steps of 8 bytes
          *reinterpret_cast<uint2*>(y) =
              a.y_bf16 ? make_uint2(w8_round2<true>(f[0], f[1]), w8_round2<true>(f[2], f[3]))
                       : make_uint2(w8_round2<false>(f[0], f[1]), w8_round2<false>(f[2], f[3]));
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < left) y[u] = a.y_bf16 ? w8_round<true>(f[u]) : w8_round<false>(f[u]);
        }
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // no block's shared memory or barriers are needed any more
  if (warp == 1) {
    tc_fence_after();
    w8_tmem_dealloc<CG>(tmem, (uint32_t)a.tmem_cols);
  }
}

}  // namespace lbq
