// Rows of routed tokens: pairs (token t, choice j) sorted by expert, token rows
// copied into that order, and back with the router's weights, with gradients.
//
//   row(t, j)  = place of pair p = t top_k + j in the order by (expert, p), or
//                -1 for a pair without an expert
//   permute:     Xs[row(t, j)] = X[t]
//   combine:     out[t] = sum_j w[t][j] Y[row(t, j)]         (FP32, j ascending)
//   gradients:   dY[row(t, j)] = w[t][j] dout[t]
//                dw[t][j]      = sum_h dout[t][h] Y[row(t, j)][h]     (FP32)
//                dX[t]         = sum_j dXs[row(t, j)]   (combine with weights 1)
// Every result is a function of its inputs alone: no atomics, fixed orders.
#pragma once

#include "common.cuh"
#include "w4a8.cuh"

namespace lbq {

constexpr int kSortThreads = 1024;

// A stable counting sort without a pass between blocks: block e reads all the
// ids, counts those below e (its first row) and compacts the pairs of its own
// expert in ascending order. Each warp owns a contiguous range of the pairs and
// walks it twice: once to count, once (from cache) to write.
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                                int32_t* __restrict__ row_of_pair,
                                                                int32_t* __restrict__ pair_of_row,
                                                                int32_t* __restrict__ offsets) {
  __shared__ int eq_sh[32], lt_sh[32];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const int e = blockIdx.x;
  const int seg = (int)((((long long)P + nw - 1) / nw + 31) / 32 * 32);
  const long long b = (long long)warp * seg;
  const int p0 = (int)(b < P ? b : P), p1 = (int)(b + seg < P ? b + seg : P);
  int eq = 0, lt = 0;
  for (int p = p0 + lane; p < p1; p += 32) {
    const uint32_t id = (uint32_t)__ldg(ids + p);
    eq += id == (uint32_t)e;
    lt += id < (uint32_t)e;
  }
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  lt = __reduce_add_sync(0xFFFFFFFFu, lt);
  if (lane == 0) {
    eq_sh[warp] = eq;
    lt_sh[warp] = lt;
  }
  __syncthreads();
  const int ev = lane < nw ? eq_sh[lane] : 0, lv = lane < nw ? lt_sh[lane] : 0;
  const int first = __reduce_add_sync(0xFFFFFFFFu, lv);               // pairs of the experts before e
  const int count = __reduce_add_sync(0xFFFFFFFFu, ev);               // pairs of e
  int at = first + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? ev : 0);
  for (int p = p0; p < p1; p += 32) {
    const bool in = p + lane < p1;
    const uint32_t id = in ? (uint32_t)__ldg(ids + p + lane) : 0xFFFFFFFFu;
    const uint32_t mine = __ballot_sync(0xFFFFFFFFu, id == (uint32_t)e);
    if (id == (uint32_t)e) {
      const int r = at + __popc(mine & ((1u << lane) - 1u));
      row_of_pair[p + lane] = r;
      pair_of_row[r] = p + lane;
    }
    at += __popc(mine);
    if (e == 0 && in && id >= (uint32_t)E) row_of_pair[p + lane] = -1;
  }
  if (tid == 0) offsets[e] = first;
  if (e == E - 1) {
    if (tid == 0) offsets[E] = first + count;
    for (int r = first + count + tid; r < P; r += blockDim.x) pair_of_row[r] = -1;
  }
}

template <int B>
struct RowVec;  // B bytes of a row
template <> struct RowVec<16> { using T = uint4; };
template <> struct RowVec<8> { using T = uint2; };
template <> struct RowVec<4> { using T = uint32_t; };
template <> struct RowVec<2> { using T = uint16_t; };
template <> struct RowVec<1> { using T = uint8_t; };

// Thread = one B-byte piece of a token's row: read once, written to the token's
// top_k places.
template <int B>
__global__ void __launch_bounds__(256) moe_permute_kernel(const void* __restrict__ X, long long pieces, int per_row,
                                                          int top_k, const int32_t* __restrict__ row_of_pair, int rows,
                                                          void* __restrict__ Xs) {
  using V = typename RowVec<B>::T;
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= pieces) return;
  const long long t = i / per_row;
  const int c = (int)(i - t * per_row);
  const V v = static_cast<const V*>(X)[i];
  const int32_t* rp = row_of_pair + t * top_k;
  for (int j = 0; j < top_k; ++j) {
    const int r = __ldg(rp + j);
    if (r >= 0 && r < rows) static_cast<V*>(Xs)[(size_t)r * per_row + c] = v;
  }
}

// N 16-bit values as FP32 and back.
template <bool BF16, int N>
__device__ __forceinline__ void unpack_row(const typename RowVec<2 * N>::T& v, float (&f)[N]) {
  const uint16_t* h = reinterpret_cast<const uint16_t*>(&v);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = x2f<BF16>(h[i]);
}
template <bool BF16, int N>
__device__ __forceinline__ typename RowVec<2 * N>::T pack_row(const float (&f)[N]) {
  typename RowVec<2 * N>::T v;
  uint16_t* h = reinterpret_cast<uint16_t*>(&v);
#pragma unroll
  for (int i = 0; i < N; ++i)
    h[i] = BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[i])) : __half_as_ushort(__float2half_rn(f[i]));
  return v;
}

// Thread = N columns of one token: its top_k rows summed in FP32, j ascending,
// rounded once. weights null: 1.
template <bool BF16, int N>
__global__ void __launch_bounds__(256) moe_combine_kernel(const void* __restrict__ Y, int rows, long long pieces,
                                                          int per_row, int top_k,
                                                          const int32_t* __restrict__ row_of_pair,
                                                          const float* __restrict__ weights, void* __restrict__ out) {
  using V = typename RowVec<2 * N>::T;
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= pieces) return;
  const long long t = i / per_row;
  const int c = (int)(i - t * per_row);
  float acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    V v[4];
    float w[4];
    bool use[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      const int r = j < top_k ? __ldg(row_of_pair + t * top_k + j) : -1;
      use[u] = r >= 0 && r < rows;
      if (use[u]) {
        v[u] = static_cast<const V*>(Y)[(size_t)r * per_row + c];
        w[u] = weights ? __ldg(weights + t * top_k + j) : 1.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (use[u]) {
        float f[N];
        unpack_row<BF16, N>(v[u], f);
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = fmaf(w[u], f[n], acc[n]);
      }
  }
  static_cast<V*>(out)[i] = pack_row<BF16, N>(acc);
}

// Block = one token. Its dout row is read once for every four choices; each
// thread keeps its part of the four dot products, which meet in shared memory
// in a fixed order. dY may be Y (a thread reads a place before it writes it), so
// neither is declared restrict.
template <bool BF16, int N>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(const void* __restrict__ dout, const void* Y, int rows,
                                                               int per_row, int top_k,
                                                               const int32_t* __restrict__ row_of_pair,
                                                               const float* __restrict__ weights, void* dY,
                                                               float* __restrict__ dweights) {
  using V = typename RowVec<2 * N>::T;
  __shared__ float red[4][8];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const long long t = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const V* d = static_cast<const V*>(dout) + t * per_row;
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    int r[4];
    float w[4], dot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      r[u] = j < top_k ? __ldg(row_of_pair + t * top_k + j) : -1;
      if (r[u] >= rows) r[u] = -1;
      w[u] = r[u] >= 0 ? __ldg(weights + t * top_k + j) : 0.0f;
      dot[u] = 0.0f;
    }
    for (int c = tid; c < per_row; c += blockDim.x) {
      float g[N];
      unpack_row<BF16, N>(d[c], g);
      V y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (r[u] >= 0) y[u] = static_cast<const V*>(Y)[(size_t)r[u] * per_row + c];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (r[u] >= 0) {
          float f[N], o[N];
          unpack_row<BF16, N>(y[u], f);
#pragma unroll
          for (int n = 0; n < N; ++n) {
            dot[u] = fmaf(g[n], f[n], dot[u]);
            o[n] = w[u] * g[n];
          }
          static_cast<V*>(dY)[(size_t)r[u] * per_row + c] = pack_row<BF16, N>(o);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], o);
      if (lane == 0) red[u][warp] = dot[u];
    }
    __syncthreads();
    if (tid < 4 && j0 + tid < top_k) {
      float s = 0.0f;
      for (int i = 0; i < nw; ++i) s += red[tid][i];
      dweights[t * top_k + j0 + tid] = s;
    }
    __syncthreads();
  }
}

}  // namespace lbq
