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
// Every result is a function of its inputs alone: fixed orders, and no atomics but
// the counts of moe_sort_kernel, whose sums do not depend on theirs.
#pragma once

#include "common.cuh"
#include "w4a8.cuh"
#include "w8a8.cuh"

namespace lbq {

constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;       // blocks of the clustered sort
constexpr int kSortBlockPairs = 16384;       // the most pairs of the block-per-expert sort
constexpr long long kSortBlockWork = 1 << 24; // ... and pairs times experts

// A stable counting sort without a pass between blocks: block e reads all the
// ids (16 bytes per thread V times, kept in registers), counts those below e (its
// first row) and compacts the pairs of its own expert in ascending order. Reads
// E P ids from L2 in all; no block waits for another. Measured against the
// clustered sort below: 128 pairs and 256 experts 1.6 us against 4.6, 8192 and 256
// 3.6 against 5.6, 4096 and 1024 5.6 against 8.2, 8192 and 2048 12.1 against 16.0;
// 32768 and 256 10.2 against 8.3, 32768 and 8 9.4 against 6.4.
template <int V>
__global__ void __launch_bounds__(kSortThreads) moe_sort_block_kernel(const int32_t* ids, int P, int E,
                                                                      int32_t* row_of_pair,
                                                                      int32_t* pair_of_row,
                                                                      int32_t* offsets) {
  __shared__ int eq_sh[32], lt_sh[32];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const uint32_t e = blockIdx.x;
  const int p0 = warp * (V * 128) + lane * 4;  // each warp: V runs of 128 pairs
  uint4 id[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int p = p0 + v * 128;
    id[v] = make_uint4(0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu);
    if (p + 3 < P) {
      id[v] = ld_v4(ids + p);
    } else {
      if (p < P) id[v].x = (uint32_t)ids[p];
      if (p + 1 < P) id[v].y = (uint32_t)ids[p + 1];
      if (p + 2 < P) id[v].z = (uint32_t)ids[p + 2];
    }
  }
  int eq = 0, lt = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    eq += (id[v].x == e) + (id[v].y == e) + (id[v].z == e) + (id[v].w == e);
    lt += (id[v].x < e) + (id[v].y < e) + (id[v].z < e) + (id[v].w < e);
  }
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  lt = __reduce_add_sync(0xFFFFFFFFu, lt);
  if (lane == 0) {
    eq_sh[warp] = eq;
    lt_sh[warp] = lt;
  }
  __syncthreads();
  const int ev = lane < nw ? eq_sh[lane] : 0, lv = lane < nw ? lt_sh[lane] : 0;
  const int first = __reduce_add_sync(0xFFFFFFFFu, lv);  // pairs of the experts before e
  const int count = __reduce_add_sync(0xFFFFFFFFu, ev);  // pairs of e
  int at = first + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? ev : 0);
  if (eq > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool m[4] = {id[v].x == e, id[v].y == e, id[v].z == e, id[v].w == e};
      if (__ballot_sync(0xFFFFFFFFu, m[0] || m[1] || m[2] || m[3]) == 0u) continue;
      int r = at;  // rows before this lane's first pair of the run
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, m[c]);
        r += __popc(b & ((1u << lane) - 1u));
        at += __popc(b);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (m[c]) {
          const int p = p0 + v * 128 + c;
          row_of_pair[p] = r;
          pair_of_row[r++] = p;
        }
    }
  }
  if (e == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t q[4] = {id[v].x, id[v].y, id[v].z, id[v].w};
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (q[c] >= (uint32_t)E && p0 + v * 128 + c < P) row_of_pair[p0 + v * 128 + c] = -1;
    }
  }
  if (tid == 0) offsets[e] = first;
  if (e == (uint32_t)E - 1) {
    if (tid == 0) offsets[E] = first + count;
    for (int r = first + count + tid; r < P; r += blockDim.x) pair_of_row[r] = -1;
  }
}

// The same order by one cluster of eight blocks. Every warp owns a contiguous
// range of the pairs: it counts its ids per expert in its own row of shared
// memory; the rows become exclusive sums over the block's warps, the blocks
// exchange their totals through distributed shared memory, and each warp walks its
// range again, 32 pairs at a time, handing out places in order (lanes with the
// same id by their rank among them). Time grows with the pairs, not with the
// experts.
// Dynamic shared memory: [warps][E] counts, [E] totals of the block, [E] bases.
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(const int32_t* ids, int P, int E,
                                                                int32_t* row_of_pair,
                                                                int32_t* pair_of_row,
                                                                int32_t* offsets) {
  extern __shared__ int sort_sm[];
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
  int* count = sort_sm;            // [nw][E]
  int* total = count + nw * E;     // [E] this block's pairs of each expert
  int* base = total + E;           // [E] first row of this block's pairs of each expert
  const int rank = (int)cluster_rank();
  w8_griddep_launch_dependents();
  for (int i = tid; i < nw * E; i += nt) count[i] = 0;
  __syncthreads();
  w8_griddep_wait();

  const long long ranges = (long long)kSortCluster * nw, range = rank * nw + warp;
  const long long seg = ((P + ranges - 1) / ranges + 31) / 32 * 32;
  const int p0 = (int)min((long long)P, range * seg), p1 = (int)min((long long)P, range * seg + seg);
  int* mine = count + warp * E;
#pragma unroll 4
  for (int p = p0 + lane; p < p1; p += 32) {
    const uint32_t id = (uint32_t)ids[p];
    if (id < (uint32_t)E) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += nt) {  // exclusive over the warps
    int sum = 0;
    for (int w = 0; w < nw; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = sum;
      sum += c;
    }
    total[e] = sum;
  }
  cluster_sync();
  // bases: all pairs of the experts before, then those of the blocks before
  const int per = (E + nt - 1) / nt, e0 = min(E, tid * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int before = 0, all = 0;
#pragma unroll
    for (int c = 0; c < kSortCluster; ++c) {
      const int v = ld_cluster(cluster_addr(smem_u32(total + e), (uint32_t)c));
      before += c < rank ? v : 0;
      all += v;
    }
    base[e] = sum + before;
    sum += all;
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  cluster_sync();  // (also the block's barrier) no block's totals are needed any more
  const int ws = lane < nw ? warp_sum[lane] : 0;
  const int rows = __reduce_add_sync(0xFFFFFFFFu, ws);
  const int o = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? ws : 0) + incl - sum;
  for (int e = e0; e < e1; ++e) base[e] += o;
  if (rank == 0) {
    // the first block's bases are the offsets (no block lies before it)
    for (int e = e0; e < e1; ++e) offsets[e] = base[e];
    if (tid == 0) offsets[E] = rows;
  }
  __syncthreads();

  // (match.any takes some 70 clocks of the SM per warp; log2 E votes are cheaper)
  const int bits = E > 1 ? 32 - __clz(E - 1) : 0;
  uint32_t next = p0 + lane < p1 ? (uint32_t)ids[p0 + lane] : 0xFFFFFFFFu;
  for (int p = p0; p < p1; p += 32) {
    const bool in = p + lane < p1;
    const uint32_t id = next;
    next = p + 32 + lane < p1 ? (uint32_t)ids[p + 32 + lane] : 0xFFFFFFFFu;
    uint32_t same = __ballot_sync(0xFFFFFFFFu, id < (uint32_t)E);  // lanes with this lane's id, bit by bit
    for (int b = 0; b < bits; ++b) {
      const uint32_t set = __ballot_sync(0xFFFFFFFFu, (id >> b) & 1u);
      same &= (id >> b) & 1u ? set : ~set;
    }
    const int before = __popc(same & ((1u << lane) - 1u));
    int r = -1;
    if (id < (uint32_t)E) {
      r = base[id] + mine[id] + before;
      pair_of_row[r] = p + lane;
    }
    __syncwarp();
    if (id < (uint32_t)E && before == 0) mine[id] += __popc(same);
    __syncwarp();
    if (in) row_of_pair[p + lane] = r;
  }
  for (int r = rows + rank * nt + tid; r < P; r += kSortCluster * nt) pair_of_row[r] = -1;
}

template <int B>
struct RowVec;  // B bytes of a row
template <> struct RowVec<16> { using T = uint4; };
template <> struct RowVec<8> { using T = uint2; };
template <> struct RowVec<4> { using T = uint32_t; };
template <> struct RowVec<2> { using T = uint16_t; };
template <> struct RowVec<1> { using T = uint8_t; };

// Threads of a block per token: 2^shift, the token's pieces strided over them.
// Copies a token's row, read once, to its top_k places; U pieces per thread and
// step, so that narrow pieces (rows that 16 bytes do not divide) still have
// several loads in flight. HBM-bound: 4096 tokens, top-8, rows of 4 KB 25.6 us (5.9
// TB/s); rows of 2006 bytes (2-byte pieces, top-2) 7.8 us (3.1 TB/s; 11.2 with four
// pieces per thread instead of eight).
template <int B, int U>
__global__ void __launch_bounds__(256) moe_permute_kernel(const void* X, int T, int per_row, int top_k,
                                                          const int32_t* row_of_pair, int rows,
                                                          void* Xs, int shift) {
  using V = typename RowVec<B>::T;
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int lanes = 1 << shift, l = threadIdx.x & (lanes - 1);
  const long long t = (((long long)blockIdx.x << 8) + threadIdx.x) >> shift;
  if (t >= T) return;
  const V* x = static_cast<const V*>(X) + t * per_row;
  const int32_t* rp = row_of_pair + t * top_k;
  for (long long c0 = l; c0 < per_row; c0 += (long long)lanes * U) {
    V v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * lanes < per_row) v[u] = x[c0 + u * lanes];
    for (int j = 0; j < top_k; ++j) {
      const int r = rp[j];
      if (r < 0 || r >= rows) continue;
      V* y = static_cast<V*>(Xs) + (size_t)r * per_row + c0;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * lanes < per_row) y[u * lanes] = v[u];
    }
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

// Threads of a block per token as in moe_permute_kernel; a piece is N columns: the
// token's top_k rows summed in FP32, j ascending, rounded once, kCombineRows rows
// times U pieces in flight per thread. weights null: 1. HBM-bound on the scattered
// rows: 4096 tokens, top-8, H = 2048 27.6 us (5.5 TB/s; with eight rows in flight,
// which do not fit the registers of four blocks per SM, 28.8, and 29.3 with three
// blocks). Registers are bounded to as many blocks per SM as pays: H = 1004 17.1 us
// (four blocks; 19.6 with three), H = 1002 19.0 (29.3), H = 1003 29.6 (three blocks;
// 43 with four, 53 with two).
constexpr int kCombineRows = 4;
template <bool BF16, int N, int U>
__global__ void __launch_bounds__(256, N == 1 ? 3 : 4) moe_combine_kernel(const void* Y, int rows, int T, int per_row,
                                                          int top_k, const int32_t* row_of_pair,
                                                          const float* weights, void* out,
                                                          int shift) {
  constexpr int J = kCombineRows;
  using V = typename RowVec<2 * N>::T;
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  const int lanes = 1 << shift, l = threadIdx.x & (lanes - 1);
  const long long t = (((long long)blockIdx.x << 8) + threadIdx.x) >> shift;
  if (t >= T) return;
  for (long long c0 = l; c0 < per_row; c0 += (long long)lanes * U) {
    float acc[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int n = 0; n < N; ++n) acc[u][n] = 0.0f;
    for (int j0 = 0; j0 < top_k; j0 += J) {
      V v[J][U];
      float w[J];
      bool use[J];
#pragma unroll
      for (int i = 0; i < J; ++i) {
        const int r = j0 + i < top_k ? row_of_pair[t * top_k + j0 + i] : -1;
        use[i] = r >= 0 && r < rows;
        const V* y = static_cast<const V*>(Y) + (size_t)(use[i] ? r : 0) * per_row + c0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (use[i] && c0 + u * lanes < per_row) v[i][u] = y[u * lanes];
        w[i] = use[i] && weights ? weights[t * top_k + j0 + i] : 1.0f;
      }
#pragma unroll
      for (int i = 0; i < J; ++i)
        if (use[i]) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float f[N];
            unpack_row<BF16, N>(v[i][u], f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[u][n] = fmaf(w[i], f[n], acc[u][n]);
          }
        }
    }
    V* o = static_cast<V*>(out) + t * per_row + c0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * lanes < per_row) o[u * lanes] = pack_row<BF16, N>(acc[u]);
  }
}

constexpr int kZeroRows = 8192;  // the most rows per zeroing block (a byte each in shared memory)

// Zero the rows of dY among r0 .. r1 - 1 (at most kZeroRows) that no entry of
// row_of_pair names: a mark per row, set from all the entries (a store each, of the
// others to a place behind: a branch per entry takes twice as long), then a warp
// per row.
template <typename V>
__device__ __forceinline__ void moe_zero_unnamed(V* dY, int per_row, const int32_t* row_of_pair, long long pairs, int r0,
                                                 int r1) {
  __shared__ uint32_t marks[kZeroRows / 4 + 1];
  uint8_t* named = reinterpret_cast<uint8_t*>(marks);
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int i = tid; i <= (r1 - r0) / 4; i += nt) marks[i] = 0u;
  __syncthreads();
  auto mark = [&](int r) {
    named[min((uint32_t)r - (uint32_t)r0, (uint32_t)(r1 - r0))] = 1;
  };
  const int4* v = reinterpret_cast<const int4*>(row_of_pair);
  const long long quads = pairs >> 2;
  for (long long q = tid; q < quads; q += 8LL * nt) {
    int4 r[8];  // requested together, then marked
#pragma unroll
    for (int u = 0; u < 8; ++u) r[u] = q + u * nt < quads ? v[q + u * nt] : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      mark(r[u].x);
      mark(r[u].y);
      mark(r[u].z);
      mark(r[u].w);
    }
  }
  if (tid < (int)(pairs & 3)) mark(row_of_pair[4 * quads + tid]);
  __syncthreads();
  for (int r = r0 + (tid >> 5); r < r1; r += nt >> 5) {
    if (named[r - r0]) continue;
    V* y = dY + (size_t)r * per_row;
    for (int i = tid & 31; i < per_row; i += 32) y[i] = V{};
  }
}

// Block = one token. Its dout row is read once for every four choices; each
// thread keeps its part of the four dot products, which meet in shared memory
// in a fixed order. HBM-bound: 4096 tokens, top-8, H = 2048 49 us (5.8 TB/s), H =
// 1002 30 (4.6), H = 1003 46 (3.0). dY may be Y (a thread reads a place before it
// writes it), so neither is declared restrict. The grid's first zero_blocks blocks,
// if any, zero the rows of dY that no entry names, zero_rows each; no other block
// touches those.
template <bool BF16, int N, int U>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(const void* dout, const void* Y, int rows,
                                                               int per_row, int top_k,
                                                               const int32_t* row_of_pair,
                                                               const float* weights, void* dY,
                                                               float* dweights, int zero_blocks, int zero_rows) {
  using V = typename RowVec<2 * N>::T;
  __shared__ float red[4][8];
  w8_griddep_launch_dependents();
  w8_griddep_wait();
  if ((int)blockIdx.x < zero_blocks) {
    const int r0 = (int)blockIdx.x * zero_rows;
    moe_zero_unnamed(static_cast<V*>(dY), per_row, row_of_pair, (long long)(gridDim.x - zero_blocks) * top_k, r0,
                     min(rows, r0 + zero_rows));
    return;
  }
  const long long t = blockIdx.x - zero_blocks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
  const V* d = static_cast<const V*>(dout) + t * per_row;
  for (int j0 = 0; j0 < top_k; j0 += 4) {
    int r[4];
    float w[4], dot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      r[u] = j < top_k ? row_of_pair[t * top_k + j] : -1;
      if (r[u] >= rows) r[u] = -1;
      w[u] = r[u] >= 0 ? weights[t * top_k + j] : 0.0f;
      dot[u] = 0.0f;
    }
    const V* y0[4];
    V* dy0[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      y0[u] = static_cast<const V*>(Y) + (size_t)max(r[u], 0) * per_row;
      dy0[u] = static_cast<V*>(dY) + (size_t)max(r[u], 0) * per_row;
    }
    for (uint32_t c0 = (uint32_t)tid; c0 < (uint32_t)per_row; c0 += blockDim.x * U) {
      V gv[U], yv[4][U];
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const uint32_t c = c0 + q * blockDim.x;
        if (c >= (uint32_t)per_row) continue;
        gv[q] = d[c];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r[u] >= 0) yv[u][q] = y0[u][c];
      }
#pragma unroll
      for (int q = 0; q < U; ++q) {
        const uint32_t c = c0 + q * blockDim.x;
        if (c >= (uint32_t)per_row) continue;
        float g[N];
        unpack_row<BF16, N>(gv[q], g);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r[u] >= 0) {
            float f[N], o[N];
            unpack_row<BF16, N>(yv[u][q], f);
#pragma unroll
            for (int n = 0; n < N; ++n) {
              dot[u] = fmaf(g[n], f[n], dot[u]);
              o[n] = w[u] * g[n];
            }
            dy0[u][c] = pack_row<BF16, N>(o);
          }
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
