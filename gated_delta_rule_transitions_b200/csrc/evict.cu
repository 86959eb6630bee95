// Eviction of cached chunks by accumulated gate weight.
//
// HLA summary page, "Methodology in Plain English" para. 4 (chunks with little routing
// weight are left out; leaving a chunk out is exact, it acts as the identity) and "Main
// Findings" (the per-chunk affine states are what a decode cache holds): a cache that has
// reached its budget drops, per (sequence, head), the chunks whose gates have carried the
// least weight so far:
//   mass_j = sum over query tokens t of the gate of t's chunk on chunk j.
// Three kernels:
//   gate_mass_kernel   column sums of a gate matrix, each row weighted by its chunk's tokens;
//   evict_select       one CTA per (sequence, head): the `recent` last chunks stay, the
//                      others compete by (mass descending, index ascending): each chunk's
//                      rank by counting up to 256 of them, else a radix select over the 32 key
//                      bits, 8 at a time; then an ordered compaction;
//   evict_move         moves every per-chunk array to its place.  A thread owns 16 bytes of
//                      the chunk and takes the kept chunks in ascending order; entry i comes
//                      from a chunk kept[i] >= i, and reads run ahead of writes, so the move
//                      is safe in place without any barrier.
// The move is bound by HBM: 16 sequences x 16 heads, 384 of 512 chunks kept, 13.0 GB in 1.97 ms,
// 1.0 of the measured copy rate; in place, where chunks that keep their index stay, 7.6 GB in
// 1.16 ms, 0.99; one sequence of 29 chunks 14.6 us, two launches' latency.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.cuh"

namespace hla {

namespace {

// ---- mass from a gate matrix -----------------------------------------------------------

// One cluster of up to eight CTAs per (sequence, head) and 32 kQ kVec columns: a lane reads kQ
// groups of kVec neighbours of a row (kVec = 4 where rows start on 16 bytes), the cluster's
// warps take the rows in turn (each its own in ascending order), and the warps' sums of a
// column are added in warp order, the other CTAs' through distributed shared memory: the same
// bits every time.  The row split evens out the triangle (a tile's rows go from all to few)
// and leaves work for every SM where heads are few.
constexpr int kMassWarps = 8;

template <int kQ, int kVec>
__global__ void __launch_bounds__(32 * kMassWarps) gate_mass_kernel(
    const float* __restrict__ gates, int N, int ncols, int C, int T, float thr, float* __restrict__ mass,
    long mass_stride) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int step = kMassWarps * ctas;
  constexpr int kCols = 32 * kQ * kVec;
  __shared__ __align__(16) float part[kMassWarps][kCols];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int tiles = (ncols + kCols - 1) / kCols;
  const long heads = gridDim.x / ctas / tiles, bh = blockIdx.x / ctas % heads;
  const int j0 = (int)(blockIdx.x / ctas / heads) * kCols;  // (tiles of many rows start first)
  const float* G = gates + bh * (long)N * N + j0 + kVec * lane;
  float acc[kQ][kVec] = {};
  // rows i > j hold a weight on chunk j; row i stands for the tokens of chunk i
  int i = j0 + 1 + rank * kMassWarps + w;
  for (; i < min(N, j0 + kCols); i += step) {  // rows that meet the diagonal
    const float wt = (float)min(C, T - i * C);
#pragma unroll
    for (int q = 0; q < kQ; ++q)
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        if (j0 + kVec * (32 * q + lane) + v < i) {
          const float g = __ldg(G + (long)i * N + 32 * kVec * q + v);
          if (thr <= 0.0f || g >= thr) acc[q][v] = fmaf(wt, g, acc[q][v]);
        }
  }
  // below it every column of the tile counts (j0 + kCols <= i < N): kRows rows in flight (32 heads
  // of 2048 chunks: 2, 4, 6, 8 rows 55, 51, 58, 76 us; left to the compiler's unrolling 57)
  constexpr int kRows = 4;
  for (; i < N; i += kRows * step) {
    float g[kRows][kQ][kVec];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const float* p = G + (long)(i + r * step) * N + 32 * kVec * q;
        if (i + r * step >= N) break;
        if constexpr (kVec == 4) {
          const float4 f = __ldg((const float4*)p);
          g[r][q][0] = f.x, g[r][q][1] = f.y, g[r][q][2] = f.z, g[r][q][3] = f.w;
        } else {
          g[r][q][0] = __ldg(p);
        }
      }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int t = i + r * step;
      const float wt = (float)min(C, T - t * C);
#pragma unroll
      for (int q = 0; q < kQ; ++q)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          if (t < N && (thr <= 0.0f || g[r][q][v] >= thr)) acc[q][v] = fmaf(wt, g[r][q][v], acc[q][v]);
    }
  }
#pragma unroll
  for (int q = 0; q < kQ; ++q)
#pragma unroll
    for (int v = 0; v < kVec; ++v) part[w][kVec * (32 * q + lane) + v] = acc[q][v];
  cluster.sync();
  // each CTA adds up its share of the columns
  for (int c = rank * (kCols / ctas) + threadIdx.x; c < (rank + 1) * (kCols / ctas); c += 32 * kMassWarps)
    if (j0 + c < ncols) {
      float s = 0.0f;
      for (int r = 0; r < ctas; ++r) {
        const float* p = cluster.map_shared_rank(&part[0][0], r);
#pragma unroll
        for (int k = 0; k < kMassWarps; ++k) s += p[k * kCols + c];
      }
      mass[bh * mass_stride + j0 + c] = s;
    }
  cluster.sync();  // the other CTAs' shared memory stays until it has been read
}

// ---- selection ------------------------------------------------------------------------

constexpr int kSelThreads = 256;

// Order-preserving key of a weight: larger weight, larger key (a NaN counts as no weight).
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.0f);  // -0 counts as +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of `flag` over the CTA's threads, in thread order; total in *sum.
__device__ __forceinline__ int block_prefix(bool flag, int* wsum, int* sum) {
  const unsigned bal = __ballot_sync(0xFFFFFFFFu, flag);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) wsum[w] = __popc(bal);
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kSelThreads / 32; ++k) {
    if (k < w) before += wsum[k];
    all += wsum[k];
  }
  *sum = all;
  return before + __popc(bal & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  // the move's blocks take their places meanwhile (they wait for this grid)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int hist[256];
  __shared__ int wsum[kSelThreads / 32];
  __shared__ int pick[2];  // digit, how many of the wanted lie above it
  const long bh = blockIdx.x;
  const int b = (int)(bh / a.H);
  const int tid = threadIdx.x;
  const int n = max(0, min(a.n_src[b], a.src_chunks));
  int32_t* kept = a.kept + bh * a.keep;
  const float* mass = a.mass + bh * a.src_chunks;
  if (n <= a.keep) {
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int old = n - a.recent;        // chunks that compete
  int want = a.keep - a.recent;        // how many of them stay (< old)
  if (n <= kSelThreads) {
    // one chunk a thread: a chunk's rank is how many come before it
    uint32_t* keys = (uint32_t*)hist;
    const uint32_t mine = tid < old ? mass_key(mass[tid]) : 0u;
    keys[tid] = mine;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < old; ++i) rank += keys[i] > mine || (keys[i] == mine && i < tid);
    const bool stays = tid < n && (tid >= old || rank < want);
    int total;
    const int at = block_prefix(stays, wsum, &total);
    if (stays) kept[at] = tid;
    return;
  }
  // the key of the last one that stays (`prefix`), and how many with that key stay (`want`)
  uint32_t prefix = 0, mask = 0;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < old; j += kSelThreads) {
        const uint32_t key = mass_key(mass[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      // thread = digit 255 - tid: how many keys have a larger one (a prefix over the threads)
      const int mine = hist[255 - tid];
      int above = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, above, o);
        if ((tid & 31) >= o) above += up;
      }
      if ((tid & 31) == 31) wsum[tid >> 5] = above;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kSelThreads / 32 - 1; ++k)
        if (k < (tid >> 5)) above += wsum[k];
      above -= mine;
      if (above < want && above + mine >= want) {
        pick[0] = 255 - tid;
        pick[1] = above;
      }
      __syncthreads();
      prefix |= (uint32_t)pick[0] << shift;
      mask |= 255u << shift;
      want -= pick[1];
      __syncthreads();
    }
  }
  // ascending compaction: larger keys, the first `want` of the equal ones, the recent ones
  int pos = 0, equal_before = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool larger = j >= old && j < n, equal = false;
    if (j < old && a.keep > a.recent) {
      const uint32_t key = mass_key(mass[j]);
      larger = key > prefix;
      equal = key == prefix;
    }
    int eq_total, total;
    const int eq = equal_before + block_prefix(equal, wsum, &eq_total);
    const bool stays = larger || (equal && eq < want);
    const int at = pos + block_prefix(stays, wsum, &total);
    if (stays) kept[at] = j;
    equal_before += eq_total;
    pos += total;
  }
}

// ---- moving ---------------------------------------------------------------------------

constexpr int kMoveThreads = 128;
// Chunks in flight per thread (8, 10, 12, 16: 16 sequences x 16 heads, 384 of 512 kept, 2012, 1995,
// 1971, 1980 us; one sequence, 21 of 29, 15.7, 14.3, 14.5, 18.3).
constexpr int kMoveBatch = 12;

// One 16-byte column of one array, over the kept chunks [i0, i1) in ascending order.
__device__ __forceinline__ void move_column(const uint4* src, uint4* dst, long pitch, const int32_t* kept, int i0,
                                            int i1, bool in_place) {
  for (int i = i0; i < i1; i += kMoveBatch) {
    uint4 r[kMoveBatch];
    int j[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      j[u] = i + u < i1 ? kept[i + u] : -1;
      if (in_place && j[u] == i + u) j[u] = -1;  // already there
      if (j[u] >= 0) r[u] = src[(long)j[u] * pitch];
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (j[u] >= 0) dst[(long)(i + u) * pitch] = r[u];
  }
}

// grid (B H (column blocks + 1), splits of the kept list).  A thread has one 16-byte column of
// the per-chunk arrays or, into another cache, of the open chunk's.  The last block of a
// (sequence, head) finishes it: the weights move with their chunks and the counters change.
// Nothing here but that last step reads the counts (the list ends at its first -1), so it
// may change them.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, unsigned blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long bh = blockIdx.x / (blocks + 1);
  const unsigned blk = blockIdx.x % (blocks + 1);
  const int tid = threadIdx.x;
  const int32_t* kept = a.kept + bh * a.keep;
  if (blk < blocks) {
    const int per = (a.keep + gridDim.y - 1) / gridDim.y;
    const int i0 = min(a.keep, (int)blockIdx.y * per), i1 = min(a.keep, i0 + per);
    long col = (long)blk * kMoveThreads + tid;
    for (int x = 0; x < a.n_arrays; ++x) {
      const long cols = a.chunk_bytes[x] / 16;
      if (col < cols) {
        move_column((const uint4*)a.src[x] + bh * a.src_chunks * cols + col,
                    (uint4*)a.dst[x] + bh * a.dst_chunks * cols + col, cols, kept, i0, i1, a.in_place);
        return;
      }
      col -= cols;
    }
    if (a.in_place || blockIdx.y != 0) return;
    for (int x = 0; x < a.n_open; ++x) {
      const long cols = a.open_bytes[x] / 16;
      if (col < cols) {
        ((uint4*)a.open_dst[x])[bh * cols + col] = ((const uint4*)a.open_src[x])[bh * cols + col];
        return;
      }
      col -= cols;
    }
    return;
  }
  if (blockIdx.y != 0) return;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  if (a.mass_dst != nullptr) {
    const float* src = a.mass + bh * a.src_chunks;
    float* dst = a.mass_dst + bh * a.dst_chunks;
    for (int i0 = 0; i0 < a.keep; i0 += kMoveThreads) {
      const int i = i0 + tid;
      const int j = i < a.keep ? kept[i] : -1;
      const float m = j >= 0 ? src[j] : 0.0f;
      __syncthreads();  // in place: this round's reads before its writes
      if (j >= 0) dst[i] = m;
    }
  }
  if (h == 0 && tid == 0) {
    if (!a.in_place) a.m_dst[b] = a.m_src[b];
    a.n_dst[b] = min(max(0, min(a.n_src[b], a.src_chunks)), a.keep);
  }
}

}  // namespace

cudaError_t launch_gate_mass(const float* gates, int B, int H, int N, int ncols, int C, int T, float thr, float* mass,
                             long mass_stride, cudaStream_t s) {
  const long BH = (long)B * H;
  auto tiles = [&](int cols) { return BH * ((ncols + cols - 1) / cols); };
  // Wide tiles while eight CTAs each reach every SM, else narrow ones; CTAs per tile until they
  // fill the GPU and a warp has at most 64 rows.  (32 heads of 2048 chunks: 49 us with four CTAs,
  // 58 with eight; 256 heads of 512: 35.9 with one, 37.4 with two; 64 heads of 512: 10.3 with
  // four, 14.4 with eight.)
  const int cols = tiles(256) * 8 >= num_sms() ? 256 : 32;
  int ctas = 1;
  while (ctas < 8 && (tiles(cols) * ctas < 2L * num_sms() || N > 64 * kMassWarps * ctas)) ctas *= 2;
  const long blocks = tiles(cols) * ctas;
  if (blocks <= 0) return cudaSuccess;
  if (blocks >= (1L << 31)) return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32 * kMassWarps);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* k = cols == 32 ? gate_mass_kernel<1, 1> : N % 4 == 0 ? gate_mass_kernel<2, 4> : gate_mass_kernel<8, 1>;
  return cudaLaunchKernelEx(&cfg, k, gates, N, ncols, C, T, thr, mass, mass_stride);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const long BH = (long)a.B * a.H;
  long cols = 0;
  for (int x = 0; x < a.n_arrays; ++x) cols += a.chunk_bytes[x] / 16;
  if (!a.in_place)
    for (int x = 0; x < a.n_open; ++x) cols += a.open_bytes[x] / 16;
  const long blocks = (cols + kMoveThreads - 1) / kMoveThreads;
  if (BH * (blocks + 1) >= (1L << 31)) return cudaErrorNotSupported;
  evict_select_kernel<<<(unsigned)BH, kSelThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // into another cache the kept list can be split as well
  unsigned split = 1;
  if (!a.in_place)
    while (blocks * BH * split < 8L * num_sms() && (long)split * 2 * kMoveBatch <= a.keep) split *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(BH * (blocks + 1)), split);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a, (unsigned)blocks);
}

}  // namespace hla
