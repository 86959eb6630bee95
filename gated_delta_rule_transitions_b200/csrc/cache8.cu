// Chunk transitions held in 8 bits.
//
// HLA summary page, "Main Findings" (affine-state memory: the per-chunk states replace the
// KV cache) and "Methodology in Plain English" para. 1.  Per closed chunk j and head:
//   A_j ~ a_j I + sA_j QA_j,   B_j ~ sB_j QB_j     (QA, QB: d x d int8 codes)
// a_j is the mean of A_j's diagonal.  A chunk's transition is a decay of the whole state
// plus edits of low rank: its diagonal is some ten times its other entries, and taking the
// diagonal's mean out lets the 254 steps cover the entries that carry the edits.  The
// scales are (largest magnitude) / 127, the codes round to nearest, ties to even, so a
// stored entry is off by at most sA / 2 or sB / 2.  A matrix of zeros has scale 0 and codes
// 0; one that holds an infinity or a NaN has such a scale, so that it does not pass for a
// number.  Half the bytes of the bf16 cache, a quarter of float32.
//
// A CTA per chunk and head reads A and B twice (the second time from L2): the scale has to be
// known before the first code.  Holding the values in registers instead leaves one CTA per SM.
// Measured: 256 chunks of 16 heads, d = 128, bf16: 144 us, 402 MB, 2.8 TB/s, bound by the
// instructions per value (327 us with the values held); a prompt's fill, 5 % of its prefill.
#include "common.cuh"
#include "kernels.cuh"

namespace hla {

namespace {

constexpr int kThreads = 256;

// Sum / largest bits over the CTA, the same value in every thread.
template <typename F>
__device__ __forceinline__ uint32_t block_reduce(uint32_t v, uint32_t* red, F op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t r = red[0];
  for (int k = 1; k < (int)(blockDim.x >> 5); ++k) r = op(r, red[k]);
  return r;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *(const uint4*)p;
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(q[e] << 16);
    x[2 * e + 1] = __uint_as_float(q[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = *(const float4*)p, w = *(const float4*)(p + 4);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float scale) {
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = scale > 0.0f ? max(-127, min(127, __float2int_rn(__fdiv_rn(x[e], scale)))) : 0;
    q[e >> 2] |= ((uint32_t)c & 255u) << (8 * (e & 3));
  }
  return make_uint2(q[0], q[1]);
}

// One chunk's A and B (d x d, row-major) into codes and (a, sA, sB, 0), by the whole CTA.
template <int D, typename Tio>
__device__ void quantise_chunk(const Tio* A, const Tio* B, uint8_t* qa, uint8_t* qb, float4* scales) {
  __shared__ uint32_t red[32];
  const int tid = threadIdx.x, nt = blockDim.x;
  // mean of the diagonal: per-warp butterflies, then the warps in order
  float dsum = 0.0f;
  for (int i = tid; i < D; i += nt) dsum += ldf(A + (long)i * D + i);
  auto fadd = [](uint32_t p, uint32_t q) { return __float_as_uint(__uint_as_float(p) + __uint_as_float(q)); };
  auto umax = [](uint32_t p, uint32_t q) { return max(p, q); };
  const float mean = __uint_as_float(block_reduce(__float_as_uint(dsum), red, fadd)) * (1.0f / D);
  // largest magnitudes, as bits: they order like the values, and a NaN is above them all
  uint32_t ma = 0u, mb = 0u;
  for (int e = tid; e < D * D / 8; e += nt) {
    const int r = e / (D / 8), c = (e % (D / 8)) * 8;
    float x[8], y[8];
    load8(A + (long)e * 8, x);
    load8(B + (long)e * 8, y);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float xa = r == c + u ? x[u] - mean : x[u];
      ma = max(ma, __float_as_uint(fabsf(xa)));
      mb = max(mb, __float_as_uint(fabsf(y[u])));
    }
  }
  const float sA = __fdiv_rn(__uint_as_float(block_reduce(ma, red, umax)), 127.0f);
  const float sB = __fdiv_rn(__uint_as_float(block_reduce(mb, red, umax)), 127.0f);
  for (int e = tid; e < D * D / 8; e += nt) {
    const int r = e / (D / 8), c = (e % (D / 8)) * 8;
    float x[8], y[8];
    load8(A + (long)e * 8, x);
    load8(B + (long)e * 8, y);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (r == c + u) x[u] -= mean;
    ((uint2*)qa)[e] = codes8(x, sA);
    ((uint2*)qb)[e] = codes8(y, sB);
  }
  if (tid == 0) *scales = make_float4(mean, sA, sB, 0.0f);
}

// Prefill hand-off: every complete chunk's transitions from the workspace.
template <int D, typename Tio>
__global__ void __launch_bounds__(kThreads) cache8_fill_kernel(Cache8Args a) {
  const long chunk = blockIdx.x;
  const int i = (int)(chunk % a.Nc);
  const long bh = chunk / a.Nc;
  const long slot = bh * a.max_chunks + i, src = (bh * a.src_stride + i) * (long)D * D;
  quantise_chunk<D, Tio>((const Tio*)a.A + src, (const Tio*)a.Bm + src, (uint8_t*)a.qa + slot * D * D,
                         (uint8_t*)a.qb + slot * D * D, (float4*)a.scales + slot);
}

// Decode close: the transition that a chunk closing this step left in the scratch (one per
// (sequence, head)) into slot n_chunks.  Launched as the transition kernel's programmatic
// dependent; the pool kernel after it waits for this grid, which waits for that one.
template <int D, typename Tio>
__global__ void __launch_bounds__(kThreads) cache8_close_kernel(Cache8Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long bh = blockIdx.x;
  const int b = (int)(bh / a.H);
  if (a.close_m[b] + 1 != a.C) return;
  const int n = a.close_n[b];
  if (n >= a.max_chunks) return;  // cache full (flagged by the pool kernel)
  const long slot = bh * a.max_chunks + n, src = bh * (long)D * D;
  quantise_chunk<D, Tio>((const Tio*)a.A + src, (const Tio*)a.Bm + src, (uint8_t*)a.qa + slot * D * D,
                         (uint8_t*)a.qb + slot * D * D, (float4*)a.scales + slot);
}

template <int D, typename Tio>
cudaError_t launch_c8(const Cache8Args& a, bool close, cudaStream_t s) {
  if (!close) {
    const long blocks = (long)a.B * a.H * a.Nc;
    if (blocks <= 0) return cudaSuccess;
    if (blocks >= (1L << 31)) return cudaErrorNotSupported;
    cache8_fill_kernel<D, Tio><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * a.H));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache8_close_kernel<D, Tio>, a);
}

}  // namespace

cudaError_t launch_cache8(const Cache8Args& a, bool close, cudaStream_t s) {
  if (a.d == 128)
    return a.dtype == HLA_BF16 ? launch_c8<128, __nv_bfloat16>(a, close, s) : launch_c8<128, float>(a, close, s);
  return a.dtype == HLA_BF16 ? launch_c8<64, __nv_bfloat16>(a, close, s) : launch_c8<64, float>(a, close, s);
}

}  // namespace hla
