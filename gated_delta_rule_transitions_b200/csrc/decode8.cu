// Decode step over a chunk cache in 8 bits (A_j ~ a_j I + sA QA, B_j ~ sB QB, int8 codes).
//
// HLA summary page, "Key Contributions" 3 (dynamic autoregressive decoding) and
// "Methodology in Plain English" paras. 3-4.  Same steps as the other decode kernels: append
// the token, sweep the open chunk right to left (x = A_p q, y = B_p q), gate every closed
// chunk, then for active j descending
//   y += g sB (QB x);   x <- (1 - g) x + g (a x + sA (QA x)).
// The chain is bound by HBM where there are enough (sequence, head) pairs: 2 d^2 bytes an
// active chunk, half of bf16's.
//
// The products are whole-number ones.  The running x is held in float32; before each chunk
// it is written as a fixed-point number of 32 bits relative to its largest entry,
//   x_c = 2^(e - 30) N_c,  |N_c| <= 127 x 2^24,  N_c = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3  (signed bytes),
// so that QA x and QB x are four exact dot products of bytes each (32-bit sums: at most
// 128 x 127 x 128 < 2^21).  The only error beside float32's own is the fixed point's half
// unit, some 2^-32 to 2^-31 of the largest entry (2^-127 where that is below 2^-96): an entry
// keeps all its bits down to 2^-6 of the largest.  (With three digits, 24 bits, entries 2^-7
// below came out with a relative error of 1e-5; the fourth is a column that the product has
// to spare.)
//
// decode_stream8_kernel (bf16, d = 128; after decode_gates_kernel): one CTA per (sequence,
// head), two per SM.  The four digit vectors are four columns of one right factor on the
// tensor cores (warp-level 16 x 8 x 32); the matrices go there from shared memory as they lie,
// 16 ldmatrix a warp and chunk, nothing is converted.  (As dp4a a chunk took 1,410
// cycles, 880 of them the products, as they are some 1,100; 64 sequences x 16 heads x 512
// chunks: 2.60 and 2.55 ms, 1.04 of the measured copy rate; 8 x 16 heads with some 90 active
// chunks: 144 and 97 us.  A ring of six units, or x and y on four warps each: no faster.)  A unit of the
// ring is one chunk: 16 KiB of QA, 16 KiB of QB (128 rows of 128 bytes, one 128-byte-swizzled
// box each) and its four scales.  Warp w has rows 32 w .. + 31 of both; lane l owns row
// 32 w + l / 4 + 8 (l % 4) of the vectors.
//
// decode_rows8_kernel (float32, d = 64): one kernel for all steps, the same products on codes
// that all threads bring in by cp.async, a ring of chunks ahead.
#include "common.cuh"
#include "kernels.cuh"
#include "routing_recipe.cuh"
#include "tc_common.cuh"

namespace hla {

HLA_DEFINE_ERROR_WORD(decode8)

cudaError_t make_tmap_2d(CUtensorMap* m, const void* base, long inner, long rows, long row_stride_bytes,
                         int box_inner, int box_rows);

namespace {

constexpr int kD = 128;
constexpr int kCompute = 128;
constexpr int kThreads = kCompute + 32;
constexpr int kU8Tile = kD * kD;                    // 16 KiB of codes
constexpr int kU8Unit = 2 * kU8Tile;                // 32 KiB
constexpr int kU8Units = 3;
constexpr uint32_t kU8Tx = kU8Unit + 16;
constexpr int kDigits = kD + 32;                    // pitch of a digit vector: four on 32 banks
constexpr int kU8Vec = 4 * kDigits;                 // digits of one x

// x (this thread's row) as digits; returns the unit 2^(e - 30).  The digits of a zero x are zero;
// one with an infinity or a NaN has unit NaN.  Contains one barrier.
__device__ __forceinline__ float write_digits(float x, int row, uint32_t* mx, uint8_t* xd) {
  const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x) & 0x7FFFFFFFu);
  if ((threadIdx.x & 31) == 0) mx[threadIdx.x >> 5] = m;
  tc::bar_sync(1, kCompute);
  const uint4 m4 = *(const uint4*)mx;
  const uint32_t big = max(max(m4.x, m4.y), max(m4.z, m4.w));
  // |x| < 127/128 2^(e + 1), so that the last digit stays a signed byte; below 2^-96 the fixed
  // point stays where it is
  const int e = max((int)((big + 0x20000u) >> 23) - 127, -96);
  const float up = __uint_as_float((uint32_t)(127 + 30 - e) << 23);
  const int n = __float2int_rn(x * up);
  const int d0 = (int)(int8_t)n;
  const int n1 = (n - d0) >> 8;
  const int d1 = (int)(int8_t)n1;
  const int n2 = (n1 - d1) >> 8;
  const int d2 = (int)(int8_t)n2;
  xd[row] = (uint8_t)d0;
  xd[kDigits + row] = (uint8_t)d1;
  xd[2 * kDigits + row] = (uint8_t)d2;
  xd[3 * kDigits + row] = (uint8_t)((n2 - d2) >> 8);
  if (big >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((uint32_t)(127 - 30 + e) << 23);
}

// Two digits' sums joined (below 2^30); the other two lie in the neighbouring lane.
__device__ __forceinline__ float join2(int lo, int hi) { return (float)(lo + 256 * hi); }
__device__ __forceinline__ float join4(float lo) {
  return fmaf(__shfl_xor_sync(0xFFFFFFFFu, lo, 1), 65536.0f, lo);
}

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Raw 16-byte words of kN values as float pairs.
template <int kN>
__device__ __forceinline__ void to_pairs(const uint4 (&w)[kN / 8], const __nv_bfloat16*, float2 (&x)[kN / 2]) {
#pragma unroll
  for (int i = 0; i < kN / 8; ++i) {
    x[4 * i] = tc::bf16x2_to_float2(w[i].x);
    x[4 * i + 1] = tc::bf16x2_to_float2(w[i].y);
    x[4 * i + 2] = tc::bf16x2_to_float2(w[i].z);
    x[4 * i + 3] = tc::bf16x2_to_float2(w[i].w);
  }
}
template <int kN>
__device__ __forceinline__ void to_pairs(const uint4 (&w)[kN / 4], const float*, float2 (&x)[kN / 2]) {
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    x[2 * i] = make_float2(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
    x[2 * i + 1] = make_float2(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
  }
}

// The open chunk right to left by one warp: x = A_p q and y = B_p q into shared memory.
//   c = k_t . x;  y += beta_t c v_t;  x <- alpha_t (x - beta_t c k_t)
// Lane l has the D / 8 channels from D / 8 (l % 8) of x (four copies, so that a dot product is
// three shuffles) and the D / 32 channels from D / 32 l of y; the rows of the tokens to come
// are on their way while these are worked on.  The step's own token (t = m) is read from the
// call's arguments, so that the sweep need not wait for its place in the open chunk.
template <int D, typename Tio, bool kChan>
__device__ __forceinline__ void sweep_warp(const DecodeArgs& a, int bh, int m, float* xs, float* ys) {
  constexpr int E = D / 8, F = D / 32;
  constexpr int W = E * (int)sizeof(Tio) / 16;  // 16-byte words of a lane's keys
  constexpr int kAhead = kChan || sizeof(Tio) == 4 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const int g = lane & 7;
  const long tok = (long)bh * D, buf = (long)bh * a.C * D;
  struct Row {
    uint4 k[W];
    float4 al[kChan ? E / 4 : 1];
    Tio v[F];
    float b;
  };
  float2 x[E / 2];
  float y[F] = {};
  {
    uint4 w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = ((const uint4*)((const Tio*)a.q + (long)bh * D + E * g))[i];
    to_pairs<E>(w, (const Tio*)nullptr, x);
  }
  Row next[kAhead];
  auto load = [&](int t, Row& r) {  // token t (nothing before the first)
    if (t < 0) return;
    const bool own = t == m;
    const long at = buf + (long)t * D, one = (long)bh * a.C + t;
    const Tio* k = (own ? (const Tio*)a.k + tok : (const Tio*)a.buf_k + at) + E * g;
    const Tio* v = (own ? (const Tio*)a.v + tok : (const Tio*)a.buf_v + at) + F * lane;
#pragma unroll
    for (int i = 0; i < W; ++i) r.k[i] = ((const uint4*)k)[i];
    if constexpr (kChan) {
      const float* al = (own ? a.alpha + tok : a.buf_alpha + at) + E * g;
#pragma unroll
      for (int i = 0; i < E / 4; ++i) r.al[i] = ((const float4*)al)[i];
    } else {
      r.al[0].x = own ? a.alpha[bh] : a.buf_alpha[one];
    }
#pragma unroll
    for (int i = 0; i < F; ++i) r.v[i] = v[i];
    r.b = own ? a.beta[bh] : a.buf_beta[one];
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(m - i, next[i]);
  for (int t0 = m; t0 >= 0; t0 -= kAhead) {
    Row cur[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      cur[i] = next[i];
      load(t0 - kAhead - i, next[i]);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t0 - i < 0) break;
      float2 k[E / 2];
      to_pairs<E>(cur[i].k, (const Tio*)nullptr, k);
      float2 d0 = make_float2(0.0f, 0.0f), d1 = d0;
#pragma unroll
      for (int e = 0; e < E / 2; e += 2) {
        d0 = tc::fma2(x[e], k[e], d0);
        d1 = tc::fma2(x[e + 1], k[e + 1], d1);
      }
      float c = (d0.x + d0.y) + (d1.x + d1.y);
      c += __shfl_xor_sync(0xFFFFFFFFu, c, 1);
      c += __shfl_xor_sync(0xFFFFFFFFu, c, 2);
      c += __shfl_xor_sync(0xFFFFFFFFu, c, 4);
      c *= cur[i].b;
#pragma unroll
      for (int f = 0; f < F; ++f) y[f] = fmaf(c, ldf(&cur[i].v[f]), y[f]);
      const float2 nc = make_float2(-c, -c);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        float2 al = make_float2(cur[i].al[0].x, cur[i].al[0].x);
        if constexpr (kChan) {
          const float4 w = cur[i].al[e >> 1];
          al = (e & 1) ? make_float2(w.z, w.w) : make_float2(w.x, w.y);
        }
        x[e] = tc::mul2(al, tc::fma2(nc, k[e], x[e]));
      }
    }
  }
  if (lane < 8) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) *(float2*)(xs + E * g + 2 * e) = x[e];
  }
#pragma unroll
  for (int f = 0; f < F; ++f) ys[F * lane + f] = y[f];
}

__global__ void __launch_bounds__(kThreads, 2)
    decode_stream8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          DecodeArgs a) {
  // launched as the gate kernel's programmatic dependent, early: the open chunk (but for the
  // step's own token, an argument) and the counters are not that kernel's, so the sweep runs
  // beside it; what it writes (the lists) is read after the wait
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float4* sc_s = (float4*)(ring + kU8Units * kU8Unit);  // [kU8Units] a, sA, sB, 0
  uint8_t* xd = (uint8_t*)(sc_s + kU8Units);             // [2][3][kDigits] digits of x
  uint32_t* mx = (uint32_t*)(xd + 2 * kU8Vec);           // [2][4]
  uint64_t* full = (uint64_t*)(mx + 8);
  uint64_t* empty = full + kU8Units;
  float* xs = (float*)(empty + kU8Units);    // [kD] x after the open chunk
  float* ys = xs + kD;                       // [kD] y of the open chunk
  volatile int* abort_s = (volatile int*)(ys + kD);

  const int bh = blockIdx.x;
  const int b = bh / a.H;
  const int tid = threadIdx.x;
  const int m = a.m_partial[b];
  const int32_t* act_idx = a.act_idx + (long)bh * a.max_chunks;
  const float* act_g = a.act_g + (long)bh * a.max_chunks;

  if (tid == 0) {
    for (int u = 0; u < kU8Units; ++u) {
      tc::mbar_init(&full[u], 1);
      tc::mbar_init(&empty[u], 1);
    }
    *abort_s = 0;
    tc::mbar_fence_init();
    tc::fence_async_smem();
  }
  __syncthreads();

  if (tid >= kCompute) {
    // ---------------- TMA producer (warp 4, lane 0): one unit per active chunk ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cnt = a.act_cnt[bh];
    if (tid == kCompute && cnt > 0) {
      tc::tma_prefetch_desc(&tmA);
      tc::tma_prefetch_desc(&tmB);
      int u = 0;
      for (int p = cnt - 1; p >= 0; --p, ++u) {
        const int st = u % kU8Units;
        const long slot = (long)bh * a.max_chunks + act_idx[p];
        if (u >= kU8Units && !tc::mbar_wait(&empty[st], ((u / kU8Units) - 1) & 1, abort_s)) break;
        const int row = (int)(slot * kD);
        tc::mbar_arrive_expect_tx(&full[st], kU8Tx);
        uint8_t* dst = ring + st * kU8Unit;
        tc::tma_load_2d(dst, &tmA, 0, row, &full[st]);
        tc::tma_load_2d(dst + kU8Tile, &tmB, 0, row, &full[st]);
        tc::bulk_load_1d(sc_s + st, a.df + slot * 4, 16, &full[st]);
      }
      if (*abort_s)
        for (int t = max(0, u - kU8Units); t < u; ++t)
          tc::mbar_wait(&full[t % kU8Units], (t / kU8Units) & 1, nullptr, 200000000ull);
    }
    __syncwarp();
  } else {
    // ---------------- compute (warps 0-3) ----------------
    const int warp = tid >> 5, lane = tid & 31;
    const int row = 32 * warp + (lane >> 2) + 8 * (lane & 3);  // this thread's row of x and y
    if (warp == 0) {
      if (a.alpha_vec)
        sweep_warp<kD, __nv_bfloat16, true>(a, bh, m, xs, ys);
      else
        sweep_warp<kD, __nv_bfloat16, false>(a, bh, m, xs, ys);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int cnt = a.act_cnt[bh];
    tc::bar_sync(1, kCompute);
    float x = xs[row], y = 0.0f;
    float g = cnt > 0 ? act_g[cnt - 1] : 0.0f;
    float unit = write_digits(x, row, mx, xd);
    // ldmatrix addresses: lane l gives row l % 16 of a 16-row tile, 16-byte piece l / 16 of a
    // 32-byte step; the swizzle of a row is l % 8 in every tile
    const uint32_t mrow = tc::smem_u32(ring) + (32 * warp + (lane & 15)) * 128;
    const int mpiece = lane >> 4, mswz = lane & 7;
    const int dcol = lane >> 2;  // digit vector of this lane's part of the right factor
    for (int p = cnt - 1, u = 0; p >= 0; --p, ++u) {
      const int st = u % kU8Units;
      const uint8_t* xc = xd + (u & 1) * kU8Vec + dcol * kDigits + 4 * (lane & 3);
      const float g_next = p > 0 ? act_g[p - 1] : 0.0f;
      if (!tc::bar_all(1, kCompute, tc::mbar_wait(&full[st], (u / kU8Units) & 1, abort_s))) break;
      uint32_t xb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) xb[e] = dcol < 4 ? *(const uint32_t*)(xc + 16 * e) : 0u;
      int acc[4][4] = {};  // QA rows 0-15, 16-31, QB rows 0-15, 16-31 of this warp's
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t at = mrow + st * kU8Unit + (((2 * ks + mpiece) ^ mswz) << 4);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t f[4];
          ldmatrix4(at + (t >> 1) * kU8Tile + (t & 1) * 2048, f);
          mma_s8(acc[t], f, xb[2 * ks], xb[2 * ks + 1]);
        }
      }
      // columns 0, 1 of a row are in lane 4 (row % 8), 2 and 3 in the lane after it: join the
      // digits there, then hand row 8 j + l / 4 to the lane with l % 4 = j
      float sa = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = j >> 1, c = 2 * (j & 1);
        float va = join4(join2(acc[t][c], acc[t][c + 1]));
        float vb = join4(join2(acc[2 + t][c], acc[2 + t][c + 1]));
        va = __shfl_sync(0xFFFFFFFFu, va, lane & 28);
        vb = __shfl_sync(0xFFFFFFFFu, vb, lane & 28);
        if ((lane & 3) == j) {
          sa = va;
          sb = vb;
        }
      }
      const float4 sc = sc_s[st];
      y = fmaf(g * sc.z, sb * unit, y);
      x = fmaf(1.0f - g, x, g * fmaf(sc.x, x, sc.y * (sa * unit)));
      g = g_next;
      // the digits of the new x; the barrier inside also says that this unit has been read
      unit = write_digits(x, row, mx + 4 * ((u + 1) & 1), xd + ((u + 1) & 1) * kU8Vec);
      if (tid == 0) tc::mbar_arrive(&empty[st]);
    }
    stf((__nv_bfloat16*)a.o + (long)bh * kD + row, y + ys[row]);
  }
  __syncthreads();
  if (tid == 0 && *abort_s) report_device_error(kErrMbarTimeout);
}

// ---- float32, or d = 64 ------------------------------------------------------------------
//
// One CTA of 4 warps per (sequence, head).  Warp 0 sweeps the open chunk while the other three
// pool the route queries and gate the closed chunks; then the chain.  Warp w has the rows
// D / 4 w .. of both matrices; of d = 64 a lane's row of the vectors is its neighbour's too.
template <int D>
constexpr int rows8_stages() { return D == 64 ? 6 : 3; }

// Byte of 16-byte piece `piece` of row r of a matrix in shared memory: pieces turned within
// 128 bytes, so that eight rows' pieces lie in eight bank groups.
template <int D>
__device__ __forceinline__ int code_at(int r, int piece) {
  return r * D + ((D == 128 ? piece ^ (r & 7) : piece ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

template <int D, typename Tio>
__global__ void __launch_bounds__(kCompute) decode_rows8_kernel(DecodeArgs a) {
  constexpr int kTiles = D / 64;               // 16-row tiles per warp and matrix
  constexpr int kMat = D * D;                  // bytes of one matrix
  constexpr int kPieces = D / 16;              // 16-byte pieces of a row
  constexpr int kGate = 96;                    // threads that pool and gate
  constexpr int kStages = rows8_stages<D>();
  extern __shared__ __align__(128) uint8_t ring[];  // [kStages][QA | QB]
  __shared__ __align__(16) float4 sc_s[kStages];
  __shared__ float g_s[kStages];
  __shared__ __align__(16) float xs[D], ys[D], rq[D];
  __shared__ __align__(16) uint8_t xd[2 * kU8Vec];
  __shared__ __align__(16) uint32_t mx[8];
  __shared__ int wcount[3];
  __shared__ int cnt_s;
  const int bh = blockIdx.x;
  const int b = bh / a.H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.C;
  const int n = a.n_chunks[b];
  const int m = a.m_partial[b];
  int32_t* act_idx = a.act_idx + (long)bh * a.max_chunks;
  float* act_g = a.act_g + (long)bh * a.max_chunks;
  // append the token to the open chunk
  const Tio* qr_in = (const Tio*)(a.q_route ? a.q_route : a.q);
  const Tio* kr_in = (const Tio*)(a.k_route ? a.k_route : a.k);
  if (tid < D) {
    const long tok = (long)bh * D + tid, slot = ((long)bh * C + m) * D + tid;
    ((Tio*)a.buf_k)[slot] = ((const Tio*)a.k)[tok];
    ((Tio*)a.buf_v)[slot] = ((const Tio*)a.v)[tok];
    ((Tio*)a.buf_qr)[slot] = qr_in[tok];
    ((Tio*)a.buf_kr)[slot] = kr_in[tok];
    if (a.alpha_vec) a.buf_alpha[slot] = a.alpha[tok];
  }
  if (tid == 0) {
    if (!a.alpha_vec) a.buf_alpha[(long)bh * C + m] = a.alpha[bh];
    a.buf_beta[(long)bh * C + m] = a.beta[bh];
    cnt_s = 0;
  }
  __syncthreads();
  if (warp == 0) {
    if (a.alpha_vec)
      sweep_warp<D, Tio, true>(a, bh, m, xs, ys);
    else
      sweep_warp<D, Tio, false>(a, bh, m, xs, ys);
  } else if (a.mode != HLA_GATES_ZERO && n > 0) {
    const int t96 = tid - 32;
    const route::Consts K = route::make_consts();
    if (a.mode == HLA_GATES_ROUTED) {
      // query pool over the open chunk's m + 1 route tokens
      const float inv_tau = __fdiv_rn(1.0f, a.tau);
      for (int c = t96; c < D; c += kGate) {
        const Tio* bq = (const Tio*)a.buf_qr + (long)bh * C * D + c;
        float top = __fmul_rn(ldf(bq), inv_tau);
#pragma unroll 8
        for (int t = 1; t <= m; ++t) top = fmaxf(top, __fmul_rn(ldf(bq + (long)t * D), inv_tau));
        float s = 0.0f;
#pragma unroll 8
        for (int t = 0; t <= m; ++t)
          s = __fadd_rn(s, route::rexp(route::pool_shift(ldf(bq + (long)t * D), inv_tau, top), K));
        rq[c] = __fmul_rn(a.tau, __fadd_rn(top, route::rlog(__fdiv_rn(s, (float)(m + 1)), K)));
      }
      tc::bar_sync(2, kGate);
    }
    const int W = a.win > 0 ? a.win : 1;
    const float* rk = a.rk + (long)bh * a.max_chunks * W * D;
    int cnt = 0;
    for (int jb = 0; jb < n; jb += kGate) {
      const int j = jb + t96;
      float g = 1.0f;
      bool keep = false;
      if (j < n) {
        if (a.mode == HLA_GATES_ROUTED && a.win > 0) {
          // log-sum-exp over the closed chunk's window representatives
          float t[kMaxWindows];
          const float top = route::window_scores(rq, rk + (long)j * W * D, a.win, D, a.c_d, t);
          g = route::gate_from_window_scores(t, a.win, top, a.bias, K);
        } else if (a.mode == HLA_GATES_ROUTED) {
          const float4* rkj = (const float4*)(rk + (long)j * D);
          float dot = 0.0f;
#pragma unroll 8
          for (int c4 = 0; c4 < D / 4; ++c4) {
            const float4 r4 = rkj[c4];
            dot = route::dot_step(dot, rq[4 * c4 + 0], r4.x);
            dot = route::dot_step(dot, rq[4 * c4 + 1], r4.y);
            dot = route::dot_step(dot, rq[4 * c4 + 2], r4.z);
            dot = route::dot_step(dot, rq[4 * c4 + 3], r4.w);
          }
          g = route::gate_from_dot(dot, a.c_d, a.bias, K);
        }
        keep = a.thr <= 0.0f || g >= a.thr;
      }
      const unsigned int bal = __ballot_sync(0xFFFFFFFFu, keep);
      if (lane == 0) wcount[warp - 1] = __popc(bal);
      tc::bar_sync(2, kGate);
      int before = 0, total = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k < warp - 1) before += wcount[k];
        total += wcount[k];
      }
      if (keep) {
        const int pos = cnt + before + __popc(bal & ((1u << lane) - 1u));
        act_idx[pos] = j;
        act_g[pos] = g;
        if (a.mass != nullptr) a.mass[(long)bh * a.max_chunks + j] += g;
      }
      cnt += total;
      tc::bar_sync(2, kGate);
    }
    if (t96 == 0) cnt_s = cnt;
  }
  __syncthreads();
  // the chain
  const int cnt = cnt_s;
  const int own = kTiles == 2 ? lane & 3 : lane & 1;  // 8-row block of this lane's row
  const int row = D / 4 * warp + (lane >> 2) + 8 * own;
  const uint8_t* A = (const uint8_t*)a.A + (long)bh * a.max_chunks * kMat;
  const uint8_t* Bm = (const uint8_t*)a.Bm + (long)bh * a.max_chunks * kMat;
  int j_next = cnt > 0 ? act_idx[cnt - 1] : 0;  // list entries come a round before their chunk
  auto issue = [&](int p, int st) {
    if (p >= 0) {
      const int j = j_next;
      if (p > 0) j_next = act_idx[p - 1];
      uint8_t* dst = ring + st * 2 * kMat;
#pragma unroll
      for (int i = 0; i < kMat / 16 / kCompute; ++i) {
        const int e = tid + i * kCompute, at = code_at<D>(e / kPieces, e % kPieces);
        cp16(dst + at, A + (long)j * kMat + 16 * e);
        cp16(dst + kMat + at, Bm + (long)j * kMat + 16 * e);
      }
      if (tid == 0) {
        cp16(&sc_s[st], a.df + ((long)bh * a.max_chunks + j) * 4);
        g_s[st] = act_g[p];
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < kStages - 1; ++i) issue(cnt - 1 - i, i);
  float x = xs[row], y = 0.0f;
  float unit = write_digits(x, row, mx, xd);
  const int dcol = lane >> 2;
  for (int p = cnt - 1, u = 0; p >= 0; --p, ++u) {
    const int st = u % kStages;
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    tc::bar_sync(1, kCompute);  // the digits and every thread's share of the chunk are there
    // the stage of the chunk before (read by all before the barrier in write_digits)
    issue(p - (kStages - 1), (u + kStages - 1) % kStages);
    const uint8_t* xc = xd + (u & 1) * kU8Vec + dcol * kDigits + 4 * (lane & 3);
    const uint32_t at = tc::smem_u32(ring) + st * 2 * kMat;
    int acc[2 * kTiles][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) {
      const uint32_t x0 = dcol < 4 ? *(const uint32_t*)(xc + 32 * ks) : 0u;
      const uint32_t x1 = dcol < 4 ? *(const uint32_t*)(xc + 32 * ks + 16) : 0u;
#pragma unroll
      for (int t = 0; t < 2 * kTiles; ++t) {
        uint32_t f[4];
        const int r = D / 4 * warp + 16 * (t % kTiles) + (lane & 15);
        ldmatrix4(at + (t / kTiles) * kMat + code_at<D>(r, 2 * ks + (lane >> 4)), f);
        mma_s8(acc[t], f, x0, x1);
      }
    }
    float sa = 0.0f, sb = 0.0f;
#pragma unroll
    for (int k = 0; k < 2 * kTiles; ++k) {  // as in decode_stream8_kernel
      const int t = k >> 1, c = 2 * (k & 1);
      float va = join4(join2(acc[t][c], acc[t][c + 1]));
      float vb = join4(join2(acc[kTiles + t][c], acc[kTiles + t][c + 1]));
      va = __shfl_sync(0xFFFFFFFFu, va, lane & 28);
      vb = __shfl_sync(0xFFFFFFFFu, vb, lane & 28);
      if (own == k) {
        sa = va;
        sb = vb;
      }
    }
    const float g = g_s[st];
    const float4 sc = sc_s[st];
    y = fmaf(g * sc.z, sb * unit, y);
    x = fmaf(1.0f - g, x, g * fmaf(sc.x, x, sc.y * (sa * unit)));
    unit = write_digits(x, row, mx + 4 * ((u + 1) & 1), xd + ((u + 1) & 1) * kU8Vec);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  stf((Tio*)a.o + (long)bh * D + row, y + ys[row]);
}

template <int D, typename Tio>
cudaError_t launch_rows8(const DecodeArgs& a, cudaStream_t s) {
  const int smem = rows8_stages<D>() * 2 * D * D;
  cudaError_t e = cudaFuncSetAttribute(decode_rows8_kernel<D, Tio>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  decode_rows8_kernel<D, Tio><<<a.B * a.H, kCompute, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode8(const DecodeArgs& a, cudaStream_t s) {
  if (a.d == 64) return a.dtype == HLA_BF16 ? launch_rows8<64, __nv_bfloat16>(a, s) : launch_rows8<64, float>(a, s);
  if (a.dtype != HLA_BF16) return launch_rows8<128, float>(a, s);
  const long rows = (long)a.B * a.H * a.max_chunks * kD;
  if (rows >= (1L << 31)) return cudaErrorNotSupported;  // tile coordinates are 32-bit
  // a row of 128 codes as 64 two-byte elements
  CUtensorMap tmA, tmB;
  cudaError_t e = make_tmap_2d(&tmA, a.A, kD / 2, rows, kD, kD / 2, kD);
  if (e == cudaSuccess) e = make_tmap_2d(&tmB, a.Bm, kD / 2, rows, kD, kD / 2, kD);
  if (e == cudaSuccess) e = launch_decode_gates(a, s);
  if (e != cudaSuccess) return e;
  const size_t smem = 1024 + kU8Units * (kU8Unit + 16) + 2 * kU8Vec + 32 + 2 * kU8Units * 8 + 2 * kD * 4 + 16;
  e = cudaFuncSetAttribute(decode_stream8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * a.H);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_stream8_kernel, tmA, tmB, a);
}

}  // namespace hla
