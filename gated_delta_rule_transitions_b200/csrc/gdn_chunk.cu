// The gated delta rule by chunks of 64 tokens on tcgen05 tensor cores (bf16, d = 128, one
// decay per head), ragged sequences, float32 state in and out.
//
// HLA summary page, "Methodology in Plain English" para. 1 (the per-token rule; affine maps
// compose); chunkwise WY/UT form (the chunkwise WY algorithm named in the Gated DeltaNet-2
// abstract on the HLA listing page).  Per chunk, with l_t = sum_{s<=t} log alpha_s,
// gamma_t = e^{l_t}, Gamma_ts = e^{l_t - l_s}:
//   L = strictly-lower(diag(beta) (Gamma o K K^T)),  T = (I + L)^{-1} diag(beta),
//   G = tril(Gamma o Q K^T) T                                     (gdn_wy_kernel)
//   R = V - diag(gamma) K S^T,  U = T R,  O = diag(gamma) Q S^T + G R,
//   S <- gamma_C S + U^T diag(gamma_C / gamma_t) K                 (gdn_scan_kernel)
// T and G do not depend on the state: gdn_wy_kernel makes them for every chunk at once.
// gdn_scan_kernel then walks the chunks of one (sequence, head) and 16, 32 or 64 of its value
// columns, three products a chunk, each waiting for the one before.
//
// What bounds it: the scan's chain of a chunk, 1.7 us with 16 columns and 3.5 with 64 (there
// shared memory's bandwidth as well); the tensor cores are active 16 % of the time.
// Measured, 16 heads: 16384 tokens of one sequence 532 us (T and G 96, the scan 443),
// four sequences of 4096 tokens 319 us (99 and 224).
//
// Precision.  The state is float32 and stays so: it is held in registers, and what goes into
// a product (S, R, U, T) goes in as three bf16 numbers, x = x1 + x2 + x3, each the eight bits
// after the one before: exactly x (two would leave 2^-16 of it out, more than float32 sums
// do).  K, Q and V are bf16 already.  Left out are the products of parts that are 2^-22 and
// less.  T and G are made of products of two tf32 numbers a factor (off by 2^-20).  G goes in as
// three parts too, and the output sums all three of S: made of single tf32 factors, in two parts
// each, it was off by 2^-12 before its own rounding and by 8e-4 of its size after it.  Decays are
// differences of 64-bit running sums of float32 logarithms: log alpha is off by 2^-24 of itself,
// so a decay e^l by at most |l| e^l 2^-24 < 2^-25.
//
// NaN and infinities.  The entries of T and G above the diagonal are zeros that are multiplied all
// the same, so a token that is no number would spoil the 63 before it.  Therefore: gdn_wy_kernel
// keeps T and G finite and writes an undefined gamma from the first token on whose key, decay or
// beta is none; gdn_scan_kernel takes such tokens, and values that are none, as zeros, and makes
// undefined what they reach.  (A bad query has a row of its own.  The checks cost 2 %: 16384
// tokens 524 -> 534 us.)
#include <climits>

#include "common.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace hla {

HLA_DEFINE_ERROR_WORD(gdn_chunk)

cudaError_t make_tmap_2d(CUtensorMap* m, const void* base, long inner, long rows, long row_stride_bytes,
                         int box_inner, int box_rows);

namespace {

constexpr int kD = 128;
constexpr int kC = 64;
constexpr int kTile = kC * 128;               // 8 KiB: 64 rows of 128 bytes, 128-byte swizzle
constexpr int kWy = 6 * kTile;                // [T1; G1], [T2; G2], [T3; G3] of a chunk, as they lie in shared memory
constexpr int kScal = 2 * kC * 4;             // gamma_t, gamma_C / gamma_t
constexpr int kSlot = kWy + kScal;            // workspace bytes per (chunk slot, head)

// Rows of a stacked left factor [X; Y] (64 rows each): 16 of X, 16 of Y, and so on, so that each
// quarter of tensor memory's lanes (one warp's reach) gets 16 rows of either product and no
// warp is without work in any step.  Row of X's row t (Y's is 16 further on):
__device__ __forceinline__ int stacked(int t) { return 32 * (t >> 4) + (t & 15); }

__device__ __forceinline__ int swz(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// Chunk slots.  Sequence s owns the slots first_slot(s) + c, c < ceil(len / 64): they never meet
// the next sequence's, so no prefix sum over the lengths is needed.  cu[s] / 64 + s is such a
// numbering (T / 64 + n_seq slots); where sequences of 32 tokens and less go by rows and need
// none, so is cu[s] / 32 (T / 32 + 1 slots).  The owner of a slot is the last sequence whose
// first slot is not above it.
__device__ __forceinline__ int first_slot(const GdnArgs& a, int seq) {
  return a.half_slots ? a.cu[seq] / (kC / 2) : a.cu[seq] / kC + seq;
}
__device__ __forceinline__ int slot_owner(const GdnArgs& a, int slot) {
  int lo = 0, hi = a.n_seq;  // owner in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_slot(a, mid) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ bool good_bounds(int t0, int t1, int T) { return t0 >= 0 && t1 >= t0 && t1 <= T; }

// The two neighbours' next eight bits each: packed, and what is left of x.
__device__ __forceinline__ uint32_t cut(float2& x) {
  const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
  x.x -= __uint_as_float(a & 0xFFFF0000u);
  x.y -= __uint_as_float(b & 0xFFFF0000u);
  return __byte_perm(a, b, 0x7632);
}
// Two neighbours as three bf16 parts by cutting: exactly x, 8 bits each.
__device__ __forceinline__ void cut3(float a, float b, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
  float2 x = make_float2(a, b);
  p1 = cut(x);
  p2 = cut(x);
  p3 = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}

// Waits for this thread's tensor-memory loads; the registers are operands, so that no use of
// them is scheduled before the wait.
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// ---- T and G of every chunk ------------------------------------------------------------

constexpr int kP = kC + 4;                    // row pitch (floats): 16-byte rows
constexpr int kMat = kC * kP * 4;             // one 64 x 64 float32 matrix
constexpr int kWyQK = 0;                      // [kb][Q | K][64 rows][128 B]; once they are multiplied:
constexpr int kWyL = 0;                       //   L, then L' (off the diagonal blocks), then P, then G
constexpr int kWyU = kMat;                    //   (I + L)^{-1}
constexpr int kWySmall = 2 * kMat;
constexpr int kWySmem = kWySmall + kC * 8 + 3 * kC * 4 + 2 * 8 + 40;
static_assert(2 * kMat >= 4 * kTile, "the tiles fit under L and U");
constexpr uint32_t kIdescWy = tc::idesc_bf16_f32(128, 64, 0, 0);
constexpr float kProductRange = 40.0f;

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// x as two tf32 numbers, cut (the instruction does not read the last 13 bits): off by 2^-21.
__device__ __forceinline__ void cut_tf32(float x, uint32_t& h, uint32_t& l) {
  h = __float_as_uint(x) & 0xFFFFE000u;
  l = __float_as_uint(x - __uint_as_float(h));
}

// acc[j] += A (16 x 16) B (16 x 8 kN)'s column tile j, float32 in shared memory (row pitches
// pa, pb), of two tf32 numbers a factor.
template <int kN>
__device__ __forceinline__ void block16(float (&acc)[kN][4], const float* A, int pa, const float* B, int pb,
                                        int lane) {
  const int g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int k0 = 0; k0 < 16; k0 += 8) {
    const float a[4] = {A[g * pa + k0 + q], A[(g + 8) * pa + k0 + q], A[g * pa + k0 + q + 4],
                        A[(g + 8) * pa + k0 + q + 4]};
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cut_tf32(a[i], ah[i], al[i]);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const float b[2] = {B[(k0 + q) * pb + 8 * j + g], B[(k0 + q + 4) * pb + 8 * j + g]};
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        cut_tf32(b[i], bh[i], bl[i]);
      mma_tf32(acc[j], ah, bl);
      mma_tf32(acc[j], al, bh);
      mma_tf32(acc[j], ah, bh);
    }
  }
}

__device__ __forceinline__ void store16(float* D, int pd, const float (&acc)[4], float s, int lane) {
  const int g = lane >> 2, q = lane & 3;
  *(float2*)(D + g * pd + 2 * q) = make_float2(s * acc[0], s * acc[1]);
  *(float2*)(D + (g + 8) * pd + 2 * q) = make_float2(s * acc[2], s * acc[3]);
}

// e^x of a 64-bit exponent, to float32's last bits.
__device__ __forceinline__ float exp64(double x) {
  const float h = (float)x;
  const float e = expf(h);
  return fmaf(e, (float)(x - (double)h), e);
}

// One CTA (4 warps) per (chunk slot, head), five per SM.  Q K^T stays in tensor memory until L'
// has been used, so that one buffer serves L and P.
__global__ void __launch_bounds__(128, 5)
    gdn_wy_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, GdnArgs a,
                  uint8_t* ws) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  float* Ls = (float*)(sm + kWyL);
  float* Us = (float*)(sm + kWyU);
  double* ell = (double*)(sm + kWySmall);
  float* beta_s = (float*)(ell + kC);
  float* gam = beta_s + kC;
  float* igam = gam + kC;
  uint64_t* bars = (uint64_t*)(igam + kC);      // tma, mma
  double* wsum = (double*)(bars + 2);
  uint32_t* lmax = (uint32_t*)(wsum + 1);       // [2]
  uint32_t* tmem_s = lmax + 2;
  volatile int* abort_s = (volatile int*)(tmem_s + 1);
  int* bad_s = (int*)tmem_s + 2;                // first token whose products with keys are no numbers

  // gdn_scan_kernel's blocks may take their places while this grid drains
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % a.H;
  const int slot = blockIdx.x / a.H;
  const int seq = slot_owner(a, slot);
  const int s0 = a.cu[seq], s1 = a.cu[seq + 1];
  const int c = slot - first_slot(a, seq);
  // launched as a programmatic dependent where gdn_recurrent_kernel has the short sequences: this
  // grid has nothing from it and waits (its first block) only so as not to end first
  auto wait_first = [] {
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (!good_bounds(s0, s1, a.T) || s1 - s0 <= a.by_row || c < 0 || c >= (s1 - s0 + kC - 1) / kC) {
    wait_first();  // a slot of no chunk
    return;
  }
  const int t0 = s0 + c * kC;
  const int n = min(kC, s1 - t0);
  const int hk = h / (a.H / a.Hk);

  if (tid == 0) {
    tc::mbar_init(&bars[0], 1);
    tc::mbar_init(&bars[1], 1);
    *abort_s = 0;
    *bad_s = kC;
    tc::mbar_fence_init();
    tc::fence_async_smem();
  }
  if (warp == 0) tc::tmem_alloc(tmem_s, 64);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = *tmem_s;
  if (tid == 0) {
    tc::mbar_arrive_expect_tx(&bars[0], 4 * kTile);
    for (int kb = 0; kb < 2; ++kb) {
      tc::tma_load_2d(sm + kWyQK + kb * 2 * kTile, &tmQ, hk * kD + 64 * kb, t0, &bars[0]);
      tc::tma_load_2d(sm + kWyQK + kb * 2 * kTile + kTile, &tmK, hk * kD + 64 * kb, t0, &bars[0]);
    }
  }
  // l_t: log decays summed in 64 bits (a decay of zero as e^-200, which is zero in float32
  // next to anything else)
  double la = 0.0;
  float be = 0.0f;
  if (tid < kC) {
    if (tid < n) {
      const long at = (long)(t0 + tid) * a.H + h;
      const float x = logf(a.alpha[at]);
      la = x < -200.0f ? -200.0 : (double)x;
      be = a.beta[at];
      // T and G have no other number than these: an infinite or undefined beta (or decay) becomes
      // an undefined gamma from its token on, by which gdn_scan_kernel knows
      if (!(fabsf(be) < INFINITY)) {
        la = (double)NAN;
        be = 0.0f;
      }
    }
    beta_s[tid] = be;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xFFFFFFFFu, la, o);
      if (lane >= o) la += y;
    }
    if (tid == 31) *wsum = la;
  }
  __syncthreads();
  if (tid < kC) {
    if (warp == 1) la += *wsum;
    ell[tid] = la;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf((float)la)));
    if (lane == 0) lmax[warp] = m;
  }
  __syncthreads();
  if (tid < kC) {
    gam[tid] = exp64(la);
    igam[tid] = exp64(-la);
  }
  bool ok = tc::bar_all(1, 128, tid == 0 ? tc::mbar_wait(&bars[0], 0, abort_s) : true);
  if (ok && n < kC) {
    // rows behind the sequence belong to another one, or to none: zero
    for (int e = tid; e < (kC - n) * 32; e += 128) {
      const int r = n + e / 32, x = e % 32;  // 4 tiles of 8 16-byte pieces
      *(uint4*)(sm + kWyQK + (x >> 3) * kTile + r * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    tc::fence_async_smem();
    __syncthreads();
  }
  // [Q; K] K^T: rows 0-63 Q K^T, rows 64-127 K K^T
  if (ok && tid == 0) {
    const uint32_t base = tc::smem_u32(sm + kWyQK);
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks) {
      const uint32_t off = (ks >> 2) * 2 * kTile + (ks & 3) * 32;
      tc::mma_ss(tm, tc::sdesc_sw128(base + off, 16, 1024), tc::sdesc_sw128(base + kTile + off, 16, 1024), kIdescWy,
                 ks > 0 ? 1u : 0u);
    }
    tc::mma_commit(&bars[1]);
  }
  if (ok) ok = tc::bar_all(1, 128, tid == 0 ? tc::mbar_wait(&bars[1], 0, abort_s) : true);
  // An entry of L or U that is no number is left out, and its token (its row) noted: as zero times
  // NaN it would reach the rows before, while its own row and those after it are undefined anyway.
  auto finite_or_note = [&](float& x, int t) {
    if (!(fabsf(x) < INFINITY)) {
      x = 0.0f;
      atomicMin(bad_s, t);
    }
  };
  // rows 0-63 (warps 0, 1): P = tril(Gamma o Q K^T); rows 64-127 (warps 2, 3): L; each when asked
  auto masked = [&](bool isL) {
    const int t = tid & (kC - 1);
    float* row = Ls + t * kP;
    const float bt = isL ? beta_s[t] : 1.0f;
    const int last = isL ? t - 1 : t;  // columns up to and with `last`
    const bool product = max(lmax[0], lmax[1]) <= __float_as_uint(kProductRange);
    const float gt = gam[t] * bt;
    float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // becomes NaN with an entry that is no number
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t x[32];
      tc::tmem_ld32(tm + ((uint32_t)(32 * warp) << 16) + 32 * half, x);
      wait_ld(x);
      if (product) {  // the pair's decay as a product of two exponentials while both stay in range
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const int s = 32 * half + e;
          const float4 i4 = *(const float4*)(igam + s);
          float4 v;
          v.x = s <= last ? gt * i4.x * __uint_as_float(x[e]) : 0.0f;
          v.y = s + 1 <= last ? gt * i4.y * __uint_as_float(x[e + 1]) : 0.0f;
          v.z = s + 2 <= last ? gt * i4.z * __uint_as_float(x[e + 2]) : 0.0f;
          v.w = s + 3 <= last ? gt * i4.w * __uint_as_float(x[e + 3]) : 0.0f;
          *(float4*)(row + s) = v;
          if (isL) z = make_float4(fmaf(v.x, 0.0f, z.x), fmaf(v.y, 0.0f, z.y), fmaf(v.z, 0.0f, z.z), fmaf(v.w, 0.0f, z.w));
        }
      } else {
        const double lt = ell[t];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int s = 32 * half + e;
          const float v = s <= last ? bt * expf((float)(lt - ell[s])) * __uint_as_float(x[e]) : 0.0f;
          row[s] = v;
          if (isL) z.x = fmaf(v, 0.0f, z.x);
        }
      }
    }
    if (isL && (z.x + z.y) + (z.z + z.w) != 0.0f) {
      for (int s = 0; s <= last; ++s) finite_or_note(row[s], t);
    }
  };
  if (ok) tc::tc_fence_after();
  if (ok && warp >= 2) masked(true);
  __syncthreads();
  // U = (I + L)^{-1} by 16 x 16 blocks: forward substitution on the diagonal blocks, then
  // U_ij = -sum_{k=j}^{i-1} (U_ii L_ik) U_kj, one level i - j after the other
  if (tid < kC) {
    const int k = tid >> 4, cc = tid & 15;
    float x[16];
#pragma unroll
    for (int tl = 0; tl < 16; ++tl) {
      const float4* Lrow = (const float4*)(Ls + (16 * k + tl) * kP + 16 * k);
      float v = tl == cc ? 1.0f : 0.0f;
#pragma unroll
      for (int s4 = 0; s4 < tl; s4 += 4) {
        const float4 w = Lrow[s4 >> 2];
        v = fmaf(-w.x, x[s4], v);
        if (s4 + 1 < tl) v = fmaf(-w.y, x[s4 + 1], v);
        if (s4 + 2 < tl) v = fmaf(-w.z, x[s4 + 2], v);
        if (s4 + 3 < tl) v = fmaf(-w.w, x[s4 + 3], v);
      }
      x[tl] = v;
    }
    float z = 0.0f;
#pragma unroll
    for (int tl = 0; tl < 16; ++tl) z = fmaf(x[tl], 0.0f, z);
    if (z != 0.0f) {
#pragma unroll
      for (int tl = 0; tl < 16; ++tl) finite_or_note(x[tl], 16 * k + tl);
    }
#pragma unroll
    for (int tl = 0; tl < 16; ++tl) Us[(16 * k + tl) * kP + 16 * k + cc] = x[tl];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 3; ++r) {  // L'_ik = U_ii L_ik in L's place: 6 blocks, 12 halves, 3 a warp
    const int u = warp + 4 * r, blk = u >> 1, nh = u & 1;
    const int ib = blk < 1 ? 1 : (blk < 3 ? 2 : 3);
    const int kb = blk - (ib * (ib - 1)) / 2;
    float acc[1][4] = {};
    float* at = Ls + 16 * ib * kP + 16 * kb + 8 * nh;
    block16<1>(acc, Us + 16 * ib * kP + 16 * ib, kP, at, kP, lane);
    __syncwarp();
    store16(at, kP, acc[0], 1.0f, lane);
  }
  __syncthreads();
#pragma unroll
  for (int lev = 1; lev <= 3; ++lev) {
    for (int u = warp; u < 2 * (4 - lev); u += 4) {
      const int jb = u >> 1, nh = u & 1;
      float acc[1][4] = {};
#pragma unroll
      for (int k = 0; k < lev; ++k)
        block16<1>(acc, Ls + 16 * (jb + lev) * kP + 16 * (jb + k), kP, Us + 16 * (jb + k) * kP + 16 * jb + 8 * nh, kP,
                   lane);
      if (acc[0][0] * 0.0f + acc[0][1] * 0.0f + acc[0][2] * 0.0f + acc[0][3] * 0.0f != 0.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) finite_or_note(acc[0][e], 16 * (jb + lev) + (lane >> 2) + 8 * (e >> 1));
      }
      __syncwarp();  // (the next product is the whole warp's)
      store16(Us + 16 * (jb + lev) * kP + 16 * jb + 8 * nh, kP, acc[0], -1.0f, lane);
    }
    __syncthreads();
  }
  // P over L' (no longer needed)
  if (ok && warp < 2) masked(false);
  tc::tc_fence_before();
  __syncthreads();
  // G = P U, blocks (i, j), j <= i, of i - j + 1 products: 5 a warp.  G_ij overwrites P_ij, which
  // a product of another warp may still want: all of them before any is stored
  float ga[4][2][4] = {};  // this warp's blocks: (3,0) (0,0) | (3,1) (3,2) | (2,0) (2,1) | (1,0) (1,1) (2,2) (3,3)
  auto g_at = [&](int u, int& i, int& j) {
    const int code = warp == 0 ? (u == 0 ? 0x30 : 0x00) : warp == 1 ? (u == 0 ? 0x31 : 0x32)
                   : warp == 2 ? (u == 0 ? 0x20 : 0x21) : (u == 0 ? 0x10 : 0x11 * u);
    i = code >> 4;
    j = code & 15;
  };
  const int blocks = warp == 3 ? 4 : 2;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < blocks) {
      int i, j;
      g_at(u, i, j);
      for (int k = j; k <= i; ++k) block16<2>(ga[u], Ls + 16 * i * kP + 16 * k, kP, Us + 16 * k * kP + 16 * j, kP, lane);
    }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < blocks) {
      int i, j;
      g_at(u, i, j);
      store16(Ls + 16 * i * kP + 16 * j, kP, ga[u][0], 1.0f, lane);
      store16(Ls + 16 * i * kP + 16 * j + 8, kP, ga[u][1], 1.0f, lane);
    }
  __syncthreads();
  // out: the parts of T and G as swizzled tiles, then gamma_t and gamma_C / gamma_t
  uint8_t* out = ws + ((long)slot * a.H + h) * kSlot;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int t = 16 * e + (tid >> 3), c8 = tid & 7;  // a warp writes four whole rows at once
    uint32_t w[6][4] = {};  // T1, G1, T2, G2, T3, G3 (blocks above the diagonal are zero)
    if ((c8 >> 1) <= (t >> 4)) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int cc = 8 * c8 + 2 * u;
        const float2 b2 = *(const float2*)(beta_s + cc);
        const float2 x = *(const float2*)(Us + t * kP + cc), y = *(const float2*)(Ls + t * kP + cc);
        cut3(x.x * b2.x, x.y * b2.y, w[0][u], w[2][u], w[4][u]);
        cut3(y.x * b2.x, y.y * b2.y, w[1][u], w[3][u], w[5][u]);
      }
    }
#pragma unroll
    for (int p = 0; p < 6; ++p) {
      const int row = stacked(t) + 16 * (p & 1);
      *(uint4*)(out + 2 * (p >> 1) * kTile + swz(row, c8)) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    }
  }
  float* sc = (float*)(out + kWy);
  if ((tid & (kC - 1)) >= *bad_s)
    sc[tid] = NAN;
  else
    sc[tid] = tid < kC ? gam[tid] : exp64(ell[kC - 1] - ell[tid - kC]);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 0) tc::tmem_dealloc(tm, 64);
  if (tid == 0 && *abort_s) report_device_error(kErrMbarTimeout);
  wait_first();
}

// ---- the walk over a sequence's chunks ---------------------------------------------------
//
// One CTA per (sequence, head, kV value columns): warp 0 loads, warp 1 issues the products,
// the others do the rest.  The parts of the right factor lie side by side, so that one
// instruction reads the left one once for all of them.
//   A  [K; Q] (128 x 128) x [S1 | S2 | S3]     -> K S^T and Q S^T (rows as in stacked())
//      R_t = V_t - gamma_t (K S^T)_t into shared memory (three parts); gamma_t (Q S^T)_t stays
//      in registers
//   B  [T1; G1] (128 x 64) x [R1 | R2 | R3], [T2; G2] x [R1 | R2], [T3; G3] x R1
//      diag(gamma_C / gamma_t) U (three parts) over R; the output is written beside the next A
//   C  K^T (128 x 64) x [U1 | U2 | U3]          -> S's update, one row k a thread:
//      S <- gamma_C S + update in registers, and its parts for the next A.
// What bounds it is the chain: three products, each with its way through tensor memory and
// registers to the next one's operand, and nothing to overlap them with but the output.

constexpr int kStKQ = 0;                      // stage: [kb][K, Q stacked: 128 rows][128 B]
constexpr int kStV = 4 * kTile;               // 64 value columns
constexpr int kStScal = kStV + kTile;
constexpr int kStage = kStScal + 1024;
constexpr int kStages = 2;
constexpr uint32_t kStTx = 5 * kTile + kScal;

// A right factor of kV columns in three parts side by side: 64-column atoms (128-byte rows).
// kV = 64: an atom per part; 32: parts 1 and 2 share the first; 16: one for all.
template <int kV>
struct Geo {
  static constexpr int kAtoms = kV == 64 ? 3 : kV == 32 ? 2 : 1;
  static constexpr int kHalf = 16;                  // columns per warp (output() counts on it)
  static constexpr int kSets = kV / kHalf;          // warps per 32 rows
  static constexpr int kThreads = 64 + 128 * kSets;
  static constexpr int kPieces = kHalf / 8;   // 16-byte pieces of a row per warp and part
  static constexpr int kWyAt = kStages * kStage;         // [T1; G1], [T2; G2], [T3; G3]
  static constexpr int kSAt = kWyAt + 6 * kTile;         // S^T: 128 rows
  static constexpr int kRAt = kSAt + kAtoms * 2 * kTile; // R, then U: 64 rows
  static constexpr int kOutAt = kRAt + kAtoms * kTile;  // 512 bytes per warp: its part of the output
  static constexpr int kSmallAt = kOutAt + 4 * kSets * 512;
  static constexpr int kSmem = kSmallAt + 128 + 4 * kV;
  static constexpr uint32_t kIdescA = tc::idesc_bf16_f32(128, 3 * kV, 0, 1);
  static constexpr uint32_t kIdescB2 = tc::idesc_bf16_f32(128, 2 * kV, 0, 1);
  static constexpr uint32_t kIdescB3 = tc::idesc_bf16_f32(128, kV, 0, 1);
  static constexpr uint32_t kIdescC = tc::idesc_bf16_f32(128, 3 * kV, 1, 1);
  // tensor memory columns: A and C, then the two accumulators of B
  static constexpr uint32_t kTmA = 0, kTmB = 3 * kV, kTmB2 = 6 * kV, kTmCols = 8 * kV;
  // byte offset of part p's atom, and the 16-byte piece its columns start at
  static __device__ __forceinline__ int atom(int p, int rows) { return (p * kV >> 6) * rows * 128; }
  static __device__ __forceinline__ int piece(int p) { return (p * kV & 63) >> 3; }
};

__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Tensor memory, 16 lanes x 16 columns in the layout of a warp-level product's result: for
// the 8-column tile j (registers 4 j ..) rows lane / 4 and lane / 4 + 8, columns 2 (lane % 4), + 1.
__device__ __forceinline__ void ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void ld_row(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Orders the uses of loaded registers after the wait above them.
template <int kN>
__device__ __forceinline__ void after_wait(uint32_t (&r)[kN]) {
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(r[i]));
}

// Two bf16 numbers times zero: zeros, or NaN where one is infinite or none.
__device__ __forceinline__ uint32_t times_zero(uint32_t w) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %2;" : "=r"(r) : "r"(w), "r"(0u));
  return r;
}

// Sum of kN accumulators, `pitch` columns apart, on 16 lanes x 16 kT columns (ld_frag's layout).
template <int kN, int kT>
__device__ __forceinline__ void sum_frag(uint32_t addr, int pitch, float (&x)[8 * kT]) {
  uint32_t y[kN][kT][8];
#pragma unroll
  for (int p = 0; p < kN; ++p)
#pragma unroll
    for (int i = 0; i < kT; ++i) ld_frag(addr + pitch * p + 16 * i, y[p][i]);
  tc::tmem_wait_ld();
#pragma unroll
  for (int p = 0; p < kN; ++p)
#pragma unroll
    for (int i = 0; i < kT; ++i) after_wait(y[p][i]);
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = __uint_as_float(y[kN - 1][i][e]);  // the smallest first
#pragma unroll
      for (int p = kN - 2; p >= 0; --p) s += __uint_as_float(y[p][i][e]);
      x[8 * i + e] = s;
    }
}

// 16 rows x kHalf columns (sum_frag's layout) into the three parts of R / U: rows 16 q .. of the
// 64-row atoms, columns half ch.
template <int kV>
__device__ __forceinline__ void store_frag(uint32_t dst, int q, int ch, int lane, const float (&x)[Geo<kV>::kHalf / 2]) {
  using G = Geo<kV>;
  const int row = 16 * q + (lane & 15);  // this lane's address: matrices (rows 0-7, 8-15) x (pieces 2 i, 2 i + 1)
#pragma unroll
  for (int i = 0; i < G::kHalf / 16; ++i) {
    uint32_t w[3][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)  // matrix m: rows 8 (m & 1), piece 2 i + (m >> 1)
      cut3(x[8 * i + 4 * (m >> 1) + 2 * (m & 1)], x[8 * i + 4 * (m >> 1) + 2 * (m & 1) + 1], w[0][m], w[1][m], w[2][m]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      stmatrix4(dst + G::atom(p, kC) + swz(row, G::piece(p) + G::kPieces * ch + 2 * i + (lane >> 4)), w[p]);
  }
}

template <int kV>
__global__ void __launch_bounds__(Geo<kV>::kThreads, 1)
    gdn_scan_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, GdnArgs a, const uint8_t* ws, bool longest_first) {
  using G = Geo<kV>;
  constexpr int kSplit = kD / kV;
  constexpr int kScThreads = G::kThreads;
  constexpr int kHalf = G::kHalf;
  constexpr int kT = kHalf / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* full = (uint64_t*)(sm + G::kSmallAt);
  uint64_t* empty = full + kStages;
  uint64_t* wfull = empty + kStages;
  uint64_t* doneA = wfull + 1;
  uint64_t* doneB = doneA + 1;   // also: T and G are free
  uint64_t* doneC = doneB + 1;
  uint64_t* s_ready = doneC + 1;
  uint64_t* r_ready = s_ready + 1;
  uint64_t* u_ready = r_ready + 1;
  uint64_t* fin = u_ready + 1;
  uint32_t* tmem_s = (uint32_t*)(fin + 1);
  volatile int* abort_s = (volatile int*)(tmem_s + 1);
  volatile int* any_bad = abort_s + 1;
  int* first_bad = (int*)(sm + G::kSmallAt + 128);  // [kV] first token of the sequence that makes a column undefined

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = (int)(blockIdx.x % kSplit) * kV;
  const int h = (int)((blockIdx.x / kSplit) % a.H);
  int seq = (int)((blockIdx.x / kSplit) / a.H);
  const int hk = h / (a.H / a.Hk);
  // Launched as gdn_wy_kernel's programmatic dependent: the loading warp waits for that grid where
  // it reads what it wrote; the first block waits in any case before it leaves, so that this grid
  // never ends before the other.
  auto wait_first = [] {
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (longest_first) {
    // more CTAs than run at once, or fewer than sequences (the short ones go by rows): blocks in
    // order of their sequences' lengths, so that the longest do not start last (block order ->
    // the sequence of that rank; ties by index)
    __shared__ int seq_s;
    int* length = (int*)sm;  // (the buffers are not in use yet)
    int longer = 0;          // than by_row
    for (int i0 = 0; i0 < a.n_seq; i0 += kScThreads) {
      const int i = i0 + tid;
      int len = -1;  // bounds that are none come last
      if (i < a.n_seq) {
        const int t0 = a.cu[i], t1 = a.cu[i + 1];
        if (good_bounds(t0, t1, a.T)) len = t1 - t0;
        length[i] = len;
      }
      longer += __syncthreads_count(len > a.by_row);
    }
    if (a.by_row >= 0 && seq >= longer) {  // the rest is gdn_recurrent_kernel's
      wait_first();
      return;
    }
    for (int s = tid; s < a.n_seq; s += kScThreads) {
      const int mine = length[s];
      int rank = 0;
      for (int i = 0; i < a.n_seq; ++i) rank += length[i] > mine || (length[i] == mine && i < s);
      if (rank == seq) seq_s = s;
    }
    __syncthreads();
    seq = seq_s;
  }
  // what the device arrays cannot mean is refused: nothing is read or written for it
  int slot = seq;
  if (a.slots != nullptr) {
    slot = a.slots[seq];
    if (slot < 0) {  // padding of the batch
      wait_first();
      return;
    }
    bool twice = false;    // an earlier sequence has the same state
    for (int i = tid; i < seq; i += kScThreads) twice |= a.slots[i] == slot;
    if (__syncthreads_or(twice) || slot >= a.n_slots) {
      if (tid == 0) report_device_error(kErrBadIndex);
      wait_first();
      return;
    }
  }
  const int s0 = a.cu[seq], s1 = a.cu[seq + 1];
  const int len = s1 - s0;
  if (len >= 0 && len <= a.by_row) {  // gdn_recurrent_kernel's
    wait_first();
    return;
  }
  const int nc = (len + kC - 1) / kC;
  const int base = first_slot(a, seq);
  // (a slot's owner is found by bisection: where the bounds are in order it is this sequence)
  if (!good_bounds(s0, s1, a.T) ||
      (nc > 0 && (slot_owner(a, base) != seq || slot_owner(a, base + nc - 1) != seq))) {
    if (tid == 0) report_device_error(kErrBadIndex);
    wait_first();
    return;
  }
  const long soff = ((long)slot * a.H + h) * kD * kD + (long)v0 * kD;  // this CTA's state rows
  if (nc == 0) {  // no tokens: the state passes through
    if (a.state_out != nullptr && a.state_out != a.state_in)
      for (int e = tid; e < kV * kD / 4; e += kScThreads) {
        float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.state_in != nullptr) w = ((const float4*)(a.state_in + soff))[e];
        ((float4*)(a.state_out + soff))[e] = w;
      }
    wait_first();
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(wfull, 1);
    tc::mbar_init(doneA, 1);
    tc::mbar_init(doneB, 1);
    tc::mbar_init(doneC, 1);
    tc::mbar_init(s_ready, 4 * G::kSets);
    tc::mbar_init(r_ready, 4 * G::kSets);
    tc::mbar_init(u_ready, 4 * G::kSets);
    tc::mbar_init(fin, 1);
    *abort_s = 0;
    *any_bad = 0;
    tc::mbar_fence_init();
  }
  if (tid < kV) first_bad[tid] = INT_MAX;
  tc::fence_async_smem();  // (lengths have been written where the copies land)
  if (warp == 1) tc::tmem_alloc(tmem_s, G::kTmCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tm = *tmem_s;

  if (warp == 0) {
    // ---------------- loads ----------------
    if (lane == 0) {
      tc::tma_prefetch_desc(&tmQ);
      tc::tma_prefetch_desc(&tmK);
      tc::tma_prefetch_desc(&tmV);
      const uint8_t* wy = ws + ((long)base * a.H + h) * kSlot;
      // the workspace (the call's inputs were there before that grid started)
      asm volatile("griddepcontrol.wait;" ::: "memory");
      auto load_stage = [&](int c) {
        const int st = c % kStages;
        if (c >= kStages && !tc::mbar_wait(&empty[st], ((c / kStages) - 1) & 1, abort_s)) return false;
        uint8_t* dst = sm + st * kStage;
        const int y = s0 + c * kC;
        tc::mbar_arrive_expect_tx(&full[st], kStTx);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint8_t* at = dst + kStKQ + kb * 2 * kTile + g * 4096;
            tc::tma_load_2d(at, &tmK, hk * kD + 64 * kb, y + 16 * g, &full[st]);
            tc::tma_load_2d(at + 2048, &tmQ, hk * kD + 64 * kb, y + 16 * g, &full[st]);
          }
        tc::tma_load_2d(dst + kStV, &tmV, h * kD + (v0 & 64), y, &full[st]);
        tc::bulk_load_1d(dst + kStScal, wy + (long)c * a.H * kSlot + kWy, kScal, &full[st]);
        return true;
      };
      int c = 0, stages = 0;  // loads issued
      if (load_stage(0)) ++stages;
      for (; c < nc; ++c) {
        if (c > 0 && !tc::mbar_wait(doneB, (c - 1) & 1, abort_s)) break;
        const uint8_t* src = wy + (long)c * a.H * kSlot;
        uint8_t* dst = sm + G::kWyAt;
        tc::mbar_arrive_expect_tx(wfull, kWy);
        tc::bulk_load_1d(dst, src, kWy, wfull);
        if (c + 1 < nc) {
          if (!load_stage(c + 1)) {
            ++c;
            break;
          }
          ++stages;
        }
      }
      if (*abort_s) {  // never leave the CTA with copies in flight
        for (int t = max(0, stages - kStages); t < stages; ++t)
          tc::mbar_wait(&full[t % kStages], (t / kStages) & 1, nullptr, 200000000ull);
        if (c > 0) tc::mbar_wait(wfull, (c - 1) & 1, nullptr, 200000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- products ----------------
    // The whole warp walks the loop and one elected lane issues, so that descriptors and
    // addresses are the same in every lane and live in uniform registers (issued from a
    // branch of one lane, an instruction took 69 cycles).
    const bool lead = tc::elect_one();
    const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0);
    // descriptors of the operands' starts; a step adds its bytes / 16 to the address field
    const uint64_t kq0 = tc::sdesc_sw128(tc::smem_u32(sm + kStKQ), 16, 1024);
    const uint64_t kt0 = tc::sdesc_sw128(tc::smem_u32(sm + kStKQ), 2 * kTile, 1024);
    const uint64_t w0 = tc::sdesc_sw128(tc::smem_u32(sm + G::kWyAt), 16, 1024);
    const uint64_t s_d = tc::sdesc_sw128(tc::smem_u32(sm + G::kSAt), 2 * kTile, 1024);
    const uint64_t r_d = tc::sdesc_sw128(tc::smem_u32(sm + G::kRAt), kTile, 1024);
    for (int c = 0; c < nc; ++c) {
      const int st = c % kStages;
      const uint32_t par = (uint32_t)c & 1;
      const uint64_t kq = kq0 + (uint64_t)(st * (kStage >> 4)), kt = kt0 + (uint64_t)(st * (kStage >> 4));
      bool go = tc::mbar_wait(&full[st], (uint32_t)(c / kStages) & 1, abort_s) && tc::mbar_wait(s_ready, par, abort_s);
      if (!__all_sync(0xFFFFFFFFu, go)) break;
      tc::tc_fence_after();
      if (lead) {
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks)
          tc::mma_ss(tmu + G::kTmA, kq + (((ks >> 2) * 2 * kTile + (ks & 3) * 32) >> 4), s_d + ((ks * 2048) >> 4),
                     G::kIdescA, ks > 0 ? 1u : 0u);
        tc::mma_commit(doneA);
      }
      __syncwarp();
      go = tc::mbar_wait(wfull, par, abort_s) && tc::mbar_wait(r_ready, par, abort_s);
      if (!__all_sync(0xFFFFFFFFu, go)) break;
      tc::tc_fence_after();
      if (lead) {
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          tc::mma_ss(tmu + G::kTmB, w0 + ((ks * 32) >> 4), r_d + ((ks * 2048) >> 4), G::kIdescA, ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          tc::mma_ss(tmu + G::kTmB2, w0 + ((2 * kTile + ks * 32) >> 4), r_d + ((ks * 2048) >> 4), G::kIdescB2,
                     ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          tc::mma_ss(tmu + G::kTmB2, w0 + ((4 * kTile + ks * 32) >> 4), r_d + ((ks * 2048) >> 4), G::kIdescB3, 1u);
        tc::mma_commit(doneB);
      }
      __syncwarp();
      go = tc::mbar_wait(u_ready, par, abort_s);
      if (!__all_sync(0xFFFFFFFFu, go)) break;
      tc::tc_fence_after();
      if (lead) {
#pragma unroll
        for (int ks = 0; ks < kC / 16; ++ks)
          tc::mma_ss(tmu + G::kTmA, kt + ((ks * 4096) >> 4), r_d + ((ks * 2048) >> 4), G::kIdescC, ks > 0 ? 1u : 0u);
        tc::mma_commit(doneC);
        tc::mma_commit(&empty[st]);
      }
      __syncwarp();
    }
    // every product issued here completes before tensor memory is freed
    if (lead) tc::mma_commit(fin);
    __syncwarp();
    tc::mbar_wait(fin, 0, nullptr, 200000000ull);
    __syncwarp();
  } else {
    // ---------------- the others: lane quarter q, column set ch of every product ----------------
    const int q = warp & 3;
    const int ch = (warp - 2) >> 2;
    const int r = 32 * q + lane;             // C and S: key channel r
    const int ta = 16 * q + (lane >> 2);     // A, B: tokens ta and ta + 8
    const uint32_t lanes = tm + ((uint32_t)(32 * q) << 16) + kHalf * ch;
    const uint32_t lanes2 = lanes + (16u << 16);  // the rows of Q and G
    const long srow = soff + (long)(kHalf * ch) * kD + r;
    const uint32_t rdst = tc::smem_u32(sm + G::kRAt);
    // V's pieces of this warp's columns in the stage's 64
    const int vpiece = ((v0 & 63) >> 3) + G::kPieces * ch;
    float S[kHalf];
#pragma unroll
    for (int v = 0; v < kHalf; ++v) S[v] = a.state_in != nullptr ? a.state_in[srow + (long)v * kD] : 0.0f;
    float ga = 0.0f, gb = 0.0f;       // gamma of tokens ta, ta + 8
    float y[kHalf / 2];                // Q S^T of the chunk, until its output is written
    // column of the CTA that register pair e of a fragment (sum_frag) starts at, and its token
    auto frag_col = [&](int e) { return kHalf * ch + 8 * (e >> 2) + 2 * (lane & 3); };
    auto frag_row = [&](int e) { return ta + ((e & 2) ? 8 : 0); };
    // the output of chunk c's tokens ta and ta + 8, with c's ga, gb and y
    auto output = [&](int c, bool undefined) {  // undefined: a column is, from some token on
      float x[kHalf / 2], z[kHalf / 2];
      sum_frag<3, kT>(lanes2 + G::kTmB, kV, x);
      sum_frag<2, kT>(lanes2 + G::kTmB2, kV, z);
      // 16 tokens x 16 columns by way of shared memory, so that two lanes write a row's 32 bytes
#pragma unroll
      for (int e = 0; e < kHalf / 2; ++e) x[e] = fmaf((e & 2) ? gb : ga, y[e], x[e] + z[e]);
      if (undefined) {
#pragma unroll
        for (int e = 0; e < kHalf / 2; ++e)
          if (c * kC + frag_row(e) >= first_bad[frag_col(e) + (e & 1)]) x[e] = NAN;
      }
      uint32_t w[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {  // matrix m: tokens 8 (m & 1) .., columns 8 (m >> 1) ..
        const int e = 4 * (m >> 1) + 2 * (m & 1);
        w[m] = tc::pack_bf16x2(x[e], x[e + 1]);
      }
      uint8_t* stage = sm + G::kOutAt + (warp - 2) * 512;
      __syncwarp();  // (the chunk before has been read)
      stmatrix4(tc::smem_u32(stage) + (lane & 15) * 32 + (lane >> 4) * 16, w);
      __syncwarp();
      const uint4 row16 = *(const uint4*)(stage + lane * 16);
      const int t = c * kC + 16 * q + (lane >> 1);
      if (t < len)
        *(uint4*)((__nv_bfloat16*)a.o + ((long)(s0 + t) * a.H + h) * kD + v0 + kHalf * ch + 8 * (lane & 1)) = row16;
    };
    bool ok = true;
    for (int c = 0; c < nc; ++c) {
      const uint32_t par = (uint32_t)c & 1;
      uint8_t* stage = sm + (c % kStages) * kStage;
      const int n = min(kC, len - c * kC);
      const bool undefined = *any_bad != 0;
      // S's parts: row r, columns of set ch
#pragma unroll
      for (int i = 0; i < G::kPieces; ++i) {
        uint32_t w[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) cut3(S[8 * i + 2 * e], S[8 * i + 2 * e + 1], w[0][e], w[1][e], w[2][e]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *(uint4*)(sm + G::kSAt + G::atom(p, kD) + swz(r, G::piece(p) + G::kPieces * ch + i)) =
              make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
      }
      if (n < kC) {
        // keys behind the sequence belong to another one, or to none: zero
        ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&full[c % kStages], (uint32_t)(c / kStages) & 1, abort_s));
        if (!ok) break;
        if (r < kC && r >= n)
          for (int kb = ch; kb < 2; kb += G::kSets)
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8)
              *(uint4*)(stage + kStKQ + kb * 2 * kTile + stacked(r) * 128 + 16 * c8) = make_uint4(0u, 0u, 0u, 0u);
      }
      tc::fence_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(s_ready);
      // while A runs: the output of the chunk before (B's accumulators are not written again
      // before r_ready), and what the next steps need of this chunk (read before r_ready: the
      // stage may be refilled once C is done)
      if (c > 0) output(c - 1, undefined);
      ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(&full[c % kStages], (uint32_t)(c / kStages) & 1, abort_s));
      if (!ok) break;
      const float* sc = (const float*)(stage + kStScal);
      ga = sc[ta], gb = sc[ta + 8];
      const float da = sc[kC + ta], db = sc[kC + ta + 8], gC = sc[kC - 1];
      uint32_t vw[kT][4];  // V: matrix m of tile pair i as in store_frag
#pragma unroll
      for (int i = 0; i < kT; ++i)
        ldmatrix4(tc::smem_u32(stage + kStV) + swz(16 * q + (lane & 15), vpiece + 2 * i + (lane >> 4)), vw[i]);
      // A value that is no number goes into the products as zero, for the tokens before it; from its
      // token on its column is undefined: output() and the end see to that.
      static_assert(kHalf == 16, "eight values a thread");
      if (((times_zero(vw[0][0]) | times_zero(vw[0][1]) | times_zero(vw[0][2]) | times_zero(vw[0][3])) & 0x7FFF7FFFu)) {
#pragma unroll
        for (int e = 0; e < kHalf / 2; ++e) {
          uint32_t& w = vw[0][2 * (e >> 2) + ((e >> 1) & 1)];
          const uint32_t mask = (e & 1) ? 0xFFFF0000u : 0xFFFFu;
          if (frag_row(e) < n && (times_zero(w & mask) & 0x7FFF7FFFu)) {
            atomicMin(&first_bad[frag_col(e) + (e & 1)], c * kC + frag_row(e));
            *any_bad = 1;
            w &= ~mask;
          }
        }
      }
      __syncwarp();
      ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(doneA, par, abort_s));
      if (!ok) break;
      tc::tc_fence_after();
      float x[kHalf / 2];
      sum_frag<3, kT>(lanes + G::kTmA, kV, x);
      {
        // R is zero behind the sequence, and where gamma is undefined: that token would reach those
        // before it as zero times NaN (its own output and the state get gamma as well)
        const bool la = ta < n && fabsf(ga) < INFINITY, lb = ta + 8 < n && fabsf(gb) < INFINITY;
#pragma unroll
        for (int i = 0; i < kT; ++i)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int e = 8 * i + 4 * (m >> 1) + 2 * (m & 1);
            const float g = (m & 1) ? gb : ga;
            const bool live = (m & 1) ? lb : la;
            x[e] = live ? fmaf(-g, x[e], tc::bf16lo(vw[i][m])) : 0.0f;
            x[e + 1] = live ? fmaf(-g, x[e + 1], tc::bf16hi(vw[i][m])) : 0.0f;
          }
      }
      store_frag<kV>(rdst, q, ch, lane, x);
      tc::fence_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(r_ready);
      sum_frag<3, kT>(lanes2 + G::kTmA, kV, y);  // Q S^T
      ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(doneB, par, abort_s));
      if (!ok) break;
      tc::tc_fence_after();
      {
        float z[kHalf / 2];
        sum_frag<3, kT>(lanes + G::kTmB, kV, x);
        sum_frag<2, kT>(lanes + G::kTmB2, kV, z);
#pragma unroll
        for (int e = 0; e < kHalf / 2; ++e) x[e] = ((e & 2) ? db : da) * (x[e] + z[e]);
      }
      store_frag<kV>(rdst, q, ch, lane, x);
      tc::fence_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(u_ready);
      ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(doneC, par, abort_s));
      if (!ok) break;
      tc::tc_fence_after();
      {
        uint32_t z[3][kT][16];
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int i = 0; i < kT; ++i) ld_row(lanes + G::kTmA + kV * p + 16 * i, z[p][i]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int i = 0; i < kT; ++i) after_wait(z[p][i]);
#pragma unroll
        for (int v = 0; v < kHalf; ++v)
          S[v] = fmaf(gC, S[v],
                      (__uint_as_float(z[2][v >> 4][v & 15]) + __uint_as_float(z[1][v >> 4][v & 15])) +
                          __uint_as_float(z[0][v >> 4][v & 15]));
      }
    }
    if (ok) output(nc - 1, *any_bad != 0);
    if (ok && a.state_out != nullptr) {
      if (*any_bad) {
#pragma unroll
        for (int v = 0; v < kHalf; ++v)
          if (first_bad[kHalf * ch + v] != INT_MAX) S[v] = NAN;
      }
#pragma unroll
      for (int v = 0; v < kHalf; ++v) a.state_out[srow + (long)v * kD] = S[v];
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tm, G::kTmCols);
  if (tid == 0 && *abort_s) report_device_error(kErrMbarTimeout);
  wait_first();
}

template <int kV>
cudaError_t launch_scan(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const GdnArgs& a,
                        const uint8_t* ws, long n, cudaStream_t s) {
  const int smem = 1024 + Geo<kV>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(gdn_scan_kernel<kV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n * a.H * (kD / kV)));
  cfg.blockDim = dim3(Geo<kV>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool longest_first = n < a.n_seq || ((long)cfg.gridDim.x > num_sms() && n > 1 && n <= kGdnRankedSeqs);
  return cudaLaunchKernelEx(&cfg, gdn_scan_kernel<kV>, tq, tk, tv, a, ws, longest_first);
}

}  // namespace

// Chunk slots of T tokens in n sequences (see first_slot).
static bool gdn_half_slots(int T, int n_seq, int by_row) {
  return by_row >= kC / 2 - 1 && T / (kC / 2) + 1L < T / kC + (long)n_seq;
}
static long gdn_slots(int T, int n_seq, int by_row) {
  return gdn_half_slots(T, n_seq, by_row) ? T / (kC / 2) + 1L : T / kC + (long)n_seq;
}

size_t gdn_chunk_workspace(int T, int n_seq, int H, int by_row) {
  return (size_t)gdn_slots(T, n_seq, by_row) * H * kSlot;
}

cudaError_t launch_gdn_chunk(const GdnArgs& in, void* ws, cudaStream_t s) {
  GdnArgs a = in;
  a.half_slots = gdn_half_slots(a.T, a.n_seq, a.by_row);
  // sequences that can be the chunks': all, or as many as fit T with more than by_row tokens
  const long n = a.by_row < 0 ? a.n_seq : min((long)a.n_seq, (long)a.T / (a.by_row + 1));
  const long wy = gdn_slots(a.T, a.n_seq, a.by_row) * a.H, pairs = n * a.H;
  if (wy >= (1L << 31) || pairs * 2 >= (1L << 31)) return cudaErrorNotSupported;
  const long rowk = (long)a.Hk * kD, rowv = (long)a.H * kD;
  CUtensorMap tq, tk, tq16, tk16, tv;
  cudaError_t e = make_tmap_2d(&tq, a.q, rowk, a.T, rowk * 2, 64, 64);
  if (e == cudaSuccess) e = make_tmap_2d(&tk, a.k, rowk, a.T, rowk * 2, 64, 64);
  if (e == cudaSuccess) e = make_tmap_2d(&tq16, a.q, rowk, a.T, rowk * 2, 64, 16);
  if (e == cudaSuccess) e = make_tmap_2d(&tk16, a.k, rowk, a.T, rowk * 2, 64, 16);
  if (e == cudaSuccess) e = make_tmap_2d(&tv, a.v, rowv, a.T, rowv * 2, 64, 64);
  if (e != cudaSuccess) return e;
  const int wsm = 1024 + kWySmem;
  e = cudaFuncSetAttribute(gdn_wy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, wsm);
  if (e != cudaSuccess) return e;
  if (a.by_row >= 0) e = launch_gdn_recurrent(a, s);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)wy);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = wsm;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.by_row >= 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, gdn_wy_kernel, tq, tk, a, (uint8_t*)ws);
  if (e != cudaSuccess) return e;
  // the value columns go to as many CTAs as all run at once: each chunk's steps get shorter
  if (pairs * 8 <= num_sms()) return launch_scan<16>(tq16, tk16, tv, a, (const uint8_t*)ws, n, s);
  if (pairs * 4 <= num_sms()) return launch_scan<32>(tq16, tk16, tv, a, (const uint8_t*)ws, n, s);
  return launch_scan<64>(tq16, tk16, tv, a, (const uint8_t*)ws, n, s);
}

}  // namespace hla
