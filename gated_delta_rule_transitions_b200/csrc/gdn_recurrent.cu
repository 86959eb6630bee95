// The gated delta rule token by token, with a state that is carried in and out
// (float32 arithmetic on CUDA cores): the one-token step of a decode batch, and the
// ragged forward of every type, head dim and decay.
//
// HLA summary page, "Methodology in Plain English" para. 1: the per-token affine rule
//   S <- S Diag(alpha_t);  u_t = beta_t (v_t - S k_t);  S <- S + u_t k_t^T;  o_t = S q_t
// (alpha_t one decay per head, or one per key channel).  Rows of S evolve on their own.
//
// A CTA of 128 threads holds 16 R rows of one (sequence, head)'s state in registers:
// 8 threads per R rows, thread g of a group on the columns 32 m + 4 g + u (u < 4), so
// that state loads and stores are 128-byte segments and the dot products over a row are
// three shuffles.  Keys, queries, values and decays of 8 to 32 tokens at a time come in by
// cp.async as they are stored (two buffers: the next tokens land while these are worked
// on); outputs leave through shared memory.
//
// A step is bound by the state's way in and out (2 d^2 floats a head): 64 sequences x 16 heads
// of 128, 23.5 us, 5.8 TB/s, 0.88 of the measured copy rate; a forward pass by the chain of
// shuffles and multiply-adds from token to token, 0.19 us a token.
#include "common.cuh"
#include "kernels.cuh"

namespace hla {

HLA_DEFINE_ERROR_WORD(gdn_recurrent)

namespace {

constexpr int kThreads = 128;
// Tokens per staged segment: as many as two buffers have room for in 40 KiB, up to 32.
template <int D, int R, typename Tio, bool kChan, bool kOne>
constexpr int seg_len() {
  const int bytes = (2 * D + 16 * R) * (int)sizeof(Tio) + 4 * (kChan ? D : 1) + 4;
  return kOne ? 1 : 64 * bytes <= 40960 ? 32 : 32 * bytes <= 40960 ? 16 : 8;
}
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// Four consecutive values as two float pairs.
__device__ __forceinline__ void ld4(const float* p, float2& lo, float2& hi) {
  const float4 w = *(const float4*)p;
  lo = make_float2(w.x, w.y);
  hi = make_float2(w.z, w.w);
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float2& lo, float2& hi) {
  const uint2 w = *(const uint2*)p;
  lo = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
  hi = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ float group_sum(float v) {
  v += __shfl_xor_sync(kFull, v, 1);
  v += __shfl_xor_sync(kFull, v, 2);
  v += __shfl_xor_sync(kFull, v, 4);
  return v;
}

template <int D, int R, typename Tio, bool kChan, int kSeg>
struct Stage {
  Tio k[kSeg][D];
  Tio q[kSeg][D];
  Tio v[kSeg][16 * R];
  float a[kSeg][kChan ? D : 1];
  float b[kSeg];
};

// Row r's dot product over this thread's columns.
template <int M>
__device__ __forceinline__ float dot_cols(const float2 (&x)[2 * M], const float2 (&k)[2 * M]) {
  float2 d0 = make_float2(0.0f, 0.0f), d1 = d0;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    d0 = __ffma2_rn(x[2 * m], k[2 * m], d0);
    d1 = __ffma2_rn(x[2 * m + 1], k[2 * m + 1], d1);
  }
  return (d0.x + d0.y) + (d1.x + d1.y);
}

// kOne: one token per sequence (the step).  Otherwise token t's output and token t + 1's dot
// product with its key are reduced together: one chain of three shuffles a token.
template <int D, int R, typename Tio, bool kChan, bool kOne>
__global__ void __launch_bounds__(kThreads) gdn_recurrent_kernel(GdnArgs a) {
  constexpr int kRows = 16 * R;
  constexpr int kSplit = D / kRows;   // CTAs per (sequence, head)
  constexpr int M = D / 32;           // 4-column groups per thread
  constexpr int kVec = 16 / (int)sizeof(Tio);
  constexpr int kSeg = seg_len<D, R, Tio, kChan, kOne>();
  __shared__ __align__(16) Stage<D, R, Tio, kChan, kSeg> st[kOne ? 1 : 2];
  __shared__ float os[kSeg][kRows];
  // launched as a programmatic dependent: the next step's blocks may take their places while
  // this grid drains; all that is read comes after the wait for the grid before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int split = blockIdx.x % kSplit;
  const long sh = blockIdx.x / kSplit;
  const int h = (int)(sh % a.H);
  const int seq = (int)(sh / a.H);
  const int hk = h / (a.H / a.Hk);
  const int p = tid >> 3, g = tid & 7;
  const int row0 = split * kRows + p * R;  // this group's rows row0 .. row0 + R - 1

  // the sequence's tokens and its state; what the device arrays cannot mean is refused
  // (nothing is read or written for that sequence)
  int t0 = seq, t1 = seq + 1;
  if (!kOne) {
    t0 = a.cu[seq];
    t1 = a.cu[seq + 1];
  }
  int slot = seq;
  if (a.slots != nullptr) {
    slot = a.slots[seq];
    if (slot < 0) return;  // padding of the batch
  }
  if (t0 < 0 || t1 < t0 || t1 > a.T || slot >= a.n_slots) {
    if (tid == 0) report_device_error(kErrBadIndex);
    return;
  }
  if (!kOne && t1 - t0 > a.by_row) return;  // gdn_scan_kernel's

  const Tio* kin = (const Tio*)a.k + ((long)t0 * a.Hk + hk) * D;
  const Tio* qin = (const Tio*)a.q + ((long)t0 * a.Hk + hk) * D;
  const Tio* vin = (const Tio*)a.v + ((long)t0 * a.H + h) * D + split * kRows;
  Tio* out = (Tio*)a.o + ((long)t0 * a.H + h) * D + split * kRows;
  const float* ain = a.alpha + ((long)t0 * a.H + h) * (kChan ? D : 1);
  const float* bin = a.beta + (long)t0 * a.H + h;
  const int len = t1 - t0;

  // tokens [s0, s0 + kSeg) into buffer w
  auto stage = [&](int s0, int w) {
    const int ns = min(kSeg, len - s0);
    for (int e = tid; e < ns * (D / kVec); e += kThreads) {
      const int t = e / (D / kVec), c = (e % (D / kVec)) * kVec;
      const long row = (long)(s0 + t) * a.Hk * D + c;
      cp16(&st[w].k[t][c], kin + row);
      cp16(&st[w].q[t][c], qin + row);
    }
    for (int e = tid; e < ns * (kRows / kVec); e += kThreads) {
      const int t = e / (kRows / kVec), c = (e % (kRows / kVec)) * kVec;
      cp16(&st[w].v[t][c], vin + (long)(s0 + t) * a.H * D + c);
    }
    if (kChan) {
      for (int e = tid; e < ns * (D / 4); e += kThreads) {
        const int t = e / (D / 4), c = (e % (D / 4)) * 4;
        cp16(&st[w].a[t][c], ain + (long)(s0 + t) * a.H * D + c);
      }
    } else if (tid >= 32 && tid < 32 + ns) {
      cp4(&st[w].a[tid - 32][0], ain + (long)(s0 + tid - 32) * a.H);
    }
    if (tid < ns) cp4(&st[w].b[tid], bin + (long)(s0 + tid) * a.H);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (len > 0) stage(0, 0);

  // the state: x[r][2 m + e] = columns 32 m + 4 g + 2 e, + 1 of row row0 + r
  const long off = (((long)slot * a.H + h) * D + row0) * D + 4 * g;
  float2 x[R][2 * M];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (a.state_in != nullptr) w = *(const float4*)(a.state_in + off + (long)r * D + 32 * m);
      x[r][2 * m] = make_float2(w.x, w.y);
      x[r][2 * m + 1] = make_float2(w.z, w.w);
    }

  if (a.slots != nullptr) {  // (the state and the first tokens are on their way)
    bool twice = false;      // an earlier sequence has the same state
    for (int i = tid; i < seq; i += kThreads) twice |= a.slots[i] == slot;
    if (__syncthreads_or(twice)) {
      if (tid == 0) report_device_error(kErrBadIndex);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      return;
    }
  }

  int w = 0;
  for (int s0 = 0; s0 < len; s0 += kSeg, w ^= (kOne ? 0 : 1)) {
    const int ns = min(kSeg, len - s0);
    if (!kOne && s0 + kSeg < len) {
      stage(s0 + kSeg, w ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    // keys (and decays) of the token at hand; p[r] = the decayed row's product with the key
    float2 kr[2 * M], ar[kChan ? 2 * M : 1];
    float p_[R];
    auto load_key = [&](int t, float2 (&k)[2 * M], float2 (&al)[kChan ? 2 * M : 1]) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        ld4(&st[w].k[t][32 * m + 4 * g], k[2 * m], k[2 * m + 1]);
        if constexpr (kChan) {
          const float4 f = *(const float4*)&st[w].a[t][32 * m + 4 * g];
          al[2 * m] = make_float2(f.x, f.y);
          al[2 * m + 1] = make_float2(f.z, f.w);
        }
      }
    };
    auto key_part = [&](const float2 (&xr)[2 * M], const float2 (&k)[2 * M], const float2 (&al)[kChan ? 2 * M : 1]) {
      if constexpr (kChan) {
        float2 ka[2 * M];
#pragma unroll
        for (int j = 0; j < 2 * M; ++j) ka[j] = __fmul2_rn(k[j], al[j]);
        return dot_cols<M>(xr, ka);
      } else {
        return dot_cols<M>(xr, k);
      }
    };
    load_key(0, kr, ar);
#pragma unroll
    for (int r = 0; r < R; ++r) p_[r] = group_sum(key_part(x[r], kr, ar));
    for (int t = 0; t < ns; ++t) {
      float2 qr[2 * M], kn[2 * M], an[kChan ? 2 * M : 1];
#pragma unroll
      for (int m = 0; m < M; ++m) ld4(&st[w].q[t][32 * m + 4 * g], qr[2 * m], qr[2 * m + 1]);
      if (!kOne) load_key(min(t + 1, ns - 1), kn, an);  // (the last token's is not used)
      const float at = kChan ? 1.0f : st[w].a[t][0];
      const float bt = st[w].b[t];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float u = bt * (ldf(&st[w].v[t][p * R + r]) - at * p_[r]);
        const float2 u2 = make_float2(u, u), a2 = make_float2(at, at);
#pragma unroll
        for (int j = 0; j < 2 * M; ++j) {
          if constexpr (kChan)
            x[r][j] = __ffma2_rn(u2, kr[j], __fmul2_rn(ar[j], x[r][j]));
          else
            x[r][j] = __ffma2_rn(u2, kr[j], __fmul2_rn(a2, x[r][j]));
        }
      }
      float y[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        y[r] = dot_cols<M>(x[r], qr);
        if (!kOne) p_[r] = key_part(x[r], kn, an);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          y[r] += __shfl_xor_sync(kFull, y[r], o);
          if (!kOne) p_[r] += __shfl_xor_sync(kFull, p_[r], o);
        }
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (g == r) os[t][p * R + r] = y[r];
      if (!kOne) {
#pragma unroll
        for (int j = 0; j < 2 * M; ++j) {
          kr[j] = kn[j];
          if constexpr (kChan) ar[j] = an[j];
        }
      }
    }
    __syncthreads();  // the segment's outputs are in shared memory and its buffer is free
    for (int e = tid; e < ns * kRows; e += kThreads) {
      const int t = e / kRows, r = e % kRows;
      stf(out + (long)(s0 + t) * a.H * D + r, os[t][r]);
    }
  }
  if (a.state_out == nullptr || (len == 0 && a.state_out == a.state_in)) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int m = 0; m < M; ++m)
      *(float4*)(a.state_out + off + (long)r * D + 32 * m) =
          make_float4(x[r][2 * m].x, x[r][2 * m].y, x[r][2 * m + 1].x, x[r][2 * m + 1].y);
}

template <int D, int R, typename Tio>
cudaError_t launch_r(const GdnArgs& a, cudaStream_t s) {
  const long blocks = (long)a.n_seq * a.H * (D / (16 * R));
  if (blocks >= (1L << 31)) return cudaErrorNotSupported;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.cu == nullptr)
    return a.alpha_vec ? cudaLaunchKernelEx(&cfg, gdn_recurrent_kernel<D, R, Tio, true, true>, a)
                       : cudaLaunchKernelEx(&cfg, gdn_recurrent_kernel<D, R, Tio, false, true>, a);
  return a.alpha_vec ? cudaLaunchKernelEx(&cfg, gdn_recurrent_kernel<D, R, Tio, true, false>, a)
                     : cudaLaunchKernelEx(&cfg, gdn_recurrent_kernel<D, R, Tio, false, false>, a);
}

template <int D, typename Tio>
cudaError_t launch_d(const GdnArgs& a, cudaStream_t s) {
  // Rows per group of threads: one while that leaves each SM a few CTAs at most (a token's
  // chain is shortest), else two (a shared-memory read then feeds two rows; four take so many
  // registers that the step slows down: 64 x 16 heads of 128, 23.5 us with two, 26 with four).
  // Measured, 16 heads of 128, bf16: 256 tokens of one sequence 49 us with one row, 78 with
  // two; of four sequences 152 and 95.  The step of 8 x 8 heads: 2.5 and 2.7; of 16 x 8: 4.1
  // and 3.5.
  const long ctas = (long)a.n_seq * a.H * (D / 16);
  return ctas <= (a.cu == nullptr ? 4L : 2L) * num_sms() ? launch_r<D, 1, Tio>(a, s) : launch_r<D, 2, Tio>(a, s);
}

}  // namespace

cudaError_t launch_gdn_recurrent(const GdnArgs& a, cudaStream_t s) {
  if (a.n_seq <= 0) return cudaSuccess;
  if (a.d == 128)
    return a.dtype == HLA_BF16 ? launch_d<128, __nv_bfloat16>(a, s) : launch_d<128, float>(a, s);
  return a.dtype == HLA_BF16 ? launch_d<64, __nv_bfloat16>(a, s) : launch_d<64, float>(a, s);
}

}  // namespace hla
