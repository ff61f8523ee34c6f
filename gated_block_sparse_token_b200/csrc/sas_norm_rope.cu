// Per-head RMSNorm of queries and keys with the position rotation in the same
// pass, and its gradient.
//
//   x^ = x / sqrt(mean_d x_d^2 + eps)           (one row = one token and head)
//   z  = gamma * x^
//   y_i = z_i cos - z_(i+64) sin,  y_(i+64) = z_(i+64) cos + z_i sin,
//         angle = pos * base^(-2i/128), i = 0 .. 63
// gradient, for dL/dy:
//   dz = rotation transposed of dy;  dgamma += dz * x^ (all rows);
//   u = gamma * dz;  dx = (u - x^ * mean_d(u x^)) / sqrt(mean x^2 + eps)
//
// Both are bound by memory: a row is read and written once (the gradient
// reads x and dy).  Eight lanes hold a row: lane j dims 8j .. 8j+7 and their
// rotate-half partners 64 + 8j .. 64 + 8j + 7, so the rotation needs no
// exchange and the mean one 8-lane reduction (three shuffles).  An 8-lane group
// keeps its token's 8 (cos, sin) pairs in registers over a chunk of heads:
// the angles are reduced in double precision (exact for any int32 position)
// and would otherwise cost more than the row.  Measured, bf16, 32 + 8 heads:
// 2 x 32,768 tokens 210 us (6.4 TB/s), one decode step of 8 sequences 2.5 us;
// gradient, with the gains' sum and the caller's zeroing of them, of 8 x 1,021
// padded tokens of 40 + 8 heads 42 us (5.4 TB/s), of 2 x 32,768 tokens 308 (6.5
// TB/s).  fp32: 462, 85 and 630 us (5.8, 5.3 and 6.4 TB/s).
#include "sas_internal.h"

namespace sas {

namespace {

constexpr int kNrRowsPerCta = kNrThreads / 8;  // token slots of a CTA

// 8 consecutive elements as loaded (16-byte aligned), and as fp32.
template <typename T>
struct Raw8 {
  uint4 r[sizeof(T) / 2];
};
// the ring of the next heads: slots, and bytes of one (16-byte pieces of x, and of dy, a thread)
constexpr int kNrStages = 4;
__host__ __device__ constexpr int nr_stage(bool back) { return (back ? 4 : 2) * 16 * kNrThreads; }

template <typename T>
__device__ __forceinline__ void load8(const T* p, Raw8<T>& x) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) x.r[i] = reinterpret_cast<const uint4*>(p)[i];
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& v, float (&x)[8]) {
  const uint4 r = v.r[0];
  x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
  x[4] = bf16_lo(r.z), x[5] = bf16_hi(r.z), x[6] = bf16_lo(r.w), x[7] = bf16_hi(r.w);
}
__device__ __forceinline__ void unpack8(const Raw8<float>& v, float (&x)[8]) {
  const uint4 a = v.r[0], b = v.r[1];
  x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
  x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y), x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ float sum8lanes(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  return v;
}

}  // namespace

// blockIdx.y: a chunk of p.chunk heads, the query heads' chunks first (a
// chunk never mixes queries and keys); blockIdx.x: tokens, 32 at a time.
template <typename T, bool kBack, bool kRing>
__global__ void __launch_bounds__(kNrThreads, kBack ? 2 : 4)
    norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, j = lane & 7;
  const bool is_q = static_cast<int>(blockIdx.y) < p.q_chunks;
  const int h0 = (is_q ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) - p.q_chunks) * p.chunk;
  const int h1 = min(h0 + p.chunk, is_q ? p.hq : p.hkv);
  const RowsView xv = is_q ? p.x_q : p.x_k, yv = is_q ? p.y_q : p.y_k, dv = is_q ? p.d_q : p.d_k;
  const float* gamma = is_q ? p.gamma_q : p.gamma_k;
  float glo[8], ghi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    glo[e] = gamma[8 * j + e];
    ghi[e] = gamma[64 + 8 * j + e];
  }
  float alo[8], ahi[8];  // gradient: this lane's share of dgamma
#pragma unroll
  for (int e = 0; e < 8; ++e) alo[e] = ahi[e] = 0.f;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  static_assert(!kRing || sizeof(T) == 2, "one 16-byte piece is eight elements");
  const uint32_t ring = kRing ? smem_u32(smem_raw) + 16 * tid : 0u;

  const int n_tok = p.batch * p.tokens;
  for (int n0 = static_cast<int>(blockIdx.x) * kNrRowsPerCta; n0 < n_tok;
       n0 += static_cast<int>(gridDim.x) * kNrRowsPerCta) {
    const int n = n0 + (tid >> 3);
    const int s = n / p.tokens, t = n - s * p.tokens;
    const int pos = n < n_tok ? (p.positions != nullptr ? p.positions[n] : t) : -1;
    const bool live = pos >= 0;  // uniform over the 8 lanes of a row
    const long long off = static_cast<long long>(s) * xv.seq + static_cast<long long>(t) * xv.token + 8 * j;
    const T* x = static_cast<const T*>(xv.data) + off;
    T* y = static_cast<T*>(const_cast<void*>(yv.data)) + static_cast<long long>(s) * yv.seq +
           static_cast<long long>(t) * yv.token + 8 * j;
    const T* dy = static_cast<const T*>(dv.data) + static_cast<long long>(s) * dv.seq +
                  static_cast<long long>(t) * dv.token + 8 * j;
    // The next heads' loads go out before this one's store, which the compiler
    // could not arrange: the output may be the input.  bf16: every lane copies its
    // pieces of the next three heads to its own places in shared memory; an SM's
    // registers hold one head ahead (2 x 32,768 tokens of 32 + 8 heads 212 against
    // 228 us, the gradient of 8 x 1,021 of 40 + 8 42 against 50).  An fp32 lane's
    // pieces are every other 16 bytes, half sectors to such a copy: through
    // registers (gradient 84 us against 138), as is a single head (a decode step:
    // 2.5 us against 2.6).
    Raw8<T> bx[2], bd[2];
    const auto slot = [&](int h) { return ring + static_cast<uint32_t>(h - h0) % kNrStages * nr_stage(kBack); };
    auto fetch = [&](int h) {
      if constexpr (kRing) {
        const uint8_t* sx = reinterpret_cast<const uint8_t*>(x + h * xv.head);
        const uint8_t* sd = reinterpret_cast<const uint8_t*>(dy + h * dv.head);
        cp_async16(slot(h), sx);
        cp_async16(slot(h) + 16 * kNrThreads, sx + 128);
        if constexpr (kBack) {
          cp_async16(slot(h) + 32 * kNrThreads, sd);
          cp_async16(slot(h) + 48 * kNrThreads, sd + 128);
        }
        return;
      }
      load8(x + h * xv.head, bx[0]);
      load8(x + h * xv.head + 64, bx[1]);
      if constexpr (kBack) {
        load8(dy + h * dv.head, bd[0]);
        load8(dy + h * dv.head + 64, bd[1]);
      }
    };
    bx[0] = bx[1] = bd[0] = bd[1] = Raw8<T>{};
    if constexpr (kRing) {
#pragma unroll
      for (int i = 0; i < kNrStages - 1; ++i) {
        if (live && h0 + i < h1) fetch(h0 + i);
        cp_async_commit();
      }
    } else {
      if (live) fetch(h0);
    }
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) rope_cos_sin(p.rope.theta_over_pi[8 * j + e], max(pos, 0), cs[e], sn[e]);
    for (int h = h0; h < h1; ++h) {
      if constexpr (kRing) {
        cp_async_wait<kNrStages - 2>();
        if (live) {
          bx[0].r[0] = lds128(slot(h));
          bx[1].r[0] = lds128(slot(h) + 16 * kNrThreads);
          if constexpr (kBack) {
            bd[0].r[0] = lds128(slot(h) + 32 * kNrThreads);
            bd[1].r[0] = lds128(slot(h) + 48 * kNrThreads);
          }
        }
        if (live && h + kNrStages - 1 < h1) fetch(h + kNrStages - 1);  // into the place of the head before
        cp_async_commit();
      }
      float lo[8], hi[8];
      unpack8(bx[0], lo);
      unpack8(bx[1], hi);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], ss));
      if constexpr (!kBack) {
        if (!kRing && live && h + 1 < h1) fetch(h + 1);
        const float r = rsqrtf(sum8lanes(ss) * (1.f / kDim) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float a = lo[e] * r * glo[e], b = hi[e] * r * ghi[e];
          lo[e] = a * cs[e] - b * sn[e];
          hi[e] = b * cs[e] + a * sn[e];
        }
      } else {
        float dlo[8], dhi[8];
        unpack8(bd[0], dlo);
        unpack8(bd[1], dhi);
        if (!kRing && live && h + 1 < h1) fetch(h + 1);
        // a row that is not live is zeros here: r 0 keeps it out of the gains' sums
        // also where eps is 0 and 1 / sqrt(mean + eps) infinite
        const float inv = rsqrtf(sum8lanes(ss) * (1.f / kDim) + p.eps);
        const float r = live ? inv : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float zl = dlo[e] * cs[e] + dhi[e] * sn[e];
          const float zh = dhi[e] * cs[e] - dlo[e] * sn[e];
          lo[e] *= r;
          hi[e] *= r;
          alo[e] = fmaf(zl, lo[e], alo[e]);
          ahi[e] = fmaf(zh, hi[e], ahi[e]);
          dlo[e] = zl * glo[e];
          dhi[e] = zh * ghi[e];
          dot = fmaf(dlo[e], lo[e], fmaf(dhi[e], hi[e], dot));
        }
        const float m = sum8lanes(dot) * (1.f / kDim);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = r * (dlo[e] - lo[e] * m);
          hi[e] = r * (dhi[e] - hi[e] * m);
        }
      }
      if (live) {
        store8(y + h * yv.head, lo);
        store8(y + h * yv.head + 64, hi);
      }
    }
  }

  if constexpr (kBack) {
    // the CTA's sum per dimension: the four rows of a warp, then the warps,
    // in a fixed order
    __shared__ float part[kNrThreads / 32][kDim];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) {
        alo[e] += __shfl_xor_sync(0xffffffffu, alo[e], o);
        ahi[e] += __shfl_xor_sync(0xffffffffu, ahi[e], o);
      }
    }
    if (lane < 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        part[tid >> 5][8 * j + e] = alo[e];
        part[tid >> 5][64 + 8 * j + e] = ahi[e];
      }
    }
    __syncthreads();
    if (tid < kDim) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kNrThreads / 32; ++w) v += part[w][tid];
      p.ws_part[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kDim + tid] = v;
    }
  }
}

// dgamma += the CTAs' partial sums, in a fixed order.  CTA (i, which): 32
// columns of the query (0) or key (1) gain; warp w sums rows w, w + 32, ..
__global__ void __launch_bounds__(1024) norm_rope_gain_kernel(const float* part, int q_rows, int k_rows,
                                                              float* dgamma_q, float* dgamma_k) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const bool is_q = blockIdx.y == 0;
  float* out = is_q ? dgamma_q : dgamma_k;
  const int rows = is_q ? q_rows : k_rows;
  const float* src = part + (is_q ? 0 : static_cast<size_t>(q_rows) * kDim) + 32 * blockIdx.x + lane;
  float v = 0.f;
  for (int r = w; r < rows; r += 32) v += src[static_cast<size_t>(r) * kDim];
  acc[w][lane] = v;
  __syncthreads();
  if (w == 0 && rows > 0) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += acc[k][lane];
    out[32 * blockIdx.x + lane] += t;
  }
}

cudaError_t launch_norm_rope(bool f32, bool back, NormRopeParams p, float* dgamma_q, float* dgamma_k,
                             cudaStream_t stream) {
  const NormRopeGrid g = norm_rope_grid(p.batch, p.tokens, p.hq, p.hkv, back);
  p.chunk = g.chunk;
  p.q_chunks = g.q_chunks;
  const dim3 grid(static_cast<unsigned>(g.x), static_cast<unsigned>(g.q_chunks + g.k_chunks));
  const bool ring = !f32 && g.chunk > 1;
  const size_t smem = ring ? kNrStages * nr_stage(back) : 0;
  const auto go = [&](auto* kernel) { return launch_pdl(kernel, grid, kNrThreads, smem, stream, 0, p); };
  if (!back)
    return f32 ? go(norm_rope_kernel<float, false, false>)
               : (ring ? go(norm_rope_kernel<__nv_bfloat16, false, true>)
                       : go(norm_rope_kernel<__nv_bfloat16, false, false>));
  const cudaError_t e = f32 ? go(norm_rope_kernel<float, true, false>)
                            : (ring ? go(norm_rope_kernel<__nv_bfloat16, true, true>)
                                    : go(norm_rope_kernel<__nv_bfloat16, true, false>));
  if (e != cudaSuccess) return e;
  int q_rows = g.q_chunks * g.x, k_rows = g.k_chunks * g.x;
  if (dgamma_q == dgamma_k && p.hq > 0 && p.hkv > 0) q_rows += k_rows, k_rows = 0;  // one gain: one sum
  return launch_pdl(norm_rope_gain_kernel, dim3(kDim / 32, 2), 1024, 0, stream, 0, p.ws_part, q_rows, k_rows, dgamma_q,
                    dgamma_k);
}

cudaError_t prepare_norm_rope_kernels() {
  return cudaFuncSetAttribute(norm_rope_kernel<__nv_bfloat16, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kNrStages * nr_stage(true));
}

}  // namespace sas
