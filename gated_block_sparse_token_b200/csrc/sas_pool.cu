// SAS key-block pooling and gate keys.
//
// Method (release pages: keys pooled per block by max, min and average, Q/K
// normalisation and gate RoPE on, gate hidden size 128): for a
// complete 64-token block b of (sequence s, KV head h)
//   P_b  = [max_j K_j ; min_j K_j ; mean_j K_j]          (384 = 3 x 128)
//   k~_b = RoPE(RMSNorm(P_b @ W_k[h]) * gamma_k, position b)
//
// One CTA handles up to kPoolBlocksPerCta consecutive blocks of one (s, h).
// W_k[h] (96 KiB bf16) comes into shared memory with one TMA bulk copy that
// overlaps the pooling; each warp pools whole blocks (16-byte loads, 16 rows
// in flight per lane, reduced in registers and across the lanes that share
// a column chunk).  The 384x128 projection of all the CTA's blocks then runs
// out of shared memory at once, thread d owning output dimension d.
#include <cmath>

#include "sas_internal.h"

namespace sas {

template <typename T>
__global__ void __launch_bounds__(kThreads) pool_keys_kernel(const __grid_constant__ PoolParams p) {
  constexpr int NB = kPoolBlocksPerCta;
  constexpr int VEC = 16 / static_cast<int>(sizeof(T));  // elements per 16-byte load
  constexpr int TPR = kDim / VEC;                       // lanes per K row
  const int s = blockIdx.z;
  const int h = blockIdx.y;
  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;

  extern __shared__ __align__(16) uint8_t smem_raw[];
  __nv_bfloat16* wk_s = reinterpret_cast<__nv_bfloat16*>(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem_raw + kPoolWkBytes);
  // pooled blocks, [pooled dim][block]; reused for the normalised u, [block][dim]
  __shared__ __align__(16) float Pt[kPool][NB];
  float (*xs)[kDim] = reinterpret_cast<float (*)[kDim]>(&Pt[0][0]);
  __shared__ float ssq[kWarps][NB];

  const int L = (p.kv.seq_lens != nullptr) ? p.kv.seq_lens[s] : p.kv.capacity;  // prefill: full length
  const int first = p.blk_begin != nullptr ? p.blk_begin[s] : 0;
  const int b0 = first + static_cast<int>(blockIdx.x) * NB;
  const int b_end = first + p.num_blocks;

  long long rows[NB];
  int nb = 0;
  bool err = false;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int b = b0 + i;
    rows[i] = -1;
    // only complete blocks that have a gate-key row are pooled
    if (b >= 0 && b < b_end && b < p.mg && L >= 1 &&
        static_cast<long long>(b + 1) * kBlock <= static_cast<long long>(L)) {
      rows[i] = p.kv.block_row(s, h, b);
      if (rows[i] < 0)
        err = true;
      else
        nb = i + 1;
    }
  }
  if (err && tid == 0) raise_status(p.status, kStatusBounds);
  if (nb == 0) return;  // uniform over the CTA

  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(bar, kPoolWkBytes);
    bulk_g2s(wk_s, p.w_k + static_cast<size_t>(h) * kPool * kDim, kPoolWkBytes, bar);
  }

  // ---- pooling: max, min, mean over the 64 tokens, per dimension.  Warp w
  // pools blocks w, w + 4, ...: lane l reads the 16-byte chunk l % TPR of
  // rows l / TPR, l / TPR + RPW, ... (16 rows' loads in flight per lane)
  {
    constexpr int RPW = 32 / TPR;          // rows per warp step (2 bf16, 1 fp32)
    constexpr int ROWS = kBlock / RPW;     // rows per lane
    const T* kbase = static_cast<const T*>(p.kv.k);
    const int cvec = lane % TPR, par = lane / TPR;
    for (int i = warp; i < NB; i += kWarps) {  // warp-uniform
      float mx[VEC], mn[VEC], sm[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        mx[v] = -INFINITY;
        mn[v] = INFINITY;
        sm[v] = 0.f;
      }
      if (rows[i] >= 0) {
        const T* blk = kbase + (rows[i] + par) * kDim + cvec * VEC;
#pragma unroll
        for (int part = 0; part < ROWS / 16; ++part) {
          uint4 raw[16];
#pragma unroll
          for (int r = 0; r < 16; ++r)
            raw[r] = *reinterpret_cast<const uint4*>(blk + static_cast<size_t>(RPW * (16 * part + r)) * kDim);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const T* e = reinterpret_cast<const T*>(&raw[r]);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
              const float x = to_float(e[v]);
              mx[v] = fmaxf(mx[v], x);
              mn[v] = fminf(mn[v], x);
              sm[v] += x;
            }
          }
        }
      }
#pragma unroll
      for (int o = TPR; o < 32; o <<= 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          mx[v] = fmaxf(mx[v], __shfl_xor_sync(0xffffffffu, mx[v], o));
          mn[v] = fminf(mn[v], __shfl_xor_sync(0xffffffffu, mn[v], o));
          sm[v] += __shfl_xor_sync(0xffffffffu, sm[v], o);
        }
      }
      if (par == 0) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const int dd = cvec * VEC + v;
          const float mean = sm[v] * (1.f / kBlock);
          Pt[dd][i] = rows[i] >= 0 ? mx[v] : 0.f;
          Pt[kDim + dd][i] = rows[i] >= 0 ? mn[v] : 0.f;
          Pt[2 * kDim + dd][i] = mean;
          if (p.pooled_raw != nullptr && rows[i] >= 0) {
            float* pr = p.pooled_raw + ((static_cast<size_t>(s) * p.hkv + h) * p.mg + (b0 + i)) * kPool;
            pr[dd] = mx[v];
            pr[kDim + dd] = mn[v];
            pr[2 * kDim + dd] = mean;
          }
        }
      }
    }
  }
  __syncthreads();

  // ---- u = P @ W_k[h] from shared memory, thread d owning output dimension d
  const bool ok = mbar_wait(bar, 0, p.status);
  const int d = tid;
  float u[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) u[i] = 0.f;
  if (ok) {
#pragma unroll 4
    for (int r = 0; r < kPool; ++r) {
      const float w = __bfloat162float(wk_s[r * kDim + d]);
      const float4* p4 = reinterpret_cast<const float4*>(&Pt[r][0]);
#pragma unroll
      for (int c = 0; c < NB / 4; ++c) {
        const float4 x = p4[c];
        u[4 * c] = fmaf(x.x, w, u[4 * c]);
        u[4 * c + 1] = fmaf(x.y, w, u[4 * c + 1]);
        u[4 * c + 2] = fmaf(x.z, w, u[4 * c + 2]);
        u[4 * c + 3] = fmaf(x.w, w, u[4 * c + 3]);
      }
    }
  }

  // ---- RMSNorm (gain gamma_k) and gate RoPE at the block index, per block
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    float sq = u[i] * u[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) ssq[warp][i] = sq;
  }
  __syncthreads();  // every Pt read is done: xs may overwrite it
  const float gk = p.gamma_k[d];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const float tot = ssq[0][i] + ssq[1][i] + ssq[2][i] + ssq[3][i];
    xs[i][d] = u[i] * (1.f / sqrtf(tot / kDim + p.eps)) * gk;
  }
  __syncthreads();
  const int j = d & 63;
  for (int i = 0; i < nb; ++i) {
    if (rows[i] < 0) continue;
    const int b = b0 + i;
    float cs, sn;
    rope_cos_sin(p.rope.theta_over_pi[j], b, cs, sn);
    const float y = (d < 64) ? xs[i][d] * cs - xs[i][d + 64] * sn : xs[i][d] * cs + xs[i][d - 64] * sn;
    const size_t gi = ((static_cast<size_t>(s) * p.hkv + h) * p.mg + b) * kDim + d;
    if (p.gk16)
      static_cast<__nv_bfloat16*>(p.gate_keys)[gi] = __float2bfloat16_rn(y);
    else
      static_cast<float*>(p.gate_keys)[gi] = y;
  }
}

cudaError_t launch_pool(bool f32_kv, const PoolParams& p, int batch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.num_blocks + kPoolBlocksPerCta - 1) / kPoolBlocksPerCta),
                  static_cast<unsigned>(p.hkv), static_cast<unsigned>(batch));
  const size_t smem = pool_smem_bytes();
  if (f32_kv)
    pool_keys_kernel<float><<<grid, kThreads, smem, stream>>>(p);
  else
    pool_keys_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

size_t pool_smem_bytes() { return static_cast<size_t>(kPoolWkBytes) + 16; }

cudaError_t prepare_pool_project_kernel();

cudaError_t prepare_pool_kernels() {
  const cudaError_t e0 = prepare_pool_project_kernel();
  if (e0 != cudaSuccess) return e0;
  cudaError_t e = cudaFuncSetAttribute(pool_keys_kernel<float>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(pool_smem_bytes()));
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(pool_keys_kernel<__nv_bfloat16>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(pool_smem_bytes()));
}

void fill_rope_table(RopeTable& t, float base) {
  // 64 powers cost a small kernel's launch: each host thread keeps the table
  // of the last base it was asked for
  thread_local float last_base = 0.f;  // no valid base
  thread_local RopeTable last;
  if (base != last_base) {
    for (int i = 0; i < 64; ++i)
      last.theta_over_pi[i] = std::pow(static_cast<double>(base), -2.0 * i / kDim) / M_PI;
    last_base = base;
  }
  t = last;
}

// ---------------------------------------------------------------- tensor-core pooling and projection
// The same pooled keys and gate keys for bf16 caches, with the projection on
// the 5th-generation tensor cores.  One CTA (256 threads) per 128 blocks of
// one (sequence, KV head):
//   1. W_k[h] (96 KiB bf16) comes in by TMA, 128-byte swizzled, as the
//      MN-major B operand [384 x 128]; tensor memory: 128 fp32 columns.
//   2. the 8 warps pool the tile's blocks straight from global memory
//      (16-byte loads, 16 per lane in flight) and write row i of the A
//      operand [128 x 512] bf16, K-major and 128-byte swizzled:
//      [max | min | mean_hi | mean_lo], where mean_hi = bf16(mean) and
//      mean_lo = bf16(mean - mean_hi).  max and min are elements of K (exact
//      in bf16) and hi + lo carries the fp32 mean to within 2^-17 of it, so
//      the bf16 x bf16 products the tensor core accumulates in fp32 give
//      u = P @ W_k to fp32 accuracy (the mean's W_k rows serve both hi and lo).
//   3. one thread issues the 32 MMAs (M = 128 blocks, N = 128, K = 16 each).
//   4. the epilogue reads u from tensor memory (a thread per block, two
//      warps per lane quarter, each half the rotate-half pairs), applies
//      RMSNorm, gamma_k and the gate RoPE at the block index, and stores the
//      gate keys.
// SRC: the cache's elements, bf16 or (an 8-bit cache) codes under one scale a
// block.  Codes and their mean are pooled in units of the scale -- exact in
// bf16, the mean as hi + lo -- and the epilogue multiplies u by the block's
// scale, so the 8-bit form reads half the bytes and rounds nothing more.  Its
// codes come through a cp.async ring in the space of W_k, which is fetched (from
// L2) once the pooling is done: with 227 KiB of shared memory taken, the L1 that
// ordinary loads return through holds too little in flight (39.4 us).
constexpr int kPpRows = 128;          // blocks per CTA (the MMA's M)
constexpr int kPpThreads = 256;
constexpr int kPpA = kPpRows * 512 * 2;           // A operand bytes (8 chunks of 16 KiB)
constexpr int kPpB = kPool * kDim * 2;            // B operand bytes (2 N-halves of 48 KiB)
constexpr int kPpSmem = kPpA + kPpB + 2 * kPpRows * 4 + 64 + 1024;

enum PoolSource : int { kSrcE4m3 = kCodeE4m3, kSrcInt8 = kCodeInt8, kSrcBf16 };

// Pooled codes of dims 4 lane .. 4 lane + 3 (a lane's four codes of each row, so
// that nothing is left to reduce across lanes): maximum and minimum as f16 pairs
// (dims 0, 1 and 2, 3), the sums in fp32 -- all exact (sums are multiples of
// 2^-9 below 2^15, or integers below 2^17).  int8 codes stay biased by 1152 until
// the end (exact in f16): taking the bias off each would cost as much as the
// maxima.
template <int CODE>
struct PooledCodes {
  uint32_t hx[2], hn[2];
  float sm[4];

  template <int ROWS>
  __device__ __forceinline__ void add(const uint32_t (&raw)[ROWS], bool first) {
    if (first) {
#pragma unroll
      for (int v = 0; v < 4; ++v) sm[v] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      uint32_t c[2];
      if constexpr (CODE == kCodeE4m3) {
        codes_f16<CODE>(raw[r], c[0], c[1]);
      } else {
        const uint32_t w = raw[r] ^ 0x80808080u;
        c[0] = __byte_perm(w, 0x64646464u, 0x4140);
        c[1] = __byte_perm(w, 0x64646464u, 0x4342);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool init = first && r == 0;
        hx[k] = init ? c[k] : max_f16x2(hx[k], c[k]);
        hn[k] = init ? c[k] : min_f16x2(hn[k], c[k]);
        add_f16x2(sm[2 * k], sm[2 * k + 1], c[k]);
      }
    }
  }
  // mx, mn, sm over all of `rows` rows
  __device__ __forceinline__ void get(int rows, float (&mx)[4], float (&mn)[4], float (&s)[4]) const {
    constexpr float bias = CODE == kCodeInt8 ? 1152.f : 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mx[2 * k] = f16_lo(hx[k]) - bias, mx[2 * k + 1] = f16_hi(hx[k]) - bias;
      mn[2 * k] = f16_lo(hn[k]) - bias, mn[2 * k + 1] = f16_hi(hn[k]) - bias;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) s[v] = sm[v] - static_cast<float>(rows) * bias;
  }
};

template <int ROWS>
__device__ __forceinline__ void load_codes(uint32_t (&raw)[ROWS], const uint8_t* src) {
#pragma unroll
  for (int r = 0; r < ROWS; ++r) raw[r] = *reinterpret_cast<const uint32_t*>(src + r * kDim);
}

// Threads of the kernel for a source: codes are pooled by sixteen warps (the
// loop over a block's words is bound by instruction issue, twice the values a
// word of bf16).
__host__ __device__ constexpr int pp_threads(int src) { return src == kSrcBf16 ? kPpThreads : 2 * kPpThreads; }

template <int SRC>
__global__ void __launch_bounds__(pp_threads(SRC), 1) pool_project_kernel(const __grid_constant__ PoolParams p,
                                                                     const __grid_constant__ CUtensorMap tmwk) {
  if constexpr (SRC != kSrcBf16) {  // launched with programmatic stream serialization
    griddep_launch_dependents();
    griddep_wait();
  }
  const int s = blockIdx.z;
  const int h = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = base;
  uint8_t* sB = base + kPpA;
  float* ssq = reinterpret_cast<float*>(sB + kPpB);  // [2][128] partial sums of squares
  uint64_t* bars = reinterpret_cast<uint64_t*>(ssq + 2 * kPpRows);  // W_k, MMA done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2);

  const int L = (p.kv.seq_lens != nullptr) ? p.kv.seq_lens[s] : p.kv.capacity;  // prefill: full length
  const int first = p.blk_begin != nullptr ? p.blk_begin[s] : 0;
  const int b0 = first + static_cast<int>(blockIdx.x) * kPpRows;
  const int b_end = first + p.num_blocks;
  auto row_of = [&](int i) -> long long {  // cache row of tile row i; -1: not pooled; -2: out of range
    const int b = b0 + i;
    if (b < 0 || b >= b_end || b >= p.mg || L < 1 || static_cast<long long>(b + 1) * kBlock > L) return -1;
    const long long r = p.kv.block_row(s, h, b);
    return r < 0 ? -2 : r;
  };
  // rows that may hold work: blocks max(b0, 0) .. min(b0 + 128, b_end, mg, L / 64) - 1
  const int hi = min(min(b0 + kPpRows, b_end), min(p.mg, L >= 1 ? L / kBlock : 0));
  if (max(b0, 0) >= hi) return;  // uniform over the CTA

  const auto fetch_wk = [&]() {  // one thread
    mbar_arrive_expect_tx(&bars[0], kPpB);
    for (int c = 0; c < 2; ++c)
      for (int r = 0; r < kPool / 64; ++r)
        tma_load_2d(sB + c * (kPool * 128) + r * 8192, &tmwk, 64 * c, h * kPool + 64 * r, &bars[0]);
  };
  if (tid == 0) {
    prefetch_tensormap(&tmwk);
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
    if (SRC == kSrcBf16) fetch_wk();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 128);
    tmem_relinquish();
  }

  // ---- pooling into the A operand
  if constexpr (SRC != kSrcBf16) {
    bool err = false;
    // a warp's blocks i, i + 16, ..: each in quarters of 16 rows through the warp's
    // ring of three; the next block's cache row known a block ahead
    constexpr int STEP = pp_threads(SRC) / 32, Q = 16, SLOTS = 3, SLOT = Q * kDim;
    static_assert(STEP * SLOTS * SLOT <= kPpB, "the rings fit W_k's space");
    const uint32_t ring = smem_u32(sB) + warp * (SLOTS * SLOT);
    const uint8_t* kb = static_cast<const uint8_t*>(p.kv.k);
    long long row = row_of(warp), row_n = row_of(warp + STEP);
    const int n_rows = hi - b0;  // rows past the last block stay unwritten: the product's
                                 // rows are independent, and theirs are not read
    const auto issue = [&](uint32_t slot, long long r, int k) {  // quarter k of the block at row r
      if (r >= 0) {
        const uint8_t* src = kb + (r + Q * k) * kDim + 16 * lane;
#pragma unroll
        for (int i = 0; i < SLOT / 512; ++i) cp_async16(slot + 512 * i + 16 * lane, src + 512 * i);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) issue(ring + k * SLOT, warp < n_rows ? row : -1, k);
    uint32_t slot = ring;
    for (int i = warp; i < n_rows; i += STEP) {  // warp-uniform
      if (row == -2) err = true;
      const long long row_2n = i + 2 * STEP < kPpRows ? row_of(i + 2 * STEP) : -1;
      const long long next = i + STEP < n_rows ? row_n : -1;
      float mx[4] = {0.f, 0.f, 0.f, 0.f}, mn[4] = {0.f, 0.f, 0.f, 0.f}, sm[4] = {0.f, 0.f, 0.f, 0.f};
      PooledCodes<SRC> pool;
#pragma unroll
      for (int k = 0; k < kBlock / Q; ++k) {
        cp_async_wait<SLOTS - 1>();
        __syncwarp();
        uint32_t r[Q];
#pragma unroll
        for (int v = 0; v < Q; ++v)
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[v]) : "r"(slot + v * kDim + 4 * lane) : "memory");
        __syncwarp();  // the slot is read: refill it
        issue(slot, k + SLOTS < kBlock / Q ? row : next, (k + SLOTS) % (kBlock / Q));
        pool.add(r, k == 0);
        slot = slot + SLOT == ring + SLOTS * SLOT ? ring : slot + SLOT;
      }
      if (row >= 0) pool.get(kBlock, mx, mn, sm);
      uint32_t pk[4][2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float m0 = sm[2 * v] * (1.f / kBlock), m1 = sm[2 * v + 1] * (1.f / kBlock);
        const float g0 = __bfloat162float(__float2bfloat16_rn(m0)), g1 = __bfloat162float(__float2bfloat16_rn(m1));
        pk[0][v] = pack_bf16x2(mx[2 * v], mx[2 * v + 1]);
        pk[1][v] = pack_bf16x2(mn[2 * v], mn[2 * v + 1]);
        pk[2][v] = pack_bf16x2(g0, g1);
        pk[3][v] = pack_bf16x2(m0 - g0, m1 - g1);
      }
      // K index sec * 128 + 4 lane: chunk 2 sec + lane / 16, 16-byte unit (lane / 2) % 8, half lane % 2
#pragma unroll
      for (int sec = 0; sec < 4; ++sec)
        *reinterpret_cast<uint2*>(sA + (2 * sec + (lane >> 4)) * (kPpRows * 128) + i * 128 +
                                  ((((lane >> 1) & 7) ^ (i & 7)) << 4) + 8 * (lane & 1)) =
            make_uint2(pk[sec][0], pk[sec][1]);
      if (p.pooled_raw != nullptr && row >= 0) {
        const float sc = p.k_scale[row / kBlock];
        float* pr = p.pooled_raw + ((static_cast<size_t>(s) * p.hkv + h) * p.mg + (b0 + i)) * kPool + lane * 4;
#pragma unroll
        for (int v = 0; v < 4; ++v) {  // 4-byte aligned: scalar stores
          pr[v] = mx[v] * sc;
          pr[kDim + v] = mn[v] * sc;
          pr[2 * kDim + v] = sm[v] * (1.f / kBlock) * sc;
        }
      }
      row = row_n;
      row_n = row_2n;
    }
    cp_async_wait<0>();
    if (err && lane == 0) raise_status(p.status, kStatusBounds);
  } else {
    constexpr int TPR = 16;             // lanes per K row (16-byte loads)
    const int cvec = lane % TPR, par = lane / TPR;
    const __nv_bfloat16* kbase = static_cast<const __nv_bfloat16*>(p.kv.k);
    bool err = false;
    for (int i = warp; i < kPpRows; i += kPpThreads / 32) {  // warp-uniform
      const long long row = row_of(i);
      if (row == -2) err = true;
      float mx[8], mn[8], sm[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        mx[v] = -INFINITY;
        mn[v] = INFINITY;
        sm[v] = 0.f;
      }
      if (row >= 0) {
        const __nv_bfloat16* blk = kbase + (row + par) * kDim + cvec * 8;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          uint4 raw[16];
#pragma unroll
          for (int r = 0; r < 16; ++r)
            raw[r] = *reinterpret_cast<const uint4*>(blk + static_cast<size_t>(2 * (16 * part + r)) * kDim);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const uint32_t w4[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float x0 = bf16_lo(w4[v]), x1 = bf16_hi(w4[v]);
              mx[2 * v] = fmaxf(mx[2 * v], x0);
              mn[2 * v] = fminf(mn[2 * v], x0);
              sm[2 * v] += x0;
              mx[2 * v + 1] = fmaxf(mx[2 * v + 1], x1);
              mn[2 * v + 1] = fminf(mn[2 * v + 1], x1);
              sm[2 * v + 1] += x1;
            }
          }
        }
      }
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        mx[v] = fmaxf(mx[v], __shfl_xor_sync(0xffffffffu, mx[v], 16));
        mn[v] = fminf(mn[v], __shfl_xor_sync(0xffffffffu, mn[v], 16));
        sm[v] += __shfl_xor_sync(0xffffffffu, sm[v], 16);
      }
      if (par == 0) {
        uint32_t pk[4][4];  // [max, min, hi, lo][4 bf16 pairs]
        float mean[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) mean[v] = (row >= 0) ? sm[v] * (1.f / kBlock) : 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float a0 = row >= 0 ? mx[2 * v] : 0.f, a1 = row >= 0 ? mx[2 * v + 1] : 0.f;
          const float n0 = row >= 0 ? mn[2 * v] : 0.f, n1 = row >= 0 ? mn[2 * v + 1] : 0.f;
          const __nv_bfloat16 h0 = __float2bfloat16_rn(mean[2 * v]), h1 = __float2bfloat16_rn(mean[2 * v + 1]);
          pk[0][v] = pack_bf16x2(a0, a1);
          pk[1][v] = pack_bf16x2(n0, n1);
          pk[2][v] = pack_bf16x2(__bfloat162float(h0), __bfloat162float(h1));
          pk[3][v] = pack_bf16x2(mean[2 * v] - __bfloat162float(h0), mean[2 * v + 1] - __bfloat162float(h1));
        }
        // K index sec * 128 + 8 cvec: chunk 2 sec + cvec / 8, 16-byte unit cvec % 8
#pragma unroll
        for (int sec = 0; sec < 4; ++sec) {
          const int kc = 2 * sec + (cvec >> 3);
          const int j = cvec & 7;
          *reinterpret_cast<uint4*>(sA + kc * (kPpRows * 128) + i * 128 + ((j ^ (i & 7)) << 4)) =
              make_uint4(pk[sec][0], pk[sec][1], pk[sec][2], pk[sec][3]);
        }
        if (p.pooled_raw != nullptr && row >= 0) {
          float* pr = p.pooled_raw + ((static_cast<size_t>(s) * p.hkv + h) * p.mg + (b0 + i)) * kPool + cvec * 8;
#pragma unroll
          for (int v = 0; v < 8; ++v) {  // 4-byte aligned: scalar stores
            pr[v] = mx[v];
            pr[kDim + v] = mn[v];
            pr[2 * kDim + v] = mean[v];
          }
        }
      }
    }
    if (err && lane == 0) raise_status(p.status, kStatusBounds);
  }
  fence_proxy_async_smem();  // the A rows written here are read by the tensor core (async proxy)
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // ---- u = A @ B on the tensor cores
  if (tid == 0) {
    if (SRC != kSrcBf16) fetch_wk();  // every thread has fenced its use of the ring
    const bool okb = mbar_wait(&bars[0], 0, p.status);
    tc_fence_after_sync();
    if (okb) {
      const uint64_t dA = umma_desc_sw128(smem_u32(sA), 16, 1024);
      const uint64_t dB = umma_desc_sw128(smem_u32(sB), kPool * 128, 1024);
      constexpr uint32_t idesc = umma_idesc_bf16(kPpRows, kDim, false, true);
#pragma unroll
      for (int kk = 0; kk < 32; ++kk) {
        const uint32_t a_off = (kk >> 2) * (kPpRows * 128) + (kk & 3) * 32;
        const uint32_t brow = (kk < 24) ? 16 * kk : 16 * (kk - 8);  // the mean rows serve hi and lo
        umma_bf16_ss(tmem, dA + (a_off >> 4), dB + ((brow * 128) >> 4), idesc, kk > 0);
      }
    }
    umma_commit(&bars[1]);  // also when nothing was issued: the barrier still completes
  }
  const bool okm = mbar_wait(&bars[1], 0, p.status);
  tc_fence_after_sync();

  // ---- epilogue: RMSNorm, gain, RoPE at the block index, store
  {
    // lane quarter; part of the rotate-half pairs, W of them
    constexpr int PARTS = pp_threads(SRC) / 128, W = 64 / PARTS;
    const int q4 = warp & 3, hf = warp >> 2;
    const int i = 32 * q4 + lane;             // tile row = block b0 + i
    const uint32_t tl = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    float* sq = SRC == kSrcBf16 ? ssq : reinterpret_cast<float*>(sA);  // four parts: over A, which is used
    float lo[W], hi[W];
    if constexpr (W == 32) {
      tmem_ld32(tl + W * hf, lo);       // columns W hf .. W hf + W - 1
      tmem_ld32(tl + 64 + W * hf, hi);  // their rotate-half partners
    } else {
      tmem_ld16(tl + W * hf, lo);
      tmem_ld16(tl + 64 + W * hf, hi);
    }
    tmem_wait_ld();
    const long long row = row_of(i);
    if constexpr (SRC != kSrcBf16) {
      const float sc = row >= 0 ? p.k_scale[row / kBlock] : 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        lo[k] *= sc;
        hi[k] *= sc;
      }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) ss = fmaf(lo[k], lo[k], fmaf(hi[k], hi[k], ss));
    sq[hf * kPpRows + i] = ss;
    __syncthreads();
    if (row >= 0 && okm) {
      const int b = b0 + i;
      float tot = sq[i] + sq[kPpRows + i];
      if constexpr (PARTS == 4) tot += sq[2 * kPpRows + i] + sq[3 * kPpRows + i];
      const float inv = 1.f / sqrtf(tot / kDim + p.eps);
      const size_t gi = ((static_cast<size_t>(s) * p.hkv + h) * p.mg + b) * kDim;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const int d = W * hf + k;
        const float x0 = lo[k] * inv * p.gamma_k[d];
        const float x1 = hi[k] * inv * p.gamma_k[d + 64];
        float cs, sn;
        rope_cos_sin(p.rope.theta_over_pi[d], b, cs, sn);
        lo[k] = x0 * cs - x1 * sn;
        hi[k] = x1 * cs + x0 * sn;
      }
      if (p.gk16) {
        __nv_bfloat16* g = static_cast<__nv_bfloat16*>(p.gate_keys) + gi;
#pragma unroll
        for (int k = 0; k < W; k += 8) {
          *reinterpret_cast<uint4*>(g + W * hf + k) =
              make_uint4(pack_bf16x2(lo[k], lo[k + 1]), pack_bf16x2(lo[k + 2], lo[k + 3]),
                         pack_bf16x2(lo[k + 4], lo[k + 5]), pack_bf16x2(lo[k + 6], lo[k + 7]));
          *reinterpret_cast<uint4*>(g + 64 + W * hf + k) =
              make_uint4(pack_bf16x2(hi[k], hi[k + 1]), pack_bf16x2(hi[k + 2], hi[k + 3]),
                         pack_bf16x2(hi[k + 4], hi[k + 5]), pack_bf16x2(hi[k + 6], hi[k + 7]));
        }
      } else {
        float* g = static_cast<float*>(p.gate_keys) + gi;
#pragma unroll
        for (int k = 0; k < W; k += 4) {
          *reinterpret_cast<float4*>(g + W * hf + k) = make_float4(lo[k], lo[k + 1], lo[k + 2], lo[k + 3]);
          *reinterpret_cast<float4*>(g + 64 + W * hf + k) = make_float4(hi[k], hi[k + 1], hi[k + 2], hi[k + 3]);
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 128);
}

cudaError_t launch_pool_project(const PoolParams& p, const CUtensorMap& tmwk, int batch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.num_blocks + kPpRows - 1) / kPpRows), static_cast<unsigned>(p.hkv),
                  static_cast<unsigned>(batch));
  pool_project_kernel<kSrcBf16><<<grid, kPpThreads, kPpSmem, stream>>>(p, tmwk);
  return cudaGetLastError();
}

cudaError_t launch_pool_project_kv8(int code, const PoolParams& p, const CUtensorMap& tmwk, int batch,
                                    cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.num_blocks + kPpRows - 1) / kPpRows), static_cast<unsigned>(p.hkv),
                  static_cast<unsigned>(batch));
  constexpr int T = pp_threads(kSrcE4m3);
  return code == kCodeE4m3 ? launch_pdl(pool_project_kernel<kSrcE4m3>, grid, T, kPpSmem, stream, 0, p, tmwk)
                           : launch_pdl(pool_project_kernel<kSrcInt8>, grid, T, kPpSmem, stream, 0, p, tmwk);
}

// ---------------------------------------------------------------- few blocks
// The gate keys of the few blocks that a decode step or a short append
// completes: one CTA (16 warps) per block instead of one per 128, so that
// nothing waits for a 128-row operand.  Warp w holds rows 24w .. 24w + 23 of
// W_k[h] in registers (requested before the block's codes are known), pools 4 of
// the block's rows, and multiplies its 24 pooled values once all are in; the
// sums over warps run in a fixed order, in fp32.
constexpr int kPfThreads = 512, kPfWarps = kPfThreads / 32, kPfRowsK = kPool / kPfWarps;

template <int CODE>
__global__ void __launch_bounds__(kPfThreads) pool_few_kernel(const __grid_constant__ PoolParams p) {
  __shared__ float part[3][kPfWarps][kDim];
  __shared__ float P[kPool];
  __shared__ float xs[kDim];
  __shared__ float ssq[kDim / 32];
  const int s = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  griddep_launch_dependents();
  griddep_wait();
  const int L = p.kv.seq_lens[s];
  const int b = (p.blk_begin != nullptr ? p.blk_begin[s] : 0) + static_cast<int>(blockIdx.x);
  if (b < 0 || b >= p.mg || L < 1 || static_cast<long long>(b + 1) * kBlock > L) return;  // uniform
  uint2 w[kPfRowsK];
  const __nv_bfloat16* wk = p.w_k + (static_cast<size_t>(h) * kPool + kPfRowsK * warp) * kDim + 4 * lane;
#pragma unroll
  for (int i = 0; i < kPfRowsK; ++i) w[i] = *reinterpret_cast<const uint2*>(wk + i * kDim);
  const long long row = p.kv.block_row(s, h, b);
  if (row < 0) {
    if (tid == 0) raise_status(p.status, kStatusBounds);
    return;
  }
  const float scale = p.k_scale[row / kBlock];
  {
    constexpr int R = kBlock / kPfWarps;
    float mx[4], mn[4], sm[4];
    uint32_t raw[R];
    load_codes(raw, static_cast<const uint8_t*>(p.kv.k) + (row + R * warp) * kDim + 4 * lane);
    PooledCodes<CODE> pool;
    pool.add(raw, true);
    pool.get(R, mx, mn, sm);
    *reinterpret_cast<float4*>(&part[0][warp][4 * lane]) = make_float4(mx[0], mx[1], mx[2], mx[3]);
    *reinterpret_cast<float4*>(&part[1][warp][4 * lane]) = make_float4(mn[0], mn[1], mn[2], mn[3]);
    *reinterpret_cast<float4*>(&part[2][warp][4 * lane]) = make_float4(sm[0], sm[1], sm[2], sm[3]);
  }
  __syncthreads();
  const size_t gi = (static_cast<size_t>(s) * p.hkv + h) * p.mg + b;
  if (tid < kPool) {
    const int sec = tid / kDim, d = tid % kDim;  // sec is the same in a warp
    float v = part[sec][0][d];
#pragma unroll
    for (int k = 1; k < kPfWarps; ++k) {
      const float x = part[sec][k][d];
      v = sec == 0 ? fmaxf(v, x) : (sec == 1 ? fminf(v, x) : v + x);
    }
    if (sec == 2) v *= 1.f / kBlock;
    P[tid] = v;
    if (p.pooled_raw != nullptr) p.pooled_raw[gi * kPool + tid] = v * scale;
  }
  __syncthreads();
  {
    float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPfRowsK; ++i) {
      const float x = P[kPfRowsK * warp + i];
      u[0] = fmaf(x, bf16_lo(w[i].x), u[0]);
      u[1] = fmaf(x, bf16_hi(w[i].x), u[1]);
      u[2] = fmaf(x, bf16_lo(w[i].y), u[2]);
      u[3] = fmaf(x, bf16_hi(w[i].y), u[3]);
    }
    *reinterpret_cast<float4*>(&part[0][warp][4 * lane]) = make_float4(u[0], u[1], u[2], u[3]);
  }
  __syncthreads();
  float u = 0.f, gain = 0.f, cs = 0.f, sn = 0.f;
  if (tid < kDim) {
    gain = p.gamma_k[tid];
    rope_cos_sin(p.rope.theta_over_pi[tid & 63], b, cs, sn);
#pragma unroll
    for (int k = 0; k < kPfWarps; ++k) u += part[0][k][tid];
    u *= scale;
    float sq = u * u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) ssq[warp] = sq;
  }
  __syncthreads();
  if (tid < kDim) {
    u *= 1.f / sqrtf((ssq[0] + ssq[1] + ssq[2] + ssq[3]) / kDim + p.eps) * gain;
    xs[tid] = u;
  }
  __syncthreads();
  if (tid < kDim) {
    const float y = tid < 64 ? u * cs - xs[tid + 64] * sn : u * cs + xs[tid - 64] * sn;
    if (p.gk16)
      static_cast<__nv_bfloat16*>(p.gate_keys)[gi * kDim + tid] = __float2bfloat16_rn(y);
    else
      static_cast<float*>(p.gate_keys)[gi * kDim + tid] = y;
  }
}

cudaError_t launch_pool_few_kv8(int code, const PoolParams& p, int batch, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.num_blocks), static_cast<unsigned>(p.hkv), static_cast<unsigned>(batch));
  return code == kCodeE4m3 ? launch_pdl(pool_few_kernel<kCodeE4m3>, grid, kPfThreads, 0, stream, 0, p)
                           : launch_pdl(pool_few_kernel<kCodeInt8>, grid, kPfThreads, 0, stream, 0, p);
}

cudaError_t prepare_pool_project_kernel() {
  for (auto* k : {pool_project_kernel<kSrcBf16>, pool_project_kernel<kSrcE4m3>, pool_project_kernel<kSrcInt8>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPpSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sas
