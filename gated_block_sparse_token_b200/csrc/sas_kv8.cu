// The 8-bit KV cache: quantising write, read-back and block-sparse decode
// attention.
//
// A complete 64-token block of one KV head is stored as 64 x 128 codes (e4m3,
// or int8) of its keys and of its values, each under one fp32 scale:
//   a = max(max |x|, 2^-100);  scale = a / qmax (448, or 127);
//   code = round-to-nearest-even(x * qmax / a)
// (a block that holds a NaN or an infinity: scale NaN, codes 0, so that it
// reads back as NaN).  The block of a sequence's last token stays in bf16 in
// the sequence's tail: codes are written once, when the block completes, from
// the bf16 values, so the cache does not depend on how many tokens came per
// call.
#include <type_traits>

#include "sas_internal.h"

namespace sas {

namespace {

constexpr float kQmaxE4m3 = 448.f, kQmaxInt8 = 127.f;
constexpr uint32_t kMinAmaxBits = 0x0d800000u;  // 2^-100
constexpr uint32_t kBf16Inf = 0x7f80u;

__device__ __forceinline__ uint16_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- write
// A CTA walks every gridDim.x-th block that the append completes for one
// (sequence, KV head): threads 0-127 the keys, 128-255 the values, 8 rows x 8
// dims per thread in registers between the maximum and the rounding, so a block
// is read once and its codes written once; the next block's loads go out as
// soon as the codes are made.  CTA 0 also writes the tail, after its first block
// has read the tail's old rows.  Bound by memory, 3 B a value: 4 x 32,768 packed
// tokens 129 us (6.3 TB/s), six ragged chunks of 1,219 to 8,190 tokens 30-33 us
// (one CTA a block: 39); one token of each of 32 sequences 4.6 us, which is latency.
__device__ __forceinline__ uint4 load_new_row(const RowsView& r, long long tok, int h, int s, int d0) {
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(r.data) + static_cast<long long>(s) * r.seq +
                           tok * r.token + static_cast<long long>(h) * r.head + d0;
  return *reinterpret_cast<const uint4*>(p);
}

template <int CODE>
__global__ void __launch_bounds__(256, 3) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int s = blockIdx.z, h = blockIdx.y;
  const int half = threadIdx.x >> 7, tid = threadIdx.x & 127, lane = tid & 31;
  const int L = p.kv.seq_lens[s];
  const int n = p.new_lens != nullptr ? p.new_lens[s] : p.max_new;
  const long long start = p.new_starts != nullptr ? p.new_starts[s] : 0;
  bool err = n < 0 || n > p.max_new || L < n || start < 0 || start + n > p.new_tokens ||
             static_cast<long long>(L) > static_cast<long long>(p.kv.blocks) * kBlock;
  if (!err && n == 0) return;  // uniform over the CTA, like every branch on n and L
  const int L0 = err ? 0 : L - n;
  const int b_first = err ? 0 : L0 / kBlock, b_done = err ? 0 : L / kBlock;  // completed: [b_first, b_done)
  const RowsView src = half == 0 ? p.k_new : p.v_new;
  __nv_bfloat16* tail = const_cast<__nv_bfloat16*>(half == 0 ? p.kv.k_tail : p.kv.v_tail) +
                        (static_cast<long long>(s) * p.kv.hkv + h) * (kBlock * kDim);
  const int d0 = 8 * (tid & 15), r0 = tid >> 4;  // 16 lanes a row, rows r0, r0 + 8, ..
  uint4 x[8];
  const auto load_block = [&](int b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = r0 + 8 * i;
      const int t = b * kBlock + row - L0;  // index among the new tokens
      x[i] = t < 0 ? *reinterpret_cast<const uint4*>(tail + row * kDim + d0)
                   : load_new_row(src, start + t, h, s, d0);
    }
  };
  int b = b_first + static_cast<int>(blockIdx.x);
  // never when err; the rows lie in the input and the tail whatever the pages are
  if (b < b_done) load_block(b);
  // a page out of range anywhere in the write skips the whole (sequence, head)
  if (p.kv.block_table != nullptr)
    for (int k = b_first + static_cast<int>(threadIdx.x); k < b_done; k += 256)
      if (p.kv.tile(s, h, k) < 0) err = true;
  __shared__ uint32_t amax_s[2][2][4];  // by the parity of the round: one barrier a block
  if (__syncthreads_or(err)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(p.status, kStatusBounds);
    return;
  }
  for (int round = 0; b < b_done; b += static_cast<int>(gridDim.x), ++round) {
    uint32_t m = 0;  // two bf16 magnitudes
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = __vmaxu2(m, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu));
      m = __vmaxu2(m, __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
    }
    m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(0xffffffffu, m);
    uint32_t* am = amax_s[round & 1][half];
    if (lane == 0) am[tid >> 5] = m;
    __syncthreads();
    m = max(max(am[0], am[1]), max(am[2], am[3]));
    const bool finite = m < kBf16Inf;
    const uint32_t abits = finite ? max(m << 16, kMinAmaxBits) : 0x3f800000u;
    const float a = __uint_as_float(abits);
    constexpr float qmax = CODE == kCodeE4m3 ? kQmaxE4m3 : kQmaxInt8;
    // The rounded quotient x qmax / a, exact where it is representable (so also
    // where it lies half-way between two codes).  qmax / a is taken as Rh + Rl, Rh
    // its leading 16 bits: x Rh is exact (8 bits by 16), and x (Rh + Rl) within
    // 2^-38 of the quotient before its one rounding.  A quotient of bf16 values
    // that is no half-way point is at least 2^-16 of its value away from one, so
    // the code is that of the exact quotient.  a is first scaled to [2, 4) and
    // the factors by the same power of two, which keeps every term in range.
    const float pw = __uint_as_float(((255u - (abits >> 23)) << 23));
    const float an = a * pw;
    const float rh = __uint_as_float(__float_as_uint(qmax / an) & 0xffffff00u);
    const float Rh = rh * pw, Rl = fmaf(-rh, an, qmax) / an * pw;
    const auto quot = [&](float v) { return fmaf(v, Rl, v * Rh); };
    uint2 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float y0 = quot(bf16_lo(w[2 * k])), y1 = quot(bf16_hi(w[2 * k]));
        const float y2 = quot(bf16_lo(w[2 * k + 1])), y3 = quot(bf16_hi(w[2 * k + 1]));
        if constexpr (CODE == kCodeE4m3) {
          c[k] = static_cast<uint32_t>(cvt_e4m3x2(y0, y1)) | (static_cast<uint32_t>(cvt_e4m3x2(y2, y3)) << 16);
        } else {
          // y + 1.5 * 2^23 rounds y to the nearest integer (even on a tie) in
          // its low bits, whose low byte is the code
          constexpr float magic = 12582912.f;
          const uint32_t p01 = __byte_perm(__float_as_uint(y0 + magic), __float_as_uint(y1 + magic), 0x0040);
          const uint32_t p23 = __byte_perm(__float_as_uint(y2 + magic), __float_as_uint(y3 + magic), 0x0040);
          c[k] = __byte_perm(p01, p23, 0x5410);
        }
      }
      code[i] = finite ? make_uint2(c[0], c[1]) : make_uint2(0u, 0u);
    }
    if (b + static_cast<int>(gridDim.x) < b_done) load_block(b + static_cast<int>(gridDim.x));
    const long long tile = p.kv.tile(s, h, b);
    uint8_t* dst = const_cast<uint8_t*>(half == 0 ? p.kv.k : p.kv.v) + tile * kTile8Bytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint2*>(dst + (r0 + 8 * i) * kDim + d0) = code[i];
    if (tid == 0)
      const_cast<float*>(half == 0 ? p.kv.k_scale : p.kv.v_scale)[tile] =
          finite ? __fdiv_rn(a, qmax) : __uint_as_float(0x7fc00000u);
  }
  if (blockIdx.x == 0) {
    __syncthreads();  // the tail's old rows have been read
    const int c = (L - 1) / kBlock;
    for (int row = r0 + max(0, (L0 - c * kBlock) & ~7); row < L - c * kBlock; row += 8) {
      const int t = c * kBlock + row - L0;
      if (t >= 0) *reinterpret_cast<uint4*>(tail + row * kDim + d0) = load_new_row(src, start + t, h, s, d0);
    }
  }
}

// ---------------------------------------------------------------- read-back
// A CTA walks every gridDim.x-th block of one (sequence, KV head)'s range,
// threads 0-127 the keys, 128-255 the values.  A lane turns as many codes as
// make 16 output bytes, so that a warp's stores fill whole sectors; the next
// block's codes are requested before this one's values are stored.  Bound by
// memory, 3 B a value into bf16: 805 MB in 129 us (6.2 TB/s); 5 B into fp32: 1.34 GB
// in 222 us (6.0 TB/s).
template <int CODE, typename OutT>
__global__ void __launch_bounds__(256, 3) kv8_read_kernel(const __grid_constant__ Kv8ReadParams p) {
  constexpr int VEC = 16 / static_cast<int>(sizeof(OutT));  // codes of a lane: 8 or 4
  constexpr int LPR = kDim / VEC;                           // lanes of a row
  constexpr int ROWS = 128 / LPR;                           // rows of a pass: 8 or 4
  constexpr int N = kBlock / ROWS;                          // passes
  using Codes = std::conditional_t<VEC == 8, uint2, uint32_t>;
  griddep_launch_dependents();
  griddep_wait();
  const int s = blockIdx.z, h = blockIdx.y;
  const int half = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int L = p.kv.seq_lens[s];
  const int begin = p.begin != nullptr ? p.begin[s] : 0;
  const RowsView o = half == 0 ? p.k_out : p.v_out;
  bool err = L < 0 || begin < 0 || static_cast<long long>(L) > static_cast<long long>(p.kv.blocks) * kBlock;
  // positions begin .. end - 1, in blocks b0 .. b1 - 1
  const int end = err ? 0 : static_cast<int>(min(static_cast<long long>(begin) + p.count, static_cast<long long>(L)));
  if (o.data != nullptr && begin < end) {
    const int c = (L - 1) / kBlock, b0 = begin / kBlock, b1 = (end - 1) / kBlock + 1;
    const int step = static_cast<int>(gridDim.x);
    const uint8_t* codes = half == 0 ? p.kv.k : p.kv.v;
    const float* scales = half == 0 ? p.kv.k_scale : p.kv.v_scale;
    const int d0 = VEC * (tid % LPR), r0 = tid / LPR;  // rows r0, r0 + ROWS, ..
    OutT* out = static_cast<OutT*>(const_cast<void*>(o.data)) + static_cast<long long>(s) * o.seq +
                static_cast<long long>(h) * o.head + d0;
    const auto store = [&](int pos, const float (&x)[VEC]) {
      if (pos < begin || pos >= end) return;
      OutT* dst = out + static_cast<long long>(pos - begin) * o.token;
      if constexpr (VEC == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[VEC - 3]), pack_bf16x2(x[VEC - 2], x[VEC - 1]));
    };
    Codes w[N];
    float sc = 0.f;
    long long tile = -1, tile_n = -1;
    const int be = min(b1, c);  // the stored ones
    const auto load_block = [&]() {
      if (tile < 0) return;
      sc = scales[tile];
#pragma unroll
      for (int i = 0; i < N; ++i)
        w[i] = *reinterpret_cast<const Codes*>(codes + tile * kTile8Bytes + (r0 + ROWS * i) * kDim + d0);
    };
    int b = b0 + static_cast<int>(blockIdx.x);
    if (b < be) {
      tile = p.kv.tile(s, h, b);
      if (b + step < be) tile_n = p.kv.tile(s, h, b + step);
      load_block();
    }
    for (; b < be; b += step) {
      Codes cur[N];
#pragma unroll
      for (int i = 0; i < N; ++i) cur[i] = w[i];
      const float cur_sc = sc;
      const bool known = tile >= 0;
      if (!known) err = true;
      tile = tile_n;
      if (b + step < be) load_block();
      if (b + 2 * step < be) tile_n = p.kv.tile(s, h, b + 2 * step);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float x[VEC];
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
          uint32_t lo, hi, word;
          if constexpr (VEC == 8)
            word = k == 0 ? cur[i].x : cur[i].y;
          else
            word = cur[i];
          codes_f16<CODE>(word, lo, hi);
          x[4 * k] = f16_lo(lo) * cur_sc;
          x[4 * k + 1] = f16_hi(lo) * cur_sc;
          x[4 * k + 2] = f16_lo(hi) * cur_sc;
          x[4 * k + 3] = f16_hi(hi) * cur_sc;
        }
        if (!known) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) x[k] = 0.f;
        }
        store(b * kBlock + r0 + ROWS * i, x);
      }
    }
    if (c < b1 && static_cast<int>(blockIdx.x) == (c - b0) % step) {  // the current block: from the tail
      const __nv_bfloat16* tail = (half == 0 ? p.kv.k_tail : p.kv.v_tail) +
                                  (static_cast<long long>(s) * p.kv.hkv + h) * (kBlock * kDim) + d0;
      for (int row = r0; row < end - c * kBlock; row += ROWS) {
        float x[VEC];
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(tail + row * kDim + 2 * k);
          x[2 * k] = bf16_lo(u);
          x[2 * k + 1] = bf16_hi(u);
        }
        store(c * kBlock + row, x);
      }
    }
  }
  if (err) raise_status(p.status, kStatusBounds);
}

// ---------------------------------------------------------------- attention
// out_g = sum_j softmax_j(q_g . k_j * scale) v_j over the tokens of the listed
// blocks (or of every block), one cluster of CTAs per (sequence, KV head).
//
// Bound by memory: 16 KiB of codes a block.  A group of four warps takes whole
// blocks, 16 keys a warp; a CTA holds two groups.  Every warp streams its own
// 4 KiB slices through its own ring of kKaStages slots (cp.async, 16 bytes a
// lane): the loop has no barrier and no producer, and 192 KiB are in flight on
// an SM whatever the register use.  (Loads into registers, one slice ahead, left
// too little in flight: 84 us for 256 pairs x 64 blocks; a ring fed by 2-D TMA
// from a lane of one of the consuming warps, which spends that warp's time on
// two copies a block: 59; this one 55.)
//   S^T = K q^T  the 16 keys are the rows, the (up to 8) heads of the group the
//                columns.  int8: m16n8k32 on the codes as they are stored, the
//                query as the three signed 8-bit digits of a fixed-point number
//                per head, in steps of 2^-21 of the power of two below the head's
//                largest value: its bf16 values stay exact down to 2^-14 of that,
//                and within 2^-22 of it below; its sums are exact.  (Two digits,
//                steps of 2^-14, cost the small channels beside a dominant one
//                their value; they save 0.9 of 13.5 us on 64 pairs x 32 blocks, 0.4
//                of 97 over 2 x 128k tokens.)  e4m3: m16n8k16 f16, the codes
//                converted (exact), the query scaled by a power of two per head
//                into f16's range (its bf16 values stay exact down to 2^-15 of the
//                largest, and off by 2^-25 of it below).  (The e4m3 form of
//                m16n8k32 with the query as two e4m3 terms ran slower than the
//                conversions it saves: 144 us against 114 for 2 x 128k tokens.)
//   softmax      per head over the columns, fp32, base 2; the running maximum
//                moves only when it grows by more than 2^kKaGrow (any factor
//                common to p and its sum cancels), so most blocks need one vote
//                and no shuffles;
//   O^T += V^T P^T  m16n8k16 f16 (codes are exact in f16), the P fragment
//                transposed in place by movmatrix.  P enters as two f16 terms, in
//                two products: 2^-22 of it.  (One term, 2^-11, left a few in a
//                hundred bf16 outputs on the other side of a rounding border; it
//                saves 2.5 of 96 us over 2 x 128k tokens, 0.5 of 11.5 on 64 pairs x
//                32 blocks, 11 of 185 over 16 x 32,000 tokens.)  It enters as
//                2^kKaShift p, so that this holds for every key down to 2^-14 of the
//                largest, and 2^-15 down to 2^-21: a few keys that take nearly all
//                the weight leave the others exact enough (unshifted, a hundred
//                thousand keys at 2^-24 were a third off).  V's scale takes the
//                factor back.  The sum of P runs over the unrounded values.
// Both products take their k index from whatever order makes a lane's 16-byte
// shared load its fragment: dims 16t .. 16t+15 and 64 + those for K, dims 16g ..
// of four keys for V.  Key g of a fragment is row 2(g/2) + g/4 (xor 4 for odd
// g) of its eight: with the swizzle both operands' loads are then free of bank
// conflicts.  The block's two scales enter as fp32 factors of S and O.
// The current block comes from the bf16 tail on bf16 products (P as a sum of
// three bf16 terms, 2^-24 of it), rows past the length masked, while the ring
// first fills.
//
// Two ways to divide the work.  Lists (and dense attention without the
// workspace for the other way): a cluster of CTAs a pair, which merge through
// distributed shared memory.  Dense attention (CHUNKS): every sequence in chunks
// of equal length, one CTA a (chunk, head), so that few or ragged long
// sequences fill the SMs; a second kernel merges the chunks' partial sums (16
// pairs x 2,000 blocks, e4m3 / int8: 95 / 94 us against 132 / 178 by clusters; 128
// pairs x 500 blocks, which are even: 185 / 197 against 170 / 180).
// Measured, e4m3: 64 pairs x 32 blocks 11.6 us (2.9 TB/s; the launch, the chain of
// length, list, table and first tile, and the merge are half of it; int8 13.6), 256
// pairs x 64 blocks 53 us (5.1 TB/s; int8 55), 128 pairs x 500 blocks dense 170 us
// (6.2 TB/s).
constexpr int kKaStages = 3;                // ring slots of a warp
constexpr int kKaSlot = 2 * 16 * kDim;      // 16 rows of K, then of V
constexpr int kKaHeadPair = 2 * kDim + 4;   // floats between head pairs of a partial (bank spread)
constexpr int kKaPart = (kMaxGroup / 2) * kKaHeadPair;
constexpr int kKaWarps = 8, kKaGroups = kKaWarps / 4;
constexpr int kKaMaxChunkBatch = 1024;      // sequences that the chunked way handles
constexpr int kKaChunkMin = 16;             // blocks of a chunk, at least
constexpr int kKaMaxCluster = 8;
// p <= 2^(kKaShift + kKaGrow) stays below f16's largest value
constexpr float kKaGrow = 4.f, kKaShift = 11.f, kKaUnshift = 1.f / 2048.f;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D(16x8) += A(16x32) * B(32x8) on signed bytes: lane (g, t) holds bytes
// 4t .. of row g (a0) and g + 8 (a1), 16 + 4t .. of both (a2, a3), and of
// column g (b0, b1).
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The query of one head (this lane: 32 of its values as 16 bf16 pairs) as B
// fragments, in units of kUnit E: E the power of two below the head's largest
// value, of biased exponent e (1 .. 254), which set() takes.
__device__ __forceinline__ float pow2_down(uint32_t e) {  // 2^(127 - e), e = 254: below the normal range
  return __uint_as_float(e < 254u ? (254u - e) << 23 : 0x00400000u);
}

template <int CODE>
struct KaQuery {  // int8: sum_n 256^n digit_n; k-step j: b[.][2j], b[.][2j + 1]
  static constexpr int kDigits = 3;
  // largest value to below 2^22, the most that `magic` leaves room for, and a bit
  // less than three signed bytes hold
  static constexpr float kUnit = 1.f / 2097152.f;
  uint32_t b[kDigits][8];

  __device__ __forceinline__ void set(const uint32_t (&raw)[16], uint32_t e) {
    constexpr float magic = 12582912.f;  // 1.5 * 2^23: its sum holds the rounded value in the low bits
    constexpr uint32_t bias = 0x808080u;
    const float dn = pow2_down(e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t u[4];  // byte n: digit n (v + bias has unsigned digits; each less 128 is signed)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = raw[2 * i + (k >> 1)];
        const float y = fmaf(((k & 1) ? bf16_hi(w) : bf16_lo(w)) * dn, 1.f / kUnit, magic);
        u[k] = (__float_as_uint(y) - __float_as_uint(magic) + bias) ^ bias;
      }
#pragma unroll
      for (int n = 0; n < kDigits; ++n) {
        const uint32_t sel = 0x0040u + 0x0011u * n;  // byte n of both words
        b[n][i] = __byte_perm(__byte_perm(u[0], u[1], sel), __byte_perm(u[2], u[3], sel), 0x5410);
      }
    }
  }
};
template <>
struct KaQuery<kCodeE4m3> {  // f16; k-step j: b[2j], b[2j + 1]
  static constexpr float kUnit = 1.f;
  uint32_t b[16];

  __device__ __forceinline__ void set(const uint32_t (&raw)[16], uint32_t e) {
    const float dn = pow2_down(e);  // q dn lies in (-2, 2)
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = pack_f16x2(bf16_lo(raw[i]) * dn, bf16_hi(raw[i]) * dn);
  }
};

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

struct KaState {
  float m[2], l[2];   // heads 2t, 2t + 1 (m: base-2 logit, the maximum within 2^kKaGrow, less kKaShift; uniform over g)
  float acc[8][4];    // O^T: dims 16g + j (0, 1) and 16g + 8 + j (2, 3), heads 2t, 2t + 1
};

__device__ __forceinline__ float weight(float m, float top) { return m == -INFINITY ? 0.f : exp2_approx(m - top); }

// Moves the running maximum to cover the 16 x 8 logits sc (this lane: keys
// g, g + 8 x heads 2t, 2t + 1).
__device__ __forceinline__ void raise_max(KaState& st, const float (&sc)[4]) {
  constexpr float room = kKaShift + kKaGrow;
  const bool grow = fmaxf(sc[0], sc[2]) > st.m[0] + room || fmaxf(sc[1], sc[3]) > st.m[1] + room;
  if (!__any_sync(0xffffffffu, grow)) return;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float x = fmaxf(sc[e], sc[e + 2]);
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
    const float top = fmaxf(st.m[e], x - kKaShift);
    const float f = weight(st.m[e], top);
    st.m[e] = top;
    st.l[e] *= f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      st.acc[j][e] *= f;
      st.acc[j][e + 2] *= f;
    }
  }
}

// One 16-key slice of a stored block: rows at ks_addr and vs_addr in shared
// memory, swizzled in 16-byte units by their row modulo 8.  kr: the K row of
// this lane (key g), vr: the V rows of keys 2t and 2t + 1 (row 8 further: keys
// g + 8, ...).  qs: E of heads 2t, 2t + 1; scale: attn_scale log2(e).
template <int CODE>
__device__ __forceinline__ void attend_codes(KaState& st, uint32_t ks_addr, uint32_t vs_addr, const KaQuery<CODE>& q,
                                             const float (&qs)[2], float scale, float ks, float vs) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int kr = (2 * (g >> 1) + (g >> 2)) ^ (4 * (g & 1)), vr = 2 * t + (t >> 1);
  uint4 x[4];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t at = ks_addr + kr * kDim + (((t + 4 * c) ^ kr) << 4);
    x[2 * c] = lds128(at);
    x[2 * c + 1] = lds128(at + 8 * kDim);
  }
  const uint32_t at0 = vs_addr + vr * kDim + ((g ^ vr) << 4), at1 = vs_addr + (vr ^ 4) * kDim + ((g ^ vr ^ 4) << 4);
  const uint4 y0 = lds128(at0), y1 = lds128(at1), y2 = lds128(at0 + 8 * kDim), y3 = lds128(at1 + 8 * kDim);
  float sc[4];
  if constexpr (CODE == kCodeInt8) {
    constexpr int N = KaQuery<CODE>::kDigits;
    int d[2][N][4] = {};  // independent chains of two products
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int n = 0; n < N; ++n) {
        mma_s8(d[c][n], x[2 * c].x, x[2 * c + 1].x, x[2 * c].y, x[2 * c + 1].y, q.b[n][4 * c], q.b[n][4 * c + 1]);
        mma_s8(d[c][n], x[2 * c].z, x[2 * c + 1].z, x[2 * c].w, x[2 * c + 1].w, q.b[n][4 * c + 2], q.b[n][4 * c + 3]);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sc[e] = fmaf(static_cast<float>(d[0][1][e] + d[1][1][e]), 256.f, static_cast<float>(d[0][0][e] + d[1][0][e]));
      sc[e] = fmaf(static_cast<float>(d[0][2][e] + d[1][2][e]), 65536.f, sc[e]);
    }
  } else {
    float d[2][4] = {};  // two chains of products
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t r0[4] = {x[2 * c].x, x[2 * c].y, x[2 * c].z, x[2 * c].w};
      const uint32_t r1[4] = {x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a0, a1, a2, a3;
        codes_f16<CODE>(r0[j], a0, a2);
        codes_f16<CODE>(r1[j], a1, a3);
        mma_f16(d[c], a0, a1, a2, a3, q.b[8 * c + 2 * j], q.b[8 * c + 2 * j + 1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = d[0][e] + d[1][e];
  }
  // V^T as f16, while those products run: a[j] = dims 16g + j and
  // 16g + 8 + j of keys 2t, 2t + 1 (0, 1) and 2t + 8, 2t + 9 (2, 3)
  uint32_t a[8][4];
  {
    const uint32_t va[4] = {y0.x, y0.y, y0.z, y0.w}, vb[4] = {y1.x, y1.y, y1.z, y1.w};
    const uint32_t vc[4] = {y2.x, y2.y, y2.z, y2.w}, vd[4] = {y3.x, y3.y, y3.z, y3.w};
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint32_t sel = hf == 0 ? 0x5140 : 0x7362;
        const int j = 4 * w + 2 * hf;
        codes_f16<CODE>(__byte_perm(va[w], vb[w], sel), a[j][0], a[j + 1][0]);
        codes_f16<CODE>(__byte_perm(va[w + 2], vb[w + 2], sel), a[j][1], a[j + 1][1]);
        codes_f16<CODE>(__byte_perm(vc[w], vd[w], sel), a[j][2], a[j + 1][2]);
        codes_f16<CODE>(__byte_perm(vc[w + 2], vd[w + 2], sel), a[j][3], a[j + 1][3]);
      }
  }
  // E and the keys' scale first, like the product of query and key: neither E nor
  // the scale alone meets a factor that could take it out of range
  const float f0 = qs[0] * ks * (scale * KaQuery<CODE>::kUnit), f1 = qs[1] * ks * (scale * KaQuery<CODE>::kUnit);
  vs *= kKaUnshift;
#pragma unroll
  for (int e = 0; e < 4; ++e) sc[e] *= (e & 1) ? f1 : f0;
  raise_max(st, sc);
  float p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = exp2_approx(sc[e] - st.m[e & 1]);
  st.l[0] = fmaf(p[0] + p[2], kKaUnshift, st.l[0]);
  st.l[1] = fmaf(p[1] + p[3], kKaUnshift, st.l[1]);
  const uint32_t h0 = pack_f16x2(p[0], p[1]), h1 = pack_f16x2(p[2], p[3]);
  const uint32_t b0 = transpose8x8(h0), b1 = transpose8x8(h1);
  const uint32_t e0 = transpose8x8(pack_f16x2(p[0] - f16_lo(h0), p[1] - f16_hi(h0)));
  const uint32_t e1 = transpose8x8(pack_f16x2(p[2] - f16_lo(h1), p[3] - f16_hi(h1)));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    mma_f16(o, a[j][0], a[j][1], a[j][2], a[j][3], b0, b1);
    mma_f16(o, a[j][0], a[j][1], a[j][2], a[j][3], e0, e1);
#pragma unroll
    for (int e = 0; e < 4; ++e) st.acc[j][e] = fmaf(o[e], vs, st.acc[j][e]);
  }
}

// One 16-key slice of the current block, from the bf16 tail: rows
// row0 .. row0 + 15 of which those below `rows` count.
__device__ __forceinline__ void attend_tail(KaState& st, const __nv_bfloat16* kt, const __nv_bfloat16* vt,
                                            const __nv_bfloat16* q, bool head_ok, int row0, int rows, float scale) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d0 = 64 * c + 16 * t + 8 * i;
      const uint4 r0 = *reinterpret_cast<const uint4*>(kt + (row0 + g) * kDim + d0);
      const uint4 r1 = *reinterpret_cast<const uint4*>(kt + (row0 + g + 8) * kDim + d0);
      const uint4 b = head_ok ? *reinterpret_cast<const uint4*>(q + d0) : make_uint4(0u, 0u, 0u, 0u);
      mma_bf16_16816(sc, r0.x, r1.x, r0.y, r1.y, b.x, b.y);
      mma_bf16_16816(sc, r0.z, r1.z, r0.w, r1.w, b.z, b.w);
    }
  }
  const bool in0 = row0 + g < rows, in1 = row0 + g + 8 < rows;
  sc[0] = in0 ? sc[0] * scale : -INFINITY;
  sc[1] = in0 ? sc[1] * scale : -INFINITY;
  sc[2] = in1 ? sc[2] * scale : -INFINITY;
  sc[3] = in1 ? sc[3] * scale : -INFINITY;
  raise_max(st, sc);
  float p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) p[e] = (e < 2 ? in0 : in1) ? exp2_approx(sc[e] - (st.m[e & 1] + kKaShift)) : 0.f;
  st.l[0] += p[0] + p[2];
  st.l[1] += p[1] + p[3];
  constexpr int kTerms = 3;  // of P
  uint32_t b[kTerms][2];
#pragma unroll
  for (int n = 0; n < kTerms; ++n) {
    const uint32_t h0 = pack_bf16x2(p[0], p[1]), h1 = pack_bf16x2(p[2], p[3]);
    b[n][0] = transpose8x8(h0);
    b[n][1] = transpose8x8(h1);
    p[0] -= bf16_lo(h0), p[1] -= bf16_hi(h0), p[2] -= bf16_lo(h1), p[3] -= bf16_hi(h1);
  }
  uint32_t v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 2 * t + (i & 1) + 8 * (i >> 1);
    const uint4* src = reinterpret_cast<const uint4*>(vt + row * kDim + 16 * g);
    const uint4 x = src[0], y = src[1];
    const bool in = row < rows;  // stale rows may hold anything, NaN included
    v[i][0] = in ? x.x : 0u, v[i][1] = in ? x.y : 0u, v[i][2] = in ? x.z : 0u, v[i][3] = in ? x.w : 0u;
    v[i][4] = in ? y.x : 0u, v[i][5] = in ? y.y : 0u, v[i][6] = in ? y.z : 0u, v[i][7] = in ? y.w : 0u;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t sel = (j & 1) ? 0x7632 : 0x5410;
    const int w = j / 2;
    const uint32_t a0 = __byte_perm(v[0][w], v[1][w], sel), a1 = __byte_perm(v[0][4 + w], v[1][4 + w], sel);
    const uint32_t a2 = __byte_perm(v[2][w], v[3][w], sel), a3 = __byte_perm(v[2][4 + w], v[3][4 + w], sel);
#pragma unroll
    for (int n = 0; n < kTerms; ++n) mma_bf16_16816(st.acc[j], a0, a1, a2, a3, b[n][0], b[n][1]);
  }
}

}  // namespace

// How dense attention is cut: sequence s of m_s blocks into ceil(m_s / size)
// chunks; chunk q of head h of it is the grid's number
// (first_s * Hkv + h * chunks_s + q), first_s the chunks of the sequences before.
struct KaChunk {
  int s, h, q, chunks, size;
};

// Called by all 256 threads; finds the grid's number `at` (s = -1: none).  The
// chunks' size is that of `target` equal ones, at least kKaChunkMin.  Every
// sequence counts, a bad length as one block.
__device__ __forceinline__ KaChunk find_chunk(const Kv8View& kv, int batch, int target, int at) {
  __shared__ int sum[8], found[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int PER = kKaMaxChunkBatch / 256;  // sequences of a thread, consecutive
  int m[PER], mine = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int s = tid * PER + k;
    m[k] = 0;
    if (s < batch) {
      const int L = kv.seq_lens[s];
      const bool bad = L < 1 || static_cast<long long>(L) > static_cast<long long>(kv.blocks) * kBlock;
      m[k] = bad ? 1 : (L - 1) / kBlock + 1;
    }
    mine += m[k];
  }
  const auto scan = [&](int v, int& before) {  // sum over the CTA, and over the threads before this one
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sum[warp] = inc;
    __syncthreads();
    int base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      base += w < warp ? sum[w] : 0;
      all += sum[w];
    }
    __syncthreads();
    before = base + inc - v;
    return all;
  };
  KaChunk c{};
  int before = 0;
  const long long tiles = static_cast<long long>(scan(mine, before)) * kv.hkv;
  c.size = static_cast<int>(max(static_cast<long long>(kKaChunkMin), (tiles + target - 1) / target));
  int n = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) n += (m[k] + c.size - 1) / c.size;
  (void)scan(n, before);
  if (tid == 0) found[0] = -1;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int chunks = (m[k] + c.size - 1) / c.size, first = before * kv.hkv;
    if (at >= first && at < first + chunks * kv.hkv) {
      found[0] = tid * PER + k;
      found[1] = (at - first) / chunks;
      found[2] = (at - first) % chunks;
      found[3] = chunks;
    }
    before += chunks;
  }
  __syncthreads();
  c.s = found[0];
  c.h = found[1];
  c.q = found[2];
  c.chunks = found[3];
  return c;
}

// Partial sums of one chunk in the workspace: [G][128] o, [8] m, [8] l, flag.
__device__ __forceinline__ size_t chunk_floats(int G) { return static_cast<size_t>(G) * kDim + 2 * kMaxGroup + 4; }

template <int CODE, bool F32OUT, bool CHUNKS>
__global__ void __launch_bounds__(32 * kKaWarps, 2)
    kv8_attend_kernel(const __grid_constant__ Kv8AttendParams p) {
  // the warps' rings; once every block is used, the warps' partials
  extern __shared__ __align__(128) uint8_t smem_raw[];
  float* part = reinterpret_cast<float*>(smem_raw);
  __shared__ float ml[kKaWarps][2][kMaxGroup];
  __shared__ float cta_ml[2][kMaxGroup];
  __shared__ int cta_bad;
  const int CS = CHUNKS ? 1 : static_cast<int>(gridDim.x), rank = CHUNKS ? 0 : static_cast<int>(blockIdx.x);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  constexpr int threads = 32 * kKaWarps;
  const int G = p.G;
  const int quarter = warp & 3;
  griddep_launch_dependents();
  griddep_wait();

  KaChunk ch{};
  int pair, s, h;
  if constexpr (CHUNKS) {
    ch = find_chunk(p.kv, p.batch, p.target, static_cast<int>(blockIdx.x));
    if (ch.s < 0) return;  // more CTAs than chunks
    s = ch.s;
    h = ch.h;
    pair = s * p.kv.hkv + h;
  } else {
    pair = static_cast<int>(blockIdx.y);
    s = pair / p.kv.hkv;
    h = pair - s * p.kv.hkv;
  }

  // ---- the list.  Stored blocks of this warp's group: entries jb, jb + js, ..
  // (n of them); lane l holds block, tile and scales of a chunk's l-th.  The
  // first chunk's block numbers are read together with the length and the count
  // (inside the list's storage whatever those turn out to be).
  const int32_t* sel = !CHUNKS && p.sel_idx != nullptr ? p.sel_idx + static_cast<size_t>(pair) * p.max_sel : nullptr;
  const int js = CS * kKaGroups, grp = rank * kKaGroups + (warp >> 2);
  const int jb = CHUNKS ? ch.q * ch.size + grp : grp;
  const int L = p.kv.seq_lens[s];
  int m = 0, first_b = 0, first_next = 0, last_b = 0;
  if (sel != nullptr) {
    const int first_j = jb + js * lane;
    m = p.sel_count[pair];
    if (first_j < p.max_sel) first_b = sel[first_j];
    if (first_j + 1 < p.max_sel) first_next = sel[first_j + 1];
  }
  const __nv_bfloat16* qrow = p.q + (static_cast<size_t>(s) * p.hq + static_cast<size_t>(h) * G + min(g, G - 1)) * kDim;
  uint32_t raw[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 x = *reinterpret_cast<const uint4*>(qrow + 64 * (i >> 1) + 16 * t + 8 * (i & 1));
    raw[4 * i] = x.x, raw[4 * i + 1] = x.y, raw[4 * i + 2] = x.z, raw[4 * i + 3] = x.w;
  }
  bool bad = L < 1 || static_cast<long long>(L) > static_cast<long long>(p.kv.blocks) * kBlock;
  const int c = bad ? 0 : (L - 1) / kBlock;
  if (sel == nullptr) {
    m = c + 1;
  } else {
    if (m < 1 || m > p.max_sel) bad = true;
    if (!bad) last_b = sel[m - 1];
  }
  const int je = CHUNKS ? min(m - 1, (ch.q + 1) * ch.size) : m - 1;  // end of this CTA's (cluster's) stored entries
  int n = bad || jb >= je ? 0 : (je - 1 - jb) / js + 1;

  int tile_c = 0, tile_n = 0;
  float ks_c = 0.f, vs_c = 0.f, ks_n = 0.f, vs_n = 0.f;
  auto fetch = [&](int i0, int& tile, float& ks, float& vs) -> bool {  // entries i0 .. i0 + 31
    const int i = i0 + lane;
    bool ok = true;
    tile = 0;
    if (i < n) {
      const int j = jb + js * i;
      const int b = sel == nullptr ? j : (i0 == 0 ? first_b : sel[j]);
      if (sel != nullptr && (i0 == 0 ? first_next : sel[j + 1]) <= b) ok = false;  // ascending, so all lie below c
      const long long at = b < c ? p.kv.tile(s, h, b) : -1;
      if (at < 0) ok = false;
      if (ok) {
        tile = static_cast<int>(at);
        ks = p.kv.k_scale[tile];
        vs = p.kv.v_scale[tile];
      }
    }
    return __all_sync(0xffffffffu, ok);
  };
  if (n > 0 && !fetch(0, tile_c, ks_c, vs_c)) {
    bad = true;
    n = 0;
  }
  // lane: 16-byte unit lane % 8 of rows lane / 8 + 4k, stored at that unit xor
  // the row modulo 8
  const uint32_t ring = smem_u32(smem_raw) + warp * (kKaStages * kKaSlot);
  const uint32_t d_even = (lane >> 3) * kDim + (((lane & 7) ^ (lane >> 3)) << 4);
  const uint32_t d_odd = d_even ^ 64u;  // rows 4 further: the unit xor 4
  const size_t src_off = static_cast<size_t>(quarter) * (16 * kDim) + 16 * lane;
  auto issue = [&](uint32_t slot, int tile) {
    const uint8_t* kp = p.kv.k + static_cast<size_t>(tile) * kTile8Bytes + src_off;
    const uint8_t* vp = p.kv.v + static_cast<size_t>(tile) * kTile8Bytes + src_off;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t dst = slot + 4 * k * kDim + ((k & 1) ? d_odd : d_even);
      cp_async16(dst, kp + 4 * k * kDim);
      cp_async16(dst + 16 * kDim, vp + 4 * k * kDim);
    }
  };
#pragma unroll
  for (int i = 0; i < kKaStages; ++i) {
    const int tile = __shfl_sync(0xffffffffu, tile_c, i);
    if (i < n) issue(ring + i * kKaSlot, tile);
    cp_async_commit();
  }

  // ---- the query, as B fragments: head g, dims 16t .. and 64 + 16t ..
  KaQuery<CODE> qf;
  float qs[2];
  {
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (g >= G) raw[i] = 0u;
      mag = __vmaxu2(mag, raw[i] & 0x7fff7fffu);
    }
    mag = max(mag & 0xffffu, mag >> 16);
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    const uint32_t e = min(max(mag >> 7, 1u), 254u);
    qf.set(raw, e);
    const float E = __uint_as_float(mag >= kBf16Inf ? 0x7fc00000u : e << 23);  // an infinity or NaN: every logit is NaN
    qs[0] = __shfl_sync(0xffffffffu, E, 8 * t);
    qs[1] = __shfl_sync(0xffffffffu, E, 8 * t + 4);
  }

  KaState st;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    st.m[e] = -INFINITY;
    st.l[e] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) st.acc[j][e] = 0.f;

  // ---- the current block: the group whose turn it is, while its ring fills
  if (sel != nullptr && last_b != c) bad = true;
  const bool tail_turn = CHUNKS ? (ch.q == ch.chunks - 1 && grp == 0) : grp == (m - 1) % js;
  if (!bad && tail_turn && 16 * quarter < L - c * kBlock) {
    const size_t off = static_cast<size_t>(pair) * (kBlock * kDim);
    attend_tail(st, p.kv.k_tail + off, p.kv.v_tail + off, qrow, g < G, 16 * quarter, L - c * kBlock, p.scale_log2);
  }

  // ---- the stored blocks
  uint32_t slot = ring;
  for (int i = 0; i < n; ++i) {
    if ((i & 31) == 0 && i + 32 < n && !fetch(i + 32, tile_n, ks_n, vs_n)) {
      bad = true;
      n = i + 32;
    }
    cp_async_wait<kKaStages - 1>();
    __syncwarp();
    attend_codes<CODE>(st, slot, slot + 16 * kDim, qf, qs, p.scale_log2, __shfl_sync(0xffffffffu, ks_c, i & 31),
                       __shfl_sync(0xffffffffu, vs_c, i & 31));
    __syncwarp();
    const int nxt = i + kKaStages;  // into the slot just used
    const int tile = __shfl_sync(0xffffffffu, ((i ^ nxt) & ~31) ? tile_n : tile_c, nxt & 31);
    if (nxt < n) issue(slot, tile);
    cp_async_commit();
    if ((i & 31) == 31) {
      tile_c = tile_n;
      ks_c = ks_n;
      vs_c = vs_n;
    }
    slot += kKaSlot;
    if (slot == ring + kKaStages * kKaSlot) slot = ring;
  }
  __syncthreads();  // every copy has landed and been used: the rings' space is free

  // ---- merge: warps, then CTAs of the cluster
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 4);
    st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 8);
    st.l[e] += __shfl_xor_sync(0xffffffffu, st.l[e], 16);
    if (g == 0) {
      ml[warp][0][2 * t + e] = st.m[e];
      ml[warp][1][2 * t + e] = st.l[e];
    }
    float* dst = part + warp * kKaPart + t * kKaHeadPair + e * kDim + 16 * g;
    float4* d4 = reinterpret_cast<float4*>(dst);
    d4[0] = make_float4(st.acc[0][e], st.acc[1][e], st.acc[2][e], st.acc[3][e]);
    d4[1] = make_float4(st.acc[4][e], st.acc[5][e], st.acc[6][e], st.acc[7][e]);
    d4[2] = make_float4(st.acc[0][e + 2], st.acc[1][e + 2], st.acc[2][e + 2], st.acc[3][e + 2]);
    d4[3] = make_float4(st.acc[4][e + 2], st.acc[5][e + 2], st.acc[6][e + 2], st.acc[7][e + 2]);
  }
  bad = __syncthreads_or(bad) != 0;
  for (int i = tid; i < G * kDim; i += threads) {
    const int hd = i / kDim, d = i % kDim;
    float top = ml[0][0][hd];
#pragma unroll
    for (int w = 1; w < kKaWarps; ++w) top = fmaxf(top, ml[w][0][hd]);
    float o = 0.f, l = 0.f;
    const int at = (hd >> 1) * kKaHeadPair + (hd & 1) * kDim + d;
#pragma unroll
    for (int w = 0; w < kKaWarps; ++w) {
      const float f = weight(ml[w][0][hd], top);
      o = fmaf(f, part[w * kKaPart + at], o);
      l = fmaf(f, ml[w][1][hd], l);
    }
    part[at] = o;  // read and written by this thread alone
    if (d == 0) {
      cta_ml[0][hd] = top;
      cta_ml[1][hd] = l;
    }
  }
  if (tid == 0) cta_bad = bad ? 1 : 0;
  const auto store = [&](int hd, int d, float v) {
    const size_t at = (static_cast<size_t>(s) * p.hq + static_cast<size_t>(h) * G + hd) * kDim + d;
    if constexpr (F32OUT)
      static_cast<float*>(p.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  };
  if constexpr (CHUNKS) {
    __syncthreads();
    if (ch.chunks == 1) {
      for (int i = tid; i < G * kDim; i += threads) {
        const int hd = i / kDim, d = i % kDim;
        store(hd, d, bad ? 0.f : part[(hd >> 1) * kKaHeadPair + (hd & 1) * kDim + d] / cta_ml[1][hd]);
      }
      if (bad && tid == 0) raise_status(p.status, kStatusBounds);
    } else {
      float* dst = p.ws_part + static_cast<size_t>(blockIdx.x) * chunk_floats(G);
      for (int i = tid; i < G * kDim; i += threads) {
        const int hd = i / kDim, d = i % kDim;
        dst[i] = part[(hd >> 1) * kKaHeadPair + (hd & 1) * kDim + d];
      }
      if (tid < G) {
        dst[G * kDim + tid] = cta_ml[0][tid];
        dst[G * kDim + kMaxGroup + tid] = cta_ml[1][tid];
      }
      if (tid == 0) dst[G * kDim + 2 * kMaxGroup] = bad ? 1.f : 0.f;
    }
    return;
  }
  // every CTA's partial is complete and visible to the cluster
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // all of an output's remote values are requested before the first is used (a
  // rank past the cluster's reads the last one again, with weight 0)
  const int dpc = kDim / CS;
  int bads[kKaMaxCluster];
#pragma unroll
  for (int r = 0; r < kKaMaxCluster; ++r) bads[r] = __float_as_int(ld_dsmem(dsmem_addr(&cta_bad, min(r, CS - 1))));
  bool any_bad = false;
  for (int i = tid; i < G * dpc; i += threads) {
    const int hd = i / dpc, d = rank * dpc + i % dpc;
    const int at = (hd >> 1) * kKaHeadPair + (hd & 1) * kDim + d;
    float ms[kKaMaxCluster], ls[kKaMaxCluster], os[kKaMaxCluster];
#pragma unroll
    for (int r = 0; r < kKaMaxCluster; ++r) {
      ms[r] = ld_dsmem(dsmem_addr(&cta_ml[0][hd], min(r, CS - 1)));
      ls[r] = ld_dsmem(dsmem_addr(&cta_ml[1][hd], min(r, CS - 1)));
      os[r] = ld_dsmem(dsmem_addr(part + at, min(r, CS - 1)));
    }
    any_bad = false;
    float top = ms[0];
#pragma unroll
    for (int r = 0; r < kKaMaxCluster; ++r) {
      any_bad = any_bad || bads[r] != 0;
      top = fmaxf(top, ms[r]);
    }
    float o = 0.f, l = 0.f;
#pragma unroll
    for (int r = 0; r < kKaMaxCluster; ++r) {
      const float f = weight(ms[r], top);
      o = r < CS ? fmaf(f, os[r], o) : o;
      l = r < CS ? fmaf(f, ls[r], l) : l;
    }
    store(hd, d, any_bad ? 0.f : o / l);
  }
  // (thread 0 has an output in every CTA)
  if (any_bad && rank == 0 && tid == 0) raise_status(p.status, kStatusBounds);
  // no CTA leaves while another may still read its shared memory
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Merges the chunks' partial sums: one CTA per (sequence, KV head, query head of
// the group), every thread one dimension of every second chunk, in order.
template <bool F32OUT>
__global__ void __launch_bounds__(256) kv8_combine_kernel(const __grid_constant__ Kv8AttendParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float red[8], half_o[kDim];
  __shared__ int first_s;
  const int pair = static_cast<int>(blockIdx.x), s = pair / p.kv.hkv, h = pair - s * p.kv.hkv;
  const int hd = static_cast<int>(blockIdx.y);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.G;
  // the same cut as the first kernel's: a pair's chunks are consecutive
  const int size = find_chunk(p.kv, p.batch, p.target, -1).size;
  const auto chunks_of = [&](int k) {
    const int L = p.kv.seq_lens[k];
    const bool bad = L < 1 || static_cast<long long>(L) > static_cast<long long>(p.kv.blocks) * kBlock;
    return ((bad ? 1 : (L - 1) / kBlock + 1) + size - 1) / size;
  };
  const int chunks = chunks_of(s);
  if (chunks == 1) return;  // written by the first kernel
  int before = 0;           // chunks of the sequences ahead
  for (int k = tid; k < s; k += 256) before += chunks_of(k);
  if (tid == 0) first_s = 0;
  __syncthreads();
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0 && before > 0) atomicAdd(&first_s, before);  // integers: any order
  __syncthreads();
  const size_t stride = chunk_floats(G);
  const float* src = p.ws_part + (static_cast<size_t>(first_s) * p.kv.hkv + static_cast<size_t>(h) * chunks) * stride;
  const float *ms = src + G * kDim + hd, *ls = ms + kMaxGroup, *flag = src + G * kDim + 2 * kMaxGroup;
  bool bad = false;
  float top = -INFINITY;
  for (int q = tid; q < chunks; q += 256) {
    top = fmaxf(top, ms[q * stride]);
    bad = bad || flag[q * stride] != 0.f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  bad = __syncthreads_or(bad) != 0;
  top = red[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) top = fmaxf(top, red[w]);
  const int d = tid & (kDim - 1), half = tid >> 7;
  const float* os = src + hd * kDim + d;
  float o = 0.f, l = 0.f;
#pragma unroll 8
  for (int q = half; q < chunks; q += 2) {
    const float f = weight(ms[q * stride], top);
    o = fmaf(f, os[q * stride], o);
    l = fmaf(f, ls[q * stride], l);
  }
  __syncthreads();  // red is read
  if (half == 1) {
    half_o[d] = o;
    if (d == 0) red[0] = l;
  }
  __syncthreads();
  if (half == 0) {
    const float v = bad ? 0.f : (o + half_o[d]) / (l + red[0]);
    const size_t at = (static_cast<size_t>(s) * p.hq + static_cast<size_t>(h) * G + hd) * kDim + d;
    if constexpr (F32OUT)
      static_cast<float*>(p.out)[at] = v;
    else
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  }
  if (bad && tid == 0) raise_status(p.status, kStatusBounds);
}

// ---------------------------------------------------------------- launches
// CTAs of one (sequence, head) that walk `blocks` blocks: four waves of three an
// SM over all pairs (a ragged batch levels out), or about four blocks a CTA if
// that makes more, at most one a block.  Read-back of 32 pairs x 513 blocks with
// 37 / 55 / 111 CTAs a pair: 138 / 135 / 130 us; of 48 pairs x 129 with 25 / 37 /
// 74: 31.6 / 30.1 / 31.4.
static unsigned walkers(long long blocks, long long pairs) {
  const long long n = std::max((148 * 12 + pairs - 1) / pairs, blocks / 4);
  return static_cast<unsigned>(std::max<long long>(1, std::min(blocks, n)));
}

cudaError_t launch_kv8_append(int code, const Kv8AppendParams& p, int batch, cudaStream_t stream) {
  // at most (63 + max_new) / 64 blocks are completed
  const long long blocks = (static_cast<long long>(p.max_new) + kBlock - 1) / kBlock;
  const dim3 grid(walkers(blocks, static_cast<long long>(batch) * p.kv.hkv), static_cast<unsigned>(p.kv.hkv),
                  static_cast<unsigned>(batch));
  return code == kCodeE4m3 ? launch_pdl(kv8_append_kernel<kCodeE4m3>, grid, 256, 0, stream, 0, p)
                           : launch_pdl(kv8_append_kernel<kCodeInt8>, grid, 256, 0, stream, 0, p);
}

cudaError_t launch_kv8_read(int code, bool f32_out, const Kv8ReadParams& p, int batch, cudaStream_t stream) {
  const long long blocks = (static_cast<long long>(p.count) + kBlock - 1) / kBlock + 1;
  const dim3 grid(walkers(blocks, static_cast<long long>(batch) * p.kv.hkv), static_cast<unsigned>(p.kv.hkv),
                  static_cast<unsigned>(batch));
  if (code == kCodeE4m3)
    return f32_out ? launch_pdl(kv8_read_kernel<kCodeE4m3, float>, grid, 256, 0, stream, 0, p)
                   : launch_pdl(kv8_read_kernel<kCodeE4m3, __nv_bfloat16>, grid, 256, 0, stream, 0, p);
  return f32_out ? launch_pdl(kv8_read_kernel<kCodeInt8, float>, grid, 256, 0, stream, 0, p)
                 : launch_pdl(kv8_read_kernel<kCodeInt8, __nv_bfloat16>, grid, 256, 0, stream, 0, p);
}

// CTAs of a cluster: as many as keep the whole grid resident at once (two of 8
// warps an SM), up to one block a group of four warps.  Measured, CTAs a cluster
// -> us: 64 pairs x 32 blocks 8 -> 17.6, 4 -> 11.7, 2 -> 14.6; 256 pairs x 64
// blocks 8 -> 92, 4 -> 70, 2 -> 60, 1 -> 55.  More pairs than that run in waves:
// two CTAs a pair shorten a last wave that is half empty or more (304 / 336 / 368 /
// 400 pairs x 64 blocks, e4m3: 67 / 75 / 78 / 81 us against 73 / 85 / 86 / 88 with
// one, int8: 74 / 76 / 79 / 87 against 81 / 83 / 83 / 84; 512 and 592 int8: 104 and
// 120 against 104 and 115).
int kv8_attend_cluster(int pairs, int max_blocks) {
  int cluster = 1;
  const int last = pairs % (2 * 148);
  if (pairs > 2 * 148 && last > 0 && last <= 148 && max_blocks >= 2 * kKaGroups) return 2;
  while (cluster < kKaMaxCluster && pairs * cluster * 2 <= 2 * 148 && cluster * 2 * kKaGroups <= max_blocks)
    cluster *= 2;
  return cluster;
}

// The grid holds target + pairs chunks at most.  Up to 74 pairs they all fit
// the GPU at once (2 x 148 CTAs); more pairs have no use for a single wave.
static long long chunk_target(long long pairs) { return pairs <= 74 ? 2 * 148 - pairs : 4 * 148; }

size_t kv8_attend_scratch_bytes(long long pairs, int G) {
  return static_cast<size_t>(chunk_target(pairs) + pairs) * (static_cast<size_t>(G) * kDim + 2 * kMaxGroup + 4) * 4;
}

cudaError_t launch_kv8_attend(int code, bool f32_out, Kv8AttendParams p, cudaStream_t stream) {
  const int pairs = p.batch * p.kv.hkv;
  constexpr int T = 32 * kKaWarps;
  constexpr size_t smem = kKaWarps * std::max(kKaStages * kKaSlot, kKaPart * 4);
  // Chunks where a sequence may be longer than a few of them and the workspace
  // holds their partial sums
  if (p.sel_idx == nullptr && p.ws_part != nullptr && p.batch <= kKaMaxChunkBatch && p.kv.blocks > 4 * kKaChunkMin) {
    p.target = static_cast<int>(chunk_target(pairs));
    const dim3 grid(static_cast<unsigned>(p.target + pairs));
    const dim3 cgrid(static_cast<unsigned>(pairs), static_cast<unsigned>(p.G));
    cudaError_t e;
    if (code == kCodeE4m3)
      e = f32_out ? launch_pdl(kv8_attend_kernel<kCodeE4m3, true, true>, grid, T, smem, stream, 0, p)
                  : launch_pdl(kv8_attend_kernel<kCodeE4m3, false, true>, grid, T, smem, stream, 0, p);
    else
      e = f32_out ? launch_pdl(kv8_attend_kernel<kCodeInt8, true, true>, grid, T, smem, stream, 0, p)
                  : launch_pdl(kv8_attend_kernel<kCodeInt8, false, true>, grid, T, smem, stream, 0, p);
    if (e != cudaSuccess) return e;
    return f32_out ? launch_pdl(kv8_combine_kernel<true>, cgrid, 256, 0, stream, 0, p)
                   : launch_pdl(kv8_combine_kernel<false>, cgrid, 256, 0, stream, 0, p);
  }
  const int cluster = kv8_attend_cluster(pairs, p.sel_idx != nullptr ? p.max_sel : p.kv.blocks);
  const dim3 grid(static_cast<unsigned>(cluster), static_cast<unsigned>(pairs));
  if (code == kCodeE4m3)
    return f32_out ? launch_pdl(kv8_attend_kernel<kCodeE4m3, true, false>, grid, T, smem, stream, cluster, p)
                   : launch_pdl(kv8_attend_kernel<kCodeE4m3, false, false>, grid, T, smem, stream, cluster, p);
  return f32_out ? launch_pdl(kv8_attend_kernel<kCodeInt8, true, false>, grid, T, smem, stream, cluster, p)
                 : launch_pdl(kv8_attend_kernel<kCodeInt8, false, false>, grid, T, smem, stream, cluster, p);
}

cudaError_t prepare_kv8_kernels() {
  constexpr int smem = kKaWarps * std::max(kKaStages * kKaSlot, kKaPart * 4);
  for (auto* k : {kv8_attend_kernel<kCodeE4m3, false, false>, kv8_attend_kernel<kCodeE4m3, true, false>,
                  kv8_attend_kernel<kCodeInt8, false, false>, kv8_attend_kernel<kCodeInt8, true, false>,
                  kv8_attend_kernel<kCodeE4m3, false, true>, kv8_attend_kernel<kCodeE4m3, true, true>,
                  kv8_attend_kernel<kCodeInt8, false, true>, kv8_attend_kernel<kCodeInt8, true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sas
