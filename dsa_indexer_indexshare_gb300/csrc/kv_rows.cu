// Writing and reading of MLA KV cache rows: the append (interleaved RoPE of the
// 64-d key, then the row in the cache's format at its place in the batch
// layout), the read-back in bf16, and the INT4 quantiser.
//
// Row formats: bf16 [576]; FP8 656 bytes (kv_fp8_quant_kernel); INT4 416 bytes:
//   [0, 256)    the 512-d latent as codes n = q + 8, q in [-7, 7], in sixteen
//               groups of 32 dims; the little-endian 32-bit word m holds dims
//               8m .. 8m+7, dim 8m+2k in bits 4k.. and dim 8m+2k+1 in bits
//               16+4k.., so that one shift and one logical operation bring a
//               pair of neighbours into the two halves of a register
//   [256, 288)  the groups' bf16 scales s, bf16(amax / 7) but at least 2^-100
//               (an all-zero group) and at most 145 * 2^118 (so that 7 s stays
//               finite)
//   [288, 416)  the 64-d RoPE key, bf16
// with q = the integer nearest to the exact x / s, ties to even.  416 bytes are
// 13 whole 32-byte sectors.  A group that holds an infinity or a NaN gets a NaN
// scale and reads back as NaN throughout.  Read back, an element is
// bf16(q * s), one rounding.  Uniform codes leave about the noise of E2M1 (relative
// power 0.0094 against 0.0102 in groups of 32 normal values, both with bf16
// scales) and widen in fewer operations.
//
// The append and the quantiser give a warp one row, the read-back two; lane l holds dims
// 8l .. 8l+7 and 256+8l .. 256+8l+7, so that every access of a warp is one contiguous run.
// Bound by HBM: the append reads 1152 bytes a row and writes 416 / 656 / 1152,
// the read-back the other way round.  Measured (times in a graph): the read-back of
// 131,072 INT4 rows in 32.4 us, 6.36 TB/s or 0.95 of the copy rate; of 16,301 INT4
// rows in 5.4 us and 27,009 FP8 rows in 6.6 us (in L2).  The append of 4096 INT4 rows
// takes 4.6 us, of 4503 FP8 rows 5.7 us, of one row 2.5 us: two thirds are the
// launch and the chain of a row (its place, its values, the group's maximum, the
// codes), as 4096 rows are seven warps a scheduler.
#include <cmath>

#include "common.cuh"
#include "rows.cuh"

namespace dsa {
namespace {

enum RowType { kRowBf16 = 0, kRowFp8 = 1, kRowInt4 = 2 };  // dsa_dtype_t

template <int RT>
__host__ __device__ constexpr int row_bytes() {
  return RT == kRowBf16 ? DSA_KV_ROW_BYTES : RT == kRowFp8 ? DSA_KV_ROW_BYTES_FP8 : DSA_KV_ROW_BYTES_INT4;
}

// ---------------------------------------------------------------- quantisation
// Eight bf16 values (one 16-byte vector) as floats.
__device__ __forceinline__ void widen8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(u[k] << 16);
    v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
  }
}

// Largest |x| of a vector's eight bf16 values as bf16 bits (NaN above infinity
// above every finite value).
__device__ __forceinline__ uint32_t absmax8_bits(const uint4& w) {
  const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                              __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ float rcp_approx(float x) {  // one unit in the last place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The INT4 word of eight values and the bf16 bits of their group's scale; the
// group is the four lanes of a quad.  amax / 7 is formed as a product (two
// roundings to 24 bits): the quotient of an 8-bit number by 7 is at least 1/14 of
// a bf16 step away from a midpoint, so the bf16 result is that of the exact
// quotient.  x / s is formed as x * (1/s) with an error below 2^-20 and first
// rounded to a multiple of 2^-12: both x and s have
// 8 significant bits, so a quotient that is not a half-integer is at least
// 2^-10 away from one, while a true half-integer is restored exactly, and the
// second rounding breaks its tie to even.  |x / s| < 7.04 (s is within 2^-9 of
// amax / 7 unless it was raised, and 145/255 * 2^118 at the upper limit), so no
// code is beyond +-7.
__device__ __forceinline__ uint32_t int4_word(const uint4& w, uint16_t& scale_bits) {
  uint32_t ab = absmax8_bits(w);
  ab = max(ab, __shfl_xor_sync(0xffffffffu, ab, 1));
  ab = max(ab, __shfl_xor_sync(0xffffffffu, ab, 2));
  if (ab >= 0x7F80u) {
    scale_bits = 0x7FC0u;
    return 0x88888888u;
  }
  const float amax = __uint_as_float(ab << 16);
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(amax, 1.f / 7.f)));
  s = fminf(fmaxf(s, 7.888609052210118e-31f), __uint_as_float(0x7E110000u));  // 2^-100, 145 * 2^118
  scale_bits = static_cast<uint16_t>(__float_as_uint(s) >> 16);
  const float r = rcp_approx(s);
  float v[8];
  widen8(w, v);
  uint32_t word = 0;
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const float t = __fsub_rn(__fmaf_rn(v[d], r, 0x1.8p11f), 0x1.8p11f);  // ulp 2^-12
    const uint32_t n = __float_as_uint(__fadd_rn(t, 0x1.8p23f)) + 8u;  // ulp 1
    word |= (n & 15u) << (4 * (d >> 1) + 16 * (d & 1));
  }
  return word;
}

// Eight E4M3 codes and their group's scale; the group is 16 lanes.  The scale is
// the fp32 nearest to amax / 448, as in every FP8 row (kv_fp8_quant_kernel): a
// cache may hold rows of both calls.  (The product amax * fp32(1/448) would be an ulp off
// in six groups of ten; 4503 rows take 5.59 us with it and 5.71 with the division.)
// A code is the E4M3 value nearest to the exact x / sc (one element in 200 of a random
// group is an exact midpoint, so it is decided for all): q = |x| * (1/sc) gives the
// interval between two codes, m is its midpoint, the sign of the fma |x| - m sc is that
// of |x| / sc - m exactly, and m or its neighbour on that side is what the conversion
// rounds.  (Where q is off by so little that it lies in the next interval, |x| / sc is
// that close to their common code, which either gives.)  Extreme scales go out of line.
static __device__ __noinline__ uint32_t e4m3_exact(float x, float sc) { return e4m3_of_quotient(x, sc); }

__device__ __forceinline__ uint2 fp8_codes8(const uint4& w, float& sc) {
  float v[8];
  widen8(w, v);
  float amax = 0.f;
#pragma unroll
  for (int d = 0; d < 8; ++d) amax = fmaxf(amax, fabsf(v[d]));
#pragma unroll
  for (int m = 1; m < 16; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  const float r = rcp_approx(sc);
  uint32_t o[4];
#pragma unroll
  for (int d = 0; d < 8; d += 2) {
    float q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float x = v[d + k], ax = fabsf(x), qa = __fmul_rn(ax, r);
      // the midpoint of the interval: three bits kept, or steps of 2^-9 below 2^-6
      const float mid = qa < 0.015625f ? __fmaf_rn(floorf(qa * 512.f), 0.001953125f, 0.0009765625f)
                                       : __uint_as_float((__float_as_uint(qa) & 0xFFF00000u) | 0x00080000u);
      const float off = __fmaf_rn(-mid, sc, ax);
      q[k] = copysignf(__uint_as_float(__float_as_uint(mid) + (off > 0.f) - (off < 0.f)), x);
    }
    o[d / 2] = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
  }
  if (!(sc > 1e-25f && sc < 1e35f)) {
#pragma unroll
    for (int d = 0; d < 8; ++d)
      o[d / 2] = (o[d / 2] & ~(0xFFu << (8 * (d & 1)))) | e4m3_exact(v[d], sc) << (8 * (d & 1));
  }
  return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// One row from a warp's registers: a, b = the lane's two latent vectors, key =
// its pair (2l, 2l+1) of the RoPE key.
template <int RT>
__device__ __forceinline__ void store_row(uint8_t* row, int lane, const uint4& a, const uint4& b,
                                          uint32_t key) {
  if constexpr (RT == kRowBf16) {
    reinterpret_cast<uint4*>(row)[lane] = a;
    reinterpret_cast<uint4*>(row)[32 + lane] = b;
    reinterpret_cast<uint32_t*>(row + 1024)[lane] = key;
  } else if constexpr (RT == kRowFp8) {
    float sa, sb;
    const uint2 ca = fp8_codes8(a, sa), cb = fp8_codes8(b, sb);
    reinterpret_cast<uint2*>(row)[lane] = ca;
    reinterpret_cast<uint2*>(row)[32 + lane] = cb;
    if ((lane & 15) == 0) {
      reinterpret_cast<float*>(row + 512)[lane >> 4] = sa;
      reinterpret_cast<float*>(row + 512)[2 + (lane >> 4)] = sb;
    }
    reinterpret_cast<uint32_t*>(row + 528)[lane] = key;
  } else {
    uint16_t sa, sb;
    const uint32_t ca = int4_word(a, sa), cb = int4_word(b, sb);
    reinterpret_cast<uint32_t*>(row)[lane] = ca;
    reinterpret_cast<uint32_t*>(row)[32 + lane] = cb;
    if ((lane & 3) == 0) {
      reinterpret_cast<uint16_t*>(row + 256)[lane >> 2] = sa;
      reinterpret_cast<uint16_t*>(row + 256)[8 + (lane >> 2)] = sb;
    }
    reinterpret_cast<uint32_t*>(row + 288)[lane] = key;
  }
}

// ---------------------------------------------------------------- dequantisation
// Four bf16 pairs bf16(q * s) of an INT4 word: a nibble n set into the mantissa
// of 128 gives 128 + n, minus 136 is q (both exact), times s rounds once.
__device__ __forceinline__ uint4 int4_values(uint32_t w, __nv_bfloat162 s2) {
  const __nv_bfloat162 off = __halves2bfloat162(__ushort_as_bfloat16(0x4308), __ushort_as_bfloat16(0x4308));
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = ((w >> (4 * k)) & 0x000F000Fu) | 0x43004300u;
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), off);
    const __nv_bfloat162 p = __hmul2(q, s2);
    o[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight bf16 values bf16(fp32(code * scale)) of eight E4M3 codes.
__device__ __forceinline__ uint4 fp8_values(uint2 c, float s) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
    o[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// What a lane reads of one row, before it is widened.
template <int RT>
struct LaneRow;
template <>
struct LaneRow<kRowBf16> {
  uint4 a, b;
  uint32_t key;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    a = __ldcs(reinterpret_cast<const uint4*>(row) + lane);
    b = __ldcs(reinterpret_cast<const uint4*>(row) + 32 + lane);
    key = __ldcs(reinterpret_cast<const uint32_t*>(row + 1024) + lane);
  }
  __device__ __forceinline__ void values(uint4& va, uint4& vb) const { va = a, vb = b; }
};
template <>
struct LaneRow<kRowFp8> {
  uint2 a, b;
  float sa, sb;
  uint32_t key;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    a = __ldcs(reinterpret_cast<const uint2*>(row) + lane);
    b = __ldcs(reinterpret_cast<const uint2*>(row) + 32 + lane);
    sa = __ldcs(reinterpret_cast<const float*>(row + 512) + (lane >> 4));
    sb = __ldcs(reinterpret_cast<const float*>(row + 512) + 2 + (lane >> 4));
    key = __ldcs(reinterpret_cast<const uint32_t*>(row + 528) + lane);
  }
  __device__ __forceinline__ void values(uint4& va, uint4& vb) const {
    va = fp8_values(a, sa);
    vb = fp8_values(b, sb);
  }
};
template <>
struct LaneRow<kRowInt4> {
  uint32_t a, b, key;
  uint16_t sa, sb;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    a = __ldcs(reinterpret_cast<const uint32_t*>(row) + lane);
    b = __ldcs(reinterpret_cast<const uint32_t*>(row) + 32 + lane);
    sa = __ldcs(reinterpret_cast<const unsigned short*>(row + 256) + (lane >> 2));
    sb = __ldcs(reinterpret_cast<const unsigned short*>(row + 256) + 8 + (lane >> 2));
    key = __ldcs(reinterpret_cast<const uint32_t*>(row + 288) + lane);
  }
  __device__ __forceinline__ void values(uint4& va, uint4& vb) const {
    const __nv_bfloat16 s0 = __ushort_as_bfloat16(sa), s1 = __ushort_as_bfloat16(sb);
    va = int4_values(a, __halves2bfloat162(s0, s0));
    vb = int4_values(b, __halves2bfloat162(s1, s1));
  }
};

// ---------------------------------------------------------------- places
// Cache row of an entry (sequence, position): >= 0; -1 for a padding entry
// (sequence -1); -2 for one outside the batch, its table or the cache.
__device__ __forceinline__ int64_t entry_row(const BatchArgs& b, int seq, int pos, int64_t kv_rows) {
  if (seq == -1) return -1;
  if (seq < 0 || seq >= b.num_seqs || pos < 0 || pos >= b.max_len) return -2;
  const int64_t r = cache_row(b, seq, seq_base_row(b, seq), pos);
  return r >= 0 && r < kv_rows ? r : -2;
}

// ---------------------------------------------------------------- RoPE
struct RopeTurns {
  double f[32];       // rotary frequencies
  uint64_t turn[32];  // f / 2 pi as a fraction of a turn, in units of 2^-64
  uint32_t usual;     // bit i: 0 < f[i] <= 1 (the fast path's error bound)
  int on;             // 0: the key is stored as given
};

// The pair where the quick path does not decide: double-float, then fp64.
static __device__ __noinline__ uint32_t rotate_key_exact(double f, int pos, float x0, float x1) {
  DF sn{0.f, 0.f}, cs{1.f, 0.f};
  const bool fast = df_sincos_pos(pos, f, sn, cs);
  return rotate_pair_df(pos, f, fast, cs, sn, x0, x1);
}

// The pair (2l, 2l+1) of the key, rotated by pos * f[l], as bf16 bits.  The angle is
// reduced as a 64-bit fixed-point fraction of a turn (an error of 2^-34 turns at
// most), its top 32 bits split into a quadrant and a rest of |t| <= pi/4, and cos t
// and sin t are the Taylor polynomials to t^10 and t^9 (truncated terms below
// 2^-31 and 2^-29).  cos and sin are off by less than 1.9 * 2^-23: the rest's two
// roundings to 24 bits (2 * pi/4 * 2^-24), the low phase bits (2^-29), the
// polynomials' last roundings (2^-24 and little) and the 2^-28 by which the fp64
// product pos * f may differ from the exact angle below 2^25; the result by less
// than 3 * 2^-23 (|x0| + |x1|).  Where that cannot decide the bf16 rounding (about
// one value in 1000) the exact path does, so that the stored bits are those of the
// fp64 rotation rounded once.
__device__ __forceinline__ uint32_t rotate_key(const RopeTurns& rt, uint64_t turn, int lane, int pos, uint32_t raw) {
  const bool usual = (rt.usual >> lane) & 1u;
  const float x0 = bf16_bits_to_float(static_cast<uint16_t>(raw & 0xFFFF));
  const float x1 = bf16_bits_to_float(static_cast<uint16_t>(raw >> 16));
  const uint32_t phase = static_cast<uint32_t>((static_cast<uint64_t>(pos) * turn) >> 32);
  const uint32_t quad = (phase + 0x20000000u) >> 30;
  const float t = static_cast<float>(static_cast<int32_t>(phase - (quad << 30))) * 1.4629180792671596e-09f;  // 2 pi / 2^32
  const float t2 = t * t;
  const float ct = __fmaf_rn(
      t2, __fmaf_rn(t2, __fmaf_rn(t2, __fmaf_rn(t2, __fmaf_rn(t2, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  const float st = __fmaf_rn(
      __fmul_rn(t, t2), __fmaf_rn(t2, __fmaf_rn(t2, __fmaf_rn(t2, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), t);
  float c = quad & 1 ? st : ct, s = quad & 1 ? ct : st;
  c = (quad + 1) & 2 ? -c : c;  // quadrants 1, 2
  s = quad & 2 ? -s : s;        // quadrants 2, 3
  const float mag = fabsf(x0) + fabsf(x1);
  const float y0 = __fmaf_rn(x0, c, -__fmul_rn(x1, s));
  const float y1 = __fmaf_rn(x0, s, __fmul_rn(x1, c));
  const float e = mag * 4.76837158203125e-07f;  // 2^-21
  if (usual && pos < (1 << 25) && mag >= 7.888609052210118e-31f && fabsf(y0) < 3.0e38f && fabsf(y1) < 3.0e38f &&
      clear_of_bf16_midpoint(y0, e) && clear_of_bf16_midpoint(y1, e)) {
    const __nv_bfloat162 r2 = __floats2bfloat162_rn(y0, y1);
    return *reinterpret_cast<const uint32_t*>(&r2);
  }
  return rotate_key_exact(rt.f[lane], pos, x0, x1);
}

// ---------------------------------------------------------------- kernels
constexpr int kAppendWarps = 4;
template <int RT>
__global__ void __launch_bounds__(kAppendWarps * 32)
    kv_append_kernel(const uint16_t* __restrict__ x, int64_t stride, const int32_t* __restrict__ seq_of,
                     const int32_t* __restrict__ pos_of, int n, const BatchArgs b,
                     const __grid_constant__ RopeTurns rt, uint8_t* __restrict__ kv, int64_t kv_rows,
                     int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  // The turns, one per lane, by way of shared memory: a lane's own entry of a kernel
  // parameter is a constant-memory access per lane, one after the other (the
  // append of 4096 rows took 2 us longer that way).
  __shared__ uint64_t turns[32];
  if (rt.on && threadIdx.x < 32) {
    uint64_t v = 0;
#pragma unroll
    for (int l = 0; l < 32; ++l) v = lane == l ? rt.turn[l] : v;
    turns[lane] = v;
  }
  __syncthreads();
  chain_wait();
  chain_release();
  if (i >= n) return;
  const uint16_t* src = x + i * stride;
  const int seq = seq_of[i], pos = pos_of[i];
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src) + lane);
  const uint4 c = __ldcs(reinterpret_cast<const uint4*>(src) + 32 + lane);
  uint32_t key = __ldcs(reinterpret_cast<const uint32_t*>(src + 512) + lane);
  const int64_t row = entry_row(b, seq, pos, kv_rows);
  if (row < 0) {  // uniform over the warp
    if (row == -2 && lane == 0) atomicOr(status, DSA_DEVERR_INDEX);
    return;
  }
  if (rt.on) key = rotate_key(rt, turns[lane], lane, pos, key);
  store_row<RT>(kv + row * row_bytes<RT>(), lane, a, c, key);
}

// The INT4 quantiser: rows in order, keys copied.
__global__ void __launch_bounds__(kAppendWarps * 32)
    kv_int4_quant_kernel(const uint16_t* __restrict__ x, int64_t rows, uint8_t* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (i >= rows) return;
  const uint16_t* src = x + i * 576;
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(src) + lane);
  const uint4 c = __ldcs(reinterpret_cast<const uint4*>(src) + 32 + lane);
  const uint32_t key = __ldcs(reinterpret_cast<const uint32_t*>(src + 512) + lane);
  store_row<kRowInt4>(out + i * DSA_KV_ROW_BYTES_INT4, lane, a, c, key);
}

constexpr int kReadWarps = 4, kReadRows = 2;  // rows a warp has in flight
template <int RT>
__global__ void __launch_bounds__(kReadWarps * 32)
    kv_read_kernel(const uint8_t* __restrict__ kv, int64_t kv_rows, const int32_t* __restrict__ seq_of,
                   const int32_t* __restrict__ pos_of, int n, const BatchArgs b,
                   uint16_t* __restrict__ out, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5)) * kReadRows;
  chain_wait();
  chain_release();
  if (i0 >= n) return;
  const int m = static_cast<int>(min(static_cast<int64_t>(kReadRows), n - i0));
  // lane u < m resolves entry i0 + u for the warp
  int64_t mine = -1;
  if (lane < m) {
    mine = entry_row(b, seq_of[i0 + lane], pos_of[i0 + lane], kv_rows);
    if (mine == -2) atomicOr(status, DSA_DEVERR_INDEX);
  }
  int64_t row[kReadRows];
  LaneRow<RT> v[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    row[u] = __shfl_sync(0xffffffffu, mine, u);
    if (row[u] >= 0) v[u].load(kv + row[u] * row_bytes<RT>(), lane);
  }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    if (u >= m) break;
    uint4 va = make_uint4(0, 0, 0, 0), vb = va;
    uint32_t key = 0;
    if (row[u] >= 0) {
      v[u].values(va, vb);
      key = v[u].key;
    }
    uint16_t* dst = out + (i0 + u) * 576;
    __stcs(reinterpret_cast<uint4*>(dst) + lane, va);
    __stcs(reinterpret_cast<uint4*>(dst) + 32 + lane, vb);
    __stcs(reinterpret_cast<uint32_t*>(dst + 512) + lane, key);
  }
}

}  // namespace

cudaError_t launch_kv_append(const void* x, int64_t stride, const int32_t* seq_of,
                             const int32_t* pos_of, int n, const dsa_batch_t& b, int row_type,
                             const double* inv_freq, void* kv, int64_t kv_rows, int* status,
                             cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  RopeTurns rt{};
  rt.on = inv_freq != nullptr;
  if (inv_freq)
    for (int i = 0; i < 32; ++i) {
      const double f = inv_freq[i];
      rt.f[i] = f;
      if (f > 0 && f <= 1) {
        rt.usual |= 1u << i;
        // f / 2 pi in (0, 0.16): below 2^62 in units of 2^-64, as a product with the
        // pair of doubles nearest to 2^64 / 2 pi (long double is software on Arm)
        const double kHi = 2935890503282001408.0, kLo = -181.50375616818447;
        const double p = f * kHi, whole = std::floor(p);
        const double rest = (p - whole) + (std::fma(f, kHi, -p) + f * kLo);
        rt.turn[i] = static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint(rest));
      }
    }
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(n) + kAppendWarps - 1) / kAppendWarps));
  const dim3 block(kAppendWarps * 32);
  prof_begin(stream);
  auto* kern = row_type == kRowBf16  ? kv_append_kernel<kRowBf16>
               : row_type == kRowFp8 ? kv_append_kernel<kRowFp8>
                                     : kv_append_kernel<kRowInt4>;
  const cudaError_t e = launch_chained(kern, grid, block, 0, stream, 1, static_cast<const uint16_t*>(x),
                                       stride, seq_of, pos_of, n, to_args(b), rt,
                                       static_cast<uint8_t*>(kv), kv_rows, status);
  prof_end(kLaunchAppend, stream);
  count_launch(kLaunchAppend);
  return e;
}

cudaError_t launch_kv_read(const void* kv, int64_t kv_rows, int row_type, const int32_t* seq_of,
                           const int32_t* pos_of, int n, const dsa_batch_t& b, void* out, int* status,
                           cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  constexpr int kPer = kReadWarps * kReadRows;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(n) + kPer - 1) / kPer));
  prof_begin(stream);
  auto* kern = row_type == kRowBf16  ? kv_read_kernel<kRowBf16>
               : row_type == kRowFp8 ? kv_read_kernel<kRowFp8>
                                     : kv_read_kernel<kRowInt4>;
  const cudaError_t e = launch_chained(kern, grid, dim3(kReadWarps * 32), 0, stream, 1,
                                       static_cast<const uint8_t*>(kv), kv_rows, seq_of, pos_of, n,
                                       to_args(b), static_cast<uint16_t*>(out), status);
  prof_end(kLaunchRead, stream);
  count_launch(kLaunchRead);
  return e;
}

cudaError_t launch_kv_int4_quantize(const void* kv, int64_t rows, uint8_t* out, cudaStream_t stream) {
  if (rows == 0) return cudaSuccess;
  const int64_t blocks = (rows + kAppendWarps - 1) / kAppendWarps;
  prof_begin(stream);
  kv_int4_quant_kernel<<<static_cast<unsigned>(blocks), kAppendWarps * 32, 0, stream>>>(
      static_cast<const uint16_t*>(kv), rows, out);
  prof_end(kLaunchQuant, stream);
  count_launch(kLaunchQuant);
  return cudaGetLastError();
}

}  // namespace dsa
