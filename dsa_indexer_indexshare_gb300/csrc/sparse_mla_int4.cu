// Absorbed-MLA sparse attention over INT4 cache rows (416 bytes a position: see
// kv_rows.cu), the same function as sparse_mla.cu on the bf16 values the rows
// stand for:
//   z_s = scale * (q_lat[t,h] . C[s,:512] + q_rope[t,h] . C[s,512:])
//   out[t,h] = sum_s softmax(z)_s C[s,:512]
//
// The products are those of the bf16 kernels, 128 keys a block:
//   S^T[128 keys, H]  = C . Q^T          (A = C, a key per TMEM lane)
//   O^T[512 dims, H] += C^T . P          (A = C^T, a dim per TMEM lane)
// in the same order of terms, so the results are bit for bit what those kernels
// give on the rows read back in bf16 (short of the range's ends, see Widen).
//
// What differs is where the operand C lives.  The bf16 kernels keep a block as
// a 144 KB tile of shared memory, which both products read (about 3400 cycles
// of shared-memory bandwidth a block) and which one block at a time can occupy.
// Here only the 4-bit rows are in shared memory (three blocks of codes, 38 KB
// each, gathered by cp.async up to two blocks ahead), and sixteen widening warps
// write the bf16 operands straight into TMEM, in slots of 128 lanes x 32
// columns:
//   - a slot of S^T: 64 dims of 128 keys; a thread is a key, reads its own codes
//     (two 16-byte loads) and stores 32 columns of neighbouring pairs of dims
//   - a slot of O^T: 128 dims of 64 keys; ldmatrix.trans gives a thread the codes
//     of four dims for pairs of keys (the row format puts the four codes of a
//     16-bit half 4 bits apart, so a transposed half-word holds one dim of two
//     keys in matching places), stored with the 16x128b fragment: lane
//     8i + r of a quarter holds dim 8 (r / 2) + 2i + r % 2 of its group of 32
// A pair of values costs one logical operation and one packed fma (see Widen).
//
// Two warps issue the products, each from a ring of slots (three, or five for up to
// 32 heads): the next block's scores are computed while this block's softmax runs,
// and the softmax of a block while the previous block's O^T products do.  Measured: an M128 N64 K16 MMA takes
// 48 cycles with both operands in shared memory (its bandwidth) and 32 with A in
// TMEM (the tensor pipe's rate), so a block of 68 takes at least 2200 cycles
// against 3260.
//
// Rows of no visible position are gathered as zeros, whatever the cache holds.
// One CTA per SM walks a list of tokens (many tokens), or a cluster of NSPLIT
// CTAs shares the blocks of one token (decode).
//
// Measured (64 heads, K = 2048; in a replayed graph): 8192 queries of one sequence in
// 2.51 ms (the bf16 kernel 2.54 ms; 2.04e12 operations, 43% of the cuBLAS rate), a decode
// step of 64 tokens in 37.5 us (bf16 rows 43.3 us; 45 and 53 us after a flush of L2), of 8
// tokens in 19.0 us (16.1 us).  A block of 128 keys takes about 6900 cycles of
// an SM, three times its 68 MMAs.  The widening bounds it: 68 slot fills of a warp
// (four warps of a scheduler fill a slot in 550 cycles
// side by side, one alone in 300), and about 190 cycles around each fill to find
// the slot free and to announce it.  Of the 600 us that 2560 queries took when parts were
// left out, the arithmetic of the widening was 13%, its stores 27%, the MMAs 9%, the
// exponentials 1% (590 us now); slots of half the size cost 25%, and neither an earlier
// release of S^T, nor P in two halves, nor fewer looks at the barriers gain any.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "mla.cuh"

namespace dsa {
namespace {

constexpr int kRow = DSA_KV_ROW_BYTES_INT4;
constexpr int kListMax = 128;    // tokens per CTA
constexpr int kCodePitch = 304;  // codes and scales of a row (288 bytes): 19 16-byte units, odd, so
constexpr int kKeyPitch = 144;   // that eight rows' units lie in different banks; RoPE key (128)

template <int H>
struct Int4Cfg {
  static constexpr int QSUB = H * 128;    // one 64-dim sub-tile of Q: H rows x 128 B
  static constexpr int Q_BYTES = 9 * QSUB;
  static constexpr int PSUB = H * 128;    // P^T sub-tile (H < 64): H rows x 64 keys
  static constexpr bool P_MN = H == 64;   // P stored MN-major: one 128-byte row of heads per key
  static constexpr int P_BYTES = 16384;
  static constexpr int CODE = 128 * kCodePitch;  // one block's codes and scales
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = (Q_BYTES + 1023) & ~1023;
  static constexpr int OFF_CODE = OFF_P + P_BYTES;
  static constexpr int OFF_KEY = OFF_CODE + 3 * CODE;
  static constexpr int OFF_SCR = OFF_KEY + 128 * kKeyPitch;
  static constexpr int SCR_FLOATS = H + 4 * H + H + H;  // m_used, red[4], lsum, fac
  static constexpr int OFF_BAR = OFF_SCR + SCR_FLOATS * 4;
  // Operand slots of 32 TMEM columns that each of the two products has: as many as
  // fit beside S^T and O^T (2560 queries of 32 heads: 545 us with three, 539 with five).
  static constexpr int SLOTS = H == 64 ? 3 : 5;
  static constexpr int NBAR = 8 + 4 * SLOTS + 6 + 2 + 3;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_VAL = (OFF_MISC + 64 + 15) & ~15;  // 3 x 128 validity bits
  static constexpr int OFF_LIST = OFF_VAL + 48;
  static constexpr int SMEM = OFF_LIST + kListMax * 16 + 1024;
  static constexpr int HW = H > 32 ? 32 : H;  // heads per softmax warp
  static constexpr int NSW = 4 * (H / HW);    // softmax warps
  static constexpr int NDW = 16;              // widening warps: two sets of four for each product
  static constexpr int NGW = 4;               // gathering warps
  static constexpr int NOW = (NSW + NDW) / 4;  // warps of a lane quarter that write a split token's O^T
  static constexpr int NT = (NSW + NDW + 4 + NGW) * 32;  // + two MMA issuers, the query loader, an idle warp
  // Registers a thread: the launch gives every thread R_LAUNCH (64K over the
  // threads, in eights); the softmax warps take more, the others give them up.
  static constexpr int R_LAUNCH = (65536 / NT) & ~7;
  static constexpr int R_SOFT = H == 64 ? 104 : 136;
  static constexpr int R_WIDEN = H == 64 ? 56 : 72;
  static constexpr int R_REST = 40;
  static_assert(NSW * 32 * R_SOFT + NDW * 32 * R_WIDEN + (4 + NGW) * 32 * R_REST <= NT * R_LAUNCH,
                "the increase must find its registers");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t TM_S = 0;     // S^T: H columns
  static constexpr uint32_t TM_R = 64;    // operand slots of S^T, then of O^T
  static constexpr uint32_t TM_O = TM_R + 2 * SLOTS * 32;  // O^T chunk c: H columns
  static_assert(TM_O + 4 * H <= TMEM_COLS && H <= TM_R, "TMEM");
  static_assert(PSUB * 2 <= P_BYTES && 16 * H * 4 <= P_BYTES, "P, and the combine's weights over it");
  static_assert(H * 512 * 4 <= OFF_SCR - OFF_CODE, "O staging over the code and key buffers");
  static_assert(SMEM <= 232448, "shared memory");
};

struct Int4Params {
  BatchArgs b;
  const uint8_t* kv;  // [kv_rows, 416]
  int64_t kv_rows;
  int direct;  // index entries are absolute rows (no causal test)
  const int32_t* idx;
  int K;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part;  // tokens split over 4, 8 or 16 CTAs: see MlaParams
  int* status;
  uint64_t timeout_ns;
};

// Widening.  A bf16 pattern below 0x0100 is its integer times 2^-133 (the
// subnormals and the first binade have one spacing), so a masked nibble n in bits
// 0..3 or 4..7 of a half is the number n * 2^-133 or n * 2^-129 as it stands, and
//   fma(n * 2^-133, s * 2^(133 - kShift), -8 s * 2^-kShift) = (n - 8) s * 2^-kShift
// is the value in one packed operation with its only rounding.  kShift keeps the
// factor finite: the operand holds every value (and RoPE key) times 2^-kShift,
// which the score scale and the output's normalisation take back, all exact.
// Scales from 2^(kShift - 6) on, whose factor would overflow, take one more
// product (n * 2^-133 * 2^kLift first).  (Values below 2^(kShift - 126) lose bits
// as subnormals.)
constexpr int kShift = 40, kLift = 100;
constexpr float kUnshift = 1099511627776.f;  // 2^kShift
__host__ __device__ constexpr uint32_t pow2_pair(int e) { return static_cast<uint32_t>((e + 127) << 7) * 0x00010001u; }
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// The factors of a pair of scales.  BIG: for scales whose x0 would overflow.
template <bool BIG>
struct Widen {
  uint32_t x0, x1, c;
  __device__ __forceinline__ explicit Widen(uint32_t s2) {
    x0 = mul2(s2, pow2_pair(133 - kShift - (BIG ? kLift : 0)));
    x1 = mul2(x0, pow2_pair(-4));
    c = mul2(s2, pow2_pair(3 - kShift) | 0x80008000u);
  }
  // pair k of a word: nibbles k and k + 4
  __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t w8, int k) const {
    uint32_t u = (k < 2 ? w : w8) & ((k & 1) ? 0x00F000F0u : 0x000F000Fu);
    if (BIG) u = mul2(u, pow2_pair(kLift));
    return fma2(u, (k & 1) ? x1 : x0, c);
  }
};
// the larger bits of each half, and whether one of them is a scale above
// 2^(kShift - 6) (or not a number)
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ bool big_scale(uint32_t bits) {
  return max_bits(bits, pow2_pair(kShift - 6)) != pow2_pair(kShift - 6);
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Four transposed 8x8 matrices of 16-bit elements (lane l: the address of row l & 7 of matrix l / 8).
__device__ __forceinline__ void ldsm4_trans(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// 16 columns of this thread's lane.
__device__ __forceinline__ void tmem_st_row16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 16 columns: register 2j + e of lane l is column 4j + l % 4 of TMEM lane 8e + l / 4.
__device__ __forceinline__ void tmem_st_frag16(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// MMA issue.  The whole warp walks the issue loop and one elected lane issues:
// control flow and operands stay uniform over the warp, so descriptors and
// addresses live in uniform registers and a wait between products costs the
// tensor pipe nothing.  (Issued from a branch of one lane, every MMA took 45 to
// 100 cycles of the issuing thread; this way 32, the pipe's rate.)
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p;
}
// D[tmem] (+)= A[tmem] * B[smem]^T, bf16 inputs, fp32 accumulation, by the elected lane.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void umma_commit_elected(uint32_t bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(elected)
      : "memory");
}

// Barrier over nthreads threads that tells each whether any came with v.
__device__ __forceinline__ int named_bar_or(int id, int nthreads, bool v) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\tselp.s32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(static_cast<int>(v))
      : "memory");
  return r;
}

// A slot of a ring and how often the ring has been gone through.
template <int N>
struct Ring {
  int i = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void step() {
    if (++i == N) {
      i = 0;
      ++round;
    }
  }
};

// SHORT: lists of at most 64 entries.  Only keys 0-63 of a block are gathered,
// widened and multiplied with P (512 queries of 16 heads over 64 entries: 24.3 us
// with whole blocks, 22.1 us this way; chosen at run time in one kernel it cost long
// lists 1.7%).
template <int H, int NSPLIT, bool PAGED, bool SHORT>
__global__ void __launch_bounds__(Int4Cfg<H>::NT, 1)
    sparse_mla_int4_kernel(const __grid_constant__ CUtensorMap qlat_map,
                           const __grid_constant__ CUtensorMap qrope_map, const Int4Params p) {
  using C = Int4Cfg<H>;
  constexpr int HW = C::HW, NSW = C::NSW, NDW = C::NDW, NT = C::NT, NST = NSW * 32;
  constexpr int W_S = NSW + NDW, W_O = W_S + 1, W_Q = W_S + 2, W_G = W_S + 4;
  constexpr bool kMergeL2 = NSPLIT >= 4;  // as in sparse_mla.cu: pairs merge through the cluster
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = NSPLIT > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const uint32_t sQ = smem_u32(sm + C::OFF_Q);
  float* m_used = reinterpret_cast<float*>(sm + C::OFF_SCR);
  float* red = m_used + H;
  float* lsum = red + 4 * H;
  float* fac = lsum + H;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + C::OFF_MISC);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + C::OFF_MISC + 8);
  int* wcnt = reinterpret_cast<int*>(sm + C::OFF_MISC + 16);  // list entries per warp
  uint8_t* vbits = sm + C::OFF_VAL;
  int4* toks = reinterpret_cast<int4*>(sm + C::OFF_LIST);  // {t, pos, first row lo, hi} or {t, pos, seq, 0}
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  // Q: the token's query landed / QD: its last S^T product done; S / SR: S^T of a
  // block done / read; P: P written; PV: the block's O^T products done; DS / DO: every
  // product done (before exit); FS, FO / RS, RO: slot of S^T, of O^T filled / consumed;
  // CF / CE: a block's codes landed / read for the last time; KF / KE: RoPE keys landed
  // / read; VF: validity bits written
  constexpr int B_Q = 0, B_QD = 1, B_S = 2, B_SR = 3, B_P = 4, B_PV = 5, B_DS = 6, B_DO = 7, B_RS = 8,
                B_RO = B_RS + C::SLOTS, B_FS = B_RO + C::SLOTS, B_FO = B_FS + C::SLOTS, B_CF = B_FO + C::SLOTS,
                B_CE = B_CF + 3, B_KF = B_CE + 3, B_KE = B_KF + 1, B_VF = B_KE + 1;
  static_assert(B_VF + 3 == C::NBAR, "");

  if (tid == 0) {
    *abort_flag = 0;
    for (int i = B_Q; i < B_FS; ++i) mbar_init(bar(i), i == B_SR || i == B_P ? NSW : 1);
    for (int i = B_FS; i < B_CF; ++i) mbar_init(bar(i), 4);
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(B_CF + i), C::NGW * 32);
      mbar_init(bar(B_CE + i), NDW);
      mbar_init(bar(B_VF + i), C::NGW);
    }
    mbar_init(bar(B_KF), C::NGW * 32);
    mbar_init(bar(B_KE), 4);
    fence_mbar_init();
  }
  if (tid < H) m_used[tid] = -INFINITY;
  if (warp == W_O) {
    tmem_alloc(smem_u32(tslot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == W_Q && lane == 0) {
    tma_prefetch_desc(&qlat_map);
    tma_prefetch_desc(&qrope_map);
  }
  chain_wait();     // the previous kernel of the stream has completed
  chain_release();  // the next one may be scheduled

  // ---- the tokens of this CTA, heaviest first (work item w: the
  // (w / num_seqs)-th latest query of sequence w % num_seqs); items are dealt
  // out in rounds, in order in even rounds and in reverse in odd ones.  A query
  // at an invalid position gets a zero output, lse = -inf and DSA_DEVERR_BATCH.
  if (tid < kListMax) {
    bool mine = false;
    int4 tk = make_int4(0, 0, 0, 0);
    const unsigned cta = blockIdx.x / NSPLIT, ctas = gridDim.x / NSPLIT;
    const int64_t w = static_cast<int64_t>(tid) * ctas + ((tid & 1) ? ctas - 1 - cta : cta);
    if (w < static_cast<int64_t>(p.b.max_q) * p.b.num_seqs) {
      const int seq = static_cast<int>(w % p.b.num_seqs);
      const int qi = p.b.max_q - 1 - static_cast<int>(w / p.b.num_seqs);
      const int qs = p.b.q_start[seq], qe = p.b.q_start[seq + 1];
      if (qs < 0 || qe < qs || qe > p.b.num_q) {
        atomicOr(p.status, DSA_DEVERR_BATCH);
      } else if (qs + qi < qe) {
        const int t = qs + qi;
        const int pos = query_pos(p.b, t, p.status);
        if (pos >= 0) {
          const int64_t r0 = PAGED ? seq : p.direct ? 0 : seq_base_row(p.b, seq);
          mine = true;
          tk = make_int4(t, pos, static_cast<int>(static_cast<uint32_t>(r0)),
                         static_cast<int>(static_cast<uint64_t>(r0) >> 32));
        } else if (rank == 0) {
          uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(t) * H * 512);
          for (int i = 0; i < H * 512 / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
          if (p.lse)
            for (int h = 0; h < H; ++h) p.lse[static_cast<int64_t>(t) * H + h] = -INFINITY;
        }
      }
    }
    const unsigned bal = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) wcnt[warp] = __popc(bal);
    named_bar_sync(1, kListMax);
    int off = 0;
    for (int w2 = 0; w2 < warp; ++w2) off += wcnt[w2];
    if (mine) toks[off + __popc(bal & ((1u << lane) - 1u))] = tk;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int ntok = 0;  // uniform over the CTA
#pragma unroll
  for (int w2 = 0; w2 < kListMax / 32; ++w2) ntok += wcnt[w2];
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tslot, 0);  // (known to be uniform)
  const uint64_t to = p.timeout_ns;
  volatile int no_abort = 0;
  auto tok_nvalid = [&](const int4& tk) { return min(p.K, tk.y + 1); };
  // this CTA's blocks of a token: [rank * nb / NSPLIT, (rank + 1) * nb / NSPLIT)
  auto tok_j0 = [&](const int4& tk) { return rank * ((tok_nvalid(tk) + 127) / 128) / NSPLIT; };
  auto tok_j1 = [&](const int4& tk) { return (rank + 1) * ((tok_nvalid(tk) + 127) / 128) / NSPLIT; };
  constexpr int two = SHORT ? 0 : 1;  // a chunk of 128 dims of O^T takes 1 << two slots
  // (only a split token, of which a CTA has one, can leave a CTA without blocks)
  auto tok_nb = [&](int i) {
    const int4 tk = toks[i];
    return tok_j1(tk) - tok_j0(tk);
  };

  // A split token's unnormalised O^T as [h][512], in the token's partial results
  // in global memory or (pairs) in shared memory.  Unit c of a lane quarter: the
  // 128-dim chunk c % 4 of the HW heads from HW * (c / 4).  TMEM lane L of a quarter
  // holds dim 8 (L % 8 / 2) + 2 (L / 8) + L % 2 of its 32.
  auto part_base = [&]() {
    return kMergeL2 ? p.part + (static_cast<int64_t>(toks[0].x) * NSPLIT + rank) * (H * 512 + 2 * H)
                    : reinterpret_cast<float*>(sm + C::OFF_CODE);
  };
  auto write_part = [&](int c) {
    const int quarter = warp & 3, h0 = (c >> 2) * HW;
    const int dim = 128 * (c & 3) + 32 * quarter + 8 * ((lane & 7) >> 1) + 2 * (lane >> 3) + (lane & 1);
    float* Od = part_base() + h0 * 512 + dim;
#pragma unroll 1
    for (int hh = 0; hh < HW; hh += 16) {
      float o[16];
      tmem_cols_load<16>(tbase + (static_cast<uint32_t>(quarter * 32) << 16) + C::TM_O + (c & 3) * H + h0 + hh, o);
#pragma unroll
      for (int h = 0; h < 16; ++h) Od[(hh + h) * 512] = o[h];
    }
  };

  if (warp >= W_S) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_REST));
    if (warp == W_S) {
    // ------------------------------------------------ issuer of S^T = C . Q^T
    constexpr uint32_t id_qk = idesc_bf16(128, H, false, false);
    const uint32_t el = elect_lane();
    const uint64_t dq = sdesc_sw128(sQ, 0, 1024);
    const uint32_t d_s = tbase + C::TM_S, ring = tbase + C::TM_R;
    bool ok = true;
    Ring<C::SLOTS> r;
    uint32_t n = 0;  // blocks of this CTA so far
    for (int i = 0; ok && i < ntok; ++i) {
      const int nb = tok_nb(i);
      ok = mbar_wait(bar(B_Q), i & 1, abort_flag, p.status, to);
      for (int u = 0; ok && u < nb; ++u, ++n) {
        if (n > 0) ok = mbar_wait(bar(B_SR), (n - 1) & 1, abort_flag, p.status, to);
#pragma unroll 1  // (short code: the roles share the instruction cache)
        for (int s = 0; s < 9; ++s) {
          ok = ok && mbar_wait(bar(B_FS + r.i), r.round & 1, abort_flag, p.status, to);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = ring + r.i * 32;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_ts(d_s, a + kk * 8, sdesc_at(dq, s * C::QSUB + kk * 32), id_qk, (s | kk) != 0, el);
          umma_commit_elected(bar(B_RS + r.i), el);
          r.step();
        }
        if (!ok) break;
        umma_commit_elected(bar(B_S), el);
        if (u == nb - 1) umma_commit_elected(bar(B_QD), el);
      }
    }
    umma_commit_elected(bar(B_DS), el);
    mbar_wait(bar(B_DS), 0, &no_abort, nullptr, to);
  } else if (warp == W_O) {
    // ------------------------------------------------ issuer of O^T += C^T . P
    constexpr uint32_t id_pv = idesc_bf16(128, H, false, C::P_MN);
    const uint32_t el = elect_lane();
    const uint64_t dp = C::P_MN ? sdesc_sw128(smem_u32(sm + C::OFF_P), 8192, 1024)
                                : sdesc_sw128(smem_u32(sm + C::OFF_P), 0, 1024);
    const uint32_t d_o = tbase + C::TM_O, ring = tbase + C::TM_R + C::SLOTS * 32;
    bool ok = true;
    Ring<C::SLOTS> r;
    uint32_t n = 0;
    for (int i = 0; ok && i < ntok; ++i) {
      const int nb = tok_nb(i);
      // a token's first block overwrites O^T: its P arrives only after the softmax
      // warps have read the previous token's O^T
      for (int u = 0; ok && u < nb; ++u, ++n) {
        ok = mbar_wait(bar(B_P), n & 1, abort_flag, p.status, to);
#pragma unroll 1
        for (int s = 0; s < 4 << two; ++s) {  // dims 128 (s >> two) .., keys 64 (s & two) ..
          ok = ok && mbar_wait(bar(B_FO + r.i), r.round & 1, abort_flag, p.status, to);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = ring + r.i * 32;
          const uint64_t db = sdesc_at(dp, (s & two) * (C::P_MN ? 8192 : C::PSUB));
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)  // key 16 k4 of these
            umma_bf16_ts(d_o + (s >> two) * H, a + k4 * 8, sdesc_at(db, k4 * (C::P_MN ? 2048 : 32)), id_pv,
                         k4 > 0 || (s & two) || u > 0, el);
          umma_commit_elected(bar(B_RO + r.i), el);
          r.step();
        }
        if (!ok) break;
        umma_commit_elected(bar(B_PV), el);
      }
    }
    umma_commit_elected(bar(B_DO), el);
    mbar_wait(bar(B_DO), 0, &no_abort, nullptr, to);
  } else if (warp == W_Q) {
    // ------------------------------------------------ the query of each token, by TMA
    if (lane == 0) {
      int nq = 0;
      for (int i = 0; i < ntok; ++i) {
        const int4 tk = toks[i];
        if (i > 0 && !mbar_wait(bar(B_QD), (i - 1) & 1, abort_flag, p.status, to)) break;
        mbar_arrive_expect_tx(bar(B_Q), C::Q_BYTES);
        for (int c = 0; c < 8; ++c) tma_load_2d(sQ + c * C::QSUB, &qlat_map, 64 * c, tk.x * H, bar(B_Q));
        tma_load_2d(sQ + 8 * C::QSUB, &qrope_map, 0, tk.x * H, bar(B_Q));
        ++nq;
        if (i + 1 < ntok) {  // the next token's query into L2
          const int tn = toks[i + 1].x;
          for (int c = 0; c < 8; ++c) tma_prefetch_l2_2d(&qlat_map, 64 * c, tn * H);
          tma_prefetch_l2_2d(&qrope_map, 0, tn * H);
        }
      }
      if (nq > 0) mbar_wait(bar(B_Q), (nq - 1) & 1, &no_abort, nullptr, to);  // the last copy landed
    }
    __syncwarp();
  } else if (warp >= W_G) {
    // ------------------------------------------------ gathering warps
    // Warp g holds the rows 32g + lane of a block (row index, -1 for none: zeros are
    // copied) and copies codes (16 chunks of two rows an instruction), scales (2 of
    // 16 rows) and keys (8 of four rows).
    const int g = warp - W_G;
    const int bps = p.b.blocks_per_seq;
    const int rshift = PAGED ? __ffs(p.b.block_rows) - 1 : 0;  // block_rows is a power of two
    const uint32_t sCode = smem_u32(sm + C::OFF_CODE), sKey = smem_u32(sm + C::OFF_KEY);
    auto place = [&](const int4& tk, int e) -> int {
      if (e < 0 || (!p.direct && e > tk.y)) return -1;
      int64_t rr;
      if constexpr (!PAGED) {
        rr = static_cast<int64_t>((static_cast<uint64_t>(static_cast<uint32_t>(tk.w)) << 32) |
                                  static_cast<uint32_t>(tk.z)) + e;
      } else {
        const int blk = e >> rshift;
        if (blk >= bps) return -1;
        const int32_t id = ld_keep_i32(p.b.block_table + static_cast<int64_t>(tk.z) * bps + blk);
        rr = id < 0 ? -1 : (static_cast<int64_t>(id) << rshift) + (e & (p.b.block_rows - 1));
      }
      return rr < 0 || rr >= p.kv_rows ? -1 : static_cast<int>(rr);  // kv_rows < 2^31
    };
    auto copy16 = [&](uint32_t dst, const uint8_t* src) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    };
    auto copy16z = [&](uint32_t dst, const uint8_t* at, int row) {  // zeros where row < 0
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                   "l"(at + static_cast<int64_t>(max(row, 0)) * kRow), "r"(row < 0 ? 0 : 16)
                   : "memory");
    };
    auto arrive_copies = [&](int b) {
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar(b)) : "memory");
    };
    int i = 0, j = 0, jend = 0;  // the block whose entry is in e
    auto fetch = [&](int& e) {  // this lane's entry of block (i, j)
      e = -1;
      if (i >= ntok) return false;
      const int4 tk = toks[i];
      const int sl = j * 128 + 32 * g + lane;
      if (sl < tok_nvalid(tk)) e = ld_stream_i32(p.idx + static_cast<int64_t>(tk.x) * p.K + sl);
      return true;
    };
    if (ntok > 0) {
      j = tok_j0(toks[0]);
      jend = tok_j1(toks[0]);
      if (j >= jend) i = ntok;
    }
    int e;
    bool have = fetch(e);
    uint32_t n = 0;
    int buf = 0;      // n % 3
    uint32_t ph = 0;  // (n / 3) & 1
    while (have) {
      const int row = place(toks[i], e);
      if (row < 0 && e != -1) atomicOr(p.status, DSA_DEVERR_INDEX);
      if (++j >= jend) {
        ++i;
        if (i < ntok) {
          j = tok_j0(toks[i]);
          jend = tok_j1(toks[i]);
        }
      }
      have = fetch(e);
      // codes and scales, once block n - 3's have been read
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_CE + buf), ph ^ 1u, abort_flag, p.status, to))) break;
      const unsigned okb = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) {
        *reinterpret_cast<uint32_t*>(vbits + buf * 16 + g * 4) = okb;
        mbar_arrive(bar(B_VF + buf));
      }
      const uint32_t dc = sCode + buf * C::CODE + (32 * g + (lane >> 4)) * kCodePitch + (lane & 15) * 16;
      const uint8_t* src = p.kv + (lane & 15) * 16;
      if (SHORT && g >= 2) {
      } else if (okb == 0xffffffffu) {
#pragma unroll 4
        for (int r = 0; r < 32; r += 2)  // rows r, r + 1
          copy16(dc + r * kCodePitch, src + static_cast<int64_t>(__shfl_sync(0xffffffffu, row, r + (lane >> 4))) * kRow);
      } else {
#pragma unroll 1
        for (int r = 0; r < 32; r += 2)
          copy16z(dc + r * kCodePitch, src, __shfl_sync(0xffffffffu, row, r + (lane >> 4)));
      }
#pragma unroll 1
      for (int r = SHORT && g >= 2 ? 32 : 0; r < 32; r += 16)
        copy16z(sCode + buf * C::CODE + (32 * g + r + (lane >> 1)) * kCodePitch + 256 + (lane & 1) * 16,
                p.kv + 256 + (lane & 1) * 16, __shfl_sync(0xffffffffu, row, r + (lane >> 1)));
      arrive_copies(B_CF + buf);
      // keys, once block n - 1's have been read
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_KE), (n & 1) ^ 1u, abort_flag, p.status, to))) break;
#pragma unroll 2
      for (int r = SHORT && g >= 2 ? 32 : 0; r < 32; r += 4)
        copy16z(sKey + (32 * g + r + (lane >> 3)) * kKeyPitch + (lane & 7) * 16, p.kv + 288 + (lane & 7) * 16,
                __shfl_sync(0xffffffffu, row, r + (lane >> 3)));
      arrive_copies(B_KF);
      ++n;
      if (++buf == 3) {
        buf = 0;
        ph ^= 1u;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp >= NSW) {
    // ------------------------------------------------ widening warps
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_WIDEN));
    // For each product two sets of four warps (one per TMEM lane quarter) fill the
    // slots in turn, each in two halves of 16 columns (all 32 would not fit in the
    // registers).  Whether the slot is free is asked before the first half is
    // widened and waited for before it is stored: that hides the 95 cycles of a look
    // (8192 queries: 2.54 -> 2.51 ms).
    const int team = (warp - NSW) >> 2;
    const bool for_o = team >= 2;
    const int set = team & 1, quarter = warp & 3;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + C::TM_R + (for_o ? C::SLOTS * 32 : 0);
    const int key = quarter * 32 + lane;
    const uint32_t sCode = smem_u32(sm + C::OFF_CODE);
    const uint32_t sKeyRow = smem_u32(sm + C::OFF_KEY) + key * kKeyPitch;
    int nblk = 0;
    for (int i = 0; i < ntok; ++i) nblk += tok_nb(i);
    // this set's slots: every other one around the ring
    const uint32_t b_free = bar(for_o ? B_RO : B_RS), b_full = bar(for_o ? B_FO : B_FS);
    uint32_t ri = set, rph = 1;  // slot, and the parity that its last use has when it is free
    bool alive = true;
    // The slot's last products are done: looked at before its first half is widened,
    // waited for before that is stored.
    auto look = [&]() { return mbar_try_wait(b_free + 8 * ri, rph); };
    auto acquire = [&](bool free) {
      alive = __all_sync(0xffffffffu, free || mbar_wait(b_free + 8 * ri, rph, abort_flag, p.status, to));
      if (alive) tc_fence_after();
      return alive;
    };
    auto publish = [&]() {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_full + 8 * ri);
      ri += 2;
      if (ri >= C::SLOTS) {
        ri -= C::SLOTS;
        rph ^= 1u;
      }
    };
    auto read_done = [&](int b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    int buf = 0;      // n % 3
    uint32_t ph = 0;  // (n / 3) & 1
    int s = set;      // this set's next slot of the block
    const int slots = for_o ? 4 << two : 8;
#pragma unroll 1
    for (int n = 0; alive && n < nblk; ++n) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_CF + buf), ph, abort_flag, p.status, to))) break;
      const uint32_t codes = sCode + buf * C::CODE;
#pragma unroll 1
      for (; s < slots; s += 2) {
        const uint32_t slot = lane_base + ri * 32;
        const bool free = look();
        if (SHORT && !for_o && quarter >= 2) {  // keys 64 .. are in no list
          if (s >= 6) read_done(B_CE + buf);
          acquire(free);
        } else if (!for_o) {  // dims 64s .. of this thread's key
          const uint32_t row = codes + key * kCodePitch;
          const uint32_t sc = lds4(row + 256 + 4 * s);
          uint4 a = lds16(row + 32 * s);
          const uint4 a1 = lds16(row + 32 * s + 16);
          if (s >= 6) read_done(B_CE + buf);  // this set's last look at the codes
          // (stored inside: a join of the two forms would copy every value)
          auto widen = [&](auto big_t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const Widen<decltype(big_t)::value> f(__byte_perm(sc, sc, hf ? 0x3232 : 0x1010));
              const uint32_t w[4] = {a.x, a.y, a.z, a.w};
              uint32_t v[16];
#pragma unroll
              for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * m + k] = f.pair(w[m], w[m] >> 8, k);
              if (hf == 0 && !acquire(free)) break;
              tmem_st_row16(slot + 16 * hf, v);
              a = a1;
            }
          };
          if (__builtin_expect(__any_sync(0xffffffffu, big_scale(sc)), 0))
            widen(std::true_type());
          else
            widen(std::false_type());
        } else {  // dims 128 (s >> two) + 32 quarter .., keys 64 (s & two) ..
          const int grp = 4 * (s >> two) + quarter;
          const uint32_t row = codes + (64 * (s & two) + lane) * kCodePitch;
          uint32_t w[8], sc[8];
          ldsm4_trans(w, row + 16 * grp);
          ldsm4_trans(sc, row + 256 + 16 * (grp >> 3));
          ldsm4_trans(w + 4, row + 32 * kCodePitch + 16 * grp);
          ldsm4_trans(sc + 4, row + 32 * kCodePitch + 256 + 16 * (grp >> 3));
          if (s >= slots - 2) read_done(B_CE + buf);
          // of the pairs of keys of eight groups, lane 4 (grp % 8) + l % 4 has this group's
#pragma unroll
          for (int j = 0; j < 8; ++j) sc[j] = __shfl_sync(0xffffffffu, sc[j], 4 * (grp & 7) + (lane & 3));
          uint32_t top = sc[0];
#pragma unroll
          for (int j = 1; j < 8; ++j) top = max_bits(top, sc[j]);
          auto widen = [&](auto big_t) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t lo[8], hi[8];  // lanes 0-15 and 16-31 of the quarter
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const Widen<decltype(big_t)::value> f(sc[4 * hf + j]);
                const uint32_t x = w[4 * hf + j];
                lo[2 * j] = f.pair(x, x >> 8, 0);
                lo[2 * j + 1] = f.pair(x, x >> 8, 1);
                hi[2 * j] = f.pair(x, x >> 8, 2);
                hi[2 * j + 1] = f.pair(x, x >> 8, 3);
              }
              if (hf == 0 && !acquire(free)) break;
              tmem_st_frag16(slot + 16 * hf, lo);
              tmem_st_frag16(slot + (16u << 16) + 16 * hf, hi);
            }
          };
          if (__builtin_expect(__any_sync(0xffffffffu, big_scale(top)), 0))
            widen(std::true_type());
          else
            widen(std::false_type());
        }
        if (!alive) break;
        publish();
      }
      if (!alive) break;
      if (!for_o && s == 8) {  // the RoPE keys
        if (!__all_sync(0xffffffffu, mbar_wait(bar(B_KF), n & 1, abort_flag, p.status, to)) || !acquire(false)) break;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t v[16];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint4 k4 = lds16(sKeyRow + 64 * hf + 16 * m);
            v[4 * m] = mul2(k4.x, pow2_pair(-kShift));
            v[4 * m + 1] = mul2(k4.y, pow2_pair(-kShift));
            v[4 * m + 2] = mul2(k4.z, pow2_pair(-kShift));
            v[4 * m + 3] = mul2(k4.w, pow2_pair(-kShift));
          }
          if (hf == 1) read_done(B_KE);
          tmem_st_row16(lane_base + ri * 32 + 16 * hf, v);
        }
        publish();
        s += 2;
      }
      s -= for_o ? slots : 9;
      if (++buf == 3) {
        buf = 0;
        ph ^= 1u;
      }
    }
    if constexpr (NSPLIT > 1) {
      // (B_DO completes once; B_PV's phases are not followed here)
      if (alive && nblk > 0 && __all_sync(0xffffffffu, mbar_wait(bar(B_DO), 0, abort_flag, p.status, to))) {
        tc_fence_after();
#pragma unroll 1
        for (int c = warp >> 2; c < 4 * NSW / 4; c += C::NOW) write_part(c);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::R_SOFT));
    // ------------------------------------------------ softmax: key = TMEM lane, HW heads
    const int quarter = warp & 3;
    const int h0 = (warp >> 2) * HW;
    const int key = quarter * 32 + lane;
    const uint32_t lane_base = tbase + (static_cast<uint32_t>(quarter * 32) << 16);
    const float sl2 = p.scale_log2 * kUnshift;  // S^T comes times 2^-kShift
    float lpart[HW];  // this thread's share of the softmax denominators
    uint32_t gu = 0;  // blocks of this CTA so far (barrier phases)
    int buf = 0;      // gu % 3
    uint32_t vph = 0;
    bool alive = true;
    // the dim within a 128-dim chunk of O^T that this thread's TMEM lane holds
    const int dl = 32 * quarter + 8 * ((lane & 7) >> 1) + 2 * (lane >> 3) + (lane & 1);
    // v[h] = v[h] * sl2 - (running maximum of head h0 + h)
    auto minus_max = [&](float (&v)[HW]) {
#pragma unroll
      for (int h = 0; h < HW; h += 4) {
        const float4 m = *reinterpret_cast<const float4*>(m_used + h0 + h);
        v[h] = fmaf(v[h], sl2, -m.x);
        v[h + 1] = fmaf(v[h + 1], sl2, -m.y);
        v[h + 2] = fmaf(v[h + 2], sl2, -m.z);
        v[h + 3] = fmaf(v[h + 3], sl2, -m.w);
      }
    };
    // After a wait that ran out, a warp goes on without waiting: every warp comes to
    // every barrier that the softmax warps share.
    auto wait = [&](int b, uint32_t parity) {
      alive = alive && __all_sync(0xffffffffu, mbar_wait(bar(b), parity, abort_flag, p.status, to));
    };
#pragma unroll 1
    for (int i = 0; i < ntok; ++i) {
      const int nb = tok_nb(i);
#pragma unroll
      for (int h = 0; h < HW; ++h) lpart[h] = 0.f;
#pragma unroll 1
      for (int u = 0; u < nb; ++u, ++gu) {
        wait(B_VF + buf, vph);
        const bool valid = (vbits[buf * 16 + (key >> 3)] >> (key & 7)) & 1;
        if (++buf == 3) {
          buf = 0;
          vph ^= 1u;
        }
        wait(B_S, gu & 1);
        tc_fence_after();
        float d[HW];
        tmem_cols_load<HW>(lane_base + C::TM_S + h0, d);
        // the first block sets the running maximum; a later one raises it only
        // when one of its scores exceeds it by more than the threshold
        int resc = 1;
        if (u > 0) {
          float dmax = -INFINITY;
          minus_max(d);
#pragma unroll
          for (int h = 0; h < HW; ++h) dmax = fmaxf(dmax, d[h]);
          resc = named_bar_or(1, NST, valid && dmax > kRescaleThreshold);
          if (resc) tmem_cols_load<HW>(lane_base + C::TM_S + h0, d);  // raw scores again
        }
        if (resc) {
#pragma unroll
          for (int h = 0; h < HW; ++h) d[h] = valid ? d[h] * sl2 : -INFINITY;
          head_reduce<HW, 16, true>(d, lane);
          if (HW == 32 || (lane & 1) == 0) red[quarter * H + h0 + (HW == 32 ? lane : lane >> 1)] = d[0];
          named_bar_sync(1, NST);
          if (tid < H) {
            const float mo = m_used[tid];
            const float mb = fmaxf(fmaxf(red[tid], red[H + tid]), fmaxf(red[2 * H + tid], red[3 * H + tid]));
            const float mn = fmaxf(mo, mb);
            fac[tid] = (mn == -INFINITY) ? 1.f : ex2(mo - mn);
            m_used[tid] = mn;
          }
          named_bar_sync(1, NST);
          tmem_cols_load<HW>(lane_base + C::TM_S + h0, d);
#pragma unroll
          for (int h = 0; h < HW; ++h) lpart[h] *= fac[h0 + h];
          minus_max(d);
        }
        // S^T is in registers: the next block's products may overwrite it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_SR));
        // exponentials while the previous block's O^T products still run
        if (!__all_sync(0xffffffffu, valid)) {
#pragma unroll
          for (int h = 0; h < HW; ++h) d[h] = valid ? d[h] : -INFINITY;
        }
        uint32_t pk[HW / 2];
#pragma unroll
        for (int h = 0; h < HW; h += 2) {
          const float p0 = ex2(d[h]);
          const float p1 = ex2(d[h + 1]);
          lpart[h] += p0;
          lpart[h + 1] += p1;
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
          pk[h / 2] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        if (gu > 0) wait(B_PV, (gu - 1) & 1);
        if (resc) {
          tc_fence_after();
          if (u > 0) {  // O^T rows of this thread: dims 128c + key, 16 heads at a time
#pragma unroll 1
            for (int c = 0; c < 4 * (HW / 16); ++c) {
              const int hh = (c % (HW / 16)) * 16;
              const uint32_t col = C::TM_O + (c / (HW / 16)) * H + h0 + hh;
              float o[16];
              tmem_cols_load<16>(lane_base + col, o);
#pragma unroll
              for (int h = 0; h < 16; ++h) o[h] *= fac[h0 + hh + h];
              tmem_cols_store<16>(lane_base + col, o);
            }
            tmem_wait_st();
          }
        }
        if constexpr (C::P_MN) {  // P[key][h] = bf16(2^d), one 128-byte swizzled row per key
          uint8_t* prow = sm + C::OFF_P + key * 128;
#pragma unroll
          for (int qv = 0; qv < HW / 8; ++qv) {
            const int chunk = ((h0 >> 3) + qv) ^ (key & 7);
            *reinterpret_cast<uint4*>(prow + (chunk << 4)) =
                make_uint4(pk[4 * qv], pk[4 * qv + 1], pk[4 * qv + 2], pk[4 * qv + 3]);
          }
        } else {  // P^T[h][key]: K-major rows of 64 keys per head
          uint8_t* pbase = sm + C::OFF_P + (key >> 6) * C::PSUB;
          const int kb = (key & 63) * 2;
#pragma unroll
          for (int h = 0; h < HW; ++h) {
            const int hg = h0 + h;
            const int off = hg * 128 + ((((kb >> 4) ^ (hg & 7)) << 4) | (kb & 15));
            *reinterpret_cast<uint16_t*>(pbase + off) = static_cast<uint16_t>(pk[h / 2] >> (16 * (h & 1)));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P));
      }
      // ---- row sums over the 128 keys, then the token's output
      head_reduce<HW, 16, false>(lpart, lane);
      if (HW == 32 || (lane & 1) == 0) red[quarter * H + h0 + (HW == 32 ? lane : lane >> 1)] = lpart[0];
      named_bar_sync(1, NST);
      if (tid < H) {
        const float L = (red[tid] + red[H + tid]) + (red[2 * H + tid] + red[3 * H + tid]);
        if constexpr (NSPLIT == 1) {
          fac[tid] = L > 0.f ? kUnshift * (1.f / L) : 0.f;
          if (p.lse)
            p.lse[static_cast<int64_t>(toks[i].x) * H + tid] =
                L > 0.f ? (m_used[tid] + log2f(L)) * kLn2 : -INFINITY;
          m_used[tid] = -INFINITY;  // the next token's running maximum
        } else {
          lsum[tid] = L;
        }
      }
      named_bar_sync(1, NST);
      if (nb > 0) wait(B_PV, (gu - 1) & 1);
      const bool have = nb > 0 && alive;
      tc_fence_after();
      if constexpr (NSPLIT == 1) {
        if (!have) continue;
        // dims 128c + dl of this thread's heads: lanes 2m and 2m+1 hold neighbours
        // and swap one value of each head pair, so that each writes one head's two
        const bool odd = lane & 1;
        uint16_t* orow = p.out + static_cast<int64_t>(toks[i].x) * H * 512 + (dl & ~1);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float o[HW];
          tmem_cols_load<HW>(lane_base + C::TM_O + c * H + h0, o);
#pragma unroll
          for (int hp = 0; hp < HW / 2; ++hp) {
            const float mine = odd ? o[2 * hp + 1] : o[2 * hp];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? o[2 * hp] : o[2 * hp + 1], 1);
            const int h = h0 + 2 * hp + (odd ? 1 : 0);
            const float f = fac[h];
            const __nv_bfloat162 b2 = odd ? __floats2bfloat162_rn(other * f, mine * f)
                                          : __floats2bfloat162_rn(mine * f, other * f);
            *reinterpret_cast<uint32_t*>(orow + h * 512 + c * 128) = *reinterpret_cast<const uint32_t*>(&b2);
          }
        }
      } else {
        if (have) {  // (with the widening warps)
#pragma unroll 1
          for (int c = warp >> 2; c < 4 * NSW / 4; c += C::NOW) write_part(c);
        }
        float* Od = part_base();
        if (kMergeL2 && have && tid < H) {
          Od[H * 512 + tid] = m_used[tid];
          Od[H * 512 + H + tid] = lsum[tid];
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_O) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }

  // ---- combine the NSPLIT partial results of the cluster's token and write
  // bf16 out (+ lse)
  if constexpr (NSPLIT > 1) {
    float* Os = reinterpret_cast<float*>(sm + C::OFF_CODE);
    float* wfac = reinterpret_cast<float*>(sm + C::OFF_P);  // [NSPLIT][H], over P
    if (kMergeL2) __threadfence();
    cluster_sync();
    if (ntok > 0) {  // the same in every CTA of the cluster
      const int t = toks[0].x, nbt = (tok_nvalid(toks[0]) + 127) / 128;
      auto has = [&](int r) { return (r + 1) * nbt / NSPLIT > r * nbt / NSPLIT; };  // CTA r had blocks
      const float* part_t = p.part + static_cast<int64_t>(t) * NSPLIT * (H * 512 + 2 * H);
      auto part4 = [&](int r, int h, int d) -> float4 {
        if constexpr (kMergeL2)
          return __ldcg(reinterpret_cast<const float4*>(part_t + r * (H * 512 + 2 * H) + h * 512 + d));
        else
          return ld_dsmem_f4(mapa_shared(smem_u32(&Os[h * 512 + d]), r));
      };
      if (tid < H) {
        float mr[NSPLIT], lr[NSPLIT];
        float M = -INFINITY;
#pragma unroll
        for (int r = 0; r < NSPLIT; ++r) {
          mr[r] = -INFINITY;
          lr[r] = 0.f;
          if (has(r)) {
            if constexpr (kMergeL2) {
              const float* pr = part_t + r * (H * 512 + 2 * H) + H * 512;
              mr[r] = __ldcg(pr + tid);
              lr[r] = __ldcg(pr + H + tid);
            } else {
              mr[r] = __uint_as_float(ld_dsmem_u32(mapa_shared(smem_u32(&m_used[tid]), r)));
              lr[r] = __uint_as_float(ld_dsmem_u32(mapa_shared(smem_u32(&lsum[tid]), r)));
            }
          }
          M = fmaxf(M, mr[r]);
        }
        float L = 0.f;
#pragma unroll
        for (int r = 0; r < NSPLIT; ++r) L += (mr[r] == -INFINITY) ? 0.f : lr[r] * ex2(mr[r] - M);
#pragma unroll
        for (int r = 0; r < NSPLIT; ++r)
          wfac[r * H + tid] = (L > 0.f && mr[r] != -INFINITY) ? kUnshift * (ex2(mr[r] - M) / L) : 0.f;
        if (rank == 0 && p.lse)
          p.lse[static_cast<int64_t>(t) * H + tid] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
      }
      __syncthreads();
      // this rank's DS dims of every head, four at a time
      constexpr int DS = 512 / NSPLIT, ITEMS = H * DS / 4, R = NSPLIT < 4 ? NSPLIT : 4;
      for (int i = tid; i < ITEMS; i += NT) {
        const int h = i / (DS / 4), d = rank * DS + (i % (DS / 4)) * 4;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r0 = 0; r0 < NSPLIT; r0 += R) {
          float4 v[R];
#pragma unroll
          for (int r = 0; r < R; ++r) v[r] = has(r0 + r) ? part4(r0 + r, h, d) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float f = wfac[(r0 + r) * H + h];
            acc.x = fmaf(f, v[r].x, acc.x);
            acc.y = fmaf(f, v[r].y, acc.y);
            acc.z = fmaf(f, v[r].z, acc.z);
            acc.w = fmaf(f, v[r].w, acc.w);
          }
        }
        __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x, acc.y);
        __nv_bfloat162 hi2 = __floats2bfloat162_rn(acc.z, acc.w);
        uint2 pk;
        pk.x = *reinterpret_cast<uint32_t*>(&lo2);
        pk.y = *reinterpret_cast<uint32_t*>(&hi2);
        *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(t) * H + h) * 512 + d) = pk;
      }
    }
    if (!kMergeL2) cluster_sync();  // this CTA's shared memory stays until every rank has read it
  }
}

template <int H, int NSPLIT, bool PAGED, bool SHORT = false>
cudaError_t launch_one(const CUtensorMap& ql, const CUtensorMap& qr, const Int4Params& p, int grid,
                       cudaStream_t stream) {
  using C = Int4Cfg<H>;
  auto* kern = sparse_mla_int4_kernel<H, NSPLIT, PAGED, SHORT>;
  static std::atomic<uint64_t> configured{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(configured.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e == cudaSuccess && NSPLIT > 8)  // 16 CTAs per cluster: beyond the portable size
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    configured.fetch_or(bit, std::memory_order_release);
  }
  prof_begin(stream);
  e = launch_chained(kern, dim3(static_cast<unsigned>(grid)), dim3(C::NT), C::SMEM, stream, NSPLIT, ql, qr, p);
  prof_end(kLaunchMla, stream);
  count_launch(kLaunchMla);
  return e;
}

template <int H, bool PAGED>
cudaError_t launch_split(int nsplit, const CUtensorMap& ql, const CUtensorMap& qr, const Int4Params& p,
                         int grid, cudaStream_t stream) {
  switch (nsplit) {
    case 1:  // (a list of one block is never split)
      return p.K <= 64 ? launch_one<H, 1, PAGED, true>(ql, qr, p, grid, stream)
                       : launch_one<H, 1, PAGED>(ql, qr, p, grid, stream);
    case 2: return launch_one<H, 2, PAGED>(ql, qr, p, grid, stream);
    case 4: return launch_one<H, 4, PAGED>(ql, qr, p, grid, stream);
    case 8: return launch_one<H, 8, PAGED>(ql, qr, p, grid, stream);
    default: return launch_one<H, 16, PAGED>(ql, qr, p, grid, stream);
  }
}

// CTAs per token: as mla_nsplit, but no more than cover the blocks that a token
// of this batch can have.
int int4_nsplit(const dsa_batch_t& b, int k) {
  int nsplit = mla_nsplit(b, k);
  const int nblk = (std::min(k, b.max_len) + 127) / 128;
  while (nsplit > 1 && nsplit / 2 >= nblk) nsplit /= 2;
  return nsplit;
}

}  // namespace

cudaError_t launch_sparse_mla_int4(const void* q_lat, const void* q_rope, const void* kv,
                                   int64_t kv_rows, const int32_t* idx, int k, int heads, float scale,
                                   const dsa_batch_t& b, void* out, float* lse, void* ws,
                                   size_t ws_bytes, int* status, cudaStream_t stream,
                                   bool direct_rows) {
  if (b.num_q == 0) return cudaSuccess;
  CUtensorMap ql, qr;
  const uint64_t qrows = static_cast<uint64_t>(b.num_q) * heads;
  if (!make_tmap_2d(&ql, q_lat, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 512, qrows, 64, heads) ||
      !make_tmap_2d(&qr, q_rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, 64, qrows, 64, heads))
    return cudaErrorInvalidValue;
  Int4Params p{};
  p.b = to_args(b);
  p.kv = static_cast<const uint8_t*>(kv);
  p.kv_rows = kv_rows;
  p.direct = direct_rows ? 1 : 0;
  p.idx = idx;
  p.K = k;
  p.scale_log2 = scale * kLog2e;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status;
  p.timeout_ns = wait_timeout_ns();
  const int64_t items = static_cast<int64_t>(b.max_q) * b.num_seqs;
  // no more CTAs a token than it can have blocks
  const int nsplit = int4_nsplit(b, k);
  if (nsplit >= 4) {  // the partial results go through the workspace
    if (!ws || ws_bytes < mla_workspace_bytes(b, heads, k)) return cudaErrorInvalidValue;
    p.part = static_cast<float*>(ws);
  }
  int64_t grid = items * nsplit;  // a cluster per token
  if (nsplit == 1) {              // one CTA per SM, or more where a list would not hold its tokens
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    grid = std::max<int64_t>(std::min<int64_t>(items, sms), (items + kListMax - 1) / kListMax);
  }
  const bool paged = b.block_table != nullptr && !direct_rows;
  const int g = static_cast<int>(grid);
  if (heads == 16)
    return paged ? launch_split<16, true>(nsplit, ql, qr, p, g, stream)
                 : launch_split<16, false>(nsplit, ql, qr, p, g, stream);
  if (heads == 32)
    return paged ? launch_split<32, true>(nsplit, ql, qr, p, g, stream)
                 : launch_split<32, false>(nsplit, ql, qr, p, g, stream);
  return paged ? launch_split<64, true>(nsplit, ql, qr, p, g, stream)
               : launch_split<64, false>(nsplit, ql, qr, p, g, stream);
}

}  // namespace dsa
