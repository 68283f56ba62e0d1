// The text model's 8-bit key / value cache: blocks of block_tokens tokens of one
// sequence, per kv head the codes of K [block_tokens, D] and of V transposed [D,
// block_tokens], and one float32 scale each. Two operators: new tokens enter it,
// and the attention of one query token per sequence reads it.
#include <cuda_fp16.h>

#include <algorithm>

#include "int8_code.cuh"
#include "internal.cuh"
#include "sm100.cuh"
#include "softmax.cuh"

namespace h3 {
namespace {

// The block a table names, or -1 (and the error word set) if there is none.
__device__ __forceinline__ int block_of(const int32_t* table, int width, int seq, int page,
                                        int n_blocks, int* err) {
  const int b = table[(size_t)seq * width + page];
  if (b >= 0 && b < n_blocks) return b;
  atomicExch(err, H3_DEVERR_LAYOUT);
  return -1;
}

// ------------------------------------------------------------- store
// A thread block per (sequence, cache block touched, kv head): the block's new
// values of K and V are read once into registers, their maxima set the scales,
// and the codes are written. Where the block holds earlier tokens and a scale
// grows, their codes are rounded again under the new one. HBM-bound for prompts
// (2 bytes in, 1 out per value), launch-bound for single tokens. A thread holds
// eight channels of four neighbouring slots, so that V's codes turn in
// registers to words of four tokens; these pass through shared memory (with the
// word's place XORed by the channel, against bank conflicts), so that global
// stores run along the tokens. Where most pairs of a sequence and a block up to
// max_new would be empty, a thread block finds its pair by a scan over the
// sequences. 18400 tokens of 8 heads x 128 in 16 sequences (113 MB in and out):
// 29.0 us (34 without the scan), six waves of one chain each (sequence, values, scale,
// codes); two thread blocks per SM 37 us, four, whose registers spill, 35 us. One
// token of each of 48 sequences: 4.5 us.
// As many threads as a block has groups of four slots and eight channels (with 256
// for all, 36000 tokens of 8 heads x 64, 32 per block: 73 us against 27).
template <int D, int BT>
constexpr int kStoreThreads = BT * D / 32 < 256 ? BT * D / 32 : 256;

struct StoreArgs {
  const int32_t *table, *lengths, *offsets;
  const uint16_t* x[2];  // k, v
  int64_t stride[2];
  uint8_t* codes[2];
  float* scales[2];
  int n_blocks, kv_heads, width, max_new, rows, n_seq, pages;
  bool search;
  int* err;
};

// The new tokens of a sequence and the cache blocks they touch.
struct Arrival {
  int before, first, count;
};

// False for lengths or offsets that make no sense: nothing of the sequence is stored.
template <int BT>
__device__ __forceinline__ bool arrival(const StoreArgs& a, int seq, Arrival& r) {
  r.before = a.lengths[seq];
  r.first = a.offsets[seq];
  r.count = a.offsets[seq + 1] - r.first;
  return r.count == 0 ||
         !(r.before < 0 || r.first < 0 || r.count < 0 || r.count > a.max_new ||
           r.first > a.rows - r.count || (long long)r.before + r.count > (long long)a.width * BT);
}

template <int BT>
__device__ __forceinline__ int blocks_touched(const Arrival& r) {
  return r.count == 0 ? 0 : (r.before + r.count - 1) / BT - r.before / BT + 1;
}

// The unit-th cache block of all that the sequences touch, in their order: a scan
// over the sequences by the thread block. False past the last.
template <int BT, int THREADS>
__device__ __forceinline__ bool find_unit(const StoreArgs& a, int unit, int* sums, int* found,
                                          Arrival* which) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int each = (a.n_seq + THREADS - 1) / THREADS;
  const int begin = min(t * each, a.n_seq), end = min(begin + each, a.n_seq);
  int mine = 0;
  for (int s = begin; s < end; ++s) {
    Arrival r;
    if (arrival<BT>(a, s, r)) mine += blocks_touched<BT>(r);
    else if (blockIdx.x == 0) atomicExch(a.err, H3_DEVERR_LAYOUT);
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) sums[warp] = upto;
  if (t == 0) found[0] = -1;
  __syncthreads();
  for (int w = 0; w < warp; ++w) upto += sums[w];
  int at = upto - mine;
  if (unit >= at && unit < upto)
    for (int s = begin; s < end; ++s) {
      Arrival r;
      const int n = arrival<BT>(a, s, r) ? blocks_touched<BT>(r) : 0;
      if (unit < at + n) {
        found[0] = s;
        found[1] = unit - at;
        *which = r;
        break;
      }
      at += n;
    }
  __syncthreads();
  return found[0] >= 0;
}

// Scale of a block and kv head, and what happens to its codes.
struct BlockScale {
  RowScale s;
  float old;
  bool zero;   // every code is 0
  bool again;  // earlier codes change
};

template <h3_type T>
__device__ __forceinline__ BlockScale block_scale(float peak, float old, bool held,
                                                  float* stored, bool writer) {
  BlockScale b;
  float scale = max_nan(peak / 127.f, old);
  // an infinity or a NaN marks the whole block: scale NaN, codes 0
  const bool bad = !(peak <= kMaxFinite) || !(old <= kMaxFinite);
  if (bad) scale = __int_as_float(0x7fc00000);
  if (writer) *stored = scale;
  b.old = old;
  b.zero = bad || scale == 0.f;
  b.s = row_scale<T>(b.zero ? 1.f : scale);
  b.again = held && (bad || scale > old);
  return b;
}

__device__ __forceinline__ uint32_t word_again(uint32_t x, const BlockScale& b) {
  if (b.zero) return 0;
  const float ratio = b.old * b.s.inv;
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = code_again((int)(int8_t)(x >> (8 * k)), b.old, b.s.scale, ratio);
  return pack4(c[0], c[1], c[2], c[3]);
}

template <h3_type T>
__device__ __forceinline__ uint2 vec_codes(const uint4& u, const BlockScale& b) {
  float f[8];
  unpack<T>(u, f);
  return codes_of_8(f, b.s);
}

template <h3_type T, int D, int BT>
__device__ __forceinline__ void store_block(const StoreArgs& a, int seq, int nth, int head,
                                            const Arrival& r, uint32_t* turned,
                                            float (*part)[kStoreThreads<D, BT> / 32]) {
  constexpr int THREADS = kStoreThreads<D, BT>;
  constexpr int RV = D / 8;                 // 16-byte vectors per token
  constexpr int WR = BT / 4;                // words of four slots per channel
  constexpr int GROUPS = WR * RV;           // (word, vector) pairs
  constexpr int NG = (GROUPS + THREADS - 1) / THREADS;
  const int t = threadIdx.x;
  if (nth >= blocks_touched<BT>(r)) return;
  const int before = r.before, first = r.first, count = r.count;
  const int page = before / BT + nth;
  const int lo = max(before, page * BT), hi = min(before + count, (page + 1) * BT);
  const int held = nth == 0 ? before % BT : 0;  // earlier tokens of the block
  const int slot0 = lo - page * BT, to = hi - page * BT;
  const bool whole = slot0 == 0 && to == BT;

  // the thread's groups: four slots from 4 word on, eight channels from 8 vec on
  const int vec = t % RV, word0 = t / RV;
  constexpr int WORDS = THREADS / RV;  // word step between a thread's groups
  uint4 u[2][NG][4];
  const long long row0 = (long long)first + page * BT - before;  // row of slot 0
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint16_t* x = a.x[w] + (row0 + 4 * word0) * a.stride[w] + head * D + vec * 8;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int slot = 4 * (word0 + i * WORDS) + j;
        u[w][i][j] = make_uint4(0, 0, 0, 0);
        if (slot >= slot0 && slot < to)
          u[w][i][j] = __ldcs(
              reinterpret_cast<const uint4*>(x + (4 * i * WORDS + j) * a.stride[w]));
      }
  }
  const int block = block_of(a.table, a.width, seq, page, a.n_blocks, a.err);
  if (block < 0) return;
  const size_t at = (size_t)block * a.kv_heads + head;
  float old[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) old[w] = held > 0 ? a.scales[w][at] : 0.f;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    AbsMax<T> peak;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) peak.add(u[w][i][j]);
    const float m = warp_peak(peak.value());
    if ((t & 31) == 0) part[w][t >> 5] = m;
  }
  __syncthreads();  // also: every thread has read the old scales
  BlockScale bs[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float m = warp_peak(part[w][t % (THREADS / 32)]);
    bs[w] = block_scale<T>(m, old[w], held > 0, a.scales[w] + at, t == 0);
  }
  uint8_t* kc = a.codes[0] + at * (BT * D);
  uint8_t* vc = a.codes[1] + at * (BT * D);

#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int word = word0 + i * WORDS;
    if (word >= WR || 4 * word + 4 <= slot0 || 4 * word >= to) continue;
    uint8_t* k = kc + 4 * word * D + vec * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint2 c = vec_codes<T>(u[0][i][j], bs[0]);
      if (bs[0].zero) c = make_uint2(0, 0);
      const int slot = 4 * word + j;
      if (whole || (slot >= slot0 && slot < to)) *reinterpret_cast<uint2*>(k + j * D) = c;
    }
    // two channels of the four slots at a time, in the order of the words
    uint32_t* dst = turned + vec * 8 * WR + (word ^ (vec & (WR - 1)));
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4& x = u[1][i][j];
        unpack_pair<T>(h == 0 ? x.x : h == 1 ? x.y : h == 2 ? x.z : x.w, f[j], f[4 + j]);
      }
      const uint2 c = codes_of_8(f, bs[1].s);
      dst[2 * h * WR] = c.x;
      dst[(2 * h + 1) * WR] = c.y;
    }
  }
  if (bs[0].again)
    for (int i = t; i < held * D / 4; i += THREADS) {
      uint32_t* p = reinterpret_cast<uint32_t*>(kc) + i;
      *p = word_again(*p, bs[0]);
    }
  __syncthreads();
  const bool zero = bs[1].zero;
  if (whole) {
#pragma unroll
    for (int i = 0; i < D * WR / 4; i += THREADS) {
      const int d = (i + t) / (WR / 4), q = (i + t) % (WR / 4) * 4;
      if (D * WR / 4 % THREADS != 0 && i + t >= D * WR / 4) break;
      const uint32_t* row = turned + d * WR;
      const int f = (d / 8) & (WR - 1);
      uint4 c = make_uint4(row[q ^ f], row[(q + 1) ^ f], row[(q + 2) ^ f], row[(q + 3) ^ f]);
      if (zero) c = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(vc + d * BT + 4 * q) = c;
    }
    return;
  }
  const bool again = bs[1].again;
  const int w0 = (again ? 0 : slot0) / 4, words = (to + 3) / 4 - w0;
  for (int i = t; i < D * words; i += THREADS) {
    const int d = i % D, word = w0 + i / D;
    uint32_t c = turned[d * WR + (word ^ ((d / 8) & (WR - 1)))];
    if (zero) c = 0;
    uint8_t* p = vc + d * BT + 4 * word;
    if (4 * word >= slot0 && 4 * word + 4 <= to) {
      *reinterpret_cast<uint32_t*>(p) = c;
      continue;
    }
    // the word also holds earlier or later tokens
    const uint32_t early =
        again && 4 * word < slot0 ? word_again(*reinterpret_cast<uint32_t*>(p), bs[1]) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int slot = 4 * word + k;
      if (slot >= slot0 && slot < to) p[k] = (uint8_t)(c >> (8 * k));
      else if (again && slot < slot0) p[k] = (uint8_t)(early >> (8 * k));
    }
  }
}

template <h3_type T, int D, int BT>
__global__ void __launch_bounds__(kStoreThreads<D, BT>,
                                  (BT * D >= 16384 ? 512 : 768) / kStoreThreads<D, BT>)
    k_kv_store(const StoreArgs a) {
  constexpr int THREADS = kStoreThreads<D, BT>;
  __shared__ uint32_t turned[D * BT / 4];
  __shared__ float part[2][THREADS / 32];
  __shared__ int sums[THREADS / 32], found[2];
  __shared__ Arrival which;
  const int head = blockIdx.x % a.kv_heads;
  const int unit = blockIdx.x / a.kv_heads;
  int seq, nth;
  Arrival r;
  if (a.search) {
    if (!find_unit<BT, THREADS>(a, unit, sums, found, &which)) return;
    seq = found[0];
    nth = found[1];
    r = which;
  } else {
    seq = unit / a.pages;
    nth = unit % a.pages;
    if (!arrival<BT>(a, seq, r)) {
      if (threadIdx.x == 0) atomicExch(a.err, H3_DEVERR_LAYOUT);
      return;
    }
    if (r.count == 0) return;
  }
  store_block<T, D, BT>(a, seq, nth, head, r, turned, part);
}

// ------------------------------------------------------------- attention
// o[s, h] = softmax_j(scale q[s, h] . k[j]) v[j] over the sequence's cached
// tokens. Bound by the bytes of the cache (2 D per token and kv head), so the
// query heads of a group share one pass over it, eight at a time: the columns of an
// MMA. (16 at a time halve the bytes of larger groups, but double a thread's
// registers and work per byte: 24 sequences of 6000 tokens, 24 heads over 1 x 128,
// 45 us against 24.)
//
// The work is the list of all (sequence, head group, cache block) units in that
// order, cut into equal ranges, one per thread block, as many as run at once:
// lengths may differ as they like, every thread block streams the same number
// of bytes, and its ring of stages runs on from one sequence to the next. A pair
// (sequence, head group) counts kPairUnits more than it has, since beginning and
// ending one costs a thread block about as much as three units (40 sequences of
// 500 to 24000 tokens, 40 over 8 heads: the last thread block ends after 84 us
// without this, most after 66). A pair that lies in one range is finished there;
// the parts of one that is cut go to the workspace and a second kernel joins
// them. At most the first and the last pair of a range are cut, so the workspace
// does not grow with the sequences.
//
// A thread block has one producer warp, which streams cache blocks into shared-
// memory stages with bulk copies, and four consumer warps in teams of two (or one)
// that take the stages in turn, a team's warps half the tokens each, every warp with its
// own running maximum, sum and accumulator (joined at the end of a segment), so
// that nothing waits but on its data.
//
// Both products have the tokens or channels on the 16-row side of the MMA and
// the query heads on the 8-column side, eight heads per column tile. (This form
// takes its operands from registers as the codes lie in shared memory; the kernel
// is bound by bytes and then by the instructions per byte, not by the tensor
// rate.) Scores: s^T = K q^T on 8-bit integers (m16n8k32), q as two 8-bit limbs of
// a 16-bit fixed-point row (an error of at most half of its largest element's
// 32512th, 2^-15.98 of that element), the sums exact. Values: o^T += V^T w^T on fp16 (m16n8k16), where the
// codes become fp16 exactly and the weights are fp16, times 2^15 so that they
// stay normal numbers down to 2^-29 of the largest, and times the block's V scale
// over the largest one met so far, so that the sums of all blocks share one
// accumulator. The K scale is applied to the scores in float32. A thread reads
// 16-byte pieces of a K row as four k-quads, since the order of the channels in a
// product is free, and the tokens are assigned to rows so that its V operand is
// one contiguous piece of a transposed V row; the weights turn between the two
// layouts by 8 x 8 transposes across the warp. 40 sequences of 500 to 24000 tokens,
// 40 heads over 8 x 128 (423 MB): 75 us, 5.6 TB/s; one of 4001 tokens: 10.9 us.
constexpr int kAttnThreads = 160, kConsumers = 4;
constexpr int kRows = 8;        // query heads that share a pass over the cache
constexpr int kListSize = 64;   // entries of the producer's list, two batches of 32
constexpr int kMinUnits = 2;    // cache blocks a range has at least, but for whole pairs
constexpr int kPairUnits = 3;

template <int D, int BT>
struct Ring {
  static constexpr int BLOCK = BT * D;  // bytes of K (or V) codes
  // thread blocks per SM: three where the accumulators leave the registers for it
  static constexpr int PER_SM = BLOCK >= 16384 ? 2 : 3;
  static constexpr int FIT = (PER_SM == 2 ? 98304 : 65536) / (2 * BLOCK);
  // Warps that share a unit (small ones are a warp's alone: 48 sequences of 3000 tokens,
  // 40 heads over 8 x 64, 34 us against 36), and how many such teams there are.
  static constexpr int TEAM = BLOCK <= 4096 ? 1 : 2, TEAMS = kConsumers / TEAM;
  // A multiple of the teams, so that a stage always serves the same one: a warp that
  // waits for a stage's next fill has then seen its last one, and cannot take an older
  // phase of the same parity for the one it waits for.
  static constexpr int STAGES = FIT < 16 ? FIT / TEAMS * TEAMS : 16;
  static constexpr int PITCH = D + 4;   // floats; the accumulators' stores meet no bank twice
  static constexpr int SUMS = 2 * kRows * PITCH * 4;  // two warps' accumulators
  static constexpr int BYTES = STAGES * 2 * BLOCK + SUMS;
  static_assert(STAGES <= kListSize - 32, "a list entry outlives its stage");
  static_assert(SUMS % 128 == 0, "stage alignment");
};

#ifdef H3_FAULT_INJECTION
// Test-only build: the unit of every range whose copies are left out, so that the
// wait of the warps that take it runs out (none where negative).
static __device__ int g_fault_skip_unit = -1;
#endif

struct Entry {
  int block, page;
  float ks, vs;
};

struct AttnArgs {
  const int32_t *table, *lengths;
  const uint8_t *k_codes, *v_codes;
  const float *k_scales, *v_scales;
  const uint16_t* q;
  uint16_t* o;
  int64_t q_stride, o_stride;
  // workspace, per thread block: two parts (0: a pair begun earlier, 1: a pair
  // that goes on) of kRows rows of averages and of (maximum, sum of weights), and
  // which pair part 1 belongs to, with the number of its parts
  float* part;    // [blocks][2][kRows][D]
  float2* stat;   // [blocks][2][kRows]
  int4* cut;      // [blocks] {sequence, head group, parts, 0}
  int n_seq, n_blocks, kv_heads, group, row_groups, width;
  float scale_log2;
  bool f16;
  int* err;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements held two a thread, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Four int8 codes as two fp16 pairs: code + 128 in the mantissa of 1024 + x.
__device__ __forceinline__ void codes_to_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  c ^= 0x80808080u;
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  const uint32_t a = __byte_perm(c, 0x64646464u, 0x4140), b = __byte_perm(c, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The tokens of a sequence, limited to what its table can name.
__device__ __forceinline__ int length_of(const AttnArgs& a, int seq, int block_tokens) {
  const int len = a.lengths[seq];
  const long long most = (long long)a.width * block_tokens;
  if (len >= 0 && len <= most) return len;
  atomicExch(a.err, H3_DEVERR_LAYOUT);
  return len < 0 ? 0 : (int)most;
}

// Division of values that hardly ever need 64 bits (which take a hundred
// instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// 1 / l of a weights' sum (0 where there were no tokens), within 2^-22 of it.
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : __fdividef(1.f, l); }

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, 128;" ::: "memory");
}

// The same; true for all of them if x is for any.
__device__ __forceinline__ bool consumers_any(bool x) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(x ? 1u : 0u)
      : "memory");
  return any != 0;
}

template <int D, int BT>
__global__ void __launch_bounds__(kAttnThreads, Ring<D, BT>::PER_SM)
    k_cache_attention(const AttnArgs a) {
  using R = Ring<D, BT>;
  constexpr int PITCH = R::PITCH;
  constexpr int HT = BT / R::TEAM;  // tokens of a warp per cache block
  constexpr int NB = HT / 8;     // its blocks of eight tokens
  constexpr int NH = D / 64;     // 64-channel halves of a K row
  constexpr int ND = D / 16;     // 16-channel row tiles of the output
  // Weights are at most 2^15: normal numbers of fp16 down to 2^-29 of that, and with
  // the smaller V scale of a block still to 2^-21 where their sum comes from them.
  constexpr float kShift = 15.f, kSmallRatio = 1.f / 256;
  constexpr float kFixed = 32512.f;  // 127 * 256: the largest element of a q row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[R::STAGES], empty[R::STAGES];
  __shared__ Entry list[kListSize];
  __shared__ float2 stat[kConsumers][kRows];
  __shared__ long long warp_sum[kAttnThreads / 32];
  __shared__ int4 s_begin;       // the range's first unit: {sequence, head group, page, 0}
  __shared__ long long s_cut[2];  // its ends among all units
  __shared__ long long s_pair_at; // where its first pair begins in the weights
  __shared__ int s_abort;

  asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel may be set up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.kv_heads * a.row_groups, q_heads = a.kv_heads * a.group;

  // ---- this thread block's range of units: a scan over the sequences' lengths
  auto pages_of = [&](int s) { return (length_of(a, s, BT) + BT - 1) / BT; };
  constexpr int kCount = 40;  // cache blocks in the low bits, sequences that have any above
  const int per = (a.n_seq + kAttnThreads - 1) / kAttnThreads;
  const int seq0 = min(a.n_seq, (int)threadIdx.x * per), seq1 = min(a.n_seq, seq0 + per);
  long long mine = 0;
  for (int s = seq0; s < seq1; ++s) {
    const int n = pages_of(s);
    if (n > 0) mine += (1ll << kCount) + n;
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_sum[warp] = upto;
  if (warp == kConsumers) {
    if (lane < R::STAGES) {
      mbar_init(&full[lane], 2);   // the copies issued, the list entry written
      mbar_init(&empty[lane], R::TEAM);  // the warps of a team
    }
    if (lane == 0) s_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  before += upto - mine;  // of the sequences before seq0
  auto units_in = [&](long long sum) { return (sum & ((1ll << kCount) - 1)) * heads; };
  auto weight_of = [&](long long sum) {
    return units_in(sum) + (sum >> kCount) * kPairUnits * heads;
  };
  const long long units = units_in(total), weight = weight_of(total);
  long long ranges = max((units + kMinUnits - 1) / kMinUnits, (total >> kCount) * heads);
  if (ranges > gridDim.x) ranges = gridDim.x;
  const bool idle = (long long)blockIdx.x >= ranges;
  if (!idle) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long at = quotient(weight * (blockIdx.x + e), ranges);
      if (at == weight && threadIdx.x == 0) s_cut[e] = units;
      if (at < weight_of(before) || at >= weight_of(before + mine)) continue;
      // this thread's sequences hold the cut
      long long sum = before;
      for (int s = seq0;; ++s) {
        const int n = pages_of(s);
        if (n == 0) continue;
        const long long in = at - weight_of(sum);
        if (in < (long long)heads * (n + kPairUnits)) {
          const int h = (int)quotient(in, n + kPairUnits);
          const int p = max(0, (int)(in - (long long)h * (n + kPairUnits)) - kPairUnits);
          s_cut[e] = units_in(sum) + (long long)h * n + p;
          if (e == 0) {
            s_begin = make_int4(s, h, p, 0);
            s_pair_at = weight_of(sum) + (long long)h * (n + kPairUnits);
          }
          break;
        }
        sum += (1ll << kCount) + n;
      }
    }
  }
  // sequences with nothing cached get zeros
  for (int s = blockIdx.x; s < a.n_seq; s += gridDim.x)
    if (length_of(a, s, BT) == 0)
      for (int i = threadIdx.x; i < q_heads * D; i += kAttnThreads) a.o[s * a.o_stride + i] = 0;
  __syncthreads();
  const long long u0 = idle ? 0 : s_cut[0], u1 = idle ? 0 : s_cut[1];
  if (u0 == u1) {
    if (threadIdx.x == 0) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
    return;
  }
  int seq = s_begin.x, hg = s_begin.y, page = s_begin.z;
  int len = length_of(a, seq, BT), pages = (len + BT - 1) / BT;
  long long pair_at = s_pair_at;
  const int n_units = (int)(u1 - u0);  // at most 2^31: a range is a fraction of the pool
  // on to the next (sequence, head group)
  auto next_pair = [&]() {
    pair_at += pages + kPairUnits;
    page = 0;
    if (++hg < heads) return;
    hg = 0;
    do ++seq; while ((len = length_of(a, seq, BT)) == 0);
    pages = (len + BT - 1) / BT;
  };
  const WaitCtx wc{a.err, &s_abort};

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    int i = 0;       // units listed and issued
    int issued = 0;  // lane 0's count of the latter
    while (i < n_units && ok) {
      const int n = min(min(32, pages - page), n_units - i);
      const int kvh = hg / a.row_groups;
      auto issue = [&](int k, int block) {  // unit k's copies; nothing for no block
        const int s = k % R::STAGES;
#ifdef H3_FAULT_INJECTION
        if (k == *(volatile int*)&g_fault_skip_unit) return;
#endif
        if (block < 0) {
          mbar_arrive(&full[s]);
          return;
        }
        const size_t at = ((size_t)block * a.kv_heads + kvh) * R::BLOCK;
        uint8_t* dst = smem + R::SUMS + s * 2 * R::BLOCK;
        mbar_arrive_expect_tx(&full[s], 2 * R::BLOCK);
        bulk_load(dst, a.k_codes + at, R::BLOCK, &full[s]);
        bulk_load(dst + R::BLOCK, a.v_codes + at, R::BLOCK, &full[s]);
      };
      // the first units' copies go out before anything else is known of them
      const int early = i == 0 ? min(n, R::STAGES) : 0;
      if (lane < n) {
        const int b = block_of(a.table, a.width, seq, page + lane, a.n_blocks, a.err);
        if (lane < early) issue(lane, b);
        const size_t at = (size_t)max(b, 0) * a.kv_heads + kvh;
        list[(i + lane) % kListSize] = Entry{b, page + lane, b < 0 ? 0.f : a.k_scales[at],
                                             b < 0 ? 0.f : a.v_scales[at]};
      }
      __syncwarp();
      if (lane == 0) {
        for (int k = i; k < i + n; ++k) {
          const int s = k % R::STAGES;
          if (k >= i + early) {
            if (!mbar_wait(&empty[s], ((k / R::STAGES) & 1) ^ 1, wc)) {
              ok = false;
              break;
            }
            issue(k, list[k % kListSize].block);
          }
          mbar_arrive(&full[s]);  // the entry is written
          issued = k + 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      i += n;
      page += n;
      if (i < n_units && page == pages) next_pair();
    }
    // Copies land before the block retires, though the consumers may have given up
    // (else they have waited for every one, later than this).
    for (int j = max(0, issued - R::STAGES); lane == 0 && j < issued; ++j)
      mbar_land(&full[j % R::STAGES], (j / R::STAGES) & 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  const int team = warp / R::TEAM, half = warp % R::TEAM;
  float* sums = reinterpret_cast<float*>(smem);  // [2][kRows][PITCH]
  int unit = 0;
  bool have_cut = false;
  while (unit < n_units) {
    const int kvh = hg / a.row_groups, h0 = (hg - kvh * a.row_groups) * kRows;
    const int rows = min(kRows, a.group - h0), head0 = kvh * a.group + h0;
    const int n = min(pages - page, n_units - unit);  // this segment's units
    const bool begins = page == 0, ends = page + n == pages;
    // q rows -> 16-bit fixed point, two limbs. Column g is head g of the group's
    // part; the thread's channels are 64 h + 16 t + 0..15.
    uint32_t qh[NH][4], ql[NH][4];
    float mul[2];  // of heads 2 t, + 1
    {
      const bool there = g < rows;
      const uint16_t* q = a.q + seq * a.q_stride + (head0 + (there ? g : 0)) * D + 16 * t;
      float x[NH][16], m = 0.f;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          const uint4 u = *reinterpret_cast<const uint4*>(q + 64 * h + e);
          if (a.f16) unpack<H3_F16>(u, &x[h][e]);
          else unpack<H3_BF16>(u, &x[h][e]);
#pragma unroll
          for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(x[h][e + k]));
        }
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const bool fine = m <= kMaxFinite;
      float up = 1.f;
      if (m < 1e-30f) {  // so small that the fixed-point factor would overflow
        up = 0x1p100f;
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int e = 0; e < 16; ++e) x[h][e] *= up;
      }
      const float inv = there && fine && m > 0.f ? kFixed / (m * up) : 0.f;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int v = fine ? __float2int_rn(x[h][4 * w + k] * inv) : 0;
            hi[k] = (uint32_t)((v + 128) >> 8);
            lo[k] = (uint32_t)v;  // its low byte, signed, is v - 256 hi
          }
          qh[h][w] = pack4(hi[0], hi[1], hi[2], hi[3]);
          ql[h][w] = pack4(lo[0], lo[1], lo[2], lo[3]);
        }
      const float f = fine ? m * a.scale_log2 * (1.f / kFixed) : __int_as_float(0x7fc00000);
      mul[0] = __shfl_sync(0xffffffffu, f, 8 * t);
      mul[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
    // rows 16 d + g (+ 8) are channels, columns heads
    float acc[ND][4];
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = 0.f;
    float v_top = 0.f;  // the accumulator holds sums over V scale / v_top
    bool ok = true;
    // unit i belongs to team i % TEAMS
    for (int i = unit + ((team - unit) & (R::TEAMS - 1)); i < unit + n; i += R::TEAMS) {
      const int s = i % R::STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (i / R::STAGES) & 1, wc))) {
        ok = false;
        break;
      }
      const Entry en = list[i % kListSize];
      if (en.block < 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
        continue;
      }
      const uint8_t* kb = smem + R::SUMS + s * 2 * R::BLOCK;
      const uint8_t* vb = kb + R::BLOCK;
      // row r of block b is token HT / 4 * (r / 2) + 2 b + r % 2 of the half
      const uint8_t* krow = kb + (half * HT + (HT / 4) * (g >> 1) + (g & 1)) * D + 16 * t;
      float sc[NB / 2][4];
#pragma unroll
      for (int b = 0; b < NB / 2; ++b) {
        int hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint4 x = *reinterpret_cast<const uint4*>(krow + 4 * b * D + 64 * h);
          const uint4 y = *reinterpret_cast<const uint4*>(krow + (4 * b + 2) * D + 64 * h);
          const uint32_t k0[4] = {x.x, y.x, x.y, y.y}, k1[4] = {x.z, y.z, x.w, y.w};
          mma_s8(hi, k0, qh[h][0], qh[h][1]);
          mma_s8(lo, k0, ql[h][0], ql[h][1]);
          mma_s8(hi, k1, qh[h][2], qh[h][3]);
          mma_s8(lo, k1, ql[h][2], ql[h][3]);
        }
        // |sum| <= 128 * 127 * (256 * 127 + 128) < 2^31
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[b][e] = (float)(hi[e] * 256 + lo[e]);
      }
      // scores in log2 units; tokens behind the end
      const int base = en.page * BT + half * HT + (HT / 4) * (g >> 1) + (g & 1);
      const bool cut = (en.page + 1) * BT > len;
      const float f[2] = {mul[0] * en.ks, mul[1] * en.ks};
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < NB / 2; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[b][e] *= f[e & 1];
          if (cut && base + 4 * b + (e & 2) >= len) sc[b][e] = -INFINITY;
          mx[e & 1] = fmaxf(mx[e & 1], sc[b][e]);
        }
      bool grows = fabsf(en.vs) > v_top;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 4));
        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 8));
        mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 16));
        grows |= mx[k] > m_run[k];
      }
      if (__any_sync(0xffffffffu, grows)) {
        // a new largest V scale with some room, so that few follow
        const float top = fabsf(en.vs) > v_top ? 1.5f * fabsf(en.vs) : v_top;
        const float vf = top > v_top ? v_top / top : 1.f;
        v_top = top;
        float by[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float to = fmaxf(m_run[k], mx[k]);
          by[k] = to > m_run[k] ? exp2_mufu(m_run[k] - to) : 1.f;
          l_run[k] *= by[k];
          m_run[k] = to;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[d][e] *= by[e & 1] * vf;
      }
      // weights, turned so that a thread has head g's tokens 2 t, 2 t + 1 of a block
      const float ratio = en.vs == 0.f ? 0.f : en.vs / v_top;
      // so small a share of the largest V scale that weights leave fp16's normal
      // numbers: their sum is then taken from the unrounded ones
      const bool small = ratio < kSmallRatio;
      uint32_t pb[NB];
      float unrounded[2] = {0.f, 0.f}, sub[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)  // a head that has seen no token has maximum -inf: weights 0
        sub[k] = kShift - (m_run[k] == -INFINITY ? 0.f : m_run[k]);
#pragma unroll
      for (int b = 0; b < NB / 2; ++b) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = exp2_mufu(sc[b][e] + sub[e & 1]);
        if (small) {
#pragma unroll
          for (int e = 0; e < 4; ++e) unrounded[e & 1] += p[e];
        }
        pb[2 * b] = transpose8(pack_f16x2(p[0] * ratio, p[1] * ratio));
        pb[2 * b + 1] = transpose8(pack_f16x2(p[2] * ratio, p[3] * ratio));
      }
      // The weights' sum from the rounded weights, as one more row of values that are
      // all 1: what rounding moves in the sums it then moves in their divisor too.
      if (small) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float z = unrounded[k];
          z += __shfl_xor_sync(0xffffffffu, z, 4);
          z += __shfl_xor_sync(0xffffffffu, z, 8);
          z += __shfl_xor_sync(0xffffffffu, z, 16);
          l_run[k] += z;
        }
      } else {
        const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) mma_f16(sum, ones, pb[2 * k], pb[2 * k + 1]);
        const float back = 1.f / ratio;
#pragma unroll
        for (int k = 0; k < 2; ++k) l_run[k] = fmaf(sum[k], back, l_run[k]);
      }
      const uint8_t* vrow = vb + g * BT + half * HT + (HT / 4) * t;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        uint32_t w[2][NB / 2];  // rows g and g + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t* v = vrow + (16 * d + 8 * r) * BT;
          if constexpr (NB == 8) {
            const uint4 x = *reinterpret_cast<const uint4*>(v);
            w[r][0] = x.x, w[r][1] = x.y, w[r][2] = x.z, w[r][3] = x.w;
          } else {
            static_assert(NB == 4, "a warp takes 32 or 64 tokens of a cache block");
            const uint2 x = *reinterpret_cast<const uint2*>(v);
            w[r][0] = x.x, w[r][1] = x.y;
          }
        }
#pragma unroll
        for (int k = 0; k < NB / 2; ++k) {
          uint32_t va[4];
          codes_to_f16(w[0][k], va[0], va[2]);
          codes_to_f16(w[1][k], va[1], va[3]);
          mma_f16(acc[d], va, pb[2 * k], pb[2 * k + 1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    // ---- the segment's end: the warps' results become one
    if (g == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) stat[warp][2 * t + k] = make_float2(m_run[k], l_run[k]);
    }
    // A wait that ran out in one warp ends all four after this segment: one that went
    // on alone would wait at the next one's barriers for good.
    ok = !consumers_any(!ok);
    float m_all[2], l_all[2], by[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, stat[w][2 * t + k].x);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float2 ml = stat[w][2 * t + k];
        // a NaN sum has to survive: its maximum may be -inf
        l = fmaf(ml.y, ml.x == m ? 1.f : exp2_mufu(ml.x - m), l);
      }
      m_all[k] = m;
      l_all[k] = l;
      by[k] = (m_run[k] == m ? 1.f : exp2_mufu(m_run[k] - m)) * inverse(l);
    }
    // Divided by the weights' sum before the V scale comes in: an average of the
    // values is in float32's range wherever they are, a sum over the tokens may not be.
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = acc[d][e] * by[e & 1] * v_top;
    auto each = [&](auto&& what) {  // (value, its place in a [kRows][PITCH] array)
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          what(acc[d][e], (2 * t + (e & 1)) * PITCH + 16 * d + g + 4 * (e & 2));
    };
    if (warp >= 2) {
      float* to = sums + (warp - 2) * kRows * PITCH;
      each([&](float& x, int at) { to[at] = x; });
    }
    consumers_sync();
    if (warp < 2) {
      float* from = sums + warp * kRows * PITCH;
      each([&](float& x, int at) { x += from[at]; });
      if (warp == 1) each([&](float& x, int at) { from[at] = x; });  // where it has just read
    }
    consumers_sync();
    const bool whole = begins && ends;
    const size_t slot = ((size_t)blockIdx.x * 2 + (begins ? 1 : 0)) * kRows;
    if (warp == 0) {
      const float* from = sums + kRows * PITCH;
      each([&](float& x, int at) { sums[at] = x + from[at]; });
      if (!whole && g == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) a.stat[slot + 2 * t + k] = make_float2(m_all[k], l_all[k]);
      }
      if (!whole && begins) {
        // the range that holds the pair's end, and so the number of parts
        const long long end = pair_at + pages + kPairUnits;
        const int to = (int)quotient(end * ranges - 1, weight);
        if (lane == 0) a.cut[blockIdx.x] = make_int4(seq, hg, to - (int)blockIdx.x + 1, 0);
        have_cut = true;
      }
    }
    consumers_sync();
    // rows as they lie in memory
    if (whole) {
      for (int i = threadIdx.x; i < rows * (D / 8); i += 32 * kConsumers) {
        const int r = i / (D / 8), d = i % (D / 8) * 8;
        const float* x = sums + r * PITCH + d;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = a.f16 ? pack_f16x2(x[2 * k], x[2 * k + 1]) : pack_bf16x2(x[2 * k], x[2 * k + 1]);
        *reinterpret_cast<uint4*>(a.o + seq * a.o_stride + (head0 + r) * D + d) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      for (int i = threadIdx.x; i < rows * (D / 4); i += 32 * kConsumers) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        *reinterpret_cast<float4*>(a.part + (slot + r) * D + d) =
            *reinterpret_cast<const float4*>(sums + r * PITCH + d);
      }
    }
    unit += n;
    page += n;
    if (!ok) break;
    if (unit < n_units) next_pair();
  }
  if (threadIdx.x == 0 && !have_cut) a.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
}

// Joins the parts of the pairs that were cut: a thread block per range, for its
// last pair. A warp takes a row, its lanes side by side along the channels; where
// pairs are few, and so have many parts, eight warps share a row's parts and a
// thread block has one row (one sequence of 4001 tokens: 10.5 us against 12.5; 48 of
// 1000 tokens, eight rows per thread block: 27 us against 31). The first parts are
// fetched before it is known whether there is anything to join (they lie in the
// workspace anyway).
constexpr int kJoinWarps = 8;

template <int D, int SLICES>  // warps that share a row
__global__ void __launch_bounds__(32 * kJoinWarps) k_cache_join(const AttnArgs a) {
  constexpr int E = D / 32, kAhead = 8;  // channels of a lane
  struct alignas(4 * E) Piece {
    float x[E];
  };
  __shared__ Piece sums[SLICES > 1 ? SLICES : 1][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the ranges' kernel is complete
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp % SLICES;
  const int r = blockIdx.y * (kJoinWarps / SLICES) + warp / SLICES;
  const int4 cut = a.cut[blockIdx.x];
  // part 1 of its own range, part 0 of the following ones
  auto at = [&](int i) {
    const int range = min((int)blockIdx.x + i, (int)gridDim.x - 1);
    return ((size_t)range * 2 + (i == 0 ? 1 : 0)) * kRows + r;
  };
  auto part = [&](int i) { return *reinterpret_cast<const Piece*>(a.part + at(i) * D + E * lane); };
  Piece x[kAhead];
  float2 ml[kAhead];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    x[k] = part(slice + k * SLICES);
    ml[k] = a.stat[at(slice + k * SLICES)];
  }
  float2 own = a.stat[at(lane)];  // a lane's part, for the maximum and the weights' sum
  const int n = cut.z, kvh = cut.y / a.row_groups, h0 = (cut.y - kvh * a.row_groups) * kRows;
  if (n == 0 || h0 + r >= a.group) return;  // with shared rows: the whole thread block
#pragma unroll
  for (int k = 2; k < kAhead; ++k) {
    const int i = slice + k * SLICES;
    if (i < n) x[k] = part(i), ml[k] = a.stat[at(i)];
  }
  if (lane >= n) own = make_float2(-INFINITY, 0.f);
  float m = own.x, l = 0.f;
  for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, a.stat[at(i)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  auto weight = [&](const float2& part) {  // of a part's average
    return part.y * (part.x == m ? 1.f : exp2_mufu(part.x - m));
  };
  l = weight(own);
  for (int i = lane + 32; i < n; i += 32) l += weight(a.stat[at(i)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = inverse(l);
  Piece sum = {};
  for (int i0 = slice; i0 < n; i0 += kAhead * SLICES) {
    if (i0 > slice) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * SLICES;
        if (i < n) x[k] = part(i), ml[k] = a.stat[at(i)];
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (i0 + k * SLICES >= n) break;
      const float f = weight(ml[k]) * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) sum.x[e] = fmaf(x[k].x[e], f, sum.x[e]);
    }
  }
  if constexpr (SLICES > 1) {
    sums[slice][lane] = sum;
    __syncthreads();
    if (slice > 0) return;
#pragma unroll
    for (int i = 1; i < SLICES; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) sum.x[e] += sums[i][lane].x[e];
  }
  uint16_t* o = a.o + cut.x * a.o_stride + (kvh * a.group + h0 + r) * D + E * lane;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    reinterpret_cast<uint32_t*>(o)[e / 2] = a.f16
                                                ? pack_f16x2(sum.x[e], sum.x[e + 1])
                                                : pack_bf16x2(sum.x[e], sum.x[e + 1]);
}

// Thread blocks of an attention call: as many as run at once, at most one per
// kMinUnits units of tables that are full, or per pair of a sequence and heads.
template <int D, int BT>
int ranges_of(int n_seq, int heads, int width) {
  const long long units = (long long)n_seq * heads * width;
  const long long most = (long long)num_sms() * Ring<D, BT>::PER_SM;
  const long long pairs = width > 0 ? (long long)n_seq * heads : 0;
  const long long n = std::max((units + kMinUnits - 1) / kMinUnits, pairs);
  return (int)(n < most ? n : most);
}

template <int D, int BT>
size_t workspace_of(int n_seq, int heads, int width) {
  return (size_t)ranges_of<D, BT>(n_seq, heads, width) *
         (2 * kRows * (D * 4 + 8) + sizeof(int4));
}

template <int D, int BT>
cudaError_t run_attention(AttnArgs& a, void* ws, cudaStream_t st) {
  using R = Ring<D, BT>;
  cudaError_t e = cudaFuncSetAttribute(k_cache_attention<D, BT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, R::BYTES);
  if (e != cudaSuccess) return e;
  const int ranges = ranges_of<D, BT>(a.n_seq, a.kv_heads * a.row_groups, a.width);
  a.part = static_cast<float*>(ws);
  a.stat = reinterpret_cast<float2*>(a.part + (size_t)ranges * 2 * kRows * D);
  a.cut = reinterpret_cast<int4*>(a.stat + (size_t)ranges * 2 * kRows);
  k_cache_attention<D, BT><<<(unsigned)ranges, kAttnThreads, R::BYTES, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.width == 1) return cudaSuccess;  // pairs of one block: none is cut
  // launched while the ranges run, to wait for them on the GPU
  cudaLaunchConfig_t cfg = {};
  const bool many_parts = 8ll * a.n_seq * a.kv_heads * a.row_groups <= ranges;
  cfg.gridDim = dim3((unsigned)ranges, (unsigned)(!many_parts ? 1 : min(a.group, kRows)));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return many_parts ? cudaLaunchKernelEx(&cfg, k_cache_join<D, kJoinWarps>, a)
                    : cudaLaunchKernelEx(&cfg, k_cache_join<D, 1>, a);
}

// F<head_dim, block_tokens>(...) for a cache.
#define H3_BY_CACHE(F, c, ...)                                       \
  ((c).head_dim == 128 ? H3_BY_BLOCK(F, 128, c, __VA_ARGS__)         \
                       : H3_BY_BLOCK(F, 64, c, __VA_ARGS__))
#define H3_BY_BLOCK(F, D, c, ...)                                    \
  ((c).block_tokens == 32   ? F<D, 32>(__VA_ARGS__)                  \
   : (c).block_tokens == 64 ? F<D, 64>(__VA_ARGS__)                  \
                            : F<D, 128>(__VA_ARGS__))

template <h3_type T, int D>
cudaError_t run_store(StoreArgs a, int block_tokens, cudaStream_t st) {
  // Where the sequences bring very different numbers of tokens, most pairs of a
  // sequence and a block up to max_new would be empty: with as many rows as there
  // are, only rows / block_tokens + 2 n_seq of them can hold one.
  long long units = (long long)a.n_seq * a.pages;
  const long long most = a.rows / block_tokens + 2LL * a.n_seq;
  a.search = most < units;
  if (a.search) units = most;
  if (units * a.kv_heads > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(units * a.kv_heads);
  if (block_tokens == 32) k_kv_store<T, D, 32><<<grid, kStoreThreads<D, 32>, 0, st>>>(a);
  else if (block_tokens == 64) k_kv_store<T, D, 64><<<grid, kStoreThreads<D, 64>, 0, st>>>(a);
  else k_kv_store<T, D, 128><<<grid, kStoreThreads<D, 128>, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_cache_store(const h3_kv_cache& c, int n_seq, int max_new,
                                  const int32_t* table, int width, const int32_t* lengths,
                                  const int32_t* offsets, bool f16, int rows, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, int* err,
                                  cudaStream_t st) {
  StoreArgs a;
  a.table = table;
  a.lengths = lengths;
  a.offsets = offsets;
  a.x[0] = static_cast<const uint16_t*>(k);
  a.x[1] = static_cast<const uint16_t*>(v);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.codes[0] = static_cast<uint8_t*>(c.k_codes);
  a.codes[1] = static_cast<uint8_t*>(c.v_codes);
  a.scales[0] = c.k_scales;
  a.scales[1] = c.v_scales;
  a.n_blocks = c.n_blocks;
  a.kv_heads = c.kv_heads;
  a.width = width;
  a.max_new = max_new;
  a.rows = rows;
  a.n_seq = n_seq;
  // max_new tokens that begin anywhere inside a block (in 64 bits: INT_MAX
  // stands for no bound)
  a.pages = (int)std::min(((long long)max_new + c.block_tokens - 2) / c.block_tokens + 1,
                          (long long)width);
  a.err = err;
  if (c.head_dim == 128)
    return f16 ? run_store<H3_F16, 128>(a, c.block_tokens, st)
               : run_store<H3_BF16, 128>(a, c.block_tokens, st);
  return f16 ? run_store<H3_F16, 64>(a, c.block_tokens, st)
             : run_store<H3_BF16, 64>(a, c.block_tokens, st);
}

size_t cache_attention_workspace(const h3_kv_cache& c, int n_seq, int q_heads, int width) {
  const int heads = c.kv_heads * ((q_heads / c.kv_heads + kRows - 1) / kRows);
  return H3_BY_CACHE(workspace_of, c, n_seq, heads, width);
}

cudaError_t launch_cache_attention(const h3_kv_cache& c, int n_seq, int q_heads,
                                   const int32_t* table, int width, const int32_t* lengths,
                                   bool f16, const void* q, int64_t q_stride, float scale,
                                   void* o, int64_t o_stride, void* ws, int* err,
                                   cudaStream_t st) {
  AttnArgs a;
  a.table = table;
  a.lengths = lengths;
  a.k_codes = static_cast<const uint8_t*>(c.k_codes);
  a.v_codes = static_cast<const uint8_t*>(c.v_codes);
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.q_stride = q_stride;
  a.o_stride = o_stride;
  a.n_seq = n_seq;
  a.n_blocks = c.n_blocks;
  a.kv_heads = c.kv_heads;
  a.group = q_heads / c.kv_heads;
  a.row_groups = (a.group + kRows - 1) / kRows;
  a.width = width;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.f16 = f16;
  a.err = err;
  return H3_BY_CACHE(run_attention, c, a, ws, st);
}

}  // namespace h3

#ifdef H3_FAULT_INJECTION
// Test-only build: the unit whose copies cache attention leaves out (-1: none).
extern "C" __attribute__((visibility("default"))) int h3_test_cache_skip_unit(int unit) {
  return cudaMemcpyToSymbol(h3::g_fault_skip_unit, &unit, sizeof(int)) == cudaSuccess ? 0 : -1;
}
#endif
