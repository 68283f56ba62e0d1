// The text model's 8-bit key / value cache: blocks of block_tokens tokens of one
// sequence, per kv head the codes of K [block_tokens, D] and of V transposed [D,
// block_tokens], and one float32 scale each. Two operators: new tokens enter it,
// and the attention of one query token per sequence reads it.
#include <cuda_fp16.h>

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
// A thread block per (sequence, cache block touched, kv head, K or V): the
// block's new values are read once into registers, their maximum sets the
// scale, and the codes are written. Where the block holds earlier tokens and
// the scale grows, their codes are rounded again under the new scale. HBM-bound
// for prompts (2 bytes in, 1 out per value), launch-bound for single tokens.
// V's codes are turned through shared memory, so that global stores run along
// the tokens.
constexpr int kStoreThreads = 256;

struct StoreArgs {
  const int32_t *table, *lengths, *offsets;
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int n_blocks, kv_heads, width, max_new, rows, pages;
  int* err;
};

template <h3_type T, int D, int BT>
__global__ void __launch_bounds__(kStoreThreads) k_kv_store(const StoreArgs a) {
  constexpr int RV = D / 8;                                // 16-byte vectors per token
  constexpr int NV = (BT * RV + kStoreThreads - 1) / kStoreThreads;
  constexpr int PITCH = BT + 4;
  __shared__ __align__(16) uint8_t turned[D * PITCH];
  __shared__ float part[kStoreThreads / 32];
  int id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int head = id % a.kv_heads;
  id /= a.kv_heads;
  const int nth = id % a.pages, seq = id / a.pages;
  const int t = threadIdx.x;

  const int before = a.lengths[seq], first = a.offsets[seq];
  const int count = a.offsets[seq + 1] - first;
  if (count == 0) return;
  // lengths or offsets that make no sense: nothing of the sequence is stored
  if (before < 0 || first < 0 || count < 0 || count > a.max_new || first > a.rows - count ||
      (long long)before + count > (long long)a.width * BT) {
    if (t == 0) atomicExch(a.err, H3_DEVERR_LAYOUT);
    return;
  }
  const int page = before / BT + nth;
  const int lo = max(before, page * BT), hi = min(before + count, (page + 1) * BT);
  if (lo >= hi) return;
  const int block = block_of(a.table, a.width, seq, page, a.n_blocks, a.err);
  if (block < 0) return;
  const int held = nth == 0 ? before % BT : 0;             // earlier tokens of the block
  const int slot0 = lo - page * BT, n = hi - lo;

  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* x = (is_v ? a.v : a.k) + (first + lo - before) * stride + head * D;
  uint4 u[NV];
  AbsMax<T> peak;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int idx = t + i * kStoreThreads;
    if (idx < n * RV)
      u[i] = __ldcs(reinterpret_cast<const uint4*>(x + (idx / RV) * stride) + idx % RV);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (t + i * kStoreThreads < n * RV) peak.add(u[i]);
  float m = peak.value();
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((t & 31) == 0) part[t >> 5] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int w = 0; w < kStoreThreads / 32; ++w) m = max_nan(m, part[w]);

  const size_t at = (size_t)block * a.kv_heads + head;
  float* scales = is_v ? a.v_scales : a.k_scales;
  uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + at * (BT * D);
  const float old = held > 0 ? scales[at] : 0.f;
  float scale = max_nan(m / 127.f, old);
  // an infinity or a NaN marks the whole block: scale NaN, codes 0
  const bool bad = !(m <= kMaxFinite) || !(old <= kMaxFinite);
  if (bad) scale = __int_as_float(0x7fc00000);
  const bool zero = bad || scale == 0.f;
  const RowScale s = row_scale(zero ? 1.f : scale);
  const bool again = held > 0 && (bad || scale > old);      // earlier codes change
  const float ratio = old * s.inv;
  __syncthreads();  // every thread has read the old scale
  if (t == 0) scales[at] = scale;

  auto vec_codes = [&](const uint4& w) {
    float f[8];
    unpack<T>(w, f);
    if (zero) return make_uint2(0, 0);
    return codes_of(f, s);
  };
  auto word_again = [&](uint32_t w) {
    if (zero) return 0u;
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = code_again((int)(int8_t)(w >> (8 * k)), old, scale, ratio);
    return pack4(c[0], c[1], c[2], c[3]);
  };

  if (!is_v) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int idx = t + i * kStoreThreads;
      if (idx < n * RV) reinterpret_cast<uint2*>(codes)[slot0 * RV + idx] = vec_codes(u[i]);
    }
    if (again)
      for (int w = t; w < held * D / 4; w += kStoreThreads) {
        uint32_t* p = reinterpret_cast<uint32_t*>(codes) + w;
        *p = word_again(*p);
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int idx = t + i * kStoreThreads;
    if (idx < n * RV) {
      const uint2 c = vec_codes(u[i]);
      uint8_t* dst = turned + (idx % RV) * 8 * PITCH + slot0 + idx / RV;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        dst[k * PITCH] = (uint8_t)((k < 4 ? c.x : c.y) >> (8 * (k & 3)));
    }
  }
  __syncthreads();
  const int from = again ? 0 : slot0, to = slot0 + n;
  const int w0 = from / 4, words = (to + 3) / 4 - w0;
  for (int i = t; i < D * words; i += kStoreThreads) {
    const int d = i / words, w = w0 + i % words;
    uint32_t* p = reinterpret_cast<uint32_t*>(codes + d * BT) + w;
    uint32_t c = *reinterpret_cast<const uint32_t*>(turned + d * PITCH + 4 * w);
    if (4 * w < slot0 || 4 * w + 4 > to) {  // the word also holds earlier or later tokens
      const uint32_t was = *p;
      const uint32_t early = again ? word_again(was) : was;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int slot = 4 * w + k;
        const uint32_t mask = 0xffu << (8 * k);
        if (slot < slot0) c = (c & ~mask) | (early & mask);
        if (slot >= to) c = (c & ~mask) | (was & mask);
      }
    }
    *p = c;
  }
}

// ------------------------------------------------------------- attention
// o[s, h] = softmax_j(scale q[s, h] . k[j]) v[j] over the sequence's cached
// tokens. Bound by the bytes of the cache (2 D per token and kv head), so the
// query heads of a group (16 at a time) share one pass over it, and the tokens
// are split over thread blocks, whose partial results a second kernel joins.
//
// A block has one producer warp, which streams cache blocks into a ring of
// shared-memory stages with bulk copies, and four consumer warps: two pairs take
// the ring's entries in turn, the warps of a pair half the tokens each, every
// warp with its own running maximum, sum and accumulator (joined at the end), so
// nothing waits but on its data. The products run on m16n8k16 fp16 MMAs (the
// query heads fill the 16 rows; the kernel is bound by bytes, and this form
// takes its operands from registers, where the codes become fp16 exactly): the
// 16-byte pieces a thread reads of a K row serve as four k-steps, since the order
// of the channels inside a product is free, and the tokens are assigned to
// columns so that the weights' registers are the A operand of the second product
// and its V operand is one contiguous piece of a transposed V row.
//
// q enters fp16 times a power of two per row (exact but for elements below 2^-14
// of the row's largest); the K scale is applied to the scores, the V scale to
// each block's sum, both in float32. Weights are stored in fp16 times 2^10, so
// that they stay normal numbers down to 2^-24 of the largest.
constexpr int kAttnThreads = 160, kConsumers = 4;
constexpr int kRows = 16;
constexpr int kMaxChunk = 64;  // cache blocks per thread block
constexpr int kRingBytes = 96 * 1024;

template <int D, int BT>
struct Ring {
  static constexpr int BLOCK = BT * D;                   // bytes of K (or V) codes
  static constexpr int STAGES = kRingBytes / (2 * BLOCK) < 16 ? kRingBytes / (2 * BLOCK) : 16;
  static constexpr int BYTES = STAGES * 2 * BLOCK;
};

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
  float* part;     // [n_seq * q_heads * splits][D] sums
  float2* stat;    // [n_seq * q_heads * splits] maximum (log2 units), sum of weights
  int n_blocks, kv_heads, group, row_groups, width, splits, chunk;
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

__device__ __forceinline__ float act_to_float(uint16_t u, bool f16) {
  return f16 ? __half2float(__ushort_as_half(u)) : __uint_as_float((uint32_t)u << 16);
}
__device__ __forceinline__ uint16_t float_to_act(float v, bool f16) {
  return f16 ? __half_as_ushort(__float2half_rn(v))
             : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// The tokens of a sequence, limited to what its table can name.
__device__ __forceinline__ int length_of(const AttnArgs& a, int seq, int block_tokens) {
  const int len = a.lengths[seq];
  const long long most = (long long)a.width * block_tokens;
  if (len >= 0 && len <= most) return len;
  atomicExch(a.err, H3_DEVERR_LAYOUT);
  return len < 0 ? 0 : (int)most;
}

template <int D, int BT>
__global__ void __launch_bounds__(kAttnThreads, 2) k_cache_attention(const AttnArgs a) {
  using R = Ring<D, BT>;
  constexpr int HT = BT / 2;     // tokens of a warp per cache block
  constexpr int NJ = HT / 8;     // its 8-token column tiles
  constexpr int KM = D / 16;     // k-steps of the score product
  constexpr int ND = D / 8;      // 8-channel column tiles of the output
  constexpr float kShift = 10.f;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) __half qs[kRows * (D + 8)];
  __shared__ uint64_t full[R::STAGES], empty[R::STAGES];
  __shared__ Entry list[kMaxChunk];
  __shared__ float q_mul[kRows];
  __shared__ float2 stat[kConsumers][kRows];
  __shared__ int s_n;
  __shared__ int s_abort;
  static_assert(kConsumers * kRows * D * 4 <= R::BYTES, "the sums reuse the stages");

  asm volatile("griddepcontrol.launch_dependents;");  // the joining kernel may be set up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int id = blockIdx.x;
  const int heads = a.kv_heads * a.row_groups;
  const int hg = id % heads;
  id /= heads;
  const int split = id % a.splits, seq = id / a.splits;
  const int kvh = hg / a.row_groups, h0 = (hg % a.row_groups) * kRows;
  const int rows = min(kRows, a.group - h0), q_heads = a.kv_heads * a.group;
  const int head0 = kvh * a.group + h0;

  const int len = length_of(a, seq, BT);
  const int pages = (len + BT - 1) / BT;
  const int p0 = split * a.chunk, p1 = min(pages, p0 + a.chunk);
  const bool alone = pages <= a.chunk;  // this block's result is the result
  if (p0 >= p1) {
    if (split == 0)  // nothing cached: zeros
      for (int i = threadIdx.x; i < rows * D; i += kAttnThreads)
        a.o[seq * a.o_stride + (head0 + i / D) * D + i % D] = 0;
    return;
  }

  auto load = [&](int i, int block) {  // entry i of the list into its stage
    const int s = i % R::STAGES;
    const size_t at = ((size_t)block * a.kv_heads + kvh) * R::BLOCK;
    mbar_arrive_expect_tx(&full[s], 2 * R::BLOCK);
    bulk_load(smem + s * 2 * R::BLOCK, a.k_codes + at, R::BLOCK, &full[s]);
    bulk_load(smem + s * 2 * R::BLOCK + R::BLOCK, a.v_codes + at, R::BLOCK, &full[s]);
  };
  if (warp == kConsumers) {  // the cache blocks of this range, those that exist
    if (lane < R::STAGES) {
      mbar_init(&full[lane], 1);
      mbar_init(&empty[lane], 2);  // the two warps of a pair
    }
    if (lane == 0) s_abort = 0;
    fence_mbar_init();
    __syncwarp();
    int n = 0;
    for (int p = p0; p < p1; p += 32) {
      const int b = p + lane < p1
                        ? block_of(a.table, a.width, seq, p + lane, a.n_blocks, a.err) : -1;
      const uint32_t mask = __ballot_sync(0xffffffffu, b >= 0);
      if (b >= 0) {
        const int i = n + __popc(mask & ((1u << lane) - 1u));
        if (i < R::STAGES) load(i, b);  // the first ones go out at once
        const size_t at = (size_t)b * a.kv_heads + kvh;
        list[i] = Entry{b, p + lane, a.k_scales[at], a.v_scales[at]};
      }
      n += __popc(mask);
    }
    if (lane == 0) s_n = n;
  } else {
    // q rows -> fp16 times a power of two, through shared memory
    for (int r = warp; r < kRows; r += kConsumers) {
      float x[D / 32], m = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        x[e] = r < rows ? act_to_float(a.q[seq * a.q_stride + (head0 + r) * D + e * 32 + lane],
                                       a.f16) : 0.f;
        m = max_nan(m, fabsf(x[e]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      // 2^e with m 2^-e in [1, 2); rows of zeros and tiny rows as they are
      const uint32_t ex = min(max(__float_as_uint(m) & 0x7f800000u, 0x01000000u), 0x7e000000u);
      const float up = __uint_as_float(ex), down = __uint_as_float(0x7f000000u - ex);
      const bool fine = m <= kMaxFinite;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        qs[r * (D + 8) + e * 32 + lane] = __float2half_rn(fine ? x[e] * down : 0.f);
      if (lane == 0) q_mul[r] = fine ? up * a.scale_log2 : __int_as_float(0x7fc00000);
    }
  }
  __syncthreads();
  const int n = s_n;
  const WaitCtx wc{a.err, &s_abort};
  const int g = lane >> 2, t = lane & 3;
  uint32_t qa[KM][4];
  if (warp < kConsumers) {
#pragma unroll
    for (int m = 0; m < KM; ++m) {
      const int d = 64 * (m >> 2) + 16 * t + 4 * (m & 3);  // the thread's four channels
      const uint2 lo = *reinterpret_cast<const uint2*>(qs + g * (D + 8) + d);
      const uint2 hi = *reinterpret_cast<const uint2*>(qs + (g + 8) * (D + 8) + d);
      qa[m][0] = lo.x;
      qa[m][1] = hi.x;
      qa[m][2] = lo.y;
      qa[m][3] = hi.y;
    }
  }

  float acc[ND][4];
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  if (warp == kConsumers) {
    if (lane == 0) {
      int i = min(n, R::STAGES);
      bool ok = true;
      for (; i < n; ++i) {
        if (!mbar_wait(&empty[i % R::STAGES], ((i / R::STAGES) & 1) ^ 1, wc)) {
          ok = false;
          break;
        }
        load(i, list[i].block);
      }
      if (!ok)  // let issued copies land before the block retires
        for (int j = i > R::STAGES ? i - R::STAGES : 0; j < i; ++j)
          mbar_drain(&full[j % R::STAGES], (j / R::STAGES) & 1);
    }
  } else {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[d][e] = 0.f;
    const int half = warp & 1;
    const float mul0 = q_mul[g], mul1 = q_mul[g + 8];
    for (int i = warp >> 1; i < n; i += kConsumers / 2) {
      const int s = i % R::STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (i / R::STAGES) & 1, wc))) break;
      const Entry en = list[i];
      const uint8_t* kb = smem + s * 2 * R::BLOCK;
      const uint8_t* vb = kb + R::BLOCK;
      // column c of tile j is token HT / 4 * (c / 2) + 2 j + c % 2 of the half
      float sc[NJ][4];
      const uint8_t* krow = kb + (half * HT + (HT / 4) * (g >> 1) + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        constexpr int JB = NJ < 4 ? NJ : 4;  // independent products in flight
#pragma unroll
        for (int j0 = 0; j0 < NJ; j0 += JB) {
          uint32_t w[JB][4];
#pragma unroll
          for (int j = 0; j < JB; ++j) {
            const uint4 x = *reinterpret_cast<const uint4*>(krow + 2 * (j0 + j) * D + 64 * h);
            w[j][0] = x.x, w[j][1] = x.y, w[j][2] = x.z, w[j][3] = x.w;
          }
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < JB; ++j) {
              uint32_t b0, b1;
              codes_to_f16(w[j][m], b0, b1);
              mma_f16(sc[j0 + j], qa[4 * h + m], b0, b1);
            }
        }
      }
      const float f0 = mul0 * en.ks, f1 = mul1 * en.ks;
      const int base = en.page * BT + half * HT + (HT / 4) * t;  // the thread's first token
      float mx0 = -INFINITY, mx1 = -INFINITY;
      if ((en.page + 1) * BT > len) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[j][e] *= e < 2 ? f0 : f1;
            if (base + 2 * j + (e & 1) >= len) sc[j][e] = -INFINITY;
          }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[j][e] *= e < 2 ? f0 : f1;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        mx0 = max3(mx0, sc[j][0], sc[j][1]);
        mx1 = max3(mx1, sc[j][2], sc[j][3]);
      }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      if (__any_sync(0xffffffffu, mx0 > m_run[0] || mx1 > m_run[1])) {
        const float n0 = fmaxf(m_run[0], mx0), n1 = fmaxf(m_run[1], mx1);
        const float a0 = n0 > m_run[0] ? exp2_mufu(m_run[0] - n0) : 1.f;
        const float a1 = n1 > m_run[1] ? exp2_mufu(m_run[1] - n1) : 1.f;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          acc[d][0] *= a0;
          acc[d][1] *= a0;
          acc[d][2] *= a1;
          acc[d][3] *= a1;
        }
        l_run[0] *= a0;
        l_run[1] *= a1;
        m_run[0] = n0;
        m_run[1] = n1;
      }
      // a row that has seen no token yet has maximum -inf: its weights are 0
      const float s0 = kShift - (m_run[0] == -INFINITY ? 0.f : m_run[0]);
      const float s1 = kShift - (m_run[1] == -INFINITY ? 0.f : m_run[1]);
      uint32_t pa[NJ / 2][4];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float p0 = exp2_mufu(sc[j][0] + s0), p1 = exp2_mufu(sc[j][1] + s0);
        const float p2 = exp2_mufu(sc[j][2] + s1), p3 = exp2_mufu(sc[j][3] + s1);
        l_run[0] += p0 + p1;
        l_run[1] += p2 + p3;
        pa[j / 2][2 * (j & 1)] = pack_f16x2(p0, p1);
        pa[j / 2][2 * (j & 1) + 1] = pack_f16x2(p2, p3);
      }
      const uint8_t* vrow = vb + g * BT + half * HT + (HT / 4) * t;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        uint32_t w[NJ / 2];
        if constexpr (NJ == 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(vrow + 8 * d * BT);
          w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else if constexpr (NJ == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(vrow + 8 * d * BT);
          w[0] = x.x, w[1] = x.y;
        } else {
          w[0] = *reinterpret_cast<const uint32_t*>(vrow + 8 * d * BT);
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < NJ / 2; ++k) {
          uint32_t b0, b1;
          codes_to_f16(w[k], b0, b1);
          mma_f16(c, pa[k], b0, b1);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[d][e] = fmaf(en.vs, c[e], acc[d][e]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 1);
      l_run[r] += __shfl_xor_sync(0xffffffffu, l_run[r], 2);
    }
  }
  __syncthreads();  // every stage has been read
  float* sums = reinterpret_cast<float*>(smem);  // [consumer][16][D]
  if (warp < kConsumers) {
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      float* p = sums + (warp * kRows + g) * D + 8 * d + 2 * t;
      *reinterpret_cast<float2*>(p) = make_float2(acc[d][0], acc[d][1]);
      *reinterpret_cast<float2*>(p + 8 * D) = make_float2(acc[d][2], acc[d][3]);
    }
    if (t == 0) {
      stat[warp][g] = make_float2(m_run[0], l_run[0]);
      stat[warp][g + 8] = make_float2(m_run[1], l_run[1]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * D; i += kAttnThreads) {
    const int r = i / D, d = i % D;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) m = fmaxf(m, stat[w][r].x);
    float sum = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kConsumers; ++w) {
      const float2 ml = stat[w][r];
      // a NaN sum has to survive: its maximum may be -inf
      const float f = ml.x == m ? 1.f : exp2_mufu(ml.x - m);
      sum = fmaf(sums[(w * kRows + r) * D + d], f, sum);
      l = fmaf(ml.y, f, l);
    }
    if (alone) {
      a.o[seq * a.o_stride + (head0 + r) * D + d] =
          float_to_act(l == 0.f ? 0.f : sum / l, a.f16);
    } else {
      const size_t at = ((size_t)seq * q_heads + head0 + r) * a.splits + split;
      a.part[at * D + d] = sum;
      if (d == 0) a.stat[at] = make_float2(m, l);
    }
  }
}

// Joins the ranges of the sequences that had more than one: a block per
// (sequence, head), kJoinParts threads per channel, each taking every
// kJoinParts-th range, so that the partial sums are fetched side by side.
constexpr int kJoinParts = 4, kJoinTile = 128;

template <int D, int BT>
__global__ void __launch_bounds__(D * kJoinParts) k_cache_join(const AttnArgs a) {
  __shared__ float factor[kJoinTile];
  __shared__ float sums[kJoinParts][D], weights[kJoinParts];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the ranges' kernel is complete
  const int q_heads = a.kv_heads * a.group;
  const int seq = blockIdx.x / q_heads, head = blockIdx.x - seq * q_heads;
  const int d = threadIdx.x % D, p = threadIdx.x / D, lane = threadIdx.x & 31;
  const long long most = (long long)a.width * BT;
  const int len = (int)min((long long)max(a.lengths[seq], 0), most);
  const int n = ((len + BT - 1) / BT + a.chunk - 1) / a.chunk;
  if (n <= 1) return;
  const size_t at = (size_t)blockIdx.x * a.splits;
  float m = -INFINITY;  // every warp for itself
  for (int i = lane; i < n; i += 32) m = fmaxf(m, a.stat[at + i].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float sum = 0.f, l = 0.f;
  for (int i0 = 0; i0 < n; i0 += kJoinTile) {
    const int k = min(kJoinTile, n - i0);
    __syncthreads();
    if (threadIdx.x < k) {
      const float2 ml = a.stat[at + i0 + threadIdx.x];
      const float f = ml.x == m ? 1.f : exp2_mufu(ml.x - m);
      factor[threadIdx.x] = f;
      l = fmaf(ml.y, f, l);
    }
    __syncthreads();
    const float* part = a.part + (at + i0) * D + d;
#pragma unroll 8
    for (int i = p; i < k; i += kJoinParts) sum = fmaf(part[(size_t)i * D], factor[i], sum);
  }
  sums[p][d] = sum;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // the threads that held a weight are the first kJoinTile = 4 warps
  if (lane == 0 && threadIdx.x < kJoinTile) weights[threadIdx.x / 32] = l;
  __syncthreads();
  if (p == 0) {
    float total = 0.f, w = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinParts; ++i) total += sums[i][d];
#pragma unroll
    for (int i = 0; i < kJoinTile / 32; ++i) w += weights[i];
    a.o[seq * a.o_stride + head * D + d] = float_to_act(w == 0.f ? 0.f : total / w, a.f16);
  }
}

// How the tokens are split: cache blocks per thread block, such that two thread
// blocks per SM exist when every sequence is as long as its table, at most
// kMaxChunk; and the number of ranges that gives.
void split_of(int n_seq, int heads, int width, int& chunk, int& splits) {
  const long long units = (long long)n_seq * heads * width;
  const long long at_once = 2 * num_sms();
  long long c = (units + at_once - 1) / at_once;
  if (c > kMaxChunk) c = kMaxChunk;
  if (c > width) c = width;
  chunk = (int)c;
  splits = (width + chunk - 1) / chunk;
}

template <int D, int BT>
cudaError_t run_attention(AttnArgs& a, int n_seq, cudaStream_t st) {
  constexpr int BYTES = Ring<D, BT>::BYTES;
  cudaError_t e = cudaFuncSetAttribute(k_cache_attention<D, BT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)n_seq * a.splits * a.kv_heads * a.row_groups;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_cache_attention<D, BT><<<(unsigned)blocks, kAttnThreads, BYTES, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.splits == 1) return e;
  const long long heads = (long long)n_seq * a.kv_heads * a.group;
  if (heads > 0x7fffffffLL) return cudaErrorInvalidValue;
  // launched while the ranges run, to wait for them on the GPU
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)heads);
  cfg.blockDim = dim3(D * kJoinParts);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_cache_join<D, BT>, a);
}

template <h3_type T, int D>
cudaError_t run_store(const StoreArgs& a, int n_seq, int block_tokens, cudaStream_t st) {
  const long long blocks = 2ll * n_seq * a.pages * a.kv_heads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)blocks;
  if (block_tokens == 32) k_kv_store<T, D, 32><<<grid, kStoreThreads, 0, st>>>(a);
  else if (block_tokens == 64) k_kv_store<T, D, 64><<<grid, kStoreThreads, 0, st>>>(a);
  else k_kv_store<T, D, 128><<<grid, kStoreThreads, 0, st>>>(a);
  return cudaGetLastError();
}

size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

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
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_codes = static_cast<uint8_t*>(c.k_codes);
  a.v_codes = static_cast<uint8_t*>(c.v_codes);
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.n_blocks = c.n_blocks;
  a.kv_heads = c.kv_heads;
  a.width = width;
  a.max_new = max_new;
  a.rows = rows;
  // max_new tokens that begin anywhere inside a block
  a.pages = (max_new + c.block_tokens - 2) / c.block_tokens + 1;
  if (a.pages > width) a.pages = width;
  a.err = err;
  if (c.head_dim == 128)
    return f16 ? run_store<H3_F16, 128>(a, n_seq, c.block_tokens, st)
               : run_store<H3_BF16, 128>(a, n_seq, c.block_tokens, st);
  return f16 ? run_store<H3_F16, 64>(a, n_seq, c.block_tokens, st)
             : run_store<H3_BF16, 64>(a, n_seq, c.block_tokens, st);
}

size_t cache_attention_workspace(const h3_kv_cache& c, int n_seq, int q_heads, int width) {
  const int group = q_heads / c.kv_heads;
  int chunk, splits;
  split_of(n_seq, c.kv_heads * ((group + kRows - 1) / kRows), width, chunk, splits);
  if (splits == 1) return 0;
  const size_t n = (size_t)n_seq * q_heads * splits;
  return align256(n * c.head_dim * 4) + align256(n * 8);
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
  a.n_blocks = c.n_blocks;
  a.kv_heads = c.kv_heads;
  a.group = q_heads / c.kv_heads;
  a.row_groups = (a.group + kRows - 1) / kRows;
  a.width = width;
  split_of(n_seq, a.kv_heads * a.row_groups, width, a.chunk, a.splits);
  a.part = static_cast<float*>(ws);
  a.stat = reinterpret_cast<float2*>(
      static_cast<uint8_t*>(ws) +
      align256((size_t)n_seq * q_heads * a.splits * c.head_dim * 4));
  a.scale_log2 = scale * 1.4426950408889634f;
  a.f16 = f16;
  a.err = err;
#define H3_RUN(D)                                                        \
  (c.block_tokens == 32 ? run_attention<D, 32>(a, n_seq, st)             \
   : c.block_tokens == 64 ? run_attention<D, 64>(a, n_seq, st)           \
                          : run_attention<D, 128>(a, n_seq, st))
  return c.head_dim == 128 ? H3_RUN(128) : H3_RUN(64);
#undef H3_RUN
}

}  // namespace h3
