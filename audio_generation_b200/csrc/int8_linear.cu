// The text model's linear layer on 8-bit integers: rows quantized to int8 codes
// with one scale each, and the product of codes
//   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k]
// with the sum in 32-bit integers on tcgen05 (kind::i8). The integer sum is
// exact whatever its order, so K may be split freely.
#include <cuda_fp16.h>
#include <limits.h>

#include <type_traits>

#include "host_util.cuh"
#include "int8_code.cuh"
#include "internal.cuh"
#include "sm100.cuh"
#include "softmax.cuh"

namespace h3 {
namespace {

// ------------------------------------------------------------- quantization
// HBM-bound: 2 (or 4) bytes in and 1 out per element. A group of G threads
// keeps its row in registers between the two passes over it (maximum, codes),
// so a row is read once; rows too long for that (K > 65536 in 16 bits) are
// read twice.
// The rounding is in int8_code.cuh.

template <h3_type T>
__device__ __forceinline__ void store_codes(const uint4& u, const RowScale& s, void* dst) {
  float v[Vec<T>::N];
  unpack<T>(u, v);
  if constexpr (T == H3_F32)
    *reinterpret_cast<uint32_t*>(dst) = codes_of_4(v, s);
  else
    *reinterpret_cast<uint2*>(dst) = codes_of_8(v, s);
}

// The maximum over the block's threads, or over each warp's alone.
template <bool BLOCK>
__device__ __forceinline__ float group_max(float m) {
  m = warp_peak(m);
  if constexpr (BLOCK) {
    __shared__ float part[32];
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = warp_peak(lane < warps ? part[lane] : 0.f);
  }
  return m;
}

// A block per row (G threads; 0: as launched), or a warp (G = 32, eight rows per
// block); NV 16-byte vectors of the row per thread in registers; NV = 0: any
// length, read twice.
template <h3_type T, int G, int NV>
__global__ void __launch_bounds__(G == 32 ? 256 : G == 0 ? 1024 : G)
    k_quantize_rows_int8(int rows, int K, const uint4* __restrict__ x, int64_t stride_vec,
                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int VE = Vec<T>::N;
  const int g = G == 0 ? blockDim.x : G;
  const int row = G == 32 ? blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (G == 32 && row >= rows) return;
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int nvec = K / VE;
  const uint4* xr = x + row * stride_vec;
  uint8_t* cr = codes + (size_t)row * K;
  uint4 u[NV > 0 ? NV : 1];
  AbsMax<T> peak;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * g < nvec) u[i] = __ldcs(xr + t + i * g);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * g < nvec) peak.add(u[i]);
  } else {
    for (int i = t; i < nvec; i += g) peak.add(xr[i]);
  }
  const float m = group_max<G != 32>(peak.value());
  if (!(m <= kMaxFinite)) {  // an infinity or a NaN in the row
    for (int i = t; i < K / 4; i += g) reinterpret_cast<uint32_t*>(cr)[i] = 0;
    if (t == 0) scales[row] = __int_as_float(0x7fc00000);
    return;
  }
  float scale = m / 127.f;
  if (scale == 0.f) scale = 1.f;  // zeros, or a maximum below the smallest scale
  const RowScale s = row_scale<T>(scale);
  if (t == 0) scales[row] = s.scale;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * g < nvec) store_codes<T>(u[i], s, cr + (t + i * g) * VE);
  } else {
    for (int i = t; i < nvec; i += g) store_codes<T>(xr[i], s, cr + (size_t)i * VE);
  }
}

// Short rows take a warp, longer ones a block of as many warps as hold them at
// eight vectors a thread (four where there are few rows, so that a row's loads
// are all in flight and little is done in turn), so that few threads idle. 8192 rows
// of 14336 bf16 elements: 53.3 us, 6.6 TB/s.
// Block sizes built in, against the one read at run time (us for 8192 rows, bf16 unless
// said): 64 threads always (K of 2560 10.8 against 11.7, 4096 16.1 : 16.3, float32 1536
// 10.0 : 11.2, 2048 12.6 : 13.1); 96, 128 and 256 where the last vectors are not all
// there (5120 19.8 : 21.6, 7168 26.5 : 28.0, 13312 51.6 : 55.0, 14336 54.3 : 57.3; float32
// 3584 21.5 : 22.2, 7168 44.1 : 45.5, but 2560 17.6 : 16.9), not where they are (6144
// 25.0 : 24.4, 8192 33.4 : 31.6, 16384 66.8 : 62.7; float32 4096 26.7 : 24.9, 8192 55.8 :
// 52.9); 160 and 192 never (10240 43.9 : 41.4, 12288 51.5 : 49.0; float32 5120 34.3 :
// 31.4), and 224 take 256 (14336 with 224 built in 62.7).
template <h3_type T>
cudaError_t quantize(int rows, int K, const void* x, int64_t stride_vec, void* codes,
                     float* scales, cudaStream_t st) {
  const int nvec = K / Vec<T>::N;
  const uint4* xv = static_cast<const uint4*>(x);
  uint8_t* c = static_cast<uint8_t*>(codes);
#define H3_Q(G, NV, GRID, THREADS)                                                     \
  k_quantize_rows_int8<T, G, NV><<<GRID, THREADS, 0, st>>>(rows, K, xv, stride_vec, c, scales)
  const int few = (nvec + 127) / 128 * 32, many = (nvec + 255) / 256 * 32;
  if (nvec <= 64) H3_Q(32, 2, (rows + 7) / 8, 256);
  else if (nvec <= 256) H3_Q(32, 8, (rows + 7) / 8, 256);
  else if (nvec <= 4096 && rows <= 4 * num_sms()) H3_Q(0, 4, rows, few);
  else if (many == 64) H3_Q(64, 8, rows, 64);
  else if (many == 96 && nvec < 768) H3_Q(96, 8, rows, 96);
  else if (many == 128 && nvec < 1024) H3_Q(128, 8, rows, 128);
  else if (many >= 224 && nvec < 2048) H3_Q(256, 8, rows, 256);
  else if (nvec <= 8192) H3_Q(0, 8, rows, many);
  else H3_Q(0, 0, rows, 1024);
#undef H3_Q
  return cudaGetLastError();
}

// ------------------------------------------------------------- matrix product

#ifdef H3_FAULT_INJECTION
// Test-only build: the K step (of a CTA's, in the order of its fetches) whose copies
// are not counted, so that the wait for it runs out (none where negative).
static __device__ int g_fault_skip_step = -1;
#endif

constexpr int BM = 128;        // rows of a CTA's operand tile = TMEM lanes
constexpr int BKB = 128;       // K bytes per stage: one 128-byte swizzled row
constexpr int NUM_THREADS = 192;
constexpr int A_STAGE = BM * BKB;  // 16 KB

struct Out {
  void* p;
  int64_t stride_m, stride_n;  // elements between rows, and between columns
  int type;
  const float* a_scale;
  const float* w_scale;
};

// A sum times its two scales in float32: three roundings, 3 x 2^-24 relative; a 16-bit
// type rounds once more. The smaller scale comes first: a product with it leaves
// float32's normal numbers only if the value does or the scale itself has (then it
// is a multiple of the subnormals' step, and exact), where the scales' product
// could have few bits, be 0 or infinite. A NaN scale gives NaN.
__device__ __forceinline__ float scaled(uint32_t sum, float a, float w) {
  float low, high;  // by magnitude; low has the sign of both
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(low) : "f"(a), "f"(w));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(high) : "f"(fabsf(a)), "f"(fabsf(w)));
  return (float)(int)sum * low * high;
}

// Two sums times a lane's own scale, then times two others, two to an instruction: the
// same, as long as the lane's scale is at most kOwnFirst, with which no sum leaves
// the range. (The form above for all values costs the epilogues 6 %: 8192 x 5120 x
// 512 44.5 us against 42.)
constexpr float kOwnFirst = 0x1p96f;
__device__ __forceinline__ void scaled_2(uint32_t sum0, uint32_t sum1, uint64_t own2,
                                         uint64_t others, float& y0, float& y1) {
  f2_unpack(f2_mul(f2_mul(f2_pack((float)(int)sum0, (float)(int)sum1), own2), others), y0, y1);
}

// One output value.
__device__ __forceinline__ void store_one(const Out& o, size_t off, float v) {
  if (o.type == H3_BF16)
    static_cast<__nv_bfloat16*>(o.p)[off] = __float2bfloat16_rn(v);
  else if (o.type == H3_F16)
    static_cast<__half*>(o.p)[off] = __float2half_rn(v);
  else
    static_cast<float*>(o.p)[off] = v;
}

// Four neighbouring values of one row, aligned to their size.
__device__ __forceinline__ void store_4(const Out& o, size_t off, const float* v) {
  if (o.type == H3_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(o.p) + off) =
        make_float4(v[0], v[1], v[2], v[3]);
  } else if (o.type == H3_BF16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.p) + off) =
        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else {
    const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.p) + off) = make_uint2(
        *reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

template <h3_type T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (T == H3_BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A warp's 32 x 32 values, row i from turn + kTurn i, to `rows` rows of out from off
// on, `cols` columns each: whole and aligned rows in pieces of 16 bytes, a row's
// pieces by neighbouring lanes; else neighbouring lanes store neighbouring columns.
constexpr int kTurn = 36;
constexpr int kTurnBytes = 4 * 32 * kTurn * 4;  // of four warps
template <h3_type T>
__device__ __forceinline__ void store_turned(const Out& o, int64_t off, int64_t stride,
                                             const float* turn, int rows, int cols, bool vec,
                                             int lane) {
  if (vec && cols >= 32) {
    constexpr int PER = T == H3_F32 ? 4 : 8;  // values of a piece
    constexpr int LANES = 32 / PER;           // lanes of a row
    const int i0 = lane / LANES, q = lane % LANES * PER;
    const float* src = turn + i0 * kTurn + q;
    off += i0 * stride + q;
#pragma unroll
    for (int i = 0; i < 32; i += 32 / LANES) {
      const float4 x = *reinterpret_cast<const float4*>(src + i * kTurn);
      uint4 w;
      if constexpr (T == H3_F32) {
        w = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                       __float_as_uint(x.w));
      } else {
        const float4 y = *reinterpret_cast<const float4*>(src + i * kTurn + 4);
        w = make_uint4(pack16<T>(x.x, x.y), pack16<T>(x.z, x.w),
                       pack16<T>(y.x, y.y), pack16<T>(y.z, y.w));
      }
      if (i0 + i < rows)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(o.p) +
                                  (off + i * stride) * (T == H3_F32 ? 4 : 2)) = w;
    }
    return;
  }
  if (stride % 2 == 0 && cols >= 32) {  // rows aligned to two values
    const int i0 = lane / 16, q = lane % 16 * 2;
    off += i0 * stride + q;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 x = *reinterpret_cast<const float2*>(turn + (i0 + i) * kTurn + q);
      if (i0 + i < rows) {
        if constexpr (T == H3_F32)
          *reinterpret_cast<float2*>(static_cast<float*>(o.p) + off) = x;
        else
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(o.p) + off) = pack16<T>(x.x, x.y);
      }
      off += 2 * stride;
    }
    return;
  }
  if (lane >= cols) return;
  off += lane;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float x = turn[i * kTurn + lane];
    if (i < rows) {
      if constexpr (T == H3_F32) static_cast<float*>(o.p)[off] = x;
      else static_cast<uint16_t*>(o.p)[off] = (uint16_t)pack16<T>(x, 0.f);
    }
    off += stride;
  }
}
// The same from a row per lane.
__device__ __forceinline__ void turn_and_store(const Out& o, int64_t off, int64_t stride,
                                               float* turn, const float* v, int rows, int cols,
                                               bool vec, int lane) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    *reinterpret_cast<float4*>(turn + lane * kTurn + 4 * q) =
        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  __syncwarp();
  if (o.type == H3_F32) store_turned<H3_F32>(o, off, stride, turn, rows, cols, vec, lane);
  else if (o.type == H3_BF16) store_turned<H3_BF16>(o, off, stride, turn, rows, cols, vec, lane);
  else store_turned<H3_F16>(o, off, stride, turn, rows, cols, vec, lane);
  __syncwarp();
}

// Many rows: the persistent CTA-pair form. A pair computes 256 x BN tiles of
// out with cta_group::2 MMAs, each CTA holding 128 rows of A and BN / 2 of the
// tile's weight rows per stage, 128 bytes of K (four K = 32 instructions), six
// stages; the accumulator is double-buffered in TMEM, so the epilogue of a tile
// overlaps the next tile's products. Warps: 0 TMA producer, 1 TMEM owner and
// MMA issuer, 2..5 epilogue (one TMEM lane = one row per thread).
// 8191 x 14336 x 5376: 372 us alone (3.4 P operations/s, the tensor pipe active in
// 97 % of the cycles), 430 to 470 us in a loop, where the board's power cap holds
// the clock down.
constexpr int PNST = 6;
template <int BN>
constexpr int p_stage() { return A_STAGE + BN / 2 * BKB; }
template <int BN>
constexpr int p_smem() { return PNST * p_stage<BN>() + 1024 + 256 + 4 * (BN + 32 * kTurn) * 4; }

template <int BN>
__device__ __forceinline__ void pair_tile(int t, int tiles_m, int tiles_n, int group_n, int& m0,
                                          int& n0) {
  const int per_group = group_n * tiles_m;
  const int g = t / per_group, r = t - g * per_group;
  const int width = min(group_n, tiles_n - g * group_n);
  m0 = (r / width) * 2 * BM;
  n0 = (g * group_n + r % width) * BN;
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NUM_THREADS, 1)
    k_int8_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                int M, int N, int kb_n, int group_n, const Out out, int* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  constexpr int STAGE = p_stage<BN>();
  static_assert(STAGE % 1024 == 0, "stage alignment");
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + PNST * STAGE);
  uint64_t* empty = full + PNST;
  uint64_t* tfull = empty + PNST;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int tiles_m = (M + 2 * BM - 1) / (2 * BM), tiles_n = (N + BN - 1) / BN;
  const int T = tiles_m * tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < PNST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 8);  // one arrival per epilogue warp of both CTAs
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{err, abort_flag};
  auto at = [&](uint64_t* bar, uint32_t r) { return mapa_shared(smem_u32(bar), r); };
  uint32_t fills = 0;  // thread 0's stages issued

  if (warp == 0) {
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int t = pair; t < T && ok; t += n_pairs) {
        int m0, n0;
        pair_tile<BN>(t, tiles_m, tiles_n, group_n, m0, n0);
        for (int kb = 0; kb < kb_n; ++kb) {
          const uint32_t s = n % PNST, ph = (n / PNST) & 1;
          if (!mbar_wait(&empty[s], ph ^ 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * STAGE;
#ifdef H3_FAULT_INJECTION
          if ((int)n != *(volatile int*)&g_fault_skip_step)
#endif
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * STAGE);
          tma_load_2d_pair(sa, &tmA, at(&full[s], 0), kb * BKB, m0 + BM * rank);
          tma_load_2d_pair(sa + A_STAGE, &tmW, at(&full[s], 0), kb * BKB, n0 + (BN / 2) * rank);
          ++n;
        }
      }
      fills = n;
    }
  } else if (warp == 1) {
    if (leader) {  // the whole warp runs the loop; one elected lane issues
      constexpr uint32_t idesc = idesc_s8_s32(2 * BM, BN);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t base_lo = sdesc_lo(smem_u32(smem), 16);
      uint32_t n = 0, it = 0;
      bool ok = true;
      for (int t = pair; t < T && ok; t += n_pairs, ++it) {
        const uint32_t acc = it & 1, aph = (it >> 1) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&tempty[acc], aph ^ 1, wc))) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < kb_n; ++kb) {
          const uint32_t s = n % PNST, ph = (n / PNST) & 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, wc))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_lo = base_lo + s * (STAGE >> 4);
          const uint32_t b_lo = a_lo + (A_STAGE >> 4);
#pragma unroll
          for (int k = 0; k < BKB / 32; ++k)
            umma_ss_w_pair_elect_i8(d, a_lo + 2 * k, hi, b_lo + 2 * k, hi, idesc,
                                    (kb | k) != 0 ? 1u : 0u);
          umma_commit_pair_elect(at(&empty[s], 0));
          umma_commit_pair_elect(at(&empty[s], 1));
          ++n;
        }
        if (!ok) break;
        umma_commit_pair_elect(at(&tfull[acc], 0));
        umma_commit_pair_elect(at(&tfull[acc], 1));
      }
      umma_commit_pair_elect(at(drain, 0));  // every MMA issued is complete past this point
      mbar_drain(drain, 0);
    }
  } else {
    const int quarter = warp & 3;
    const uint32_t tempty0 = at(&tempty[0], 0), tempty1 = at(&tempty[1], 0);
    const bool vec = out.stride_m % (out.type == H3_F32 ? 4 : 8) == 0;
    // the tile's column scales, and 32 x 32 values to turn
    float* scales = reinterpret_cast<float*>(smem + PNST * STAGE + 256) + (warp - 2) * BN;
    float* turn =
        reinterpret_cast<float*>(smem + PNST * STAGE + 256) + 4 * BN + (warp - 2) * 32 * kTurn;
    uint32_t it = 0;
    for (int t = pair; t < T; t += n_pairs, ++it) {
      const uint32_t acc = it & 1, aph = (it >> 1) & 1;
      int m0, n0;
      pair_tile<BN>(t, tiles_m, tiles_n, group_n, m0, n0);
      m0 += BM * rank + quarter * 32;
      const int m = m0 + lane;
      const bool row_ok = m < M;
      const float sa = row_ok ? __ldg(out.a_scale + m) : 0.f;
      const uint64_t sa2 = f2_pack(sa, sa);
#pragma unroll
      for (int k = 4 * lane; k < BN; k += 128) {
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        const float* src = out.w_scale + n0 + k;
        if (n0 + k + 4 <= N) {
          w = __ldg(reinterpret_cast<const float4*>(src));
        } else {
          if (n0 + k < N) w.x = __ldg(src);
          if (n0 + k + 1 < N) w.y = __ldg(src + 1);
          if (n0 + k + 2 < N) w.z = __ldg(src + 2);
        }
        *reinterpret_cast<float4*>(scales + k) = w;
      }
      __syncwarp();
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], aph, wc))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
#pragma unroll 1
      for (int c = 0; c < BN / 32; ++c) {
        const int n = n0 + 32 * c;
        if (n >= N || m0 >= M) break;
        uint32_t r[32];
        tmem_ld32(taddr + 32 * c, r);
        tmem_wait_ld();
        float v[32];
        const ulonglong2* w4 = reinterpret_cast<const ulonglong2*>(scales + 32 * c);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const ulonglong2 w = w4[q];
          scaled_2(r[4 * q], r[4 * q + 1], sa2, w.x, v[4 * q], v[4 * q + 1]);
          scaled_2(r[4 * q + 2], r[4 * q + 3], sa2, w.y, v[4 * q + 2], v[4 * q + 3]);
        }
        // (A lane per row would store 16 bytes of 32 rows at a time: 63 us for 2031 x
        // 18992 x 256 to float32, against 43 us; 50 us against 11 for 4517 x 275 x 224.)
        turn_and_store(out, m0 * out.stride_m + n, out.stride_m, turn, v, min(32, M - m0),
                       min(32, N - n), vec, lane);
      }
      if (__any_sync(0xffffffffu, fabsf(sa) > kOwnFirst)) {  // the same places once more
#pragma unroll 1
        for (int n = n0; n < n0 + BN && n < N && m0 < M; n += 32) {
          uint32_t r[32];
          tmem_ld32(taddr + n - n0, r);
          tmem_wait_ld();
          __syncwarp();  // the turned values of before have been read, and stored
          float* row = turn + lane * kTurn;
#pragma unroll
          for (int k = 0; k < 32; ++k) row[k] = __uint_as_float(r[k]);
#pragma unroll 1
          for (int k = 0; k < 32 && n + k < N; ++k)
            if (row_ok)
              store_one(out, m * out.stride_m + n + k,
                        scaled(__float_as_uint(row[k]), sa, scales[n - n0 + k]));
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acc ? tempty1 : tempty0);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && leader && *abort_flag) {  // both CTAs' issued copies land first
    for (uint32_t i = fills > PNST ? fills - PNST : 0; i < fills; ++i)
      mbar_drain(&full[i % PNST], (i / PNST) & 1);
  }
  cluster_sync();  // no CTA leaves while the pair's MMAs or signals may still reach it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * BN);
  }
}

// Few rows: bound by the bytes of the weights, or by how many SMs have work. The
// weights take the MMA's 128-row side and NT tokens its N side, so a CTA streams
// tiles of 128 weight rows through a ring that fills most of its SM's shared
// memory (the bytes in flight are what carries the bandwidth), one CTA per SM,
// the ring running on from tile to tile (token tiles first, so that a weight tile
// stays in L2 for its others). With few tiles the CTAs of a cluster share the K
// axis of one and add their integer sums through distributed shared memory,
// each finishing a share of the tokens. Neighbouring lanes store neighbouring
// columns of out. Warps as above; the accumulator is double-buffered.
// 1 x 14336 x 5120: 13.6 to 15 us (73 MB: 5 TB/s, 3 to 4 us of it launch, fill and
// tail); 48 x 32003 x 5120 with float32 out: 32.0 us (170 MB: 5.3 TB/s).
template <int NT>
constexpr int s_stage() { return A_STAGE + NT * BKB; }
template <int NT>
constexpr int s_stages() { return 200 * 1024 / s_stage<NT>(); }
template <int NT, bool TURN>
constexpr int s_smem() {
  return s_stages<NT>() * s_stage<NT>() + 1024 + 512 + (TURN ? kTurnBytes : 0);
}

constexpr int kMaxSplit = 8;  // CTAs that share a K axis

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int NT, bool TURN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_int8_skinny(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                  int M, int N, int kb_n, int split, const Out out, int* err) {
  constexpr int NST = s_stages<NT>(), STAGE = s_stage<NT>();
  static_assert(STAGE % 1024 == 0, "stage alignment");
  static_assert(NT * BM * 4 <= NST * STAGE, "the partial sums reuse the stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + NST * STAGE);
  uint64_t* empty = full + NST;
  uint64_t* tfull = empty + NST;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t ACC = NT < 32 ? 32 : NT;  // columns of one accumulator

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int m_tiles = (M + NT - 1) / NT;
  const int tiles = (N + BM - 1) / BM * m_tiles;
  const int tile0 = (int)(blockIdx.x / split), step = (int)(gridDim.x / split);
  const int kb0 = (int)((long long)kb_n * rank / split);
  const int kb1 = (int)((long long)kb_n * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 4);  // one arrival per epilogue warp
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * ACC);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{err, abort_flag};
  uint32_t fills = 0;  // thread 0's stages issued

  if (warp == 0) {
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int t = tile0; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb, ++n) {
          const uint32_t s = n % NST, ph = (n / NST) & 1;
          if (!mbar_wait(&empty[s], ph ^ 1, wc)) {
            ok = false;
            break;
          }
          uint8_t* sw = smem + s * STAGE;
#ifdef H3_FAULT_INJECTION
          if ((int)n != *(volatile int*)&g_fault_skip_step)
#endif
          mbar_arrive_expect_tx(&full[s], STAGE);
          tma_load_2d(sw, &tmW, &full[s], kb * BKB, t / m_tiles * BM);
          tma_load_2d(sw + A_STAGE, &tmA, &full[s], kb * BKB, t % m_tiles * NT);
        }
      }
      fills = n;
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_s8_s32(BM, NT);
    constexpr uint32_t hi = sdesc_hi_sw128(1024);
    const uint32_t base_lo = sdesc_lo(smem_u32(smem), 16);
    uint32_t n = 0, it = 0;
    bool ok = true;
    for (int t = tile0; t < tiles && ok; t += step, ++it) {
      const uint32_t acc = it & 1, aph = (it >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&tempty[acc], aph ^ 1, wc))) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * ACC;
      for (int kb = kb0; kb < kb1; ++kb, ++n) {
        const uint32_t s = n % NST, ph = (n / NST) & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], ph, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a_lo = base_lo + s * (STAGE >> 4);
        const uint32_t b_lo = a_lo + (A_STAGE >> 4);
#pragma unroll
        for (int k = 0; k < BKB / 32; ++k)
          umma_ss_w_elect_i8(d, a_lo + 2 * k, hi, b_lo + 2 * k, hi, idesc,
                             (kb > kb0 || k > 0) ? 1u : 0u);
        umma_commit_elect(&empty[s]);
      }
      if (!ok) break;
      umma_commit_elect(&tfull[acc]);
    }
    umma_commit_elect(drain);  // every MMA issued is complete past this point
    mbar_drain(drain, 0);
  } else {
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // weight row of the tile
    float* turn = reinterpret_cast<float*>(smem + NST * STAGE + 512) + (warp - 2) * 32 * kTurn;
    const bool vec = out.stride_n % (out.type == H3_F32 ? 4 : 8) == 0;
    uint32_t it = 0;
    for (int t = tile0; t < tiles; t += step, ++it) {
      const uint32_t acc = it & 1, aph = (it >> 1) & 1;
      const int n = t / m_tiles * BM + r, m0 = t % m_tiles * NT;
      const int rows = min(NT, M - m0);
      const float sw = n < N ? __ldg(out.w_scale + n) : 0.f;
      float sa_next = lane < rows ? __ldg(out.a_scale + m0 + lane) : 0.f;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], aph, wc))) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + acc * ACC;
      // with a shared K axis: [NT][128] sums of this CTA, over its stages (the
      // one tile's products are complete, so nothing reads them any more)
      uint32_t* part = reinterpret_cast<uint32_t*>(smem);
#pragma unroll 1
      for (int c = 0; c < (NT + 31) / 32; ++c) {
        const float sa = sa_next;  // of token 32 c + lane
        sa_next = 32 * c + 32 + lane < rows ? __ldg(out.a_scale + m0 + 32 * c + 32 + lane) : 0.f;
        uint32_t v[32];
        tmem_ld32(taddr + 32 * c, v);
        tmem_wait_ld();
        if (split > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < rows) part[(32 * c + i) * BM + r] = v[i];
        } else {
          float y[32];
          if constexpr (TURN) {
            const uint64_t sw2 = f2_pack(sw, sw);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              scaled_2(v[i], v[i + 1], sw2, f2_pack(__shfl_sync(0xffffffffu, sa, i),
                                                    __shfl_sync(0xffffffffu, sa, i + 1)),
                       y[i], y[i + 1]);
            if (n - lane < N)
              turn_and_store(out, (n - lane) * out.stride_n + m0 + 32 * c, out.stride_n, turn, y,
                             min(32, N - (n - lane)), min(32, rows - 32 * c), vec, lane);
            if (__any_sync(0xffffffffu, fabsf(sw) > kOwnFirst)) {  // the same places once more
              tmem_ld32(taddr + 32 * c, v);
              tmem_wait_ld();
              float* row = turn + lane * kTurn;
#pragma unroll
              for (int i = 0; i < 32; ++i) row[i] = __uint_as_float(v[i]);
#pragma unroll 1
              for (int i = 0; i < 32 && 32 * c + i < rows; ++i) {
                const float a = __shfl_sync(0xffffffffu, sa, i);
                if (n < N)
                  store_one(out, n * out.stride_n + m0 + 32 * c + i,
                            scaled(__float_as_uint(row[i]), a, sw));
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i] = scaled(v[i], __shfl_sync(0xffffffffu, sa, i), sw);
            if (n < N) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i < rows)
                  store_one(out, (m0 + 32 * c + i) * out.stride_m + n, y[i]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
    }
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();
    const int n = tile0 / m_tiles * BM + 4 * lane;  // four columns of a token per thread
    if (warp >= 2 && n < N) {
      const int m0 = tile0 % m_tiles * NT, rows = min(NT, M - m0);
      const int first = rows * rank / split, last = rows * (rank + 1) / split;
      const bool vec = n + 4 <= N && out.stride_n == 1 && out.stride_m % 4 == 0;
      float sw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sw[e] = n + e < N ? __ldg(out.w_scale + n + e) : 0.f;
      const uint32_t mine = smem_u32(smem) + lane * 16;
      // U tokens of a warp side by side, each from at most Q CTAs: the latency of the
      // fetches is what the join takes
      auto join = [&](auto tokens, auto ctas) {
        constexpr int U = decltype(tokens)::value, Q = decltype(ctas)::value;
        for (int i0 = first + warp - 2; i0 < last; i0 += 4 * U) {
          uint4 v[U][Q];
          float sa[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = min(i0 + 4 * u, last - 1);
            sa[u] = __ldg(out.a_scale + m0 + i);
#pragma unroll
            for (int q = 0; q < Q; ++q)
              v[u][q] = q < split ? ld_cluster_v4(mapa_shared(mine, q) + i * BM * 4)
                                  : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = i0 + 4 * u;
            if (i >= last) break;
            uint4 sum = v[u][0];
#pragma unroll
            for (int q = 1; q < Q; ++q)
              sum.x += v[u][q].x, sum.y += v[u][q].y, sum.z += v[u][q].z, sum.w += v[u][q].w;
            const float y[4] = {scaled(sum.x, sa[u], sw[0]), scaled(sum.y, sa[u], sw[1]),
                                scaled(sum.z, sa[u], sw[2]), scaled(sum.w, sa[u], sw[3])};
            const size_t at = (m0 + i) * out.stride_m + n * out.stride_n;
            if (vec) {
              store_4(out, at, y);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < N) store_one(out, at + e * out.stride_n, y[e]);
            }
          }
        }
      };
      if (!TURN && split <= 3)
        join(std::integral_constant<int, 4>(), std::integral_constant<int, 3>());
      else
        join(std::integral_constant<int, 1>(), std::integral_constant<int, kMaxSplit>());
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
  }
  if (threadIdx.x == 0 && *abort_flag) {  // issued copies land before the CTA retires
    for (uint32_t i = fills > NST ? fills - NST : 0; i < fills; ++i)
      mbar_drain(&full[i % NST], (i / NST) & 1);
  }
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * ACC);
  }
}

bool tmap_codes(CUtensorMap* t, const void* p, int rows, int K, uint32_t box_rows) {
  const uint64_t d[2] = {(uint64_t)K, (uint64_t)rows}, s[1] = {(uint64_t)K};
  const uint32_t b[2] = {BKB, box_rows};
  return make_tmap(t, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, d, s, b);
}

template <int BN>
cudaError_t run_pair(int M, int N, int K, const void* a, const void* w, const Out& out, int* err,
                     cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_int8_pair<BN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, p_smem<BN>());
  if (e != cudaSuccess) return e;
  CUtensorMap ta, tw;
  if (!tmap_codes(&ta, a, M, K, BM) || !tmap_codes(&tw, w, N, K, BN / 2))
    return cudaErrorInvalidValue;
  const long long tiles_n = (N + BN - 1) / BN;
  const long long T = (long long)((M + 2 * BM - 1) / (2 * BM)) * tiles_n;
  if (T > 0x3fffffff) return cudaErrorInvalidValue;
  const int max_pairs = num_sms() / 2;
  const int n_pairs = T < max_pairs ? (int)T : max_pairs;
  // Weight tiles kept L2-resident per group: about 48 MB.
  long long group_n = (48ll << 20) / ((long long)BN * K);
  if (group_n < 1) group_n = 1;
  if (group_n > tiles_n) group_n = tiles_n;
  k_int8_pair<BN><<<2 * n_pairs, NUM_THREADS, p_smem<BN>(), st>>>(
      ta, tw, M, N, (K + BKB - 1) / BKB, (int)group_n, out, err);
  return cudaGetLastError();
}

// Clusters of `split` CTAs that the current device runs at once (asked once).
template <int NT, bool TURN>
int clusters_at_once(int split) {
  static int known[64][kMaxSplit + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (known[dev][split] == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(NUM_THREADS);
    cfg.dynamicSmemBytes = s_smem<NT, TURN>();
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(k_int8_skinny<NT, TURN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             s_smem<NT, TURN>()) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k_int8_skinny<NT, TURN>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev][split] = n > 0 ? n : -1;
  }
  return known[dev][split];
}

// How a launch of the few-row kernel looks, and about how many cycles it takes.
struct Plan {
  long long cycles;
  int split, ctas;
  int tokens;  // of a tile: NT
};

// Cycles, from measurements at 1.9 GHz: a K step of a CTA costs its MMAs (2 NT) or
// the fetch of its operands at 44 bytes a cycle, all weights together at least
// 3440 bytes a cycle (HBM); 6000 go to launch, fill and last tile, and joining a
// shared K axis costs 1500 and 90 for each token that a CTA finishes (350 with out
// turned, whose columns are then stored one by one). (5120 x 5120, one row: 8 us;
// 128 rows: 11.5 us; 256 rows: 15.6 us in tiles of 256 against 18.3 by pairs of CTAs;
// 1024 x 5120, 512 rows: 10 us against 20.)
template <int NT, bool TURN>
Plan plan_skinny(int M, int N, int K) {
  Plan p{};
  p.tokens = NT;
  const int kb_n = (K + BKB - 1) / BKB, sms = num_sms();
  const long long tiles = (long long)((N + BM - 1) / BM) * ((M + NT - 1) / NT);
  // As many CTAs share a tile's K axis as leave every tile a cluster that runs at
  // once, each with two K steps at least; with more tiles a CTA takes whole ones.
  int split = tiles < sms ? (int)(sms / tiles) : 1;
  if (split > kb_n / 2) split = kb_n / 2;
  if (split > kMaxSplit) split = kMaxSplit;
  while (split > 1 && clusters_at_once<NT, TURN>(split) < tiles) --split;
  if (split < 1) split = 1;
  const long long step = 2 * NT > (A_STAGE + NT * BKB) / 44 ? 2 * NT : (A_STAGE + NT * BKB) / 44;
  const long long bytes = (long long)N * K / 3440;
  for (;; split = 1) {
    const long long run = (tiles * split + sms - 1) / sms * ((kb_n + split - 1) / split) * step;
    const long long join = split > 1 ? 1500 + (TURN ? 350 : 90) * (M < NT ? M : NT) / split : 0;
    const long long cycles = (run > bytes ? run : bytes) + 6000 + join;
    if (p.split == 0 || cycles < p.cycles) {
      p.cycles = cycles;
      p.split = split;
      p.ctas = split > 1 ? (int)tiles * split : (int)(tiles < sms ? tiles : sms);
    }
    if (split == 1) return p;
  }
}

// The same for the pair kernel: 700 cycles a K step and wave, 8000 around.
long long pair_cycles(int M, int N, int K) {
  const long long tiles =
      (long long)((M + 2 * BM - 1) / (2 * BM)) * ((N + 255) / 256), pairs = num_sms() / 2;
  const long long run = (tiles + pairs - 1) / pairs * ((K + BKB - 1) / BKB) * 700;
  const long long bytes = (long long)N * K / 3440;
  return (run > bytes ? run : bytes) + 8000;
}

template <int NT, bool TURN>
cudaError_t run_skinny(const Plan& p, int M, int N, int K, const void* a, const void* w,
                       const Out& out, int* err, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(k_int8_skinny<NT, TURN>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       s_smem<NT, TURN>());
  if (e != cudaSuccess) return e;
  CUtensorMap ta, tw;
  if (!tmap_codes(&ta, a, M, K, NT) || !tmap_codes(&tw, w, N, K, BM)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = s_smem<NT, TURN>();
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_int8_skinny<NT, TURN>, tw, ta, M, N, (K + BKB - 1) / BKB,
                            p.split, out, err);
}

// The narrowest token tile that holds all tokens, or tiles of 128 of them, or of 256
// where those are so few that their K axis is shared.
template <bool TURN>
Plan plan_any(int M, int N, int K) {
  if (M <= 16) return plan_skinny<16, TURN>(M, N, K);
  if (M <= 32) return plan_skinny<32, TURN>(M, N, K);
  if (M <= 64) return plan_skinny<64, TURN>(M, N, K);
  const Plan p = plan_skinny<128, TURN>(M, N, K);
  if constexpr (!TURN) {
    if (M > 128) {
      const Plan wide = plan_skinny<256, TURN>(M, N, K);
      if (wide.split > 1 && wide.cycles < p.cycles) return wide;
    }
  }
  return p;
}
template <bool TURN>
cudaError_t run_any(const Plan& p, int M, int N, int K, const void* a, const void* w,
                    const Out& out, int* err, cudaStream_t st) {
  switch (p.tokens) {
    case 16: return run_skinny<16, TURN>(p, M, N, K, a, w, out, err, st);
    case 32: return run_skinny<32, TURN>(p, M, N, K, a, w, out, err, st);
    case 64: return run_skinny<64, TURN>(p, M, N, K, a, w, out, err, st);
    case 128: return run_skinny<128, TURN>(p, M, N, K, a, w, out, err, st);
  }
  if constexpr (!TURN) return run_skinny<256, TURN>(p, M, N, K, a, w, out, err, st);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_quantize_rows_int8(h3_type type, int rows, int K, const void* x,
                                      int64_t x_stride, void* codes, float* scales,
                                      cudaStream_t st) {
  switch (type) {
    case H3_BF16: return quantize<H3_BF16>(rows, K, x, x_stride / 8, codes, scales, st);
    case H3_F16: return quantize<H3_F16>(rows, K, x, x_stride / 8, codes, scales, st);
    case H3_F32: return quantize<H3_F32>(rows, K, x, x_stride / 4, codes, scales, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_matmul_int8(int M, int N, int K, const void* a, const float* a_scale,
                               const void* w, const float* w_scale, h3_type out_type, void* out,
                               int64_t out_stride, int* err, cudaStream_t st) {
  const Out o{out, out_stride, 1, (int)out_type, a_scale, w_scale};
  // The few-row kernel with a's rows as tokens (up to 2048 of them), or, where out
  // is narrower than long, with w's rows as tokens and out turned. Pairs of CTAs
  // where they are estimated to be faster. (2290 x 10 x 9040: 7.7 us turned, 30 us by
  // pairs, of which there are only nine.)
  const bool few = M <= 2048, turn = N <= 128 && N < M;
  Plan p{}, q{};
  if (few) p = plan_any<false>(M, N, K);
  if (turn) q = plan_any<true>(N, M, K);
  const long long pairs = M <= 128 ? LLONG_MAX : pair_cycles(M, N, K);
  if (turn && q.cycles < pairs && (!few || q.cycles < p.cycles)) {
    const Out t{out, 1, out_stride, (int)out_type, w_scale, a_scale};
    return run_any<true>(q, N, M, K, w, a, t, err, st);
  }
  if (few && p.cycles < pairs) return run_any<false>(p, M, N, K, a, w, o, err, st);
  return run_pair<256>(M, N, K, a, w, o, err, st);
}

}  // namespace h3

#ifdef H3_FAULT_INJECTION
extern "C" __attribute__((visibility("default"))) int h3_test_int8_skip_step(int step) {
  return cudaMemcpyToSymbol(h3::g_fault_skip_step, &step, sizeof(int)) == cudaSuccess ? 0 : -1;
}
#endif
