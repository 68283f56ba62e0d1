// Causal attention over packed prompts of different lengths, grouped heads:
//   o[i, h] = sum_{j <= i} softmax_j(scale q[i, h] . k[j, h / G]) v[j, h / G]
// over the tokens of i's own prompt, G = q_heads / kv_heads.
//
// Flash style on tcgen05, one pass over the keys with a running maximum and
// sum, the roles and tensor-memory plan of the packed-sequence attention kernel:
// a CTA takes two 128-row query tiles of one kv head, so that the tensor core
// works on one tile while the other's softmax runs. Warps 0..3 and 4..7 are the
// tiles' softmax (one row per thread = one TMEM lane), warp 8 the TMA producer,
// warp 9 the TMEM owner and MMA issuer, warps 10 and 11 idle (their registers go
// to the softmax). S_i takes 128 TMEM columns, P overwrites its first 64, O_i
// takes D.
//
// A tile's rows are (position, head of the group): 128 / G positions with all G
// heads that share the K and V tile. Compared with 128 positions of one head, a
// short prompt fills its tiles G times better, the diagonal costs G times fewer
// masked keys, and K and V are fetched once per group. One 3-D TMA box (64
// channels, G heads, 128 / G tokens) lays such a tile down as 128-byte rows.
// Where G does not divide 128 the last rows of a tile are idle.
//
// Work items (two tiles each, or one where that leaves no SM idle) come from the
// prompts object, longest key range first. One CTA per SM takes them in turn (there
// and back over the list's rounds, so that no CTA always gets the longer one), every
// role running on into the next item: its first keys and its q are fetched and a query tile's first
// scores computed right after the tile's last product of the item before, while
// that is still being divided and stored. A q tile is given back after the item's
// last score product with it, an O accumulator when its rows have been read.
//
// Bound by the softmax's chain: 1650 cycles per 128 x 128 tile against 1024 of tensor
// work at D = 128. One prompt of 8192 tokens, 56 heads over 8 x 128: 810 us at full
// clock (1190 TFLOP/s), 925 us in a loop of seconds, whose power cap brings the clock
// to 1.63 GHz; 12 prompts of 120 to 2500 tokens, 40 over 8: 131 and 148 us. An item
// costs about 4 us beyond its key tiles, from its first fetch to its last store.
#include <cuda_fp16.h>

#include <algorithm>
#include <new>
#include <vector>

#include "host_util.cuh"
#include "internal.cuh"
#include "sm100.cuh"
#include "softmax.cuh"

namespace h3 {
namespace {

#ifdef H3_FAULT_INJECTION
// Test-only build: the key tile (of a CTA's, in the order of its fetches) whose copies
// are not counted, so that the wait for it runs out (none where negative).
static __device__ int g_fault_skip_keys = -1;
#endif

constexpr int HALF = 128 * 64 * 2;  // 128 rows x 64 channels: 16 KB
constexpr int NUM_THREADS = 384;
// 2 * 128 * kSoftmaxRegs + 128 * kControlRegs must not exceed the 384 * 168
// registers of the launch.
constexpr uint32_t kSoftmaxRegs = 216, kControlRegs = 72;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs <= 384 * 168, "register split");
constexpr int TMEM_COLS = 512;
constexpr float kLazyRescale = 8.0f;  // log2 units

struct Bars {
  uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2],
      p_half[2], p_full[2], o_final[2], o_free[2], drain;
};

// 2^f on the FMA pipe, f in [-1/2, 1/2]: the cubic of least largest relative error
// (1.02e-4) among those that are 1 at 0, and which of 32 key pairs take it. With
// arguments limited to -127 and more it then gives 0 there, and so to masked keys
// (2^-126, say, times the largest v would be more than 1). A NaN gives the largest
// number, which as a weight becomes infinite and so marks its row.
constexpr float kExpC3 = 0.05500905961f, kExpC2 = 0.24221096933f, kExpC1 = 0.69328290224f,
                kExpC0 = 1.f, kExpLowest = -127.f;
constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23
constexpr uint32_t kCubicPairs = 0x20820820u;  // every sixth

// smem: Q0 Q1 | K0 K1 | V0 V1 | barriers
template <int D>
constexpr int tile_bytes() { return D / 64 * HALF; }
template <int D>
constexpr int smem_bytes() { return 6 * tile_bytes<D>() + 256 + 1024; }

struct Item {
  int kvh, start, pos0, len, n0, n1;
};

struct Args {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const int4* items;  // {first row of the prompt, first position (row), length, 0}
  int n_work;         // items * kv_heads
  int rows;           // of the packed buffers
  bool single;        // items of one query tile
  int kv_heads, group, tile_pos;  // tile_pos = 128 / group positions per tile
  float scale_log2;
  int* err;
};

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}
template <bool F16>
__device__ __forceinline__ float to_float(uint16_t u) {
  if constexpr (F16) return __half2float(__ushort_as_half(u));
  return __uint_as_float((uint32_t)u << 16);
}

// One output row by plain arithmetic, a warp together: for rows whose tiles gave
// an infinity or a NaN that they should not have. A key outside the row's range
// carries the weight 0, but 0 times an infinite or NaN v of a later or a
// neighbouring prompt's token is NaN in a matrix product; here only the row's own
// keys are touched, so what they give is the row's true result. 32 keys at a time, D / 8 lanes to a row of k
// or v: a lane multiplies its eight channels of as many keys as rows have lanes,
// the sums are passed on by halves until each lane holds one key's score, and the
// values' sums meet at the end. The weights stay float32, times 2^-32, so that no
// sum of finite values leaves the range. A score that is NaN or infinite makes the
// whole row NaN.
constexpr float kPlainShift = -32.f;

template <bool F16>
__device__ __forceinline__ void to_floats(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = to_float<F16>((uint16_t)w[k]);
    x[2 * k + 1] = to_float<F16>((uint16_t)(w[k] >> 16));
  }
}

template <int D, bool F16>
__device__ __noinline__ void plain_row(const Args& a, int start, int pos, int head) {
  constexpr int LANES = D / 8, ROWS = 32 / LANES;  // lanes of a row, rows of a load
  const int lane = threadIdx.x & 31, c = lane % LANES, g = lane / LANES;
  const int kvh = head / a.group;
  const uint16_t* k = a.k + kvh * D + 8 * c;
  const uint16_t* v = a.v + kvh * D + 8 * c;
  uint4* o = reinterpret_cast<uint4*>(a.o + (start + pos) * a.o_stride + head * D + 8 * c);
  float q[8], acc[8];
  to_floats<F16>(*reinterpret_cast<const uint4*>(a.q + (start + pos) * a.q_stride + head * D +
                                                 8 * c), q);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;  // l: of this lane's keys
  for (int j0 = 0; j0 <= pos; j0 += 32) {
    uint4 x[LANES];
#pragma unroll
    for (int t = 0; t < LANES; ++t)  // key j0 + t ROWS + g
      x[t] = *reinterpret_cast<const uint4*>(
          k + (long long)(start + min(j0 + t * ROWS + g, pos)) * a.k_stride);
    float part[LANES];
#pragma unroll
    for (int t = 0; t < LANES; ++t) {
      float y[8], s0 = 0.f, s1 = 0.f;
      to_floats<F16>(x[t], y);
#pragma unroll
      for (int e = 0; e < 8; e += 2) s0 = fmaf(q[e], y[e], s0), s1 = fmaf(q[e + 1], y[e + 1], s1);
      part[t] = s0 + s1;
    }
#pragma unroll
    for (int t = 0; t < LANES; ++t)  // asked for before the scores are needed
      x[t] = *reinterpret_cast<const uint4*>(
          v + (long long)(start + min(j0 + t * ROWS + g, pos)) * a.v_stride);
#pragma unroll
    for (int w = LANES / 2; w; w >>= 1)
#pragma unroll
      for (int t = 0; t < w; ++t) {
        const bool high = lane & w;
        const float give = high ? part[t] : part[t + w], keep = high ? part[t + w] : part[t];
        part[t] = keep + __shfl_xor_sync(0xffffffffu, give, w);
      }
    // the lane's key is j0 + c ROWS + g
    const float s = j0 + c * ROWS + g <= pos ? part[0] * a.scale_log2 : -INFINITY;
    if (__any_sync(0xffffffffu, !(s < INFINITY))) {
      const uint32_t nan = F16 ? 0x7e007e00u : 0x7fc07fc0u;
      if (g == 0) *o = make_uint4(nan, nan, nan, nan);
      return;
    }
    float to = s;
#pragma unroll
    for (int d = 16; d; d >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
    if (to > m) {
      const float alpha = exp2_mufu(m - to);
      l *= alpha;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= alpha;
      m = to;
    }
    const float p = s == -INFINITY ? 0.f : exp2_mufu(s - m + kPlainShift);
    l += p;
#pragma unroll
    for (int t = 0; t < LANES; ++t) {
      const float w = __shfl_sync(0xffffffffu, p, g * LANES + t);
      float y[8];
      to_floats<F16>(x[t], y);
      if (j0 + t * ROWS + g <= pos) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, y[e], acc[e]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
  for (int d = LANES; d < 32; d <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], d);
  if (g == 0)
    *o = make_uint4(pack2<F16>(acc[0] / l, acc[1] / l), pack2<F16>(acc[2] / l, acc[3] / l),
                    pack2<F16>(acc[4] / l, acc[5] / l), pack2<F16>(acc[6] / l, acc[7] / l));
}

// Which of eight neighbouring values are infinities or NaN, a bit for each.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite_8(const uint16_t* x) {
  constexpr uint32_t kExp = F16 ? 0x7c00u : 0x7f80u;
  const uint4 u = *reinterpret_cast<const uint4*>(x);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t bad = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if ((w[k] & kExp) == kExp) bad |= 1u << (2 * k);
    if ((w[k] >> 16 & kExp) == kExp) bad |= 2u << (2 * k);
  }
  return bad;
}

template <int D, bool F16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    k_prompt_attention(const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ Args a) {
  constexpr int TILE = tile_bytes<D>();
  constexpr int OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE, OFF_BAR = 6 * TILE;
  // fp16 P: weights are stored times 2^7 (at most 2^15 with the lazy maximum),
  // so that they stay normal numbers down to 2^-21 of the largest. bfloat16 P: times
  // 2^-24, so that up to 65536 products with the largest v stay within float32.
  constexpr float kShift = F16 ? 7.f : -24.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = a.tile_pos;
  // the w-th piece of work of this CTA; false past the last
  auto piece = [&](int w, Item& x) {
    const int i = (w & 1) ? (w + 1) * (int)gridDim.x - 1 - (int)blockIdx.x
                          : w * (int)gridDim.x + (int)blockIdx.x;
    if (i >= a.n_work) return false;
    const int item = i / a.kv_heads;
    const int4 it = __ldg(a.items + item);
    x.kvh = i - item * a.kv_heads;
    x.start = it.x;
    x.pos0 = it.y;
    x.len = it.z;
    // key tiles each query tile visits: up to its last existing position
    x.n0 = (min(x.pos0 + P, x.len) - 1) / 128 + 1;
    x.n1 = !a.single && x.pos0 + P < x.len ? (min(x.pos0 + 2 * P, x.len) - 1) / 128 + 1 : 0;
    return true;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_half[i], 4);  // one arrival per softmax warp
      mbar_init(&bars->p_full[i], 4);
      mbar_init(&bars->o_final[i], 1);
      mbar_init(&bars->o_free[i], 4);
    }
    mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{a.err, abort_flag};

  if (warp >= 8) {
    setmaxnreg_dec<kControlRegs>();
    if (warp == 8) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        int nk = 0, nv = 0, nq[2] = {0, 0};  // fills so far
        bool ok = true;
        Item x;
        for (int w = 0; ok && piece(w, x); ++w) {
          const int n = max(x.n0, x.n1);
          for (int j = 0; j < n; ++j) {
            int st = nk & 1;
            if (!mbar_wait(&bars->k_empty[st], ((nk >> 1) & 1) ^ 1, wc)) { ok = false; break; }
#ifdef H3_FAULT_INJECTION
            if (nk != *(volatile int*)&g_fault_skip_keys)
#endif
            mbar_arrive_expect_tx(&bars->k_full[st], TILE);
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(smem + OFF_K + st * TILE + h * HALF, &tk, &bars->k_full[st], 64 * h,
                          x.kvh, x.start + j * 128);
            ++nk;
            for (int i = 0; j == 0 && i < (x.n1 > 0 ? 2 : 1) && ok; ++i) {
              if (!mbar_wait(&bars->q_empty[i], (nq[i] & 1) ^ 1, wc)) { ok = false; break; }
              mbar_arrive_expect_tx(&bars->q_full[i], (D / 64) * P * a.group * 128);
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(smem + OFF_Q + i * TILE + h * HALF, &tq, &bars->q_full[i], 64 * h,
                            x.kvh * a.group, x.start + x.pos0 + i * P);
              ++nq[i];
            }
            if (!ok) break;
            st = nv & 1;
            if (!mbar_wait(&bars->v_empty[st], ((nv >> 1) & 1) ^ 1, wc)) { ok = false; break; }
            mbar_arrive_expect_tx(&bars->v_full[st], TILE);
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(smem + OFF_V + st * TILE + h * HALF, &tv, &bars->v_full[st], 64 * h,
                          x.kvh, x.start + j * 128);
            ++nv;
          }
        }
        // issued copies land before the CTA retires, whoever has given up
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) mbar_land(&bars->q_full[i], (nq[i] - 1) & 1);
        for (int j = nk > 2 ? nk - 2 : 0; j < nk; ++j)
          mbar_land(&bars->k_full[j & 1], (j >> 1) & 1);
        for (int j = nv > 2 ? nv - 2 : 0; j < nv; ++j)
          mbar_land(&bars->v_full[j & 1], (j >> 1) & 1);
      }
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_s = idesc_f16_f32(128, 128, false, false, !F16);
      constexpr uint32_t idesc_pv = idesc_f16_f32(128, D, false, true, !F16);
      constexpr uint32_t hi = sdesc_hi_sw128(1024);
      const uint32_t q_lo = sdesc_lo(smem_u32(smem + OFF_Q), 16);
      const uint32_t k_lo = sdesc_lo(smem_u32(smem + OFF_K), 16);
      const uint32_t v_lo = sdesc_lo(smem_u32(smem + OFF_V), HALF);
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc));
      };
      // One step per key tile of each item in turn, the c-th of all. Tile 0 uses a
      // step's key tile first where it visits it, tile 1 last: its range is the
      // item's (n tiles) unless it is empty, and tile 0's is that or one less.
      uint32_t p_ph[2] = {0, 0}, q_ph[2] = {0, 0}, o_ph[2] = {1, 1};  // parities to wait for
      // S_i = Q_i K^T: the tile's first and last of the item, the key tile's last use
      auto issue_s = [&](int i, int c, bool first, bool last, bool free) -> bool {
        const int st = c & 1;
        if (first) {
          if (!wait_all(&bars->q_full[i], q_ph[i])) return false;
          q_ph[i] ^= 1;
        }
        if (!wait_all(&bars->k_full[st], (c >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t kl = k_lo + st * (TILE >> 4);
        const uint32_t ql = q_lo + i * (TILE >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
          umma_ss_w_elect(tmem + i * 128, ql + off, hi, kl + off, hi, idesc_s, kk > 0 ? 1u : 0u);
        }
        umma_commit_elect(&bars->s_full[i]);
        if (free) umma_commit_elect(&bars->k_empty[st]);
        if (last) umma_commit_elect(&bars->q_empty[i]);
        return true;
      };
      // O_i += P_i V in two halves of the keys, each as soon as it is stored
      auto issue_pv = [&](int i, int c, bool first, bool last, bool free) -> bool {
        const int st = c & 1;
        if (first) {
          if (!wait_all(&bars->o_free[i], o_ph[i])) return false;
          o_ph[i] ^= 1;
        }
        if (!wait_all(&bars->p_half[i], p_ph[i])) return false;
        if (!wait_all(&bars->v_full[st], (c >> 1) & 1)) return false;
        tc_fence_after();
        const uint32_t vl = v_lo + st * (TILE >> 4);
        const uint32_t o = tmem + 256 + i * 128, p = tmem + i * 128;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ts_w_elect(o, p + kk * 8, vl + kk * (2048 >> 4), hi, idesc_pv,
                          (!first || kk > 0) ? 1u : 0u);
        if (!wait_all(&bars->p_full[i], p_ph[i])) return false;
        p_ph[i] ^= 1;
        tc_fence_after();
#pragma unroll
        for (int kk = 4; kk < 8; ++kk)
          umma_ts_w_elect(o, p + kk * 8, vl + kk * (2048 >> 4), hi, idesc_pv, 1u);
        if (free) umma_commit_elect(&bars->v_empty[st]);
        if (last) umma_commit_elect(&bars->o_final[i]);
        return true;
      };
      bool ok = true;
      Item x;
      // (the shuffles only tell the compiler that the ranges are the same in every
      // lane: its MMA operands then stay in uniform registers)
      int z0 = 0, z1 = 0;  // the next item's ranges, 0 past the last
      auto next = [&](int w) {
        const bool have = piece(w, x);
        z0 = __shfl_sync(0xffffffffu, have ? x.n0 : 0, 0);
        z1 = __shfl_sync(0xffffffffu, have ? x.n1 : 0, 0);
      };
      next(0);
      int n0 = 0, n1 = 0, c = -1;  // the item before the first
      for (int w = 1; ok && (n0 > 0 || z0 > 0); ++w) {
        // an item's last step and the next one's first scores
        const int n = max(n0, n1);
        if (n0 > 0 && n0 == n) ok = issue_pv(0, c, n == 1, true, n1 == 0);
        if (ok && z0 > 0) ok = issue_s(0, c + 1, true, z0 == 1, z1 == 0);
        if (ok && n1 > 0) ok = issue_pv(1, c, n == 1, true, true);
        if (ok && z1 > 0) ok = issue_s(1, c + 1, true, z1 == 1, true);
        if (!ok) break;
        // the next item's steps but the last
        n0 = z0;
        n1 = z1;
        next(w);
        const int m = max(n0, n1);
        ++c;
        for (int j = 0; j + 1 < m; ++j, ++c) {
          ok = issue_pv(0, c, j == 0, j + 1 == n0, n1 == 0);
          if (ok && j + 1 < n0) ok = issue_s(0, c + 1, false, j + 2 == n0, n1 == 0);
          if (n1 > 0) {
            if (ok) ok = issue_pv(1, c, j == 0, false, true);
            if (ok) ok = issue_s(1, c + 1, false, j + 2 == n1, true);
          }
          if (!ok) break;
        }
      }
      umma_commit_elect(&bars->drain);  // every MMA issued is complete past this point
      mbar_drain(&bars->drain, 0);
    }
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax (warps 0..7)
    const int i = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;  // row in the tile = TMEM lane
    const int rp = r / a.group;         // its position in the tile, its head in the group
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lane_base + i * 128;
    const uint32_t o_col = lane_base + 256 + i * 128;
    const uint64_t scale2 = f2_pack(a.scale_log2, a.scale_log2);
    bool ok = true;
    uint32_t marked = 0;  // bit w % 32: piece w has rows with an infinity or a NaN
    int done = 0, rounds = 0;  // score tiles, and items with work, so far
    Item x;
    for (int w = 0; ok && piece(w, x); ++w) {
    const int my_n = i == 0 ? x.n0 : x.n1;
    if (my_n == 0) continue;
    const int tile0 = x.pos0 + i * P, pos = tile0 + rp;
    float m_run = -INFINITY, l_run = 0.f;
    for (int j = 0; j < my_n; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(&bars->s_full[i], (done + j) & 1, wc))) {
        ok = false;
        break;
      }
      tc_fence_after();
      float sc[128];
      {
        uint32_t rr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, rr[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) sc[32 * c + e] = __uint_as_float(rr[c][e]);
      }
      if (128 * j + 127 > tile0) {  // the diagonal: keys after the row's own position
        const int last = pos - 128 * j;
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e > last) sc[e] = -INFINITY;
      }
      float pm[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) pm[k] = max3(sc[2 * k], sc[2 * k + 1], sc[16 + 2 * k]);
#pragma unroll
      for (int e = 32; e < 128; e += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k) pm[k] = max3(pm[k], sc[e + 2 * k], sc[e + 2 * k + 1]);
#pragma unroll
      for (int k = 0; k < 8; ++k) pm[k] = fmaxf(pm[k], sc[16 + 2 * k + 1]);
      float mx = max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
      mx *= a.scale_log2;
      // O_i is stable here: the commit that signalled S_i(j) follows PV_i(j-1).
      const bool need = mx > m_run + kLazyRescale;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? mx : m_run;
        if (j > 0) {
          const float alpha = need ? exp2_mufu(m_run - m_new) : 1.f;
          l_run *= alpha;
          uint32_t rr[32];
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            tmem_ld32(o_col + 32 * c, rr);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st32(o_col + 32 * c, rr);
          }
        }
        m_run = m_new;
      }
      // P = 2^(s * scale - m + shift) in the type of v, over S columns already
      // held in registers, in two halves (one arrival per warp each).
      // (Scores that are all -inf so far have weight 0.)
      const float sub = kShift - (m_run == -INFINITY ? 0.f : m_run);
      const uint64_t negm2 = f2_pack(sub, sub);
      uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int key = 64 * h + 2 * e;
          const uint64_t x2 = f2_fma(f2_pack(sc[key], sc[key + 1]), scale2, negm2);
          float p0, p1;
          if ((kCubicPairs >> e) & 1u) {
            f2_unpack(x2, p0, p1);
            exp2_cubic2_clamped(f2_pack(max_nan(p0, kExpLowest), max_nan(p1, kExpLowest)),
                                Cubic{kExpC3, kExpC2, kExpC1, kExpC0, kRoundMagic}, p0, p1);
          } else {
            f2_unpack(x2, p0, p1);
            p0 = exp2_mufu(p0);
            p1 = exp2_mufu(p1);
          }
          sum2[e & 3] = f2_add(sum2[e & 3], f2_pack(p0, p1));
          pk[e] = pack2<F16>(p0, p1);
        }
        tmem_st32(s_col + 32 * h, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(h == 0 ? &bars->p_half[i] : &bars->p_full[i]);
      }
      float a0, a1, b0, b1;
      f2_unpack(f2_add(sum2[0], sum2[1]), a0, a1);
      f2_unpack(f2_add(sum2[2], sum2[3]), b0, b1);
      // A NaN or an infinity among the tile's own scores makes weights NaN, or the
      // largest number by the cubic; from here on the row's sum is NaN, whatever the
      // running maximum does.
      const float sum = (a0 + a1) + (b0 + b1);
      l_run += sum < 1e37f ? sum : __int_as_float(0x7fc00000);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_final[i], rounds & 1, wc));
    if (!ok) break;
    done += my_n;
    ++rounds;
    tc_fence_after();
    const int head = x.kvh * a.group + r - rp * a.group;
    const bool row_ok = rp < P && pos < x.len;
    const bool scores_ok = l_run >= 0.f;  // else the row is NaN, and needs no other look
    const float inv_l = 1.f / l_run;
    // A row's 64 bytes at a time; four lanes turn their pieces of 16 so that a
    // store covers 64 bytes of eight rows instead of 16 of 32.
    const long long mine = row_ok ? (x.start + pos) * a.o_stride + head * D : -1;
    long long dst[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[k] = __shfl_sync(0xffffffffu, mine, (lane & 28) + k);
    const bool odd = lane & 1, high = lane & 2;
    float worst = 0.f;  // NaN or infinite if any value of the row is
    uint32_t rr[32];
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      tmem_ld32(o_col + 32 * c, rr);
      tmem_wait_ld();
      if (c == D / 32 - 1) {  // the row is in registers: the accumulator may go
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free[i]);
      }
      uint32_t u[4][4];  // [piece][word]
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v0 = __uint_as_float(rr[2 * e]) * inv_l;
        const float v1 = __uint_as_float(rr[2 * e + 1]) * inv_l;
        worst = max_nan(worst, fabsf(v0));
        worst = max_nan(worst, fabsf(v1));
        u[e / 4][e % 4] = pack2<F16>(v0, v1);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int h = 0; h < 4; h += 2) {  // lanes l and l ^ 1: pieces h, h + 1
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? u[h][k] : u[h + 1][k], 1);
          if (odd) u[h][k] = got; else u[h + 1][k] = got;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // lanes l and l ^ 2: pieces h, h + 2
          const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? u[h][k] : u[h + 2][k], 2);
          if (high) u[h][k] = got; else u[h + 2][k] = got;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)  // piece lane % 4 of row k of the four
        if (dst[k] >= 0)
          *reinterpret_cast<uint4*>(a.o + dst[k] + 32 * c + 8 * (lane & 3)) =
              make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
    }
    if (__any_sync(0xffffffffu, row_ok && scores_ok && !(worst <= 3.4028235e38f)))
      marked |= 1u << (w & 31);
    }
    // A row with an infinity or a NaN is computed again if a v outside its range has
    // one too, in the same channel and in a key tile that the row's tile visits. (Any
    // other comes from the row's own keys.) That happens when no other warp waits for
    // this one any more, so that no wait runs out over it, however long the prompts.
    // 8192 tokens, 56 heads over 8 x 128: 0.82 ms without a bad v, 0.87 with one at
    // token 3, 8.4 at token 4000, 16 at token 8000 (32 rows of a warp over all keys).
    __syncwarp();  // rows are stored by other lanes: that comes before
    for (int w = 0; ok && marked != 0 && piece(w, x); ++w) {
      const int tiles = i == 0 ? x.n0 : x.n1;
      if ((marked >> (w & 31) & 1) == 0 || tiles == 0) continue;
      const int tile0 = x.pos0 + i * P, pos = tile0 + rp;
      const int head = x.kvh * a.group + r - rp * a.group;
      const bool row_ok = rp < P && pos < x.len;
      const int end = min(tiles * 128, a.rows - x.start);
      bool again = false;
      for (int c = 0; c < D; c += 8) {
        const uint32_t mine =
            row_ok ? not_finite_8<F16>(a.o + (x.start + pos) * a.o_stride + head * D + c) : 0;
        if (!__any_sync(0xffffffffu, mine != 0)) continue;
        int last[8];  // the last key with a bad v, of each channel
#pragma unroll
        for (int e = 0; e < 8; ++e) last[e] = -1;
        for (int j0 = tile0; j0 < end; j0 += 32) {
          const int j = j0 + lane;
          const uint32_t bad =
              j < end ? not_finite_8<F16>(a.v + (x.start + j) * a.v_stride + x.kvh * D + c) : 0;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            last[e] = max(last[e], __reduce_max_sync(0xffffffffu, (bad >> e & 1) ? j : -1));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) again |= (mine >> e & 1) && last[e] > pos;
      }
      uint32_t rows = __ballot_sync(0xffffffffu, again);
      while (rows) {
        const int src = __ffs(rows) - 1;
        rows &= rows - 1;
        plain_row<D, F16>(a, x.start, __shfl_sync(0xffffffffu, pos, src),
                          __shfl_sync(0xffffffffu, head, src));
      }
    }
  }
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

bool tmap_heads(CUtensorMap* t, const void* p, bool f16, int D, int heads, int rows,
                int64_t stride, int box_heads, int box_rows) {
  const uint64_t d[3] = {(uint64_t)D, (uint64_t)heads, (uint64_t)rows};
  const uint64_t s[2] = {(uint64_t)D * 2, (uint64_t)stride * 2};
  const uint32_t b[3] = {64, (uint32_t)box_heads, (uint32_t)box_rows};
  return make_tmap(t, p, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   3, d, s, b);
}

// ---------------------------------------------------------- short prompts only
// Where every prompt has at most 256 tokens the time is a chain of latencies, and
// the form above makes it long: one item at a time per SM, its tiles mostly empty.
// Here a thread block takes 64 (position, head) rows of a prompt and kv head, many
// per SM; keys and values up to its last row's position go to shared memory at
// once, and each of four warps takes 16 rows through warp-level MMAs, 32 keys at a
// time with a running maximum and sum.
constexpr int kShortKeys = 256;  // the longest prompt of a batch that comes here
constexpr int kShortRows = 64;

__device__ __forceinline__ void copy_16(uint32_t dst, const void* src, bool there) {
  const int bytes = there ? 16 : 0;  // the rest of 16 becomes 0
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool F16>
__global__ void __launch_bounds__(128) k_short_prompts(const __grid_constant__ Args a) {
  constexpr int CH = D / 8;                      // 16-byte chunks of a row
  constexpr float kShift = F16 ? 7.f : 0.f;      // as above
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t smem = smem_u32(smem_raw);
  const int item = blockIdx.x / a.kv_heads, kvh = blockIdx.x - item * a.kv_heads;
  const int4 it = __ldg(a.items + item);
  const int start = it.x, r0 = it.y, total = it.z * a.group;  // rows of the prompt and kv head
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int keys = (min(r0 + kShortRows, total) - 1) / a.group + 1, padded = (keys + 31) & ~31;
  // rows of D elements, a chunk's place XORed by its row, against bank conflicts
  auto place = [&](int row, int chunk) { return (row * CH + (chunk ^ (row & 7))) * 16; };
  const uint32_t sk = smem + kShortRows * D * 2, sv = sk + padded * D * 2;
  {
    const int c = threadIdx.x % CH;
    for (int row = threadIdx.x / CH; row < kShortRows; row += 128 / CH) {
      const int r = min(r0 + row, total - 1), pos = r / a.group;
      copy_16(smem + place(row, c),
              a.q + (start + pos) * a.q_stride + (kvh * a.group + r - pos * a.group) * D + 8 * c,
              r0 + row < total);
    }
    for (int row = threadIdx.x / CH; row < padded; row += 128 / CH) {
      const long long from = start + min(row, keys - 1);
      copy_16(sk + place(row, c), a.k + from * a.k_stride + kvh * D + 8 * c, row < keys);
      copy_16(sv + place(row, c), a.v + from * a.v_stride + kvh * D + 8 * c, row < keys);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  const int first = r0 + 16 * warp;  // the warp's rows; lane / 4 and that plus 8 are a lane's
  if (first >= total) return;
  const int pos[2] = {(first + (lane >> 2)) / a.group, (first + (lane >> 2) + 8) / a.group};
  const int last = (min(first + 16, total) - 1) / a.group;

  uint32_t q[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    ldmatrix4<false>(smem + place(16 * warp + (lane & 15), 2 * k + (lane >> 4)), q[k]);
  float acc[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
  for (int key0 = 0; key0 <= last; key0 += 32) {
    float s[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int n = 0; n < 4; n += 2) {
        uint32_t b[4];
        ldmatrix4<false>(sk + place(key0 + 8 * n + (lane & 7) + (lane >> 4) * 8,
                                    2 * k + ((lane >> 3) & 1)), b);
        mma_16816<F16>(s[n], q[k], b[0], b[1]);
        mma_16816<F16>(s[n + 1], q[k], b[2], b[3]);
      }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] *= a.scale_log2;
        if (key0 + 8 * n + 2 * (lane & 3) + (e & 1) > pos[e >> 1]) s[n][e] = -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
    float by[2], sub[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      by[h] = exp2_mufu(m[h] - mx[h]);
      m[h] = mx[h];
      sub[h] = kShift - mx[h];
      l[h] *= by[h];
    }
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] *= by[e >> 1];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2_mufu(s[n][e] + sub[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t p[4] = {
          pack2<F16>(s[2 * j][0], s[2 * j][1]), pack2<F16>(s[2 * j][2], s[2 * j][3]),
          pack2<F16>(s[2 * j + 1][0], s[2 * j + 1][1]),
          pack2<F16>(s[2 * j + 1][2], s[2 * j + 1][3])};
#pragma unroll
      for (int n = 0; n < D / 8; n += 2) {
        uint32_t b[4];
        ldmatrix4<true>(sv + place(key0 + 16 * j + (lane & 15), n + (lane >> 4)), b);
        mma_16816<F16>(acc[n], p, b[0], b[1]);
        mma_16816<F16>(acc[n + 1], p, b[2], b[3]);
      }
    }
  }
  // out through the warp's own q rows
  float worst[2] = {0.f, 0.f};  // NaN or infinite if any value of the row is
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    const float inv = 1.f / l[h];
    const int row = 16 * warp + (lane >> 2) + 8 * h;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      const float x = acc[n][2 * h] * inv, y = acc[n][2 * h + 1] * inv;
      worst[h] = max_nan(worst[h], max_nan(fabsf(x), fabsf(y)));
      *reinterpret_cast<uint32_t*>(smem_raw + place(row, n) + 4 * (lane & 3)) = pack2<F16>(x, y);
    }
  }
  __syncwarp();
  for (int i = lane; i < 16 * CH; i += 32) {
    const int row = i / CH, c = i % CH, r = first + row, at = r / a.group;
    if (r < total)
      *reinterpret_cast<uint4*>(a.o + (start + at) * a.o_stride +
                                (kvh * a.group + r - at * a.group) * D + 8 * c) =
          *reinterpret_cast<const uint4*>(smem_raw + place(16 * warp + row, c));
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t again = __ballot_sync(0xffffffffu, !(worst[h] <= 3.4028235e38f));
    for (int g = 0; g < 8; ++g) {
      const int r = first + g + 8 * h;
      if ((again >> (4 * g) & 15u) == 0 || r >= total) continue;
      plain_row<D, F16>(a, start, r / a.group, kvh * a.group + r % a.group);
    }
  }
}

template <int D, bool F16>
cudaError_t run_short(const h3_prompts* p, const Args& a, cudaStream_t st) {
  constexpr int most = (kShortRows + 2 * kShortKeys) * D * 2;
  cudaError_t e = cudaFuncSetAttribute(k_short_prompts<D, F16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  const int bytes = (kShortRows + 2 * ((p->longest + 31) & ~31)) * D * 2;
  k_short_prompts<D, F16><<<(unsigned)a.n_work, 128, bytes, st>>>(a);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t run(const h3_prompts* p, const Args& a, cudaStream_t st) {
  if (p->brief) return run_short<D, F16>(p, a, st);
  cudaError_t e = cudaFuncSetAttribute(k_prompt_attention<D, F16>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes<D>());
  if (e != cudaSuccess) return e;
  CUtensorMap tq, tk, tv;
  if (!tmap_heads(&tq, a.q, F16, D, p->q_heads, p->rows, a.q_stride, a.group, a.tile_pos) ||
      !tmap_heads(&tk, a.k, F16, D, p->kv_heads, p->rows, a.k_stride, 1, 128) ||
      !tmap_heads(&tv, a.v, F16, D, p->kv_heads, p->rows, a.v_stride, 1, 128))
    return cudaErrorInvalidValue;
  const int ctas = a.n_work < num_sms() ? a.n_work : num_sms();
  k_prompt_attention<D, F16><<<(unsigned)ctas, NUM_THREADS, smem_bytes<D>(), st>>>(tq, tk, tv, a);
  return cudaGetLastError();
}

// Of a batch of short prompts: nanoseconds of the chip, from measurements. A thread
// block of the short form costs with its keys and channels, an item of the other 20
// or 30, and 2.3 us more come before and behind its items. (64 prompts of 3 to 77
// tokens, 14 heads over 2 x 64: 6.3 us against 10.2; 31 of 8, 40 over 8 x 64: 4.6
// against 9.2; 32 of 100, 40 over 8 x 128: 48 against 24; one of 256, 40 over 8 x 64:
// 8.3 against 8.7.)
bool short_is_faster(const h3_prompts* p, long long pairs, long long blocks) {
  return p->kv_heads * blocks * (p->head_dim / 64) * (4.5 + 0.05 * p->longest) <
         p->kv_heads * pairs * (p->head_dim == 128 ? 30. : 20.) + 2300.;
}

}  // namespace

h3_status build_prompts(h3_prompts* p, const int32_t* offsets, int n_prompts) {
  // an item: two query tiles of 128 / group positions, one, or kShortRows rows
  const int group = p->q_heads / p->kv_heads, tile = 128 / group;
  long long pairs = 0, tiles = 0, blocks = 0;
  for (int i = 0; i < n_prompts; ++i) {
    const long long len = (long long)offsets[i + 1] - offsets[i];
    p->longest = std::max(p->longest, (int)len);
    pairs += (len + 2 * tile - 1) / (2 * tile);
    tiles += (len + tile - 1) / tile;
    blocks += (len * group + kShortRows - 1) / kShortRows;
  }
  p->brief = p->longest <= kShortKeys && short_is_faster(p, pairs, blocks);
  const long long work = (p->brief ? blocks : pairs) * p->kv_heads;
  if (work > 0x7fff0000LL) return H3_ERR_SHAPE;  // rounds of the grid fit an int
  if (work == 0) return H3_OK;
  const int ctas = num_sms();
  std::vector<int4> items, other;
  auto list = [&](std::vector<int4>& to, int step) {
    for (int i = 0; i < n_prompts; ++i) {
      const int len = offsets[i + 1] - offsets[i];
      for (long long pos = 0; pos < (long long)len * (p->brief ? group : 1); pos += step)
        to.push_back(make_int4(offsets[i], (int)pos, len, 0));
    }
    std::stable_sort(to.begin(), to.end(),
                     [](const int4& x, const int4& y) { return x.y > y.y; });
  };
  // the longest that a CTA takes, in steps of two tiles
  auto span = [&](const std::vector<int4>& of, int step, double cost) {
    std::vector<double> busy(ctas, 0.);
    long long i = 0;
    for (const int4& it : of)
      for (int h = 0; h < p->kv_heads; ++h, ++i) {
        const int at = (int)(i % ctas);
        const int keys = (int)std::min<long long>((long long)it.y + step, it.z);
        busy[(i / ctas) & 1 ? ctas - 1 - at : at] += ((keys - 1) / 128 + 1) * cost + 0.8;
      }
    return *std::max_element(busy.begin(), busy.end());
  };
  try {
    list(items, p->brief ? kShortRows : 2 * tile);
    // A step of one tile takes 0.86 of one of two: less time where there are few items
    // (one prompt of 2000 tokens, 16 heads over 4 x 128: 31 us against 35; 40 over 8:
    // 75 against 50).
    if (!p->brief && tiles * p->kv_heads <= 4ll * ctas) {
      list(other, tile);
      if (span(other, tile, 0.86) < span(items, 2 * tile, 1.)) {
        items.swap(other);
        p->single = true;
      }
    }
  } catch (...) {
    return H3_ERR_CUDA;
  }
  const size_t count = items.size();
  p->n_items = (int)count;
  if (cudaMalloc(&p->items, count * sizeof(int4)) != cudaSuccess) return H3_ERR_CUDA;
  // the copy may still be under way when cudaMemcpy returns, and a stream that
  // does not follow the default one would not wait for it
  if (cudaMemcpy(p->items, items.data(), count * sizeof(int4), cudaMemcpyHostToDevice) !=
          cudaSuccess ||
      cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) {
    cudaFree(p->items);
    p->items = nullptr;
    return H3_ERR_CUDA;
  }
  return H3_OK;
}

cudaError_t launch_prompt_attention(const h3_prompts* p, bool f16, const void* q,
                                    int64_t q_stride, const void* k, int64_t k_stride,
                                    const void* v, int64_t v_stride, float scale, void* o,
                                    int64_t o_stride, int* err, cudaStream_t st) {
  Args a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.o = static_cast<uint16_t*>(o);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.o_stride = o_stride;
  a.items = static_cast<const int4*>(p->items);
  a.n_work = p->n_items * p->kv_heads;
  a.rows = p->rows;
  a.kv_heads = p->kv_heads;
  a.group = p->q_heads / p->kv_heads;
  a.tile_pos = 128 / a.group;
  a.single = p->single;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = err;
  if (p->head_dim == 128) return f16 ? run<128, true>(p, a, st) : run<128, false>(p, a, st);
  return f16 ? run<64, true>(p, a, st) : run<64, false>(p, a, st);
}

}  // namespace h3

#ifdef H3_FAULT_INJECTION
extern "C" __attribute__((visibility("default"))) int h3_test_prompt_skip_keys(int tile) {
  return cudaMemcpyToSymbol(h3::g_fault_skip_keys, &tile, sizeof(int)) == cudaSuccess ? 0 : -1;
}
#endif
