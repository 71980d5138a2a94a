// attend_back_few.cu -- attention backward when a bag has few query rows
// (queries times heads of a group <= 64): one pass over the keys.
//
//   p = exp(s - lse), dp = dO V^T, ds = p (dp - delta), delta = sum(dO * O),
//   dV = p^T dO,  dK = scale ds^T Q,  dQ = scale ds K.
//
// With all the bag's rows in one tile, a key tile's dK and dV need no sum over
// query tiles, and the scores are computed once: K and V are read once, dK and
// dV written once, which is what bounds this pass.  A block takes the rows of
// one key head and a part of the bag's keys, 128 keys a step:
//
//   S^T = K Q^T, dP^T = V dO^T      (128 keys x NR rows, tensor memory)
//   P^T, dS^T as 16-bit values over them; dS also to shared memory
//   dV = P^T dO, dK = dS^T Q        (128 keys x D), stored
//   dQ += dS K                      (NR rows x D, kept in tensor memory)
//
// Measured on B200: 256 bags of 0-16 queries over 1000-5000 keys, 2 heads of 64,
// 161-181 us with the join (4.9 to 4.3 TB/s of K, V, dK and dV); one query, 8 heads of
// 128 over 2, 303 us (one block an SM, and the chain of a tile's steps shows).
//
// Bags of few keys (SPLIT, as in the other backward) have dS go into its products
// as two 16-bit values, its rounding and what that leaves out: for dQ the second
// values are rows NR .. 2 NR - 1 of the 128 that a product takes anyway, for dK a
// product of NR more values.  (On long bags, where it is not needed, it takes 170
// us instead of 152 for 0-16 queries over 256 bags of 1000-5000 keys.)
//
// fp16 (kShiftP in attend.cuh): ds takes a power of two of the block's own that
// follows its largest |ds| so far.  When a tile passes what fp16 holds, all compute
// warps lower the power, and dQ in tensor memory with it; the barrier that every
// tile has before P and dS are stored carries the question.  (One query, 8 heads of
// 128 over 2: 306 us, bf16 303; up to 64 rows of 64: 101 and 99.)
//
// While the compute warps store dV and dK of one tile, the scores of the next
// are made; the copies run further ahead.  Parts of dQ (several blocks a bag)
// are joined in order by join_q_kernel.
#include <algorithm>
#include <type_traits>

#include "attend.cuh"
#include "tc.cuh"

namespace recis {

namespace {

constexpr int kKeys = 128;
constexpr int kCompute = 256;
constexpr int kThreads = kCompute + 64;

template <int DP, int NR>
struct FewBackCfg {
  static constexpr bool kTwo = DP == 64 && NR <= 32;   // two blocks an SM
  static constexpr int kBlocks = DP / 64;
  static constexpr int kTile = kBlocks * kKeys * 128;  // K or V
  static constexpr int kRows = kBlocks * NR * 128;     // Q or dO
  static constexpr int kStages = DP == 64 && !kTwo ? 4 : 2;
  static constexpr uint32_t kDp = kTwo ? 32 : 64, kDv = 2 * kDp, kDk = kDv + DP, kDq = kDk + DP;
  static constexpr uint32_t kCols = kTwo ? 256 : 512;
  // K and V stages, dS [128 rows][128 keys], Q, dO, alignment, barriers, lse, delta
  static constexpr int kTotal = 2 * kStages * kTile + 2 * 16384 + 2 * kRows + 1024 + 128 + 2 * NR * 4;
};

// fp16: the power of two that dS begins with, above any tile's; `scale` and what
// takes it and P's out of the accumulators
constexpr int kHalfUp = 60;
template <typename T>
__device__ __forceinline__ float half_down(int up, float scale) {
  return kShiftP<T> > 0 ? pow2_times(-up - kShiftP<T>, scale) : scale;
}
// whether a pair of halves holds an infinity (NaN aside)
template <int N>
__device__ __forceinline__ bool any_infinite(const uint32_t (&v)[N]) {
  __half2 m = __float2half2_rn(0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&v[i])));
  return __hisinf(__low2half(m)) || __hisinf(__high2half(m));
}
// whether `v` holds in any compute thread; a barrier of them all
__device__ __forceinline__ bool block_any(bool v) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 5, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"((uint32_t)v), "n"(kCompute)
      : "memory");
  return any != 0;
}

struct FewMaps {
  CUtensorMap q, o, k, v;  // o: grad_out
};

// One block's work: the rows of key head h of a bag against part sp of its keys
template <typename T, int DP, int NR, bool SPLIT>
__device__ __forceinline__ void few_back_block(const AttendParams& p, const FewMaps& maps, int spin_max, const Bag& bag,
                                               int h, int sp) {
  using C = FewBackCfg<DP, NR>;
  constexpr int NS = C::kStages, H = NR / 2;  // H: columns a compute warpgroup takes
  extern __shared__ uint8_t s_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *skv = base, *sds = skv + 2 * NS * C::kTile, *sq = sds + 2 * 16384, *so = sq + C::kRows;
  uint64_t* bar = reinterpret_cast<uint64_t*>(so + C::kRows);
  uint64_t *q_raw = bar, *q_full = bar + 1, *s_full = bar + 2, *e_full = bar + 3, *o_full = bar + 4, *all_done = bar + 5;
  uint64_t *kv_full = bar + 6, *kv_empty = kv_full + NS;
  float* s_lse = reinterpret_cast<float*>(so + C::kRows + 128);  // [NR] lse * log2(e) - kShiftP
  float* s_delta = s_lse + NR;                                   // [NR] delta (fp16: times ds's scale)
  __shared__ uint32_t s_tmem;
  __shared__ float s_max[kCompute / 32];

  const int rows = bag.nq * p.G;  // <= NR
  const int ks = sp * p.split_keys, ke = min(ks + p.split_keys, bag.nk);
  if (sp > 0 && ks >= bag.nk) return;
  const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (rows == 0) {  // keys without queries: zero gradients
    // a thread keeps its piece of the rows: the pieces of all rows may pass 2^31
    const int per = p.D / 8, step = kThreads / per, d = tid % per * 8;
    for (int i = tid < step * per ? tid / per : ke - ks; i < ke - ks; i += step) {
      const int64_t t = bag.k0 + ks + i;
      *reinterpret_cast<uint4*>(static_cast<T*>(p.gk) + t * p.gks + h * p.gkh + d) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(static_cast<T*>(p.gv) + t * p.gvs + h * p.gvh + d) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int n = ke > ks ? (ke - ks + kKeys - 1) / kKeys : 0;

  constexpr int kLoader = kCompute / 32, kIssuer = kLoader + 1;
  if (w == kIssuer) tmem_alloc(&s_tmem, C::kCols);
  if (tid == kLoader * 32) {
    mbar_init(q_raw, 1);
    mbar_init(q_full, 1);
    mbar_init(s_full, 1);
    mbar_init(e_full, kCompute);
    mbar_init(o_full, 1);
    mbar_init(all_done, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;  // false: a wait gave up

  if (w == kLoader) {
    if (n > 0) {
      int asked = 0;
      auto ask = [&](int j) {
        const int st = j % NS, row = (int)(bag.k0 + ks + j * kKeys);
        uint8_t* at = skv + 2 * st * C::kTile;
        mbar_arrive_expect(kv_full + st, 2 * C::kTile);
        for (int i = 0; i < C::kBlocks; ++i) {
          tma_load3(at + i * kKeys * 128, &maps.k, 64 * i, h, row, kv_full + st);
          tma_load3(at + C::kTile + i * kKeys * 128, &maps.v, 64 * i, h, row, kv_full + st);
        }
        asked = j + 1;
      };
      if (lane == 0) {
        mbar_arrive_expect(q_raw, (unsigned)(2 * C::kBlocks * p.max_q * p.G * 128));
        for (int i = 0; i < C::kBlocks; ++i) {
          tma_load3(sq + i * NR * 128, &maps.q, 64 * i, h * p.G, (int)bag.q0, q_raw);
          tma_load3(so + i * NR * 128, &maps.o, 64 * i, h * p.G, (int)bag.q0, q_raw);
        }
        for (int j = 0; j < min(n, NS); ++j) ask(j);
      }
      ok = mbar_wait(q_raw, 0, spin_max);
      for (int r = rows + lane; r < NR; r += 32)  // rows of other bags, or of none
        for (int i = 0; i < C::kBlocks; ++i)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            reinterpret_cast<uint4*>(sq + (i * NR + r) * 128)[u] = make_uint4(0, 0, 0, 0);
            reinterpret_cast<uint4*>(so + (i * NR + r) * 128)[u] = make_uint4(0, 0, 0, 0);
          }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(q_full);
        for (int j = NS; j < n && ok; ++j) {
          if (!(ok = mbar_wait(kv_empty + j % NS, ((j / NS) & 1) ^ 1, spin_max))) break;
          ask(j);
        }
        // copies in flight end before the block does
        for (int j = max(asked - NS, 0); j < asked; ++j) ok = mbar_wait(kv_full + j % NS, (j / NS) & 1, spin_max) && ok;
      }
      __syncwarp();
    }
  } else if (w == kIssuer) {
    if (n > 0) {
      constexpr uint32_t id_s = mma_desc<T>(kKeys, NR, false, false), id_o = mma_desc<T>(kKeys, DP, false, true);
      // descriptors count 16 bytes
      const uint64_t dq = smem_desc(smem_u32(sq), 16), dg = smem_desc(smem_u32(so), 16);
      const uint64_t tq = smem_desc(smem_u32(sq), NR * 128), tg = smem_desc(smem_u32(so), NR * 128);
      const uint64_t dds = smem_desc(smem_u32(sds), 16);
      const uint64_t dkv = smem_desc(smem_u32(skv), 16), tkv = smem_desc(smem_u32(skv), kKeys * 128);
      const bool one = elect_one();
      auto scores = [&](int j) {
        const int st = j % NS;
        if (!warp_wait(kv_full + st, (j / NS) & 1, spin_max)) return false;
        tc_fence_after();
        const uint64_t dk = dkv + st * (2 * C::kTile >> 4), dv = dk + (C::kTile >> 4);
        if (one) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(tmem, dk + (((k >> 2) * kKeys * 128 + (k & 3) * 32) >> 4),
                   dq + (((k >> 2) * NR * 128 + (k & 3) * 32) >> 4), id_s, k > 0);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(tmem + C::kDp, dv + (((k >> 2) * kKeys * 128 + (k & 3) * 32) >> 4),
                   dg + (((k >> 2) * NR * 128 + (k & 3) * 32) >> 4), id_s, k > 0);
          mma_commit(s_full);
        }
        __syncwarp();
        return true;
      };
      ok = warp_wait(q_full, 0, spin_max) && scores(0);
      for (int j = 0; j < n && ok; ++j) {
        const uint64_t tk = tkv + (j % NS) * (2 * C::kTile >> 4);
        if (!(ok = warp_wait(e_full, j & 1, spin_max))) break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int k = 0; k < NR / 16; ++k) mma_ts(tmem + C::kDv, tmem + 8 * k, tg + (k * 2048 >> 4), id_o, k > 0);
#pragma unroll
          for (int k = 0; k < NR / 16; ++k)
            mma_ts(tmem + C::kDk, tmem + C::kDp + 8 * k, tq + (k * 2048 >> 4), id_o, k > 0);
#pragma unroll
          for (int k = 0; SPLIT && k < NR / 16; ++k)
            mma_ts(tmem + C::kDk, tmem + C::kDp + NR / 2 + 8 * k, tq + (k * 2048 >> 4), id_o, true);
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            mma_ss(tmem + C::kDq, dds + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), tk + (k * 2048 >> 4), id_o,
                   j > 0 || k > 0);
          mma_commit(o_full);
          mma_commit(kv_empty + j % NS);
        }
        __syncwarp();
        if (j + 1 < n) ok = scores(j + 1);
      }
      if (one) mma_commit(all_done);
      ok = warp_wait(all_done, 0, spin_max) && ok;
    }
    __syncwarp();
  } else {
    const int wg = w >> 2, key = tid & 127;
    const uint32_t mine = tmem + ((uint32_t)(w & 3) << 21);
    // the rows' lse and delta
    for (int r = w; r < NR; r += kCompute / 32) {
      float lse = INFINITY, s = 0.f;
      if (r < rows) {
        const int64_t t = bag.q0 + r / p.G;
        const int hq = h * p.G + r % p.G, d = lane * 4;
        if (d < p.D) {
          const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.out) + t * p.os + hq * p.oh + d);
          const uint2 y = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.go) + t * p.gos + hq * p.goh + d);
          const float2 x0 = unpack2<T>(x.x), x1 = unpack2<T>(x.y), y0 = unpack2<T>(y.x), y1 = unpack2<T>(y.y);
          s = x0.x * y0.x + x0.y * y0.y + x1.x * y1.x + x1.y * y1.y;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        lse = fmaf(p.lse[t * p.Hq + hq], 1.4426950408889634f, -(float)kShiftP<T>);
        if (lse == -INFINITY) lse = INFINITY;  // a row without keys: p = 0
      }
      if (lane == 0) {
        s_lse[r] = lse;
        s_delta[r] = kShiftP<T> > 0 ? s * pow2(kHalfUp) : s;
      }
    }
    asm volatile("bar.sync 5, 256;" ::: "memory");
    const float c = p.scale_log2;
    // where the thread's key lies in dS's rows: its 16-byte chunk is swizzled by the row
    uint8_t* ds_at = sds + (key >> 6) * 16384 + (key & 7) * 2;
    const int chunk = (key & 63) >> 3;
    // whether the thread's key of tile j takes part: not 0 (the byte is not looked at before its turn)
    auto mask_at = [&](int j) -> unsigned {
      const int i = ks + j * kKeys + key;
      unsigned m = i < ke;
      if (m && p.mask) m = __ldg(p.mask + bag.k0 + i);
      return m;
    };
    unsigned takes_next = mask_at(0);
    int up = kHalfUp;  // fp16: ds 2^(up + kShiftP) is what is rounded
    float scaled = kShiftP<T> > 0 ? pow2(kHalfUp) : 1.f;  // 2^up
    for (int j = 0; j < n; ++j) {
      const int k0 = ks + j * kKeys;
      const bool takes = takes_next != 0;
      takes_next = mask_at(j + 1);
      // a warp that gave up goes on without waiting: the block's barriers need it
      ok = ok && mbar_wait(s_full, j & 1, spin_max);
      __syncwarp();
      tc_fence_after();
      uint32_t s[H], d[H], pk[H / 2], dk[H / 2], dl[H / 2];
      tmem_ld(mine + wg * H, s);
      tmem_ld(mine + C::kDp + wg * H, d);
      tmem_wait_ld();
      // both warps of these lanes have read before P and dS go over S and dP (fp16: all warps, below)
      if (kShiftP<T> == 0) asm volatile("bar.sync %0, 64;" ::"r"(1 + (w & 3)) : "memory");
      float f[H];
#pragma unroll
      for (int i = 0; i < H; i += 4) {
        const float4 ls = *reinterpret_cast<const float4*>(s_lse + wg * H + i);
        const float4 de = *reinterpret_cast<const float4*>(s_delta + wg * H + i);
        const float l4[4] = {ls.x, ls.y, ls.z, ls.w}, d4[4] = {de.x, de.y, de.z, de.w};
        float e[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float dp = __uint_as_float(d[i + u]);
          e[u] = ex2(fmaf(__uint_as_float(s[i + u]), c, -l4[u]));
          f[i + u] = takes ? e[u] * (kShiftP<T> > 0 ? fmaf(dp, scaled, -d4[u]) : dp - d4[u]) : 0.f;
        }
        pk[i / 2] = pack2<T>(e[0], e[1]);
        pk[i / 2 + 1] = pack2<T>(e[2], e[3]);
        dk[i / 2] = pack2<T>(f[i], f[i + 1]);
        dk[i / 2 + 1] = pack2<T>(f[i + 2], f[i + 3]);
      }
      if constexpr (kShiftP<T> > 0) {
        if (block_any(any_infinite(dk))) {
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < H; ++i) most = finite_max(most, fabsf(f[i]));
          most = warp_max(most);
          if (lane == 0) s_max[w] = most;
          asm volatile("bar.sync 5, 256;" ::: "memory");
#pragma unroll
          for (int i = 0; i < kCompute / 32; ++i) most = fmaxf(most, s_max[i]);
          if (most >= 65520.f) {  // what rounds to infinity (not if only infinities did)
            const int by = half_exponent(most);
            const float lower = pow2(by);
            up += by;
            scaled *= lower;
            if (tid < NR) s_delta[tid] *= lower;
            if (wg == 0 && j > 0) {  // dQ so far; the tile before is done with it
#pragma unroll
              for (int q = 0; q < DP / 8; ++q) {
                uint32_t r[8];
                tmem_ld(mine + C::kDq + 8 * q, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * lower);
                tmem_st(mine + C::kDq + 8 * q, r);
              }
            }
#pragma unroll
            for (int i = 0; i < H; i += 2) {
              f[i] *= lower;
              f[i + 1] *= lower;
              dk[i / 2] = pack2<T>(f[i], f[i + 1]);
            }
          }
        }
      }
      if (SPLIT) {
#pragma unroll
        for (int i = 0; i < H; i += 2) {
          const float2 r = unpack2<T>(dk[i / 2]);
          dl[i / 2] = pack2<T>(f[i] - r.x, f[i + 1] - r.y);
        }
      }
      tmem_st(mine + wg * (H / 2), pk);
      tmem_st(mine + C::kDp + wg * (H / 2), dk);
      if (SPLIT) tmem_st(mine + C::kDp + NR / 2 + wg * (H / 2), dl);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const int r = wg * H + i;
        uint8_t* at = ds_at + r * 128 + ((chunk ^ (r & 7)) << 4);
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)(i & 1 ? dk[i / 2] >> 16 : dk[i / 2]);
        if (SPLIT) *reinterpret_cast<uint16_t*>(at + NR * 128) = (uint16_t)(i & 1 ? dl[i / 2] >> 16 : dl[i / 2]);
      }
      if (wg == 0 && !takes)  // a row of K that another bag or a masked key holds: 0 * NaN is NaN
        for (int i = 0; i < C::kBlocks; ++i) {
          uint4* row = reinterpret_cast<uint4*>(skv + 2 * (j % NS) * C::kTile + (i * kKeys + key) * 128);
#pragma unroll
          for (int u = 0; u < 8; ++u) row[u] = make_uint4(0, 0, 0, 0);
        }
      fence_async_smem();
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(e_full);
      ok = ok && mbar_wait(o_full, j & 1, spin_max);
      __syncwarp();
      tc_fence_after();
      // warpgroup 0 stores dV, warpgroup 1 dK, 64 columns at a time: the thread's
      // row goes to shared memory (its warpgroup's half of dS, whose product is
      // done), and 8 lanes store a row's 128 bytes together
      T* out = wg == 0 ? static_cast<T*>(p.gv) + h * p.gvh : static_cast<T*>(p.gk) + h * p.gkh;
      const int64_t stride = wg == 0 ? p.gvs : p.gks;
      const float mul = wg == 0 ? pow2(-kShiftP<T>) : half_down<T>(up, p.scale);
      uint8_t* stage = sds + wg * 16384;
#pragma unroll
      for (int half = 0; half < C::kBlocks; ++half) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t r[32];
          tmem_ld(mine + (wg == 0 ? C::kDv : C::kDk) + 64 * half + 32 * q, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 u;
            uint32_t* v = &u.x;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = takes ? pack2<T>(__uint_as_float(r[8 * i + 2 * e]) * mul, __uint_as_float(r[8 * i + 2 * e + 1]) * mul)
                           : 0u;
            *reinterpret_cast<uint4*>(stage + key * 128 + (((4 * q + i) ^ (key & 7)) << 4)) = u;
          }
        }
        if (half == C::kBlocks - 1) tc_fence_before();
        asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
        const int ch = lane & 7, d = 64 * half + 8 * ch;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = (w & 3) * 32 + 4 * i + (lane >> 3);
          const uint4 u = *reinterpret_cast<const uint4*>(stage + row * 128 + ((ch ^ (row & 7)) << 4));
          if (k0 + row < ke && d < p.D) *reinterpret_cast<uint4*>(out + (bag.k0 + k0 + row) * stride + d) = u;
        }
        // the rows are out before the next half, or the next tile's dS, takes their place
        if (half < C::kBlocks - 1) asm volatile("bar.sync %0, 128;" ::"r"(6 + wg) : "memory");
        else asm volatile("bar.sync 5, 256;" ::: "memory");
      }
    }
    // dQ: lane r of tensor memory is row r with dS rounded; lane NR + r (SPLIT) is
    // the same row with the rest, and is added through shared memory (K and V are
    // done with)
    if (wg == 0) {
      constexpr int LD = DP + 4;
      float* rest = reinterpret_cast<float*>(skv);
      const int row = tid & 127;
      const bool have = n > 0 && ok;
      const float mul = half_down<T>(up, p.scale);
      tc_fence_after();
      if (SPLIT) {
        if (have && (w & 3) * 32 < 2 * NR) {
#pragma unroll
          for (int q = 0; q < DP / 32; ++q) {
            uint32_t r[32];
            tmem_ld(mine + C::kDq + 32 * q, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (row >= NR && row < 2 * NR)
                *reinterpret_cast<float4*>(rest + (row - NR) * LD + 32 * q + i) =
                    make_float4(__uint_as_float(r[i]), __uint_as_float(r[i + 1]), __uint_as_float(r[i + 2]),
                                __uint_as_float(r[i + 3]));
          }
        }
        asm volatile("bar.sync 6, 128;" ::: "memory");
      }
      if ((w & 3) * 32 < NR) {
        const int64_t t = bag.q0 + row / p.G;
        const int hq = h * p.G + row % p.G;
#pragma unroll
        for (int q = 0; q < DP / 32; ++q) {
          uint32_t r[32];
          if (have) {
            tmem_ld(mine + C::kDq + 32 * q, r);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = 32 * q + 8 * i;
            float f[8], e[8] = {};
            if (SPLIT && have && row < NR) {
              RawVec<float, 8> x;
              x.load(rest + row * LD + d);
              x.unpack(e);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) f[u] = have ? (__uint_as_float(r[8 * i + u]) + e[u]) * mul : 0.f;
            if (row < rows && d < p.D) {
              if (p.splits == 1) store_vec(static_cast<T*>(p.gq) + t * p.gqs + hq * p.gqh + d, f);
              else store_vec(p.po + (((int64_t)sp * p.Tq + t) * p.Hq + hq) * p.D + d, f);
            }
          }
        }
      }
    }
  }
  if (!ok) atomicOr(p.status, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == kIssuer) tmem_free(tmem, C::kCols);
}

template <typename T, int DP, int NR>
__global__ void __launch_bounds__(kThreads, FewBackCfg<DP, NR>::kTwo ? 2 : 1)
    attend_back_few_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ FewMaps maps, int spin_max) {
  unsigned id = blockIdx.x;
  const int h = id % p.Hkv;
  id /= p.Hkv;
  const int sp = id % p.splits, b = id / p.splits;
  pdl_wait();
  pdl_trigger();  // the join may be brought in; it waits for this grid's end
  const Bag bag = load_bag(p, b);
  if (bag.nk <= kSplitKeys) few_back_block<T, DP, NR, true>(p, maps, spin_max, bag, h, sp);
  else few_back_block<T, DP, NR, false>(p, maps, spin_max, bag, h, sp);
}

template <typename T, int DP, int NR>
cudaError_t few_back_go(const AttendParams& p, const FewMaps& m, int64_t grid, cudaStream_t s) {
  using C = FewBackCfg<DP, NR>;
  auto kernel = attend_back_few_kernel<T, DP, NR>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(kernel, C::kTotal, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, (unsigned)grid, kThreads, C::kTotal, s, p, m, kSpinLimit);
}

}  // namespace

recis_status launch_attend_back_few(const AttendParams& p, bool bf16, cudaStream_t s) {
  const int64_t grid = (int64_t)p.B * p.splits * p.Hkv;
  if (grid >= ((int64_t)1 << 31)) {
    set_error("attend_backward: too many blocks (bags times longest bag times heads)");
    return RECIS_ERR_INVALID_ARG;
  }
  FewMaps m = {};
  // a map is made only where its array has rows; without rows no block uses it
  bool ok = true;
  if (p.Tq > 0)
    ok = rows_map(&m.q, p.q, bf16, p.D, p.Hq, p.Tq, p.qs, p.qh, p.G, p.max_q) &&
         rows_map(&m.o, p.go, bf16, p.D, p.Hq, p.Tq, p.gos, p.goh, p.G, p.max_q);
  if (p.Tk > 0)
    ok = ok && rows_map(&m.k, p.k, bf16, p.D, p.Hkv, p.Tk, p.ks, p.kh, 1, kKeys) &&
         rows_map(&m.v, p.v, bf16, p.D, p.Hkv, p.Tk, p.vs, p.vh, 1, kKeys);
  if (!ok) {
    set_error("attend_backward: the driver refused a tensor map");
    return RECIS_ERR_CUDA;
  }
  const int rows = p.max_q * p.G;
  LaunchScope ls("attend_back_few", s);
  auto go = [&](auto t) {
    using T = decltype(t);
    if (p.D <= 64)
      return rows <= 16   ? few_back_go<T, 64, 16>(p, m, grid, s)
             : rows <= 32 ? few_back_go<T, 64, 32>(p, m, grid, s)
                          : few_back_go<T, 64, 64>(p, m, grid, s);
    return rows <= 16   ? few_back_go<T, 128, 16>(p, m, grid, s)
           : rows <= 32 ? few_back_go<T, 128, 32>(p, m, grid, s)
                        : few_back_go<T, 128, 64>(p, m, grid, s);
  };
  const cudaError_t e = bf16 ? go(__nv_bfloat16()) : go(__half());
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "attend_back_few launch");
}

}  // namespace recis
