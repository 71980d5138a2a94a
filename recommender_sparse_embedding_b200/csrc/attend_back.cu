// attend_back.cu -- attention backward, on the tensor cores.
//
//   p = exp(s - lse), dp = dO V^T, ds = p (dp - delta), delta = sum(dO * O),
//   dV = p^T dO,  dK = scale ds^T Q,  dQ = scale ds K.
//
// Two passes of one kernel.  Each block keeps a pair of 128-row tiles X1, X2 in
// shared memory and streams pairs of 64-row tiles Y1, Y2 past them:
//
//   keys:    X = (K, V) of 128 keys,  Y = (Q, dO);  A1 = dV += P^T Y2, A2 = dK += dS^T Y1
//   queries: X = (Q, dO) of 128 rows, Y = (K, V);                      A2 = dQ += dS Y1
//
// S = X1 Y1^T and dP = X2 Y2^T go to tensor memory, the compute warps (one row
// of X a thread) write P and dS over them as 16-bit values, and the second
// products take them from there; the accumulators stay in tensor memory.  The
// scores are thus computed twice (7 products instead of 5), but no block adds
// to another's output: no atomics, and the result does not depend on
// scheduling.  The query heads that share a key head are rows of one matrix
// (row r: query r / G, head r % G), so dK and dV sum over them in the
// accumulator.
//
// Measured on B200, bf16: 4 bags of 4096 queries over 4096 keys, 8 heads of 128, 771
// us, 891 TFLOP/s counted as 5 products (keys 405 us, queries 353); heads of 64, 546-
// 578 us, 630-595.  A step of 64 rows takes 1750 cycles over keys, 1400 over queries; its
// products take 1294 and 1038 (64 columns a product from shared memory take 49
// cycles instead of 32), issuing them and their waits and commits about 1400.
//
// Bags of few keys (SPLIT, by the bag's own length, so that its gradients do not
// depend on its neighbours) have dS go into its products as two 16-bit values,
// its rounding and what that leaves out (over the two halves of dP's columns):
// there the rounding of dS and that of `out` in delta would add up to more than
// 1.5 times the gradients' own rounding.  The more keys, the more the second
// averages out, and one value is enough.
//
// fp16 (kShiftP in attend.cuh): a thread's row of X is a row of the accumulators, so
// each thread scales ds by a power of two of its own, from |ds| <= |dO| |V| + |delta|:
// over keys its own |V| and the largest |dO| and |delta| of the bag's rows, over
// queries its own |dO| and delta and the largest |V| of the bag's keys, which the
// pass over keys has left.  (16 bags of 512-1024 over 1024-4096 keys, 8 heads of 128
// over 4: 560 us, bf16 531; the product more a pair of scores over keys costs most.)
//
// Rows of a tile that belong to another bag, or to masked keys, are overwritten
// with zeros before the products (0 * NaN is NaN) by the warp that issues the
// copies, which waits for such a tile's data itself.
#include <algorithm>
#include <type_traits>

#include "attend.cuh"
#include "tc.cuh"

namespace recis {

namespace {

constexpr int kX = 128;  // resident rows
constexpr int kY = 64;   // streamed rows a step

template <int DP, bool KEYS>
struct BackCfg {
  static constexpr int kBlocks = DP / 64;
  static constexpr int kXBytes = kBlocks * kX * 128, kYBytes = kBlocks * kY * 128;  // one tile
  // One block an SM.  S and dP are kept kBuf times: one's exponentials run under
  // another's products.  kNS streamed tiles: those in use (kBuf) and enough in
  // flight to cover a copy's latency, which a step (about 1000 cycles of
  // products) is shorter than.
  static constexpr int kBuf = DP == 64 ? 3 : 2;
  static constexpr int kNS = DP == 64 ? 7 : 5;
  static constexpr int kWG = 2;      // compute warpgroups
  static constexpr int kThreads = kWG * 128 + 64;
  static constexpr uint32_t kCols = 512;
  static constexpr uint32_t kAcc1 = kBuf * 128, kAcc2 = kAcc1 + (KEYS ? DP : 0);
  // tiles, barriers, the warps' maxima, lse and delta (or masks) of the streamed rows
  static constexpr int kBars = 2 * kXBytes + 2 * kNS * kYBytes, kMax = kBars + 256, kRowData = kMax + 64;
  static constexpr int kTotal = kRowData + kNS * (KEYS ? 2 * kY * 4 : 8);
};

struct BackMaps {
  CUtensorMap x1, x2, y1, y2;
};

// One block's work: tile `tile` of key head h of a bag, against part sp of its keys
template <typename T, int DP, bool KEYS, bool SPLIT>
__device__ __forceinline__ void attend_back_block(const AttendParams& p, const BackMaps& maps, int spin_max,
                                                  const Bag& bag, int b, int tile, int h, int sp) {
  using C = BackCfg<DP, KEYS>;
  constexpr int NB = C::kBuf, WG = C::kWG, kNS = C::kNS;
  extern __shared__ __align__(1024) uint8_t base[];  // nothing else is in shared memory: it starts at a tile's boundary
  uint8_t *x1 = base, *x2 = x1 + C::kXBytes, *y1 = x2 + C::kXBytes, *y2 = y1 + kNS * C::kYBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + C::kBars);
  uint64_t *x_full = bar, *acc_full = bar + 1, *s_full = bar + 2, *e_full = s_full + NB;
  uint64_t *y_full = e_full + NB, *y_empty = y_full + kNS, *y_raw = y_empty + kNS;
  static_assert(2 + 2 * NB + 3 * kNS < 32, "barriers and the address of tensor memory in 256 bytes");
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar + 31);
  float* s_lse = reinterpret_cast<float*>(base + C::kRowData);  // KEYS: [kNS][kY] -lse * log2(e)
  float* s_delta = s_lse + kNS * kY;                            // KEYS: [kNS][kY] -delta
  uint32_t(*s_valid)[2] = reinterpret_cast<uint32_t(*)[2]>(base + C::kRowData);  // queries: the keys that take part

  // the block's tile: of keys, or of (query, head) rows against a part of the keys
  const int TQ = kX / p.G;                                  // queries: queries a tile
  const int first = tile * (KEYS ? kX : TQ);                // first key, or query, of the tile
  const int ks = KEYS ? 0 : sp * p.split_keys, ke = KEYS ? bag.nk : min(ks + p.split_keys, bag.nk);
  if (first >= (KEYS ? bag.nk : bag.nq) || (!KEYS && sp > 0 && ks >= bag.nk)) return;
  // streamed tiles; keys: heads in chunks of at most 64, the queries of a chunk's tile
  const int gc = min(p.G, kY), chunks = (p.G + gc - 1) / gc, tq = kY / gc;
  const int n = KEYS ? (bag.nq + tq - 1) / tq * chunks : ke > ks ? (ke - ks + kY - 1) / kY : 0;

  const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
  constexpr int kLoader = WG * 4, kIssuer = kLoader + 1;
  if (w == kIssuer) tmem_alloc(s_tmem, C::kCols);
  if (tid == kLoader * 32) {
    mbar_init(x_full, 1);
    mbar_init(acc_full, 1);
    for (int i = 0; i < NB; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(e_full + i, 128);
    }
    for (int i = 0; i < kNS; ++i) {
      // a tile: its copies' bytes, the warp's word that it is finished, the lanes' copies of lse and delta
      mbar_init(y_full + i, KEYS ? 34 : 2);
      mbar_init(y_empty + i, 1);
      mbar_init(y_raw + i, 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  bool ok = true;  // false: a wait gave up

  if (w == kLoader) {
    if (n > 0) {
      if (elect_one()) {
        const int rows = KEYS ? kX : TQ * p.G;
        mbar_arrive_expect(x_full, (unsigned)(2 * C::kBlocks * rows * 128));
        for (int i = 0; i < C::kBlocks; ++i) {
          const int y = KEYS ? h : h * p.G, z = (int)((KEYS ? bag.k0 : bag.q0) + first);
          tma_load3(x1 + i * kX * 128, &maps.x1, 64 * i, y, z, x_full);
          tma_load3(x2 + i * kX * 128, &maps.x2, 64 * i, y, z, x_full);
        }
      }
      // the lane's rows of a tile: lane and lane + 32
      int rq[2], rg[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rq[i] = (lane + 32 * i) / gc;
        rg[i] = (lane + 32 * i) % gc;
      }
      // a tile's first query and head (keys), or key: advanced without divisions,
      // which would take longer than the step
      struct At {
        int a, g;
      };
      auto next = [&](At& t) {
        if (!KEYS) {
          t.a += kY;
        } else if ((t.g += gc) >= p.G) {
          t.g = 0;
          t.a += tq;
        }
      };
      // whether the lane's i-th row of the tile takes part: not 0 (a mask's byte is not looked at before its turn)
      auto takes = [&](const At& t, int i) -> unsigned {
        if (KEYS) return rq[i] < tq && t.a + rq[i] < bag.nq && t.g + rg[i] < p.G;
        const int key = t.a + lane + 32 * i;
        unsigned m = key < ke;
        if (m && p.mask) m = __ldg(p.mask + bag.k0 + key);
        return m;
      };
      auto special = [&](const At& t) {  // whether it holds rows that must be zeroed
        if (!KEYS) return t.a + kY > ke || p.mask != nullptr;
        return tq * gc < kY || t.a + tq > bag.nq || t.g + gc > p.G;
      };
      const unsigned bytes = 2 * C::kBlocks * 128 * (KEYS ? tq * gc : kY);
      // a special tile is finished a step after it is asked for; what its
      // finishing needs (masks) is read a step before that
      At at = {KEYS ? 0 : ks, 0}, ahead = at;
      unsigned v[2] = {0, 0}, v_next[2] = {takes(at, 0), takes(at, 1)};
      bool last_special = false;
      next(ahead);
      int st = 0, last_st = 0, asked = 0;
      unsigned ph = 0, last_ph = 0, raw = 0;  // raw: stages whose tile is a special one
      for (int j = 0; j <= n; ++j) {
        if (last_special) {
          if (!KEYS)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const unsigned bits = __ballot_sync(0xffffffffu, v[i] != 0);
              if (lane == 0) s_valid[last_st][i] = bits;
            }
          ok = mbar_wait(y_raw + last_st, last_ph, spin_max) && ok;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!v[i])
              for (int k = 0; k < C::kBlocks; ++k) {
                uint4* a = reinterpret_cast<uint4*>(y1 + last_st * C::kYBytes + (k * kY + lane + 32 * i) * 128);
                uint4* c = reinterpret_cast<uint4*>(y2 + last_st * C::kYBytes + (k * kY + lane + 32 * i) * 128);
#pragma unroll
                for (int u = 0; u < 8; ++u) a[u] = c[u] = make_uint4(0, 0, 0, 0);
              }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(y_full + last_st);
        }
        if (j == n) break;
        v[0] = v_next[0];
        v[1] = v_next[1];
        if (j + 1 < n) {
          v_next[0] = takes(ahead, 0);
          v_next[1] = takes(ahead, 1);
          next(ahead);
        }
        if (j >= kNS) ok = mbar_wait(y_empty + st, ph ^ 1, spin_max) && ok;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        last_special = special(at);
        raw = (raw & ~(1u << st)) | (last_special ? 1u << st : 0u);
        asked = j + 1;
        if (elect_one()) {
          uint64_t* full = y_full + st;
          if (last_special) {
            mbar_arrive(full);
            full = y_raw + st;
          } else {
            if (!KEYS) s_valid[st][0] = s_valid[st][1] = 0xffffffffu;
            mbar_arrive(y_raw + st);  // keeps the stage's phases in step
            mbar_arrive(full);
          }
          mbar_arrive_expect(full, bytes);
          const int y = KEYS ? h * p.G + at.g : h, z = (int)(KEYS ? bag.q0 : bag.k0) + at.a;
          for (int i = 0; i < C::kBlocks; ++i) {
            tma_load3(y1 + st * C::kYBytes + i * kY * 128, &maps.y1, 64 * i, y, z, full);
            tma_load3(y2 + st * C::kYBytes + i * kY * 128, &maps.y2, 64 * i, y, z, full);
          }
        }
        __syncwarp();
        if (KEYS) {
          // the rows' -lse and -delta; zeros for rows that do not take part, whose
          // Q and dO are zeros too (p = 1, but p^T dO and ds are 0)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t r = v[i] ? (bag.q0 + at.a + rq[i]) * p.Hq + h * p.G + at.g + rg[i] : 0;
            copy4(s_lse + st * kY + lane + 32 * i, p.nlse + r, v[i] != 0);
            copy4(s_delta + st * kY + lane + 32 * i, p.delta + r, v[i] != 0);
          }
          copy_arrive(y_full + st);
        }
        last_st = st;
        last_ph = ph;
        next(at);
        if (++st == kNS) {
          st = 0;
          ph ^= 1;
        }
      }
      if (KEYS) copy_wait_all();
      // copies in flight end before the block does
      ok = mbar_wait(x_full, 0, spin_max) && ok;
      if (!ok)
        for (int j = max(asked - kNS, 0); j < asked; ++j)
          mbar_wait((raw >> (j % kNS) & 1 ? y_raw : y_full) + j % kNS, (j / kNS) & 1, spin_max);
    }
  } else if (w == kIssuer) {
    if (n > 0) {
      constexpr uint32_t id_s = mma_desc<T>(kX, kY, false, false), id_a = mma_desc<T>(kX, DP, false, true);
      // descriptors count 16 bytes
      const uint64_t dx1 = smem_desc(smem_u32(x1), 16), dx2 = smem_desc(smem_u32(x2), 16);
      const uint64_t dy1 = smem_desc(smem_u32(y1), 16), dy2 = smem_desc(smem_u32(y2), 16);
      const uint64_t ty1 = smem_desc(smem_u32(y1), kY * 128), ty2 = smem_desc(smem_u32(y2), kY * 128);
      const bool one = elect_one();
      auto scores = [&](int j) {
        const int st = j % kNS, bf = j % NB;
        if (!warp_wait(y_full + st, (j / kNS) & 1, spin_max)) return false;
        tc_fence_after();
        const uint32_t d = tmem + bf * 128;
        const uint64_t b1 = dy1 + st * (C::kYBytes >> 4), b2 = dy2 + st * (C::kYBytes >> 4);
        if (one) {
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(d, dx1 + (((k >> 2) * kX * 128 + (k & 3) * 32) >> 4), b1 + (((k >> 2) * kY * 128 + (k & 3) * 32) >> 4),
                   id_s, k > 0);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k)
            mma_ss(d + 64, dx2 + (((k >> 2) * kX * 128 + (k & 3) * 32) >> 4),
                   b2 + (((k >> 2) * kY * 128 + (k & 3) * 32) >> 4), id_s, k > 0);
          mma_commit(s_full + bf);
        }
        __syncwarp();
        return true;
      };
      // the scores run NB - 1 tiles ahead of the products that use them
      ok = warp_wait(x_full, 0, spin_max);
      for (int j = 0; j < NB - 1 && j < n && ok; ++j) ok = scores(j);
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % kNS, bf = j % NB;
        if (j + NB - 1 < n && !(ok = scores(j + NB - 1))) break;
        if (!(ok = warp_wait(e_full + bf, (j / NB) & 1, spin_max))) break;
        tc_fence_after();
        const uint32_t e = tmem + bf * 128;
        const uint64_t b1 = ty1 + st * (C::kYBytes >> 4), b2 = ty2 + st * (C::kYBytes >> 4);
        if (one) {
#pragma unroll
          for (int k = 0; k < kY / 16; ++k) {
            const uint32_t at = (k >> 1) * 32 + (k & 1) * 8;
            if (KEYS) mma_ts(tmem + C::kAcc1, e + at, b2 + (k * 2048 >> 4), id_a, j > 0 || k > 0);
            mma_ts(tmem + C::kAcc2, e + 64 + at, b1 + (k * 2048 >> 4), id_a, j > 0 || k > 0);
            if (SPLIT) mma_ts(tmem + C::kAcc2, e + 80 + at, b1 + (k * 2048 >> 4), id_a, true);
          }
          mma_commit(y_empty + st);
        }
        __syncwarp();
      }
      if (one) mma_commit(acc_full);
      ok = warp_wait(acc_full, 0, spin_max) && ok;
    }
    __syncwarp();
  } else {
    const int row = tid & 127, wg = tid >> 7;  // the thread's row of X
    const uint32_t mine = tmem + ((uint32_t)(w & 3) << 21);
    bool live;
    int64_t t;       // its row in memory
    int hx;          // its head
    float lse = -INFINITY, delta = 0.f;  // queries: the row's -lse * log2(e) and -delta
    if (KEYS) {
      live = first + row < bag.nk;
      t = bag.k0 + first + row;
      hx = h;
    } else {
      live = row < TQ * p.G && first + row / p.G < bag.nq;
      t = bag.q0 + first + row / p.G;
      hx = h * p.G + row % p.G;
      if (live) {
        lse = p.nlse[t * p.Hq + hx];
        delta = p.delta[t * p.Hq + hx];
      }
    }
    const bool any = __any_sync(0xffffffffu, live);
    const float c = p.scale_log2;
    float up = 1.f;  // fp16: ds 2^kShiftP to its own scale
    if constexpr (kShiftP<T> > 0) {
      float bound = 0.f;
      if (KEYS && n > 0) {
        float* s_max = reinterpret_cast<float*>(base + C::kMax);
        float go = 0.f, de = 0.f;
        const int rows = bag.nq * p.G;
        for (int r = tid; r < rows; r += 4 * WG * 128) {
          float a[4], c[4];  // 8 loads in flight
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int at = min(r + u * WG * 128, rows - 1);
            const int64_t i = (bag.q0 + at / p.G) * p.Hq + h * p.G + at % p.G;
            a[u] = p.gnorm[i];
            c[u] = p.delta[i];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            go = finite_max(go, a[u]);
            de = finite_max(de, fabsf(c[u]));
          }
        }
        go = warp_max(go);
        de = warp_max(de);
        if (lane == 0) {
          s_max[w] = go;
          s_max[8 + w] = de;
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");
#pragma unroll
        for (int i = 0; i < WG * 4; ++i) {
          go = fmaxf(go, s_max[i]);
          de = fmaxf(de, s_max[8 + i]);
        }
        ok = mbar_wait(x_full, 0, spin_max);
        float v = 0.f;
        for (int i = 0; i < C::kBlocks; ++i)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            RawVec<T, 8> raw;
            raw.load(reinterpret_cast<const T*>(x2 + (i * kX + row) * 128 + ((u ^ (row & 7)) << 4)));
            float f[8];
            raw.unpack(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v = fmaf(f[e], f[e], v);
          }
        v = live && (!p.mask || p.mask[t]) && v < INFINITY ? sqrtf(v) : 0.f;
        bound = fmaf(go, v, de);
        v = warp_max(v);
        if (wg == 0 && lane == 0) p.vnorm[value_slots(p.B, p.Tk) * h + value_slot(bag.k0, b) + 4 * tile + w] = v;
      } else if (!KEYS) {
        float v = 0.f;
        const float* slots = p.vnorm + value_slots(p.B, p.Tk) * h + value_slot(bag.k0, b);
        for (int i = ks / kX * 4 + lane; i < (ke + kX - 1) / kX * 4; i += 32) v = fmaxf(v, slots[i]);
        v = warp_max(v);
        if (live) bound = fmaf(p.gnorm[t * p.Hq + hx], v, fabsf(delta));
      }
      up = pow2(half_exponent(bound) - kShiftP<T>);
      delta *= up;
    }
    // two warpgroups take every other tile, each its own S and dP, so that one's
    // exponentials run under the other's products
    for (int j = wg; j < n; j += WG) {
      const int st = j % kNS, bf = j % NB;
      ok = mbar_wait(y_full + st, (j / kNS) & 1, spin_max) && mbar_wait(s_full + bf, (j / NB) & 1, spin_max);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (any) {
        uint32_t sd[2][2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          tmem_ld32(mine + bf * 128 + 32 * q, sd[0][q]);
          tmem_ld32(mine + bf * 128 + 64 + 32 * q, sd[1][q]);
        }
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col = q * 32;
          const uint32_t(&s)[32] = sd[0][q];
          const uint32_t(&d)[32] = sd[1][q];
          uint32_t valid = 0xffffffffu;
          if (!KEYS) valid = s_valid[st][col >> 5];
          uint32_t pk[16], dk[16], dl[16];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float4 ls = make_float4(lse, lse, lse, lse), de = make_float4(delta, delta, delta, delta);
            if (KEYS) {
              ls = *reinterpret_cast<const float4*>(s_lse + st * kY + col + i);
              de = *reinterpret_cast<const float4*>(s_delta + st * kY + col + i);
            }
            const float2 c2 = make_float2(c, c);
            float2 e0 = fma2(as_f2(s[i], s[i + 1]), c2, make_float2(ls.x, ls.y));
            float2 e1 = fma2(as_f2(s[i + 2], s[i + 3]), c2, make_float2(ls.z, ls.w));
            e0 = make_float2(ex2(e0.x), ex2(e0.y));
            e1 = make_float2(ex2(e1.x), ex2(e1.y));
            float2 f0, f1;
            if constexpr (kShiftP<T> > 0) {
              const float2 u2 = make_float2(up, up);
              if (KEYS) {
                f0 = mul2(e0, mul2(add2(as_f2(d[i], d[i + 1]), make_float2(de.x, de.y)), u2));
                f1 = mul2(e1, mul2(add2(as_f2(d[i + 2], d[i + 3]), make_float2(de.z, de.w)), u2));
              } else {  // delta is scaled already
                f0 = mul2(e0, fma2(as_f2(d[i], d[i + 1]), u2, make_float2(de.x, de.y)));
                f1 = mul2(e1, fma2(as_f2(d[i + 2], d[i + 3]), u2, make_float2(de.z, de.w)));
              }
            } else {
              f0 = mul2(e0, add2(as_f2(d[i], d[i + 1]), make_float2(de.x, de.y)));
              f1 = mul2(e1, add2(as_f2(d[i + 2], d[i + 3]), make_float2(de.z, de.w)));
            }
            if (!KEYS && valid != 0xffffffffu) {
              if (!(valid >> i & 1)) f0.x = 0.f;
              if (!(valid >> (i + 1) & 1)) f0.y = 0.f;
              if (!(valid >> (i + 2) & 1)) f1.x = 0.f;
              if (!(valid >> (i + 3) & 1)) f1.y = 0.f;
            }
            if (KEYS) {
              pk[i / 2] = pack2<T>(e0.x, e0.y);
              pk[i / 2 + 1] = pack2<T>(e1.x, e1.y);
            }
            dk[i / 2] = pack2<T>(f0.x, f0.y);
            dk[i / 2 + 1] = pack2<T>(f1.x, f1.y);
            if (SPLIT) {
              const float2 r0 = unpack2<T>(dk[i / 2]), r1 = unpack2<T>(dk[i / 2 + 1]);
              dl[i / 2] = pack2<T>(f0.x - r0.x, f0.y - r0.y);
              dl[i / 2 + 1] = pack2<T>(f1.x - r1.x, f1.y - r1.y);
            }
          }
          if (KEYS) tmem_st16(mine + bf * 128 + col, pk);
          tmem_st16(mine + bf * 128 + 64 + col, dk);
          if (SPLIT) tmem_st16(mine + bf * 128 + 80 + col, dl);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(e_full + bf);
    }
    if (n > 0) ok = mbar_wait(acc_full, 0, spin_max) && ok;
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    const bool have = n > 0 && ok;
    const bool takes = !KEYS || !p.mask || (live && p.mask[t]);  // a masked key's gradients are zero
    float back = p.scale;  // takes ds's scale out of its sums again
    if constexpr (kShiftP<T> > 0) back = pow2_times(127 - (int)(__float_as_uint(up) >> 23) - kShiftP<T>, p.scale);
    // 2 accumulators (keys) or 1 (queries) of DP columns, in pieces of 64: the
    // thread's row goes to shared memory (X's tiles are done with), 8 lanes store
    // a row's 128 bytes together.  Parts of grad_q are stored directly, in fp32.
    constexpr int kPieces = (KEYS ? 2 : 1) * C::kBlocks;
#pragma unroll
    for (int piece = wg; piece < kPieces; piece += WG) {
      const bool acc1 = KEYS && piece < C::kBlocks;
      const int d0 = piece * 64 % DP;
      const float mul = acc1 ? pow2(-kShiftP<T>) : back;
      uint8_t* stage = x1 + piece * kX * 128;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t r[32];
        if (have) {
          tmem_ld32(mine + (acc1 ? C::kAcc1 : C::kAcc2) + d0 + 32 * q, r);
          tmem_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = have && takes ? __uint_as_float(r[8 * i + e]) * mul : 0.f;
          const int d = d0 + 32 * q + 8 * i;
          if (KEYS || p.splits == 1)
            *reinterpret_cast<uint4*>(stage + row * 128 + (((4 * q + i) ^ (row & 7)) << 4)) = make_uint4(
                pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
          else if (live && d < p.D)
            store_vec(p.po + (((int64_t)sp * p.Tq + t) * p.Hq + hx) * p.D + d, f);
        }
      }
      if (!KEYS && p.splits > 1) continue;
      asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
      T* out = static_cast<T*>(KEYS ? acc1 ? p.gv : p.gk : p.gq);
      const int64_t rs = KEYS ? acc1 ? p.gvs : p.gks : p.gqs, hs = KEYS ? acc1 ? p.gvh : p.gkh : p.gqh;
      const int ch = lane & 7, d = d0 + 8 * ch;
      for (int i = 0; i < 8; ++i) {
        const int rr = (w & 3) * 32 + 4 * i + (lane >> 3);
        const int q = KEYS ? rr : rr / p.G, hh = KEYS ? h : h * p.G + rr - q * p.G;
        const bool lives = KEYS ? first + rr < bag.nk : rr < TQ * p.G && first + q < bag.nq;
        const uint4 u = *reinterpret_cast<const uint4*>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
        if (lives && d < p.D)
          *reinterpret_cast<uint4*>(out + ((KEYS ? bag.k0 : bag.q0) + first + q) * rs + hh * hs + d) = u;
      }
    }
  }
  if (!ok) atomicOr(p.status, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == kIssuer) tmem_free(tmem, C::kCols);
}

template <typename T, int DP, bool KEYS>
__global__ void __launch_bounds__(BackCfg<DP, KEYS>::kThreads, 1)
    attend_back_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ BackMaps maps, int spin_max) {
  const int TQ = kX / p.G;
  const int per_bag = KEYS ? (p.max_k + kX - 1) / kX : (p.max_q + TQ - 1) / TQ;
  unsigned id = blockIdx.x;
  const int tile = id % per_bag;
  id /= per_bag;
  const int h = id % p.Hkv;
  id /= p.Hkv;
  pdl_wait();
  pdl_trigger();  // the next kernel may be brought in; it waits for this grid's end
  const int sp = KEYS ? 0 : id % p.splits, b = KEYS ? id : id / p.splits;
  const Bag bag = load_bag(p, b);
  // (two whole bodies: with a branch around the second values alone, or two loops
  // in the compute warps, both passes of long bags take 5 % longer)
  if (bag.nk <= kSplitKeys) attend_back_block<T, DP, KEYS, true>(p, maps, spin_max, bag, b, tile, h, sp);
  else attend_back_block<T, DP, KEYS, false>(p, maps, spin_max, bag, b, tile, h, sp);
}

// What the passes need of a row: -delta, delta[t][h] = sum_d grad_out * out,
// -lse * log2(e) + kShiftP (-inf for a row without keys: p = 0), for fp16 |grad_out|.
// 16 lanes a (query, head), 8 columns each.
template <typename T>
__global__ void __launch_bounds__(256) delta_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15, d = lane * 8;
  const int64_t i = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  float s = 0.f, g = 0.f;
  if (i < p.Tq * p.Hq && d < p.D) {
    const int64_t t = i / p.Hq;
    const int h = (int)(i - t * p.Hq);
    RawVec<T, 8> a, b;
    a.load(static_cast<const T*>(p.out) + t * p.os + h * p.oh + d);
    b.load(static_cast<const T*>(p.go) + t * p.gos + h * p.goh + d);
    float x[8], y[8];
    a.unpack(x);
    b.unpack(y);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s = fmaf(x[j], y[j], s);
      if (kShiftP<T> > 0) g = fmaf(y[j], y[j], g);
    }
  }
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, off);
    if (kShiftP<T> > 0) g += __shfl_xor_sync(0xffffffffu, g, off);
  }
  if (lane == 0 && i < p.Tq * p.Hq) {
    const float lse = p.lse[i];
    p.delta[i] = -s;
    p.nlse[i] = lse == -INFINITY ? -INFINITY : fmaf(-lse, 1.4426950408889634f, (float)kShiftP<T>);
    if (kShiftP<T> > 0) p.gnorm[i] = sqrtf(g);
  }
}

// grad_q from the parts of the keys, added in order: one warp a (query, head)
template <typename T>
__global__ void __launch_bounds__(128) join_q_kernel(const __grid_constant__ AttendParams p) {
  const int lane = threadIdx.x & 31, d = lane * 4;
  const int tiles = (p.max_q * p.Hq + 3) / 4;
  const int b = blockIdx.x / tiles, i = (blockIdx.x % tiles) * 4 + (threadIdx.x >> 5);
  pdl_wait();
  const Bag bag = load_bag(p, b);
  if (i >= bag.nq * p.Hq || d >= p.D) return;
  const int64_t t = bag.q0 + i / p.Hq, step = p.Tq * p.Hq;
  const int hq = i % p.Hq, n = max(1, (bag.nk + p.split_keys - 1) / p.split_keys);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < n; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(p.po + (s * step + t * p.Hq + hq) * p.D + d);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  *reinterpret_cast<uint2*>(static_cast<T*>(p.gq) + t * p.gqs + hq * p.gqh + d) =
      make_uint2(pack2<T>(a.x, a.y), pack2<T>(a.z, a.w));
}

template <typename T, int DP, bool KEYS>
cudaError_t back_go(const AttendParams& p, const BackMaps& m, int64_t grid, cudaStream_t s) {
  using C = BackCfg<DP, KEYS>;
  auto kernel = attend_back_kernel<T, DP, KEYS>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(kernel, C::kTotal, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, (unsigned)grid, C::kThreads, C::kTotal, s, p, m, kSpinLimit);
}

template <typename T, bool KEYS>
cudaError_t back_launch(const AttendParams& p, const BackMaps& m, int64_t grid, cudaStream_t s) {
  return p.D <= 64 ? back_go<T, 64, KEYS>(p, m, grid, s) : back_go<T, 128, KEYS>(p, m, grid, s);
}

// joins the parts of grad_q
template <typename T>
recis_status join_q(const AttendParams& p, cudaStream_t s) {
  if (p.splits == 1 || p.Tq == 0) return RECIS_OK;
  const int64_t grid = (int64_t)p.B * (((int64_t)p.max_q * p.Hq + 3) / 4);
  if (grid >= ((int64_t)1 << 31)) {
    set_error("attend_backward: too many blocks (bags times longest bag times heads)");
    return RECIS_ERR_INVALID_ARG;
  }
  LaunchScope ls("attend_join_q", s);
  const cudaError_t e = launch_pdl(join_q_kernel<T>, (unsigned)grid, 128, 0, s, p);
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "attend_join_q launch");
}

template <typename T>
recis_status back(const AttendParams& p, cudaStream_t s) {
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  if (few_back_rows(p.max_q, p.G)) {
    const recis_status st = launch_attend_back_few(p, bf16, s);
    return st == RECIS_OK ? join_q<T>(p, s) : st;
  }
  const int TQ = kX / p.G, gc = std::min(p.G, kY), tq = kY / gc;
  const int64_t kgrid = (int64_t)p.B * p.Hkv * (((int64_t)p.max_k + kX - 1) / kX);
  const int64_t qgrid = (int64_t)p.B * p.splits * p.Hkv * (((int64_t)p.max_q + TQ - 1) / TQ);
  const int64_t dgrid = (p.Tq * p.Hq + 15) / 16;
  for (int64_t g : {kgrid, qgrid, dgrid})
    if (g >= ((int64_t)1 << 31)) {
      set_error("attend_backward: too many blocks (bags times longest bag times heads)");
      return RECIS_ERR_INVALID_ARG;
    }
  BackMaps mk = {}, mq = {};
  bool ok = true;
  // a map is made only where its array has rows; without rows no block uses it
  if (p.Tq > 0)
    ok = ok && rows_map(&mk.y1, p.q, bf16, p.D, p.Hq, p.Tq, p.qs, p.qh, gc, tq) &&
         rows_map(&mk.y2, p.go, bf16, p.D, p.Hq, p.Tq, p.gos, p.goh, gc, tq) &&
         rows_map(&mq.x1, p.q, bf16, p.D, p.Hq, p.Tq, p.qs, p.qh, p.G, TQ) &&
         rows_map(&mq.x2, p.go, bf16, p.D, p.Hq, p.Tq, p.gos, p.goh, p.G, TQ);
  if (p.Tk > 0)
    ok = ok && rows_map(&mk.x1, p.k, bf16, p.D, p.Hkv, p.Tk, p.ks, p.kh, 1, kX) &&
         rows_map(&mk.x2, p.v, bf16, p.D, p.Hkv, p.Tk, p.vs, p.vh, 1, kX) &&
         rows_map(&mq.y1, p.k, bf16, p.D, p.Hkv, p.Tk, p.ks, p.kh, 1, kY) &&
         rows_map(&mq.y2, p.v, bf16, p.D, p.Hkv, p.Tk, p.vs, p.vh, 1, kY);
  if (!ok) {
    set_error("attend_backward: the driver refused a tensor map");
    return RECIS_ERR_CUDA;
  }
  cudaError_t e;
  if (dgrid > 0) {
    LaunchScope ls("attend_delta", s);
    e = launch_pdl(delta_kernel<T>, (unsigned)dgrid, 256, 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "attend_delta launch");
  }
  if (kgrid > 0) {
    LaunchScope ls("attend_back_keys", s);
    e = back_launch<T, true>(p, mk, kgrid, s);
    if (e != cudaSuccess) return cuda_fail(e, "attend_back_keys launch");
  }
  if (qgrid > 0) {
    LaunchScope ls("attend_back_queries", s);
    e = back_launch<T, false>(p, mq, qgrid, s);
    if (e != cudaSuccess) return cuda_fail(e, "attend_back_queries launch");
  }
  return join_q<T>(p, s);
}

}  // namespace

recis_status launch_attend_back(const AttendParams& p, bool bf16, cudaStream_t s) {
  return bf16 ? back<__nv_bfloat16>(p, s) : back<__half>(p, s);
}

}  // namespace recis
