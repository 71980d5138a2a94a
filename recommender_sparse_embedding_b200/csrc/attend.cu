// attend.cu -- attention of each bag's queries over the bag's keys: argument
// checks, the plan of a call, and the forward pass for few rows.
//
//   s = scale q k^T over the bag's unmasked keys, out = softmax(s) v,
//   lse = log sum exp s;  a bag without keys: out 0, lse -inf.
//
// The query heads that share a key head are rows of one matrix: row r of key
// head h is query r / G, head h G + r % G, so K and V are read once for all of
// them.
//
// Measured on B200: one query over 256 bags of 1000-5000 keys, 8 heads of 128 over
// 2, 129 us with the join in passes in a row (its floor is 122), 140 with L2 flushed
// before each; up to 16 queries, 2 heads of 64, 83 us (4.6 TB/s).
#include <algorithm>
#include <type_traits>

#include "attend.cuh"
#include "tc.cuh"

namespace recis {

namespace {

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

constexpr int kRowTile = kFewRows;  // rows (query, head of the group) a block of few_kernel takes
constexpr int kFewWarps = 4;        // warps of products, 16 keys of a tile each
constexpr int kFewKeys = 64;        // keys a tile

template <int DP>
struct FewCfg {
  static constexpr int kBlocks = DP / 64;
  static constexpr int kBytes = kBlocks * kFewKeys * 128;  // one tile of K or V
  static constexpr int kStages = DP == 64 ? 4 : 3;         // 64 and 96 KB in flight: three and two blocks an SM
  static constexpr int kTotal = 2 * kStages * kBytes + 1024 + 128;
};

// One block: 16 rows of one key head against one part of the bag's keys, bound
// by reading K and V.  A fifth warp keeps tiles of 64 keys coming by
// tensor-map copies, kStages deep; warp w takes 16 keys of each tile with a
// softmax of its own (one m16n8k16 step of p v), and the warps' results are
// joined in shared memory at the end, so the warps never wait for one another
// in between.
template <typename T, int DP>  // DP: D rounded up to 64 or 128
__global__ void __launch_bounds__(kFewWarps * 32 + 32)
    few_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, int spin_max) {
  using C = FewCfg<DP>;
  constexpr int NS = C::kStages, LD = DP + 4;
  extern __shared__ uint8_t s_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + 2 * NS * C::kBytes);
  uint64_t* empty = full + NS;
  __shared__ float s_m[kFewWarps][kRowTile], s_l[kFewWarps][kRowTile];
  const int rtiles = (p.max_q * p.G + kRowTile - 1) / kRowTile;
  unsigned id = blockIdx.x;
  const int rt = id % rtiles;
  id /= rtiles;
  const int h = id % p.Hkv;
  id /= p.Hkv;
  const int sp = id % p.splits, b = id / p.splits;
  pdl_wait();
  pdl_trigger();  // the join may be brought in; it waits for this grid's end
  const Bag bag = load_bag(p, b);
  const int rows = bag.nq * p.G, r0 = rt * kRowTile;
  const int ks = sp * p.split_keys, ke = min(ks + p.split_keys, bag.nk);
  if (r0 >= rows || (ks >= bag.nk && sp > 0)) return;
  const int n = ke > ks ? (ke - ks + kFewKeys - 1) / kFewKeys : 0;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2, c = lane & 3;
  if (tid == kFewWarps * 32) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kFewWarps);
    }
  }
  __syncthreads();
  bool ok = true;  // false: a wait gave up
  if (w == kFewWarps) {
    if (lane == 0) {
      int asked = 0;
      for (int j = 0; j < n; ++j) {
        const int st = j % NS;
        if (j >= NS && !(ok = mbar_wait(empty + st, ((j / NS) & 1) ^ 1, spin_max))) break;
        mbar_arrive_expect(full + st, 2 * C::kBytes);
        const int row = (int)(bag.k0 + ks + j * kFewKeys);
        for (int i = 0; i < C::kBlocks; ++i) {
          tma_load3(base + 2 * st * C::kBytes + i * kFewKeys * 128, &mk, 64 * i, h, row, full + st);
          tma_load3(base + (2 * st + 1) * C::kBytes + i * kFewKeys * 128, &mv, 64 * i, h, row, full + st);
        }
        asked = j + 1;
      }
      // copies in flight end before the block does
      for (int j = max(asked - NS, 0); j < asked; ++j) ok = mbar_wait(full + j % NS, (j / NS) & 1, spin_max) && ok;
    }
  } else {
    uint32_t qa[DP / 16][4];
#pragma unroll
    for (int i = 0; i < DP / 16; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + g + 8 * (u & 1), d = 16 * i + 2 * c + 8 * (u >> 1);
        qa[i][u] = 0;
        if (d < p.D && r < rows)
          qa[i][u] = *reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + (bag.q0 + r / p.G) * p.qs +
                                                        (h * p.G + r % p.G) * p.qh + d);
      }
    float o[DP / 8][4];
#pragma unroll
    for (int j = 0; j < DP / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // the lane's rows of K and V for the matrix loads, and its swizzle
    const int krow = w * 16 + (lane >> 4) * 8 + (lane & 7), vrow = w * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
    const int kch = (lane >> 3) & 1, vch = lane >> 4, sw = lane & 7;
    // whether the lane's key (of 16) of tile j takes part: not 0 (the byte is not looked at before its turn)
    auto takes = [&](int j) -> unsigned {
      const int key = ks + j * kFewKeys + w * 16 + (lane & 15);
      unsigned m = key < ke;
      if (m && p.mask) m = __ldg(p.mask + bag.k0 + key);
      return m;
    };
    unsigned v_next = takes(0);
    for (int j = 0; j < n; ++j) {
      const int st = j % NS, k0 = ks + j * kFewKeys + w * 16;  // the warp's first key
      const unsigned v = v_next;
      v_next = takes(j + 1);
      ok = mbar_wait(full + st, (j / NS) & 1, spin_max);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t ak = smem_u32(base + 2 * st * C::kBytes) + krow * 128;
      const uint32_t av = smem_u32(base + (2 * st + 1) * C::kBytes) + vrow * 128;
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        uint32_t kf[4];
        ldsm4(kf, ak + (i >> 2) * kFewKeys * 128 + ((((i & 3) * 2 + kch) ^ sw) << 4));
        mma16816<T>(s[0], qa[i], kf[0], kf[1]);
        mma16816<T>(s[1], qa[i], kf[2], kf[3]);
      }
      uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // the lane's pairs of keys in V's registers
      const bool some = k0 + 16 > ke || p.mask;
      if (some) {
        // keys that take no part: their scores -inf, their values zeros (0 * NaN is NaN)
        const unsigned bits = __ballot_sync(0xffffffffu, v != 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const unsigned pair = bits >> (t * 8 + 2 * c);
          keep[t] = (pair & 1 ? 0x0000ffffu : 0u) | (pair & 2 ? 0xffff0000u : 0u);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] = pair >> (i & 1) & 1 ? s[t][i] * p.scale_log2 : -INFINITY;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] *= p.scale_log2;
      }
      float mx[2] = {fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                     fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))};
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float mn = fmaxf(m[r], mx[r]);
        mx[r] = mn == -INFINITY ? 0.f : mn;
        corr[r] = ex2(m[r] - mx[r]);
        m[r] = mn;
        l[r] *= corr[r];
      }
      uint32_t pa[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] = ex2(s[t][i] - mx[i >> 1]);
          l[i >> 1] += s[t][i];
        }
        pa[t * 2] = pack2<T>(s[t][0], s[t][1]);
        pa[t * 2 + 1] = pack2<T>(s[t][2], s[t][3]);
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          o[i][0] *= corr[0];
          o[i][1] *= corr[0];
          o[i][2] *= corr[1];
          o[i][3] *= corr[1];
        }
      }
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        uint32_t vf[4];
        ldsm4t(vf, av + (i >> 2) * kFewKeys * 128 + ((((i & 3) * 2 + vch) ^ sw) << 4));
        if (some) {
          vf[0] &= keep[0];
          vf[1] &= keep[1];
          vf[2] &= keep[0];
          vf[3] &= keep[1];
        }
        mma16816<T>(o[2 * i], pa, vf[0], vf[1]);
        mma16816<T>(o[2 * i + 1], pa, vf[2], vf[3]);
      }
      // the tile's reads are done before a copy may overwrite it: an arrival alone does
      // not order them before writes of the copy engine's
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + st);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) {
        s_m[w][g + 8 * r] = m[r];
        s_l[w][g + 8 * r] = l[r];
      }
    }
    // every tile was waited for by every warp before it passes this barrier,
    // so the tiles' memory takes the warps' results
    asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
    float* s_o = reinterpret_cast<float*>(base);
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        *reinterpret_cast<float2*>(s_o + (w * kRowTile + g + 8 * r) * LD + 8 * i + 2 * c) =
            make_float2(o[i][2 * r], o[i][2 * r + 1]);
    asm volatile("bar.sync 1, %0;" ::"n"(kFewWarps * 32) : "memory");
    // join the warps: 8 threads a row, each every eighth group of 8 columns
    const int row = tid >> 3, r = r0 + row;
    if (r < rows) {
      float mm = s_m[0][row];
#pragma unroll
      for (int q = 1; q < kFewWarps; ++q) mm = fmaxf(mm, s_m[q][row]);
      const float mb = mm == -INFINITY ? 0.f : mm;
      float f[kFewWarps], ll = 0.f;
#pragma unroll
      for (int q = 0; q < kFewWarps; ++q) {
        f[q] = ex2(s_m[q][row] - mb);
        ll = fmaf(s_l[q][row], f[q], ll);
      }
      const float inv = ll == 0.f ? 0.f : 1.0f / ll;
      const float lse = ll == 0.f ? -INFINITY : (mb + log2f(ll)) * 0.6931471805599453f;
      const int64_t t = bag.q0 + r / p.G;
      const int hq = h * p.G + r % p.G;
      for (int d = (tid & 7) * 8; d < p.D; d += 64) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
        for (int q = 0; q < kFewWarps; ++q) {
          RawVec<float, 8> raw;
          raw.load(s_o + (q * kRowTile + row) * LD + d);
          float x[8];
          raw.unpack(x);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = fmaf(x[j], f[q], v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv;
        if (p.splits == 1) store_vec(static_cast<T*>(p.out) + t * p.os + hq * p.oh + d, v);
        else store_vec(p.po + (((int64_t)sp * p.Tq + t) * p.Hq + hq) * p.D + d, v);
      }
      if ((tid & 7) == 0) {
        if (p.splits == 1) p.lse[t * p.Hq + hq] = lse;
        else p.pl[((int64_t)sp * p.Tq + t) * p.Hq + hq] = lse;
      }
    }
  }
  if (!ok) atomicOr(p.status, kErrTimeout);
}

// Joins the parts of the keys: out = sum_s exp(lse_s - lse) out_s; one warp a
// (query, head), 4 columns a lane.
template <typename T>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ AttendParams p) {
  const int lane = threadIdx.x & 31;
  const int tiles = (p.max_q * p.Hq + 3) / 4;
  const int b = blockIdx.x / tiles, i = (blockIdx.x % tiles) * 4 + (threadIdx.x >> 5);
  pdl_wait();
  const Bag bag = load_bag(p, b);
  if (i >= bag.nq * p.Hq) return;
  const int64_t t = bag.q0 + i / p.Hq;
  const int hq = i % p.Hq;
  const int n = max(1, (bag.nk + p.split_keys - 1) / p.split_keys);
  const int64_t step = p.Tq * p.Hq, at = t * p.Hq + hq;
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, p.pl[s * step + at]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int d = lane * 4;
  for (int s = 0; s < n; ++s) {
    const float f = expf(p.pl[s * step + at] - base);
    sum += f;
    if (d < p.D) {
      const float4 v = *reinterpret_cast<const float4*>(p.po + (s * step + at) * p.D + d);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  if (d < p.D) {
    uint2 u = make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + t * p.os + hq * p.oh + d) = u;
  }
  if (lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : base + logf(sum);
}

// ---------------------------------------------------------------- host
struct AttendPlan {
  int splits, split_keys;
  int64_t po_bytes, pl_bytes, delta_bytes, vnorm_bytes;  // delta_bytes: one array of rows
  int64_t bytes;
};

// The call with bounds of 0 raised to 1: the blocks that look at every bag's
// offsets run all the same.  The checks, the plan and the launches all take
// their sizes from this, so that a launch never needs more than its plan gave.
recis_attend_args launch_sizes(const recis_attend_args& a) {
  recis_attend_args c = a;
  if (c.max_q == 0) c.max_q = 1;
  if (c.max_k == 0) c.max_k = 1;
  return c;
}

// a: of launch_sizes
AttendPlan attend_plan(const recis_attend_args& a, bool backward) {
  AttendPlan g = {};
  g.splits = 1;
  g.split_keys = (int)a.max_k;
  if (backward) {
    // parts of the keys for grad_q.  Few rows: the keys' pass makes it, three
    // rounds of blocks on every SM even out the bags' lengths; many: a pass
    // over query tiles of its own, two blocks an SM.  At least 512 keys a part.
    const int64_t G = a.Hq / a.Hkv, rows = a.max_q * G;
    const bool few = few_back_rows(a.max_q, G);
    if (!few) g.delta_bytes = align256(a.Tq * a.Hq * 4);
    if (!few && a.type == RECIS_F16) g.vnorm_bytes = align256(value_slots(a.B, a.Tk) * a.Hkv * 4);
    const int64_t blocks = std::max<int64_t>(1, a.B * a.Hkv * (few ? 1 : (a.max_q + 128 / G - 1) / (128 / G)));
    const int64_t target = kSMs * (few ? 3 * few_back_per_sm(a.D, rows) : 2);
    const int64_t want = std::min<int64_t>((target + blocks - 1) / blocks, (a.max_k + 511) / 512);
    if (want > 1) {
      g.split_keys = (int)((a.max_k + want - 1) / want + 127) / 128 * 128;
      g.splits = (int)((a.max_k + g.split_keys - 1) / g.split_keys);
    }
    if (g.splits > 1) g.po_bytes = align256(g.splits * a.Tq * a.Hq * a.D * 4);
  } else {
    // parts of the keys: enough blocks for every SM to hold a few, each part
    // at least 256 keys (few rows: 4 tiles) or 512 (tiles: 4 steps)
    const int64_t G = a.Hq / a.Hkv;
    const bool few = few_rows(a.max_q, G);
    const int64_t tile = few ? std::max<int64_t>(kRowTile / G, 1) : 128 / G;  // queries a block
    const int64_t blocks = std::max<int64_t>(1, a.B * a.Hkv * ((a.max_q + tile - 1) / tile));
    const int64_t least = few ? 256 : 512;
    const int64_t want = std::min<int64_t>((kSMs * (few ? 8 : 4) + blocks - 1) / blocks, (a.max_k + least - 1) / least);
    if (want > 1) {
      g.split_keys = (int)((a.max_k + want - 1) / want + 127) / 128 * 128;
      g.splits = (int)((a.max_k + g.split_keys - 1) / g.split_keys);
    }
    if (g.splits > 1) {
      g.po_bytes = align256(g.splits * a.Tq * a.Hq * a.D * 4);
      g.pl_bytes = align256(g.splits * a.Tq * a.Hq * 4);
    }
  }
  g.bytes = g.po_bytes + g.pl_bytes + (g.vnorm_bytes ? 3 : 2) * g.delta_bytes + g.vnorm_bytes;
  return g;
}

recis_status check_sizes(const recis_attend_args* a, const char* what) {
  // room below 2^31 for coordinates and counts rounded up to tiles
  const int64_t top = INT32_MAX - 65536, bound = (int64_t)1 << 30;
  if ((a->type != RECIS_BF16 && a->type != RECIS_F16) || a->D < 8 || a->D > 128 || a->D % 8 != 0 || a->Hkv < 1 ||
      a->Hq < a->Hkv || a->Hq % a->Hkv != 0 || a->Hq / a->Hkv > 128 || a->B < 0 || a->Tq < 0 || a->Tk < 0 ||
      a->max_q < 0 || a->max_k < 0 || a->B >= top || a->Tq >= top || a->Tk >= top || a->max_q >= top ||
      a->max_k >= top || a->max_q * a->Hq > bound || a->max_k * a->Hkv > bound || !(a->scale > -1e30 && a->scale < 1e30)) {
    set_error(std::string(what) + ": bad arguments (bf16 or fp16, D a multiple of 8 up to 128, Hq a multiple of Hkv, max_q * Hq and max_k * Hkv up to 2^30)");
    return RECIS_ERR_INVALID_ARG;
  }
  return RECIS_OK;
}

// rows of heads of D elements: aligned for 16-byte accesses
bool bad_array(const void* p, int64_t stride, int64_t head_stride, int64_t rows) {
  return rows > 0 && (!p || misaligned(p, 16) || stride % 8 != 0 || head_stride % 8 != 0 || stride <= 0 ||
                      head_stride <= 0);
}

// bags, rows and blocks of a launch fit its grid
bool grid_fits(int64_t n) { return n < ((int64_t)1 << 31); }

// a: of launch_sizes; `given`: the caller's
recis_status fill(const recis_attend_args* a, const recis_attend_args* given, AttendParams* p, const AttendPlan& g,
                  void* ws) {
  int* st = sequence_status();
  if (!st) {
    set_error("the sequence operators' status word is not reachable (no usable sm_100 device?)");
    return RECIS_ERR_NO_DEVICE;
  }
  *p = AttendParams{};
  p->q = a->q; p->k = a->k; p->v = a->v; p->go = a->grad_out;
  p->out = a->out; p->gq = a->grad_q; p->gk = a->grad_k; p->gv = a->grad_v;
  p->lse = a->lse;
  p->qo = a->q_offsets; p->ko = a->k_offsets; p->mask = a->key_mask;
  p->qs = a->q_stride; p->qh = a->q_head_stride; p->ks = a->k_stride; p->kh = a->k_head_stride;
  p->vs = a->v_stride; p->vh = a->v_head_stride; p->os = a->out_stride; p->oh = a->out_head_stride;
  p->gos = a->grad_out_stride; p->goh = a->grad_out_head_stride;
  p->gqs = a->grad_q_stride; p->gqh = a->grad_q_head_stride; p->gks = a->grad_k_stride; p->gkh = a->grad_k_head_stride;
  p->gvs = a->grad_v_stride; p->gvh = a->grad_v_head_stride;
  p->Tq = a->Tq; p->Tk = a->Tk;
  p->B = (int)a->B; p->Hq = a->Hq; p->Hkv = a->Hkv; p->G = a->Hq / a->Hkv; p->D = a->D;
  p->max_q = (int)a->max_q; p->max_k = (int)a->max_k;
  p->bound_q = (int)given->max_q; p->bound_k = (int)given->max_k;
  p->scale = (float)a->scale;
  p->scale_log2 = (float)(a->scale * 1.4426950408889634);
  // a scale of 0 makes every score 0; 1e-30 does too, and keeps the -inf of keys that take no part
  if (p->scale_log2 == 0.f) p->scale_log2 = 1e-30f;
  p->splits = g.splits;
  p->split_keys = g.split_keys;
  char* at = static_cast<char*>(ws);
  p->po = reinterpret_cast<float*>(at);
  p->pl = reinterpret_cast<float*>(at + g.po_bytes);
  at += g.po_bytes + g.pl_bytes;
  p->delta = reinterpret_cast<float*>(at);
  p->nlse = reinterpret_cast<float*>(at + g.delta_bytes);
  p->gnorm = reinterpret_cast<float*>(at + 2 * g.delta_bytes);
  p->vnorm = reinterpret_cast<float*>(at + 3 * g.delta_bytes);
  p->status = st;
  return RECIS_OK;
}

template <typename T, int DP>
cudaError_t few_launch(const AttendParams& p, const CUtensorMap& mk, const CUtensorMap& mv, int64_t grid,
                       cudaStream_t s) {
  auto kernel = few_kernel<T, DP>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(kernel, FewCfg<DP>::kTotal, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, (unsigned)grid, kFewWarps * 32 + 32, FewCfg<DP>::kTotal, s, p, mk, mv, kSpinLimit);
}

template <typename T>
recis_status forward(const AttendParams& p, cudaStream_t s) {
  const bool few = few_rows(p.max_q, p.G);
  const int64_t rtiles = ((int64_t)p.max_q * p.G + kRowTile - 1) / kRowTile;
  const int64_t grid = (int64_t)p.B * p.splits * p.Hkv * rtiles, jgrid = (int64_t)p.B * (((int64_t)p.max_q * p.Hq + 3) / 4);
  if ((few && !grid_fits(grid)) || (p.splits > 1 && !grid_fits(jgrid))) {
    set_error("attend: too many blocks (bags times max_q times heads)");
    return RECIS_ERR_INVALID_ARG;
  }
  if (!few) {
    const recis_status st = launch_attend_tc(p, std::is_same<T, __nv_bfloat16>::value, s);
    if (st != RECIS_OK) return st;
  } else {
    LaunchScope ls("attend_few", s);
    constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap mk = {}, mv = {};
    if (p.Tk > 0 && (!rows_map(&mk, p.k, bf16, p.D, p.Hkv, p.Tk, p.ks, p.kh, 1, kFewKeys) ||
                     !rows_map(&mv, p.v, bf16, p.D, p.Hkv, p.Tk, p.vs, p.vh, 1, kFewKeys))) {
      set_error("attend: the driver refused a tensor map");
      return RECIS_ERR_CUDA;
    }
    const cudaError_t e = p.D <= 64 ? few_launch<T, 64>(p, mk, mv, grid, s) : few_launch<T, 128>(p, mk, mv, grid, s);
    if (e != cudaSuccess) return cuda_fail(e, "attend launch");
  }
  cudaError_t e;
  if (p.splits > 1) {
    LaunchScope ls("attend_join", s);
    e = launch_pdl(join_kernel<T>, (unsigned)jgrid, 128, 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "attend_join launch");
  }
  return RECIS_OK;
}

}  // namespace
}  // namespace recis

using namespace recis;

// null pointers are refused with the sizes
static recis_attend_args sizes_of(const recis_attend_args* a) { return a ? launch_sizes(*a) : recis_attend_args{}; }

extern "C" recis_status recis_attend_workspace(const recis_attend_args* args, int32_t backward, int64_t* bytes_out) {
  const recis_attend_args c = sizes_of(args), *a = &c;
  recis_status st = check_sizes(a, "attend_workspace");
  if (st != RECIS_OK) return st;
  if (!bytes_out) {
    set_error("attend_workspace: null argument");
    return RECIS_ERR_INVALID_ARG;
  }
  *bytes_out = attend_plan(*a, backward != 0).bytes;
  return RECIS_OK;
}

static recis_status check_call(const recis_attend_args* a, bool backward, void* ws, int64_t ws_bytes, const char* what) {
  const recis_status st = check_sizes(a, what);
  if (st != RECIS_OK) return st;
  bool bad = (a->B > 0 && (!a->q_offsets || !a->k_offsets)) || misaligned(a->q_offsets, 8) ||
             misaligned(a->k_offsets, 8) || misaligned(a->lse, 4) || (a->Tq > 0 && !a->lse);
  bad = bad || bad_array(a->q, a->q_stride, a->q_head_stride, a->Tq) ||
        bad_array(a->k, a->k_stride, a->k_head_stride, a->Tk) || bad_array(a->v, a->v_stride, a->v_head_stride, a->Tk) ||
        bad_array(a->out, a->out_stride, a->out_head_stride, a->Tq);
  if (backward)
    bad = bad || bad_array(a->grad_out, a->grad_out_stride, a->grad_out_head_stride, a->Tq) ||
          bad_array(a->grad_q, a->grad_q_stride, a->grad_q_head_stride, a->Tq) ||
          bad_array(a->grad_k, a->grad_k_stride, a->grad_k_head_stride, a->Tk) ||
          bad_array(a->grad_v, a->grad_v_stride, a->grad_v_head_stride, a->Tk);
  if (bad) {
    set_error(std::string(what) + ": null or misaligned array, or a stride that is not a multiple of 8 elements");
    return RECIS_ERR_INVALID_ARG;
  }
  const int64_t need = attend_plan(*a, backward).bytes;
  if (misaligned(ws, 256) || (need > 0 && (!ws || ws_bytes < need))) {
    set_error(std::string(what) + ": workspace too small or not 256-byte aligned");
    return RECIS_ERR_INVALID_ARG;
  }
  return RECIS_OK;
}

extern "C" recis_status recis_attend(const recis_attend_args* args, void* workspace, int64_t workspace_bytes,
                                     recis_stream_t stream) {
  const recis_attend_args c = sizes_of(args), *a = &c;
  recis_status st = check_call(a, false, workspace, workspace_bytes, "attend");
  if (st != RECIS_OK) return st;
  if (a->B == 0 || a->Tq == 0) return RECIS_OK;
  AttendParams p;
  if ((st = fill(a, args, &p, attend_plan(*a, false), workspace)) != RECIS_OK) return st;
  return a->type == RECIS_BF16 ? forward<__nv_bfloat16>(p, (cudaStream_t)stream)
                               : forward<__half>(p, (cudaStream_t)stream);
}

extern "C" recis_status recis_attend_backward(const recis_attend_args* args, void* workspace, int64_t workspace_bytes,
                                              recis_stream_t stream) {
  const recis_attend_args c = sizes_of(args), *a = &c;
  recis_status st = check_call(a, true, workspace, workspace_bytes, "attend_backward");
  if (st != RECIS_OK) return st;
  if (a->B == 0) return RECIS_OK;
  AttendParams p;
  if ((st = fill(a, args, &p, attend_plan(*a, true), workspace)) != RECIS_OK) return st;
  return launch_attend_back(p, a->type == RECIS_BF16, (cudaStream_t)stream);
}
