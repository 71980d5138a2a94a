// attend_tc.cu -- attention forward for many queries, on the tensor cores.
//
// One block (CTA) takes 128 rows of one key head -- row r is query r / G, head
// r % G of the group -- against one part of the bag's keys, 128 keys a step:
//
//   S = Q K^T        128 x 128, fp32, tensor memory
//   P = exp2(c S - m), row sums l;  P overwrites S as 16-bit values
//   O = O + P V      128 x D, fp32, tensor memory; P is read from there
//
// Warps 0-3 do the softmax, one row a thread, so a row's maximum and sum need
// no exchange; warp 4 issues the tensor-map copies, warp 5 the products.  Two
// blocks share an SM (half of tensor memory and less than half of shared
// memory each): one's products run under the other's exponentials.  O is
// rescaled only when a row's maximum has grown by more than 2^8 since the last
// time (P then stays below 2^8 and sums stay fp32), which after the first
// steps is rare.  (Attention kernels commonly rescale so seldom; the bound and its
// place here are this kernel's own.)
//
// Measured on B200, bf16: 4 bags of 4096 queries over 4096 keys, 8 heads of 128,
// 249 us, 1105 TFLOP/s (0.66 of the measured matrix peak); heads of 64, 205 us, 670
// TFLOP/s.  Products and exponentials each fill about half of the time (1024
// cycles a tile each); what is left is the chain scores - softmax - values, which
// two blocks an SM overlap only in part.
//
// A copy brings whole tiles of 128 rows, so the last one of a bag holds rows of
// the next bag.  Their scores are replaced by -inf, and their V rows (like
// those of masked keys) are overwritten with zeros before the product, because
// 0 * NaN is NaN.
#include "attend.cuh"
#include "tc.cuh"

namespace recis {

namespace {

constexpr int kTile = 128;              // rows of Q, keys a step
constexpr int kTcThreads = 192;
constexpr uint32_t kTmemCols = 256;     // S (then P) 0..127, O 128..255
constexpr float kLazy = 8.0f;           // growth of the maximum (log2) that O is rescaled at

template <int DP>
struct FwdSmem {
  static constexpr int kBlocks = DP / 64;                 // 64-element blocks of a row
  static constexpr int kBytes = kBlocks * kTile * 128;    // one tile
  static constexpr int kStages = DP == 64 ? 2 : 1;        // K and V tiles each
  static constexpr int kTiles = (1 + 2 * kStages) * kBytes;
  static constexpr int kTotal = kTiles + 1024 + 256;      // alignment, barriers
};

template <typename T, int DP>
__global__ void __launch_bounds__(kTcThreads, 2)
    attend_tc_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap mq,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, int spin_max) {
  using L = FwdSmem<DP>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t s_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sq = base;
  uint8_t* sk = sq + L::kBytes;
  uint8_t* sv = sk + NS * L::kBytes;
  uint64_t* bar = reinterpret_cast<uint64_t*>(sv + NS * L::kBytes);
  uint64_t *q_full = bar, *s_full = bar + 1, *o_full = bar + 2, *p_full = bar + 3;  // p_full: two halves of a tile
  uint64_t *k_full = bar + 5, *k_empty = k_full + NS, *v_full = k_empty + NS, *v_empty = v_full + NS;
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_valid[2][4];

  const int TQ = kTile / p.G;  // queries a tile
  const int qtiles = (p.max_q + TQ - 1) / TQ;
  unsigned id = blockIdx.x;
  const int qt = id % qtiles;
  id /= qtiles;
  const int h = id % p.Hkv;
  id /= p.Hkv;
  pdl_wait();
  pdl_trigger();  // the join may be brought in; it waits for this grid's end
  const int sp = id % p.splits, b = id / p.splits;
  const Bag bag = load_bag(p, b);
  const int t0 = qt * TQ;
  const int ks = sp * p.split_keys, ke = min(ks + p.split_keys, bag.nk);
  if (t0 >= bag.nq || (ks >= bag.nk && sp > 0)) return;
  const int n = ke > ks ? (ke - ks + kTile - 1) / kTile : 0;  // steps

  const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (w == 5) tmem_alloc(&s_tmem, kTmemCols);
  if (tid == 128) {
    mbar_init(q_full, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, kTile);
    mbar_init(p_full + 1, kTile);
    mbar_init(o_full, 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;  // false: a wait gave up

  if (w == 4) {  // copies
    if (lane == 0 && n > 0) {
      prefetch_map(&mq);
      prefetch_map(&mk);
      prefetch_map(&mv);
      mbar_arrive_expect(q_full, (unsigned)(L::kBlocks * TQ * p.G * 128));
      for (int i = 0; i < L::kBlocks; ++i)
        tma_load3(sq + i * kTile * 128, &mq, 64 * i, h * p.G, (int)(bag.q0 + t0), q_full);
      int nk = 0, nv = 0;  // K and V tiles asked for
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % NS, ph = (j / NS) & 1;
        const int row = (int)(bag.k0 + ks + j * kTile);
        if (j >= NS) ok = mbar_wait(k_empty + st, ph ^ 1, spin_max);
        if (!ok) break;
        mbar_arrive_expect(k_full + st, L::kBytes);
        for (int i = 0; i < L::kBlocks; ++i)
          tma_load3(sk + st * L::kBytes + i * kTile * 128, &mk, 64 * i, h, row, k_full + st);
        nk = j + 1;
        if (j >= NS) ok = mbar_wait(v_empty + st, ph ^ 1, spin_max);
        if (!ok) break;
        mbar_arrive_expect(v_full + st, L::kBytes);
        for (int i = 0; i < L::kBlocks; ++i)
          tma_load3(sv + st * L::kBytes + i * kTile * 128, &mv, 64 * i, h, row, v_full + st);
        nv = j + 1;
      }
      // copies in flight end before the block does
      ok = mbar_wait(q_full, 0, spin_max) && ok;
      for (int j = max(nk - NS, 0); j < nk; ++j) ok = mbar_wait(k_full + j % NS, (j / NS) & 1, spin_max) && ok;
      for (int j = max(nv - NS, 0); j < nv; ++j) ok = mbar_wait(v_full + j % NS, (j / NS) & 1, spin_max) && ok;
    }
    __syncwarp();
  } else if (w == 5) {  // products
    if (n > 0) {
      constexpr uint32_t id_s = mma_desc<T>(kTile, kTile, false, false), id_o = mma_desc<T>(kTile, DP, false, true);
      // descriptors count 16 bytes
      const uint64_t dq = smem_desc(smem_u32(sq), 16), dk = smem_desc(smem_u32(sk), 16);
      const uint64_t dv = smem_desc(smem_u32(sv), kTile * 128);
      const bool one = elect_one();
      ok = warp_wait(q_full, 0, spin_max);
      for (int j = 0; j < n && ok; ++j) {
        const int st = j % NS, ph = (j / NS) & 1;
        if (!(ok = warp_wait(k_full + st, ph, spin_max))) break;
        tc_fence_after();
        if (one) {
          const uint64_t b = dk + st * (L::kBytes >> 4);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint32_t off = ((k >> 2) * kTile * 128 + (k & 3) * 32) >> 4;
            mma_ss(tmem, dq + off, b + off, id_s, k > 0);
          }
          mma_commit(s_full);
          mma_commit(k_empty + st);
        }
        __syncwarp();
        if (!(ok = warp_wait(v_full + st, ph, spin_max))) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!(ok = warp_wait(p_full + half, j & 1, spin_max))) break;
          tc_fence_after();
          if (one) {
            const uint64_t b = dv + st * (L::kBytes >> 4);
#pragma unroll
            for (int k = half * kTile / 32; k < (half + 1) * kTile / 32; ++k)
              mma_ts(tmem + 128, tmem + 8 * k, b + (k * 2048 >> 4), id_o, j > 0 || k > 0);
            if (half == 1) mma_commit(v_empty + st);
          }
          __syncwarp();
        }
      }
      if (one) mma_commit(o_full);
      ok = warp_wait(o_full, 0, spin_max) && ok;
    }
    __syncwarp();
  } else {  // softmax: thread tid is row tid
    const uint32_t mine = tmem + ((uint32_t)w << 21);  // lane 32 w
    const float c = p.scale_log2;
    // the score of a key that takes no part: -inf once scaled (c is never 0)
    const uint32_t out_of = __float_as_uint(c >= 0.f ? -INFINITY : INFINITY);
    // whether key tid of step j takes part: not 0 (the byte is not looked at before its turn)
    auto takes = [&](int j) -> unsigned {
      const int key = ks + j * kTile + tid;
      unsigned m = key < ke;
      if (m && p.mask) m = __ldg(p.mask + bag.k0 + key);
      return m;
    };
    unsigned v_next = takes(0);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const int k0 = ks + j * kTile;
      const bool tail = k0 + kTile > ke || p.mask;
      const unsigned v = v_next;
      v_next = takes(j + 1);
      if (tail) {  // which of the tile's keys take part
        const unsigned bits = __ballot_sync(0xffffffffu, v != 0);
        if (lane == 0) s_valid[j & 1][w] = bits;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        // Rows of V that take no part are zeroed.  The scores come first: they were
        // asked for after the tile before had taken its V, so that only then the wait
        // for V's copy is one for this tile's (earlier, with the V of the tile before
        // still on its way, the parity of the one before that would pass).
        const int st = j % NS;
        ok = ok && mbar_wait(s_full, j & 1, spin_max) && mbar_wait(v_full + st, (j / NS) & 1, spin_max);
        if (!v)
          for (int i = 0; i < L::kBlocks; ++i) {
            uint4* row = reinterpret_cast<uint4*>(sv + st * L::kBytes + (i * kTile + tid) * 128);
#pragma unroll
            for (int c = 0; c < 8; ++c) row[c] = make_uint4(0, 0, 0, 0);
          }
        fence_async_smem();
      }
      // a warp that gave up goes on without waiting: the others' barrier needs it
      ok = ok && mbar_wait(s_full, j & 1, spin_max);
      __syncwarp();
      tc_fence_after();
      uint32_t r[kTile];  // the row's scores, in registers from here on
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(mine + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * q));
      tmem_wait_ld();
      if (tail) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t bits = s_valid[j & 1][q];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(bits >> i & 1)) r[32 * q + i] = out_of;
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (c >= 0.f) {
#pragma unroll
        for (int i = 0; i < kTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(r[i]));
      } else {
#pragma unroll
        for (int i = 0; i < kTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], -__uint_as_float(r[i]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // the maximum that P is taken against: kept while it is near enough
      const float grown = fmaxf(m, top == -INFINITY ? top : top * fabsf(c));
      const bool move = j == 0 || grown > m + kLazy;
      if (__any_sync(0xffffffffu, move)) {
        // each row by its own maximum: the warp's other rows, which may be another
        // bag's or none, do not show in it
        const float next = move && grown != -INFINITY ? grown : m;
        const float f = !move ? 1.f : m == -INFINITY ? 0.f : ex2(m - next);
        m = next;
        l *= f;
        if (j > 0) {
#pragma unroll
          for (int q = 0; q < DP / 16; ++q) {
            uint32_t o[16];
            tmem_ld16(mine + 128 + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(mine + 128 + 16 * q, o);
          }
        }
      }
      const float mb = m == -INFINITY ? 0.f : -m;
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float2 a = fma2(as_f2(r[32 * q + i], r[32 * q + i + 1]), make_float2(c, c), make_float2(mb, mb));
          float2 b = fma2(as_f2(r[32 * q + i + 2], r[32 * q + i + 3]), make_float2(c, c), make_float2(mb, mb));
          a = make_float2(ex2(a.x), ex2(a.y));
          b = make_float2(ex2(b.x), ex2(b.y));
          s0 = add2(s0, a);
          s1 = add2(s1, b);
          pk[i / 2] = pack2<T>(a.x, a.y);
          pk[i / 2 + 1] = pack2<T>(b.x, b.y);
        }
        tmem_st16(mine + 16 * q, pk);
        if (q & 1) {  // half of the row is there: its product may start
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_full + (q >> 1));
        }
      }
      s0 = add2(s0, s1);
      l += s0.x + s0.y;
    }
    if (n > 0) ok = ok && mbar_wait(o_full, 0, spin_max);
    tc_fence_after();
    const int r = tid;
    const bool live = r < TQ * p.G && t0 + r / p.G < bag.nq;
    const int64_t t = bag.q0 + t0 + r / p.G;
    const int hq = h * p.G + r % p.G;
    const float inv = l == 0.f ? 0.f : 1.0f / l;
    const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    const bool have = n > 0 && ok;
    // the thread's row goes to shared memory (Q is done with), 8 lanes store a
    // row's 128 bytes together; parts are stored directly, in fp32
#pragma unroll
    for (int q = 0; q < DP / 32; ++q) {
      uint32_t o[32];
      if (have) {
        tmem_ld32(mine + 128 + 32 * q, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 32 * q + 8 * i;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = !have || l == 0.f ? 0.f : __uint_as_float(o[8 * i + e]) * inv;
        if (p.splits == 1)
          *reinterpret_cast<uint4*>(sq + (q >> 1) * kTile * 128 + r * 128 + (((4 * (q & 1) + i) ^ (r & 7)) << 4)) =
              make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
        else if (live && d < p.D)
          store_vec(p.po + (((int64_t)sp * p.Tq + t) * p.Hq + hq) * p.D + d, f);
      }
    }
    if (p.splits == 1) {
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int blk = 0; blk < L::kBlocks; ++blk)
        for (int i = 0; i < 8; ++i) {
          const int rr = w * 32 + 4 * i + (lane >> 3), ch = lane & 7, d = 64 * blk + 8 * ch;
          const int qq = rr / p.G, g = rr - qq * p.G;
          const uint4 u = *reinterpret_cast<const uint4*>(sq + blk * kTile * 128 + rr * 128 + ((ch ^ (rr & 7)) << 4));
          if (rr < TQ * p.G && t0 + qq < bag.nq && d < p.D)
            *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (bag.q0 + t0 + qq) * p.os + (h * p.G + g) * p.oh + d) = u;
        }
    }
    if (live) {
      if (p.splits == 1) p.lse[t * p.Hq + hq] = lse;
      else p.pl[((int64_t)sp * p.Tq + t) * p.Hq + hq] = lse;
    }
  }
  if (!ok) atomicOr(p.status, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 5) tmem_free(tmem, kTmemCols);
}

}  // namespace

bool rows_map(CUtensorMap* map, const void* p, bool bf16, int D, int H, int64_t T, int64_t stride, int64_t head_stride,
              int heads, int rows) {
  using Encode = decltype(&::cuTensorMapEncodeTiled);
  static Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return (Encode)fn;
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)rows};
  const cuuint32_t one[3] = {1, 1, 1};
  auto make = [&] {
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  if (make() == CUDA_SUCCESS) return true;
  // A host thread's first CUDA call: it has no context yet, which the runtime's
  // calls make current and the driver's do not.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && make() == CUDA_SUCCESS;
}

template <typename T, int DP>
static cudaError_t tc_launch(const AttendParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                             int64_t grid, cudaStream_t s) {
  auto kernel = attend_tc_kernel<T, DP>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e =
      allow_smem(kernel, FwdSmem<DP>::kTotal, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, (unsigned)grid, kTcThreads, FwdSmem<DP>::kTotal, s, p, mq, mk, mv, kSpinLimit);
}

recis_status launch_attend_tc(const AttendParams& p, bool bf16, cudaStream_t s) {
  const int TQ = kTile / p.G;
  const int64_t grid = (int64_t)p.B * p.splits * p.Hkv * (((int64_t)p.max_q + TQ - 1) / TQ);
  if (grid >= ((int64_t)1 << 31)) {
    set_error("attend: too many blocks (bags times max_q times heads)");
    return RECIS_ERR_INVALID_ARG;
  }
  CUtensorMap mq = {}, mk = {}, mv = {};
  // without keys the maps of K and V are never used
  if (!rows_map(&mq, p.q, bf16, p.D, p.Hq, p.Tq, p.qs, p.qh, p.G, TQ) ||
      (p.Tk > 0 && (!rows_map(&mk, p.k, bf16, p.D, p.Hkv, p.Tk, p.ks, p.kh, 1, kTile) ||
                    !rows_map(&mv, p.v, bf16, p.D, p.Hkv, p.Tk, p.vs, p.vh, 1, kTile)))) {
    set_error("attend: the driver refused a tensor map");
    return RECIS_ERR_CUDA;
  }
  LaunchScope ls("attend_tc", s);
  cudaError_t e;
  if (p.D <= 64)
    e = bf16 ? tc_launch<__nv_bfloat16, 64>(p, mq, mk, mv, grid, s) : tc_launch<__half, 64>(p, mq, mk, mv, grid, s);
  else
    e = bf16 ? tc_launch<__nv_bfloat16, 128>(p, mq, mk, mv, grid, s) : tc_launch<__half, 128>(p, mq, mk, mv, grid, s);
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "attend launch");
}

}  // namespace recis
