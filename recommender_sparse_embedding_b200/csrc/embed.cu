// embed.cu -- dense embedding tables: rows of a [V][D] weight looked up by
// token with a scale, and the weight's gradient by sorted tokens.
//
//   out[i] = scale * W[t_i]            dW[v] = scale * sum_{i : t_i = v} dout[i]
//
// Both are bound by memory: the lookup reads N rows and writes N, the
// gradient reads N rows of dout and writes the V rows of dW.
//
// The gradient sorts (token, position) by a stable radix sort, so that a row's
// terms are added in occurrence order whatever the scheduling.  The sort moves
// little and is bound by latency; its kernels carry extra blocks that write
// the zeros of dW beside it.  The sorted positions are cut into spans; a group
// of lanes walks one span, 8 columns a lane, adds the rows of equal tokens in
// fp32, and goes on into the next span to finish a run that ends there.  A
// longer run (a hot token) leaves one fp32 partial per span, and a second
// kernel adds those in span order in fp64: no float atomic is used.
//
// Measured on B200 (L2 flushed): 1.5M tokens over 1M rows of 128, fp32 weight to
// bf16 rows, 125-130 us, 5.5 TB/s of DRAM traffic; their gradient (bf16 to fp32, dW
// of 512 MB) 278 us, of which the spans 127 us at 4.5 TB/s, the sort about 125 us
// with the 77 us worth of zeros beside it, the join 20 us.
#include <algorithm>

#include "seqops.cuh"

namespace recis {

namespace {

__device__ int g_seq_status;

// up to here one kernel finds and sums each token's rows (1000 tokens over 1000
// rows of 64: 9.5 us, 19.7 by sorting)
constexpr int kSmallN = 1024;
constexpr int kSortThreads = 256;
constexpr int kMaxDigit = 10;     // bits a pass sorts by
constexpr int kMaxSpan = 64;      // sorted positions a group of lanes walks: 16, 32 or 64
constexpr int kMaxSpans = 64;     // spans a block takes

// ---------------------------------------------------------------- lookup
struct LookupParams {
  const void* w;
  const int64_t* tok;
  void* out;
  int64_t V, N, out_stride, padding;
  int D, units, lanes;  // lanes: threads a row (a power of two)
  float scale;
  int* status;
};

// `lanes` threads walk the columns of R rows at once, so R independent row
// loads a thread are in flight; the next rows' tokens are read meanwhile.
template <typename TW, typename TO, int VEC, int R>
__global__ void __launch_bounds__(256, R == 1 ? 6 : 4) embed_lookup_kernel(const __grid_constant__ LookupParams p) {
  const int lane = threadIdx.x & (p.lanes - 1);
  const int64_t step = (int64_t)gridDim.x * (256 / p.lanes) * R;
  int64_t r0 = ((int64_t)blockIdx.x * (256 / p.lanes) + threadIdx.x / p.lanes) * R;
  int64_t t[R];
  auto tokens = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < R; ++i) t[i] = r + i < p.N ? __ldg(p.tok + r + i) : p.padding;
  };
  tokens(r0);
  for (; r0 < p.N; r0 += step) {
    int row[R];  // -1: zeros
#pragma unroll
    for (int i = 0; i < R; ++i) {
      row[i] = t[i] >= 0 && t[i] < p.V && t[i] != p.padding ? (int)t[i] : -1;
      if (row[i] < 0 && t[i] != p.padding && lane == 0) atomicOr(p.status, kErrTagOverflow);
    }
    tokens(r0 + step);
    for (int c = lane; c < p.units; c += p.lanes) {
      RawVec<TW, VEC> v[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (row[i] >= 0) v[i].load(static_cast<const TW*>(p.w) + (int64_t)row[i] * p.D + c * VEC);
      TO* out = static_cast<TO*>(p.out) + r0 * p.out_stride + c * VEC;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (r0 + i >= p.N) break;
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = 0.f;
        if (row[i] >= 0) {
          v[i].unpack(f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[j] *= p.scale;
        }
        store_vec(out + i * p.out_stride, f);
      }
    }
  }
}

template <typename TW, typename TO, int VEC>
cudaError_t lookup_launch(LookupParams p, cudaStream_t s) {
  p.units = p.D / VEC;
  p.lanes = 1;
  while (p.lanes < p.units && p.lanes < 256) p.lanes *= 2;
  // four rows a group once that still fills the machine, one row each below
  // (1.5M rows of 128: 122 and 134 us; 64 rows of 1024: 2.9 and 2.5)
  const bool many = p.N / 4 * p.lanes >= (int64_t)kSMs * 1024;
  const int64_t groups = many ? (p.N + 3) / 4 : p.N;
  const int64_t blocks = std::min<int64_t>((groups * p.lanes + 255) / 256, kSMs * (many ? 4 : 6));
  LaunchScope ls("embed_lookup", s);
  if (many) embed_lookup_kernel<TW, TO, VEC, 4><<<(unsigned)blocks, 256, 0, s>>>(p);
  else embed_lookup_kernel<TW, TO, VEC, 1><<<(unsigned)blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- gradient: radix sort
// Sort key of a token: itself, or V for padding and tokens out of range (they
// end up behind every row).
__device__ __forceinline__ uint32_t sort_key(int64_t t, int64_t V, int64_t padding, int* status, bool report) {
  if (t == padding) return (uint32_t)V;
  if (t < 0 || t >= V) {
    if (report) atomicOr(status, kErrTagOverflow);
    return (uint32_t)V;
  }
  return (uint32_t)t;
}

// Zeros written by the blocks behind a kernel's own: [at, at + bytes), 16-byte
// aligned, kZeroBytes a block.
constexpr int kZeroBytes = 64 * 1024;
struct ZeroSlice {
  char* at;
  int64_t bytes;
};
__device__ __forceinline__ void zero_block(const ZeroSlice& z, int64_t block) {
  const int64_t lo = block * kZeroBytes, hi = lo + kZeroBytes < z.bytes ? lo + kZeroBytes : z.bytes;
  for (int64_t i = lo + (int64_t)threadIdx.x * 16; i < hi; i += (int64_t)blockDim.x * 16)
    *reinterpret_cast<uint4*>(z.at + i) = make_uint4(0, 0, 0, 0);
}

struct PassParams {
  const int64_t* tok;       // first pass: the tokens; later passes read `in`
  const uint2* in;          // {key, position}
  uint2* out;
  int64_t N, V, padding;
  int shift, bits;          // the pass's digit
  int tiles;
  uint32_t* hist;           // [tiles][bins]: counts, then exclusive prefixes over tiles
  uint32_t* total;          // [bins]
  int* listed;              // runs listed for the join: cleared by the first pass
  int* status;
  ZeroSlice zero[3];        // beside the count, the scan and the scatter
};

__device__ __forceinline__ uint2 pass_item(const PassParams& p, int64_t i, bool report) {
  if (p.in) return p.in[i];  // written by the kernel before: no read-only path
  return make_uint2(sort_key(__ldg(p.tok + i), p.V, p.padding, p.status, report), (uint32_t)i);
}

// digit counts of each tile
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) grad_count_kernel(const __grid_constant__ PassParams p) {
  __shared__ uint32_t s_h[1 << kMaxDigit];
  const int bins = 1 << p.bits;
  pdl_wait();
  if ((int)blockIdx.x >= p.tiles) {
    zero_block(p.zero[0], blockIdx.x - p.tiles);
    return;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && !p.in) *p.listed = 0;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) s_h[b] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * (kSortThreads * ITEMS);
  uint32_t key[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int64_t i = base + j * kSortThreads + threadIdx.x;
    key[j] = i < p.N ? pass_item(p, i, true).x : 0;
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j)
    if (base + j * kSortThreads + threadIdx.x < p.N) atomicAdd(&s_h[(key[j] >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  pdl_trigger();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) p.hist[(size_t)blockIdx.x * bins + b] = s_h[b];
}

// exclusive prefix over tiles of each bin's counts, and its total; a block
// takes 32 bins, warp w the w-th part of the tiles
__global__ void __launch_bounds__(1024) grad_scan_kernel(const __grid_constant__ PassParams p) {
  __shared__ uint32_t s_part[32][33];
  const int bins = 1 << p.bits, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int b = blockIdx.x * 32 + lane;
  const int per = (p.tiles + 31) / 32;
  const int t0 = min(w * per, p.tiles), t1 = min(t0 + per, p.tiles);
  pdl_wait();
  if (blockIdx.x * 32 >= bins) {
    zero_block(p.zero[1], blockIdx.x - (bins + 31) / 32);
    return;
  }
  uint32_t sum = 0;
  if (b < bins)
#pragma unroll 8
    for (int t = t0; t < t1; ++t) sum += p.hist[(size_t)t * bins + b];
  s_part[w][lane] = sum;
  __syncthreads();
  uint32_t run = 0;
  for (int q = 0; q < w; ++q) run += s_part[q][lane];
  if (b < bins) {
    for (int t = t0; t < t1; ++t) {
      const uint32_t c = p.hist[(size_t)t * bins + b];
      p.hist[(size_t)t * bins + b] = run;
      run += c;
    }
    if (w == 31) p.total[b] = run;
  }
  pdl_trigger();
}

// stable move: a key's place = keys of lower digits + the same digit's keys in
// earlier tiles, earlier warps of the tile, and before it in its warp
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) grad_scatter_kernel(const __grid_constant__ PassParams p) {
  constexpr int kWarps = kSortThreads / 32;
  extern __shared__ uint32_t s_cnt[];  // [kWarps][bins], then the digits' bases [bins]
  __shared__ uint32_t s_w[kWarps];
  const int bins = 1 << p.bits, tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint32_t* s_base = s_cnt + kWarps * bins;
  if ((int)blockIdx.x < p.tiles)
    for (int b = tid; b < kWarps * bins; b += kSortThreads) s_cnt[b] = 0;
  pdl_wait();
  if ((int)blockIdx.x >= p.tiles) {
    zero_block(p.zero[2], blockIdx.x - p.tiles);
    return;
  }
  // the tile's keys and counts, all in flight at once
  const int64_t base = (int64_t)blockIdx.x * (kSortThreads * ITEMS) + (int64_t)w * 32 * ITEMS + lane;
  uint2 v[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j)
    v[j] = base + j * 32 < p.N ? pass_item(p, base + j * 32, false) : make_uint2(0, 0);
  // exclusive scan of the digit totals: 4 (at most) consecutive bins a thread
  constexpr int kPer = (1 << kMaxDigit) / kSortThreads;
  uint32_t tot[kPer], pre[kPer], mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = tid * kPer + j;
    tot[j] = b < bins ? p.total[b] : 0;
    pre[j] = b < bins ? p.hist[(size_t)blockIdx.x * bins + b] : 0;
    mine += tot[j];
  }
  uint32_t x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) s_w[w] = x;
  __syncthreads();
  uint32_t run = x - mine;
  for (int q = 0; q < w; ++q) run += s_w[q];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int b = tid * kPer + j;
    if (b < bins) s_base[b] = run + pre[j];
    run += tot[j];
  }
  // ranks within the warp's keys, in order
  uint32_t* cnt = s_cnt + w * bins;
  uint32_t rank[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const bool ok = base + j * 32 < p.N;
    const uint32_t d = (v[j].x >> p.shift) & (bins - 1);
    unsigned peers = __ballot_sync(0xffffffffu, ok);
    for (int b = 0; b < p.bits; ++b) {
      const unsigned m = __ballot_sync(0xffffffffu, d >> b & 1);
      peers &= (d >> b & 1) ? m : ~m;
    }
    if (!ok) peers = 0;
    const uint32_t before = ok ? cnt[d] : 0;
    rank[j] = before + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (ok && lane == __ffs(peers) - 1) cnt[d] = before + __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  for (int b = tid; b < bins; b += kSortThreads) {
    uint32_t at = s_base[b], c[kWarps];
#pragma unroll
    for (int q = 0; q < kWarps; ++q) c[q] = s_cnt[q * bins + b];
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      s_cnt[q * bins + b] = at;
      at += c[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < ITEMS; ++j)
    if (base + j * 32 < p.N) p.out[cnt[(v[j].x >> p.shift) & (bins - 1)] + rank[j]] = v[j];
  pdl_trigger();
}

// ---------------------------------------------------------------- gradient: sums
struct SumParams {
  const uint2* pairs;   // sorted {token, position}
  const int64_t* tok;   // small path: the tokens
  const void* g;
  void* dw;
  float* partial;       // [spans][2][D]: parts of runs that the join adds up, 0 begun before the span, 1 in it
  int2* list;           // those runs' first spans and tokens, *listed of them
  int* listed;
  int* run_last;        // [V]: the span each of them ends in, by token
  int64_t N, V, g_stride, padding;
  int D, units, lanes;
  int span, spb;        // positions a span; spans a block
  int accumulate;
  float scale;
  int* status;
};

// dw[row][c ..] (+)= scale * f
template <typename TO, int VEC>
__device__ __forceinline__ void grad_store(const SumParams& p, int64_t row, int c, float (&f)[VEC]) {
  TO* at = static_cast<TO*>(p.dw) + row * p.D + (int64_t)c * VEC;
  if (p.accumulate) {
    RawVec<TO, VEC> old;
    old.load(at);
    float o[VEC];
    old.unpack(o);
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] = fmaf(p.scale, f[j], o[j]);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) f[j] *= p.scale;
  }
  store_vec(at, f);
}

// One group of `lanes` lanes (at most a warp) walks one span; blockIdx.y picks
// the group's columns.  The block's sorted pairs are brought to shared memory
// at once, so that a group's row loads, 8 at a time, wait for nothing else.  A
// run belongs to the span it begins in; one that ends in the next span is
// finished by its owner (the next span's group passes over it), one that goes
// on further is listed and left in parts.
template <typename TG, typename TO, int VEC>
__global__ void __launch_bounds__(256, 3) grad_span_kernel(const __grid_constant__ SumParams p) {
  constexpr int U = 8;
  // pairs from one span and a position before the block's first span to one span behind its last
  __shared__ uint2 s_pair[(kMaxSpans + 2) * kMaxSpan + 2];
  const int lane = threadIdx.x & (p.lanes - 1), S = p.span;
  const int64_t b0 = (int64_t)blockIdx.x * p.spb * S, lo = b0 - S - 1;
  const uint32_t none = (uint32_t)p.V;  // key of positions without a row
  pdl_wait();
  for (int i = threadIdx.x; i < (p.spb + 2) * S + 2; i += blockDim.x) {
    const int64_t at = lo + i;
    s_pair[i] = at >= 0 && at < p.N ? p.pairs[at] : make_uint2(none, 0);
  }
  __syncthreads();
  const int64_t span = (int64_t)blockIdx.x * p.spb + threadIdx.x / p.lanes;
  const int64_t p0 = span * S;
  if (p0 >= p.N) return;
  const uint2* pr = s_pair + (p0 - lo);  // pr[i]: position p0 + i, -S - 1 <= i <= 2 S
  const int len = p.N - p0 < S ? (int)(p.N - p0) : S;
  const int c = blockIdx.y * p.lanes + lane;
  const bool in = c < p.units;
  // the keys around the span's ends
  const uint32_t first = pr[0].x, last = pr[len - 1].x, before = pr[-1].x, after = pr[len].x;
  // a run begun before the span: finished by its owner if that is the span
  // before and the run ends in this one; else this span's part of it
  const bool head = before == first && first < none;
  const bool head_part = head && (after == first || pr[-S - 1].x == first);
  // the run that goes on past the span, if it is this span's: finished here if
  // it ends in the next span, else in parts
  const bool tail = after == last && last < none && !(head && last == first);
  const bool tail_part = tail && pr[2 * S].x == last;
  const int end = tail && !tail_part ? 2 * S : len;
  int q = 0;
  if (head && !head_part)
    while (q < len && pr[q].x == first) ++q;
  bool in_head = head_part;
  const TG* g = static_cast<const TG*>(p.g) + (int64_t)c * VEC;
  float acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  uint32_t cur = q < len ? pr[q].x : none;
  for (; q < end && cur < none; q += U) {
    RawVec<TG, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint2 e = q + u < end ? pr[q + u] : make_uint2(none, 0);
      if (in && e.x < none) r[u].load(g + (int64_t)e.y * p.g_stride);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t key = q + u < end ? pr[q + u].x : none;
      if (key != cur) {  // the run of `cur` ends
        if (q + u >= end) break;
        if (in) {
          if (!in_head) grad_store<TO, VEC>(p, cur, c, acc);
          else store_vec(p.partial + span * 2 * p.D + (int64_t)c * VEC, acc);
        }
        in_head = false;
        // past the span only its own last run is taken; keys without a row come last
        cur = q + u < len ? key : none;
        if (cur >= none) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
      }
      if (in) {
        float f[VEC];
        r[u].unpack(f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += f[j];
      }
    }
  }
  // (a run in parts has one last span: where its head ends)
  if (head_part && after != first && c == 0) p.run_last[first] = (int)span;
  if (cur >= none) return;
  if (tail_part || in_head) {
    if (in) store_vec(p.partial + (span * 2 + (tail_part ? 1 : 0)) * p.D + (int64_t)c * VEC, acc);
    if (tail_part && c == 0) p.list[atomicAdd(p.listed, 1)] = make_int2((int)span, (int)cur);
  } else if (in) {
    grad_store<TO, VEC>(p, cur, c, acc);
  }
}

// Adds the parts of the listed runs: a block takes a run, `256 / lanes` strided
// groups of lanes add its spans' parts in fp64, eight loads in flight, then the
// groups' sums are added in a fixed order.  The list's order, the only thing that
// scheduling decides, does not enter the sums.  (Few parts a run, many runs: with
// 512 threads a block it takes 29 us instead of 23 on 1.5M tokens.)
constexpr int kJoinThreads = 256;
template <typename TO, int VEC>
__global__ void __launch_bounds__(kJoinThreads) grad_join_kernel(const __grid_constant__ SumParams p) {
  __shared__ double s_sum[kJoinThreads / 32][32][VEC];
  const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, groups = kJoinThreads / p.lanes;
  const int c = blockIdx.y * p.lanes + lane;
  pdl_wait();
  const int n = *p.listed;
  for (int item = blockIdx.x; item < n; item += gridDim.x) {
    const int64_t span = p.list[item].x;
    const uint32_t key = (uint32_t)p.list[item].y;
    const int64_t last = p.run_last[key];
    double sum[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum[j] = 0.0;
    if (c < p.units) {
      for (int64_t t0 = span + group; t0 <= last; t0 += 8 * groups) {
        RawVec<float, VEC> r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int64_t t = t0 + u * groups;
          if (t <= last) r[u].load(p.partial + (t * 2 + (t == span ? 1 : 0)) * p.D + (int64_t)c * VEC);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (t0 + u * groups > last) break;
          float f[VEC];
          r[u].unpack(f);
#pragma unroll
          for (int j = 0; j < VEC; ++j) sum[j] += (double)f[j];
        }
      }
    }
    // the groups of a warp, then the warps
    for (int off = p.lanes; off < 32; off <<= 1)
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
    if ((threadIdx.x & 31) < p.lanes)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s_sum[threadIdx.x >> 5][lane][j] = sum[j];
    __syncthreads();
    if (threadIdx.x < p.lanes && c < p.units) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        double t = 0.0;
#pragma unroll
        for (int q = 0; q < kJoinThreads / 32; ++q) t += s_sum[q][lane][j];
        f[j] = (float)t;
      }
      grad_store<TO, VEC>(p, key, c, f);
    }
    __syncthreads();
  }
}

// Few tokens: block i takes the run of tok[i] if no earlier position holds the
// token, lists its positions in order and adds their rows, `256 / lanes` rows
// at a time; the groups' sums are joined in group order in fp64.
template <typename TG, typename TO, int VEC>
__global__ void __launch_bounds__(256) grad_small_kernel(const __grid_constant__ SumParams p) {
  __shared__ int s_pos[kSmallN];
  __shared__ int s_warp[8];
  __shared__ double s_sum[256][VEC];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int i = blockIdx.x, N = (int)p.N;
  const int64_t t = p.tok[i];
  if (t == p.padding) return;
  if (t < 0 || t >= p.V) {
    if (tid == 0) atomicOr(p.status, kErrTagOverflow);
    return;
  }
  bool earlier = false;
  for (int j = tid; j < i; j += 256) earlier |= p.tok[j] == t;
  if (__syncthreads_or(earlier)) return;
  int n = 0;
  for (int j0 = i; j0 < N; j0 += 256) {
    const int j = j0 + tid;
    const bool hit = j < N && p.tok[j] == t;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (lane == 0) s_warp[w] = __popc(m);
    __syncthreads();
    int at = n, all = 0;
    for (int q = 0; q < 8; ++q) {
      if (q < w) at += s_warp[q];
      all += s_warp[q];
    }
    if (hit) s_pos[at + __popc(m & ((1u << lane) - 1u))] = j;
    n += all;
    __syncthreads();
  }
  const int gl = tid & (p.lanes - 1), group = tid / p.lanes, groups = 256 / p.lanes;
  for (int c0 = 0; c0 < p.units; c0 += p.lanes) {
    const int c = c0 + gl;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
    if (c < p.units) {
#pragma unroll 4
      for (int q = group; q < n; q += groups) {
        RawVec<TG, VEC> r;
        r.load(static_cast<const TG*>(p.g) + (int64_t)s_pos[q] * p.g_stride + (int64_t)c * VEC);
        float f[VEC];
        r.unpack(f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += f[j];
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) s_sum[tid][j] = (double)acc[j];
    __syncthreads();
    if (group == 0 && c < p.units) {
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        double s = 0.0;
        for (int q = 0; q < groups && q < n; ++q) s += s_sum[q * p.lanes + gl][j];
        f[j] = (float)s;
      }
      grad_store<TO, VEC>(p, t, c, f);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gradient: host
struct GradPlan {
  int items, tiles, passes, bits;  // the sort
  int span;
  int64_t pairs_bytes, hist_bytes, total_bytes, partial_bytes, list_bytes, last_bytes;
  int64_t bytes;
};

GradPlan grad_plan(int64_t N, int64_t V, int D) {
  GradPlan g = {};
  if (N <= kSmallN) return g;
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;  // keys 0 .. V
  // Fewest passes, of at most 10 bits: a pass costs three launches (65536 tokens of
  // 18 bits: 46 us in two passes, 52 in three of 6; 1.5M: 198 and 212; 1.5M of 19
  // bits: 237 and 243).  Only two full digits of 10 bits, whose bins cost a block as
  // much as its keys, fall behind three of 7 where there are many tokens (20 bits:
  // 800000 tokens 202 and 208, 1.5M 308 and 292).
  const int most = N >= 1000000 && bits == 20 ? 8 : kMaxDigit;
  g.passes = (bits + most - 1) / most;
  g.bits = (bits + g.passes - 1) / g.passes;
  if (g.bits < 5) g.bits = 5;  // the scan takes 32 bins at a time
  // 8 keys a thread once they make two tiles for every SM, 4 below (1M rows: 500000
  // tokens 171 us at 8 and 167 at 4, 650000 179 and 198, 1.5M 288 and 308)
  g.items = N >= (int64_t)kSMs * kSortThreads * 16 ? 8 : 4;
  const int64_t tile = (int64_t)kSortThreads * g.items;
  g.tiles = (int)((N + tile - 1) / tile);
  g.pairs_bytes = align256(N * 8);
  g.hist_bytes = align256(((int64_t)g.tiles << g.bits) * 4);
  g.total_bytes = align256(((int64_t)1 << g.bits) * 4 + 4);  // and the number of listed runs
  // long spans leave fewer parts, short ones make enough groups to fill the
  // machine, 8 columns a lane (30000 tokens over rows of 128: 33 us with spans of
  // 16, 51 of 64)
  g.span = kMaxSpan;
  while (g.span > 16 && N / g.span * ((D + 7) / 8) < (int64_t)kSMs * 2048) g.span /= 2;
  const int64_t spans = (N + g.span - 1) / g.span;
  g.partial_bytes = align256(spans * 2 * D * 4);
  g.list_bytes = align256(spans * 8);
  g.last_bytes = align256(V * 4);
  g.bytes = 2 * g.pairs_bytes + g.hist_bytes + g.total_bytes + g.partial_bytes + g.list_bytes + g.last_bytes;
  return g;
}

unsigned zero_blocks(const ZeroSlice& z) { return (unsigned)((z.bytes + kZeroBytes - 1) / kZeroBytes); }

template <int ITEMS>
cudaError_t sort_pass_launch(const PassParams& pp, cudaStream_t s) {
  const int bins = 1 << pp.bits;
  cudaError_t e;
  {
    LaunchScope ls("embed_grad_count", s);
    e = launch_pdl(grad_count_kernel<ITEMS>, (unsigned)pp.tiles + zero_blocks(pp.zero[0]), kSortThreads, 0, s, pp);
    if (e != cudaSuccess) return e;
  }
  {
    LaunchScope ls("embed_grad_scan", s);
    e = launch_pdl(grad_scan_kernel, (unsigned)((bins + 31) / 32) + zero_blocks(pp.zero[1]), 1024, 0, s, pp);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls("embed_grad_scatter", s);
  return launch_pdl(grad_scatter_kernel<ITEMS>, (unsigned)pp.tiles + zero_blocks(pp.zero[2]), kSortThreads,
                    (size_t)(kSortThreads / 32 + 1) * bins * 4, s, pp);
}

template <typename TG, typename TO, int VEC>
cudaError_t grad_launch(SumParams p, const int64_t* tok, char* ws, cudaStream_t s) {
  p.units = p.D / VEC;
  p.lanes = 1;
  while (p.lanes < p.units && p.lanes < 32) p.lanes *= 2;
  cudaError_t e;
  const int64_t dw_bytes = (int64_t)p.V * p.D * sizeof(TO);
  // the sort's kernels write the zeros where it runs and 16-byte stores fit
  const bool beside = p.N > kSmallN && dw_bytes % 16 == 0 && !misaligned(p.dw, 16);
  if (!p.accumulate && !beside) {
    if ((e = cudaMemsetAsync(p.dw, 0, (size_t)dw_bytes, s)) != cudaSuccess) return e;
  }
  if (p.N == 0) return cudaSuccess;
  if (p.N <= kSmallN) {
    LaunchScope ls("embed_grad_small", s);
    grad_small_kernel<TG, TO, VEC><<<(unsigned)p.N, 256, 0, s>>>(p);
    return cudaGetLastError();
  }
  const GradPlan g = grad_plan(p.N, p.V, p.D);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(ws), reinterpret_cast<uint2*>(ws + g.pairs_bytes)};
  char* at = ws + 2 * g.pairs_bytes;
  PassParams pp = {};
  pp.tok = tok;
  pp.N = p.N;
  pp.V = p.V;
  pp.padding = p.padding;
  pp.bits = g.bits;
  pp.tiles = g.tiles;
  pp.hist = reinterpret_cast<uint32_t*>(at);
  at += g.hist_bytes;
  pp.total = reinterpret_cast<uint32_t*>(at);
  pp.listed = reinterpret_cast<int*>(pp.total + ((int64_t)1 << g.bits));
  at += g.total_bytes;
  pp.status = p.status;
  // the zeros in equal slices, one a kernel of the sort
  const int slices = 3 * g.passes;
  const int64_t slice = (dw_bytes / slices + 16) / 16 * 16;
  int64_t done = 0;
  for (int i = 0; i < g.passes; ++i) {
    pp.shift = i * g.bits;
    pp.in = i == 0 ? nullptr : pairs[(i + 1) & 1];
    pp.out = pairs[i & 1];
    for (ZeroSlice& z : pp.zero) {
      z.at = static_cast<char*>(p.dw) + done;
      z.bytes = beside && !p.accumulate ? std::min(slice, dw_bytes - done) : 0;
      done += z.bytes;
    }
    e = g.items == 8 ? sort_pass_launch<8>(pp, s) : sort_pass_launch<4>(pp, s);
    if (e != cudaSuccess) return e;
  }
  p.pairs = pairs[(g.passes - 1) & 1];
  p.partial = reinterpret_cast<float*>(at);
  p.list = reinterpret_cast<int2*>(at + g.partial_bytes);
  p.run_last = reinterpret_cast<int*>(at + g.partial_bytes + g.list_bytes);
  p.listed = pp.listed;
  p.span = g.span;
  const int64_t spans = (p.N + p.span - 1) / p.span;
  p.spb = std::min(256 / p.lanes, kMaxSpans);
  const int cols = (p.units + p.lanes - 1) / p.lanes;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cfg.stream = s;
  {
    LaunchScope ls("embed_grad_span", s);
    cfg.gridDim = dim3((unsigned)((spans + p.spb - 1) / p.spb), (unsigned)cols);
    cfg.blockDim = dim3((unsigned)(p.spb * p.lanes));
    if ((e = cudaLaunchKernelEx(&cfg, grad_span_kernel<TG, TO, VEC>, p)) != cudaSuccess) return e;
  }
  if (spans > 2) {  // a run in parts covers a whole span between two others
    LaunchScope ls("embed_grad_join", s);
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(spans / 2, kSMs * 8), (unsigned)cols);
    cfg.blockDim = dim3(kJoinThreads);
    if ((e = cudaLaunchKernelEx(&cfg, grad_join_kernel<TO, VEC>, p)) != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

// Clears the bits of the status word that a caller has read, no others: another
// stream's kernel may have set one since.
__global__ void status_clear_kernel(int* status, int bits) { atomicAnd(status, ~bits); }

}  // namespace

int* sequence_status() {
  static int* at[128] = {nullptr};  // per device; every writer stores the same address
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return nullptr;
  int* p = __atomic_load_n(&at[dev], __ATOMIC_ACQUIRE);
  if (!p) {
    void* q = nullptr;
    if (cudaGetSymbolAddress(&q, g_seq_status) != cudaSuccess) return nullptr;
    p = static_cast<int*>(q);
    __atomic_store_n(&at[dev], p, __ATOMIC_RELEASE);
  }
  return p;
}

static recis_status status_missing() {
  set_error("the sequence operators' status word is not reachable (no usable sm_100 device?)");
  return RECIS_ERR_NO_DEVICE;
}

}  // namespace recis

using namespace recis;

extern "C" recis_status recis_sequence_status_sync(recis_stream_t stream) {
  int* st = sequence_status();
  if (!st) return status_missing();
  cudaStream_t s = (cudaStream_t)stream;
  int h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, st, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (!h) return RECIS_OK;
  status_clear_kernel<<<1, 1, 0, s>>>(st, h);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail(e, "status clear");
  if ((e = cudaStreamSynchronize(s)) != cudaSuccess) return cuda_fail(e, "status clear");
  if (h & kErrTimeout) {
    set_error("a bounded device-side wait gave up");
    return RECIS_ERR_TIMEOUT;
  }
  set_error(h & kErrBadOffsets ? "bag offsets decrease, leave their array or pass the given bound"
                               : "a token is neither padding nor a row of the weight");
  return RECIS_ERR_INVALID_ARG;
}

extern "C" recis_status recis_embed_lookup(const void* weight, int32_t weight_type, int64_t V, int32_t D,
                                           const int64_t* tokens, int64_t N, double scale, int64_t padding, void* out,
                                           int32_t out_type, int64_t out_stride, recis_stream_t stream) {
  if (!float_type(weight_type) || !float_type(out_type) || V < 1 || V > INT32_MAX || D < 1 || D > 65536 || N < 0 ||
      N > INT32_MAX || !weight || out_stride < D || (N > 0 && (!tokens || !out))) {
    set_error("embed_lookup: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  if (misaligned(weight, type_bytes(weight_type)) || misaligned(out, type_bytes(out_type)) || misaligned(tokens, 8)) {
    set_error("embed_lookup: misaligned array");
    return RECIS_ERR_INVALID_ARG;
  }
  if (N == 0) return RECIS_OK;
  int* st = sequence_status();
  if (!st) return status_missing();
  LookupParams p = {weight, tokens, out, V, N, out_stride, padding, D, 0, 0, (float)scale, st};
  // 16-byte accesses where every row of both arrays allows them
  const bool vec = D % 8 == 0 && rows_aligned16(weight, D, weight_type) && rows_aligned16(out, out_stride, out_type);
  const cudaError_t e = with_type(weight_type, [&](auto w) {
    return with_type(out_type, [&](auto o) {
      using TW = decltype(w);
      using TO = decltype(o);
      return vec ? lookup_launch<TW, TO, 8>(p, (cudaStream_t)stream) : lookup_launch<TW, TO, 1>(p, (cudaStream_t)stream);
    });
  });
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "embed_lookup launch");
}

static bool grad_sizes_ok(int64_t N, int64_t V, int32_t D) {
  return V >= 1 && V < INT32_MAX && D >= 1 && D <= 65536 && N >= 0 && N < ((int64_t)1 << 30);
}

extern "C" recis_status recis_embed_grad_workspace(int64_t N, int64_t V, int32_t D, int64_t* bytes_out) {
  if (!bytes_out || !grad_sizes_ok(N, V, D)) {
    set_error("embed_grad_workspace: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  *bytes_out = grad_plan(N, V, D).bytes;
  return RECIS_OK;
}

extern "C" recis_status recis_embed_grad(const int64_t* tokens, int64_t N, const void* grad_out, int32_t grad_type,
                                         int64_t grad_stride, int64_t V, int32_t D, double scale, int64_t padding,
                                         int32_t accumulate, void* grad_weight, int32_t weight_type, void* workspace,
                                         int64_t workspace_bytes, recis_stream_t stream) {
  if (!float_type(grad_type) || !float_type(weight_type) || !grad_sizes_ok(N, V, D) || !grad_weight ||
      grad_stride < D || (accumulate != 0 && accumulate != 1) || (N > 0 && (!tokens || !grad_out))) {
    set_error("embed_grad: bad arguments");
    return RECIS_ERR_INVALID_ARG;
  }
  if (misaligned(grad_out, type_bytes(grad_type)) || misaligned(grad_weight, type_bytes(weight_type)) ||
      misaligned(tokens, 8) || misaligned(workspace, 256)) {
    set_error("embed_grad: misaligned array");
    return RECIS_ERR_INVALID_ARG;
  }
  const int64_t need = grad_plan(N, V, D).bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) {
    set_error("embed_grad: workspace too small");
    return RECIS_ERR_INVALID_ARG;
  }
  int* st = sequence_status();
  if (!st) return status_missing();
  SumParams p = {};
  p.tok = tokens;
  p.g = grad_out;
  p.dw = grad_weight;
  p.N = N;
  p.V = V;
  p.g_stride = grad_stride;
  p.padding = padding;
  p.D = D;
  p.accumulate = accumulate;
  p.scale = (float)scale;
  p.status = st;
  const bool vec =
      D % 8 == 0 && rows_aligned16(grad_out, grad_stride, grad_type) && rows_aligned16(grad_weight, D, weight_type);
  char* ws = static_cast<char*>(workspace);
  const cudaError_t e = with_type(grad_type, [&](auto g) {
    return with_type(weight_type, [&](auto o) {
      using TG = decltype(g);
      using TO = decltype(o);
      return vec ? grad_launch<TG, TO, 8>(p, tokens, ws, (cudaStream_t)stream)
                 : grad_launch<TG, TO, 1>(p, tokens, ws, (cudaStream_t)stream);
    });
  });
  return e == cudaSuccess ? RECIS_OK : cuda_fail(e, "embed_grad launch");
}
