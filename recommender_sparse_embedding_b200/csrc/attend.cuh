// attend.cuh -- shared by the attention kernels (attend.cu, attend_back.cu).
#pragma once
#include "seqops.cuh"

namespace recis {

// What every attention kernel is given: recis_attend_args with the group size
// and the plan of the call.
struct AttendParams {
  const void *q, *k, *v, *go;
  void *out, *gq, *gk, *gv;
  float* lse;
  const int64_t *qo, *ko;
  const uint8_t* mask;
  int64_t qs, qh, ks, kh, vs, vh, os, oh, gos, goh, gqs, gqh, gks, gkh, gvs, gvh;  // strides: row, head
  int64_t Tq, Tk;
  int B, Hq, Hkv, G, D;
  int max_q, max_k;         // at least 1 (launch_sizes in attend.cu)
  int bound_q, bound_k;     // what no bag may pass: the caller's max_q and max_k
  float scale, scale_log2;  // scale, scale * log2(e)
  int splits, split_keys;   // parts of a bag's keys, keys a part
  float* po;                // splits > 1: [splits][Tq][Hq][D] each part's output ...
  float* pl;                // ... and [splits][Tq][Hq] its lse
  float* delta;             // backward, many rows: [Tq][Hq] -sum(grad_out * out) ...
  float* nlse;              // ... and [Tq][Hq] -lse * log2(e) (plus kShiftP)
  float* gnorm;             // fp16 too: [Tq][Hq] |grad_out| ...
  float* vnorm;             // ... and value_slots() maxima of |v|, one a warp of a key tile
  int* status;
};

struct Bag {
  int64_t q0, k0;
  int nq, nk;
};

// Bag b's rows; a bag whose offsets are malformed or that passes its bound is
// reported and has none, so no access leaves the arrays.
__device__ __forceinline__ Bag load_bag(const AttendParams& p, int b) {
  const int64_t q0 = __ldg(p.qo + b), q1 = __ldg(p.qo + b + 1), k0 = __ldg(p.ko + b), k1 = __ldg(p.ko + b + 1);
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.Tq && q1 - q0 <= p.bound_q && k0 >= 0 && k1 >= k0 && k1 <= p.Tk &&
                  k1 - k0 <= p.bound_k;
  if (!ok) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrBadOffsets);
    return Bag{0, 0, 0, 0};
  }
  return Bag{q0, k0, (int)(q1 - q0), (int)(k1 - k0)};
}

// More rows (queries times heads of a group) than this in a bag: tiles of 128 rows
// in the forward (64 bags of 1000-5000 keys, 2 heads of 128: at 16 rows 62 us
// without them, 65 with; at 32 rows 73 and 64; 256 bags of up to 16 rows of 64: 83
// and 112).
constexpr int kFewRows = 16;
inline bool few_rows(int64_t max_q, int64_t G) { return max_q * G <= kFewRows; }
// At most this many keys in a bag (its own, whatever max_k is): the backward takes
// ds as two 16-bit values.
// (The gradients of q and k are then within 1.4 times their own rounding of 64
// bits, at 8 keys as at 128; with one value they are at 1.7 times at 8 keys and
// at 1.45 from 128 on.)
constexpr int kSplitKeys = 128;
// At most this many rows in a bag: the backward takes them all at once, in one
// pass over the keys (64 bags of 1000-5000 keys, 64 rows, 2 heads of 128: 140 us,
// 213 in two passes; 256 bags of up to 16 rows, 2 heads of 64: 161 and 609).
constexpr int kFewBackRows = 64;
inline bool few_back_rows(int64_t max_q, int64_t G) { return max_q * G <= kFewBackRows; }
// blocks of that pass an SM holds
inline int few_back_per_sm(int D, int64_t rows) { return D <= 64 && rows <= 32 ? 2 : 1; }

// fp16 has no normal numbers below 2^-14, and p and ds of a long bag lie there
// (5000 keys: p about 2^-12, times a gradient of 10^-3).  Its backward therefore
// rounds p 2^kShiftP and ds 2^e, e from a bound on |ds| so that ds 2^e stays below
// 2^14 (or the block's largest so far is followed, attend_back_few.cu); the
// accumulators take the powers of two out again.  bf16 has fp32's range: 0.
template <typename T>
constexpr int kShiftP = 0;
template <>
constexpr int kShiftP<__half> = 14;
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// 2^e * scale, finite (a zero accumulator stays zero)
__device__ __forceinline__ float pow2_times(int e, float scale) {
  return fminf(fmaxf(pow2(e) * scale, -3e38f), 3e38f);
}
// e with 2^13 <= bound * 2^e < 2^14; 0 where bound is 0 or not finite
__device__ __forceinline__ int half_exponent(float bound) {
  if (!(bound > 0.f && bound < INFINITY)) return 0;
  return min(13 + 127 - (int)(__float_as_uint(bound) >> 23), 100);
}
__device__ __forceinline__ float finite_max(float a, float b) { return b < INFINITY ? fmaxf(a, b) : a; }  // b >= 0
__device__ __forceinline__ float warp_max(float v) {  // of values >= 0
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}
// The maxima of |v| of a bag's key tiles (of 128, 4 warps each), bags and tiles in
// order of their keys: tile i of bag b begins at value_slot(k0, b) + 4 i.
__host__ __device__ inline int64_t value_slots(int64_t B, int64_t Tk) { return (Tk / 128 + B + 1) * 4; }
__device__ __forceinline__ int64_t value_slot(int64_t k0, int b) { return (k0 / 128 + b) * 4; }

recis_status launch_attend_back_few(const AttendParams& p, bool bf16, cudaStream_t s);
recis_status launch_attend_tc(const AttendParams& p, bool bf16, cudaStream_t s);
recis_status launch_attend_back(const AttendParams& p, bool bf16, cudaStream_t s);

}  // namespace recis
