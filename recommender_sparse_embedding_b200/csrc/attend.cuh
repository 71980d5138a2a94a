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
  int max_q, max_k;
  float scale, scale_log2;  // scale, scale * log2(e)
  int splits, split_keys;   // parts of a bag's keys, keys a part
  float* po;                // splits > 1: [splits][Tq][Hq][D] each part's output ...
  float* pl;                // ... and [splits][Tq][Hq] its lse
  float* delta;             // backward, many rows: [Tq][Hq] -sum(grad_out * out) ...
  float* nlse;              // ... and [Tq][Hq] -lse * log2(e)
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
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.Tq && q1 - q0 <= p.max_q && k0 >= 0 && k1 >= k0 && k1 <= p.Tk &&
                  k1 - k0 <= p.max_k;
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
recis_status launch_attend_back_few(const AttendParams& p, bool bf16, cudaStream_t s);
recis_status launch_attend_tc(const AttendParams& p, bool bf16, cudaStream_t s);
recis_status launch_attend_back(const AttendParams& p, bool bf16, cudaStream_t s);

}  // namespace recis
