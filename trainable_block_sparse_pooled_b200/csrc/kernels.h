// Internal launcher declarations of libspa2 (not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spa2.h"

namespace spa2 {

// timing.cu: per-kernel event timing (spa2_timing_*). One id per kernel kind.
enum KernelId : int {
  KID_POOL = 0,
  KID_SELECT,
  KID_LOGITS,
  KID_CSC,
  KID_PBAR_SELECT,
  KID_V16,
  KID_FWD,
  KID_BWD_PRE,
  KID_BWD_DKDV,
  KID_BWD_DQ,
  KID_PROBE,
  KID_TILES,
  KID_ROTARY,
  KID_PACK8,
  KID_UNPACK8,
  KID_BWD_DQ_CKPT,
  KID_COUNT
};

// Brackets one kernel launch with two CUDA events recorded on `s` while timing
// is on (construct it just before the launch, in the launch's scope).
class KernelTimer {
 public:
  KernelTimer(int kid, cudaStream_t s);
  ~KernelTimer();
  KernelTimer(const KernelTimer&) = delete;
  KernelTimer& operator=(const KernelTimer&) = delete;

 private:
  int slot_;
  cudaStream_t s_;
};

struct MaskOut {
  int* row_cnt;
  int* row_idx;
  float* pbar;       // may be null
  uint8_t* bitmap;   // may be null
};

// mask.cu
// qbar, kbc: Qbar and Kbar workspaces in chunks of 64 blocks,
// [BH, kbar_chunks(Tm), d, 64] and [BH, kbar_chunks(Tn), d, 64] fp32;
// lg: logit workspace [BH, Tm, Tn] fp32
int kbar_chunks(int Tn);
cudaError_t launch_mask(const void* q, const void* k, float* qbar, float* kbc, float* lg, int BH, int N, int d,
                        int Tm, int Tn, int bq, int bkv, int K, unsigned long long thr, const MaskOut& out,
                        int* col_cnt, int* col_idx, uint32_t* bits, int W, int* status,
                        unsigned long long wait_limit_ns, cudaStream_t s);
cudaError_t launch_select(const float* pbar, int BH, int Tm, int Tn, int K, unsigned long long thr,
                          const MaskOut& out, uint32_t* bits, int W, int* status, cudaStream_t s);
cudaError_t launch_csc(const uint32_t* bits, int BH, int Tm, int Tn, int W, int* col_cnt, int* col_idx,
                       cudaStream_t s);

// attn_fwd.cu
struct FwdArgs {
  const CUtensorMap* tm_q;   // box {64, 128, 1}
  const CUtensorMap* tm_k;   // box {64, 64, 1}
  const CUtensorMap* tm_v;   // box {64, 64, 1}, fp16 copy of V
  const CUtensorMap* tm_o;   // box {64, 128, 1}
  const CUtensorMap* tm_olo; // box {64, 128, 1}; O residual, used when has_olo
  int has_olo;
  const int* row_cnt;
  const int* row_idx;
  float* lse;         // may be null
  int BH, N, Tm, Tn;
  float scale_log2;   // softmax_scale * log2(e)
  int* status;
  unsigned long long wait_limit_ns;
  int tiled;          // list entries may carry tile exclusion bits
};
cudaError_t launch_fwd(const FwdArgs& a, int d, cudaStream_t s);
cudaError_t launch_v_to_f16(const void* v, void* v16, long long elems, int* status, cudaStream_t s);

// attn_bwd.cu
// The backward on 8-bit checkpoints: the `ranks` longest columns of every head are taken by the dK/dV
// pass in up to `parts` parts, whose sums meet in `partial` [ranks * heads, parts, 2, 16, d, 4]
struct ColumnSplit {
  int ranks, parts, heads;
  float* partial;
  int* done;  // [ranks * heads, 4]: parts that are there, by quarter of 32 features; zero before the pass
};
struct BwdArgs {
  const CUtensorMap* tm_q;    // Q bf16, box {64, 128, 1}
  const CUtensorMap* tm_k;    // K bf16, box {64, 64, 1}
  const CUtensorMap* tm_v;    // V bf16, box {64, 64, 1}
  const CUtensorMap* tm_do;   // fp16 copy of dO, box {64, 128, 1}
  const CUtensorMap* tm_q16;  // fp16 copy of Q, box {64, 128, 1}
  const CUtensorMap* tm_dq;   // dQ output: fp32 box {32, 128, 1} or bf16 box {64, 128, 1}, 128-byte swizzle
  const void* q;      // null with q8
  const void* k;
  const void* o;      // null with q8
  const void* o_lo;   // may be null
  const void* dout;
  const void* v;
  float* lse;         // given, or (q8) written by the dQ pass
  const int* row_cnt;
  const int* row_idx;
  const int* col_cnt;
  const int* col_idx;
  float* dvec;     // [BH, N]
  void* do16;      // [BH, N, d] fp16
  void* q16;       // [BH, N, d] fp16
  void* dq;
  void* dk;
  void* dv;
  int grad_f32;       // 1: dq/dk/dv are fp32, 0: bf16
  int BH, N, Tm, Tn;
  float scale;        // softmax_scale
  float scale_log2;   // softmax_scale * log2(e)
  int* status;
  int* ticket;        // zero at launch: the persistent dK/dV kernel's column counter
  unsigned long long wait_limit_ns;
  int tiled;          // list entries may carry tile exclusion bits
  int* col_order;     // [BH * Tn]: the dK/dV pass's columns, head by head, long columns first (pre-pass)
  // on 8-bit checkpoints (otherwise null): Q's codes and exponents; tm_k and tm_v are fp16, col_order
  // and do_most are there, and the dQ pass writes lse, dvec, do16, q16 and unscale
  const int8_t* q8;
  const uint8_t *qe, *ke, *ve;
  const uint32_t* do_most;    // [BH, DO_PARTS]
  float* unscale;             // [BH]: do16 and dvec are dO and D divided by this power of two
  ColumnSplit split;
};
cudaError_t launch_bwd(const BwdArgs& a, int d, cudaStream_t s);

// attn_bwd_ckpt.cu: the dQ pass on 8-bit checkpoints, which also finds LSE and D
cudaError_t launch_dq_ckpt(const BwdArgs& a, int d, cudaStream_t s);

// pack8.cu. The checkpoints of a step's q, k, v [rows, d] bf16 (d = 64 or 128, 16-byte aligned),
// with an fp16 copy of v; |v| > 65504 is clamped and reported to status
cudaError_t launch_pack8_step(const spa2_pack8_tensor (&t)[3], void* v16, int* status, cudaStream_t s);
// and what the backward starts from: k, v as fp16, the dK/dV pass's columns in order, the largest |dO|
constexpr int DO_PARTS = 32;  // parts of a head whose largest |dO| are found apart
struct Unpack8Step {
  spa2_pack8_tensor k, v;
  uint32_t *k16, *v16;
  const void* dout;   // bf16, 16-byte aligned
  uint32_t* do_most;  // [heads, DO_PARTS]: the largest |dO|'s bf16 bits, and in the low half V's largest exponent
  const int* col_cnt;
  int* col_order;
  int N, d, Tn;
  ColumnSplit split;
  long long heads, per_head;  // N * d elements to a head
};
cudaError_t launch_unpack8_step(const Unpack8Step& a, cudaStream_t s);

// api.cu
cudaError_t launch_timeout_probe(int* status, unsigned long long limit_ns, cudaStream_t s);

// tiles.cu: block CSR (and CSC when csc_cnt is not NULL) -> tile lists of 128-row query tiles x 64-row key
// tiles (TMt = ceil(N / 128), TNt = ceil(N / 64)); see the tile-list notes in common.cuh
cudaError_t launch_tile_lists(const int* row_cnt, const int* row_idx, const int* col_cnt, const int* col_idx, int BH,
                              int Tm, int Tn, int TMt, int TNt, int bq, int bkv, int* csr_cnt, int* csr_idx,
                              int* csc_cnt, int* csc_idx, int* status, cudaStream_t s);

}  // namespace spa2
