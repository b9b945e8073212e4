// Launch arguments of the operators on rows of logits (sample.cu, distill.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dflash.h"

namespace df {

struct SampleLeft {               // a row that one pass did not decide
  uint64_t about;                 // about its mass, 0: not known
  uint32_t largest, on;           // key of its largest logit; 0: decided
};
struct SampleArgs {
  df_rows x;
  int group, row0;                // row r's setting: (row0 + r) / group
  const float *temperature, *top_p, *min_p;   // [rows / group], each may be null
  const int32_t* top_k;
  const float* u;                 // [rows], or null:
  const uint32_t* draw_key;       // [rows] keys of the draws (without logprob and n_kept; see as_unset in sample.cu)
  int32_t* token;                 // [rows]
  float* logprob;                 // [rows], may be null
  int32_t* n_kept;                // [rows], may be null
  SampleLeft* left;               // [rows]
  int* status;
};
int launch_sample(const SampleArgs& a, cudaStream_t st);

struct TopArgs {
  df_rows x;
  int K;
  float temperature;
  int32_t* id;                    // [rows][K]
  float *val, *lse;               // [rows][K]; [rows], may be null
  int* status;
};
int launch_top_logits(const TopArgs& a, cudaStream_t st);

struct DistillArgs {
  df_rows x;                      // the student's logits
  int K, n_teacher;
  const int32_t* id;              // [n_teacher][K]
  const float *val, *lse;         // [n_teacher][K]; [n_teacher] or null
  const int32_t* teacher_row;     // [rows] or null
  float temperature;
  const float *weight, *grad_loss;  // [rows] or null
  float *loss, *stats;            // [rows]; [rows][4]
  void* grad;                     // [rows][ld_grad] in the type of x, may be null (backward: not)
  long long ld_grad;
  int* status;
};
int launch_distill(const DistillArgs& a, cudaStream_t st);
int launch_distill_backward(const DistillArgs& a, cudaStream_t st);

// dflash_path_rows
int launch_path_rows(int b, int D, int n_tree, const int32_t* n_new, const int32_t* src_slot, int max_src,
                     const int32_t* cache_len, int32_t* teacher_row, cudaStream_t st);

// CTAs that share a row of V logits (one cluster): a power of two up to 8 with which all rows have at
// most `most` of them, and at least 2048 elements each.  One wave of CTAs that share rows beats a
// second wave by far (draws of 40 rows of 151936: 4 CTAs each 16 us, 8 of them 27; of 80 rows: 2 CTAs
// 21 us, 8 of them 41), and more CTAs on a row beat idle SMs (of 20 rows: 1 CTA 18 us, 8 of them 14).
int row_ctas(int rows, int V, int most);

}  // namespace df
