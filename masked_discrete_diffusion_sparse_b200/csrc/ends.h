// Host-side interface of the training-form RMSNorm and embedding kernels (see ends.cu).
#pragma once
#include "kernels.cuh"

namespace smdm {

struct RmsArgs {
  int rows, d;
  bool x_f32, f32;             // type of x, grad_x, add; type of gain, y, grad_y, grad_gain
  long long ld_x, ld_y;        // row strides in elements of x and of y (grad_y)
  float eps;
  const void* x;
  const void* gain;
  void* y;
  float* rstd_out;             // optional
  // gradient
  const float* rstd;
  const void* grad_y;
  const void* add;             // optional [rows][d]
  void* grad_x;                // [rows][d]
  void* grad_gain;             // [d]
  float* ws;
};

struct EmbedArgs {
  int rows, d, n_emb;
  bool f32, out_f32;           // type of the table (and its gradient); type of the rows
  long long ld_table;          // forward
  long long ld_grad;           // gradient: row stride of grad_out
  float scale;
  const int* ids;
  const void* table;
  void* out;
  const void* grad_out;
  void* grad_table;
  void* ws;
  uint32_t* status;            // optional
};

constexpr int kMaxNormWidth = 8192;   // a row is held in the registers of 256 threads

cudaError_t launch_train_rmsnorm(const RmsArgs& a, cudaStream_t st);
size_t rmsnorm_grad_bytes(int rows, int d);
int rmsnorm_grad_launches(int rows, int d);   // kernels that the gradient launches
cudaError_t launch_train_rmsnorm_grad(const RmsArgs& a, cudaStream_t st);
cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t st);
size_t embed_grad_bytes(int rows, int d, int n_emb);
cudaError_t launch_embed_grad(const EmbedArgs& a, cudaStream_t st);
// (id << 32 | row) of n rows in order, ids outside [0, n_ids) as n_ids; in a or b, n words each (b
// is used above kSortChunk rows).  Bytes at `clear` are set to 0 meanwhile.
constexpr int kSortChunk = 2048;
int sort_ids_launches(int n);
cudaError_t launch_sort_ids(const int* ids, int n, int n_ids, unsigned long long* a,
                            unsigned long long* b, void* clear, size_t clear_bytes,
                            uint32_t* status, cudaStream_t st, const unsigned long long** sorted);
// out[i] = x[index[i]], rows of d fp32 (index out of [0, n): row 0 and kStatusBounds).
cudaError_t launch_gather_f32(const float* x, const int* index, int rows, int n, int d, float* out,
                              uint32_t* status, cudaStream_t st);

}  // namespace smdm
