// Host-side interface of the LM-head loss kernels (see head.cu).
#pragma once
#include "kernels.cuh"

namespace smdm {

struct HeadArgs {
  int rows, d, vocab;
  bool f32;                  // hidden, lm_head and their gradients: fp32 (else bf16)
  long long ld_hidden, ld_head;   // row strides in elements
  const void* hidden;
  const void* head;
  const int* target;         // [rows], negative = the row takes no part
  float* nll;                // loss: [rows]
  float* lse_out;            // loss: [rows]
  const float* lse;          // gradient: [rows]
  const float* grad_nll;     // gradient: [rows]
  void* grad_hidden;         // gradient: [rows][d] or null
  void* grad_head;           // gradient: [vocab][d] or null
  // Logits from fp16 operands: the loss's hidden and head are fp16; the gradient makes its logits
  // from these two (contiguous, on 16 bytes, d a multiple of 8), its products from hidden and head.
  bool half;
  const void* hidden16;
  const void* head16;
  void* ws;
  uint32_t* status;          // optional
};

// Bytes of workspace for one call (grad: the gradient's, else the loss's; half as in HeadArgs).
size_t head_workspace_bytes(int rows, int d, int vocab, bool f32, bool grad, bool half = false);
// True when lm_head must start on a 16-byte boundary (its rows are then read by TMA in place).
bool head_needs_aligned_weight(int d, long long ld_head, bool f32);
// Kernels that a call launches.
int head_loss_launches(const HeadArgs& a);
int head_grad_launches(const HeadArgs& a);
cudaError_t launch_head_loss(const HeadArgs& a, cudaStream_t st);
cudaError_t launch_head_grad(const HeadArgs& a, cudaStream_t st);

// The same for a handful of rows (head_few.cu); `sms`: SMs of the device.
constexpr int kFewRows = 16;
constexpr int kFewSmem = 200 * 1024;     // the hidden rows of a launch in fp32
bool head_few_fits(int rows, int d);
int head_few_groups(int rows, int d);    // launches that make the logits
size_t head_few_bytes(int rows, int d, int vocab, int sms);
cudaError_t launch_head_few_loss(const HeadArgs& a, int sms, cudaStream_t st);
cudaError_t launch_head_few_grad(const HeadArgs& a, int sms, cudaStream_t st);

}  // namespace smdm
