/* What tensors.cpp tells binding.c of a tensor. */
#ifndef TLQ_TENSORS_H_
#define TLQ_TENSORS_H_

enum { TLQ_TENSOR_F16 = 1, TLQ_TENSOR_F32, TLQ_TENSOR_I32, TLQ_TENSOR_I64, TLQ_TENSOR_U8 };

typedef struct {
  void* data;
  long long numel, size[4], step[4];
  int type, dims, contiguous;
} tlq_tensor;

#endif
