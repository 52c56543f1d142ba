// The weight gradient from 8-bit checkpoints: what its entry (flce_ckpt8.cu) and its
// tensor-core kernel (flce_ckpt8_tc.cu) share.
#pragma once

#include "flce_ops.cuh"

namespace flce {

struct DwArgs {
  int64_t M, N, K, nblk;   // nblk: scales per row
  const void* dy;
  int64_t lddy;
  const uint8_t* q;
  int64_t ldq;
  const float* scale;
  void* dW;
  int64_t lddW;
  int ovw;
};

// Workspace bytes of the tensor-core path, and its launch, which zeroes the status word first.
// `dt`: dtype of dy; `wdt`: of dW.
size_t dw_tc_workspace(const DwArgs& a, int dt);
bool dw_tc_supported();
cudaError_t launch_dw_tc8(const DwArgs& a, int dt, int wdt, void* workspace, int* status, uint64_t timeout_ns,
                          bool stall, cudaStream_t s);

}  // namespace flce
