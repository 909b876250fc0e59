// fa_host.h - host helpers that the library's two translation units share: fa_api.cu, which
// defines them with the entry points for plain scores, and fa_api_score.cu, which holds the
// entry points for changed scores and the 4-bit cache.  (Two units build side by side, and
// what one instantiates leaves the other's code as it is.)
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_bwd.cuh"

namespace fa_host {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool debug_enabled();
bool cuda_ok(cudaError_t e, const char *what);
EncodeTiled encode_fn();
// The current device is an sm_100 and the kernels of fa_api.cu are set up on it.
bool device_ready();
bool make_map_bf16(CUtensorMap *m, const void *ptr, int d, int N, long long heads, int box_rows);
bool aligned16(const void *p);
int timer_start(int which, cudaStream_t s);
void timer_stop(int which, int slot, cudaStream_t s);
int check_sizes(int B, int Hq, int Hkv, int N, int d, float scale);
int check_decode_sizes(int B, int Hq, int Hkv, int Nq, int Nk, int d, float scale);
size_t decode_workspace(int B, int Hq, int Nq, int d, int splits);
int decode_rows_padded(int R);
void launch_merge(const float *o_part, const float *lse_part, void *o, float *lse, int S, long long rows, int d,
                  cudaStream_t s);
fa::BwdOrder bwd_order(int B, int Hkv, int N, int left, int right);
constexpr int kMaxDecodeSplits = 1024;
constexpr int kMaxDevices = 64;

// Defined in fa_api_score.cu: the status word of its kernels on the current device, cleared
// when it is not FA_OK (FA_OK without a look at the device before the first of them).
int take_score_status();

// A kernel that rebalances registers with setmaxnreg must have been compiled for the launch
// register count its split assumes (see fa_api.cu).
template <typename K>
bool regs_at_least(K kernel, int regs) {
  cudaFuncAttributes attr;
  return cuda_ok(cudaFuncGetAttributes(&attr, kernel), "cudaFuncGetAttributes") && attr.numRegs >= regs;
}

template <typename K>
bool set_smem(K kernel, int bytes) {
  return cuda_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                 "cudaFuncSetAttribute(max dynamic shared memory)");
}

}  // namespace fa_host
