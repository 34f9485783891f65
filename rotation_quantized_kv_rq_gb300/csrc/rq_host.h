// What the host sides of the library's calls share: the device scope of a call, argument checks, and the
// handles that several of them take.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rq.h"
#include "rq_internal.h"

namespace rq {

// Makes `dev` current for the scope and restores the previous device afterwards.
class DeviceScope {
 public:
  explicit DeviceScope(int dev) {
    ok_ = cudaGetDevice(&prev_) == cudaSuccess;
    if (ok_ && dev >= 0 && dev != prev_) {
      ok_ = cudaSetDevice(dev) == cudaSuccess;
      switched_ = ok_;
    }
  }
  ~DeviceScope() {
    if (switched_) cudaSetDevice(prev_);
  }
  bool ok() const { return ok_; }

 private:
  int prev_ = 0;
  bool ok_ = false, switched_ = false;
};

inline bool misaligned16(const void* p) { return (uintptr_t)p % 16 != 0; }
inline int to_status(cudaError_t e) { return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA; }

}  // namespace rq

struct rq_rope {
  rq::RopeTable table;
  uint64_t* d_pairs;
  int device;
  int num_sms;
};
