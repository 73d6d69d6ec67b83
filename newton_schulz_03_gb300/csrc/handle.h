// handle.h -- what the host files beside muon_api.cpp see of a handle.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

#include "moe.h"

struct muon_handle_s;

namespace muon {

struct HandleInfo {
  int num_sms;
  Fp8Pairs fp8_pairs;
  int* dev_err;   // device error word (kDevErr* bits)
};

// Status of the handle (MUON_OK, or MUON_ERR_INVALID_ARG with its message);
// makes the handle's device current.
int handle_info(muon_handle_s* h, HandleInfo* out);

// Device scratch of at least `bytes`, apart from the step's workspace.  Its
// address outlives the call: a buffer that has become too small is kept until
// the handle goes, since a captured graph may still write to it.
int handle_scratch(muon_handle_s* h, size_t bytes, void** out);

// What muon_selftest_loss_wait asked of this call, which takes it off.
int take_loss_stall(muon_handle_s* h);

// Counts one kernel launch of class `kind` and, with timing on, brackets it
// with events.
class LaunchMark {
 public:
  LaunchMark(muon_handle_s* h, int kind, cudaStream_t s);
  ~LaunchMark();
  LaunchMark(const LaunchMark&) = delete;
  LaunchMark& operator=(const LaunchMark&) = delete;

 private:
  muon_handle_s* h_;
  int kind_;
  cudaStream_t s_;
  cudaEvent_t a_;
};

}  // namespace muon
