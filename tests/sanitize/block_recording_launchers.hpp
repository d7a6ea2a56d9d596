// block_recording_launchers.hpp -- what the recording launchers of the linear layer's and the router's calls
// were called with, and what the plans answer.
#pragma once
#include <cstddef>
#include <string>
#include <vector>

struct BlockRecorded {
  std::vector<std::string> launches;   // names, in order
  const void* left = nullptr;          // the last product's left operand
  const void* workspace = nullptr;     // ... and workspace
  const void* pre = nullptr;           // the epilogue's gradient: pre, padded copy, counters, partial sums
  const void* padded = nullptr;
  const void* counters = nullptr;
  const void* partials = nullptr;
};
extern BlockRecorded g_rec;

struct BlockAnswers {
  bool one_row = true, four_rows = true;   // the decode kernels take the call
  bool skinny_fits = true;                 // the weight-streaming kernels do
  bool grad_fits = false;                  // the epilogue's gradient is made within the product
  size_t product = 0;                      // workspace of the products
  size_t sums = 0;                         // ... of the column sums
  size_t moe = 0;
};
extern BlockAnswers g_ans;
