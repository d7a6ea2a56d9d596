// recording_launchers.hpp -- what the recording launchers were called with.
#pragma once
#include <cstddef>
#include <string>
#include <vector>

struct Recorded {
  std::vector<std::string> launches;   // names, in order
  const void* left = nullptr;          // the last product's left operand
  const void* workspace = nullptr;     // ... and workspace
  const void* padded = nullptr;        // the padded copy given to the pairs' gradient
};
extern Recorded g_rec;

// what the size queries and the plans' checks answer
struct Answers {
  size_t workspace = 0;                // every workspace query of the block's operators
  bool skinny_fits = true;             // the weight-streaming kernels take the call
  bool grad_fits = false;              // the pairs' gradient is made within the product
};
extern Answers g_ans;
