// The layer for a few tokens (few.hip).
#pragma once

#include "common.h"

namespace moe {

constexpr int kFewTokens = 16;
// experts in use: at most one for each pair, and the shared one
constexpr int kFewEntries = kFewTokens * MOE_KMAX + 1;

// The experts in use, as the first kernel leaves them for the second.
struct FewList {
  int32_t n;
  int32_t entry[kFewEntries];             // physical id, num_physical: shared
  uint32_t mask[kFewEntries];             // bit t: token t uses it
  float w[kFewEntries][kFewTokens];       // its weight there
};

struct FewCall {
  const float* logits;       // softmax top-k inside (E <= 256), or null:
  const float* bias;
  const int32_t* ids;        // the routes
  const float* w;
  const bf16_t* x;
  const moe_weights* weights;
  const int32_t* l2p;
  const int32_t* rep;
  int32_t* counts;           // or null
  FewList* list;
  bf16_t* h;                 // [few_entries][kFewTokens][I]
  void* out;
};
int few_entries(const moe_problem* p);    // for every T up to kFewTokens
hipError_t launch_few(const moe_problem* p, const FewCall& c, hipStream_t s);

}  // namespace moe
