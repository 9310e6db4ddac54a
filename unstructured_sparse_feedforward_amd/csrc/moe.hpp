// A mixture-of-experts layer for few tokens (moe.hip), as api_moe.hip
// launches it.
#pragma once

#include "mx.hpp"

namespace sffn {

constexpr int kMoeMaxT = 256;      // tokens a call
constexpr int kMoeMaxE = 1024;     // experts
constexpr int kMoeMaxK = 32;       // experts a token

struct MoeArgs {
  const uint16_t* x;         // [T, d] bf16
  const uint16_t* router;    // [E, d] bf16
  const void* wg;            // [E, F, d] bf16, or the codes of [E F, d]
  const void* wu;            // nullptr: non-gated
  const void* wd;
  const uint8_t* sg;         // MXFP4 scales
  const uint8_t* su;
  const uint8_t* sd;
  int T, d, F, E, k;
  int normalize;
  const int32_t* t_dev;      // nullable: the number of valid tokens
  const int32_t* in_ids;     // [T, k] the tokens' experts and their weights as given by the
  const float* in_probs;     // caller, in place of the router (nullable, both)
  // A unit is an expert, or, when the (token, rank) pairs are fewer than the
  // experts, a pair (the pair of an expert's first token works for all of
  // the expert's tokens, the others have no tokens): Y of them.
  int Y;
  int by_pair;
  int one;                   // a single token, routed by the hidden kernel
  int nb;                    // neurons a workgroup of the hidden kernel
  int chunks;                // column chunks of the down kernel
  int ntk;                   // blocks of 16 tokens a pass of the hidden kernel
  int zh;                    // workgroups that share out a unit's passes there
  int zd;                    // workgroups that share out its blocks of 16 tokens in the down
                             // kernel (both powers of two)
  int split, fs;             // ranges of neurons there, of fs each
  // workspace
  long long* keys;           // [T, E] the logits as ordered integers
  int32_t* expert;           // [T k] the experts of each token by rank
  float* weight;             // [T k] their softmax weights
  uint8_t* on;               // [zh, Y, F] neuron active for one of the passes' tokens
  float* h;                  // [F, T k] hidden activations, the pairs in the order of their
                             // experts: those of a unit's tokens side by side
  float* part;               // [split, T k, d] output of each pair, by ranges of neurons
  float* y;                  // [T, d]
  int32_t* ids;              // [T, k] (nullable)
  float* probs;              // [T, k] (nullable)
};

// fills Y .. fs from the sizes (and whether the experts are given)
void moe_plan(bool mx, MoeArgs* a);
hipError_t launch_moe(bool mx, const MoeArgs& a, hipStream_t s);

}  // namespace sffn
