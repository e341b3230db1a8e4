// score.h -- the parameters of scores beyond the plain scale * q . k (score.cuh),
// for host code too.
#pragma once

#include <stdint.h>

namespace pkv {

struct ScoreParams {
  float cap2;                // softcap * log2 e; 0: no cap
  float inv_cap2;            // 1 / cap2
  float cap_k;               // 2 / softcap
  int32_t window;            // 0: none
  const float* slopes;       // [Hq], or null
  const int32_t* first_key;  // decode [B], prefill [T], or null
  const int32_t* prefix;     // [B], or null (prefill)
};

}  // namespace pkv
