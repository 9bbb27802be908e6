// Prompt attention, causal or full.
#include "prompt.hpp"

namespace dspark {

namespace {

template <int HD, int NW, int KT>
hipError_t launch(const Work& w, hipStream_t stream) {
  if (w.a.lse)
    return w.a.causal ? launch_one<HD, NW, KT, true, true, false>(w, stream) : launch_one<HD, NW, KT, false, true, false>(w, stream);
  return w.a.causal ? launch_one<HD, NW, KT, true, false, false>(w, stream) : launch_one<HD, NW, KT, false, false, false>(w, stream);
}

}  // namespace

hipError_t launch_prompt_attention(const PromptArgs& a, int hd, hipStream_t stream) {
  const Work w = work_of(a);
  // Workgroups of four waves, two on a compute unit, where sequences are short: one begins
  // or ends, which is memory's time, while the other multiplies.  Eight waves where they are
  // long: half the tiles to load.  32/8 heads of 128, causal, four waves against eight: 192
  // sequences of 64 59 and 76 us, 24 of 512 107 and 112, 12 of 1024 170 and 161, one of 8192
  // 611 and 536; 16/2 heads of 64: 64 of 256 35 and 36 us, one of 1024 18 and 23, two of 4096
  // 100 and 92.  Heads of 256 leave registers for four waves only.  The host knows the mean
  // length alone, and these were equal lengths: one of 8192 among 31 of some 100 takes 641 us by
  // four waves, 560 alone by eight and the others 23.
  switch (hd) {
    case 64: return a.T <= (int64_t)1024 * a.B ? launch<64, 4, 64>(w, stream) : launch<64, 8, 64>(w, stream);
    case 128: return a.T <= (int64_t)512 * a.B ? launch<128, 4, 32>(w, stream) : launch<128, 8, 64>(w, stream);
    case 256: return launch<256, 4, 32>(w, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
