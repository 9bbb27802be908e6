// Causal prompt attention under a window with sinks.
#include "prompt.hpp"

namespace dspark {

namespace {

template <int HD, int NW, int KT>
hipError_t launch(const Work& w, hipStream_t stream) {
  return w.a.lse ? launch_one<HD, NW, KT, true, true, true>(w, stream) : launch_one<HD, NW, KT, true, false, true>(w, stream);
}

}  // namespace

hipError_t launch_prompt_window(const PromptArgs& a, int hd, hipStream_t stream) {
  const Work w = work_of(a);
  switch (hd) {
    case 64: return a.T <= (int64_t)1024 * a.B ? launch<64, 4, 64>(w, stream) : launch<64, 8, 64>(w, stream);
    case 128: return a.T <= (int64_t)512 * a.B ? launch<128, 4, 32>(w, stream) : launch<128, 8, 64>(w, stream);
    case 256: return launch<256, 4, 32>(w, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dspark
