#include "gr_mixer.h"
namespace gr {
bool mix_tc_supported(const MixArgs&) { return false; }
size_t mix_tc_workspace(int64_t, int, int, int, int) { return 0; }
cudaError_t launch_mix_tc(const MixArgs&, void*, cudaStream_t) { return cudaErrorNotSupported; }
int mixer_status(bool) { return 0; }
}  // namespace gr
