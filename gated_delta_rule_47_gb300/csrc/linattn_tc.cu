#include "linattn.cuh"
namespace gdn {
bool linattn_tc_supported(const LinAttnArgs &) { return false; }
size_t linattn_tc_fwd_workspace(const LinAttnArgs &) { return 0; }
int launch_linattn_tc_fwd(const LinAttnArgs &, cudaStream_t) { return GDN_ERR_UNSUPPORTED; }
size_t linattn_tc_bwd_workspace(const LinAttnArgs &) { return 0; }
int launch_linattn_tc_bwd(const LinAttnArgs &, cudaStream_t) { return GDN_ERR_UNSUPPORTED; }
int linattn_tc_read_clear_error() { return GDN_OK; }
}
