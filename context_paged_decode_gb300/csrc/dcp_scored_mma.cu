#include "dcp_scored.cuh"
namespace dcp {
bool scored_mma_ok(const ScoredArgs&, CacheKind, bool) { return false; }
int scored_mma_ctas(int, int, CacheKind) { return 0; }
int launch_scored_mma(const ScoredArgs&, CacheKind, cudaStream_t) { return DCP_EUNSUPPORTED; }
}  // namespace dcp
