// Stand-ins for what the host layer of the sequence operators and the history
// layer calls on the device side. Launches are counted, not made; the plans of
// workspaces are sizes to check arguments against.
#include <cstdio>
#include <cstdlib>

#include "seq_internal.h"

int g_launches = 0;
emb::Buckets g_buckets;  // of the last attention's launch

extern "C" int stub_launches(void) { return g_launches; }
extern "C" int stub_bucket_start(int i) { return g_buckets.first[i]; }

namespace emb {
static hipError_t count() {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_norm_rotary(const NormRotaryArgs&, const RotTable&, hipStream_t) { return count(); }
hipError_t launch_norm_rotary_back(const NormRotaryBackArgs&, const RotTable&, hipStream_t) { return count(); }
hipError_t launch_kv_append(const AppendArgs&, const RotTable&, hipStream_t) { return count(); }
hipError_t launch_prefix_attention(const PrefixArgs&, const PrefixPlan&, char*, hipStream_t) { return count(); }
hipError_t launch_layer_norm(const LayerNormArgs&, hipStream_t) { return count(); }
int layer_norm_back_blocks(long long rows) { return (int)(rows < 256 ? rows : 256); }
hipError_t launch_layer_norm_back(const LayerNormBackArgs&, hipStream_t) { return count(); }
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t) {
  if (a.threshold > 1ull << 32 || !(a.scale >= 0.f)) std::abort();
  return count();
}
hipError_t launch_history(const HistoryArgs& a, hipStream_t) {
  g_buckets = a.h.buckets;
  return count();
}
HistoryBackPlan history_back_plan(const HistoryView&, long long tokens, int seqs) {
  return HistoryBackPlan{256, (size_t)(256 + tokens + seqs)};
}
hipError_t launch_history_back(const HistoryBackArgs& a, hipStream_t) {
  if (a.f.tokens > 0 && (!a.rows || reinterpret_cast<char*>(a.part) - reinterpret_cast<char*>(a.rows) != 256)) std::abort();
  return count();
}
int history_step_parts(const HistoryView&, const KvView&, int seqs, int) { return seqs ? 3 : 1; }
hipError_t launch_history_step(const HistoryStepArgs&, hipStream_t) { return count(); }
}  // namespace emb
