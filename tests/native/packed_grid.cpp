// How many work shares the attention of packed rows cuts, by the device (no CUDA).
#include "packed_plan.cuh"

using namespace pkv;

extern "C" {
int workspace_shares() { return kPackedShares; }
int launch_shares(int num_sms) { return packed_most_shares(num_sms); }
int used_shares(long long total, int min_steps, int num_sms) { return packed_share_count(total, min_steps, packed_most_shares(num_sms)); }
}
