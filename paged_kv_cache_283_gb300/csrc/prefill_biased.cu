// Paged prefill on the tensor cores with changed scores and masks: the variants
// of the kernel (prefill_kernel.cuh) that pa_prefill_biased launches.  A variant
// for each pair of cap and bias: the softmax threads' code is what bounds the
// kernel, and with both as run-time flags of one variant the 16 x 512-token step
// below took 974 us.  16 x 512 new tokens after up to 3450 (32 query / 8 KV heads,
// scores below a fifth of the cap): no change 314 to 328 us, cap 372 to 386, bias 347
// to 359, both 430, over several GPUs.

#include "prefill_kernel.cuh"

namespace pa {

namespace {

template <int RULE>
cudaError_t launch_rule(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                        const PrefillParams& p, int group, int max_query_len, int num_seqs,
                        cudaStream_t stream) {
  switch (group) {
    case 1: return launch_prefill_g<1, RULE>(tq, tk, tv, p, max_query_len, num_seqs, stream);
    case 2: return launch_prefill_g<2, RULE>(tq, tk, tv, p, max_query_len, num_seqs, stream);
    case 4: return launch_prefill_g<4, RULE>(tq, tk, tv, p, max_query_len, num_seqs, stream);
    default: return launch_prefill_g<8, RULE>(tq, tk, tv, p, max_query_len, num_seqs, stream);
  }
}

}  // namespace

cudaError_t launch_prefill_biased(const CUtensorMap& tq, const CUtensorMap& tk,
                                  const CUtensorMap& tv, const PrefillParams& p, int group,
                                  int max_query_len, int num_seqs, cudaStream_t stream) {
  const bool cap = p.rule.softcap > 0.f, bias = p.rule.slopes != nullptr;
  if (cap && bias)
    return launch_rule<kRuled | kCap | kBias>(tq, tk, tv, p, group, max_query_len, num_seqs,
                                              stream);
  if (cap)
    return launch_rule<kRuled | kCap>(tq, tk, tv, p, group, max_query_len, num_seqs, stream);
  if (bias)
    return launch_rule<kRuled | kBias>(tq, tk, tv, p, group, max_query_len, num_seqs, stream);
  return launch_rule<kRuled>(tq, tk, tv, p, group, max_query_len, num_seqs, stream);
}

}  // namespace pa
