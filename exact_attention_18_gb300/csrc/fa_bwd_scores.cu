// The backward with modified scores: the kernel of fa_bwd_main.cuh in both passes.
// With S' = y ln 2 the modified scores, t = tanh(scale x / cap):
//   P = exp(S' - L),  dS' = P o (dP - Delta),  dS = dS' o (1 - t^2),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// The bias is a constant of the call: it enters P alone.
//
// Roundings to 16 bits, as in the plain backward: P and dS as operands (half a step of
// each), the stored O that Delta is taken from, the results.  With scores far apart P
// is near 1 and dP - Delta a difference of like numbers, so the error of O in Delta is
// the largest part of dQ's and dK's.
//
// What bounds it (causal B1 H16/4 S4096 D128 bf16, capped): 159 us for the dK/dV pass
// and 120 for the dQ pass, tensor pipes 39 % active, instructions issued 44 %: the
// products of a block wait for its scores' arithmetic and the other way round, two
// groups of eight warps apart.  D = 64 with a bias (H16 fp16): 86 and 66 us, issue 63 %.
#include "fa_bwd_main.cuh"

namespace fa {

namespace {

template <int D, bool BF16>
cudaError_t launch_scored_t(bool kv_outer, const BwdMaps& m, const WithScores<BwdParams>& p, cudaStream_t stream) {
  return kv_outer ? launch_main_t<D, BF16, true, true, true>(m.k128, m.v128, m.q64, m.do64, p, stream, true)
                  : launch_main_t<D, BF16, false, true, true>(m.q128, m.do128, m.k64, m.v64, p, stream, true);
}

}  // namespace

cudaError_t launch_bwd_scored(int D, bool bf16, bool kv_outer, const BwdMaps& m, const WithScores<BwdParams>& p,
                              cudaStream_t stream) {
#define FA_SCORED_CASE(DD) \
  case DD: return bf16 ? launch_scored_t<DD, true>(kv_outer, m, p, stream) : launch_scored_t<DD, false>(kv_outer, m, p, stream);
  switch (D) {
    FA_SCORED_CASE(16)
    FA_SCORED_CASE(32)
    FA_SCORED_CASE(64)
    FA_SCORED_CASE(128)
    default: return cudaErrorInvalidValue;
  }
#undef FA_SCORED_CASE
}

}  // namespace fa
