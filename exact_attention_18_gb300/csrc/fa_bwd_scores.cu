// The backward with modified scores: the kernel of fa_bwd_main.cuh in both passes.
// With S' = y ln 2 the modified scores, t = tanh(scale x / cap):
//   P = exp(S' - L),  dS' = P o (dP - Delta),  dS = dS' o (1 - t^2),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO.
// The bias is a constant of the call: it enters P alone.
//
// Delta.  rowsum(dO o O) of the stored O is off by half a 16-bit step of O, and where a
// row's weight lies on few keys dP - Delta is small against that: dQ and dK were off by
// 3.4e-3 of their size at scores of deviation 4 (bf16; 5.7e-3 at 8), where 16-bit
// operands and results alone make 2.4e-3.  So the dQ pass, which goes first, sums the
// row's P . dP in fp32 on its way and corrects what it has formed with the other:
//   Delta' = sum_j P_j dP_j,  dQ = scale (dS K - (Delta' - Delta) M),  M = (P o f) K,
// one product more, and the dK/dV pass reads Delta'.  Without / with it (us): causal
// B1 H32/4 S4096 D128 with a bias 382 / 421, capped (a degree less than now) 512 / 511;
// B2 H16 S4096 D64 286 / 303, 386 / 396.
//
// Roundings to 16 bits: P, P o f and dS as operands (half a step of each), the results.
//
// What bounds it (causal B1 H16/4 S4096 D128 bf16, capped): 137 us for the dQ pass and
// 157 for the dK/dV pass, tensor pipes 45 and 40 % active, instructions issued 45 %: the
// products of a block wait for its scores' arithmetic and the other way round, two
// groups of eight warps apart.  D = 64 with a bias (H16 fp16): 75 and 86 us, issue 61 and
// 63 %.
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
