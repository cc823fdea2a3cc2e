// attn_decode_q4.cu -- instantiations of the few-row attention over a cache held in 4 bits.
#include "attn_kernel_decode_q4.cuh"

namespace attn {

template <int DK, int DV, bool CTA>
static cudaError_t launch_rows(const DecodeQ4Params& p, cudaStream_t stream)
{
    if (p.R > 8) return dq4::launch<DK, DV, 2, false, CTA>(p, stream);
    if (DV == 128 && p.R <= 4) return dq4::launch<DK, DV, 1, DV == 128, CTA>(p, stream);
    return dq4::launch<DK, DV, 1, false, CTA>(p, stream);
}

template <int DK, int DV>
static cudaError_t launch_mode(const DecodeQ4Params& p, cudaStream_t stream)
{
    return p.mode == Q4_CTA ? launch_rows<DK, DV, true>(p, stream) : launch_rows<DK, DV, false>(p, stream);
}

cudaError_t launch_decode_q4(int d_k, int d_v, const DecodeQ4Params& p, cudaStream_t stream)
{
    if (d_k == 64 && d_v == 64) return launch_mode<64, 64>(p, stream);
    if (d_k == 128 && d_v == 128) return launch_mode<128, 128>(p, stream);
    if (d_k == 64 && d_v == 128) return launch_mode<64, 128>(p, stream);
    if (d_k == 128 && d_v == 64) return launch_mode<128, 64>(p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace attn
