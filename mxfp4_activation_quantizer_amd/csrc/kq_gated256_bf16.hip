// The gated feed-forward products on large tiles for bf16 outputs (a source for each type, so that they compile side by
// side).
#include "kq_gated256.hpp"

namespace kqhost {
kq_status gated256_bf16(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_g, const uint8_t *scales_g,
                       int packed, int64_t k, const kq::GatedEpi &ep, kq_stream_t stream) {
    return launch_gated256<uint16_t>(codes_a, scales_a, codes_g, scales_g, packed, k, ep, stream);
}
}  // namespace kqhost
