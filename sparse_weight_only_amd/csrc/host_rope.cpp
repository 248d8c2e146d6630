// sgemv_rope_table: frequencies of rotary positions (host).
#include <math.h>

#include "internal.hpp"

extern "C" int sgemv_rope_table(int32_t rot_dim, double base, double factor, double context, double low, double high,
                                double* turns_out) {
  if (!turns_out || rot_dim < 2 || rot_dim > 256 || rot_dim % 2) return SGEMV_EINVAL;
  if (!(base > 0.0) || !isfinite(base) || !(factor > 0.0) || !isfinite(factor)) return SGEMV_EINVAL;
  if (!(context >= 0.0) || !isfinite(context)) return SGEMV_EINVAL;
  if (context > 0.0 && (!isfinite(low) || !isfinite(high) || !(high > low) || !isfinite(high - low))) return SGEMV_EINVAL;
  for (int32_t j = 0; j < rot_dim / 2; ++j) {
    const double f = pow(base, -2.0 * j / rot_dim) / (2.0 * M_PI);
    double g = 0.0;                       // share of the frequency that stays
    if (context > 0.0) {
      g = (context * f - low) / (high - low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
    }
    turns_out[j] = f * (g + (1.0 - g) / factor);
    if (!isfinite(turns_out[j])) return SGEMV_EINVAL;
  }
  return SGEMV_OK;
}
