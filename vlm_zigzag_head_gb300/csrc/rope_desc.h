// Checks and device form of the angles in a descriptor (cp_norm_rope_t, cp_rope_t).
#pragma once
#include <cmath>

#include "entry.h"
#include "rope.h"

namespace cpattn {

template <typename Desc>
cp_status_t rope_check_angles(const Desc* p) {
  if (p->rot_dim < 0 || p->rot_dim > p->d || p->rot_dim % 16 != 0)
    return entry_fail(CP_ERR_SHAPE, "rot_dim must be a multiple of 16 in [0, head_dim]");
  if (p->n_axes < 1 || p->n_axes > kRopeMaxAxes)
    return entry_fail(CP_ERR_SHAPE, "n_axes must be in [1, 4]");
  int pairs = 0;
  for (int i = 0; i < p->n_axes; ++i) {
    if (p->sections[i] < 0 || p->sections[i] > 64)
      return entry_fail(CP_ERR_SHAPE, "a section is negative or larger than the head");
    pairs += p->sections[i];
  }
  if (pairs != p->rot_dim / 2)
    return entry_fail(CP_ERR_SHAPE, "sections must add up to rot_dim / 2");
  if (p->rot_dim > 0 && !p->inv_freq)
    return entry_fail(CP_ERR_INVALID_ARG, "inv_freq is NULL");
  for (int i = 0; i < p->rot_dim / 2; ++i)
    if (!std::isfinite(p->inv_freq[i]))
      return entry_fail(CP_ERR_INVALID_ARG, "inv_freq must be finite");
  return CP_OK;
}

// On a checked descriptor.
template <typename Desc>
void rope_fill_angles(const Desc* p, const int32_t* pos, RopeAngles* a) {
  int end = 0;
  for (int i = 0; i < kRopeMaxAxes; ++i) {
    if (i < p->n_axes) end += p->sections[i];
    a->sec_end[i] = end;
  }
  a->pos = pos;
  a->n_axes = p->n_axes;
  a->T = p->T;
  a->rot = p->rot_dim;
  for (int i = 0; i < 64; ++i) a->freq[i] = 0;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    const double turns = p->inv_freq[i] / 6.283185307179586476925;
    const double frac = (turns - std::floor(turns)) * 18446744073709551616.0;   // exact
    a->freq[i] = frac < 18446744073709551616.0 ? (uint64_t)frac : 0;
  }
}

}  // namespace cpattn
