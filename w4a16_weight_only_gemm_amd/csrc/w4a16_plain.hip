// w4a16_plain.hip -- w4a16_gemm's small-M forms (the kernel is in w4a16_plain.h)
// and the time model that picks one per shape.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/w4a16.h"
#include "w4a16_device.h"
#include "w4a16_launch.h"
#include "w4a16_plain.h"

namespace w4a16_internal {
namespace {

constexpr PlainForm kXsForms[] = {kXs1x2, kXs1x4, kXs1x5, kXs2x2,
                                  kXs2x3, kXs2x4, kXs2x5, kXs4x4};

// Modelled time of an XS form (microseconds): from 9 rows each
// workgroup streams its MB x 16 activation rows (from L2) and NB weight
// columns over all of K at about 45 GB/s per compute unit, after a fixed
// start of 4 us (8 waves), 1.5 us (16 waves: more loads in flight from the
// first group) or 2 us (4 waves); a compute unit that holds n workgroups takes
// n times as long. Fitted to the decode layer set and its tensor-parallel
// shard (qkv 5120x896, o 768x5120, gate_up 5120x4352, down 2176x5120) at M =
// 17 to 320, where the form it puts first is within 1 % of the fastest of
// every form measured, summed over the shapes (above 320 rows it runs 5-11 %
// under the measured time of the shard's qkv, 12.4 and 19.7 against 13.0 and
// 22.1 us at 512 and 1024 rows, still far from the tile engine's 30 us); at 9
// to 16 rows (the rows past M repeat row M - 1 and are read from the caches)
// it puts first the fastest XS form of each decode projection.
double xs_estimate_us(PlainForm f, int M, int N, int K) {
  const PlainFormInfo& i = kPlainFormInfo[f];
  const long long ncb = (static_cast<long long>(N) + 15) / 16;
  const long long wgs = (ncb + i.nb - 1) / i.nb * ((static_cast<long long>(M) + 16 * i.mb - 1) / (16 * i.mb));
  const long long rounds = (wgs + kModelCUs - 1) / kModelCUs;
  const double bytes = static_cast<double>(K) * (32.0 * i.mb + 8.0 * i.nb);
  const double t0 = i.waves == 16 ? 1.5 : i.waves == 4 ? 2.0 : 4.0;
  return static_cast<double>(rounds) * (bytes / 45000.0 + t0);
}

// The XS form of least modelled time; with wide4 and wide N (1024 column
// blocks or more) the 4-wave 32-row form is a candidate too.
PlainForm best_xs_form(int M, int N, int K, bool wide4, double* est_out) {
  PlainForm best = kXsForms[0];
  double best_est = xs_estimate_us(best, M, N, K);
  for (PlainForm f : kXsForms) {
    const double e = xs_estimate_us(f, M, N, K);
    if (e < best_est) {
      best_est = e;
      best = f;
    }
  }
  if (wide4 && (N + 15) / 16 >= 1024) {
    const double e = xs_estimate_us(kXs2x5w4, M, N, K);
    if (e < best_est) {
      best_est = e;
      best = kXs2x5w4;
    }
  }
  if (est_out) *est_out = best_est;
  return best;
}

}  // namespace

int plain_form(int M, int N, int K, int group) {
  const bool wide = (N + 15) / 16 >= 1024;
  const size_t xlds_rows = static_cast<size_t>(M < 16 ? M : 16) * (static_cast<size_t>(K) + 8) * 2 +
                           static_cast<size_t>(K / group) * 64;
  // From 9 rows at group 128 the XS forms win on the decode layer set and its
  // tensor-parallel shard (M = 16: 76.6 -> 61.8 us per layer set as four
  // calls); at 8 rows and fewer the forms below (measured at M = 4, 6 and 8).
  // At group 128 and up to 16 rows, wide N takes the 4-wave XS forms, and a
  // short K (at most 8 groups: the shard's o 768x5120, 4.2-4.4 -> 3.6-3.8 us)
  // the 8-wave two-block XS form, at every row count.
  if (group == 128 && M <= 16) {
    if (wide) return M <= 4 ? kXs1x3w4 : kXs1x5w4;
    if (K <= 1024 && (N + 15) / 16 >= 128) return kXs1x2;
  }
  if (group == 128 && M >= 9) {
    const PlainForm f = best_xs_form(M, N, K, true, nullptr);
    return f == kXs1x2 && M <= 12 && K > 1024 ? kXs1x2p2 : f;
  }
  if (M <= 16) {
    if (wide) {
      if (M <= 2 && xlds_rows + 4 * 2 * 1024 <= kPlainLdsLimit) return kWideStaged;
      return M <= 4 ? kWide2 : kWide4;
    }
    if (M <= 2 && K >= 12288 && xlds_rows + 16 * 2 * 1024 <= kPlainLdsLimit) return kDeepStaged;
    if (M <= 8 && (N + 15) / 16 < 128) return kOne16;
    if (M == 1 && xlds_rows + 16 * 1024 <= kPlainLdsLimit) return kOne16Staged;
    if (group == 128 && M >= 7 && K > 1024) return kXs1x2p2;
    return M <= 8 ? kSmall8 : kWide2;
  }
  if (M <= 32) return wide ? kOp2x4 : kOp2x2;
  return wide ? kOp4x4 : kOp4x2;
}

void plain_form_shape(int form, int* rows, int* cols, int* waves) {
  const PlainFormInfo& i = kPlainFormInfo[form >= 0 && form < kPlainForms ? form : 0];
  *rows = 16 * i.mb;
  *cols = 16 * i.nb;
  *waves = i.waves;
}

// The best XS form's modelled time; at other group sizes the forms load their
// activation fragments in operand order, measured 1.3x slower than XS at 64
// rows on the decode layer set.
double plain_estimate_us(int M, int N, int K, int group) {
  double est = 0.0;
  best_xs_form(M, N, K, group == 128, &est);
  return group == 128 ? est : 1.3 * est;
}

hipError_t launch_skinny(const GemmArgs& a, hipStream_t stream) {
  const int form = plain_form(a.M, a.N, a.K, a.group);
  switch (a.group) {
    case 32: return launch_plain_form<32, kEpiNone>(form, a, Epilogue{}, stream);
    case 64: return launch_plain_form<64, kEpiNone>(form, a, Epilogue{}, stream);
    case 128: return launch_plain_form<128, kEpiNone>(form, a, Epilogue{}, stream);
    case 256: return launch_plain_form<256, kEpiNone>(form, a, Epilogue{}, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace w4a16_internal
