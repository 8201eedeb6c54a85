// Host-only parts of the paged KV cache: rotary frequencies and steps, and
// the bookkeeping of pages on the caller's arrays. No CUDA, no allocation.
#include <cmath>
#include <cstdint>

#include "exq.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925;

int pages_of(int32_t n_tokens, int32_t page_size) { return (n_tokens + page_size - 1) / page_size; }

}  // namespace

extern "C" exq_status exq_rope_freqs(int32_t R, double base, int32_t scaling, double factor, double orig_ctx, double low,
                                     double high, double* inv_freq_out, double* gain_out) {
  if (!inv_freq_out || !gain_out || R < 2 || R % 2 || !(base > 1) || !std::isfinite(base)) return EXQ_ERR_INVALID_ARG;
  if (scaling < EXQ_ROPE_SCALE_NONE || scaling > EXQ_ROPE_SCALE_BANDS) return EXQ_ERR_INVALID_ARG;
  if (scaling != EXQ_ROPE_SCALE_NONE && (!(factor > 0) || !std::isfinite(factor))) return EXQ_ERR_INVALID_ARG;
  if (scaling == EXQ_ROPE_SCALE_NTK && R == 2) return EXQ_ERR_INVALID_ARG;
  const bool banded = scaling == EXQ_ROPE_SCALE_YARN || scaling == EXQ_ROPE_SCALE_BANDS;
  if (banded && (!(orig_ctx > 0) || !(low > 0) || !(high > low) || !std::isfinite(orig_ctx) || !std::isfinite(high)))
    return EXQ_ERR_INVALID_ARG;
  *gain_out = 1.0;
  if (scaling == EXQ_ROPE_SCALE_NTK) base *= std::pow(factor, static_cast<double>(R) / (R - 2));
  double ramp0 = 0, ramp1 = 1;
  if (scaling == EXQ_ROPE_SCALE_YARN) {
    // the (real) pair index that turns n times over orig_ctx: base^(-2j/R) = 2 pi n / orig_ctx
    const auto index = [&](double n) { return R * std::log(orig_ctx / (n * kTwoPi)) / (2 * std::log(base)); };
    ramp0 = std::fmax(std::floor(index(high)), 0.0);
    ramp1 = std::fmin(std::ceil(index(low)), R - 1.0);
    if (ramp1 - ramp0 < 1e-3) ramp1 = ramp0 + 1e-3;
    if (factor > 1) *gain_out = 0.1 * std::log(factor) + 1.0;
  }
  for (int32_t j = 0; j < R / 2; ++j) {
    const double f = std::pow(base, -2.0 * j / R);
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == EXQ_ROPE_SCALE_LINEAR) keep = 0.0;
    if (scaling == EXQ_ROPE_SCALE_YARN) keep = 1.0 - std::fmin(std::fmax((j - ramp0) / (ramp1 - ramp0), 0.0), 1.0);
    if (scaling == EXQ_ROPE_SCALE_BANDS)
      keep = std::fmin(std::fmax((orig_ctx * f / kTwoPi - low) / (high - low), 0.0), 1.0);
    const bool stretched = scaling != EXQ_ROPE_SCALE_NONE && scaling != EXQ_ROPE_SCALE_NTK;
    inv_freq_out[j] = stretched ? (1.0 - keep) * (f / factor) + keep * f : f;
  }
  return EXQ_OK;
}

extern "C" exq_status exq_rope_steps(const double* inv_freq, int32_t n, uint64_t* steps_out) {
  if (!inv_freq || !steps_out || n <= 0) return EXQ_ERR_INVALID_ARG;
  for (int32_t j = 0; j < n; ++j)
    if (!std::isfinite(inv_freq[j])) return EXQ_ERR_INVALID_ARG;
  for (int32_t j = 0; j < n; ++j) {
    const double turns = inv_freq[j] / kTwoPi;
    const double r = std::rint(std::ldexp(turns - std::floor(turns), 64));  // 0 .. 2^64
    steps_out[j] = r >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(r);
  }
  return EXQ_OK;
}

extern "C" exq_status exq_pages_alloc(int32_t* refs, int32_t n_pages, int32_t n, int32_t* ids_out) {
  if (!refs || n_pages <= 0 || n < 0 || (n > 0 && !ids_out)) return EXQ_ERR_INVALID_ARG;
  int32_t found = 0;
  for (int32_t p = 0; p < n_pages && found < n; ++p)
    if (refs[p] == 0) ids_out[found++] = p;
  if (found < n) return EXQ_ERR_FULL;
  for (int32_t i = 0; i < n; ++i) refs[ids_out[i]] = 1;
  return EXQ_OK;
}

extern "C" exq_status exq_pages_free(int32_t* refs, int32_t n_pages, const int32_t* ids, int32_t n) {
  if (!refs || n_pages <= 0 || n < 0 || (n > 0 && !ids)) return EXQ_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (ids[i] < 0 || ids[i] >= n_pages) return EXQ_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (--refs[ids[i]] < 0) {  // named more often than held: give back what was taken
      for (int32_t j = i; j >= 0; --j) ++refs[ids[j]];
      return EXQ_ERR_INVALID_ARG;
    }
  return EXQ_OK;
}

extern "C" exq_status exq_pages_fork(int32_t* refs, int32_t n_pages, int32_t page_size, const int32_t* ids,
                                     int32_t n_tokens, int32_t* ids_out, int32_t* pair_out, int32_t* n_pairs_out) {
  if (!refs || n_pages <= 0 || page_size <= 0 || n_tokens < 0 || !pair_out || !n_pairs_out) return EXQ_ERR_INVALID_ARG;
  if (n_tokens > INT32_MAX - page_size) return EXQ_ERR_INVALID_ARG;
  const int32_t n = pages_of(n_tokens, page_size);
  if (n > 0 && (!ids || !ids_out)) return EXQ_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (ids[i] < 0 || ids[i] >= n_pages || refs[ids[i]] <= 0) return EXQ_ERR_INVALID_ARG;
  const int32_t whole = n_tokens / page_size;
  int32_t own = -1;
  if (whole < n) {
    const exq_status st = exq_pages_alloc(refs, n_pages, 1, &own);
    if (st != EXQ_OK) return st;
  }
  for (int32_t i = 0; i < whole; ++i) {
    ++refs[ids[i]];
    ids_out[i] = ids[i];
  }
  *n_pairs_out = 0;
  if (own >= 0) {
    pair_out[0] = ids[whole];
    pair_out[1] = own;
    ids_out[whole] = own;
    *n_pairs_out = 1;
  }
  return EXQ_OK;
}

extern "C" exq_status exq_pages_compact(int32_t* refs, int32_t n_pages, int32_t* tables, int64_t n_entries,
                                        int32_t* pairs_out, int32_t* n_pairs_out) {
  if (!refs || n_pages <= 0 || n_entries < 0 || (n_entries > 0 && !tables) || !n_pairs_out || (n_pages > 1 && !pairs_out))
    return EXQ_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n_entries; ++i)
    if (tables[i] >= 0 && (tables[i] >= n_pages || refs[tables[i]] <= 0)) return EXQ_ERR_INVALID_ARG;
  int32_t n = 0;
  for (int32_t lo = 0, hi = n_pages - 1;; ++lo, --hi) {
    while (lo < hi && refs[lo] != 0) ++lo;
    while (lo < hi && refs[hi] == 0) --hi;
    if (lo >= hi) break;
    refs[lo] = refs[hi];
    refs[hi] = 0;
    pairs_out[2 * n] = hi;  // falling src, rising dst
    pairs_out[2 * n + 1] = lo;
    ++n;
  }
  for (int64_t i = 0; i < n_entries && n > 0; ++i) {
    if (tables[i] < pairs_out[2 * (n - 1)]) continue;  // below every moved page, or none
    int32_t a = 0, b = n - 1;
    while (a < b) {  // the first pair whose src is at most the entry
      const int32_t m = (a + b) / 2;
      if (pairs_out[2 * m] <= tables[i]) b = m; else a = m + 1;
    }
    if (pairs_out[2 * a] == tables[i]) tables[i] = pairs_out[2 * a + 1];
  }
  *n_pairs_out = n;
  return EXQ_OK;
}
