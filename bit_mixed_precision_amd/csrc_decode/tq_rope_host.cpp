// Host side of the rotary positions: the table of cosines and sines, in fp64.

#include <math.h>
#include <stdint.h>

#include <system_error>
#include <thread>
#include <vector>

#include "tq.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

bool positive(double v) { return isfinite(v) && v > 0; }

void fill(float* table, const double* freq, int64_t half, int64_t p0, int64_t p1, double gain) {
  for (int64_t p = p0; p < p1; ++p)
    for (int64_t i = 0; i < half; ++i) {
      const double a = (double)p * freq[i];
      table[2 * (p * half + i)] = (float)(cos(a) * gain);
      table[2 * (p * half + i) + 1] = (float)(sin(a) * gain);
    }
}

}  // namespace

extern "C" int tq_rope_table(int64_t n_pos, int64_t rot, double theta, int scaling, double factor,
                             double trained, double fast, double slow, double gain, float* table) {
  if (!table && n_pos != 0) return TQ_ERR_NULL;
  if (n_pos < 0 || n_pos > (int64_t(1) << 30) || rot < 2 || rot % 2 || rot > (int64_t(1) << 16) ||
      (rot == 2 && scaling == TQ_ROPE_BASE))
    return TQ_ERR_SHAPE;
  if (scaling < TQ_ROPE_NONE || scaling > TQ_ROPE_PARTS || !positive(theta) || !positive(gain))
    return TQ_ERR_VALUE;
  if (scaling != TQ_ROPE_NONE && !positive(factor)) return TQ_ERR_VALUE;
  if (scaling == TQ_ROPE_PARTS &&
      (!positive(trained) || !isfinite(fast) || !isfinite(slow) || fast <= slow))
    return TQ_ERR_VALUE;
  const int64_t half = rot / 2;
  try {
    std::vector<double> freq(half);
    const double base =
        scaling == TQ_ROPE_BASE ? theta * pow(factor, (double)rot / (double)(rot - 2)) : theta;
    if (!positive(base)) return TQ_ERR_VALUE;
    for (int64_t i = 0; i < half; ++i) {
      double f = pow(base, -2.0 * (double)i / (double)rot);
      if (scaling == TQ_ROPE_LINEAR) f /= factor;
      if (scaling == TQ_ROPE_PARTS) {
        double keep = (trained * f / kTwoPi - slow) / (fast - slow);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        f = f * keep + f / factor * (1 - keep);
      }
      freq[i] = f;
    }
    // a table of 2^20 entries takes some 50 ms on one thread
    int64_t threads = n_pos * half >> 18;
    const int64_t cores = std::thread::hardware_concurrency();
    if (threads > cores) threads = cores;
    if (threads > 8) threads = 8;
    if (threads < 1) threads = 1;
    std::vector<std::thread> pool;
    pool.reserve(8);  // nothing may throw once a thread runs
    int64_t done = 0;  // positions handed to started threads
    for (int64_t t = 1; t < threads; ++t) {
      const int64_t to = n_pos * t / threads;
      try {
        pool.emplace_back(fill, table, freq.data(), half, done, to, gain);
      } catch (const std::system_error&) {
        break;  // the rest is filled here
      }
      done = to;
    }
    fill(table, freq.data(), half, done, n_pos, gain);
    for (auto& t : pool) t.join();
  } catch (...) {
    return TQ_ERR_DEVICE;  // no host memory: nothing was started
  }
  return TQ_OK;
}
