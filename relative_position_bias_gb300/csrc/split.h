// How the compact-bias backward's units are cut for the last, partly filled wave of CTAs.  Plain C++, so that it is
// tested on the host by itself.
#pragma once

namespace dera {

// Whole units and pieces per remaining unit, of `units` tiles.
struct CbSplit {
  int full, split;
  int tail(int units) const { return split > 1 ? units - full : 0; }
  int blocks(int units) const { return full + (units - full) * split; }
};

// Padded width of the rows kernel's key steps, and its steps for H grid rows.
inline int cb_width(int W) { return W <= 16 ? 16 : (W <= 32 ? 32 : (W <= 48 ? 48 : 64)); }
inline int cb_rows_steps(int H, int W) {
  const int per = W <= 16 ? 4 : (W <= 32 ? 2 : 1);   // CbKeys<cb_width(W)>::KHT
  return (H + per - 1) / per;
}

// A unit takes rows_steps steps in the rows kernel, cols_steps in the cols kernel.
inline void cb_split(int units, int rows_steps, int cols_steps, int sms, CbSplit* rows, CbSplit* cols) {
  // One CTA an SM, first the rows kernel's units, then the cols kernel's, whose CTAs start where the
  // rows kernel's run out: the 2 * units CTAs leave one last wave that is only partly filled.
  // Its units, all of them cols' unless there are fewer CTAs than SMs, are cut into as many pieces as
  // finish them soonest; a piece costs kStart steps more than the steps it takes (its tiles, the
  // pieces' partial results and the join).
  constexpr int kStart = 10, kMinSteps = 4;
  *rows = {units, 1};
  *cols = {units, 1};
  if (sms <= 0) return;
  const long long all = 2ll * units;
  const int tail = static_cast<int>(all % sms);
  if (tail == 0) return;
  const bool few = all < sms;   // every unit is of the last wave
  const int steps = few ? (rows_steps < cols_steps ? rows_steps : cols_steps) : cols_steps;
  int pieces = 1;
  long long best = steps + kStart;
  for (int p = 2; p <= steps / kMinSteps; ++p) {
    const long long waves = (static_cast<long long>(tail) * p + sms - 1) / sms;
    const long long cost = waves * ((steps + p - 1) / p + kStart);
    if (cost < best) {
      best = cost;
      pieces = p;
    }
  }
  if (pieces == 1) return;
  if (few) *rows = {0, pieces};
  *cols = {few ? 0 : units - (tail < units ? tail : units), pieces};
}

}  // namespace dera
