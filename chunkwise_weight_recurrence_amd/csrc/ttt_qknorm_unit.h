// The columns and pairs of one lane's unit of a row of d columns, `rot` of them in turned pairs.
// Host code can include it too, so that the places are checked without a GPU.
#pragma once

namespace ttt {

// Where a lane's unit u lies: pieces of V columns at a and b (d: none), and its turned pairs' table entries
// t .. t + pairs - 1.  HALF: pair (j, j + rot / 2); the columns behind rot, and interleaved pairs, are pieces side by
// side, and a row of an odd number of pieces ends in a unit that has a piece at a only.
template <int V, bool HALF> struct Unit {
  int a, b, t, pairs;
  __device__ __forceinline__ Unit(int u, int d, int rot) {
    const int nr = HALF ? rot / 2 / V : 0;
    if (HALF && u < nr) {
      a = t = u * V;
      b = a + rot / 2;
      pairs = V;
    } else {
      a = (HALF ? rot : 0) + (u - nr) * 2 * V;
      a = a < d ? a : d;
      b = a + V < d ? a + V : d;
      t = a / 2;
      const int left = HALF || rot / 2 < t ? 0 : rot / 2 - t;
      pairs = left < V ? left : V;
    }
  }
};

}  // namespace ttt
