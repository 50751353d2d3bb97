// node_dense_rows.hip -- the products of node_dense.hpp for one data type and
// mode (TPCONV_DOUBLE, TPCONV_MODE), so that they compile side by side.
#include "node_dense.hpp"

namespace tpconv {
namespace dense {

template <class T, int MODE, bool X8>
hipError_t run_dense(DenseArgs& a, hipStream_t s) {
  if (a.n_rows == 0 || a.n_jobs == 0) return hipSuccess;
  // The fewest channels a block that hold the widest side: a narrow map in a wide block multiplies zeros.  (Gated, 2048
  // fp64 rows of 16 channels l <= 4 with 16: 15 us, 32: 22; 4096 fp32 rows of 32 channels l <= 3 with 32: 12 us, 64: 18.)
  // fp64 has no registers for 64.
  int widest = 1;
  // The gates' rows that a transposed product reads as well go by chunks in any case, so they count for no more than
  // makes 8 chunks in turn.  (Such products of these two by their number, 80 and 128: 17.6 and 14.2 us, by an eighth
  // 15.8 and 12.2; the gradients of 4096 fp32 rows of 16 channels l <= 3 with 208 gates, by an eighth 61 us, by the
  // rows' channels alone 68.)
  for (int i = 0; i < a.n_jobs; ++i) {
    const int gates = a.job[i].gate.src.K;
    widest = std::max({widest, a.job[i].N, a.job[i].main.src.K, MODE == kTransposed ? gates / 8 : gates});
  }
  if (widest <= 16) return launch_jobs<T, 16, MODE, X8>(a, s);
  if constexpr (sizeof(T) == 4)
    if (widest > 32) return launch_jobs<T, 64, MODE, X8>(a, s);
  return launch_jobs<T, 32, MODE, X8>(a, s);
}

#if TPCONV_DOUBLE
using Real = double;
#else
using Real = float;
#endif
template hipError_t run_dense<Real, TPCONV_MODE, false>(DenseArgs&, hipStream_t);
#if !TPCONV_DOUBLE && (TPCONV_MODE == 2 || TPCONV_MODE == 3)
template hipError_t run_dense<Real, TPCONV_MODE, true>(DenseArgs&, hipStream_t);
#endif

}  // namespace dense
}  // namespace tpconv
