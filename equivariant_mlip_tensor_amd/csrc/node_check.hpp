// node_check.hpp -- what the node operators' C entry points check their
// arguments and report their errors with.
#pragma once

#include <exception>
#include <string>

#include "node_internal.hpp"

namespace tpconv {

constexpr int64_t kMaxRows = int64_t(1) << 31;

// Runs an entry point's body; no C++ exception leaves the library.
template <class F>
tpconv_status guarded(F&& body) noexcept {
  try {
    return body();
  } catch (const std::exception& e) {
    try {
      return fail(TPCONV_E_INVALID_ARG, e.what());
    } catch (...) {
      return TPCONV_E_INVALID_ARG;
    }
  } catch (...) {
    return TPCONV_E_INVALID_ARG;
  }
}

inline tpconv_status bad(const std::string& msg) { return fail(TPCONV_E_INVALID_ARG, msg); }

inline tpconv_status launched(hipError_t he, const char* what) {
  if (he != hipSuccess) return fail(TPCONV_E_HIP, std::string(what) + " launch: " + hipGetErrorString(he));
  return TPCONV_OK;
}

inline bool known(tpconv_dtype dt) { return dt == TPCONV_F32 || dt == TPCONV_F64; }

inline tpconv_status check_workspace(const void* ws, size_t have, size_t need, const char* what) {
  if (need == 0) return TPCONV_OK;
  if (ws == nullptr || have < need)
    return fail(TPCONV_E_WORKSPACE,
                std::string(what) + " holds " + std::to_string(have) + " bytes, needs " + std::to_string(need));
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return fail(TPCONV_E_WORKSPACE, std::string(what) + " must be 256-byte aligned");
  return TPCONV_OK;
}

}  // namespace tpconv
