// What the paged 4-bit cache's kernels share: the host checks of a pool and
// the address of a token-head's row in it.
#pragma once

#include <cstdint>

#include "sf_internal.h"

namespace sf {

inline bool pow2_in(int v, int lo, int hi) { return v >= lo && v <= hi && (v & (v - 1)) == 0; }

inline int log2i(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

// SF_OK, or SF_EINVAL with a message for a pool outside the contract.
inline sf_status check_paged_kv(const sf_paged_kv* kv, const char* what) {
  SF_REQUIRE(kv, "%s: kv is null", what);
  SF_REQUIRE(kv->k_codes && kv->k_param && kv->v_codes && kv->v_param, "%s: kv has a null array", what);
  SF_REQUIRE(aligned(kv->k_codes, 16) && aligned(kv->k_param, 16) && aligned(kv->v_codes, 16) &&
                 aligned(kv->v_param, 16),
             "%s: kv's arrays must be 16-byte aligned", what);
  SF_REQUIRE(kv->d == 64 || kv->d == 128 || kv->d == 256, "%s: d must be 64, 128 or 256", what);
  SF_REQUIRE(pow2_in(kv->page_size, 16, 256), "%s: page_size must be a power of two in [16, 256]", what);
  SF_REQUIRE(kv->Hkv >= 1 && kv->Hkv <= 256, "%s: Hkv must be in [1, 256]", what);
  SF_REQUIRE(kv->num_pages >= 1 && static_cast<int64_t>(kv->num_pages) * kv->page_size < (1ll << 31),
             "%s: need num_pages >= 1 and num_pages * page_size < 2^31", what);
  SF_REQUIRE(kv->page_rows == 0 ||
                 (kv->page_rows >= static_cast<int64_t>(kv->Hkv) * kv->page_size && kv->page_rows % 4 == 0),
             "%s: page_rows must be 0 or a multiple of 4 of at least Hkv * page_size", what);
  return SF_OK;
}

inline int64_t page_rows(const sf_paged_kv* kv) {
  return kv->page_rows ? kv->page_rows : static_cast<int64_t>(kv->Hkv) * kv->page_size;
}

}  // namespace sf
