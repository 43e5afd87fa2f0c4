#include "scan_common.hpp"
extern "C" size_t ssu_scan_backward_workspace(const rssm_scan_dims* dims) { return 0; }
extern "C" int ssu_scan_backward(const rssm_scan_dims*, const void*, const void*, const void*,
                      const float*, const void*, const void*, const float*,
                      const float*, const int32_t*,
                      const void*, const uint8_t*,
                      const int32_t*, const float*, void*,
                      void*, void*, void*, float*, float*,
                      float*, float*, void*,
                      size_t, int32_t*, hipStream_t) { return RSSM_ESHAPE; }
