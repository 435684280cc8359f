// How the layer norm's kernels divide a row of `width` elements.
//
// A row is held in registers, so that it is read once: EPT = VE * NV elements
// a thread, VE of them consecutive (one load). VE is the widest load that
// every row's start is aligned to: 16 bytes where the width allows, else one
// element (an odd width leaves every other row unaligned). G lanes of a warp
// share a row where it is short, so that no lane is without elements; longer
// rows take a whole CTA (G = 0).
#pragma once

#include "gdn_vec.cuh"

namespace gdn {
namespace ln {

constexpr int kEpt = 16;          // elements per thread at most
constexpr int kWarpWidth = 512;   // widest row of one warp: 32 x kEpt
constexpr int kRowThreads = 256;  // threads of a CTA whose warps take rows of their own

struct Shape {
    int ve, nv, g;     // elements per load, loads per thread, lanes per row (0: the CTA)
    int threads;       // of a CTA
    int rows_per_cta;  // rows in work at a time
};

template <typename T>
inline Shape shape_of(int width) {
    constexpr int kVec = 16 / int(sizeof(T));
    Shape s;
    s.ve = width % kVec == 0 ? kVec : 1;
    const int small = s.ve == 1 ? 4 : 1;  // loads a thread of the variant for short rows
    const int large = kEpt / s.ve;
    if (width <= 16 * s.ve * small) {
        s.nv = small, s.g = 16;
    } else if (width <= 32 * s.ve * small) {
        s.nv = small, s.g = 32;
    } else if (width <= kWarpWidth) {
        s.nv = large, s.g = 32;
    } else {
        s.nv = large, s.g = 0;
    }
    s.threads = s.g ? kRowThreads : ((width + s.ve * s.nv - 1) / (s.ve * s.nv) + 31) / 32 * 32;
    s.rows_per_cta = s.g ? kRowThreads / s.g : 1;
    return s;
}

// calls F<VE, NV, G>(...) for the shape
#define GDN_LN_DISPATCH(T, s, F, ...)                                                  \
    do {                                                                               \
        constexpr int kV = 16 / int(sizeof(T));                                        \
        if ((s).ve == kV) {                                                            \
            if ((s).g == 16) F<T, kV, 1, 16>(__VA_ARGS__);                             \
            else if ((s).g == 32 && (s).nv == 1) F<T, kV, 1, 32>(__VA_ARGS__);         \
            else if ((s).g == 32) F<T, kV, ln::kEpt / kV, 32>(__VA_ARGS__);            \
            else F<T, kV, ln::kEpt / kV, 0>(__VA_ARGS__);                              \
        } else {                                                                       \
            if ((s).g == 16) F<T, 1, 4, 16>(__VA_ARGS__);                              \
            else if ((s).g == 32 && (s).nv == 4) F<T, 1, 4, 32>(__VA_ARGS__);          \
            else if ((s).g == 32) F<T, 1, ln::kEpt, 32>(__VA_ARGS__);                  \
            else F<T, 1, ln::kEpt, 0>(__VA_ARGS__);                                    \
        }                                                                              \
    } while (0)

}  // namespace ln
}  // namespace gdn
