// The partials of tree attention's cut units: where they lie, and which records of
// them may be followed.  Plain C++ on the host too, so that it is tested there.
#pragma once

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

// A CTA leaves at most two partials: that of the unit that a CTA before it began, then
// that of the unit which it begins itself.
PKV_HOST_DEVICE int tree_partials(int ctas) { return 2 * ctas; }
PKV_HOST_DEVICE int tree_partial(int cta, bool begins) { return 2 * cta + (begins ? 1 : 0); }

// Whether a unit's record names CTAs of the launch.  The attention kernel writes every
// unit's record while it runs to its end; a CTA whose bounded wait expired writes none of
// its later units', and the workspace then holds what it held before the call.
PKV_HOST_DEVICE bool tree_parts_valid(int first, int last, int ctas) {
    return first >= 0 && first <= last && last < ctas;
}

}  // namespace pkv
