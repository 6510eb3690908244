// Reading the pair of index maps (moe_layer_ops.h) on the device.
#pragma once

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace mfr {

// Row of pair (t, j), or -1 where the pair has none: its entry is out of
// range, or the row does not name the pair in turn.  Only that check makes
// each row the business of one pair, so that no two writers meet whatever the
// maps hold.  `report`: this caller raises the status bit.
__device__ __forceinline__ int pair_row(const MapParams& m, int64_t t, int j, bool report) {
    const int64_t s = t * m.k + j;
    const int32_t r = m.row_of[s];
    bool ok = r >= 0 && static_cast<int64_t>(r) < m.R;
    if (ok) ok = m.slot_of[r] == s;
    if (!ok && report && !(m.sentinel && r < 0)) atomicOr(m.status, MFR_STATUS_BAD_INDEX);
    return ok ? r : -1;
}

// What row r is from its own side: true where it is to be written with
// zeros.  Raises the status bit for a row whose pair does not name it in turn.
__device__ __forceinline__ bool row_is_padding(const MapParams& m, int64_t r) {
    const int32_t s = m.slot_of[r];
    if (s >= 0) {
        if (s >= m.T * m.k || m.row_of[s] != r) atomicOr(m.status, MFR_STATUS_BAD_INDEX);
        return false;
    }
    if (s < MFR_ROW_UNUSED) atomicOr(m.status, MFR_STATUS_BAD_INDEX);
    return s == MFR_ROW_PADDING;
}

}  // namespace mfr
