// attn_range.h -- which keys a row of an attention problem sees and which rows see a key, for host and device.
#pragma once
#include "../../include/sdtw.h"

#ifdef __CUDACC__
#define SDTW_BOTH __host__ __device__ __forceinline__
#else
#define SDTW_BOTH inline
#endif

namespace sdtw {

SDTW_BOTH int least(int a, int b) { return a < b ? a : b; }
SDTW_BOTH int most(int a, int b) { return a > b ? a : b; }

// Keys that row n of batch element b sees: [lo(n), hi(n)), empty where lo >= hi.
// Row n of n_b stands at key n + (m_b - n_b): the last row at the last key.
struct RowRange {
    int n_b, m_b, shift, left, right;
    SDTW_BOTH RowRange(const sdtw_attention& a, int b) {
        n_b = a.q_lengths ? least(most(a.q_lengths[b], 0), a.N) : a.N;
        m_b = a.k_lengths ? least(most(a.k_lengths[b], 0), a.M) : a.M;
        shift = m_b - n_b;
        left = a.window_left;
        right = a.window_right;
    }
    SDTW_BOTH int lo(int n) const { return left < 0 ? 0 : most(0, n + shift - left); }
    SDTW_BOTH int hi(int n) const { return right < 0 ? m_b : least(m_b, n + shift + right + 1); }
    // rows that see key j: [row_lo, row_hi). Both lie within [0, n_b], so that their places among the packed rows,
    // G times as many, fit 32 bits as N * G does: old keys of a long cache are up to M rows out of a window's reach.
    SDTW_BOTH int row_lo(int j) const { return right < 0 ? 0 : least(n_b, most(0, j - shift - right)); }
    SDTW_BOTH int row_hi(int j) const { return left < 0 ? n_b : most(0, least(n_b, j - shift + left + 1)); }
    // Rows before this one stand before the first key and see none. Those from it on, up to n_b, each see one: a window
    // takes in a row's own place, and the last row stands at the last key.
    SDTW_BOTH int first_row() const { return m_b > 0 ? row_lo(0) : n_b; }
    // packed rows (G a position) that see any of the keys [j0, j1): [lo, hi), both 0 where there is none
    struct Rows {
        int lo, hi;
    };
    SDTW_BOTH Rows seeing(int j0, int j1, int G) const {
        const int j_last = least(j1, m_b) - 1;
        if (j0 > j_last) return {0, 0};
        const int first = row_lo(j0), end = row_hi(j_last);
        if (first >= end) return {0, 0};
        return {first * G, end * G};
    }
};

}  // namespace sdtw
