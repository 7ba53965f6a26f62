// TMA maps of the selective scan's inputs.
#pragma once
#include "kernels.h"
#include "tc_common.cuh"

namespace linattn {

struct ScanMaps {
  CUtensorMap x, dt, z, B, C, dy;
};

// Boxes of `tokens` rows by `channels` (x, dt, z, dy) or by one group's N
// states (B, C).  z and dy may be null: their maps are left alone.
inline bool make_scan_maps(ScanMaps *m, const ScanArgs &a, const void *dy, int elem_bytes,
                           int channels, int tokens) {
  if (a.L == 0) return true;
  auto map = [&](CUtensorMap *t, const void *p, int64_t width, int64_t ld, int box) {
    return !p || make_tmap_rows(t, p, elem_bytes, width, a.L, a.B, ld, box, tokens);
  };
  const int64_t GN = (int64_t)a.G * a.N;
  return map(&m->x, a.x, a.E, a.ldx, channels) && map(&m->dt, a.dt, a.E, a.lddt, channels) &&
         map(&m->z, a.z, a.E, a.ldz, channels) && map(&m->B, a.Bm, GN, a.ldb, a.N) &&
         map(&m->C, a.Cm, GN, a.ldc, a.N) && map(&m->dy, dy, a.E, a.E, channels);
}

}  // namespace linattn
