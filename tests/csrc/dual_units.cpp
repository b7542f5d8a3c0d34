// The dual-path linear's unit order for the host tests (no CUDA).
#include "dual_units.h"

extern "C" void dual_split_unit(int j, int k, int* tile, int* piece) {
  const dual_units::SplitUnit u = dual_units::split_unit(j, k);
  *tile = u.tile;
  *piece = u.piece;
}

extern "C" void dual_split_plan(long long t_units, long long main_tiles, long long resident,
                                int kb_total, int few_too, int* tiles, int* k) {
  const dual_units::Split s =
      dual_units::split_plan(t_units, main_tiles, resident, kb_total, few_too != 0);
  *tiles = s.tiles;
  *k = s.k;
}
