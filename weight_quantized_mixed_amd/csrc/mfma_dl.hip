// Direct-load MFMA path (M > 8): the choice of its tile and its launches.  The kernel is in
// mfma_dl_kernel.hpp; its instances for gated plans are compiled in mfma_dl_gated.hip.
#include "mfma_dl_kernel.hpp"

namespace qg {

void dl_tile_dims(int tile, int* bm, int* bn) {
  static const int dims[DL_NUM][2] = {{32, 64},  {32, 128},  {32, 256},  {64, 128},
                                      {64, 256}, {128, 256}, {256, 256}, {128, 128}};
  *bm = dims[tile][0];
  *bn = dims[tile][1];
}

int choose_dl_tile(int fmt, int64_t M, int64_t N, int k_parts, int smode, bool gated) {
  const bool packed = fmt == FMT_I4 || fmt == FMT_U4 || fmt == FMT_I2;
  if (packed && smode == SC_PIECE) return -1;  // one scale slot per stage holds one group per column
  const int cap = M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  static const int order[] = {DL_256x256, DL_128x256, DL_128x128, DL_64x256, DL_64x128, DL_32x256, DL_32x128, DL_32x64};
#ifdef QG_FORCE_DL_TILE
  if (QG_FORCE_DL_TILE >= 0) return QG_FORCE_DL_TILE;
#endif
  // Gated fp16 of 129 to 256 rows: the tile whose waves of 256 workgroups, each at the cost
  // measured for a wave of it, are soonest done.  (The rule below jumps from one wave of
  // large tiles that fill a little under 60 % of the CUs to three of the smallest: N = 6306,
  // K = 2624, M = 186 67 us, so 36 us; N = 2900, K = 2560, M = 186 43 and 21 us.)
  if (gated && fmt == FMT_F16 && M > 128 && M <= 256) {
    static const struct { int tile, cost; } waves_of[] = {{DL_128x256, 170}, {DL_64x256, 145}, {DL_64x128, 100},
                                                         {DL_32x128, 88},  {DL_32x64, 68}};
    int best = -1;
    int64_t least = 0;
    for (const auto& w : waves_of) {
      int bm, bn;
      dl_tile_dims(w.tile, &bm, &bn);
      const int64_t t = (((M + bm - 1) / bm) * ((N + bn - 1) / bn) * k_parts + 255) / 256 * w.cost;
      if (best < 0 || t < least) {
        best = w.tile;
        least = t;
      }
    }
    return best;
  }
  // The largest tile whose last wave of workgroups still occupies at least 60% of
  // the 256 CUs: larger tiles re-read less of A and B, idle CUs cost in proportion.
  int pick = -1;
  for (int t : order) {
    // 128 x 128 only for int4 / int2 weights, whose upcast it shares over 128 rows
    // (measured at M = 128, N = 32000: 58 -> 50 us for int4; not measured for int8 and fp16)
    if (t == DL_128x128 && !packed) continue;
    int bm, bn;
    dl_tile_dims(t, &bm, &bn);
    if (bm > cap) continue;
    pick = t;
    const int64_t wgs = ((M + bm - 1) / bm) * ((N + bn - 1) / bn) * k_parts;
    const int64_t waves = (wgs + 255) / 256;
    if (wgs * 10 >= waves * 256 * 6) break;
  }
  return pick;
}

hipError_t launch_mfma_dl(int fmt, int tile, const RunArgs& a0, hipStream_t st) {
  // One scale group over K and no zero points: the column scale factors out of the
  // whole sum, so the tiles take the unscaled upcast (exact q rather than q * s rounded
  // to fp16) and the epilogue scales the fp32 sum; W4A16 g = -1 at 16384^3 then runs
  // like g = 0
  RunArgs a = a0;
  if ((fmt == FMT_I4 || fmt == FMT_U4) && a.smode == SC_BLOCK && a.group_size < 0 && !a.zeros) {
    a.epi_scale = static_cast<const _Float16*>(a.S);
    a.smode = SC_NONE;
  }
  // fp16 and int4 / uint4 without zero points: four waves of 128 x 128 (measured
  // at 16384^3: fp16 6.66 -> 6.41 ms, int4 6.34 -> 5.82 ms); the others keep
  // eight waves of 128 x 64, which measured faster for them
  if (tile == DL_256x256 && QG_BIG4 && big_tile_takes(fmt, a)) return launch_mfma_big(fmt, a, st);
  if (fmt == FMT_F16 && a.row_scale) return launch_mfma_dl_rows(tile, a, st);
  return a.out_mode == OUT_GATE ? launch_mfma_dl_gated(fmt, tile, a, st) : launch_any_tile<false>(fmt, tile, a, st);
}

}  // namespace qg
