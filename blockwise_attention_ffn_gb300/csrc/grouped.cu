// grouped.cu -- grouped_gemm(): tensor maps, parameters and the choice of the
// tile for the grouped GEMM (grouped_kernel.cuh), and the public products over
// ragged groups.
#include "grouped_kernel.cuh"

namespace bpt {

using namespace gg;

int64_t grouped_part_tiles(int64_t N) { return (N + 255) / 256; }

int grouped_gemm(const GroupedOp& op, cudaStream_t st) {
  Params p;
  memset(&p, 0, sizeof(p));
  const bool tn = op.form == GROUPED_TN;
  const bool dual = op.form == GROUPED_NT && op.w2 != nullptr;
  const bool two = op.form == GROUPED_NN && op.a2 != nullptr;
  if (op.groups < 1 || op.groups > GROUPED_MAX_GROUPS || op.rows < 1) return 1;
  // Tiles, by the rows a group has on average (what each has, only the device
  // knows).  A pair of SMs takes 256 rows at a time: its product reads two thirds
  // of the bytes from L2 and shared memory, but leaves 128 rows idle in a group's
  // last tile on average against one SM's 64.  Few rows: the weights' bytes bound
  // the product; 64-column tiles of 32 rows give the SMs more units to share them
  // and a ring of little but weights.  us at 16, 32, 64, 256, 384, 512 rows, 64
  // groups of 1024 x 2048: few-row tiles 61, 70, 104, 326, 467, 619; one SM 64,
  // 64, 64, 90, 101, 124; a pair 68, 68, 70, 79, 96, 117; 16 of 2048 x 2048: 37,
  // 39, 53, 166, 238, 313; 37, 37, 37, 47, 57, 68; 41, 41, 41, 49, 57, 59.
  const bool small = op.form == GROUPED_NT && op.mean_rows <= 24;
  bool pair = tn ? op.M > BM : op.mean_rows >= 384;
  if (pair && gk::pair_units() <= 0) pair = false;
  // One SM a tile and few rounds of tiles: half as wide ones, of three quarters of
  // the time, where that takes less time in whole rounds, on average over tile
  // counts around the one of even groups.  NT, us at 64 rows: 12 groups of 1000 x
  // 2744 27.2 and 19.7, 3 of 2000 x 640 6.9 and 5.6 (one round either way); 40 of
  // 776 x 1304 at 256 rows 46.6 and 49.1 (three rounds, four), at 66 very uneven
  // ones 20.7 and 23.7 (one, two).
  bool half = false;
  if (!tn && !dual && op.epi == GROUPED_STORE && !small && !pair) {
    const int64_t mt = std::min<int64_t>(op.groups, op.rows) * ((op.mean_rows + BM - 1) / BM), sms = std::max(1, sm_count());
    auto rounds = [&](int64_t bn) {
      double r = 0;
      for (double by : {0.85, 1.0, 1.15}) r += ceil(by * (double)(mt * ((op.N + bn - 1) / bn)) / (double)sms);
      return r;
    };
    half = 0.75 * rounds(128) < rounds(256);
  }
  const int BN = small ? 64 : dual || half ? 128 : 256;
  const int TM = small ? 32 : pair ? 2 * BM : BM;
  const int BNS = pair ? BN / 2 : BN;
  p.offsets = op.offsets;
  p.groups = op.groups;
  p.rows = (int)op.rows;
  p.N = (int)op.N;
  p.nt = (int)((op.N + BN - 1) / BN);
  p.order = op.order;
  p.by_k = ((1ull << 37) + op.top_k - 1) / op.top_k;
  p.a_cols = (int)(tn ? op.M : op.K);
  p.pairs = (int)op.rows;
  p.out = op.out;
  p.out2 = op.out2;
  p.out3 = op.out3;
  p.out_f32 = op.out_f32;
  p.beta = op.beta;
  p.aux = reinterpret_cast<const __nv_bfloat16*>(op.aux);
  p.aux2 = reinterpret_cast<const __nv_bfloat16*>(op.aux2);
  p.row_weight = op.row_weight;
  p.row_weight_f32 = op.row_weight_f32;
  p.part = op.part;
  p.span = op.span;
  p.err = device_error_word();
  if (!p.err) return 3;
  int64_t units, mt_all;
  const int64_t some = std::min<int64_t>(op.groups, op.rows);  // groups that can hold a row
  int rc = 0;
  if (!tn) {
    p.segs = two ? 2 : 1;
    p.nkt = (int)((op.K + BK - 1) / BK);
    for (int i = 0; i < p.segs; ++i) {
      const void* a = i ? op.a2 : op.a;
      rc |= make_map_2d(&p.map_a[i], a, op.a_rows, op.K, op.K, BK, BM, 128);
      p.a[i] = reinterpret_cast<const __nv_bfloat16*>(a);
    }
    for (int i = 0; i < (dual || two ? 2 : 1); ++i) {
      const void* w = i ? op.w2 : op.w;
      rc |= op.form == GROUPED_NT ? make_map_stack(&p.map_b[i], w, op.groups, op.N, op.K, BK, BNS)
                                  : make_map_stack(&p.map_b[i], w, op.groups, op.K, op.N, 64, BK);
    }
    mt_all = std::min<int64_t>(op.rows, op.rows / TM + some);
    units = mt_all * p.nt;
  } else {
    p.segs = op.a2 ? 2 : 1;
    p.M = (int)op.M;
    p.mt = (int)((op.M + TM - 1) / TM);
    for (int i = 0; i < p.segs; ++i) {
      const void* a = i ? op.a2 : op.a;
      rc |= make_map_2d(&p.map_a[i], a, op.a_rows, op.M, op.M, 64, BK, 128);
      p.a[i] = reinterpret_cast<const __nv_bfloat16*>(a);
    }
    rc |= make_map_2d(&p.map_b[0], op.b, op.b_rows, op.N, op.N, 64, BK, 128);
    p.b = reinterpret_cast<const __nv_bfloat16*>(op.b);
    p.b_cols = (int)op.N;
    mt_all = (int64_t)op.groups * p.segs * p.mt;
    units = mt_all * p.nt;
  }
  if (rc) return 1;
  if (units > INT32_MAX) return 5;
  // bands of 4096 rows (TN: of 4096 of M): the wave in flight shares the
  // band's rows in L2 while the other operand streams through once a band
  p.band = 4096 / TM;
  ProfScope prof(PROF_GEMM, 2.0 * (double)op.rows * (double)op.N * (double)(tn ? op.M * p.segs : op.K * p.segs) * (dual ? 2 : 1), 0.0, st);
  if (op.form == GROUPED_NT) return launch_nt(p, op.epi, op.act, op.a_gather || small, pair, BN, units, st);
  if (op.form == GROUPED_NN) return launch_nn(p, op.epi, op.act, pair, BN, units, st);
  return launch_tn(p, op.a_gather, op.b_gather, pair, units, st);
}

}  // namespace bpt
