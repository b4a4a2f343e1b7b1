// The grids of the gated delta rule's launches, with the stand-ins of
// delta_checks.cpp: a launch counts threads in 32 bits, so a call is refused
// where any of its launches would have more.
#define main delta_checks_main
#include "delta_checks.cpp"
#undef main

// Threads of the widest launch of a call (see launch_shape in delta_chunk.h).
static double most_threads(const DeltaArgs& a, bool backward) {
  const double heads = a.H, pieces = heads * a.pieces, blocks = heads * (double)a.slots;
  double most = std::max((blocks + 3) / 4, pieces * (a.tiles + (a.seg_slots > 0 ? a.move_tiles : 0))) * 256;
  if (a.seg_slots > 0 && a.segments > 2) most = std::max(most, heads * a.B * ((a.pitch + 15) / 16) * 256);
  if (backward) most = std::max(most, heads * (double)a.group_slots * (a.Dk > 64 ? 512 : 256));
  return most;
}

int main() {
  int taken = 0, refused = 0;
  for (prnnDataType_t type : {PRNN_DATA_FLOAT, PRNN_DATA_HALF, PRNN_DATA_BFLOAT})
    for (int Dk : {8, 64, 65, 128, 129, 256})
      for (int Dv : {1, 64, 65, 200})
        for (int T : {1, 32, 33, 64, 65, 300})
          for (int B : {1, 1 << 16, 1 << 18, (1 << 19) - 1, (1 << 19) + 1, 786432, (1 << 20) - 1})
            for (int rows = 0; rows < 2; ++rows)
              for (int backward = 0; backward < 2; ++backward) {
                Case c(1, T, 16, 16, Dk, Dv, type);
                c.d.B = B;
                uintptr_t far = 1ull << 46;  // (batch first, and far apart)
                for (prnnSequence_t* x : {&c.q, &c.k, &c.v, &c.g, &c.beta, &c.o, &c.dq, &c.dk, &c.dv, &c.dg, &c.dbeta}) {
                  x->data = at<void>(far += 1ull << 46);
                  x->batch = x->token * T;
                }
                c.S0 = at<float>(far += 1ull << 46);
                c.S1 = at<float>(far += 1ull << 46);
                if (rows) {
                  c.d.offsets = at<int32_t>(0x1000);
                  c.d.rows = (int64_t)B * T;
                }
                launches = 0;
                const prnnStatus_t st = backward ? c.backward() : c.forward();
                if (st != PRNN_STATUS_SUCCESS) {
                  CHECK(st == PRNN_STATUS_NOT_SUPPORTED && launches == 0, "status %d", (int)st);
                  ++refused;
                  continue;
                }
                ++taken;
                CHECK(most_threads(args, backward) <= 4294967295., "type %d Dk %d Dv %d T %d B %d rows %d backward %d: %.0f threads",
                      (int)type, Dk, Dv, T, B, rows, backward, most_threads(args, backward));
              }
  CHECK(taken > 1000 && refused > 1000, "%d calls taken, %d refused", taken, refused);
  if (failures == 0) std::printf("all checks passed\n");
  return failures == 0 ? 0 : 1;
}
