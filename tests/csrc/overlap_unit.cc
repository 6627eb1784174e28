// Host functions of csrc/overlap.cuh for tests/test_overlap.py.
#include "../../gated_delta_rule_16_gb300/csrc/overlap.cuh"

static gdn::Pieces make(const int64_t *x) { return gdn::pieces((const void *)(uintptr_t)x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]); }

extern "C" int overlap_unit(const int64_t *a, const int64_t *b) { return gdn::overlap(make(a), make(b)); }
extern "C" int overlaps_itself_unit(const int64_t *a) { return gdn::overlaps_itself(make(a)); }
