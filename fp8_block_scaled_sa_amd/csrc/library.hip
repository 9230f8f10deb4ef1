// library.hip -- the library as one translation unit: both files of entry
// points, the second with the first one's host checks and error record.
#include "dg_fp8.hip"

#include "moe_step.hip"
