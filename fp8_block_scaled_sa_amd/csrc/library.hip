// library.hip -- the library as one translation unit: the files of entry
// points, the later ones with the first one's host checks and error record.
#include "dg_fp8.hip"

#include "moe_step.hip"

#include "attention_step.hip"
