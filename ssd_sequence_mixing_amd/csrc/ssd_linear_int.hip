// The products of 8-bit integers (kInt), built as a translation unit of their own so
// that they compile in parallel with the others. Everything else in the included
// file is compiled out here.
#define SSD_INT_TU 1
#include "ssd_linear.hip"
