// placeholder
#include "paged.cuh"
