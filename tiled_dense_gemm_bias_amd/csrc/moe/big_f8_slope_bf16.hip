#include "gm_launch.hpp"

GBM_BIG_TABLE(big_f8_slope_bf16, 1, EPI_SLOPE)
