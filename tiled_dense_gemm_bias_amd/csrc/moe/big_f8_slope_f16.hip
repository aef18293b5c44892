#include "gm_launch.hpp"

GBM_BIG_TABLE(big_f8_slope_f16, 0, EPI_SLOPE)
