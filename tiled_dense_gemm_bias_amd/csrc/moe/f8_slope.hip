#include "gm_launch.hpp"

GBM_RING_TABLE(f8_slope, EPI_SLOPE)
