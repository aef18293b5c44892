#include "gx_launch.hpp"

GBX_RING_TABLE(slope_nt, EPI_SLOPE, true)
