#include "gx_launch.hpp"

GBX_RING_TABLE(slope_nn, EPI_SLOPE, false)
