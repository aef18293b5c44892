#include "gx_launch.hpp"

GBX_RING_TABLE(fwd_nn, EPI_ACT, false)
