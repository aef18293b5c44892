#include "gx_launch.hpp"

GBX_RING_TABLE(fwd_nt, EPI_ACT, true)
