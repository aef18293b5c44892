#include "gx_launch.hpp"

GBX_RING_MX4_TABLE(mx4_nt)
