#include "gx_launch.hpp"

GBX_RING_WGRAD_TABLE(wgrad_tn)
