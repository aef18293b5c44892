#include "gx_launch.hpp"

GBX_BIG_WGRAD_TABLE(big_wgrad_tn)
